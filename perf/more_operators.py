"""Cases of the 8-bit operators: quantising by blocks of 128, the matrix product of such codes, the latent store into rows of
blocks, and reading cached latents back.

Each case is one call of one operator.  ``run`` computes it in elementary torch operations, or with ``own`` set through
this package's public calls; ``exact`` computes it in 64 bits from the definition.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
SMALLEST = 2.0 ** -100  # a block whose largest magnitude is below is scaled as if it were this


# --------------------------------------------------------------------------------------------------------- the cases
def listed():
    """Twelve cases: two or more of each operator, the DeepSeek-V3 widths of this package's workloads among them."""
    return [
        # one decode step's hidden states, normalised and quantised for the projections into queries and latents
        dict(name="quantize_decode", op="quantize", M=64, K=7168, norm=True, rows=1, pad=0),
        # the values that a prompt's attention leaves (128 heads x 128), for the output projection
        dict(name="quantize_prompt", op="quantize", M=4096, K=16384, norm=False, rows=1, pad=0),
        # the output projection's weight, quantised once when a model is loaded
        dict(name="quantize_weight", op="quantize", M=7168, K=16384, norm=False, rows=128, pad=0),
        # the output projection of a decode step, added to the residual stream
        dict(name="product_decode", op="product", M=64, K=16384, N=7168, bias=False, act="none", residual=True, pad=0),
        # an odd middle size with everything in the epilogue
        dict(name="product_odd", op="product", M=333, K=1008, N=1544, bias=True, act="gelu_tanh", residual=True, pad=16),
        # the query projection (7168 -> 128 heads x 192) of a verification step, 4 tokens for each of 64 sequences
        dict(name="product_verify", op="product", M=256, K=7168, N=24576, bias=False, act="none", residual=False, pad=0),
        # the output projection of a prompt
        dict(name="product_prompt", op="product", M=4096, K=16384, N=7168, bias=False, act="none", residual=True, pad=0),
        # the new latents of a decode step of 64 sequences, into the slots of a paged cache
        dict(name="store_decode", op="store", tokens=64, d_c=512, d_rope=64, page_size=64, norm=True,
             layout="interleaved", far=32768, lead=0),
        # a batch of prompts, a slice of a wider projection's rows
        dict(name="store_prompt", op="store", tokens=32768, d_c=512, d_rope=64, page_size=64, norm=True,
             layout="half", far=32768, lead=1536),
        # a short history of a few sequences, kept with one scale, read back before a chunk of a prompt
        dict(name="load_chunk", op="load", B=3, T=333, rows=333, d_c=512, d_rope=64, page_size=64, kv="e4m3", listed=False),
        # the histories of a batch, kept in blocks, read back for a prefill in the expanded form
        dict(name="load_history", op="load", B=64, T=4096, rows=4096, d_c=512, d_rope=64, page_size=64, kv="blocks",
             listed=False),
        # the tokens that a selector picked for each sequence, of a long history kept in blocks
        dict(name="load_selected", op="load", B=32, T=16384, rows=2048, d_c=512, d_rope=64, page_size=64, kv="blocks",
             listed=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["quantize", "product", "product", "store", "load"])
    if op == "quantize":
        rows = rng.choice([1, 1, 1, 128])
        return dict(op=op, M=_log_int(rng, 1, 4096), K=16 * _log_int(rng, 1, 1024), norm=rows == 1 and rng.random() < 0.5,
                    rows=rows, pad=rng.choice([0, 0, 8, 64]))
    if op == "product":
        return dict(op=op, M=_log_int(rng, 1, 4096), K=16 * _log_int(rng, 4, 1024), N=8 * _log_int(rng, 4, 896),
                    bias=rng.random() < 0.5, act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                    residual=rng.random() < 0.5, pad=rng.choice([0, 0, 16, 64]))
    if op == "store":
        return dict(op=op, tokens=_log_int(rng, 1, 32768), d_c=64 * rng.choice([1, 2, 3, 4, 5, 8, 8, 8]),
                    d_rope=16 * rng.choice([0, 1, 2, 3, 4, 4, 4]), page_size=64 * rng.randint(1, 3),
                    norm=rng.random() < 0.8, layout=rng.choice(["interleaved", "half"]), far=_log_int(rng, 256, 1 << 28),
                    lead=rng.choice([0, 0, 8, 200, 1024]))
    B = _log_int(rng, 1, 64)
    T = _log_int(rng, 1, min(16384, 262144 // B))
    pick = rng.random() < 0.5
    return dict(op=op, B=B, T=T, rows=_log_int(rng, 1, min(T, 4096)) if pick else T, d_c=64 * rng.choice([1, 2, 3, 4, 5, 8, 8, 8]),
                d_rope=16 * rng.choice([1, 2, 3, 4, 4, 4]), page_size=64 * rng.randint(1, 3),
                kv=rng.choice(["bf16", "e4m3", "blocks", "blocks"]), listed=pick)


def _row_bytes(case):
    d_c, d_rope = case["d_c"], case["d_rope"]
    return {"bf16": 2 * (d_c + d_rope), "e4m3": d_c + d_rope, "blocks": d_c + 16 + 2 * d_rope}[case.get("kv", "blocks")]


def work(case):
    op = case["op"]
    if op == "quantize":
        M, K, b = case["M"], case["K"], -(-case["K"] // 128)
        return {"bytes": 3 * M * K + 4 * b * -(-M // case["rows"]) + 2 * K * case["norm"],
                "flops": M * K * (6 if case["norm"] else 2)}
    if op == "product":
        M, K, N, b = case["M"], case["K"], case["N"], -(-case["K"] // 128)
        return {"bytes": M * K + N * K + 4 * b * (M + -(-N // 128)) + 2 * M * N * (2 if case["residual"] else 1)
                + 2 * N * case["bias"], "flops": 2 * M * K * N}
    if op == "store":
        width = case["d_c"] + case["d_rope"]
        return {"bytes": case["tokens"] * (2 * width + 8 + _row_bytes(case)) + 2 * case["d_c"] * case["norm"],
                "flops": case["tokens"] * (6 * case["d_c"] + 3 * case["d_rope"])}
    # about what the drawn lengths come to
    width, rows = case["d_c"] + case["d_rope"], case["B"] * (case["rows"] if case["listed"] else 0.75 * case["rows"])
    return {"bytes": rows * (_row_bytes(case) + 2 * width + (4 if case["listed"] else 4 / case["page_size"])),
            "flops": 0 if case["kv"] == "bf16" else rows * width}


# -------------------------------------------------------------------------------------------------------- the inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _hidden(g, M, K):
    """Activations: channels differ in size, as a model's do."""
    return (torch.randn((M, K), generator=g, device=DEV) * torch.exp(0.7 * torch.randn((K,), generator=g, device=DEV))).to(
        torch.bfloat16)


def _blocks(y, rows):
    """y [M, K] in fp32 as codes [M, K] and scales [M / rows, K / 128], a scale for each block of rows x 128 values."""
    M, K = y.shape
    mb, kb = -(-M // rows), -(-K // 128)
    full = y.new_zeros((mb * rows, kb * 128))
    full[:M, :K] = y
    full = full.view(mb, rows, kb, 128)
    top = full.abs().amax(dim=(1, 3), keepdim=True).clamp(min=SMALLEST)
    codes = (full * (448.0 / top)).clamp(-448.0, 448.0).to(E4M3)
    return codes.view(mb * rows, kb * 128)[:M, :K], (top / 448.0).view(mb, kb)


def prepare(case, seed):
    return {"quantize": _prepare_quantize, "product": _prepare_product, "store": _prepare_store,
            "load": _prepare_load}[case["op"]](case, seed)


def _mla():
    from mla_decode_attention_absorbed_gb300 import mla
    return mla


def _prepare_quantize(case, seed):
    g = _generator(seed)
    M, K = case["M"], case["K"]
    x = _hidden(g, M, K + case["pad"]) if case["rows"] == 1 else _normal(g, (M, K + case["pad"]), K ** -0.5)
    weight = (1.0 + 0.2 * torch.randn((K,), generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None
    return dict(case=case, x=x[:, :K], weight=weight, eps=1e-6)


def _prepare_product(case, seed):
    g = _generator(seed)
    M, K, N = case["M"], case["K"], case["N"]
    codes, scale = _blocks(_hidden(g, M, K).float(), 1)
    x = torch.zeros((M, K + case["pad"]), device=DEV, dtype=E4M3)[:, :K]
    x.copy_(codes)
    w, w_scale = _blocks(_normal(g, (N, K), K ** -0.5).float(), 128)
    return dict(case=case, x=x, x_scale=scale.t().contiguous(), w=w.contiguous(), w_scale=w_scale.contiguous(),
                bias=_normal(g, (N,)) if case["bias"] else None,
                residual=_normal(g, (M, N)) if case["residual"] else None)


def _frequencies(d):
    """Angular frequencies of the d / 2 pairs, in 64 bits: what a program works out once per model."""
    return torch.exp(torch.arange(d // 2, dtype=torch.float64) * (-2.0 / d * math.log(10000.0))).to(DEV)


def _prepare_store(case, seed):
    g = _generator(seed)
    T, d_c, d_rope, ps, lead = case["tokens"], case["d_c"], case["d_rope"], case["page_size"], case["lead"]
    rows = _normal(g, (T, lead + d_c + d_rope))[:, lead:]
    weight = (1.0 + 0.2 * torch.randn((d_c,), generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None
    at = torch.randint(0, case["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
    pages = -(-T // ps) + 2
    slots = torch.randperm(pages * ps, generator=g, device=DEV)[:T].to(torch.int32)
    kv = torch.zeros((pages, ps, _row_bytes(case)), device=DEV, dtype=torch.uint8)
    st = dict(case=case, rows=rows, weight=weight, at=at, slots=slots, kv=kv, eps=1e-6)
    if d_rope:
        st["f"] = _frequencies(d_rope)
    if own:
        m = _mla()
        st["lens"] = torch.ones((T,), device=DEV, dtype=torch.int32)
        st["table"] = torch.zeros((T, 1), device=DEV, dtype=torch.int32)
        st["prob"] = m.Problem(T, 128, 1, d_c, d_rope, 128, 128, 1.0)
        st["cache"] = m.make_cache(st["prob"], kv, st["lens"], st["table"], ps)
        layout = {"interleaved": m.ROPE_INTERLEAVED, "half": m.ROPE_HALF}[case["layout"]]
        st["plan"] = m.rope_plan(d_rope, layout=layout) if d_rope else None
    return st


def _prepare_load(case, seed):
    g = _generator(seed)
    B, T, rows, d_c, d_rope, ps = (case[k] for k in ("B", "T", "rows", "d_c", "d_rope", "page_size"))
    width, kind = d_c + d_rope, case["kv"]
    cols = -(-T // ps)
    pages = B * cols + 3
    table = torch.randperm(pages, generator=g, device=DEV)[:B * cols].to(torch.int32).view(B, cols)
    # lengths between half of T and T; the table's entries behind a length are never reached
    lens = T // 2 + (torch.rand((B,), generator=g, device=DEV) * (T - T // 2 + 1)).floor().clamp(max=T - T // 2)
    lens = lens.clamp(min=1).to(torch.int32)
    st = dict(case=case, table=table, lens=lens, at=None, kv_scale=0.04)
    if kind == "bf16":
        kv = _normal(g, (pages, ps, width))
    else:
        kv = torch.zeros((pages, ps, _row_bytes(case)), device=DEV, dtype=torch.uint8)
        values = d_c if kind == "blocks" else width
        codes = torch.randn((pages, ps, values), generator=g, device=DEV).mul_(100.0 if kind == "blocks" else 32.0)
        kv[:, :, :values] = codes.clamp_(-448.0, 448.0).to(E4M3).view(torch.uint8)
        del codes
        if kind == "blocks":
            scales = torch.exp(0.3 * torch.randn((pages, ps, 4), generator=g, device=DEV)) * 0.01
            scales[:, :, -(-d_c // 128):] = 0.0
            kv[:, :, d_c:d_c + 16].view(torch.float32).copy_(scales)
            kv[:, :, d_c + 16:].view(torch.bfloat16).copy_(_normal(g, (pages, ps, d_rope)))
    st["kv"] = kv
    if case["listed"]:
        # positions in a history, some places empty where the selector had no more
        at = (torch.rand((B, rows), generator=g, device=DEV) * lens[:, None]).floor().to(torch.int32)
        st["at"] = torch.where(torch.rand((B, rows), generator=g, device=DEV) < 0.02, -1, at)
    st["out"] = torch.zeros((B, rows, width), device=DEV, dtype=torch.bfloat16)
    if own:
        m = _mla()
        st["prob"] = m.Problem(B, 128, 1, d_c, d_rope, 128, 128, 1.0)
        st["cache"] = m.make_cache(st["prob"], kv, lens, table, ps, kv_scale=st["kv_scale"] if kind == "e4m3" else None)
    return st


# ---------------------------------------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"quantize": _own_quantize, "product": _own_product, "store": _own_store, "load": _own_load}[op](state)
    return {"quantize": _plain_quantize, "product": _plain_product, "store": _plain_store, "load": _plain_load}[op](state)


def _own_quantize(st):
    return _mla().quantize(st["x"], norm_weight=st["weight"], eps=st["eps"], block_rows=st["case"]["rows"])


def _own_product(st):
    m = _mla()
    act = {"none": m.ACT_NONE, "relu": m.ACT_RELU, "silu": m.ACT_SILU, "gelu": m.ACT_GELU,
           "gelu_tanh": m.ACT_GELU_TANH}[st["case"]["act"]]
    return m.linear_fp8(st["x"], st["x_scale"], st["w"], st["w_scale"], bias=st["bias"], residual=st["residual"], act=act)


def _own_store(st):
    _mla().latent_store(st["prob"], st["rows"], st["cache"], plan=st["plan"], norm_weight=st["weight"], eps=st["eps"],
                        positions=st["at"], slots=st["slots"])
    return _parts(st)


def _own_load(st):
    return _mla().latent_load(st["prob"], st["cache"], st["case"]["rows"], positions=st["at"], out=st["out"])


def _parts(st):
    """The pool's three parts: codes, the scales in use, keys."""
    kv, d_c = st["kv"], st["case"]["d_c"]
    return dict(codes=kv[:, :, :d_c].view(E4M3), scales=kv[:, :, d_c:d_c + 4 * -(-d_c // 128)].view(torch.float32),
                keys=kv[:, :, d_c + 16:].view(torch.bfloat16) if st["case"]["d_rope"] else None)


def _norm(x, weight, eps):
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + eps) * weight.float()


def _plain_quantize(st):
    y = st["x"].float()
    if st["weight"] is not None:
        y = _norm(y, st["weight"], st["eps"])
    codes, scales = _blocks(y, st["case"]["rows"])
    return codes, scales.t().contiguous() if st["case"]["rows"] == 1 else scales


def _plain_product(st):
    K, N = st["case"]["K"], st["case"]["N"]
    x = st["x"].float() * st["x_scale"].t().repeat_interleave(128, dim=1)[:, :K]
    w = st["w"].float() * st["w_scale"].repeat_interleave(128, dim=0)[:N].repeat_interleave(128, dim=1)[:, :K]
    y = x @ w.t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    act = st["case"]["act"]
    if act == "relu":
        y = y.clamp(min=0.0)
    elif act == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif act == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(torch.bfloat16)


def _plain_store(st):
    case, rows, d_c = st["case"], st["rows"], st["case"]["d_c"]
    c = rows[:, :d_c].float()
    if st["weight"] is not None:
        c = _norm(c, st["weight"], st["eps"])
    codes, scales = _blocks(c, 1)
    flat, to = st["kv"].view(-1, st["kv"].shape[-1]), st["slots"].long()
    flat[to, :d_c] = codes.contiguous().view(torch.uint8)
    flat[to, d_c:d_c + 4 * scales.shape[1]] = scales.view(torch.uint8)
    if case["d_rope"]:
        angle = st["at"].to(torch.float64)[:, None] * st["f"]
        cos, sin, k = torch.cos(angle).float(), torch.sin(angle).float(), rows[:, d_c:].float()
        half = case["d_rope"] // 2
        if case["layout"] == "interleaved":
            a, b = k[:, 0::2], k[:, 1::2]
            k = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(1)
        else:
            a, b = k[:, :half], k[:, half:]
            k = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
        flat[to, d_c + 16:] = k.to(torch.bfloat16).view(torch.uint8)
    return _parts(st)


def _where(st):
    """For each row asked for: whether it is there, and its row of the pool."""
    case, table = st["case"], st["table"]
    ps = case["page_size"]
    at = st["at"]
    if at is None:
        at = torch.arange(case["rows"], device=table.device).expand(case["B"], -1)
    there = (at >= 0) & (at < st["lens"][:, None])
    at = at.clamp(0, case["T"] - 1).long()
    return there, table.long().gather(1, at // ps) * ps + at % ps


def _plain_load(st):
    case, d_c = st["case"], st["case"]["d_c"]
    there, at = _where(st)
    rows = st["kv"].view(-1, st["kv"].shape[-1])[at]
    if case["kv"] == "blocks":
        scales = rows[:, :, d_c:d_c + 16].view(torch.float32).repeat_interleave(128, dim=2)[:, :, :d_c]
        c = rows[:, :, :d_c].view(E4M3).float() * scales
        rows = torch.cat((c.to(torch.bfloat16), rows[:, :, d_c + 16:].view(torch.bfloat16)), dim=2)
    elif case["kv"] == "e4m3":
        rows = (rows.view(E4M3).float() * st["kv_scale"]).to(torch.bfloat16)
    st["out"].copy_(torch.where(there[:, :, None], rows, st["out"]))
    return st["out"]


# ------------------------------------------------------------------------------------------- from the definition, 64 bits
def _exact_blocks(y, rows):
    """The quotients that are rounded to codes, and the scales, block column by block column."""
    M, K = y.shape
    q, scales = torch.empty_like(y), torch.empty((-(-M // rows), -(-K // 128)), dtype=torch.float64, device=DEV)
    row = torch.arange(M, device=DEV) // rows
    for j in range(scales.shape[1]):
        part = y[:, 128 * j:128 * j + 128]
        top = torch.zeros((scales.shape[0],), dtype=torch.float64, device=DEV)
        top.scatter_reduce_(0, row, torch.linalg.vector_norm(part, ord=math.inf, dim=1), "amax")
        scales[:, j] = torch.maximum(top, torch.full_like(top, SMALLEST)) / 448.0
        q[:, 128 * j:128 * j + 128] = part / scales[row, j, None]
    return q, scales


def _exact_norm(x, weight, eps):
    root = (torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / x.shape[1] + eps) ** 0.5
    return x / root * weight.double()


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        y = st["x"].double()
        if case["norm"]:
            y = _exact_norm(y, st["weight"], st["eps"])
        q, scales = _exact_blocks(y, case["rows"])
        return q, scales.t().contiguous() if case["rows"] == 1 else scales
    if case["op"] == "product":
        # each operand's values, then one product
        x, w = st["x"].double(), st["w"].double()
        for j in range(-(-case["K"] // 128)):
            x[:, 128 * j:128 * j + 128] *= st["x_scale"][j, :, None].double()
            w[:, 128 * j:128 * j + 128] *= st["w_scale"][torch.arange(case["N"], device=DEV) // 128, j, None].double()
        y = torch.matmul(x, w.t())
        if case["bias"]:
            y += st["bias"].double()
        if case["act"] == "relu":
            y = torch.maximum(y, torch.zeros_like(y))
        if case["act"] == "silu":
            y = y * torch.special.expit(y)
        if case["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        if case["act"] == "gelu_tanh":
            # (1 + tanh u) / 2 is the logistic function of 2 u
            y = y * torch.special.expit(2.0 * (2.0 / math.pi) ** 0.5 * (y + 0.044715 * y ** 3))
        return y + st["residual"].double() if case["residual"] else y
    if case["op"] == "store":
        d_c, d, x = case["d_c"], case["d_rope"], st["rows"].double()
        c = x[:, :d_c]
        if case["norm"]:
            c = _exact_norm(c, st["weight"], st["eps"])
        q, scales = _exact_blocks(c, 1)
        k = torch.empty_like(x[:, d_c:])
        for i in range(d // 2):
            p, r = (2 * i, 2 * i + 1) if case["layout"] == "interleaved" else (i, i + d // 2)
            angle = st["at"].double() * 10000.0 ** (-2.0 * i / d)
            z = torch.complex(x[:, d_c + p], x[:, d_c + r]) * torch.polar(torch.ones_like(angle), angle)
            k[:, p], k[:, r] = z.real, z.imag
        pages, ps, to = st["kv"].shape[0], case["page_size"], st["slots"].long()

        def pool(v):
            return torch.zeros((pages * ps, v.shape[1]), dtype=torch.float64, device=DEV).index_copy_(0, to, v).view(
                pages, ps, v.shape[1])
        return dict(codes=pool(q), scales=pool(scales), keys=pool(k) if d else None)
    there, at = _where(st)
    d_c, out = case["d_c"], torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        rows = st["kv"].view(-1, st["kv"].shape[-1])[at[b, there[b]]]
        if case["kv"] == "blocks":
            v = torch.empty((rows.shape[0], out.shape[2]), dtype=torch.float64, device=DEV)
            v[:, d_c:] = rows[:, d_c + 16:].view(torch.bfloat16).double()
            for j in range(-(-d_c // 128)):
                part = slice(128 * j, min(128 * j + 128, d_c))
                v[:, part] = rows[:, part].view(E4M3).double() * rows[:, d_c + 4 * j:d_c + 4 * j + 4].view(torch.float32).double()
        else:
            v = rows.double() if case["kv"] == "bf16" else rows.view(E4M3).double() * st["kv_scale"]
        out[b, there[b]] = v
    return out
