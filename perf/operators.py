"""Cases of the operators around the latent attention: rotary positions, page tables with slot maps, the normalised and
rotated latent store, and the matrix product with bias, activation and residual.

Each case is one call of one operator.  ``run`` computes it in elementary torch operations, or with ``own`` set through
this package's public calls; ``exact`` computes it in 64 bits from the definition.
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------------------------------------- the cases
def listed():
    """Twelve cases: three of each operator, the DeepSeek-V3 widths of this package's workloads among them."""
    return [
        # one decode step's queries: 64 sequences, 128 heads, split into the two parts the attention takes and rotated
        dict(name="rope_decode", op="rope", B=64, s_q=1, H=128, d_nope=128, d_rope=64, layout="interleaved",
             scaling="yarn", factor=40.0, original=4096, base=10000.0, mscale=1.0, far=8192, given=False, pad=0),
        # verification of a few tokens per sequence far into a stretched context, half layout, rows of a wider projection
        dict(name="rope_verify_far", op="rope", B=37, s_q=3, H=40, d_nope=80, d_rope=48, layout="half",
             scaling="linear", factor=8.0, original=0, base=500000.0, mscale=1.25, far=1 << 27, given=True, pad=24),
        # a long prompt's queries
        dict(name="rope_prompt", op="rope", B=1, s_q=8192, H=128, d_nope=128, d_rope=64, layout="interleaved",
             scaling="plain", factor=1.0, original=0, base=10000.0, mscale=1.0, far=8192, given=False, pad=0),
        # a decode step of 64 requests: one token each, now and then a new page
        dict(name="pages_step", op="pages", B=64, page_size=64, longest=8192, grow=1, release=0.0, fresh=0.0),
        # a scheduler's turn on 512 requests: prompts admitted, some requests finished, drafts taken back
        dict(name="pages_turn", op="pages", B=512, page_size=64, longest=16384, grow=4, release=0.1, fresh=0.1),
        # 8,191 requests admitted at once: millions of new tokens
        dict(name="pages_admit", op="pages", B=8191, page_size=128, longest=2048, grow=700, release=0.02, fresh=0.4),
        # the new latents of a decode step of 64 sequences, into a paged bf16 cache
        dict(name="store_decode", op="store", tokens=64, d_c=512, d_rope=64, page_size=64, kv="bf16", norm=True,
             layout="interleaved", far=32768, lead=0),
        # the new latents of a speculative step with an FP8 cache, a slice of a wider projection's rows
        dict(name="store_verify_fp8", op="store", tokens=501, d_c=512, d_rope=64, page_size=64, kv="e4m3", norm=True,
             layout="interleaved", far=131072, lead=1024),
        # a batch of prompts
        dict(name="store_prompt", op="store", tokens=32768, d_c=512, d_rope=64, page_size=64, kv="bf16", norm=True,
             layout="half", far=32768, lead=0),
        # the output projection of a decode step (128 heads x 128 values -> 7168), added to the residual stream
        dict(name="linear_decode", op="linear", M=64, K=16384, N=7168, bias=False, act="none", residual=True, pad=0),
        # an odd middle size with everything in the epilogue
        dict(name="linear_odd", op="linear", M=333, K=1000, N=1544, bias=True, act="gelu_tanh", residual=True, pad=8),
        # the output projection of a prompt
        dict(name="linear_prompt", op="linear", M=4096, K=16384, N=7168, bias=False, act="none", residual=True, pad=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["rope", "pages", "store", "linear"])
    if op == "rope":
        s_q = rng.choice([1, 1, 2, 3, 4, 7, _log_int(rng, 16, 4096)])
        scaling = rng.choice(["plain", "linear", "ntk", "yarn"])
        B, H = _log_int(rng, 1, 256), rng.choice([1, 5, 16, 40, 64, 128, 128])
        if B * s_q * H > 8192 * 128:
            B = max(1, 8192 * 128 // (s_q * H))
        return dict(op=op, B=B, s_q=s_q, H=H, d_nope=16 * rng.choice([0, 1, 3, 4, 8, 8, 8]),
                    d_rope=16 * rng.randint(1, 4), layout=rng.choice(["interleaved", "half"]), scaling=scaling,
                    factor=1.0 if scaling == "plain" else rng.choice([2.0, 4.0, 8.0, 40.0]),
                    original=rng.choice([2048, 4096, 8192]), base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    mscale=rng.choice([1.0, 1.0, 1.1386]), far=max(2 * s_q, _log_int(rng, 512, 1 << 30)),
                    given=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 24]))
    if op == "pages":
        B = _log_int(rng, 1, 8192)
        grow = _log_int(rng, 1, max(2, min(4096, 4000000 // B)))
        return dict(op=op, B=B, page_size=64 * rng.choice([1, 1, 1, 2, 4]),
                    longest=max(256, 2 * grow, min(_log_int(rng, 512, 32768), 16 * 1024 * 1024 // B)), grow=grow,
                    release=rng.choice([0.0, 0.05, 0.2]), fresh=rng.choice([0.0, 0.1, 0.5]))
    if op == "store":
        return dict(op=op, tokens=_log_int(rng, 1, 32768), d_c=64 * rng.choice([1, 2, 4, 5, 8, 8, 8]),
                    d_rope=16 * rng.choice([0, 1, 2, 3, 4, 4, 4]), page_size=64 * rng.randint(1, 3),
                    kv=rng.choice(["bf16", "e4m3"]), norm=rng.random() < 0.8,
                    layout=rng.choice(["interleaved", "half"]), far=_log_int(rng, 256, 1 << 28),
                    lead=rng.choice([0, 0, 8, 200, 1024]))
    M = _log_int(rng, 1, 4096)
    return dict(op=op, M=M, K=8 * _log_int(rng, 8, 2048), N=8 * _log_int(rng, 4, 896), bias=rng.random() < 0.5,
                act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), residual=rng.random() < 0.5,
                pad=rng.choice([0, 0, 8, 64]))


def work(case):
    op = case["op"]
    if op == "rope":
        tokens, width = case["B"] * case["s_q"], case["d_nope"] + case["d_rope"]
        return {"bytes": tokens * (4 * case["H"] * width + 4), "flops": 3 * tokens * case["H"] * case["d_rope"]}
    if op == "pages":
        # about what the drawn lengths come to: two lengths in, length, start and two words a token's entry out, the pages
        tokens = _room(case)
        pages = tokens / case["page_size"] + case["B"] * case["release"] * case["longest"] / 4 / case["page_size"]
        return {"bytes": 16 * case["B"] + 8 * tokens + 8 * pages, "flops": 0}
    if op == "store":
        width = case["d_c"] + case["d_rope"]
        return {"bytes": case["tokens"] * (2 * width + 8 + width * (2 if case["kv"] == "bf16" else 1))
                + 2 * case["d_c"] * case["norm"], "flops": case["tokens"] * (4 * case["d_c"] + 3 * case["d_rope"])}
    M, K, N = case["M"], case["K"], case["N"]
    return {"bytes": 2 * (M * K + K * N + M * N * (2 if case["residual"] else 1) + N * case["bias"]),
            "flops": 2 * M * K * N}


# -------------------------------------------------------------------------------------------------------- the inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _frequencies(case, d):
    """Angular frequencies of the d / 2 pairs, in 64 bits: what a program works out once per model."""
    i = torch.arange(d // 2, dtype=torch.float64)
    base, s = case.get("base", 10000.0), case.get("factor", 1.0)
    scaling = case.get("scaling", "plain")
    if scaling == "ntk":
        base = base * s ** (d / (d - 2))
    f = torch.exp(-(2.0 * i / d) * math.log(base))
    if scaling == "linear":
        f = f / s
    if scaling == "yarn":
        turns = [d * math.log(case["original"] / (n * 2.0 * math.pi)) / (2.0 * math.log(base)) for n in (32.0, 1.0)]
        low, high = max(math.floor(turns[0]), 0), min(math.ceil(turns[1]), d - 1)
        ramp = torch.clamp((i - low) / max(high - low, 0.001), 0.0, 1.0)
        f = f / s * ramp + f * (1.0 - ramp)
    return f.to(DEV)


def _room(case):
    """Entries of the token arrays: what the requests come to with four standard deviations to spare, as a captured step
    has a fixed room that it hardly ever fills."""
    B, grow = case["B"], case["grow"]
    return min(B * grow, int(B * (grow + 1) / 2 + 1.2 * grow * math.sqrt(B))) + 5


def prepare(case, seed):
    return {"rope": _prepare_rope, "pages": _prepare_pages, "store": _prepare_store,
            "linear": _prepare_linear}[case["op"]](case, seed)


def _mla():
    from mla_decode_attention_absorbed_gb300 import mla
    return mla


def _plan(case, d):
    m = _mla()
    return m.rope_plan(d, layout={"interleaved": m.ROPE_INTERLEAVED, "half": m.ROPE_HALF}[case["layout"]],
                       base=case.get("base", 10000.0),
                       scaling={"plain": m.ROPE_PLAIN, "linear": m.ROPE_LINEAR, "ntk": m.ROPE_NTK,
                                "yarn": m.ROPE_YARN}[case.get("scaling", "plain")],
                       factor=case.get("factor", 1.0), original_len=case.get("original", 0),
                       mscale=case.get("mscale", 1.0))


def _prepare_rope(case, seed):
    g = _generator(seed)
    B, s_q, H, width = case["B"], case["s_q"], case["H"], case["d_nope"] + case["d_rope"]
    x = _normal(g, (B, s_q, H * width + case["pad"]))[:, :, :H * width].unflatten(2, (H, width))
    lens = torch.randint(s_q, case["far"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    at = None
    if case["given"]:  # positions of their own: trees of drafts, packed prompts
        at = torch.randint(0, case["far"], (B, s_q), generator=g, device=DEV, dtype=torch.int32)
    st = dict(case=case, x=x, lens=lens, at=at, f=_frequencies(case, case["d_rope"]))
    if own:
        m = _mla()
        st["prob"] = m.Problem(B, H, s_q, 512, case["d_rope"], max(case["d_nope"], 16), 128, 1.0)
        st["plan"] = _plan(case, case["d_rope"])
    return st


def _prepare_pages(case, seed):
    g = _generator(seed)
    B, ps, longest, grow = case["B"], case["page_size"], case["longest"], case["grow"]

    def uniform():
        return torch.rand((B,), generator=g, device=DEV, dtype=torch.float64)

    old = (uniform() * (longest - grow)).floor()
    old = torch.where(uniform() < case["fresh"], torch.zeros_like(old), old)
    new = old + 1 + (uniform() * grow).floor()
    kind = uniform()
    # some requests end (all their pages come back), others give a few rejected tokens back
    new = torch.where(kind < case["release"] / 2, torch.zeros_like(new), new)
    back = torch.clamp(old - (uniform() * 100).floor(), min=0)
    new = torch.where((kind >= case["release"] / 2) & (kind < case["release"]), back, new)
    old, new = old.to(torch.int32), new.to(torch.int32)
    max_pages = -(-longest // ps)
    held = (old.long() + ps - 1) // ps
    pool = B * max_pages + 7
    ids = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    first = torch.cumsum(held, 0) - held
    col = torch.arange(max_pages, device=DEV)
    table = torch.where(col < held[:, None], ids[(first[:, None] + col).clamp(max=pool - 1)],
                        torch.full((), -1, device=DEV, dtype=torch.int32))
    n_held = int(held.sum())
    head = int(torch.randint(0, pool, (1,), generator=g, device=DEV))
    ring = torch.full((pool,), -1, device=DEV, dtype=torch.int32)
    ring[(head + torch.arange(pool - n_held, device=DEV)) % pool] = ids[n_held:]
    state = torch.tensor([head, pool - n_held], device=DEV, dtype=torch.int32)
    st = dict(case=case, old=old, new=new, table=table, ring=ring, state=state, max_tokens=_room(case))
    if own:
        st["pages"] = _mla().Pages(table, ring, page_size=ps)
    return st


def _prepare_store(case, seed):
    g = _generator(seed)
    T, d_c, d_rope, ps, lead = case["tokens"], case["d_c"], case["d_rope"], case["page_size"], case["lead"]
    width = d_c + d_rope
    rows = _normal(g, (T, lead + width))[:, lead:]
    weight = (1.0 + 0.2 * torch.randn((d_c,), generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None
    at = torch.randint(0, case["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
    pages = -(-T // ps) + 2
    slots = torch.randperm(pages * ps, generator=g, device=DEV)[:T].to(torch.int32)
    kv = torch.zeros((pages, ps, width), device=DEV,
                     dtype=torch.bfloat16 if case["kv"] == "bf16" else torch.float8_e4m3fn)
    st = dict(case=case, rows=rows, weight=weight, at=at, slots=slots, kv=kv, eps=1e-6, kv_scale=1.0 / 16.0)
    if d_rope:
        st["f"] = _frequencies(case, d_rope)
    if own:
        m = _mla()
        st["lens"] = torch.ones((T,), device=DEV, dtype=torch.int32)
        st["table"] = torch.zeros((T, 1), device=DEV, dtype=torch.int32)
        st["prob"] = m.Problem(T, 128, 1, d_c, d_rope, 128, 128, 1.0)
        st["cache"] = m.make_cache(st["prob"], kv, st["lens"], st["table"], ps, kv_scale=st["kv_scale"])
        st["plan"] = _plan(case, d_rope) if d_rope else None
    return st


def _prepare_linear(case, seed):
    g = _generator(seed)
    M, K, N = case["M"], case["K"], case["N"]
    return dict(case=case, x=_normal(g, (M, K + case["pad"]))[:, :K], w=_normal(g, (K, N), K ** -0.5),
                bias=_normal(g, (N,)) if case["bias"] else None,
                residual=_normal(g, (M, N)) if case["residual"] else None)


# ---------------------------------------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "pages": _own_pages, "store": _own_store, "linear": _own_linear}[op](state)
    return {"rope": _plain_rope, "pages": _plain_pages, "store": _plain_store, "linear": _plain_linear}[op](state)


def _own_rope(st):
    case = st["case"]
    out = _mla().rope(st["prob"], st["plan"], st["x"], positions=st["at"], seq_lens=None if case["given"] else st["lens"])
    return out


def _own_pages(st):
    new_state = _mla().pages_update(st["pages"], st["state"], st["old"], st["new"], st["max_tokens"])
    return dict(lens=new_state.seq_lens, state=new_state.ring_state, start=new_state.token_start,
                positions=new_state.positions, slots=new_state.slots, table=st["table"], ring=st["ring"])


def _own_store(st):
    _mla().latent_store(st["prob"], st["rows"], st["cache"], plan=st["plan"], norm_weight=st["weight"], eps=st["eps"],
                        positions=st["at"], slots=st["slots"])
    return st["kv"]


def _own_linear(st):
    m = _mla()
    act = {"none": m.ACT_NONE, "relu": m.ACT_RELU, "silu": m.ACT_SILU, "gelu": m.ACT_GELU,
           "gelu_tanh": m.ACT_GELU_TANH}[st["case"]["act"]]
    return m.linear(st["x"], st["w"], bias=st["bias"], residual=st["residual"], act=act)


def _rotate(x, at, f, layout, mscale):
    """x [..., d] rotated by the angles at * f: at broadcasts against x's leading dimensions."""
    angle = at.to(torch.float64)[..., None] * f
    cos, sin = (mscale * torch.cos(angle)).float(), (mscale * torch.sin(angle)).float()
    half = x.shape[-1] // 2
    x = x.float()
    if layout == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)


def _plain_rope(st):
    case, x = st["case"], st["x"]
    at = st["at"]
    if at is None:
        at = st["lens"][:, None] - case["s_q"] + torch.arange(case["s_q"], device=x.device)
    turned = _rotate(x[..., case["d_nope"]:], at[:, :, None], st["f"], case["layout"], case["mscale"])
    if case["d_nope"] == 0:
        return turned.to(torch.bfloat16)
    return x[..., :case["d_nope"]].contiguous(), turned.to(torch.bfloat16)


def _plain_pages(st):
    ps, table, ring = st["case"]["page_size"], st["table"], st["ring"]
    old, new, pool = st["old"].long(), st["new"].long(), ring.numel()
    B, max_pages = table.shape
    head, count = st["state"][0].long(), st["state"][1].long()
    valid = (old >= 0) & (new >= 0) & (old <= max_pages * ps) & (new <= max_pages * ps)
    zero = torch.zeros_like(old)
    had, has = (old + ps - 1) // ps, (new + ps - 1) // ps
    fresh = torch.where(valid, (new - old).clamp(min=0), zero)
    need = torch.where(valid, (has - had).clamp(min=0), zero)
    freed = torch.where(valid, (had - has).clamp(min=0), zero)
    token_end, need_end, freed_end = fresh.cumsum(0), need.cumsum(0), freed.cumsum(0)
    fits = valid & ((need == 0) | (need_end <= count)) & ((fresh == 0) | (token_end <= st["max_tokens"]))
    taken = torch.where(fits & (need > 0), need_end, zero).amax()
    lens = torch.where(fits, new, old).to(torch.int32)
    start = torch.cat((zero[:1], token_end)).to(torch.int32)
    # pages taken from the ring's head, into the columns after the ones held
    col = torch.arange(max_pages, device=table.device)[None, :]
    take = fits[:, None] & (col >= had[:, None]) & (col < has[:, None])
    page = ring[((head + (need_end - need)[:, None] + col - had[:, None]) % pool)]
    give = valid[:, None] & (col >= has[:, None]) & (col < had[:, None])
    after = torch.where(take, page, table)
    # pages given back, behind the ring's tail; entry `pool` takes what is not given back
    to = torch.where(give, (head + count + (freed_end - freed)[:, None] + col - has[:, None]) % pool, pool)
    ring_after = torch.cat((ring, ring[:1])).scatter(0, to.flatten(), table.flatten())[:pool]
    state = torch.stack(((head + taken) % pool, count - taken + freed_end[-1])).to(torch.int32)
    # every new token's position and row of the pool
    t = torch.arange(st["max_tokens"], device=table.device)
    of = torch.searchsorted(token_end, t, right=True)
    at = of.clamp(max=B - 1)
    pos = old[at] + t - (token_end - fresh)[at]
    there = (of < B) & fits[at]
    held_page = after[at, (pos // ps).clamp(0, max_pages - 1)].long()
    positions = torch.where(there, pos, -1).to(torch.int32)
    slots = torch.where(there, held_page * ps + pos % ps, -1).to(torch.int32)
    return dict(lens=lens, state=state, start=start, positions=positions, slots=slots, table=after, ring=ring_after)


def _plain_store(st):
    case, rows = st["case"], st["rows"]
    c = rows[:, :case["d_c"]].float()
    if st["weight"] is not None:
        c = c * torch.rsqrt(c.square().mean(dim=-1, keepdim=True) + st["eps"]) * st["weight"].float()
    if case["d_rope"]:
        k = _rotate(rows[:, case["d_c"]:], st["at"], st["f"], case["layout"], case.get("mscale", 1.0))
        c = torch.cat((c, k), dim=-1)
    kv = st["kv"]
    flat = kv.view(-1, kv.shape[-1])
    if kv.dtype == torch.bfloat16:
        flat[st["slots"].long()] = c.to(torch.bfloat16)
    else:
        codes = (c / st["kv_scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        flat.view(torch.uint8)[st["slots"].long()] = codes.view(torch.uint8)
    return kv


def _plain_linear(st):
    y = st["x"].float() @ st["w"].float()
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


# ------------------------------------------------------------------------------------------- from the definition, 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        x = st["x"].double()
        turned = torch.empty(x.shape[:-1] + (case["d_rope"],), dtype=torch.float64, device=DEV)
        if st["at"] is not None:
            at = st["at"].double()
        else:
            at = st["lens"].double()[:, None] + torch.arange(-case["s_q"], 0, device=DEV)
        _exact_turn(case, x[..., case["d_nope"]:], at[:, :, None], turned)
        return (x[..., :case["d_nope"]].clone(), turned) if case["d_nope"] else turned
    if case["op"] == "store":
        d_c, x = case["d_c"], st["rows"].double()
        row = torch.empty_like(x)
        row[:, :d_c] = x[:, :d_c]
        if case["norm"]:
            row[:, :d_c] /= (torch.linalg.vector_norm(x[:, :d_c], dim=1, keepdim=True) ** 2 / d_c + st["eps"]) ** 0.5
            row[:, :d_c] *= st["weight"].double()
        if case["d_rope"]:
            _exact_turn(case, x[:, d_c:], st["at"].double(), row[:, d_c:])
        if case["kv"] != "bf16":
            row = torch.clamp(row / st["kv_scale"], -448.0, 448.0)
        kv = torch.zeros(st["kv"].shape, dtype=torch.float64, device=DEV)
        kv.view(-1, kv.shape[-1]).index_copy_(0, st["slots"].long(), row)
        return kv
    if case["op"] == "linear":
        y = torch.matmul(st["x"].double(), st["w"].double())
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
    return None  # pages: whole numbers


def _exact_turn(case, x, at, out):
    """out = x with pair i of the layout multiplied, as a complex number, by mscale * exp(i * at * f_i)."""
    d = case["d_rope"]
    base, s, scaling = case.get("base", 10000.0), case.get("factor", 1.0), case.get("scaling", "plain")
    for i in range(d // 2):
        f = base ** (-2.0 * i / d)
        if scaling == "linear":
            f = f / s
        elif scaling == "ntk":
            f = (base * s ** (d / (d - 2.0))) ** (-2.0 * i / d)
        elif scaling == "yarn":
            # pairs that turn more than 32 times within the original length keep their frequency, those that turn
            # less than once are stretched by s, the ones between go over linearly in their index
            fast = d * math.log(case["original"] / (64.0 * math.pi)) / math.log(base) / 2.0
            slow = d * math.log(case["original"] / (2.0 * math.pi)) / math.log(base) / 2.0
            fast, slow = max(math.floor(fast), 0), min(math.ceil(slow), d - 1)
            kept = 1.0 - min(max((i - fast) / max(slow - fast, 0.001), 0.0), 1.0)
            f = f * kept + (f / s) * (1.0 - kept)
        p, q = (2 * i, 2 * i + 1) if case["layout"] == "interleaved" else (i, i + d // 2)
        z = torch.complex(x[..., p], x[..., q]) * torch.polar(torch.full_like(at, case.get("mscale", 1.0)), at * f)
        out[..., p], out[..., q] = z.real, z.imag
