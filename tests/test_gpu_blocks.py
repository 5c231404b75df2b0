"""The 8-bit operators with scales by blocks of 128 on the GPU against plain 64-bit implementations (oracle/layer.py):
mla_quantize, mla_linear_fp8, mla_latent_store into rows of blocks, mla_latent_load, and a run of them together with the
attention.

Tolerances count roundings: half a step is 2^-8 of a bf16 value, 2^-4 of an E4M3 code (2^-10 among its subnormals) and 2^-24
of an fp32 value."""
import math
import threading

import pytest
import torch

from helpers import LINEAR_FP8_FORMS, linear_fp8_form, within_tolerance
from mla_decode_attention_absorbed_gb300 import build, mla
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = "cuda"
ACTS = {"none": mla.ACT_NONE, "relu": mla.ACT_RELU, "silu": mla.ACT_SILU, "gelu": mla.ACT_GELU,
        "gelu_tanh": mla.ACT_GELU_TANH}
BF16, I32, F32, E4M3 = torch.bfloat16, torch.int32, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.load()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF16)


def close(got, want, tol, what=""):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN differ"
    ok = torch.isnan(want) | (got == want) | ((got - want).abs() <= tol)
    if not bool(ok.all()):
        at = tuple(int(i) for i in (~ok).nonzero()[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} off, first at {at}: {got[at]} for {want[at]}, "
                             f"allowed {tol[at] if torch.is_tensor(tol) else tol}")


def close_codes(got, want, rel=0.0, what=""):
    """Codes of quotients that fp32 arithmetic has off by `rel` of their value: half a step more."""
    close(got.float(), want, want.abs() * (2.0 ** -4 + 1.1 * rel) + 2.0 ** -10, what)


def wide_rows(t, pad, fill):
    """t's values on the GPU in rows that are `pad` wider, and those whole rows."""
    w = torch.full((t.shape[0], t.shape[1] + pad), fill).to(t.dtype)
    w[:, :t.shape[1]] = t
    w = w.to(DEV)
    return w[:, :t.shape[1]], w


def f32(v):
    """v rounded to fp32."""
    return float(torch.tensor(v, dtype=F32))


LEAST = f32(2.0 ** -100 / 448)  # the scale of a block of zeros


def problem(B=2, H=16, s_q=1, d_c=512, d_rope=64, d_nope=128, d_v=128):
    return mla.Problem(B, H, s_q, d_c, d_rope, d_nope, d_v, (d_nope + d_rope) ** -0.5)


# --------------------------------------------------------------------------------------------------------- quantize
def fp32_blocks(x, rows):
    """Codes and scales of bf16 values in fp32, operation by operation as documented (CPU)."""
    M, K = x.shape
    top = torch.empty(-(-M // rows), -(-K // 128))
    for i in range(top.shape[0]):
        for j in range(top.shape[1]):
            top[i, j] = x[rows * i:rows * i + rows, 128 * j:128 * j + 128].float().abs().max()
    top = top.clamp(min=2.0 ** -100)
    # (448.0 / top would be top's reciprocal times 448, two roundings)
    unit = torch.full_like(top, 448.0).div(top).repeat_interleave(rows, 0)[:M].repeat_interleave(128, 1)[:, :K]
    return (x.float() * unit).to(E4M3), top / 448.0


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("M,K,px,pc", [
    (1, 16, 0, 0), (1, 128, 8, 16), (7, 144, 0, 0), (8, 112, 24, 16), (9, 1008, 8, 0), (127, 256, 0, 32), (128, 128, 0, 0),
    (129, 400, 8, 16), (300, 272, 0, 0), (64, 7168, 0, 0), (3, 16400, 0, 0)])
def test_quantize(M, K, px, pc, rows):
    """Without a norm every step is one fp32 operation of known rounding: bit for bit."""
    g = gen(M + K)
    x = (torch.randn(M, K, generator=g) * torch.exp(2 * torch.randn(M, K, generator=g))).to(BF16)
    xd, _ = wide_rows(x, px, float("nan"))
    codes, whole = wide_rows(torch.zeros(M, K).to(E4M3), pc, 1.5)
    scales = torch.zeros((-(-K // 128), M) if rows == 1 else (-(-M // 128), -(-K // 128)), device=DEV)
    got = mla.quantize(xd, block_rows=rows, codes=codes, scales=scales)
    assert got[0] is codes and got[1] is scales
    want, want_scales = fp32_blocks(x, rows)
    assert torch.equal(codes.cpu().view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(scales.cpu(), want_scales.t() if rows == 1 else want_scales)
    assert bool((whole[:, K:].float() == 1.5).all()), "bytes behind K are left as they were"
    quotient, exact = layer.blocks(x, rows)
    close(scales.t() if rows == 1 else scales, exact, exact * 2.0 ** -24)
    close_codes(codes, quotient, 2.0 ** -22)
    again = mla.quantize(xd, block_rows=rows)
    assert torch.equal(again[0].view(torch.uint8), codes.contiguous().view(torch.uint8)) and torch.equal(again[1], scales)


@pytest.mark.parametrize("M,K,px", [
    (1, 16, 0), (2, 128, 8), (9, 256, 0), (17, 272, 0), (33, 512, 24), (5, 1008, 0), (6, 1024, 0), (7, 1040, 8), (40, 2048, 0), (3, 4112, 0),
    (64, 7168, 0), (5, 8192, 0), (4, 8208, 8), (3, 16384, 0), (2, 16400, 0), (2, 40000, 0), (1, 1 << 20, 0)])
def test_quantize_after_the_norm(M, K, px):
    """The sum of K squares in fp32 is off by at most K 2^-24 of it (each addition by 2^-24 of a part of it), its root by half
    that; 2^-21 covers the root's estimate, the division by K and two products."""
    g = gen(M + K + 1)
    x = (torch.randn(M, K, generator=g) * torch.exp(torch.randn(K, generator=g))).to(BF16)
    weight = (1 + 0.3 * torch.randn(K, generator=g)).to(BF16)
    xd, _ = wide_rows(x, px, float("nan"))
    codes, scales = mla.quantize(xd, norm_weight=weight.to(DEV), eps=1e-5)
    quotient, exact = layer.blocks(layer.rms_norm(x, weight, 1e-5), 1)
    rel = K * 2.0 ** -25 + 2.0 ** -21
    close(scales.t(), exact, exact * (rel + 2.0 ** -24), "scales")
    # a quotient is a value over its own block's largest: the row's factor falls out but for its rounding
    close_codes(codes, quotient, 2.0 ** -21, "codes")


def test_quantize_special_values():
    """Zeros, values below 2^-100, the largest ones, NaN and infinities, each in a block of its own."""
    x = torch.zeros(8, 256, dtype=BF16)
    x[1, :3] = torch.tensor([2.0 ** -120, -2.0 ** -126, 2.0 ** -133])
    x[2, 5], x[2, 6] = 3.3895e38, -1.0
    x[3, 0], x[3, 1], x[3, 2] = float("nan"), 2.0, -0.5
    x[4, 0], x[4, 1] = float("inf"), 2.0
    x[5, 0] = float("-inf")
    x[6, :128] = float("nan")
    x[7, :128] = torch.arange(128) / 128
    x[:, 128:] = 1.0  # the second block knows nothing of the first
    for norm in (False, True):
        kw = dict(norm_weight=torch.ones(256, dtype=BF16, device=DEV), eps=0.0) if norm else {}
        if norm:
            x[3:7] = 1.0  # a NaN or an infinity is in the row's sum: the whole row's
            x[6, 200] = float("nan")
        codes, scales = mla.quantize(x.to(DEV), **kw)
        codes, scales = codes.cpu().float(), scales.cpu()
        assert bool((codes[0, :128] == 0).all()) and float(scales[0, 0]) == LEAST and bool((codes[0, 128:] == 448).all())
        if norm:
            assert bool(torch.isnan(codes[6]).all())
            continue
        # 2^-120 in units of 2^-100 / 448 is 448 2^-20: below half the smallest code
        assert bool((codes[1, :128] == 0).all()) and float(scales[0, 1]) == LEAST
        assert float(codes[2, 5]) == 448 and float(codes[2, 6]) == 0 and math.isfinite(float(scales[0, 2]))
        assert bool(torch.isnan(codes[3, 0])) and codes[3, 1:4].tolist() == [448.0, -112.0, 0.0] and float(scales[0, 3]) == f32(2.0 / 448)
        for r in (4, 5):  # an infinity's block: infinite scale, its own code NaN, the others 0
            assert float(scales[0, r]) == math.inf and bool(torch.isnan(codes[r, 0])) and bool((codes[r, 1:128] == 0).all())
        assert bool(torch.isnan(codes[6, :128]).all()) and float(scales[0, 6]) == LEAST
        assert bool((codes[:, 128:] == 448).all()) and bool((scales[1] == 1 / 448).all())


def test_quantize_squares_special_values():
    x = torch.zeros(130, 144, dtype=BF16)
    x[3, 5], x[3, 6], x[129, 0], x[129, 143] = float("nan"), 4.0, float("inf"), -2.0
    codes, scales = (t.cpu() for t in mla.quantize(x.to(DEV), block_rows=128))
    assert scales.tolist() == [[f32(4 / 448), LEAST], [math.inf, f32(2 / 448)]]
    assert bool(torch.isnan(codes.float()[3, 5])) and float(codes.float()[3, 6]) == 448 and float(codes.float()[129, 143]) == -448
    assert bool(torch.isnan(codes.float()[129, 0])) and int((codes.float() != 0).sum()) == 4


def test_quantize_no_rows():
    for rows in (1, 128):
        codes, scales = mla.quantize(torch.empty(0, 256, dtype=BF16, device=DEV), block_rows=rows)
        assert codes.shape == (0, 256) and scales.shape == ((2, 0) if rows == 1 else (0, 2))


@pytest.mark.parametrize("M,K", [(65535 * 128, 16), (1, 1 << 20), (300, 1 << 20)])
def test_quantize_longest_sides(M, K):
    """The ends of the ranges, compared at rows and columns spread over them."""
    g = torch.Generator(device=DEV).manual_seed(M + K)
    x = torch.randn(M, K, generator=g, device=DEV).to(BF16)
    for rows in (1, 128):
        codes, scales = mla.quantize(x, block_rows=rows)
        for i in {0, M // 2 // rows, (M - 1) // rows}:
            for j in {0, K // 2 // 128, (K - 1) // 128}:
                part = (slice(rows * i, rows * i + rows), slice(128 * j, 128 * j + 128))
                want, want_scale = fp32_blocks(x[part].cpu(), rows)
                assert torch.equal(codes[part].cpu().float(), want.float())
                assert float(scales[j, i] if rows == 1 else scales[i, j]) == float(want_scale)


# ------------------------------------------------------------------------------------------------------- linear_fp8
def whole_codes(g, *shape, most=4):
    return torch.randint(-most, most + 1, shape, generator=g).float().to(E4M3)


def powers(g, *shape, least=-2, most=2):
    return torch.exp2(torch.randint(least, most + 1, shape, generator=g).float())


def operands(g, M, K, N, exact):
    """Codes and scales: whole numbers and powers of two (every sum exact in fp32 while K times 16 times 16 is below 2^24),
    or values as quantising leaves them."""
    if exact:
        return whole_codes(g, M, K), powers(g, -(-K // 128), M), whole_codes(g, N, K), powers(g, -(-N // 128), -(-K // 128))
    x, xs = fp32_blocks(randn(g, M, K), 1)
    w, ws = fp32_blocks(randn(g, N, K, std=K ** -0.5), 128)
    return x, xs.t().contiguous(), w, ws


def product_tolerance(x, xs, w, ws, pre, want):
    """fp32 sums of K terms are off by at most K 2^-23 of the terms' absolute sum (as those of mla_linear), a block's scale
    and its product by 2^-22; the activations stretch that by at most 1.13 and add 2^-17 of their value; one rounding."""
    terms = layer.linear_fp8(x.float().abs(), xs, w.float().abs(), ws)
    tol = 1.13 * (x.shape[1] * 2.0 ** -23 + 2.0 ** -22) * terms + pre.abs() * 2.0 ** -17 + 2.0 ** -22
    return tol + want.abs() * 2.0 ** -8 * 1.01


PRODUCT_CASES = [
    # M, K, N, bias, act, residual, paddings of x (bytes), out and residual rows
    (1, 16, 8, False, "none", False, 0, 0, 0), (1, 128, 128, True, "relu", True, 16, 8, 8), (2, 144, 136, True, "silu", False, 0, 16, 0),
    (7, 1008, 264, False, "gelu", True, 16, 0, 8), (8, 4096, 128, True, "gelu_tanh", True, 0, 0, 0), (15, 256, 72, True, "none", True, 0, 8, 0),
    (17, 128, 1544, False, "none", True, 0, 8, 0), (32, 192, 64, True, "none", False, 0, 0, 0), (33, 528, 2056, True, "gelu", True, 48, 8, 8),
    (64, 16384, 256, False, "none", True, 0, 0, 0), (65, 272, 392, True, "silu", True, 0, 0, 0), (127, 2048, 1000, False, "relu", False, 0, 0, 64),
    (128, 64, 8, True, "gelu_tanh", True, 0, 0, 0), (129, 1008, 136, True, "none", True, 16, 0, 0), (256, 128, 4096, False, "none", False, 0, 0, 0),
    (333, 1008, 1544, True, "gelu_tanh", True, 16, 8, 8), (1025, 80, 520, True, "silu", True, 0, 24, 0),
    (4096, 512, 2048, False, "none", True, 0, 0, 0), (5000, 144, 1160, True, "gelu", True, 0, 0, 0),
    (5000, 1040, 6000, True, "silu", True, 16, 8, 8), (700, 2064, 6024, False, "none", True, 0, 0, 0),
    (250, 8208, 7000, True, "gelu_tanh", True, 0, 8, 8), (1264, 6800, 416, False, "none", True, 16, 0, 0), (8, 1008, 20480, True, "relu", True, 0, 8, 0),
]


def check_product(M, K, N, bias, act, residual, px, po, pr, exact, seed=0):
    g = gen(M + K + N + seed)
    x, xs, w, ws = operands(g, M, K, N, exact)
    b = randn(g, N) if bias else None
    r = randn(g, M, N, std=2.0) if residual else None
    out, whole = wide_rows(torch.full((M, N), 5.0, dtype=BF16), po, 9.0)
    got = mla.linear_fp8(wide_rows(x, px, float("nan"))[0], xs.to(DEV), w.to(DEV), ws.to(DEV), bias=None if b is None else b.to(DEV),
                         residual=None if r is None else wide_rows(r, pr, float("nan"))[0], act=ACTS[act], out=out)
    assert bool((whole[:, N:] == 9).all()), "columns behind N are left as they were"
    if exact and act in ("none", "relu"):
        full = layer.linear_fp8(x, xs, w, ws).float()  # exact
        if b is not None:
            full = full + b.float()
        full = full.clamp(min=0) if act == "relu" else full
        if r is not None:
            full = full + r.float()
        assert torch.equal(got.cpu(), full.to(BF16))
        return
    want = layer.linear_fp8(x, xs, w, ws, b, r, act)
    close(got, want, product_tolerance(x, xs, w, ws, layer.linear_fp8(x, xs, w, ws, b, None, act), want))


@pytest.mark.parametrize("M,K,N,bias,act,residual,px,po,pr", PRODUCT_CASES)
def test_linear_fp8(M, K, N, bias, act, residual, px, po, pr):
    for exact in (True, False):
        check_product(M, K, N, bias, act, residual, px, po, pr, exact)


@pytest.mark.parametrize("form", LINEAR_FP8_FORMS, ids=lambda f: "x".join(map(str, f)))
def test_linear_fp8_every_form(form):
    """Each way a product is cut (on 152 SMs; on another card the same sizes, cut as it has it), rows, K and columns ending
    inside a tile."""
    M, K, N = LINEAR_FP8_FORMS[form]
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert linear_fp8_form(M, K, N) == form
    check_product(M, K, N, True, "none", True, 16, 8, 8, True, 1)
    check_product(M, K, N, True, "silu", True, 0, 0, 0, False, 2)


@pytest.mark.parametrize("M", [1025, 2305, 4360])
def test_linear_fp8_many_tiles_of_tokens(M):
    """More tiles of tokens than go through the columns together, and a rest of them."""
    check_product(M, 144, 1160, True, "none", True, 16, 8, 8, True, 3)
    check_product(M, 272, 520, False, "none", False, 0, 0, 0, False, 4)


def test_linear_fp8_of_what_quantize_gives():
    """The two calls one after the other, with nothing between them, against the product of the codes read back."""
    g = gen(5)
    for M, K, N in ((64, 7168, 576), (333, 1008, 1544), (1, 16384, 136)):
        x, weight = randn(g, M, K).to(DEV), (1 + 0.2 * torch.randn(K, generator=g)).to(BF16).to(DEV)
        w, ws = mla.quantize(randn(g, N, K, std=K ** -0.5).to(DEV), block_rows=128)
        for _ in range(3):
            c, s = mla.quantize(x, norm_weight=weight)
            got = mla.linear_fp8(c, s, w, ws)
        args = [t.cpu() for t in (c, s, w, ws)]
        want = layer.linear_fp8(*args)
        close(got, want, product_tolerance(*args, want, want))


def test_linear_fp8_in_place_on_the_residual_stream():
    g = gen(31)
    for M, K, N in ((3, 4096, 264), (300, 64, 520), (4096, 128, 1536), (64, 16384, 1024), (250, 8208, 7000)):
        x, xs, w, ws = (t.to(DEV) for t in operands(g, M, K, N, False))
        rd = randn(g, M, N).to(DEV)
        apart = mla.linear_fp8(x, xs, w, ws, residual=rd)
        mla.linear_fp8(x, xs, w, ws, residual=rd, out=rd)
        assert torch.equal(rd, apart)


def test_linear_fp8_repeats_bit_for_bit():
    g = gen(32)
    for M, K, N in ((64, 16384, 1024), (333, 1008, 1544), (1, 8192, 264), (8, 1008, 20480), (529, 2928, 8232), (166, 2912, 20104)):
        args = [t.to(DEV) for t in operands(g, M, K, N, False)]
        a = mla.linear_fp8(*args)
        for _ in range(4):
            assert torch.equal(mla.linear_fp8(*args), a)


def test_linear_fp8_rows_do_not_know_their_neighbours():
    """A row of x gives the same alone, among 7 and among 128 others whose rows are NaN: what lies in a tile beside it is
    never part of its sums (the same cut: K in one part)."""
    g = gen(34)
    K, N = 256, 136
    x, xs, w, ws = operands(g, 130, K, N, False)
    w, ws = w.to(DEV), ws.to(DEV)
    alone = mla.linear_fp8(x[:1].to(DEV), xs[:, :1].contiguous().to(DEV), w, ws)
    x = x.clone()
    x[1:] = torch.full((129, K), float("nan")).to(E4M3)
    for M in (2, 7, 8, 9, 128, 130):
        y = mla.linear_fp8(x[:M].to(DEV), xs[:, :M].contiguous().to(DEV), w, ws)
        assert torch.equal(y[:1], alone) and bool(torch.isnan(y[1:]).all()), M


def test_linear_fp8_special_values():
    """NaN codes and infinite scales show in the rows (of x) or columns (of w) they belong to, and nowhere else."""
    g = gen(33)
    M, K, N = 20, 272, 264
    x, xs, w, ws = operands(g, M, K, N, False)
    x, xs, w, ws = x.float(), xs.clone(), w.float(), ws.clone()
    x[3, 5], x[7, 271], w[70, 9] = float("nan"), float("nan"), float("nan")
    xs[1, 11], ws[2, 0] = float("inf"), float("nan")
    x, w = x.to(E4M3), w.to(E4M3)
    got = mla.linear_fp8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV)).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[3], bad[7], bad[11], bad[:, 70], bad[:, 256:] = True, True, True, True, True
    assert torch.equal(~torch.isfinite(got), bad)
    assert bool(torch.isnan(got[3]).all()) and bool(torch.isnan(got[:, 256:]).all())


def test_linear_fp8_no_rows():
    out = mla.linear_fp8(torch.empty(0, 128, dtype=E4M3, device=DEV), torch.empty(1, 0, device=DEV),
                         torch.zeros(128, 128, device=DEV).to(E4M3), torch.ones(1, 1, device=DEV))
    assert out.shape == (0, 128)


@pytest.mark.parametrize("M,K,N", [(1, 1 << 20, 8), (1, 16, 1 << 20), (65535 * 128, 16, 8), (130, 64, 8 * 131071)])
def test_linear_fp8_longest_sides(M, K, N):
    """Whole numbers, so that every sum is exact: the ends of each size's range."""
    g = torch.Generator(device=DEV).manual_seed(M + K)
    x = torch.randint(-1, 2, (M, K), generator=g, device=DEV).float().to(E4M3)
    w = torch.randint(-1, 2, (N, K), generator=g, device=DEV).float().to(E4M3)
    xs = torch.ones(-(-K // 128), M, device=DEV)
    ws = torch.ones(-(-N // 128), -(-K // 128), device=DEV)
    want = (x.to(BF16).double() @ w.to(BF16).double().t()).to(F32).to(BF16)
    assert torch.equal(mla.linear_fp8(x, xs, w, ws), want)


def test_linear_fp8_offsets_past_32_bits():
    """140,000 x 32,768 outputs (4.6e9) and the last rows of x far into memory, against the same rows alone."""
    g = torch.Generator(device=DEV).manual_seed(92)
    M, K, N = 140000, 128, 32768
    x = torch.randn(M, K, generator=g, device=DEV).to(E4M3)
    w = torch.randn(N, K, generator=g, device=DEV).to(E4M3)
    xs, ws = torch.rand(1, M, generator=g, device=DEV), torch.rand(N // 128, 1, generator=g, device=DEV)
    y = mla.linear_fp8(x, xs, w, ws)
    for rows in (slice(0, 300), slice(M - 300, M)):
        assert torch.equal(y[rows], mla.linear_fp8(x[rows], xs[:, rows].contiguous(), w, ws))
    del y
    wide = torch.empty(200, 1 << 25, dtype=E4M3, device=DEV)  # rows 32 MB apart: 6.7e9 bytes
    wide[:, :K] = x[:200]
    assert torch.equal(mla.linear_fp8(wide[:, :K], xs[:, :200].contiguous(), w, ws),
                       mla.linear_fp8(x[:200], xs[:, :200].contiguous(), w, ws))


TIMEOUT_CASES = [
    # M, K, N: whole tiles, clusters, pairs in several rounds, whole tiles and a shared one, clusters of pairs
    (333, 1008, 1544), (64, 16384, 1024), (3, 65536, 136), (8, 4112, 20480), (5000, 1040, 6000), (250, 8208, 7000),
    (529, 2928, 8232), (171, 9664, 3088), (1039, 4544, 4904), (397, 18272, 1352), (166, 2912, 20104), (153, 3872, 1448),
    (262, 10896, 3768), (130, 11632, 23432), (993, 11760, 608), (140, 7536, 5032), (145, 4304, 20296), (135, 8144, 2472),
]


@pytest.mark.parametrize("M,K,N", TIMEOUT_CASES)
def test_linear_fp8_wait_timeout_reported_and_recovered(M, K, N):
    """With a short bound on the waits for work, some of them run out, at once or on the way: the call ends, the status
    word says so, every output is NaN or what it should be (whole numbers: exact sums), and calls after it are clean."""
    g = gen(M + K + N + 7)
    x, w = whole_codes(g, M, K, most=1).to(DEV), whole_codes(g, N, K, most=1).to(DEV)
    xs, ws = torch.ones(-(-K // 128), M, device=DEV), torch.ones(-(-N // 128), -(-K // 128), device=DEV)
    residual = torch.randint(-8, 9, (M, N), generator=g).to(BF16).to(DEV)
    status = torch.zeros(1, dtype=I32, device=DEV)
    want = mla.linear_fp8(x, xs, w, ws, residual=residual, status=status)
    assert int(status) == 0
    seen = 0
    try:
        for ns in (1, 200, 1000, 3000, 10000):
            mla.set_wait_limit_ns(ns)
            for _ in range(3):
                status.zero_()
                out = torch.full((M, N), 77.0, dtype=BF16, device=DEV)
                start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
                start.record()
                mla.linear_fp8(x, xs, w, ws, residual=residual, status=status, out=out)
                end.record()
                torch.cuda.synchronize()
                assert start.elapsed_time(end) < 1000.0
                lost = torch.isnan(out)
                assert torch.equal(torch.where(lost, want, out), want)
                assert int(status) in (0, 8) and (int(status) == 8 or not bool(lost.any()))
                seen += int(status) == 8
    finally:
        mla.set_wait_limit_ns(0)
    assert seen > 0
    status.zero_()
    assert torch.equal(mla.linear_fp8(x, xs, w, ws, residual=residual, status=status), want) and int(status) == 0


# ------------------------------------------------------------------------------------------------------------ store
def blocks_of(rows, d_c, d_rope):
    """Codes, scales (all four) and keys of rows of blocks, uint8 [..., row] on the CPU."""
    rows = rows.cpu()
    return (rows[..., :d_c].contiguous().view(E4M3).double(), rows[..., d_c:d_c + 16].contiguous().view(F32).double(),
            rows[..., d_c + 16:].contiguous().view(BF16).double())


def store_case(g, T, d_c, d_rope, norm, lead):
    rows = randn(g, T, lead + d_c + d_rope)
    weight = (1 + 0.3 * torch.randn(d_c, generator=g)).to(BF16) if norm else None
    return rows, rows[:, lead:], weight


def check_store(new, x, weight, at, freq, half, d_c, d_rope):
    """As test_quantize for the latent; the key as mla_latent_store's bf16 rows: half a step, and 2^-20 of the pair's length for
    angle and products."""
    codes, scales, keys = blocks_of(new, d_c, d_rope)
    quotient, exact = layer.blocks(layer.rms_norm(x[:, :d_c], weight, 1e-5), 1)
    rel = d_c * 2.0 ** -25 + 2.0 ** -21 if weight is not None else 2.0 ** -23
    n = exact.shape[1]
    close(scales[:, :n], exact, exact * rel, "scales")
    assert bool((scales[:, n:] == 0).all()), "scales of no value are 0"
    close_codes(codes, quotient, rel, "codes")
    if d_rope:
        k = x[:, d_c:].double()
        if freq is None:
            assert torch.equal(keys, k)
        else:
            want = layer.rotate(x[:, d_c:], at, freq, half)
            p, q = layer.pairs(d_rope, half)
            slack = torch.empty_like(k)
            slack[:, p] = slack[:, q] = (k[:, p].abs() + k[:, q].abs()) * (2.0 ** -20 + at.double()[:, None] * torch.tensor(freq).double() * 2.0 ** -51)
            close(keys, want, want.abs() * 2.0 ** -8 * 1.01 + slack, "keys")


@pytest.mark.parametrize("B,s_q,d_c,d_rope,ps,norm,half,turned,with_slots,lead", [
    (1, 1, 64, 0, 64, False, False, False, True, 0), (3, 2, 64, 16, 64, True, False, True, True, 8), (5, 1, 128, 32, 128, True, True, True, True, 0),
    (7, 3, 192, 48, 64, True, False, True, False, 16), (64, 1, 512, 64, 64, True, False, True, True, 0), (40, 5, 512, 64, 192, True, True, True, True, 1024),
    (9, 4, 320, 64, 0, True, True, True, False, 0), (3, 300, 512, 64, 64, False, False, True, True, 200), (2, 7, 448, 16, 0, False, False, False, False, 0),
    (6, 1, 384, 0, 64, True, False, False, False, 0)])
def test_store_in_blocks(B, s_q, d_c, d_rope, ps, norm, half, turned, with_slots, lead):
    """Paged (ps > 0) and contiguous caches, by slots and by the lengths; rows of no token are left as they were."""
    g = gen(B + s_q + d_c)
    T, prob = B * s_q, problem(B, 16, s_q, d_c=d_c, d_rope=d_rope)
    row = mla.latent_row_bytes(prob)
    whole, x, weight = store_case(g, T, d_c, d_rope, norm, lead)
    cap = 3 * max(ps, 64) if s_q < 100 else 320 // max(ps, 64) * max(ps, 64) + max(ps, 64)
    lens = torch.randint(s_q, cap + 1, (B,), generator=g, dtype=I32)
    at = (lens.long()[:, None] - s_q + torch.arange(s_q)).flatten()
    if ps:
        cols = cap // ps
        pages = B * cols + 2
        table = torch.randperm(pages, generator=g)[:B * cols].view(B, cols)
        kv = torch.randint(0, 256, (pages, ps, row), generator=g, dtype=torch.uint8)
        b = torch.arange(T) // s_q
        slot = table[b, at // ps] * ps + at % ps
        rows_at = slot
    else:
        kv, table = torch.randint(0, 256, (B, cap, row), generator=g, dtype=torch.uint8), None
        rows_at = torch.arange(T) // s_q * cap + at
    kw = {}
    if with_slots:
        kw["slots"] = slot.to(I32).to(DEV)
        at = torch.randint(0, 2 ** 31 - 1, (T,), generator=g)
        kw["positions"] = at.to(I32).to(DEV)
    plan = mla.rope_plan(d_rope, layout=mla.ROPE_HALF if half else mla.ROPE_INTERLEAVED) if turned else None
    freq = layer.frequencies(d_rope) if turned else None
    kv_d, lens_d, table_d = kv.to(DEV), lens.to(DEV), None if table is None else table.to(I32).to(DEV)
    status = torch.zeros(1, dtype=I32, device=DEV)
    cache = mla.make_cache(prob, kv_d, lens_d, table_d, ps or 64)
    mla.latent_store(prob, whole.to(DEV)[:, lead:], cache, plan=plan, norm_weight=None if weight is None else weight.to(DEV), eps=1e-5,
                     status=status, **kw)
    assert int(status) == 0
    got = kv_d.cpu().view(-1, row)
    check_store(got[rows_at], x, weight, at, freq, half, d_c, d_rope)
    other = torch.ones(got.shape[0], dtype=torch.bool)
    other[rows_at] = False
    assert torch.equal(got[other], kv.view(-1, row)[other])


def test_store_in_blocks_skips_and_flags():
    g = gen(21)
    T, d_c, d_rope, ps, pages = 12, 128, 32, 64, 4
    x = randn(g, T, d_c + d_rope)
    prob = problem(T, 16, 1, d_c=d_c, d_rope=d_rope)
    slots = torch.arange(T, dtype=I32) * 9
    slots[2], slots[5], slots[6], slots[7] = -1, pages * ps, 2 ** 31 - 1, -2 ** 31
    at = torch.arange(T, dtype=I32)
    at[9] = -1
    written = torch.tensor([i for i in range(T) if i not in (2, 5, 6, 7, 9)])
    kv, status = torch.zeros(pages, ps, 208, dtype=torch.uint8, device=DEV), torch.zeros(1, dtype=I32, device=DEV)
    lens, table = torch.ones(T, dtype=I32, device=DEV), torch.zeros(T, 1, dtype=I32, device=DEV)
    mla.latent_store(prob, x.to(DEV), mla.make_cache(prob, kv, lens, table, ps), plan=mla.rope_plan(d_rope), positions=at.to(DEV),
                     slots=slots.to(DEV), status=status)
    assert int(status) == layer.PAGE
    touched = (kv.cpu().view(-1, 208).float().abs().sum(1) > 0).nonzero().flatten()
    assert torch.equal(touched, slots[written].long())
    lens[0], lens[1], table[2] = 0, 65, pages  # by the lengths: too short, too long, a page outside the pool
    for first, code in ((slice(0, 12), (layer.SEQLEN, layer.PAGE)),):
        status.zero_()
        kv.zero_()
        mla.latent_store(prob, x.to(DEV), mla.make_cache(prob, kv, lens, table, ps), status=status)
        assert int(status) in code
        assert (kv.cpu().view(-1, 208).float().abs().sum(1) > 0).nonzero().flatten().tolist() == [0]  # the others: token 0 of page 0


def test_store_in_blocks_special_values():
    """A block of zeros, NaN and infinities: the latent's stay in their block (with a norm in their row), the key's in their
    value; and the row reads back as the documents say."""
    d_c, d_rope = 256, 16
    x = torch.zeros(5, d_c + d_rope, dtype=BF16)
    x[1, 3], x[1, 4], x[1, d_c] = float("nan"), 8.0, float("inf")
    x[2, 130] = float("inf")
    x[3, :] = 1e30
    x[4, :128] = torch.arange(128)
    prob = problem(5, 16, 1, d_c=d_c, d_rope=d_rope)
    lens, table = torch.full((5,), 5, dtype=I32, device=DEV), torch.zeros(5, 1, dtype=I32, device=DEV)
    for weight in (None, torch.ones(d_c, dtype=BF16, device=DEV)):
        kv = torch.full((1, 64, 304), 0x55, dtype=torch.uint8, device=DEV)
        cache = mla.make_cache(prob, kv, lens, table, 64)
        mla.latent_store(prob, x.to(DEV), cache, norm_weight=weight, slots=torch.arange(5, dtype=I32, device=DEV))
        codes, scales, keys = blocks_of(kv[0, :5], d_c, d_rope)
        assert bool((codes[0] == 0).all()) and scales[0].tolist() == [LEAST] * 2 + [0.0, 0.0]
        assert float(keys[1, 0]) == math.inf and bool((keys[1, 1:] == 0).all())
        back = mla.latent_load(prob, cache, 5)[0].cpu().float()
        assert bool((back[0] == 0).all())
        if weight is None:
            assert bool(torch.isnan(back[1, 3])) and float(back[1, 4]) == 8.0 and bool((back[1, 5:128] == 0).all())
            assert bool((back[2, :128] == 0).all()) and bool(torch.isnan(back[2, 128:d_c]).all())  # 0 x infinity
            assert bool((back[3, :d_c] == float(x[3, 0])).all())
        else:
            assert bool(torch.isnan(back[1, :d_c]).all())
            assert bool((back[3, :d_c] == 0).all())  # 1e30 squared passes fp32
        assert float(back[4, 128:d_c].abs().sum()) == 0


# ------------------------------------------------------------------------------------------------------------- load
def cache_bytes(g, kind, shape, d_c, d_rope):
    """Random rows of a cache (CPU), and the values they stand for: codes of every kind but NaN."""
    codes = lambda n: torch.randint(0, 256, (*shape, n), generator=g, dtype=torch.uint8)  # noqa: E731

    def no_nan(c):
        return torch.where((c & 0x7F) == 0x7F, c - 1, c)
    if kind == "bf16":
        kv = randn(g, *shape, d_c + d_rope)
        return kv, kv.double(), None
    if kind == "e4m3":
        kv = no_nan(codes(d_c + d_rope))
        return kv, kv.view(E4M3).double() * float(torch.tensor(0.03)), 0.03
    c, s, k = no_nan(codes(d_c)), torch.exp(torch.randn(*shape, 4, generator=g)) * 0.01, randn(g, *shape, d_rope)
    kv = torch.cat((c, s.view(torch.uint8), k.view(torch.uint8)), -1)
    return kv, torch.cat((c.view(E4M3).double() * s.double().repeat_interleave(128, -1)[..., :d_c], k.double()), -1), None


LOAD_CASES = [
    # B, rows, longest, d_c, d_rope, page size (0: contiguous), positions given, extra stride of out
    (1, 1, 1, 64, 0, 64, False, 0), (3, 5, 130, 64, 16, 64, True, 0), (2, 130, 130, 128, 32, 128, False, 8), (5, 33, 70, 192, 48, 64, True, 24),
    (4, 64, 64, 512, 64, 64, False, 0), (3, 333, 333, 512, 64, 192, False, 0), (7, 17, 1000, 320, 64, 0, True, 8), (2, 257, 300, 448, 16, 0, False, 0),
    (65, 3, 200, 512, 64, 64, True, 0), (2, 16, 5, 512, 64, 0, False, 16),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "blocks"])
@pytest.mark.parametrize("B,rows,T,d_c,d_rope,ps,given,extra", LOAD_CASES)
def test_load(kind, B, rows, T, d_c, d_rope, ps, given, extra):
    """fp32 values rounded once: scale times code (2^-24) and half a bf16 step; a bf16 row bit for bit.  Rows of no token
    (behind a length, padding, positions out of range) and the memory between sequences stay as they were."""
    g = gen(B + rows + d_c)
    prob, W = problem(B, 16, 1, d_c=d_c, d_rope=d_rope), d_c + d_rope
    lens = torch.randint(0, T + 1, (B,), generator=g, dtype=I32)
    lens[0] = T
    if ps:
        cols = -(-T // ps)
        pages = B * cols + 2
        table = torch.randperm(pages, generator=g)[:B * cols].view(B, cols)
        kv, values, scale = cache_bytes(g, kind, (pages, ps), d_c, d_rope)
        values = values[table].reshape(B, cols * ps, W)
        table = torch.where(torch.arange(cols) * ps < lens[:, None], table, -1).to(I32)  # no page behind a length
    else:
        table = None
        kv, values, scale = cache_bytes(g, kind, (B, T), d_c, d_rope)
    at = torch.arange(rows).expand(B, -1)
    if given:
        at = torch.randint(-2, T + 3, (B, rows), generator=g)
        at[0, 0], at[-1, -1] = 2 ** 31 - 1, -2 ** 31
    there = (at >= 0) & (at < lens[:, None])
    out = torch.full((B, rows * W + extra), 7.0, dtype=BF16, device=DEV)
    kv_d, lens_d, table_d = kv.to(DEV), lens.to(DEV), None if table is None else table.to(DEV)
    status = torch.zeros(1, dtype=I32, device=DEV)
    cache = mla.make_cache(prob, kv_d, lens_d, table_d, ps or 64, kv_scale=scale)
    view = out[:, :rows * W].unflatten(1, (rows, W))
    got = mla.latent_load(prob, cache, rows, positions=at.to(I32).to(DEV) if given else None, out=view, status=status)
    assert got is view and int(status) == 0
    want = torch.full((B, rows, W), 7.0, dtype=torch.float64)
    want[there] = values[torch.arange(B)[:, None].expand(-1, rows)[there], at[there]]
    close(view, want, want.abs() * (0 if kind == "bf16" else 2.0 ** -8 * (1 + 2.0 ** -14)) + 2.0 ** -134)
    assert bool((out[:, rows * W:] == 7).all())
    assert torch.equal(kv_d.cpu().view(torch.uint8), kv.view(torch.uint8)), "the cache is not written"
    if bool(there.all()):
        assert torch.equal(mla.latent_load(prob, cache, rows, positions=at.to(I32).to(DEV) if given else None), view)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "blocks"])
def test_load_skips_and_flags(kind):
    """Lengths and pages out of range: recorded, the rows left as they were, the others read."""
    g = gen(77)
    B, d_c, d_rope, ps, pages = 6, 64, 16, 64, 5
    prob = problem(B, 16, 1, d_c=d_c, d_rope=d_rope)
    kv, values, scale = cache_bytes(g, kind, (pages, ps), d_c, d_rope)
    lens = torch.tensor([0, 129, -1, 100, 70, 128], dtype=I32, device=DEV)
    table = torch.tensor([[0, 0], [0, 0], [0, 0], [1, -1], [pages, 2], [3, 4]], dtype=I32, device=DEV)
    kv = kv.to(DEV)
    for keep, code in ((range(6), (layer.SEQLEN, layer.PAGE)), ((0, 5), (0,)), ((1, 0, 0, 0, 0, 0), (layer.SEQLEN,)), ((3,), (layer.PAGE,))):
        pick = torch.tensor(list(keep), device=DEV)
        p = problem(len(pick), 16, 1, d_c=d_c, d_rope=d_rope)
        status = torch.zeros(1, dtype=I32, device=DEV)
        some_lens, some_table = lens[pick].contiguous(), table[pick].contiguous()
        out = torch.full((len(pick), 128, 80), 7.0, dtype=BF16, device=DEV)
        mla.latent_load(p, mla.make_cache(p, kv, some_lens, some_table, ps, kv_scale=scale), 128, out=out, status=status)
        assert int(status) in code
        for i, b in enumerate(pick.tolist()):
            left = {0: range(128), 1: range(128), 2: range(128), 3: range(64, 128), 4: [*range(64), *range(70, 128)], 5: []}[b]
            same = (out[i].cpu() == 7).all(1)
            assert same.nonzero().flatten().tolist() == list(left), b
    # no status word: the same, nothing recorded
    out = torch.full((B, 128, 80), 7.0, dtype=BF16, device=DEV)
    mla.latent_load(prob, mla.make_cache(prob, kv, lens, table, ps, kv_scale=scale), 128, out=out)
    assert bool((out[:3] == 7).all())


def test_load_of_nothing():
    prob = problem(2, 16, 1, d_c=64, d_rope=16)
    kv, lens = torch.zeros(2, 10, 112, dtype=torch.uint8, device=DEV), torch.full((2,), 10, dtype=I32, device=DEV)
    cache = mla.make_cache(prob, kv, lens)
    assert mla.latent_load(prob, cache, 0).shape == (2, 0, 80)


def test_offsets_past_32_bits():
    """The last slots of a pool of 6.6e9 bytes and the last rows of an output of 2.5e9 values."""
    pages = 156000
    prob = problem(4, 16, 1)
    g = torch.Generator(device=DEV).manual_seed(93)
    kv = torch.empty(pages, 64, 656, dtype=torch.uint8, device=DEV)
    kv[0].zero_()
    kv[-2:].zero_()
    x = torch.randn(4, 576, generator=g, device=DEV).to(BF16)
    slots = torch.tensor([pages * 64 - 1, 5, pages * 64 - 65, pages * 64 - 64], dtype=I32, device=DEV)
    lens, table = torch.ones(4, dtype=I32, device=DEV), torch.zeros(4, 1, dtype=I32, device=DEV)
    mla.latent_store(prob, x, mla.make_cache(prob, kv, lens, table, 64), slots=slots)
    small = torch.zeros(1, 64, 656, dtype=torch.uint8, device=DEV)
    mla.latent_store(prob, x, mla.make_cache(prob, small, lens, table, 64), slots=torch.arange(4, dtype=I32, device=DEV))
    flat = kv.view(-1, 656)
    assert torch.equal(flat[slots.long()], small[0, :4])
    around = torch.cat((flat[:64], flat[-128:])).float().abs().sum(1)
    assert int((around > 0).sum()) == 4
    # read back by a table whose pages are the last ones
    one = problem(1, 16, 1)
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=I32, device=DEV)
    at = torch.tensor([[63, 64 + 5, 128 + 63, 0]], dtype=I32, device=DEV)
    full = torch.full((1,), 192, dtype=I32, device=DEV)
    back = mla.latent_load(one, mla.make_cache(one, kv, full, table, 64), 4, positions=at)
    page, first = torch.full((1,), 64, dtype=I32, device=DEV), torch.zeros(1, 1, dtype=I32, device=DEV)
    want = mla.latent_load(one, mla.make_cache(one, small, page, first, 64), 4)
    assert torch.equal(back, want)
    del kv, flat, around
    # a contiguous cache of 2 x 4.5e9 bytes, into outputs 2.4e9 values apart
    T = 6900000
    two = problem(2, 16, 1)
    kv = torch.empty(2, T, 656, dtype=torch.uint8, device=DEV)
    kv[:, -4:] = small[0, :4]
    lens = torch.full((2,), T, dtype=I32, device=DEV)
    wide = torch.empty(2, 2400000 * 1000 // 8 * 8, dtype=BF16, device=DEV)
    out = wide[:, :4 * 576].unflatten(1, (4, 576))
    at = torch.tensor([[T - 4, T - 3, T - 2, T - 1]] * 2, dtype=I32, device=DEV)
    mla.latent_load(two, mla.make_cache(two, kv, lens), 4, positions=at, out=out)
    assert torch.equal(out, want.expand(2, -1, -1))


# ------------------------------------------------------------------------------------------------------------ together
class Layer8:
    """One MLA layer's step in 8 bits, x = x + attention(norm(x)) . W_O: weights, activations and cache rows in blocks of 128; the
    attention reads what latent_load gives.  Every stage's inputs are kept, so that each can be held against 64 bits."""

    def __init__(self, B, H, d_model, d_c, d_rope, d_nope, d_v, ps, max_pages, seed):
        g = gen(seed)
        self.B, self.H, self.ps, self.cap = B, H, ps, max_pages * ps
        self.dims = dict(d_c=d_c, d_rope=d_rope, d_nope=d_nope, d_v=d_v)
        self.norm = (1 + 0.1 * torch.randn(d_model, generator=g)).to(BF16).to(DEV)
        self.c_norm = (1 + 0.1 * torch.randn(d_c, generator=g)).to(BF16).to(DEV)
        sizes = dict(q=(H * (d_nope + d_rope), d_model), kv=(d_c + d_rope, d_model), o=(d_model, H * d_v))
        self.full = {k: randn(g, *n, std=n[1] ** -0.5) for k, n in sizes.items()}
        self.w = {k: mla.quantize(v.to(DEV), block_rows=128) for k, v in self.full.items()}
        self.w_uk, self.w_uv = (randn(g, H, d_c, n, std=d_c ** -0.5).to(DEV) for n in (d_nope, d_v))
        self.plan, self.freq = mla.rope_plan(d_rope), layer.frequencies(d_rope)
        self.pages, self.state = mla.Pages.empty(B, max_pages, B * max_pages, ps)
        self.kv = torch.zeros(B * max_pages, ps, d_c + 16 + 2 * d_rope, dtype=torch.uint8, device=DEV)
        self.read = torch.zeros(B, self.cap, d_c + d_rope, dtype=BF16, device=DEV)
        self.lens = torch.zeros(B, dtype=I32, device=DEV)

    def step(self, x, new_lens, status):
        s_q = x.shape[0] // self.B
        prob = mla.Problem(self.B, self.H, s_q, scale=(self.dims["d_nope"] + self.dims["d_rope"]) ** -0.5, **self.dims)
        up = mla.pages_update(self.pages, self.state, self.lens, new_lens, x.shape[0], status=status)
        h = mla.quantize(x, norm_weight=self.norm)
        q = mla.linear_fp8(*h, *self.w["q"], status=status)
        q_nope, q_rope = mla.rope(prob, self.plan, q.view(self.B, s_q, self.H, -1), positions=up.positions)
        c = mla.linear_fp8(*h, *self.w["kv"], status=status)
        kept = mla.make_cache(prob, self.kv, up.seq_lens, self.pages.block_table, self.ps)
        mla.latent_store(prob, c, kept, plan=self.plan, norm_weight=self.c_norm, positions=up.positions, slots=up.slots, status=status)
        mla.latent_load(prob, kept, self.cap, out=self.read, status=status)
        cache = mla.make_cache(prob, self.read, up.seq_lens)
        q_cat = mla.absorb_q(prob, q_nope, q_rope, self.w_uk)
        o_lat, _, ws = mla.decode_attn(prob, q_cat, cache)
        out = mla.out_proj(prob, o_lat, self.w_uv)
        a = mla.quantize(out.view(x.shape[0], -1))
        y = mla.linear_fp8(*a, *self.w["o"], residual=x, status=status)
        self.keep = dict(up=up, h=h, q=q, c=c, q_nope=q_nope, q_rope=q_rope, kept=kept, cache=cache, q_cat=q_cat, o_lat=o_lat, ws=ws, out=out, a=a)
        self.state, self.lens = up.ring_state, up.seq_lens
        return y


def check_step(L, x, y, s_q, n):
    """Every stage of a step against 64 bits on the stage's own inputs, and the whole against the layer without 8 bits."""
    k = {n_: tuple(t.cpu() for t in v) if isinstance(v, tuple) else v.cpu() if torch.is_tensor(v) else v for n_, v in L.keep.items()}
    D, B, H = L.dims, L.B, L.H
    rel = x.shape[1] * 2.0 ** -25 + 2.0 ** -21
    quotient, exact = layer.blocks(layer.rms_norm(x, L.norm.cpu(), 1e-6), 1)
    close(k["h"][1].t(), exact, exact * (rel + 2.0 ** -24))
    close_codes(k["h"][0], quotient, 2.0 ** -21)
    w = {name: [t.cpu() for t in v] for name, v in L.w.items()}
    for name, codes, got, res in (("q", k["h"], k["q"], None), ("kv", k["h"], k["c"], None), ("o", k["a"], y, x)):
        want = layer.linear_fp8(*codes, *w[name], None, res)
        close(got, want, product_tolerance(*codes, *w[name], want, want), name)
    # the rows written, and the rows read back
    at = (n - s_q + torch.arange(s_q)).repeat(B)
    slot = k["up"].slots.cpu().long()
    new = L.kv.cpu().view(-1, L.kv.shape[-1])[slot]
    rel_c = D["d_c"] * 2.0 ** -25 + 2.0 ** -21
    codes, scales, keys = blocks_of(new, D["d_c"], D["d_rope"])
    quotient, exact = layer.blocks(layer.rms_norm(k["c"][:, :D["d_c"]], L.c_norm.cpu(), 1e-6), 1)
    close(scales[:, :exact.shape[1]], exact, exact * (rel_c + 2.0 ** -24))
    close_codes(codes, quotient, 2.0 ** -20)
    rows = L.read.cpu()[:, :n]
    values = torch.cat((codes * layer.spread(scales[:, :exact.shape[1]], 1, B * s_q, D["d_c"]), keys), 1).view(B, s_q, -1)
    close(rows[:, n - s_q:], values, values.abs() * 2.0 ** -8 * 1.001)
    # the attention on the rows read back
    rows = rows.double()
    limit = (n - s_q + torch.arange(s_q))[None, :, None, None]
    s = torch.einsum("bihc,bjc->bihj", k["q_cat"].double(), rows) * (D["d_nope"] + D["d_rope"]) ** -0.5
    p = torch.softmax(s.masked_fill(torch.arange(n) > limit, -math.inf), -1)
    within_tolerance(k["o_lat"], torch.einsum("bihj,bjc->bihc", p, rows[:, :, :D["d_c"]]), "o_lat")


@pytest.mark.parametrize("H,d_c,d_rope,d_nope,d_v", [(16, 64, 16, 32, 32), (128, 512, 64, 128, 128)])
def test_a_layer_in_8_bits_step_after_step(H, d_c, d_rope, d_nope, d_v):
    L = Layer8(3, H, 512, d_c, d_rope, d_nope, d_v, 64, 4, 41)
    g = gen(42)
    status = torch.zeros(1, dtype=I32, device=DEV)
    lens = 0
    for s_q in (60, 1, 3, 1, 130 if d_c == 64 else 65, 1):
        lens += s_q
        x = randn(g, 3 * s_q, 512)
        y = L.step(x.to(DEV), torch.full((3,), lens, dtype=I32, device=DEV), status)
        assert int(status) == 0 and mla.read_status(L.keep["ws"]) == 0
        check_step(L, x, y, s_q, lens)
        assert L.lens.tolist() == [lens] * 3


def test_a_prefill_on_a_cache_of_blocks():
    """A chunk of a prompt on a history kept in blocks: read back, then the expanded form, which takes bf16 rows alone, against
    64 bits on the rows read.  K and V are rounded to bf16: a score is off by e = 2^-8 scale sum |q K| at most, a
    probability by a factor of exp(2 e), and with its own rounding, V's and the result's 2^-8 each, the sum of p V by
    (exp(2 e) - 1 + 3 2^-8) sum p |V| (2^-12 for fp32 sums; random codes make scores of 50, and e up to a few tenths)."""
    g = gen(71)
    B, H, s_q, T = 2, 128, 130, 300
    prob = mla.Problem(B, H, s_q, 512, 64, 128, 128, 192 ** -0.5)
    kv, values, _ = cache_bytes(g, "blocks", (B, T), 512, 64)
    kv, lens = kv.to(DEV), torch.tensor([T, 200], dtype=I32, device=DEV)
    read = mla.latent_load(prob, mla.make_cache(prob, kv, lens), T)  # a cache holds addresses: its tensors are kept here
    cache = mla.make_cache(prob, read, lens)
    q_nope, q_rope = randn(g, B, s_q, H, 128).to(DEV), randn(g, B, s_q, H, 64).to(DEV)
    w_uk, w_uv = (randn(g, H, 512, 128, std=512 ** -0.5).to(DEV) for _ in range(2))
    out, _, ws = mla.prefill_expand(prob, q_nope, q_rope, cache, w_uk, w_uv)
    assert mla.read_status(ws) == 0
    for b, n in enumerate(lens.tolist()):
        c, k_rope = read[b, :n, :512].double(), read[b, :n, 512:].double()
        k, v = torch.einsum("jc,hcn->hjn", c, w_uk.double()), torch.einsum("jc,hcv->hjv", c, w_uv.double())
        qn, qr = q_nope[b].double(), q_rope[b].double()
        s = (torch.einsum("ihn,hjn->ihj", qn, k) + torch.einsum("ihr,jr->ihj", qr, k_rope)) * prob.scale
        seen = torch.arange(n, device=DEV) <= (n - s_q + torch.arange(s_q, device=DEV))[:, None, None]
        p = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
        e = 2.0 ** -8 * prob.scale * (torch.einsum("ihn,hjn->ihj", qn.abs(), k.abs()) * seen).amax(-1, keepdim=True)
        tol = (torch.exp(2 * e) - 1 + 3 * 2.0 ** -8 + 2.0 ** -12) * torch.einsum("ihj,hjv->ihv", p, v.abs())
        close(out[b], torch.einsum("ihj,hjv->ihv", p, v).cpu(), tol.cpu(), f"sequence {b}")


def test_the_tokens_of_a_selector():
    """latent_load of listed tokens, then attention over them alone, against the sparse attention on the whole cache."""
    g = gen(72)
    B, H, T, k = 3, 128, 500, 64
    prob = mla.Problem(B, H, 1, 512, 64, 128, 128, 192 ** -0.5)
    kv = (torch.randn(B, T, 576, generator=g)).to(BF16).to(DEV)
    lens = torch.tensor([500, 300, 64], dtype=I32, device=DEV)
    at = torch.stack([torch.randperm(int(n), generator=g)[:k] for n in lens.tolist()]).to(I32).to(DEV)
    q_cat = randn(g, B, 1, H, 576, std=0.3).to(DEV)
    whole = mla.make_cache(prob, kv, lens)
    want, _, _ = mla.decode_attn_sparse(prob, q_cat, whole, at.view(B, 1, k))
    some = mla.latent_load(prob, whole, k, positions=at)
    all_k = torch.full((B,), k, dtype=I32, device=DEV)
    o_lat, _, ws = mla.decode_attn(prob, q_cat, mla.make_cache(prob, some, all_k))
    assert mla.read_status(ws) == 0
    within_tolerance(o_lat, want.cpu(), "listed tokens")


def test_a_step_captured_and_replayed():
    """Two graphs of the 8-bit calls, each on its own layer, replayed in turn, against the same steps run eagerly."""
    def make(seed):
        L = Layer8(2, 16, 256, 64, 16, 32, 32, 64, 3, seed)
        status = torch.zeros(1, dtype=I32, device=DEV)
        L.step(randn(gen(seed), 2 * 62, 256).to(DEV), torch.full((2,), 62, dtype=I32, device=DEV), status)
        return L, status

    def capture(L, status):
        x = torch.zeros(2, 256, dtype=BF16, device=DEV)
        lens, state, new = L.lens.clone(), L.state.clone(), L.lens + 1
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            L.lens, L.state = lens, state
            y = L.step(x, new, status)
            lens.copy_(L.lens)
            state.copy_(L.state)
            new.add_(1)
        L.buffers = (lens, state, new)
        return graph, x, y

    (a, sa), (b, sb), (ea, se), (eb, sf) = make(51), make(52), make(51), make(52)
    torch.cuda.synchronize()
    ga, xa, ya = capture(a, sa)
    gb, xb, yb = capture(b, sb)
    g = gen(53)
    for i in range(4):
        x = randn(g, 2, 256).to(DEV)
        for graph, xs, ys, eager, st in ((ga, xa, ya, ea, se), (gb, xb, yb, eb, sf)):
            xs.copy_(x)
            graph.replay()
            assert torch.equal(ys, eager.step(x, eager.lens + 1, st)), i
    assert int(sa) == 0 and int(sb) == 0 and torch.equal(a.kv, ea.kv) and torch.equal(b.read, eb.read)


def calls(g):
    """One call of each operator with buffers of its own, as functions that give tensors."""
    x = randn(g, 200, 1008).to(DEV)
    weight = randn(g, 1008).to(DEV)
    many = [t.to(DEV) for t in operands(g, 300, 2064, 1544, False)]
    few = [t.to(DEV) for t in operands(g, 5, 8192, 264, False)]
    prob = problem(3, 16, 1, d_c=128, d_rope=32)
    rows, lens = randn(g, 3, 160).to(DEV), torch.full((3,), 7, dtype=I32, device=DEV)

    def kept():
        kv = torch.zeros(3, 64, 208, dtype=torch.uint8, device=DEV)
        cache = mla.make_cache(prob, kv, lens)
        mla.latent_store(prob, rows, cache, norm_weight=weight[:128].contiguous())
        out = torch.zeros(3, 7, 160, dtype=BF16, device=DEV)
        return kv, mla.latent_load(prob, cache, 7, out=out)
    return (lambda: [t.view(torch.uint8) for t in mla.quantize(x, norm_weight=weight)], lambda: [mla.linear_fp8(*many)],
            lambda: [mla.linear_fp8(*few)], kept)


def test_calls_on_two_streams_at_once():
    """Calls with buffers of their own on two streams, many in flight, give what they give alone."""
    g = gen(61)
    fs = calls(g)
    want = [[t.clone() for t in f()] for f in fs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(20):
        for s, order in zip(streams, (1, -1)):
            with torch.cuda.stream(s):
                got += [(j, fs[j]()) for j in range(len(fs))[::order]]
    torch.cuda.synchronize()
    for j, tensors in got:
        assert all(torch.equal(a, b) for a, b in zip(tensors, want[j])), j


def test_calls_from_several_threads():
    g = gen(62)
    fs = calls(g)
    want = [[t.clone() for t in f()] for f in fs]
    torch.cuda.synchronize()
    wrong = []

    def work(j):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = [fs[j % len(fs)]() for _ in range(50)]
            s.synchronize()
        wrong.extend(j for tensors in got if not all(torch.equal(a, b) for a, b in zip(tensors, want[j % len(fs)])))

    threads = [threading.Thread(target=work, args=(j,)) for j in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_a_long_chain_without_a_pause():
    """Each product is launched while the one before it ends, and reads its result: the chain gives what it gives with a
    wait after every call."""
    g = gen(63)
    w = [mla.quantize(randn(g, n, k, std=k ** -0.5).to(DEV), block_rows=128) for n, k in ((1536, 512), (512, 1536), (4096, 512), (512, 4096))]
    x = randn(g, 70, 512).to(DEV)

    def chain(pause):
        y = x
        for i in range(40):
            y = mla.linear_fp8(*mla.quantize(y), *w[i % 4], residual=x if i % 2 else None, act=mla.ACT_SILU)
            pause()
        return y
    want = chain(torch.cuda.synchronize)
    for _ in range(5):
        assert torch.equal(chain(lambda: None), want)


def test_stream_argument():
    """Calls under stream=s behind a long wait there, while the current stream fills memory of the outputs' sizes; tensors
    that a call makes under stream= come from that stream's memory."""
    g = gen(64)
    x = randn(g, 64, 4096).to(DEV)
    w = mla.quantize(randn(g, 520, 4096, std=1 / 64).to(DEV), block_rows=128)
    prob = problem(3, 16, 1, d_c=128, d_rope=32)
    kv, lens = torch.zeros(3, 64, 208, dtype=torch.uint8, device=DEV), torch.full((3,), 64, dtype=I32, device=DEV)
    cache = mla.make_cache(prob, kv, lens)
    want = mla.linear_fp8(*mla.quantize(x), *w)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    c, cs = mla.quantize(x, stream=s)
    y = mla.linear_fp8(c, cs, *w, stream=s)
    rows = mla.latent_load(prob, cache, 64, stream=s)
    taken = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for n in (64 * 4096, 64 * 32 * 4, 64 * 520 * 2) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(y, want) and bool((rows == 0).all()) and all(bool((t == 0x7F).all()) for t in taken)
    segments = torch.cuda.memory_snapshot()
    for t in (c, cs, y, rows):
        at = [seg for seg in segments if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]]
        assert len(at) == 1 and at[0]["stream"] == s.cuda_stream
