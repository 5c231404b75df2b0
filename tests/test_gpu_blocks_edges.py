"""The 8-bit operators with scales by blocks of 128 at the ends of what they are defined for: scales whose product is no normal
number, or nearly infinite."""
import pytest
import torch

from mla_decode_attention_absorbed_gb300 import build, mla
from oracle import layer
from test_gpu_blocks import BF16, DEV, E4M3, cache_bytes, close, gen, operands, powers, problem, randn, whole_codes

pytestmark = pytest.mark.gpu

# A tile of each form on a single CTA and on a pair, whole and shared (M, K, N).
SIZES = [(3, 208, 136), (121, 1968, 136), (3, 208, 10328), (135, 208, 10840), (137, 208, 16408), (140, 7536, 5032)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.load()


# ------------------------------------------------------------------------------------------------- scales, far from 1
# Half a step of bf16 is 2^-8 of a normal value and 2^-134 of a subnormal one; an fp32 subnormal on the way to it is off
# by 2^-150.
STEP, LEAST = 2.0 ** -8 * (1 + 2.0 ** -12), 2.0 ** -134 + 2.0 ** -150


@pytest.mark.parametrize("low", [-122, -136, -150, -164])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_linear_fp8_of_small_scales(M, K, N, low):
    """Powers of two whose products go down to 2^low, of whole codes: every sum is exact, however small the scales'
    product."""
    g = gen(M + K - low)
    x, w = whole_codes(g, M, K), whole_codes(g, N, K)
    kb, half = -(-K // 128), low // 2
    xs, ws = powers(g, kb, M, least=half, most=half + 2), powers(g, -(-N // 128), kb, least=low - half, most=low - half + 2)
    r = (randn(g, M, N).double() * 2.0 ** (low + 10)).to(BF16)
    want = layer.linear_fp8(x, xs, w, ws, None, r)
    got = mla.linear_fp8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), residual=r.to(DEV))
    close(got, want, want.abs() * STEP + LEAST)


@pytest.mark.parametrize("low", [-110, -118, -125])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_linear_fp8_of_small_values(M, K, N, low):
    """Values as quantising leaves them, of 2^low together: as product_tolerance has it, without its absolute part."""
    g = gen(M + N - low)
    x, xs, w, ws = operands(g, M, K, N, False)
    xs, ws = xs * 2.0 ** (low // 2), ws * 2.0 ** (low - low // 2)
    want = layer.linear_fp8(x, xs, w, ws)
    terms = layer.linear_fp8(x.float().abs(), xs, w.float().abs(), ws)
    got = mla.linear_fp8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV))
    close(got, want, (K * 2.0 ** -23 + 2.0 ** -22) * terms + want.abs() * STEP + LEAST)


def test_linear_fp8_of_the_smallest_scales():
    """The scale that a block of values below 2^-100 has, 2^-100 / 448, on either side, and fp32's smallest number: what codes
    of 448 make of them shows in bf16."""
    M, K, N = 5, 4096, 136
    x, w = torch.full((M, K), 448.0).to(E4M3), torch.full((N, K), 448.0).to(E4M3)
    for a, b in ((2.0 ** -100 / 448, 2.0 ** -46), (2.0 ** -46, 2.0 ** -100 / 448), (2.0 ** -149, 1.0), (2.0 ** -149, 2.0 ** -8), (2.0 ** -75, 2.0 ** -81)):
        xs, ws = torch.full((32, M), a), torch.full((2, 32), b)
        want = layer.linear_fp8(x, xs, w, ws)
        assert float(want[0, 0]) > 2.0 ** -128
        # a block's scale and 32 of them added in fp32
        close(mla.linear_fp8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV)), want, want * (STEP + 2.0 ** -18) + LEAST)


@pytest.mark.parametrize("M,K,N", SIZES)
def test_linear_fp8_of_scales_far_apart(M, K, N):
    """Blocks of one row up to 2^200 apart, in an order of their own in each row: as test_linear_fp8, of all terms; where a block's scale is
    past 2^16, the others' may be off by half an fp32 step of 2^-149, which is 2^-125 of codes' sum at most."""
    g = gen(M + N)
    x, w = whole_codes(g, M, K), whole_codes(g, N, K)
    kb = -(-K // 128)
    xs, ws = powers(g, kb, M, least=-80, most=45), powers(g, -(-N // 128), kb, least=-60, most=10)
    want = layer.linear_fp8(x, xs, w, ws)
    terms = layer.linear_fp8(x.float().abs(), xs, w.float().abs(), ws)
    close(mla.linear_fp8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV)), want,
          terms * (K * 2.0 ** -23) + want.abs() * STEP + LEAST + kb * 2.0 ** -125)


@pytest.mark.parametrize("M,K,N", SIZES)
def test_linear_fp8_of_large_scales(M, K, N):
    """Scales' products around 2^85 of sums below 2^17 units (K times 16), of 2^2 at most between blocks: exact in fp32."""
    g = gen(M + K)
    x, w = whole_codes(g, M, K), whole_codes(g, N, K)
    kb = -(-K // 128)
    xs, ws = powers(g, kb, M, least=40, most=41), powers(g, -(-N // 128), kb, least=43, most=44)
    want = layer.linear_fp8(x, xs, w, ws)
    got = mla.linear_fp8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV))
    assert torch.equal(got.cpu(), want.float().to(BF16))


@pytest.mark.parametrize("M,K,N", SIZES)
def test_linear_fp8_of_large_scales_beside_zeros(M, K, N):
    """A scale of 2^66 or 2^120 beside a zero one is a block of zeros, whichever side it is on."""
    g = gen(M + K + 1)
    K += 256
    x, w = whole_codes(g, M, K), whole_codes(g, N, K)
    kb = -(-K // 128)
    xs, ws = powers(g, kb, M, least=0, most=1), powers(g, -(-N // 128), kb, least=0, most=1)
    xs[0], ws[:, 0] = 0.0, 2.0 ** 66
    xs[2], ws[:, 2] = 2.0 ** 120, 0.0
    want = layer.linear_fp8(x, xs, w, ws)
    assert bool((want != 0).any())
    got = mla.linear_fp8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV))
    assert torch.equal(got.cpu(), want.float().to(BF16))


# ----------------------------------------------------------------------------------------------------- waits that run out
@pytest.mark.parametrize("M,K,N", [(4000, 16, 7160), (515, 208, 12760), (1039, 80, 20000), (3, 16, 41000), (2, 912, 20568), (262, 10896, 3768)])
def test_linear_fp8_waits_for_the_residual_within_the_limit(M, K, N):
    """Few blocks of K and several tiles a CTA: of a tile's time most goes to its residual, and to the copy of the tile before.
    Limits that end those waits leave NaN, never a sum beside a residual that had not come, nor a tile as it was; the
    next call knows nothing of it."""
    g = gen(M + N)
    x, xs, w, ws = (t.to(DEV) for t in operands(g, M, K, N, False))
    r = randn(g, M, N, std=64.0).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = mla.linear_fp8(x, xs, w, ws, residual=r)
    seen = 0
    try:
        for ns in (1, 300, 1000, 2000, 4000, 8000, 16000):
            mla.set_wait_limit_ns(ns)
            for inplace in (False, True, False):
                status.zero_()
                out = r.clone() if inplace else torch.full((M, N), 77.0, dtype=BF16, device=DEV)
                start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
                start.record()
                mla.linear_fp8(x, xs, w, ws, residual=out if inplace else r, status=status, out=out)
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
    assert torch.equal(mla.linear_fp8(x, xs, w, ws, residual=r, status=status), want) and int(status) == 0


# ------------------------------------------------------------------------------------------------------- rows of no token
@pytest.mark.parametrize("on_stream", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "blocks"])
def test_load_without_out_gives_zeros_for_rows_of_no_token(kind, on_stream):
    """Behind a length, of an empty sequence, of a position of -1 in a list, of a length or page out of range: 0 in a tensor that the call
    makes, whatever lay in its memory before."""
    g = gen(81)
    B, rows, T, d_c, d_rope = 5, 1300, 320, 128, 32
    prob, W = problem(B, 16, 1, d_c=d_c, d_rope=d_rope), d_c + d_rope
    kv, values, scale = cache_bytes(g, kind, (B * 5, 64), d_c, d_rope)
    table = torch.arange(B * 5, dtype=torch.int32).view(B, 5)
    values = values.view(B, T, W)
    lens = torch.tensor([320, 0, 130, 321, 320], dtype=torch.int32)
    table[4, 1] = B * 5
    kv, table_d, lens_d = kv.to(DEV), table.to(DEV), lens.to(DEV)
    cache = mla.make_cache(prob, kv, lens_d, table_d, 64, kv_scale=scale)
    at = torch.randint(0, T, (B, rows), generator=g)
    at[:, ::7] = -1
    stream = torch.cuda.Stream() if on_stream else None
    torch.cuda.synchronize()
    for positions in (None, at):
        with torch.cuda.stream(stream):  # what the call gets next
            torch.full((B, rows, W), float("nan"), dtype=BF16, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        got = mla.latent_load(prob, cache, rows, positions=None if positions is None else at.to(torch.int32).to(DEV), status=status,
                              stream=stream)
        torch.cuda.synchronize()
        assert int(status) in (layer.SEQLEN, layer.PAGE)
        p = torch.arange(rows).expand(B, -1) if positions is None else at
        there = (p >= 0) & (p < lens[:, None])
        there[3] = False
        there[4] &= p[4] // 64 != 1
        want = torch.zeros(B, rows, W, dtype=torch.float64)
        want[there] = values[torch.arange(B)[:, None].expand(-1, rows)[there], p[there]]
        close(got, want, want.abs() * (0 if kind == "bf16" else 2.0 ** -8 * (1 + 2.0 ** -14)) + 2.0 ** -134)


# -------------------------------------------------------------------------------------------------- some of quantised rows
def test_linear_fp8_of_some_of_the_rows():
    """A part of a batch, and its scales where they lie among the others', gives what it gives with a copy of them."""
    g = gen(91)
    x, weight = randn(g, 300, 1040).to(DEV), randn(g, 1040).to(DEV)
    w, ws = mla.quantize(randn(g, 520, 1040, std=1040 ** -0.5).to(DEV), block_rows=128)
    codes, scales = mla.quantize(x, norm_weight=weight)
    for a, b in ((0, 300), (3, 4), (7, 150), (290, 300), (299, 300)):
        want = mla.linear_fp8(codes[a:b].clone(), scales[:, a:b].clone(memory_format=torch.contiguous_format), w, ws)
        assert torch.equal(mla.linear_fp8(codes[a:b], scales[:, a:b], w, ws), want), (a, b)
        assert torch.equal(mla.linear_fp8(*mla.quantize(x[a:b], norm_weight=weight), w, ws), want), (a, b)


# ------------------------------------------------------------------------------------------------ the sum within a block
def test_linear_fp8_keeps_small_terms_beside_large_ones():
    """448 x 448 and its negative in one block of K, with a small term.  Where the large ones are among the same 32 values, which are one
    instruction's, the smallest code survives beside them; across instructions the sum is an fp32 number, whose step at
    200704 is 2^-6.  (What the card does; the contract is a sum in fp32.)"""
    def one(terms):
        x, w = torch.zeros(1, 128), torch.zeros(8, 128)
        for k, a, b in terms:
            x[0, k], w[:, k] = a, b
        ones = torch.ones(1, 1, device=DEV)
        got = mla.linear_fp8(x.to(E4M3).to(DEV), ones, w.to(E4M3).to(DEV), ones).cpu().float()
        assert bool((got == got[0, 0]).all())
        return float(got[0, 0])

    for group in range(0, 128, 32):
        for k, l, m in ((0, 1, 2), (31, 0, 17), (5, 30, 31), (16, 15, 0)):
            assert one([(group + k, 448.0, 448.0), (group + l, 448.0, -448.0), (group + m, 2.0 ** -9, 1.0)]) == 2.0 ** -9
    for first, second, small in ((0, 32, 64), (0, 127, 64), (96, 1, 33), (40, 70, 3)):
        assert one([(first, 448.0, 448.0), (second, 448.0, -448.0), (small, 2.0 ** -6, 1.0)]) == 2.0 ** -6
