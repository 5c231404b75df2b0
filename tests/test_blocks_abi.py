"""The 8-bit operators with scales by blocks of 128 (mla_quantize, mla_linear_fp8, caches of MLA_KV_E4M3_BLOCKS,
mla_latent_load): what they refuse on the host, before anything is launched.  No GPU needed."""
import ctypes

import pytest
import torch

from helpers import LINEAR_FP8_FORMS, linear_fp8_form
from mla_decode_attention_absorbed_gb300 import build, mla

NUL, A, B_, C_ = (ctypes.c_void_p(v) for v in (0, 0x40000, 0x50000, 0x60000))
ODD, ODD4 = ctypes.c_void_p(0x40008), ctypes.c_void_p(0x40002)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mla.load()


def dims(B=4, H=16, s_q=1, d_c=512, d_rope=64, d_nope=128, d_v=128):
    return mla.Problem(B, H, s_q, d_c, d_rope, d_nope, d_v, 0.1).dims()


def cache(T=4096, paged=True, kind=mla.KV_E4M3_BLOCKS, scale=0.5, page_size=64, num_pages=1000, kv=0x10000, lens=0x20000, row=656):
    if paged:
        return mla.Cache(kv, 0, 0, 0x30000, T // 64, page_size, num_pages, lens, 0, kind, scale)
    return mla.Cache(kv, T * row, T, None, 0, 64, 0, lens, 0, kind, scale)


# --------------------------------------------------------------------------------------------------------- quantize
def test_quantize_refusals(lib):
    def desc(M=4, K=256, rows=1, xs=256, cs=256, ss=4):
        return mla.QuantizeDesc(M, K, rows, xs, cs, ss)

    def call(d=None, x=A, w=NUL, eps=1e-6, codes=B_, scales=C_):
        return lib.mla_quantize(ctypes.byref(desc() if d is None else d), x, w, eps, codes, scales, NUL)

    assert lib.mla_quantize(None, A, NUL, 0.0, B_, C_, NUL) == 1
    for name in ("x", "codes", "scales"):
        assert call(**{name: NUL}) == 1, name
    for name in ("x", "w", "codes"):
        assert call(**{name: ODD}) == 4, name
    assert call(scales=ODD4) == 4
    for bad, code in ((dict(M=-1), 2), (dict(K=0), 2), (dict(K=248), 4), (dict(rows=0), 6), (dict(rows=64), 6), (dict(xs=248), 2),
                      (dict(cs=240), 2), (dict(xs=260), 4), (dict(cs=264), 4), (dict(ss=3), 2), (dict(rows=128, ss=1), 2),
                      (dict(K=(1 << 20) + 16, xs=1 << 21, cs=1 << 21), 6), (dict(M=65535 * 128 + 1, ss=1 << 40), 6)):
        assert call(desc(**bad)) == code, bad
    assert call(desc(rows=128, ss=2), w=A) == 6  # a norm is of rows
    assert call(w=A, eps=-1.0) == 2 and call(w=A, eps=float("nan")) == 2 and call(w=A, eps=float("inf")) == 2
    assert call(codes=A) == 6 and call(scales=A) == 6 and call(scales=B_) == 6  # outputs that are one another, or the input
    assert call(desc(M=0), x=NUL) == 0


# ------------------------------------------------------------------------------------------------------- linear_fp8
def fp8_desc(M=4, K=256, N=128, act=0, xs=256, ss=4, os=128, rs=128):
    return mla.LinearFp8Desc(M, K, N, act, xs, ss, os, rs)


BAD_FP8 = ((dict(M=-1), 2), (dict(K=0), 2), (dict(N=0), 2), (dict(K=248), 4), (dict(N=124), 4), (dict(act=5), 6), (dict(act=-1), 6),
           (dict(xs=240), 2), (dict(ss=3), 2), (dict(os=120), 2), (dict(xs=264), 4), (dict(os=132), 4), (dict(xs=1 << 40), 6),
           (dict(os=1 << 39), 6), (dict(K=(1 << 20) + 16, xs=1 << 21), 6), (dict(N=(1 << 20) + 8, os=1 << 21), 6),
           (dict(M=65535 * 128 + 1, ss=1 << 30), 6))


def test_linear_fp8_refusals(lib):
    def call(d=None, x=A, xs=A, w=A, ws=A, bias=NUL, residual=NUL, out=C_, status=NUL):
        return lib.mla_linear_fp8(ctypes.byref(fp8_desc() if d is None else d), x, xs, w, ws, bias, residual, out, status, NUL)

    assert lib.mla_linear_fp8(None, A, A, A, A, NUL, NUL, C_, NUL, NUL) == 1
    for name in ("x", "xs", "w", "ws", "out"):
        assert call(**{name: NUL}) == 1, name
    for name in ("x", "w", "bias", "residual", "out"):
        assert call(**{name: ODD}) == 4, name
    for name in ("xs", "ws", "status"):
        assert call(**{name: ODD4}) == 4, name
    for bad, code in BAD_FP8:
        assert call(fp8_desc(**bad)) == code, bad
    assert call(fp8_desc(rs=120), residual=B_) == 2 and call(fp8_desc(rs=132), residual=B_) == 4
    assert call(fp8_desc(rs=1 << 39), residual=B_) == 6
    assert call(x=C_) == 6 and call(w=C_) == 6  # out over an operand
    assert call(fp8_desc(rs=136), residual=C_) == 6  # residual in place, but with another stride
    assert call(fp8_desc(M=0), x=NUL) == 0


def test_linear_fp8_cuts(lib):
    """Every form is reached, at the sizes that the tests on the GPU use; sizes out of range are refused."""
    for form, size in LINEAR_FP8_FORMS.items():
        assert linear_fp8_form(*size) == form, size
    cut = mla.LinearCut()
    assert lib.mla_linear_fp8_query_cut(None, ctypes.byref(cut)) == 1
    assert lib.mla_linear_fp8_query_cut(ctypes.byref(fp8_desc()), None) == 1
    assert lib.mla_linear_fp8_query_cut(ctypes.byref(fp8_desc(M=0)), ctypes.byref(cut)) == 2
    for bad, code in BAD_FP8:
        assert lib.mla_linear_fp8_query_cut(ctypes.byref(fp8_desc(**bad)), ctypes.byref(cut)) == code, bad


def test_linear_fp8_cuts_hold_over_the_range(lib):
    """A cut's CTAs fit the card at once, and its parts and rounds cover every tile."""
    for M in (1, 7, 64, 128, 129, 300, 4096, 65535 * 128):
        for K in (16, 128, 144, 1008, 16384, 1 << 20):
            for N in (8, 72, 136, 7168, 1 << 20):
                c = mla.linear_fp8_cut(M, K, N)
                pair = c.tile_rows == 256
                assert (c.tile_rows, c.tile_columns) in ((128, 64), (128, 128), (256, 192), (256, 256)) and c.runs == 0
                assert M > 128 or not pair
                assert 1 <= c.k_parts <= (4 if pair else 8) and -(-K // 128) >= (2 * c.k_parts if c.k_parts > 1 else 1)
                units, tiles = c.ctas // (2 if pair else 1), -(-M // c.tile_rows) * -(-N // c.tile_columns)
                assert 1 <= c.ctas <= 152 and units % c.k_parts == 0
                if c.k_parts > 1:
                    assert tiles % units <= units // c.k_parts, (M, K, N)


# ------------------------------------------------------------------------------------------------------------ cache
def test_row_bytes(lib):
    assert mla.latent_row_bytes(mla.Problem(1, 1, 1, 512, 64, 128, 128, 1.0)) == 656
    assert mla.latent_row_bytes(mla.Problem(1, 1, 1, 64, 0, 128, 128, 1.0)) == 80
    for bad in (dict(d_c=96), dict(d_c=576), dict(d_c=0), dict(d_rope=8), dict(d_rope=80), dict(d_rope=-16)):
        assert lib.mla_latent_row_bytes(ctypes.byref(dims(**bad))) == 0
        with pytest.raises(ValueError):
            mla.latent_row_bytes(mla.Problem(1, 1, 1, **{"d_c": 512, "d_rope": 64, **bad}, d_nope=128, d_v=128, scale=1.0))
    assert lib.mla_latent_row_bytes(None) == 0


def test_make_cache_knows_rows_of_blocks():
    prob = mla.Problem(2, 16, 1, 128, 32, 64, 64, 1.0)
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    row = 128 + 16 + 64
    c = mla.make_cache(prob, torch.zeros(6, 64, row, dtype=torch.uint8), lens, table)
    assert (c.kv_dtype, c.page_size, c.num_pages) == (mla.KV_E4M3_BLOCKS, 64, 6)
    c = mla.make_cache(prob, torch.zeros(2, 100, row, dtype=torch.uint8), lens)
    assert (c.kv_dtype, c.seq_stride, c.capacity) == (mla.KV_E4M3_BLOCKS, 100 * row, 100)
    c = mla.make_cache(prob, torch.zeros(2, 100, 160, dtype=torch.uint8), lens, kv_scale=0.5)
    assert c.kv_dtype == mla.KV_E4M3
    for bad in (torch.zeros(2, 100, row, dtype=torch.float8_e4m3fn), torch.zeros(2, 100, row, dtype=torch.bfloat16),
                torch.zeros(2, 100, row + 16, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            mla.make_cache(prob, bad, lens)


def test_attention_refuses_rows_of_blocks(lib):
    """Rows of blocks are read back with mla_latent_load: the attention's entry points do not take them."""
    d, big = dims(), 1 << 40
    for c in (cache(), cache(paged=False)):
        r = ctypes.byref(c)
        assert lib.mla_decode_workspace_size(ctypes.byref(d), r, 0) == 0
        assert lib.mla_decode_attn(ctypes.byref(d), A, r, A, A, A, big, 0, NUL) == 6
        assert lib.mla_decode_attn_sparse(ctypes.byref(d), A, r, A, 64, A, A, A, big, 0, NUL) == 6
        assert lib.mla_decode_step(ctypes.byref(d), A, A, r, A, A, A, A, A, A, A, big, 0, NUL) == 6
        assert lib.mla_prefill(ctypes.byref(d), A, A, r, A, A, A, A, A, big, None, NUL) == 6
        assert lib.mla_prefill_expand(ctypes.byref(d), A, A, r, A, A, A, A, A, big, NUL) == 6
        assert lib.mla_naive_decode(ctypes.byref(d), A, A, r, A, A, A, A, A, big, NUL) == 6
        assert lib.mla_cache_append(ctypes.byref(d), 512, A, A, A, r, A, big, NUL) == 6


def test_store_refuses_bad_rows_of_blocks(lib):
    def call(c, d=None, slots=NUL):
        d = dims() if d is None else d
        return lib.mla_latent_store(ctypes.byref(d), None, A, 576, NUL, 0.0, NUL, slots, ctypes.byref(c), NUL, NUL)

    assert call(cache(kv=0)) == 1 and call(cache(kv=0x10008)) == 4 and call(cache(page_size=32)) == 6
    flat = cache(paged=False)
    flat.seq_stride = 4096 * 656 - 16
    assert call(flat) == 2  # shorter than its rows
    flat.seq_stride = 4096 * 656 + 8
    assert call(flat) == 4
    assert call(cache(paged=False), slots=A) == 6
    none = cache()
    none.kv_dtype = 2
    assert call(none) == 6


# ------------------------------------------------------------------------------------------------------------- load
def test_load_refusals(lib):
    def call(d=None, c=None, rows=8, positions=A, out=B_, stride=8 * 576, status=NUL):
        d = dims() if d is None else d
        c = cache() if c is None else c
        return lib.mla_latent_load(ctypes.byref(d), ctypes.byref(c), rows, positions, out, stride, status, NUL)

    d, c = dims(), cache()
    assert lib.mla_latent_load(None, ctypes.byref(c), 8, A, B_, 8 * 576, NUL, NUL) == 1
    assert lib.mla_latent_load(ctypes.byref(d), None, 8, A, B_, 8 * 576, NUL, NUL) == 1
    assert call(out=NUL) == 1 and call(c=cache(kv=0)) == 1 and call(c=cache(lens=0)) == 1
    assert call(out=ODD) == 4 and call(positions=ODD4) == 4 and call(status=ODD4) == 4 and call(c=cache(kv=0x10008)) == 4
    assert call(rows=-1) == 2 and call(stride=8 * 576 - 8) == 2 and call(stride=8 * 576 + 4) == 4
    assert call(rows=(1 << 30) + 8, stride=1 << 50) == 6
    assert call(d=dims(d_c=96)) == 6 and call(d=dims(d_c=0)) == 2 and call(d=dims(d_rope=80)) == 6 and call(d=dims(B=65536)) == 6
    assert call(c=cache(page_size=32)) == 6 and call(c=cache(num_pages=0)) == 2
    for kind in (mla.KV_BF16, mla.KV_E4M3):
        assert call(c=cache(paged=False, kind=kind, row=575)) == 2
    assert call(c=cache(kind=mla.KV_E4M3, scale=0.0)) == 2
    assert call(out=ctypes.c_void_p(0x10000)) == 6  # over the cache
    bad = cache()
    bad.kv_dtype = 2
    assert call(c=bad) == 6
    assert call(rows=0, out=NUL) == 0 and call(d=dims(B=0), out=NUL) == 0 and call(d=dims(B=-1)) == 2
    assert call(d=dims(B=65535, s_q=1 << 21, H=-1), rows=0, out=NUL) == 0  # of the sizes, B and the widths alone are read


# ---------------------------------------------------------------------------------------------------------- python
class OnDevice:
    """A CPU tensor that says it lies on a device: for checks that end before a pointer is used."""

    def __init__(self, t, dev=0):
        self.t, self.dev = t, dev

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.dev


@pytest.fixture
def device0(monkeypatch):
    monkeypatch.setattr(mla, "_current_device", lambda: 0)
    monkeypatch.setattr(mla, "_raw_stream", lambda dev, stream: 0)


def on(*shape, dtype=torch.bfloat16, dev=0):
    return OnDevice(torch.zeros(*shape, dtype=dtype), dev)


E4M3, F32 = torch.float8_e4m3fn, torch.float32


def test_quantize_checks_its_tensors(lib, device0):
    ok = dict(x=on(8, 256), codes=on(8, 256, dtype=E4M3), scales=on(2, 8, dtype=F32))
    for name, bad in (("x", on(8, 256, dtype=F32)), ("x", on(8, 256, dev=1)), ("x", on(8, 256, dev=-1)), ("x", on(8, 16, 16)),
                      ("x", OnDevice(torch.zeros(256, 8, dtype=torch.bfloat16).t())), ("norm_weight", on(255)),
                      ("norm_weight", on(256, dtype=F32)), ("codes", on(8, 256, dtype=torch.uint8)), ("codes", on(8, 128, dtype=E4M3)),
                      ("codes", on(8, 256, dtype=E4M3, dev=1)), ("scales", on(8, 2, dtype=F32)), ("scales", on(2, 8)),
                      ("scales", OnDevice(torch.zeros(8, 2).t())), ("scales", on(2, 8, dtype=F32, dev=1))):
        with pytest.raises(ValueError):
            mla.quantize(**{**ok, name: bad})


def test_linear_fp8_checks_its_tensors(lib, device0):
    ok = dict(x=on(8, 256, dtype=E4M3), x_scale=on(2, 8, dtype=F32), w=on(136, 256, dtype=E4M3), w_scale=on(2, 2, dtype=F32), out=on(8, 136))
    for name, bad in (("x", on(8, 256, dtype=torch.uint8)), ("x", on(8, 128, dtype=E4M3)), ("x", on(8, 256, dtype=E4M3, dev=1)),
                      ("x_scale", on(8, 2, dtype=F32)), ("x_scale", on(2, 8)), ("x_scale", OnDevice(torch.zeros(8, 2).t())),
                      ("w", on(136, 256)), ("w", OnDevice(torch.zeros(256, 136).to(E4M3).t())), ("w", on(136, 256, dtype=E4M3, dev=1)),
                      ("w_scale", on(1, 2, dtype=F32)), ("w_scale", on(2, 2, dtype=F32, dev=1)), ("bias", on(128)), ("bias", on(136, dtype=F32)),
                      ("residual", on(8, 128)), ("residual", on(8, 136, dev=1)), ("out", on(8, 128)), ("out", on(8, 136, dtype=F32)),
                      ("status", on(1)), ("status", on(0, dtype=torch.int32))):
        with pytest.raises(ValueError):
            mla.linear_fp8(**{**ok, name: bad})


def test_latent_load_checks_its_tensors(lib, device0):
    prob = mla.Problem(2, 16, 1, 64, 16, 64, 64, 1.0)
    c = cache(row=112)
    for name, bad in (("out", on(2, 5, 96)), ("out", on(2, 4, 80)), ("out", on(2, 5, 80, dtype=F32)), ("out", on(2, 5, 80, dev=1)),
                      ("out", OnDevice(torch.zeros(2, 10, 80, dtype=torch.bfloat16)[:, ::2])),
                      ("positions", on(2, 5, dtype=torch.int64)), ("positions", on(2, 4, dtype=torch.int32)),
                      ("positions", on(2, 5, dtype=torch.int32, dev=1)), ("status", on(1))):
        with pytest.raises(ValueError):
            mla.latent_load(prob, c, 5, **{**dict(out=on(2, 5, 80)), name: bad})
