"""The operators around the attention (mla_rope, mla_pages_update, mla_latent_store, mla_linear): what they refuse on the
host, before anything is launched, and the rotation's frequencies.  No GPU needed."""
import copy
import ctypes
import dataclasses
import math
import pickle
import random
import weakref

import pytest
import torch

from helpers import LINEAR_FORMS
from mla_decode_attention_absorbed_gb300 import build, mla
from oracle import layer

NUL, A = ctypes.c_void_p(0), ctypes.c_void_p(0x40000)
ODD, ODD4 = ctypes.c_void_p(0x40008), ctypes.c_void_p(0x40002)
NAMES = {"plain": mla.ROPE_PLAIN, "linear": mla.ROPE_LINEAR, "ntk": mla.ROPE_NTK, "yarn": mla.ROPE_YARN}


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mla.load()


def dims(B=4, H=16, s_q=1, d_c=512, d_rope=64, d_nope=128, d_v=128):
    return mla.Problem(B, H, s_q, d_c, d_rope, d_nope, d_v, 0.1).dims()


def test_problem_keeps_its_structure_up_to_date():
    """The ctypes structure made once per Problem follows its fields, and copies and pickles do without it."""
    p = mla.Problem(4, 16, 1, 512, 64, 128, 128, 0.5)

    def seen(q):
        return ctypes.cast(q.dims_ref(), ctypes.POINTER(mla.Dims)).contents

    assert seen(p).B == 4 and p.dims_ref() is p.dims_ref()
    q, r, s = copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p))
    p.B, q.H, r.scale = 7, 3, 0.25
    assert (seen(p).B, seen(p).H) == (7, 16) and (seen(q).B, seen(q).H) == (4, 3) and seen(r).scale == 0.25
    assert s == mla.Problem(4, 16, 1, 512, 64, 128, 128, 0.5) and seen(s).scale == 0.5


def test_problem_holds_its_fields_alone():
    """What dims_ref() keeps is no field: vars() and copies by them are the sizes, before and after a call."""
    p = mla.Problem(4, 16, 1, 512, 64, 128, 128, 0.5)
    fields = dict(B=4, H=16, s_q=1, d_c=512, d_rope=64, d_nope=128, d_v=128, scale=0.5)
    assert vars(p) == fields and p.dims_ref() is not None and vars(p) == fields
    assert mla.Problem(**vars(p)) == p and dataclasses.replace(p, B=2).dims().B == 2 and weakref.ref(p)() is p
    vars(p)["B"] = 3
    assert ctypes.cast(p.dims_ref(), ctypes.POINTER(mla.Dims)).contents.B == 3


def test_problem_field_set_while_another_thread_makes_the_structure(monkeypatch):
    """A field set between the structure's making and its keeping (as by another thread): the next call sees it."""
    p = mla.Problem(4, 16, 1, 512, 64, 128, 128, 0.5)
    make = mla.Dims

    class Interrupted(make):
        def __init__(self, *values):
            super().__init__(*values)
            if p.B == 4:
                p.B = 7

    with monkeypatch.context() as m:
        m.setattr(mla, "Dims", Interrupted)
        p.dims_ref()
    assert ctypes.cast(p.dims_ref(), ctypes.POINTER(make)).contents.B == 7


# ------------------------------------------------------------------------------------------------------------- rope
@pytest.mark.parametrize("scaling", list(NAMES))
@pytest.mark.parametrize("d,base,factor,original", [(64, 10000.0, 40.0, 4096), (48, 500000.0, 8.0, 8192),
                                                    (16, 1e6, 2.5, 300), (32, 10000.0, 4.0, 7)])
def test_rope_plan_holds_the_frequencies(lib, scaling, d, base, factor, original):
    """turn[i] = f_i / 2 pi in units of 2^-64.  pow and log are right to a few units of 2^-53, and so is f (2^-48 of
    it); rounding to whole units is off by half of one, pi 2^-64 < 2^-62 radians.  The two add up."""
    plan = mla.rope_plan(d, base=base, scaling=NAMES[scaling], factor=factor, original_len=original)
    want = layer.frequencies(d, base, scaling, factor, original)
    for i, f in enumerate(want):
        assert abs(plan.turn[i] / 2.0 ** 64 * 2 * math.pi - f) <= 2.0 ** -48 * f + 2.0 ** -62, i
    assert all(plan.turn[i] == 0 for i in range(d // 2, 32))


def test_rope_plan_takes_a_table(lib):
    table = [0.5, 7.0, -0.25, 1e-6, 0.0, 1.0, 2.0, 3.0]  # whole turns and signs fold into [0, 1) turns
    plan = mla.rope_plan(16, layout=mla.ROPE_HALF, mscale=1.5, inv_freq=table)
    assert plan.layout == mla.ROPE_HALF and plan.mscale == 1.5
    for i, f in enumerate(table):
        turns = f / (2 * math.pi)
        assert abs(plan.turn[i] / 2.0 ** 64 - (turns - math.floor(turns))) <= 2.0 ** -51
    with pytest.raises(ValueError):
        mla.rope_plan(16, inv_freq=table[:-1])


@pytest.mark.parametrize("bad,code", [
    (dict(d_rope=0), 6), (dict(d_rope=24), 6), (dict(d_rope=80), 6), (dict(layout=2), 6), (dict(scaling=4), 6),
    (dict(base=1.0), 2), (dict(base=float("nan")), 2), (dict(base=float("inf")), 2), (dict(mscale=0.0), 2),
    (dict(mscale=float("inf")), 2), (dict(mscale=1e60), 2), (dict(scaling=1, factor=0.0), 2),
    (dict(scaling=2, factor=float("nan")), 2), (dict(scaling=2, factor=1e308), 2), (dict(scaling=3, factor=2.0), 2),
    (dict(scaling=3, factor=2.0, original_len=4096, beta_fast=0.0), 2),
    (dict(scaling=3, factor=2.0, original_len=4096, beta_slow=float("inf")), 2),
    (dict(inv_freq=[float("nan")] * 32), 2)])
def test_rope_plan_refusals(lib, bad, code):
    with pytest.raises(mla.MLAError) as e:
        mla.rope_plan(**{"d_rope": 64, **bad})
    assert e.value.code == code
    assert lib.mla_rope_init(None, None) == 1


def test_rope_refusals(lib):
    plan = mla.rope_plan(64)
    p = ctypes.byref(plan)
    W = 192

    def call(d=None, plan=p, x=A, ts=16 * W, hs=W, pos=A, lens=NUL, q_nope=ctypes.c_void_p(0x60000),
             q_rope=ctypes.c_void_p(0x70000)):
        d = dims() if d is None else d
        return lib.mla_rope(ctypes.byref(d), plan, x, ts, hs, pos, lens, q_nope, q_rope, 0, NUL)

    assert lib.mla_rope(None, p, A, 1, 1, A, A, A, A, 0, NUL) == 1
    assert call(plan=None) == 1
    assert call(x=NUL) == 1 and call(q_rope=NUL) == 1 and call(pos=NUL, lens=NUL) == 1
    assert call(x=ODD) == 4 and call(q_nope=ODD) == 4 and call(q_rope=ODD) == 4 and call(pos=ODD4) == 4
    assert call(lens=ODD4) == 4
    assert call(hs=W - 8) == 2 and call(ts=16 * W - 8) == 2 and call(ts=16 * W + 4) == 4 and call(hs=W + 4, ts=1 << 20) == 4
    assert call(d=dims(d_rope=48)) == 2  # another width than the plan's
    assert call(d=dims(d_nope=24)) == 6 and call(d=dims(d_nope=272)) == 6 and call(d=dims(B=65536)) == 6
    assert call(d=dims(B=65535, s_q=129)) == 6 and call(d=dims(B=-1)) == 2 and call(d=dims(s_q=0)) == 2
    assert call(d=dims(B=0), x=NUL) == 0  # nothing to do
    B_ = ctypes.c_void_p(0x50000)
    for over in (dict(x=A, q_nope=A, q_rope=B_), dict(x=B_, q_nope=A, q_rope=A), dict(x=A, q_nope=B_, q_rope=A),
                 dict(x=A, q_nope=NUL, q_rope=A)):  # in place only where x is dense rows of d_rope
        assert call(**over) == 6, over
    broken = mla.rope_plan(64)
    broken.d_rope = 80
    assert call(plan=ctypes.byref(broken)) == 6


# ------------------------------------------------------------------------------------------------------------ pages
def pool(B=4, page_size=64, max_pages=16, num_pages=100, table=0x40000, ring=0x50000, state=0x60000, state_out=0x60010):
    return mla.PagePool(B, page_size, max_pages, num_pages, table, ring, state, state_out)


def test_pages_refusals(lib):
    def call(p=None, old=A, new=ctypes.c_void_p(0x41000), n=10, lens=ctypes.c_void_p(0x42000), start=A, pos=A, slots=A,
             status=NUL):
        p = pool() if p is None else p
        return lib.mla_pages_update(ctypes.byref(p), old, new, n, lens, start, pos, slots, status, NUL)

    assert lib.mla_pages_update(None, A, A, 1, A, A, A, A, A, NUL) == 1
    for bad in (dict(table=0), dict(ring=0), dict(state=0), dict(state_out=0)):
        assert call(pool(**bad)) == 1, bad
    for name in ("old", "new", "lens", "start", "pos", "slots"):
        assert call(**{name: NUL}) == 1, name
    for name in ("old", "new", "lens", "start", "pos", "slots", "status"):
        assert call(**{name: ODD4}) == 4, name
    for bad, code in ((dict(B=-1), 2), (dict(page_size=0), 2), (dict(max_pages=0), 2), (dict(num_pages=0), 2),
                      (dict(page_size=32), 6), (dict(B=65536), 6), (dict(max_pages=1 << 25), 6),
                      (dict(num_pages=1 << 25), 6)):
        assert call(pool(**bad)) == code, bad
    assert call(n=-1) == 2 and call(n=(1 << 30) + 1) == 6
    # outputs that are inputs
    assert call(pool(state_out=0x60000)) == 6
    assert call(lens=A) == 6 and call(lens=ctypes.c_void_p(0x41000)) == 6


# ------------------------------------------------------------------------------------------------------------ store
def cache(T=4096, paged=True, fp8=False, scale=0.5, page_size=64, num_pages=1000, kv=0x10000, lens=0x20000):
    dt = 1 if fp8 else 0
    if paged:
        return mla.Cache(kv, 0, 0, 0x30000, T // 64, page_size, num_pages, lens, 0, dt, scale)
    return mla.Cache(kv, T * 576, T, None, 0, 64, 0, lens, 0, dt, scale)


def test_store_refusals(lib):
    plan = mla.rope_plan(64)

    def call(d=None, plan=ctypes.byref(plan), x=A, ts=576, w=A, eps=1e-6, pos=A, slots=A, c=None, status=A):
        d = dims() if d is None else d
        c = cache() if c is None else c
        return lib.mla_latent_store(ctypes.byref(d), plan, x, ts, w, eps, pos, slots, ctypes.byref(c), status, NUL)

    d = dims()
    assert lib.mla_latent_store(None, None, A, 576, A, 0.0, A, A, ctypes.byref(cache()), A, NUL) == 1
    assert lib.mla_latent_store(ctypes.byref(d), None, A, 576, A, 0.0, A, A, None, A, NUL) == 1
    assert call(x=NUL) == 1 and call(c=cache(kv=0)) == 1 and call(c=cache(lens=0)) == 1
    for name in ("x", "w"):
        assert call(**{name: ODD}) == 4, name
    for name in ("pos", "slots", "status"):
        assert call(**{name: ODD4}) == 4, name
    assert call(ts=575) == 2 and call(ts=580) == 4
    assert call(eps=-1.0) == 2 and call(eps=float("nan")) == 2 and call(eps=float("inf")) == 2
    assert call(d=dims(d_c=96)) == 6 and call(d=dims(d_c=576)) == 6 and call(d=dims(d_rope=48)) == 2
    assert call(d=dims(d_rope=80), plan=None) == 6 and call(d=dims(B=65536)) == 6
    assert call(c=cache(paged=False)) == 6  # slots are rows of a pool
    assert call(c=cache(page_size=32)) == 6 and call(c=cache(num_pages=1 << 25)) == 6 and call(c=cache(num_pages=0)) == 2
    assert call(c=cache(fp8=True, scale=1e-39)) == 6
    assert call(c=cache(fp8=True, scale=0.0)) == 2 and call(c=cache(fp8=True, scale=float("nan"))) == 2
    bad = cache()
    bad.kv_dtype = 2
    assert call(c=bad) == 6
    assert call(d=dims(B=0), x=NUL) == 0


# ----------------------------------------------------------------------------------------------------------- linear
def test_linear_refusals(lib):
    def desc(M=4, K=64, N=128, act=0, xs=64, os=128, rs=128):
        return mla.LinearDesc(M, K, N, act, xs, os, rs)

    def call(d=None, x=A, w=A, bias=NUL, residual=NUL, out=ctypes.c_void_p(0x60000), ws=A, nbytes=1 << 30):
        d = desc() if d is None else d
        return lib.mla_linear(ctypes.byref(d), x, w, bias, residual, out, ws, nbytes, NUL)

    assert lib.mla_linear(None, A, A, A, A, A, A, 0, NUL) == 1
    for name in ("x", "w", "out"):
        assert call(**{name: NUL}) == 1, name
    runs = desc(M=8, K=4104, N=20480, xs=4104, os=20480)  # 160 tiles: cut along K, with pieces in the workspace
    assert lib.mla_linear_workspace_size(ctypes.byref(runs)) > 256 and call(runs, ws=NUL) == 1
    for name in ("x", "w", "bias", "residual", "out", "ws"):
        assert call(**{name: ODD}) == 4, name
    for bad, code in ((dict(M=-1), 2), (dict(K=0), 2), (dict(N=0), 2), (dict(K=60, xs=64), 4), (dict(N=124), 4),
                      (dict(act=5), 6), (dict(act=-1), 6), (dict(xs=56), 2), (dict(os=120), 2), (dict(xs=68), 4),
                      (dict(os=132), 4), (dict(K=(1 << 20) + 8, xs=1 << 21), 6), (dict(N=(1 << 20) + 8, os=1 << 21), 6),
                      (dict(M=65535 * 128 + 1), 6), (dict(xs=1 << 39), 6)):
        assert call(desc(**bad)) == code, bad
        assert lib.mla_linear_workspace_size(ctypes.byref(desc(**bad))) == 0, bad
    assert call(desc(rs=120), residual=A) == 2 and call(desc(rs=132), residual=A) == 4
    B_ = ctypes.c_void_p(0x50000)
    assert call(x=A, w=B_, out=A) == 6 and call(x=B_, w=A, out=A) == 6  # out over an operand
    assert call(desc(rs=136), x=B_, w=B_, residual=A, out=A) == 6  # residual in place, but with another stride
    need = lib.mla_linear_workspace_size(ctypes.byref(desc()))
    assert need > 0 and call(nbytes=need - 1) == 5
    assert call(desc(M=0), x=NUL) == 0  # nothing to do


def test_linear_workspace_stays_bounded(lib):
    """Two fp32 tiles a CTA at most, whatever the shape."""
    for M in (1, 17, 64, 300, 4096, 65535):
        for K in (8, 64, 1000, 16384):
            for N in (8, 136, 7168, 65536):
                assert 0 < mla.linear_workspace_size(M, K, N) <= 2 * 152 * 128 * 256 * 4, (M, K, N)


# ---------------------------------------------------------------------------------------------------------- python
def test_a_stream_of_another_device_is_refused():
    class Stream:
        device_index, device, cuda_stream = 1, "cuda:1", 0x1234

    assert mla._raw_stream(1, Stream()) == 0x1234
    with pytest.raises(ValueError):
        mla._raw_stream(0, Stream())


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


def test_linear_checks_its_workspace(lib, device0):
    x, w, out = (OnDevice(torch.zeros(*n, dtype=torch.bfloat16)) for n in ((8, 64), (64, 128), (8, 128)))
    for ws in (OnDevice(torch.zeros(512, dtype=torch.uint8), -1), OnDevice(torch.zeros(512, dtype=torch.uint8), 1),
               OnDevice(torch.zeros(1024, dtype=torch.uint8)[::2])):
        with pytest.raises(ValueError, match="workspace"):
            mla.linear(x, w, out=out, workspace=ws)


def test_pages_update_checks_fields_assigned_later(lib, device0):
    i32 = lambda *n: OnDevice(torch.zeros(*n, dtype=torch.int32))  # noqa: E731
    table, ring, lens = i32(2, 4), i32(8), i32(2)
    bad = [("free_ring", r) for r in (OnDevice(ring.t.long()), OnDevice(ring.t, -1), OnDevice(ring.t, 1),
                                      OnDevice(torch.zeros(16, dtype=torch.int32)[::2]), i32(2, 4))]
    bad += [("block_table", t) for t in (OnDevice(table.t.long()), OnDevice(table.t, -1), i32(8),
                                         OnDevice(torch.zeros(4, 2, dtype=torch.int32).t()))]
    out = mla.PagesStep(i32(2), i32(2), i32(3), i32(4), i32(4))
    for name, value in bad:
        pages = mla.Pages(table, ring, 64)
        setattr(pages, name, value)
        with pytest.raises(ValueError):
            mla.pages_update(pages, i32(2), lens, i32(2), 4, out=out)


def test_linear_status_is_checked_like_the_rest(lib, device0):
    d, out = mla.LinearDesc(4, 64, 128, 0, 64, 128, 128), ctypes.c_void_p(0x60000)
    assert lib.mla_linear_status(ctypes.byref(d), A, A, NUL, NUL, out, A, 1 << 30, ODD4, NUL) == 4
    assert lib.mla_linear_status(None, A, A, NUL, NUL, out, A, 1 << 30, A, NUL) == 1
    x, w, y = (OnDevice(torch.zeros(*n, dtype=torch.bfloat16)) for n in ((8, 64), (64, 128), (8, 128)))
    for word in (OnDevice(torch.zeros(1, dtype=torch.int64)), OnDevice(torch.zeros(1, dtype=torch.int32), -1)):
        with pytest.raises(ValueError, match="status"):
            mla.linear(x, w, out=y, status=word)


# ------------------------------------------------------------------------------------------------- how products are cut
@pytest.mark.parametrize("form", LINEAR_FORMS)
def test_linear_forms_are_reached(lib, form):
    """The shapes that the GPU tests compare, form by form, are still cut that way (without a GPU the plan is that of 152
    SMs); together they hold every form there is."""
    cut = mla.linear_cut(*LINEAR_FORMS[form])
    assert (cut.tile_rows, cut.tile_columns, cut.k_parts, cut.runs) == form and 1 <= cut.ctas <= 152


def test_linear_forms_are_all_there(lib):
    rng = random.Random(5)
    seen = set()
    for _ in range(20000):
        M, K, N = int(math.exp(rng.uniform(0, 9))), 8 * int(math.exp(rng.uniform(0, 7.8))), 8 * int(math.exp(rng.uniform(0, 8)))
        cut = mla.linear_cut(M, K, N)
        seen.add((cut.tile_rows, cut.tile_columns, cut.k_parts, cut.runs))
        assert (mla.linear_workspace_size(M, K, N) > 256) == bool(cut.runs)
    assert seen <= set(LINEAR_FORMS)


def test_linear_cut_refusals(lib):
    cut = mla.LinearCut()
    assert lib.mla_linear_query_cut(None, ctypes.byref(cut)) == 1
    assert lib.mla_linear_query_cut(ctypes.byref(mla.LinearDesc(4, 64, 128, 0, 64, 128, 128)), None) == 1
    for M, K, N, code in ((0, 64, 128, 2), (-1, 64, 128, 2), (4, 60, 128, 4), (4, 64, 1 << 21, 6)):
        assert lib.mla_linear_query_cut(ctypes.byref(mla.LinearDesc(M, K, N, 0, 64, N, N)), ctypes.byref(cut)) == code
