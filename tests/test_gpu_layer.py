"""The operators around the attention on the GPU against plain 64-bit implementations (oracle/layer.py): rotary positions,
page tables, the latent store, the matrix product with its epilogue, and a run of them together with the attention.

Tolerances count roundings.  A bf16 result is off by at most half a step, 2^-8 of its value (E4M3: 2^-4, and 2^-10 in
units of the code among its subnormals); what is computed before that in fp32 adds a few times 2^-24 of the terms."""
import math
import threading

import pytest
import torch

import oracle
from helpers import LINEAR_FORMS, within_tolerance
from mla_decode_attention_absorbed_gb300 import build, mla
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = "cuda"
ROPE = {"plain": mla.ROPE_PLAIN, "linear": mla.ROPE_LINEAR, "ntk": mla.ROPE_NTK, "yarn": mla.ROPE_YARN}
ACTS = {"none": mla.ACT_NONE, "relu": mla.ACT_RELU, "silu": mla.ACT_SILU, "gelu": mla.ACT_GELU,
        "gelu_tanh": mla.ACT_GELU_TANH}
BF16, I32 = torch.bfloat16, torch.int32


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


# ------------------------------------------------------------------------------------------------------------- rope
def problem(B=2, H=16, s_q=1, d_c=512, d_rope=64, d_nope=128, d_v=128):
    return mla.Problem(B, H, s_q, d_c, d_rope, d_nope, d_v, (d_nope + d_rope) ** -0.5)


def rope_tolerance(x, positions, freq, half, mscale, want):
    """Half a bf16 step; the angle: 2^-25 half turns from its conversion to fp32 and 2^-23 from sincospi, 2^-22 together
    with the fp32 products, and the frequency's own 2^-51 (plan and oracle each work it out in 64 bits, and the oracle
    rounds angles of that size) times the position.  Either coordinate of a pair moves by that times the pair's length."""
    p, q = layer.pairs(x.shape[-1], half)
    xd = x.double()
    length = mscale * (xd[..., p].abs() + xd[..., q].abs())
    angle = positions.double()[..., None] * torch.tensor(freq, dtype=torch.float64).abs()
    tol = 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8)
    slack = length * (2.0 ** -21 + angle * 2.0 ** -51)
    tol[..., p] += slack
    tol[..., q] += slack
    return tol


ROPE_CASES = [
    # B, s_q, H, d_nope, d_rope, half, scaling, mscale, positions given, row padding, longest position
    (1, 1, 1, 16, 16, False, "plain", 1.0, False, 0, 100),
    (1, 1, 1, 0, 64, True, "plain", 1.0, True, 8, 2 ** 31 - 1),
    (3, 2, 128, 128, 64, False, "yarn", 1.0, False, 0, 160000),
    (2, 1, 128, 128, 64, True, "plain", 1.1386, True, 24, 2 ** 31 - 1),
    (37, 3, 5, 80, 48, False, "ntk", 0.75, False, 8, 2 ** 30),
    (5, 7, 40, 256, 32, True, "linear", 1.0, True, 0, 2 ** 27),
    (65, 2, 1, 0, 64, False, "plain", 1.0, False, 512, 32768),
    (1, 300, 1, 0, 16, True, "yarn", 2.0, False, 0, 4096),
    (2, 1, 200, 48, 64, False, "plain", 1.0, True, 8, 8192),
    (1, 129, 130, 16, 48, True, "plain", 1.0, False, 0, 8192),
]


@pytest.mark.parametrize("B,s_q,H,d_nope,d_rope,half,scaling,mscale,given,pad,far", ROPE_CASES)
def test_rope(B, s_q, H, d_nope, d_rope, half, scaling, mscale, given, pad, far):
    g = gen(B + s_q + H)
    width = d_nope + d_rope
    rows = randn(g, B, s_q, H * width + pad)
    x = rows[:, :, :H * width].unflatten(2, (H, width))
    lens = torch.randint(s_q, far, (B,), generator=g, dtype=I32) if far > s_q else torch.full((B,), s_q, dtype=I32)
    lens[0] = far
    at = lens.long()[:, None] - s_q + torch.arange(s_q)
    if given:
        at = torch.randint(0, far, (B, s_q), generator=g)
        at[0, 0], at[-1, -1] = 0, far
    kw = dict(base=10000.0, scaling=scaling, factor=8.0, original_len=4096)
    freq = layer.frequencies(d_rope, **kw)
    plan = mla.rope_plan(d_rope, layout=mla.ROPE_HALF if half else mla.ROPE_INTERLEAVED, mscale=mscale,
                         **{**kw, "scaling": ROPE[scaling]})
    prob = problem(B, H, s_q, d_rope=d_rope, d_nope=max(d_nope, 16))
    xd = rows.to(DEV)[:, :, :H * width].unflatten(2, (H, width))
    pos = dict(positions=at.to(I32).to(DEV)) if given else dict(seq_lens=lens.to(DEV))
    for transpose in (False, True):
        out = mla.rope(prob, plan, xd, transpose=transpose, **pos)
        if d_nope:
            assert torch.equal(out[0].cpu(), x[..., :d_nope])
            out = out[1]
        want = layer.rotate(x[..., d_nope:], at[:, :, None], freq, half, float(plan.mscale), transpose)
        close(out, want, rope_tolerance(x[..., d_nope:], at[:, :, None], freq, half, mscale, want), f"transpose {transpose}")


def test_rope_in_place_and_padding():
    """x is its own output; tokens at negative positions (given, or before a short sequence) keep what was there."""
    g = gen(3)
    prob = problem(B=3, H=4, s_q=2, d_rope=32)
    plan = mla.rope_plan(32, layout=mla.ROPE_HALF)
    x = randn(g, 3, 2, 4, 32)
    lens = torch.tensor([0, 1, 9], dtype=I32)  # positions -2, -1 | -1, 0 | 7, 8
    freq = layer.frequencies(32)
    for kw in (dict(seq_lens=lens.to(DEV)), dict(positions=torch.tensor([[-2, -1], [-1, 0], [7, 8]], dtype=I32, device=DEV))):
        y = x.to(DEV)
        out = mla.rope(prob, plan, y, q_rope=y, **kw)
        assert out.data_ptr() == y.data_ptr()
        at = torch.tensor([[-2, -1], [-1, 0], [7, 8]])
        want = layer.rotate(x, at[:, :, None], freq, True)
        tol = rope_tolerance(x, at[:, :, None], freq, True, 1.0, want)
        keep = at < 0
        want[keep], tol[keep] = x.double()[keep], 0.0
        close(y, want, tol)
    # the split: neither part of a padded token is written
    x = randn(g, 3, 2, 4, 160)
    q_nope = torch.full((3, 2, 4, 128), 7.0, dtype=BF16, device=DEV)
    q_rope = torch.full((3, 2, 4, 32), 7.0, dtype=BF16, device=DEV)
    mla.rope(prob, plan, x.to(DEV), seq_lens=lens.to(DEV), q_nope=q_nope, q_rope=q_rope)
    assert bool((q_nope[0] == 7).all()) and bool((q_rope[0] == 7).all()) and bool((q_rope[1, 0] == 7).all())
    assert torch.equal(q_nope[1:].cpu()[:, 1], x[1:, 1, :, :128]) and bool((q_rope[2] != 7).any())


def test_rope_gradient_is_the_transposed_call():
    """d<y, rope(x)>/dx by autograd through the plain formula in 64 bits, and by differences: the map is linear, so the
    difference quotient of any step is the derivative; both against the transposed call."""
    g = gen(4)
    B, s_q, H, d = 2, 3, 5, 48
    x, y = randn(g, B, s_q, H, d), randn(g, B, s_q, H, d)
    at = torch.randint(0, 100000, (B, s_q), generator=g)
    freq = layer.frequencies(d, scaling="ntk", factor=4.0)
    plan = mla.rope_plan(d, scaling=mla.ROPE_NTK, factor=4.0, mscale=1.25)
    got = mla.rope(problem(B, H, s_q, d_rope=d), plan, y.to(DEV), positions=at.to(I32).to(DEV), transpose=True)
    xr = x.double().requires_grad_(True)
    f = (layer.rotate(xr, at[:, :, None], freq, False, 1.25) * y.double()).sum()
    f.backward()
    tol = rope_tolerance(y, at[:, :, None], freq, False, 1.25, xr.grad)
    close(got, xr.grad, tol)
    for at_xyz in ((0, 0, 0, 0), (1, 2, 4, 47), (0, 1, 3, 24)):
        step = x.double().clone()
        step[at_xyz] += 1.0
        diff = (layer.rotate(step, at[:, :, None], freq, False, 1.25) * y.double()).sum() - f.detach()
        assert abs(float(got[at_xyz]) - float(diff)) <= float(tol[at_xyz]) + 1e-9


def test_rope_carries_infinities_and_nan():
    x = torch.zeros(1, 1, 2, 16, dtype=BF16)
    x[0, 0, 0, 2], x[0, 0, 1, 5] = float("inf"), float("nan")
    out = mla.rope(problem(1, 2, 1, d_rope=16), mla.rope_plan(16), x.to(DEV),
                   positions=torch.tensor([[1000]], dtype=I32, device=DEV)).cpu()
    assert bool(torch.isinf(out[0, 0, 0, 2:4]).all()) and bool(torch.isnan(out[0, 0, 1, 4:6]).all())
    assert int((~torch.isfinite(out)).sum()) == 4


# ------------------------------------------------------------------------------------------------------------ pages
CODES = {0: "ok", 2: "shape", 3: "length", 9: "page"}


def pages_case(B, ps, max_pages, seed, grow, spare=3):
    """A consistent pool: requests of random lengths hold random pages, the others lie in the ring."""
    g = gen(seed)
    most = ps * max_pages
    old = torch.randint(0, most + 1, (B,), generator=g)
    old[torch.rand(B, generator=g) < 0.2] = 0
    new = (old + torch.randint(0, grow + 1, (B,), generator=g)).clamp(max=most)
    kind = torch.rand(B, generator=g)
    new[kind < 0.15] = 0
    shrink = (kind >= 0.15) & (kind < 0.3)
    new[shrink] = (old[shrink] - 70).clamp(min=0)
    had, has = -(-old // ps), -(-new // ps)
    held, need = int(had.sum()), int((has - had).clamp(min=0).sum())
    P = max(held + max(need + spare, 0), 1)
    ids = torch.randperm(P, generator=g)
    table = torch.full((B, max_pages), -1, dtype=torch.int64)
    n = 0
    for b in range(B):
        table[b, :had[b]] = ids[n:n + had[b]]
        n += int(had[b])
    head = int(torch.randint(0, P, (1,), generator=g))
    ring = torch.full((P,), -5, dtype=torch.int64)
    ring[(head + torch.arange(P - held)) % P] = ids[held:]
    return table, ring, [head, P - held], old, new


def pages_check(table, ring, state, old, new, ps, max_tokens, codes=None, status0=0):
    """The call against the plain loop, bit for bit, once and again on the same inputs."""
    want = layer.pages_update(table.tolist(), ring.tolist(), state, old.tolist(), new.tolist(), ps, max_tokens)
    dev = lambda t: torch.as_tensor(t).to(I32).to(DEV)  # noqa: E731
    pages = mla.Pages(dev(table), dev(ring), ps)
    st, o, n = dev(state), dev(old), dev(new)
    status = torch.full((1,), status0, dtype=I32, device=DEV)
    for _ in range(2):
        out = mla.pages_update(pages, st, o, n, max_tokens, status=status)
        got = (pages.block_table, pages.free_ring, out.ring_state, out.seq_lens, out.token_start, out.positions, out.slots)
        names = ("block_table", "free_ring", "ring_state", "seq_lens", "token_start", "positions", "slots")
        for name, t, w in zip(names, got, want):
            assert torch.equal(t.cpu().long().flatten(), torch.tensor(w, dtype=torch.int64).flatten()), name
    for t, w in ((st, state), (o, old), (n, new)):
        assert torch.equal(t.cpu().long(), torch.as_tensor(w).long()), "inputs are left as they are"
    s = int(status)
    if status0:
        assert s == status0
    else:
        assert s in want[-1] if want[-1] else s == 0, (CODES.get(s, s), want[-1])
    if codes is not None:
        assert want[-1] == codes
    return out


@pytest.mark.parametrize("B,ps,max_pages,grow", [
    (1, 64, 1, 1), (1, 64, 40, 2000), (3, 128, 4, 1), (31, 64, 9, 70), (64, 64, 128, 1), (255, 64, 33, 300),
    (1000, 64, 16, 4), (1024, 192, 3, 64), (1025, 64, 5, 130), (3000, 64, 3, 2), (8191, 128, 4, 9), (20000, 64, 2, 60)])
def test_pages(B, ps, max_pages, grow):
    table, ring, state, old, new = pages_case(B, ps, max_pages, B + grow, grow)
    n = int((new - old).clamp(min=0).sum())
    pages_check(table, ring, state, old, new, ps, n + 13, codes=set())
    pages_check(table, ring, state, old, new, ps, n, codes=set())


def test_pages_one_long_among_many():
    """One prompt of 200,000 tokens among requests that grow by nothing or one."""
    table, ring, state, old, new = pages_case(700, 64, 3200, 5, 1)
    old[300], new[300] = 17, 200017
    ids = list(range(len(ring) + 3200))
    had = -(-old // 64)
    n = 0
    for b in range(700):
        table[b] = -1
        table[b, :had[b]] = torch.tensor(ids[n:n + had[b]])
        n += int(had[b])
    ring = torch.full((len(ids),), -5, dtype=torch.int64)
    ring[(torch.arange(len(ids) - n) + 11) % len(ids)] = torch.tensor(ids[n:])
    pages_check(table, ring, [11, len(ids) - n], old, new, 64, 210000, codes=set())


@pytest.mark.parametrize("B,ps,max_pages,grow,short", [
    (3, 64, 1100, 60000, -3), (3, 256, 300, 60000, 40), (2000, 192, 5, 400, -3), (2000, 64, 16, 400, 1500),
    (4000, 64, 20, 129, -3), (900, 128, 40, 3000, 5000)])
def test_pages_many_tokens(B, ps, max_pages, grow, short):
    """Tokens by warps: long requests, short ones, both, some of them without pages; with room to spare, with too
    little, and into arrays that start between two 16-byte boundaries."""
    table, ring, state, old, new = pages_case(B, ps, max_pages, B + grow, grow, spare=-short)
    if B == 4000:  # every other request grows by a token or not at all, in long stretches
        new[500:2500] = torch.where(torch.arange(2000) % 3 == 0, old[500:2500] + 1, old[500:2500]).clamp(max=ps * max_pages)
    n = int((new - old).clamp(min=0).sum())
    assert n > 38912 * (4 if B > 992 else 1) * 0.5
    room = max(n + 5, 152 * 1024 + 1)
    codes = {layer.PAGE} if short > 0 else set()
    out = pages_check(table, ring, state, old, new, ps, room, codes=codes)
    if short < 0:
        pages_check(table, ring, state, old, new, ps, n - 777 if n - 777 > 152 * 1024 else n, codes=None)
    # into views that begin one element after an allocation
    dev = lambda t: torch.as_tensor(t).to(I32).to(DEV)  # noqa: E731
    buf = torch.full((2, room + 2), -9, dtype=I32, device=DEV)
    views = mla.PagesStep(dev(old), dev(state), torch.empty(B + 1, dtype=I32, device=DEV), buf[0, 1:-1], buf[1, 1:-1])
    mla.pages_update(mla.Pages(dev(table), dev(ring), ps), dev(state), dev(old), dev(new), room, out=views)
    assert torch.equal(views.positions, out.positions) and torch.equal(views.slots, out.slots)
    assert bool((buf[:, 0] == -9).all()) and bool((buf[:, -1] == -9).all())


@pytest.mark.parametrize("B,short", [(2, 1), (40, 1), (40, 25), (3000, 700)])
def test_pages_ring_runs_out(B, short):
    """Requests are served in order as long as pages last; those that need none always are."""
    table, ring, state, old, new = pages_case(B, 64, 8, B + 1, 150, spare=-short)
    n = int((new - old).clamp(min=0).sum())
    pages_check(table, ring, state, old, new, 64, n + 5, codes={layer.PAGE})


def test_pages_tokens_run_out():
    table, ring, state, old, new = pages_case(100, 64, 8, 8, 150)
    n = int((new - old).clamp(min=0).sum())
    pages_check(table, ring, state, old, new, 64, n // 2, codes={layer.SHAPE})
    pages_check(table, ring, state, old, new, 64, 0, codes={layer.SHAPE})
    pages_check(table, ring, state, old, new, 64, n // 2, status0=77)  # a status word in use is kept


def test_pages_bad_lengths():
    table, ring, state, old, new = pages_case(50, 64, 8, 9, 90)
    old[3], new[7], new[20], old[49], old[12], new[12] = -1, -2 ** 31, 64 * 8 + 1, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1
    n = int((new - old).clamp(min=0, max=1000).sum())
    pages_check(table, ring, state, old, new, 64, n + 5, codes={layer.SEQLEN})


@pytest.mark.parametrize("state", [[-1, 5], [0, -1], [10 ** 6, 5], [0, 10 ** 6], [2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, 0]])
def test_pages_bad_state(state):
    table, ring, _, old, new = pages_case(50, 64, 8, 10, 90)
    pages_check(table, ring, state, old, new, 64, 5000, codes={layer.PAGE})


def test_pages_bad_entries():
    """Ids outside the pool, in the ring and in the table: entered as -1, their tokens without a slot, nothing faults."""
    table, ring, state, old, new = pages_case(60, 64, 8, 11, 150)
    ring[state[0]], ring[(state[0] + 3) % len(ring)] = 10 ** 9, -7
    grows = [b for b in range(60) if new[b] > old[b] and old[b] % 64]
    table[grows[0], old[grows[0]] // 64] = len(ring)
    n = int((new - old).clamp(min=0).sum())
    pages_check(table, ring, state, old, new, 64, n, codes={layer.PAGE})


def test_pages_more_given_back_than_the_ring_holds():
    """A table that claims more pages than the pool has (a broken caller): the ring never grows past the pool."""
    ring = torch.arange(10)
    table = torch.arange(40).view(4, 10) % 10
    pages_check(table, ring, [4, 8], torch.tensor([640, 640, 10, 640]), torch.tensor([0, 64, 64, 0]), 64, 60,
                codes={layer.PAGE})


def test_pages_empty_batch():
    pages = mla.Pages(torch.empty(0, 4, dtype=I32, device=DEV), torch.arange(6, dtype=I32, device=DEV), 64)
    empty = torch.empty(0, dtype=I32, device=DEV)
    out = mla.pages_update(pages, torch.tensor([5, 6], dtype=I32, device=DEV), empty, empty.clone(), 3)
    assert out.token_start.tolist() == [0] and out.ring_state.tolist() == [5, 6]
    assert out.positions.tolist() == [-1] * 3 and out.slots.tolist() == [-1] * 3


# ------------------------------------------------------------------------------------------------------------ store
def store_reference(x, weight, eps, at, freq, half, mscale, d_c):
    c = layer.rms_norm(x[:, :d_c], weight, eps)
    k = x[:, d_c:].double()
    if freq is not None:
        k = layer.rotate(x[:, d_c:], at, freq, half, mscale)
    return torch.cat((c, k), 1)


def store_tolerance(want, x, weight, at, freq, half, mscale, d_c, scale=None):
    """fp32 before the rounding: 22 additions deep a mean square, then root, quotient and two products, 2^-19 of a value;
    the key as in rope_tolerance."""
    tol = want.abs() * 2.0 ** -19
    if weight is None:
        tol[:, :d_c] = 0.0
    tol[:, d_c:] = 0.0
    if freq is not None:
        zero = torch.zeros_like(want[:, d_c:])
        tol[:, d_c:] = rope_tolerance(x[:, d_c:], at, freq, half, mscale, zero)
    if scale is None:
        return tol * 1.01 + want.abs() * 2.0 ** -8
    return tol * 1.01 + (want.abs() * (2.0 ** -4 + 2.0 ** -22)).clamp(min=scale * 2.0 ** -10)


STORE_CASES = [
    # B, s_q, d_c, d_rope, page, fp8 scale, norm, half, rotate, slots, lead
    (1, 1, 64, 0, 64, None, True, False, False, True, 0),
    (3, 2, 512, 64, 64, None, True, False, True, True, 0),
    (5, 1, 512, 64, 64, None, True, True, True, False, 8),
    (65, 3, 512, 64, 128, 1 / 16, True, False, True, True, 1024),
    (7, 4, 320, 48, 64, 0.0371, True, True, True, False, 24),
    (130, 1, 448, 16, 0, None, False, False, True, False, 0),
    (9, 5, 128, 32, 0, 0.01, False, False, False, False, 200),
    (4, 1, 64, 16, 192, None, False, True, True, True, 0),
]


@pytest.mark.parametrize("B,s_q,d_c,d_rope,ps,scale,norm,half,turned,with_slots,lead", STORE_CASES)
def test_latent_store(B, s_q, d_c, d_rope, ps, scale, norm, half, turned, with_slots, lead):
    g = gen(B * s_q + d_c)
    T, W = B * s_q, d_c + d_rope
    rows = randn(g, T, lead + W)
    rows[:, lead] *= 8.0
    x = rows[:, lead:]
    weight = (1 + 0.3 * torch.randn(d_c, generator=g)).to(BF16) if norm else None
    lens = torch.randint(s_q, 500, (B,), generator=g, dtype=I32)
    cap = 512
    dt = BF16 if scale is None else torch.uint8
    if ps:
        n_pages = cap // ps + (cap % ps > 0)
        pool = B * n_pages + 3
        table = torch.randperm(pool, generator=g)[:B * n_pages].view(B, n_pages).to(I32)
        kv = torch.randint(0, 100, (pool, ps, W), generator=g).to(dt)
        slot = torch.stack([table[b, j // ps] * ps + j % ps for b in range(B) for j in range(int(lens[b]) - s_q, int(lens[b]))])
        rows_at = slot.long()
    else:
        table = None
        kv = torch.randint(0, 100, (B, cap, W), generator=g).to(dt)
        rows_at = torch.tensor([b * cap + j for b in range(B) for j in range(int(lens[b]) - s_q, int(lens[b]))])
    prob = problem(B, 16, s_q, d_c=d_c, d_rope=d_rope)
    at = (lens.long()[:, None] - s_q + torch.arange(s_q)).flatten()
    kw, pos = {}, {}
    if with_slots:
        kw["slots"] = slot.to(I32).to(DEV)
        at = torch.randint(0, 2 ** 31 - 1, (T,), generator=g)  # positions of their own go with slots
        kw["positions"] = at.to(I32).to(DEV)
    plan = mla.rope_plan(d_rope, layout=mla.ROPE_HALF if half else mla.ROPE_INTERLEAVED, mscale=1.125) if turned else None
    freq = layer.frequencies(d_rope) if turned else None
    lens_d, table_d, kv_d = lens.to(DEV), None if table is None else table.to(DEV), kv.to(DEV)
    status = torch.zeros(1, dtype=I32, device=DEV)
    cache = mla.make_cache(prob, kv_d, lens_d, table_d, ps or 64, kv_scale=scale)
    mla.latent_store(prob, rows.to(DEV)[:, lead:], cache, plan=plan, norm_weight=None if weight is None else weight.to(DEV),
                     eps=1e-5, status=status, **kw)
    assert int(status) == 0
    want = store_reference(x, weight, 1e-5, at, freq, half, 1.125, d_c)
    tol = store_tolerance(want, x, weight, at, freq, half, 1.125, d_c, scale)
    got = kv_d.cpu().view(-1, W)
    new = got[rows_at]
    if scale is not None:
        new = new.view(torch.float8_e4m3fn).double() * float(torch.tensor(scale))
        want = want.clamp(-448 * scale, 448 * scale)
    close(new, want, tol)
    other = torch.ones(got.shape[0], dtype=torch.bool)
    other[rows_at] = False
    assert torch.equal(got[other], kv.view(-1, W)[other]), "rows of no token are left as they were"


@pytest.mark.parametrize("fp8", [False, True])
def test_latent_store_skips_and_flags(fp8):
    g = gen(21)
    T, d_c, d_rope, ps, pages = 12, 128, 32, 64, 4
    W = d_c + d_rope
    x = randn(g, T, W)
    kv = torch.zeros(pages, ps, W, dtype=torch.uint8 if fp8 else BF16)
    prob = problem(T, 16, 1, d_c=d_c, d_rope=d_rope)
    lens, table = torch.ones(T, dtype=I32), torch.zeros(T, 1, dtype=I32)
    slots = torch.arange(T, dtype=I32) * 9
    slots[2], slots[5], slots[6], slots[7] = -1, pages * ps, 2 ** 31 - 1, -2 ** 31
    at = torch.arange(T, dtype=I32)
    at[9] = -1
    written = torch.tensor([i for i in range(T) if i not in (2, 5, 6, 7, 9)])
    lens_d, table_d, kv_d, status = lens.to(DEV), table.to(DEV), kv.to(DEV), torch.zeros(1, dtype=I32, device=DEV)
    cache = mla.make_cache(prob, kv_d, lens_d, table_d, ps, kv_scale=1.0)
    mla.latent_store(prob, x.to(DEV), cache, plan=mla.rope_plan(d_rope), norm_weight=torch.ones(d_c, dtype=BF16, device=DEV),
                     positions=at.to(DEV), slots=slots.to(DEV), status=status)
    assert int(status) == layer.PAGE
    touched = (kv_d.cpu().view(-1, W).float().abs().sum(1) > 0).nonzero().flatten()
    assert torch.equal(touched, slots[written].long())
    # by the lengths: too short, too long, a page outside the pool; the word keeps the first error
    lens = torch.tensor([0, 65, -3, 64] + [1] * 8, dtype=I32)
    table[4], table[5] = -1, pages
    table[6:, 0] = 3
    lens[6:] = torch.arange(6, dtype=I32) + 10
    kv_d.zero_()
    lens_d, table_d = lens.to(DEV), table.to(DEV)
    for slot_kw in ({}, dict(slots=slots.to(DEV))):  # with slots, the lengths give the positions
        kv_d.zero_()
        status.zero_()
        cache = mla.make_cache(prob, kv_d, lens_d, table_d, ps, kv_scale=1.0)
        mla.latent_store(prob, x.to(DEV), cache, plan=mla.rope_plan(d_rope), status=status, **slot_kw)
        assert int(status) in (layer.SEQLEN, layer.PAGE)
        touched = (kv_d.cpu().view(-1, W).float().abs().sum(1) > 0).nonzero().flatten().tolist()
        if slot_kw:
            assert touched == sorted(int(slots[i]) for i in (3, 4, 8, 9, 10, 11))
        else:
            assert touched == [63] + [3 * 64 + 9 + i for i in range(6)]


def test_latent_store_special_values():
    """Infinities and NaN stay in their token; zeros and the smallest values with eps."""
    d_c, d_rope = 64, 16
    x = torch.zeros(4, d_c + d_rope, dtype=BF16)
    x[1, 3], x[1, d_c] = float("nan"), float("inf")
    x[2, :d_c] = 1e-30
    x[3, :] = 1e30
    prob = problem(4, 16, 1, d_c=d_c, d_rope=d_rope)
    for fp8 in (False, True):
        kv = torch.zeros(1, 64, d_c + d_rope, dtype=torch.uint8 if fp8 else BF16, device=DEV)
        lens, table = torch.ones(4, dtype=I32, device=DEV), torch.zeros(4, 1, dtype=I32, device=DEV)
        cache = mla.make_cache(prob, kv, lens, table, 64, kv_scale=1.0)
        mla.latent_store(prob, x.to(DEV), cache, norm_weight=torch.ones(d_c, dtype=BF16, device=DEV), eps=1e-6,
                         slots=torch.arange(4, dtype=I32, device=DEV))
        got = (kv.view(torch.float8_e4m3fn) if fp8 else kv).cpu().float()[0, :4]
        assert bool((got[0] == 0).all())
        assert bool(torch.isnan(got[1, :d_c]).all())
        assert float(got[1, d_c]) == (448.0 if fp8 else math.inf) and bool((got[1, d_c + 1:] == 0).all())
        assert bool((got[2, :d_c].abs() <= 1e-20).all())
        # 1e30 squared passes fp32: the mean is infinite and the row is 0, as the formula in fp32 gives it
        assert bool((got[3, :d_c] == 0).all()) and float(got[3, d_c]) == (448.0 if fp8 else float(x[3, 0]))


def test_latent_store_fp8_smallest_scale():
    """kv_scale 2^-126, whose inverse is 2^126, with weights that times it pass fp32: zeros stay zeros (a row of them, and
    beside other values), what is not zero saturates with its sign, and values of the scale's own size are held as such."""
    d_c, d_rope = 64, 16
    x = torch.zeros(3, d_c + d_rope, dtype=BF16)
    x[1, :4] = torch.tensor([1.0, -2.0, 0.0, 0.5])
    x[2, :4] = torch.tensor([2.0 ** -126, -3 * 2.0 ** -126, 0.0, 2.0 ** -125])
    x[:, d_c:d_c + 2] = torch.tensor([2.0 ** -124, -1.0])
    weight = torch.full((d_c,), 4.0)
    weight[1], weight[5] = 1e30, -8.0
    want = torch.zeros(3, d_c + d_rope)
    want[:, d_c:d_c + 2] = torch.tensor([4.0, -448.0])
    prob = problem(3, 16, 1, d_c=d_c, d_rope=d_rope)
    lens, table = torch.ones(3, dtype=I32, device=DEV), torch.zeros(3, 1, dtype=I32, device=DEV)
    for norm in (weight.to(BF16).to(DEV), None):
        kv = torch.full((1, 64, d_c + d_rope), 0x55, dtype=torch.uint8, device=DEV)
        cache = mla.make_cache(prob, kv, lens, table, 64, kv_scale=2.0 ** -126)
        mla.latent_store(prob, x.to(DEV), cache, norm_weight=norm, eps=1e-6, slots=torch.arange(3, dtype=I32, device=DEV))
        got = kv.view(torch.float8_e4m3fn).cpu().float()[0, :3]
        want[1, :4] = torch.tensor([448.0, -448.0, 0.0, 448.0])
        # without a norm the row's own values; with one they are 1000 times that (1 / sqrt(eps)) and their weight
        want[2, :4] = torch.tensor([1.0, -3.0, 0.0, 2.0]) if norm is None else torch.tensor([448.0, -448.0, 0.0, 448.0])
        assert torch.equal(got, want)


# ----------------------------------------------------------------------------------------------------------- linear
LINEAR_CASES = [
    # M, K, N, bias, act, residual, paddings of x, out and residual rows
    (1, 8, 8, False, "none", False, 0, 0, 0), (1, 64, 128, True, "relu", True, 8, 8, 8), (2, 72, 136, True, "silu", False, 0, 16, 0),
    (15, 1000, 264, False, "gelu", True, 24, 0, 8), (16, 4096, 128, True, "gelu_tanh", True, 0, 0, 0),
    (17, 128, 1544, False, "none", True, 0, 8, 0), (32, 192, 64, True, "none", False, 0, 0, 0),
    (33, 520, 2056, True, "gelu", True, 8, 8, 8), (64, 16384, 256, False, "none", True, 0, 0, 0),
    (65, 264, 392, True, "silu", True, 0, 0, 0), (127, 2048, 1000, False, "relu", False, 0, 0, 64),
    (128, 64, 8, True, "gelu_tanh", True, 0, 0, 0), (129, 1000, 136, True, "none", True, 8, 0, 0),
    (256, 128, 4096, False, "none", False, 0, 0, 0), (333, 1000, 1544, True, "gelu_tanh", True, 8, 8, 8),
    (1025, 72, 520, True, "silu", True, 0, 24, 0), (4096, 512, 2048, False, "none", True, 0, 0, 0),
    (5000, 136, 1160, True, "gelu", True, 0, 0, 0),
    # pairs of CTAs: several rounds of tiles, the last ones cut by every edge; one round
    (5000, 1032, 6000, True, "silu", True, 8, 8, 8), (700, 2056, 6024, False, "none", True, 0, 0, 0),
    # clusters of two and of four pairs share K
    (250, 8200, 7000, True, "gelu_tanh", True, 0, 8, 8), (1264, 6792, 416, False, "none", True, 8, 0, 0),
    # tiles over a little more than a wave: whole, and cut into runs
    (8, 1000, 20480, True, "relu", True, 0, 8, 0), (8, 4104, 20480, True, "silu", True, 8, 8, 0), (150, 2048, 19464, False, "none", True, 0, 0, 0),
]


def strided(t, pad, fill=None):
    """t's values in rows that are `pad` wider (CPU tensor)."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), 3.0 if fill is None else fill, dtype=t.dtype)
    wide[:, :t.shape[1]] = t
    return wide


@pytest.mark.parametrize("M,K,N,bias,act,residual,px,po,pr", LINEAR_CASES)
def test_linear(M, K, N, bias, act, residual, px, po, pr):
    """Once with small whole numbers, whose sums are exact in fp32, so that only the epilogue rounds (bit-equal without
    an activation), and once with normal values: fp32 accumulation of K terms is off by at most K 2^-23 of the terms'
    absolute sum, the activations stretch that by at most 1.13 and add 2^-17 of their value, and the result rounds once."""
    for exact in (True, False):
        g = gen(M + K + N)
        if exact:
            x = torch.randint(-4, 5, (M, K), generator=g).to(BF16)
            w = torch.randint(-4, 5, (K, N), generator=g).to(BF16)
        else:
            x, w = randn(g, M, K), randn(g, K, N, std=K ** -0.5)
        b = randn(g, N) if bias else None
        r = randn(g, M, N, std=2.0) if residual else None
        out = strided(torch.full((M, N), 5.0, dtype=BF16), po, 9.0).to(DEV)
        got = mla.linear(strided(x, px).to(DEV)[:, :K], w.to(DEV), bias=None if b is None else b.to(DEV),
                         residual=None if r is None else strided(r, pr).to(DEV)[:, :N], act=ACTS[act], out=out[:, :N])
        assert bool((out[:, N:] == 9).all()), "columns behind N are left as they were"
        want = layer.linear(x, w, b, r, act)
        if exact and act in ("none", "relu"):
            full = (x.float().double() @ w.double()).float()  # exact
            if b is not None:
                full = full + b.float()
            full = full.clamp(min=0) if act == "relu" else full
            if r is not None:
                full = full + r.float()
            assert torch.equal(got.cpu(), full.to(BF16))
            continue
        terms = x.double().abs() @ w.double().abs()
        pre = layer.linear(x, w, b, None, act)
        tol = 1.13 * (0.0 if exact else 1.0) * K * 2.0 ** -23 * terms + pre.abs() * 2.0 ** -17 + 2.0 ** -22
        close(got, want, tol + want.abs() * 2.0 ** -8 * 1.01)


def test_linear_in_place_on_the_residual_stream():
    g = gen(31)
    for M, K, N in ((3, 4096, 264), (300, 64, 520), (4096, 128, 1536)):
        x, w, r = randn(g, M, K), randn(g, K, N, std=K ** -0.5), randn(g, M, N)
        rd = r.to(DEV)
        apart = mla.linear(x.to(DEV), w.to(DEV), residual=rd)
        mla.linear(x.to(DEV), w.to(DEV), residual=rd, out=rd)
        assert torch.equal(rd, apart)


def test_linear_repeats_bit_for_bit_with_a_dirty_workspace():
    g = gen(32)
    for M, K, N in ((64, 16384, 1024), (333, 1000, 1544), (1, 8192, 264), (8, 4104, 20480)):
        x, w = randn(g, M, K).to(DEV), randn(g, K, N, std=K ** -0.5).to(DEV)
        ws = torch.full((mla.linear_workspace_size(M, K, N),), 0xFF, dtype=torch.uint8, device=DEV)
        a = mla.linear(x, w, workspace=ws)
        for _ in range(3):
            assert torch.equal(mla.linear(x, w, workspace=ws), a)


def test_linear_special_values():
    """An infinite or NaN input stays in its row (of x) or column (of w); columns and rows behind the ends, which the
    tiles read as zeros, bring nothing in."""
    g = gen(33)
    M, K, N = 20, 72, 136
    x, w = randn(g, M, K), randn(g, K, N)
    x[3, 5], x[7, 71], w[70, 9] = float("inf"), float("nan"), float("inf")
    got = mla.linear(strided(x, 8, float("nan")).to(DEV)[:, :K], w.to(DEV)).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[3], bad[7], bad[:, 9] = True, True, True
    assert torch.equal(~torch.isfinite(got), bad | ~torch.isfinite(layer.linear(x, w)))
    assert torch.equal(torch.isnan(got), torch.isnan(layer.linear(x, w)))


def test_linear_no_rows():
    out = mla.linear(torch.empty(0, 64, dtype=BF16, device=DEV), torch.zeros(64, 128, dtype=BF16, device=DEV))
    assert out.shape == (0, 128)


# --------------------------------------------------------------------------------------------- argument checks in python
def test_wrappers_refuse():
    prob, plan = problem(2, 4, 1, d_rope=32), mla.rope_plan(32)
    x = torch.zeros(2, 1, 4, 32, dtype=BF16, device=DEV)
    lens = torch.ones(2, dtype=I32, device=DEV)
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(x=x[:, :, :, :16]), dict(x=x[:1]), dict(seq_lens=lens.long()),
                dict(seq_lens=lens[:1]), dict(seq_lens=lens.cpu()), dict(q_rope=x.float()), dict(q_nope=x)):
        with pytest.raises(ValueError):
            mla.rope(prob, plan, **{"x": x, "seq_lens": lens, **bad})
    a = torch.zeros(4, 64, dtype=BF16, device=DEV)
    w = torch.zeros(64, 128, dtype=BF16, device=DEV)
    for bad in (dict(x=a.float()), dict(w=w.t()), dict(w=w[:32]), dict(bias=w[0, :64]), dict(residual=w[:4, :64]),
                dict(out=w[:3]), dict(x=w.t()[:4, :64])):
        with pytest.raises(ValueError):
            mla.linear(**{"x": a, "w": w, **bad})
    with pytest.raises(mla.MLAError):
        mla.linear(a, w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


# ------------------------------------------------------------------------------------------------------------ together
class Layer:
    """One MLA layer's step on a paged cache from these operators and the attention, x = x + attention(x) . W_O."""

    def __init__(self, B, H, d_model, d_c, d_rope, d_nope, d_v, ps, max_pages, seed, fp8=False):
        g = gen(seed)
        self.B, self.H, self.d_model, self.ps = B, H, d_model, ps
        self.dims = dict(d_c=d_c, d_rope=d_rope, d_nope=d_nope, d_v=d_v)
        self.w_q = randn(g, d_model, H * (d_nope + d_rope), std=d_model ** -0.5)
        self.w_kv = randn(g, d_model, d_c + d_rope, std=d_model ** -0.5)
        self.w_norm = (1 + 0.1 * torch.randn(d_c, generator=g)).to(BF16)
        self.w_uk, self.w_uv = randn(g, H, d_c, d_nope, std=d_c ** -0.5), randn(g, H, d_c, d_v, std=d_c ** -0.5)
        self.w_o = randn(g, H * d_v, d_model, std=(H * d_v) ** -0.5)
        self.dev = {k: v.to(DEV) for k, v in vars(self).items() if torch.is_tensor(v)}
        self.plan = mla.rope_plan(d_rope, base=10000.0)
        self.freq = layer.frequencies(d_rope)
        self.pages, self.state = mla.Pages.empty(B, max_pages, B * max_pages, ps)
        self.kv_scale = 1 / 16 if fp8 else None
        self.kv = torch.zeros(B * max_pages, ps, d_c + d_rope, dtype=torch.uint8 if fp8 else BF16, device=DEV)
        self.lens = torch.zeros(B, dtype=I32, device=DEV)
        self.history = [torch.empty(0, d_c + d_rope, dtype=torch.float64) for _ in range(B)]

    def problem(self, s_q):
        return mla.Problem(self.B, self.H, s_q, scale=(self.dims["d_nope"] + self.dims["d_rope"]) ** -0.5, **self.dims)

    def step(self, x, new_lens, status):
        """x [B * s_q, d_model]: every request grows by s_q tokens."""
        s_q = x.shape[0] // self.B
        prob, w = self.problem(s_q), self.dev
        up = mla.pages_update(self.pages, self.state, self.lens, new_lens, x.shape[0], status=status)
        q = mla.linear(x, w["w_q"]).view(self.B, s_q, self.H, -1)
        q_nope, q_rope = mla.rope(prob, self.plan, q, positions=up.positions)
        cache = mla.make_cache(prob, self.kv, up.seq_lens, self.pages.block_table, self.ps, kv_scale=self.kv_scale)
        mla.latent_store(prob, mla.linear(x, w["w_kv"]), cache, plan=self.plan, norm_weight=w["w_norm"],
                         positions=up.positions, slots=up.slots, status=status)
        q_cat = mla.absorb_q(prob, q_nope, q_rope, w["w_uk"])
        o_lat, _, ws = mla.decode_attn(prob, q_cat, cache)
        out = mla.out_proj(prob, o_lat, w["w_uv"])
        y = mla.linear(out.view(x.shape[0], -1), w["w_o"], residual=x)
        self.keep = (up, q, q_nope, q_rope, cache, q_cat, o_lat, ws, out)
        self.state, self.lens = up.ring_state, up.seq_lens
        return y

    def reference(self, x):
        """The same step in 64 bits on its own history of rows."""
        s_q, D = x.shape[0] // self.B, self.dims
        x = x.double()
        q = (x @ self.w_q.double()).view(self.B, s_q, self.H, -1)
        kv = x @ self.w_kv.double()
        c = layer.rms_norm(kv[:, :D["d_c"]], self.w_norm, 1e-6).view(self.B, s_q, -1)
        k = kv[:, D["d_c"]:].view(self.B, s_q, -1)
        outs = torch.empty(self.B, s_q, self.H * D["d_v"], dtype=torch.float64)
        for b in range(self.B):
            n = self.history[b].shape[0]
            at = n + torch.arange(s_q)
            rows = torch.cat((c[b], layer.rotate(k[b], at, self.freq, False)), 1)
            self.history[b] = torch.cat((self.history[b], rows))
            qr = layer.rotate(q[b, :, :, D["d_nope"]:], at[:, None], self.freq, False)
            qa = torch.einsum("ihn,hcn->ihc", q[b, :, :, :D["d_nope"]], self.w_uk.double())
            s = torch.einsum("ihc,jc->ihj", torch.cat((qa, qr), 2), self.history[b]) * (D["d_nope"] + D["d_rope"]) ** -0.5
            s = s.masked_fill(torch.arange(n + s_q)[None, None, :] > at[:, None, None], -math.inf)
            o = torch.einsum("ihj,jc->ihc", torch.softmax(s, -1), self.history[b][:, :D["d_c"]])
            outs[b] = torch.einsum("ihc,hcv->ihv", o, self.w_uv.double()).flatten(1)
        return x + outs.view(x.shape[0], -1) @ self.w_o.double()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,d_c,d_rope,d_nope,d_v", [(16, 64, 16, 32, 32), (128, 512, 64, 128, 128)])
def test_a_layer_step_after_step(H, d_c, d_rope, d_nope, d_v, fp8):
    """Prompt, decode, verification and decode steps of one layer on a growing paged cache, each against the step in 64
    bits on the same inputs (the tolerance of the end-to-end attention tests; FP8 rows carry 2^-4 of rounding, which the
    softmax averages and the residual dwarfs)."""
    L = Layer(3, H, 512, d_c, d_rope, d_nope, d_v, 64, 4, 41, fp8)
    g = gen(42)
    status = torch.zeros(1, dtype=I32, device=DEV)
    lens = 0
    for s_q in (60, 1, 3, 1, 130 if d_c == 64 else 65, 1):
        lens += s_q
        x = randn(g, 3 * s_q, 512)
        y = L.step(x.to(DEV), torch.full((3,), lens, dtype=I32, device=DEV), status)
        assert int(status) == 0 and mla.read_status(L.keep[7]) == 0
        within_tolerance(y, L.reference(x), f"step of {s_q} tokens", rel=2e-2 if not fp8 else 4e-2)
        assert L.lens.tolist() == [lens] * 3


def test_a_decode_step_captured_and_replayed():
    """One graph of the whole step (fixed buffers, the state flipped by copies), replayed over several tokens, against
    the same steps run eagerly, bit for bit; a second graph on its own layer replays between them."""
    def make(seed):
        L = Layer(2, 16, 256, 64, 16, 32, 32, 64, 3, seed)
        status = torch.zeros(1, dtype=I32, device=DEV)
        x = randn(gen(seed), 2 * 62, 256).to(DEV)
        L.step(x, torch.full((2,), 62, dtype=I32, device=DEV), status)
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
        L.buffers = (lens, state, new)  # the graph's own: they live as long as it
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
            want = eager.step(x, eager.lens + 1, st)
            assert torch.equal(ys, want), i
    assert int(sa) == 0 and int(sb) == 0
    assert torch.equal(a.kv, ea.kv) and torch.equal(b.pages.block_table, eb.pages.block_table)


def test_calls_on_two_streams_at_once():
    """Calls with buffers of their own on two streams, many in flight, give what they give alone."""
    g = gen(61)
    x, w = randn(g, 64, 4096).to(DEV), randn(g, 4096, 520, std=1 / 64).to(DEV)
    x2, w2 = randn(g, 200, 512).to(DEV), randn(g, 512, 1032, std=1 / 23).to(DEV)
    table, ring, state, old, new = pages_case(500, 64, 8, 62, 90)
    n = int((new - old).clamp(min=0).sum())
    dev = lambda t: torch.as_tensor(t).to(I32).to(DEV)  # noqa: E731
    pages = mla.Pages(dev(table), dev(ring), 64)
    st, o, nw = dev(state), dev(old), dev(new)
    alone = mla.linear(x, w), mla.linear(x2, w2), mla.pages_update(pages, st, o, nw, n)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        with torch.cuda.stream(s1):
            outs.append((0, mla.linear(x, w)))
            outs.append((2, mla.pages_update(pages, st, o, nw, n)))
        with torch.cuda.stream(s2):
            outs.append((1, mla.linear(x2, w2)))
    torch.cuda.synchronize()
    for k, got in outs:
        if k < 2:
            assert torch.equal(got, alone[k])
        else:
            assert torch.equal(got.slots, alone[2].slots) and torch.equal(got.ring_state, alone[2].ring_state)


# ------------------------------------------------------------------------------------- sizes at the ends of the ranges
def test_offsets_past_32_bits():
    """Rows whose element offsets pass 2^32: the last tokens of a rotation, the last slots of a pool, the last rows of a
    product, each against the same call on those rows alone (whose results the other tests check)."""
    torch.manual_seed(91)
    # rotation: 100,000 tokens x 128 heads x 192 = 2.46e9 values in, as many out
    T, H = 100000, 128
    x = torch.empty(1, T, H, 192, dtype=BF16, device=DEV)
    x[0, :3] = torch.randn(3, H, 192, device=DEV)
    x[0, -3:] = torch.randn(3, H, 192, device=DEV)
    plan = mla.rope_plan(64)
    at = torch.arange(T, dtype=I32, device=DEV)
    nope, turned = mla.rope(problem(1, H, T), plan, x, positions=at)
    for rows in (slice(0, 3), slice(T - 3, T)):
        n1, t1 = mla.rope(problem(1, H, 3), plan, x[:, rows], positions=at[rows].contiguous())
        assert torch.equal(nope[:, rows], n1) and torch.equal(turned[:, rows], t1)
    del x, nope, turned
    # store: 150,000 pages of 64 rows of 576 values
    pages, W = 150000, 576
    kv = torch.empty(pages, 64, W, dtype=BF16, device=DEV)
    kv[0].zero_()
    kv[-2:].zero_()
    rows = torch.randn(4, W, device=DEV).to(BF16)
    slots = torch.tensor([pages * 64 - 1, 5, pages * 64 - 65, pages * 64 - 64], dtype=I32, device=DEV)
    lens, table = torch.ones(4, dtype=I32, device=DEV), torch.zeros(4, 1, dtype=I32, device=DEV)
    prob = problem(4, 16, 1)
    kw = dict(plan=plan, positions=torch.arange(4, dtype=I32, device=DEV), norm_weight=torch.ones(512, dtype=BF16, device=DEV))
    mla.latent_store(prob, rows, mla.make_cache(prob, kv, lens, table, 64), slots=slots, **kw)
    small = torch.zeros(1, 64, W, dtype=BF16, device=DEV)
    mla.latent_store(prob, rows, mla.make_cache(prob, small, lens, table, 64), slots=torch.arange(4, dtype=I32, device=DEV), **kw)
    flat = kv.view(-1, W)
    assert torch.equal(flat[slots.long()], small[0, :4])
    around = torch.cat((flat[:64], flat[-128:])).float().abs().sum(1)
    assert int((around > 0).sum()) == 4
    del kv, flat, around
    # product: 140,000 x 32,768 outputs = 4.6e9
    M, K, N = 140000, 64, 32768
    x, w = torch.randn(M, K, device=DEV).to(BF16), torch.randn(K, N, device=DEV).to(BF16)
    y = mla.linear(x, w)
    for rows in (slice(0, 300), slice(M - 300, M)):
        assert torch.equal(y[rows], mla.linear(x[rows], w))


@pytest.mark.parametrize("M,K,N", [(1, 1 << 20, 8), (1, 8, 1 << 20), (65535 * 128, 8, 8), (2, 64, 8 * 131071)])
def test_linear_longest_sides(M, K, N):
    """Whole numbers, so that every sum is exact: the ends of each size's range."""
    g = torch.Generator(device=DEV).manual_seed(M + K)
    x = torch.randint(-1, 2, (M, K), generator=g, device=DEV).to(BF16)
    w = torch.randint(-1, 2, (K, N), generator=g, device=DEV).to(BF16)
    want = (x.double() @ w.double()).to(torch.float32).to(BF16)
    assert torch.equal(mla.linear(x, w), want)


def test_most_tokens_of_rope_and_store():
    """65535 sequences of 128 tokens, the most a call takes, padding among them."""
    B, s_q = 65535, 128
    prob = problem(B, 1, s_q, d_c=64, d_rope=16, d_nope=16)
    plan = mla.rope_plan(16, layout=mla.ROPE_HALF)
    g = torch.Generator(device=DEV).manual_seed(71)
    x = torch.randn(B, s_q, 1, 16, generator=g, device=DEV).to(BF16)
    at = torch.randint(-3, 1000, (B, s_q), generator=g, device=DEV).to(I32)
    out = torch.full_like(x, 9.0)
    mla.rope(prob, plan, x, positions=at, q_rope=out)
    assert bool((out[at < 0] == 9).all())
    pick = torch.randint(0, B * s_q, (2000,), generator=g, device=DEV)
    pick = torch.cat((pick, torch.tensor([0, B * s_q - 1], device=DEV)))
    pick = pick[at.flatten()[pick] >= 0]
    few = x.view(-1, 16)[pick]
    want = layer.rotate(few.cpu(), at.flatten()[pick].cpu().long(), layer.frequencies(16), True)
    close(out.view(-1, 16)[pick], want,
          rope_tolerance(few.cpu(), at.flatten()[pick].cpu().long(), layer.frequencies(16), True, 1.0, want))
    rows = torch.randn(B * s_q, 80, generator=g, device=DEV).to(BF16)
    kv = torch.zeros(B * s_q // 64, 64, 80, dtype=BF16, device=DEV)
    slots = torch.randperm(B * s_q, generator=g, device=DEV).to(I32)
    lens, table = torch.full((B,), s_q, dtype=I32, device=DEV), torch.zeros(B, 2, dtype=I32, device=DEV)
    mla.latent_store(prob, rows, mla.make_cache(prob, kv, lens, table, 64), slots=slots)  # neither norm nor rotation: a copy
    assert torch.equal(kv.view(-1, 80)[slots.long()], rows)


def test_one_workspace_in_two_graphs():
    """Two captured products share a workspace: replayed one after another on a stream, each gives its own result."""
    g = gen(81)
    M, K, N = 8, 4104, 20480  # cut along K, its pieces in the workspace
    w = randn(g, K, N, std=K ** -0.5).to(DEV)
    xs = [randn(g, M, K).to(DEV) for _ in range(2)]
    ws = torch.empty(mla.linear_workspace_size(M, K, N), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 256
    want = [mla.linear(x, w) for x in xs]
    graphs, outs = [], []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(mla.linear(x, w, workspace=ws))
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], want[i])


# ------------------------------------------------------------------------------------------------- a stream as an argument
def test_stream_argument_while_the_current_stream_allocates():
    """linear(stream=s) of a shape that is cut into runs, held up on s, while the current stream takes and fills buffers
    of the workspace's and of the output's size: neither side writes into the other's memory."""
    g = gen(101)
    M, K, N = 8, 4104, 20480
    x, w = randn(g, M, K).to(DEV), randn(g, K, N, std=K ** -0.5).to(DEV)
    nbytes = mla.linear_workspace_size(M, K, N)
    assert nbytes > 256
    want = mla.linear(x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = [mla.linear(x, w, stream=s) for _ in range(3)]
        taken = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for n in (nbytes, nbytes, 2 * M * N)]
        for _ in range(20):
            for t in taken:
                t.fill_(0x7F)
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for y in got)
        assert all(bool((t == 0x7F).all()) for t in taken)
        del got, taken


def test_tensors_made_for_a_stream_belong_to_it():
    """Outputs that rope, pages_update and linear make under stream= come from that stream's memory."""
    s = torch.cuda.Stream()
    prob, plan = problem(2, 4, 1, d_rope=32, d_nope=64), mla.rope_plan(32)
    q = torch.zeros(2, 1, 4, 96, dtype=BF16, device=DEV)
    lens = torch.ones(2, dtype=I32, device=DEV)
    pages, state = mla.Pages.empty(2, 4, 8)
    x, w = torch.zeros(4, 64, dtype=BF16, device=DEV), torch.zeros(64, 128, dtype=BF16, device=DEV)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    made = [*mla.rope(prob, plan, q, seq_lens=lens, stream=s), mla.linear(x, w, stream=s)]
    up = mla.pages_update(pages, state, lens, lens + 1, 2, stream=s)
    made += [up.seq_lens, up.ring_state, up.token_start, up.positions, up.slots]
    torch.cuda.synchronize()
    segments = torch.cuda.memory_snapshot()
    for t in made:
        at = [seg for seg in segments if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]]
        assert len(at) == 1 and at[0]["stream"] == s.cuda_stream


# ------------------------------------------------------------------------------------------------------ more refusals
def test_linear_refuses_a_workspace_it_cannot_use():
    """On the host or strided it is refused before anything is launched; its size counts in bytes, whatever its type."""
    g = gen(111)
    M, K, N = 8, 4104, 20480
    x, w = randn(g, M, K).to(DEV), randn(g, K, N, std=K ** -0.5).to(DEV)
    need = mla.linear_workspace_size(M, K, N)
    for bad in (torch.empty(need, dtype=torch.uint8), torch.empty(2 * need, dtype=torch.uint8, device=DEV)[::2],
                torch.empty(2, need, dtype=torch.uint8, device=DEV).t()):
        with pytest.raises(ValueError):
            mla.linear(x, w, workspace=bad)
    words = torch.empty((need + 3) // 4, dtype=torch.float32, device=DEV)
    assert torch.equal(mla.linear(x, w, workspace=words), mla.linear(x, w))
    with pytest.raises(mla.MLAError):
        mla.linear(x, w, workspace=words[:-64])


# -------------------------------------------------------------------------------------------- waits that run out
TIMEOUT_CASES = [
    # M, K, N: whole tiles, clusters, runs, pairs in several rounds, clusters of two and of four pairs
    (333, 1000, 1544), (64, 16384, 1024), (3, 65536, 136), (8, 4104, 20480), (5000, 1032, 6000), (250, 8200, 7000),
    (1264, 6792, 416), (2000, 16384, 256),
]


@pytest.mark.parametrize("M,K,N", TIMEOUT_CASES)
def test_linear_wait_timeout_reported_and_recovered(M, K, N):
    """With a short bound on the waits for work, some of them run out, at once or on the way: the call ends, the status
    word says so, every output is NaN or what it should be (whole numbers: exact sums), and calls after it are clean."""
    g = gen(M + K + N + 7)
    x, w = (torch.randint(-3, 4, n, generator=g).to(BF16).to(DEV) for n in ((M, K), (K, N)))
    status = torch.zeros(1, dtype=I32, device=DEV)
    want = mla.linear(x, w, status=status)
    assert int(status) == 0
    assert torch.equal(want, (x.float().double() @ w.float().double()).float().to(BF16))
    seen = []
    try:
        for ns in (1, 1, 300, 1000, 3000, 4000, 5000, 6500, 8000, 10000):
            mla.set_wait_limit_ns(ns)
            status.zero_()
            out = torch.full((M, N), 7.25, dtype=BF16, device=DEV)  # no sum of whole numbers
            mla.linear(x, w, out=out, status=status)
            torch.cuda.synchronize()
            bad = torch.isnan(out)
            assert torch.equal(out[~bad], want[~bad]), ns
            assert int(status) in (0, 8) and (int(status) == 8 or not bool(bad.any())), ns
            seen.append((int(status), int(bad.sum())))
    finally:
        mla.set_wait_limit_ns(0)
    print(seen)
    assert (8 in [c for c, _ in seen]) and any(n for _, n in seen), seen  # MLA_ERR_TIMEOUT
    for _ in range(2):
        status.zero_()
        assert torch.equal(mla.linear(x, w, status=status), want) and int(status) == 0


# ----------------------------------------------------------------------------------------- activations over their range
def exact_activation(act, v):
    """In 64 bits without cancellation: v Phi(v) by erfc, the others by the logistic function of z."""
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2))
    z = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    e = torch.exp(-z.abs())
    return torch.where(z < 0, v * e, v) / (1 + e)


@pytest.mark.parametrize("act,least", [("silu", -94.0), ("gelu", -13.75), ("gelu_tanh", -10.5)])
def test_linear_activations_to_the_end_of_bf16(act, least):
    """One non-zero weight of 1, so that the activation gets x itself, from where its result leaves bf16 to 14.  A result
    rounds once, half a step of 2^-8 of it (2^-134 among the subnormals) beside 2^-16 for the activation in fp32 (an
    exponent near -126 rounds to 2^-18, ln 2 of which is 2^-18.5, three times; tanh's cube twice that).  With the rounded
    result taken off again by the residual, what is left is that error in fp32 and half a step of a remainder that is
    itself at most half a step: 2^-16 twice."""
    v = torch.cat((torch.linspace(least, 0, 6000), torch.linspace(0, 14, 3000), -torch.logspace(-30, 1, 3000))).to(BF16)
    v = torch.unique(v.float()).to(BF16)
    M, N = v.numel(), 8
    x, w = torch.zeros(M, 8, dtype=BF16), torch.zeros(8, N, dtype=BF16)
    x[:, 3], w[3] = v, 1.0
    want = exact_activation(act, v.double())[:, None].expand(M, N)
    got = mla.linear(x.to(DEV), w.to(DEV), act=ACTS[act])
    close(got, want, want.abs() * (2.0 ** -8 + 2.0 ** -16) + 2.0 ** -134)
    tail = (want.abs() > 2.0 ** -126) & (want < 0)
    assert bool((got.cpu()[tail] < 0).all()) and int(tail.sum()) > 1000
    taken = -want.to(BF16)
    left = mla.linear(x.to(DEV), w.to(DEV), act=ACTS[act], residual=taken.contiguous().to(DEV))
    close(left, want + taken.double(), want.abs() * 2.0 ** -15 + 2.0 ** -133)


# ------------------------------------------------------------------------------------------------- every form of a product
@pytest.mark.parametrize("form", LINEAR_FORMS, ids=lambda f: "x".join(map(str, f)))
def test_linear_every_form(form):
    """Each way a product is cut, with ends inside tiles: small whole numbers, whose sums are exact in fp32, so that only
    the epilogue rounds and the result is bit-equal; rows in wider ones, bias and residual; and again, bit for bit."""
    M, K, N = LINEAR_FORMS[form]
    cut = mla.linear_cut(M, K, N)
    assert (cut.tile_rows, cut.tile_columns, cut.k_parts, cut.runs) == form
    g = torch.Generator(device=DEV).manual_seed(sum(form) + M)
    x = torch.randint(-4, 5, (M, K + 8), generator=g, device=DEV).to(BF16)[:, :K]
    w = torch.randint(-4, 5, (K, N), generator=g, device=DEV).to(BF16)
    b, r = torch.randn(N, generator=g, device=DEV).to(BF16), torch.randn(M, N + 16, generator=g, device=DEV).to(BF16)[:, :N]
    full = (x.double() @ w.double()).float()  # exact
    status = torch.zeros(1, dtype=I32, device=DEV)
    assert torch.equal(mla.linear(x, w, status=status), full.to(BF16))
    out = torch.full((M, N + 8), 9.0, dtype=BF16, device=DEV)
    for _ in range(2):
        mla.linear(x, w, bias=b, residual=r, act=mla.ACT_RELU, out=out[:, :N], status=status)
        assert torch.equal(out[:, :N], ((full + b.float()).clamp(min=0) + r.float()).to(BF16))
        assert bool((out[:, N:] == 9).all())
    stream = r.clone(memory_format=torch.contiguous_format)  # in place on the residual
    mla.linear(x, w, bias=b, residual=stream, act=mla.ACT_RELU, out=stream, status=status)
    assert torch.equal(stream, out[:, :N]) and int(status) == 0


def test_calls_from_several_threads():
    """Four threads, each on a stream of its own given as an argument, through one Problem, plan and set of weights: every
    result is what the call gives alone."""
    g = gen(121)
    prob, plan = problem(6, 16, 2, d_c=128, d_rope=32, d_nope=64), mla.rope_plan(32)
    q, at = randn(g, 6, 2, 16, 96).to(DEV), torch.arange(12, dtype=I32, device=DEV).view(6, 2)
    x, w = randn(g, 8, 4104).to(DEV), randn(g, 4104, 20480, std=1 / 64).to(DEV)
    x2, w2 = randn(g, 300, 520).to(DEV), randn(g, 520, 1032, std=1 / 23).to(DEV)
    rows, norm = randn(g, 12, 160).to(DEV), randn(g, 128).to(DEV)
    lens, table = torch.full((6,), 40, dtype=I32, device=DEV), torch.arange(6, dtype=I32, device=DEV).view(6, 1)
    slots = (torch.arange(12, dtype=I32, device=DEV) * 29).contiguous()

    def calls(stream):
        with torch.cuda.stream(stream):
            kv = torch.zeros(6, 64, 160, dtype=BF16, device=DEV)
            pages, state = mla.Pages.empty(6, 4, 24)
            old = torch.zeros(6, dtype=I32, device=DEV)
            torch.cuda.current_stream().synchronize()
        prob.scale = prob.scale  # fields set and structures made at the same time
        n, r = mla.rope(prob, plan, q, positions=at, stream=stream)
        y, y2 = mla.linear(x, w, stream=stream), mla.linear(x2, w2, act=mla.ACT_GELU, stream=stream)
        mla.latent_store(prob, rows, mla.make_cache(prob, kv, lens, table, 64), plan=plan, norm_weight=norm, positions=at,
                         slots=slots, stream=stream)
        up = mla.pages_update(pages, state, old, lens, 240, stream=stream)
        return n, r, y, y2, kv, up.slots, up.positions, up.ring_state, pages.block_table

    alone = calls(torch.cuda.Stream())
    torch.cuda.synchronize()
    wrong = []

    def work():
        try:
            s = torch.cuda.Stream()
            kept = [calls(s) for _ in range(15)]
            s.synchronize()
            wrong.extend(k for got in kept for k, (a, b) in enumerate(zip(got, alone)) if not torch.equal(a, b))
        except Exception as e:  # noqa: BLE001 - shown by the assertion below
            wrong.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
