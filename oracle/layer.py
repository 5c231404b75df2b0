"""Plain 64-bit implementations of the operators around the attention, from their definitions: rotary positions, page
tables, the latent store, the matrix product with its epilogue, and values in blocks of 128 with a scale each.  Test
infrastructure only."""
from __future__ import annotations

import math

import torch


def frequencies(d: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0, original_len: int = 0,
                beta_fast: float = 32.0, beta_slow: float = 1.0) -> list[float]:
    """Radians a position of each of the d / 2 pairs."""
    if scaling == "ntk":
        base = base * factor ** (d / (d - 2))
    f = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if scaling == "linear":
        f = [v / factor for v in f]
    if scaling == "yarn":
        def index(turns):
            return d * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))
        low, high = max(math.floor(index(beta_fast)), 0), min(math.ceil(index(beta_slow)), d - 1)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(d // 2)]
        f = [v / factor * r + v * (1 - r) for v, r in zip(f, ramp)]
    return f


def pairs(d: int, half: bool):
    i = torch.arange(d // 2)
    return (i, i + d // 2) if half else (2 * i, 2 * i + 1)


def rotate(x: torch.Tensor, positions: torch.Tensor, freq: list[float], half: bool, mscale: float = 1.0,
           transpose: bool = False) -> torch.Tensor:
    """x [..., d] turned by positions (broadcast against x's leading dimensions) * freq; differentiable."""
    angle = positions.to(torch.float64)[..., None] * torch.tensor(freq, dtype=torch.float64)
    c, s = mscale * torch.cos(angle), mscale * torch.sin(angle) * (-1.0 if transpose else 1.0)
    p, q = pairs(x.shape[-1], half)
    u, v = x.double()[..., p], x.double()[..., q]
    out = torch.empty(torch.broadcast_shapes(x.shape, angle.shape[:-1] + x.shape[-1:]), dtype=torch.float64)
    out[..., p] = u * c - v * s
    out[..., q] = u * s + v * c
    return out


def rms_norm(c: torch.Tensor, weight, eps: float) -> torch.Tensor:
    c = c.double()
    if weight is None:
        return c
    return c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps) * weight.double()


def act(name: str, v: torch.Tensor) -> torch.Tensor:
    if name == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return v * torch.special.ndtr(v)
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def linear(x, w, bias=None, residual=None, name: str = "none") -> torch.Tensor:
    y = x.double() @ w.double()
    if bias is not None:
        y = y + bias.double()
    y = act(name, y)
    return y if residual is None else y + residual.double()


def spread(scales: torch.Tensor, rows: int, M: int, K: int) -> torch.Tensor:
    """Scales of blocks of rows x 128 as one a value."""
    return scales.double().repeat_interleave(rows, 0)[:M].repeat_interleave(128, 1)[:, :K]


def blocks(y: torch.Tensor, rows: int = 1):
    """The quotients that are rounded to codes (their largest 448 in a block) and the scales [M / rows, K / 128]; a NaN
    is left out of its block's scale."""
    y = y.double()
    M, K = y.shape
    scales = torch.empty(-(-M // rows), -(-K // 128), dtype=torch.float64)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            part = y[rows * i:rows * i + rows, 128 * j:128 * j + 128].abs()
            part = part[~torch.isnan(part)]
            scales[i, j] = max(float(part.max()) if part.numel() else 0.0, 2.0 ** -100) / 448
    return y / spread(scales, rows, M, K), scales


def linear_fp8(x, x_scale, w, w_scale, bias=None, residual=None, name: str = "none") -> torch.Tensor:
    """x [M, K], w [N, K] codes, x_scale [K / 128, M], w_scale [N / 128, K / 128]."""
    (M, K), N = x.shape, w.shape[0]
    xv = x.double() * spread(x_scale.t(), 1, M, K)
    return linear(xv, (w.double() * spread(w_scale, 128, N, K)).t(), bias, residual, name)


SEQLEN, PAGE, SHAPE = 3, 9, 2


def pages_update(table, ring, state, old, new, page_size: int, max_tokens: int):
    """One request after another on lists of ints; returns the new (table, ring, state, seq_lens, token_start,
    positions, slots) and the set of status codes that arose."""
    table, ring = [list(r) for r in table], list(ring)
    P, most = len(ring), (len(table[0]) * page_size if table else 0)
    head, count = state
    codes = set()
    state_ok = 0 <= head < P and 0 <= count <= P
    if not state_ok:
        codes.add(PAGE)
    lens, start, positions, slots = [], [0], [-1] * max_tokens, [-1] * max_tokens
    asked = taken = given = tokens = 0
    out_ring = list(ring)
    for b, (o, n) in enumerate(zip(old, new)):
        if not (0 <= o <= most and 0 <= n <= most):
            codes.add(SEQLEN)
            lens.append(o)
            start.append(tokens)
            continue
        had, has = -(-o // page_size), -(-n // page_size)
        grow, need, back = max(n - o, 0), max(has - had, 0), max(had - has, 0)
        first, tokens = tokens, tokens + grow
        asked += need
        start.append(min(tokens, 2 ** 31 - 1))
        short = need > 0 and state_ok and asked > count
        late = grow > 0 and tokens > max_tokens
        if short or late or (not state_ok and (need or back)):
            codes.add(SHAPE if late and not short and state_ok else PAGE)
            lens.append(o)
            continue
        lens.append(n)
        for k in range(need):
            page = ring[(head + taken) % P]
            taken += 1
            if not 0 <= page < P:
                codes.add(PAGE)
                page = -1
            table[b][had + k] = page
        for k in range(back):
            if count + given < P:
                out_ring[(head + count + given) % P] = table[b][has + k]
                given += 1
            else:
                codes.add(PAGE)
        for k in range(grow):
            page = table[b][(o + k) // page_size]
            positions[first + k] = o + k
            if 0 <= page < P:
                slots[first + k] = page * page_size + (o + k) % page_size
            else:
                codes.add(PAGE)
    new_state = [(head + taken) % P, count - taken + given] if state_ok else [head, count]
    return table, out_ring, new_state, lens, start, positions, slots, codes
