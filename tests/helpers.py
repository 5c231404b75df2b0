"""Shared helpers of the test suite: run the CUDA path, compare with the oracle."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from mla_decode_attention_absorbed_gb300 import mla
from mla_decode_attention_absorbed_gb300.workloads import MLAConfig, make_inputs

# Spec tolerance per output tensor: max|gpu - ref| <= 2e-2 * max|ref| + 1e-3
REL_TOL = 2e-2
ABS_TOL = 1e-3


def within_tolerance(gpu: torch.Tensor, ref: torch.Tensor, what: str = "", rel=REL_TOL, abs_=ABS_TOL):
    g = gpu.detach().to("cpu", torch.float64)
    r = ref.detach().to("cpu", torch.float64)
    assert g.shape == r.shape, (what, g.shape, r.shape)
    fin = torch.isfinite(r)
    assert torch.equal(torch.isfinite(g), fin), f"{what}: non-finite values differ"
    if fin.sum() == 0:
        return 0.0
    err = (g[fin] - r[fin]).abs().max().item()
    bound = rel * r[fin].abs().max().item() + abs_
    assert err <= bound, f"{what}: max|gpu-ref| = {err:.3e} > {bound:.3e}"
    return err / max(bound, 1e-30)


# lse is an fp32 output of the normaliser: besides the per-tensor bound above it must
# agree with the oracle to 1e-2 nats everywhere (the relative bound alone would allow
# about 0.2 nats at lse ~ 9)
LSE_ABS_TOL = 1e-2


def lse_close(gpu: torch.Tensor, ref: torch.Tensor, what: str = "lse"):
    within_tolerance(gpu, ref, what)
    g = gpu.detach().to("cpu", torch.float64)
    r = ref.detach().to("cpu", torch.float64)
    fin = torch.isfinite(r)
    if fin.any():
        err = (g[fin] - r[fin]).abs().max().item()
        assert err <= LSE_ABS_TOL, f"{what}: max|gpu-ref| = {err:.3e} nats > {LSE_ABS_TOL}"


def to_dev(inp: dict, device="cuda") -> dict:
    out = {}
    for k, v in inp.items():
        out[k] = v.to(device) if isinstance(v, torch.Tensor) else v
    return out


def gpu_cache(cfg: MLAConfig, d: dict, max_seq_len=0):
    prob = mla.Problem.of(cfg)
    cache = mla.make_cache(prob, d["kv"], d["seq_lens"], d["block_table"], cfg.page_size, max_seq_len)
    return prob, cache


def run_gpu(cfg: MLAConfig, inp: dict, num_splits: int = 0, max_seq_len: int = 0):
    """absorb_q -> decode_attn -> out_proj on the GPU; returns CPU tensors and the status word."""
    d = to_dev(inp)
    prob, cache = gpu_cache(cfg, d, max_seq_len)
    q_cat = mla.absorb_q(prob, d["q_nope"], d["q_rope"], d["w_uk"])
    o_lat, lse, ws = mla.decode_attn(prob, q_cat, cache, num_splits=num_splits)
    out = mla.out_proj(prob, o_lat, d["w_uv"])
    status = mla.read_status(ws)
    torch.cuda.synchronize()
    return dict(q_cat=q_cat.cpu(), o_lat=o_lat.cpu(), lse=lse.cpu(), out=out.cpu(), status=status)


def oracle_args(cfg, inp):
    return (inp["q_nope"], inp["q_rope"], inp["kv"], inp["seq_lens"], inp["w_uk"], inp["w_uv"])


def check_against_oracle(cfg: MLAConfig, inp: dict, g: dict, rows=None):
    """Stage-isolated and end-to-end comparison (all rows, or the listed flat rows)."""
    ref_q = oracle.absorb_q(cfg, inp["q_nope"], inp["q_rope"], inp["w_uk"])
    within_tolerance(g["q_cat"], ref_q, "q_cat")
    # attention from the GPU's own q_cat (stage-isolated)
    o_ref, lse_ref = oracle.attend(cfg, g["q_cat"], inp["kv"], inp["seq_lens"], inp["block_table"],
                                   cfg.page_size, rows=rows)
    sel = slice(None) if rows is None else torch.as_tensor(np.asarray(rows, dtype=np.int64))
    within_tolerance(g["o_lat"].view(-1, cfg.d_c)[sel], o_ref.view(-1, cfg.d_c)[sel], "o_lat")
    lse_close(g["lse"].view(-1)[sel], lse_ref.view(-1)[sel], "lse")
    # projection from the GPU's own o_lat (stage-isolated)
    out_ref = oracle.out_proj(cfg, g["o_lat"], inp["w_uv"])
    within_tolerance(g["out"].view(-1, cfg.d_v)[sel], out_ref.view(-1, cfg.d_v)[sel], "out (stage)")
    # end to end from the inputs in fp64
    e2e = oracle.decode(cfg, *oracle_args(cfg, inp), block_table=inp["block_table"], page_size=cfg.page_size,
                        rows=rows)
    within_tolerance(g["out"].view(-1, cfg.d_v)[sel], e2e["out"].view(-1, cfg.d_v)[sel], "out (end to end)")
    lse_close(g["lse"].view(-1)[sel], e2e["lse"].view(-1)[sel], "lse (end to end)")


def sample_rows(cfg: MLAConfig, n: int, seed: int = 1):
    """n flat rows spread over sequences, query positions and heads, always
    including the first and the last row."""
    total = cfg.B * cfg.s_q * cfg.H
    g = np.random.default_rng(seed)
    rows = set(g.choice(total, size=min(n, total), replace=False).tolist())
    rows |= {0, total - 1}
    return sorted(rows)


# A product for every way mla_linear cuts one on a GPU of 152 SMs, (rows a tile, columns a tile, parts of K, runs) to
# (M, K, N), each with rows, K and columns that end inside a tile.
LINEAR_FORMS = {
    (16, 128, 1, 0): (3, 136, 136), (16, 128, 2, 0): (3, 456, 4680), (16, 128, 4, 0): (3, 456, 136),
    (16, 128, 8, 0): (3, 976, 136), (16, 128, 1, 1): (3, 1520, 19856),
    (32, 128, 1, 0): (1256, 136, 136), (32, 128, 2, 0): (619, 840, 136), (32, 128, 4, 0): (293, 648, 136),
    (32, 128, 8, 0): (114, 1288, 136), (32, 128, 1, 1): (17, 2016, 19512),
    (64, 128, 1, 0): (2460, 136, 136), (64, 128, 2, 0): (1241, 1352, 136), (64, 128, 4, 0): (43, 16320, 3224),
    (64, 128, 8, 0): (293, 2888, 136), (64, 128, 1, 1): (141, 17712, 944),
    (128, 128, 1, 0): (5178, 328, 136), (128, 128, 2, 0): (323, 2544, 1952), (128, 128, 4, 0): (1241, 2792, 144),
    (128, 128, 8, 0): (583, 5624, 136), (128, 128, 1, 1): (794, 18704, 1400),
    (256, 128, 1, 0): (565, 480, 12816), (256, 128, 2, 0): (1001, 14000, 2368), (256, 128, 4, 0): (1276, 12360, 880),
    (256, 128, 8, 0): (1237, 14288, 136), (256, 128, 1, 1): (2869, 13720, 864),
    (256, 256, 1, 0): (5234, 904, 392), (256, 256, 2, 0): (3310, 4648, 280), (256, 256, 4, 0): (1604, 5968, 272),
}

# The same of mla_linear_fp8, (rows a tile, columns a tile, parts of K, rounds of whole tiles: 0, 1 or 2 for more) to (M, K, N).
LINEAR_FP8_FORMS = {
    (128, 64, 1, 1): (3, 208, 136), (128, 64, 2, 0): (2, 2512, 4704), (128, 64, 4, 0): (5, 1728, 72),
    (128, 64, 4, 1): (2, 12480, 9952), (128, 64, 8, 0): (121, 1968, 136), (128, 128, 1, 1): (3, 208, 10328),
    (128, 128, 1, 2): (3, 208, 20552), (128, 128, 2, 0): (2, 4272, 4904), (128, 128, 2, 1): (3, 1520, 23480),
    (128, 128, 4, 0): (2, 1936, 2352), (128, 128, 4, 1): (2, 912, 20568), (128, 128, 8, 0): (2, 2016, 968),
    (256, 192, 1, 1): (135, 208, 10840), (256, 192, 1, 2): (1039, 4544, 4904), (256, 192, 2, 0): (140, 7536, 5032),
    (256, 192, 2, 1): (145, 4304, 20296), (256, 192, 4, 0): (135, 8144, 2472),
    (256, 256, 1, 1): (137, 208, 16408), (256, 256, 1, 2): (515, 208, 12760), (256, 256, 2, 0): (262, 10896, 3768),
    (256, 256, 2, 1): (5799, 4432, 1784), (256, 256, 4, 0): (397, 18272, 1352),
}


def linear_fp8_form(M: int, K: int, N: int):
    """The form that mla_linear_fp8 takes for a product."""
    c = mla.linear_fp8_cut(M, K, N)
    tiles = -(-M // c.tile_rows) * -(-N // c.tile_columns)
    units = c.ctas // (2 if c.tile_rows == 256 else 1)
    if c.k_parts == 1:
        return c.tile_rows, c.tile_columns, 1, 1 if tiles <= units else 2
    return c.tile_rows, c.tile_columns, c.k_parts, 0 if units == tiles * c.k_parts else 1
