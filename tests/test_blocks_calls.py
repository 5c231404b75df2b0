"""What the Python calls of the 8-bit operators take and refuse, where nothing is launched.  No GPU needed."""
import pytest
import torch

from mla_decode_attention_absorbed_gb300 import mla


@pytest.mark.parametrize("paged", [False, True])
def test_rows_of_blocks_take_no_scale(paged):
    """Their width alone tells them from codes with one scale: a scale beside them is one or the other gone wrong."""
    prob = mla.Problem(2, 16, 1, 128, 32, 64, 64, 1.0)
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1, dtype=torch.int32) if paged else None
    rows = torch.zeros(2, 64, 128 + 16 + 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="kv_scale"):
        mla.make_cache(prob, rows, lens, table, kv_scale=0.5)
    assert mla.make_cache(prob, rows, lens, table).kv_dtype == mla.KV_E4M3_BLOCKS
    assert mla.make_cache(prob, rows[:, :, :160].contiguous(), lens, table, kv_scale=0.5).kv_dtype == mla.KV_E4M3


class OnDevice:
    """A CPU tensor that says it lies on device 0."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return 0


def test_linear_fp8_takes_the_scales_of_some_rows(monkeypatch):
    """The rows [a, b) of quantised values and their scales, a slice of each, without a copy."""
    seen = []

    class Library:
        def mla_linear_fp8(self, desc, x, x_scale, *rest):
            seen.append((desc._obj.M, x, desc._obj.x_stride, x_scale, desc._obj.x_scale_stride))
            return 0

    monkeypatch.setattr(mla, "_lib", Library())
    monkeypatch.setattr(mla, "_current_device", lambda: 0)
    monkeypatch.setattr(mla, "_raw_stream", lambda dev, stream: 0)
    x, scales = torch.zeros(40, 272).to(torch.float8_e4m3fn), torch.zeros(3, 40)
    w, w_scale = OnDevice(torch.zeros(136, 272).to(torch.float8_e4m3fn)), OnDevice(torch.zeros(2, 3))
    for a, b in ((0, 40), (8, 24), (39, 40), (5, 5)):
        out = OnDevice(torch.zeros(b - a, 136, dtype=torch.bfloat16))
        mla.linear_fp8(OnDevice(x[a:b]), OnDevice(scales[:, a:b]), w, w_scale, out=out)
        M, at, _, scale_at, stride = seen.pop()
        assert M == b - a
        if M:
            assert at == x.data_ptr() + 272 * a and scale_at == scales.data_ptr() + 4 * a and stride == 40
    for bad in (scales.t().contiguous().t(), scales[:2], scales[:, :39], scales.double(), scales[:, ::2].repeat(1, 2)[:, ::2]):
        with pytest.raises(ValueError):
            mla.linear_fp8(OnDevice(x), OnDevice(bad), w, w_scale, out=OnDevice(torch.zeros(40, 136, dtype=torch.bfloat16)))
    assert not seen


def test_whole_operands_sum_exactly():
    """The products compared bit for bit: their codes' products are whole and their scales' at least 2^-4, so every sum is exact in fp32
    while the absolute terms come to less than 2^24 times 2^-4.  16 x 16 a term holds that up to K = 4096; beyond, by the
    data."""
    from helpers import LINEAR_FP8_FORMS
    from test_gpu_blocks import PRODUCT_CASES, gen, operands
    sizes = [(M, K, N, 1) for M, K, N in LINEAR_FP8_FORMS.values()] + [(*case[:3], 0) for case in PRODUCT_CASES]
    long = [s for s in sizes if s[1] > 4096]
    assert long
    for M, K, N, seed in long:
        x, xs, w, ws = operands(gen(M + K + N + seed), M, K, N, True)
        xv = x.float().abs() * xs.t().repeat_interleave(128, 1)[:, :K]
        wv = w.float().abs() * ws.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        assert float((xv @ wv.t()).max()) * 2.0 ** 4 < 2.0 ** 24 * 0.99, (M, K, N)
