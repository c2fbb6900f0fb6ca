"""The scaled product on scales and outputs that start at any byte their type
allows, and on row counts of every kernel: the bits of the aligned call."""
import numpy as np
import pytest

import routing_grouped_expert_amd as moe
from gpu_util import dev, note, sync, torch
from test_gpu_mx import mx_inputs

pytestmark = pytest.mark.gpu


def shifted(a, by):
    """The same values `by` elements into an allocation, and none behind them."""
    t = torch()
    d = dev(a)
    buf = t.full((d.numel() + by,), 0xFF if d.dtype == t.uint8 else 0, dtype=d.dtype, device="cuda:0")
    v = buf[by:].view(d.shape)
    v.copy_(d)
    return v


@pytest.mark.parametrize("xbits", [4, 8])
@pytest.mark.parametrize("K,M", [(32, 24), (96, 40), (288, 264), (512, 31), (1184, 16)])
@pytest.mark.parametrize("counts", [[7, 0, 32], [50, 64], [100, 128, 3], [300, 20, 90, 40]])
def test_scales_and_outputs_anywhere(K, M, counts, xbits):
    t = torch()
    off, xc, xs, wc, ws, rows, n, N, T = mx_inputs(counts, 2, K, M, xbits, 1, True, K + M)
    g = [dev(a) for a in (off, xc, wc, rows)]
    ref = {}
    for f32 in (False, True):
        kind = t.float32 if f32 else t.bfloat16
        for by in (0, 1, 2, 3, 5):
            y = t.zeros(N * M + by, dtype=kind, device="cuda:0")[by:].view(N, M)
            note(f"anywhere K={K} M={M} {counts} xbits={xbits} f32={f32} by={by}")
            moe.grouped_matmul_mx(g[1], shifted(xs, by), g[0], g[2], shifted(ws, by), y,
                                  permuted_rows=g[3], k=1)
            sync()
            got = y.double().cpu().numpy()
            assert np.array_equal(got, ref.setdefault(f32, got)), (f32, by)
    assert np.any(ref[True])


@pytest.mark.parametrize("bits", [4, 8])
def test_quantised_scales_anywhere(bits):
    t = torch()
    rng = np.random.default_rng(bits)
    x = dev(rng.standard_normal((9, 160)).astype(np.float32))
    gu = dev(rng.standard_normal((9, 320)).astype(np.float32))
    ref = []
    for by in (0, 1, 2, 3):
        out = []
        for f in (moe.quantize_mx, moe.swiglu_quantize_mx):
            c = t.zeros((9, 160 * bits // 8), dtype=t.uint8, device="cuda:0")
            s = t.zeros(45 + by, dtype=t.uint8, device="cuda:0")[by:].view(9, 5)
            f(x if f is moe.quantize_mx else gu, c, s)
            o = t.zeros((9, 160), dtype=t.float32, device="cuda:0")
            moe.dequantize_mx(c, s, o)
            out += [a.cpu().numpy() for a in (c, s, o)]
        sync()
        ref = ref or out
        assert all(np.array_equal(a, b) for a, b in zip(ref, out)), by
