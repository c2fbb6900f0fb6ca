"""What the operators around the layer refuse, on the host: the library's
status codes (nothing launched) and the binding's checks."""
import ctypes

import pytest

import routing_grouped_expert_amd as moe
from test_abi import _FakeGpuTensor as F

P = ctypes.c_void_p(0x1000)    # never dereferenced
ODD = ctypes.c_void_p(0x1008)  # not 16-byte aligned
OK, BAD, LIMIT, WS = 0, 1, 2, 3
BIG = 1 << 20


def gm(x=P, rows=P, off=P, L=4, T=8, k=2, N=16, K=64, M=32, w=P, y=P):
    return moe.lib().moe_grouped_matmul(x, rows, off, L, T, k, N, K, M, w, y, 0, None)


def dx(dy=P, off=P, L=4, N=16, K=64, M=32, w=P, out=P):
    return moe.lib().moe_grouped_matmul_dx(dy, off, L, N, K, M, w, out, 0, None)


def dw(dy=P, x=P, rows=P, off=P, L=4, T=8, k=2, N=16, K=64, M=32, out=P):
    return moe.lib().moe_grouped_matmul_dw(dy, x, rows, off, L, T, k, N, K, M, out, 0, None)


def mx(xq=P, xs=P, bits=8, rows=P, off=P, L=4, T=8, k=2, N=16, K=64, M=32, wq=P, ws=P, y=P):
    return moe.lib().moe_grouped_matmul_mx(xq, xs, bits, rows, off, L, T, k, N, K, M, wq, ws, y, 0,
                                           None)


def norm(x=P, res=P, w=P, eps=1e-6, T=4, H=64, h=P, y=P, q=P, s=P):
    return moe.lib().moe_rms_norm(x, res, w, eps, T, H, h, y, q, s, None)


def norm_bwd(dy=P, h=P, w=P, eps=1e-6, T=4, H=64, dres=P, out=P, dg=P, ws=P, n=1 << 20):
    return moe.lib().moe_rms_norm_backward(dy, h, w, eps, T, H, dres, out, dg, ws, n, None)


def quant(x=P, R=4, K=64, bits=4, c=P, s=P):
    return moe.lib().moe_quantize_mx(x, 0, R, K, bits, c, s, None)


def swiglu(x=P, N=4, I=64, rows=None, bits=4, c=P, s=P):
    return moe.lib().moe_swiglu_quantize_mx(x, 0, N, I, rows, bits, c, s, None)


def dequant(c=P, s=P, R=4, K=64, bits=4, out=P):
    return moe.lib().moe_dequantize_mx(c, s, R, K, bits, out, 0, None)


CASES = [
    # negative, zero and missing arguments
    *[(f, d, BAD) for f in (gm, mx) for d in (
        dict(L=-1), dict(T=-1), dict(N=-1), dict(k=0), dict(K=0), dict(M=0), dict(off=None),
        dict(y=None), dict(rows=None), dict(rows=None, k=1, N=9))],
    (gm, dict(x=None), BAD), (gm, dict(w=None), BAD),
    (mx, dict(xq=None), BAD), (mx, dict(xs=None), BAD), (mx, dict(wq=None), BAD),
    (mx, dict(ws=None), BAD), (mx, dict(bits=6), BAD),
    *[(dx, d, BAD) for d in (dict(L=-1), dict(N=-1), dict(K=0), dict(M=0), dict(dy=None),
                             dict(off=None), dict(w=None), dict(out=None))],
    *[(dw, d, BAD) for d in (dict(L=-1), dict(N=-1), dict(dy=None), dict(x=None), dict(off=None),
                             dict(out=None), dict(rows=None))],
    *[(norm, d, BAD) for d in (dict(T=-1), dict(H=0), dict(eps=-1.0), dict(eps=float("nan")),
                               dict(x=None), dict(w=None), dict(q=None), dict(s=None),
                               dict(h=None, y=None, q=None, s=None))],
    *[(norm_bwd, d, BAD) for d in (dict(T=-1), dict(H=0), dict(eps=-1.0), dict(dy=None),
                                   dict(h=None), dict(w=None), dict(out=None), dict(dg=None))],
    *[(f, d, BAD) for f in (quant, dequant, swiglu) for d in (dict(bits=5), dict(c=None),
                                                              dict(s=None))],
    (quant, dict(R=-1), BAD), (quant, dict(x=None), BAD), (dequant, dict(out=None), BAD),
    (swiglu, dict(N=-1), BAD), (swiglu, dict(x=None), BAD),
    # limits
    *[(f, d, LIMIT) for f in (gm, mx) for d in (
        dict(L=4097), dict(k=33), dict(K=BIG + 32), dict(M=BIG + 1), dict(T=1 << 30, k=2),
        dict(T=1 << 25, K=64), dict(N=1 << 26, M=32), dict(K=1 << 16, M=1 << 15))],
    (dx, dict(L=4097), LIMIT), (dx, dict(K=BIG + 1), LIMIT), (dx, dict(N=1 << 25), LIMIT),
    (dw, dict(L=4097), LIMIT), (dw, dict(M=BIG + 1), LIMIT),
    (norm, dict(T=1 << 25), LIMIT), (norm, dict(H=48), LIMIT), (norm_bwd, dict(T=1 << 25), LIMIT),
    (mx, dict(K=48), LIMIT), (mx, dict(xq=ODD), LIMIT), (mx, dict(wq=ODD), LIMIT),
    (quant, dict(K=33), LIMIT), (quant, dict(x=ODD), LIMIT), (quant, dict(c=ODD), LIMIT),
    (swiglu, dict(I=40), LIMIT), (swiglu, dict(x=ODD), LIMIT), (dequant, dict(out=ODD), LIMIT),
    (quant, dict(R=1 << 29, K=32), LIMIT),
    # workspace
    (norm_bwd, dict(ws=None), WS), (norm_bwd, dict(n=4 * 64 * 4 - 1), WS),
    (norm_bwd, dict(ws=ctypes.c_void_p(0x1010)), WS),
    # nothing to do
    *[(f, dict(N=0), OK) for f in (gm, mx)], *[(f, dict(L=0), OK) for f in (gm, mx, dx, dw)],
    (dx, dict(N=0), OK), (norm, dict(T=0), OK), (quant, dict(R=0), OK), (dequant, dict(R=0), OK),
    (swiglu, dict(N=0), OK),
]


@pytest.mark.parametrize("f,kw,status", CASES)
def test_status(f, kw, status):
    assert f(**kw) == status


def test_backward_workspace_size():
    assert moe.rms_norm_backward_workspace_size(0, 64) == 0
    a, b = (moe.rms_norm_backward_workspace_size(t, 4096) for t in (1, 1 << 16))
    assert a == 4096 * 4 and a < b <= 4096 * 4 * 1024 and b % 256 == 0
    for bad in ((-1, 64), (4, 0)):
        with pytest.raises(moe.MoeError) as e:
            moe.rms_norm_backward_workspace_size(*bad)
        assert e.value.status == 1


def test_binding_refuses_before_calling():
    T, K, M, L, k, N = 8, 64, 32, 4, 2, 16
    b = dict(esize=2)
    x, w, y, off, rows = F((T, K), **b), F((L, M, K), **b), F((N, M), **b), F((L + 1,)), F((N,))
    q, s, wq, ws = F((T, K), 1), F((T, K // 32), 1), F((L, M, K // 2), 1), F((L, M, K // 32), 1)
    cases = [
        lambda: moe.grouped_matmul(F((T, K), 2, cuda=False), off, w, y, rows, k),
        lambda: moe.grouped_matmul(F((T, K), 2, contiguous=False), off, w, y, rows, k),
        lambda: moe.grouped_matmul(F((T, K), 4), off, w, y, rows, k),
        lambda: moe.grouped_matmul(x, off, F((L + 1, M, K), 2), y, rows, k),
        lambda: moe.grouped_matmul(x, off, w, F((N, M), 1), rows, k),
        lambda: moe.grouped_matmul(x, off, w, y, F((N + 1,)), k),
        lambda: moe.grouped_matmul(x, off, w, y),                      # T != N, no rows
        lambda: moe.grouped_matmul(F((N, K), 2), off, w, y, None, 2),  # k without rows
        lambda: moe.grouped_matmul_dx(F((N + 1, M), 2), off, w, F((N, K), 2)),
        lambda: moe.grouped_matmul_dx(F((N, M), 2), off, F((L, K, M), 2), F((N, K), 2)),
        lambda: moe.grouped_matmul_dw(F((N, M), 4), x, off, F((L, M, K), 2), rows, k),
        lambda: moe.grouped_matmul_dw(F((N, M), 2), x, off, F((L, K, M), 2), rows, k),
        lambda: moe.grouped_matmul_mx(q, F((T, 3), 1), off, wq, ws, y, rows, k),
        lambda: moe.grouped_matmul_mx(F((T, K - 1), 1), s, off, wq, ws, y, rows, k),
        lambda: moe.grouped_matmul_mx(q, s, off, wq, F((L, M, 3), 1), y, rows, k),
        lambda: moe.rms_norm(x, F((K + 1,)), 1e-6, y=F((T, K), 2)),
        lambda: moe.rms_norm(x, F((K,), 2), 1e-6, y=F((T, K), 2)),
        lambda: moe.rms_norm(x, F((K,)), 1e-6, y=F((T, K), 4)),
        lambda: moe.rms_norm(x, F((K,)), 1e-6, yq=q, ys=F((T, 3), 1)),
        lambda: moe.rms_norm_backward(x, x, F((K,)), 1e-6, F((T, K), 4), F((K,)), None),
        lambda: moe.rms_norm_backward(x, x, F((K,)), 1e-6, x, F((K,), 2), None),
        lambda: moe.quantize_mx(x, F((T, K // 4), 1), s),
        lambda: moe.quantize_mx(F((T, K), 1), q, s),
        lambda: moe.quantize_mx(x, q, F((T, 1), 1)),
        lambda: moe.swiglu_quantize_mx(F((T, 65), 2), q, s),
        lambda: moe.swiglu_quantize_mx(F((T, 2 * K), 2), q, s, rows=F((2,))),
        lambda: moe.dequantize_mx(q, s, F((T, K + 1), 2)),
    ]
    for i, c in enumerate(cases):
        with pytest.raises(ValueError):
            c()
            raise AssertionError(f"case {i} was let through")


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    """A call launches on the current device: tensors of another one are
    refused before the library is reached."""
    import torch

    class On(F):
        def get_device(self):
            return 1

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    T, K = 4, 64
    x, q, s = On((T, K), 2), On((T, K), 1), On((T, K // 32), 1)
    for call in (lambda: moe.rms_norm(x, On((K,)), 1e-6, y=x),
                 lambda: moe.quantize_mx(x, q, s),
                 lambda: moe.grouped_matmul(x, On((3,)), On((2, 8, K), 2), On((T, 8), 2))):
        with pytest.raises(ValueError, match="device"):
            call()


def test_norm_width_limit():
    for call in (lambda: norm(T=1, H=BIG + 32), lambda: norm_bwd(T=1, H=BIG + 32)):
        assert call() == LIMIT
    with pytest.raises(moe.MoeError) as e:
        moe.rms_norm_backward_workspace_size(1, BIG + 1)
    assert e.value.status == LIMIT


@pytest.mark.parametrize("name", ["float16", "float8_e5m2", "float8_e4m3fnuz"])
def test_binding_refuses_types_of_the_same_size(monkeypatch, name):
    """A float16 tensor where bf16 is read, another 8-bit type where E4M3 is."""
    import torch

    class On(F):
        dtype = torch.bfloat16

        def get_device(self):
            return 0

    class Other(On):
        dtype = getattr(torch, name)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    T, K = 4, 64
    if name == "float16":
        x = Other((T, K), 2)
        calls = [lambda: moe.rms_norm(x, On((K,)), 1e-6, y=On((T, K), 2)),
                 lambda: moe.quantize_mx(x, On((T, K), 1), On((T, 2), 1)),
                 lambda: moe.grouped_matmul(x, On((3,)), On((2, 8, K), 2), On((T, 8), 2)),
                 lambda: moe.grouped_matmul_dx(On((T, 8), 2), On((3,)), On((2, 8, K), 2), x)]
    else:
        q = Other((T, K), 1)
        calls = [lambda: moe.quantize_mx(On((T, K), 2), q, On((T, 2), 1)),
                 lambda: moe.dequantize_mx(q, On((T, 2), 1), On((T, K), 2)),
                 lambda: moe.rms_norm(On((T, K), 2), On((K,)), 1e-6, yq=q, ys=On((T, 2), 1))]
    for call in calls:
        with pytest.raises(ValueError, match="type"):
            call()


def test_binding_refuses_floats_for_whole_numbers_and_back(monkeypatch):
    """float32 offsets, selections and row counts, int32 norm weights, values
    and outputs: the same size, but their bits mean something else. A workspace
    may have any type."""
    import torch

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def on(shape, dtype):
        class On(F):
            def get_device(self):
                return 0
        t = On(shape, dtype.itemsize)
        t.dtype = dtype
        return t

    bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    T, K, M, L = 4, 64, 8, 2
    x, y, w = on((T, K), bf), on((T, M), bf), on((L, M, K), bf)
    off, rows = on((L + 1,), i32), on((T,), i32)
    q, s, wq, ws = on((T, K), u8), on((T, 2), u8), on((L, M, K // 2), u8), on((L, M, 2), u8)
    reached = []
    monkeypatch.setattr(moe, "lib", lambda: reached.append(1) or (_ for _ in ()).throw(KeyError()))
    calls = [
        lambda o, r: moe.grouped_matmul(x, o, w, y, r),
        lambda o, r: moe.grouped_matmul_dw(y, x, o, on((L, M, K), bf), r),
        lambda o, r: moe.grouped_matmul_mx(q, s, o, wq, ws, y, r),
    ]
    bad = [lambda c=c: c(on((L + 1,), f32), rows) for c in calls]
    bad += [lambda c=c: c(off, on((T,), f32)) for c in calls]
    bad += [
        lambda: moe.grouped_matmul_dx(y, on((L + 1,), f32), w, x),
        lambda: moe.grouped_matmul(x, off, w, on((T, M), i32), rows),
        lambda: moe.rms_norm(x, on((K,), i32), 1e-6, y=x),
        lambda: moe.rms_norm_backward(x, x, on((K,), f32), 1e-6, x, on((K,), i32), None),
        lambda: moe.quantize_mx(on((T, K), i32), q, s),
        lambda: moe.dequantize_mx(q, s, on((T, K), i32)),
        lambda: moe.swiglu_quantize_mx(on((T, 2 * K), bf), q, s, rows=on((1,), f32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError, match="type"):
            call()
        assert not reached, f"case {i} was let through"
    good = [lambda c=c: c(off, rows) for c in calls]
    good += [lambda: moe.rms_norm(x, on((K,), f32), 1e-6, y=on((T, K), torch.int16)),
             lambda: moe.rms_norm_backward(x, x, on((K,), f32), 1e-6, x, on((K,), f32), off)]
    for call in good:
        with pytest.raises(KeyError):
            call()
