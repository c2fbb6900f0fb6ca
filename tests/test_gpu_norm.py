"""The root-mean-square norm with the residual's addition, its 8-bit output and
its backward, against float64."""
import numpy as np
import pytest

import ops_plain as plain
import routing_grouped_expert_amd as moe
from gpu_util import bf16_to_f64, dev, host, note, sync, torch

pytestmark = pytest.mark.gpu
EPS = 1e-6
SHAPES = [(1, 8), (1, 7168), (3, 32), (5, 512), (9, 520), (2, 2048), (3, 2080), (2, 4096),
          (2, 4128), (3, 8192), (2, 8224), (1, 16384), (2, 16416), (7, 1), (4, 33), (3, 1001),
          (600, 96), (1030, 40)]


def rel(H):
    """fp32 roundings on the longest way from an input to y, each 2^-24: a
    thread's chain, 6 wave steps, 16 waves, and the division, root and
    products. (The root halves the sum's error; that is left in hand.)"""
    return (max(32, H // 256 + 1) + 6 + 16 + 8) * plain.F32


def buf(shape, esize):
    t = torch()
    dt = {1: t.uint8, 2: t.int16, 4: t.float32}[esize]
    return t.full(tuple(shape), 1, dtype=dt, device="cuda:0")


def draw(T, H, seed):
    rng = np.random.default_rng(seed)
    x = plain.to_bf16(rng.standard_normal((T, H)))
    r = plain.to_bf16(rng.standard_normal((T, H)) * 3)
    w = (1 + 0.2 * rng.standard_normal(H)).astype(np.float32)
    return x, r, w


def check_quantised(q, s, y, e, what):
    """MXFP8 of a y known to the relative error e: the scale is that of the
    block's largest magnitude (its neighbour only where that lies within e of a
    power of two), and each value is the nearest code's, cut at 448."""
    a = np.abs(y).reshape(*y.shape[:-1], -1, 32).max(-1)
    lo, hi = (plain.mx_quantize(np.repeat(a * f, 32, -1), 8)[1] for f in (1 - e, 1 + e))
    assert ((s == lo) | (s == hi)).all(), what
    sc = np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, -1)
    v = plain.mx_decode(q, s, 8)
    cut = np.maximum(np.abs(y) * (1 + e) - 448 * sc, 0)
    bound = np.maximum(np.abs(y) * (2.0 ** -4), sc * 2.0 ** -10) + 2 * e * np.abs(y)
    bad = np.abs(v - y) > np.maximum(bound, cut)
    assert not bad.any(), f"{what}: {bad.sum()}"


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(T, H, residual):
    x, r, w = draw(T, H, T * 10000 + H)
    res = r if residual else None
    q = H % 32 == 0
    h_, y_ = buf((T, H), 2), buf((T, H), 2)
    yq, ys = (buf((T, H), 1), buf((T, H // 32), 1)) if q else (None, None)
    note(f"norm T={T} H={H} residual={residual}")
    moe.rms_norm(dev(x), dev(w), EPS, y=y_, yq=yq, ys=ys,
                 residual=None if res is None else dev(res), residual_out=h_)
    sync()
    h, _, y = plain.norm(x, res, w.astype(np.float64), EPS)
    assert np.array_equal(host(h_).view(np.uint16), h)
    e = rel(H)
    plain.check(bf16_to_f64(host(y_).view(np.uint16)), y,
                np.abs(y) * (plain.BF16 + 2 * e) + 1e-40, "y")
    if q:
        check_quantised(host(yq), host(ys), y, e, f"T={T} H={H}")


def test_outputs_are_optional_and_independent():
    """Each output alone has the bits it has beside the others."""
    T, H = 5, 320
    x, r, w = (dev(a) for a in draw(T, H, 4))
    full = [buf((T, H), 2), buf((T, H), 2), buf((T, H), 1), buf((T, 10), 1)]
    moe.rms_norm(x, w, EPS, y=full[1], yq=full[2], ys=full[3], residual=r, residual_out=full[0])
    h, y, yq, ys = buf((T, H), 2), buf((T, H), 2), buf((T, H), 1), buf((T, 10), 1)
    moe.rms_norm(x, w, EPS, residual=r, residual_out=h)
    moe.rms_norm(x, w, EPS, residual=r, y=y)
    moe.rms_norm(x, w, EPS, residual=r, yq=yq, ys=ys)
    sync()
    for a, b in zip(full, (h, y, yq, ys)):
        assert np.array_equal(host(a), host(b))


@pytest.mark.parametrize("H", [64, 1000, 1001, 7168])
def test_in_place(H):
    """residual_out on residual and y on x, as a serving loop keeps them."""
    x, r, w = (dev(a) for a in draw(6, H, H))
    h, y = buf((6, H), 2), buf((6, H), 2)
    moe.rms_norm(x, w, EPS, y=y, residual=r, residual_out=h)
    moe.rms_norm(x, w, EPS, y=x, residual=r, residual_out=r)
    sync()
    assert np.array_equal(host(r), host(h)) and np.array_equal(host(x), host(y))
    d, g0, g1 = dev(draw(6, H, 9)[0]), buf((H,), 4), buf((H,), 4)
    ws = torch().empty(max(256, moe.rms_norm_backward_workspace_size(6, H)), dtype=torch().uint8,
                       device="cuda:0")
    dx = buf((6, H), 2)
    moe.rms_norm_backward(d, h, w, EPS, dx, g0, ws, dresidual=y)
    moe.rms_norm_backward(d, h, w, EPS, d, g1, ws, dresidual=y)
    sync()
    assert np.array_equal(host(dx), host(d)) and np.array_equal(host(g0), host(g1))


def test_zero_and_special_rows():
    """A row of zeros gives zeros (eps keeps the root finite), a row with a NaN
    or an infinity gives NaN or zero where the formula does, other rows keep
    their values."""
    T, H = 4, 64
    x, _, w = draw(T, H, 2)
    x[1] = 0
    x[2, 5] = 0x7FC0
    x[3, 7] = 0x7F80
    y, yq, ys = buf((T, H), 2), buf((T, H), 1), buf((T, 2), 1)
    moe.rms_norm(dev(x), dev(w), EPS, y=y, yq=yq, ys=ys)
    sync()
    v = bf16_to_f64(host(y).view(np.uint16))
    assert (v[1] == 0).all() and np.isnan(v[2]).all()
    assert np.isnan(v[3, 7]) and (np.delete(v[3], 7) == 0).all()
    assert (host(ys)[1] == 0).all() and (host(yq)[1] & 127 == 0).all()
    assert (host(ys)[2] == 255).all() and (host(ys)[3] == [255, 0]).all()
    ref = plain.norm(x[:1], None, w.astype(np.float64), EPS)[2]
    plain.check(v[:1], ref, np.abs(ref) * (plain.BF16 + 2 * rel(H)), "row 0")


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("with_dres", [False, True])
def test_backward(T, H, with_dres):
    x, r, w = draw(T, H, T + H)
    dy, dr = draw(T, H, T + H + 1)[:2]
    dres = dr if with_dres else None
    dx, dg = buf((T, H), 2), buf((H,), 4)
    ws = torch().empty(max(256, moe.rms_norm_backward_workspace_size(T, H)),
                       dtype=torch().uint8, device="cuda:0")
    ws.fill_(0xFF)
    note(f"norm backward T={T} H={H} dres={with_dres}")
    moe.rms_norm_backward(dev(dy), dev(x), dev(w), EPS, dx, dg, ws,
                          dresidual=None if dres is None else dev(dres))
    sync()
    h, d, W = bf16_to_f64(x), bf16_to_f64(dy), w.astype(np.float64)
    D = None if dres is None else bf16_to_f64(dres)
    rx, rg = plain.norm_backward(d, h, W, EPS, D)
    s = 1 / np.sqrt((h * h).mean(1, keepdims=True) + EPS)
    # each factor of the two terms is off by at most rel(H) of its magnitudes
    size = s * (np.abs(W * d) + np.abs(h) * s * s * np.abs(W * d * h).mean(1, keepdims=True))
    size = size + (0 if D is None else np.abs(D))
    plain.check(bf16_to_f64(host(dx).view(np.uint16)), rx,
                4 * rel(H) * size + plain.BF16 * np.abs(rx) * (1 + 1e-3) + 1e-40, "dx")
    # a block's rows in turn, then up to 32 blocks a slice and 16 slices
    chain = (T / 512 + 1 + 32 + 16 + 4) * plain.F32 + 2 * rel(H)
    plain.check(host(dg).astype(np.float64), rg, chain * np.abs(d * h * s).sum(0) + 1e-40, "dweight")


def test_backward_against_differences():
    """The formula's derivative, by central differences of the norm in 64 bits
    (the kernel's y is rounded to bf16, too coarse to difference)."""
    T, H = 3, 40
    x, _, w = draw(T, H, 77)
    dy = draw(T, H, 78)[0]
    h, d, W = bf16_to_f64(x), bf16_to_f64(dy), w.astype(np.float64)
    dx, dg = buf((T, H), 2), buf((H,), 4)
    ws = torch().empty(moe.rms_norm_backward_workspace_size(T, H), dtype=torch().uint8,
                       device="cuda:0")
    moe.rms_norm_backward(dev(dy), dev(x), dev(w), EPS, dx, dg, ws)
    sync()

    def loss(h, W):
        return (d * h / np.sqrt((h * h).mean(1, keepdims=True) + EPS) * W).sum()

    got, gg = bf16_to_f64(host(dx).view(np.uint16)), host(dg)
    for t, c in ((0, 0), (2, 39), (1, 17)):
        u = np.zeros_like(h)
        u[t, c] = 1e-4
        q = (loss(h + u, W) - loss(h - u, W)) / 2e-4
        assert abs(q - got[t, c]) <= plain.BF16 * abs(q) + 1e-5
    for c in (0, 39):
        u = np.zeros(H)
        u[c] = 1e-4
        q = (loss(h, W + u) - loss(h, W - u)) / 2e-4
        assert abs(q - gg[c]) <= 1e-5 * max(1, abs(q))


def test_no_rows():
    t = torch()
    e = t.empty((0, 64), dtype=t.bfloat16, device="cuda:0")
    dg = buf((64,), 4)
    moe.rms_norm_backward(e, e, buf((64,), 4), EPS, e, dg, None)
    moe.rms_norm(e, buf((64,), 4), EPS, y=e)
    sync()
    assert (host(dg) == 0).all()


def test_misaligned_rows_match():
    """Views off 16 bytes run element by element: within the same bounds."""
    t = torch()
    x, r, w = draw(4, 128, 8)
    ref = plain.norm(x, r, w.astype(np.float64), EPS)
    v = []
    for a in (x, r):
        d = t.empty(4 * 128 + 1, dtype=t.int16, device="cuda:0")[1:].view(4, 128)
        d.copy_(dev(a))
        v.append(d)
    h, y, yq, ys = buf((4, 128), 2), buf((4, 128), 2), buf((4, 128), 1), buf((4, 4), 1)
    moe.rms_norm(v[0], dev(w), EPS, y=y, yq=yq, ys=ys, residual=v[1], residual_out=h)
    sync()
    assert np.array_equal(host(h).view(np.uint16), ref[0])
    plain.check(bf16_to_f64(host(y).view(np.uint16)), ref[2],
                np.abs(ref[2]) * (plain.BF16 + 2 * rel(128)), "y")
    check_quantised(host(yq), host(ys), ref[2], rel(128), "misaligned")


@pytest.mark.parametrize("T,H", [((1 << 24) + 5, 3), ((1 << 26) + 5, 8)])
def test_more_rows_than_a_launch_holds(T, H):
    """A block (or wave) for every row would be 2^32 threads: the bits are those
    of the rows called in parts."""
    t = torch()
    note(f"norm T={T} H={H}")
    x = t.randint(0, 0x4000, (T, H), dtype=t.int16, device="cuda:0")  # bf16 in [0, 2)
    w = t.linspace(0.5, 1.5, H, dtype=t.float32, device="cuda:0")
    y, h, part = (t.zeros((T, H), dtype=t.int16, device="cuda:0") for _ in range(3))
    moe.rms_norm(x, w, EPS, y=y, residual=x, residual_out=h)
    step = 1 << 21
    for a in range(0, T, step):
        b = min(T, a + step)
        moe.rms_norm(x[a:b], w, EPS, y=part[a:b], residual=x[a:b])
    sync()
    assert t.equal(y, part)
    assert t.equal(h.view(t.bfloat16), x.view(t.bfloat16) * 2)
    ref = plain.norm(host(h[-3:]).view(np.uint16), None, host(w).astype(np.float64), EPS)[2]
    plain.check(bf16_to_f64(host(y[-3:]).view(np.uint16)), ref,
                np.abs(ref) * (plain.BF16 + 2 * rel(H)) + 1e-40, "last rows")


@pytest.mark.parametrize("H", [8, 1])
def test_reciprocal_root_is_rounded_once(H):
    """The row's 1 / sqrt(mean + eps) is the nearest fp32 value but for cases that
    lie within 2^-6 of a step of the middle between two (a first value off by at most
    4 steps, corrected once: the correction's own roundings and its second order are
    below that). Seen in dweight: with one row h = (1, 0, ..) and dy = 1 it is the
    root itself. The mean is 1 / H and eps a multiple of 2^-24 that makes their sum
    exact."""
    t = torch()
    n = 256
    rng = np.random.default_rng(H)
    eps = rng.integers(1, 1 << 20, n) * 2.0 ** -24 * (1 if H == 8 else 2)
    h = np.zeros((1, H), np.uint16)
    h[0, 0] = 0x3F80
    one = np.full((1, H), 0x3F80, np.uint16)
    dg, dx = buf((n, H), 4), buf((1, H), 2)
    ws = t.empty(max(256, moe.rms_norm_backward_workspace_size(1, H)), dtype=t.uint8, device="cuda:0")
    gh, gdy, gw = dev(h), dev(one), dev(np.ones(H, np.float32))
    note(f"reciprocal root H={H}")
    for i in range(n):
        moe.rms_norm_backward(gdy, gh, gw, float(eps[i]), dx, dg[i], ws)
    sync()
    got = host(dg)[:, 0].astype(np.float64)
    s = 1 / np.sqrt(1 / H + eps)
    step = 2.0 ** (np.floor(np.log2(s)) - 23)
    assert (np.abs(got - s) <= (0.5 + 2.0 ** -6) * step).all(), (np.abs(got - s) / step).max()
