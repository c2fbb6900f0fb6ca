"""The large-tile kernels of the grouped products where a block has several
tiles of several stages each, whole ones (whose stores stay in flight while the
next tile is multiplied) and cut ones: against float64 on the GPU, with bounds
from the number of roundings."""
import numpy as np
import pytest

import ops_plain as plain
import routing_grouped_expert_amd as moe
from gpu_util import note, sync, torch
from test_gpu_grouped import out_tensor, untouched

pytestmark = pytest.mark.gpu

# rows per expert: whole tiles of 256 and cut ones, more tiles than blocks at 16 or
# more tiles the other way; hundreds of experts with a whole narrow tile of 128 or
# 64 rows, and one row more
WIDE = [512, 768, 600, 256, 0, 700, 511, 257, 1024]
NARROW = {n: [n] * 300 for n in (64, 65, 128)}
NARROW["mixed"] = [128, 64, 65, 127, 33, 128] * 60


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def gpu(a):
    return torch().from_numpy(a).to("cuda:0")


def normal(*shape, seed, sigma=1.0):
    t = torch()
    g = t.Generator(device="cuda:0")
    g.manual_seed(seed)
    return (t.randn(shape, generator=g, device="cuda:0") * sigma).bfloat16()


def check(got, ref, bound, what):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds"


def bound(ref, sums, terms, f32):
    """As ops_plain.product_bound: `terms` additions, each off by at most 2^-23 of
    a partial sum, and the output's rounding."""
    acc = terms * 2.0 ** -23 * sums
    return acc + (0.0 if f32 else plain.BF16 * (ref.abs() + acc)) + 1e-40


def picked(N, T, k, seed, gather):
    """Selections of N rows (every one a row of x), and the rows they name."""
    t = torch()
    if not gather:
        return None, t.arange(N, device="cuda:0")
    rows = np.random.default_rng(seed).integers(0, T * k, N).astype(np.int32)
    return gpu(rows), gpu(rows).long() // k


def products(counts, K, M, f32, gather, which, what):
    t = torch()
    k = 2 if gather else 1
    off = offsets(counts)
    n = int(off[-1])
    N, L = n + 3, len(counts)
    T = N // 2 if gather else N
    x, dy = normal(T, K, seed=1), normal(N, M, seed=2)
    rows, src = picked(N, T, k, 3, gather)
    goff = gpu(off)
    if which == "dw":
        o = out_tensor((L, M, K), f32)
    else:
        w = normal(L, M, K, seed=4, sigma=0.1)
        o = out_tensor((N, M if which == "y" else K), f32)
    note(what)
    for _ in range(2):
        if which == "y":
            moe.grouped_matmul(x, goff, w, o, permuted_rows=rows, k=k)
        elif which == "dx":
            moe.grouped_matmul_dx(dy, goff, w, o)
        else:
            moe.grouped_matmul_dw(dy, x, goff, o, permuted_rows=rows, k=k)
    sync()
    for e in range(L):
        a = slice(int(off[e]), int(off[e + 1]))
        X, D = x[src[a]].double(), dy[a].double()
        if which == "dw":
            A, B, terms, got = D.t(), X, max(a.stop - a.start, 1), o[e]
        else:
            A, B = (X, w[e].double().t()) if which == "y" else (D, w[e].double())
            terms, got = A.shape[1], o[a]
        ref = A @ B
        check(got, ref, bound(ref, A.abs() @ B.abs(), terms, f32), f"{what}, expert {e}")
    assert which == "dw" or untouched(o, n), what + ": rows behind the last expert"
    t.cuda.empty_cache()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("which,K,M,gather", [
    ("y", 320, 8192, True), ("y", 320, 8200, False), ("y", 32, 8192, True), ("y", 1000, 4096, False),
    ("dx", 8192, 320, False), ("dx", 8200, 328, False), ("dx", 4096, 1000, False),
    ("dw", 2048, 2560, True), ("dw", 2048, 2560, False), ("dw", 2056, 2568, True)])
def test_several_wide_tiles(which, K, M, gather, f32):
    products(WIDE, K, M, f32, gather, which, f"wide {which} K={K} M={M} gather={gather} f32={f32}")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("counts", [128, "mixed"])
@pytest.mark.parametrize("which,K,M", [("y", 192, 512), ("y", 64, 520), ("y", 456, 768),
                                       ("dx", 512, 192), ("dx", 520, 64), ("dx", 768, 456)])
def test_several_narrow_tiles(which, K, M, counts, f32):
    products(NARROW[counts], K, M, f32, which == "y", which,
             f"narrow {which} {counts} K={K} M={M} f32={f32}")


@pytest.mark.parametrize("gather", [False, True])
def test_dw_of_many_whole_tiles_with_few_stages(gather):
    """Rows for one to five stages of a dw tile, in whole tiles."""
    products([1, 32, 33, 64, 96, 97, 128, 160] * 6, 768, 1024, False, gather, "dw",
             f"short dw gather={gather}")


# ------------------------------------------------------------ microscaled

def codes(*shape, bits, seed):
    """Random codes (of 8 bits: no NaN) as bytes, scale codes, and their values."""
    t = torch()
    g = t.Generator(device="cuda:0")
    g.manual_seed(seed)
    K = shape[-1]
    s = t.randint(118, 132, shape[:-1] + (K // 32,), generator=g, device="cuda:0", dtype=t.uint8)
    if bits == 8:
        c = t.randint(0, 127, shape, generator=g, device="cuda:0", dtype=t.uint8)
        c |= t.randint(0, 2, shape, generator=g, device="cuda:0", dtype=t.uint8) << 7
    else:
        c = t.randint(0, 256, shape[:-1] + (K // 2,), generator=g, device="cuda:0", dtype=t.uint8)
    return c, s


def decoded(c, s, bits):
    t = torch()
    if bits == 8:
        v = t.from_numpy(plain.E4M3).to("cuda:0")[c.long()]
    else:
        v = t.from_numpy(plain.E2M1).to("cuda:0")[t.stack([c & 15, c >> 4], -1).flatten(-2).long()]
    return v * t.exp2(s.double() - 127).repeat_interleave(32, -1)


def mx(counts, K, M, xbits, f32, gather, what):
    t = torch()
    k = 2 if gather else 1
    off = offsets(counts)
    n = int(off[-1])
    N, L = n + 3, len(counts)
    T = N // 2 if gather else N
    xq, xs = codes(T, K, bits=xbits, seed=5)
    wq, ws = codes(L, M, K, bits=4, seed=6)
    rows, src = picked(N, T, k, 7, gather)
    goff, o = gpu(off), out_tensor((N, M), f32)
    note(what)
    for _ in range(2):
        moe.grouped_matmul_mx(xq, xs, goff, wq, ws, o, permuted_rows=rows, k=k)
    sync()
    X = decoded(xq, xs, xbits)
    for e in range(L):
        a = slice(int(off[e]), int(off[e + 1]))
        A, B = X[src[a]], decoded(wq[e], ws[e], 4)
        ref = A @ B.t()
        check(o[a], ref, bound(ref, A.abs() @ B.t().abs(), K, f32), f"{what}, expert {e}")
    assert untouched(o, n), what + ": rows behind the last expert"
    t.cuda.empty_cache()


@pytest.mark.parametrize("xbits", [4, 8])
@pytest.mark.parametrize("K,M,f32,gather", [
    (640, 8192, False, True),   # five stages: runs of three and two
    (640, 8200, True, False),
    (1152, 4096, False, False),  # nine: four, three, two
    (1184, 4101, True, True),   # ten, the last cut; element stores
    (128, 8192, False, True),   # one, and one of zeros
    (2080, 2048, True, False)])
def test_mx_several_wide_tiles(K, M, f32, gather, xbits):
    mx(WIDE, K, M, xbits, f32, gather, f"mx wide K={K} M={M} f32={f32} gather={gather} xbits={xbits}")


@pytest.mark.parametrize("xbits", [4, 8])
@pytest.mark.parametrize("counts", [64, 65, 128, "mixed"])
@pytest.mark.parametrize("K,M,f32", [(640, 512, False), (288, 520, True), (1024, 256, False)])
def test_mx_several_narrow_tiles(K, M, f32, counts, xbits):
    mx(NARROW[counts], K, M, xbits, f32, False, f"mx narrow {counts} K={K} M={M} f32={f32} xbits={xbits}")
