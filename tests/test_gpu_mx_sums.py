"""Sums of the scaled product are those of fp32 whatever the magnitudes beside
each other: small E4M3 values next to the largest, in every kernel's class of
row counts."""
import numpy as np
import pytest

import ops_plain as plain
import routing_grouped_expert_amd as moe
from gpu_util import dev, note, sync, torch
from test_gpu_grouped import out_tensor, values

pytestmark = pytest.mark.gpu

# rows per expert: the kernel for few, tiles of 64, 128 and 256 rows
COUNTS = {"one": [1], "few": [9, 25, 0, 32], "narrow": [33, 64], "middle": [65, 128], "wide": [129, 300]}


def product(xc, wc, counts):
    """fp32 y of E4M3 codes xc [N, K] and E2M1 codes wc [L, M, K], scales 1."""
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    N, K = xc.shape
    L, M, _ = wc.shape
    y = out_tensor((N, M), True)
    moe.grouped_matmul_mx(dev(xc), dev(np.full((N, K // 32), 127, np.uint8)), dev(off),
                          dev(plain.pack4(wc)), dev(np.full((L, M, K // 32), 127, np.uint8)), y)
    sync()
    return off, values(y)


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("K", [32, 96, 128, 288])
@pytest.mark.parametrize("top", [0x7E, 0x6D, 0x40, 0x3F])
def test_small_values_beside_a_large_one(name, K, top):
    """One value of 448, 104, 2 or 1.875 in each 8 consecutive places, the others
    any smaller ones, weights any, all products positive (what is cut from them
    adds up). Sums of K products: fp32 with one rounding (2^-23, if it cuts) for
    each addition."""
    counts = COUNTS[name]
    rng = np.random.default_rng(K + top)
    N, M, L = sum(counts), 40, len(counts)
    x = rng.integers(0, top, (N, K)).astype(np.uint8)
    x[np.arange(N)[:, None], np.arange(0, K, 8) + rng.integers(0, 8, (N, K // 8))] = top
    w = rng.integers(0, 8, (L, M, K)).astype(np.uint8)
    note(f"sums {name} K={K} top={top:#x}")
    off, y = product(x, w, counts)
    ref, s = plain.grouped(plain.E4M3[x], plain.E2M1[w], off, M)
    plain.check(y, ref, plain.product_bound(ref, s, K, True), f"{name} K={K} top={top:#x}")


def test_every_pair_beside_the_largest():
    """Each code (either sign) times each weight code beside 448 x 6 and beside the
    largest of its own part, 1.875 x 6: two products, whose sum fp32 holds."""
    for big in (0x7E, 0x3F):
        codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
        N, M = len(codes), 16
        x = np.zeros((N, 32), np.uint8)
        x[:, 0], x[:, 5] = codes, big
        w = np.zeros((1, M, 32), np.uint8)
        w[0, :, 0], w[0, :, 5] = np.arange(16), 7
        for n in (N, 100, 40, 20):  # every kernel
            _, y = product(x[:n], w, [n])
            ref = plain.E4M3[x[:n]] @ plain.E2M1[w[0]].T
            assert np.array_equal(y, ref), (big, n, np.abs(y - ref).max())


@pytest.mark.parametrize("counts", [[20], [50], [100], [300]])
def test_normal_values_in_fp32(counts):
    """Normal values at K 4096 against what 4096 random roundings of partial sums
    come to: each 2^-24 / sqrt(3) of a sum no larger than the result's size, 64 times
    that together."""
    K, M = 4096, 64
    rng = np.random.default_rng(3)
    n = sum(counts)
    x, xs = plain.mx_quantize(rng.standard_normal((n, K)), 8)
    w, ws = plain.mx_quantize(rng.standard_normal((1, M, K)), 4)
    y = out_tensor((n, M), True)
    off = np.array([0, n], np.int32)
    moe.grouped_matmul_mx(dev(x), dev(xs), dev(off), dev(plain.pack4(w)), dev(ws), y)
    sync()
    ref = plain.mx_decode(x, xs, 8) @ plain.mx_decode(plain.pack4(w), ws, 4)[0].T
    err = np.linalg.norm(values(y) - ref) / np.linalg.norm(ref)
    assert err <= 64 * 2.0 ** -24 / np.sqrt(3), err
