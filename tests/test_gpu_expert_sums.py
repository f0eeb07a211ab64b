"""The experts' E4M3 product sums in 32 bits, whatever the sizes of the channels' products are."""
import numpy as np
import pytest
import torch

import experts_oracle as oracle64
from combine_ep_get_02_amd import experts

pytestmark = pytest.mark.gpu
U = oracle64.U


def _codes(v):
    return torch.from_numpy(np.asarray(v, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)


def _run(sizes, n, k, x, xs, w, ws):
    E, M = len(sizes), x.shape[0]
    out = torch.full((M, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    experts.ep_expert_gemm_fp8(E, n, k, x.cuda(), torch.from_numpy(xs).cuda(), w.cuda(), torch.from_numpy(ws).cuda(),
                               torch.from_numpy(np.asarray(sizes, np.int32)).cuda(), M, out)
    return out.double().cpu().numpy()


# (sizes, n, k) that reach each kernel: few rows and few or many columns, some rows of many experts, many rows
CASES = [([3], 256, 640), ([20], 1024, 1152), ([40], 2048, 896), ([9] * 40, 1024, 384), ([20] * 40, 2048, 256),
         ([50] * 8, 2056, 640), ([130, 200, 7], 4096, 768), ([1100, 900], 4104, 512),
         ([50] * 8, 4104, 640), ([1100, 900], 2056, 384)]


@pytest.mark.parametrize("sizes,n,k", CASES, ids=str)
def test_small_products_beside_large_ones_that_cancel(sizes, n, k):
    """In each group of eight channels one product is the largest there is, 448 * 448, and the group's opposite takes it
    back in the next one; the others are small integers, a few 2^-17 of it.  Every sum is exact in f32."""
    rng = np.random.default_rng(n + k)
    E, M = len(sizes), sum(sizes)
    xv = rng.integers(-3, 4, size=(M, k)).astype(np.float32)
    wv = rng.integers(-3, 4, size=(E, n, k)).astype(np.float32)
    at = np.arange(0, k, 16) + rng.integers(0, 8, size=k // 16)
    xv[:, at] = 448.0
    wv[:, :, at] = 448.0
    back = np.arange(8, k, 16) + rng.integers(0, 8, size=k // 16)
    xv[:, back] = -448.0
    wv[:, :, back] = 448.0
    x, w = _codes(xv), _codes(wv)
    xs, ws = np.full((M, k // 128), 0.5, np.float32), np.full((E, -(-n // 128), k // 128), 2.0, np.float32)
    got = _run(sizes, n, k, x, xs, w, ws)
    owner = np.repeat(np.arange(E), sizes)
    rows = np.unique(np.r_[0:min(M, 150), max(M - 150, 0):M])  # the first and last tiles whole
    for e in np.unique(owner[rows]):
        r = rows[owner[rows] == e]
        want = xv[r].astype(np.float64) @ wv[e].astype(np.float64).T
        # partial sums are integers below 2^24 (a step of 448 * 448 and at most 9 * 128 beside it): one rounding
        assert np.array_equal(got[r], oracle64.bf16_round(want))


@pytest.mark.parametrize("sizes,n,k", CASES, ids=str)
def test_codes_of_all_sizes(sizes, n, k):
    """Codes spread over all exponents, against f32 sums' bound: no part of a product is dropped."""
    rng = np.random.default_rng(n * k)
    E, M = len(sizes), sum(sizes)
    x = _codes(rng.standard_normal((M, k)) * 2.0 ** rng.integers(-9, 8, size=(M, k)))
    w = _codes(rng.standard_normal((E, n, k)) * 2.0 ** rng.integers(-9, 8, size=(E, n, k)))
    xs = (rng.random((M, k // 128)) * 0.02 + 1e-3).astype(np.float32)
    ws = (rng.random((E, -(-n // 128), k // 128)) * 0.02 + 1e-3).astype(np.float32)
    got = _run(sizes, n, k, x, xs, w, ws)
    want, mag = oracle64.product(x, xs, w, ws, sizes, M)
    # the rounding to bf16, and K products and K / 128 scaled sums in f32, each step off by at most 2 U of the sum of
    # magnitudes (the matrix unit may truncate), the scales' product by U
    off = (2 * (k + k // 128) + 2) * U * mag
    tol = oracle64.BF16_HALF * np.abs(want) + off * (1 + oracle64.BF16_HALF)
    # the widest draws lie outside the type's range and are NaN codes: they make their row and column NaN, no more
    number = ~np.isnan(want)
    assert number.any() and not number.all() and np.array_equal(np.isnan(got), ~number)
    assert np.all(np.abs(got - want)[number] <= tol[number])
