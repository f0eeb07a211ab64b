"""The experts' E4M3 products against their definitions in binary64."""
import numpy as np
import pytest
import torch

import experts_oracle as oracle64
from combine_ep_get_02_amd import ep, experts
from gpu_harness import bf16_host, to_dev_bf16

pytestmark = pytest.mark.gpu
U = oracle64.U


def _codes(rng, shape, exact):
    """E4M3 codes of normal values, or of the integers -2 .. 2 (sums of products are then exact)."""
    v = rng.integers(-2, 3, size=shape).astype(np.float32) if exact else rng.standard_normal(shape).astype(np.float32) * 40
    return torch.from_numpy(v).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(rng, shape, exact):
    if exact:
        return (2.0 ** rng.integers(-3, 3, size=shape)).astype(np.float32)
    return (rng.random(shape) * 0.02 + 1e-3).astype(np.float32)


def _inputs(rng, E, N, K, num_rows, exact):
    x = _codes(rng, (num_rows, K), exact)
    w = _codes(rng, (E, N, K), exact)
    xs = _scales(rng, (num_rows, K // 128), exact)
    ws = _scales(rng, (E, -(-N // 128), K // 128), exact)
    return x, xs, w, ws


def _product(E, n, k, x, xs, w, ws, rows, num_rows, swiglu=False, stream=None):
    """Outputs in buffers with a guard row behind them, and the device status."""
    drows = None if rows is None else torch.from_numpy(np.asarray(rows, np.int32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (E, n, k, x.cuda(), torch.from_numpy(xs).cuda(), w.cuda(), torch.from_numpy(ws).cuda(), drows, num_rows)
    if swiglu:
        out = torch.full((num_rows + 1, n), 0xAB, dtype=torch.uint8, device="cuda")
        outs = torch.full((num_rows + 1, n // 128), -2.0, device="cuda")
        experts.ep_expert_gemm_swiglu_fp8(*args, out, outs, status)
        torch.cuda.synchronize()
        assert bool((out[num_rows] == 0xAB).all()) and bool((outs[num_rows] == -2.0).all())
        return out[:num_rows], outs[:num_rows].cpu().numpy(), int(status.item())
    out = torch.full((num_rows + 1, n), -1, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    experts.ep_expert_gemm_fp8(*args, out, status)
    torch.cuda.synchronize()
    assert np.all(bf16_host(out[num_rows]) == 0xFFFF)
    return out[:num_rows], int(status.item())


def _values(t):
    return t.double().cpu().numpy()


def _check_product(got, want, mag, K, exact, cut=None):
    rows = ~np.isnan(want[:, 0])
    if exact:  # every partial sum is an integer times a power of two, far below 2^24 units: one rounding
        assert np.array_equal(_values(got)[rows], oracle64.bf16_round(want[rows]))
    else:
        # the rounding to bf16, and K products and K / 128 scaled sums in f32, each step off by at
        # most 2 U of the sum of magnitudes (the matrix unit may truncate), the scale's product by U;
        # and in each group of eight channels up to eight products cut below 2^-13 of the largest
        off = (2 * (K + K // 128) + 2) * U * mag[rows] + 8 * 2.0 ** -13 * cut[rows]
        tol = oracle64.BF16_HALF * np.abs(want[rows]) + off * (1 + oracle64.BF16_HALF)
        assert np.all(np.abs(_values(got)[rows] - want[rows]) <= tol)
    # rows that no segment holds are left as they were
    assert np.all(bf16_host(got)[~rows] == 0xFFFF)


SEGMENTS = {
    "one row": [1], "ragged": [5, 0, 17, 1, 33, 16, 0], "empty": [0, 0, 0], "tile edges": [128, 127, 129, 256, 1],
    "one expert many rows": [700], "last": [0, 0, 0, 40],
}


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("n,k", [(8, 128), (128, 256), (264, 384), (1000, 128), (512, 1024)])
@pytest.mark.parametrize("name", sorted(SEGMENTS))
def test_product(name, n, k, exact):
    rows = SEGMENTS[name]
    rng = np.random.default_rng(n + k)
    num_rows = sum(rows) + 5  # some rows behind the last segment
    print(f"[product] {name} n={n} k={k} exact={exact}", flush=True)
    x, xs, w, ws = _inputs(rng, len(rows), n, k, num_rows, exact)
    got, status = _product(len(rows), n, k, x, xs, w, ws, rows, num_rows)
    want, mag = oracle64.product(x, xs, w, ws, rows, num_rows)
    _check_product(got, want, mag, k, exact, None if exact else oracle64.product_cut(x, xs, w, ws, rows, num_rows))
    assert status == 0


@pytest.mark.parametrize("rows,E", [(1, 300), (64, 300), (513, 65)])
def test_product_many_experts(rows, E):
    """More experts than a wave has lanes, most of them without rows."""
    rng = np.random.default_rng(rows)
    sizes = rng.multinomial(rows, np.ones(E) / E)
    x, xs, w, ws = _inputs(rng, E, 136, 128, rows, True)
    got, status = _product(E, 136, 128, x, xs, w, ws, sizes, rows)
    want, mag = oracle64.product(x, xs, w, ws, sizes, rows)
    _check_product(got, want, mag, 128, True)
    assert status == 0


# (experts, rows, n, k): every kernel of the product (16 rows by 16 and 64 columns, 32 rows by 64 and 128, 128 and
# 256 rows a block) and of the SwiGLU form (16, 32, 64 and 128 rows a block); the last ones give every wave that shares
# the channels several blocks of them
KERNELS = [(1, 3, 256, 640), (3, 90, 256, 640), (40, 130, 1024, 384), (70, 100, 2048, 128), (6, 700, 2048, 256),
           (3, 900, 1024, 128), (2, 1300, 8192, 128), (1, 4400, 2048, 128), (40, 700, 2048, 384),
           (1, 20, 256, 4096), (2, 40, 2048, 2176), (2, 300, 2048, 2304)]


@pytest.mark.parametrize("case", KERNELS, ids=str)
@pytest.mark.parametrize("exact", [True, False])
def test_each_kernel(case, exact):
    """Both outputs, segments uneven around their mean, some empty."""
    E, rows, n, k = case
    rng = np.random.default_rng(rows)
    print(f"[product] kernels {case} exact={exact}", flush=True)
    share = rng.random(E) * (rng.random(E) < 0.8) + 1e-9
    sizes = rng.multinomial(rows, share / share.sum())
    x, xs, w, ws = _inputs(rng, E, n, k, rows, exact)
    got, status = _product(E, n, k, x, xs, w, ws, sizes, rows)
    want, mag = oracle64.product(x, xs, w, ws, sizes, rows)
    if exact:
        _check_product(got, want, mag, k, True)
    else:  # the cut is measured for the first rows and the last alone: it is k / 8 products of the whole
        at = np.r_[0:min(rows, 20), max(rows - 20, 0):rows]
        ends = np.cumsum(sizes)
        owner = np.searchsorted(ends, at, side="right")
        cut = np.stack([oracle64.product_cut(x[r:r + 1], xs[r:r + 1], w[e:e + 1], ws[e:e + 1], [1], 1)[0]
                        for r, e in zip(at, owner)])
        _check_product(got[torch.from_numpy(at).cuda()], want[at], mag[at], k, False, cut)
    assert status == 0
    if exact:
        xs, want = xs / 64, want / 64
    n //= 2
    codes, scales, _ = _product(E, n, k, x, xs, w, ws, sizes, rows, swiglu=True)
    slack = np.zeros_like(want) if exact else (2 * (k + k // 128) + 2) * U * mag
    _check_swiglu(codes, scales, want, slack, np.ones(rows, bool))


def test_odd_numbers_of_blocks_of_channels():
    rng = np.random.default_rng(30)
    for k in (128, 256, 384, 512, 1152):
        for sizes in ([5], [20], [200]):
            x, xs, w, ws = _inputs(rng, 1, 256, k, sizes[0], True)
            got, _ = _product(1, 256, k, x, xs, w, ws, sizes, sizes[0])
            want, mag = oracle64.product(x, xs, w, ws, sizes, sizes[0])
            _check_product(got, want, mag, k, True)
            xs = xs / 64
            codes, scales, _ = _product(1, 128, k, x, xs, w, ws, sizes, sizes[0], swiglu=True)
            _check_swiglu(codes, scales, want / 64, np.zeros_like(want), np.ones(sizes[0], bool))


def test_dense_product_needs_no_sizes():
    rng = np.random.default_rng(9)
    for rows in (1, 15, 130, 300):
        x, xs, w, ws = _inputs(rng, 1, 392, 640, rows, True)
        got, _ = _product(1, 392, 640, x, xs, w, ws, None, rows)
        want, mag = oracle64.product(x, xs, w, ws, [rows], rows)
        _check_product(got, want, mag, 640, True)


def test_sizes_that_pass_the_buffers_or_are_negative():
    rng = np.random.default_rng(10)
    for rows, over in (([10, -3, 20], 0), ([10, 60, 20], ep.EP_DEV_RECV_OVERFLOW), ([2147483647] * 3, ep.EP_DEV_RECV_OVERFLOW),
                       ([0, 0, 51], ep.EP_DEV_RECV_OVERFLOW), ([50, 0, 0], 0), ([-2147483648] * 3, 0)):
        x, xs, w, ws = _inputs(rng, 3, 264, 256, 50, True)
        got, status = _product(3, 264, 256, x, xs, w, ws, rows, 50)
        want, mag = oracle64.product(x, xs, w, ws, rows, 50)
        _check_product(got, want, mag, 256, True)
        assert status == over
        codes, scales, status = _product(3, 256, 256, x, xs, torch.cat([w, w], 1)[:, :512], np.concatenate([ws, ws], 1)[:, :4],
                                         rows, 50, swiglu=True)
        assert status == over
        untouched = np.isnan(want[:, 0])
        assert np.all(codes.cpu().numpy()[untouched] == 0xAB) and np.all(scales[untouched] == -2.0)
        assert not np.any(scales[~untouched] == -2.0)


def test_nan_codes_stay_in_their_row_and_column():
    rng = np.random.default_rng(12)
    x, xs, w, ws = _inputs(rng, 1, 264, 256, 40, True)
    x[3, 200] = 0x7F
    w[0, 17, 5] = 0xFF
    got, _ = _product(1, 264, 256, x, xs, w, ws, [40], 40)
    bad = np.isnan(_values(got))
    assert bad[3].all() and bad[:, 17].all() and bad.sum() == 264 + 40 - 1


def test_rows_behind_the_last_segment_are_not_read_into_results():
    """NaN codes and scales in the rows behind the segments, and in the rows of other segments."""
    rng = np.random.default_rng(13)
    sizes = [7, 3, 20]
    x, xs, w, ws = _inputs(rng, 3, 128, 128, 64, True)
    x[30:] = 0x7F
    xs[30:] = np.nan
    x[7:10] = 0x7F
    got, _ = _product(3, 128, 128, x, xs, w, ws, sizes, 64)
    v = _values(got)[:30]
    assert np.isnan(v[7:10]).all() and np.isfinite(np.delete(v, [7, 8, 9], 0)).all()


def _check_swiglu(codes, scales, gate_up, slack, rows):
    """slack: how far gate and up may be off, in the shape of gate_up."""
    n = gate_up.shape[1] // 2
    a = oracle64.swiglu(gate_up[rows])
    g, u = np.abs(gate_up[rows][:, :n]), np.abs(gate_up[rows][:, n:])
    dg, du = slack[rows][:, :n], slack[rows][:, n:]
    # silu's slope is below 1.1 and silu(g) below |g| in magnitude; an exponential, a sum, a quotient and a product: 8 U
    da = 1.1 * dg * (u + du) + g * du + 8 * U * np.abs(a)
    blocks = a.reshape(a.shape[0], n // 128, 128)
    top = np.maximum(np.abs(blocks).max(2), 2.0 ** -64)
    dtop = da.reshape(blocks.shape).max(2)
    assert np.all(np.abs(scales[rows] - top / 448) <= (dtop + 2 * U * top) / 448)
    got = oracle64.e4m3_values(codes)[rows] * np.repeat(scales[rows].astype(np.float64), 128, 1)
    # half a step of the code: 2^-4 of the value (counting the step from the value's own size), or
    # 2^-10 of the scale for the smallest; the quotient, product and clamp before it: 4 U
    s = np.repeat(scales[rows].astype(np.float64), 128, 1)
    tol = oracle64.E4M3_HALF * (np.abs(a) + da) + 2.0 ** -10 * s + da + 4 * U * np.abs(a) + np.repeat(dtop, 128, 1) * E4M3_EDGE
    assert np.all(np.abs(got - a) <= tol)


E4M3_EDGE = 1.0 + 2.0 ** -4  # a value at the edge of the range moves with the block's largest


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("n,k", [(128, 128), (256, 384), (640, 256)])
@pytest.mark.parametrize("name", sorted(SEGMENTS))
def test_swiglu(name, n, k, exact):
    sizes = SEGMENTS[name]
    rng = np.random.default_rng(n * k)
    num_rows = sum(sizes) + 3
    print(f"[swiglu] {name} n={n} k={k} exact={exact}", flush=True)
    x, xs, w, ws = _inputs(rng, len(sizes), 2 * n, k, num_rows, exact)
    if exact:  # values small enough that the activation is neither linear nor zero
        xs /= 64
    codes, scales, status = _product(len(sizes), n, k, x, xs, w, ws, sizes, num_rows, swiglu=True)
    want, mag = oracle64.product(x, xs, w, ws, sizes, num_rows)
    rows = ~np.isnan(want[:, 0])
    slack = np.zeros_like(want) if exact else (2 * (k + k // 128) + 2) * U * mag
    _check_swiglu(codes, scales, want, slack, rows)
    assert np.all(codes.cpu().numpy()[~rows] == 0xAB) and np.all(scales[~rows] == -2.0)
    assert status == 0


def test_swiglu_extremes():
    """Gates far below and above zero, and rows of zeros: no NaN, the smallest scale."""
    E, n, k = 1, 128, 128
    x = torch.zeros(4, k, dtype=torch.uint8)
    x[:3, 0] = 0x38  # 1.0
    w = torch.zeros(1, 2 * n, k, dtype=torch.uint8)
    w[0, :n, 0] = torch.from_numpy(np.full(n, 448.0, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
    w[0, n:, 0] = 0x38
    ws = np.ones((1, 2, 1), np.float32)
    xs = np.array([[1.0], [-1.0], [-1e30], [1.0]], np.float32)
    codes, scales, _ = _product(E, n, k, x, xs, w, ws, [4], 4, swiglu=True)
    v = oracle64.e4m3_values(codes) * np.repeat(scales.astype(np.float64), 128, 1)
    assert np.isfinite(v).all()
    assert np.allclose(v[0], 448.0, rtol=2.0 ** -4) and np.all(np.abs(v[1]) < 1e-100) and np.all(v[2:] == 0.0)
    assert np.all(scales[1:] == np.float32(2.0 ** -64 / 448))


def test_input_gradient_is_the_product_with_transposed_weights():
    """dX = (dY per block of 128, quantised) times the transposed codes with transposed block scales."""
    rng = np.random.default_rng(21)
    E, N, K, rows = 3, 256, 384, [20, 0, 33]
    M = sum(rows)
    _, _, w, ws = _inputs(rng, E, N, K, M, False)
    dy = rng.standard_normal((M, N)).astype(np.float32)
    d = to_dev_bf16((torch.from_numpy(dy).to(torch.bfloat16).view(torch.int16).numpy()).view(np.uint16))
    codes = torch.empty(M, N, dtype=torch.uint8, device="cuda")
    scales = torch.empty(M, N // 128, device="cuda")
    ep.ep_quantize_fp8(d, M, N, N // 128, codes, scales)
    wt, wst = w.transpose(1, 2).contiguous(), np.ascontiguousarray(ws.transpose(0, 2, 1))
    got, _ = _product(E, K, N, codes.cpu(), scales.cpu().numpy(), wt, wst, rows, M)
    want, mag = oracle64.product(codes.cpu(), scales.cpu().numpy(), wt, wst, rows, M)
    _check_product(got, want, mag, N, False, oracle64.product_cut(codes.cpu(), scales.cpu().numpy(), wt, wst, rows, M))
    # and against the gradient of sum(dY * (X W^T)) written out: dX[m][i] = sum_c dY[m][c] W[c][i], dY within half a step
    at = 0
    for e, n in enumerate(rows):
        wv = oracle64.e4m3_values(w[e]) * np.repeat(np.repeat(ws[e].astype(np.float64), 128, 0), 128, 1)
        seg = slice(at, at + n)
        dyv = d.double().cpu().numpy()[seg]
        step = oracle64.E4M3_HALF * np.abs(dyv) + 2.0 ** -10 * np.repeat(scales.cpu().numpy()[seg].astype(np.float64), 128, 1)
        tol = 1.01 * step @ np.abs(wv) + 2.0 ** -7 * np.abs(dyv) @ np.abs(wv)
        assert np.all(np.abs(_values(got)[seg] - dyv @ wv) <= tol)
        at += n
