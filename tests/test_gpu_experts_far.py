"""The expert-layer calls on buffers whose offsets pass 32 bits: a sample of rows against the same
rows in a small call or against sums that are exact, and nothing written elsewhere."""
import numpy as np
import pytest
import torch

from combine_ep_get_02_amd import ep, experts

pytestmark = pytest.mark.gpu
CODES = torch.tensor([0xC0, 0xB8, 0x00, 0x38, 0x40], dtype=torch.uint8)  # E4M3 of -2 .. 2
VALUES = torch.tensor([-2.0, -1.0, 0.0, 1.0, 2.0], dtype=torch.float64)


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def _sample(rng, rows, count=64):
    """Sorted rows, the first and the last among them."""
    at = np.unique(np.concatenate([[0, rows - 1], rng.integers(0, rows, size=count)]))
    return torch.from_numpy(at).cuda()


def _draw(rng, shape):
    pick = torch.from_numpy(rng.integers(0, 5, size=shape))
    return CODES[pick], VALUES[pick]


@pytest.mark.parametrize("rows,n,k", [((1 << 22) + 333, 8, 1024), ((1 << 20) + 77, 4096, 128)])
def test_product_rows(rows, n, k):
    assert rows * max(k, n) > 1 << 32
    rng = np.random.default_rng(1)
    at = _sample(rng, rows)
    codes, values = _draw(rng, (len(at), k))
    wcodes, wvalues = _draw(rng, (n, k))
    x = torch.zeros((rows, k), dtype=torch.uint8, device="cuda")
    x[at] = codes.cuda()
    xs = torch.full((rows, k // 128), 0.5, device="cuda")
    ws = torch.full((-(-n // 128), k // 128), 2.0, device="cuda")
    out = torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    experts.ep_expert_gemm_fp8(1, n, k, x, xs, wcodes.cuda(), ws, None, rows, out)
    # sums of k products of integers up to 4 are exact in f32: one rounding to bf16
    want = (values @ wvalues.T).to(torch.float32).to(torch.bfloat16)
    assert torch.equal(out[at].cpu(), want)
    out[at] = 0
    assert not out.any()


@pytest.mark.parametrize("swiglu", [False, True])
def test_experts_weights(swiglu):
    E, n, k = 300, 2048, 4096
    wide = 2 * n if swiglu else 2 * n + 8
    assert E * wide * k > 1 << 32
    rng = np.random.default_rng(2)
    sizes = np.zeros(E, np.int32)
    sizes[[0, 100, 256, 299]] = 3, 20, 1, 40
    rows = int(sizes.sum())
    codes, values = _draw(rng, (rows, k))
    w = torch.zeros((E, wide, k), dtype=torch.uint8, device="cuda")
    ws = torch.ones((E, -(-wide // 128), k // 128), device="cuda")
    xs = torch.full((rows, k // 128), 2.0 ** -6, device="cuda")
    drawn = {int(e): _draw(rng, (wide, k)) for e in np.flatnonzero(sizes)}
    for e, (wc, _) in drawn.items():
        w[e] = wc.cuda()
    x, sized = codes.cuda(), torch.from_numpy(sizes).cuda()
    if swiglu:
        out = torch.zeros((rows, n), dtype=torch.uint8, device="cuda")
        outs = torch.zeros((rows, n // 128), device="cuda")
        experts.ep_expert_gemm_swiglu_fp8(E, n, k, x, xs, w, ws, sized, rows, out, outs)
        got = out.view(torch.float8_e4m3fn).double().cpu() * outs.double().cpu().repeat_interleave(128, dim=1)
    else:
        out = torch.zeros((rows, wide), dtype=torch.bfloat16, device="cuda")
        experts.ep_expert_gemm_fp8(E, wide, k, x, xs, w, ws, sized, rows, out)
    first = 0
    for e, (_, wv) in drawn.items():
        here = slice(first, first + int(sizes[e]))
        first = here.stop
        product = values[here] @ wv.T * 2.0 ** -6
        if not swiglu:
            assert torch.equal(out[here].cpu(), product.to(torch.float32).to(torch.bfloat16))
            continue
        gate, up = product[:, :n], product[:, n:]
        want = gate / (1 + torch.exp(-gate)) * up
        top = want.abs().reshape(-1, n // 128, 128).amax(2).repeat_interleave(128, dim=1)
        # half a step of E4M3 relative to the value (2^-4), or half its least code (2^-10 of top / 448);
        # the f32 of the activation, the scale and its inverse are far below the spare 2^-12 of the value
        assert bool(((got[here] - want).abs() <= (2.0 ** -4 + 2.0 ** -12) * want.abs() + top * 2.0 ** -10 / 448 * 1.01).all())


@pytest.mark.parametrize("rows,n,k", [((1 << 22) + 333, 128, 1024), ((1 << 20) + 77, 4096, 128)])
def test_swiglu_rows(rows, n, k):
    assert rows * max(k, n) > 1 << 32
    rng = np.random.default_rng(3)
    at = _sample(rng, rows)
    codes, _ = _draw(rng, (len(at), k))
    wcodes, _ = _draw(rng, (2 * n, k))
    w, ws = wcodes.cuda(), torch.ones((2 * n // 128, k // 128), device="cuda")
    x = torch.zeros((rows, k), dtype=torch.uint8, device="cuda")
    x[at] = codes.cuda()
    out = torch.full((rows, n), 0xAB, dtype=torch.uint8, device="cuda")
    outs = torch.full((rows, n // 128), -2.0, device="cuda")
    experts.ep_expert_gemm_swiglu_fp8(1, n, k, x, torch.full((rows, k // 128), 0.25, device="cuda"), w, ws, None, rows,
                                      out, outs)
    few, fews = torch.empty((len(at), n), dtype=torch.uint8, device="cuda"), torch.empty((len(at), n // 128), device="cuda")
    experts.ep_expert_gemm_swiglu_fp8(1, n, k, codes.cuda(), torch.full((len(at), k // 128), 0.25, device="cuda"), w, ws,
                                      None, len(at), few, fews)
    assert torch.equal(out[at], few) and torch.equal(outs[at], fews)
    out[at], outs[at] = 0, 2.0 ** -64 / 448  # a block of zeros has the floor's scale
    assert not out.any() and bool((outs == outs[0, 0]).all())


def test_route_rows():
    T, E, k = 2_097_200, 2048, 8
    assert T * E > 1 << 32
    rng = np.random.default_rng(4)
    at = _sample(rng, T)
    shape, few = ep.make_shape(T, 8, k, E, 1, 1), ep.make_shape(len(at), 8, k, E, 1, 1)
    r = experts.make_router(experts.EP_SCORE_SOFTMAX, 8, 4, 2, True, 2.5)
    logits = torch.empty((T, E), dtype=torch.bfloat16, device="cuda").normal_()
    idx, w = torch.empty((T, k), dtype=torch.int64, device="cuda"), torch.empty((T, k), device="cuda")
    experts.ep_route(shape, r, logits, None, None, idx, w)
    sample = logits[at]
    idx2, w2 = torch.empty((len(at), k), dtype=torch.int64, device="cuda"), torch.empty((len(at), k), device="cuda")
    experts.ep_route(few, r, sample, None, None, idx2, w2)
    assert torch.equal(idx[at], idx2) and torch.equal(w[at], w2)
    grad_w = torch.randn((T, k), device="cuda")
    grad = torch.full((T, E), float("nan"), dtype=torch.bfloat16, device="cuda")
    experts.ep_route_backward(shape, r, logits, idx, grad_w, grad)
    grad2 = torch.empty((len(at), E), dtype=torch.bfloat16, device="cuda")
    experts.ep_route_backward(few, r, sample, idx2, grad_w[at], grad2)
    assert torch.equal(grad[at], grad2) and not grad[T // 2:].isnan().any() and not grad[:T // 2].isnan().any()


def test_combine_rows():
    """Outputs and gradients of a few tokens whose rows are spread over 9 GiB of grouped rows."""
    T, H, K, E, R, rows = 300, 16384, 4, 8, 2, 280_000
    assert rows * H > 1 << 32
    rng = np.random.default_rng(5)
    idx = torch.from_numpy(np.stack([rng.choice(E, K, replace=False) for _ in range(T)]))
    pos = torch.from_numpy(np.concatenate([[0, rows - 1], rng.choice(np.arange(1, rows - 1), T * K - 2, replace=False)]).reshape(T, K))
    send_slot = torch.arange(T).reshape(T, 1).repeat(1, R).to(torch.int32).cuda()  # receive row t, for either rank
    weights = torch.from_numpy(rng.integers(1, 5, (T, K)).astype(np.float32))
    values = torch.from_numpy(rng.integers(-3, 4, (T, K, H)).astype(np.float32))
    grads = torch.from_numpy(rng.integers(-3, 4, (T, H)).astype(np.float32))
    shape = ep.make_shape(T, H, K, E, R, 1)
    y = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
    y[pos.reshape(-1).cuda()] = values.reshape(-1, H).to(torch.bfloat16).cuda()
    maps = (idx.cuda(), weights.cuda(), send_slot, pos.to(torch.int32).cuda())
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    experts.ep_combine_grouped(shape, y, *maps, T, rows, out, status)
    want = (values * weights[:, :, None]).sum(1)  # integers up to 48: exact in f32 and bf16
    assert torch.equal(out.float().cpu(), want)
    # row 1 and row rows - 2 are padding, the others not named are rows of other tokens: left alone
    owner = torch.zeros(rows, dtype=torch.int32)
    free = [r for r in (1, 2, rows - 2, rows - 3) if not bool((pos == r).any())]
    owner[free] = -1
    gy = torch.full((rows, H), 7.0, dtype=torch.bfloat16, device="cuda")
    gw = torch.full((T, K), float("nan"), device="cuda")
    experts.ep_combine_grouped_backward(shape, grads.to(torch.bfloat16).cuda(), y, *maps, owner.cuda(),
                                        torch.tensor([rows], dtype=torch.int32, device="cuda"), T, rows, gy, gw, status)
    assert torch.equal(gw.cpu(), (values * grads[:, None, :]).sum(2))  # integers up to 9 * 16384: exact
    assert torch.equal(gy[pos.reshape(-1).cuda()].float().cpu(), (weights[:, :, None] * grads[:, None, :]).reshape(-1, H))
    assert free and not gy[torch.tensor(free).cuda()].any()
    gy[pos.reshape(-1).cuda()] = 7.0
    gy[torch.tensor(free).cuda()] = 7.0
    assert bool((gy == 7.0).all()) and int(status.item()) == 0
