"""The combine of grouped rows and its gradient against their definitions in binary64."""
import numpy as np
import pytest
import torch

import experts_oracle as oracle64
from combine_ep_get_02_amd import ep, experts
from gpu_harness import bf16_host

pytestmark = pytest.mark.gpu
U = oracle64.U


def _placed(rng, T, E, R, K, masked, align, duplicates=False):
    """A routing and the library's own grouping of it: (b, g-like tensors, idx, weights)."""
    idx = np.stack([rng.choice(E, K, replace=duplicates) for _ in range(T)]).astype(np.int64).reshape(T, K)
    idx[rng.random((T, K)) < masked] = -1
    return idx, rng.random((T, K)).astype(np.float32) * (idx >= 0)


def _group(idx, w, H, E, R, align, slack=0):
    T, K = idx.shape
    shape = ep.make_shape(T, H, K, E, R, 4, expert_alignment=align)
    didx, dw = torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda()
    probe = ep.allocate(shape, 0)
    n = ep.run_layout_notify(probe, didx, read_back=True)
    b = ep.allocate(shape, n + slack)
    ep.run_layout_notify(b, didx)
    cap = int(b.recv_per_expert.sum().item()) + slack
    g = ep.allocate_group(b, cap)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    ep.run_dispatch_grouped(b, g, x, didx, dw)
    torch.cuda.synchronize()
    return shape, b, g, didx, dw


def _bf16(rng, shape, exact):
    v = rng.integers(-4, 5, size=shape) if exact else rng.standard_normal(shape)
    return torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16)


CASES = [  # T, H, K, E, R, masked, align, slack
    (1, 8, 1, 1, 1, 0.0, 1, 0), (1, 7168, 8, 256, 16, 0.0, 1, 0), (17, 264, 3, 12, 4, 0.3, 1, 2),
    (64, 256, 2, 16, 8, 0.0, 4, 0), (130, 1032, 8, 64, 64, 0.5, 16, 7), (33, 520, 32, 64, 8, 0.1, 1, 0),
    (300, 4096, 6, 64, 16, 0.0, 1, 3), (40, 8192, 4, 8, 2, 0.2, 128, 0), (9, 16392, 2, 8, 8, 0.0, 1, 0),
    (5, 64, 4, 8, 8, 1.0, 1, 4),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("exact", [True, False])
def test_combine_and_gradient(case, exact):
    T, H, K, E, R, masked, align, slack = case
    rng = np.random.default_rng(T + H)
    print(f"[combine grouped] {case} exact={exact}", flush=True)
    idx, w = _placed(rng, T, E, R, K, masked, align)
    if exact:  # powers of two: every sum is exact
        w = (2.0 ** rng.integers(-3, 1, size=w.shape) * (idx >= 0)).astype(np.float32)
    shape, b, g, didx, dw = _group(idx, w, H, E, R, align, slack)
    y = _bf16(rng, (g.capacity, H), exact)
    dy = y.cuda()
    out = torch.full((T + 1, H), -1, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    experts.ep_combine_grouped(shape, dy, didx, dw, b.send_slot, g.slot_pos, b.capacity, g.capacity, out, status)
    torch.cuda.synchronize()
    pos = oracle64.positions(idx, b.send_slot.cpu().numpy(), g.slot_pos.cpu().numpy(), E, R, b.capacity, g.capacity)
    assert np.array_equal(pos >= 0, idx >= 0)
    yv = y.double().numpy()
    want, mag = oracle64.combine(yv, w, pos)
    got = out[:T].double().cpu().numpy()
    if exact:
        assert np.array_equal(got, oracle64.bf16_round(want))
    else:  # K fused steps of half a step each, and the rounding
        assert np.all(np.abs(got - want) <= oracle64.BF16_HALF * np.abs(want) + 2 * K * U * mag)
    assert np.all(bf16_host(out[T]) == 0xFFFF) and int(status.item()) == 0

    grad = _bf16(rng, (T, H), exact)
    gy = torch.full((g.capacity + 1, H), -1, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    gw = torch.full((T + 1, K), -3.0, device="cuda")
    experts.ep_combine_grouped_backward(shape, grad.cuda(), dy, didx, dw, b.send_slot, g.slot_pos, g.grouped_row,
                                        g.num_grouped, b.capacity, g.capacity, gy, gw, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    used = int(g.num_grouped.item())
    want_gy = np.zeros((used, H))
    gv = grad.double().numpy()
    want_gw, mag_gw = np.zeros((T, K)), np.zeros((T, K))
    for t, j in zip(*np.nonzero(pos >= 0)):
        want_gy[pos[t, j]] = oracle64.bf16_round(w[t, j] * grad[t].float().numpy())  # one product, one rounding
        want_gw[t, j] = yv[pos[t, j]] @ gv[t]
        mag_gw[t, j] = np.abs(yv[pos[t, j]]) @ np.abs(gv[t])
    assert np.array_equal(gy[:used].double().cpu().numpy(), want_gy)  # padding rows are zeros
    assert np.all(bf16_host(gy[used:]) == 0xFFFF)
    got_gw = gw[:T].double().cpu().numpy()
    assert np.all(np.abs(got_gw - want_gw) <= (0 if exact else H * U * mag_gw))
    assert np.all(got_gw[pos < 0] == 0.0)
    assert bool((gw[T] == -3.0).all())


def test_gradient_against_differences():
    """d sum(grad * out) / d weight and / d y, by differences of the definition in binary64."""
    rng = np.random.default_rng(8)
    T, H, K, E, R = 6, 16, 3, 8, 4
    idx, w = _placed(rng, T, E, R, K, 0.2, 1)
    shape, b, g, didx, dw = _group(idx, w, H, E, R, 2)
    y, grad = _bf16(rng, (g.capacity, H), False), _bf16(rng, (T, H), False)
    gy = torch.zeros(g.capacity, H, dtype=torch.bfloat16, device="cuda")
    gw = torch.empty(T, K, device="cuda")
    experts.ep_combine_grouped_backward(shape, grad.cuda(), y.cuda(), didx, dw, b.send_slot, g.slot_pos, g.grouped_row,
                                        g.num_grouped, b.capacity, g.capacity, gy, gw)
    pos = oracle64.positions(idx, b.send_slot.cpu().numpy(), g.slot_pos.cpu().numpy(), E, R, b.capacity, g.capacity)
    yv, gv, wv = y.double().numpy(), grad.double().numpy(), w.astype(np.float64)
    value = lambda y_, w_: (oracle64.combine(y_, w_, pos)[0] * gv).sum()  # noqa: E731
    h = 2.0 ** -10
    for t in range(T):
        for j in range(K):
            up, down = wv.copy(), wv.copy()
            up[t, j] += h
            down[t, j] -= h
            d = (value(yv, up) - value(yv, down)) / (2 * h)
            assert abs(gw[t, j].item() - d) <= 1e-5  # linear: 16 f32 steps of values below 20, rounding of the differences
    for r in range(g.capacity):
        for i in (0, 7, 15):
            up, down = yv.copy(), yv.copy()
            up[r, i] += h
            down[r, i] -= h
            d = (value(up, wv) - value(down, wv)) / (2 * h)
            assert abs(gy[r, i].item() - d) <= oracle64.BF16_HALF * abs(d) + 1e-9


def test_bad_entries_are_skipped_and_flagged():
    rng = np.random.default_rng(14)
    T, H, K, E, R = 12, 64, 4, 16, 4
    idx, w = _placed(rng, T, E, R, K, 0.0, 1)
    shape, b, g, didx, dw = _group(idx, w, H, E, R, 1)
    y, grad = _bf16(rng, (g.capacity, H), True), _bf16(rng, (T, H), True)
    slot, sp = b.send_slot.clone(), g.slot_pos.clone()
    row = int(slot[3, idx[3, 1] // (E // R)].item())

    def check(idx_, slot_, sp_, bits):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        di = torch.from_numpy(idx_).cuda()
        experts.ep_combine_grouped(shape, y.cuda(), di, dw, slot_, sp_, b.capacity, g.capacity, out, status)
        assert int(status.item()) == bits
        pos = oracle64.positions(idx_, slot_.cpu().numpy(), sp_.cpu().numpy(), E, R, b.capacity, g.capacity)
        want, mag = oracle64.combine(y.double().numpy(), w, pos)
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= oracle64.BF16_HALF * np.abs(want) + 2 * K * U * mag)
        status.zero_()
        gy = torch.zeros(g.capacity, H, dtype=torch.bfloat16, device="cuda")
        gw = torch.empty(T, K, device="cuda")
        experts.ep_combine_grouped_backward(shape, grad.cuda(), y.cuda(), di, dw, slot_, sp_, g.grouped_row,
                                            g.num_grouped, b.capacity, g.capacity, gy, gw, status)
        assert int(status.item()) == bits
        assert np.all(gw.cpu().numpy()[pos < 0] == 0.0) and (pos < 0).any()

    for value in (E, -2, 1 << 40, -(1 << 40)):
        bad = idx.copy()
        bad[3, 1] = value
        check(bad, slot, sp, ep.EP_DEV_BAD_TOPK_IDX)
    for value in (b.capacity, -2, 2147483647, -2147483648):
        s2 = slot.clone()
        s2[3, idx[3, 1] // (E // R)] = value
        check(idx, s2, sp, ep.EP_DEV_BAD_SEND_SLOT)
    for value in (g.capacity, -2, 2147483647, -2147483648):
        p2 = sp.clone()
        p2[row, 1] = value
        check(idx, slot, p2, ep.EP_DEV_BAD_SEND_SLOT)
    p2 = sp.clone()
    p2[row, 1] = -1  # dropped by the grouping: no flag
    check(idx, slot, p2, 0)


def test_an_expert_twice_in_a_token():
    """The grouping gives each slot a row of its own, and so does the combine."""
    rng = np.random.default_rng(15)
    T, H, K, E, R = 20, 72, 4, 8, 4
    idx, w = _placed(rng, T, E, R, K, 0.0, 1, duplicates=True)
    idx[0] = 5
    shape, b, g, didx, dw = _group(idx, w, H, E, R, 1)
    y = _bf16(rng, (g.capacity, H), False)
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    experts.ep_combine_grouped(shape, y.cuda(), didx, dw, b.send_slot, g.slot_pos, b.capacity, g.capacity, out)
    pos = oracle64.positions(idx, b.send_slot.cpu().numpy(), g.slot_pos.cpu().numpy(), E, R, b.capacity, g.capacity)
    assert len(set(pos.reshape(-1).tolist())) == T * K
    want, mag = oracle64.combine(y.double().numpy(), w, pos)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= oracle64.BF16_HALF * np.abs(want) + 2 * K * U * mag)


def test_rows_that_are_not_placed_are_not_read():
    """NaN in padding rows, in rows behind the last and under dropped slots never reaches an output."""
    rng = np.random.default_rng(16)
    T, H, K, E, R = 30, 128, 4, 8, 2
    idx, w = _placed(rng, T, E, R, K, 0.3, 16)
    shape, b, g, didx, dw = _group(idx, w, H, E, R, 16, slack=9)
    y = _bf16(rng, (g.capacity, H), True)
    placed = (g.grouped_row >= 0).cpu()
    placed[int(g.num_grouped.item()):] = False
    y[~placed] = float("nan")
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    experts.ep_combine_grouped(shape, y.cuda(), didx, dw, b.send_slot, g.slot_pos, b.capacity, g.capacity, out)
    assert bool(out.isfinite().all())
    gy = torch.full((g.capacity, H), 1.0, dtype=torch.bfloat16, device="cuda")
    gw = torch.empty(T, K, device="cuda")
    experts.ep_combine_grouped_backward(shape, _bf16(rng, (T, H), True).cuda(), y.cuda(), didx, dw, b.send_slot, g.slot_pos,
                                        g.grouped_row, g.num_grouped, b.capacity, g.capacity, gy, gw)
    assert bool(gw.isfinite().all()) and bool(gy.isfinite().all())


def test_no_tokens_and_padding_alone():
    shape = ep.make_shape(0, 64, 4, 8, 2, 1, expert_alignment=8)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    e64, f32 = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    bf = torch.empty(0, dtype=torch.bfloat16, device="cuda")
    experts.ep_combine_grouped(shape, bf, e64, f32, e, e, 0, 0, bf)
    for rows in (1, 24, 5000):
        gy = torch.full((rows, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        grouped_row = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        n = torch.tensor([max(rows - 1, 1)], dtype=torch.int32, device="cuda")
        experts.ep_combine_grouped_backward(shape, bf, bf, e64, f32, e, e, grouped_row, n, 0, rows, gy, f32)
        assert not gy[:int(n.item())].any() and bool((gy[int(n.item()):] == 3.0).all())
