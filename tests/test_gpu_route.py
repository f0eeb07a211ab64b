"""The router and its gradient against their definitions in binary64."""
import itertools

import numpy as np
import pytest
import torch

import experts_oracle as oracle64
from combine_ep_get_02_amd import ep, experts

pytestmark = pytest.mark.gpu
KINDS = {"sigmoid": experts.EP_SCORE_SIGMOID, "softmax": experts.EP_SCORE_SOFTMAX}
U = oracle64.U


def _logits(rng, T, E, dtype):
    """Values as the type holds them, and the tensor."""
    t = torch.from_numpy((rng.standard_normal((T, E)) * 1.5).astype(np.float32)).to(dtype)
    return t.to(torch.float32).numpy(), t.cuda()


def _route(logits, bias, kind, k, groups=1, kept=1, best=1, renorm=True, scale=1.0, mask=None, ranks=1):
    T, E = logits.shape
    shape = ep.make_shape(T, 8, k, E, ranks, 1)
    r = experts.make_router(KINDS[kind], groups, kept, best, renorm, scale)
    idx = torch.full((T + 1, k), -777, dtype=torch.int64, device="cuda")
    w = torch.full((T + 1, k), -3.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    experts.ep_route(shape, r, logits, bias, mask, idx[:T], w[:T], status)
    torch.cuda.synchronize()
    assert bool((idx[T] == -777).all()) and bool((w[T] == -3.0).all())
    return idx[:T].cpu().numpy(), w[:T].cpu().numpy(), int(status.item())


def _weights_near(got, want, kind, renorm):
    # numerators and their sum are formed in 64 bits and rounded once (a step is 2 U, half of it U).
    # A softmax that is not renormalised also divides by a sum of E 32-bit exponentials: an
    # exponential of d <= 0 is off by (|d| + 4) U, the terms' weights average |d| + 4 to under 16
    # here, and a tree over up to 2048 terms (32 in a lane, 6 steps across) adds at most 38 U.
    tol = 2 * U if kind == "sigmoid" or renorm else 56 * U
    assert np.all(np.abs(got - want) <= tol * np.abs(want) + 1e-44)


@pytest.mark.parametrize("E", [1, 2, 5, 16, 60, 64, 65, 128, 160, 256, 384, 1000, 2048])
@pytest.mark.parametrize("kind,dtype,renorm", [("sigmoid", torch.float32, True), ("softmax", torch.bfloat16, False),
                                               ("softmax", torch.float32, True)])
def test_choice_and_weights(E, kind, dtype, renorm):
    rng = np.random.default_rng(E)
    k = min(8, E)
    for T, with_bias in ((1, False), (37, True), (130, False)):
        print(f"[route] E={E} {kind} {dtype} T={T} bias={with_bias}", flush=True)
        values, logits = _logits(rng, T, E, dtype)
        bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if with_bias else None
        got_i, got_w, status = _route(logits, None if bias is None else torch.from_numpy(bias).cuda(), kind, k,
                                      renorm=renorm, scale=1.0 if renorm else 2.5)
        want_i, want_w = oracle64.route(values, bias, kind, k, 1, 1, 1, renorm, 1.0 if renorm else 2.5)
        assert np.array_equal(got_i, want_i)
        _weights_near(got_w, want_w, kind, renorm)
        assert status == 0


# 4096 tokens and more go 16 lanes to a token, where they hold its experts (128), slots (16) and groups (16), or 32
# (256 experts)
MANY = [(16, 2, 1, 1), (60, 6, 1, 1), (64, 6, 8, 3), (65, 4, 5, 2), (128, 8, 16, 5), (160, 8, 8, 3), (192, 3, 6, 2),
        (256, 8, 8, 4), (256, 16, 16, 16), (256, 17, 4, 2), (256, 8, 32, 9), (257, 8, 1, 1), (12, 16, 3, 2)]


@pytest.mark.parametrize("E,k,groups,kept", MANY)
@pytest.mark.parametrize("kind,dtype,with_bias", [("sigmoid", torch.float32, True), ("softmax", torch.bfloat16, False),
                                                  ("softmax", torch.float32, True), ("sigmoid", torch.bfloat16, True)])
@pytest.mark.parametrize("T", [2049, 4099])
def test_many_tokens(E, k, groups, kept, kind, dtype, with_bias, T):
    rng = np.random.default_rng(E + k)
    print(f"[route] many tokens E={E} k={k} G={groups} {kind} {dtype} bias={with_bias}", flush=True)
    values, logits = _logits(rng, T, E, dtype)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if with_bias else None
    mask = (rng.random(T) < 0.9).astype(np.uint8)
    best = 2 if groups > 1 else 1
    got_i, got_w, status = _route(logits, None if bias is None else torch.from_numpy(bias).cuda(), kind, k, groups,
                                  kept, best, kind == "sigmoid", 1.5, torch.from_numpy(mask).cuda())
    # the first tokens, the last ones and some between
    at = np.unique(np.concatenate([np.arange(40), rng.integers(0, T, 60), np.arange(T - 20, T)]))
    want_i, want_w = oracle64.route(values[at], bias, kind, k, groups, kept, best, kind == "sigmoid", 1.5, mask[at])
    assert np.array_equal(got_i[at], want_i) and status == 0
    _weights_near(got_w[at], want_w, kind, kind == "sigmoid")
    gw = rng.standard_normal((T, k)).astype(np.float32)
    out = torch.full((T, E), float("nan"), dtype=dtype, device="cuda")
    experts.ep_route_backward(ep.make_shape(T, 8, k, E, 1, 1), experts.make_router(KINDS[kind], 1, 1, 1, kind == "sigmoid", 1.5),
                              logits, torch.from_numpy(got_i).cuda(), torch.from_numpy(gw).cuda(), out)
    assert bool(out.isfinite().all())
    _check_gradient(out[torch.from_numpy(at).cuda()], values[at], got_i[at], gw[at], kind, kind == "sigmoid", 1.5)


@pytest.mark.parametrize("T", [70, 2100, 4100])
@pytest.mark.parametrize("kind", sorted(KINDS))
def test_near_ties_among_many_and_few_tokens(T, kind):
    """Biases that undo the scores' differences to a few steps of f32: every token's order is a near tie."""
    rng = np.random.default_rng(T)
    E, k = 64, 6
    base = rng.standard_normal(E).astype(np.float32)
    values = np.repeat(base[None], T, 0)
    values += (rng.integers(-3, 4, size=(T, E)) * 2.0 ** -22).astype(np.float32)
    p = oracle64.scores(base[None], kind)[0]
    bias = (0.7 - p).astype(np.float32)
    for groups, kept, best in ((1, 1, 1), (8, 3, 2), (8, 3, 1)):
        got_i, got_w, _ = _route(torch.from_numpy(values).cuda(), torch.from_numpy(bias).cuda(), kind, k, groups, kept, best)
        at = np.unique(np.concatenate([np.arange(40), rng.integers(0, T, 40)]))
        want_i, want_w = oracle64.route(values[at], bias, kind, k, groups, kept, best, True, 1.0)
        assert np.array_equal(got_i[at], want_i)
        _weights_near(got_w[at], want_w, kind, True)


@pytest.mark.parametrize("T", [500, 2100, 4100])
@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("k", [1, 2, 3])
def test_near_tie_behind_equal_experts(T, kind, k):
    """Experts 5 and 9 are equal and fill the last slot and the one behind it; expert 2 is a hair above or below."""
    rng = np.random.default_rng(T + k)
    E = 64
    values = np.full((T, E), -6.0, np.float32)
    bias = np.zeros(E, np.float32)
    bias[2] = 0.1
    s = 0.2 + 0.1 * rng.random(T)  # of experts 5 and 9; the others' scores are far below
    if kind == "sigmoid":
        values[:, 5] = values[:, 9] = np.log(s / (1 - s))
        v5 = 1 / (1 + np.exp(-values[:, 5].astype(np.float64)))
        values[:, 2] = np.log((v5 - 0.1) / (1.1 - v5))
    else:
        # scores p5 = p9 = s and p2 = s - bias, the rest shared out
        rest = (1 - 3 * s + float(bias[2])) / (E - 3)
        values[:] = np.log(rest)[:, None]
        values[:, 5] = values[:, 9] = np.log(s)
        values[:, 2] = np.log(s - float(bias[2]))
    steps = rng.integers(-2, 3, size=T)
    for _ in range(2):  # a step or two of f32 either way
        values[:, 2] = np.where(steps > 0, np.nextafter(values[:, 2], np.float32(9)),
                                np.where(steps < 0, np.nextafter(values[:, 2], np.float32(-99)), values[:, 2]))
        steps -= np.sign(steps)
    got_i, _, _ = _route(torch.from_numpy(values).cuda(), torch.from_numpy(bias).cuda(), kind, k)
    want_i, _ = oracle64.route(values, bias, kind, k, 1, 1, 1, True, 1.0)
    assert len(np.unique(want_i[:, 0])) > 1  # both orders occur
    assert np.array_equal(got_i, want_i)


@pytest.mark.parametrize("T,E,k", [(130, 200, 8), (130, 200, 32), (2100, 200, 16), (2100, 60, 3), (40, 1500, 8), (4100, 60, 3),
                                   (4100, 120, 16), (4100, 200, 32), (4100, 240, 8)])
@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("groups,kept,best", [(1, 1, 1), (10, 4, 2), (20, 7, 1)])
def test_more_near_ties_than_candidates(T, E, k, kind, groups, kept, best):
    """Every expert of a token is within a few steps of f32 of every other, or of a part of them."""
    rng = np.random.default_rng(E + k)
    base = rng.standard_normal(E).astype(np.float32)
    values = np.repeat(base[None], T, 0) + (rng.integers(-3, 4, size=(T, E)) * 2.0 ** -23).astype(np.float32)
    values = values.astype(np.float32)
    bias = (0.7 - oracle64.scores(base[None], kind)[0]).astype(np.float32)
    bias[rng.random(E) < 0.5] -= np.float32(0.25)
    at = np.unique(np.concatenate([np.arange(30), rng.integers(0, T, 30)]))
    got_i, got_w, _ = _route(torch.from_numpy(values).cuda(), torch.from_numpy(bias).cuda(), kind, k, groups, kept, best)
    want_i, want_w = oracle64.route(values[at], bias, kind, k, groups, kept, best, True, 1.0)
    assert np.array_equal(got_i[at], want_i)
    _weights_near(got_w[at], want_w, kind, True)


@pytest.mark.parametrize("E,groups,kept", [(256, 8, 4), (64, 64, 9), (160, 8, 3), (12, 4, 4), (96, 2, 1), (1024, 16, 1)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("with_bias", [False, True])
def test_groups(E, groups, kept, best, kind, with_bias):
    rng = np.random.default_rng(E + best)
    print(f"[route] groups E={E} G={groups} kept={kept} best={best} {kind} bias={with_bias}", flush=True)
    values, logits = _logits(rng, 70, E, torch.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if with_bias else None
    k = 8  # more than the groups kept hold, in some cases: the rest of the slots stay empty
    got_i, got_w, _ = _route(logits, None if bias is None else torch.from_numpy(bias).cuda(), kind, k, groups, kept,
                             best, True, 2.5)
    want_i, want_w = oracle64.route(values, bias, kind, k, groups, kept, best, True, 2.5)
    assert np.array_equal(got_i, want_i)
    _weights_near(got_w, want_w, kind, True)


@pytest.mark.parametrize("T", [300, 2100, 4100])
@pytest.mark.parametrize("kind", sorted(KINDS))
def test_group_ratings_that_cancel(T, kind):
    """The two best of each group are about 64 and -64: their sum is far smaller than what f32 makes of each is off by."""
    rng = np.random.default_rng(T)
    E, groups = 16, 8
    values = np.repeat(rng.standard_normal((T, 1)), E, 1).astype(np.float32)
    values += (rng.integers(-8, 9, size=(T, E)) * 2.0 ** -21).astype(np.float32)
    bias = np.tile(np.array([64, -64], np.float32), groups)
    got_i, got_w, _ = _route(torch.from_numpy(values).cuda(), torch.from_numpy(bias).cuda(), kind, 3, groups, 3, 2)
    want_i, want_w = oracle64.route(values, bias, kind, 3, groups, 3, 2, True, 1.0)
    assert np.array_equal(got_i, want_i)
    _weights_near(got_w, want_w, kind, True)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("with_bias", [False, True])
def test_ties_go_to_the_lowest_expert(kind, with_bias):
    """Few distinct values: nearly every choice and every group rating is a tie."""
    rng = np.random.default_rng(3)
    values = rng.integers(-2, 3, size=(200, 64)).astype(np.float32)
    bias = (rng.integers(0, 2, size=64) * 0.25).astype(np.float32) if with_bias else None
    dbias = None if bias is None else torch.from_numpy(bias).cuda()
    for dtype, (groups, kept, best) in itertools.product((torch.float32, torch.bfloat16), ((1, 1, 1), (8, 3, 2), (8, 3, 1))):
        got_i, got_w, _ = _route(torch.from_numpy(values).to(dtype).cuda(), dbias, kind, 6, groups, kept, best)
        want_i, want_w = oracle64.route(values, bias, kind, 6, groups, kept, best, True, 1.0)
        assert np.array_equal(got_i, want_i)
        _weights_near(got_w, want_w, kind, True)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_near_ties_are_decided_as_in_64_bits(kind):
    """Choices that differ by less than a step of f32, and logits so large that scores saturate."""
    rng = np.random.default_rng(11)
    T, E = 64, 256
    values = np.repeat(rng.standard_normal((T, 1)), E, 1).astype(np.float32)
    values = np.nextafter(values, np.where(rng.random((T, E)) < 0.5, 9, -9).astype(np.float32)).astype(np.float32)
    bias = np.zeros(E, np.float32)
    bias[rng.integers(0, E, 20)] = np.float32(1e-9)
    logits = torch.from_numpy(values).cuda()
    for b in (None, bias):
        got_i, got_w, _ = _route(logits, None if b is None else torch.from_numpy(b).cuda(), kind, 8, 8, 4, 2)
        want_i, want_w = oracle64.route(values, b, kind, 8, 8, 4, 2, True, 1.0)
        assert np.array_equal(got_i, want_i)
        _weights_near(got_w, want_w, kind, True)
    big = (30 + 60 * rng.random((T, E))).astype(np.float32)
    for v in (big, -big):
        got_i, _, _ = _route(torch.from_numpy(v).cuda(), None, kind, 8)
        assert np.array_equal(got_i, oracle64.route(v, None, kind, 8, 1, 1, 1, True, 1.0)[0])


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_experts_tokens_and_bad_values(kind, renorm, groups):
    rng = np.random.default_rng(5)
    T, E, k = 24, 32, 6
    values = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    values[0] = -np.inf                                   # nothing to choose
    values[1, 3:] = -np.inf                               # three experts for six slots
    values[2, :] = np.finfo(np.float32).min               # the type's lowest value is a value
    values[3, ::2] = np.finfo(np.float32).min
    values[4, 0], values[4, 1] = np.nan, np.inf
    values[5] = np.nan
    values[6, 5] = np.finfo(np.float32).max
    values[7] = -800.0                                    # every sigmoid is 0 in 64 bits: no sum to divide by
    values[8, 0] = -np.nan
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    bias[7] = -np.inf
    mask = np.ones(T, np.uint8)
    mask[20:] = 0
    for b in (None, bias):
        got_i, got_w, status = _route(torch.from_numpy(values).cuda(), None if b is None else torch.from_numpy(b).cuda(),
                                      kind, k, groups, max(1, groups - 2), 2 if groups > 1 else 1, renorm, 1.0,
                                      torch.from_numpy(mask).cuda())
        want_i, want_w = oracle64.route(values, b, kind, k, groups, max(1, groups - 2), 2 if groups > 1 else 1, renorm,
                                        1.0, mask)
        assert np.array_equal(got_i, want_i)
        assert np.all(np.isfinite(got_w))
        _weights_near(got_w, want_w, kind, renorm)
        assert status == experts.EP_DEV_BAD_LOGIT
    # rows switched off are not read: their bad values are not flagged
    values[:20] = 0.0
    values[20:] = np.nan
    _, _, status = _route(torch.from_numpy(values).cuda(), None, kind, k, mask=torch.from_numpy(mask).cuda())
    assert status == 0
    bias[3] = np.nan
    got_i, _, status = _route(torch.from_numpy(values[:20]).cuda(), torch.from_numpy(bias).cuda(), kind, k)
    assert status == experts.EP_DEV_BAD_LOGIT and not np.isin(got_i, (3, 7)).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_apart(dtype):
    """Logits and their gradient as columns of wider tensors, at offsets that break 16-byte alignment."""
    rng = np.random.default_rng(7)
    T, E, k = 50, 60, 4
    values, _ = _logits(rng, T, E, dtype)
    for lead, extra in ((0, 0), (1, 0), (3, 7), (4, 4)):
        wide = torch.full((T, lead + E + extra), float("nan"), dtype=dtype, device="cuda")
        view = wide[:, lead:lead + E]
        view.copy_(torch.from_numpy(values))
        got_i, got_w, status = _route(view, None, "sigmoid", k)
        want_i, want_w = oracle64.route(values, None, "sigmoid", k, 1, 1, 1, True, 1.0)
        assert np.array_equal(got_i, want_i) and status == 0
        _weights_near(got_w, want_w, "sigmoid", True)
        out = torch.full_like(wide, 7.0)
        gw = rng.standard_normal((T, k)).astype(np.float32)
        shape = ep.make_shape(T, 8, k, E, 1, 1)
        experts.ep_route_backward(shape, experts.make_router(1), view, torch.from_numpy(got_i).cuda(),
                                  torch.from_numpy(gw).cuda(), out[:, lead:lead + E])
        assert bool((out[:, :lead] == 7.0).all()) and bool((out[:, lead + E:] == 7.0).all())
        _check_gradient(out[:, lead:lead + E], values, got_i, gw, "sigmoid", True, 1.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E", [(50, 100), (50, 200), (30, 471), (2100, 61), (2100, 120), (2100, 255), (9, 1501), (4100, 61), (4100, 120),
                                 (4100, 255)])
def test_rows_apart_equal_rows_together(T, E, dtype):
    """Rows that start on any element, of whole and of part lanes: the same bits as rows without gaps."""
    rng = np.random.default_rng(T + E)
    k = 5
    _, logits = _logits(rng, T, E, dtype)
    bias = torch.from_numpy((rng.standard_normal(E) * 0.1).astype(np.float32)).cuda()
    gw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    shape, r = ep.make_shape(T, 8, k, E, 1, 1), experts.make_router(experts.EP_SCORE_SOFTMAX)
    want_i, want_w, status = _route(logits, bias, "softmax", k)
    idx = torch.from_numpy(want_i).cuda()
    grad = torch.empty_like(logits)
    experts.ep_route_backward(shape, r, logits, idx, gw, grad)
    for lead, extra in ((1, 0), (2, 1), (3, 6), (0, 1)):
        wide = torch.full((T, lead + E + extra), float("nan"), dtype=dtype, device="cuda")
        wide[:, lead:lead + E] = logits
        shifted = torch.full((E + lead,), float("nan"), device="cuda")
        shifted[lead:] = bias
        got_i, got_w, status = _route(wide[:, lead:lead + E], shifted[lead:], "softmax", k)
        assert np.array_equal(got_i, want_i) and np.array_equal(got_w, want_w) and status == 0
        out = torch.full_like(wide, 7.0)
        experts.ep_route_backward(shape, r, wide[:, lead:lead + E], idx, gw, out[:, lead:lead + E])
        assert torch.equal(out[:, lead:lead + E], grad)
        assert bool((out[:, :lead] == 7.0).all()) and bool((out[:, lead + E:] == 7.0).all())


def _check_gradient(got, values, idx, gw, kind, renorm, scale):
    want, size, before = oracle64.route_backward(values, idx, gw, kind, renorm, scale)
    # sigmoid: two 32-bit sigmoids of at most 8 U each (an exponential, a sum, a quotient), the slots'
    # sum and two products: under 24 U of `size`.  Softmax: a score of at most 56 U (as for the
    # weights, with its own exponential) times a difference off by 3 U of `size`.
    # Renormalising takes g_j - sum g_i s_i / S in binary64, where up to k + 6 steps of 2^-53 each
    # leave up to 40 * 2^-53 of what is subtracted even where the difference is 0 (one slot alone).
    tol = (24 if kind == "sigmoid" else 64) * U * size + 40 * 2.0 ** -53 * before
    if got.dtype == torch.bfloat16:
        tol = tol + oracle64.BF16_HALF * np.abs(want)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol + 1e-37), float((err - tol).max())


@pytest.mark.parametrize("E", [1, 7, 64, 160, 256, 2048])
@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_against_the_formula(E, kind, renorm, dtype):
    rng = np.random.default_rng(E + 1)
    T, k = 33, min(8, E)
    print(f"[route] gradient E={E} {kind} renorm={renorm} {dtype}", flush=True)
    values, logits = _logits(rng, T, E, dtype)
    idx = np.stack([rng.choice(E, k, replace=False) for _ in range(T)]).astype(np.int64)
    idx[0] = -1
    idx[1, 0] = -1
    idx[2, :] = idx[2, 0]  # one expert in every slot
    gw = rng.standard_normal((T, k)).astype(np.float32)
    gw[3] = 0.0
    out = torch.full((T, E), float("nan"), dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    experts.ep_route_backward(ep.make_shape(T, 8, k, E, 1, 1), experts.make_router(KINDS[kind], 1, 1, 1, renorm, 2.5), logits,
                              torch.from_numpy(idx).cuda(), torch.from_numpy(gw).cuda(), out, status)
    assert int(status.item()) == 0
    assert not out[0].any() and not out[3].any()
    _check_gradient(out, values, idx, gw, kind, renorm, 2.5)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(kind, renorm):
    """Central differences of the weights in binary64, the choice held fixed."""
    rng = np.random.default_rng(2)
    T, E, k = 6, 24, 4
    values, logits = _logits(rng, T, E, torch.float32)
    idx, _ = oracle64.route(values, None, kind, k, 1, 1, 1, renorm, 1.5)
    gw = rng.standard_normal((T, k)).astype(np.float32)

    def value(v):
        p = np.take_along_axis(oracle64.scores(v, kind), idx, 1)
        w = 1.5 * (p / p.sum(1, keepdims=True) if renorm else p)
        return (w * gw).sum()

    h = 1e-5
    want = np.zeros((T, E))
    for t, e in itertools.product(range(T), range(E)):
        up, down = values.astype(np.float64), values.astype(np.float64)
        up[t, e] += h
        down[t, e] -= h
        want[t, e] = (value(up) - value(down)) / (2 * h)
    out = torch.empty(T, E, device="cuda")
    experts.ep_route_backward(ep.make_shape(T, 8, k, E, 1, 1), experts.make_router(KINDS[kind], 1, 1, 1, renorm, 1.5), logits,
                              torch.from_numpy(idx).cuda(), torch.from_numpy(gw).cuda(), out)
    # truncation h^2 times a third derivative below 10, rounding 2^-53 * 20 / h, and 64 U of values below 4
    assert np.allclose(out.cpu().numpy(), want, rtol=0, atol=2e-5)


def test_gradient_of_masked_and_bad_logits():
    T, E, k = 4, 8, 3
    values = np.random.default_rng(1).standard_normal((T, E)).astype(np.float32)
    values[0, :4] = -np.inf
    values[1] = -np.inf
    values[2, 0] = np.finfo(np.float32).min
    idx = np.array([[5, 6, -1], [0, 1, 2], [0, 1, 2], [1, 99, -5]], np.int64)
    gw = np.ones((T, k), np.float32)
    gw[:, 1] = -2.0
    for kind, renorm in itertools.product(sorted(KINDS), (False, True)):
        out = torch.full((T, E), float("nan"), device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        experts.ep_route_backward(ep.make_shape(T, 8, k, E, 1, 1), experts.make_router(KINDS[kind], 1, 1, 1, renorm),
                                  torch.from_numpy(values).cuda(), torch.from_numpy(idx).cuda(),
                                  torch.from_numpy(gw).cuda(), out, status)
        assert int(status.item()) == ep.EP_DEV_BAD_TOPK_IDX
        _check_gradient(out, values, idx, gw, kind, renorm, 1.0)
        bad = values.copy()
        bad[3, 7] = np.nan
        status.zero_()
        experts.ep_route_backward(ep.make_shape(T, 8, k, E, 1, 1), experts.make_router(KINDS[kind], 1, 1, 1, renorm),
                                  torch.from_numpy(bad).cuda(), torch.from_numpy(idx).cuda(),
                                  torch.from_numpy(gw).cuda(), out, status)
        assert int(status.item()) == ep.EP_DEV_BAD_TOPK_IDX | experts.EP_DEV_BAD_LOGIT
        _check_gradient(out, bad, idx, gw, kind, renorm, 1.0)


@pytest.mark.parametrize("T", [40, 2100, 4100])
def test_gradient_of_tokens_without_slots_reads_no_logits(T):
    """A padded batch: NaN logits where the mask left no slot are neither flagged nor passed on."""
    rng = np.random.default_rng(6)
    E, k = 60, 4
    values, logits = _logits(rng, T, E, torch.float32)
    mask = (rng.random(T) < 0.5).astype(np.uint8)
    logits[torch.from_numpy(mask == 0).cuda()] = float("nan")
    for kind, renorm in itertools.product(sorted(KINDS), (False, True)):
        idx, _, status = _route(logits, None, kind, k, renorm=renorm, mask=torch.from_numpy(mask).cuda())
        assert status == 0 and np.all(idx[mask == 0] == -1)
        gw = rng.standard_normal((T, k)).astype(np.float32)
        out = torch.full((T, E), float("nan"), device="cuda")
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        experts.ep_route_backward(ep.make_shape(T, 8, k, E, 1, 1), experts.make_router(KINDS[kind], 1, 1, 1, renorm), logits,
                                  torch.from_numpy(idx).cuda(), torch.from_numpy(gw).cuda(), out, word)
        assert int(word.item()) == 0 and not out[torch.from_numpy(mask == 0).cuda()].any()
        at = np.flatnonzero(mask)[:30]
        _check_gradient(out[torch.from_numpy(at).cuda()], values[at], idx[at], gw[at], kind, renorm, 1.0)


def test_no_tokens_and_many_slots():
    empty = torch.empty(0, 16, device="cuda")
    idx, w, status = _route(empty, None, "sigmoid", 4)
    assert idx.shape == (0, 4) and status == 0
    rng = np.random.default_rng(4)
    values, logits = _logits(rng, 9, 40, torch.float32)
    got_i, got_w, _ = _route(logits, None, "softmax", 32)
    want_i, want_w = oracle64.route(values, None, "softmax", 32, 1, 1, 1, True, 1.0)
    assert np.array_equal(got_i, want_i)
    _weights_near(got_w, want_w, "softmax", True)
    values, logits = _logits(rng, 9, 5, torch.float32)
    got_i, _, _ = _route(logits, None, "softmax", 32)
    assert np.array_equal(got_i, oracle64.route(values, None, "softmax", 32, 1, 1, 1, True, 1.0)[0])
    assert np.all(got_i[:, 5:] == -1)
