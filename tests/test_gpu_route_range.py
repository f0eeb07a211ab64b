"""The router's gradient where scores are far below the range of f32, against its definition worked
out in logarithms: binary64 holds these, whatever the scores are."""
import numpy as np
import pytest
import torch

import experts_oracle as oracle64
from combine_ep_get_02_amd import ep, experts

pytestmark = pytest.mark.gpu
KINDS = {"sigmoid": experts.EP_SCORE_SIGMOID, "softmax": experts.EP_SCORE_SOFTMAX}
U = oracle64.U


def _log_scores(l, kind):
    """Logarithms of the scores, and 1 - score (a sigmoid's), in binary64."""
    l = l.astype(np.float64)
    if kind == "sigmoid":
        return -np.logaddexp(0.0, -l), np.exp(-np.logaddexp(0.0, l))
    top = l.max(1, keepdims=True)
    return l - top - np.log(np.exp(l - top).sum(1, keepdims=True)), None


def _gradient(values, idx, gw, kind, renorm, scale):
    """(gradient, size of what is added up in it): the slots' terms with their scores as exponentials of
    logarithms, the ratios of renormalised ones as exponentials of differences."""
    T, E = values.shape
    log_s, rest = _log_scores(values, kind)
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        ls = log_s[t, idx[t]]
        g = gw[t].astype(np.float64)
        if renorm:
            r = np.exp(ls - ls.max())
            r /= r.sum()
            part = scale * (g - (g * r).sum()) * r
            whole = scale * (np.abs(g) + (np.abs(g) * r).sum()) * r
        else:
            part = scale * g * np.exp(ls)
            whole = np.abs(part)
        if kind == "sigmoid":
            part, whole = part * rest[t, idx[t]], whole * rest[t, idx[t]]
        elif not renorm:
            out[t] -= np.exp(log_s[t]) * part.sum()
            size[t] += np.exp(log_s[t]) * whole.sum()
        for j, e in enumerate(idx[t]):
            out[t, e] += part[j]
            size[t, e] += whole[j]
    return out, size


def _backward(logits, idx, gw, kind, renorm, scale):
    T, E = logits.shape
    out = torch.full((T, E), float("nan"), dtype=logits.dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    experts.ep_route_backward(ep.make_shape(T, 8, idx.shape[1], E, 1, 1),
                              experts.make_router(KINDS[kind], 1, 1, 1, renorm, scale), logits,
                              torch.from_numpy(idx).cuda(), torch.from_numpy(gw).cuda(), out, status)
    assert int(status.item()) == 0
    return out


def _check(out, values, idx, gw, kind, renorm, scale):
    want, size = _gradient(values, idx, gw, kind, renorm, scale)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    # A slot's term is formed in binary64 and rounded to f32 once, and up to k of them are added: k + 1 steps of U.
    # A softmax that is not renormalised divides by a sum of f32 exponentials, 56 U of a score, and rounds its mean
    # and two products.  Logarithms of up to 800 leave 1e-13 of a score in the definition here.  An f32 is a
    # multiple of 2^-149.
    k = idx.shape[1]
    tol = (k + 1 + (60 if kind == "softmax" and not renorm else 0)) * U * size + 1e-12 * size + 2.0 ** -149
    if out.dtype == torch.bfloat16:
        tol = tol + oracle64.BF16_HALF * (np.abs(want) + tol) + 2.0 ** -133  # the least bf16
    err = np.abs(got - want)
    assert np.all(err <= tol), float((err - tol).max())


def _case(rng, T, E, k, level, dtype):
    """Logits whose chosen ones lie within a few units of `level`, the others far below or about it."""
    t = torch.from_numpy((level + rng.standard_normal((T, E)) * 2.0).astype(np.float32)).to(dtype)
    idx = np.stack([rng.choice(E, k, replace=False) for _ in range(T)]).astype(np.int64)
    return t.to(torch.float32).numpy(), t.cuda(), idx


# T, E, k: every width of a token, rows in one turn of the lanes and in several
SIZES = [(37, 24, 2), (37, 256, 8), (9, 600, 8), (4100, 60, 6), (4100, 120, 8), (4100, 250, 8)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("level", [-60.0, -84.0, -88.0, -95.0, -110.0, -300.0, -690.0, 60.0, 95.0])
@pytest.mark.parametrize("kind,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
def test_gradient_at_any_level_of_the_logits(T, E, k, level, kind, renorm):
    rng = np.random.default_rng(E + int(abs(level)))
    for dtype, size in ((torch.float32, 1.0), (torch.bfloat16, 1.0), (torch.float32, 1e4)):
        values, logits, idx = _case(rng, T, E, k, level, dtype)
        gw = (rng.standard_normal((T, k)) * size).astype(np.float32)
        out = _backward(logits, idx, gw, kind, renorm, 2.5)
        at = np.unique(np.concatenate([np.arange(min(T, 30)), [T - 1]]))
        _check(out[torch.from_numpy(at).cuda()], values[at], idx[at], gw[at], kind, renorm, 2.5)


def test_gradient_of_two_small_sigmoids():
    """Chosen logits -95 and -96: weights 0.731 and 0.269, and a gradient of 0.731 * 0.269 each way."""
    values = np.zeros((1, 8), np.float32)
    values[0, 2:4] = -95.0, -96.0
    idx = np.array([[2, 3]], np.int64)
    out = _backward(torch.from_numpy(values).cuda(), idx, np.array([[1.0, 0.0]], np.float32), "sigmoid", True, 1.0)
    r = 1.0 / (1.0 + np.exp(-1.0))
    want = np.zeros(8)
    want[2:4] = r * (1 - r), -r * (1 - r)
    assert np.all(np.abs(out.double().cpu().numpy()[0] - want) <= 4 * U)


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("below", [80.0, 90.0, 104.0, 300.0, 700.0])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_softmax_choices_far_below_the_top(T, E, k, below, renorm):
    """What a bias does: the experts chosen are `below` under the row's largest logit, which is not chosen."""
    rng = np.random.default_rng(E + int(below))
    values, _, idx = _case(rng, T, E, k, 0.0, torch.float32)
    values[np.arange(T)[:, None], idx] -= np.float32(below)
    logits = torch.from_numpy(values).cuda()
    for size in (1.0, 1e4):
        gw = (rng.standard_normal((T, k)) * size).astype(np.float32)
        out = _backward(logits, idx, gw, "softmax", renorm, 1.0)
        at = np.unique(np.concatenate([np.arange(min(T, 30)), [T - 1]]))
        _check(out[torch.from_numpy(at).cuda()], values[at], idx[at], gw[at], "softmax", renorm, 1.0)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_an_expert_in_several_slots(kind, renorm):
    rng = np.random.default_rng(8)
    T, E, k = 33, 40, 5
    for level in (0.0, -95.0):
        values, logits, idx = _case(rng, T, E, k, level, torch.float32)
        idx[:, 3] = idx[:, 1]
        idx[:16, 4] = idx[:16, 1]
        gw = rng.standard_normal((T, k)).astype(np.float32)
        _check(_backward(logits, idx, gw, kind, renorm, 1.5), values, idx, gw, kind, renorm, 1.5)


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("below", [300.0, 800.0, 1e6, 1e37])
@pytest.mark.parametrize("renorm", [True, False])
def test_softmax_weights_and_gradient_agree_however_far_below_the_top(T, E, k, below, renorm):
    """A bias picks experts whose scores binary64 cannot hold: renormalised weights are ratios to each other, and the
    gradient is that of these ratios; others are 0, and so is their gradient."""
    rng = np.random.default_rng(E)
    values, _, idx = _case(rng, T, E, k, 0.0, torch.float32)
    values[np.arange(T)[:, None], idx] -= np.float32(below)
    # the same experts in every token, so that a bias can pick them
    values[:, idx[0]] = np.float32(-below) * (1 + rng.integers(0, 2, (T, k)) * 2.0 ** -23) - rng.random((T, k)).astype(np.float32)
    rest = np.setdiff1d(np.arange(E), idx[0])
    values[:, rest] = rng.standard_normal((T, len(rest)))
    values = values.astype(np.float32)
    bias = np.zeros(E, np.float32)
    bias[idx[0]] = 2.0 + np.arange(k)  # in this order: scores are 0 and 1 at most
    logits = torch.from_numpy(values).cuda()
    got_i = torch.empty(T, k, dtype=torch.int64, device="cuda")
    got_w = torch.empty(T, k, device="cuda")
    experts.ep_route(ep.make_shape(T, 8, k, E, 1, 1), experts.make_router(0, 1, 1, 1, renorm, 2.5), logits,
                     torch.from_numpy(bias).cuda(), None, got_i, got_w)
    order = np.repeat(idx[:1, ::-1], T, 0)
    assert np.array_equal(got_i.cpu().numpy(), order)
    chosen = np.take_along_axis(values.astype(np.float64), order, 1)
    r = np.exp(chosen - chosen.max(1, keepdims=True))
    r /= r.sum(1, keepdims=True)
    if not renorm:
        r = np.exp(_log_scores(values, "softmax")[0])[np.arange(T)[:, None], order]
    # formed in binary64 and rounded once, but for a sum of f32 exponentials, 56 U
    assert np.all(np.abs(got_w.double().cpu().numpy() - 2.5 * r) <= (2 if renorm else 58) * U * 2.5 * r + 2.0 ** -149)
    gw = rng.standard_normal((T, k)).astype(np.float32)
    at = np.unique(np.concatenate([np.arange(min(T, 30)), [T - 1]]))
    out = _backward(logits, order, gw, "softmax", renorm, 2.5)
    _check(out[torch.from_numpy(at).cuda()], values[at], order[at], gw[at], "softmax", renorm, 2.5)


@pytest.mark.parametrize("level", [-705.0, -800.0, -1e30])
def test_sigmoid_weights_and_gradient_where_scores_end(level):
    """Below about -709 a sigmoid is 0 in binary64: weights and gradient are 0; above, both are those of the ratios."""
    rng = np.random.default_rng(3)
    T, E, k = 20, 16, 3
    values = np.full((T, E), -1e35, np.float32)
    idx = np.stack([np.sort(rng.choice(E, k, replace=False)) for _ in range(T)]).astype(np.int64)
    np.put_along_axis(values, idx, np.float32(level) - np.arange(k, dtype=np.float32), 1)
    logits = torch.from_numpy(values).cuda()
    got_i, got_w = torch.empty(T, k, dtype=torch.int64, device="cuda"), torch.empty(T, k, device="cuda")
    experts.ep_route(ep.make_shape(T, 8, k, E, 1, 1), experts.make_router(1, 1, 1, 1, True, 1.0), logits, None, None, got_i, got_w)
    assert np.array_equal(got_i.cpu().numpy(), idx)
    gw = rng.standard_normal((T, k)).astype(np.float32)
    out = _backward(logits, idx, gw, "sigmoid", True, 1.0)
    if level < -709:
        assert not got_w.any() and not out.any()
        return
    r = np.exp(-np.arange(k))
    assert np.all(np.abs(got_w.double().cpu().numpy() - r / r.sum()) <= 2 * U * r / r.sum())
    _check(out, values, idx, gw, "sigmoid", True, 1.0)
