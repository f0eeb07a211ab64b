"""The operators together: a layer from router logits to combined rows, its gradient back to the
logits, captured and replayed, and on two streams."""
import numpy as np
import pytest
import torch

import experts_oracle as oracle64
import oracle
from combine_ep_get_02_amd import ep, experts
from gpu_harness import bf16_host, random_rows, to_dev_bf16

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, T, H, I, E, R, K, align=1, seed=0, groups=1, kept=1):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.I, self.E, self.R, self.K = T, H, I, E, R, K
        self.shape = ep.make_shape(T, H, K, E, R, 4, expert_alignment=align)
        self.router = experts.make_router(experts.EP_SCORE_SIGMOID, groups, kept, 2, True, 1.5)
        self.bias_np = (rng.standard_normal(E) * 0.05).astype(np.float32)
        self.groups, self.kept = groups, kept
        self.w_in = self._weights(rng, (E, 2 * I, H))
        self.w_out = self._weights(rng, (E, H, I))
        self.w_in_s = (rng.random((E, 2 * I // 128, H // 128)) * 1e-3 + 1e-4).astype(np.float32)
        self.w_out_s = (rng.random((E, H // 128, I // 128)) * 1e-3 + 1e-4).astype(np.float32)
        self.dev = dict(w_in=self.w_in.cuda(), w_out=self.w_out.cuda(), w_in_s=torch.from_numpy(self.w_in_s).cuda(),
                        w_out_s=torch.from_numpy(self.w_out_s).cuda(), bias=torch.from_numpy(self.bias_np).cuda())
        self.b = ep.allocate(self.shape, T * min(R, K))
        self.e = experts.allocate_experts(self.b, I, T * K + E * (align - 1))
        self.logits = torch.zeros(T, E, device="cuda")
        self.x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")

    @staticmethod
    def _weights(rng, shape):
        v = (rng.standard_normal(shape) * 60).astype(np.float32)
        return torch.from_numpy(v).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    def draw(self, seed):
        rng = np.random.default_rng(seed)
        self.logits.copy_(torch.from_numpy(rng.standard_normal((self.T, self.E)).astype(np.float32)))
        self.x.copy_(torch.from_numpy(rng.standard_normal((self.T, self.H)).astype(np.float32)))

    def run(self, stream=None):
        d = self.dev
        experts.run_route(self.b, self.e, self.router, self.logits, d["bias"], stream=stream)
        experts.run_experts(self.b, self.e, self.x, d["w_in"], d["w_in_s"], d["w_out"], d["w_out_s"], stream=stream)

    def outputs(self):
        torch.cuda.synchronize()
        n = int(self.e.num_grouped.item())
        assert int(self.b.dev_status.item()) == 0
        return [t.cpu().clone() for t in (self.b.combined_x.view(torch.int16), self.e.topk_idx, self.e.topk_weights,
                                          self.e.act[:n], self.e.act_scales[:n], self.e.y[:n].view(torch.int16))]


@pytest.mark.parametrize("shape", [dict(T=1, H=256, I=128, E=16, R=8, K=2), dict(T=70, H=512, I=256, E=32, R=8, K=4, align=4),
                                   dict(T=200, H=256, I=384, E=64, R=16, K=8, groups=8, kept=3)], ids=str)
def test_layer_against_binary64(shape):
    layer = Layer(**shape)
    layer.draw(1)
    layer.run()
    combined, idx, w, act, act_s, y = layer.outputs()
    T, H, I, E, R, K = layer.T, layer.H, layer.I, layer.E, layer.R, layer.K
    want_i, want_w = oracle64.route(layer.logits.cpu().numpy(), layer.bias_np, "sigmoid", K, layer.groups, layer.kept,
                                    2, True, 1.5)
    assert np.array_equal(idx.numpy(), want_i)
    assert np.all(np.abs(w.numpy() - want_w) <= 2 * oracle64.U * np.abs(want_w))

    # token by token from x as the quantiser has it (bit-exact), everything after it in binary64
    o = oracle.Oracle()
    codes, scales = o.quantize_e4m3(bf16_host(layer.x), H // 128)
    xv = oracle64.e4m3_values(codes) * np.repeat(scales.astype(np.float64), 128, 1)
    w1 = oracle64.e4m3_values(layer.w_in) * np.repeat(np.repeat(layer.w_in_s.astype(np.float64), 128, 1), 128, 2)
    w2 = oracle64.e4m3_values(layer.w_out) * np.repeat(np.repeat(layer.w_out_s.astype(np.float64), 128, 1), 128, 2)
    got = layer.b.combined_x.double().cpu().numpy()
    for t in range(T):
        out, tol = np.zeros(H), np.zeros(H)
        for j in range(K):
            e = want_i[t, j]
            a = oracle64.swiglu((w1[e] @ xv[t])[None])[0]
            top = np.abs(a.reshape(-1, 128)).max(1)
            # the second product's input: half a code's step off; 1 % covers the f32 sums before it
            da = oracle64.E4M3_HALF * np.abs(a) + 2.0 ** -10 * np.repeat(top / 448, 128) + 0.01 * np.repeat(top, 128)
            v = w2[e] @ a
            dv = np.abs(w2[e]) @ da
            out += want_w[t, j] * v
            tol += want_w[t, j] * (dv + oracle64.BF16_HALF * (np.abs(v) + dv))
        tol += oracle64.BF16_HALF * (np.abs(out) + tol) + 1e-6 * tol
        assert np.all(np.abs(got[t] - out) <= tol)
    # the second half again, from the codes that the first half made
    pos = oracle64.positions(want_i, layer.b.send_slot.cpu().numpy(), layer.e.slot_pos.cpu().numpy(), E, R, layer.b.capacity,
                             layer.e.capacity)
    sizes = layer.b.recv_per_expert.cpu().numpy()
    want_y, mag = oracle64.product(act, act_s.numpy(), layer.w_out, layer.w_out_s, sizes, act.shape[0])
    yv = y.view(torch.bfloat16).double().numpy()
    cut = oracle64.product_cut(act, act_s.numpy(), layer.w_out, layer.w_out_s, sizes, act.shape[0])
    tol = oracle64.BF16_HALF * np.abs(want_y) + ((2 * (I + I // 128) + 2) * oracle64.U * mag + 8 * 2.0 ** -13 * cut) * 1.01
    assert np.all(np.abs(yv - want_y) <= tol)
    want, cmag = oracle64.combine(yv, w.numpy(), pos)
    assert np.all(np.abs(got - want) <= oracle64.BF16_HALF * np.abs(want) + 2 * K * oracle64.U * cmag)


def test_gradient_from_outputs_to_logits():
    """grad of sum(G * combined) with respect to the logits, with y held, through both backward calls."""
    layer = Layer(T=40, H=256, I=128, E=16, R=4, K=3, align=2, seed=3)
    layer.draw(4)
    layer.run()
    T, E, K = layer.T, layer.E, layer.K
    rng = np.random.default_rng(5)
    grad = torch.from_numpy(rng.standard_normal((T, layer.H)).astype(np.float32)).to(torch.bfloat16).cuda()
    gy = torch.empty_like(layer.e.y)
    gw = torch.empty(T, K, device="cuda")
    gl = torch.empty_like(layer.logits)
    experts.run_combine_grouped_backward(layer.b, layer.e, grad, gy, gw)
    experts.ep_route_backward(layer.shape, layer.router, layer.logits, layer.e.topk_idx, gw, gl)
    torch.cuda.synchronize()
    idx = layer.e.topk_idx.cpu().numpy()
    pos = oracle64.positions(idx, layer.b.send_slot.cpu().numpy(), layer.e.slot_pos.cpu().numpy(), E, layer.R,
                             layer.b.capacity, layer.e.capacity)
    yv, gv = layer.e.y.double().cpu().numpy(), grad.double().cpu().numpy()
    want_gw = np.stack([[yv[pos[t, j]] @ gv[t] for j in range(K)] for t in range(T)])
    mag_gw = np.stack([[np.abs(yv[pos[t, j]]) @ np.abs(gv[t]) for j in range(K)] for t in range(T)])
    want, size, _ = oracle64.route_backward(layer.logits.cpu().numpy(), idx, want_gw, "sigmoid", True, 1.5)
    # a weight's gradient off by H U of its magnitudes moves each logit's by at most 1.5 (1 + 1) s (1 - s) / S of that,
    # and S is at least the largest score: under 4 times the largest of the token's
    tol = 24 * oracle64.U * size + 4 * layer.H * oracle64.U * mag_gw.max(1, keepdims=True)
    assert np.all(np.abs(gl.double().cpu().numpy() - want) <= tol)


def test_replays_of_a_captured_layer_equal_the_eager_one():
    layer = Layer(T=130, H=512, I=256, E=32, R=8, K=4, align=4, seed=6, groups=4, kept=2)
    gy, gw = torch.empty_like(layer.e.y), torch.empty(layer.T, layer.K, device="cuda")
    gl, grad = torch.empty_like(layer.logits), torch.empty(layer.T, layer.H, dtype=torch.bfloat16, device="cuda")

    def step():
        layer.run()
        experts.run_combine_grouped_backward(layer.b, layer.e, grad, gy, gw)
        experts.ep_route_backward(layer.shape, layer.router, layer.logits, layer.e.topk_idx, gw, gl)

    def everything():
        out = layer.outputs()
        n = int(layer.e.num_grouped.item())
        return out + [gy[:n].view(torch.int16).cpu().clone(), gw.cpu().clone(), gl.cpu().clone()]

    layer.draw(10)
    grad.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (11, 12, 13):
        layer.draw(seed)
        grad.normal_()
        step()
        want = everything()
        for t in (layer.b.combined_x, layer.e.y, gy, gw, gl, layer.e.topk_weights):
            t.zero_()
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            for got, ref in zip(everything(), want):
                assert torch.equal(got, ref)


def test_two_layers_at_once_on_two_streams():
    a = Layer(T=300, H=512, I=256, E=32, R=8, K=4, seed=7)
    c = Layer(T=90, H=256, I=384, E=64, R=16, K=8, seed=8)
    a.draw(1)
    c.draw(2)
    want = []
    for layer in (a, c):
        layer.run()
        want.append(layer.outputs())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for layer in (a, c):
            layer.b.combined_x.zero_()
            layer.e.y.zero_()
        torch.cuda.synchronize()
        for layer, s in zip((a, c), streams):
            layer.run(stream=s)
        torch.cuda.synchronize()
        for layer, ref in zip((a, c), want):
            for got, r in zip(layer.outputs(), ref):
                assert torch.equal(got, r)


def test_a_layer_whose_tokens_are_all_masked():
    layer = Layer(T=20, H=256, I=128, E=16, R=8, K=2, seed=9)
    layer.draw(3)
    mask = torch.zeros(20, dtype=torch.uint8, device="cuda")
    experts.run_route(layer.b, layer.e, layer.router, layer.logits, layer.dev["bias"], mask)
    d = layer.dev
    layer.b.combined_x.fill_(5.0)
    experts.run_experts(layer.b, layer.e, layer.x, d["w_in"], d["w_in_s"], d["w_out"], d["w_out_s"])
    torch.cuda.synchronize()
    assert int(layer.e.num_grouped.item()) == 0 and not layer.b.combined_x.any()


def test_rows_of_random_bits_through_the_layer():
    """x of widely differing magnitudes: every output finite, combine and products as above for shape only."""
    layer = Layer(T=33, H=256, I=128, E=8, R=2, K=2, seed=10)
    layer.draw(5)
    layer.x.copy_(to_dev_bf16(random_rows(np.random.default_rng(1), 33, 256)))
    layer.run()
    layer.outputs()
    assert bool(layer.b.combined_x.isfinite().all())


def test_a_layer_without_tokens():
    layer = Layer(T=0, H=256, I=128, E=8, R=2, K=2, seed=11)
    layer.run()
    torch.cuda.synchronize()
    assert int(layer.b.dev_status.item()) == 0


def test_a_layer_whose_buffers_are_larger_than_its_rows():
    """Receive and grouped capacity far above what the routing fills: the same outputs."""
    layer = Layer(T=50, H=256, I=128, E=16, R=4, K=3, align=2, seed=12)
    layer.draw(2)
    layer.run()
    want = layer.outputs()
    layer.b = ep.allocate(layer.shape, 50 * 4 + 300)
    layer.e = experts.allocate_experts(layer.b, 128, 5000)
    layer.e.y.fill_(float("nan"))
    layer.run()
    for got, ref in zip(layer.outputs(), want):
        assert torch.equal(got, ref)


def test_few_received_rows_are_dropped_and_flagged():
    """A receive capacity below the routing: the tokens that fit come out, nothing reads past the buffers."""
    layer = Layer(T=50, H=256, I=128, E=16, R=4, K=3, seed=13)
    layer.draw(2)
    layer.run()
    whole = layer.outputs()[0]
    n = int(layer.b.num_recv.item())
    layer.b = ep.allocate(layer.shape, n - 20)
    layer.e = experts.allocate_experts(layer.b, 128, 150)
    layer.run()
    torch.cuda.synchronize()
    assert int(layer.b.dev_status.item()) == ep.EP_DEV_RECV_OVERFLOW
    kept = (layer.b.send_slot >= 0).cpu().numpy()
    idx = layer.e.topk_idx.cpu().numpy()
    fits = np.array([all(kept[t, e // 4] for e in idx[t]) for t in range(50)])
    assert fits.any() and not fits.all()
    got = layer.b.combined_x.view(torch.int16).cpu()
    assert torch.equal(got[torch.from_numpy(fits)], whole[torch.from_numpy(fits)])
