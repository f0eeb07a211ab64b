"""Every kernel of the experts' E4M3 products over numbers of blocks of channels that fill its buffers once,
not quite, and several times, at its whole width and with columns that end inside a block.  Which kernel a
case reaches is checked on the CPU, by test_expert_kernel_choice.py."""
import numpy as np
import pytest
import torch

from combine_ep_get_02_amd import experts

pytestmark = pytest.mark.gpu
CODES = torch.tensor([0xC0, 0xB8, 0x00, 0x38, 0x40], dtype=torch.uint8)  # E4M3 of -2 .. 2
MANY = [1100, 0, 900, 1, 128, 129]  # tiles filled whole, to one row, to their half and one row past it
SOME = [130, 200, 7]

# kernel: (swiglu, rows and columns of a block, threads), segments, n, numbers of blocks of 128 channels
KERNELS = {
    "product, 16 rows, 16 columns": ((False, 16, 16, 512), [3], 264, (1, 7, 8, 9, 23, 24, 25, 49)),
    "product, 16 rows, 64 columns": ((False, 16, 64, 512), [20], 2056, (1, 7, 8, 9, 15, 16, 17, 33)),
    "product, 32 rows, 64 columns": ((False, 32, 64, 512), [40], 8200, (1, 8, 9, 15, 16, 17, 25)),
    "product, 32 rows, 128 columns": ((False, 32, 128, 256), SOME, 4104, (1, 2, 3, 4, 5, 6, 9)),
    "product, 64 rows": ((False, 64, 256, 512), [50, 64, 0, 63, 65, 1, 80, 77], 4104, (1, 2, 3, 4, 5, 6, 7, 16)),
    "product, 128 rows": ((False, 128, 256, 512), MANY, 2056, (1, 2, 3, 4, 5, 6, 7, 16)),
    "swiglu, 16 rows": ((True, 16, 128, 512), [20], 256, (1, 2, 3, 4, 5, 6, 9)),
    "swiglu, 32 rows": ((True, 32, 128, 512), SOME, 1664, (1, 2, 3, 4, 5, 6, 9)),
    "swiglu, 64 rows": ((True, 64, 128, 512), SOME, 2816, (1, 2, 3, 4, 5, 6, 7, 16)),
    "swiglu, 128 rows": ((True, 128, 128, 512), MANY, 1024, (1, 2, 3, 4, 5, 6, 7, 16)),
}
CASES = [(name, blocks) for name in KERNELS for blocks in KERNELS[name][3]]


def _draw(rng, shape):
    pick = torch.from_numpy(rng.integers(0, 5, size=shape))
    return CODES[pick].cuda(), pick.cuda().to(torch.float64) - 2.0


@pytest.mark.parametrize("name,blocks", CASES)
def test_kernel_over_blocks_of_channels(name, blocks):
    """Integers and scales that are powers of two: every partial sum is exact in f32, so results round once."""
    (swiglu, *_), sizes, n, _ = KERNELS[name]
    rng = np.random.default_rng(blocks)
    E, rows, k, wide = len(sizes), sum(sizes), 128 * blocks, n * (2 if swiglu else 1)
    print(f"[loops] {name}, {blocks} blocks", flush=True)
    x, xv = _draw(rng, (rows, k))
    w, wv = _draw(rng, (E, wide, k))
    # scales of the rows' blocks and of the weights' differ from block to block, so that one taken from another shows
    xs = 2.0 ** torch.from_numpy(rng.integers(-3, 3, size=(rows, blocks))).cuda().to(torch.float64)
    ws = 2.0 ** torch.from_numpy(rng.integers(-3, 3, size=(E, -(-wide // 128), blocks))).cuda().to(torch.float64)
    xv = xv * xs.repeat_interleave(128, 1)
    held = torch.from_numpy(np.array(sizes, np.int32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if swiglu:
        xs, xv = xs / 64, xv / 64
        out = torch.zeros(rows, n, dtype=torch.uint8, device="cuda")
        outs = torch.zeros(rows, n // 128, device="cuda")
        experts.ep_expert_gemm_swiglu_fp8(E, n, k, x, xs.float(), w, ws.float(), held, rows, out, outs, status)
        got = out.view(torch.float8_e4m3fn).double() * outs.double().repeat_interleave(128, 1)
    else:
        out = torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device="cuda")
        experts.ep_expert_gemm_fp8(E, n, k, x, xs.float(), w, ws.float(), held, rows, out, status)
    assert int(status.item()) == 0
    first = 0
    for e, size in enumerate(sizes):
        here = slice(first, first + size)
        first += size
        if size == 0:
            continue
        weights = wv[e] * ws[e].repeat_interleave(128, 0)[:wide].repeat_interleave(128, 1)
        y = torch.matmul(xv[here], weights.t().contiguous())
        if not swiglu:
            # multiples of 2^-6, of either sign, whose sums stay far below 2^24 of it
            assert torch.equal(out[here], y.to(torch.float32).to(torch.bfloat16)), f"expert {e}"
            continue
        a = y[:, :n] / (1.0 + torch.exp(-y[:, :n])) * y[:, n:]
        top = a.abs().view(size, n // 128, 128).amax(2).clamp_(min=2.0 ** -64)
        # gate and up are exact; the activation is an exponential, a sum, a quotient and a product, the scale a quotient
        assert bool(((outs[here].double() - top / 448).abs() <= 10 * 2.0 ** -24 * top / 448).all()), f"expert {e}"
        step = 2.0 ** -4 * a.abs() + (2.0 ** -10 * outs[here].double()).repeat_interleave(128, 1)
        assert bool(((got[here] - a).abs() <= step * (1 + 2.0 ** -4) + 2.0 ** -18 * a.abs()).all()), f"expert {e}"
