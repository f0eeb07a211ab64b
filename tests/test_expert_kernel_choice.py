"""The rule that picks a product's kernel, compiled for the host: the cases of test_gpu_expert_loops.py reach
the kernels that they are for, and there is one for each kernel that the rule can pick (no GPU needed)."""
import os
import subprocess

import pytest

import test_gpu_expert_loops as loops
from combine_ep_get_02_amd import build as hip_build

PROGRAM = r"""
#include <stdio.h>
#include "ep_expert_gemm.hip"
int main() {
    int experts, n, k, rows, swiglu;
    while (scanf("%d %d %d %d %d", &experts, &n, &k, &rows, &swiglu) == 5) {
        ep::GemmArgs a = {};
        int32_t sizes = 0;
        a.num_experts = experts, a.n = n, a.k = k, a.num_rows = rows, a.swiglu = swiglu != 0;
        a.expert_rows = &sizes;
        const ep::Plan p = ep::plan(a);
        printf("%d %d %d\n", p.rows, p.cols, p.threads);
    }
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    where = tmp_path_factory.mktemp("choice")
    src, exe = where / "choice.hip", where / "choice"
    src.write_text(PROGRAM)
    flags = [f for f in hip_build.FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run(["hipcc", *flags, str(src), "-o", str(exe)], check=True, capture_output=True)

    def run(cases):
        text = "\n".join(" ".join(str(v) for v in c) for c in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]

    return run


def test_cases_reach_their_kernels(choose):
    names = sorted(loops.KERNELS)
    cases = []
    for name in names:
        (swiglu, *_), sizes, n, blocks = loops.KERNELS[name]
        cases += [(len(sizes), n, 128 * b, sum(sizes), int(swiglu)) for b in blocks]
    got = iter(choose(cases))
    for name in names:
        (_, *block), _, _, blocks = loops.KERNELS[name]
        for b in blocks:
            assert next(got) == tuple(block), (name, b)


def test_every_kernel_has_a_case(choose):
    sizes = [1, 2, 5, 12, 16, 20, 32, 40, 64, 90, 128, 200, 500, 1000, 3000, 10000]
    cases = [(e, n, 1024, r * e, s) for e in (1, 2, 8, 32, 64, 300) for n in (128, 512, 2048, 8192) for r in sizes for s in (0, 1)]
    picked = {(s, *block) for (_, _, _, _, s), block in zip(cases, choose(cases))}
    assert picked == {(int(kernel[0]), *kernel[1:]) for kernel, *_ in loops.KERNELS.values()}
