"""The expert-layer part of the C ABI without a GPU: the library exports what include/ep_experts.h
declares, and malformed arguments are refused on the host before anything is launched."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ep_experts.h")


@pytest.fixture(scope="module")
def ep():
    from combine_ep_get_02_amd import ep as ep_mod

    if not os.path.exists(ep_mod.LIBRARY):
        import __graft_entry__

        __graft_entry__.build()
    return ep_mod


@pytest.fixture(scope="module")
def lib(ep):
    from combine_ep_get_02_amd import experts

    return experts.load()


def _declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return set(re.findall(r"\b(ep_[a-z0-9_]+)\s*\(", text))


def test_header_binding_and_library_agree(ep, lib):
    from combine_ep_get_02_amd import experts

    assert _declared() == set(experts.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", ep.LIBRARY], capture_output=True, text=True, check=True)
    assert _declared() <= set(re.findall(r"\bT (ep_\w+)", out.stdout))


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "ep_experts.h"\n_Static_assert(sizeof(ep_router_t) == 24, "six words");\n'
                   "int main(void) { return EP_DEV_BAD_LOGIT != 32; }\n")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", "/opt/rocm/include", "-fsyntax-only", str(src)], check=True)
    from combine_ep_get_02_amd import experts

    assert ctypes.sizeof(experts.ep_router_t) == 24


P = ctypes.c_void_p(256)    # never dereferenced: every call must fail its host checks first
ODD8 = ctypes.c_void_p(264)  # 8- but not 16-byte aligned
ODD4 = ctypes.c_void_p(260)
ODD2 = ctypes.c_void_p(258)
ODD1 = ctypes.c_void_p(257)


def _shape(ep, **kw):
    base = dict(num_tokens=64, hidden=256, num_topk=4, num_experts=64, num_ranks=8, num_channels=4)
    base.update(kw)
    return ep.make_shape(**base)


def _route(lib, s, r, logits=P, kind=0, stride=64, bias=P, mask=P, idx=P, w=P):
    return lib.ep_route(ctypes.byref(s), None if r is None else ctypes.byref(r), logits, kind, stride, bias, mask, idx,
                        w, None, None)


def _route_bwd(lib, s, r, logits=P, kind=0, stride=64, idx=P, g=P, out=P, out_stride=64):
    return lib.ep_route_backward(ctypes.byref(s), None if r is None else ctypes.byref(r), logits, kind, stride, idx, g,
                                 out, out_stride, None, None)


ROUTERS = {
    "score": dict(score=2), "no group": dict(num_groups=0), "uneven groups": dict(num_groups=7, groups_kept=2),
    "none kept": dict(num_groups=8, groups_kept=0), "too many kept": dict(num_groups=8, groups_kept=9),
    "best 0": dict(group_best=0), "best 3": dict(group_best=3), "scale inf": dict(weight_scale=float("inf")),
    "scale nan": dict(weight_scale=float("nan")),
}


@pytest.mark.parametrize("name", sorted(ROUTERS))
def test_bad_routers_refused(ep, lib, name):
    from combine_ep_get_02_amd import experts

    r = experts.make_router(**{"score": 1, **ROUTERS[name]})
    s = _shape(ep)
    assert _route(lib, s, r) == ep.EP_ERR_INVALID_ARG
    assert _route_bwd(lib, s, r) == ep.EP_ERR_INVALID_ARG


def test_bad_route_arguments_refused(ep, lib):
    from combine_ep_get_02_amd import experts

    r = experts.make_router(1)
    s = _shape(ep)
    bad = ep.EP_ERR_INVALID_ARG
    for kw in (dict(logits=None), dict(kind=2), dict(stride=63), dict(idx=None), dict(w=None), dict(logits=ODD2),
               dict(logits=ODD1, kind=1), dict(idx=ODD4), dict(w=ODD2), dict(bias=ODD2)):
        assert _route(lib, s, r, **kw) == bad, kw
    for kw in (dict(logits=None), dict(kind=2), dict(stride=63), dict(idx=None), dict(g=None), dict(out=None),
               dict(out_stride=63), dict(logits=ODD2), dict(out=ODD2), dict(out=ODD1, kind=1), dict(idx=ODD4),
               dict(g=ODD2)):
        assert _route_bwd(lib, s, r, **kw) == bad, kw
    assert _route(lib, s, None) == bad and _route_bwd(lib, s, None) == bad
    assert _route(lib, _shape(ep, hidden=12), r) == bad
    many = _shape(ep, num_experts=2056)
    assert _route(lib, many, r, stride=2056) == ep.EP_ERR_UNSUPPORTED
    assert _route_bwd(lib, many, r, stride=2056, out_stride=2056) == ep.EP_ERR_UNSUPPORTED
    groups = _shape(ep, num_experts=128 * 8)
    assert _route(lib, groups, experts.make_router(1, num_groups=128), stride=1024) == ep.EP_ERR_UNSUPPORTED
    many = _shape(ep, num_tokens=(1 << 25) + 1, num_ranks=1)
    assert _route(lib, many, r) == ep.EP_ERR_UNSUPPORTED and _route_bwd(lib, many, r) == ep.EP_ERR_UNSUPPORTED
    none = _shape(ep, num_tokens=0)
    assert _route(lib, none, r, logits=None, idx=None, w=None, bias=None, mask=None) == ep.EP_OK
    assert _route_bwd(lib, none, r, logits=None, idx=None, g=None, out=None) == ep.EP_OK


def _gemm(lib, swiglu=False, experts=4, n=256, k=256, x=P, xs=P, w=P, ws=P, rows=P, num_rows=64, out=P, outs=P):
    if swiglu:
        return lib.ep_expert_gemm_swiglu_fp8(experts, n, k, x, xs, w, ws, rows, num_rows, out, outs, None, None)
    return lib.ep_expert_gemm_fp8(experts, n, k, x, xs, w, ws, rows, num_rows, out, None, None)


@pytest.mark.parametrize("swiglu", [False, True])
def test_bad_product_arguments_refused(ep, lib, swiglu):
    bad = ep.EP_ERR_INVALID_ARG
    for kw in (dict(experts=0), dict(n=0), dict(n=252), dict(k=0), dict(k=192), dict(num_rows=-1), dict(x=None),
               dict(xs=None), dict(w=None), dict(ws=None), dict(out=None), dict(rows=None), dict(x=ODD8), dict(w=ODD8),
               dict(out=ODD8), dict(xs=ODD2), dict(ws=ODD2), dict(rows=ODD2)):
        assert _gemm(lib, swiglu, **kw) == bad, kw
    if swiglu:
        for kw in (dict(n=192), dict(outs=None), dict(outs=ODD2)):
            assert _gemm(lib, swiglu, **kw) == bad, kw
    for kw in (dict(experts=16385), dict(n=1 << 16, k=1 << 15), dict(k=(1 << 20) + 128),
               dict(n=1 << 14, num_rows=2147483647)):
        assert _gemm(lib, swiglu, **kw) == ep.EP_ERR_UNSUPPORTED, kw
    empty = dict(x=None, xs=None, w=None, ws=None, out=None, outs=None, num_rows=0)
    assert _gemm(lib, swiglu, **empty) == ep.EP_OK


def _combine(lib, s, y=P, idx=P, w=P, slot=P, pos=P, recv=8, rows=8, out=P):
    return lib.ep_combine_grouped(ctypes.byref(s), y, idx, w, slot, pos, recv, rows, out, None, None)


def _combine_bwd(lib, s, g=P, y=P, idx=P, w=P, slot=P, pos=P, row=P, num=P, recv=8, rows=8, gy=P, gw=P):
    return lib.ep_combine_grouped_backward(ctypes.byref(s), g, y, idx, w, slot, pos, row, num, recv, rows, gy, gw, None,
                                           None)


def test_bad_combine_arguments_refused(ep, lib):
    s = _shape(ep)
    bad = ep.EP_ERR_INVALID_ARG
    both = (dict(y=None), dict(idx=None), dict(w=None), dict(slot=None), dict(pos=None), dict(recv=-1), dict(rows=-1),
            dict(y=ODD8), dict(idx=ODD4), dict(w=ODD2), dict(slot=ODD2), dict(pos=ODD2))
    for kw in both + (dict(out=None), dict(out=ODD8)):
        assert _combine(lib, s, **kw) == bad, kw
    for kw in both + (dict(g=None), dict(g=ODD8), dict(row=None), dict(row=ODD2), dict(num=None), dict(num=ODD2),
                      dict(gy=None), dict(gy=ODD8), dict(gw=None), dict(gw=ODD2)):
        assert _combine_bwd(lib, s, **kw) == bad, kw
    assert _combine(lib, _shape(ep, num_experts=60)) == bad
    huge = _shape(ep, num_tokens=1 << 25, num_ranks=1)
    assert _combine(lib, huge) == ep.EP_ERR_UNSUPPORTED and _combine_bwd(lib, huge) == ep.EP_ERR_UNSUPPORTED
    none = _shape(ep, num_tokens=0)
    assert _combine(lib, none, y=None, idx=None, w=None, slot=None, pos=None, out=None) == ep.EP_OK
    assert _combine_bwd(lib, none, g=None, y=None, idx=None, w=None, slot=None, pos=None, row=None, num=None, recv=0,
                        rows=0, gy=None, gw=None) == ep.EP_OK


def test_binding_refuses_tensors_the_library_cannot_check(ep):
    from combine_ep_get_02_amd import experts

    s = _shape(ep)
    r = experts.make_router(experts.EP_SCORE_SIGMOID)
    cpu = torch.zeros(64, 64)
    idx, w = torch.zeros(64, 4, dtype=torch.int64), torch.zeros(64, 4)
    for logits in (None, cpu, cpu.double(), cpu[:32], cpu[:, :32], cpu.view(-1)):
        with pytest.raises(ValueError):
            experts.ep_route(s, r, logits, None, None, idx, w)
    with pytest.raises(ValueError):
        experts.ep_expert_gemm_fp8(1, 8, 128, torch.zeros(4, 128), None, None, None, None, 4, None)
    with pytest.raises(ValueError):
        experts.ep_combine_grouped(s, None, idx, w, None, None, 8, 8, None)
