"""Host-side checks of the 16-bit-activation and routed-layer entry points (no GPU): what they refuse,
empty calls, workspace sizes; and the ABI layer under AddressSanitizer and
UndefinedBehaviorSanitizer with host stand-ins for the kernels."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import w4a4_rank_gemm_amd as twq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 6
A = ctypes.c_void_p(4096)
MIS = ctypes.c_void_p(4096 + 8)
MIS4 = ctypes.c_void_p(4096 + 2)  # ids, weights and bias need 4 bytes
BIG = 1 << 46


def _a16(b=4, m=256, n=32, r=16, g=128, type=0, x=A, qw=A, sw=A, l1t=A, l2t=A, y=A, ws=A, wsb=BIG):
    return twq.lib().twq_linear_a16(x, qw, sw, l1t, l2t, r, y, b, m, n, g, type, ws, wsb, None)


def _route(b=4, m=256, experts=8, k=2, score=0, norm=1, scale=1.0, type=0, x=A, wr=A, bias=A, ids=A, w=A, ws=A, wsb=BIG):
    return twq.lib().twq_moe_route(x, wr, bias, b, m, experts, k, score, norm, scale, type, ids, w, ws, wsb, None)


def _experts(b=4, m=256, f=128, experts=8, k=2, g=128, type=0, x=A, ids=A, w=A, q1=A, s1=A, q2=A, s2=A, y=A, ws=A, wsb=BIG):
    return twq.lib().twq_moe_experts(x, ids, w, q1, s1, q2, s2, y, b, m, f, experts, k, g, type, ws, wsb, None)


def _moe(b=4, m=256, f=128, experts=8, k=2, g=128, score=0, norm=1, scale=1.0, type=0, x=A, wr=A, bias=A, q1=A, s1=A, q2=A,
         s2=A, y=A, ws=A, wsb=BIG):
    return twq.lib().twq_moe(x, wr, bias, q1, s1, q2, s2, y, b, m, f, experts, k, g, score, norm, scale, type, ws, wsb, None)


def test_refused_shapes_and_types():
    for bad in (dict(m=100), dict(m=0), dict(m=131200), dict(n=24), dict(n=-16), dict(n=(1 << 22) + 16), dict(r=8),
                dict(r=272), dict(r=-16), dict(b=-1), dict(b=(1 << 24) + 1), dict(b=1 << 24, n=1 << 20)):
        assert _a16(**bad) == SHAPE, bad
    for call in (_a16, _route, _experts, _moe):
        assert call(type=2) == UNSUPPORTED and call(type=-1) == UNSUPPORTED
    for call in (_a16, _experts, _moe):
        assert call(g=64) == UNSUPPORTED
    for call in (_route, _moe):
        assert call(score=2) == UNSUPPORTED and call(score=-1) == UNSUPPORTED
        assert call(k=9) == SHAPE  # more than experts
    for call in (_route, _experts, _moe):
        for bad in (dict(m=100), dict(m=0), dict(m=131200), dict(b=-1), dict(b=257), dict(experts=0), dict(experts=513),
                    dict(k=0), dict(k=17), dict(k=-1)):
            assert call(**bad) == SHAPE, bad
    for call in (_experts, _moe):
        for bad in (dict(f=0), dict(f=64), dict(f=-128), dict(f=131200), dict(experts=512, f=16512), dict(experts=512, m=32896)):
            assert call(**bad) == SHAPE, bad


def test_outputs_of_one_call():
    """b n at most 2^37."""
    assert _a16(b=1 << 24, n=(1 << 13) + 16) == SHAPE and _a16(b=1 << 16, n=(1 << 21) + 16) == SHAPE
    assert twq.lib().twq_linear_a16_workspace_bytes(1 << 24, 128, (1 << 13) + 16, 0, 128) == 0
    assert twq.lib().twq_linear_a16_workspace_bytes(1 << 24, 128, 1 << 13, 0, 128) > 0


def test_refused_pointers():
    for call, names, optional in ((_a16, ("x", "qw", "sw", "l1t", "l2t", "y"), ()),
                                  (_route, ("x", "wr", "ids", "w"), ("bias",)),
                                  (_experts, ("x", "ids", "w", "q1", "s1", "q2", "s2", "y"), ()),
                                  (_moe, ("x", "wr", "q1", "s1", "q2", "s2", "y"), ("bias",))):
        for name in names:
            assert call(**{name: None}) == NULL, (call, name)
        for name in names + optional + ("ws",):
            assert call(**{name: MIS4 if name in ("ids", "w", "bias") else MIS}) == ALIGN, (call, name)


def test_workspaces():
    L = twq.lib()
    assert L.twq_linear_a16_workspace_bytes(1, 4096, 4096, 0, 128) == 0  # one launch
    assert L.twq_linear_a16_workspace_bytes(9, 512, 4096, 16, 128) == 0
    for b, m, n, r in ((1, 4096, 4096, 16), (16, 4096, 64, 32), (61, 14336, 4096, 0), (500, 256, 16384, 0), (3000, 4096, 512, 64)):
        need = L.twq_linear_a16_workspace_bytes(b, m, n, r, 128)
        assert need > 0 and _a16(b, m, n, r, wsb=need - 1) == WORKSPACE and _a16(b, m, n, r, ws=None) == WORKSPACE
    assert L.twq_linear_a16_workspace_bytes(500, 256, 16384, 0, 128) >= 500 * 256 * 2
    assert L.twq_linear_a16_workspace_bytes(500, 256, 16384, 0, 64) == 0 and L.twq_linear_a16_workspace_bytes(4, 100, 32, 0, 128) == 0
    need = L.twq_moe_route_workspace_bytes(9, 4096, 77, 3)
    assert need >= 9 * 77 * 8 and _route(9, 4096, 77, 3, wsb=need - 1) == WORKSPACE and _route(9, 4096, 77, 3, ws=None) == WORKSPACE
    part = L.twq_moe_experts_workspace_bytes(9, 256, 384, 77, 3)
    assert part >= 27 * 384 * 4 and _experts(9, 256, 384, 77, 3, wsb=part - 1) == WORKSPACE
    need = L.twq_moe_workspace_bytes(9, 256, 384, 77, 3)
    assert need >= part + 27 * 8 and _moe(9, 256, 384, 77, 3, wsb=need - 1) == WORKSPACE
    assert L.twq_moe_experts_workspace_bytes(2, 256, 128, 2, 3) > 0  # a given choice may name an expert twice
    assert L.twq_moe_workspace_bytes(2, 256, 128, 2, 3) == 0 and L.twq_moe_route_workspace_bytes(257, 256, 8, 2) == 0


def test_empty_calls_launch_nothing():
    assert _a16(b=0, x=None, qw=None, sw=None, l1t=None, l2t=None, y=None, ws=None, wsb=0) == OK
    assert _a16(n=0, x=None, qw=None, sw=None, l1t=None, l2t=None, y=None, ws=None, wsb=0) == OK
    assert _route(b=0, x=None, wr=None, bias=None, ids=None, w=None, ws=None, wsb=0) == OK
    assert _experts(b=0, x=None, ids=None, w=None, q1=None, s1=None, q2=None, s2=None, y=None, ws=None, wsb=0) == OK
    assert _moe(b=0, x=None, wr=None, bias=None, q1=None, s1=None, q2=None, s2=None, y=None, ws=None, wsb=0) == OK


def test_binding_refuses_cpu_tensors_and_wrong_types():
    h, q = torch.zeros(4, 256, dtype=torch.float16), torch.zeros(32, 128, dtype=torch.uint8)
    q3 = torch.zeros(8, 256, 128, dtype=torch.uint8)
    for call in (lambda x: twq.linear_a16(x, q, torch.zeros(2, 32)), lambda x: twq.moe_route(x, x, 1),
                 lambda x: twq.moe_experts(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), (q3, x), (q3, x)),
                 lambda x: twq.moe(x, x, 1, (q3, x), (q3, x))):
        with pytest.raises(ValueError):
            call(h)
        with pytest.raises(TypeError):
            call(h.float())
        with pytest.raises(TypeError):
            call([h])
    with pytest.raises(ValueError):
        twq.pack_experts(torch.zeros(2, 32, 128))


def test_moe_abi_under_asan_ubsan(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    exe = tmp_path / "moe_driver"
    csrc = os.path.join(ROOT, "w4a4_rank_gemm_amd", "csrc")
    san = os.path.join(ROOT, "tests", "sanitize")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-fno-omit-frame-pointer", "-g", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"), "-I" + csrc, os.path.join(csrc, "moe_api.cpp"),
                    os.path.join(csrc, "plan.cpp"), os.path.join(san, "moe_driver.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    assert "all calls returned the expected status" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
