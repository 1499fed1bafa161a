"""Host-side checks of the adapter, checkpoint and input-gradient entry points (no GPU): what
they refuse, empty calls, workspace sizes; and the ABI layer under AddressSanitizer and
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
BIG = 1 << 40


def _forward(b=4, m=256, n=32, r=16, count=2, type=0, x=A, at=A, bt=A, scale=A, plan=A, pb=BIG, y=A, out=A, h=A, ws=A,
             wsb=BIG):
    return twq.lib().twq_adapters(x, at, bt, scale, plan, pb, y, out, h, b, m, n, r, count, type, ws, wsb, None)


def _grad(b=4, m=256, n=32, r=16, count=2, type=0, dy=A, x=A, qc=None, sc=None, h=A, at=A, bt=A, scale=A, plan=A, pb=BIG,
          dx=A, dxo=A, dat=A, dbt=A, ws=A, wsb=BIG):
    return twq.lib().twq_adapters_grad(dy, x, qc, sc, h, at, bt, scale, plan, pb, dx, dxo, dat, dbt, b, m, n, r, count,
                                       type, ws, wsb, None)


def _dx(b=4, m=256, n=32, r=16, type=0, dy=A, qw=A, sw=A, l1t=A, l2t=A, dx=A, ws=A, wsb=BIG):
    return twq.lib().twq_linear_dx(dy, qw, sw, l1t, l2t, r, dx, b, m, n, type, ws, wsb, None)


@pytest.mark.parametrize("call", [_forward, _grad, _dx])
def test_refused_shapes_and_types(call):
    for bad in (dict(m=100), dict(m=0), dict(m=131200), dict(n=0), dict(n=24), dict(n=-16), dict(n=(1 << 22) + 16),
                dict(r=8), dict(r=272), dict(r=-16), dict(b=-1), dict(b=(1 << 24) + 1), dict(b=1 << 24, n=1 << 20)):
        assert call(**bad) == SHAPE, bad
    assert call(type=2) == UNSUPPORTED and call(type=-1) == UNSUPPORTED
    if call is not _dx:
        assert call(r=0) == SHAPE and call(count=-1) == SHAPE and call(count=4097) == SHAPE


def test_refused_pointers():
    for name in ("x", "at", "bt", "plan", "out"):
        assert _forward(**{name: None}) == NULL, name
    for name in ("x", "at", "bt", "plan", "out", "scale", "y", "h", "ws"):
        assert _forward(**{name: MIS}) == ALIGN, name
    for name in ("dy", "h", "at", "bt", "plan", "dxo", "dat", "dbt", "x"):
        assert _grad(**{name: None}) == NULL, name
    assert _grad(x=None, qc=A) == NULL and _grad(x=None, sc=A) == NULL
    assert _grad(qc=A, sc=A) == UNSUPPORTED  # whole and 8-bit activations at once
    for name in ("dy", "h", "at", "bt", "plan", "dxo", "dat", "dbt", "x", "scale", "dx", "ws"):
        assert _grad(**{name: MIS}) == ALIGN, name
    for name in ("dy", "qw", "sw", "dx", "l1t", "l2t"):
        assert _dx(**{name: None}) == NULL, name
        assert _dx(**{name: MIS}) == ALIGN, name
    L = twq.lib()
    assert L.twq_adapter_plan(None, 4, 2, A, BIG, None) == NULL
    assert L.twq_adapter_plan(A, 4, 2, None, BIG, None) == NULL
    assert L.twq_adapter_plan(MIS, 4, 2, A, BIG, None) == ALIGN
    assert L.twq_adapter_plan(A, -1, 2, A, BIG, None) == SHAPE
    assert L.twq_adapter_plan(A, 4, 5000, A, BIG, None) == SHAPE
    for fn, args in ((L.twq_checkpoint_act, lambda x, q, s, b=4, m=256, t=0: (x, b, m, t, q, s, None)),
                     (L.twq_restore_act, lambda x, q, s, b=4, m=256, t=0: (q, s, b, m, t, x, None))):
        assert fn(*args(None, A, A)) == NULL and fn(*args(A, None, A)) == NULL and fn(*args(A, A, None)) == NULL
        assert fn(*args(MIS, A, A)) == ALIGN and fn(*args(A, MIS, A)) == ALIGN and fn(*args(A, A, MIS)) == ALIGN
        assert fn(*args(A, A, A, m=192)) == SHAPE and fn(*args(A, A, A, b=-1)) == SHAPE
        assert fn(*args(A, A, A, t=7)) == UNSUPPORTED
        assert fn(*args(None, None, None, b=0)) == OK


def test_workspaces_and_plan_sizes():
    L = twq.lib()
    need = L.twq_adapter_plan_bytes(64, 5)
    assert need >= 64 * 4 and L.twq_adapter_plan_bytes(-1, 5) == 0 and L.twq_adapter_plan_bytes(4, 5000) == 0
    assert L.twq_adapter_plan(A, 64, 5, A, need - 1, None) == WORKSPACE
    need = L.twq_adapters_workspace_bytes(300, 4096, 512, 64, 5)
    assert need >= 300 * 64 * 4 and L.twq_adapters_workspace_bytes(300, 100, 512, 64, 5) == 0
    assert _forward(300, 4096, 512, 64, 5, wsb=need - 1) == WORKSPACE
    assert _forward(300, 4096, 512, 64, 5, ws=None) == WORKSPACE
    assert _forward(300, 4096, 512, 64, 5, pb=64) == WORKSPACE
    need = L.twq_adapters_grad_workspace_bytes(300, 4096, 512, 64, 5)
    assert need > 0 and _grad(300, 4096, 512, 64, 5, wsb=need - 1) == WORKSPACE
    need = L.twq_linear_dx_workspace_bytes(16, 4096, 4096, 32)
    assert need >= 16 * 4096 * 2 and _dx(16, 4096, 4096, 32, wsb=need - 1) == WORKSPACE
    assert L.twq_linear_dx_workspace_bytes(16, 4096, 4100, 32) == 0


def test_refused_launch_sizes():
    """(b / 64 + count + 1) ((m + n) / 128 + 2) stays below 2^24."""
    L = twq.lib()
    n = 128 * (2 ** 24 // 4161 - 2) // 16 * 16 - 256  # 4096 rows of 4096 adapters: 4160 tiles
    assert L.twq_adapters_workspace_bytes(4096, 256, n, 16, 4096) > 0
    assert L.twq_adapters_grad_workspace_bytes(4096, 256, n, 16, 4096) > 0
    n += 2048
    assert L.twq_adapters_workspace_bytes(4096, 256, n, 16, 4096) == 0
    assert L.twq_adapters_grad_workspace_bytes(4096, 256, n, 16, 4096) == 0
    assert _forward(4096, 256, n, 16, 4096) == SHAPE and _grad(4096, 256, n, 16, 4096) == SHAPE
    assert L.twq_adapters_workspace_bytes(4096, 256, n, 16, 4000) > 0  # fewer adapters


def test_empty_calls_launch_nothing():
    nothing = dict(x=None, at=None, bt=None, scale=None, plan=None, pb=0, y=None, out=None, h=None, ws=None, wsb=0)
    assert _forward(b=0, **nothing) == OK
    assert _grad(b=0, count=0, dy=None, x=None, h=None, at=None, bt=None, scale=None, plan=None, pb=0, dx=None, dxo=None,
                 dat=None, dbt=None, ws=None, wsb=0) == OK
    assert _dx(b=0, dy=None, qw=None, sw=None, l1t=None, l2t=None, dx=None, ws=None, wsb=0) == OK


def test_binding_refuses_cpu_tensors_and_wrong_types():
    h = torch.zeros(4, 256, dtype=torch.float16)
    with pytest.raises(ValueError):
        twq.checkpoint_act(h)
    with pytest.raises(TypeError):
        twq.checkpoint_act(h.float())
    with pytest.raises(ValueError):
        twq.restore_act(torch.zeros(4, 256, dtype=torch.int8), torch.zeros(2, 4))
    with pytest.raises(ValueError):
        twq.adapter_plan(torch.zeros(4, dtype=torch.int32), 2)
    plan = twq.AdapterPlan(torch.zeros(64, dtype=torch.uint8), 4, 1)
    with pytest.raises(ValueError):
        twq.adapters(h, h.view(1, 4, 256), h.view(1, 256, 4), plan, h)
    with pytest.raises(ValueError):
        twq.adapters_grad(h, h, h, h.view(1, 4, 256), h.view(1, 256, 4), plan)
    with pytest.raises(ValueError):
        twq.linear_dx(h, torch.zeros(256, 128, dtype=torch.uint8), torch.zeros(256))


def test_adapter_abi_under_asan_ubsan(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    exe = tmp_path / "adapters_driver"
    csrc = os.path.join(ROOT, "w4a4_rank_gemm_amd", "csrc")
    san = os.path.join(ROOT, "tests", "sanitize")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-fno-omit-frame-pointer", "-g", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"), "-I" + csrc, os.path.join(csrc, "adapters_api.cpp"),
                    os.path.join(csrc, "plan.cpp"), os.path.join(san, "adapters_stub.cpp"),
                    os.path.join(san, "adapters_driver.cpp"), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    assert "all calls returned the expected status" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
