"""The launch rules of plan.cpp and twq_adapters.h, evaluated on the host (tests/plan_driver.cpp)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def build(folder):
    exe = os.path.join(str(folder), "plan_driver")
    csrc = os.path.join(ROOT, "w4a4_rank_gemm_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + csrc,
                    os.path.join(csrc, "plan.cpp"), os.path.join(ROOT, "tests", "plan_driver.cpp"), "-o", exe],
                   check=True, capture_output=True, text=True)
    return exe


def ask(exe, lines):
    """One list of numbers a line."""
    text = "\n".join(" ".join(str(v) for v in line) for line in lines) + "\n"
    out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout
    return [[int(v) for v in line.split()] for line in out.splitlines()]
