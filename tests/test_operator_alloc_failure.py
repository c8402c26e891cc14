"""The C entry points of the training-step operators with host allocations that
fail: no exception leaves them, whichever allocation it is. Runs on the CPU:
no call reaches a GPU."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_exception_leaves_a_c_entry(tmp_path):
    from bf16_fp8_weight_amd import build

    exe = tmp_path / "alloc_failure"
    libdir = os.path.dirname(build.LIB_PATH)
    rocm = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "lib")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", build.INCLUDE,
                    os.path.join(ROOT, "tests", "c_abi", "alloc_failure.cpp"), "-o", str(exe), f"-L{libdir}", "-l:libwt.so",
                    f"-Wl,-rpath,{libdir}", f"-L{rocm}", "-lamdhip64", f"-Wl,-rpath,{rocm}"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "alloc failure ok" in r.stdout, r.stdout + r.stderr
