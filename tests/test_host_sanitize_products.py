"""The host code of the 8-bit integer and grouped products under AddressSanitizer and
UndefinedBehaviorSanitizer: their sources are compiled with both on the host
code, linked with tests/sanitize/product_checks.cpp, and run on the CPU.  No GPU
is used."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gradient_compression_distributed_lc_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang++"


@pytest.mark.timeout(300)
def test_product_host_code_under_address_and_ub_sanitizers(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANG)):
        pytest.skip("ROCm compilers not installed")
    common = ["-O1", "-g", "-std=c++17", "-I", os.path.join(ROOT, "include")]
    objects, running = [], []
    for name in ("q8.hip", "products.hip", "ckpt8_matrix.hip"):
        objects.append(str(tmp_path / (name + ".o")))
        running.append(subprocess.Popen(
            [HIPCC, "--offload-arch=gfx950", *common, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-fno-gpu-flush-denormals-to-zero", "-ffp-contract=off", "-Xarch_host", "-fsanitize=address",
             "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-omit-frame-pointer", "-c", "-x", "hip",
             os.path.join(CSRC, name), "-o", objects[-1]], stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL))
    assert [r.wait() for r in running] == [0, 0, 0]
    host_flags = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    drv, exe = str(tmp_path / "checks.o"), str(tmp_path / "checks")
    subprocess.run([CLANG, *common, *host_flags, "-fno-omit-frame-pointer", "-c",
                    os.path.join(ROOT, "tests", "sanitize", "product_checks.cpp"), "-o", drv], check=True,
                   capture_output=True)
    subprocess.run([CLANG, *host_flags, drv, *objects, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib",
                    "-o", exe], check=True, capture_output=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "product host checks ok" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
