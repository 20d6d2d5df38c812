"""The host's rules of the 8-bit products, on the CPU: tests/q8c_host_rules.cu
calls them over types, sizes and addresses.  No GPU is touched."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_host_rules(tmp_path):
    from gguf_block_quantized_qmatmul_gb300 import build
    build.build()
    exe = str(tmp_path / "q8c_host_rules")
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.CSRC, "-o", exe, os.path.join(ROOT, "tests", "q8c_host_rules.cu"),
                    build.LIB, "-Xlinker", "-rpath", "-Xlinker", build.BUILD], check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-4000:]
    assert r.stdout.startswith("ok "), r.stdout
