"""A mixture-of-experts plan runs on the GPU that it was made for: with another one current every call is
refused on the host, before any launch.  The host side of csrc/moe.cu runs here over a fake of
cudaGetDevice (moe_device_client.cu), its kernels compiled to PTX only and with no GPU visible."""
import os
import subprocess

from tile_scheduled_tensor_gb300 import build

TESTS = os.path.dirname(os.path.abspath(__file__))


def test_calls_with_another_gpu_current_are_refused(tmp_path):
    exe = str(tmp_path / "moe_device_client")
    subprocess.check_call([build._nvcc(), "-arch=compute_103a", "-code=compute_103a", "-Xcicc", "-O0", "-std=c++17", "-diag-suppress", "177",
                           f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-o", exe, os.path.join(TESTS, "moe_device_client.cu")])
    r = subprocess.run([exe], env=dict(os.environ, CUDA_VISIBLE_DEVICES=""), capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
