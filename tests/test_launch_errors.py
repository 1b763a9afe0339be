"""launch_after (gq_sm100.cuh) reports a launch that the runtime refuses and
takes the error from it, so that the next call of the library, or of anything
else in the process, does not report it again.  The launch is refused on any
machine: by its block size, or for want of a device."""
import subprocess

SOURCE = r"""
#include "gq_sm100.cuh"
#include <cstdio>
__global__ void kernel(int) {}
int main() {
  const int status = gq::launch_after(kernel, dim3(1), dim3(2048), 0, nullptr, 1);
  std::printf("%d %d", status, (int)cudaPeekAtLastError());
  return 0;
}
"""


def test_a_refused_launch_leaves_no_error_behind(tmp_path):
    from quantized_gnn_message_gb300 import build
    src, exe = tmp_path / "refused.cu", tmp_path / "refused"
    src.write_text(SOURCE)
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I" + build.INCLUDE, "-I" + build.CSRC, str(src), "-o",
                    str(exe)], check=True, capture_output=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    status, left = map(int, out.split())
    assert status == 4 and left == 0  # GQ_ERR_CUDA, cudaSuccess
