"""launch_after (gq_sm100.cuh) reports a launch that the runtime refuses and
takes the error from it, so that the next call of the library, or of anything
else in the process, does not report it again.  Host code with a fake of the
runtime's launch and error calls."""
import subprocess

SOURCE = r"""
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdio>
static cudaError_t refuse = cudaErrorInvalidConfiguration, last = cudaSuccess;
template <typename... A>
static cudaError_t fake_launch(A&&...) { return refuse == cudaSuccess ? refuse : last = refuse; }
static cudaError_t fake_last() { const cudaError_t e = last; last = cudaSuccess; return e; }
#define cudaLaunchKernelEx fake_launch
#define cudaGetLastError fake_last
#include "gq_sm100.cuh"
static void kernel(int) {}
int main() {
  int status = gq::launch_after(kernel, dim3(1), dim3(2048), 0, nullptr, 1);
  std::printf("%d %d ", status, (int)last);
  refuse = cudaSuccess;
  last = cudaErrorInvalidValue;  // of an earlier call: not this one's to take
  status = gq::launch_after(kernel, dim3(1), dim3(32), 0, nullptr, 1);
  std::printf("%d %d", status, (int)last);
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
    # GQ_ERR_CUDA and nothing left behind; GQ_OK and cudaErrorInvalidValue
    assert out.split() == ["4", "0", "0", "1"]


def test_kernels_that_wait_for_the_one_before_promise_nothing_about_their_inputs():
    """A `const T* __restrict__` parameter says that its data do not change
    while the kernel runs, so its loads may be moved up past grid_wait(),
    behind which alone the kernel before has written them."""
    import glob
    import re
    from quantized_gnn_message_gb300 import build
    seen = 0
    for path in glob.glob(build.CSRC + "/*.cu"):
        with open(path, encoding="utf-8") as f:
            text = build._code_only(f.read())
        for kernel in re.split(r"\b__global__\b", text)[1:]:
            head, _, rest = kernel.partition("{")
            body = re.split(r"\n}", rest)[0]
            if "grid_wait()" in body:
                seen += 1
                assert "__restrict__" not in head, f"{path}: {head.split('(')[0].split()[-1]}"
    assert seen >= 6
