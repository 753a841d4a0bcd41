// Host checks shared by the streaming-block operators.
#include "stream_ops.cuh"

#include <atomic>

namespace gam {
namespace ops {

gam_status check_device(int* sms) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];  // 0: not asked yet, -1: not a B200, else its SMs
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess)
    return op_fail(GAM_ERR_UNSUPPORTED_DEVICE, std::string("no CUDA device: ") + cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return op_fail(GAM_ERR_UNSUPPORTED_DEVICE, "device index above 63");
  int v = known[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    int major = 0, minor = 0, n = 0;
    e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
      return op_fail(GAM_ERR_CUDA, std::string("cudaDeviceGetAttribute: ") + cudaGetErrorString(e));
    v = major == 10 && minor == 0 ? n : -1;
    known[dev].store(v, std::memory_order_relaxed);
  }
  if (v < 0) return op_fail(GAM_ERR_UNSUPPORTED_DEVICE, "device is not compute capability 10.0 (B200 / sm_100a)");
  *sms = v;
  return GAM_OK;
}

gam_status launch_status(cudaError_t e) {
  if (e == cudaSuccess) return GAM_OK;
  cudaGetLastError();  // reported here, so not to the caller's next check
  return op_fail(GAM_ERR_CUDA, std::string("launch: ") + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")");
}

}  // namespace ops
}  // namespace gam
