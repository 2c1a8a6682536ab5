// csrc/moe_device.cuh with a CUDA runtime of several devices that only remembers what it was asked.
enum cudaError_t { cudaSuccess = 0, cudaErrorInvalidValue = 1, cudaErrorNoDevice = 100 };
enum cudaFuncAttribute { cudaFuncAttributeMaxDynamicSharedMemorySize = 8 };

namespace {
int g_device, g_calls, g_bytes[100];
cudaError_t g_device_error, g_set_error;
cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return g_device_error;
}
template <class K>
cudaError_t cudaFuncSetAttribute(K*, cudaFuncAttribute, int bytes) {
  ++g_calls;
  if (g_set_error == cudaSuccess) g_bytes[g_device] = bytes;
  return g_set_error;
}
}  // namespace
#include "../nvfp4_expert_gemms_gb300/csrc/moe_device.cuh"

namespace {
void kernel() {}
moe::SmemOptIn g_opt_in;
moe::PerDevice g_number;
}  // namespace

extern "C" {
// One opt-in on device `dev` while the runtime's two functions return these errors: what it returns; calls: how often
// the attribute was set so far; bytes: what the device has.
int opt_in(int dev, int device_error, int set_error, int bytes, int* calls, int* has) {
  g_device = dev;
  g_device_error = (cudaError_t)device_error;
  g_set_error = (cudaError_t)set_error;
  const int e = g_opt_in(kernel, bytes);
  *calls = g_calls;
  *has = g_bytes[dev];
  return e;
}
// The number of device `dev` after adding `by` to it; -1: there is none.
int number(int dev, int by) {
  g_device = dev;
  g_device_error = cudaSuccess;
  std::atomic<int>* at;
  if (g_number.here(&at) != cudaSuccess || !at) return -1;
  return *at += by;
}
}
