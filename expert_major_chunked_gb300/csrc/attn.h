// Internal declarations of the attention operators: the kernels (attn_prefill.cu, attn_decode.cu, kv_cache.cu) and
// their C entries (attention.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "../../include/moe_attention.h"

namespace moe {

constexpr int kAssignMaxRequests = 16384;

cudaError_t launch_kv_assign(const moe_kv_assign_args& a, cudaStream_t stream);
cudaError_t launch_kv_append(const moe_kv_append_args& a, cudaStream_t stream);
cudaError_t launch_attn_prefill(const moe_attn_prefill_args& a, cudaStream_t stream);
size_t attn_decode_workspace(int n_requests, int n_heads, int n_kv_heads, int head_dim);
cudaError_t launch_attn_decode(const moe_attn_decode_args& a, cudaStream_t stream);

// Waits for the stream, reads moe_attn_prefill's error word and clears it (0: no wait in the kernel gave up).
cudaError_t attn_prefill_take_error(int* site, cudaStream_t stream);

constexpr int kMaxDevices = 64;  // ordinals that the C entries take

// What has to be done once on each device, such as a kernel's attributes; an attempt that fails is made again. (Threads
// that come first together may both do it.)
class OncePerDevice {
 public:
  template <class F>
  cudaError_t operator()(F prepare) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = prepare();
    if (e == cudaSuccess) done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<bool> done_[kMaxDevices] = {};
};

// Launches a kernel whose set-up may run beside the end of the work before it in the stream: the kernel waits for that
// work (griddepcontrol.wait) before it touches global memory. Back to back, a call of a few microseconds otherwise takes
// whole multiples of 2 us (64 single tokens into the cache: 6.1 us a call against 3.1). Letting the next kernel in at the
// start of this one (let_next_start) gained nothing more, as CTAs that wait take room and issue slots (that call 3.6 us;
// slots of 1024 requests 10.0 us against 7.7); only the decode kernel does it, for its join.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);  // (the runtime's last error may be some earlier call's)
}

// cuTensorMapEncodeTiled of the driver, or nullptr
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();

}  // namespace moe
