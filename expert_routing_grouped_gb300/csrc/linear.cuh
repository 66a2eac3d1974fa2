// linear.cuh -- parameters and epilogue arithmetic shared by the kernels of
// moe_linear.
#pragma once

#include <atomic>

#include "moe_internal.cuh"

namespace moe {

// Runs f (a function attribute that lasts as long as the context) once for
// each device; again after an error.
struct DeviceOnce {
  std::atomic<unsigned long long> done{0};
  template <class F>
  cudaError_t run(F f) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    err = f();
    if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return err;
  }
};

struct LinearParams {
  const void *x, *w;
  const float *x_scale, *w_scale;   // e4m3: [T], [rows of w]
  const float *bias;                // [rows of w] or nullptr
  const void *resid;                // of out's type, or nullptr; may be out
  void *out;
  int T, N, K, act, out_dtype;
  long long ldx, ldw, ldr, ldo;     // row strides in elements
  int32_t *status;
};

// linear_tc.cu: more than kFewTokens tokens.
constexpr int kFewTokens = 16;
// The wait limit of what this host thread launches (moe_linear_wait_limit), and the
// current device's word for kernels without a status word (moe_linear_status).
unsigned long long linear_wait_ns();
cudaError_t linear_gave_up(int32_t **word);
cudaError_t launch_linear_tc(const LinearParams &p, int dtype, cudaStream_t st);

// sx sw acc + bias, the pre-activation of row n of w.
static __device__ __forceinline__ float finish_acc(const LinearParams &p, float acc, float sx, int n) {
  if (p.w_scale) acc *= sx * p.w_scale[n];
  return p.bias ? acc + p.bias[n] : acc;
}

// kFast, for a bf16 output: the hardware exponential (2 units and |v| 2^-24),
// far below the 2^-9 of the rounding that follows.  The quotient is the fast
// one (2 units of f32) either way.
template <bool kFast = false>
static __device__ __forceinline__ float silu(float v) {
  return __fdividef(v, 1.0f + (kFast ? __expf(-v) : expf(-v)));
}

static __device__ __forceinline__ float activate(int act, float v) {
  if (act == MOE_ACT_SILU) return silu(v);
  if (act == MOE_ACT_GELU) return 0.5f * v * erfcf(-v * 0.70710678118654752f);
  return v;
}

template <bool kFast = false>
static __device__ __forceinline__ float swiglu(float gate, float up) {
  return silu<kFast>(gate) * up;
}

// Residual and output elements, kBf16 the output type (of the whole kernel: a
// branch at each element would make every residual load wait for itself).
template <bool kBf16>
static __device__ __forceinline__ float load_resid(const LinearParams &p, int t, int n) {
  const size_t i = (size_t)t * p.ldr + n;
  if constexpr (kBf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.resid)[i]);
  return reinterpret_cast<const float *>(p.resid)[i];
}

template <bool kBf16>
static __device__ __forceinline__ void store_out(const LinearParams &p, int t, int n, float y) {
  const size_t i = (size_t)t * p.ldo + n;
  if constexpr (kBf16) reinterpret_cast<__nv_bfloat16 *>(p.out)[i] = __float2bfloat16_rn(y);
  else reinterpret_cast<float *>(p.out)[i] = y;
}

}  // namespace moe
