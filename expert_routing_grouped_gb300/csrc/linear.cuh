// linear.cuh -- parameters and epilogue arithmetic shared by the kernels of
// moe_linear.
#pragma once

#include "moe_internal.cuh"

namespace moe {

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
cudaError_t launch_linear_tc(const LinearParams &p, int dtype, cudaStream_t st);

// sx sw acc + bias, the pre-activation of row n of w.
static __device__ __forceinline__ float finish_acc(const LinearParams &p, float acc, float sx, int n) {
  if (p.w_scale) acc *= sx * p.w_scale[n];
  return p.bias ? acc + p.bias[n] : acc;
}

static __device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

static __device__ __forceinline__ float activate(int act, float v) {
  if (act == MOE_ACT_SILU) return silu(v);
  if (act == MOE_ACT_GELU) return 0.5f * v * erfcf(-v * 0.70710678118654752f);
  return v;
}

static __device__ __forceinline__ float swiglu(float gate, float up) { return silu(gate) * up; }

static __device__ __forceinline__ float load_resid(const LinearParams &p, int t, int n) {
  if (!p.resid) return 0.f;
  const size_t i = (size_t)t * p.ldr + n;
  return p.out_dtype == MOE_BF16
             ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.resid)[i])
             : reinterpret_cast<const float *>(p.resid)[i];
}

static __device__ __forceinline__ void store_out(const LinearParams &p, int t, int n, float y) {
  const size_t i = (size_t)t * p.ldo + n;
  if (p.out_dtype == MOE_BF16) reinterpret_cast<__nv_bfloat16 *>(p.out)[i] = __float2bfloat16_rn(y);
  else reinterpret_cast<float *>(p.out)[i] = y;
}

}  // namespace moe
