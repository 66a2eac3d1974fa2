// norm.cu -- the RMS norm that adds into the residual stream and can round to
// 8 bits (moe_add_rmsnorm in include/moe.h).
//
//   r = resid + x (rounded to resid's type; without resid r = x), resid_out = r
//   n_i = r_i * rstd * gain_i,  rstd = 1 / sqrt(mean(r^2) + eps)
//   bf16 out: bf16(n_i)
//   e4m3 out: per group g (the row, or 32 / 64 / 128 values of it)
//             s_g = max(max |n_i| / 448, 2^-126), q_i = e4m3(n_i / s_g)
//
// Since max |n_i| = rstd * max |r_i gain_i|, the sum of squares and the
// largest |r gain| of a row are reduced together, and the row is read once and
// held in registers from its load to its last store: one block per row, 8
// values (16 bytes of bf16, 32 of f32) per thread and step.
//
// Memory bound: 4096 rows of 6144, f32 onto an f32 stream with bf16 out, take
// 53.3 us (6.6 TB/s, 0.97 of a copy's rate); bf16 onto f32 with e4m3 out 48.1
// us (5.8 TB/s).  One row takes 2.7 us: launch and one memory round trip.
#include <algorithm>

#include "area.cuh"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kNormMaxH = 32768;   // 1024 threads x 4 steps x 8 values
constexpr int kNoResid = 2;        // RT: no residual stream (else 0 f32, 1 bf16)

struct NormParams {
  const void *x, *resid;
  void *resid_out;
  const float *gain;     // [H] or nullptr
  void *out;
  float *scale;          // [T][H / group] (e4m3 out)
  int H, group;          // group: values per scale, H for one scale a row
  float eps;
  long long ldx, ldr, ldro, ldo;   // row strides in elements
};

template <int DT>
__device__ __forceinline__ void load8(const void *base, size_t i, float v[8]) {
  if constexpr (DT == MOE_BF16) {
    const uint4 u = *reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(base) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v[2 * c] = __uint_as_float(w[c] << 16);
      v[2 * c + 1] = __uint_as_float(w[c] & 0xFFFF0000u);
    }
  } else {
    const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(base) + i);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Four values in 8 bits (e4m3, to nearest, saturating; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// The bits of |v|: as unsigned numbers they order finite values, then
// infinity, then NaN, so an integer maximum carries a NaN through.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// XT, RT, OT: MOE_F32 / MOE_BF16 (RT also kNoResid), OT MOE_BF16 / MOE_E4M3.
// Thread i holds the row's 8-value pieces i, i + blockDim.x, ... (NV of them).
template <int XT, int RT, int OT, int NV>
__global__ void __launch_bounds__(NV == 8 ? 512 : 1024) add_rmsnorm_kernel(const NormParams p) {
  __shared__ float part[32];
  __shared__ uint32_t part_max[32];
  const int H = p.H, n8 = H / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const size_t t = blockIdx.x;
  const bool by_row = p.group == H;
  float r[NV][8];
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
#pragma unroll
    for (int c = 0; c < 8; ++c) r[j][c] = 0.f;
    if (i >= n8) continue;
    load8<XT>(p.x, t * p.ldx + (size_t)i * 8, r[j]);
    if constexpr (RT != kNoResid) {
      float a[8];
      load8<RT>(p.resid, t * p.ldr + (size_t)i * 8, a);
#pragma unroll
      for (int c = 0; c < 8; ++c) r[j][c] += a[c];
      if constexpr (RT == MOE_BF16) {
        // The norm is of the stream as it is kept: rounded to bf16.
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          w[c] = pack_bf16(r[j][2 * c], r[j][2 * c + 1]);
          r[j][2 * c] = __uint_as_float(w[c] << 16);
          r[j][2 * c + 1] = __uint_as_float(w[c] & 0xFFFF0000u);
        }
        *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(p.resid_out) + t * p.ldro +
                                   (size_t)i * 8) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        float4 *o = reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.resid_out) +
                                               t * p.ldro + (size_t)i * 8);
        o[0] = make_float4(r[j][0], r[j][1], r[j][2], r[j][3]);
        o[1] = make_float4(r[j][4], r[j][5], r[j][6], r[j][7]);
      }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) ss = fmaf(r[j][c], r[j][c], ss);
  }
  // Gain, and the largest |r gain| of this thread's pieces.
  uint32_t mx[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    mx[j] = 0u;
    if (i >= n8) continue;
    if (p.gain) {
      const float4 *g = reinterpret_cast<const float4 *>(p.gain + (size_t)i * 8);
      const float4 ga = __ldg(g), gb = __ldg(g + 1);
      r[j][0] *= ga.x, r[j][1] *= ga.y, r[j][2] *= ga.z, r[j][3] *= ga.w;
      r[j][4] *= gb.x, r[j][5] *= gb.y, r[j][6] *= gb.z, r[j][7] *= gb.w;
    }
    if constexpr (OT == MOE_E4M3) {
#pragma unroll
      for (int c = 0; c < 8; ++c) mx[j] = max(mx[j], abs_bits(r[j][c]));
    }
  }
  // Row sums in a fixed order: lanes, then warps.
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) part[warp] = ss;
  if constexpr (OT == MOE_E4M3) {
    if (by_row) {
      uint32_t m = mx[0];
#pragma unroll
      for (int j = 1; j < NV; ++j) m = max(m, mx[j]);
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) part_max[warp] = m;
    }
  }
  __syncthreads();
  float tot = 0.f;
  for (int w = 0; w < nw; ++w) tot += part[w];
  const float rstd = 1.0f / sqrtf(tot / (float)H + p.eps);
  if constexpr (OT == MOE_BF16) {
    __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16 *>(p.out) + t * p.ldo;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      if (i >= n8) continue;
      uint32_t w[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) w[c] = pack_bf16(r[j][2 * c] * rstd, r[j][2 * c + 1] * rstd);
      *reinterpret_cast<uint4 *>(o + (size_t)i * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    uint8_t *o = reinterpret_cast<uint8_t *>(p.out) + t * p.ldo;
    float sc, f, back;
    auto scale_of = [&](uint32_t m) {
      // NaN fails the comparison and stays.
      const float amax = __uint_as_float(m) * rstd / 448.0f;
      sc = amax < 1.17549435e-38f ? 1.17549435e-38f : amax;
      f = 1.0f / sc;
      back = f == 0.0f ? 0.0f : -sc;   // sc infinite: 0 or NaN
    };
    if (by_row) {
      uint32_t m = 0u;
      for (int w = 0; w < nw; ++w) m = max(m, part_max[w]);
      scale_of(m);
      if (threadIdx.x == 0) p.scale[t] = sc;
    }
    const int lanes = p.group / 8;   // threads of one group (4, 8 or 16 of a warp)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      uint32_t m = mx[j];
      if (!by_row)   // pieces of a group sit in neighbouring lanes (H is a multiple of the group)
        for (int d = 1; d < lanes; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
      if (i >= n8) continue;
      if (!by_row) scale_of(m);
      // n / sc as a product with 1 / sc and one correction by the remainder,
      // which makes the f32 quotient the nearest one (Markstein 1990): bf16 rows
      // meet ties between codes often, r / max being a ratio of 8-bit numbers,
      // and a product's rounding would decide them (1037 x 4096 in groups of
      // 128: 2 codes of 10^4).  rstd / sc alone could pass f32's range (a row
      // of zeros).
      float n[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float v = r[j][c] * rstd, q0 = v * f;
        n[c] = fmaf(fmaf(q0, back, v), f, q0);
      }
      uint2 q;
      q.x = pack_e4m3(n[0], n[1], n[2], n[3]);
      q.y = pack_e4m3(n[4], n[5], n[6], n[7]);
      *reinterpret_cast<uint2 *>(o + (size_t)i * 8) = q;
      if (!by_row && i % lanes == 0) p.scale[t * (size_t)(H / p.group) + i / lanes] = sc;
    }
  }
}

template <int XT, int RT, int OT>
cudaError_t launch_norm(const NormParams &p, int T, cudaStream_t st) {
  // Threads a row: 1024 at most, and 512 where every SM has rows enough for
  // several blocks, whose loads and stores then overlap (4096 rows of 6144,
  // e4m3: 47.7 us with 384 threads, 53.0 with 768; 64 rows: 3.4 either way).
  const int n8 = p.H / 8, most = T >= 304 ? 512 : 1024;
  const int nv = n8 <= most ? 1 : n8 <= 2 * most ? 2 : n8 <= 4 * most ? 4 : 8;
  const int threads = ((n8 + nv - 1) / nv + 31) / 32 * 32;
  auto k = nv == 1 ? add_rmsnorm_kernel<XT, RT, OT, 1>
                   : nv == 2 ? add_rmsnorm_kernel<XT, RT, OT, 2>
                   : nv == 4 ? add_rmsnorm_kernel<XT, RT, OT, 4> : add_rmsnorm_kernel<XT, RT, OT, 8>;
  return launch_k(false, k, dim3(T), dim3(threads), 0, st, p);
}

template <int XT, int RT>
cudaError_t launch_norm_o(const NormParams &p, int T, int out_dtype, cudaStream_t st) {
  return out_dtype == MOE_BF16 ? launch_norm<XT, RT, MOE_BF16>(p, T, st)
                               : launch_norm<XT, RT, MOE_E4M3>(p, T, st);
}

template <int XT>
cudaError_t launch_norm_r(const NormParams &p, int T, int rt, int out_dtype, cudaStream_t st) {
  if (rt == MOE_F32) return launch_norm_o<XT, MOE_F32>(p, T, out_dtype, st);
  if (rt == MOE_BF16) return launch_norm_o<XT, MOE_BF16>(p, T, out_dtype, st);
  return launch_norm_o<XT, kNoResid>(p, T, out_dtype, st);
}

}  // namespace
}  // namespace moe

extern "C" __attribute__((visibility("default"))) int moe_add_rmsnorm(
    const void *x, const void *resid, void *resid_out, const float *gain, int T, int H, float eps,
    int x_dtype, int resid_dtype, int out_dtype, int group, void *out, float *scale,
    int64_t x_stride, int64_t resid_stride, int64_t resid_out_stride, int64_t out_stride,
    moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || H < 8 || H % (out_dtype == MOE_E4M3 ? 16 : 8) || H > kNormMaxH || !(eps >= 0.f)) return MOE_ERR_ARG;
  if ((x_dtype != MOE_F32 && x_dtype != MOE_BF16) ||
      (resid_dtype != MOE_F32 && resid_dtype != MOE_BF16) ||
      (out_dtype != MOE_BF16 && out_dtype != MOE_E4M3))
    return MOE_ERR_ARG;
  if (out_dtype == MOE_E4M3) {
    if (group != 0 && group != 32 && group != 64 && group != 128) return MOE_ERR_ARG;
    if (group && H % group) return MOE_ERR_ARG;
  } else if (group) {
    return MOE_ERR_ARG;
  }
  const size_t xe = x_dtype == MOE_F32 ? 4 : 2, re = resid_dtype == MOE_F32 ? 4 : 2,
               oe = out_dtype == MOE_BF16 ? 2 : 1;
  const long long ldx = x_stride ? x_stride : H, ldr = resid_stride ? resid_stride : H,
                  ldro = resid_out_stride ? resid_out_stride : H, ldo = out_stride ? out_stride : H;
  constexpr long long kMaxStride = 1LL << 32;
  if (ldx < H || ldr < H || ldro < H || ldo < H || ldx > kMaxStride || ldr > kMaxStride ||
      ldro > kMaxStride || ldo > kMaxStride)
    return MOE_ERR_ARG;
  // Rows are read and written 16 bytes at a time (8 for the e4m3 output).
  if (((size_t)ldx * xe | (size_t)ldr * re | (size_t)ldro * re | (size_t)ldo * oe) & 15)
    return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !out || (out_dtype == MOE_E4M3 && !scale)) return MOE_ERR_ARG;
  if ((resid == nullptr) != (resid_out == nullptr)) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(resid) |
       reinterpret_cast<uintptr_t>(resid_out) | reinterpret_cast<uintptr_t>(out) |
       reinterpret_cast<uintptr_t>(gain)) & 15)
    return MOE_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(scale) & 3) return MOE_ERR_ARG;
  // Blocks run in any order, so what one writes no other may read: the output
  // and the scales are apart from everything else, and resid_out is either
  // resid itself (the same rows) or apart from what is read.
  const size_t n = T, h = H;
  const Area ax{x, n, h * xe, (size_t)ldx * xe}, ar{resid, n, h * re, (size_t)ldr * re},
      aro{resid_out, n, h * re, (size_t)ldro * re}, ao{out, n, h * oe, (size_t)ldo * oe},
      ag = area(gain, h * 4),
      as = area(scale, out_dtype == MOE_E4M3 ? n * (group ? h / group : 1) * 4 : 0);
  if (meet(ao, ax) || meet(ao, ar) || meet(ao, aro) || meet(ao, ag) || meet(as, ao) || meet(as, ax) ||
      meet(as, ar) || meet(as, aro) || meet(as, ag) || meet(aro, ax) || meet(aro, ag))
    return MOE_ERR_ARG;
  if (!(resid_out == resid && ldro == ldr) && meet(aro, ar)) return MOE_ERR_ARG;
  NormParams p{x, resid, resid_out, gain, out, scale, H, group ? group : H, eps,
               ldx, ldr, ldro, ldo};
  const int rt = resid ? resid_dtype : kNoResid;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = x_dtype == MOE_F32 ? launch_norm_r<MOE_F32>(p, T, rt, out_dtype, st)
                                             : launch_norm_r<MOE_BF16>(p, T, rt, out_dtype, st);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_DEVICE;
}
