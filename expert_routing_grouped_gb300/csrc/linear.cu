// linear.cu -- the matrix product with bias, activation and residual in its
// epilogue (moe_linear in include/moe.h).
//
//   y[t][n] = act(sx[t] sw[n] sum_k x[t][k] w[n][k] + bias[n]) + resid[t][n]
//
// x and w both bf16, or both e4m3 with one f32 scale per row; f32 accumulation.
// SwiGLU takes 2N rows of w: y = silu(row n) * (row N + n).
#include <algorithm>

#include "area.cuh"
#include "linear.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------ few tokens --
// Warp-level MMAs with the weights as the B operand (8 rows) and the tokens as
// A (16 rows).  K order inside an MMA is free as long as both operands agree,
// so each lane takes 16 consecutive bytes of its row -- lane 4 g + q piece q of
// every 64 bytes of row g -- straight from memory into two MMAs' fragments.
// A block owns 8 outputs and splits K over its warps, 64 U bytes of each row
// at a time; partial sums meet in shared memory in warp order.  Reading w is
// the time: one bf16 token at K = 4096, SwiGLU of 14336, takes 34.9 us (6.7
// TB/s).  A ring of cp.async pieces in shared memory in place of the registers
// was slower at every size (K = 14336, N = 4096: 23.1 against 19.4 us), and so
// were 16 outputs a block.

template <int DT>
__device__ __forceinline__ void mma_m16n8(float c[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (DT == MOE_BF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// 16 bytes at `off` of a row of `bytes` (0: no row); w is read once and passes
// L1 by.
template <bool kOnce>
__device__ __forceinline__ uint4 load_piece(const uint8_t *row, int off, int bytes) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (off < bytes) {
    if constexpr (kOnce)
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "l"(row + off));
    else
      v = __ldg(reinterpret_cast<const uint4 *>(row + off));
  }
  return v;
}

// NB: row blocks of 8 per warp -- 1, or 2 (SwiGLU: the gate rows, then the up
// rows).  HI: more than 8 tokens.  W: warps.  kFold (bf16 operands, f32
// output): the MMAs truncate as they add, 1.8e-8 of the result each, so every
// four steps their sums are added in f32 to nearest (K = 14336: error 4.5e-7 in
// place of 1.8e-6, 19.7 us in place of 19.5); a bf16 output does not see it, and
// e4m3 operands lose too little to need it (4.5e-7 at K = 2^19).
// Each lane has four 16-byte pieces of w in flight whatever NB.
template <int DT, int NB, bool HI, int W, bool kFold>
__global__ void __launch_bounds__(W * 32, 32 / W) linear_few_kernel(const LinearParams p) {
  constexpr int TT = HI ? 16 : 8;
  __shared__ float red[W][TT][8 * NB];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int n0 = blockIdx.x * 8;
  constexpr int es = DT == MOE_BF16 ? 2 : 1;
  const int kb = p.K * es;                       // bytes of a row, a multiple of 16
  const int row_kb = n0 + g < p.N ? kb : 0;
  const int lo_kb = g < p.T ? kb : 0, hi_kb = HI && g + 8 < p.T ? kb : 0;
  const uint8_t *wr[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
    wr[b] = reinterpret_cast<const uint8_t *>(p.w) + ((size_t)(n0 + g) + (size_t)b * p.N) * p.ldw * es;
  const uint8_t *xl = reinterpret_cast<const uint8_t *>(p.x) + (size_t)g * p.ldx * es;
  const uint8_t *xh = xl + (size_t)8 * p.ldx * es;
  float c[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[b][i] = 0.f;
  // bf16: U units are fetched, then multiplied.  e4m3, whose MMAs take longer
  // beside half the bytes: two buffers of half as many, one on its way while
  // the other is at work (K = 14336, N = 4096: 13.1 us in place of 14.8; bf16
  // the other way round, 23.5 in place of 19.4).
  constexpr int B = DT == MOE_E4M3 ? 2 : 1, U = 4 / NB / B;
  uint4 wv[B][NB][U], lo[B][U], hi[B][U];
  auto fetch = [&](int s, int u) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int off = (u + i) * 64 + q * 16;
#pragma unroll
      for (int b = 0; b < NB; ++b) wv[s][b][i] = load_piece<true>(wr[b], off, row_kb);
      lo[s][i] = load_piece<false>(xl, off, lo_kb);
      hi[s][i] = HI ? load_piece<false>(xh, off, hi_kb) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  float sum[kFold ? NB : 1][4] = {};
  int steps = 0;
  auto fold = [&] {
    if constexpr (kFold) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[b][i] += c[b][i];
          c[b][i] = 0.f;
        }
    }
  };
  auto work = [&](int s) {
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        mma_m16n8<DT>(c[b], lo[s][i].x, hi[s][i].x, lo[s][i].y, hi[s][i].y, wv[s][b][i].x, wv[s][b][i].y);
        mma_m16n8<DT>(c[b], lo[s][i].z, hi[s][i].z, lo[s][i].w, hi[s][i].w, wv[s][b][i].z, wv[s][b][i].w);
      }
    if (kFold && (++steps & 3) == 0) fold();
  };
  // The warp's units: U of every W U.
  constexpr int kStep = W * U;
  int u = warp * U;
  if constexpr (B == 2) fetch(0, u);
  while (u * 64 < kb) {
    fetch(B - 1, u + (B - 1) * kStep);
    work(0);
    u += kStep;
    if constexpr (B == 2) {
      if (u * 64 >= kb) break;
      fetch(0, u + kStep);
      work(1);
      u += kStep;
    }
  }
  if constexpr (kFold) {
    fold();
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) c[b][i] = sum[b][i];
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    *reinterpret_cast<float2 *>(&red[warp][g][b * 8 + 2 * q]) = make_float2(c[b][0], c[b][1]);
    if constexpr (HI)
      *reinterpret_cast<float2 *>(&red[warp][g + 8][b * 8 + 2 * q]) = make_float2(c[b][2], c[b][3]);
  }
  __syncthreads();
  const int t = threadIdx.x >> 3, col = threadIdx.x & 7, n = n0 + col;
  if (t >= TT || t >= p.T || n >= p.N) return;
  float acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    acc[b] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) acc[b] += red[w][t][b * 8 + col];
  }
  const float sx = p.x_scale ? p.x_scale[t] : 1.f;
  const bool bf = p.out_dtype == MOE_BF16;
  const float res = !p.resid ? 0.f : bf ? load_resid<true>(p, t, n) : load_resid<false>(p, t, n);
  float y;
  if constexpr (NB == 2)
    y = swiglu(finish_acc(p, acc[0], sx, n), finish_acc(p, acc[1], sx, p.N + n));
  else
    y = activate(p.act, finish_acc(p, acc[0], sx, n));
  if (bf) store_out<true>(p, t, n, y + res);
  else store_out<false>(p, t, n, y + res);
}

// Warps per block: 8 where there are two blocks for every SM, 16 where there
// are fewer (more bytes in flight).  bf16, one token: N = 4096, K = 4096 6.7 us
// with 8, 7.4 with 16; N = 256, K = 6144 3.8 us with 8, 3.1 with 16.
template <int DT, int NB, bool HI, bool kFold>
cudaError_t launch_few_w(const LinearParams &p, cudaStream_t st) {
  const int blocks = (p.N + 7) / 8;
  return blocks > 304 ? launch_k(false, linear_few_kernel<DT, NB, HI, 8, kFold>, dim3(blocks), dim3(256), 0, st, p)
                      : launch_k(false, linear_few_kernel<DT, NB, HI, 16, kFold>, dim3(blocks), dim3(512), 0, st, p);
}

template <int DT, bool kFold>
cudaError_t launch_few(const LinearParams &p, cudaStream_t st) {
  if (p.act == MOE_ACT_SWIGLU)
    return p.T > 8 ? launch_few_w<DT, 2, true, kFold>(p, st) : launch_few_w<DT, 2, false, kFold>(p, st);
  return p.T > 8 ? launch_few_w<DT, 1, true, kFold>(p, st) : launch_few_w<DT, 1, false, kFold>(p, st);
}

}  // namespace
}  // namespace moe

extern "C" __attribute__((visibility("default"))) int moe_linear(
    const void *x, const float *x_scale, const void *w, const float *w_scale, const float *bias,
    const void *resid, void *out, int T, int N, int K, int dtype, int out_dtype, int act,
    int64_t x_stride, int64_t w_stride, int64_t resid_stride, int64_t out_stride, int32_t *status,
    moe_stream_t stream) {
  using namespace moe;
  constexpr int kMaxDim = 1 << 19;
  if ((dtype != MOE_BF16 && dtype != MOE_E4M3) || (out_dtype != MOE_F32 && out_dtype != MOE_BF16) ||
      act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU)
    return MOE_ERR_ARG;
  const size_t es = dtype == MOE_BF16 ? 2 : 1, os = out_dtype == MOE_F32 ? 4 : 2;
  if (T < 0 || T > kMaxDim || N < 1 || N > kMaxDim || K < 1 || K > kMaxDim || (size_t)K * es % 16)
    return MOE_ERR_ARG;
  if (act == MOE_ACT_SWIGLU && N % 16) return MOE_ERR_ARG;
  const int rows = act == MOE_ACT_SWIGLU ? 2 * N : N;
  const long long ldx = x_stride ? x_stride : K, ldw = w_stride ? w_stride : K,
                  ldr = resid_stride ? resid_stride : N, ldo = out_stride ? out_stride : N;
  constexpr long long kMaxStride = 1LL << 31;
  if (ldx < K || ldw < K || ldr < N || ldo < N || ldx > kMaxStride || ldw > kMaxStride ||
      ldr > kMaxStride || ldo > kMaxStride)
    return MOE_ERR_ARG;
  // Rows of x and w are read 16 bytes at a time.
  if (((size_t)ldx * es | (size_t)ldw * es) & 15) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !w || !out) return MOE_ERR_ARG;
  if ((dtype == MOE_E4M3) != (x_scale != nullptr) || (dtype == MOE_E4M3) != (w_scale != nullptr))
    return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w)) & 15) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(x_scale) | reinterpret_cast<uintptr_t>(w_scale) |
       reinterpret_cast<uintptr_t>(bias) | reinterpret_cast<uintptr_t>(status)) & 3)
    return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(resid)) & (os - 1))
    return MOE_ERR_ARG;
  // Blocks run in any order: out is apart from everything they read, but for
  // resid, which may be out itself (each element is read by the thread that
  // writes it).
  const Area ao{out, (size_t)T, N * os, (size_t)ldo * os}, ar{resid, (size_t)T, N * os, (size_t)ldr * os},
      ax{x, (size_t)T, K * es, (size_t)ldx * es}, aw{w, (size_t)rows, K * es, (size_t)ldw * es};
  if (meet(ao, ax) || meet(ao, aw) || meet(ao, area(x_scale, (size_t)T * 4)) ||
      meet(ao, area(w_scale, (size_t)rows * 4)) || meet(ao, area(bias, (size_t)rows * 4)) ||
      meet(ao, area(status, 4)))
    return MOE_ERR_ARG;
  if (!(resid == out && ldr == ldo) && meet(ao, ar)) return MOE_ERR_ARG;
  LinearParams p{x, w, x_scale, w_scale, bias, resid, out, T, N, K, act, out_dtype,
                 ldx, ldw, ldr, ldo, status};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = T > kFewTokens            ? launch_linear_tc(p, dtype, st)
                          : dtype == MOE_E4M3       ? launch_few<MOE_E4M3, false>(p, st)
                          : out_dtype == MOE_F32    ? launch_few<MOE_BF16, true>(p, st)
                                                    : launch_few<MOE_BF16, false>(p, st);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_DEVICE;
}
