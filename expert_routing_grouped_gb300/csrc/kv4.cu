// kv4.cu -- the rows of K and V into the 4-bit paged cache (moe_kv4_append in
// include/moe.h), and the calls' argument checks.
//
//   of 64 values x:  lo = f16(min x), step = f16(max(max x - lo, 0) / 15),
//                    c = clamp(rint((x - lo) / step), 0, 15)
//
// Eight lanes hold a group, 16 or 32 bytes each, so its smallest and largest are
// three exchanges away; each lane writes its 8 codes as one word.  The row's
// place (sequence, length, page) is looked up while its values are on the way.
//
// The floor is the rows in and 9/32 of a bfloat16's bytes out.  8192 rows of 8 heads
// of 128: 14.2 us (3.0 TB/s), bound by instructions (schedulers 69 % busy).  Rows are read
// once, past what L2 holds (13.7 us against 14.6 with plain loads, before the look at the
// offsets that keeps rows of no sequence unread, 0.4 us); two exact quotients share an
// instruction (15.3 us one at a time); several groups a warp and packed conversions (24.3
// us without).  64 rows: 1.9 us.
#include <algorithm>
#include <cmath>

#include "area.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

constexpr int kAppendWarps = 8;

struct AppendParams {
  const void *k, *v;
  uint8_t *cache;
  KvBatch b;
  long long ldk, ldv;   // row strides in elements
  int warps_row;        // warps of one row
};

// x held in float16 terms: +-60000 leaves room for lo + 15 step.
__device__ __forceinline__ float kv_clamp(float x) { return fminf(fmaxf(x, -60000.f), 60000.f); }

__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 1 / v of a float16 number v to nearest: the hardware's approximation and one Newton
// step.
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return fmaf(fmaf(-v, r, 1.f), r, r);
}
// a / b to nearest from r = 1 / b: a product, corrected by its remainder (Markstein
// 1990).
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(-q, b, a), r, q);
}
// The same twice (minus_b: -b).
__device__ __forceinline__ float2 quotient_2(float2 a, float2 minus_b, float2 r) {
  const float2 q = mul_2(a, r);
  return fma_2(fma_2(q, minus_b, a), r, q);
}
// v shifted up by a byte, below it hi and lo limited to 0 .. 15.
__device__ __forceinline__ uint32_t pack_u4(int hi, int lo, uint32_t v) {
  uint32_t d;
  asm("cvt.pack.sat.u4.s32.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(hi), "r"(lo), "r"(v));
  return d;
}

// A lane's 8 values of one group, as they came.
template <int DT>
struct Raw8 {
  uint4 v[DT == MOE_BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void *src, size_t at) {
    if constexpr (DT == MOE_BF16) {
      v[0] = __ldcs(reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(src) + at));
    } else {
      const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(src) + at);
      v[0] = __ldcs(p), v[1] = __ldcs(p + 1);
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (DT == MOE_BF16) {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(v[i].x), x[4 * i + 1] = __uint_as_float(v[i].y);
        x[4 * i + 2] = __uint_as_float(v[i].z), x[4 * i + 3] = __uint_as_float(v[i].w);
      }
    }
  }
};

// A warp takes NU rounds of 4 groups of a row: the row's place is looked up once for
// them, while all their loads are on the way.
template <int DT, int D, int NU>
__global__ void __launch_bounds__(kAppendWarps * 32) kv4_append_kernel(const AppendParams p) {
  constexpr int NG = D / kKvGroup;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int t = (int)(w / p.warps_row);
  if (t >= p.b.T) return;
  // Rows of no sequence are not read: they lie before the first offset or from the last on.
  if (p.b.q_off && (t < __ldg(p.b.q_off) || t >= __ldg(p.b.q_off + p.b.n_seq))) return;
  const int groups = p.b.Hkv * NG;   // of K, then as many of V
  const int u0 = (int)(w - (long long)t * p.warps_row) * 4 * NU + (lane >> 3);
  Raw8<DT> raw[NU];
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    const int u = u0 + 4 * n, which = u >= groups, r = u - which * groups;
    if (u < 2 * groups)
      raw[n].load(which ? p.v : p.k, (size_t)t * (which ? p.ldv : p.ldk) + r * kKvGroup + (lane & 7) * 8);
  }
  const int s = kv_seq_of(p.b, t, lane);
  int page = -1, pos = -1;
  if (s < p.b.n_seq) {
    const KvSeq q = kv_seq_at(p.b, s);
    const int i = t - q.t0;
    pos = q.len - q.nq + i;
    if (i >= 0 && i < q.nq && pos >= 0) page = kv_page_at(p.b, s, pos);
  }
  if (page < 0) return;   // the whole warp's row
  const int slot = pos & ((1 << p.b.log_page) - 1);
  uint8_t *const first = p.cache + (size_t)page * p.b.Hkv * KvBlock<D>::bytes(p.b.log_page);
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    const int u = u0 + 4 * n;
    const bool mine = u < 2 * groups;
    float x[8];
    if (mine) {
      raw[n].get(x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
    // A NaN stays in the smallest and the largest.
    float lo = min3_nan(min3_nan(min3_nan(x[0], x[1], x[2]), x[3], x[4]), min3_nan(x[5], x[6], x[7]), x[5]);
    float hi = max3_nan(max3_nan(max3_nan(x[0], x[1], x[2]), x[3], x[4]), max3_nan(x[5], x[6], x[7]), x[5]);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const float a = __shfl_xor_sync(0xffffffffu, lo, o), c = __shfl_xor_sync(0xffffffffu, hi, o);
      lo = min3_nan(lo, a, a), hi = max3_nan(hi, c, c);
    }
    if (!mine) continue;
    bool nan = false;
    if (!(lo >= -60000.f && hi <= 60000.f)) {   // far values or a NaN
      nan = lo != lo;
      lo = kv_clamp(lo), hi = kv_clamp(hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = kv_clamp(x[i]);
    }
    const __half l16 = __float2half_rn(lo);
    const float l = __half2float(l16), range = fmaxf(hi - l, 0.f);
    const __half s16 = __float2half_rn(quotient(range, 15.f, 0.06666667f));
    const float st = __half2float(s16), inv = st > 0.f ? reciprocal(st) : 0.f;
    // c = rint((x - lo) / step): 1.5 2^23 more than the quotient is rounded to whole
    // numbers, which are then its lowest bits.
    int c[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 a = add_2(make_float2(x[i], x[i + 1]), make_float2(-l, -l));
      const float2 q = add_2(quotient_2(a, make_float2(-st, -st), make_float2(inv, inv)),
                             make_float2(12582912.f, 12582912.f));
      c[i] = __float_as_int(q.x) - 0x4B400000, c[i + 1] = __float_as_int(q.y) - 0x4B400000;
    }
    uint32_t word = pack_u4(c[1], c[0], pack_u4(c[3], c[2], pack_u4(c[5], c[4], pack_u4(c[7], c[6], 0u))));
    if (nan) word = 0;
    const int which = u >= groups, r = u - which * groups, head = r / NG, g = r % NG;
    uint8_t *block = first + (size_t)head * KvBlock<D>::bytes(p.b.log_page);
    *reinterpret_cast<uint32_t *>(block + KvBlock<D>::codes(p.b.log_page, which, slot) + g * (kKvGroup / 2) +
                                  (lane & 7) * 4) = word;
    if ((lane & 7) == 0) {
      const uint32_t pair = __half_as_ushort(s16) | (uint32_t)__half_as_ushort(l16) << 16;
      *reinterpret_cast<uint32_t *>(block + KvBlock<D>::scales(p.b.log_page, which, slot) + g * 4) =
          nan ? 0x7FFF7FFFu : pair;
    }
  }
}

template <int DT, int D>
cudaError_t launch_append(AppendParams p, int n_kv_heads, cudaStream_t st) {
  // Rounds of a warp: one where there are few rows (latency), four where the rows
  // alone fill the SMs.
  const int rounds = (2 * n_kv_heads * (D / kKvGroup) + 3) / 4;
  const bool many = (long long)p.b.T * rounds >= 152 * 64 && rounds > 1;
  p.warps_row = many ? (rounds + 3) / 4 : rounds;
  const long long warps = (long long)p.b.T * p.warps_row;   // at most 2^29
  const dim3 grid((unsigned)((warps + kAppendWarps - 1) / kAppendWarps)), block(kAppendWarps * 32);
  return launch_k(false, many ? kv4_append_kernel<DT, D, 4> : kv4_append_kernel<DT, D, 1>, grid, block, 0, st, p);
}

}  // namespace
}  // namespace moe

extern "C" __attribute__((visibility("default"))) size_t moe_kv4_page_bytes(int page_size,
                                                                            int n_kv_heads,
                                                                            int head_dim) {
  if (!moe::kv4_good_page(page_size) || n_kv_heads < 1 || n_kv_heads > 1024 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return (size_t)page_size * head_dim / 8 * 9 * n_kv_heads;
}

extern "C" __attribute__((visibility("default"))) int moe_kv4_append(
    const void *k, const void *v, void *cache, const int32_t *pages, const int32_t *q_off,
    const int32_t *kv_len, int T, int n_seq, int n_kv_heads, int head_dim, int page_size,
    int n_pages, int max_pages, int dtype, int64_t k_stride, int64_t v_stride,
    moe_stream_t stream) {
  using namespace moe;
  if (!kv4_good_batch(T, 1 << 24, n_seq, q_off != nullptr, n_kv_heads, head_dim, page_size, n_pages, max_pages) ||
      (long long)T * n_kv_heads > (1 << 28) || (dtype != MOE_F32 && dtype != MOE_BF16))
    return MOE_ERR_ARG;
  const long long row = (long long)n_kv_heads * head_dim, ldk = k_stride ? k_stride : row,
                  ldv = v_stride ? v_stride : row;
  const size_t es = dtype == MOE_F32 ? 4 : 2;
  if (ldk < row || ldv < row || ldk > (1LL << 32) || ldv > (1LL << 32) ||
      (((size_t)ldk | (size_t)ldv) * es & 15))
    return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!k || !v || !cache || !pages || !kv_len) return MOE_ERR_ARG;
  if (kv4_off_by(k, 15) || kv4_off_by(v, 15) || kv4_off_by(cache, 15) || kv4_off_by(pages, 3) || kv4_off_by(q_off, 3) ||
      kv4_off_by(kv_len, 3))
    return MOE_ERR_ARG;
  const Area ac = area(cache, moe_kv4_page_bytes(page_size, n_kv_heads, head_dim) * n_pages);
  if (meet(ac, Area{k, (size_t)T, (size_t)row * es, (size_t)ldk * es}) ||
      meet(ac, Area{v, (size_t)T, (size_t)row * es, (size_t)ldv * es}) ||
      meet(ac, area(pages, (size_t)n_seq * max_pages * 4)) || meet(ac, area(kv_len, (size_t)n_seq * 4)) ||
      meet(ac, area(q_off, ((size_t)n_seq + 1) * 4)))
    return MOE_ERR_ARG;
  AppendParams p{k, v, static_cast<uint8_t *>(cache),
                 KvBatch{pages, q_off, kv_len, T, n_seq, kv4_log2(page_size), n_pages, max_pages, n_kv_heads},
                 ldk, ldv, 0};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (dtype == MOE_F32)
    err = head_dim == 64 ? launch_append<MOE_F32, 64>(p, n_kv_heads, st)
                         : launch_append<MOE_F32, 128>(p, n_kv_heads, st);
  else
    err = head_dim == 64 ? launch_append<MOE_BF16, 64>(p, n_kv_heads, st)
                         : launch_append<MOE_BF16, 128>(p, n_kv_heads, st);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_DEVICE;
}
