// kv4.cu -- the rows of K and V into the 4-bit paged cache (moe_kv4_append in
// include/moe.h), and the calls' argument checks.
//
//   of 64 values x:  lo = f16(min x), step = f16(max(max x - lo, 0) / 15),
//                    c = clamp(rint((x - lo) / step), 0, 15)
//
// Eight lanes hold a group, 16 or 32 bytes each, so its smallest and largest are
// three exchanges away; each lane writes its 8 codes as one word.  The row's
// place (sequence, length, page) is looked up while its values are on the way.
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
  int warps_row;        // warps of one row: 4 groups each
};

// x held in float16 terms: +-60000 leaves room for lo + 15 step.
__device__ __forceinline__ float kv_clamp(float x) { return fminf(fmaxf(x, -60000.f), 60000.f); }

template <int DT, int D>
__global__ void __launch_bounds__(kAppendWarps * 32) kv4_append_kernel(const AppendParams p) {
  constexpr int NG = D / kKvGroup;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int t = (int)(w / p.warps_row);
  if (t >= p.b.T) return;
  const int groups = p.b.Hkv * NG;   // of K, then as many of V
  const int u = (int)(w - (long long)t * p.warps_row) * 4 + (lane >> 3);
  const bool mine = u < 2 * groups;
  const int which = u >= groups, r = u - which * groups;
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0.f;
  if (mine) {
    const size_t at = (size_t)t * (which ? p.ldv : p.ldk) + r * kKvGroup + (lane & 7) * 8;
    const void *src = which ? p.v : p.k;
    if constexpr (DT == MOE_BF16) {
      const uint4 q = *reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(src) + at);
      const uint32_t v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
      }
    } else {
      const float4 *f = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(src) + at);
      const float4 a = f[0], c = f[1];
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
      x[4] = c.x, x[5] = c.y, x[6] = c.z, x[7] = c.w;
    }
  }
  const int s = kv_seq_of(p.b, t, lane);
  int page = -1, pos = -1;
  if (s < p.b.n_seq) {
    const KvSeq q = kv_seq_at(p.b, s);
    const int i = t - q.t0;
    pos = q.len - q.nq + i;
    if (i < q.nq && pos >= 0) page = kv_page_at(p.b, s, pos);
  }
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    nan |= x[i] != x[i];
    x[i] = kv_clamp(x[i]);
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  nan = __ballot_sync(0xffffffffu, nan) >> (lane & 24) & 0xFF;
  if (!mine || page < 0) return;
  const __half l16 = __float2half_rn(lo);
  const float l = __half2float(l16);
  const __half s16 = __float2half_rn(__fdiv_rn(fmaxf(hi - l, 0.f), 15.f));
  const float st = __half2float(s16), inv = st > 0.f ? __frcp_rn(st) : 0.f;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // The quotient to nearest: a product with 1 / step, corrected by its
    // remainder (Markstein 1990).
    const float d = x[i] - l, q0 = d * inv, q = fmaf(fmaf(-q0, st, d), inv, q0);
    const uint32_t c = (uint32_t)fminf(fmaxf(rintf(q), 0.f), 15.f);
    word |= c << (4 * i);
  }
  if (nan) word = 0;
  const int slot = pos & ((1 << p.b.log_page) - 1), head = r / NG, g = r % NG;
  uint8_t *block = p.cache + ((size_t)page * p.b.Hkv + head) * KvBlock<D>::bytes(p.b.log_page);
  *reinterpret_cast<uint32_t *>(block + KvBlock<D>::codes(p.b.log_page, which, slot) + g * (kKvGroup / 2) +
                                (lane & 7) * 4) = word;
  if ((lane & 7) == 0) {
    const uint32_t pair = __half_as_ushort(s16) | (uint32_t)__half_as_ushort(l16) << 16;
    *reinterpret_cast<uint32_t *>(block + KvBlock<D>::scales(p.b.log_page, which, slot) + g * 4) =
        nan ? 0x7FFF7FFFu : pair;
  }
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
                 ldk, ldv, (2 * n_kv_heads * (head_dim / kKvGroup) + 3) / 4};
  const long long warps = (long long)T * p.warps_row;   // at most 2^29
  const dim3 grid((unsigned)((warps + kAppendWarps - 1) / kAppendWarps)), block(kAppendWarps * 32);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto kernel = dtype == MOE_F32 ? (head_dim == 64 ? kv4_append_kernel<MOE_F32, 64> : kv4_append_kernel<MOE_F32, 128>)
                                 : (head_dim == 64 ? kv4_append_kernel<MOE_BF16, 64> : kv4_append_kernel<MOE_BF16, 128>);
  return launch_k(false, kernel, grid, block, 0, st, p) == cudaSuccess ? MOE_OK : MOE_ERR_DEVICE;
}
