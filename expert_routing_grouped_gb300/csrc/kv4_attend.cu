// kv4_attend.cu -- attention over the 4-bit paged cache (moe_kv4_attention in
// include/moe.h).
//
// One block per row and query head: its warps take the row's tokens in turn, a
// lane holds D / 32 neighbouring dimensions, and each warp keeps the running
// maximum, sum and output of an online softmax; the warps' parts are joined at
// the end.
#include <algorithm>
#include <cmath>

#include "area.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

template <int D>
__global__ void __launch_bounds__(128) kv4_attend_kernel(const AttendParams p) {
  constexpr int N = D / 32, NG = D / kKvGroup;
  __shared__ float part[4][D], pm[4], pl[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, h = blockIdx.y, hk = h / (p.H / p.b.Hkv);
  const int s = kv_seq_of(p.b, t, lane);
  if (s >= p.b.n_seq) return;
  const AttendSeq sq = attend_seq_at(p, s);
  const int i = t - sq.t0;
  if (i >= sq.rows || sq.rows * p.G <= kFewColumns) return;
  const int pos = sq.len - sq.nq + i;
  const int end = p.causal ? min(sq.len, pos + 1) : sq.len;
  const int first = p.window ? max(0, pos - p.window + 1) : 0;
  float q[N], o[N];
#pragma unroll
  for (int c = 0; c < N; ++c) {
    q[c] = __bfloat162float(p.q[(size_t)t * p.ldq + h * D + lane * N + c]);
    o[c] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int g = lane * N / kKvGroup, lp = p.b.log_page;
  for (int j = first + warp; j < end; j += 4) {
    const int page = kv_page_at(p.b, s, j);
    if (page < 0) continue;
    const int slot = j & ((1 << lp) - 1);
    const uint8_t *block = p.cache + ((size_t)page * p.b.Hkv + hk) * KvBlock<D>::bytes(lp);
    float kv[2][N];
    bool nan = false;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint8_t *c = block + KvBlock<D>::codes(lp, w, slot) + lane * N / 2;
      const __half2 sl = *reinterpret_cast<const __half2 *>(block + KvBlock<D>::scales(lp, w, slot) + g * 4);
      const float st = __low2float(sl), lo = __high2float(sl);
      nan |= st != st;
#pragma unroll
      for (int e = 0; e < N; ++e) kv[w][e] = fmaf(st, (float)(c[e / 2] >> (4 * (e & 1)) & 15), lo);
    }
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) x = fmaf(q[e], kv[0][e], x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= p.scale;
    if (p.softcap > 0.f) x = p.softcap * tanhf(x / p.softcap);
    if (__any_sync(0xffffffffu, nan)) x = NAN;
    const float top = fmaxf(m, x), keep = m > -INFINITY ? expf(m - top) : 0.f, w = expf(x - top);
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = o[e] * keep + w * kv[1][e];
    m = top;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) part[warp][lane * N + e] = o[e];
  if (lane == 0) pm[warp] = m, pl[warp] = l;
  __syncthreads();
  if (threadIdx.x >= D) return;
  const float top = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
  float sum = 0.f, y = 0.f;
  for (int w = 0; w < 4; ++w) {
    const float f = pl[w] != 0.f ? expf(pm[w] - top) : 0.f;
    sum += pl[w] * f;
    y += part[w][threadIdx.x] * f;
  }
  p.out[(size_t)t * p.ldo + h * D + threadIdx.x] = __float2bfloat16_rn(sum != 0.f ? y / sum : 0.f);
}

// Sizes that the call and its workspace are refused for.
bool good_sizes(int T, int n_seq, bool rows_given, int max_q, int n_heads, int n_kv_heads, int head_dim,
                int page_size, int n_pages, int max_pages) {
  return kv4_good_batch(T, 1 << 19, n_seq, rows_given, n_kv_heads, head_dim, page_size, n_pages, max_pages) &&
         max_q >= 0 && n_heads >= 1 && n_heads <= 1024 && n_heads % n_kv_heads == 0;
}

// Where the partial results of a call lie in its workspace.
struct Scratch {
  size_t o, ml, bytes;
};
Scratch workspace_of(const AttendParams &p, int D) {
  const size_t columns = (p.G <= kFewColumns ? few_slots(p) : 0) * kFewColumns;
  Scratch w;
  w.o = 0;
  w.ml = columns * D * sizeof(float);
  w.bytes = w.ml + columns * sizeof(float2);
  return w;
}

}  // namespace
}  // namespace moe

extern "C" __attribute__((visibility("default"))) size_t moe_kv4_workspace(
    int T, int n_seq, int max_q, int n_heads, int n_kv_heads, int head_dim, int page_size,
    int max_pages) {
  if (T < 1 || !moe::good_sizes(T, n_seq, true, max_q, n_heads, n_kv_heads, head_dim, page_size, 1, max_pages))
    return 0;
  moe::AttendParams p{};
  p.b.n_seq = n_seq, p.b.Hkv = n_kv_heads, p.b.max_pages = max_pages, p.b.log_page = moe::kv4_log2(page_size);
  p.b.T = T, p.H = n_heads, p.G = n_heads / n_kv_heads, p.max_q = max_q;
  return moe::workspace_of(p, head_dim).bytes;
}

extern "C" __attribute__((visibility("default"))) int moe_kv4_attention(
    const void *q, const void *cache, const int32_t *pages, const int32_t *q_off,
    const int32_t *kv_len, int T, int n_seq, int max_q, int n_heads, int n_kv_heads, int head_dim,
    int page_size, int n_pages, int max_pages, float scale, float softcap, int window, int causal,
    void *out, int64_t q_stride, int64_t out_stride, void *workspace, size_t workspace_bytes,
    int32_t *status, moe_stream_t stream) {
  using namespace moe;
  if (!good_sizes(T, n_seq, q_off != nullptr, max_q, n_heads, n_kv_heads, head_dim, page_size, n_pages,
                  max_pages) ||
      !std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0)
    return MOE_ERR_ARG;
  const long long row = (long long)n_heads * head_dim, ldq = q_stride ? q_stride : row,
                  ldo = out_stride ? out_stride : row;
  if (ldq < row || ldo < row || ldq > (1LL << 31) || ldo > (1LL << 31) || (ldq | ldo) & 7) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!q || !cache || !pages || !kv_len || !out) return MOE_ERR_ARG;
  if (kv4_off_by(q, 15) || kv4_off_by(cache, 15) || kv4_off_by(out, 15) || kv4_off_by(workspace, 15) ||
      kv4_off_by(pages, 3) || kv4_off_by(q_off, 3) || kv4_off_by(kv_len, 3) || kv4_off_by(status, 3))
    return MOE_ERR_ARG;
  const size_t need = moe_kv4_workspace(T, n_seq, max_q, n_heads, n_kv_heads, head_dim, page_size, max_pages);
  if (need && !workspace) return MOE_ERR_ARG;
  if (workspace_bytes < need) return MOE_ERR_NOMEM;
  const size_t rb = (size_t)row * 2;
  const Area ins[] = {
      Area{q, (size_t)T, rb, (size_t)ldq * 2},
      area(cache, moe_kv4_page_bytes(page_size, n_kv_heads, head_dim) * n_pages),
      area(pages, (size_t)n_seq * max_pages * 4),
      area(kv_len, (size_t)n_seq * 4),
      area(q_off, ((size_t)n_seq + 1) * 4),
      area(status, 4)};
  const Area ao{out, (size_t)T, rb, (size_t)ldo * 2}, aw = area(workspace, need);
  for (const Area &a : ins)
    if (meet(ao, a) || meet(aw, a)) return MOE_ERR_ARG;
  if (meet(ao, aw)) return MOE_ERR_ARG;
  AttendParams p{};
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.cache = static_cast<const uint8_t *>(cache);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.b = KvBatch{pages, q_off, kv_len, T, n_seq, kv4_log2(page_size), n_pages, max_pages, n_kv_heads};
  p.ldq = ldq, p.ldo = ldo, p.H = n_heads, p.G = n_heads / n_kv_heads, p.max_q = max_q;
  p.window = window, p.causal = causal != 0, p.scale = scale, p.softcap = softcap, p.status = status;
  const Scratch w = workspace_of(p, head_dim);
  if (w.bytes) {
    p.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + w.o);
    p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) + w.ml);
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t err = cudaSuccess;
  const long long rows = q_off ? (max_q ? std::min(max_q, T) : T) : 1;   // of one sequence, at most
  if (p.G <= kFewColumns) err = launch_few(p, head_dim, st);
  if (err == cudaSuccess && rows * p.G > kFewColumns)
    err = launch_k(false, head_dim == 64 ? kv4_attend_kernel<64> : kv4_attend_kernel<128>, dim3(T, n_heads),
                   dim3(128), 0, st, p);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_DEVICE;
}
