// kv4_attend.cu -- moe_kv4_attention's argument checks, workspace and choice of
// kernels (include/moe.h): sequences of up to 16 columns (rows times query heads
// of a KV head) in kv4_few.cu, which reads the cache once, larger ones in kv4_many.cu
// on the 5th-gen tensor cores, which decodes it once for 256 columns.  Each kernel leaves the
// other's sequences alone, so a batch may mix them.
#include <algorithm>
#include <cmath>

#include "area.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

// Sizes that the call and its workspace are refused for.
bool good_sizes(int T, int n_seq, bool rows_given, int max_q, int n_heads, int n_kv_heads, int head_dim,
                int page_size, int n_pages, int max_pages) {
  return kv4_good_batch(T, 1 << 19, n_seq, rows_given, n_kv_heads, head_dim, page_size, n_pages, max_pages) &&
         max_q >= 0 && n_heads >= 1 && n_heads <= 1024 && n_heads % n_kv_heads == 0;
}

// Whether some sequence may have more than kFewColumns columns.
bool may_have_many(const AttendParams &p) {
  const long long rows = p.b.q_off ? (p.max_q ? std::min(p.max_q, p.b.T) : p.b.T) : 1;
  return rows * p.G > kFewColumns;
}

// Where the partial results of a call lie in its workspace.
struct Scratch {
  size_t o, ml, bytes;
};
Scratch workspace_of(const AttendParams &p, int D) {
  // The kernels run one after the other: one area serves both.
  size_t rows = p.G <= kFewColumns ? few_slots(p) * kFewColumns : 0;
  if (may_have_many(p)) rows = std::max(rows, many_rows(p));
  Scratch w;
  w.o = 0;
  w.ml = rows * D * sizeof(float);
  w.bytes = w.ml + rows * sizeof(float2);
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
  // Enough with q_off and without.
  p.b.q_off = nullptr;
  const size_t without = T == n_seq ? moe::workspace_of(p, head_dim).bytes : 0;
  p.b.q_off = reinterpret_cast<const int32_t *>(uintptr_t(4));
  return std::max(without, moe::workspace_of(p, head_dim).bytes);
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
  // Tokens end before 2^30: no window shows more, and positions less it stay in 32 bits.
  p.window = std::min(window, 1 << 30), p.causal = causal != 0, p.scale = scale, p.status = status;
  // A cap past 10^38 (whose product with log2 e leaves f32) moves no score below 10^34.
  p.softcap = softcap <= 1e38f ? softcap : 0.f;
  const Scratch w = workspace_of(p, head_dim);
  if (w.bytes) {
    p.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + w.o);
    p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) + w.ml);
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t err = cudaSuccess;
  p.wait_ns = linear_wait_ns();
  if (!p.status) err = linear_gave_up(&p.status);
  if (err == cudaSuccess && p.G <= kFewColumns) err = launch_few(p, head_dim, st);
  if (err == cudaSuccess && may_have_many(p)) err = launch_many(p, head_dim, st);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_DEVICE;
}
