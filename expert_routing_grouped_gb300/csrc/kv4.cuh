// kv4.cuh -- the 4-bit cache's geometry and a batch's, shared by the kernels that
// fill the cache and attend over it (layout: include/moe.h).
#pragma once

#include "linear.cuh"
#include "moe_internal.cuh"

namespace moe {

constexpr int kKvGroup = 64;   // values per (step, lo)

// A batch over the cache: which rows are whose, and where tokens live.
struct KvBatch {
  const int32_t *pages, *q_off, *kv_len;
  int T, n_seq;
  int log_page;              // page_size = 1 << log_page
  int n_pages, max_pages;
  int Hkv;
};

// One sequence: rows t0 .. t0 + nq - 1 are the last nq of its len tokens.
struct KvSeq {
  int t0, nq, len;
};

static __device__ __forceinline__ int clamp_int(int v, int lo, int hi) { return min(max(v, lo), hi); }

static __device__ __forceinline__ int kv_len_at(const KvBatch &b, int s) {
  return clamp_int(__ldg(b.kv_len + s), 0, b.max_pages << b.log_page);
}

static __device__ __forceinline__ KvSeq kv_seq_at(const KvBatch &b, int s) {
  KvSeq q;
  if (b.q_off) {
    q.t0 = clamp_int(__ldg(b.q_off + s), 0, b.T);
    q.nq = clamp_int(__ldg(b.q_off + s + 1), q.t0, b.T) - q.t0;
  } else {
    q.t0 = s;
    q.nq = 1;
  }
  q.len = kv_len_at(b, s);
  return q;
}

// The page of a sequence's token, -1 for a hole.
static __device__ __forceinline__ int kv_page_at(const KvBatch &b, int s, int token) {
  const int id = __ldg(b.pages + (size_t)s * b.max_pages + (token >> b.log_page));
  return (unsigned)id < (unsigned)b.n_pages ? id : -1;
}

// The sequence of row t (n_seq: none), found by a whole warp, 32 offsets at a time.
static __device__ __forceinline__ int kv_seq_of(const KvBatch &b, int t, int lane) {
  if (!b.q_off) return t;
  int base = 0, n = b.n_seq + 1;   // how many offsets are at most t: base .. base + n
  while (n > 32) {
    const int step = (n + 31) / 32, i = lane * step;
    const int k = __popc(__ballot_sync(0xffffffffu, i < n && __ldg(b.q_off + base + i) <= t));
    if (k == 0) return b.n_seq;
    const int skip = (k - 1) * step;
    base += skip;
    n = min(step, n - skip);
  }
  const int s = base - 1 + __popc(__ballot_sync(0xffffffffu, lane < n && __ldg(b.q_off + base + lane) <= t));
  return s < 0 ? b.n_seq : s;
}

// Byte offsets inside one block (a page's tokens of one KV head).
template <int D>
struct KvBlock {
  static constexpr int kCodes = D / 2;                  // bytes of a token's codes
  static constexpr int kScales = D / kKvGroup * 4;      // bytes of its (step, lo)
  static __device__ __forceinline__ size_t bytes(int log_page) {
    return (size_t)(2 * (kCodes + kScales)) << log_page;
  }
  // which: 0 K, 1 V
  static __device__ __forceinline__ uint32_t codes(int log_page, int which, int slot) {
    return ((which << log_page) + slot) * kCodes;
  }
  static __device__ __forceinline__ uint32_t scales(int log_page, int which, int slot) {
    return ((2 * kCodes) << log_page) + ((which << log_page) + slot) * kScales;
  }
};

// What attention's kernels share.
struct AttendParams {
  const __nv_bfloat16 *q;
  const uint8_t *cache;
  __nv_bfloat16 *out;
  KvBatch b;
  long long ldq, ldo;        // row strides in elements
  int H, G;                  // query heads, and those of one KV head
  int max_q;                 // 0: not known
  int window, causal;
  float scale, softcap;
  float *part_o;             // [slot][column][D] partial outputs
  float2 *part_ml;           // [slot][column] (maximum, sum)
  int target;                // blocks that a batch is spread over
  int32_t *status;
  unsigned long long wait_ns;
};

// A sequence as attention takes it: `rows` of its nq rows are worked out.
struct AttendSeq : KvSeq {
  int rows;
};
static __device__ __forceinline__ AttendSeq attend_seq_at(const AttendParams &p, int s) {
  AttendSeq q;
  static_cast<KvSeq &>(q) = kv_seq_at(p.b, s);
  q.rows = p.max_q ? min(q.nq, p.max_q) : q.nq;
  return q;
}

// Sequences of at most this many columns (rows times query heads of a KV head)
// take kv4_few.cu's kernels, the others kv4_many.cu's.
constexpr int kFewColumns = 16;
size_t few_slots(const AttendParams &p);
cudaError_t launch_few(const AttendParams &p, int D, cudaStream_t st);

size_t many_rows(const AttendParams &p);
cudaError_t launch_many(const AttendParams &p, int D, cudaStream_t st);

// Two f32 operations in one instruction.
static __device__ __forceinline__ float2 fma_2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
static __device__ __forceinline__ float2 mul_2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
static __device__ __forceinline__ float2 add_2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
static __device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

static __device__ __forceinline__ uint2 pack_out(float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoScore = -3e38f;   // a maximum before any score

static __device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A score's factor held finite (an infinite one would make NaN of scores of 0).
static __device__ __forceinline__ float finite(float x) { return fminf(fmaxf(x, -3.4028235e38f), 3.4028235e38f); }
static __device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// cap tanh(x / cap) of two scores, x and the result in units of log2 e; with z = 2 x / cap
// in these units it is
//   x (1 + a z^2 + b z^4 + c z^6)      |z| < 1: tanh(y) / y to 4e-8 where y < 0.35
//   cap - 2 cap / (1 + 2^z)            else; there it is a third of cap at least
// so that it is off by at most 2^-20 of itself, however large the cap is.
static __device__ __forceinline__ float2 capped_2(float2 x, float two_by_cap, float cap_log2) {
  const float2 one = make_float2(1.f, 1.f), z = mul_2(x, make_float2(two_by_cap, two_by_cap)), t = mul_2(z, z);
  float2 p = fma_2(t, make_float2(-8.51692959e-05f, -8.51692959e-05f), make_float2(0.00191879156f, 0.00191879156f));
  p = fma_2(p, t, make_float2(-0.0400369462f, -0.0400369462f));
  p = mul_2(x, fma_2(p, t, one));
  const float2 e = add_2(make_float2(ex2(z.x), ex2(z.y)), one);
  const float2 far = fma_2(make_float2(rcp_approx(e.x), rcp_approx(e.y)), make_float2(-2.f * cap_log2, -2.f * cap_log2),
                           make_float2(cap_log2, cap_log2));
  return make_float2(fabsf(z.x) < 1.f ? p.x : far.x, fabsf(z.y) < 1.f ? p.y : far.y);
}

// A running (maximum, sum, output) of one row, four dimensions of it in a lane.
struct RowPart {
  float top = kNoScore, sum = 0.f;
  float4 y = {0.f, 0.f, 0.f, 0.f};
  // Takes N partial results at(0) .. at(n - 1), n <= N, asked for all at once.
  template <int N, int D, class At>
  __device__ __forceinline__ void take(const float *po, const float2 *pml, int n, int lane, At at) {
    float2 ml[N];
    float4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      ml[i] = make_float2(kNoScore, 0.f);
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const size_t k = at(i);
        ml[i] = __ldcg(pml + k);
        if (lane < D / 4) v[i] = __ldcg(reinterpret_cast<const float4 *>(po + k * D) + lane);
      }
    }
    float now = top;
#pragma unroll
    for (int i = 0; i < N; ++i) now = fmaxf(now, ml[i].x);
    scale(ex2(top - now));
    top = now;
#pragma unroll
    for (int i = 0; i < N; ++i) add(ml[i].y, v[i], ex2(ml[i].x - now));
  }
  __device__ __forceinline__ void scale(float f) {
    sum *= f;
    y.x *= f, y.y *= f, y.z *= f, y.w *= f;
  }
  __device__ __forceinline__ void add(float l, const float4 &v, float f) {
    sum += l * f;
    y.x += v.x * f, y.y += v.y * f, y.z += v.z * f, y.w += v.w * f;
  }
  __device__ __forceinline__ uint2 result() const {
    const float f = sum != 0.f ? 1.f / sum : 0.f;
    return pack_out(make_float4(y.x * f, y.y * f, y.z * f, y.w * f));
  }
};

// ------------------------------------------------- argument checks (host) --

static inline bool kv4_good_page(int page_size) {
  return page_size >= 16 && page_size <= 256 && (page_size & (page_size - 1)) == 0;
}

static inline int kv4_log2(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

// The sizes of a batch over a cache.
static inline bool kv4_good_batch(int T, int max_T, int n_seq, bool rows_given, int n_kv_heads,
                                  int head_dim, int page_size, int n_pages, int max_pages) {
  return T >= 0 && T <= max_T && n_seq >= 1 && n_seq <= 65535 && (rows_given || T == n_seq || T == 0) &&
         n_kv_heads >= 1 && n_kv_heads <= 1024 && (head_dim == 64 || head_dim == 128) &&
         kv4_good_page(page_size) && n_pages >= 1 && max_pages >= 1 &&
         (long long)max_pages * page_size <= (1 << 30);
}

static inline bool kv4_off_by(const void *p, uintptr_t mask) {
  return (reinterpret_cast<uintptr_t>(p) & mask) != 0;
}

}  // namespace moe
