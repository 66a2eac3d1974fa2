// balance.cu -- the router's balance loss, its per-expert counts and the
// gradient of the logits (moe_balance_loss in include/moe.h).
//
//   p[t]  = softmax(z[t] + b)  or  sigmoid(z[t]) / sum sigmoid(z[t])
//   segment s (a sequence): its tokens that the mask keeps, T_s of them
//   c[s][e] = assignments of e,  P[s][e] = 1/T_s sum_t p[t][e]
//   loss[s] = alpha E / (k T_s) sum_e c[s][e] P[s][e]
//   dz_i    = p_i (a_i - sum_e p_e a_e)  (times 1 - sigmoid_i in sigmoid mode),
//             a_e = grad[s] alpha E / (k T_s^2) c[s][e]
//
// The counts come from the selection alone, so they are taken first, and then
// ONE pass over the logits gives both the sums of p and the gradient: z is
// read once and dz written once, which is what the operator cannot do without.
// Counts are integers; every floating sum runs in a fixed order: rows of a
// chunk by warp, warps of a block, chunks of a segment.
//
// Up to three kernels, chained by programmatic dependent launch:
//   count   (gradient only) a block per long chunk of consecutive tokens: a
//           histogram in shared memory for each segment that it meets;
//   pass    a block per short chunk; its first rows of z are on their way
//           before it waits for the histograms.  Without a gradient a
//           ninth warp counts the block's tokens and there is no count kernel;
//   finish  a cluster per segment: counts, P and the loss from the partials.
// Chunk c and segment s meet in at most one run of tokens, and along the
// tokens both only grow, so c + s names each meeting once: a block writes its
// partials of a segment to slot c + s, and no slot has two writers.  Nothing
// needs clearing before a call, and no atomic leaves a block.
//
// For short segments one kernel does all three steps, a cluster per segment
// with cluster barriers between them: there the launches are the time.
//
// Memory bound when large: T = 65536, E = 256, f32 logits take 32.9 us with the
// gradient (134 MB: 20 us at a copy's rate; the count and finish kernels and
// their hand-over are about 8), 20.4 us without (10).  64 x 64: 6.1 us.
#include <algorithm>

#include "area.cuh"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalBlocks = 456;          // most chunks of a call: 3 blocks on each of 152 SMs
constexpr int kMaxAssign = 1 << 26;      // T * k of a call
constexpr int kMaxSeq = 65535;
constexpr int kCountThreads = 1024;
constexpr int kCluster = 8;              // PeerWords reads as many
constexpr long long kSmallElems = 1 << 16;   // logits of a mean segment, see is_small

struct BalParams {
  const void *z;
  const float *bias;          // [E] or nullptr (softmax modes)
  const int32_t *idx;         // [T][k]
  const uint8_t *mask;        // [T] or nullptr
  const int32_t *seq_off;     // [S + 1] or nullptr (one segment of T tokens)
  const float *grad;          // [S] or nullptr (1)
  float *loss;                // [S]
  int32_t *counts;            // [S][E]
  int32_t *tokens;            // [S]
  float *prob;                // [S][E]
  void *dz;                   // [T][E] or nullptr
  float *part;                // [chunks + S][E4] partial sums of p
  int32_t *cnt;               // [count chunks + S][E4 + 4] partial counts, kept tokens at E4
  long long ldz, lddz;
  int T, E, k, S;
  int E4;                     // E rounded up to 4: whole 16-byte pieces
  int chunk, cchunk;          // tokens per block of the pass, and of what counts
  int idx_vec;                // idx rows are whole 16-byte pieces
  float alpha;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_nctarank;" : "=r"(r));
  return r;
}
// Called by all threads of all CTAs of the cluster, converged.
__device__ __forceinline__ void cluster_sync() {
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// The same barrier in two halves: every CTA of the cluster has started once
// the wait returns, so its shared memory may be written.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The 32-bit word at p (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t ld_peer(const void *p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// The words at p of all CTAs (r < ranks, at most kCluster), all asked for before
// the first is used.
struct PeerWords {
  uint32_t w[8];
  __device__ __forceinline__ PeerWords(const void *p, int ranks) {
#pragma unroll
    for (int r = 0; r < 8; ++r) w[r] = r < ranks ? ld_peer(p, r) : 0u;
  }
  __device__ __forceinline__ int sum() const {
    int c = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) c += (int)w[r];
    return c;
  }
  __device__ __forceinline__ float fsum() const {   // in rank order
    float c = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) c += __uint_as_float(w[r]);
    return c;
  }
};

// First and past-the-last token of segment s, inside [0, T] whatever seq_off holds.
__device__ __forceinline__ int seg_begin(const BalParams &p, int s) {
  return p.seq_off ? min(max(p.seq_off[s], 0), p.T) : 0;
}
__device__ __forceinline__ int seg_end(const BalParams &p, int s) {
  return p.seq_off ? min(max(p.seq_off[s + 1], 0), p.T) : p.T;
}

// The first segment that ends past token t (S if there is none), for a whole
// warp: seq_off is non-decreasing, so each step tests 32 segments at once.  In
// any order of seq_off's values, a segment that is returned ends past t (it was
// tested itself), so a walk that goes on from its end always moves.
__device__ __forceinline__ int seg_of(const BalParams &p, int t) {
  if (!p.seq_off) return t < p.T ? 0 : 1;
  const int lane = threadIdx.x & 31;
  int lo = 0, n = p.S;                       // the answer is in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int s = lo + min((lane + 1) * step, n) - 1;   // last of this lane's piece
    const unsigned open = __ballot_sync(0xffffffffu, seg_end(p, s) > t);
    if (!open) return lo + n;
    const int hi = lo + n;
    lo += (__ffs(open) - 1) * step;
    n = min(step, hi - lo) - 1;              // that piece's last one ends past t
  }
  return lo;
}

// ---------------------------------------------------------------- counts --

// Adds the assignments of tokens [a, b) that the mask keeps, this thread's
// share of them (thread i of n takes rows a + i, a + i + n, ..), to hist[E]
// and the kept tokens to hist[E].
__device__ __forceinline__ void count_rows(const BalParams &p, int a, int b, int i, int n, int32_t *hist) {
  int kept = 0;
  for (int t = a + i; t < b; t += n) {
    if (p.mask && !p.mask[t]) continue;
    ++kept;
    const int32_t *row = p.idx + (size_t)t * p.k;
    if (p.idx_vec) {
      for (int j = 0; j < p.k; j += 4) {
        const int4 v = __ldg(reinterpret_cast<const int4 *>(row + j));
        if ((uint32_t)v.x < (uint32_t)p.E) atomicAdd(&hist[v.x], 1);
        if ((uint32_t)v.y < (uint32_t)p.E) atomicAdd(&hist[v.y], 1);
        if ((uint32_t)v.z < (uint32_t)p.E) atomicAdd(&hist[v.z], 1);
        if ((uint32_t)v.w < (uint32_t)p.E) atomicAdd(&hist[v.w], 1);
      }
    } else {
      for (int j = 0; j < p.k; ++j) {
        const int e = __ldg(row + j);
        if ((uint32_t)e < (uint32_t)p.E) atomicAdd(&hist[e], 1);
      }
    }
  }
  kept = __reduce_add_sync(0xffffffffu, kept);
  if ((threadIdx.x & 31) == 0 && kept) atomicAdd(&hist[p.E], kept);
}

// The histogram of tokens [a, b) of segment s into slot blockIdx.x + s, by
// threads i of n with `sync` between them; hist[E + 1] is shared memory.
template <class F>
__device__ __forceinline__ void count_chunk(const BalParams &p, int s, int a, int b, int32_t *hist, int i,
                                            int n, F sync) {
  for (int e = i; e <= p.E; e += n) hist[e] = 0;
  sync();
  count_rows(p, a, b, i, n, hist);
  sync();
  int32_t *dst = p.cnt + (size_t)(blockIdx.x + s) * (p.E4 + 4);
  for (int e = i; e < p.E4; e += n) dst[e] = e < p.E ? hist[e] : 0;
  if (i == 0) dst[p.E4] = hist[p.E];
  sync();
}

// Calls f(s, a, b) for every segment s and its tokens [a, b) inside [t0, t1).
template <class F>
__device__ __forceinline__ void each_segment(const BalParams &p, int t0, int t1, F f) {
  for (int at = t0; at < t1;) {
    const int s = seg_of(p, at);
    if (s >= p.S) break;
    const int a = max(at, seg_begin(p, s)), b = min(t1, seg_end(p, s));
    if (a >= t1) break;
    at = b;                                  // past `at`: the segment ends after it
    if (a < b) f(s, a, b);
  }
}

__global__ void __launch_bounds__(kCountThreads) balance_count_kernel(const BalParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int32_t hist[kMaxExperts + 1];
  const int t0 = blockIdx.x * p.cchunk, t1 = min(p.T, t0 + p.cchunk);
  each_segment(p, t0, t1, [&](int s, int a, int b) {
    count_chunk(p, s, a, b, hist, threadIdx.x, blockDim.x, [] { __syncthreads(); });
  });
}

// The slots that hold segment s's partial counts: first and past the last.
__device__ __forceinline__ int2 count_slots(const BalParams &p, int s) {
  const int a = seg_begin(p, s), b = seg_end(p, s);
  const int c0 = a / p.cchunk;
  return make_int2(c0 + s, a < b ? (b - 1) / p.cchunk + 1 + s : c0 + s);
}

// Segment s's counts added up into sum[E4 + 4] (shared memory, kept tokens at
// E4) by the whole block: a warp per slot, integer atomics.
__device__ __forceinline__ void total_counts(const BalParams &p, int s, int32_t *sum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  for (int e = threadIdx.x; e < p.E4 + 4; e += blockDim.x) sum[e] = 0;
  __syncthreads();
  const int2 sl = count_slots(p, s);
  const int row = p.E4 + 4;
  int n = 0;
  for (int i = sl.x + (int)threadIdx.x; i < sl.y; i += blockDim.x)
    n += __ldcg(p.cnt + (size_t)i * row + p.E4);
  for (int e = 4 * lane; e < p.E4; e += 256) {   // two pieces of a slot at a time
    int4 c = make_int4(0, 0, 0, 0), d = make_int4(0, 0, 0, 0);
    const bool two = e + 128 < p.E4;
#pragma unroll 4
    for (int i = sl.x + warp; i < sl.y; i += nw) {
      const int32_t *src = p.cnt + (size_t)i * row + e;
      const int4 u = __ldcg(reinterpret_cast<const int4 *>(src));
      const int4 v = two ? __ldcg(reinterpret_cast<const int4 *>(src + 128)) : make_int4(0, 0, 0, 0);
      c.x += u.x, c.y += u.y, c.z += u.z, c.w += u.w;
      d.x += v.x, d.y += v.y, d.z += v.z, d.w += v.w;
    }
    if (c.x) atomicAdd(&sum[e], c.x);
    if (c.y) atomicAdd(&sum[e + 1], c.y);
    if (c.z) atomicAdd(&sum[e + 2], c.z);
    if (c.w) atomicAdd(&sum[e + 3], c.w);
    if (d.x) atomicAdd(&sum[e + 128], d.x);
    if (d.y) atomicAdd(&sum[e + 129], d.y);
    if (d.z) atomicAdd(&sum[e + 130], d.z);
    if (d.w) atomicAdd(&sum[e + 131], d.w);
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0 && n) atomicAdd(&sum[p.E4], n);
  __syncthreads();
}

// -------------------------------------------------------------- one token --

// A token's logits over LPR lanes (a power of two) of a warp, 32 / LPR tokens
// at a time: VPL vectors of VEC neighbouring experts per lane.
template <int DT_, int VEC_, int VPL_, int LPR_, bool kSig_>
struct Lay {
  static constexpr int DT = DT_, VEC = VEC_, VPL = VPL_, LPR = LPR_, NE = VEC * VPL;
  static constexpr bool kSig = kSig_;
  // First expert of vector i in this lane.
  static __device__ __forceinline__ int first(int i) {
    return (i * LPR + (int)(threadIdx.x & (LPR - 1))) * VEC;
  }
  static __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  static __device__ __forceinline__ float max(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
  // Raw registers of one lane's logits; -infinity (p = 0) where there is none,
  // so that nothing later asks whether an expert exists.
  struct Raw {
    static constexpr int N = DT == MOE_F32 ? NE : (VEC == 1 ? NE : NE / 2);
    uint32_t w[N];
  };
  static constexpr uint32_t kNone = DT == MOE_F32 ? 0xFF800000u : 0xFF80FF80u;
  static constexpr int ES = DT == MOE_F32 ? 4 : 2;
  // row: the token's first logit of this lane, i.e. of expert first(0).
  static __device__ __forceinline__ void load(const BalParams &p, const char *row, bool there, Raw &r) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool in = there && first(i) < p.E;
      const char *at = row + i * (LPR * VEC * ES);
      if constexpr (VEC == 1) {
        r.w[i] = kNone;
        if (in) {
          if constexpr (DT == MOE_F32) r.w[i] = __float_as_uint(__ldcs(reinterpret_cast<const float *>(at)));
          else r.w[i] = __ldcs(reinterpret_cast<const unsigned short *>(at));
        }
      } else {
        uint4 u = make_uint4(kNone, kNone, kNone, kNone);
        if (in) u = __ldcs(reinterpret_cast<const uint4 *>(at));
        r.w[4 * i] = u.x, r.w[4 * i + 1] = u.y, r.w[4 * i + 2] = u.z, r.w[4 * i + 3] = u.w;
      }
    }
  }
  static __device__ __forceinline__ float get(const Raw &r, int j) {   // logit j of the lane
    if constexpr (DT == MOE_F32) return __uint_as_float(r.w[j]);
    if constexpr (VEC == 1) return __uint_as_float(r.w[j] << 16);
    const uint32_t w = r.w[j / 2];
    return __uint_as_float((j & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  static __device__ __forceinline__ void store(const BalParams &p, char *row, const float (&d)[NE]) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (first(i) >= p.E) continue;
      char *at = row + i * (LPR * VEC * ES);
      if constexpr (VEC == 1) {
        if constexpr (DT == MOE_F32) __stcs(reinterpret_cast<float *>(at), d[i]);
        else *reinterpret_cast<__nv_bfloat16 *>(at) = __float2bfloat16_rn(d[i]);
      } else if constexpr (DT == MOE_F32) {
        __stcs(reinterpret_cast<float4 *>(at), make_float4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]));
      } else {
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          // the gradient's one rounding, to the logits' own type
          const __nv_bfloat162 h = __floats2bfloat162_rn(d[8 * i + 2 * c], d[8 * i + 2 * c + 1]);
          w[c] = *reinterpret_cast<const uint32_t *>(&h);
        }
        __stcs(reinterpret_cast<uint4 *>(at), make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
  }
};

// p of the lane's token added to acc, and (kGrad) the token's gradient written
// from coef, the counts less their mean, in shared memory.  valid: the token
// exists and the mask keeps it; write: it exists (a masked token's gradient is
// 0).  Every lane of the warp takes part.  bias and coef cover the layout's
// experts (0 past E).
//
// The mean taken off the counts cancels in a_i - sum_e p_e a_e, and small
// differences keep their digits.
//
// exp is the hardware one (2 units and |z| 2^-24, 0 below 2^-126) and the
// reciprocal good to a unit: p is a sum's share, held in f32.
__device__ __forceinline__ float exp_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// With u the sigmoid (or exp(z - max)) and inv 1 / sum u: p = u inv, and
//   dz_i = scale inv u_i (1 - sigmoid_i) (coef_i - dot),  dot = inv sum u_e coef_e
template <class L, bool kGrad>
__device__ __forceinline__ void one_token(const BalParams &p, const typename L::Raw &raw, char *dst, bool valid,
                                          bool write, const float *bias, const float *coef, float scale,
                                          float (&acc)[L::NE]) {
  float u[L::NE], w[L::kSig && kGrad ? L::NE : 1];   // w: u (1 - sigmoid)
  if constexpr (L::LPR == 32) {   // the warp's one token
    if (!valid) {
      if (kGrad && write) {
#pragma unroll
        for (int j = 0; j < L::NE; ++j) u[j] = 0.f;
        L::store(p, dst, u);
      }
      return;
    }
  }
  float tot = 0.f;
  if constexpr (L::kSig) {
#pragma unroll
    for (int j = 0; j < L::NE; ++j) {
      const float ex = exp_fast(-L::get(raw, j));
      u[j] = rcp_fast(1.0f + ex);   // 0 from 2^126 on
      // 1 - sigmoid as exp(-z) sigmoid: its digits stay where the sigmoid is
      // near 1.  The bound keeps infinity times 0 out; a NaN is in u.
      if constexpr (kGrad) w[j] = u[j] * (fminf(ex, 8.5e37f) * u[j]);
      tot += u[j];
    }
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < L::NE; ++j) {
      u[j] = L::get(raw, j);
      if (bias) u[j] += bias[L::first(j / L::VEC) + j % L::VEC];
      m = fmaxf(m, u[j]);
    }
    m = L::max(m);
    if (m == -INFINITY) m = 0.f;   // a row with nothing left: p = 0
#pragma unroll
    for (int j = 0; j < L::NE; ++j) {
      u[j] = exp_fast(u[j] - m);
      tot += u[j];
    }
  }
  if constexpr (L::LPR < 32) {
    // Beside other tokens of the warp: nothing of a masked one is used, whatever
    // its logits, the bias or the gradient from above hold.
    if (!valid) {
#pragma unroll
      for (int j = 0; j < L::NE; ++j) {
        u[j] = 0.f;
        if constexpr (L::kSig && kGrad) w[j] = 0.f;
      }
      tot = 0.f;
    }
  }
  tot = L::sum(tot);
  if constexpr (L::kSig && kGrad) {
    // A row of sigmoids that are all tiny is scaled up by 2^64: 1 / tot, its
    // product with a large gradient, and tiny times small counts all stay in
    // f32's range, and p = u / tot is the same to the bit.
    if (tot < 0x1p-32f) {
#pragma unroll
      for (int j = 0; j < L::NE; ++j) u[j] *= 0x1p64f, w[j] *= 0x1p64f;
      tot *= 0x1p64f;
    }
  }
  const float inv = tot == 0.f ? 0.f : rcp_fast(tot);   // tot >= 2^-126 otherwise
#pragma unroll
  for (int j = 0; j < L::NE; ++j) acc[j] = fmaf(u[j], inv, acc[j]);
  if constexpr (kGrad) {
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < L::NE; ++j) dot = fmaf(u[j], coef[L::first(j / L::VEC) + j % L::VEC], dot);
    dot = L::sum(dot) * inv;
    const float k = inv == 0.f ? 0.f : scale * inv;   // no probabilities: no gradient
#pragma unroll
    for (int j = 0; j < L::NE; ++j) {
      const float c = (coef[L::first(j / L::VEC) + j % L::VEC] - dot) * k;
      u[j] = c * (L::kSig ? w[j] : u[j]);
    }
    if (write) L::store(p, dst, u);
  }
}

// A warp's rows first, first + step, .. below b, with the loads of kAhead steps
// under way where a lane's share is short (65536 x 256 step: 32.8 us with 2,
// 33.6 with 3, 35.6 with 4, whose registers cost more than they hide).
template <class L>
struct Rows {
  static constexpr int RPW = 32 / L::LPR;   // rows per warp and step
  static constexpr int kAhead = L::NE <= 16 ? 2 : 1;
  typename L::Raw raw[kAhead];
  bool valid[kAhead];
  int t;              // the next token to fetch, its logits, and its mask
  const char *z;
  // The logits' load does not wait for the mask's.
  __device__ __forceinline__ void fetch(const BalParams &p, int i, int step, int b) {
    valid[i] = t < b && (!p.mask || p.mask[t]);
    L::load(p, z, t < b, raw[i]);
    t += step;
    z += (size_t)step * p.ldz * L::ES;
  }
  __device__ __forceinline__ void start(const BalParams &p, int first, int step, int b) {
    t = first + (int)(threadIdx.x & 31) / L::LPR;
    z = reinterpret_cast<const char *>(p.z) + ((size_t)t * p.ldz + L::first(0)) * L::ES;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(p, i, step, b);
  }
  template <bool kGrad>
  __device__ __forceinline__ void run(const BalParams &p, int first, int step, int b, const float *bias,
                                      const float *coef, float scale, float (&acc)[L::NE]) {
    int now = first + (int)(threadIdx.x & 31) / L::LPR;
    char *dst = reinterpret_cast<char *>(p.dz) + ((size_t)now * p.lddz + L::first(0)) * L::ES;
    for (int row0 = first; row0 < b; row0 += kAhead * step) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (row0 + i * step < b) {   // the same for the whole warp
          typename L::Raw mine = raw[i];
          const bool ok = valid[i];
          fetch(p, i, step, b);
          one_token<L, kGrad>(p, mine, dst, ok, now < b, bias, coef, scale, acc);
          now += step;
          if constexpr (kGrad) dst += (size_t)step * p.lddz * L::ES;
        }
      }
    }
  }
};

// The bias over the layout's EP experts, 0 past E, into shared memory.
template <int EP>
__device__ __forceinline__ void stage_bias(const BalParams &p, float *bias) {
  if (p.bias)
    for (int e = threadIdx.x; e < EP; e += blockDim.x) bias[e] = e < p.E ? __ldg(p.bias + e) : 0.f;
}

__device__ __forceinline__ float grad_scale(const BalParams &p, int s, int tokens) {
  const float n = (float)tokens;
  return n > 0.f ? (p.grad ? p.grad[s] : 1.f) * p.alpha * (float)p.E / (float)p.k / n / n : 0.f;
}

// Adds the subgroups of a warp (the same experts) and leaves the warp's sums
// in sums[warp][NE * LPR].
template <class L>
__device__ __forceinline__ void warp_sums(float (&acc)[L::NE], float *sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < L::NE; ++j) {
#pragma unroll
    for (int o = 16; o >= L::LPR; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    if (lane < L::LPR) sums[warp * (L::NE * L::LPR) + L::first(j / L::VEC) + j % L::VEC] = acc[j];
  }
}

// -------------------------------------------------------------- main pass --

template <class L, bool kGrad>
__global__ void __launch_bounds__(kBalThreads + (kGrad ? 0 : 32), L::NE <= 8 ? 3 : 1) balance_pass_kernel(const BalParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int EP = L::NE * L::LPR;   // experts of the layout, >= E
  __shared__ float sums[kBalWarps * EP];
  __shared__ __align__(16) float coef[kGrad ? EP : 1], bias[L::kSig ? 1 : EP];
  // kGrad: the segment's counts, before sums holds anything; else the ninth
  // warp's histogram of the block's own tokens.
  __shared__ int32_t hist[kGrad ? 1 : EP + 1];
  int32_t *ints = kGrad ? reinterpret_cast<int32_t *>(sums) : hist;
  const int warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  constexpr int kStep = kBalWarps * Rows<L>::RPW;
  bool waited = false;
  if constexpr (!L::kSig) {
    stage_bias<EP>(p, bias);
    __syncthreads();
  }
  each_segment(p, t0, t1, [&](int s, int a, int b) {
    const int first = a + warp * Rows<L>::RPW;
    Rows<L> rows;
    if (kGrad || warp < kBalWarps) rows.start(p, first, kStep, b);
    float scale = 0.f;
    if constexpr (kGrad) {
      if (!waited) {
        asm volatile("griddepcontrol.wait;" ::: "memory");   // the partial counts
        waited = true;
      }
      total_counts(p, s, ints);
      scale = grad_scale(p, s, ints[p.E4]);
      int sum = 0;   // every warp for itself: all assignments of the segment
      for (int e = threadIdx.x & 31; e < p.E; e += 32) sum += ints[e];
      const float mean = (float)__reduce_add_sync(0xffffffffu, sum) / (float)p.E;
      for (int e = threadIdx.x; e < EP; e += blockDim.x)
        coef[e] = e < p.E ? (float)ints[e] - mean : 0.f;
      __syncthreads();
    }
    if (kGrad || warp < kBalWarps) {
      float acc[L::NE];
#pragma unroll
      for (int j = 0; j < L::NE; ++j) acc[j] = 0.f;
      rows.template run<kGrad>(p, first, kStep, b, p.bias ? bias : nullptr, coef, scale, acc);
      warp_sums<L>(acc, sums);
    } else {
      count_chunk(p, s, a, b, ints, threadIdx.x & 31, 32, [] { __syncwarp(); });
    }
    __syncthreads();
    float *dst = p.part + (size_t)(blockIdx.x + s) * p.E4;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
      float tsum = 0.f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) tsum += sums[w * EP + e];
      dst[e] = tsum;
    }
    __syncthreads();
  });
  // The finish kernel waits for this grid alone: leave only after the counts.
  if (kGrad && !waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// -------------------------------------------------------------- finish ----

// The loss of a segment from each CTA's share of sum_e c_e P_e, which warp 0
// holds in its lanes: every rank puts its sum into rank 0's shares[], and after
// the one cluster barrier rank 0 adds them in rank order.
__device__ __forceinline__ void finish_loss(const BalParams &p, int s, float dot, float inv, float *shares) {
  const int ranks = cluster_size(), rank = cluster_rank();
  if (threadIdx.x < 32) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (threadIdx.x == 0) {
      uint32_t a;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                   : "=r"(a)
                   : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(shares + rank))), "r"(0));
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(dot) : "memory");
    }
  }
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    float tot = 0.f;
    for (int r = 0; r < ranks; ++r) tot += shares[r];
    p.loss[s] = p.alpha * (float)p.E / (float)p.k * inv * tot;
  }
}

// A cluster per segment: rank r takes experts 32 r .. 32 r + 31, 32 (r +
// ranks) .., four to a lane; a warp reads four slots at a time, and the sums of
// its quarters and of the warps are added in that order.
constexpr int kFinishWarps = 16;

__global__ void __launch_bounds__(kFinishWarps * 32) balance_finish_kernel(const BalParams p) {
  cluster_arrive();
  const int ranks = cluster_size(), rank = cluster_rank(), s = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quarter = lane >> 3, piece = (lane & 7) * 4;
  const int a = seg_begin(p, s), b = seg_end(p, s);
  const int c0 = a / p.chunk + s, c1 = a < b ? (b - 1) / p.chunk + 1 + s : c0;
  const int2 sl = count_slots(p, s);
  const int row = p.E4 + 4;
  __shared__ float4 part[kFinishWarps][8];
  __shared__ int32_t counts[32], kept;
  __shared__ float shares[kCluster];
  if (threadIdx.x < 32) counts[threadIdx.x] = 0;
  if (threadIdx.x == 0) kept = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int n = 0;
  for (int i = sl.x + (int)threadIdx.x; i < sl.y; i += blockDim.x)
    n += __ldcg(p.cnt + (size_t)i * row + p.E4);
  float dot = 0.f, inv = 0.f;
  for (int e0 = rank * 32; e0 < p.E; e0 += ranks * 32) {
    const int e = e0 + piece;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    int4 c = make_int4(0, 0, 0, 0);
    if (e < p.E4) {
#pragma unroll 8
      for (int i = c0 + warp * 4 + quarter; i < c1; i += kFinishWarps * 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.part + (size_t)i * p.E4 + e));
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
      }
#pragma unroll 8
      for (int i = sl.x + warp * 4 + quarter; i < sl.y; i += kFinishWarps * 4) {
        const int4 v = __ldcg(reinterpret_cast<const int4 *>(p.cnt + (size_t)i * row + e));
        c.x += v.x, c.y += v.y, c.z += v.z, c.w += v.w;
      }
    }
#pragma unroll
    for (int o = 8; o <= 16; o <<= 1) {
      sum.x += __shfl_xor_sync(0xffffffffu, sum.x, o), sum.y += __shfl_xor_sync(0xffffffffu, sum.y, o);
      sum.z += __shfl_xor_sync(0xffffffffu, sum.z, o), sum.w += __shfl_xor_sync(0xffffffffu, sum.w, o);
    }
    if (quarter == 0) part[warp][lane] = sum;
    if (c.x) atomicAdd(&counts[piece], c.x);
    if (c.y) atomicAdd(&counts[piece + 1], c.y);
    if (c.z) atomicAdd(&counts[piece + 2], c.z);
    if (c.w) atomicAdd(&counts[piece + 3], c.w);
    if (e0 == rank * 32) {
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0 && n) atomicAdd(&kept, n);
    }
    __syncthreads();
    if (warp == 0) {
      n = kept;
      inv = n > 0 ? 1.0f / (float)n : 0.f;
      float tot = 0.f;
#pragma unroll
      for (int w = 0; w < kFinishWarps; ++w) tot += reinterpret_cast<const float *>(part[w])[lane];
      tot *= inv;
      if (e0 + lane < p.E) {
        p.prob[(size_t)s * p.E + e0 + lane] = tot;
        p.counts[(size_t)s * p.E + e0 + lane] = counts[lane];
        dot = fmaf((float)counts[lane], tot, dot);
      }
      counts[lane] = 0;
    }
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) p.tokens[s] = n;   // rank 0 always has experts
  __syncthreads();
  cluster_wait();
  finish_loss(p, s, dot, inv, shares);
}

// ---------------------------------------------------------- small batches --

// In an order that seq_off must not have, every segment could be all T tokens
// long and the call n_seq * T rows of work.  So a segment of more than kLongSeg
// tokens and more than kLongSeg mean segments has its array's order checked
// first, and counts as empty where the order is wrong: no call works on more
// than kLongSeg * (T + n_seq) rows.
constexpr int kLongSeg = 64;

template <class L>
__global__ void __launch_bounds__(kBalThreads, L::NE <= 8 ? 3 : 1) balance_small_kernel(const BalParams p) {
  constexpr int EP = L::NE * L::LPR;
  __shared__ float sums[kBalWarps * EP];
  __shared__ __align__(16) float coef[EP], bias[L::kSig ? 1 : EP];
  float *mine = sums;   // the block's sums, in place of warp 0's
  __shared__ int32_t hist[EP + 1];
  __shared__ float shares[kCluster];
  __shared__ int total;
  const int ranks = cluster_size(), rank = cluster_rank(), s = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5;
  const int a = seg_begin(p, s);
  int b = seg_end(p, s);
  // The same for all CTAs of the cluster; never with one segment (no seq_off).
  if (b - a > kLongSeg && (long long)(b - a) * p.S > (long long)kLongSeg * p.T) {
    int bad = 0;
    for (int i = threadIdx.x; i < p.S; i += blockDim.x) bad |= p.seq_off[i + 1] < p.seq_off[i];
    if (__syncthreads_or(bad)) b = a;
  }
  constexpr int kStep = kBalWarps * Rows<L>::RPW;
  const int first = a + (rank * kBalWarps + warp) * Rows<L>::RPW;
  Rows<L> rows;
  rows.start(p, first, ranks * kStep, b);
  if (!L::kSig) stage_bias<EP>(p, bias);
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) hist[e] = 0;
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  count_rows(p, a, b, rank * blockDim.x + threadIdx.x, ranks * blockDim.x, hist);
  cluster_sync();
  // Every CTA adds up the whole segment's counts for itself (coef: as floats).
  int sum = 0;
  const int n = PeerWords(&hist[p.E], ranks).sum();
  for (int e = threadIdx.x; e < EP; e += blockDim.x) {
    const int c = e < p.E ? PeerWords(&hist[e], ranks).sum() : 0;
    coef[e] = (float)c;
    sum += c;
    if (rank == 0 && e < p.E) p.counts[(size_t)s * p.E + e] = c;
  }
  if (rank == 0 && threadIdx.x == 0) p.tokens[s] = n;
  sum = __reduce_add_sync(0xffffffffu, sum);
  if ((threadIdx.x & 31) == 0) atomicAdd(&total, sum);
  __syncthreads();
  const float mean = (float)total / (float)p.E;
  const float scale = grad_scale(p, s, n), inv = n > 0 ? 1.0f / (float)n : 0.f;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) coef[e] -= mean;
  __syncthreads();
  float acc[L::NE];
#pragma unroll
  for (int j = 0; j < L::NE; ++j) acc[j] = 0.f;
  const float *sb = p.bias ? bias : nullptr;
  if (p.dz) rows.template run<true>(p, first, ranks * kStep, b, sb, coef, scale, acc);
  else rows.template run<false>(p, first, ranks * kStep, b, sb, coef, scale, acc);
  warp_sums<L>(acc, sums);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    float tsum = 0.f;
#pragma unroll
    for (int w = 0; w < kBalWarps; ++w) tsum += sums[w * EP + e];
    mine[e] = tsum;
  }
  cluster_sync();
  float dot = 0.f;
  for (int e = rank + ranks * (int)threadIdx.x; e < p.E; e += ranks * blockDim.x) {
    const float tot = PeerWords(&mine[e], ranks).fsum() * inv;
    p.prob[(size_t)s * p.E + e] = tot;
    sums[EP + e] = (coef[e] + mean) * tot;   // past `mine`, which the peers read
  }
  __syncthreads();
  if (warp == 0)   // this rank's experts, in their order
    for (int e = rank + ranks * (int)(threadIdx.x & 31); e < p.E; e += ranks * 32) dot += sums[EP + e];
  finish_loss(p, s, dot, inv, shares);
}

// ----------------------------------------------------------------- launch --

template <typename... KArgs>
cudaError_t launch_cluster(bool pdl, void (*kernel)(KArgs...), int blocks, int threads, int ranks,
                           cudaStream_t st, const BalParams &p) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

int balance_chunk(int T) {
  // One block's tokens: 32 (four per warp) until that makes kBalBlocks blocks.
  return std::max(32, (T + kBalBlocks - 1) / kBalBlocks);
}

// Tokens per histogram: what a block of the pass has when it counts for itself;
// the count kernel's blocks take 256, or more to stay at 64 blocks (each block
// of the pass reads every histogram of its segment).
int balance_count_chunk(int T, bool grad) {
  return grad ? std::max(256, (T + 63) / 64) : balance_chunk(T);
}

// One kernel where a mean segment has at most 2^16 logits: a block of the three
// takes its segments one after the other, about 4 us each.  With a gradient, us
// in one kernel and in three: T = 512, E = 64, one segment 6.1 and 7.9; 1024 x
// 256, one segment 14.5 and 9.7; 4096 x 256, 24 segments 11.4 and 19.6, 8
// segments 15.4 and 14.8; 16389 x 256, 64 segments 18.7 and 25.6, 24 segments
// 23.6 and 19.1; 65536 x 256, 256 segments 56 and 71, 1024 segments 146 and 191;
// 32768 x 256, 4096 segments of 8 tokens 110 and 607.  One segment with nearly
// all the tokens costs both: 65536 x 256 in 256 segments then 511 and 769.
bool is_small(int T, int E, int S) { return (long long)T * E <= kSmallElems * S; }

template <class L>
cudaError_t launch_layout(const BalParams &p, cudaStream_t st) {
  if (is_small(p.T, p.E, p.S)) {
    // CTAs of a segment: one for every two steps of its share of the rows
    // (four times the mean segment: they differ in length).
    const int rows = std::min<long long>(p.T, 4LL * ((p.T + p.S - 1) / p.S));
    const int step = 2 * kBalWarps * Rows<L>::RPW;
    int ranks = 1;
    while (ranks < kCluster && ranks * step < rows) ranks *= 2;
    return launch_cluster(false, balance_small_kernel<L>, p.S * ranks, kBalThreads, ranks, st, p);
  }
  const int chunks = (p.T + p.chunk - 1) / p.chunk;
  cudaError_t err = cudaSuccess;
  if (p.dz) {
    err = launch_k(false, balance_count_kernel, dim3((p.T + p.cchunk - 1) / p.cchunk),
                   dim3(kCountThreads), 0, st, p);
    if (err == cudaSuccess)
      err = launch_k(true, balance_pass_kernel<L, true>, dim3(chunks), dim3(kBalThreads), 0, st, p);
  } else {
    err = launch_k(false, balance_pass_kernel<L, false>, dim3(chunks), dim3(kBalThreads + 32), 0, st, p);
  }
  if (err == cudaSuccess)
    err = launch_cluster(true, balance_finish_kernel, p.S * kCluster, kFinishWarps * 32, kCluster, st, p);
  return err;
}

// Vectors where rows are whole 16-byte pieces, as few lanes a row as hold it.
template <int DT, bool kSig>
cudaError_t launch_balance(const BalParams &p, bool vec, cudaStream_t st) {
  constexpr int V = DT == MOE_F32 ? 4 : 8;
  if (vec) {
    if (p.E <= 8 * V) return launch_layout<Lay<DT, V, 1, 8, kSig>>(p, st);
    if (p.E <= 16 * V) return launch_layout<Lay<DT, V, 1, 16, kSig>>(p, st);
    if (p.E <= 32 * V) return launch_layout<Lay<DT, V, 1, 32, kSig>>(p, st);
    if (p.E <= 64 * V) return launch_layout<Lay<DT, V, 2, 32, kSig>>(p, st);
    if (p.E <= 128 * V) return launch_layout<Lay<DT, V, 4, 32, kSig>>(p, st);
    if constexpr (DT == MOE_F32) return launch_layout<Lay<DT, V, 8, 32, kSig>>(p, st);
  }
  if (p.E <= 64) return launch_layout<Lay<DT, 1, 2, 32, kSig>>(p, st);
  if (p.E <= 256) return launch_layout<Lay<DT, 1, 8, 32, kSig>>(p, st);
  return launch_layout<Lay<DT, 1, 32, 32, kSig>>(p, st);
}

}  // namespace
}  // namespace moe

extern "C" __attribute__((visibility("default"))) size_t moe_balance_workspace(int T, int num_experts,
                                                                              int n_seq) {
  using namespace moe;
  if (T < 1 || T > kMaxAssign || num_experts < 1 || num_experts > kMaxExperts || n_seq < 1 ||
      n_seq > kMaxSeq)
    return 0;
  // Partial sums of p, and partial counts in the form that has more of them.
  const int chunk = balance_chunk(T);
  const size_t slots = (size_t)(T + chunk - 1) / chunk + n_seq, E4 = (num_experts + 3) / 4 * 4;
  return slots * (2 * E4 + 4) * sizeof(float);
}

extern "C" __attribute__((visibility("default"))) int moe_balance_loss(
    const void *z, const float *bias, const int32_t *idx, const uint8_t *mask,
    const int32_t *seq_off, int T, int num_experts, int top_k, int n_seq, int z_dtype,
    int router_mode, float alpha, const float *grad, int64_t z_stride, float *loss,
    int32_t *counts, int32_t *tokens, float *prob, void *dz, int64_t dz_stride, void *workspace,
    size_t workspace_bytes, moe_stream_t stream) {
  using namespace moe;
  if (num_experts < 1 || num_experts > kMaxExperts || top_k < 1 || top_k > num_experts ||
      top_k > kMaxTopK || router_mode < 0 || router_mode > 2)
    return MOE_ERR_ROUTING;
  if (T < 0 || n_seq < 1 || n_seq > kMaxSeq || (!seq_off && n_seq != 1) ||
      (z_dtype != MOE_F32 && z_dtype != MOE_BF16) || !(alpha - alpha == 0.f) ||
      (long long)T * top_k > kMaxAssign)
    return MOE_ERR_ARG;
  const int E = num_experts;
  const long long ldz = z_stride ? z_stride : E, lddz = dz_stride ? dz_stride : E;
  if (ldz < E || lddz < E || ldz > (1LL << 32) || lddz > (1LL << 32)) return MOE_ERR_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {   // every segment is empty
    if (!loss || !counts || !tokens || !prob) return MOE_OK;
    const size_t S4 = (size_t)n_seq * 4, SE4 = S4 * E;
    const Area wr[] = {area(loss, S4), area(counts, SE4), area(tokens, S4), area(prob, SE4)};
    for (int i = 0; i < 4; ++i) {
      if (reinterpret_cast<uintptr_t>(wr[i].p) & 3) return MOE_ERR_ARG;
      for (int j = 0; j < i; ++j)
        if (meet(wr[i], wr[j])) return MOE_ERR_ARG;
    }
    for (const Area &a : wr)
      if (cudaMemsetAsync(const_cast<void *>(a.p), 0, a.bytes, st) != cudaSuccess) return MOE_ERR_DEVICE;
    return MOE_OK;
  }
  if (!loss || !counts || !tokens || !prob || !z || !idx) return MOE_ERR_ARG;
  if (workspace_bytes < moe_balance_workspace(T, E, n_seq)) return MOE_ERR_NOMEM;
  if (!workspace) return MOE_ERR_ARG;
  const uintptr_t za = z_dtype == MOE_F32 ? 3 : 1;
  if (((reinterpret_cast<uintptr_t>(z) | reinterpret_cast<uintptr_t>(dz)) & za) ||
      ((reinterpret_cast<uintptr_t>(bias) | reinterpret_cast<uintptr_t>(idx) |
        reinterpret_cast<uintptr_t>(seq_off) | reinterpret_cast<uintptr_t>(grad) |
        reinterpret_cast<uintptr_t>(loss) | reinterpret_cast<uintptr_t>(counts) |
        reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(prob) |
        0) & 3) ||
      (reinterpret_cast<uintptr_t>(workspace) & 15))
    return MOE_ERR_ARG;
  // What the kernels write is apart from everything else that the call
  // touches; dz may be z itself (a row is read whole before it is written).
  {
    const size_t ze = z_dtype == MOE_F32 ? 4 : 2, S = n_seq, SE = S * E * 4;
    const Area in[] = {{z, (size_t)T, E * ze, (size_t)ldz * ze},
                       area(idx, (size_t)T * top_k * 4),
                       area(bias, (size_t)E * 4),
                       area(mask, T),
                       area(seq_off, (S + 1) * 4),
                       area(grad, S * 4)};
    const Area wr[] = {{dz, (size_t)T, E * ze, (size_t)lddz * ze},
                       area(loss, S * 4),
                       area(counts, SE),
                       area(tokens, S * 4),
                       area(prob, SE),
                       area(workspace, moe_balance_workspace(T, E, n_seq))};
    for (int i = 0; i < 6; ++i) {
      for (int j = 0; j < 6; ++j)
        if (!(i == 0 && j == 0 && dz == z && lddz == ldz) && meet(wr[i], in[j])) return MOE_ERR_ARG;
      for (int j = 0; j < i; ++j)
        if (meet(wr[i], wr[j])) return MOE_ERR_ARG;
    }
  }
  BalParams p{z, router_mode == 1 ? nullptr : bias, idx, mask, seq_off, grad, loss, counts, tokens,
              prob, dz, static_cast<float *>(workspace), nullptr, ldz, lddz, T, E, top_k, n_seq,
              (E + 3) / 4 * 4, balance_chunk(T), balance_count_chunk(T, dz != nullptr), top_k % 4 == 0 && !(reinterpret_cast<uintptr_t>(idx) & 15), alpha};
  p.cnt = reinterpret_cast<int32_t *>(p.part + ((size_t)(T + p.chunk - 1) / p.chunk + n_seq) * p.E4);
  const long long v = z_dtype == MOE_F32 ? 4 : 8;
  const bool vec = E % v == 0 && ldz % v == 0 && !(reinterpret_cast<uintptr_t>(z) & 15) &&
                   (!dz || (lddz % v == 0 && !(reinterpret_cast<uintptr_t>(dz) & 15)));
  const bool sig = router_mode == 1;
  const cudaError_t err =
      z_dtype == MOE_F32 ? (sig ? launch_balance<MOE_F32, true>(p, vec, st) : launch_balance<MOE_F32, false>(p, vec, st))
                         : (sig ? launch_balance<MOE_BF16, true>(p, vec, st) : launch_balance<MOE_BF16, false>(p, vec, st));
  return err == cudaSuccess ? MOE_OK : MOE_ERR_DEVICE;
}
