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
// Counts are integers (their atomics commute); every floating sum runs in a
// fixed order: rows of a chunk by warp, warps of a block, chunks of a segment.
//
// A chunk is a run of consecutive tokens, one block's work.  Chunk c and
// segment s meet in at most one run of tokens, and along the tokens both only
// grow, so c + s names each meeting once: the block writes its partial sums of
// a segment to slot c + s, and no slot has two writers.
#include <algorithm>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalChunks = 3 * 1024;   // most chunks of a call

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
  float *part;                // [chunks + S][E] partial sums of p
  long long ldz, lddz;
  int T, E, k, S, chunk;      // chunk: tokens per block
  float alpha;
};

// First and past-the-last token of segment s, inside [0, T] whatever seq_off holds.
__device__ __forceinline__ int seg_begin(const BalParams &p, int s) {
  return p.seq_off ? min(max(p.seq_off[s], 0), p.T) : 0;
}
__device__ __forceinline__ int seg_end(const BalParams &p, int s) {
  return p.seq_off ? min(max(p.seq_off[s + 1], 0), p.T) : p.T;
}

// The first segment that ends past token t (S if there is none): by halving,
// seq_off being non-decreasing.
__device__ __forceinline__ int seg_of(const BalParams &p, int t) {
  int lo = 0, hi = p.S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seg_end(p, mid) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// ---------------------------------------------------------------- counts --
// Block = chunk of tokens: a histogram in shared memory per segment that the
// chunk meets, added to the segment's counts.
__global__ void __launch_bounds__(kBalThreads) balance_count_kernel(const BalParams p, int chunk) {
  extern __shared__ int32_t hist[];   // [E + 1]: counts, then the kept tokens
  const int t0 = blockIdx.x * chunk, t1 = min(p.T, t0 + chunk);
  for (int s = seg_of(p, t0); s < p.S; ++s) {
    const int a = max(t0, seg_begin(p, s)), b = min(t1, seg_end(p, s));
    if (seg_begin(p, s) >= t1) break;
    if (a >= b) continue;
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int32_t *idx = p.idx + (size_t)a * p.k;
    const int n = (b - a) * p.k;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int row = i / p.k;
      if (p.mask && !p.mask[a + row]) continue;
      const int e = idx[i];
      if (e >= 0 && e < p.E) atomicAdd(&hist[e], 1);
      if (i == row * p.k) atomicAdd(&hist[p.E], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x)
      if (hist[e]) atomicAdd(&p.counts[(size_t)s * p.E + e], hist[e]);
    if (threadIdx.x == 0 && hist[p.E]) atomicAdd(&p.tokens[s], hist[p.E]);
    __syncthreads();
  }
}

// -------------------------------------------------------------- main pass --

template <int DT>
__device__ __forceinline__ float load_z(const void *z, size_t i) {
  if constexpr (DT == MOE_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(z)[i]);
  return reinterpret_cast<const float *>(z)[i];
}

template <int DT>
__device__ __forceinline__ void store_z(void *z, size_t i, float v) {
  if constexpr (DT == MOE_BF16) reinterpret_cast<__nv_bfloat16 *>(z)[i] = __float2bfloat16_rn(v);
  else reinterpret_cast<float *>(z)[i] = v;
}

// One warp per token; expert e lives in lane e % 32, slot e / 32 (EPL slots).
template <int DT, int EPL, bool kSigmoid>
__global__ void __launch_bounds__(kBalThreads) balance_pass_kernel(const BalParams p) {
  pdl_enter();
  extern __shared__ float sums[];   // [kBalWarps][E]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  for (int s = seg_of(p, t0); s < p.S; ++s) {
    const int a = max(t0, seg_begin(p, s)), b = min(t1, seg_end(p, s));
    if (seg_begin(p, s) >= t1) break;
    if (a >= b) continue;
    float acc[EPL], ce[EPL];
    const int32_t *counts = p.counts + (size_t)s * p.E;
    float scale = 0.f;
    if (p.dz) {
      // Gradient coefficients with the mean taken off the counts: the term
      // it adds cancels in a_i - sum_e p_e a_e, and small differences keep
      // their digits.
      const float n = (float)__ldcg(p.tokens + s);
      scale = n > 0.f ? (p.grad ? p.grad[s] : 1.f) * p.alpha * (float)p.E / (float)p.k / n / n : 0.f;
      int sum = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i < p.E) sum += __ldcg(counts + lane + 32 * i);
      sum = __reduce_add_sync(0xffffffffu, sum);
      const float mean = (float)sum / (float)p.E;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        ce[i] = lane + 32 * i < p.E ? (float)__ldcg(counts + lane + 32 * i) - mean : 0.f;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = 0.f;
    for (int t = a + warp; t < b; t += kBalWarps) {
      const bool keep = !p.mask || p.mask[t];
      if (!keep) {
        if (p.dz) {
#pragma unroll
          for (int i = 0; i < EPL; ++i)
            if (lane + 32 * i < p.E) store_z<DT>(p.dz, (size_t)t * p.lddz + lane + 32 * i, 0.f);
        }
        continue;
      }
      float v[EPL], om[EPL];
      float tot = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        v[i] = e < p.E ? load_z<DT>(p.z, (size_t)t * p.ldz + e) : -INFINITY;
      }
      if constexpr (kSigmoid) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          // 0 past E: expf(inf) = inf.  1 - sigmoid is taken as e sigmoid,
          // which keeps its digits where the sigmoid is near 1.
          const float ex = expf(-v[i]);
          v[i] = 1.0f / (1.0f + ex);
          om[i] = ex < 1e30f ? ex * v[i] : 1.0f - v[i];
          tot += v[i];
        }
      } else {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          if (p.bias && lane + 32 * i < p.E) v[i] += p.bias[lane + 32 * i];
          m = fmaxf(m, v[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (m == -INFINITY) m = 0.f;   // a row with nothing left: p = 0
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          v[i] = lane + 32 * i < p.E ? expf(v[i] - m) : 0.f;
          tot += v[i];
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
      const float inv = tot == 0.f ? 0.f : 1.0f / tot;
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        v[i] *= inv;
        acc[i] += v[i];
        if (p.dz) dot = fmaf(v[i], ce[i], dot);
      }
      if (p.dz) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = lane + 32 * i;
          float d = scale * v[i] * (ce[i] - dot);
          if constexpr (kSigmoid) d *= om[i];
          if (e < p.E) store_z<DT>(p.dz, (size_t)t * p.lddz + e, d);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 32 * i < p.E) sums[warp * p.E + lane + 32 * i] = acc[i];
    __syncthreads();
    float *dst = p.part + (size_t)(blockIdx.x + s) * p.E;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
      float tsum = 0.f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) tsum += sums[w * p.E + e];
      dst[e] = tsum;
    }
    __syncthreads();
  }
}

// -------------------------------------------------------------- finish ----
// Block = segment: P from the chunks' partial sums in chunk order, then loss.
__global__ void __launch_bounds__(1024) balance_finish_kernel(const BalParams p) {
  pdl_enter();
  __shared__ float red[32];
  const int s = blockIdx.x;
  const int a = seg_begin(p, s), b = seg_end(p, s);
  const int n = __ldcg(p.tokens + s);
  const float inv = n > 0 ? 1.0f / (float)n : 0.f;
  float dot = 0.f;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    float sum = 0.f;
    if (a < b)
      for (int c = a / p.chunk; c <= (b - 1) / p.chunk; ++c)
        sum += __ldcg(p.part + (size_t)(c + s) * p.E + e);
    sum *= inv;
    p.prob[(size_t)s * p.E + e] = sum;
    dot = fmaf((float)__ldcg(p.counts + (size_t)s * p.E + e), sum, dot);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    float tot = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) tot += red[w];
    p.loss[s] = p.alpha * (float)p.E / (float)p.k * inv * tot;
  }
}

int balance_chunk(int T) {
  // One block's tokens: 32 (four per warp) until that makes kBalChunks blocks.
  return std::max(32, (T + kBalChunks - 1) / kBalChunks);
}

template <int DT, bool kSigmoid>
cudaError_t launch_pass(const BalParams &p, int chunks, cudaStream_t st) {
  const size_t smem = (size_t)kBalWarps * p.E * sizeof(float);
  const int epl = (p.E + 31) / 32;
  auto k = epl <= 1    ? balance_pass_kernel<DT, 1, kSigmoid>
           : epl <= 2  ? balance_pass_kernel<DT, 2, kSigmoid>
           : epl <= 4  ? balance_pass_kernel<DT, 4, kSigmoid>
           : epl <= 8  ? balance_pass_kernel<DT, 8, kSigmoid>
           : epl <= 16 ? balance_pass_kernel<DT, 16, kSigmoid>
                       : balance_pass_kernel<DT, 32, kSigmoid>;
  return launch_k(true, k, dim3(chunks), dim3(kBalThreads), smem, st, p);
}

}  // namespace
}  // namespace moe

extern "C" __attribute__((visibility("default"))) size_t moe_balance_workspace(int T, int num_experts,
                                                                              int n_seq) {
  using namespace moe;
  if (T < 1 || num_experts < 1 || num_experts > kMaxExperts || n_seq < 1) return 0;
  const int chunk = balance_chunk(T);
  const size_t slots = (size_t)(T + chunk - 1) / chunk + n_seq;
  return slots * num_experts * sizeof(float);
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
  if (T < 0 || n_seq < 1 || n_seq > 65535 || (!seq_off && n_seq != 1) ||
      (z_dtype != MOE_F32 && z_dtype != MOE_BF16) || !(alpha - alpha == 0.f) ||
      (long long)T * top_k > (1LL << 26))
    return MOE_ERR_ARG;
  const int E = num_experts;
  const long long ldz = z_stride ? z_stride : E, lddz = dz_stride ? dz_stride : E;
  if (ldz < E || lddz < E || ldz > (1LL << 32) || lddz > (1LL << 32)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!loss || !counts || !tokens || !prob || !z || !idx) return MOE_ERR_ARG;
  if (workspace_bytes < moe_balance_workspace(T, E, n_seq)) return MOE_ERR_NOMEM;
  if (!workspace) return MOE_ERR_ARG;
  const uintptr_t za = z_dtype == MOE_F32 ? 3 : 1;
  if (((reinterpret_cast<uintptr_t>(z) | reinterpret_cast<uintptr_t>(dz)) & za) ||
      ((reinterpret_cast<uintptr_t>(bias) | reinterpret_cast<uintptr_t>(idx) |
        reinterpret_cast<uintptr_t>(seq_off) | reinterpret_cast<uintptr_t>(grad) |
        reinterpret_cast<uintptr_t>(loss) | reinterpret_cast<uintptr_t>(counts) |
        reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(prob) |
        reinterpret_cast<uintptr_t>(workspace)) & 3))
    return MOE_ERR_ARG;
  // What the kernels write is apart from everything else that the call
  // touches; dz may be z itself (a row is read whole before it is written).
  {
    const size_t ze = z_dtype == MOE_F32 ? 4 : 2, SE = (size_t)n_seq * E * 4;
    struct Area {
      const void *p;
      size_t n;
    };
    const Area in[] = {{z, ((size_t)(T - 1) * ldz + E) * ze},
                       {idx, (size_t)T * top_k * 4},
                       {bias, bias ? (size_t)E * 4 : 0},
                       {mask, mask ? (size_t)T : 0},
                       {seq_off, seq_off ? (size_t)(n_seq + 1) * 4 : 0},
                       {grad, grad ? (size_t)n_seq * 4 : 0}};
    const Area wr[] = {{dz, dz ? ((size_t)(T - 1) * lddz + E) * ze : 0},
                       {loss, (size_t)n_seq * 4},
                       {counts, SE},
                       {tokens, (size_t)n_seq * 4},
                       {prob, SE},
                       {workspace, moe_balance_workspace(T, E, n_seq)}};
    auto meet = [](const Area &a, const Area &b) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
      return a.n && b.n && x < y + b.n && y < x + a.n;
    };
    for (int i = 0; i < 6; ++i) {
      for (int j = 0; j < 6; ++j)
        if (!(i == 0 && j == 0 && dz == z && lddz == ldz) && meet(wr[i], in[j])) return MOE_ERR_ARG;
      for (int j = 0; j < i; ++j)
        if (meet(wr[i], wr[j])) return MOE_ERR_ARG;
    }
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  BalParams p{z, router_mode == 1 ? nullptr : bias, idx, mask, seq_off, grad, loss,
              counts, tokens, prob, dz, static_cast<float *>(workspace), ldz, lddz, T, E, top_k,
              n_seq, balance_chunk(T), alpha};
  cudaError_t err = cudaMemsetAsync(counts, 0, (size_t)n_seq * E * sizeof(int32_t), st);
  if (err == cudaSuccess) err = cudaMemsetAsync(tokens, 0, (size_t)n_seq * sizeof(int32_t), st);
  if (err == cudaSuccess) {
    const int cc = std::max(64, (T + 1023) / 1024);   // count kernel: at most 1024 blocks
    err = launch_k(false, balance_count_kernel, dim3((T + cc - 1) / cc), dim3(kBalThreads),
                   (size_t)(E + 1) * sizeof(int32_t), st, p, cc);
    const int chunks = (T + p.chunk - 1) / p.chunk;
    const bool sig = router_mode == 1;
    if (err == cudaSuccess)
      err = z_dtype == MOE_F32
                ? (sig ? launch_pass<MOE_F32, true>(p, chunks, st) : launch_pass<MOE_F32, false>(p, chunks, st))
                : (sig ? launch_pass<MOE_BF16, true>(p, chunks, st) : launch_pass<MOE_BF16, false>(p, chunks, st));
  }
  if (err == cudaSuccess)
    err = launch_k(true, balance_finish_kernel, dim3(n_seq), dim3(E <= 256 ? 256 : 1024), 0, st, p);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_DEVICE;
}
