// rope.cu -- rotary positions (moe_rope in include/moe.h).
//
//   a = pos f_i;  u' = m (u cos a - v sin a),  v' = m (u sin a + v cos a)
//
// Angles: f_i / (2 pi) is kept as a 64-bit fraction of a turn, so that pos times
// it, modulo 2^64, is the angle modulo a turn without any reduction: off by
// 2^-64 turns for each position and by the double's own 2^-53, where an f32
// product at position 10^6 is off by a sixteenth of a radian.  The two highest bits are
// the quadrant; the sine and cosine of what is left come as a float and what the float
// lacks, so that mscale times them is rounded once: in all half a unit and 2^-25.4.
//
// A block turns some heads of one token.  Its threads first ask for their
// elements, then work out the token's sines and cosines once into shared
// memory, so both latencies overlap and a pair's angle is computed once for all
// of the block's heads.
//
// The floor is one read and one write.  4096 tokens of 40 heads of 128, bfloat16:
// 15.7 us (5.3 TB/s), in place 15.3; 17.9 and 18.0 without streaming loads, which leave
// L2 to what is written.  Half the warps' slots are taken; capping registers for more
// blocks an SM (18.4 us and up), 128 threads (16.2 against 15.8) and, before the streaming loads,
// one or four units a thread (18.8, 23.5 against 17.9) were slower.  104 heads of one
// token: 2.1 us, a launch and one trip to memory.
#include <algorithm>
#include <cmath>

#include "area.cuh"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kRopeMaxD = 1024;
constexpr int kRopeThreads = 256;

struct RopeParams {
  const void *x;
  const int32_t *pos;
  const double *freqs;
  void *out;
  long long ldx, ldxh, ldo, ldoh;   // strides in elements: token rows, heads
  int heads, D, R;
  int turns;         // units of V pairs in the turned part of a head
  int units;         // units of a head (the turned ones, then 2 V copied elements each)
  int heads_block;   // heads of one block
  float mscale;
  bool inverse;
};

// f radians as a fraction of a turn, in 2^-64 (two's complement, modulo 1): right to that,
// and to 2^-127 of f where f is many turns.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
  const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
  const int e = (int)(bits >> 52) & 0x7FF;
  if (e == 0) return 0ull;   // zero, and subnormals: less than 2^-64 turns at any position
  // f = m 2^(e - 1086) with m's top bit set; times 2^66 / (2 pi) is m k 2^(e - 1086).
  const unsigned long long m = (1ull << 63) | (bits << 11);
  // k: 2^66 / (2 pi) in 64 bits and 64 more.
  const unsigned long long k = 0xA2F9836E4E441529ull, k_low = 0xFC2757D1F534DDC0ull;
  const unsigned long long more = __umul64hi(m, k_low), lo = m * k + more;
  const unsigned long long hi = __umul64hi(m, k) + (lo < more);   // hi, lo: m k 2^-64
  const int shift = e - 1024;                                     // 2^64 turns = hi 2^(e - 1024)
  const unsigned long long r = shift <= -64 ? 0ull
                               : shift <= 0 ? hi >> -shift
                               : shift < 64 ? hi << shift | lo >> (64 - shift)
                               : shift < 128 ? lo << (shift - 64)
                                             : 0ull;
  return bits >> 63 ? 0ull - r : r;
}

// m cos and m sin of turn 2^-64 turns.  The angle beyond the nearest quarter turn is
// a + b, a float and what it lacks; Taylor's series to a^11 and a^10 (2e-9 at an eighth
// of a turn), each result a float and what it lacks until m is in it.
__device__ __forceinline__ float2 turn_cos_sin(unsigned long long turn, float m) {
  const unsigned long long q = (turn + (1ull << 61)) >> 62;
  const unsigned long long r = turn - (q << 62);   // -2^61 .. 2^61
  const int top = (int)(r >> 32);
  const float h = (float)top, l = (float)(top - (int)h) + (float)(uint32_t)r * 2.3283064365386963e-10f;
  const float k = 1.46291807927e-9f, k_low = -4.07094027e-17f;   // 2 pi 2^-32
  const float a = h * k, b = fmaf(h, k, -a) + fmaf(h, k_low, l * k);
  const float z = a * a;
  float p = fmaf(z, -2.5052108e-8f, 2.7557319e-6f);
  p = fmaf(p, z, -1.9841270e-4f);
  p = fmaf(p, z, 8.3333333e-3f);
  p = fmaf(p, z, -0.16666667f);
  const float t = fmaf(p * z, a, fmaf(-0.5f * z, b, b));
  const float s = a + t, s_low = (a - s) + t;
  const float w = fmaf(-0.5f, z, 1.f), left = fmaf(-0.5f, z, 1.f - w);
  p = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  p = fmaf(p, z, -1.3888889e-3f);
  p = fmaf(p, z, 0.041666667f);
  const float u = fmaf(z * z, p, left) - fmaf(0.5f, fmaf(a, a, -z), a * b);
  const float c = w + u, c_low = (w - c) + u;
  const float mc = fmaf(m, c, m * c_low), ms = fmaf(m, s, m * s_low);
  const float x = q & 1 ? ms : mc, y = q & 1 ? mc : ms;
  return make_float2((q + 1) & 2 ? -x : x, q & 2 ? -y : y);
}

template <int B>
struct Raw;
template <> struct Raw<2> { typedef unsigned short T; };
template <> struct Raw<4> { typedef uint32_t T; };
template <> struct Raw<8> { typedef uint2 T; };
template <> struct Raw<16> { typedef uint4 T; };

// N elements of one type, moved in pieces of at most 16 bytes.
template <int DT, int N>
struct Piece {
  static constexpr int kBytes = N * (DT == MOE_BF16 ? 2 : 4);
  static constexpr int kWord = kBytes < 16 ? kBytes : 16;
  typedef typename Raw<kWord>::T Word;
  Word w[kBytes / kWord];
  __device__ __forceinline__ void load(const void *base, long long i) {
    const Word *p = reinterpret_cast<const Word *>(reinterpret_cast<const char *>(base) +
                                                   i * (DT == MOE_BF16 ? 2 : 4));
#pragma unroll
    for (int c = 0; c < kBytes / kWord; ++c) w[c] = __ldcs(p + c);   // read once
  }
  __device__ __forceinline__ void store(void *base, long long i) const {
    Word *p = reinterpret_cast<Word *>(reinterpret_cast<char *>(base) + i * (DT == MOE_BF16 ? 2 : 4));
#pragma unroll
    for (int c = 0; c < kBytes / kWord; ++c) p[c] = w[c];
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == MOE_F32) return reinterpret_cast<const float *>(w)[i];
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(w)[i]);
  }
  __device__ __forceinline__ void set(int i, float v) {
    if constexpr (DT == MOE_F32) reinterpret_cast<float *>(w)[i] = v;
    else reinterpret_cast<__nv_bfloat16 *>(w)[i] = __float2bfloat16_rn(v);
  }
};

// V pairs per unit; NU units per thread.
template <int DT, int V, bool kInterleaved, int NU>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  __shared__ float cs[kRopeMaxD / 2], sn[kRopeMaxD / 2];
  const long long t = blockIdx.x;
  const int h0 = blockIdx.y * p.heads_block, nh = min(p.heads_block, p.heads - h0);
  const int n = nh * p.units;
  // A unit's elements: V and V of the halves, or 2 V in a row (also the copied ones).
  Piece<DT, V> a[NU], b[NU];
  long long dst[NU];
  int pair[NU];   // first pair of the unit; -1: copied; -2: none; -3: V elements copied
  for (int base = 0; base < n; base += NU * blockDim.x) {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const int u = base + threadIdx.x + j * blockDim.x;
      pair[j] = -2;
      if (u >= n) continue;
      const int h = u / p.units, i = u - h * p.units;
      long long src = t * p.ldx + (h0 + h) * p.ldxh;
      dst[j] = t * p.ldo + (h0 + h) * p.ldoh;
      if (i < p.turns) {
        pair[j] = i * V;
        const int first = kInterleaved ? 2 * i * V : i * V;
        src += first, dst[j] += first;
        a[j].load(p.x, src);
        b[j].load(p.x, src + (kInterleaved ? V : p.R / 2));
      } else {
        const int first = p.R + (i - p.turns) * 2 * V;
        src += first, dst[j] += first;
        pair[j] = first + V < p.D ? -1 : -3;
        a[j].load(p.x, src);
        if (pair[j] == -1) b[j].load(p.x, src + V);
      }
    }
    if (base == 0) {
      const long long pos = __ldg(p.pos + t);
      for (int i = threadIdx.x; i < p.R / 2; i += blockDim.x) {
        const double f = __ldg(p.freqs + i);
        const unsigned long long turn = turn_fraction(f) * (unsigned long long)pos;
        float2 t = turn_cos_sin(turn, p.mscale);
        if (!isfinite(f)) t.x = t.y = __int_as_float(0x7fffffff);
        cs[i] = t.x;
        sn[i] = p.inverse ? -t.y : t.y;
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      if (pair[j] >= 0) {
        const float *c = cs + pair[j], *s = sn + pair[j];
        if constexpr (kInterleaved) {
          // element 2 i and 2 i + 1 of the 2 V in a and b
          float e[2 * V];
#pragma unroll
          for (int i = 0; i < V; ++i) e[i] = a[j].get(i), e[V + i] = b[j].get(i);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float u = e[2 * i], v = e[2 * i + 1];
            e[2 * i] = u * c[i] - v * s[i];
            e[2 * i + 1] = u * s[i] + v * c[i];
          }
#pragma unroll
          for (int i = 0; i < V; ++i) a[j].set(i, e[i]), b[j].set(i, e[V + i]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float u = a[j].get(i), v = b[j].get(i);
            a[j].set(i, u * c[i] - v * s[i]);
            b[j].set(i, u * s[i] + v * c[i]);
          }
        }
      }
      if (pair[j] == -2) continue;
      a[j].store(p.out, dst[j]);
      if (pair[j] != -3) b[j].store(p.out, dst[j] + (kInterleaved || pair[j] < 0 ? V : p.R / 2));
    }
  }
}

template <int DT, int V>
cudaError_t launch_rope(RopeParams p, int T, bool interleaved, bool in_place, cudaStream_t st) {
  p.turns = p.R / (2 * V);
  p.units = p.turns;
  // In place the elements past R stay where they are.
  if (!in_place) p.units += (p.D - p.R + 2 * V - 1) / (2 * V);
  if (p.units == 0) return cudaSuccess;
  // Two units a thread where there are tokens enough for every SM, else one;
  // heads are split over blocks where one block does not hold them.
  const int nu = (long long)T * p.heads * p.units >= 2 * 152 * 2048 ? 2 : 1;
  const int per = std::max(1, kRopeThreads * nu / p.units);
  const int ny = (p.heads + per - 1) / per;
  p.heads_block = (p.heads + ny - 1) / ny;
  const int threads = std::min(kRopeThreads, (p.heads_block * p.units + 32 * nu - 1) / (32 * nu) * 32);
  auto k = nu == 2 ? (interleaved ? rope_kernel<DT, V, true, 2> : rope_kernel<DT, V, false, 2>)
                   : (interleaved ? rope_kernel<DT, V, true, 1> : rope_kernel<DT, V, false, 1>);
  return launch_k(false, k, dim3(T, ny), dim3(threads), 0, st, p);
}

}  // namespace
}  // namespace moe

extern "C" __attribute__((visibility("default"))) int moe_rope(
    const void *x, const int32_t *pos, const double *freqs, int T, int n_heads, int head_dim,
    int rot_dim, int interleaved, int inverse, float mscale, int dtype, void *out,
    int64_t x_stride, int64_t x_head_stride, int64_t out_stride, int64_t out_head_stride,
    moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || T > (1 << 24) || n_heads < 1 || head_dim < 2 || head_dim > kRopeMaxD ||
      (long long)n_heads * head_dim > (1 << 20) || rot_dim < 2 || rot_dim % 2 || rot_dim > head_dim ||
      !std::isfinite(mscale) || (dtype != MOE_F32 && dtype != MOE_BF16))
    return MOE_ERR_ARG;
  const long long ldxh = x_head_stride ? x_head_stride : head_dim,
                  ldoh = out_head_stride ? out_head_stride : head_dim,
                  ldx = x_stride ? x_stride : n_heads * ldxh,
                  ldo = out_stride ? out_stride : n_heads * ldoh;
  // Either order: heads inside a token's row, or tokens inside a head's.
  constexpr long long kMaxStride = 1LL << 32;
  auto apart = [&](long long ld, long long ldh) {
    if (ld < head_dim || ldh < head_dim || ld > kMaxStride || ldh > kMaxStride) return false;
    return n_heads == 1 || T <= 1 || ld >= (n_heads - 1) * ldh + head_dim ||
           ldh >= (T - 1) * ld + head_dim;
  };
  if (!apart(ldx, ldxh) || !apart(ldo, ldoh)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  const size_t es = dtype == MOE_F32 ? 4 : 2;
  if (!x || !pos || !freqs || !out) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & (es - 1)) return MOE_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(pos) & 3 || reinterpret_cast<uintptr_t>(freqs) & 7) return MOE_ERR_ARG;
  // Rows as wide as a token's heads where these lie inside it, else the whole.
  auto rows = [&](const void *p, long long ld, long long ldh) {
    const size_t wide = ((size_t)(n_heads - 1) * ldh + head_dim) * es;
    if (wide <= (size_t)ld * es) return Area{p, (size_t)T, wide, (size_t)ld * es};
    return area(p, (size_t)(T - 1) * ld * es + wide);
  };
  const Area ax = rows(x, ldx, ldxh), ao = rows(out, ldo, ldoh), ap = area(pos, (size_t)T * 4),
             af = area(freqs, (size_t)rot_dim * 4);
  const bool in_place = x == out && ldx == ldo && ldxh == ldoh;
  if ((!in_place && meet(ao, ax)) || meet(ao, ap) || meet(ao, af)) return MOE_ERR_ARG;
  RopeParams p{x, pos, freqs, out, ldx, ldxh, ldo, ldoh, n_heads, head_dim, rot_dim, 0, 0, 0, mscale,
               inverse != 0};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // The widest unit that every piece of a head is a multiple of, in whole
  // aligned words.
  auto fits = [&](int v) {
    const size_t word = std::min<size_t>(16, v * es);
    return rot_dim % (2 * v) == 0 && head_dim % v == 0 && ((size_t)ldx * es) % word == 0 &&
           ((size_t)ldxh * es) % word == 0 && ((size_t)ldo * es) % word == 0 &&
           ((size_t)ldoh * es) % word == 0 &&
           ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & (word - 1)) == 0;
  };
  cudaError_t err;
  const bool il = interleaved != 0;
  if (dtype == MOE_F32)
    err = fits(4) ? launch_rope<MOE_F32, 4>(p, T, il, in_place, st) : launch_rope<MOE_F32, 1>(p, T, il, in_place, st);
  else
    err = fits(8) ? launch_rope<MOE_BF16, 8>(p, T, il, in_place, st)
          : fits(4) ? launch_rope<MOE_BF16, 4>(p, T, il, in_place, st)
                    : launch_rope<MOE_BF16, 1>(p, T, il, in_place, st);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

extern "C" __attribute__((visibility("default"))) int moe_rope_freqs(
    int rot_dim, double theta, int scaling, double factor, double context, double beta_fast,
    double beta_slow, double *freqs, float *mscale) {
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > moe::kRopeMaxD || !std::isfinite(theta) || theta < 1.0 ||
      !std::isfinite(factor) || factor < 1.0 || scaling < MOE_ROPE_PLAIN || scaling > MOE_ROPE_PARTS ||
      !freqs)
    return MOE_ERR_ARG;
  if (scaling == MOE_ROPE_BASE && rot_dim == 2) return MOE_ERR_ARG;
  if (scaling == MOE_ROPE_PARTS &&
      (!std::isfinite(context) || context < 1.0 || !std::isfinite(beta_fast) || !(beta_slow >= 0.0) ||
       !(beta_slow < beta_fast)))
    return MOE_ERR_ARG;
  const double base = scaling == MOE_ROPE_BASE
                          ? theta * std::pow(factor, rot_dim / (rot_dim - 2.0)) : theta;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == MOE_ROPE_LINEAR) f /= factor;
    if (scaling == MOE_ROPE_PARTS) {
      const double r = context * f / 6.283185307179586476925;
      const double keep = std::min(1.0, std::max(0.0, (r - beta_slow) / (beta_fast - beta_slow)));
      f *= keep + (1.0 - keep) / factor;
    }
    freqs[i] = f;
  }
  if (mscale) *mscale = scaling == MOE_ROPE_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return MOE_OK;
}
