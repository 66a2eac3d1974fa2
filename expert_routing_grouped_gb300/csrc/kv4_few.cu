// kv4_few.cu -- attention of a few rows a sequence over the 4-bit cache: decoded
// tokens, and drafted ones, up to 16 columns (rows times query heads of a KV head).
//
//   S^T[token][column] = K . q^T,  O^T[dim][column] = V^T . P^T
//
// on warp-level MMAs (m16n8k16, float16): 16 tokens, then 16 dimensions, are the
// rows, columns the 8-wide side: 8 query heads of a KV head waste nothing, one alone
// uses an eighth.
//
//   Codes: a code in the lowest bits of a float16 is the subnormal number c 2^-24,
//      four bits further up c 2^-20: one AND makes a pair of exact operands, with
//      nothing to add or take away.  The factors 2^24 and 16 go into q, the scales
//      and the output.
//   K: a lane's 16 codes of a token and group are 4 k-steps of the MMA as they lie
//      (which dimension is which k is free as long as q agrees), one accumulator
//      for each group: s = sum_g step_g acc_g + lo_g sum(q of g), no rounding of K.
//   q: float16 after a power of two per column that brings its largest just under
//      2^15: exact to 2^-25 of that.
//   P: for each group w step times a power of two, rounded to float16 (2^-11 at
//      most), in the accumulator's layout, transposed by movmatrix: the B operand.
//      V's codes are exact, and sum w lo is kept beside in f32.
//
// Each warp streams its own tiles of 32 tokens through a private ring in shared
// memory by cp.async (no barrier, no waiting but its own), with a running
// maximum that moves only when a score passes it by 8, so most tiles exchange
// nothing.  The power of two of w step is each column's and group's own: it brings
// the largest product that the column has met to 2^7 .. 2^15, so that what other
// groups hold, or tokens of little weight or that the column does not see, takes no
// bits from it (2^-25 of float16's subnormals is 2^-32 of the largest product).
// Maxima are whole numbers: where one moves, the powers move with it and the
// outputs stay as they are.  The block's warps join at the end.
//
// The tiles of all sequences and KV heads lie in one line that is cut into equal
// spans, one for each block, whatever the lengths; a second kernel joins what was cut.
//
// The floor is the cache, 9/16 bytes an element; what bounds it is latency: 878
// instructions for 32 tokens of 16 columns, issued at 2.1 of the 4 a clock and SM by
// three warps a scheduler (four with 8 columns), too few to cover one another's chains.
// One token of 96 query and 8 KV heads over 131072 tokens: 50.2 us (3.0 TB/s); 64 tokens
// of 32 and 8 heads over up to 8192 each: 52.6 us (3.6 TB/s); one over 4096: 10.8 us,
// mostly launches, the plan and the joining.  One power of two for both groups and all
// tokens took 46.9, 49.4 and 10.2 us and lost small values beside large ones.  An
// earlier form (52.5 us over 131072) took 34.6 us with the copies alone.  Tried: codes
// in 16 mantissa bits and V's scales on the values (57.9 us against 52.8), the codes as
// the A side of tcgen05 MMAs (69 against 53), four blocks an SM with shorter rings for
// 16 columns (67.2 against 52.7).
#include <algorithm>

#include "kv4.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kTile = 32;                   // tokens of a ring slot
constexpr int kMinTiles = 4;                // tiles of a span, at least: one for each warp
constexpr int kPlanSeqs = 1024;             // sequences of a batch that is cut into spans
constexpr int kColumns = kFewColumns;
constexpr int kFewSms = 152;                // blocks are sized for the GB300's SMs
constexpr int kMostUp = 100;                // the largest exponent of w step's factors

template <int D>
struct Slot {
  static constexpr int kK = 0, kV = kTile * D / 2, kKs = kTile * D, kVs = kKs + kTile * D / 16;
  static constexpr int kBytes = kVs + kTile * D / 16;
};
// Four warps to a block: up to 8 columns four blocks on an SM; up to 16, whose
// outputs take twice the registers, three.
constexpr int kWarps = 4;
template <int NT>
constexpr int kBlocks = NT == 1 ? 4 : 3;
template <int D>
constexpr int kRing = D == 64 ? 6 : 3;      // slots of a warp
template <int D>
constexpr int kSmem = kWarps * kRing<D> * Slot<D>::kBytes;

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same onto zeros.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Four pairs of codes of w (nibbles i and i + 4 of it: a pair's halves) as float16
// operands: c 2^-24, c 2^-20 in turn.
__device__ __forceinline__ void four_pairs(uint32_t w, uint32_t (&o)[4]) {
  const uint32_t w8 = w >> 8;
  o[0] = w & 0x000F000Fu;
  o[1] = w & 0x00F000F0u;
  o[2] = w8 & 0x000F000Fu;
  o[3] = w8 & 0x00F000F0u;
}
__device__ __forceinline__ float2 xor_2(float2 v, int d) {
  return make_float2(__shfl_xor_sync(0xffffffffu, v.x, d), __shfl_xor_sync(0xffffffffu, v.y, d));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ uint32_t max2_f16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// 2^e and back (of a normal number: the exponent below; of 0: -127).
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int exponent(float v) { return (__float_as_int(v) >> 23) - 127; }
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// ------------------------------------------------------------------ plan --
//
// The tiles of all sequences and KV heads in one line, each (sequence, head) with
// its own, are cut into equal spans, one for each block, whatever the lengths: a
// block works through the segments of its span.  A segment that is a whole
// (sequence, head) is finished by its block; the others leave partial results, at
// most two for each block: slot 2 b for the one at the start of its span, 2 b + 1
// for one that starts later and goes on in the next.

// What a segment costs beside its tiles, in tiles: start and end take about as
// long as ten tiles of a block.
constexpr int kSegmentCost = 8;

struct SeqTiles {
  int first, n;   // the tiles that any row sees (one at least); n = 0: none of this kernel's sequences
};

__device__ __forceinline__ SeqTiles tiles_of(const AttendParams &p, const AttendSeq &q) {
  if (q.rows < 1 || q.rows * p.G > kColumns) return SeqTiles{0, 0};
  int lo = 0;
  if (p.window) lo = max(0, q.len - q.nq - p.window + 1) / kTile;
  return SeqTiles{lo, max(1, (q.len + kTile - 1) / kTile - lo)};
}

// Tiles of a sequence's line, for one head.
__device__ __forceinline__ int span_of(const SeqTiles &t) { return t.n ? t.n + kSegmentCost : 0; }

// Exclusive prefix of v over the block's threads, and the total.
__device__ __forceinline__ long long block_scan(long long v, long long *warp_sums, long long &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += a;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  long long before = x - v;
  total = 0;
  for (int w = 0; w < nw; ++w) {
    const long long s = warp_sums[w];
    if (w < warp) before += s;
    total += s;
  }
  return before;
}

// The line: its length per block, and of a sequence where it starts.
struct Line {
  long long total, cut, start;
  int s;
};

// With seq < 0 the sequence in which block `block`'s span starts, else that of
// sequence seq.  line.s < 0: none.  kOne: there is one sequence only, and nothing to add
// up (a token over 4096 takes 10.0 us for 10.4).
template <bool kOne>
__device__ __forceinline__ Line find_line(const AttendParams &p, int block, int seq) {
  if constexpr (kOne) {
    Line line;
    line.total = (long long)span_of(tiles_of(p, attend_seq_at(p, 0))) * p.b.Hkv;
    line.cut = max((line.total + p.target - 1) / p.target, (long long)kMinTiles);
    line.s = seq >= 0 || line.cut * block < line.total ? 0 : -1;
    line.start = 0;
    return line;
  }
  __shared__ long long sums[32];
  __shared__ long long start;
  __shared__ int where;
  const int per = (p.b.n_seq + blockDim.x - 1) / blockDim.x, s0 = threadIdx.x * per;
  long long mine = 0;
  for (int s = s0; s < min(s0 + per, p.b.n_seq); ++s)
    mine += (long long)span_of(tiles_of(p, attend_seq_at(p, s))) * p.b.Hkv;
  if (threadIdx.x == 0) where = -1;
  Line line;
  long long at = block_scan(mine, sums, line.total);
  line.cut = max((line.total + p.target - 1) / p.target, (long long)kMinTiles);
  const long long u = line.cut * block;
  if (seq >= 0 ? seq >= s0 && seq < s0 + per : u >= at && u < at + mine) {
    for (int s = s0;; ++s) {
      const long long span = (long long)span_of(tiles_of(p, attend_seq_at(p, s))) * p.b.Hkv;
      if (seq >= 0 ? s == seq : u < at + span) {
        where = s;
        start = at;
        break;
      }
      at += span;
    }
  }
  __syncthreads();
  line.s = where;
  line.start = start;
  return line;
}

// A segment: tiles first .. first + n - 1 of a sequence and KV head; whole: all of them.
struct Segment {
  int s, hk, first, n, slot;
  bool whole;
};

// ---------------------------------------------------------------- kernel --

template <int NT>
struct Joined {
  float m[kWarps][8 * NT], l[kWarps][8 * NT];
  uint4 q[NT == 1 ? 1 : NT][NT == 1 ? 1 : 2][2][NT == 1 ? 1 : 32];   // two column tiles: q's B operands
};

template <int D, int NT>
__device__ __forceinline__ void do_segment(const AttendParams &p, const Segment part, uint8_t *smem,
                                           Joined<NT> &jn) {
  constexpr int NG = D / kKvGroup, MT = D / 16, SB = Slot<D>::kBytes, NS = kRing<D>, W = kWarps;
  constexpr int kPieces = D / 32;            // 16-byte pieces of a token's codes
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const AttendSeq sq = attend_seq_at(p, part.s);
  const int cols = sq.rows * p.G, lp = p.b.log_page;

  // ---- the ring: this warp's tiles are first + warp, + W, ...
  const int n_mine = part.n > warp ? (part.n - warp + W - 1) / W : 0;
  uint8_t *ring = smem + warp * (NS * SB);
  const uint32_t ring_s = smem_u32(ring);
  const int32_t *pages = p.b.pages + (size_t)part.s * p.b.max_pages;
  const uint8_t *head = p.cache + (size_t)part.hk * KvBlock<D>::bytes(lp);
  const size_t page_bytes = KvBlock<D>::bytes(lp) * p.b.Hkv;
  // Pages of the halves (16 tokens) of the warp's i-th tile; -1 also past the end.
  auto page_pair = [&](int i) {
    int2 r = make_int2(-1, -1);
    if (i >= n_mine) return r;
    const int tok = (part.first + warp + i * W) * kTile;
    auto get = [&](int token) {
      if (token >= sq.len) return -1;
      const int id = __ldg(pages + (token >> lp));
      return (unsigned)id < (unsigned)p.b.n_pages ? id : -1;
    };
    r.x = get(tok);
    r.y = lp > 4 ? (tok + 16 < sq.len ? r.x : -1) : get(tok + 16);
    return r;
  };
  // A lane's share of a tile's copies.  Codes: rows of D / 2 bytes, K's in the order
  // of the S rows; of 64-byte rows every other pair has its halves exchanged, so
  // that no loads below meet in a bank.  Whole rows wherever there is a page: a
  // row past the length holds some codes or other, and every code is a finite
  // number.  Scales: zeros past the length, whatever lies there.
  constexpr int kRows = 32 / kPieces;        // tokens of a round of copies: 8 or 16
  constexpr int kTok = 16 / (NG * 4);        // tokens of a 16-byte piece of scales
  constexpr int kSp = kTile / kTok;          // pieces of K's, and of V's: 16 or 8
  const int c_tk = lane / kPieces, c_pc = lane % kPieces;
  const uint32_t c_kr = (c_tk & 8) + 2 * (c_tk & 3) + ((c_tk >> 2) & 1);
  const uint32_t dst_k = ring_s + Slot<D>::kK + c_kr * (D / 2) + (D == 128 ? c_pc ^ (c_kr & 2) : c_pc) * 16;
  const uint32_t dst_v = ring_s + Slot<D>::kV + c_tk * (D / 2) + (D == 128 ? c_pc ^ (c_tk & 2) : c_pc) * 16;
  const int s_which = lane >= kSp, s_tk = (lane - s_which * kSp) * kTok, s_half = s_tk >= 16;
  const uint32_t dst_s = ring_s + (s_which ? Slot<D>::kVs : Slot<D>::kKs) + (lane - s_which * kSp) * 16;
  const uint32_t src_c = c_tk * (D / 2) + c_pc * 16, src_v = (uint32_t)(D / 2) << lp;
  const uint32_t src_s = ((uint32_t)D << lp) + ((uint32_t)(s_which * (D / 16)) << lp) + (s_tk & 15) * (D / 16);
  auto issue = [&](int i, int2 pg) {
    if (i < n_mine) {
      const int tok = (part.first + warp + i * W) * kTile, mask = (1 << lp) - 1;
      const uint32_t to = (i % NS) * SB;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int id = h ? pg.y : pg.x, ok = id >= 0 ? 16 : 0;
        const uint32_t slot = (tok + 16 * h) & mask;
        const uint8_t *blk = head + (size_t)max(id, 0) * page_bytes;
        const uint8_t *src = blk + slot * (D / 2) + src_c;
#pragma unroll
        for (int c = 0; c < 16 / kRows; ++c) {
          copy16(dst_k + to + (16 * h + c * kRows) * (D / 2), src + c * kRows * (D / 2), ok);
          copy16(dst_v + to + (16 * h + c * kRows) * (D / 2), src + src_v + c * kRows * (D / 2), ok);
        }
        if (lane < 2 * kSp && s_half == h)
          copy16(dst_s + to, blk + slot * (D / 16) + src_s,
                 ok ? min(16, max(0, (sq.len - tok - s_tk) * (NG * 4))) : 0);
      }
    }
    copy_commit();
  };
  uint32_t holes = 0;   // two bits a ring slot: halves without a page
  auto note = [&](int i, int2 pg) {
    const int sh = (i % NS) * 2;
    holes = (holes & ~(3u << sh)) | ((pg.x < 0) | (pg.y < 0) << 1) << sh;
  };
  {
    int2 pg[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) pg[i] = page_pair(i);
#pragma unroll
    for (int i = 0; i < NS; ++i) issue(i, pg[i]), note(i, pg[i]);
  }
  int2 next = page_pair(NS);

  // ---- q as B operands: lane (g, t4) holds column 8 nt + g, dimensions 16 t4 ..
  // + 15 of each group
  // (two column tiles: kept in shared memory, where registers are short)
  uint32_t qb[1][NG][8];
  float2 qsum[NT][NG], cs[NT];   // of the columns 8 nt + 2 t4, + 1 of the accumulators
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int c = 8 * nt + g;
    uint4 raw[NG][2];
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) raw[gr][0] = raw[gr][1] = make_uint4(0, 0, 0, 0);
    if (c < cols) {
      const int i = c / p.G, h = part.hk * p.G + c - i * p.G;
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (size_t)(sq.t0 + i) * p.ldq + (size_t)h * D);
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) raw[gr][0] = src[gr * 8 + 2 * t4], raw[gr][1] = src[gr * 8 + 2 * t4 + 1];
    }
    float v[NG][16];
    uint32_t top = 0;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      const uint32_t *r = reinterpret_cast<const uint32_t *>(raw[gr]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[gr][2 * e] = __uint_as_float(r[e] << 16);
        v[gr][2 * e + 1] = __uint_as_float(r[e] & 0xFFFF0000u);
        top = max(top, max((r[e] << 16) & 0x7FFFFFFFu, r[e] & 0x7FFF0000u));
      }
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^up times the largest is under 2^15; rows with an infinity or NaN as they are
    const int eb = (int)(top >> 23);
    const int up = eb == 255 ? 0 : min(15 + 126 - max(eb, 1), 127);
    const float f = __int_as_float((up + 127) << 23), f16th = f * 0.0625f;
    float back = p.scale * kLog2e * 16777216.f;   // 2^24
    back = up > 100 ? back * 7.888609052210118e-31f * __int_as_float((227 - up) << 23)   // 2^-100
                    : back * __int_as_float((127 - up) << 23);
    back = finite(back);
    float sum[NG];
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      sum[gr] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const int d = 8 * (ks / 2) + 2 * (ks & 1);
        // the second pair meets codes 16 times as large
        qb[0][gr][2 * ks] = pack_f16(v[gr][d] * f, v[gr][d + 4] * f);
        qb[0][gr][2 * ks + 1] = pack_f16(v[gr][d + 1] * f16th, v[gr][d + 5] * f16th);
        const float2 a = unpack_f16(qb[0][gr][2 * ks]), b = unpack_f16(qb[0][gr][2 * ks + 1]);
        sum[gr] += (a.x + a.y) + 16.f * (b.x + b.y);
      }
      sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
      sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 2);
      sum[gr] *= 5.9604644775390625e-08f;   // 2^-24, as the products of codes
    }
    if constexpr (NT > 1) {
      if (warp == 0) {
#pragma unroll
        for (int gr = 0; gr < NG; ++gr)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            jn.q[nt][gr][i][lane] =
                make_uint4(qb[0][gr][4 * i], qb[0][gr][4 * i + 1], qb[0][gr][4 * i + 2], qb[0][gr][4 * i + 3]);
      }
    }
    // from column g's lanes to those of the accumulators' columns 2 t4, 2 t4 + 1
#pragma unroll
    for (int gr = 0; gr < NG; ++gr)
      qsum[nt][gr] =
          make_float2(__shfl_sync(0xffffffffu, sum[gr], 8 * t4), __shfl_sync(0xffffffffu, sum[gr], 8 * t4 + 4));
    cs[nt] = make_float2(__shfl_sync(0xffffffffu, back, 8 * t4), __shfl_sync(0xffffffffu, back, 8 * t4 + 4));
  }
  if constexpr (NT > 1) __syncthreads();
  int all_lo = 0, all_hi = sq.len;   // the tokens that every column sees
  if (p.causal) all_hi = max(0, sq.len - sq.nq + 1);
  if (p.window) all_lo = max(0, sq.len - p.window);

  float2 nm[NT], l[NT];   // less the running maxima, whole numbers; the sums
  float2 low[NG][NT];     // sums of w lo
  float2 up[NG][NT];      // powers of two: w step enters the product times this
  float o[MT][NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    nm[nt] = both(-kNoScore), l[nt] = both(0.f);
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) low[gr][nt] = both(0.f), up[gr][nt] = both(pow2(kMostUp));
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][nt][c] = 0.f;
  }
  const float cap_log2 = p.softcap * kLog2e, two_by_cap = finite(2.f / p.softcap);

  for (int it = 0; it < n_mine; ++it) {
    copy_wait<NS - 1>();
    __syncwarp();
    uint8_t *sl = ring + (it % NS) * SB;
    const int tok = (part.first + warp + it * W) * kTile;
    const uint32_t hole = holes >> ((it % NS) * 2) & 3u;
    {
      // A token whose V holds a NaN: its K becomes NaN, its V zeros, so that only
      // the rows that see it know.
      uint32_t *vs = reinterpret_cast<uint32_t *>(sl + Slot<D>::kVs) + lane * NG;
      bool bad = false;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) bad |= (vs[gr] & 0x7FFFu) > 0x7C00u;
      if (__any_sync(0xffffffffu, bad)) {
        if (bad) {
          uint32_t *ks = reinterpret_cast<uint32_t *>(sl + Slot<D>::kKs) + lane * NG;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) vs[gr] = 0u, ks[gr] = 0x7FFF7FFFu;
        }
        __syncwarp();
      }
    }
    float2 s[2][NT][2];
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      uint32_t bq[NT][8];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (NT == 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) bq[nt][i] = qb[0][gr][i];
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 u = jn.q[nt][gr][i][lane];
            bq[nt][4 * i] = u.x, bq[nt][4 * i + 1] = u.y, bq[nt][4 * i + 2] = u.z, bq[nt][4 * i + 3] = u.w;
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        // rows g and g + 8 of the S tile: 8 bytes of the group each
        uint32_t pr[2][2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t row = 16 * mt + 8 * r + g;
          const uint32_t pc = D == 128 ? (2 * gr + (t4 >> 1)) ^ (row & 2) : (t4 >> 1);
          const uint2 w = *reinterpret_cast<const uint2 *>(sl + Slot<D>::kK + row * (D / 2) + pc * 16 + (t4 & 1) * 8);
          four_pairs(w.x, pr[r][0]);
          four_pairs(w.y, pr[r][1]);
        }
        float acc[NT][4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t a[4] = {pr[0][ks / 2][2 * (ks & 1)], pr[1][ks / 2][2 * (ks & 1)],
                                 pr[0][ks / 2][2 * (ks & 1) + 1], pr[1][ks / 2][2 * (ks & 1) + 1]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (ks == 0) mma_f16_first(acc[nt], a, bq[nt][0], bq[nt][1]);
            else mma_f16(acc[nt], a, bq[nt][2 * ks], bq[nt][2 * ks + 1]);
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          // the token of S row 8 r + g
          const int tk = 16 * mt + 8 * r + (g >> 1) + 4 * (g & 1);
          const float2 k = unpack_f16(reinterpret_cast<const uint32_t *>(sl + Slot<D>::kKs)[tk * NG + gr]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 a = make_float2(acc[nt][2 * r], acc[nt][2 * r + 1]);
            const float2 x = gr ? fma_2(both(k.y), qsum[nt][gr], s[mt][nt][r]) : mul_2(both(k.y), qsum[nt][gr]);
            s[mt][nt][r] = fma_2(both(k.x), a, x);
          }
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) s[mt][nt][r] = mul_2(s[mt][nt][r], cs[nt]);
    if (p.softcap > 0.f) {
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i) {
        float2 &x = s[i / (2 * NT)][i / 2 % NT][i & 1];
        x = capped_2(x, two_by_cap, cap_log2);
      }
    }
    if (tok < all_lo || tok + kTile > all_hi || hole) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int j0 = tok + 16 * mt + 8 * r + (g >> 1) + 4 * (g & 1);
          const bool in = j0 < sq.len && !(hole >> mt & 1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int pos = sq.len - sq.nq + min(8 * nt + 2 * t4 + j, cols - 1) / p.G;
              const bool see = in && (!p.causal || j0 <= pos) && (!p.window || j0 > pos - p.window);
              if (!see) (j ? s[mt][nt][r].y : s[mt][nt][r].x) = -INFINITY;
            }
        }
    }
    // The running maxima, when some score passes theirs by 8: whole numbers, so that what
    // is kept needs no scaling for them but the factors `up` move along.
    bool over = false;
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      top[nt][0] = fmaxf(fmaxf(s[0][nt][0].x, s[0][nt][1].x), fmaxf(s[1][nt][0].x, s[1][nt][1].x));
      top[nt][1] = fmaxf(fmaxf(s[0][nt][0].y, s[0][nt][1].y), fmaxf(s[1][nt][0].y, s[1][nt][1].y));
      const float2 x = add_2(make_float2(top[nt][0], top[nt][1]), nm[nt]);
      over |= x.x > 8.f || x.y > 8.f;
    }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = top[nt][j];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          float &nmj = j ? nm[nt].y : nm[nt].x;
          const float now = fminf(nmj, -ceilf(x)), by = nmj - now;   // first time: 3e38
          const float f = ex2(-by);
          nmj = now;
          (j ? l[nt].y : l[nt].x) *= f;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            (j ? low[gr][nt].y : low[gr][nt].x) *= f;
            float &u = j ? up[gr][nt].y : up[gr][nt].x;
            const int e = exponent(u);
            const float rise = fminf(by, (float)(kMostUp - e)), held = ex2(rise - by);   // 1 but at kMostUp
            u = pow2(e + (int)rise);
#pragma unroll
            for (int i = 4 * gr; i < 4 * gr + 4; ++i) o[i][nt][j] *= held, o[i][nt][2 + j] *= held;
          }
        }
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      // Weights, their sums and those of w lo.
      float2 w[2][NT];
      uint32_t vsc[2][NG];   // V's scales of the S rows' tokens
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t *vs = reinterpret_cast<const uint32_t *>(sl + Slot<D>::kVs) +
                             (16 * mt + 8 * r + (g >> 1) + 4 * (g & 1)) * NG;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) vsc[r][gr] = vs[gr];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 x = add_2(s[mt][nt][r], nm[nt]);
          w[r][nt] = make_float2(ex2(x.x), ex2(x.y));
          l[nt] = add_2(l[nt], w[r][nt]);
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) low[gr][nt] = fma_2(w[r][nt], both(unpack_f16(vsc[r][gr]).y), low[gr][nt]);
        }
      }
      // For each group w step as float16: the B operands, before they are transposed.
      uint32_t pb[NG][NT][2];
      auto products = [&] {
        uint32_t most = 0;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int gr = 0; gr < NG; ++gr)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float2 ws = mul_2(mul_2(w[r][nt], both(unpack_f16(vsc[r][gr]).x)), up[gr][nt]);
              pb[gr][nt][r] = pack_f16(ws.x, ws.y);
              most = max2_f16(most, pb[gr][nt][r]);
            }
        return most;
      };
      // Where one reaches 2^15 (0x7800), the factors fall: the largest is then under 2^8.
      if (__any_sync(0xffffffffu, ((products() + 0x08000800u) & 0x80008000u) != 0)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int gr = 0; gr < NG; ++gr)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float x = 0.f;
#pragma unroll
              for (int r = 0; r < 2; ++r)
                x = fmaxf(x, (j ? w[r][nt].y : w[r][nt].x) * unpack_f16(vsc[r][gr]).x);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
              float &u = j ? up[gr][nt].y : up[gr][nt].x;
              const int e = exponent(u), to = min(e, 7 - exponent(x));
              const float f = ex2((float)(to - e));
              u = pow2(to);
#pragma unroll
              for (int i = 4 * gr; i < 4 * gr + 4; ++i) o[i][nt][j] *= f, o[i][nt][2 + j] *= f;
            }
        products();
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) pb[gr][nt][r] = transpose8x8(pb[gr][nt][r]);
      // V: the k-pairs are tokens t4, t4 + 4 (rows 2 t4, 2 t4 + 1) and 8 further; a lane
      // holds dimensions 8 g .. 8 g + 7 of each group.
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        uint32_t w[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t row = 16 * mt + 8 * r + t4 + 4 * e;
            const uint32_t pc = D == 128 ? (2 * gr + (g >> 2)) ^ (row & 2) : g >> 2;
            w[r][e] = *reinterpret_cast<const uint32_t *>(sl + Slot<D>::kV + row * (D / 2) + pc * 16 + (g & 3) * 4);
          }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // four dimensions: two row pairs of the MMA's A
          uint32_t c[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) four_pairs(__byte_perm(w[r][0], w[r][1], half ? 0x7632 : 0x5410), c[r]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a[4] = {c[0][2 * i], c[0][2 * i + 1], c[1][2 * i], c[1][2 * i + 1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[gr * 4 + half * 2 + i][nt], a, pb[gr][nt][0], pb[gr][nt][1]);
          }
        }
      }
    }
    __syncwarp();
    issue(it + NS, next);
    note(it + NS, next);
    next = page_pair(it + NS + 1);
  }
  copy_wait<0>();

  // ---- join the warps: column sums, a common maximum, then the outputs
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1)
      l[nt] = add_2(l[nt], xor_2(l[nt], d));
#pragma unroll
    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) low[gr][nt] = add_2(low[gr][nt], xor_2(low[gr][nt], d));
    if (g == 0) {
      jn.m[warp][8 * nt + 2 * t4] = -nm[nt].x, jn.m[warp][8 * nt + 2 * t4 + 1] = -nm[nt].y;
      jn.l[warp][8 * nt + 2 * t4] = l[nt].x, jn.l[warp][8 * nt + 2 * t4 + 1] = l[nt].y;
    }
  }
  __syncthreads();   // also: the rings are free
  constexpr int kRow = D + 4;
  float *joined = reinterpret_cast<float *>(smem);   // [warp][column][kRow]
  static_assert(W * 8 * NT * kRow * 4 <= kSmem<D>, "the joined outputs fit the rings");
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = 8 * nt + 2 * t4 + j;
      float top = jn.m[0][c];
#pragma unroll
      for (int w = 1; w < W; ++w) top = fmaxf(top, jn.m[w][c]);
      const float f = ex2(-(j ? nm[nt].y : nm[nt].x) - top);
      float *dst = joined + (warp * 8 * NT + c) * kRow + g * 8;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        // the codes' 2^-24 and 2^-20, and w step's factor
        const float f24 = f * pow2(24 - exponent(j ? up[gr][nt].y : up[gr][nt].x)), f20 = f24 * 0.0625f;
        const float lo = (j ? low[gr][nt].y : low[gr][nt].x) * f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float(&a)[4] = o[gr * 4 + 2 * h][nt], (&b)[4] = o[gr * 4 + 2 * h + 1][nt];
          *reinterpret_cast<float4 *>(dst + gr * 64 + h * 4) =
              make_float4(fmaf(a[j], f24, lo), fmaf(a[2 + j], f20, lo), fmaf(b[j], f24, lo), fmaf(b[2 + j], f20, lo));
        }
      }
    }
  __syncthreads();
  for (int u = threadIdx.x; u < cols * (D / 4); u += W * 32) {
    const int c = u / (D / 4), d = u % (D / 4) * 4;
    float top = jn.m[0][c];
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, jn.m[w][c]);
    float sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      sum += jn.l[w][c] * ex2(jn.m[w][c] - top);
      const float4 v = *reinterpret_cast<const float4 *>(joined + (w * 8 * NT + c) * kRow + d);
      y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
    }
    if (part.whole) {
      const float f = sum != 0.f ? 1.f / sum : 0.f;
      const int i = c / p.G, h = part.hk * p.G + c - i * p.G;
      *reinterpret_cast<uint2 *>(p.out + (size_t)(sq.t0 + i) * p.ldo + (size_t)h * D + d) =
          pack_out(make_float4(y.x * f, y.y * f, y.z * f, y.w * f));
    } else {
      const size_t at = (size_t)part.slot * kColumns + c;
      *reinterpret_cast<float4 *>(p.part_o + at * D + d) = y;
      if (d == 0) p.part_ml[at] = make_float2(top, sum);
    }
  }
}

// kCut: blocks take equal spans of the line; otherwise block u is (sequence, head) u.
template <int D, int NT, bool kCut, bool kOne>
__global__ void __launch_bounds__(kWarps * 32, kBlocks<NT>) kv4_few_kernel(const AttendParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Joined<NT> jn;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the joining blocks may wait beside these
  if constexpr (!kCut) {
    Segment g;
    g.s = blockIdx.x / p.b.Hkv, g.hk = blockIdx.x - g.s * p.b.Hkv;
    const SeqTiles t = tiles_of(p, attend_seq_at(p, g.s));
    if (t.n == 0) return;
    g.first = t.first, g.n = t.n, g.slot = 0, g.whole = true;
    do_segment<D, NT>(p, g, smem, jn);
  } else {
    const Line line = find_line<kOne>(p, blockIdx.x, -1);
    if (line.s < 0) return;
    const long long begin = line.cut * blockIdx.x, end = min(begin + line.cut, line.total);
    long long u = begin, start = line.start;   // start: of sequence s in the line
    for (int s = line.s; s < p.b.n_seq && u < end; ++s) {
      const SeqTiles t = tiles_of(p, attend_seq_at(p, s));
      const int span = span_of(t);
      for (int hk = span ? (int)((u - start) / span) : p.b.Hkv; hk < p.b.Hkv && u < end; ++hk) {
        const long long first = start + (long long)hk * span;   // this head's tiles: first .. first + t.n
        const int a = (int)(u - first), b = (int)min((long long)t.n, end - first);
        if (a < b) {
          const Segment g{s, hk, t.first + a, b - a, 2 * (int)blockIdx.x + (first > begin), a == 0 && b == t.n};
          do_segment<D, NT>(p, g, smem, jn);
          __syncthreads();   // the joined outputs are read before the next tiles come
        }
        u = first + span;
      }
      start += (long long)span * p.b.Hkv;
    }
  }
}

// Joins the parts of rows and query heads of one sequence, WR warps to each: a warp
// takes eight parts in one go.
constexpr int kJoinWarps = 8;
template <int D, int WR, bool kOne>
__global__ void __launch_bounds__(kJoinWarps * 32) kv4_join_kernel(const AttendParams p, int max_cols) {
  __shared__ float4 ys[kJoinWarps][D / 4];
  __shared__ float2 mls[kJoinWarps];
  constexpr int kRowsBlock = kJoinWarps / WR;
  const int per_seq = p.b.Hkv * max_cols, blocks_seq = (per_seq + kRowsBlock - 1) / kRowsBlock;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % WR;
  const int s = blockIdx.x / blocks_seq, u = (blockIdx.x - s * blocks_seq) * kRowsBlock + warp / WR;
  const AttendSeq sq = attend_seq_at(p, s);
  const int cols = sq.rows * p.G, hk = u / max_cols, c = u - hk * max_cols;
  const SeqTiles t = tiles_of(p, sq);
  int b0 = 0, b1 = 0;
  Line line{};
  long long head = 0;
  if (t.n > 0) {   // the whole block
    line = find_line<kOne>(p, 0, s);
    head = line.start + (long long)hk * span_of(t);
    b0 = (int)(head / line.cut), b1 = (int)((head + t.n - 1) / line.cut);
  }
  // Every block waits: this grid must not be over before the one it joins.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (WR == kJoinWarps && (b0 == b1 || u >= per_seq || c >= cols)) return;   // the whole block
  const bool mine = b0 < b1 && u < per_seq && c < cols;
  RowPart row;
  if (mine) {
    const float *po = after_wait(p.part_o);
    const float2 *pml = after_wait(p.part_ml);
    // Slot of block b's part: its span's first segment, or one that starts inside it.
    for (int b = b0 + part; b <= b1; b += 8 * WR)
      row.take<8, D>(po, pml, (b1 - b) / WR + 1, lane, [&](int i) {
        return (size_t)(2 * (b + i * WR) + (head > line.cut * (b + i * WR))) * kColumns + c;
      });
  }
  if constexpr (WR > 1) {
    if (lane < D / 4) ys[warp][lane] = row.y;
    if (lane == 0) mls[warp] = make_float2(row.top, row.sum);
    __syncthreads();
    if (part) return;
    float now = row.top;
#pragma unroll
    for (int w = 1; w < WR; ++w) now = fmaxf(now, mls[warp + w].x);
    row.scale(ex2(row.top - now));
#pragma unroll
    for (int w = 1; w < WR; ++w)
      row.add(mls[warp + w].y, ys[warp + w][lane % (D / 4)], ex2(mls[warp + w].x - now));
  }
  if (!mine || lane >= D / 4) return;
  const int i = c / p.G, h = hk * p.G + c - i * p.G;
  *reinterpret_cast<uint2 *>(p.out + (size_t)(sq.t0 + i) * p.ldo + (size_t)h * D + lane * 4) = row.result();
}

template <int D, int NT, bool kCut, bool kOne>
cudaError_t launch(const AttendParams &p, int grid, cudaStream_t st) {
  auto kernel = kv4_few_kernel<D, NT, kCut, kOne>;
  static DeviceOnce once;
  const cudaError_t err = once.run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D>);
  });
  if (err != cudaSuccess) return err;
  return launch_k(false, kernel, dim3(grid), dim3(kWarps * 32), kSmem<D>, st, p);
}

template <int D, int NT>
cudaError_t launch(AttendParams p, bool cut, int max_cols, cudaStream_t st) {
  if (!cut) return launch<D, NT, false, false>(p, p.b.n_seq * p.b.Hkv, st);
  p.target = kFewSms * kBlocks<NT>;
  const bool one = p.b.n_seq == 1;
  const cudaError_t err =
      one ? launch<D, NT, true, true>(p, p.target, st) : launch<D, NT, true, false>(p, p.target, st);
  if (err != cudaSuccess) return err;
  // Eight warps to a row where its parts are many (one or two heads have a good part
  // of all blocks), else one.
  const int per_seq = p.b.Hkv * max_cols;
  const bool wide = p.target >= 4 * p.b.n_seq * p.b.Hkv;
  const int blocks_seq = wide ? per_seq : (per_seq + kJoinWarps - 1) / kJoinWarps;
  auto join = one ? (wide ? kv4_join_kernel<D, kJoinWarps, true> : kv4_join_kernel<D, 1, true>)
                  : (wide ? kv4_join_kernel<D, kJoinWarps, false> : kv4_join_kernel<D, 1, false>);
  return launch_k(true, join,
                  dim3((unsigned)(p.b.n_seq * blocks_seq)), dim3(kJoinWarps * 32), 0, st, p, max_cols);
}

// Whether the line of tiles is cut: not for more sequences than a block can look
// over at its start, nor where no sequence is longer than a span's least.
bool is_cut(const AttendParams &p) {
  return p.b.n_seq <= kPlanSeqs && ((long long)p.b.max_pages << p.b.log_page) > kMinTiles * kTile;
}

}  // namespace

// Slots of partial results: two for each block.
size_t few_slots(const AttendParams &p) { return is_cut(p) ? 2 * kFewSms * kBlocks<1> : 0; }

cudaError_t launch_few(const AttendParams &p, int D, cudaStream_t st) {
  // Columns that some sequence may have.
  const long long rows = p.b.q_off ? (p.max_q ? std::min(p.max_q, p.b.T) : p.b.T) : 1;
  const int max_cols = (int)std::min<long long>(kColumns / p.G * p.G, rows * p.G);
  const bool cut = is_cut(p);
  if (D == 128)
    return max_cols > 8 ? launch<128, 2>(p, cut, max_cols, st) : launch<128, 1>(p, cut, max_cols, st);
  return max_cols > 8 ? launch<64, 2>(p, cut, max_cols, st) : launch<64, 1>(p, cut, max_cols, st);
}

}  // namespace moe
