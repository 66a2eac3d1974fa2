// kv4_few.cu -- attention of a few rows a sequence over the 4-bit cache: decoded
// tokens, and drafted ones, up to 16 columns (rows times query heads of a KV
// head).
//
//   S^T[token][column] = K . q^T,  O^T[dim][column] = V^T . P^T
//
// on warp-level MMAs (m16n8k16, float16): 16 tokens, then 16 dimensions, are the
// rows, columns the 8-wide side, so 8 query heads waste nothing.  Bound by
// reading the cache, 9/16 bytes an element: the design keeps instructions per
// code low and loads in flight many.
//
//   K: a lane's 16 codes of a token and group are 4 k-steps of the MMA as they lie
//      (which dimension is which k is free as long as q agrees).  They enter as
//      exact integers c - 8, one accumulator for each group, and
//      s = sum_g step_g acc_g + (lo_g + 8 step_g) sum(q of g): no rounding of K.
//   q: float16 after a power of two per column that brings its largest just under
//      2^15: exact to 2^-29 of that.
//   P: the accumulator's layout, transposed by movmatrix, is the B operand.
//   V: lo + step c in float16 (pairs of tokens of one dimension, so step and lo are
//      pairs as they come), rounded once: 2^-12 of the value.
//
// Each warp streams its own tiles of 32 tokens through a private ring in shared
// memory by cp.async (no barrier, no waiting but its own), with a running
// maximum that moves only when a score passes it by 2^8 (weights up to 256 are
// float16 as well as those up to 1), so most tiles exchange nothing.  The block's
// warps join at the end.  A batch is cut into parts of about equal length over
// the tokens of all its sequences; a second kernel joins the parts of sequences
// that have several.
#include <algorithm>

#include "kv4.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kTile = 32;                   // tokens of a ring slot
constexpr int kMinTiles = kWarps;           // tiles of a part, at least
constexpr int kPlanSeqs = 1024;             // sequences of a batch that is cut into parts
constexpr int kColumns = kFewColumns;

template <int D>
struct Slot {
  static constexpr int kK = 0, kV = kTile * D / 2, kKs = kTile * D, kVs = kKs + kTile * D / 16;
  static constexpr int kBytes = kVs + kTile * D / 16;
};
template <int D>
constexpr int kRing = D == 128 ? 3 : 5;     // slots of a warp
template <int D>
constexpr int kSmem = kWarps * kRing<D> * Slot<D>::kBytes;

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// (w & mask) | magic: 1024 + c from bits 0-3 of each half, 64 + c from bits 4-7.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  uint32_t d;
  asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  uint32_t d;
  asm("lop3.b32 %0, %1, 0x00F000F0, 0x54005400, 0xEA;" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Four pairs of codes of w (nibbles i and i + 4 of it: a pair's halves), less `less`.
__device__ __forceinline__ void four_pairs(uint32_t w, uint32_t lo_bias, uint32_t hi_bias, uint32_t (&o)[4]) {
  const uint32_t w8 = w >> 8;
  o[0] = sub2(codes_lo(w), lo_bias);
  o[1] = sub2(codes_hi(w), hi_bias);
  o[2] = sub2(codes_lo(w8), lo_bias);
  o[3] = sub2(codes_hi(w8), hi_bias);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// ------------------------------------------------------------------ plan --

// A part of the batch: tiles first .. first + n - 1 of sequence s.
struct Part {
  int s, hk, part, parts, first, n, slot;   // slot: of the sequence's first part and KV head 0
};

struct SeqTiles {
  int first, n;   // tiles that any row of the sequence sees; n = 0 with first < 0: none of this kernel's
};

__device__ __forceinline__ SeqTiles tiles_of(const AttendParams &p, const AttendSeq &q) {
  if (q.rows < 1 || q.rows * p.G > kColumns) return SeqTiles{-1, 0};
  int lo = 0;
  if (p.window) lo = max(0, q.len - q.nq - p.window + 1) / kTile;
  return SeqTiles{lo, (q.len + kTile - 1) / kTile - lo};
}

// Exclusive prefix of v over the block's threads, and the total.
__device__ __forceinline__ int2 block_scan(int2 v, int2 *warp_sums, int2 &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int2 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) x.x += a, x.y += b;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int2 before = make_int2(x.x - v.x, x.y - v.y);
  total = make_int2(0, 0);
  for (int w = 0; w < nw; ++w) {
    const int2 s = warp_sums[w];
    if (w < warp) before.x += s.x, before.y += s.y;
    total.x += s.x, total.y += s.y;
  }
  return before;
}

// Which part `item` is (seq < 0), or the parts of sequence `seq`: false if there
// is none.  Every block works it out from the lengths: cutting all sequences into
// parts of at most `cut` tiles, which makes at least about `target` parts of a
// large batch.  Only sequences of several parts have slots, twice `target` at
// most (n / cut > 1 rounds up to less than twice itself).
__device__ bool find_part(const AttendParams &p, int item, int seq, Part &out) {
  __shared__ int2 sums[32];
  __shared__ Part found;
  const int Hkv = p.b.Hkv;
  if (p.b.n_seq > kPlanSeqs) {   // whole sequences
    const int s = seq >= 0 ? seq : item / Hkv;
    if (s >= p.b.n_seq) return false;
    const SeqTiles t = tiles_of(p, attend_seq_at(p, s));
    if (t.first < 0) return false;
    out = Part{s, item - s * Hkv, 0, 1, t.first, t.n, 0};
    return true;
  }
  constexpr int kMost = kPlanSeqs / 128;   // sequences of a thread, 128 threads at least
  const int per = (p.b.n_seq + blockDim.x - 1) / blockDim.x;
  SeqTiles t[kMost];
  long long mine = 0;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int s = threadIdx.x * per + i;
    t[i] = SeqTiles{-1, 0};
    if (i < per && s < p.b.n_seq) t[i] = tiles_of(p, attend_seq_at(p, s));
    mine += t[i].n;
  }
  // 1024 sequences of 2^30 / 32 tiles and 1024 KV heads need 45 bits: counted in
  // units that leave 31, rounded up.
  const int unit = (int)(mine >> 20), rest = (int)(mine & 0xFFFFF);
  int2 total;
  block_scan(make_int2(unit, rest), sums, total);
  const long long tiles = ((long long)total.x << 20) + total.y;
  const long long want = (tiles * Hkv + p.target - 1) / p.target;
  const int cut = (int)max(want, (long long)kMinTiles);
  int2 n = make_int2(0, 0);
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    if (t[i].first < 0) continue;
    const int parts = max(1, (t[i].n + cut - 1) / cut);
    n.x += parts, n.y += parts > 1 ? parts : 0;
  }
  int2 all;
  int2 at = block_scan(n, sums, all);
  if (threadIdx.x == 0) found.s = -1;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    if (t[i].first < 0) continue;
    const int s = threadIdx.x * per + i;
    const int parts = max(1, (t[i].n + cut - 1) / cut);
    if (seq >= 0 ? s == seq : item / Hkv >= at.x && item / Hkv < at.x + parts) {
      // Parts of a sequence are nearly equal: the first n % parts have a tile more.
      const int part = seq >= 0 ? 0 : item / Hkv - at.x, each = t[i].n / parts, more = t[i].n % parts;
      found = Part{s, item % Hkv, part, parts, t[i].first + part * each + min(part, more),
                   each + (part < more), at.y * Hkv};
    }
    at.x += parts, at.y += parts > 1 ? parts : 0;
  }
  __syncthreads();
  out = found;
  return out.s >= 0;
}

// ---------------------------------------------------------------- kernel --

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, 2) kv4_few_kernel(const AttendParams p) {
  constexpr int NG = D / kKvGroup, MT = D / 16, SB = Slot<D>::kBytes, NS = kRing<D>;
  constexpr int kPieces = D / 32;            // 16-byte pieces of a token's codes
  constexpr int VW = D / 64;                 // words of V codes a lane holds of a token
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float warp_m[kWarps][8 * NT], warp_l[kWarps][8 * NT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the joining blocks may wait beside these
  Part part;
  if (!find_part(p, blockIdx.x, -1, part)) return;
  const AttendSeq sq = attend_seq_at(p, part.s);
  const int cols = sq.rows * p.G, lp = p.b.log_page;

  // ---- the ring: this warp's tiles are first + warp, + kWarps, ...
  const int n_mine = part.n > warp ? (part.n - warp + kWarps - 1) / kWarps : 0;
  uint8_t *ring = smem + warp * (NS * SB);
  const uint32_t ring_s = smem_addr(ring);
  const int32_t *pages = p.b.pages + (size_t)part.s * p.b.max_pages;
  const uint8_t *head = p.cache + (size_t)part.hk * KvBlock<D>::bytes(lp);
  const size_t page_bytes = KvBlock<D>::bytes(lp) * p.b.Hkv;
  // Pages of the halves (16 tokens) of the warp's i-th tile; -1 also past the end.
  auto page_pair = [&](int i) {
    int2 r = make_int2(-1, -1);
    if (i >= n_mine) return r;
    const int tok = (part.first + warp + i * kWarps) * kTile;
    auto get = [&](int token) {
      if (token >= sq.len) return -1;
      const int id = __ldg(pages + (token >> lp));
      return (unsigned)id < (unsigned)p.b.n_pages ? id : -1;
    };
    r.x = get(tok);
    r.y = lp > 4 ? (tok + 16 < sq.len ? r.x : -1) : get(tok + 16);
    return r;
  };
  auto issue = [&](int i, int2 pg) {
    if (i < n_mine) {
      const int tok = (part.first + warp + i * kWarps) * kTile, mask = (1 << lp) - 1;
      const uint32_t dst = ring_s + (i % NS) * SB;
      const uint8_t *blk[2];
      int slot[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int id = h ? pg.y : pg.x;
        blk[h] = head + (size_t)max(id, 0) * page_bytes;
        slot[h] = (tok + 16 * h) & mask;
      }
      // Codes: whole rows where there is a page (rows past the length hold some
      // codes or other, and every code is a finite number); K rows in the order
      // of the S rows, and 16-byte pieces 2 and 3 in place of 0 and 1 in every
      // other pair of rows, for loads without bank conflicts.
      constexpr int kRows = 32 / kPieces;      // tokens of one round of copies
#pragma unroll
      for (int c = 0; c < kTile / kRows; ++c) {
        const int h = c * kRows / 16;
        const int tk = c * kRows % 16 + lane / kPieces, pc = lane % kPieces;   // token in the half, piece
        const int ok = (h ? pg.y : pg.x) >= 0 ? 16 : 0;
        const uint32_t kr = 16 * h + (tk & 8) + 2 * (tk & 3) + ((tk >> 2) & 1);   // S row of the token
        const uint32_t vr = 16 * h + tk;
        const uint32_t kp = D == 128 ? pc ^ (kr & 2) : pc, vp = D == 128 ? pc ^ (vr & 2) : pc;
        copy16(dst + Slot<D>::kK + kr * (D / 2) + kp * 16,
               blk[h] + KvBlock<D>::codes(lp, 0, slot[h] + tk) + pc * 16, ok);
        copy16(dst + Slot<D>::kV + vr * (D / 2) + vp * 16,
               blk[h] + KvBlock<D>::codes(lp, 1, slot[h] + tk) + pc * 16, ok);
      }
      // Scales: zeros past the length, whatever lies there.
      constexpr int kTok = 16 / (NG * 4);      // tokens of a piece
      constexpr int kSp = kTile / kTok;        // pieces of K's, and of V's: 16 or 8
      if (lane < 2 * kSp) {
        const int which = lane >= kSp, pc = lane - which * kSp, tk = pc * kTok, h = tk / 16;
        const int left = (sq.len - tok - tk) * (NG * 4);
        copy16(dst + (which ? Slot<D>::kVs : Slot<D>::kKs) + pc * 16,
               (h ? blk[1] : blk[0]) + KvBlock<D>::scales(lp, which, (h ? slot[1] : slot[0]) + (tk & 15)),
               (h ? pg.y : pg.x) >= 0 ? min(16, max(0, left)) : 0);
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
  uint32_t qb[NT][NG][8];
  float qsum[NT][NG][2], cs[NT][2];   // of the columns 8 nt + 2 t4, + 1 of the accumulators
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
    const float f = __int_as_float((up + 127) << 23);
    float back = p.scale * kLog2e * (p.softcap > 0.f ? 2.f / p.softcap : 1.f);
    back = up > 100 ? back * 7.888609052210118e-31f * __int_as_float((227 - up) << 23)   // 2^-100
                    : back * __int_as_float((127 - up) << 23);
    float sum[NG];
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      sum[gr] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const int d = 8 * (ks / 2) + 2 * (ks & 1);
        qb[nt][gr][2 * ks] = pack_f16(v[gr][d] * f, v[gr][d + 4] * f);
        qb[nt][gr][2 * ks + 1] = pack_f16(v[gr][d + 1] * f, v[gr][d + 5] * f);
        const float2 a = unpack_f16(qb[nt][gr][2 * ks]), b = unpack_f16(qb[nt][gr][2 * ks + 1]);
        sum[gr] += (a.x + a.y) + (b.x + b.y);
      }
      sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
      sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 2);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int src = (2 * t4 + j) * 4;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) qsum[nt][gr][j] = __shfl_sync(0xffffffffu, sum[gr], src);
      cs[nt][j] = __shfl_sync(0xffffffffu, back, src);
    }
  }
  // Position of each accumulator column's row; the tokens that every column sees.
  int pos[NT][2];
  int all_lo = 0, all_hi = sq.len;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) pos[nt][j] = sq.len - sq.nq + min(8 * nt + 2 * t4 + j, cols - 1) / p.G;
  if (p.causal) all_hi = max(0, sq.len - sq.nq + 1);
  if (p.window) all_lo = max(0, sq.len - p.window);

  float m[NT][2], l[NT][2], o[MT][NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) m[nt][j] = kNoScore, l[nt][j] = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][nt][c] = 0.f;
  }
  const float cap_log2 = p.softcap * kLog2e;
  const uint32_t c1032 = 0x64086408u, c72 = 0x54805480u;   // less 1024 + 8 and 64 + 8
  const uint32_t c1024 = 0x64006400u, c64 = 0x54005400u;

  for (int it = 0; it < n_mine; ++it) {
    copy_wait<NS - 1>();
    __syncwarp();
    uint8_t *sl = ring + (it % NS) * SB;
    const int tok = (part.first + warp + it * kWarps) * kTile;
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
    float s[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      float acc[NG][NT][4];
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[gr][nt][c] = 0.f;
        // rows g and g + 8 of the S tile: 8 bytes of the group each
        uint32_t pr[2][2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t row = 16 * mt + 8 * r + g;
          const uint32_t pc = D == 128 ? (2 * gr + (t4 >> 1)) ^ (row & 2) : (t4 >> 1);
          const uint2 w = *reinterpret_cast<const uint2 *>(sl + Slot<D>::kK + row * (D / 2) + pc * 16 + (t4 & 1) * 8);
          four_pairs(w.x, c1032, c72, pr[r][0]);
          four_pairs(w.y, c1032, c72, pr[r][1]);
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t a[4] = {pr[0][ks / 2][2 * (ks & 1)], pr[1][ks / 2][2 * (ks & 1)],
                                 pr[0][ks / 2][2 * (ks & 1) + 1], pr[1][ks / 2][2 * (ks & 1) + 1]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(acc[gr][nt], a, qb[nt][gr][2 * ks], qb[nt][gr][2 * ks + 1]);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        // the token of S row 8 r + g
        const int tk = 16 * mt + 8 * r + (g >> 1) + 4 * (g & 1);
        const uint32_t *ks = reinterpret_cast<const uint32_t *>(sl + Slot<D>::kKs) + tk * NG;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const float2 k = unpack_f16(ks[gr]);
          const float mid = fmaf(8.f, k.x, k.y);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float x = fmaf(k.x, acc[gr][nt][2 * r + j], mid * qsum[nt][gr][j]);
              s[mt][nt][2 * r + j] = gr ? s[mt][nt][2 * r + j] + x : x;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) s[mt][nt][2 * r + j] *= cs[nt][j];
      }
    }
    if (p.softcap > 0.f) {
#pragma unroll
      for (int i = 0; i < 2 * NT * 4; ++i) (&s[0][0][0])[i] = capped((&s[0][0][0])[i], cap_log2);
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
              const bool see = in && (!p.causal || j0 <= pos[nt][j]) && (!p.window || j0 > pos[nt][j] - p.window);
              if (!see) s[mt][nt][2 * r + j] = -INFINITY;
            }
        }
    }
    // The running maximum, when some score passes it by 8.
    bool over = false;
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        top[nt][j] = fmaxf(fmaxf(s[0][nt][j], s[0][nt][2 + j]), fmaxf(s[1][nt][j], s[1][nt][2 + j]));
        over |= top[nt][j] > m[nt][j] + 8.f;
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = top[nt][j];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          x = fmaxf(x, m[nt][j]);
          const float f = ex2(m[nt][j] - x);
          m[nt][j] = x;
          l[nt][j] *= f;
#pragma unroll
          for (int i = 0; i < MT; ++i) o[i][nt][j] *= f, o[i][nt][2 + j] *= f;
        }
    }
    // Weights, and their B operands for the two blocks of 16 tokens.
    uint32_t pb[2][NT][2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float a = ex2(s[mt][nt][2 * r] - m[nt][0]), b = ex2(s[mt][nt][2 * r + 1] - m[nt][1]);
          l[nt][0] += a, l[nt][1] += b;
          pb[mt][nt][r] = transpose8x8(pack_f16(a, b));
        }
    // V: tokens t4, t4 + 4 (k-pair of rows 2 t4, 2 t4 + 1), + 8 and + 12 of each block;
    // dimensions VW * 8 g .. of each.
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t st[2], lo[2], w[2][2][VW];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t sc[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t row = 16 * mt + 8 * r + t4 + 4 * e;
          sc[e] = *(reinterpret_cast<const uint32_t *>(sl + Slot<D>::kVs) + row * NG + (NG == 2 ? g >> 2 : 0));
          if constexpr (D == 128) {
            const uint32_t pc = (g >> 1) ^ (row & 2);
            const uint2 u = *reinterpret_cast<const uint2 *>(sl + Slot<D>::kV + row * 64 + pc * 16 + (g & 1) * 8);
            w[r][e][0] = u.x, w[r][e][VW - 1] = u.y;
          } else {
            w[r][e][0] = *reinterpret_cast<const uint32_t *>(sl + Slot<D>::kV + row * 32 + g * 4);
          }
        }
        st[r] = __byte_perm(sc[0], sc[1], 0x5410);
        lo[r] = __byte_perm(sc[0], sc[1], 0x7632);
      }
#pragma unroll
      for (int v = 0; v < VW; ++v)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // four dimensions: two row pairs of the MMA's A
          uint32_t c[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            four_pairs(__byte_perm(w[r][0][v], w[r][1][v], half ? 0x7632 : 0x5410), c1024, c64, c[r]);
#pragma unroll
            for (int e = 0; e < 4; ++e) c[r][e] = fma2(c[r][e], st[r], lo[r]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a[4] = {c[0][2 * i], c[0][2 * i + 1], c[1][2 * i], c[1][2 * i + 1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[v * 4 + half * 2 + i][nt], a, pb[mt][nt][0], pb[mt][nt][1]);
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
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], d);
      if (g == 0) {
        warp_m[warp][8 * nt + 2 * t4 + j] = m[nt][j];
        warp_l[warp][8 * nt + 2 * t4 + j] = l[nt][j];
      }
    }
  __syncthreads();   // also: the rings are free
  constexpr int kRow = D + 4;
  float *joined = reinterpret_cast<float *>(smem);   // [warp][column][kRow]
  static_assert(kWarps * 8 * NT * kRow * 4 <= kSmem<D>, "the joined outputs fit the rings");
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = 8 * nt + 2 * t4 + j;
      float top = warp_m[0][c];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, warp_m[w][c]);
      const float f = ex2(m[nt][j] - top);
      float *dst = joined + (warp * 8 * NT + c) * kRow + g * (D / 8);
#pragma unroll
      for (int i = 0; i < MT; i += 2)
        *reinterpret_cast<float4 *>(dst + 2 * i) =
            make_float4(o[i][nt][j] * f, o[i][nt][2 + j] * f, o[i + 1][nt][j] * f, o[i + 1][nt][2 + j] * f);
    }
  __syncthreads();
  for (int u = threadIdx.x; u < cols * (D / 4); u += kWarps * 32) {
    const int c = u / (D / 4), d = u % (D / 4) * 4;
    float top = warp_m[0][c];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, warp_m[w][c]);
    float sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sum += warp_l[w][c] * ex2(warp_m[w][c] - top);
      const float4 v = *reinterpret_cast<const float4 *>(joined + (w * 8 * NT + c) * kRow + d);
      y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
    }
    if (part.parts == 1) {
      const float f = sum != 0.f ? 1.f / sum : 0.f;
      const int i = c / p.G, h = part.hk * p.G + c - i * p.G;
      *reinterpret_cast<uint2 *>(p.out + (size_t)(sq.t0 + i) * p.ldo + (size_t)h * D + d) =
          pack_out(make_float4(y.x * f, y.y * f, y.z * f, y.w * f));
    } else {
      const size_t at = (size_t)(part.slot + part.part * p.b.Hkv + part.hk) * kColumns + c;
      *reinterpret_cast<float4 *>(p.part_o + at * D + d) = y;
      if (d == 0) p.part_ml[at] = make_float2(top, sum);
    }
  }
}

// One block per sequence, row and query head: joins its parts, four at a time in
// four warps.
template <int D>
__global__ void __launch_bounds__(128) kv4_join_kernel(const AttendParams p, int max_cols) {
  __shared__ float4 ys[4][D / 4];
  __shared__ float2 mls[4];
  const int per_seq = p.b.Hkv * max_cols;
  const int s = blockIdx.x / per_seq, u = blockIdx.x - s * per_seq;
  const AttendSeq sq = attend_seq_at(p, s);
  const int cols = sq.rows * p.G, hk = u / max_cols, c = u - hk * max_cols;
  if (cols > kColumns || c >= cols) return;
  Part part;
  if (!find_part(p, 0, s, part) || part.parts == 1) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float *po = after_wait(p.part_o);
  const float2 *pml = after_wait(p.part_ml);
  const size_t first = (size_t)(part.slot + hk) * kColumns + c, step = (size_t)p.b.Hkv * kColumns;
  float top = kNoScore;
  for (int i = lane; i < part.parts; i += 32) top = fmaxf(top, __ldcg(pml + first + i * step).x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  float sum = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = warp; i < part.parts; i += 4) {
    const float2 ml = __ldcg(pml + first + i * step);
    const float f = ex2(ml.x - top);
    sum += ml.y * f;
    if (lane < D / 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(po + (first + i * step) * D) + lane);
      y.x += v.x * f, y.y += v.y * f, y.z += v.z * f, y.w += v.w * f;
    }
  }
  if (lane < D / 4) ys[warp][lane] = y;
  if (lane == 0) mls[warp].x = sum;
  __syncthreads();
  if (warp || lane >= D / 4) return;
  sum = (mls[0].x + mls[1].x) + (mls[2].x + mls[3].x);
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    const float4 v = ys[w][lane];
    y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
  }
  const float f = sum != 0.f ? 1.f / sum : 0.f;
  const int i = c / p.G, h = hk * p.G + c - i * p.G;
  *reinterpret_cast<uint2 *>(p.out + (size_t)(sq.t0 + i) * p.ldo + (size_t)h * D + lane * 4) =
      pack_out(make_float4(y.x * f, y.y * f, y.z * f, y.w * f));
}

template <int D, int NT>
cudaError_t launch(const AttendParams &p, int grid, cudaStream_t st) {
  auto kernel = kv4_few_kernel<D, NT>;
  static DeviceOnce once;
  const cudaError_t err = once.run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D>);
  });
  if (err != cudaSuccess) return err;
  return launch_k(false, kernel, dim3(grid), dim3(kWarps * 32), kSmem<D>, st, p);
}

}  // namespace

int few_target(int sms) { return sms * 4; }

// Slots of partial results: none where no sequence can have two parts.
size_t few_slots(const AttendParams &p) {
  if (p.b.n_seq > kPlanSeqs || ((long long)p.b.max_pages << p.b.log_page) <= kMinTiles * kTile) return 0;
  return 2 * (size_t)p.target + 2 * p.b.Hkv;
}

cudaError_t launch_few(const AttendParams &p, int D, cudaStream_t st) {
  // Columns that some sequence may have.
  const long long rows = p.b.q_off ? (p.max_q ? std::min(p.max_q, p.b.T) : p.b.T) : 1;
  const int max_cols = (int)std::min<long long>(kColumns / p.G * p.G, rows * p.G);
  const bool two = max_cols > 8;
  const size_t slots = few_slots(p);
  const long long pairs = (long long)p.b.n_seq * p.b.Hkv;
  const int grid = (int)(pairs + (slots ? p.target : 0));
  cudaError_t err;
  if (D == 128) err = two ? launch<128, 2>(p, grid, st) : launch<128, 1>(p, grid, st);
  else err = two ? launch<64, 2>(p, grid, st) : launch<64, 1>(p, grid, st);
  if (err != cudaSuccess || !slots) return err;
  return launch_k(true, D == 128 ? kv4_join_kernel<128> : kv4_join_kernel<64>,
                  dim3((unsigned)(p.b.n_seq * p.b.Hkv * max_cols)), dim3(128), 0, st, p, max_cols);
}

}  // namespace moe
