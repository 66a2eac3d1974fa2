// kv4_many.cu -- attention of many rows a sequence over the 4-bit cache: prompts,
// drafted tokens of many heads, on the 5th-gen tensor cores.
//
// A block takes 256 rows (tokens times query heads of one KV head, which read the
// same keys) in two tiles of 128, and walks the keys that they see, decoded 128 at a
// time, in steps of 64:
//
//   S_i = Q_i . K^T (tcgen05, both operands in shared memory), softmax, and
//   O_i += P_i . V  (P_i float16 in tensor memory over S_i's columns)
//
//   warps 0-3, 4-7   the softmax of tile 0 and 1: a thread owns a row, so maxima
//                    and sums need no exchange
//   warps 8-11       turn codes into lo + step c in float16, 128-byte swizzled, once
//                    for 256 rows; the next tile's codes are on the way meanwhile
//   warps 12, 13     issue the MMAs of tile 0 and 1: scores run two steps ahead of
//                    the softmax, in two buffers of tensor memory
//
// 8192 tokens of 32 query and 8 KV heads, causal: 429 us, 1282 TFLOP/s of what
// counts (0.67 of a large matrix product's rate); the tensor pipe is busy 55 % of the
// clocks, the schedulers 54 %.  No single part bounds it.  In an earlier form (441 us)
// the codes' role was at work for 3760 of the 3836 clocks of a tile of 128 keys, beside
// the softmax on the same schedulers and with shared memory's pipe 75 to 90 % busy; it took
// 404 us without the exponentials, 419 without the masks, 340 without the softmax's
// arithmetic and the decoded tiles' stores.  Slower: more warps for the codes (481 us
// against 450) or for the softmax (516 against 441), codes shared by two blocks of a
// cluster (824 against 441: remote stores), two tiles of codes in flight in registers
// (625 against 450: spills), both softmax groups on one tile of rows where there is only
// one (57.9 against 56.5 for 4 rows of 96/8 heads in each of 4 sequences of 16384),
// blocks that work through several tiles of rows, the next one's decoding beside the last
// one's end (447 against 426).
//
// The running maximum moves only when a score passes it by 8: weights up to 2^8 are
// float16 as well as those up to 1, and the outputs in tensor memory need scaling
// rarely.  Rounded to float16 (2^-11 at most): keys, values and weights; queries enter
// after a power of two per row that brings the largest just under 2^15.
//
// The 8 dimensions of a word of codes lie in the order 0 4 1 5 2 6 3 7 (pairs of
// nibbles i and i + 4 decode together), in Q as in K; the output puts V's back.
//
// Where a call has fewer blocks than SMs the keys are cut into parts, whose results
// a second kernel joins: as many as fit the SMs, counting a place too many for each
// sequence, also for those that kv4_few.cu takes, so batches of many short sequences
// beside a long one are not cut.  (One line of all key tiles cut into equal spans, as for few
// rows, was slower: 512 rows of 32/8 heads over 16384 keys 163 us against 125.)
#include <algorithm>

#include "kv4.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;      // rows of a tile
constexpr int kKeys = 128;      // keys of a tile
constexpr int kSub = 64;        // keys of a softmax step
constexpr int kBlockRows = 2 * kRows;
constexpr int kThreads = 512;
constexpr int kMinPart = 4;     // key tiles of a part, at least
constexpr int kSms = 152;

// Capped scores.  cap - 2 cap / (1 + e^(2 x / cap)) is off by up to cap 2^-22: 2^-16 at
// the most for a near cap, where the keys' rounding to float16 costs a score far more.
// Past it capped_2 (kv4.cuh), off by 2^-20 of the score, however large the cap (a prompt
// of 4096, 32/8 heads: 248 us against 194 us for a near cap, 131 without one).
enum Cap { kNoCap, kNearCap, kFarCap };
constexpr float kMostNear = 64.f;

// Registers a thread: 512 x 128 at launch, then by warpgroup; the shares add up to
// what the block was launched with.
constexpr int kSoftmaxRegs = 176, kDecodeRegs = 112, kIssueRegs = 48;
static_assert(2 * kSoftmaxRegs + kDecodeRegs + kIssueRegs == 4 * 128 && kSoftmaxRegs >= 128 && kDecodeRegs <= 128 &&
                  kIssueRegs <= 128,
              "the block's registers; inc only up, dec only down");

template <int D>
struct Smem {
  static constexpr int kQ = kRows * D * 2, kK = kKeys * D * 2;   // one tile of Q; of K or V
  static constexpr int kBytes = 2 * kQ + 4 * kK;                 // two stages of K and V
};

// What a block works out: some key tiles of a tile of rows.
struct Job {
  int s, hk;          // sequence, KV head
  int q0, nq, len;    // the sequence's first row of q, its rows, its tokens
  int row0, rows;     // the first row (token x head of the KV head), how many
  int t0, n, end;     // key tiles t0 .. t0 + n - 1; the last key's successor, of all parts
  int parts;
  // Steps of 64 keys.
  __device__ __forceinline__ int steps() const { return min(n * 2, max(0, (end - t0 * kKeys + kSub - 1) / kSub)); }
};

struct Bars {
  uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2][2], p_full[2][2], o_done[2][2];   // [tile of rows][step % 2]
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort;
  uint8_t holes[4][4];   // [tile % 4][decoding warp]: two bits, 16 tokens each without a page
};

__device__ __forceinline__ bool wait_loop(uint64_t *bar, uint32_t parity, int *abort, int32_t *status,
                                          unsigned long long limit_ns) {
  const unsigned long long t0 = globaltimer();
  for (;;) {
    if (limit_ns && mbar_try_wait_sleep(bar, parity)) return true;
    if (*reinterpret_cast<volatile int *>(abort)) return false;
    if (globaltimer() - t0 >= limit_ns) {
      atomicExch(abort, 1);
      atomicExch(status, kStatusTimeout);
      return false;
    }
  }
}
// One thread's wait (the issuer): a limit of 0 gives up where the phase is not
// complete when first tested.
__device__ __forceinline__ bool wait_one(uint64_t *bar, uint32_t parity, int *abort, int32_t *status,
                                         unsigned long long limit_ns) {
  return mbar_test_wait(bar, parity) || wait_loop(bar, parity, abort, status, limit_ns);
}
// A whole warp's: the lanes vote, for what follows is warp-collective.  All these are for
// MMAs that an issuer has committed or is about to: the issuers' limit is the caller's,
// these have the full one and leave when an issuer has given up.
__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity, int *abort, int32_t *status) {
  const bool ok = mbar_try_wait(bar, parity) || wait_loop(bar, parity, abort, status, kWaitNs);
  return __all_sync(0xffffffffu, ok);
}

// K-major operand of 128 rows: as sw128_desc.  MN-major (V: dimensions run along
// the rows of 128 bytes, tokens are K): 64 dimensions by 8 tokens in 1024 bytes,
// the next 8 tokens 1024 bytes on (stride), the next 64 dimensions a block of 128
// tokens on (leading).
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFF) >> 4);
  d |= (uint64_t)((kKeys * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// The MMAs take the descriptors' lower words and constants to add to them: left to
// itself the compiler keeps the sums of all MMAs in registers, more than there are.
template <uint32_t A, uint32_t B>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 u, v;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "add.u32 x, %1, %7;\n\tadd.u32 y, %3, %8;\n\tmov.b64 u, {x, %2};\n\tmov.b64 v, {y, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], u, v, %5, p;\n\t}" ::"r"(d),
      "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(acc), "n"(A), "n"(B)
      : "memory");
}
template <uint32_t B>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 y;\n\t.reg .b64 v;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "add.u32 y, %2, %6;\n\tmov.b64 v, {y, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], v, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "r"(acc), "n"(B)
      : "memory");
}
template <int V>
struct Int {
  static constexpr int value = V;
};
// f(Int<0>) .. f(Int<N - 1>).
template <int N, int I = 0, class F>
__device__ __forceinline__ void each(F f) {
  if constexpr (I < N) {
    f(Int<I>{});
    each<N, I + 1>(f);
  }
}

__device__ __forceinline__ uint32_t fma2_f16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// 64 + c of the codes in bits 4-7 and 20-23.
__device__ __forceinline__ uint32_t code_pair_hi(uint32_t w) {
  uint32_t d;
  asm("lop3.b32 %0, %1, 0x00F000F0, 0x54005400, 0xEA;" : "=r"(d) : "r"(w));
  return d;
}
// lo + step c of the 8 codes of w, in the order 0 4 1 5 2 6 3 7: c is exact, and
// the sum is rounded once.
__device__ __forceinline__ uint4 decode_word(uint32_t w, uint32_t step, uint32_t lo) {
  const uint32_t w8 = w >> 8;
  uint4 r;
  r.x = fma2_f16(hsub2_f16(lop_nib16_lo(w), 0x64006400u), step, lo);
  r.y = fma2_f16(hsub2_f16(code_pair_hi(w), 0x54005400u), step, lo);
  r.z = fma2_f16(hsub2_f16(lop_nib16_lo(w8), 0x64006400u), step, lo);
  r.w = fma2_f16(hsub2_f16(code_pair_hi(w8), 0x54005400u), step, lo);
  return r;
}
// 32 lanes x 64 consecutive columns: both loads on the way at once, and their wait, in
// one statement (as tmem_ld32).
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float *v) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,"
      "%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]),
        "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
        "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]),
        "=r"(r[63])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int R>
__device__ __forceinline__ void more_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void fewer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// ------------------------------------------------------------------ plan --
//
// Sequence s has its tiles of 256 rows at u = floor(q_off[s] G / 256) + s and on:
// places enough for them all, found without the other sequences' lengths.

__device__ __forceinline__ long long tile_base(const AttendParams &p, int s) {
  const long long row = p.b.q_off ? clamp_int(__ldg(p.b.q_off + s), 0, p.b.T) : s;
  return row * p.G / kBlockRows + s;
}

// The tile of rows at place u, of sequence s (the last that starts at or before it),
// with all its key tiles; rows 0: none.
__device__ __forceinline__ Job tile_at(const AttendParams &p, int s, int u) {
  Job g{};
  if (s < 0 || s >= p.b.n_seq) return g;
  const AttendSeq sq = attend_seq_at(p, s);
  const int rows = sq.rows * p.G;
  const long long first = (u - tile_base(p, s)) * kBlockRows;
  // (Offsets out of order can name a sequence that starts later.)
  if (rows <= kFewColumns || first < 0 || first >= rows) return g;
  g.s = s, g.q0 = sq.t0, g.nq = sq.nq, g.len = sq.len;
  g.row0 = (int)first, g.rows = min(rows - g.row0, kBlockRows);
  const int pos0 = sq.len - sq.nq + g.row0 / p.G, pos1 = sq.len - sq.nq + (g.row0 + g.rows - 1) / p.G;
  g.end = p.causal ? min(sq.len, max(0, pos1 + 1)) : sq.len;
  g.t0 = p.window ? max(0, pos0 - p.window + 1) / kKeys : 0;
  g.n = max(0, (g.end + kKeys - 1) / kKeys - g.t0);
  return g;
}

// The sequence of place u, found by a whole warp.
__device__ __forceinline__ int seq_of_place(const AttendParams &p, int u) {
  const int lane = threadIdx.x & 31;
  int base = 0, n = p.b.n_seq + 1;
  while (n > 32) {
    const int step = (n + 31) / 32, i = lane * step;
    const int k = __popc(__ballot_sync(0xffffffffu, i < n && tile_base(p, base + i) <= u));
    if (k == 0) return -1;
    const int skip = (k - 1) * step;
    base += skip;
    n = min(step, n - skip);
  }
  return base - 1 + __popc(__ballot_sync(0xffffffffu, lane < n && tile_base(p, base + lane) <= u));
}

// The block's job: part `part` of the tile of rows at place u; rows 0: none.
__device__ __forceinline__ Job find_job(const AttendParams &p, int u, int hk, int nsplit, int part) {
  Job job = tile_at(p, seq_of_place(p, u), u);
  job.hk = hk;
  job.parts = min(nsplit, max(1, job.n / kMinPart));
  if (part >= job.parts) job.rows = 0;
  const int n = job.n;
  const long long a = (long long)n * part / job.parts, z = (long long)n * (part + 1) / job.parts;
  job.t0 += (int)a, job.n = (int)(z - a);
  return job;
}

// The codes' role, a warpgroup (wd the warp in it): the key tiles, decoded into their
// stages.  It is busy nearly all of a prompt: what it need not wait for is asked for a
// tile ahead.
template <int D>
__device__ __forceinline__ void decode_tiles(const AttendParams &p, const Job &job, Bars &sm, uint8_t *k_s,
                                             uint8_t *v_s, int wd) {
  const int t0 = job.t0, n_tiles = job.n;
  // A warp has 32 tokens of the tile, in rounds of 512 neighbouring bytes of codes: a
  // lane has 16 of them, 32 dimensions of one token.
  constexpr int kPieces = D / 32, kPer = 32 / kPieces, kRounds = 32 / kPer;   // tokens of a round: 8 (D = 64: 16)
  const int lane = threadIdx.x & 31;
  const int lp = p.b.log_page, w0 = wd * 32, tk = lane / kPieces, pc = lane % kPieces, g = pc / 2;
  const int32_t *pages = p.b.pages + (size_t)job.s * p.b.max_pages;
  const uint8_t *head = p.cache + (size_t)job.hk * KvBlock<D>::bytes(lp);
  const size_t page_bytes = KvBlock<D>::bytes(lp) * p.b.Hkv;
  // The page numbers of the warp's first and last 16 tokens of tile j as they stand in
  // the table (looked at a tile later, when they have come).
  auto pages_of = [&](int j) {
    const int token = (t0 + j) * kKeys + w0;
    int2 r = make_int2(-1, -1);
    if (j < n_tiles && token < job.len) r.x = __ldg(pages + (token >> lp));
    if (lp == 4 && j < n_tiles && token + 16 < job.len) r.y = __ldg(pages + (token >> lp) + 1);
    return r;
  };
  struct Codes {
    uint4 c[kRounds];
    uint32_t sc[kRounds];
  };
  const uint32_t codes_at = KvBlock<D>::codes(lp, 0, tk) + pc * 16, codes_v = KvBlock<D>::codes(lp, 1, 0);
  const uint32_t scales_at = KvBlock<D>::scales(lp, 0, tk) + g * 4;
  const uint32_t scales_v = KvBlock<D>::scales(lp, 1, 0) - KvBlock<D>::scales(lp, 0, 0);
  // Codes and scales of K (which 0) or V; zeros where there is no page or no token.
  auto load = [&](int j, int2 page, int which, Codes &x) {
    const int token0 = (t0 + j) * kKeys + w0, left = j < n_tiles ? job.len - token0 - tk : 0;
    if (lp > 4) page.y = page.x;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int id = h ? page.y : page.x;
      const bool ok = (unsigned)id < (unsigned)p.b.n_pages;
      const int slot = (token0 + 16 * h) & ((1 << lp) - 1);
      const uint8_t *blk = head + (size_t)(ok ? id : 0) * page_bytes;
      const uint8_t *codes = blk + slot * (D / 2) + codes_at + (which ? codes_v : 0);
      const uint8_t *scales = blk + slot * (D / 16) + scales_at + (which ? scales_v : 0);
#pragma unroll
      for (int c = h * kRounds / 2; c < (h + 1) * kRounds / 2; ++c) {
        const int t = c * kPer - 16 * h;   // of the half's tokens
        x.c[c] = make_uint4(0, 0, 0, 0);
        x.sc[c] = 0;
        if (ok && 16 * h + t < left) {
          x.c[c] = __ldg(reinterpret_cast<const uint4 *>(codes + t * (D / 2)));
          x.sc[c] = __ldg(reinterpret_cast<const uint32_t *>(scales + t * (D / 16)));
        }
      }
    }
  };
  // 64 bytes of a row of 128, by 16-byte pieces exchanged as the swizzle has it; lanes
  // of the second 64 dimensions take their words in another order, so that a store
  // meets itself in no bank.
  const int row = w0 + tk;
  uint32_t at[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    at[e] = g * (kKeys * 128) + row * 128 + ((((pc & 1) * 4 + (e ^ (2 * g))) ^ (row & 7)) * 16);
  auto write = [&](uint8_t *dst, const Codes &x) {
#pragma unroll
    for (int c = 0; c < kRounds; ++c) {
      const uint32_t step = __byte_perm(x.sc[c], 0, 0x1010), lo = __byte_perm(x.sc[c], 0, 0x3232);
      const uint4 q = g ? make_uint4(x.c[c].z, x.c[c].w, x.c[c].x, x.c[c].y) : x.c[c];
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      uint4 d[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = decode_word(w[e], step, lo);
      // Rounds are a multiple of 8 rows apart: the swizzle is the same.
#pragma unroll
      for (int e = 0; e < 4; ++e) *reinterpret_cast<uint4 *>(dst + at[e] + c * kPer * 128) = d[e];
    }
  };
  Codes k, v;
  int2 page = pages_of(0), next = pages_of(1);
  load(0, page, 0, k);
  load(0, page, 1, v);
  for (int j = 0; j < n_tiles; ++j) {
    const int st = j & 1, parity = ((j >> 1) & 1) ^ 1;
    // A token whose V holds a NaN: its K becomes NaN, its V zeros, so that only the
    // rows that see it know.
    bool nan = false;
#pragma unroll
    for (int c = 0; c < kRounds; ++c) nan |= (v.sc[c] & 0x7FFFu) > 0x7C00u;
    if (__any_sync(0xffffffffu, nan)) {
#pragma unroll
      for (int c = 0; c < kRounds; ++c) {
        const uint32_t other = D == 128 ? __shfl_xor_sync(0xffffffffu, v.sc[c], 2) : v.sc[c];
        if ((v.sc[c] & 0x7FFFu) > 0x7C00u || (other & 0x7FFFu) > 0x7C00u) k.sc[c] = 0x7FFF7FFFu, v.sc[c] = 0u;
      }
    }
    // (The issuers order what is written here before the MMAs.)
    if (!wait_all(&sm.k_empty[st], parity, &sm.abort, p.status)) return;
    if (lane == 0) {
      const int left = job.len - (t0 + j) * kKeys - w0, y = lp > 4 ? page.x : page.y;
      sm.holes[j & 3][wd] = (left > 0 && (unsigned)page.x >= (unsigned)p.b.n_pages ? 1 : 0) |
                            (left > 16 && (unsigned)y >= (unsigned)p.b.n_pages ? 2 : 0);
    }
    write(k_s + st * Smem<D>::kK, k);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.k_full[st]);
    load(j + 1, next, 0, k);
    if (!wait_all(&sm.v_empty[st], parity, &sm.abort, p.status)) return;
    write(v_s + st * Smem<D>::kK, v);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.v_full[st]);
    load(j + 1, next, 1, v);
    page = next;
    next = pages_of(j + 2);
  }
}

// The MMAs of tile i of rows, issued by one thread.
template <int D, int i>
__device__ __forceinline__ void issue_tile(const AttendParams &p, Bars &sm, uint8_t *q_s, uint8_t *k_s, uint8_t *v_s,
                                           int n_tiles, int n_sub) {
  // Everything that differs between the MMAs of two steps is a constant: they take 32
  // to 64 clocks each, and the issue of one, beside three busy warps of the scheduler,
  // takes about as long.
  const uint32_t id_s = idesc_f16(kRows, kSub), id_o = idesc_f16(kRows, D) | 1u << 16;   // B transposed
  const uint64_t dq = sw128_desc(smem_u32(q_s)), dk = sw128_desc(smem_u32(k_s)), dv = v_desc(smem_u32(v_s));
  const uint32_t q0 = (uint32_t)dq, k0 = (uint32_t)dk, v0 = (uint32_t)dv;
  const uint32_t kmajor = (uint32_t)(dq >> 32), mnmajor = (uint32_t)(dv >> 32);
  bool ok = true;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    return ok = ok && wait_one(bar, parity, &sm.abort, p.status, p.wait_ns);
  };
  // Scores against half h of the keys of stage st.
  auto scores = [&](auto st_, auto h_) {
    constexpr int st = decltype(st_)::value, h = decltype(h_)::value;
    each<D / 16>([&](auto k_) {
      constexpr int kk = decltype(k_)::value;
      constexpr uint32_t off = (kk / 4) * ((kRows * 128) >> 4) + (kk & 3) * 2;
      mma_ss<i * (Smem<D>::kQ >> 4) + off, st * (Smem<D>::kK >> 4) + h * ((kSub * 128) >> 4) + off>(
          i * kKeys + h * kSub, q0, kmajor, k0, kmajor, id_s, kk > 0);
    });
    mma_commit(&sm.s_full[i][h]);
  };
  auto outputs = [&](auto st_, auto h_, int t) {
    constexpr int st = decltype(st_)::value, h = decltype(h_)::value;
    each<kSub / 16>([&](auto k_) {
      constexpr int kk = decltype(k_)::value;
      mma_ts<st * (Smem<D>::kK >> 4) + (h * kSub / 16 + kk) * (2048 >> 4)>(
          2 * kKeys + i * D, i * kKeys + h * kSub + kk * 8, v0, mnmajor, id_o, kk > 0 ? 1u : (uint32_t)(t > 0));
    });
    mma_commit(&sm.o_done[i][h]);
  };
  constexpr Int<0> c0{};
  constexpr Int<1> c1{};
  // Key tile j, in stage st: its outputs, and the scores of the next one (stage nx) in
  // its place.
  auto tile = [&](int j, auto st_, auto nx_) {
    constexpr int st = decltype(st_)::value, nx = decltype(nx_)::value;
    wait(&sm.v_full[st], (j >> 1) & 1);
    if (j + 1 < n_tiles) wait(&sm.k_full[nx], ((j + 1) >> 1) & 1);
    fence_proxy_async();
    auto half = [&](auto h_) {
      constexpr int h = decltype(h_)::value;
      const int t = 2 * j + h;
      if (t >= n_sub || !wait(&sm.p_full[i][h], j & 1)) return;
      tc_fence_after();
      outputs(st_, h_, t);
      if (t + 2 < n_sub) scores(nx_, h_);
    };
    half(c0);
    half(c1);
    mma_commit(&sm.v_empty[st]);
    if (j + 1 < n_tiles) mma_commit(&sm.k_empty[nx]);
  };
  if (n_tiles > 0 && wait(&sm.k_full[0], 0) && wait(&sm.q_full[i], 0)) {
    fence_proxy_async();
    tc_fence_after();
    scores(c0, c0);
    if (n_sub > 1) scores(c0, c1);
    mma_commit(&sm.k_empty[0]);
  }
  for (int j = 0; ok && j < n_tiles; j += 2) {
    tile(j, c0, c1);
    if (ok && j + 1 < n_tiles) tile(j + 1, c1, c0);
  }
  // One more commit covers every MMA issued; tensor memory is freed after it.
  mma_commit(&sm.drain[i]);
  drain_bar(&sm.drain[i], 0, globaltimer());
}

template <int D, Cap kCap>
__global__ void __launch_bounds__(kThreads, 1) kv4_many_kernel(const AttendParams p, int nsplit) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Bars sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Heads of one place are neighbours, the last places (of a prompt: the rows that
  // see most keys) come first.
  const int unit = gridDim.x - 1 - blockIdx.x, u = unit / p.b.Hkv, part = blockIdx.y;
  const Job job = find_job(p, u, unit - u * p.b.Hkv, nsplit, part);
  if (job.rows == 0) return;
  const int tiles = job.rows > kRows ? 2 : 1;   // tiles of rows

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 4);
      mbar_init(&sm.k_full[i], 4);
      mbar_init(&sm.k_empty[i], tiles);
      mbar_init(&sm.v_full[i], 4);
      mbar_init(&sm.v_empty[i], tiles);
      mbar_init(&sm.s_full[i][0], 1);
      mbar_init(&sm.s_full[i][1], 1);
      mbar_init(&sm.p_full[i][0], 4);
      mbar_init(&sm.p_full[i][1], 4);
      mbar_init(&sm.o_done[i][0], 1);
      mbar_init(&sm.o_done[i][1], 1);
    }
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&sm.tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;   // all 512 columns are this block's
  uint8_t *q_s = smem, *k_s = smem + 2 * Smem<D>::kQ, *v_s = k_s + 2 * Smem<D>::kK;
  const uint32_t o_col = 2 * kKeys;   // S_0, S_1 in columns 0 and 128; then O_0, O_1

  if (warp < 8) {
    // ------------------------------------------------------------- softmax
    more_regs<kSoftmaxRegs>();
    const int n_sub = job.steps();
    const int i = warp >> 2, r = (warp & 3) * 32 + lane;   // tile, row of the tile
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int row = job.row0 + i * kRows + r;
    const bool mine = row < job.row0 + job.rows;
    const int tok = min(row, job.row0 + job.rows - 1) / p.G, h = job.hk * p.G + row - tok * p.G;
    bool ok = true;
    if (i < tiles) {
      // The row of Q: scaled, in the codes' order, into the swizzled tile.
      float cs = fabsf(p.scale) * kLog2e * (kCap == kNearCap ? 2.f / p.softcap : 1.f);
      if (p.scale == 0.f) cs = 1.f;
      if (n_sub > 0) {
        uint4 raw[D / 8];
        const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (size_t)(job.q0 + tok) * p.ldq + (size_t)h * D);
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          raw[c] = mine ? src[c] : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max((w[e] << 16) & 0x7FFFFFFFu, w[e] & 0x7FFF0000u));
        }
        const int eb = (int)(top >> 23);
        const int up = eb == 255 ? 0 : min(15 + 126 - max(eb, 1), 127);
        float f = __int_as_float((up + 127) << 23);
        cs = up > 100 ? cs * 7.888609052210118e-31f * __int_as_float((227 - up) << 23)   // 2^-100
                      : cs * __int_as_float((127 - up) << 23);
        cs = fmaxf(finite(cs), 1.17549435e-38f);
        // s = cs (q f) . k with cs > 0: the scale's sign goes to q
        if (p.scale < 0.f) f = -f;
        if (p.scale == 0.f) f = 0.f;
        uint8_t *dst = q_s + i * Smem<D>::kQ + r * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(w[e] << 16) * f;
            v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u) * f;
          }
          const uint4 o = make_uint4(pack_f16(v[0], v[4]), pack_f16(v[1], v[5]), pack_f16(v[2], v[6]),
                                     pack_f16(v[3], v[7]));
          *reinterpret_cast<uint4 *>(dst + (c / 8) * (kRows * 128) + (((c & 7) ^ (r & 7)) * 16)) = o;
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full[i]);
      }
      // Keys first .. end - 1 are the row's.
      const int pos = job.len - job.nq + tok;
      const int end = p.causal ? min(job.len, pos + 1) : job.len;
      const int first = p.window ? max(0, pos - p.window + 1) : 0;
      const float cap_log2 = p.softcap * kLog2e, two_by_cap = finite(2.f / p.softcap);
      const uint32_t s_col = tmem + lane_base + i * kKeys, o_at = tmem + lane_base + o_col + i * D;
      // Steps free_lo .. free_hi - 1 of the part hide nothing from this warp's rows.
      const int free_lo = (__reduce_max_sync(0xffffffffu, first) + kSub - 1) / kSub - 2 * job.t0;
      const int free_hi = __reduce_min_sync(0xffffffffu, end) / kSub - 2 * job.t0;
      float m = kNoScore;
      float2 l = make_float2(0.f, 0.f);
      for (int t = 0; t < n_sub; ++t) {
        const int h = t & 1;
        if (!(ok = wait_all(&sm.s_full[i][h], (t >> 1) & 1, &sm.abort, p.status))) break;
        tc_fence_after();
        const uint32_t at = s_col + h * kSub;
        float s[kSub];
        tmem_ld64(at, s);
        // A near cap: cap tanh(x / cap) = cap - 2 cap r, r = 1 / (1 + e^(2 x / cap)), so r stands
        // for the score, and the least r for the largest.
        constexpr float kUnseen = kCap == kNearCap ? INFINITY : -INFINITY;
        if constexpr (kCap != kNoCap) {
#pragma unroll
          for (int c = 0; c < kSub; c += 2) {
            float2 x = mul_2(make_float2(s[c], s[c + 1]), make_float2(cs, cs));
            if constexpr (kCap == kNearCap) {
              x = add_2(make_float2(ex2(x.x), ex2(x.y)), make_float2(1.f, 1.f));
              x = make_float2(rcp_approx(x.x), rcp_approx(x.y));
            } else {
              x = capped_2(x, two_by_cap, cap_log2);
            }
            s[c] = x.x, s[c + 1] = x.y;
          }
        }
        const uint32_t holes = *reinterpret_cast<const volatile uint16_t *>(&sm.holes[(t >> 1) & 3][2 * h]);
        if (t < free_lo || t >= free_hi || holes) {
          const int k0 = job.t0 * kKeys + t * kSub, a = first - k0, b = end - k0;
#pragma unroll
          for (int c = 0; c < kSub; ++c) {
            const bool see = c >= a && c < b && !(holes >> (c / 32 * 8 + c / 16 % 2) & 1);
            s[c] = see ? s[c] : kUnseen;
          }
        }
        auto most = [](float a, float b, float c) { return kCap == kNearCap ? min3(a, b, c) : max3(a, b, c); };
        float t8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t8[e] = most(s[e], s[e + 8], s[e + 16]);
#pragma unroll
        for (int e = 0; e < 8; ++e) t8[e] = most(t8[e], s[e + 24], s[e + 32]);
#pragma unroll
        for (int e = 0; e < 8; ++e) t8[e] = most(t8[e], s[e + 40], s[e + 48]);
#pragma unroll
        for (int e = 0; e < 8; ++e) t8[e] = most(t8[e], t8[e], s[e + 56]);
        const float far = most(most(t8[0], t8[1], t8[2]), most(t8[3], t8[4], t8[5]), most(t8[6], t8[7], t8[7]));
        // A score is scale s + base.
        const float scale = kCap == kNearCap ? -2.f * cap_log2 : kCap == kFarCap ? 1.f : cs;
        const float base = kCap == kNearCap ? cap_log2 : 0.f;
        const float top = fmaf(far, scale, base);
        const bool over = top > m + 8.f;
        if (__any_sync(0xffffffffu, over)) {
          const float now = over ? top : m, f = ex2(m - now);
          m = now;
          l.x *= f, l.y *= f;
          if (t > 0) {
            // The outputs so far: the last step's MMAs are done first.  (The one before's are:
            // these scores came after them.)
            if (!(ok = wait_all(&sm.o_done[i][h ^ 1], ((t - 1) >> 1) & 1, &sm.abort, p.status))) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D; c += 16) {
              float o[16];
              uint32_t v[16];
              tmem_ld16(o_at + c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(o[e] * f);
              tmem_st16(o_at + c, v);
            }
          }
        }
        const float2 sc = make_float2(scale, scale), nm = make_float2(base - m, base - m);
        uint32_t v[kSub / 2];
#pragma unroll
        for (int e = 0; e < kSub / 2; ++e) {
          const float2 x = fma_2(make_float2(s[2 * e], s[2 * e + 1]), sc, nm);
          const float2 w = make_float2(ex2(x.x), ex2(x.y));
          l = add_2(l, w);
          v[e] = pack_f16(w.x, w.y);
        }
        tmem_st32(at, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[i][h]);
      }
      if (ok && n_sub > 0) ok = wait_all(&sm.o_done[i][(n_sub - 1) & 1], ((n_sub - 1) >> 1) & 1, &sm.abort, p.status);
      if (ok) {
        tc_fence_after();
        const float sum = l.x + l.y;
        const bool whole = job.parts == 1;
        const float f = !whole ? 1.f : sum != 0.f ? 1.f / sum : 0.f;
        const size_t at = ((size_t)unit * nsplit + part) * kBlockRows + i * kRows + r;
        float *const po = p.part_o + (whole ? 0 : at * D);
        __nv_bfloat16 *const dst = p.out + (size_t)(job.q0 + tok) * p.ldo + (size_t)h * D;
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          float o[16];
          if (n_sub > 0) {
            tmem_ld16(o_at + c, o);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            // columns 0 4 1 5 2 6 3 7
            const float4 x = make_float4(o[e] * f, o[e + 2] * f, o[e + 4] * f, o[e + 6] * f);
            const float4 y = make_float4(o[e + 1] * f, o[e + 3] * f, o[e + 5] * f, o[e + 7] * f);
            if (!mine) continue;
            if (whole) {
              const uint2 v = pack_out(x), w = pack_out(y);
              *reinterpret_cast<uint4 *>(dst + c + e) = make_uint4(v.x, v.y, w.x, w.y);
            } else {
              *reinterpret_cast<float4 *>(po + c + e) = x;
              *reinterpret_cast<float4 *>(po + c + e + 4) = y;
            }
          }
        }
        if (!whole && mine) p.part_ml[at] = make_float2(m, sum);
      }
    }
  } else if (warp < 12) {
    // -------------------------------------------------------------- decode
    fewer_regs<kDecodeRegs>();
    if (p.wait_ns == 0) {   // a limit of 0 is there to show the way out: the first operands come late
      const unsigned long long start = globaltimer();
      while (globaltimer() - start < 20000ull) {
      }
    }
    decode_tiles<D>(p, job, sm, k_s, v_s, warp - 8);
  } else {
    // --------------------------------------------------------------- issue
    fewer_regs<kIssueRegs>();
    // A warp for each tile of rows: they wait for their own softmax only.
    if (warp == 12 && elect_one()) issue_tile<D, 0>(p, sm, q_s, k_s, v_s, job.n, job.steps());
    if (warp == 13 && tiles > 1 && elect_one()) issue_tile<D, 1>(p, sm, q_s, k_s, v_s, job.n, job.steps());
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sm.tmem_base) : "memory");
  }
}

// Joins the parts of a block's rows, a warp a row.
constexpr int kJoinWarps = 8, kJoinBlocks = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) kv4_many_join_kernel(const AttendParams p, int nsplit) {
  const int unit = blockIdx.x, u = unit / p.b.Hkv, lane = threadIdx.x & 31;
  const Job job = find_job(p, u, unit - u * p.b.Hkv, nsplit, 0);
  // Every block waits: this grid must not be over before the one it joins.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (job.rows == 0 || job.parts == 1) return;
  const float *po = after_wait(p.part_o);
  const float2 *pml = after_wait(p.part_ml);
  for (int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); r < job.rows; r += gridDim.y * kJoinWarps) {
    const size_t first = (size_t)unit * nsplit * kBlockRows + r;
    RowPart rp;
    for (int i = 0; i < job.parts; i += 8)
      rp.take<8, D>(po, pml, job.parts - i, lane, [&](int k) { return first + (size_t)(i + k) * kBlockRows; });
    if (lane >= D / 4) continue;
    const int row = job.row0 + r, tok = row / p.G, h = job.hk * p.G + row - tok * p.G;
    *reinterpret_cast<uint2 *>(p.out + (size_t)(job.q0 + tok) * p.ldo + (size_t)h * D + lane * 4) = rp.result();
  }
}

// Places of all sequences' tiles of rows, and the parts that keys may be cut into.
long long places(const AttendParams &p) {
  const long long rows = (p.b.q_off ? (long long)p.b.T : p.b.n_seq) * p.G;
  return rows / kBlockRows + p.b.n_seq;
}
int split_of(const AttendParams &p) {
  const long long keys = (long long)p.b.max_pages << p.b.log_page;
  const long long most = std::max<long long>(1, (keys + kKeys - 1) / kKeys / kMinPart);
  return (int)std::max<long long>(1, std::min<long long>(kSms / (places(p) * p.b.Hkv), most));
}

template <int D, Cap kCap>
cudaError_t launch(const AttendParams &p, cudaStream_t st) {
  auto kernel = kv4_many_kernel<D, kCap>;
  static DeviceOnce once;
  cudaError_t err = once.run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
  });
  if (err != cudaSuccess) return err;
  const int nsplit = split_of(p);
  const unsigned units = (unsigned)(places(p) * p.b.Hkv);
  err = launch_k(false, kernel, dim3(units, nsplit), dim3(kThreads), Smem<D>::kBytes, st, p, nsplit);
  if (err != cudaSuccess || nsplit == 1) return err;
  // Rows that a tile may have.
  const long long rows = (long long)(p.max_q ? std::min(p.max_q, p.b.T) : p.b.T) * p.G;
  const int ny = (int)std::min<long long>(kJoinBlocks, (rows + kJoinWarps - 1) / kJoinWarps);
  return launch_k(true, kv4_many_join_kernel<D>, dim3(units, ny), dim3(kJoinWarps * 32), 0, st, p, nsplit);
}

}  // namespace

// Partial results of a call, in rows of D and of (maximum, sum).
size_t many_rows(const AttendParams &p) {
  const int nsplit = split_of(p);
  return nsplit == 1 ? 0 : (size_t)places(p) * p.b.Hkv * nsplit * kBlockRows;
}

cudaError_t launch_many(const AttendParams &p, int D, cudaStream_t st) {
  const Cap cap = p.softcap == 0.f ? kNoCap : p.softcap <= kMostNear ? kNearCap : kFarCap;
  if (D == 64)
    return cap == kNoCap     ? launch<64, kNoCap>(p, st)
           : cap == kNearCap ? launch<64, kNearCap>(p, st)
                             : launch<64, kFarCap>(p, st);
  return cap == kNoCap     ? launch<128, kNoCap>(p, st)
         : cap == kNearCap ? launch<128, kNearCap>(p, st)
                           : launch<128, kFarCap>(p, st);
}

}  // namespace moe
