// linear_tc.cu -- moe_linear above 16 tokens, on the 5th-gen tensor cores.
//
// D[128 rows of w][BN tokens] = w_tile . x_tile^T: the weights are the MMA's M
// side, so a short batch wastes no tensor rows on absent tokens (BN follows T
// in steps of 16) and an epilogue lane owns one output feature, whose bias and
// scale it loads once.  Both operands come by TMA, 128 bytes of K a row and
// stage (64 bf16 or 128 e4m3 values), 128-byte swizzled.
//
// Per CTA: warp 0 the TMA producer, warp 1 the MMA issuer (tcgen05.mma, M = 128,
// N = BN, f32 accumulators in TMEM), warps 4 and up the epilogue (two or three
// to a lane quadrant).  Two accumulators in TMEM: the epilogue of one
// tile runs under the main loop of the next.
//
// Sums: the tensor cores truncate when they add to an accumulator, measured
// 1.8e-8 of the result per addition (16 bf16 products): 1.6e-5 at K = 14336.
// That is nothing beside a bf16 output's 2^-9, but for f32 output the
// accumulator is handed over every kSegBlocks K blocks (kSegs) and the epilogue
// adds the segments in f32 to nearest, in registers: under 1e-6 of the result
// whatever K, for operands of both signs.  (All of one sign, every loss adds up:
// up to 1.5e-6 for bf16; e4m3 1.1e-6 at K = 14336, 5e-6 for SwiGLU at 6144.)
// Reading an accumulator takes TMEM from the MMAs, about 300 clocks: 2048 x
// 14336 x 4096 onto an f32 stream takes 147 us in one segment, 164 in segments
// of 12.
//
// Three forms (kMode):
//   pair   large products: two CTAs on neighbouring SMs form one 256-row tile
//          (cta_group::2): each loads its 128 rows of w and half of the
//          tokens, and the leader's MMAs read both halves, so a K block costs
//          each SM (128 + BN / 2) rows of operand traffic in place of
//          128 + BN -- what bounds the solo form: 0.00091 us a row;
//   solo   one CTA per tile;
//   split  few tiles (short batches, narrow outputs): K is split over a cluster
//          of 2 to 8 CTAs; each writes its partial tile to its own shared
//          memory, and after a cluster barrier each finishes its share of the
//          columns, reading the peers' partials over distributed shared memory
//          in rank order -- no workspace, no atomics, the same bits on every
//          call.
// The tokens are cut into n_tb nearly equal tiles (a difference of one unit of
// 16, in pairs 32), so that the tiles fill whole waves of the SMs.
//
// Measured on the device, in graphs of calls: 8192^3 bf16 566 to 580 us (1.94 to
// 1.89 PFLOP/s, a library product's burst rate; 647 us in the solo form), 4096 x
// 6144 x 6144 165 us, 4096 x 4096 x 14336 e4m3 SwiGLU 270 us (3.56 PFLOP/s; 315
// in a long loop of calls, at the card's power limit); 64 x 6144 x 1024, split
// in 8, 8.7 us, of which about 6 are start, exchange and end.
//
// Every mbarrier wait is bounded: one that gives up sets the status word (the
// caller's, or the device's where there is none), and
// the roles stop, drain their copies and MMAs, and return.
#include <algorithm>
#include <cuda.h>

#include "linear.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int BM = 128;             // rows of w per tile
constexpr int kRowBytes = 128;      // K bytes per row and stage
constexpr int kMaxStages = 8;
constexpr int kEpiWarp0 = 4;
// K blocks per accumulator segment; SwiGLU multiplies two sums, and their errors
// add.  e4m3 products have 8 significant bits, so their sums lose little (4e-7
// of the result at K = 6144, 7e-7 for SwiGLU, 1e-6 at 14336 in one segment):
// they go without up to kPlainBlocks K blocks.
template <int DT, bool kSwiglu>
constexpr int kSegBlocks = DT == MOE_BF16 ? (kSwiglu ? 7 : 12) : (kSwiglu ? 24 : 48);
constexpr int kPlainBlocks = 48;
constexpr int kMaxBN = 256;
constexpr int kSegMaxBN = 192;      // with segment sums in registers
// Epilogue warps per lane quadrant: they take turns at blocks of 16 columns.
// With segments there are three, so that a thread's segment sums (64 at BN =
// 192) fit its registers: spilled, they share the path that feeds the MMAs.
// (Seven or eight scalars of a tile do spill in the solo and pair forms without
// SwiGLU, at the 128 registers that 512 threads leave.)
template <bool kSegs>
constexpr int kEpiGroups = kSegs ? 3 : 2;
template <bool kSegs>
constexpr int kThreads = (kEpiWarp0 + 4 * kEpiGroups<kSegs>) * 32;

constexpr size_t kSmemMax = 227 * 1024;

enum Mode { kSolo, kPair, kSplit };

struct TcLinear {
  CUtensorMap map_w;       // [rows][K], box 128 x 128 bytes; SwiGLU: [N/16][2][16][K]
  CUtensorMap map_x;       // [T][K], box of a CTA's tokens x 128 bytes
  LinearParams p;
  int unit, units_tb;      // tokens come in units of 16 (pairs: 32), units_tb to a tile
  int n_wide;              // and one more to the first n_wide
  int bn;                  // most tokens of a tile
  int x_rows;              // tokens a CTA loads per tile (bn, in pairs bn / 2)
  int n_fb, n_tb;          // tiles along the outputs (in pairs: of 256 rows) and the tokens
  int group_tb;            // token tiles per raster group
  int nkb;                 // K blocks of the whole product
  int stages;
  unsigned long long wait_ns;   // limit of each role wait
};

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// Set by the products on this device that gave up and had no status word of
// their caller's; moe_linear_status reads it.
__device__ int32_t gave_up;

template <int DT>
__device__ __forceinline__ uint32_t linear_idesc(int m, int n) {
  // kind::f8f6f4: format fields 0 = e4m3 for A and B, f32 accumulator
  if constexpr (DT == MOE_BF16) return idesc_bf16(m, n);
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

#define MOE_LINEAR_MMA(GROUP, KIND)                                                       \
  asm volatile(                                                                           \
      "{\n\t.reg .pred p;\n\t"                                                            \
      "setp.ne.b32 p, %4, 0;\n\t"                                                         \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(d), \
      "l"(da), "l"(db), "r"(idesc), "r"(acc)                                              \
      : "memory")
template <int DT, int kMode>
__device__ __forceinline__ void linear_mma(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc,
                                           uint32_t acc) {
  if constexpr (DT == MOE_BF16) {
    if constexpr (kMode == kPair) MOE_LINEAR_MMA("2", "f16");
    else MOE_LINEAR_MMA("1", "f16");
  } else {
    if constexpr (kMode == kPair) MOE_LINEAR_MMA("2", "f8f6f4");
    else MOE_LINEAR_MMA("1", "f8f6f4");
  }
}
#undef MOE_LINEAR_MMA

// Arrives on `bar` when the MMAs issued so far are done; in pairs on the
// barrier at the same place in both CTAs.
template <int kMode>
__device__ __forceinline__ void linear_commit(uint64_t *bar) {
  if constexpr (kMode == kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    mma_commit(bar);
}

// The address of p in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}

// TMA loads into this CTA's shared memory; in pairs the bytes are counted on
// the leader's barrier (`bar` its cluster address).
template <int kMode>
__device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  if constexpr (kMode == kPair)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <int kMode>
__device__ __forceinline__ void load_4d(void *dst, const CUtensorMap *map, int x, int w, uint32_t bar) {
  if constexpr (kMode == kPair)
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(w), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(w), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ float ld_peer(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// Tile t of the raster: output tile fb, tokens c0 .. c0 + w - 1.  The first
// n_wide token tiles have a unit more than the others, and all of theirs come
// first: dealt out in turn, the wide tiles then spread over the CTAs.  Token
// tiles run fastest within groups of group_tb, so the CTAs of a wave share few
// w and x tiles and both stay in L2.
struct Tile {
  int fb, c0, w;
};
__device__ __forceinline__ Tile tile_at(const TcLinear &q, int t) {
  const int wide = q.n_fb * q.n_wide;
  const int first = t < wide ? 0 : q.n_wide, n_tb = t < wide ? q.n_wide : q.n_tb - q.n_wide;
  if (t >= wide) t -= wide;
  const int per = q.group_tb * q.n_fb;
  const int g = t / per, r = t - g * per;
  const int width = min(q.group_tb, n_tb - g * q.group_tb);
  Tile tl;
  tl.fb = r / width;
  const int tb = first + g * q.group_tb + (r - tl.fb * width);
  tl.c0 = (tb * q.units_tb + min(tb, q.n_wide)) * q.unit;
  tl.w = (q.units_tb + (tb < q.n_wide ? 1 : 0)) * q.unit;
  return tl;
}

// One lane's accumulator column block: W values of columns (tokens) t0 ..,
// its own row's sums in v.  Rows of w: lane r of the tile holds row
// fb * 128 + r; for SwiGLU, quadrant q's lanes 0-15 the gate rows of features
// fb * 64 + 16 q + lane, lanes 16-31 their up rows.
template <bool kSwiglu>
struct LaneRow {
  int n;          // output feature of this lane
  bool ok;        // inside N
  float sw, b;    // scale and bias of this lane's row of w
};

template <bool kSwiglu>
__device__ __forceinline__ LaneRow<kSwiglu> lane_row(const LinearParams &p, int fb, int quad, int lane) {
  LaneRow<kSwiglu> r;
  int row;
  if constexpr (kSwiglu) {
    r.n = fb * 64 + quad * 16 + (lane & 15);
    row = r.n + (lane >= 16 ? p.N : 0);
  } else {
    r.n = fb * BM + quad * 32 + lane;
    row = r.n;
  }
  r.ok = r.n < p.N;
  r.sw = r.ok && p.w_scale ? __ldg(p.w_scale + row) : 1.f;
  r.b = r.ok && p.bias ? __ldg(p.bias + row) : 0.f;
  return r;
}

// The residual of a block of W columns, raw, loaded ahead of its use: a
// conversion at each load would make it wait for itself.  SwiGLU: the lane's
// own token of each column pair.
template <bool kSwiglu, bool kBf16, int W>
struct Resid {
  uint32_t v[kSwiglu ? W / 2 : W];
  __device__ __forceinline__ void load(const LinearParams &p, const LaneRow<kSwiglu> &r, int t0, int n_cols) {
    if (!p.resid) return;
    const int up = kSwiglu && (threadIdx.x & 31) >= 16 ? 1 : 0;
    const int end = r.ok ? min(p.T - t0, n_cols) - up : 0;   // columns this lane stores
    const size_t i0 = (size_t)(t0 + up) * p.ldr + r.n;
#pragma unroll
    for (int j = 0; j < W; j += kSwiglu ? 2 : 1) {
      uint32_t u = 0u;
      if (j < end)
        u = kBf16 ? reinterpret_cast<const unsigned short *>(p.resid)[i0 + (size_t)j * p.ldr]
                  : reinterpret_cast<const uint32_t *>(p.resid)[i0 + (size_t)j * p.ldr];
      v[kSwiglu ? j / 2 : j] = u;
    }
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(kBf16 ? v[i] << 16 : v[i]);
  }
};

template <bool kSwiglu, bool kBf16, int W>
__device__ __forceinline__ void finish_columns(const LinearParams &p, const LaneRow<kSwiglu> &r,
                                               float (&v)[W], const Resid<kSwiglu, kBf16, W> &res,
                                               int t0, int n_cols) {
  static_assert(W <= 32 && W % 2 == 0, "columns of one block");
  const int lane = threadIdx.x & 31;
  if (p.x_scale) {
    const float sx = lane < W && t0 + lane < p.T ? __ldg(p.x_scale + t0 + lane) : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] *= r.sw * __shfl_sync(0xffffffffu, sx, j);
  }
#pragma unroll
  for (int j = 0; j < W; ++j) v[j] += r.b;
  if constexpr (kSwiglu) {
    // One exchange per column pair: lanes 0-15 finish token j (their gate,
    // the partner's up), lanes 16-31 token j + 1.
    const bool lo = lane < 16;
#pragma unroll
    for (int j = 0; j < W; j += 2) {
      const float recv = __shfl_xor_sync(0xffffffffu, lo ? v[j + 1] : v[j], 16);
      const int jc = j + (lo ? 0 : 1);
      if (r.ok && jc < n_cols && t0 + jc < p.T) {
        float y = swiglu<kBf16>(lo ? v[j] : recv, lo ? recv : v[j + 1]);
        if (p.resid) y += res.get(j / 2);
        store_out<kBf16>(p, t0 + jc, r.n, y);
      }
    }
  } else {
    if (p.act == MOE_ACT_SILU) {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = silu<kBf16>(v[j]);
    } else if (p.act == MOE_ACT_GELU) {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = activate(MOE_ACT_GELU, v[j]);
    }
    if (p.resid) {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] += res.get(j);
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (r.ok && j < n_cols && t0 + j < p.T) store_out<kBf16>(p, t0 + j, r.n, v[j]);
  }
}

template <bool kBf16>
__device__ __forceinline__ void prefetch_resid(const LinearParams &p, int t, int n) {
  const char *a = reinterpret_cast<const char *>(p.resid) + ((size_t)t * p.ldr + n) * (kBf16 ? 2 : 4);
  asm volatile("prefetch.global.L2 [%0];" ::"l"(a));
}

// A role's wait: false if the CTA is stopping or the wait ran past its limit,
// and then *status and *abort are set.
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
__device__ __noinline__ bool wait_call(uint64_t *bar, uint32_t parity, int *abort, int32_t *status,
                                       unsigned long long limit_ns) {
  return wait_loop(bar, parity, abort, status, limit_ns);
}
// The producer's and the MMA issuer's, one thread each.  A limit of 0 gives up
// wherever the phase is not complete when first tested (test_wait does not
// hold the thread, and costs these loops nothing).
__device__ __forceinline__ bool wait_role(uint64_t *bar, uint32_t parity, int *abort, int32_t *status,
                                          unsigned long long limit_ns) {
  return mbar_test_wait(bar, parity) || wait_call(bar, parity, abort, status, limit_ns);
}
// The epilogue's, by whole warps, without a call, because it holds sums in
// registers across it; it waits long and ends with the other roles.  The lanes
// vote: one may see the phase complete where another sees the CTA stop, and the
// tensor-memory loads that follow are warp-collective.
__device__ __forceinline__ bool wait_inline(uint64_t *bar, uint32_t parity, int *abort, int32_t *status) {
  const bool ok = mbar_try_wait(bar, parity) || wait_loop(bar, parity, abort, status, kWaitNs);
  return __all_sync(0xffffffffu, ok);
}

// A persistent CTA (pair) walks the tiles; kSplit: one tile per cluster.
// kBf16: the output type.  kSegs: K in segments.
template <int DT, bool kSwiglu, int kMode, bool kBf16, bool kSegs>
__global__ void __launch_bounds__(kThreads<kSegs>, 1) linear_tc_kernel(const __grid_constant__ TcLinear q) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars sm;
  // Pairs: the buffers lie at the same place in both CTAs (the same launch).
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const LinearParams &p = q.p;
  int32_t *status = p.status ? p.status : &gave_up;
  constexpr int G = kEpiGroups<kSegs>;
  constexpr int kBlockElems = kRowBytes / (DT == MOE_BF16 ? 2 : 1);
  const uint32_t stage_bytes = (BM + q.x_rows) * kRowBytes;
  const uint32_t acc_cols = q.bn <= 32 ? 32 : q.bn <= 64 ? 64 : q.bn <= 128 ? 128 : 256;
  const int S = q.stages;
  int ranks = 1, rank = 0;
  if constexpr (kMode != kSolo) {
    asm volatile("mov.u32 %0, %cluster_nctarank;" : "=r"(ranks));
    rank = cluster_rank();
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.acc_full[i], 1);
      mbar_init(&sm.acc_empty[i], (kMode == kPair ? 2 : 1) * 4 * G);
    }
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if constexpr (kMode == kPair) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&sm.tmem_base)),
                   "r"(2 * acc_cols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&sm.tmem_base)),
                   "r"(2 * acc_cols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kMode == kPair) cluster_sync();   // the peer's barriers are ready too
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  // This CTA's tiles and its share of K.
  const int n_tiles = q.n_fb * q.n_tb;
  const int t_first = blockIdx.x / ranks, t_step = gridDim.x / ranks;
  const int kb0 = kMode == kSplit ? (int)((long long)q.nkb * rank / ranks) : 0;
  const int kb1 = kMode == kSplit ? (int)((long long)q.nkb * (rank + 1) / ranks) : q.nkb;
  constexpr int kSeg = kSegBlocks<DT, kSwiglu>;
  const int n_seg = kSegs ? (kb1 - kb0 + kSeg - 1) / kSeg : 1;
  auto seg_at = [&](int s) { return kb0 + (int)((long long)(kb1 - kb0) * s / n_seg); };
  // The 128-row block of w and the tokens that this CTA loads of a tile.
  auto block_of = [&](const Tile &tl) { return kMode == kPair ? 2 * tl.fb + rank : tl.fb; };
  auto x_row_of = [&](const Tile &tl) { return kMode == kPair ? tl.c0 + rank * (tl.w / 2) : tl.c0; };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      int s = 0;
      uint32_t ph = 0, armed = 0, par = 0;
      bool ok = true;
      // A limit of 0 is there to show the way out: operands that happen to be at
      // hand when first tested (40 x 8192 x 256 out of L2, two calls of three)
      // would not, so they come late.
      if (q.wait_ns == 0) {
        const unsigned long long start = globaltimer();
        while (globaltimer() - start < 20000ull) {
        }
      }
      for (int t = t_first; ok && t < n_tiles; t += t_step) {
        const Tile tl = tile_at(q, t);
        const int fb = block_of(tl), x_row = x_row_of(tl);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = wait_role(&sm.empty[s], ph ^ 1, &sm.abort, status, q.wait_ns))) break;
          uint8_t *a = smem + s * stage_bytes;
          uint32_t bar = smem_u32(&sm.full[s]);
          if constexpr (kMode == kPair) bar = peer_addr(&sm.full[s], 0);
          // The leader expects both CTAs' bytes.
          if (kMode != kPair || rank == 0)
            mbar_expect_tx(&sm.full[s], kMode == kPair ? 2 * stage_bytes : stage_bytes);
          if constexpr (kSwiglu) load_4d<kMode>(a, &q.map_w, kb * kBlockElems, fb * 4, bar);
          else load_2d<kMode>(a, &q.map_w, kb * kBlockElems, fb * BM, bar);
          load_2d<kMode>(a + BM * kRowBytes, &q.map_x, kb * kBlockElems, x_row, bar);
          armed |= 1u << s;
          par = (par & ~(1u << s)) | (ph << s);
          if (++s == S) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // Every copy that was issued has landed before the CTA goes on.  A pair's
      // second CTA cannot watch the leader's barriers: its copies are done when
      // the leader's MMAs have read them and their commits have arrived here; if
      // it stopped early it gives them a millisecond.
      const unsigned long long t0 = globaltimer();
      if (kMode != kPair || rank == 0) {
        for (int i = 0; i < S; ++i)
          if ((armed >> i) & 1) drain_bar(&sm.full[i], (par >> i) & 1, t0);
      } else if (ok) {
        for (int i = 0; i < S; ++i)
          if ((armed >> i) & 1) drain_bar(&sm.empty[i], (par >> i) & 1, t0);
      } else {
        while (globaltimer() - t0 < 1000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 && (kMode != kPair || rank == 0)) {
    // ---------------------------------------------------------- MMA issuer
    if (elect_one()) {
      int s = 0;
      uint32_t ph = 0, it = 0;
      const uint64_t da0 = sw128_desc(smem_u32(smem));
      const uint32_t stage_desc = stage_bytes >> 4;
      bool ok = true;
      for (int t = t_first; ok && t < n_tiles; t += t_step) {
        const Tile tl = tile_at(q, t);
        const uint32_t idesc = linear_idesc<DT>(kMode == kPair ? 2 * BM : BM, tl.w);
        for (int sg = 0; ok && sg < n_seg; ++sg, ++it) {
          const int buf = it & 1;
          if (!(ok = wait_role(&sm.acc_empty[buf], ((it >> 1) & 1) ^ 1, &sm.abort, status, q.wait_ns))) break;
          tc_fence_after();
          const uint32_t d = tmem + buf * acc_cols;
          const int ka = seg_at(sg), ke = seg_at(sg + 1);
          for (int kb = ka; kb < ke; ++kb) {
            if (!(ok = wait_role(&sm.full[s], ph, &sm.abort, status, q.wait_ns))) break;
            tc_fence_after();
            const uint64_t da = da0 + (uint64_t)(s * stage_desc);
            const uint64_t db = da + ((BM * kRowBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              linear_mma<DT, kMode>(d, da + 2 * kk, db + 2 * kk, idesc, kb > ka || kk > 0);
            linear_commit<kMode>(&sm.empty[s]);
            if (++s == S) {
              s = 0;
              ph ^= 1;
            }
          }
          if (!ok) break;
          linear_commit<kMode>(&sm.acc_full[buf]);
        }
      }
      // One more commit covers every MMA issued, also those of a tile that was
      // left in the middle; TMEM is freed only after it has arrived.
      linear_commit<kMode>(&sm.drain);
      drain_bar(&sm.drain, 0, globaltimer());
    }
    __syncwarp();
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3, turn = (warp - kEpiWarp0) >> 2;
    // Block c of this warp: columns (c G + turn) 16 .. + 15.
    auto col_of = [&](int c) { return (c * G + turn) * 16; };
    auto release = [&](int buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kMode == kPair)
          asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(
                           peer_addr(&sm.acc_empty[buf], 0))
                       : "memory");
        else
          mbar_arrive(&sm.acc_empty[buf]);
      }
    };
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    uint32_t it = 0;
    bool ok = true;
    for (int t = t_first; ok && t < n_tiles; t += t_step) {
      const Tile tl = tile_at(q, t);
      const LaneRow<kSwiglu> row = lane_row<kSwiglu>(p, block_of(tl), quad, lane);
      if constexpr (kMode != kSplit) {
        // The tile's residual comes to L2 under the main loop.
        if (p.resid && row.ok)
          for (int c = turn; c < tl.w; c += G)
            if (tl.c0 + c < p.T && (lane & 7) == 0) prefetch_resid<kBf16>(p, tl.c0 + c, row.n);
      }
      constexpr int kChunks = kSegs ? kSegMaxBN / 16 / G : 1;
      float acc[kChunks][16];
      if constexpr (kSegs) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[c][j] = 0.f;
        for (int sg = 0; sg + 1 < n_seg; ++sg, ++it) {
          const int buf = it & 1;
          if (!(ok = wait_inline(&sm.acc_full[buf], (it >> 1) & 1, &sm.abort, status))) break;
          tc_fence_after();
          const uint32_t col = tmem + lane_base + buf * acc_cols;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            if (col_of(c) < tl.w) {
              float v[16];
              tmem_ld16(col + col_of(c), v);
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[c][j] += v[j];
            }
          }
          release(buf);
        }
        if (!ok) break;
      }
      const int buf = it & 1;
      if (!(ok = wait_inline(&sm.acc_full[buf], (it >> 1) & 1, &sm.abort, status))) break;
      tc_fence_after();
      const uint32_t col = tmem + lane_base + buf * acc_cols;
      auto chunk = [&](int c, const float *more) {
        float v[16];
        Resid<kSwiglu, kBf16, 16> res;
        if constexpr (kMode != kSplit) res.load(p, row, tl.c0 + col_of(c), 16);
        tmem_ld16(col + col_of(c), v);
        if (more) {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] += more[j];
        }
        if constexpr (kMode == kSplit) {
          float *dst = reinterpret_cast<float *>(smem) + col_of(c) * BM + quad * 32 + lane;
#pragma unroll
          for (int j = 0; j < 16; ++j) dst[j * BM] = v[j];
        } else {
          finish_columns<kSwiglu, kBf16>(p, row, v, res, tl.c0 + col_of(c), 16);
        }
      };
      if constexpr (kSegs) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (col_of(c) < tl.w) chunk(c, acc[c]);
      } else {
        for (int c = 0; col_of(c) < tl.w; ++c) chunk(c, nullptr);
      }
      release(buf);
      ++it;
    }
  }

  if constexpr (kMode == kSplit) {
    __syncthreads();          // the roles are reconverged for the aligned barrier
    cluster_sync();           // every CTA's partial tile is in its shared memory
    if (warp >= kEpiWarp0 && !*reinterpret_cast<volatile int *>(&sm.abort)) {
      const int quad = warp & 3, turn = (warp - kEpiWarp0) >> 2;
      const Tile tl = tile_at(q, t_first);
      const LaneRow<kSwiglu> row = lane_row<kSwiglu>(p, tl.fb, quad, lane);
      const int share = ((tl.w + ranks - 1) / ranks + 1) & ~1;   // columns per rank, even
      const int cols = min(share, tl.w - rank * share);
      for (int c = turn * 4; c < cols; c += 4 * G) {
        const int n_cols = min(4, cols - c), col = rank * share + c;
        Resid<kSwiglu, kBf16, 4> res;
        res.load(p, row, tl.c0 + col, n_cols);
        // All ranks' partials are asked for before the first is added.
        const uint32_t src = smem_u32(smem) + ((uint32_t)col * BM + quad * 32 + lane) * 4;
        float part[8][4];
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[r][j] = r < ranks && j < n_cols ? ld_peer(src + j * BM * 4, r) : 0.f;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] += part[r][j];
        finish_columns<kSwiglu, kBf16>(p, row, v, res, tl.c0 + col, n_cols);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kMode == kPair) {
    // The leader's last commit arrives on the second CTA's drain barrier too, as
    // an access of its own that the cluster barrier below does not order: that
    // CTA's shared memory may be another block's once it has left.
    if (rank != 0 && threadIdx.x == 0) drain_bar(&sm.drain, 0, globaltimer());
    __syncwarp();
  }
  // No CTA leaves while a peer may read its shared memory or tensor memory.
  if constexpr (kMode != kSolo) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kMode == kPair)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(2 * acc_cols)
                   : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(2 * acc_cols)
                   : "memory");
  }
}

// ----------------------------------------------------------------- launch --

struct Plan {
  int mode, n_tb, split;
};

int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

int up(int v, int m) { return (v + m - 1) / m; }

// moe_linear_wait_limit's, for the products that this host thread launches.
thread_local unsigned long long wait_limit_ns = kWaitNs;

// Clusters of 1 .. 8 CTAs, one CTA to an SM, that run at once on 152 SMs
// (cudaOccupancyMaxActiveClusters): a split into more takes a second wave,
// which costs more than it gains (48 clusters of 3 for N = 6144: 28 us; of 2:
// 18 us).
constexpr int kClusters[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};

// The form and the tiles with the least estimated time, in clocks of an SM.  A
// K block costs the larger of its MMAs (4 of w / 2 clocks for w tokens, not
// under 59 each, and 12 more) and its operand rows at 1.74 clocks each; the
// whole costs at least its bytes from memory; each form has its start and end.
// All measured: within 15% of the best of all forms and tilings for T = 32 ..
// 1024 and N = 256 .. 14336.
Plan plan_of(int T, int rows, int nkb, int sms, int max_bn) {
  Plan best{kSolo, 1, 1};
  double best_cost = 1e300;
  auto consider = [&](int mode, int n_tb, int split) {
    const int unit = mode == kPair ? 32 : 16, units = up(T, unit);
    if (n_tb > units) return;
    const int w = up(units, n_tb) * unit;
    if (w > max_bn) return;
    const long long tiles = (long long)up(rows, mode == kPair ? 2 * BM : BM) * n_tb;
    if (mode == kSplit && tiles > (long long)kClusters[split] * sms / 152) return;
    // The CTA with most work takes every slots-th tile from the first: as many
    // columns as blocks of MMAs, each block with its own floor and 12 clocks.
    const long long slots = mode == kSplit ? tiles : mode == kPair ? sms / 2 : sms;
    const long long waves = (tiles + slots - 1) / slots, wide = (long long)(tiles / n_tb) * (units % n_tb);
    const long long wide_waves = std::min(waves, (wide + slots - 1) / slots);
    auto block = [&](int w1) {
      return std::max(4.0 * std::max((w1 + 24.0) / 2.0, 59.0),
                      1.74 * (BM + (mode == kPair ? w1 / 2 : w1)));
    };
    const int narrow = units / n_tb * unit;
    const double clocks = wide_waves * block(narrow + unit) + (waves - wide_waves) * block(narrow);
    const double bytes = ((double)rows + T) * nkb * kRowBytes / 3500.0;
    const double start = mode == kSolo ? 8500.0 : mode == kPair ? 10500.0 : 11500.0;
    const double cost = std::max(clocks * std::max(1.0, (double)nkb / split), bytes) + start + 12.0 * w;
    if (cost < best_cost) {
      best_cost = cost;
      best = Plan{mode, n_tb, split};
    }
  };
  const int least = up(T, max_bn), n_fb = up(rows, BM);
  for (int n_tb = least; n_tb <= std::min(least + 32, 2 * least + 8); ++n_tb) {
    consider(kSolo, n_tb, 1);
    if (n_fb >= 2) consider(kPair, n_tb, 1);
    for (int split = 2; split <= 8 && n_fb * n_tb <= kClusters[split] && nkb / split >= 4; ++split)
      consider(kSplit, n_tb, split);
  }
  return best;
}

template <int DT, bool kSwiglu, int kMode, bool kBf16, bool kSegs>
cudaError_t launch(const TcLinear &q, int grid, int cluster, cudaStream_t st) {
  auto kernel = linear_tc_kernel<DT, kSwiglu, kMode, kBf16, kSegs>;
  static DeviceOnce once;
  const cudaError_t err = once.run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(kSmemMax - sizeof(Bars) - 64));
  });
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads<kSegs>);
  cfg.dynamicSmemBytes = (size_t)q.stages * (BM + q.x_rows) * kRowBytes + 1024;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = kMode == kSolo ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, q);
}

template <int DT, bool kSwiglu, bool kBf16, bool kSegs>
cudaError_t launch_mode(const TcLinear &q, const Plan &plan, int sms, cudaStream_t st) {
  const int tiles = q.n_fb * q.n_tb;
  if (plan.mode == kPair)
    return launch<DT, kSwiglu, kPair, kBf16, kSegs>(q, 2 * std::min(tiles, sms / 2), 2, st);
  if (plan.mode == kSplit)
    return launch<DT, kSwiglu, kSplit, kBf16, kSegs>(q, tiles * plan.split, plan.split, st);
  return launch<DT, kSwiglu, kSolo, kBf16, kSegs>(q, std::min(tiles, sms), 1, st);
}

template <int DT, bool kSwiglu>
cudaError_t launch_out(const TcLinear &q, const Plan &plan, bool segs, int sms, cudaStream_t st) {
  if (q.p.out_dtype == MOE_BF16) return launch_mode<DT, kSwiglu, true, false>(q, plan, sms, st);
  if constexpr (DT == MOE_E4M3)
    if (!segs) return launch_mode<DT, kSwiglu, false, false>(q, plan, sms, st);
  return launch_mode<DT, kSwiglu, false, true>(q, plan, sms, st);
}

template <int DT>
cudaError_t launch_type(const TcLinear &q, const Plan &plan, bool segs, int sms, cudaStream_t st) {
  return q.p.act == MOE_ACT_SWIGLU ? launch_out<DT, true>(q, plan, segs, sms, st)
                                   : launch_out<DT, false>(q, plan, segs, sms, st);
}

}  // namespace

unsigned long long linear_wait_ns() { return wait_limit_ns; }

cudaError_t linear_gave_up(int32_t **word) {
  static std::atomic<int32_t *> known[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 64 && (*word = known[dev].load(std::memory_order_acquire))) return cudaSuccess;
  void *at = nullptr;
  err = cudaGetSymbolAddress(&at, gave_up);
  if (err != cudaSuccess) return err;
  *word = static_cast<int32_t *>(at);
  if (dev < 64) known[dev].store(*word, std::memory_order_release);
  return cudaSuccess;
}

cudaError_t launch_linear_tc(const LinearParams &p, int dtype, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const bool sw = p.act == MOE_ACT_SWIGLU;
  const int es = dtype == MOE_BF16 ? 2 : 1, rows = sw ? 2 * p.N : p.N;
  const CUtensorMapDataType dt =
      dtype == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  TcLinear q;
  q.p = p;
  q.nkb = up(p.K * es, kRowBytes);
  const bool segs = p.out_dtype == MOE_F32 && (dtype == MOE_BF16 || q.nkb > kPlainBlocks);
  const Plan plan = plan_of(p.T, rows, q.nkb, sms, segs ? kSegMaxBN : kMaxBN);
  const bool pair = plan.mode == kPair;
  q.unit = pair ? 32 : 16;
  const int units = up(p.T, q.unit);
  q.n_tb = plan.n_tb;
  q.units_tb = units / q.n_tb;
  q.n_wide = units % q.n_tb;
  q.bn = up(units, q.n_tb) * q.unit;
  q.x_rows = pair ? q.bn / 2 : q.bn;
  q.n_fb = up(rows, pair ? 2 * BM : BM);
  q.group_tb = std::min(q.n_tb, 16);
  q.wait_ns = wait_limit_ns;
  const size_t stage = (size_t)(BM + q.x_rows) * kRowBytes;
  q.stages = (int)std::min<size_t>(kMaxStages, (kSmemMax - sizeof(Bars) - 64 - 1024) / stage);
  if (sw) {
    if (!make_map_4d(&q.map_w, p.w, dt, p.K, 16, 2, p.N / 16, (uint64_t)p.ldw * es,
                     (uint64_t)p.ldw * es * p.N, (uint64_t)p.ldw * es * 16, kRowBytes / es, 16, 2, 4))
      return cudaErrorInvalidValue;
  } else if (!make_map(&q.map_w, p.w, dt, es, p.K, rows, p.ldw, kRowBytes / es, BM)) {
    return cudaErrorInvalidValue;
  }
  if (!make_map(&q.map_x, p.x, dt, es, p.K, p.T, p.ldx, kRowBytes / es, q.x_rows))
    return cudaErrorInvalidValue;
  return dtype == MOE_BF16 ? launch_type<MOE_BF16>(q, plan, segs, sms, st)
                           : launch_type<MOE_E4M3>(q, plan, segs, sms, st);
}

}  // namespace moe

extern "C" __attribute__((visibility("default"))) int moe_linear_wait_limit(int us) {
  if (us < 0) return MOE_ERR_ARG;
  moe::wait_limit_ns = (unsigned long long)us * 1000ull;
  return MOE_OK;
}

extern "C" __attribute__((visibility("default"))) int moe_linear_status(int32_t *status) {
  if (!status) return MOE_ERR_ARG;
  int32_t none = 0;
  if (cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpyFromSymbol(status, moe::gave_up, 4) != cudaSuccess ||
      (*status && cudaMemcpyToSymbol(moe::gave_up, &none, 4) != cudaSuccess))
    return MOE_ERR_DEVICE;
  return MOE_OK;
}
