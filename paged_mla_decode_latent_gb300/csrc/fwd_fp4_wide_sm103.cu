// fwd_fp4_wide_sm103.cu -- the decode over a 4-bit cache for more than 32 score
// rows: a pair of CTAs per (sequence, block of 128 rows, KV split), one MMA over both.
//
// With K a tile's 256 keys, Q the N = 64 or 128 query rows and V the first 512 dims of
// K, the pair computes, transposed as in the kernel for fewer rows,
//
//   S = K Q^T     [256 keys x N]   CTA r has keys 128 r .. (K from TMEM) and half of Q's rows
//   O^T += V^T P  [512 dims x N]   CTA r has dims 256 r .. of V and half of P's rows
//
// so that O^T takes 2 N TMEM columns of each CTA and both operands' other halves come
// from the partner's shared memory.  What the two CTAs trade is half of the weights in
// f16 (16 KB each way for 256 keys at N = 128), a bit a warp on whether a tile raises the
// running maxima, and the maxima where it does.  Contracting the dims in halves instead,
// as the 128-row kernel of the wider caches does, trades partial scores, 128 KB for 256
// keys: at 28 GB/s each way it was bound by that (197 us where this takes 143, below).
// Scores are summed in fp32 in one place.
//
// Per tile, all at once:
//   rows warp     looks up the rows of later tiles, and fetches them to L2
//   K warps (8)   codes to f16, 16 keys a warp, 128 dims at a time into TMEM
//   QK warp       (even CTA) S as soon as a slab of K is there
//   softmax warps a key a thread, half of the rows: the scores go to registers at once,
//   (8)           so that the next tile's MMAs may start; weights relative to a running
//                 maximum that is raised (and O rescaled) only when a weight would pass
//                 2^8, in both CTAs or neither
//   relay warp    passes on that the partner's weights have landed
//   V warps (8)   codes to f16, the CTA's 256 dims of 32 keys at a time
//   PV warp       (even CTA) O^T += V^T P, 32 keys at a time
// K and V read the cache into registers (a key's pieces side by side in a quad of lanes):
// no shared memory is left for a ring of codes, and less of it leaves more L1 for the
// reads that come back to a line (five units of V took 184 us where three took 163).
//
// What bounds it: no unit, but the chain of handoffs; a tile takes 7700 cycles at N =
// 128, its MMAs 4400 and its shared-memory traffic 3500.  Batch 64 x 128 heads x 8192:
// 143 us (1.53 TB/s; 53 % of what cuBLAS reaches in bf16), batch 8 x 128 x 65536: 138;
// batch 64 x 64 heads x 8192: 111 us.  Steps to there from 277: four lanes a key instead
// of one 234, slabs of 128 dims instead of 64 232, rows fetched to L2 ahead 208, scores
// to registers, K and V in eight warps each and the rows looked up by a warp of their
// own 184, three units of V 163, fewer registers spilled 146, six query loads in flight
// instead of nine (the last registers) 143.
//
// Precision is that of the kernel for fewer rows: queries and weights in f16.
//
// Every wait is bounded (2 s unless the plan sets another limit); one that runs out
// sets MLA_DEVFLAG_TIMEOUT and the pair winds down.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/mla_decode.h"
#include "fp4.cuh"
#include "internal.h"
#include "kv.h"
#include "ptx.cuh"

namespace {

constexpr int T = 256;                  // keys per tile, 128 of them scored by each CTA
constexpr int kVSlab = 32 * 128;        // 64 dims of 32 keys
constexpr int kVUnit = 4 * kVSlab;      // a CTA's 256 dims of 32 keys: 16 KB
constexpr int kUnits = T / 32;          // of a tile
constexpr int kQSlabs = 9;
constexpr int kRowTiles = 4;            // tiles whose rows are looked up ahead

// Warps.  Those that work on TMEM lanes 32 q ... are warps q modulo 4.
constexpr int kVWarp0 = 8, kSoftmaxWarp0 = 16, kQkWarp = 24, kPvWarp = 25, kRelayWarp = 26, kRowsWarp = 27;
constexpr int kSoftmaxWarps = 8, kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kThreads = 28 * 32;
constexpr int kLaunchRegs = 72;         // a thread

template <int N>
struct Layout {
  // Registers a thread of each group of four warps, of the launch's 72.
  static constexpr int kKRegs = N <= 64 ? 80 : 64, kVRegs = N <= 64 ? 80 : 64;
  static constexpr int kSoftmaxRegs = N <= 64 ? 64 : 104, kOtherRegs = N <= 64 ? 56 : 40;
  static_assert(2 * kKRegs + 2 * kVRegs + 2 * kSoftmaxRegs + kOtherRegs <= 7 * kLaunchRegs, "no more than the launch gives");
  static constexpr int kRows = N / 2;        // query rows that a CTA holds for the MMAs
  static constexpr int kVUnits = N <= 64 ? 4 : 3;  // in the ring of V
  static constexpr int kSBufs = N <= 64 ? 2 : 1;   // tiles of scores: what TMEM holds
  static constexpr int kPBufs = 2;           // tiles of weights (one: 175 us instead of 155)
  static constexpr int kQSlab = kRows * 128;
  static constexpr int kP = T * kRows * 2;   // a tile's weights of the CTA's rows
  static constexpr int OFF_V = 0;
  static constexpr int OFF_Q = OFF_V + kVUnits * kVUnit;
  static constexpr int OFF_P = OFF_Q + kQSlabs * kQSlab;
  static constexpr int OFF_X = OFF_P + kPBufs * kP;
  // [4][N] maxima or sums, then [N] each: the partner's maxima, its sums, minus the
  // running maxima, factors of O, the scores that raise them, visible keys; votes
  static constexpr int OFF_ROWS = OFF_X + 10 * N * 4 + 128;  // row indices of kRowTiles tiles
  static constexpr int OFF_BAR = OFF_ROWS + kRowTiles * T * 4;
  static constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;
  // TMEM columns: O^T (2 blocks of N), scores, and K as f16 pairs: a ring of slabs of
  // 128 dims (64 columns), 5 a tile, the last one half as long.
  static constexpr uint32_t TM_O = 0, TM_S = 2 * N, TM_K = (2 + kSBufs) * N;
  static constexpr int kKSlabs = (512 - (2 + kSBufs) * N) / 64;  // 2 or 4
  static_assert((kKSlabs & (kKSlabs - 1)) == 0 && kKSlabs <= 8 && kVUnits <= 4, "barriers");
  static_assert(SMEM_BYTES <= 232448 && OFF_Q % 1024 == 0 && OFF_P % 1024 == 0 && OFF_BAR % 8 == 0, "fits");
};

constexpr float kRescaleThreshold = 8.0f;
constexpr float kMaxSentinel = -1.0e30f;
constexpr uint64_t kDrainNs = 500000000ull;
constexpr uint64_t kSettleNs = 50000;  // far longer than a store to the partner takes
constexpr uint32_t kSleepNs = 20000;

// Barriers marked "0" are waited on in the even CTA, which issues the MMAs; both
// CTAs' warps arrive there.  The MMAs' own arrivals go to both CTAs.
struct Bars {
  uint64_t rows_full[kRowTiles];   // a tile's rows are looked up
  uint64_t rows_empty[kRowTiles];  // and taken by the K and V warps
  uint64_t k_full[8];    // 0: K's slab is in TMEM (eight warps of each CTA)
  uint64_t k_empty[8];   // the scores of a slab are done
  uint64_t v_full[4];    // 0: V of 32 keys is in shared memory (four warps of each)
  uint64_t v_empty[4];   // and used
  uint64_t s_full[2];    // scores done
  uint64_t s_free[2];    // 0: scores read (eight warps of each)
  uint64_t p_full[2];    // 0: weights written, O rescaled (eight warps and the relay of each)
  uint64_t p_done[2];    // the tile's values are summed
  uint64_t recv[2];      // the partner's weights of this CTA's rows have landed
  uint64_t vote[2];      // all sixteen warps' votes on the tile
  uint64_t raise;        // the softmax warps are here
  uint64_t max_full;     // the partner's maxima
  uint64_t sum_full;     // its sums
  uint64_t q_ready;      // 0: Q is in shared memory (eight warps of each)
  uint64_t drain[2];
  uint32_t tmem_base;
  int32_t abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");
// The address in shared memory of barrier i of those called `name`.
#define BAR(name, i) (sbase + L::OFF_BAR + (uint32_t)offsetof(Bars, name) + 8 * (i))

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) { return __uint_as_float(ld_shared_u32(addr)); }
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) { st_shared_u32(addr, __float_as_uint(v)); }

struct Ctx {
  int32_t* status;
  uint64_t limit_ns;
  uint32_t abort;  // the CTA's word, set when a wait ran out
};

// Bounded wait: false if the phase did not complete in time or another warp gave up.
__device__ __forceinline__ bool wait(const Ctx& c, uint32_t bar, uint32_t parity) {
  if (ptx::mbar_test_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
    if (ptx::mbar_try_wait_sleep(bar, parity, (uint32_t)min(c.limit_ns, (uint64_t)kSleepNs))) return true;
    if (ld_shared_u32(c.abort) != 0) return false;
    if (ptx::globaltimer_ns() - t0 > c.limit_ns) {
      atomicOr(c.status, MLA_DEVFLAG_TIMEOUT);
      st_shared_u32(c.abort, 1);
      return false;
    }
  }
}

__device__ __forceinline__ bool wait_all(const Ctx& c, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(c, bar, parity));
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ void st_shared_u4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}


// 16 consecutive TMEM columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}

// The ring position and phase of the u-th of a sequence of units.
template <int R>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int by = 1) {
    slot += by;
    if (slot >= R) {
      slot -= R;
      phase ^= 1u;
    }
  }
};

// D[tmem] (+)= A[tmem] * B[smem desc]^T over the pair, A K-major in TMEM.
__device__ __forceinline__ void mma_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same on a barrier that the partner's warps arrive on, too.
__device__ __forceinline__ bool wait_pair(const Ctx& c, uint32_t bar, uint32_t parity) {
  if (!wait_all(c, bar, parity)) return false;
  ptx::mbar_acquire_cluster(bar, parity);
  return true;
}

// A barrier of the CTA's softmax warps.
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, 256;" ::: "memory"); }

// This warp group's share of the launch's registers from here on.
template <int kRegs>
__device__ __forceinline__ void take_registers() {
  if constexpr (kRegs > kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
  if constexpr (kRegs < kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Loads that stay where they are written, ahead of the conversion that they feed.  (Plain
// ones: the newest rows may come from the kernel that this one is launched behind.)
__device__ __forceinline__ uint4 ld_ahead_u4(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_ahead_u32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_ahead_u16(const void* p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ void st_shared_u2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void tmem_ld16f(uint32_t addr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 16 lanes x 32 TMEM columns: thread i holds columns 8 j + 2 (i % 4) + e of lane i / 4 in
// r[4 j + e], and of lane i / 4 + 8 in r[4 j + 2 + e].
__device__ __forceinline__ void tmem_st16x256b_x4(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

template <int N>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fwd_fp4_wide_kernel(mla::FwdParams p) {
  using L = Layout<N>;
  constexpr int R = L::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem + L::OFF_BAR);
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const uint32_t peer = rank ^ 1u;

  // The work unit: (sequence b, row block rb, key range [k0, k1)), its context, and
  // where its result goes, as in the 128-row kernel.
  int rb, b, ctx, k0, k1;
  bool single;
  size_t part;
  if (p.units != nullptr) {
    // Both CTAs of a pair read the same unit and take the same branches.
    ptx::grid_dependency_wait();
    const int u = blockIdx.x >> 1;
    if (u >= *p.n_units) return;
    const int4 d = p.units[u];
    const int4 si = p.seq_info[d.x];
    b = d.x;
    rb = d.y & 0xFF;
    k0 = d.z;
    k1 = d.w;
    ctx = si.x;
    single = si.z == 1;
    part = (size_t)si.y + (d.y >> 8);
  } else {
    rb = blockIdx.x >> 1;
    b = blockIdx.y;
    const int split = blockIdx.z;
    ctx = p.seq_lens[b];
    if (ctx < 0 || ctx > p.max_ctx) {
      if (threadIdx.x == 0 && rank == 0 && split == 0) atomicOr(p.status, MLA_DEVFLAG_CTX_RANGE);
      ctx = ctx < 0 ? 0 : p.max_ctx;
    }
    k0 = p.key_begin + split * p.chunk_len;
    k1 = min(k0 + p.chunk_len, ctx);
    single = p.num_splits == 1 && !p.partials;
    part = (size_t)b * p.num_splits + split;
  }
  const int row0 = rb * mla::kRowTile;
  const int n_rows = min(p.rows - row0, N);
  const int n_tiles = k1 > k0 ? (k1 - k0 + T - 1) / T : 0;
  const int vdim0 = (int)rank * 256;  // this CTA's value dims
  const float s_kv = p.kv_scale ? *p.kv_scale : 1.f;

  if (n_tiles == 0) {
    // Both CTAs of the pair take this branch together, before any cluster traffic.
    ptx::grid_dependency_wait();
    for (int i = threadIdx.x; i < n_rows * 32; i += kThreads) {
      const size_t row = row0 + (i >> 5);
      if (single) {
        reinterpret_cast<uint4*>(p.out + ((size_t)b * p.rows + row) * mla::kDV + vdim0)[i & 31] = make_uint4(0, 0, 0, 0);
        if (rank == 0 && (i & 31) == 0) p.lse[(size_t)b * p.rows + row] = -INFINITY;
      } else if (rank == 0 && (i & 31) == 0) {
        p.part_lse[part * p.rows + row] = -INFINITY;
      }
    }
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      ptx::mbar_init(BAR(k_full, i), 16);
      ptx::mbar_init(BAR(k_empty, i), 1);
    }
    for (int i = 0; i < L::kVUnits; ++i) {
      ptx::mbar_init(BAR(v_full, i), 8);
      ptx::mbar_init(BAR(v_empty, i), 1);
    }
    for (int i = 0; i < kRowTiles; ++i) {
      ptx::mbar_init(BAR(rows_full, i), 1);
      ptx::mbar_init(BAR(rows_empty, i), kSoftmaxWarp0);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(BAR(s_full, i), 1);
      ptx::mbar_init(BAR(s_free, i), 2 * kSoftmaxWarps);
      ptx::mbar_init(BAR(p_full, i), 2 * kSoftmaxWarps + 2);
      ptx::mbar_init(BAR(p_done, i), 1);
      ptx::mbar_init(BAR(recv, i), 1);
      ptx::mbar_init(BAR(vote, i), 1);
      ptx::mbar_init(BAR(drain, i), 1);
    }
    ptx::mbar_init(BAR(raise, 0), kSoftmaxWarps);
    ptx::mbar_init(BAR(max_full, 0), 1);
    ptx::mbar_init(BAR(sum_full, 0), 1);
    ptx::mbar_init(BAR(q_ready, 0), 2 * kSoftmaxWarps);
    bars.abort = 0;
    ptx::fence_mbar_init_cluster();
  }
  if (warp == kQkWarp) {
    ptx::tmem_alloc_pair(BAR(tmem_base, 0), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync_all();  // barriers of both CTAs initialised before any remote arrive
  ptx::tc_fence_after();
  ptx::grid_dependency_wait();
  const uint32_t tmem = bars.tmem_base;
  const Ctx c{p.status, p.wait_ns, BAR(abort, 0)};
  // One lane's arrival, for its warp, on a barrier of the even CTA.
  auto arrive0 = [&](uint32_t bar) {
    __syncwarp();
    if (lane == 0) {
      if (rank == 0) ptx::mbar_arrive(bar);
      else ptx::mbar_arrive_cluster(ptx::mapa(bar, 0));
    }
  };

  const uint8_t* cache = static_cast<const uint8_t*>(p.cache);
  auto row_addr = [&](int t, int key) { return sbase + L::OFF_ROWS + 4 * ((t % kRowTiles) * T + key); };
  auto rows_wait = [&](int t) { return wait_all(c, BAR(rows_full, t % kRowTiles), (t / kRowTiles) & 1); };
  auto rows_taken = [&](int t) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(BAR(rows_empty, t % kRowTiles));
  };

  if (warp < kVWarp0) {
    take_registers<L::kKRegs>();
    // ----------------------------------------------------------------- K ---
    // 16 keys a warp, of the CTA's half of every tile.  Four lanes read a key, so that a
    // load touches 8 rows, not 32 (with a key a lane a tile took a fifth longer): lane c
    // of a quad takes dims 32 c .. of each 128, dims 16 c .. of the rope ones.  In the
    // TMEM store's layout it owns four of each 16 dims that an MMA contracts, so MMA j of
    // a slab sums over dims 32 c + 4 j .. + 3 (c = 0 .. 3), those four later over the same
    // + 16: Q is laid out in that order.
    const int key0 = 32 * (warp & 3) + 16 * (warp >> 2) + (lane >> 2), cq = lane & 3;  // and key0 + 8
    const uint32_t kcol = tmem + ((uint32_t)(32 * (warp & 3) + 16 * (warp >> 2)) << 16) + L::TM_K;
    // A row in six blocks, two ahead: four of 128 dims, then the rope dims of key0 and
    // those of key0 + 8.
    struct Block {
      uint4 x[2];
      uint32_t s[2];  // two scales
    } b0, b1;
    uint32_t row[2];
    auto take_rows = [&](int t) -> bool {
      if (!rows_wait(t)) return false;
#pragma unroll
      for (int o = 0; o < 2; ++o) row[o] = ld_shared_u32(row_addr(t, 128 * rank + key0 + 8 * o));
      rows_taken(t);
      return true;
    };
    auto fetch = [&](int i, Block& to) {
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const uint8_t* at = cache + (size_t)row[i < 4 ? o : i - 4] * fp4::kRow;
        if (i < 4) {
          to.x[o] = ld_ahead_u4(at + 64 * i + 16 * cq);
          to.s[o] = ld_ahead_u16(at + fp4::kScales + 8 * i + 2 * cq);
        } else {
          to.x[o] = ld_ahead_u4(at + fp4::kRope + 32 * cq + 16 * o);
        }
      }
    };
    bool ok = take_rows(0);
    if (ok) {
      fetch(0, b0);
      fetch(1, b1);
    }
    uint32_t n = 0;  // slabs so far
    for (int t = 0; ok && t < n_tiles; ++t) {
#pragma unroll
      for (int i = 0; i < 5; ++i, ++n) {
        const uint32_t slot = n % L::kKSlabs, column = kcol + 64 * slot;
        ok = ok && (n < L::kKSlabs || wait_all(c, BAR(k_empty, slot), (n / L::kKSlabs - 1) & 1));
        ptx::tc_fence_after();
        if (i < 4) {
          Block& at = i & 1 ? b1 : b0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t r[16];
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const uint4& x = at.x[o];
              const uint32_t sc = fp4::scale_pair(at.s[o], e);
              const uint4 lo = fp4::scaled(e ? x.z : x.x, sc), hi = fp4::scaled(e ? x.w : x.y, sc);
              r[2 * o] = lo.x;
              r[2 * o + 1] = lo.y;
              r[2 * o + 4] = lo.z;
              r[2 * o + 5] = lo.w;
              r[2 * o + 8] = hi.x;
              r[2 * o + 9] = hi.y;
              r[2 * o + 12] = hi.z;
              r[2 * o + 13] = hi.w;
            }
            tmem_st16x256b_x4(column + 32 * e, r);
          }
          fetch(i + 2, at);
        } else {
          const uint4 &a0 = b0.x[0], &a1 = b0.x[1], &c0 = b1.x[0], &c1 = b1.x[1];
          const uint32_t r[16] = {a0.x, a0.y, c0.x, c0.y, a0.z, a0.w, c0.z, c0.w,
                                  a1.x, a1.y, c1.x, c1.y, a1.z, a1.w, c1.z, c1.w};
          tmem_st16x256b_x4(column, r);
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        if (ok) arrive0(BAR(k_full, slot));
      }
      if (t + 1 < n_tiles && (ok = ok && take_rows(t + 1))) {
        fetch(0, b0);
        fetch(1, b1);
      }
    }
  } else if (warp < kSoftmaxWarp0) {
    take_registers<L::kVRegs>();
    // ----------------------------------------------------------------- V ---
    // Two groups of four warps take turns, 32 keys each; 8 keys a warp, four lanes a key:
    // lane c of a quad has dims 64 c .. (a slab) of the CTA's 256.  The loads are two of
    // the group's units ahead.
    const int group = (warp - kVWarp0) >> 2;
    const int key0 = 8 * (warp & 3) + (lane >> 2), cq = lane & 3;
    const int n_units = kUnits * n_tiles;
    // The four slabs lie a multiple of 128 bytes apart, so the lanes of a quad write
    // their pieces of 8 dims in different orders (piece i is the lane's i ^ 2 c): the
    // eight lanes that store together then hit different banks.
    const uint32_t order = cq == 0 ? 0x3210u : cq == 1 ? 0x2301u : cq == 2 ? 0x1032u : 0x0123u;
    const int first = 128 * (int)rank + 32 * cq + 16 * (cq >> 1), second = (cq & 2) ? -16 : 16;
    const int its_scales = fp4::kScales + 16 * (int)rank + 4 * cq - first;
    const uint8_t* codes = cache + first;
    struct Codes {
      uint4 x[2];
      uint32_t s;
    } c0, c1;
    auto fetch = [&](int u, Codes& to) -> bool {
      const int t = u / kUnits;
      if (u % kUnits == group && !rows_wait(t)) return false;
      const uint8_t* row = codes + (size_t)ld_shared_u32(row_addr(t, 32 * (u % kUnits) + key0)) * fp4::kRow;
      if (u % kUnits == group + kUnits - 2) rows_taken(t);
      to.x[0] = ld_ahead_u4(row);
      to.x[1] = ld_ahead_u4(row + second);
      to.s = ld_ahead_u32(row + its_scales);
      return true;
    };
    Ring<L::kVUnits> ring;
    ring.next(group);
    auto step = [&](int u, Codes& from) -> bool {
      if (u >= L::kVUnits && !wait_all(c, BAR(v_empty, ring.slot), ring.phase ^ 1u)) return false;
      const uint32_t dst = sbase + L::OFF_V + ring.slot * kVUnit + cq * kVSlab + key0 * 128;
      const uint32_t scales = __byte_perm(from.s, 0u, order);
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // 32 dims
        uint4 x[4];
        const uint4& in = from.x[i];
        const bool odd = cq & 1;
        fp4::convert(make_uint4(odd ? in.z : in.x, odd ? in.w : in.y, odd ? in.x : in.z, odd ? in.y : in.w),
                     scales >> (16 * i), x);
#pragma unroll
        for (int e = 0; e < 4; ++e) st_shared_u4(dst + (((4 * i + e) ^ (2 * cq) ^ (key0 & 7)) * 16), x[e]);
      }
      ptx::fence_proxy_async_smem();
      arrive0(BAR(v_full, ring.slot));
      ring.next(2);
      return u + 4 >= n_units || fetch(u + 4, from);
    };
    if (fetch(group, c0) && fetch(group + 2, c1))
      for (int u = group; u < n_units; u += 4)
        if (!step(u, c0) || !step(u + 2, c1)) break;
  } else if (warp < kQkWarp) {
    take_registers<L::kSoftmaxRegs>();
    // ----------------------------------------------------------- softmax ---
    // A key a thread (TMEM lane tid), rows [R h, R h + R): those that the MMAs take
    // from CTA h's shared memory, where this warp's weights go.
    const int q = warp & 3, h = (warp - kSoftmaxWarp0) >> 2;
    const int tid = 32 * q + lane, st = threadIdx.x - 32 * kSoftmaxWarp0;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const bool away = (uint32_t)h != rank;
    auto at = [&](int array, int i) { return sbase + L::OFF_X + 4 * (array * N + i); };
    constexpr int kPartnerMax = 4, kPartnerSum = 5, kMinusMax = 6, kFactor = 7, kTop = 8, kVisible = 9, kVotes = 10;
    const uint32_t nm_at = at(kMinusMax, R * h), top_at = at(kTop, R * h);
    // Q to f16, K-major: this CTA's R rows, 72 pieces of 8 dims each; rows past the
    // problem's are zero.
    {
      bool range = false;
      constexpr int kPieces = N <= 64 ? 9 : 6;  // in flight a thread
      static_assert(R * 72 % (kPieces * kSoftmaxThreads) == 0, "whole rounds");
#pragma unroll 1
      for (int i0 = st; i0 < R * 72; i0 += kPieces * kSoftmaxThreads) {
        uint4 x[kPieces];
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          const int i = i0 + kSoftmaxThreads * j, r = i / 72, ch = i - 72 * r, row = R * (int)rank + r;
          x[j] = make_uint4(0, 0, 0, 0);
          if (row < n_rows) x[j] = reinterpret_cast<const uint4*>(p.q + ((size_t)b * p.rows + row0 + row) * mla::kDQK)[ch];
        }
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          const int i = i0 + kSoftmaxThreads * j, r = i / 72, ch = i - 72 * r;
          uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xFFFF0000u);
            range |= fabsf(lo) > 65504.f || fabsf(hi) > 65504.f;
            w[e] = pack_f16(lo, hi);
          }
#pragma unroll
          for (int f = 0; f < 2; ++f) {  // four dims at a time, in the order that K has
            const int d = 8 * ch + 4 * f, jj = (d >> 2) & 3;
            const int slab = d < 512 ? 2 * (d >> 7) + ((d >> 4) & 1) : 8, cq = d < 512 ? (d >> 5) & 3 : (d >> 4) & 3;
            st_shared_u2(sbase + L::OFF_Q + slab * L::kQSlab + r * 128 + (((2 * jj + (cq >> 1)) ^ (r & 7)) * 16) + 8 * (cq & 1),
                         w[2 * f], w[2 * f + 1]);
          }
        }
      }
      if (range) atomicOr(p.status, MLA_DEVFLAG_Q_RANGE);
      ptx::fence_proxy_async_smem();
      arrive0(BAR(q_ready, 0));
    }
    auto visible = [&](int r) {  // keys before it are seen by row r
      const int tok = (row0 + r) / p.heads;
      const int n = p.causal ? ctx - p.sq + tok + 1 : ctx;
      return min(max(0, min(n, ctx)), k1);
    };
    if (st < N) {
      const int n = st < n_rows ? visible(st) : 0;
      st_shared_u32(at(kVisible, st), n > k0 ? n : 0);  // 0: none of this unit's
      st_shared_f32(at(kMinusMax, st), -kMaxSentinel);
      st_shared_f32(at(kTop, st), kRescaleThreshold + kMaxSentinel);
    }
    const int all_see = visible(0);  // by every row: the first one sees the fewest
    softmax_sync();

    const float c2 = p.softmax_scale * s_kv * 1.4426950408889634f;
    constexpr int kMine = R / 32;
    float l[kMine] = {};  // the warp's part of the sums of rows row_of_sum + i
    const int row_of_sum = kMine * lane;
    constexpr int G = R / 16;
    uint32_t raises = 0;
    // A barrier of the eight warps, for the tiles that raise the maxima.
    uint32_t syncs = 0;
    auto raise_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(BAR(raise, 0));
      return wait_all(c, BAR(raise, 0), syncs++ & 1);
    };
    // No barrier here that a wait that ran out could leave short: from then on a warp only
    // walks to the end of the loop.
    bool ok = true;
    for (int t = 0; ok && t < n_tiles; ++t) {
      const int buf = t & 1, sb = t % L::kSBufs;
      ok = wait_all(c, BAR(s_full, sb), (t / L::kSBufs) & 1);
      if (!ok) break;
      ptx::tc_fence_after();
      // The scores to registers at once, so that the next tile's can follow.
      float s[R];
#pragma unroll
      for (int g = 0; g < G; ++g) tmem_ld16f(tmem + lanes + L::TM_S + sb * N + R * h + 16 * g, s + 16 * g);
      ptx::tmem_ld_wait();
      ptx::tc_fence_before();
      arrive0(BAR(s_free, sb));
      const int first = k0 + t * T + 128 * (int)rank, key = first + tid;
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] *= c2;
      if (first + 128 > all_see) {
#pragma unroll
        for (int r = 0; r < R; ++r) s[r] = key < (int)ld_shared_u32(at(kVisible, R * h + r)) ? s[r] : -INFINITY;
      }
      bool over = false;
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const float4 m = ld_shared_f4(top_at + 4 * r);
        over |= s[r] > m.x | s[r + 1] > m.y | s[r + 2] > m.z | s[r + 3] > m.w;
      }
      // All sixteen warps raise a tile's maxima or none does: O sums over the keys of both CTAs.
      const bool mine = __any_sync(0xffffffffu, over);
      if (lane < 2)  // each warp's vote goes to both CTAs, 16 words a tile
        ptx::st_async_b32(ptx::mapa(at(kVotes, 16 * buf + 8 * rank + (warp - kSoftmaxWarp0)), lane),
                          mine ? 1u : 0u, ptx::mapa(BAR(vote, buf), lane));
      if (st == 0) ptx::mbar_arrive_expect_tx(BAR(vote, buf), 4 * 2 * kSoftmaxWarps);
      ok = wait_all(c, BAR(vote, buf), (t >> 1) & 1);
      if (!ok) break;
      if (__any_sync(0xffffffffu, ld_shared_u32(at(kVotes, 16 * buf + (lane & 15))) != 0)) {
        // New maxima: of each row over the tile, kept where they are no higher.
#pragma unroll
        for (int r = 0; r < R; ++r) {
          // the order of signed integers, a NaN left out
          const int x = __float_as_int(fmaxf(s[r], -INFINITY));
          const int m = __reduce_max_sync(0xffffffffu, x ^ ((x >> 31) & 0x7FFFFFFF));
          if (lane == 0) st_shared_u32(at(q, R * h + r), m ^ ((m >> 31) & 0x7FFFFFFF));
        }
        ok = raise_sync();
        float m = 0.f;
        if (ok && st < N) {
          m = fmaxf(fmaxf(ld_shared_f32(at(0, st)), ld_shared_f32(at(1, st))),
                    fmaxf(ld_shared_f32(at(2, st)), ld_shared_f32(at(3, st))));
          ptx::st_async_b32(ptx::mapa(at(kPartnerMax, st), peer), __float_as_uint(m),
                            ptx::mapa(BAR(max_full, 0), peer));
          if (st == 0) ptx::mbar_arrive_expect_tx(BAR(max_full, 0), 4 * N);
        }
        ok = ok && wait_all(c, BAR(max_full, 0), raises & 1);
        if (ok && st < N) {
          const float old = ld_shared_f32(at(kMinusMax, st));
          const float to = fminf(old, -fmaxf(m, ld_shared_f32(at(kPartnerMax, st))));
          st_shared_f32(at(kFactor, st), exp2f(to - old));
          st_shared_f32(at(kMinusMax, st), to);
          st_shared_f32(at(kTop, st), kRescaleThreshold - to);
        }
        if (t > 0)  // O is the tile before's
          ok = ok && wait_all(c, BAR(p_done, (t - 1) % L::kPBufs), ((t - 1) / L::kPBufs) & 1);
        ok = ok && raise_sync();
        ++raises;
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int i = 0; i < kMine; ++i) l[i] *= ld_shared_f32(at(kFactor, R * h + row_of_sum + i));
        if (t > 0) {
#pragma unroll 1
          for (int i = 0; i < 4 * G; ++i) {  // 8 columns at a time
            uint32_t o[8];
            const int r0 = 8 * (i % (2 * G));
            const uint32_t col = tmem + lanes + L::TM_O + (i / (2 * G)) * N + R * h + r0;
            tmem_ld8(col, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * ld_shared_f32(at(kFactor, R * h + r0 + j)));
            tmem_st8(col, o);
          }
          ptx::tmem_st_wait();
        }
      }
      // The weights' buffer is free, here and at the partner, once its last tile's values are summed.
      const int pb = t % L::kPBufs;
      if (t >= L::kPBufs) ok = wait_all(c, BAR(p_done, pb), (t / L::kPBufs - 1) & 1);
      if (!ok) break;
      const int kk = 128 * (int)rank + tid;
      const uint32_t recv = ptx::mapa(BAR(recv, pb), peer);
      uint32_t to = sbase + L::OFF_P + pb * L::kP + (kk >> 3) * (16 * R) + (kk & 7) * 16;
      if (away) to = ptx::mapa(to, peer);
#pragma unroll
      for (int g = 0; g < R / 8; ++g) {
        uint32_t w[4];
#pragma unroll
        for (int r = 0; r < 8; r += 4) {
          const float4 m = ld_shared_f4(nm_at + (8 * g + r) * 4);
          s[8 * g + r] = fast_exp2(s[8 * g + r] + m.x);
          s[8 * g + r + 1] = fast_exp2(s[8 * g + r + 1] + m.y);
          s[8 * g + r + 2] = fast_exp2(s[8 * g + r + 2] + m.z);
          s[8 * g + r + 3] = fast_exp2(s[8 * g + r + 3] + m.w);
          w[r / 2] = pack_f16(s[8 * g + r], s[8 * g + r + 1]);
          w[r / 2 + 1] = pack_f16(s[8 * g + r + 2], s[8 * g + r + 3]);
        }
        if (away) ptx::st_async_u4(to + g * 128, w[0], w[1], w[2], w[3], recv);
        else st_shared_u4(to + g * 128, make_uint4(w[0], w[1], w[2], w[3]));
      }
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      arrive0(BAR(p_full, pb));
      // The warp's sums over its 32 keys: half of the rows go to the lane across, five
      // times, so that a lane ends with the sums of R / 32 rows (sums of R rows in every
      // thread, added up at the end, would be R registers).
#pragma unroll
      for (int half = R / 2, across = 16; across > 0; half >>= 1, across >>= 1) {
        const bool upper = lane & across;
#pragma unroll
        for (int r = 0; r < half; ++r) {
          const float keep = upper ? s[r + half] : s[r], give = upper ? s[r] : s[r + half];
          s[r] = keep + __shfl_xor_sync(0xffffffffu, give, across);
        }
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i) l[i] += s[i];
    }

    // ---------------------------------------------------------- epilogue ---
    softmax_sync();  // xmax's last readers
#pragma unroll
    for (int i = 0; i < kMine; ++i) st_shared_f32(at(q, R * h + row_of_sum + i), l[i]);
    softmax_sync();
    float sum = 0.f;
    if (st < N) {
      sum = ld_shared_f32(at(0, st)) + ld_shared_f32(at(1, st)) + ld_shared_f32(at(2, st)) + ld_shared_f32(at(3, st));
      ptx::st_async_b32(ptx::mapa(at(kPartnerSum, st), peer), __float_as_uint(sum),
                        ptx::mapa(BAR(sum_full, 0), peer));
      if (st == 0) ptx::mbar_arrive_expect_tx(BAR(sum_full, 0), 4 * N);
    }
    ok = ok && wait_all(c, BAR(sum_full, 0), 0);
    if (st < N) {
      sum += ld_shared_f32(at(kPartnerSum, st));  // the same in both CTAs
      // keys whose scores are all -inf, not a row without any
      if (sum == 0.f && ld_shared_u32(at(kVisible, st)) != 0) sum = NAN;
      st_shared_f32(at(kFactor, st), sum == 0.f ? 0.f : s_kv / sum);
      if (ok && rank == 0 && st < n_rows) {
        const float lse = sum == 0.f ? -INFINITY : (log2f(sum) - ld_shared_f32(at(kMinusMax, st))) * 0.6931471805599453f;
        if (single) p.lse[(size_t)b * p.rows + row0 + st] = lse;
        else p.part_lse[part * p.rows + row0 + st] = lse;
      }
    }
    softmax_sync();
    if (ok && wait_all(c, BAR(p_done, (n_tiles - 1) % L::kPBufs), ((n_tiles - 1) / L::kPBufs) & 1)) {
      ptx::tc_fence_after();
#pragma unroll 1
      for (int dg = 0; dg < 2 * G; ++dg) {  // 16 rows at a time; lane: dim 128 d + tid
        const int d = dg / G, r0 = R * h + 16 * (dg % G);
        uint32_t o[16];
        tmem_ld16(tmem + lanes + L::TM_O + d * N + r0, o);
        ptx::tmem_ld_wait();
        const int dim = vdim0 + 128 * d + tid;
        if (single) {
          uint16_t* out = p.out + ((size_t)b * p.rows + row0 + r0 + (lane & 1)) * mla::kDV + (dim & ~1);
#pragma unroll
          for (int r = 0; r < 16; r += 2) {
            // even lanes store row r's two dims, odd lanes row r + 1's
            const float a = __uint_as_float(o[r]) * ld_shared_f32(at(kFactor, r0 + r));
            const float b2 = __uint_as_float(o[r + 1]) * ld_shared_f32(at(kFactor, r0 + r + 1));
            const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? a : b2, 1);
            if (r0 + r + (lane & 1) < n_rows)
              *reinterpret_cast<uint32_t*>(out + r * mla::kDV) = (lane & 1) ? pack_bf16(got, b2) : pack_bf16(a, got);
          }
        } else {
          float* out = p.part_o + (part * p.rows + row0 + r0) * mla::kDV + dim;
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (r0 + r < n_rows) out[r * mla::kDV] = __uint_as_float(o[r]) * ld_shared_f32(at(kFactor, r0 + r));
        }
      }
    }
  } else {
    take_registers<L::kOtherRegs>();
    if (warp == kQkWarp && rank == 0) {
      // -------------------------------------------------------------- QK ---
      // The whole warp walks the loop, one lane issues: in a branch that one lane
      // takes alone an MMA costs about 64 cycles to issue.
      const bool leader = ptx::elect_one();
      constexpr uint32_t id_qk = ptx::idesc_f16(256, N, 0, false, false);
      const uint64_t dq = ptx::smem_desc(sbase + L::OFF_Q, 16, 1024, 2);  // K-major, 128-byte swizzle
      bool ok = wait_pair(c, BAR(q_ready, 0), 0);
      uint32_t n = 0;  // slabs so far
      for (int t = 0; ok && t < n_tiles; ++t) {
        const int sb = t % L::kSBufs;
        if (t >= L::kSBufs) ok = wait_pair(c, BAR(s_free, sb), (t / L::kSBufs - 1) & 1);
        const uint32_t d = tmem + L::TM_S + sb * N;
#pragma unroll 1
        for (int a = 0; a < kQSlabs; a += 2, ++n) {
          const uint32_t slot = n % L::kKSlabs;
          ok = ok && wait_pair(c, BAR(k_full, slot), (n / L::kKSlabs) & 1);
          ptx::tc_fence_after();
          if (ok && leader) {
            const uint32_t k = tmem + L::TM_K + 64 * slot;
            const uint64_t qa = dq + (uint32_t)(a * L::kQSlab / 16);
#pragma unroll
            for (int s = 0; s < 4; ++s) mma_ts_pair(d, k + 8 * s, qa + 2 * s, id_qk, (a | s) != 0);
            if (a + 1 < kQSlabs) {
#pragma unroll
              for (int s = 0; s < 4; ++s) mma_ts_pair(d, k + 32 + 8 * s, qa + L::kQSlab / 16 + 2 * s, id_qk, 1);
            } else {
              ptx::mma_commit_pair(BAR(s_full, sb));
            }
            ptx::mma_commit_pair(BAR(k_empty, slot));
          }
          __syncwarp();
        }
      }
    } else if (warp == kPvWarp && rank == 0) {
      // -------------------------------------------------------------- PV ---
      const bool leader = ptx::elect_one();
      constexpr uint32_t id_pv = ptx::idesc_f16(256, N, 0, true, true);
      // V: dims contiguous, 64-dim slabs kVSlab apart, 8-key groups 1 KB apart.  P: rows
      // contiguous in groups of 8, no swizzle; a group of 8 keys x 8 rows is 128 bytes,
      // 8-key groups lie 16 R bytes apart.
      const uint64_t dv = ptx::smem_desc(sbase + L::OFF_V, kVSlab, 1024, 2);
      const uint64_t dp = ptx::smem_desc(sbase + L::OFF_P, 16 * R, 128, 0);
      bool ok = true;
      Ring<L::kVUnits> unit;
      for (int u = 0; ok && u < kUnits * n_tiles; ++u, unit.next()) {
        const int t = u / kUnits, i = u % kUnits;
        ok = (i != 0 || wait_pair(c, BAR(p_full, t % L::kPBufs), (t / L::kPBufs) & 1)) &&
             wait_pair(c, BAR(v_full, unit.slot), unit.phase);
        ptx::tc_fence_after();
        if (ok && leader) {
          const uint64_t a = dv + unit.slot * (kVUnit / 16);
          const uint64_t w = dp + (t % L::kPBufs * L::kP + i * 64 * R) / 16;
#pragma unroll
          for (int s = 0; s < 2; ++s)  // 16 keys
#pragma unroll
            for (int d = 0; d < 2; ++d)
              ptx::mma_ss_pair(tmem + L::TM_O + d * N, a + (d * 2 * kVSlab + s * 2048) / 16, w + s * 2 * R, id_pv, (u | s) != 0);
          ptx::mma_commit_pair(BAR(v_empty, unit.slot));
          if (i == kUnits - 1) ptx::mma_commit_pair(BAR(p_done, t % L::kPBufs));
        }
        __syncwarp();
      }
    } else if (warp == kRelayWarp) {
      // ----------------------------------------------------------- relay ---
      // The partner's weights: once they have landed the MMAs may read them.
      for (int t = 0; t < n_tiles; ++t) {
        const uint32_t bar = BAR(recv, t % L::kPBufs);
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar, 128 * R * 2);
        if (!wait_all(c, bar, (t / L::kPBufs) & 1)) break;
        ptx::fence_proxy_async_smem();
        arrive0(BAR(p_full, t % L::kPBufs));
      }
    } else if (warp == kRowsWarp) {
      // ------------------------------------------------------------ rows ---
      // Rows of the cache, up to four tiles ahead.  A key past the split's last one
      // repeats it (its weight is zero), so every row read lies in [k0, k1).
      const int32_t* bt = p.bt + (p.bt_indptr ? (size_t)p.bt_indptr[b] : (size_t)b * p.bt_stride);
      // key / page_size: Granlund and Montgomery, "Division by invariant integers using
      // multiplication" (PLDI 1994), exact for every 32-bit key
      const uint32_t pdiv = (uint32_t)p.page_size;
      const uint32_t plog = 32u - __clz(pdiv - 1u);
      const uint32_t pmul = (uint32_t)(((1ull << 32) * ((1ull << plog) - pdiv)) / pdiv) + 1u;
      const uint32_t pshift = plog > 0 ? plog - 1u : 0u;
      auto page_of = [&](uint32_t key) -> uint32_t {
        const uint32_t t = __umulhi(pmul, key);
        return pdiv == 1u ? key : (t + ((key - t) >> 1)) >> pshift;
      };
      auto page_at = [&](int key) -> int { return __ldg(&bt[page_of((uint32_t)key)]); };
      for (int t = 0; t < n_tiles; ++t) {
        const int slot = t % kRowTiles;
        if (t >= kRowTiles && !wait_all(c, BAR(rows_empty, slot), (t / kRowTiles - 1) & 1)) break;
#pragma unroll 2
        for (int i = 0; i < T / 32; ++i) {
          const int key = min(k0 + t * T + 32 * i + lane, k1 - 1);
          int64_t page = page_at(key);
          if (page < 0 || page >= p.num_pages) {
            atomicOr(p.status, MLA_DEVFLAG_BAD_PAGE);
            page = 0;
          }
          const uint32_t row = (uint32_t)page * pdiv + ((uint32_t)key - page_of((uint32_t)key) * pdiv);  // num_pages * page_size < 2^31
          st_shared_u32(row_addr(t, 32 * i + lane), row);
          // The K and V warps' loads are far enough ahead for L2's latency, not for DRAM's:
          // this CTA's keys are fetched to L2 here.
          if ((i >> 2) == (int)rank) {
            const uint8_t* at = cache + (size_t)row * fp4::kRow;
            prefetch_l2(at);
            prefetch_l2(at + 128);
            prefetch_l2(at + 256);
            prefetch_l2(at + 384);
          }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(BAR(rows_full, slot));
      }
    }
  }

  // ------------------------------------------------------------ teardown ---
  ptx::tc_fence_before();
  __syncthreads();
  if (bars.abort) {
    // Nothing is issued any more.  The MMAs in flight are waited for, and stores to
    // either CTA, or arrivals still on their way, get far longer than they take.
    if (rank == 0 && (warp == kQkWarp || warp == kPvWarp) && ptx::elect_one()) {
      const uint32_t bar = BAR(drain, warp - kQkWarp);
      ptx::mma_commit_pair(bar);
      const uint64_t start = ptx::globaltimer_ns();
      while (!ptx::mbar_try_wait(bar, 0))
        if (ptx::globaltimer_ns() - start > kDrainNs) break;
    }
    __syncwarp();
    const uint64_t start = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - start < kSettleNs) __nanosleep(1000);
    __syncthreads();
  }
  ptx::cluster_sync_all();  // no CTA leaves, or frees TMEM, while the pair still works
  if (warp == kQkWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace

int mla_launch_fwd_fp4_wide_sm103(const mla::FwdParams& p, void* stream) {
  const bool half = p.rows <= 64;
  auto kernel = half ? fwd_fp4_wide_kernel<64> : fwd_fp4_wide_kernel<128>;
  const int smem = half ? Layout<64>::SMEM_BYTES : Layout<128>::SMEM_BYTES;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  e = mla::opt_in_smem(reinterpret_cast<const void*>(kernel), smem, dev, half ? 12 : 13);
  if (e != cudaSuccess) return (int)e;
  // Splits vary slowest, so every sequence's first chunk is dispatched
  // before any second chunk (the planner simulates this order).  Launched as
  // a programmatic dependent: behind the decode epilogue the prologue
  // (barrier set-up, TMEM allocation) overlaps that kernel's tail.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = p.units != nullptr ? dim3(2 * p.unit_capacity, 1, 1)
                                  : dim3(p.row_blocks * 2, p.batch, p.num_splits);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, p);
}
