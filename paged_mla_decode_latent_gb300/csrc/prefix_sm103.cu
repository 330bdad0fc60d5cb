// prefix_sm103.cu -- decode attention over the keys that every sequence of a
// batch shares, for the query rows of the whole batch at once.
//
// The batch's B * Sq * H query rows are one [rows, 576] matrix and the shared
// keys one [P, 576] matrix, so the scores are a plain product: a key is loaded
// once per 128 rows instead of once per sequence.  Row r sees the first
// min(P, n_r) shared keys, n_r its own causal or ragged limit.  The own keys
// of the sequences in a 128-row block may follow as further tiles of that
// block (laid end to end; each row sees its own sequence's stretch), so that
// one softmax runs over both:
//
//   z_j = c <q_r, k_j>;   lse = ln sum_j e^z_j;   o = sum_j e^(z_j - lse) k_j[0:512]
//
// A row block that one pair holds is finished here; the parts of a cut one go
// to the workspace as partials (o, lse) for the merge.
//
// Queries and keys come staged: contiguous f16 rows of 576 (the staging kernel
// walks the block tables and converts the cache once, instead of once per row
// block).  f16 keeps every bf16 and e4m3 value of ordinary size exactly, and
// gives the weights 11 significant bits, so no second pass for heavy keys is
// needed.  Keys that f16 cannot hold are staged as zeros and remembered; rows
// that see one come out NaN.
//
// Rows of small values come multiplied by a power of two: a query row's is taken
// back in its own c, a key's 2^e in its score and its weight,
//
//   z_j = c 2^-e_j <q_r, k'_j>,   p_j = 2^(z_j - e_j - m),   o = sum_j p_j k'_j / sum_j p_j 2^e_j
//
// with m the running maximum of z_j - e_j, so that the weights keep their bits
// whatever the keys' magnitudes are.  Only tiles that hold such a key pay.
//
// Split over a CTA pair.  An fp32 accumulator of 128 rows x 512 value dims
// fills the TMEM of one SM, so a pair shares the 128 rows: `cta_group::2` MMAs
// with M = 128 give each CTA 64 rows and put the two halves of N on the two
// halves of its TMEM lanes.  64 rows x 512 dims are then 256 columns, a
// 256-key score tile 128 columns, and two score buffers fit beside O.  Nothing
// is exchanged between the CTAs except operands the MMA itself reads.  At N =
// 256 such an MMA runs at the full rate (64 cycles measured; N = 128: 50).
//
// Every operand streams through one ring of 16 KB slabs, each worth four MMAs
// (256 cycles): per 256-key tile and CTA 9 score slabs [128 keys x 64 dims]
// and 8 value slabs [64 keys x 128 dims].  The values are loaded again instead
// of kept from the score slabs: a slab's offset must mean the same operand in
// both CTAs, and for scores the pair splits the keys, for values the dims.
//
// Warps: 0-7 softmax (warp w: TMEM lane quarter w % 4, score columns 64 (w /
// 4) .. + 63), 8 loads, 9 (even CTA) issues the MMAs: scores of tile t + 1,
// then values of tile t, so the softmax of a tile has the length of both in
// which to finish.
//
// Work: the tiles of all row blocks laid end to end are dealt to the pairs in
// equal contiguous shares (counted on the device, since the own keys grow); a
// pair walks its segments (row block, tile range) in one launch.
//
// Every wait is bounded; one that runs out sets MLA_DEVFLAG_TIMEOUT.  Loads,
// MMAs and their commits are issued only while every wait of their warp has
// passed: a commit for MMAs that were not issued would free a slab whose copy
// has not landed, and the load warp would arm its barrier twice in one phase.
// The softmax warps, which share named barriers, run their loops to the end
// without waiting.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/mla_decode.h"
#include "internal.h"
#include "ptx.cuh"

namespace {

constexpr int T = mla::kPrefixTile;  // 256 keys per tile
constexpr int kSlots = 7;            // ring slabs
constexpr int SLAB = 16384;
constexpr int QSLAB = 64 * 128;      // 64 rows x 64 dims
constexpr int PSLAB = 64 * 128;      // 64 rows x 64 keys
constexpr int OFF_Q = 0;                          // 9 slabs, 72 KB
constexpr int OFF_P = OFF_Q + 9 * QSLAB;          // 4 slabs, 32 KB
constexpr int OFF_RING = OFF_P + 4 * PSLAB;       // 7 slabs, 112 KB
constexpr int OFF_X = OFF_RING + kSlots * SLAB;   // row maxima / sums: [2][4][64] floats
constexpr int OFF_BAR = OFF_X + 2 * 4 * 64 * 4;
constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;
static_assert(SMEM_BYTES <= 232448, "smem");

constexpr int kSoftmaxWarps = 8;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 32 * 10;

constexpr uint32_t TM_O = 0;    // 2 x 128 columns: dims 128 j .. of each value half
constexpr uint32_t TM_S = 256;  // two 128-column score buffers
constexpr uint32_t TM_COLS = 512;

// Weights are 2^(z - m + kHead) in f16: kHead leaves the weights of rows whose
// maximum is current at 2^kHead, so 21 binary orders below it keep all 11
// bits; the running maximum may lag by kLag before O is rescaled, and 2^(kHead
// + kLag) = 32768 stays below the largest f16.
//
// 11 bits put an output off by about 1e-4 in norm, against the 1.65e-3 of its
// own rounding to bf16 (the sum keeps the weights unrounded).  The decode
// kernels' two bf16 terms give heavy keys 16 bits and light ones 8; a second
// f16 term would cost eight more value slabs beside a tile's seventeen.
constexpr float kHead = 7.f, kLag = 8.f;
constexpr float kMaxSentinel = -1.0e30f;
constexpr uint64_t kDrainNs = 500000000ull;
constexpr uint64_t kSettleNs = 100000ull;
constexpr uint32_t kSleepNs = 20000;

struct Bars {
  uint64_t full[kSlots];   // slab landed in both CTAs (even CTA)
  uint64_t empty[kSlots];  // slab read by the MMAs (both)
  uint64_t q_empty;        // the segment's last score MMA is done (both)
  uint64_t s_full[2];      // scores written (both)
  uint64_t p_full;         // weights written by the 16 softmax warps of the pair (even CTA)
  uint64_t o_done;         // values of the tile accumulated (both)
  uint64_t o_free;         // the segment's O read by the 16 softmax warps (even CTA)
  uint64_t drain;
  uint32_t tmem_base;
  int32_t abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

struct Ctx {
  int32_t* status;
  volatile int32_t* abort;
  uint64_t limit_ns;
};

// A wait that does not pass at its first try.  It sleeps on its barrier
// (polling warps slow the MMA and load loops down) and reads the timer, which
// costs hundreds of cycles, only once a whole sleep has passed in vain.  Out
// of line, so that the loops around the waits stay short: with this inlined
// and the slab loops unrolled batch 64 x 8192 took 136 us against 107 (the
// instruction cache's misses, probably).
// kPoll: a limit below a sleep; every try returns at once.
template <bool kPoll>
__device__ __noinline__ bool wait_slow(const Ctx& c, uint32_t bar, uint32_t parity) {
  auto done = [&] {
    return kPoll ? ptx::mbar_test_wait(bar, parity) : ptx::mbar_try_wait_sleep(bar, parity, kSleepNs);
  };
  if (done()) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
    if (*c.abort) return false;
    if (done()) return true;
    if (ptx::globaltimer_ns() - t0 > c.limit_ns) {
      atomicOr(c.status, MLA_DEVFLAG_TIMEOUT);
      *c.abort = 1;
      return false;
    }
  }
}

// True when the phase completed; false once any wait of this CTA has run out.
template <bool kPoll>
__device__ __forceinline__ bool wait_for(const Ctx& c, uint32_t bar, uint32_t parity) {
  return (kPoll ? ptx::mbar_test_wait(bar, parity) : ptx::mbar_try_wait(bar, parity)) ||
         wait_slow<kPoll>(c, bar, parity);
}

// 2^-22 relative, far inside the 11 bits that the weights keep.
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

__device__ __forceinline__ void st_shared(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// K-major, 128B-swizzled operand (8-row groups 1 KB apart).
__device__ __forceinline__ uint64_t kdesc(uint32_t addr) { return ptx::smem_desc(addr, 16, 1024, 2); }
// MN-major values: 64-dim halves of a slab 8 KB apart, 8-key groups 1 KB apart.
__device__ __forceinline__ uint64_t vdesc(uint32_t addr) { return ptx::smem_desc(addr, 8192, 1024, 2); }

// The four warps that hold one set of 32 rows.
__device__ __forceinline__ void group_sync(int g) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory");
}

// A loaded value that is the same in every lane, as a uniform one.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// A pair's walk over its segments (the whole warp's, with loop bounds made
// uniform by a shuffle: without it batch 128 x 23333 took 517 us against 459,
// probably for the MMA loop's addresses, which then need vector registers):
// tiles [t0, t1) of row block rb, which has n.
struct Walk {
  const mla::PrefixShape& g;
  int next_rb, next_t, next_n, end_rb, end_t;
  int rb, t0, t1, n;
  __device__ __forceinline__ Walk(const mla::PrefixShape& shape, int pair) : g(shape) {
    const int4 s = g.pair_start[pair], e = g.pair_start[pair + 1];
    next_rb = uniform(s.x);
    next_t = uniform(s.y);
    next_n = uniform(s.z);
    end_rb = uniform(e.x);
    end_t = uniform(e.y);
  }
  __device__ __forceinline__ bool more() const {
    return next_rb < end_rb || (next_rb == end_rb && next_t < end_t);
  }
  __device__ __forceinline__ bool next() {
    if (!more()) return false;
    rb = next_rb;
    t0 = next_t;
    n = next_n;
    t1 = rb == end_rb ? end_t : n;
    next_rb = rb + 1;
    next_t = 0;
    if (more()) next_n = uniform(g.block_tiles[next_rb]);
    return true;
  }
  // The staged key that tile t starts at.
  __device__ __forceinline__ int key_row(int t) const {
    return t < g.tiles ? t * T : (t + rb * (g.block_keys / T)) * T;
  }
};

// The note of key i of a warp's 64 (four in each of 16 lanes, twice).
__device__ __forceinline__ uint32_t note_of(uint32_t notes, int i) {
  return __shfl_sync(0xffffffffu, notes, i / 4) >> (8 * (i % 4)) & 0xFFu;
}

// Reports the marks of a warp's 64 keys; returns the row's sum of weights, NaN
// if it sees a key that f16 cannot hold, [from, lim) being those that it sees.
// Rare, so out of line.
__device__ __noinline__ float marked_keys(const mla::PrefixShape& g, uint32_t notes, int from, int lim, float l) {
  uint32_t all = 0;
  for (int i = 0; i < 64; ++i) {
    const uint32_t f = note_of(notes, i);
    all |= f;
    if ((f & mla::kStagedRange) && i >= from && i < lim) l = NAN;
  }
  if ((threadIdx.x & 31) == 0)
    atomicOr(g.status, (all & mla::kStagedBadPage ? MLA_DEVFLAG_BAD_PAGE : 0) |
                           (all & mla::kStagedRange ? MLA_DEVFLAG_KV_RANGE : 0));
  return l;
}

constexpr uint32_t kMarks = (mla::kStagedBadPage | mla::kStagedRange) * 0x01010101u;  // of four rows

// The binary orders that a row was lifted by, and 2^e.
__device__ __forceinline__ int lift_of(uint32_t note) { return (int)(note >> mla::kStagedLift) * mla::kLiftStep; }
__device__ __forceinline__ float power2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

template <bool kPoll>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefix_kernel(mla::PrefixParams p, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem + OFF_BAR);
  const uint32_t sbase = ptx::smem_u32(smem);
  // Through a shuffle, so that the compiler can take the warp index as uniform,
  // and the MMA and load loops' addresses with it.
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1;  // the CTA's rank in its cluster, as a uniform value
  const int pair = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    ptx::prefetch_tensormap(&kmap);
    ptx::prefetch_tensormap(&vmap);
    ptx::prefetch_tensormap(&qmap);
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(ptx::smem_u32(&bars.full[i]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars.empty[i]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(&bars.q_empty), 1);
    for (int i = 0; i < 2; ++i) ptx::mbar_init(ptx::smem_u32(&bars.s_full[i]), 1);
    ptx::mbar_init(ptx::smem_u32(&bars.p_full), 2 * kSoftmaxWarps);
    ptx::mbar_init(ptx::smem_u32(&bars.o_done), 1);
    ptx::mbar_init(ptx::smem_u32(&bars.o_free), 2 * kSoftmaxWarps);
    ptx::mbar_init(ptx::smem_u32(&bars.drain), 1);
    bars.abort = 0;
    ptx::fence_mbar_init_cluster();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc_pair(ptx::smem_u32(&bars.tmem_base), TM_COLS);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync_all();  // both CTAs' barriers are initialised before any remote arrive
  ptx::tc_fence_after();
  ptx::grid_dependency_wait();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem_base, 0);
  const Ctx c{p.g.status, &bars.abort, p.wait_ns};
  auto wait = [](const Ctx& ctx, uint32_t bar, uint32_t parity) { return wait_for<kPoll>(ctx, bar, parity); };
  Walk w(p.g, pair);

  if (warp == kLoadWarp) {
    // -------------------------------------------------------------- loads ---
    // The whole warp walks the slabs (uniform control flow), one lane issues.
    const bool leader = ptx::elect_one();
    const uint32_t full0 = __shfl_sync(0xffffffffu, ptx::mapa(ptx::smem_u32(&bars.full[0]), 0), 0);
    const uint32_t full_own = ptx::smem_u32(&bars.full[0]), empty_own = ptx::smem_u32(&bars.empty[0]);
    int slot = 0, issued = 0;
    uint32_t ph = 1;  // a fresh barrier passes the wait for the phase before its first
    bool ok = true;
    auto reserve = [&](int bytes) {
      ok = ok && wait(c, empty_own + 8 * slot, ph);
      if (ok && leader && rank == 0) ptx::mbar_arrive_expect_tx(full_own + 8 * slot, 2 * bytes);
    };
    auto advance = [&] {
      issued += ok;
      if (++slot == kSlots) {
        slot = 0;
        ph ^= 1u;
      }
    };
    // A segment's first score slabs bring the same dims of its query rows along.
    auto scores = [&](int t, bool head) {
      const int y = w.key_row(t) + 128 * (int)rank, rows = w.rb * mla::kRowTile + 64 * (int)rank;
#pragma unroll 3
      for (int d = 0; d < 9; ++d) {
        reserve(head ? SLAB + QSLAB : SLAB);
        if (ok && leader) {
          if (head) ptx::tma_load_3d_pair(sbase + OFF_Q + d * QSLAB, &qmap, 0, rows, d, full0 + 8 * slot);
          ptx::tma_load_2d_pair(sbase + OFF_RING + slot * SLAB, &kmap, 64 * d, y, full0 + 8 * slot);
        }
        advance();
      }
    };
    for (int seg = 0; w.next(); ++seg) {
      if (seg > 0) ok = ok && wait(c, ptx::smem_u32(&bars.q_empty), (seg - 1) & 1);
      scores(w.t0, true);
      for (int t = w.t0; t < w.t1; ++t) {
        if (t + 1 < w.t1) scores(t + 1, false);
        const int y = w.key_row(t);
#pragma unroll 4
        for (int v = 0; v < 8; ++v) {  // 64-key group v / 2, dims 128 (v % 2) of the CTA's half
          reserve(SLAB);
          if (ok && leader)
            ptx::tma_load_3d_pair(sbase + OFF_RING + slot * SLAB, &vmap, 0, y + 64 * (v >> 1),
                                  4 * (int)rank + 2 * (v & 1), full0 + 8 * slot);
          advance();
        }
      }
    }
    // After a wait ran out, copies may still be landing: the even CTA, whose
    // barriers count both CTAs' bytes, waits for the last ones.
    if (!ok && rank == 0 && leader) {
      const uint64_t start = ptx::globaltimer_ns();
      for (int i = max(0, issued - kSlots); i < issued; ++i)
        while (!ptx::mbar_try_wait(full_own + 8 * (i % kSlots), (i / kSlots) & 1))
          if (ptx::globaltimer_ns() - start > kDrainNs) break;
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA ---
    // The whole warp walks the slabs of the even CTA, one lane issues.  A slab
    // is 256 cycles of MMAs, so what the loop does between two slabs' MMAs is
    // kept short: the next slab's barrier is tried while they run.
    if (rank == 0) {
      const bool leader = ptx::elect_one();
      constexpr uint32_t id_qk = ptx::idesc_f16(128, T, 0u, false, false);
      constexpr uint32_t id_pv = ptx::idesc_f16(128, 256, 0u, false, true);
      // A slab, a 32-byte step of 16 dims or a 2 KB step of 16 keys is an add
      // to the descriptor's start address (16-byte units, no carry).
      const uint64_t dq = kdesc(sbase + OFF_Q), dp = kdesc(sbase + OFF_P);
      const uint64_t dk = kdesc(sbase + OFF_RING), dv = vdesc(sbase + OFF_RING);
      const uint32_t full0 = ptx::smem_u32(&bars.full[0]), empty0 = ptx::smem_u32(&bars.empty[0]);
      bool ready = false, next = false;  // the current slab, the one after it has landed
      int slot = 0;
      uint32_t ph = 0;
      uint32_t it = 0;  // tiles whose scores this pair has issued, over all segments
      // The current slab: false once a wait has run out (the same in all
      // lanes, as a vote, which keeps the control flow uniform).
      auto pass = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait(c, bar, parity)) != 0;
      };
      // A barrier that both CTAs' softmax warps arrive on: what they wrote (their
      // halves of P, their rows of O) comes before the MMAs that follow.
      auto pass_pair = [&](uint32_t bar, uint32_t parity) {
        if (!pass(bar, parity)) return false;
        ptx::mbar_acquire_cluster(bar, parity);
        return true;
      };
      auto take = [&] {
        if (!ready && !pass(full0 + 8 * slot, ph)) return false;
        ptx::tc_fence_after();
        const bool wrap = slot == kSlots - 1;
        next = ptx::mbar_test_wait(wrap ? full0 : full0 + 8 * (slot + 1), wrap ? ph ^ 1u : ph);
        return true;
      };
      auto advance = [&] {
        if (leader) ptx::mma_commit_pair(empty0 + 8 * slot);
        if (++slot == kSlots) {
          slot = 0;
          ph ^= 1u;
        }
        ready = next;
      };
      for (int seg = 0; w.next(); ++seg) {
        const int n = w.t1 - w.t0;
        for (int t = 0; t <= n; ++t) {
          if (t < n) {
#pragma unroll 3
            for (int d = 0; d < 9; ++d) {
              if (!take()) goto mma_end;
              if (leader) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  ptx::mma_ss_pair(tmem + TM_S + 128 * (it & 1), dq + d * (QSLAB >> 4) + 2 * k,
                                   dk + slot * (SLAB >> 4) + 2 * k, id_qk, (d | k) != 0);
              }
              advance();
            }
            if (leader) {
              ptx::mma_commit_pair(ptx::smem_u32(&bars.s_full[it & 1]));
              if (t == n - 1) ptx::mma_commit_pair(ptx::smem_u32(&bars.q_empty));
            }
            ++it;
          }
          if (t == 0) continue;
          // O is free once the segment before is read.
          if (t == 1 && seg > 0 && !pass_pair(ptx::smem_u32(&bars.o_free), (seg - 1) & 1)) goto mma_end;
          if (!pass_pair(ptx::smem_u32(&bars.p_full), (it - 1 - (t < n)) & 1)) goto mma_end;
#pragma unroll 8
          for (int v = 0; v < 8; ++v) {  // 64-key group v / 2, O columns 128 (v % 2)
            if (!take()) goto mma_end;
            if (leader) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                ptx::mma_ss_pair(tmem + TM_O + 128 * (v & 1), dp + (v >> 1) * (PSLAB >> 4) + 2 * k,
                                 dv + slot * (SLAB >> 4) + k * (2048 >> 4), id_pv,
                                 !(t == 1 && v < 2 && k == 0));
            }
            advance();
          }
          if (leader) ptx::mma_commit_pair(ptx::smem_u32(&bars.o_done));
        }
      }
    }
  mma_end:
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax ---
    // This thread: TMEM lane l = 32 q4 + lane, i.e. row l % 64 of the CTA's 64
    // and half l / 64 of N; score columns 64 ch .. 64 ch + 63, so the 64-key
    // group kg of its row, and O columns 128 ch .. + 127, so 128 value dims.
    const int q4 = warp & 3, ch = warp >> 2;
    const int r = 32 * (q4 & 1) + lane;
    const int kg = 2 * (q4 >> 1) + ch;
    const int dim0 = 256 * (q4 >> 1) + 128 * ch;
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
    const float s_kv = p.kv_scale != nullptr ? *p.kv_scale : 1.f;
    const uint32_t p_full = ptx::mapa(ptx::smem_u32(&bars.p_full), 0);
    const uint32_t o_free = ptx::mapa(ptx::smem_u32(&bars.o_free), 0);
    volatile float* xch = reinterpret_cast<volatile float*>(smem + OFF_X);
    const uint32_t p_row = sbase + OFF_P + kg * PSLAB + r * 128;
    const uint32_t* key_notes = reinterpret_cast<const uint32_t*>(p.g.key_flags + 64 * kg) + (lane & 15);
    uint32_t it = 0;
    while (w.next()) {
      const int row = w.rb * mla::kRowTile + 64 * (int)rank + r;
      // The row sees the first `shared` keys of the prefix and, of its row
      // block's own keys, [own0, own1).
      int shared = 0, own0 = 0, own1 = 0;
      uint32_t row_note = 0;
      if (row < p.g.rows) {
        row_note = p.g.row_flags[row];
        const int b = row / p.g.rows_per_seq, n_vis = p.g.visible(row, b);
        shared = min(n_vis, p.g.prefix_len);
        if (p.g.fold) {
          own0 = p.g.own_off[w.rb * p.g.block_seqs + b - p.g.first_seq(w.rb)];
          own1 = own0 + max(0, n_vis - p.g.prefix_len);
        }
      }
      if (kg == 0 && (row_note & mla::kStagedRange)) atomicOr(p.g.status, MLA_DEVFLAG_Q_RANGE);
      // A scale of zero is taken as the smallest that keeps -inf * c2 = -inf.
      const float c2 = fmaxf(p.softmax_scale * s_kv * 1.4426950408889634f * power2(-lift_of(row_note)), 1.0e-37f);
      float m = kMaxSentinel, l = 0.f;
      for (int t = w.t0; t < w.t1; ++t, ++it) {
        const uint32_t notes = key_notes[w.key_row(t) / 4];  // of four of this warp's 64 keys
        wait(c, ptx::smem_u32(&bars.s_full[it & 1]), (it >> 1) & 1);
        __syncwarp();
        ptx::tc_fence_after();
        uint32_t s[2][32];
        ptx::tmem_ld32(tmem + lanes + TM_S + 128 * (it & 1) + 64 * ch, s[0]);
        ptx::tmem_ld32(tmem + lanes + TM_S + 128 * (it & 1) + 64 * ch + 32, s[1]);
        ptx::tmem_ld_wait();
        // Of this thread's 64 keys the row sees [from, lim).
        const int at = (t < p.g.tiles ? t : t - p.g.tiles) * T + 64 * kg;
        const int from = (t < p.g.tiles ? 0 : own0) - at, lim = (t < p.g.tiles ? shared : own1) - at;
        const bool all = __all_sync(0xffffffffu, from <= 0 && lim >= 64);
        if (!all) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * h + i < from || 32 * h + i >= lim) s[h][i] = 0xFF800000u;  // -inf: weight 0
        }
        const bool noted = __any_sync(0xffffffffu, notes != 0);
        float by = c2;  // s times this: z - e
        if (noted) {
          by = 1.f;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int e = lift_of(note_of(notes, 32 * h + i));
              s[h][i] = __float_as_uint(fmaf(__uint_as_float(s[h][i]) * power2(-e), c2, (float)-e));
            }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[h][i]));
        const float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        volatile float* x = xch + (it & 1) * 256;
        x[kg * 64 + r] = mine * by;
        group_sync(q4 & 1);
        const float mt = fmaxf(fmaxf(x[r], x[64 + r]), fmaxf(x[128 + r], x[192 + r]));
        // The row's maximum moves only when it lags by more than kLag; a row
        // that has seen no key yet keeps the sentinel.
        const bool need = mt > m + kLag;
        const float mn = need ? mt : m;
        const float alpha = need ? exp2f(m - mn) : 1.f;
        m = mn;
        l *= alpha;
        const float base = kHead - m;
        float lifted_sum = 0.f;  // of 2^e_j p_j
        if (noted) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              lifted_sum = fmaf(fast_exp2(__uint_as_float(s[h][i]) + base),
                                power2(lift_of(note_of(notes, 32 * h + i))), lifted_sum);
        }
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pk[32];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float a = fast_exp2(fmaf(__uint_as_float(s[h][i]), by, base));
            const float b2 = fast_exp2(fmaf(__uint_as_float(s[h][i + 1]), by, base));
            sum[i & 3] += a;
            sum[(i & 3) + 1] += b2;
            pk[16 * h + i / 2] = pack_f16(a, b2);
          }
        l += noted ? lifted_sum : (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (__any_sync(0xffffffffu, (notes & kMarks) != 0)) l = marked_keys(p.g, notes, from, lim, l);
        // The weights' buffer and O are free once the values of the tile
        // before are accumulated (a segment's first tile waited for that at
        // the end of the segment before).
        if (t > w.t0) {
          wait(c, ptx::smem_u32(&bars.o_done), (it - 1) & 1);
          __syncwarp();
          if (__any_sync(0xffffffffu, need)) {
            ptx::tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc) {
              uint32_t o[32];
              const uint32_t col = tmem + lanes + TM_O + 128 * ch + 32 * cc;
              ptx::tmem_ld32(col, o);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              ptx::tmem_st32(col, o);
            }
            ptx::tmem_st_wait();
          }
        }
#pragma unroll
        for (int v = 0; v < 8; ++v)
          st_shared(p_row + ((v ^ (r & 7)) * 16), pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(p_full);
      }
      // The segment's partial: O / l and the log-sum-exp.
      group_sync(q4 & 1);  // the exchange buffer's last maxima are read
      xch[kg * 64 + r] = l;
      group_sync(q4 & 1);
      l = (xch[r] + xch[64 + r]) + (xch[128 + r] + xch[192 + r]);
      const bool good = wait(c, ptx::smem_u32(&bars.o_done), (it - 1) & 1);
      __syncwarp();
      ptx::tc_fence_after();
      // A row block that this pair holds whole is final; another's goes to the
      // partial of this segment, pair + row block.
      const bool final = !p.partials && w.t0 == 0 && w.t1 == w.n;
      // No key: 0 and -inf.  A sum that is NaN (a query that f16 cannot hold) stays
      // so, and one of zero over keys that the row sees (scores of minus infinity
      // only, from such a query) becomes it.
      const int key0 = w.t0 * T, key1 = w.t1 * T, own = p.g.tiles * T;
      if (l == 0.f && (key0 < min(shared, key1) || max(own + own0, key0) < min(own + own1, key1))) l = NAN;
      float inv = l == 0.f ? 0.f : s_kv / l;
      float lse = l == 0.f ? -INFINITY : (m - kHead + log2f(l)) * 0.6931471805599453f;
      const size_t seg = (size_t)(pair + w.rb) * mla::kRowTile;
      const int local0 = 64 * (int)rank + 32 * (q4 & 1);  // the warp's first row of the block
      const int rows_left = good ? p.g.rows - w.rb * mla::kRowTile - local0 : 0;
      // The 16x256b shape gives a lane pairs of columns of two rows, four lanes 32
      // contiguous bytes of a row: whole sectors, without a detour through shared
      // memory (through the 32x32b shape, one row a lane, every store touched 32
      // lines: 11 us a segment instead of 3).
      const int cq = lane & 3;
      float inv4[4];  // of rows 8 i + lane / 4
#pragma unroll
      for (int i = 0; i < 4; ++i) inv4[i] = __shfl_sync(0xffffffffu, inv, 8 * i + (lane >> 2));
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        const int half = cc & 1, col = 64 * (cc >> 1);  // 16 rows x 64 columns
        uint32_t o[32];
        ptx::tmem_ld16x256b_x8(tmem + lanes + ((uint32_t)(16 * half) << 16) + TM_O + 128 * ch + col, o);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = 16 * half + 8 * e + (lane >> 2);
          const float by = half ? inv4[2 + e] : inv4[e];
          if (rr >= rows_left) continue;
          if (final) {
            uint16_t* dst = p.out + ((size_t)w.rb * mla::kRowTile + local0 + rr) * mla::kDV + dim0 + col + 2 * cq;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint32_t*>(dst + 8 * j) =
                  pack_bf16(__uint_as_float(o[4 * j + 2 * e]) * by, __uint_as_float(o[4 * j + 2 * e + 1]) * by);
          } else {
            float* dst = p.part_o + (seg + local0 + rr) * mla::kDV + dim0 + col + 2 * cq;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float2*>(dst + 8 * j) =
                  make_float2(__uint_as_float(o[4 * j + 2 * e]) * by, __uint_as_float(o[4 * j + 2 * e + 1]) * by);
          }
        }
      }
      if (lane < rows_left && kg == 0) {
        if (final) p.lse[row] = lse;
        else p.part_lse[seg + local0 + lane] = lse;
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster(o_free);
      group_sync(q4 & 1);  // the sums are read before the next segment's maxima
    }
  }

  // ------------------------------------------------------------ teardown ---
  ptx::tc_fence_before();
  __syncthreads();
  if (bars.abort) {
    // Nothing is issued any more.  The MMAs in flight are waited for, and
    // copies of either CTA still landing, or arrivals still on their way to
    // the other CTA, get far longer than they take.
    if (warp == kMmaWarp && rank == 0 && lane == 0) {
      ptx::mma_commit_pair(ptx::smem_u32(&bars.drain));
      const uint64_t start = ptx::globaltimer_ns();
      while (!ptx::mbar_try_wait(ptx::smem_u32(&bars.drain), 0))
        if (ptx::globaltimer_ns() - start > kDrainNs) break;
    }
    __syncwarp();
    const uint64_t start = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - start < kSettleNs) __nanosleep(1000);
    __syncthreads();
  }
  ptx::cluster_sync_all();  // no CTA leaves, or frees TMEM, while the pair still works
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, TM_COLS);
  }
}

}  // namespace

int mla_launch_prefix_sm103(const mla::PrefixParams& p, const void* keys, int64_t key_rows,
                            const void* rows, void* stream) {
  // Score slabs: 128 keys x 64 dims.  Value slabs: 64 keys x 2 x 64 dims and
  // query slabs: 64 rows x 64 dims, the 64-dim groups of a row as a third
  // dimension, so that one copy fills a slab group by group.
  CUtensorMap kmap, vmap, qmap;
  if (!mla::tensor_map_rows(&kmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, keys, key_rows, mla::kDQK, 128) ||
      !mla::tensor_map_groups(&vmap, keys, key_rows, 2) ||
      !mla::tensor_map_groups(&qmap, rows, p.g.rows, 1))
    return (int)cudaErrorUnknown;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  const bool poll = p.wait_ns < (uint64_t)kSleepNs;
  auto* kernel = poll ? prefix_kernel<true> : prefix_kernel<false>;
  e = mla::opt_in_smem(reinterpret_cast<const void*>(kernel), SMEM_BYTES, dev, poll ? 9 : 8);
  if (e != cudaSuccess) return (int)e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.g.pairs, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, p, kmap, vmap, qmap);
}
