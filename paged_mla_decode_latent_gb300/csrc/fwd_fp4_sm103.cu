// fwd_fp4_sm103.cu -- the decode over a 4-bit cache: keys as the rows of the
// MMAs, one CTA per (sequence, KV split) of up to 32 query rows a sequence.
//
// With K the tile's 128 keys (576 dims), Q the N query rows and V the
// first 512 dims of K, the CTA computes, transposed,
//
//   S = K Q^T     [128 keys x N]     A = K from TMEM (a key a lane), B = Q
//   O^T += V^T P  [512 dims x N]     A = V from shared memory, read dim-major in
//                                    four blocks of 128 dims, B = the weights
//
// Why transposed: an MMA costs what its larger operand side costs.  With the
// few query rows of a head-parallel shard on the N side, QK^T takes 13
// (N = 16) to 18 (N = 32) cycles a 16-dim step from TMEM and PV 39 to 40 a 128
// dims x 16 keys (bound by the 4 KB of A that it reads); with the keys on the N
// side each took 64 to 128 whatever the number of rows (all measured back to
// back).  All rows then fit one CTA: O^T takes 4 N TMEM columns, so
// there is no partner to swap partial scores with, and scores are summed in fp32
// throughout.
//
// A row of the cache is converted twice, by different warps, which takes the
// scores off the path of the values: K (576 dims) goes to TMEM as soon as the
// scores of the tile before are done, V (512 dims) to a short ring in shared
// memory as soon as the MMAs have read what was there.  The codes wait in
// shared memory for both.  Per 128-key tile, all at once:
//   copy warps (2) the rows of later tiles, 16-byte cp.async, 32 keys (a part)
//                  at a time into a ring
//   K warps (4)    part q of the tile: codes to f16, into TMEM lanes 32 q ...
//   QK warp        S as soon as K is there
//   softmax warps  a key a thread, all N rows: weights relative to a running
//   (4)            maximum that is raised (and O rescaled) only when a weight
//                  would pass 2^8, as one vote of the four warps decides
//   V warps (8)    two groups that take turns, a part each; 128 dims a warp
//   PV warp        O^T += V^T P, 32 keys at a time
//
// What bounds it: the chain of these handoffs and conversions, not one unit.  A
// tile takes about 4500 cycles an SM, of which its shared-memory traffic (codes in
// and out twice, V in and out, the MMAs' operands) needs 3300, issue slots half and
// DRAM 40 %.  Batch 8 x 16 heads x 109440 keys: 107 us (3.4 TB/s of 6.7); batch 64 x
// 32 heads x 8192: 102 us.  With eight K warps (24 warps at 80 registers) 106 and
// 105 us, with one group of V warps (16 warps at 128) 117 and 100 us.  With waits
// that poll in place of the suspended ones 109 (the MMA warps only) to 119 us (all).
//
// f16 holds a code times its scale exactly, and a bf16 query value between 2^-17 and
// 65504 in size.  Above (MLA_DEVFLAG_Q_RANGE) the row comes out NaN, below a value is off
// by up to 2^-25, which a key of 2688 kv_scale turns into 2^-13 kv_scale of a score.
// Scores and outputs are summed in fp32; weights are rounded to f16, 2^-11 of themselves
// (the output's own bf16 is eight times as coarse), as the MMA takes them.
//
// Every wait is bounded (2 s unless the plan sets another limit).  A wait that
// runs out sets MLA_DEVFLAG_TIMEOUT; the warps then run through their loops
// without waiting or issuing and leave together.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/mla_decode.h"
#include "fp4.cuh"
#include "internal.h"
#include "kv.h"
#include "ptx.cuh"

namespace {

constexpr int T = 128;                    // keys per tile
constexpr int kRaw = fp4::kRow + 16;      // a row in the ring: 27 pieces, so that eight keys' lie in different banks
constexpr int kPart = 32 * kRaw;          // 32 keys: 13.5 KB
constexpr int kVSlab = 32 * 128;          // 64 dims of 32 keys
constexpr int kVUnit = 8 * kVSlab;        // a part's V: 32 KB
constexpr int kQSlabs = 9;

// Warps.  Those that work on TMEM lanes 32 q ... are warps q modulo 4.
constexpr int kVWarp0 = 4, kSoftmaxWarp0 = 12, kQkWarp = 16, kPvWarp = 17, kCopyWarp0 = 18, kCopyWarps = 2;
constexpr int kThreads = 20 * 32;
// Registers a thread of each group of four warps; the launch gives 96 each.
constexpr int kLaunchRegs = 96, kKRegs = 96, kVRegs = 72, kSoftmaxRegs = 160, kOtherRegs = 80;
static_assert(kKRegs + 2 * kVRegs + kSoftmaxRegs + kOtherRegs <= 5 * kLaunchRegs, "no more than the launch gives");

template <int N>
struct Layout {
  static constexpr int kParts = N <= 16 ? 10 : 8;  // parts in the ring of codes
  static constexpr int kVUnits = 2;                // and in the ring of V
  static constexpr int kQSlab = N * 128;
  static constexpr int kP = T * N * 2;             // one tile's weights
  static constexpr int OFF_V = 0;
  static constexpr int OFF_Q = OFF_V + kVUnits * kVUnit;
  static constexpr int OFF_P = OFF_Q + kQSlabs * kQSlab;
  static constexpr int OFF_RAW = OFF_P + 2 * kP;
  static constexpr int OFF_X = OFF_RAW + kParts * kPart;  // [4][N] maxima or sums, [N] visible keys, [N] 1 / sum
  static constexpr int OFF_BAR = OFF_X + 6 * N * 4;
  static constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;
  // TMEM columns: O^T (4 blocks of N), two score buffers, and K as f16 pairs: a
  // ring of slabs of 64 dims (32 columns), 9 a tile, so that the next tile's
  // first ones need not wait for this one's scores.
  static constexpr uint32_t TM_O = 0, TM_S = 4 * N, TM_K = 6 * N;
  static constexpr int kKSlabs = (512 - 6 * N) / 32;  // 13 or 10
  static_assert(kKSlabs >= 9 && kKSlabs < 17 && SMEM_BYTES <= 232448 && OFF_Q % 1024 == 0 && OFF_BAR % 8 == 0, "fits");
};

constexpr float kRescaleThreshold = 8.0f;
constexpr float kMaxSentinel = -1.0e30f;
constexpr uint64_t kDrainNs = 500000000ull;
constexpr uint32_t kSleepNs = 20000;

struct Bars {
  uint64_t raw_full[10];   // a part has landed (32 lanes of a copy warp)
  uint64_t raw_empty[10];  // its K warp and four V warps have read it
  uint64_t v_full[2], v_empty[2];
  uint64_t k_full[2];      // K of a tile is in TMEM (four warps)
  uint64_t s_full[2];      // scores done, and K read
  uint64_t p_full[2];      // weights written, and scores read (four warps)
  uint64_t p_done[2];      // the tile's values are summed
  uint64_t q_ready;
  uint64_t drain[2];
  uint32_t tmem_base;
  int32_t abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

struct Ctx {
  int32_t* status;
  volatile int32_t* abort;
  uint64_t limit_ns;
  uint32_t sleep_ns;
};

// Bounded wait: false if the phase did not complete in time or another warp gave up.
__device__ __forceinline__ bool wait(const Ctx& c, uint32_t bar, uint32_t parity) {
  if (ptx::mbar_test_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
    if (ptx::mbar_try_wait_sleep(bar, parity, c.sleep_ns)) return true;
    if (*c.abort) return false;
    if (ptx::globaltimer_ns() - t0 > c.limit_ns) {
      atomicOr(c.status, MLA_DEVFLAG_TIMEOUT);
      *c.abort = 1;
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

__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void st_shared_u4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// Counts on `bar` once this thread's cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A vote of the softmax warps' 128 threads, which is also their barrier.
__device__ __forceinline__ bool any_of_softmax(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

// This warp group's share of the launch's registers from here on.
template <int kRegs>
__device__ __forceinline__ void take_registers() {
  if constexpr (kRegs > kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
  if constexpr (kRegs < kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
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

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void words(const uint4 (&v)[4], uint32_t (&r)[16]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    r[4 * e] = v[e].x;
    r[4 * e + 1] = v[e].y;
    r[4 * e + 2] = v[e].z;
    r[4 * e + 3] = v[e].w;
  }
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

template <int N>
__global__ void __launch_bounds__(kThreads, 1) fwd_fp4_kernel(mla::FwdParams p) {
  using L = Layout<N>;
  constexpr int R = L::kParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem + L::OFF_BAR);
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // The work unit, as in the other decode kernels.
  int b, ctx, k0, k1;
  bool single;
  size_t part;
  if (p.units != nullptr) {
    ptx::grid_dependency_wait();
    const int u = blockIdx.x;
    if (u >= *p.n_units) return;
    const int4 d = p.units[u];
    const int4 si = p.seq_info[d.x];
    b = d.x;
    k0 = d.z;
    k1 = d.w;
    ctx = si.x;
    single = si.z == 1;
    part = (size_t)si.y + (d.y >> 8);
  } else {
    b = blockIdx.y;
    const int split = blockIdx.z;
    ctx = p.seq_lens[b];
    if (ctx < 0 || ctx > p.max_ctx) {
      if (threadIdx.x == 0 && split == 0) atomicOr(p.status, MLA_DEVFLAG_CTX_RANGE);
      ctx = ctx < 0 ? 0 : p.max_ctx;
    }
    k0 = p.key_begin + split * p.chunk_len;
    k1 = min(k0 + p.chunk_len, ctx);
    single = p.num_splits == 1 && !p.partials;
    part = (size_t)b * p.num_splits + split;
  }
  const int n_rows = p.rows;  // <= N
  const int n_tiles = k1 > k0 ? (k1 - k0 + T - 1) / T : 0;
  const float s_kv = p.kv_scale ? *p.kv_scale : 1.f;

  if (n_tiles == 0) {
    ptx::grid_dependency_wait();
    for (int i = threadIdx.x; i < n_rows * 64; i += kThreads) {
      const size_t row = i >> 6;
      if (single) {
        reinterpret_cast<uint4*>(p.out + ((size_t)b * p.rows + row) * mla::kDV)[i & 63] = make_uint4(0, 0, 0, 0);
        if ((i & 63) == 0) p.lse[(size_t)b * p.rows + row] = -INFINITY;
      } else if ((i & 63) == 0) {
        p.part_lse[part * p.rows + row] = -INFINITY;
      }
    }
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < R; ++i) {
      ptx::mbar_init(ptx::smem_u32(&bars.raw_full[i]), 32);
      ptx::mbar_init(ptx::smem_u32(&bars.raw_empty[i]), 5);
    }
    for (int i = 0; i < L::kVUnits; ++i) {
      ptx::mbar_init(ptx::smem_u32(&bars.v_full[i]), 4);
      ptx::mbar_init(ptx::smem_u32(&bars.v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_u32(&bars.k_full[i]), 4);
      ptx::mbar_init(ptx::smem_u32(&bars.s_full[i]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars.p_full[i]), 4);
      ptx::mbar_init(ptx::smem_u32(&bars.p_done[i]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(&bars.q_ready), 128);
    for (int i = 0; i < 2; ++i) ptx::mbar_init(ptx::smem_u32(&bars.drain[i]), 1);
    bars.abort = 0;
    ptx::fence_mbar_init_cluster();
  }
  if (warp == kQkWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&bars.tmem_base), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  ptx::grid_dependency_wait();
  const uint32_t tmem = bars.tmem_base;
  Ctx c{p.status, &bars.abort, p.wait_ns,
        (uint32_t)(p.wait_ns < (uint64_t)kSleepNs ? p.wait_ns : (uint64_t)kSleepNs)};

  if (warp < kVWarp0) {
    take_registers<kKRegs>();
    // ----------------------------------------------------------------- K ---
    // Warp q: part q of every tile, a key a lane, in slabs of 64 dims.
    const int q = warp;
    const uint32_t kcol = tmem + ((uint32_t)(32 * q) << 16) + L::TM_K;
    Ring<R> ring;
    ring.next(q);
    int first = 0;  // the tile's first slab in the ring of slabs
    constexpr int kEarly = L::kKSlabs - 9;  // slabs before it take the place of tile t - 2's, the others tile t - 1's
    for (int t = 0; t < n_tiles; ++t, ring.next(4)) {
      auto column = [&](int a) {
        const int at = first + a;
        return kcol + 32 * (at < L::kKSlabs ? at : at - L::kKSlabs);
      };
      if (!wait_all(c, ptx::smem_u32(&bars.raw_full[ring.slot]), ring.phase)) break;
      const uint32_t raw = sbase + L::OFF_RAW + ring.slot * kPart + lane * kRaw;
      const uint4 s0 = ld_shared_u4(raw + fp4::kScales), s1 = ld_shared_u4(raw + fp4::kScales + 16);
      const uint32_t sc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
      bool ok = true;
#pragma unroll
      for (int a = 0; a < 8; ++a) {
        if (a == kEarly) {
          ok = t < 1 || wait_all(c, ptx::smem_u32(&bars.s_full[(t - 1) & 1]), ((t - 1) >> 1) & 1);
          if (!ok) break;
          ptx::tc_fence_after();
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // 32 dims
          uint4 v[4];
          uint32_t r[16];
          fp4::convert(ld_shared_u4(raw + 32 * a + 16 * e), sc[a] >> (16 * e), v);
          words(v, r);
          tmem_st16(column(a) + 16 * e, r);
        }
      }
      if (!ok) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 v[4];
        uint32_t r[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = ld_shared_u4(raw + fp4::kRope + 64 * h + 16 * e);
        words(v, r);
        tmem_st16(column(8) + 16 * h, r);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars.raw_empty[ring.slot]));
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars.k_full[t & 1]));
      first += 9;
      if (first >= L::kKSlabs) first -= L::kKSlabs;
    }
  } else if (warp < kSoftmaxWarp0) {
    take_registers<kVRegs>();
    // ----------------------------------------------------------------- V ---
    // Two groups of four warps take turns, a part each; warp v of a
    // group: dims 128 v .. (slabs 2 v and 2 v + 1) of the part's 32 keys, a key a lane.
    const int v = warp & 3, g = (warp - kVWarp0) >> 2;
    Ring<R> ring;
    ring.next(g);
    Ring<L::kVUnits> unit;
    unit.next(g);
    const int n_units = 4 * n_tiles;
    for (int u = g; u < n_units; u += 2, ring.next(2), unit.next(2)) {
      if (!wait_all(c, ptx::smem_u32(&bars.raw_full[ring.slot]), ring.phase)) break;
      const uint32_t raw = sbase + L::OFF_RAW + ring.slot * kPart + lane * kRaw;
      uint32_t sc[2];
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(sc[0]), "=r"(sc[1]) : "r"(raw + fp4::kScales + 8 * v) : "memory");
      uint4 codes[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) codes[i] = ld_shared_u4(raw + 64 * v + 16 * i);
      if (u >= L::kVUnits && !wait_all(c, ptx::smem_u32(&bars.v_empty[unit.slot]), unit.phase ^ 1u)) break;
      const uint32_t dst = sbase + L::OFF_V + unit.slot * kVUnit + 2 * v * kVSlab + lane * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // 32 dims
        uint4 x[4];
        fp4::convert(codes[i], sc[i >> 1] >> (16 * (i & 1)), x);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          st_shared_u4(dst + (i >> 1) * kVSlab + (((4 * (i & 1) + e) ^ (lane & 7)) * 16), x[e]);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(ptx::smem_u32(&bars.v_full[unit.slot]));
        ptx::mbar_arrive(ptx::smem_u32(&bars.raw_empty[ring.slot]));
      }
    }
  } else if (warp < kQkWarp) {
    take_registers<kSoftmaxRegs>();
    // ----------------------------------------------------------- softmax ---
    const int q = warp - kSoftmaxWarp0;
    const int tid = 32 * q + lane;  // the thread's key in a tile, its lane of TMEM
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    float* xmax = reinterpret_cast<float*>(smem + L::OFF_X);  // [4][N]
    int* vis = reinterpret_cast<int*>(xmax + 4 * N);          // [N]
    float* inv = reinterpret_cast<float*>(vis + N);           // [N]
    // Q to f16, K-major: 72 pieces of 8 dims a row; rows past the problem's are zero.
    static_assert(N % 16 == 0, "9 x 128 pieces are 16 rows");
    {
      // Nine loads in flight a thread, then their stores: 16 rows a round.
      bool range = false;
#pragma unroll 1
      for (int i0 = tid; i0 < N * 72; i0 += 9 * 128) {
        uint4 x[9];
#pragma unroll
        for (int j = 0; j < 9; ++j) {
          const int i = i0 + 128 * j, r = i / 72, ch = i - 72 * r;
          x[j] = make_uint4(0, 0, 0, 0);
          if (r < n_rows) x[j] = reinterpret_cast<const uint4*>(p.q + ((size_t)b * p.rows + r) * mla::kDQK)[ch];
        }
#pragma unroll
        for (int j = 0; j < 9; ++j) {
          const int i = i0 + 128 * j, r = i / 72, ch = i - 72 * r;
          uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xFFFF0000u);
            range |= fabsf(lo) > 65504.f || fabsf(hi) > 65504.f;
            w[e] = pack_f16(lo, hi);
          }
          st_shared_u4(sbase + L::OFF_Q + (ch >> 3) * L::kQSlab + r * 128 + (((ch & 7) ^ (r & 7)) * 16),
                       make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
      if (range) atomicOr(p.status, MLA_DEVFLAG_Q_RANGE);
      if (tid < N) {  // keys that a row sees
        int n = 0;
        if (tid < n_rows) {
          const int tok = tid / p.heads;
          n = p.causal ? ctx - p.sq + tok + 1 : ctx;
          n = min(max(0, min(n, ctx)), k1);
          if (n <= k0) n = 0;  // none of this unit's
        }
        vis[tid] = n;
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_u32(&bars.q_ready));
    }
    softmax_sync();
    int all_see = k1;  // keys before it are seen by every row
    for (int r = 0; r < n_rows; ++r) all_see = min(all_see, vis[r]);

    const float c2 = p.softmax_scale * s_kv * 1.4426950408889634f;
    float nm[N], l[N];  // minus the running maximum (log2), and this thread's part of the row sums
#pragma unroll
    for (int r = 0; r < N; ++r) {
      nm[r] = -kMaxSentinel;
      l[r] = 0.f;
    }
    // Every pass holds one vote of all four warps, so no warp leaves the loop
    // early: after a wait that ran out the others' return at once.  The scores of
    // 16 rows are in registers at a time.
    constexpr int G = N / 16;
    for (int t = 0; t < n_tiles; ++t) {
      const int buf = t & 1;
      bool ok = wait_all(c, ptx::smem_u32(&bars.s_full[buf]), (t >> 1) & 1);
      ptx::tc_fence_after();
      const int key = k0 + t * T + tid;
      const bool masked = k0 + t * T + T > all_see;
      float s[16];
      auto load = [&](int g) {  // scaled scores of rows 16 g .., -inf where hidden
        uint32_t raw[16];
        tmem_ld16(tmem + lanes + L::TM_S + buf * N + 16 * g, raw);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = __uint_as_float(raw[r]) * c2;
        if (masked) {
#pragma unroll
          for (int r = 0; r < 16; ++r) s[r] = key < vis[16 * g + r] ? s[r] : -INFINITY;
        }
      };
      float over = -INFINITY;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        load(g);
#pragma unroll
        for (int r = 0; r < 16; ++r) over = fmaxf(over, s[r] + nm[16 * g + r]);
      }
      if (any_of_softmax(over > kRescaleThreshold)) {
        // New maxima: of each row over the tile, kept where they are no higher.
#pragma unroll
        for (int g = 0; g < G; ++g) {
          if (G > 1) load(g);
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            float m = s[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == 0) xmax[q * N + 16 * g + r] = m;
          }
        }
        softmax_sync();
        if (t > 0) {  // O is the tile before's
          ok = wait_all(c, ptx::smem_u32(&bars.p_done[buf ^ 1]), ((t - 1) >> 1) & 1) && ok;
          ptx::tc_fence_after();
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float al[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = 16 * g + i;
            const float m = fmaxf(fmaxf(xmax[r], xmax[N + r]), fmaxf(xmax[2 * N + r], xmax[3 * N + r]));
            const float to = fminf(nm[r], -m);
            al[i] = exp2f(to - nm[r]);
            nm[r] = to;
            l[r] *= al[i];
          }
          if (t > 0) {
#pragma unroll 1
            for (int d = 0; d < 4; ++d) {
              uint32_t o[16];
              const uint32_t col = tmem + lanes + L::TM_O + d * N + 16 * g;
              tmem_ld16(col, o);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al[i]);
              tmem_st16(col, o);
            }
            ptx::tmem_st_wait();
          }
        }
      }
      // The weights' buffer is free once the values of tile t - 2 are summed.
      if (t >= 2) ok = wait_all(c, ptx::smem_u32(&bars.p_done[buf]), ((t >> 1) - 1) & 1) && ok;
      const uint32_t dst = sbase + L::OFF_P + buf * L::kP + (tid >> 3) * (16 * N) + (tid & 7) * 16;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (G > 1) load(g);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const int r = 16 * g + i;
          const float a = fast_exp2(s[i] + nm[r]), b2 = fast_exp2(s[i + 1] + nm[r + 1]);
          l[r] += a;
          l[r + 1] += b2;
          w[i / 2] = pack_f16(a, b2);
        }
        st_shared_u4(dst + 2 * g * 128, make_uint4(w[0], w[1], w[2], w[3]));
        st_shared_u4(dst + 2 * g * 128 + 128, make_uint4(w[4], w[5], w[6], w[7]));
      }
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars.p_full[buf]));
    }

    // ---------------------------------------------------------- epilogue ---
    float m_mine = 0.f;
    softmax_sync();  // xmax's last readers
#pragma unroll
    for (int r = 0; r < N; ++r) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
      if (lane == 0) xmax[q * N + r] = l[r];
      m_mine = r == tid ? nm[r] : m_mine;
    }
    softmax_sync();
    if (tid < N) {
      float sum = xmax[tid] + xmax[N + tid] + xmax[2 * N + tid] + xmax[3 * N + tid];
      if (sum == 0.f && vis[tid] > 0) sum = NAN;  // keys whose scores are all -inf, not a row without any
      inv[tid] = sum == 0.f ? 0.f : s_kv / sum;
      const float lse = sum == 0.f ? -INFINITY : (log2f(sum) - m_mine) * 0.6931471805599453f;
      if (tid < n_rows) {
        if (single) p.lse[(size_t)b * p.rows + tid] = lse;
        else p.part_lse[part * p.rows + tid] = lse;
      }
    }
    softmax_sync();
    if (wait_all(c, ptx::smem_u32(&bars.p_done[(n_tiles - 1) & 1]), ((n_tiles - 1) >> 1) & 1)) {
      ptx::tc_fence_after();
#pragma unroll 1
      for (int dg = 0; dg < 4 * G; ++dg) {  // 16 rows at a time; lane: dim 128 d + tid
        const int d = dg / G, r0 = 16 * (dg % G);
        uint32_t o[16];
        tmem_ld16(tmem + lanes + L::TM_O + d * N + r0, o);
        ptx::tmem_ld_wait();
        const int dim = 128 * d + tid;
        if (single) {
          uint16_t* out = p.out + ((size_t)b * p.rows + r0 + (lane & 1)) * mla::kDV + (dim & ~1);
#pragma unroll
          for (int r = 0; r < 16; r += 2) {
            // even lanes store row r's two dims, odd lanes row r + 1's
            const float a = __uint_as_float(o[r]) * inv[r0 + r], b2 = __uint_as_float(o[r + 1]) * inv[r0 + r + 1];
            const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? a : b2, 1);
            if (r0 + r + (lane & 1) < n_rows)
              *reinterpret_cast<uint32_t*>(out + r * mla::kDV) = (lane & 1) ? pack_bf16(got, b2) : pack_bf16(a, got);
          }
        } else {
          float* out = p.part_o + (part * p.rows + r0) * mla::kDV + dim;
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (r0 + r < n_rows) out[r * mla::kDV] = __uint_as_float(o[r]) * inv[r0 + r];
        }
      }
    }
    ptx::tc_fence_before();
  } else {
  take_registers<kOtherRegs>();
  if (warp == kQkWarp) {
    // ---------------------------------------------------------------- QK ---
    // The whole warp walks the loop, one lane issues: in a branch that one lane
    // takes alone an MMA costs about 64 cycles to issue.
    const bool leader = ptx::elect_one();
    constexpr uint32_t id_qk = ptx::idesc_f16(128, N, 0, false, false);
    const uint64_t dq = ptx::smem_desc(sbase + L::OFF_Q, 16, 1024, 2);  // K-major, 128-byte swizzle
    bool ok = wait_all(c, ptx::smem_u32(&bars.q_ready), 0);
    int first = 0;  // the tile's first slab in the ring of slabs
    for (int t = 0; ok && t < n_tiles; ++t) {
      // K is there, and the softmax has read the scores of tile t - 2.
      ok = wait_all(c, ptx::smem_u32(&bars.k_full[t & 1]), (t >> 1) & 1) &&
           (t < 2 || wait_all(c, ptx::smem_u32(&bars.p_full[t & 1]), ((t >> 1) - 1) & 1));
      if (!ok) break;
      ptx::tc_fence_after();
      if (leader) {
        const uint32_t d = tmem + L::TM_S + (t & 1) * N;
#pragma unroll
        for (int a = 0; a < kQSlabs; ++a) {
          const int at = first + a;
          const uint32_t k = tmem + L::TM_K + 32 * (at < L::kKSlabs ? at : at - L::kKSlabs);
#pragma unroll
          for (int s = 0; s < 4; ++s) ptx::mma_ts(d, k + 8 * s, dq + (a * L::kQSlab + 32 * s) / 16, id_qk, (a | s) != 0);
        }
        ptx::mma_commit(ptx::smem_u32(&bars.s_full[t & 1]));
      }
      __syncwarp();
      first += 9;
      if (first >= L::kKSlabs) first -= L::kKSlabs;
    }
  } else if (warp == kPvWarp) {
    // ---------------------------------------------------------------- PV ---
    const bool leader = ptx::elect_one();
    constexpr uint32_t id_pv = ptx::idesc_f16(128, N, 0, true, true);
    // V: dims contiguous, 64-dim slabs kVSlab apart, 8-key groups 1 KB apart.  P:
    // rows contiguous in groups of 8, no swizzle; a group of 8 keys x 8 rows is 128
    // bytes, 8-key groups lie 16 N bytes apart.
    const uint64_t dv = ptx::smem_desc(sbase + L::OFF_V, kVSlab, 1024, 2);
    const uint64_t dp = ptx::smem_desc(sbase + L::OFF_P, 16 * N, 128, 0);
    bool ok = true;
    Ring<L::kVUnits> unit;
    for (int u = 0; ok && u < 4 * n_tiles; ++u, unit.next()) {
      const int t = u >> 2;
      ok = ((u & 3) != 0 || wait_all(c, ptx::smem_u32(&bars.p_full[t & 1]), (t >> 1) & 1)) &&
           wait_all(c, ptx::smem_u32(&bars.v_full[unit.slot]), unit.phase);
      if (!ok) break;
      ptx::tc_fence_after();
      if (leader) {
        const uint64_t a = dv + unit.slot * (kVUnit / 16);
        const uint64_t w = dp + ((t & 1) * L::kP + (u & 3) * 64 * N) / 16;
#pragma unroll
        for (int s = 0; s < 2; ++s)  // 16 keys
#pragma unroll
          for (int d = 0; d < 4; ++d)
            ptx::mma_ss(tmem + L::TM_O + d * N, a + (d * 2 * kVSlab + s * 2048) / 16, w + s * 2 * N, id_pv, (u | s) != 0);
        ptx::mma_commit(ptx::smem_u32(&bars.v_empty[unit.slot]));
        if ((u & 3) == 3) ptx::mma_commit(ptx::smem_u32(&bars.p_done[t & 1]));
      }
      __syncwarp();
    }
  } else {
    // -------------------------------------------------------------- copy ---
    // Lane i looks up key i of the part; keys past the split's last one repeat
    // it (their weights are zero), so every row read lies in [k0, k1).
    const int32_t* bt = p.bt + (p.bt_indptr ? (size_t)p.bt_indptr[b] : (size_t)b * p.bt_stride);
    const uint8_t* cache = static_cast<const uint8_t*>(p.cache);
    // key / page_size: Granlund and Montgomery, "Division by invariant integers
    // using multiplication" (PLDI 1994), exact for every 32-bit key
    const uint32_t pdiv = (uint32_t)p.page_size;
    const uint32_t plog = 32u - __clz(pdiv - 1u);
    const uint32_t pmul = (uint32_t)(((1ull << 32) * ((1ull << plog) - pdiv)) / pdiv) + 1u;
    const uint32_t pshift = plog > 0 ? plog - 1u : 0u;
    auto page_of = [&](uint32_t key) -> uint32_t {
      const uint32_t t = __umulhi(pmul, key);
      return pdiv == 1u ? key : (t + ((key - t) >> 1)) >> pshift;
    };
    auto key_of = [&](int u) -> uint32_t { return (uint32_t)min(k0 + 32 * u + lane, k1 - 1); };
    const int n_parts = 4 * n_tiles;
    const int w = warp - kCopyWarp0;  // parts w, w + kCopyWarps, ...
    const int g = lane >> 3, sub = lane & 7;
    int page = __ldg(&bt[page_of(key_of(w))]);
    Ring<R> ring;
    ring.next(w);
    for (int u = w; u < n_parts; u += kCopyWarps, ring.next(kCopyWarps)) {
      const uint32_t key = key_of(u);
      int64_t at = page;
      if (u + kCopyWarps < n_parts) page = __ldg(&bt[page_of(key_of(u + kCopyWarps))]);
      if (at < 0 || at >= p.num_pages) {
        atomicOr(p.status, MLA_DEVFLAG_BAD_PAGE);
        at = 0;
      }
      const uint32_t row = (uint32_t)at * pdiv + (key - page_of(key) * pdiv);
      const uint32_t full = ptx::smem_u32(&bars.raw_full[ring.slot]);
      const uint32_t dst = sbase + L::OFF_RAW + ring.slot * kPart;
      // Eight lanes a key, keys g, g + 4, ... of the part: pieces sub, sub + 8 and
      // sub + 16 of each row, then the last two pieces of four keys at a time.
      // The rows are traded before the copies begin: a shuffle between them would
      // queue behind them.
      const uint8_t* src[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        src[i] = cache + (size_t)__shfl_sync(0xffffffffu, row, 4 * i + g) * fp4::kRow + sub * 16;
      if (u >= R && !wait_all(c, ptx::smem_u32(&bars.raw_empty[ring.slot]), ring.phase ^ 1u)) break;
      const uint32_t mine = dst + g * kRaw + sub * 16;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 3; ++j) ptx::cp_async_16(mine + 4 * i * kRaw + 128 * j, src[i] + 128 * j);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int of = sub >> 1;  // key 4 (4 i + of) + g, piece 24 + sub % 2
        const uint8_t* p01 = (of & 1) ? src[4 * i + 1] : src[4 * i];
        const uint8_t* p23 = (of & 1) ? src[4 * i + 3] : src[4 * i + 2];
        const uint8_t* from = ((of & 2) ? p23 : p01) - sub * 16;
        ptx::cp_async_16(dst + (4 * (4 * i + of) + g) * kRaw + (24 + (sub & 1)) * 16, from + (24 + (sub & 1)) * 16);
      }
      cp_async_arrive(full);
    }
    ptx::cp_async_commit();
    ptx::cp_async_wait<0>();
  }
  }

  // ------------------------------------------------------------ teardown ---
  __syncthreads();
  if (bars.abort) {
    if ((warp == kQkWarp || warp == kPvWarp) && ptx::elect_one()) {  // every MMA that this thread issued
      const uint32_t bar = ptx::smem_u32(&bars.drain[warp - kQkWarp]);
      ptx::mma_commit(bar);
      const uint64_t t0 = ptx::globaltimer_ns();
      while (!ptx::mbar_try_wait(bar, 0))
        if (ptx::globaltimer_ns() - t0 > kDrainNs) break;
    }
    __syncthreads();
  }
  if (warp == kQkWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace

int mla_launch_fwd_fp4_sm103(const mla::FwdParams& p, void* stream) {
  const bool few = p.rows <= 16;
  auto kernel = few ? fwd_fp4_kernel<16> : fwd_fp4_kernel<32>;
  const int smem = few ? Layout<16>::SMEM_BYTES : Layout<32>::SMEM_BYTES;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  e = mla::opt_in_smem(reinterpret_cast<const void*>(kernel), smem, dev, few ? 10 : 11);
  if (e != cudaSuccess) return (int)e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = p.units != nullptr ? dim3(p.unit_capacity, 1, 1) : dim3(1, p.batch, p.num_splits);
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
