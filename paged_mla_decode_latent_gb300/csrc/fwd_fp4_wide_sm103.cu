// fwd_fp4_wide_sm103.cu -- the decode over a 4-bit cache for more than 32 score
// rows: a pair of CTAs per (sequence, block of 128 rows, KV split).
//
// The division of the work is the 128-row kernel's (fwd_sm103.cu): CTA r of the
// pair owns value dims [256 r, 256 r + 256), contracts those and rope dims [32 r,
// 32 r + 32) for the scores, and the two add up each other's partial scores, which
// travel over distributed shared memory.  Three things differ.
//
//   * The loaders convert 4-bit rows to f16 operands (fp4.cuh), a key a lane.
//   * The MMA warp walks its loop as a whole and one elected lane issues.  In a
//     branch that one lane takes alone an MMA costs about 64 cycles to issue,
//     here what the tensor cores need (N = 64 with A from TMEM: 32, N = 256: 128).
//   * The swap of partial scores goes through two receive buffers (32 KB each), in
//     fp32, and a tile's own scores stay in registers while the partner's block
//     travels, instead of being read from TMEM again.  The buffers fit because a
//     4-bit tile's codes are 13 KB, and because the rope half of a key is kept in
//     64-byte rows (a stage of 36 KB instead of 40).
//
// What bounds it: distributed shared memory, of which a pair swaps 32 KB each way a
// tile (1.15 of the tile's 1.5 us).  Batch 64 x 128 heads x 8192: 197 us, 38 % of what
// cuBLAS reaches in bf16; x 64 heads: 174 us.  With the scores rounded to 24 bits for
// the swap 187 and 180 us, but the log-sum-exp then loses four bits to a plain form
// in fp32.
//
// Per 64-key tile, in each CTA:
//   loader warps  : six, two for each operand stage: 16-byte cp.async of the
//                   tile's codes, scales and rope dims into the warp's raw stage,
//                   then f16 into the operand stage once the value MMAs have read
//                   what was there.
//   MMA warp      : S_part = Q_part K_part^T (A = Q from TMEM, the rope part's from
//                   shared memory), O_half += P V_half (A = P from TMEM, B = the
//                   same stage read MN-major).
//   softmax warps : eight, 16 whole rows each, as in the 128-row kernel.
//
// Every wait is bounded (2 s unless the plan sets another limit); one that runs out
// sets MLA_DEVFLAG_TIMEOUT and the CTA winds down.

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

constexpr int T = mla::kKeyTile;          // 64 keys per tile
constexpr int ATOM = T * 128;             // one 64-dim latent slab of a stage: 64 keys x 128 B
constexpr int RATOM = T * 64;             // the CTA's rope half, 64-byte rows
constexpr int STAGE = 4 * ATOM + RATOM;   // 36 KB of f16 operands
constexpr int NS = 3;                     // operand stages = loader warps
constexpr int RAW_PART = 32 * fp4::kRawRow;  // a loader's 6.5 KB of codes, scales and rope
constexpr int QROPE = 128 * 64;           // the CTA's 32 rope dims of Q, 64-byte rows
// Exchange with the partner CTA: each softmax warp sends and receives the partial
// scores of its 16 rows x 64 keys per tile; a buffer for even tiles and one for odd
// ones.
constexpr int kSoftmaxWarps = 8;
constexpr int RECV_W = 32 * 32 * 4;               // one warp's block (4 KB)
constexpr int RECV = kSoftmaxWarps * RECV_W;      // one tile (32 KB)
// Warps: 0..5 loaders (warps 2 w and 2 w + 1 fill operand stage w, 32 keys each), 6
// MMA, 7 without work, 8..15 softmax.
constexpr int kLoaders = 2 * NS;
constexpr int kSoftmaxWarp0 = 8;
constexpr int kMmaWarp = 6;
constexpr int kThreads = 32 * 16;
// Registers a thread of each group of four warps; the launch gives 128 each.
constexpr int kLoaderRegs = 80, kMixedRegs = 88, kSoftmaxRegs = 168;
static_assert(kLoaderRegs + kMixedRegs + 2 * kSoftmaxRegs <= 4 * 128, "no more than the launch gives");

constexpr int OFF_STAGE = 0;
constexpr int OFF_QROPE = OFF_STAGE + NS * STAGE;
constexpr int OFF_RAW = OFF_QROPE + QROPE;
constexpr int OFF_RECV = OFF_RAW + kLoaders * RAW_PART;
constexpr int OFF_XFREE = OFF_RECV + 2 * RECV;    // [2][8] words that the "buffer free" signals land in
constexpr int OFF_BAR = OFF_XFREE + 128;
constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;  // + barriers + alignment slack
static_assert(SMEM_BYTES <= 232448 && STAGE % 1024 == 0 && OFF_QROPE % 1024 == 0 && OFF_RAW % 16 == 0 &&
                  OFF_RECV % 16 == 0 && OFF_BAR % 8 == 0, "shared memory");

// TMEM columns
constexpr uint32_t TM_O = 0;     // 256 fp32 columns: this CTA's value half
constexpr uint32_t TM_Q = 256;   // 128 columns: 256 f16 of Q, packed in pairs
constexpr uint32_t TM_S = 384;   // two 64-column score buffers; P overwrites them
constexpr uint32_t TM_COLS = 512;

constexpr float kRescaleThreshold = 8.0f;  // log2 units: P may grow to 2^8 before a rescale
constexpr float kMaxSentinel = -1.0e30f;
constexpr uint64_t kDrainNs = 500000000ull;  // bound of the wind-down waits after an abort
constexpr uint32_t kSleepNs = 20000;  // suspend-time hint of a waiting thread

struct Bars {
  uint64_t kv_full[NS];   // operand stage ready (its two loader warps arrive)
  uint64_t kv_empty[NS];  // operand stage consumed by the MMAs
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t recv_full[2][kSoftmaxWarps];  // the partner warp's partial scores landed (4 KB)
  uint64_t recv_free[2][kSoftmaxWarps];  // the partner warp has read what this warp sent
  uint64_t o_done;
  uint64_t o_final;  // the last PV has drained (one phase)
  uint64_t q_ready;
  uint64_t drain;
  uint32_t tmem_base;
  int32_t abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

struct Ctx {
  int32_t* status;
  volatile int32_t* abort;
  uint64_t limit_ns;  // bound of every pipeline wait (FwdParams::wait_ns)
  uint32_t sleep_ns;  // suspend hint of a wait: no longer than the limit, so any limit is reachable
};

// Wait used only while winding down after an abort: ignores the abort word,
// gives up after 0.5 s.
__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (ptx::globaltimer_ns() - t0 > kDrainNs) return false;
  }
  return true;
}

// Bounded wait on an mbarrier phase.  Returns false (and flags the status
// word and the CTA's abort word) if the phase did not complete in time or
// another warp of this CTA already gave up.
__device__ __forceinline__ bool wait(const Ctx& c, uint32_t bar, uint32_t parity) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
    // Sleep on the barrier rather than spin: waiting warps would otherwise
    // take issue slots from the warps that share their sub-partition.  A
    // failed try suspends the thread for up to kSleepNs (the wait limit
    // if that is shorter), so reading the timer after each one costs
    // nothing that matters.
    if (ptx::mbar_try_wait_sleep(bar, parity, c.sleep_ns)) return true;
    if (*c.abort) return false;
    if (ptx::globaltimer_ns() - t0 > c.limit_ns) {
      atomicOr(c.status, MLA_DEVFLAG_TIMEOUT);
      *c.abort = 1;
      return false;
    }
  }
}

// The same, decided for the whole warp: true only if every lane's wait
// succeeded, so warp-collective tcgen05 instructions stay convergent.
__device__ __forceinline__ bool wait_all(const Ctx& c, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(c, bar, parity));
}

// 2^x with the SFU's approximate exp2 (inputs below -126 flush to +0, -inf
// gives +0).  Its relative error is far below the 16-bit rounding the
// weights get next.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// This warp group's share of the launch's registers from here on.
template <int kRegs>
__device__ __forceinline__ void take_registers() {
  if constexpr (kRegs > 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
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

// Eight bf16 -> eight f16 (exact for |x| in [2^-14, 65504]; flags larger values).
__device__ __forceinline__ uint4 bf16x8_to_f16x8(uint4 x, bool& out_of_range) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xFFFF0000u);
    out_of_range |= fabsf(lo) > 65504.f || fabsf(hi) > 65504.f;
    w[i] = pack_f16(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// K-major, 128B-swizzled operand: rows 128 B apart, 8-row groups 1 KB apart.
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t addr) {
  return ptx::smem_desc(addr, 16, 1024, 2);
}

// K-major, 64B-swizzled operand (the rope halves): rows 64 B apart, 8-row groups 512 B apart.
__device__ __forceinline__ uint64_t rope_desc(uint32_t addr) { return ptx::smem_desc(addr, 16, 512, 4); }
__device__ __forceinline__ uint32_t sw64(int r, int c) { return r * 64 + ((c ^ ((r >> 1) & 3)) * 16); }

// The same stage read MN-major as V (N = 256 value dims over 4 slabs 8 KB
// apart, K = keys in 8-row groups 1 KB apart).
__device__ __forceinline__ uint64_t vmajor_desc(uint32_t addr) {
  return ptx::smem_desc(addr, ATOM, 1024, 2);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fwd_fp4_wide_kernel(mla::FwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem + OFF_BAR);
  const uint32_t sbase = ptx::smem_u32(smem);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const uint32_t peer = rank ^ 1u;
  // The work unit: (sequence b, row block rb, key range [k0, k1)), its
  // context, and where its result goes (the final output when the unit
  // covers the whole sequence, else partial slot `part` for the merge).
  int rb, b, ctx, k0, k1;
  bool single;
  size_t part;
  if (p.units != nullptr) {
    // Device-planned: the unit list was written by the planning kernel this
    // one is launched behind, so wait for it first.  Both CTAs of a pair
    // read the same unit and take the same branches.
    ptx::grid_dependency_wait();
    const int u = blockIdx.x >> 1;
    if (u >= *p.n_units) return;
    const int4 d = p.units[u];
    const int4 si = p.seq_info[d.x];
    b = d.x;
    rb = d.y & 0xFF;
    k0 = d.z;
    k1 = d.w;
    ctx = si.x;  // already clamped to what the table holds
    single = si.z == 1;
    part = (size_t)si.y + (d.y >> 8);
  } else {
    rb = blockIdx.x >> 1;
    b = blockIdx.y;
    const int split = blockIdx.z;
    // A context the plan does not cover is clamped to [0, max_ctx] and
    // flagged.  max_ctx keys fit the block table (bt_stride * page_size >=
    // max_ctx is checked on the host) and the splits (num_splits *
    // chunk_len >= max_ctx), so no table entry past the sequence's row is
    // read.
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
  const int n_tiles = k1 > k0 ? (k1 - k0 + T - 1) / T : 0;
  const int vdim0 = (int)rank * 256;  // this CTA's value dims
  const float s_kv = p.kv_scale ? *p.kv_scale : 1.f;

  if (n_tiles == 0) {
    // No key of this split: the row results are out = 0, lse = -inf.  Both
    // CTAs of the pair take this branch together, before any cluster traffic.
    ptx::grid_dependency_wait();
    for (int i = threadIdx.x; i < mla::kRowTile; i += kThreads) {
      const int row = rb * mla::kRowTile + i;
      if (row >= p.rows) break;
      if (single) {
        uint4* o = reinterpret_cast<uint4*>(p.out + ((size_t)b * p.rows + row) * mla::kDV + vdim0);
        for (int c = 0; c < 32; ++c) o[c] = make_uint4(0, 0, 0, 0);
        if (rank == 0) p.lse[(size_t)b * p.rows + row] = -INFINITY;
      } else if (rank == 0) {
        p.part_lse[part * p.rows + row] = -INFINITY;
      }
    }
    return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars.kv_full[s]), 2);
      ptx::mbar_init(ptx::smem_u32(&bars.kv_empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_u32(&bars.s_full[i]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars.p_full[i]), kSoftmaxWarps);
    }
    for (int i = 0; i < 2; ++i)
      for (int w = 0; w < kSoftmaxWarps; ++w) {
        ptx::mbar_init(ptx::smem_u32(&bars.recv_full[i][w]), 1);
        ptx::mbar_init(ptx::smem_u32(&bars.recv_free[i][w]), 1);
      }
    ptx::mbar_init(ptx::smem_u32(&bars.o_done), 1);
    ptx::mbar_init(ptx::smem_u32(&bars.o_final), 1);
    ptx::mbar_init(ptx::smem_u32(&bars.q_ready), 32 * kSoftmaxWarps);
    ptx::mbar_init(ptx::smem_u32(&bars.drain), 1);
    bars.abort = 0;
    ptx::fence_mbar_init_cluster();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&bars.tmem_base), TM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync_all();  // barriers of both CTAs initialised before any remote arrive
  ptx::tc_fence_after();
  // q and the newest cache rows may come from the kernel this one is
  // launched behind (the decode epilogue): nothing past this point reads
  // them, or writes an output, before that kernel has completed.  A no-op
  // when the launch is not a programmatic dependent one.
  ptx::grid_dependency_wait();
  const uint32_t tmem = bars.tmem_base;
  Ctx c{p.status, &bars.abort, p.wait_ns,
        (uint32_t)(p.wait_ns < (uint64_t)kSleepNs ? p.wait_ns : (uint64_t)kSleepNs)};

  // The loaders of both warp groups run this.
  auto load = [&]() {
    // ------------------------------------------------------------ loader ---
    // Loader warps 2 w and 2 w + 1 own operand stage w and copy tiles w, w + NS, ...,
    // 32 keys each, a key a lane: its row's index, then the copies (128 bytes of codes
    // by 8 lanes, 64 of rope by 4 and 16 of scales by 1 a key; 16-byte cp.async, L2
    // only), then its conversion.  The next tile's copies are in flight while the
    // stage waits for its value MMAs.
    const int lw = warp >> 1;   // the operand stage this warp fills
    const int half = 32 * (warp & 1);
    // This sequence's page ids: a row of the padded table, or (CSR form)
    // kv_indices from kv_indptr[b] on.
    const int32_t* bt = p.bt + (p.bt_indptr ? (size_t)p.bt_indptr[b] : (size_t)b * p.bt_stride);
    const uint8_t* cache = static_cast<const uint8_t*>(p.cache);
    auto key_of = [&](int tile) -> int {  // this lane's key, clamped to the split
      const int start = k0 + tile * T;
      return start + min(half + lane, min(T, k1 - start) - 1);
    };
    // key / page_size by a multiply and shifts: the unsigned form of
    // Granlund and Montgomery, "Division by invariant integers using
    // multiplication" (PLDI 1994), exact for every 32-bit key.  With
    // l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
    // q = (t + ((n - t) >> 1)) >> (l - 1) where t = mulhi(m, n); d = 1 is n.
    const uint32_t pdiv = (uint32_t)p.page_size;
    const uint32_t plog = 32u - __clz(pdiv - 1u);
    const uint32_t pmul = (uint32_t)(((1ull << 32) * ((1ull << plog) - pdiv)) / pdiv) + 1u;
    const uint32_t pshift = plog > 0 ? plog - 1u : 0u;
    auto page_of = [&](uint32_t key) -> uint32_t {
      const uint32_t t = __umulhi(pmul, key);
      return pdiv == 1u ? key : (t + ((key - t) >> 1)) >> pshift;
    };
    const uint32_t raw0 = sbase + OFF_RAW + warp * RAW_PART;
    auto page_at = [&](int tile) { return tile < n_tiles ? __ldg(&bt[page_of((uint32_t)key_of(tile))]) : 0; };
    int next_page = page_at(lw);
    for (int t = lw; t < n_tiles; t += NS) {
      int64_t page = next_page;
      next_page = page_at(t + NS);
      if (page < 0 || page >= p.num_pages) {
        atomicOr(p.status, MLA_DEVFLAG_BAD_PAGE);
        page = 0;
      }
      const uint32_t key = (uint32_t)key_of(t);
      const uint32_t rix = (uint32_t)page * pdiv + (key - page_of(key) * pdiv);  // num_pages * page_size < 2^31
      __syncwarp();  // every lane has converted the codes that these replace
      const uint8_t* src[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        src[i] = cache + (size_t)__shfl_sync(0xffffffffu, rix, 4 * i + (lane >> 3)) * fp4::kRow;
      const uint32_t dst = raw0 + (lane >> 3) * fp4::kRawRow + (lane & 7) * 16;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        ptx::cp_async_16(dst + 4 * i * fp4::kRawRow, src[i] + 128 * (int)rank + (lane & 7) * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int kk = 8 * i + (lane >> 2), ch = lane & 3;
        const uint8_t* from = cache + (size_t)__shfl_sync(0xffffffffu, rix, kk) * fp4::kRow;
        ptx::cp_async_16(raw0 + kk * fp4::kRawRow + fp4::kRawRope + ch * 16,
                         from + fp4::kRope + 64 * (int)rank + ch * 16);
      }
      ptx::cp_async_16(raw0 + lane * fp4::kRawRow + fp4::kRawScales,
                       cache + (size_t)rix * fp4::kRow + fp4::kScales + 16 * (int)rank);
      ptx::cp_async_commit();
      ptx::cp_async_wait<0>();
      __syncwarp();  // the other lanes' copies
      if (t >= NS && !wait_all(c, ptx::smem_u32(&bars.kv_empty[lw]), ((t / NS) - 1) & 1)) break;
      const uint32_t out = sbase + OFF_STAGE + lw * STAGE;
      const int kk = half + lane;
      const uint32_t raw = raw0 + lane * fp4::kRawRow, rowp = out + kk * 128;
      const uint4 scales = ld_shared_u4(raw + fp4::kRawScales);
      const uint32_t sc[4] = {scales.x, scales.y, scales.z, scales.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint4 v[4];
        fp4::convert(ld_shared_u4(raw + j * 16), sc[j >> 1] >> (16 * (j & 1)), v);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          st_shared_u4(rowp + (j >> 1) * ATOM + (((4 * (j & 1) + e) ^ (kk & 7)) * 16), v[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        st_shared_u4(out + 4 * ATOM + sw64(kk, e), ld_shared_u4(raw + fp4::kRawRope + e * 16));
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars.kv_full[lw]));
    }
    ptx::cp_async_wait<0>();  // nothing of this warp is in flight when it leaves
  };
  if (warp < 4) {
    take_registers<kLoaderRegs>();
    load();
  } else if (warp < kSoftmaxWarp0) {
    take_registers<kMixedRegs>();
    if (warp < kLoaders) {
      load();
    } else if (warp == kMmaWarp) {
    // --------------------------------------------------------------- MMA ---
    const bool leader = ptx::elect_one();
    constexpr uint32_t id_qk = ptx::idesc_f16(128, T, 0, false, false);
    constexpr uint32_t id_pv = ptx::idesc_f16(128, 256, 0, false, true);
    bool ok = wait_all(c, ptx::smem_u32(&bars.q_ready), 0);
    ptx::tc_fence_after();
    const uint64_t dk = kmajor_desc(sbase + OFF_STAGE);  // slab 0 of stage 0
    const uint64_t dv = vmajor_desc(sbase + OFF_STAGE);  // V of stage 0
    const uint64_t dkr = rope_desc(sbase + OFF_STAGE + 4 * ATOM), dqr = rope_desc(sbase + OFF_QROPE);
    constexpr uint32_t kStageU = STAGE >> 4, kAtomU = ATOM >> 4;
    auto issue_qk = [&](int u, int s) {  // tile u from stage s (u % NS)
      if (!leader) return;
      const uint32_t d = tmem + TM_S + (u & 1) * T;
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          ptx::mma_ts(d, tmem + TM_Q + a * 32 + kk * 8, dk + s * kStageU + a * kAtomU + 2 * kk, id_qk, (a | kk) != 0);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)  // this CTA's 32 rope dims
        ptx::mma_ss(d, dqr + 2 * kk, dkr + s * kStageU + 2 * kk, id_qk, 1);
      ptx::mma_commit(ptx::smem_u32(&bars.s_full[u & 1]));
    };
    auto issue_pv = [&](int t, int s) {  // tile t from stage s (t % NS)
      if (!leader) return;
      const uint32_t pa = tmem + TM_S + (t & 1) * T;
#pragma unroll
      for (int kk = 0; kk < T / 16; ++kk)
        ptx::mma_ts(tmem + TM_O, pa + kk * 8, dv + s * kStageU + kk * (2048 >> 4), id_pv, (t | kk) != 0);
      ptx::mma_commit(ptx::smem_u32(&bars.o_done));
      if (t == n_tiles - 1) ptx::mma_commit(ptx::smem_u32(&bars.o_final));
      ptx::mma_commit(ptx::smem_u32(&bars.kv_empty[s]));
    };
    // Issue whichever is ready: QK^T of tile nq (its stage has landed and its
    // score buffer is free, i.e. the PV of tile nq - 2 is issued; the tensor pipe
    // runs one thread's MMAs in order) or PV of tile np (its weights are written).
    int nq = 0, np = 0;
    int sq = 0, sp = 0;  // stages of tiles nq and np (t % NS)
    uint32_t phq = 0;    // phase parity of tile nq's stage barrier
    uint64_t t_last = ptx::globaltimer_ns();
    uint32_t idle = 0;
    while (ok && np < n_tiles) {
      bool progress = false;
      if (np < nq && __all_sync(0xffffffffu, ptx::mbar_test_wait(ptx::smem_u32(&bars.p_full[np & 1]), (np >> 1) & 1))) {
        ptx::tc_fence_after();
        issue_pv(np++, sp);
        __syncwarp();
        sp = sp == NS - 1 ? 0 : sp + 1;
        progress = true;
      }
      if (nq < n_tiles && nq <= np + 1 &&
          __all_sync(0xffffffffu, ptx::mbar_test_wait(ptx::smem_u32(&bars.kv_full[sq]), phq))) {
        ptx::tc_fence_after();
        issue_qk(nq++, sq);
        __syncwarp();
        if (sq == NS - 1) {
          sq = 0;
          phq ^= 1u;
        } else {
          ++sq;
        }
        progress = true;
      }
      if (progress) {
        idle = 0;
        t_last = 0;
        continue;
      }
      if ((++idle & 63) == 0) {
        const uint64_t now = ptx::globaltimer_ns();
        if (t_last == 0) t_last = now;
        if (*c.abort) {
          ok = false;
        } else if (now - t_last > c.limit_ns) {
          atomicOr(c.status, MLA_DEVFLAG_TIMEOUT);
          *c.abort = 1;
          ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    __syncwarp();
    }
  } else {
    take_registers<kSoftmaxRegs>();
    // ----------------------------------------------------------- softmax ---
    // Softmax warp sw (0..7) owns 16 whole rows of the 128-row block: TMEM
    // lanes lbase .. lbase + 15 with lbase = 32 (warp % 4) + 16 (sw / 4) (a
    // warp reaches the lane quarter warp % 4 only).  Through the 16x256b
    // access shape thread i holds rows rA = lbase + i/4 and rB = rA + 8, and
    // of every 8-key group j the keys 8j + 2(i%4) and 8j + 2(i%4) + 1: a row's
    // 64 keys are spread over the 4 threads of a quad, whose shuffles give the
    // row max and sum.  The partner CTA's warp sw holds the same elements.
    const int sw = warp - kSoftmaxWarp0;
    const int q4 = warp & 3;                   // TMEM lane quarter of this warp
    const int g = sw >> 2;                     // which half of the quarter
    const int lbase = q4 * 32 + g * 16;
    const int cq = lane & 3;                   // column pair within each 8-key group
    const int rA = lbase + (lane >> 2), rB = rA + 8;
    const uint32_t lanes16 = (uint32_t)lbase << 16;
    auto visible = [&](int r) {  // keys [k0, visible) of this split that row r sees
      const int row = rb * mla::kRowTile + r;
      if (row >= p.rows) return 0;
      const int tok = row / p.heads;
      int nvis = p.causal ? ctx - p.sq + tok + 1 : ctx;
      nvis = max(0, min(nvis, ctx));
      return min(nvis, k1);
    };
    const int visA = visible(rA), visB = visible(rB);

    // Q (this CTA's 256 latent dims) -> TMEM as 16-bit pairs: thread i of
    // the two warps of a lane quarter writes row 32 q4 + i, two 64-dim chunks
    // each; in both CTAs the second warp also puts the CTA's 32 rope dims into
    // shared memory (64B-swizzled K-major).
    {
      const int r = q4 * 32 + lane;
      const int row = rb * mla::kRowTile + r;
      const bool valid_row = row < p.rows;
      const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
      const uint4* qv = reinterpret_cast<const uint4*>(p.q + ((size_t)b * p.rows + row) * mla::kDQK);
      uint32_t buf[32];
      bool q_range = false;
      for (int chunk = 2 * g; chunk < 2 * g + 2; ++chunk) {
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          uint4 x = valid_row ? qv[(vdim0 + chunk * 64) / 8 + v] : make_uint4(0, 0, 0, 0);
          x = bf16x8_to_f16x8(x, q_range);
          buf[v * 4 + 0] = x.x;
          buf[v * 4 + 1] = x.y;
          buf[v * 4 + 2] = x.z;
          buf[v * 4 + 3] = x.w;
        }
        ptx::tmem_st32(tmem + lanes + TM_Q + chunk * 32, buf);
      }
      if (g == 1) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint4 x = valid_row ? qv[512 / 8 + 4 * (int)rank + v] : make_uint4(0, 0, 0, 0);
          x = bf16x8_to_f16x8(x, q_range);
          *reinterpret_cast<uint4*>(smem + OFF_QROPE + sw64(r, v)) = x;
        }
        ptx::fence_proxy_async_smem();
      }
      if (q_range) atomicOr(p.status, MLA_DEVFLAG_Q_RANGE);
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      ptx::mbar_arrive(ptx::smem_u32(&bars.q_ready));
    }

    const float c2 = p.softmax_scale * s_kv * 1.4426950408889634f;
    float mA = kMaxSentinel, mB = kMaxSentinel;  // running maxima (log2 domain), quad-uniform
    float lA = 0.f, lB = 0.f;                     // exact row sums over this thread's keys
    // Of receive buffer i: this warp's block, and the partner's addresses.
    auto my_recv = [&](int i) { return sbase + OFF_RECV + i * RECV + sw * RECV_W; };
    const uint32_t peer_recv0 = ptx::mapa(sbase + OFF_RECV + sw * RECV_W, peer);
    const uint32_t peer_xfree0 = ptx::mapa(sbase + OFF_XFREE + sw * 4, peer);
    const uint32_t peer_full0 = ptx::mapa(ptx::smem_u32(&bars.recv_full[0][sw]), peer);
    const uint32_t peer_free0 = ptx::mapa(ptx::smem_u32(&bars.recv_free[0][sw]), peer);
    // A warp whose 16 rows are all past the problem's rows swaps nothing and
    // computes nothing; it only keeps the barrier phases moving.  Both CTAs skip the
    // same warps.  Its TMEM lanes hold garbage that no output reads (the MMAs keep
    // rows apart).
    const bool live = rb * mla::kRowTile + lbase < p.rows;
    // s[4j + e]: e = 0, 1 -> row A keys 8j + 2cq + e; e = 2, 3 -> row B
    auto load_scores = [&](int t, float (&s)[32]) {
      uint32_t raw[32];
      ptx::tmem_ld16x256b_x8(tmem + lanes16 + TM_S + (t & 1) * T, raw);
      ptx::tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(raw[i]);
    };
    bool ok = true;
    for (int t = 0; t < n_tiles; ++t) {
      const int buf = t & 1;
      if (!wait_all(c, ptx::smem_u32(&bars.s_full[buf]), (t >> 1) & 1)) { ok = false; break; }
      if (!live) {
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars.p_full[buf]));
        continue;
      }
      ptx::tc_fence_after();
      float s[32];
      load_scores(t, s);
      // The partner has read the block of tile t - 2 from this tile's buffer.
      if (t >= 2) {
        const uint32_t free_bar = ptx::smem_u32(&bars.recv_free[buf][sw]);
        if (lane == 0) ptx::mbar_arrive_expect_tx(free_bar, 4);
        if (!wait_all(c, free_bar, ((t >> 1) - 1) & 1)) { ok = false; break; }
      }
      {
        const uint32_t dst = peer_recv0 + buf * RECV + lane * 16;
        const uint32_t bar = peer_full0 + buf * (8 * kSoftmaxWarps);
#pragma unroll
        for (int v = 0; v < 8; ++v)
          ptx::st_async_u4(dst + v * 512, __float_as_uint(s[4 * v]), __float_as_uint(s[4 * v + 1]),
                           __float_as_uint(s[4 * v + 2]), __float_as_uint(s[4 * v + 3]), bar);
      }
      {
        const uint32_t full = ptx::smem_u32(&bars.recv_full[buf][sw]);
        if (lane == 0) ptx::mbar_arrive_expect_tx(full, RECV_W);
        if (!wait_all(c, full, (t >> 1) & 1)) { ok = false; break; }
        const uint32_t src = my_recv(buf) + lane * 16;
        uint32_t fold = 0;
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const uint4 x = ld_shared_u4(src + v * 512);
          fold ^= x.x ^ x.y ^ x.z ^ x.w;
          s[4 * v] += __uint_as_float(x.x);
          s[4 * v + 1] += __uint_as_float(x.y);
          s[4 * v + 2] += __uint_as_float(x.z);
          s[4 * v + 3] += __uint_as_float(x.w);
        }
        // The buffer is read (the vote needs every lane's loaded words): the
        // partner may send the tile after next.
        const bool any = __any_sync(0xffffffffu, fold == 0x9E3779B9u);
        if (t + 2 < n_tiles && lane == 0)
          ptx::st_async_b32(peer_xfree0 + buf * 32, any ? 1u : 0u, peer_free0 + buf * (8 * kSoftmaxWarps));
      }
      // Row maxima over the visible keys of this tile (log2 domain).  Only the
      // last tile of a split and causal rows need the mask.
      const int tile0 = k0 + t * T;
      const int limA = visA - tile0, limB = visB - tile0;  // visible keys of this tile
      const bool fullA = limA >= T, fullB = limB >= T;
      // Every key of the tile visible to every row of the warp (all tiles but
      // a split's last, outside causal masking): the mask-free path.
      const bool all_full = __all_sync(0xffffffffu, fullA && fullB);
      float mxA = -INFINITY, mxB = -INFINITY;
      if (all_full) {
        float xa[4], xb[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          xa[u] = fmaxf(fmaxf(s[8 * u], s[8 * u + 1]), fmaxf(s[8 * u + 4], s[8 * u + 5]));
          xb[u] = fmaxf(fmaxf(s[8 * u + 2], s[8 * u + 3]), fmaxf(s[8 * u + 6], s[8 * u + 7]));
        }
        mxA = fmaxf(fmaxf(xa[0], xa[1]), fmaxf(xa[2], xa[3]));
        mxB = fmaxf(fmaxf(xb[0], xb[1]), fmaxf(xb[2], xb[3]));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = 8 * j + 2 * cq + e;
            if (k < limA) mxA = fmaxf(mxA, s[4 * j + e]);
            if (k < limB) mxB = fmaxf(mxB, s[4 * j + 2 + e]);
          }
      }
      mxA = fmaxf(mxA, __shfl_xor_sync(0xffffffffu, mxA, 1));
      mxB = fmaxf(mxB, __shfl_xor_sync(0xffffffffu, mxB, 1));
      mxA = fmaxf(mxA, __shfl_xor_sync(0xffffffffu, mxA, 2));
      mxB = fmaxf(mxB, __shfl_xor_sync(0xffffffffu, mxB, 2));
      const float mtA = limA > 0 ? mxA * c2 : -INFINITY;
      const float mtB = limB > 0 ? mxB * c2 : -INFINITY;
      const bool needA = mtA > mA + kRescaleThreshold, needB = mtB > mB + kRescaleThreshold;
      if (__any_sync(0xffffffffu, needA || needB)) {
        const float nA = needA ? fmaxf(mA, mtA) : mA, nB = needB ? fmaxf(mB, mtB) : mB;
        const float alA = exp2f(mA - nA), alB = exp2f(mB - nB);
        if (t > 0) {
          // This warp's rows of the CTA's O half; the PV of the previous tile
          // must have finished accumulating.  One parity wait on o_done is
          // enough: QK^T of this tile was issued after PV of tile t - 2 and
          // the pipe runs in order, so that PV has finished and o_done is at
          // most one phase short.  (A deeper score ring breaks this.)
          if (!wait_all(c, ptx::smem_u32(&bars.o_done), (t - 1) & 1)) { ok = false; break; }
          ptx::tc_fence_after();
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t o[32];
            const uint32_t col = tmem + lanes16 + TM_O + ch * 64;
            ptx::tmem_ld16x256b_x8(col, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * ((i & 2) ? alB : alA));
            ptx::tmem_st16x256b_x8(col, o);
          }
        }
        lA *= alA;
        lB *= alB;
        mA = nA;
        mB = nB;
      }
      // Weights p = 2^(s*c2 - m) (s now holds them); the row sums are exact.
      uint32_t pk[16];  // weights as 16-bit pairs (16x128b order)
      {
        const float nmA = -mA, nmB = -mB;
        float sA = 0.f, sB = 0.f;
        if (all_full) {
          float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            s[i] = fast_exp2(fmaf(s[i], c2, (i & 2) ? nmB : nmA));
            ps[i & 3] += s[i];
          }
          sA = ps[0] + ps[1];
          sB = ps[2] + ps[3];
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int k = 8 * j + 2 * cq;
            const float a0 = fast_exp2(fmaf(s[4 * j], c2, nmA));
            const float a1 = fast_exp2(fmaf(s[4 * j + 1], c2, nmA));
            const float b0 = fast_exp2(fmaf(s[4 * j + 2], c2, nmB));
            const float b1 = fast_exp2(fmaf(s[4 * j + 3], c2, nmB));
            s[4 * j] = k < limA ? a0 : 0.f;
            s[4 * j + 1] = k + 1 < limA ? a1 : 0.f;
            s[4 * j + 2] = k < limB ? b0 : 0.f;
            s[4 * j + 3] = k + 1 < limB ? b1 : 0.f;
            sA += s[4 * j] + s[4 * j + 1];
            sB += s[4 * j + 2] + s[4 * j + 3];
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          pk[2 * j] = pack_f16(s[4 * j], s[4 * j + 1]);
          pk[2 * j + 1] = pack_f16(s[4 * j + 2], s[4 * j + 3]);
        }
        lA += sA;
        lB += sB;
      }
      // P columns of this tile: key pair (2m, 2m + 1) at column m; thread i
      // holds pairs 4j + i%4, which is where the 16x128b shape writes.
      const uint32_t pcol = tmem + lanes16 + TM_S + buf * T;
      ptx::tmem_st16x128b_x8(pcol, pk);
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars.p_full[buf]));
    }

    // ---------------------------------------------------------- epilogue ---
    // Row sums over the quad, in the same order in both CTAs.
    lA += __shfl_xor_sync(0xffffffffu, lA, 1);
    lB += __shfl_xor_sync(0xffffffffu, lB, 1);
    lA += __shfl_xor_sync(0xffffffffu, lA, 2);
    lB += __shfl_xor_sync(0xffffffffu, lB, 2);
    if (ok && live && wait_all(c, ptx::smem_u32(&bars.o_final), 0)) {
      // O is final once the last PV has drained (a barrier of its own: a
      // parity wait on o_done only tells the current phase from the one
      // before it, and o_done may be one phase short or already complete).
      ptx::tc_fence_after();
      const bool someA = !(lA <= 0.f), someB = !(lB <= 0.f);  // a sum that is NaN is no empty row
      const float invA = someA ? s_kv / lA : 0.f, invB = someB ? s_kv / lB : 0.f;
      const int rowA = rb * mla::kRowTile + rA, rowB = rb * mla::kRowTile + rB;
      const bool okA = rowA < p.rows, okB = rowB < p.rows;
      const size_t pA = part * p.rows + rowA;
      const size_t pB = part * p.rows + rowB;
#pragma unroll 1
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t o[32];
        ptx::tmem_ld16x256b_x8(tmem + lanes16 + TM_O + ch * 64, o);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int dim = vdim0 + ch * 64 + 8 * j + 2 * cq;
          const float a0 = __uint_as_float(o[4 * j]) * invA, a1 = __uint_as_float(o[4 * j + 1]) * invA;
          const float b0 = __uint_as_float(o[4 * j + 2]) * invB, b1 = __uint_as_float(o[4 * j + 3]) * invB;
          if (single) {
            if (okA) *reinterpret_cast<uint32_t*>(p.out + ((size_t)b * p.rows + rowA) * mla::kDV + dim) = pack_bf16(a0, a1);
            if (okB) *reinterpret_cast<uint32_t*>(p.out + ((size_t)b * p.rows + rowB) * mla::kDV + dim) = pack_bf16(b0, b1);
          } else {
            if (okA) *reinterpret_cast<float2*>(p.part_o + pA * mla::kDV + dim) = make_float2(a0, a1);
            if (okB) *reinterpret_cast<float2*>(p.part_o + pB * mla::kDV + dim) = make_float2(b0, b1);
          }
        }
      }
      if (rank == 0 && cq == 0) {
        const float lseA = someA ? (mA + log2f(lA)) * 0.6931471805599453f : -INFINITY;
        const float lseB = someB ? (mB + log2f(lB)) * 0.6931471805599453f : -INFINITY;
        if (single) {
          if (okA) p.lse[(size_t)b * p.rows + rowA] = lseA;
          if (okB) p.lse[(size_t)b * p.rows + rowB] = lseB;
        } else {
          if (okA) p.part_lse[pA] = lseA;
          if (okB) p.part_lse[pB] = lseB;
        }
      }
    }
    ptx::tc_fence_before();
  }

  // ------------------------------------------------------------ teardown ---
  __syncthreads();
  if (warp == kMmaWarp) {
    if (bars.abort) {
      // wait for every tcgen05 op this CTA issued before giving TMEM back
      if (ptx::elect_one()) {
        ptx::mma_commit(ptx::smem_u32(&bars.drain));
        wait_drain(ptx::smem_u32(&bars.drain), 0);
      }
      __syncwarp();
    }
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, TM_COLS);
  }
  ptx::cluster_sync_all();  // no CTA leaves while its partner may still write into it
}

}  // namespace

int mla_launch_fwd_fp4_wide_sm103(const mla::FwdParams& p, void* stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  e = mla::opt_in_smem(reinterpret_cast<const void*>(fwd_fp4_wide_kernel), SMEM_BYTES, dev, 12);
  if (e != cudaSuccess) return (int)e;
  // Splits vary slowest, so every sequence's first chunk is dispatched
  // before any second chunk (the planner simulates this order).  Launched as
  // a programmatic dependent: behind the decode epilogue the prologue
  // (barrier set-up, TMEM allocation) overlaps that kernel's tail.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = p.units != nullptr ? dim3(2 * p.unit_capacity, 1, 1)
                                  : dim3(p.row_blocks * 2, p.batch, p.num_splits);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, fwd_fp4_wide_kernel, p);
}
