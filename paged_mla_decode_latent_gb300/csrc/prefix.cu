// prefix.cu -- decode attention for a batch that shares a prefix: the plan,
// the staging of keys and queries, the merge and the entry points.
//
// With P shared keys, sequence b's query rows attend to the shared keys and to
// its own keys [P, ctx_b) under one softmax.  One call queues:
//   stage   shared keys (through prefix_table), query rows and, where they are
//           folded in, the own keys -> f16 rows in the workspace; the
//           partition of the tiles over the CTA pairs
//   prefix  prefix_sm103.cu
//   own     where they are not folded in: the decode kernels over keys [P,
//           ctx_b) of each sequence
//   merge   the partials of a row:
//             L = ln sum_s e^lse_s,   out = sum_s e^(lse_s - L) o_s

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/mla_decode.h"
#include "internal.h"
#include "ptx.cuh"

namespace {

constexpr uint64_t kDefaultWaitNs = 2000000000ull;
constexpr int kPieces = 72;  // 8-element pieces of a 576-wide row
constexpr int kMaxPairs = 256;
constexpr int kChunk = 32;  // rows a staging CTA copies
constexpr int kStageThreads = 256;
constexpr int kStageIters = kChunk * kPieces / kStageThreads;  // 9 pieces a thread
static_assert(kStageThreads == 8 * kChunk, "eight threads a row");
constexpr int kLatentIters = MLA_D_V / 64;  // of them latent values
static_assert(kLatentIters == kStageIters - 1, "the last piece is the rope dims");
constexpr int kLowExponent = -8;  // bf16 rows whose latent values are all below 2^-8 are lifted
constexpr float kLowLatent = 0x1p-8f;
constexpr int kPadChunks = mla::kPrefixTile / kChunk;
constexpr int kManyParts = 8;  // partials a row from which the merge takes eight warps a row
// Own keys are folded in while they are at most this many, and their row
// blocks' regions (whole tiles) at most that many rows of 1152 bytes.
constexpr int64_t kMaxOwnRows = 1 << 18, kMaxRegionRows = 1 << 20;

struct StageParams {
  mla::PrefixShape g;
  const void* cache;
  int64_t num_pages;
  const int32_t* prefix_table;
  const int32_t* block_table;
  int64_t bt_stride;
  const uint16_t* q;
  uint16_t* k_out;  // f16 [tiles * 256 + row blocks * block_keys, 576]
  uint16_t* q_out;  // f16 [rows, 576]
  int page_size, fp8;
  int prefix_chunks, q_chunks, own_chunks;  // own_chunks: per (row block, sequence)
};

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  const __half2 v = __floats2half2_rn(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// True if one of two f16 values is infinite or NaN: what a bf16 value beyond
// 65504 (or itself not finite) becomes.
__device__ __forceinline__ bool not_finite(uint32_t w) {
  return (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u;
}

__device__ __forceinline__ uint4 to_f16(uint4 v, bool fp8) {
  if (!fp8)
    return make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z), bf16x2_to_f16x2(v.w));
  const uint32_t c[2] = {v.x, v.y};
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)  // exact for every code; NaN codes become NaN
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(w[e]) : "h"((uint16_t)(c[e >> 1] >> (16 * (e & 1)))));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The binary orders that a row of small values is lifted by: as few steps as bring
// its largest latent value to kLowLatent, while its largest of all, `top`, stays
// below 2^15 (both a float's bits; for a query, whose latent values are nothing by
// themselves, and for a row without any, `latent` is `top`).  No more than that: a
// key's weight shrinks by as much, and has to stand beside those of keys that are
// just not lifted (with lifted rows brought to 2^15, light keys beside such a one
// were lost, 6% of the output).
__device__ __forceinline__ int lift_of(uint32_t latent, uint32_t top) {
  const int want = kLowExponent - ((int)(latent >> 23) - 127);
  const int room = 14 - ((int)(top >> 23) - 127);
  const int e = (max(0, want) + mla::kLiftStep - 1) / mla::kLiftStep * mla::kLiftStep;
  return min(min(e, mla::kMaxLift), max(0, room) / mla::kLiftStep * mla::kLiftStep);
}

__device__ __forceinline__ uint32_t lifted(uint32_t w, float by) {
  const __half2 v = __floats2half2_rn(__uint_as_float(w << 16) * by, __uint_as_float(w & 0xFFFF0000u) * by);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ __half2 abs2(uint32_t w) { return __habs2(*reinterpret_cast<const __half2*>(&w)); }

__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
  if ((w & 0x7C00u) == 0x7C00u) w &= 0xFFFF0000u;
  if ((w & 0x7C000000u) == 0x7C000000u) w &= 0xFFFFu;
  return w;
}

// Stages a row again that is not as it should be, and returns its note.  Called by
// the row's eight lanes, pieces as in the staging; rare, so out of line.  `src`:
// the row in bf16, looked at only where all lanes find it low.
__device__ __noinline__ uint32_t stage_again(const uint16_t* src, uint16_t* dst, bool over, bool low, bool query) {
  const uint32_t row_lanes = 0xFFu << (threadIdx.x & 24);
  uint4* out = reinterpret_cast<uint4*>(dst) + (threadIdx.x & 7);
  if (__any_sync(row_lanes, over)) {
    // A query value spoils its own row only; a key goes without what f16 cannot
    // hold (0 x NaN would spoil rows that do not see it).
#pragma unroll 1
    for (int i = 0; over && !query && i < kStageIters; ++i) {
      const uint4 w = out[8 * i];
      out[8 * i] = make_uint4(finite_or_zero(w.x), finite_or_zero(w.y), finite_or_zero(w.z), finite_or_zero(w.w));
    }
    return mla::kStagedRange;
  }
  if (!__all_sync(row_lanes, low)) return 0;
  const uint4* from = reinterpret_cast<const uint4*>(src) + (threadIdx.x & 7);
  uint32_t latent = 0, most = 0;  // largest magnitudes, as a float's bits
#pragma unroll 1
  for (int i = 0; i < kStageIters; ++i) {
    const uint4 w = from[8 * i];
    const uint32_t a = max(w.x & 0x7FFF0000u, w.x << 17 >> 1), b = max(w.y & 0x7FFF0000u, w.y << 17 >> 1);
    const uint32_t c = max(w.z & 0x7FFF0000u, w.z << 17 >> 1), d = max(w.w & 0x7FFF0000u, w.w << 17 >> 1);
    most = max(most, max(max(a, b), max(c, d)));
    if (i < kLatentIters) latent = most;
  }
  latent = __reduce_max_sync(row_lanes, latent);
  most = __reduce_max_sync(row_lanes, most);
  if (query || latent == 0) latent = most;
  const int lift = most == 0 ? 0 : lift_of(latent, most);
  const float by = __uint_as_float((uint32_t)(127 + lift) << 23);
#pragma unroll 1
  for (int i = 0; lift > 0 && i < kStageIters; ++i) {
    const uint4 w = from[8 * i];
    out[8 * i] = make_uint4(lifted(w.x, by), lifted(w.y, by), lifted(w.z, by), lifted(w.w, by));
  }
  return (uint32_t)(lift / mla::kLiftStep) << mla::kStagedLift;
}

// The tiles of each row block, where each pair starts and where each sequence's
// own keys lie in its row blocks' regions.
__device__ void partition(const StageParams& p) {
  __shared__ int64_t warp_sum[kStageThreads / 32];
  __shared__ int64_t carry_s;
  const mla::PrefixShape& g = p.g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    carry_s = 0;
    *g.status = 0;  // the only bits that the staging sets itself are below
  }
  __syncthreads();
  int64_t mine = 0;
  int mine_n = 0;
  for (int j0 = 0; j0 < g.row_blocks; j0 += kStageThreads) {
    const int j = j0 + threadIdx.x;
    int64_t n = 0;
    if (j < g.row_blocks) {
      int own = 0;
      if (g.fold) {
        const int b0 = g.first_seq(j), b1 = g.last_seq(j);
        for (int b = b0; b <= b1; b += 8) {  // eight loads in flight
          int keys[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) keys[k] = b + k <= b1 ? g.own(b + k) : 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (b + k <= b1) g.own_off[j * g.block_seqs + b + k - b0] = own;
            own += keys[k];
          }
        }
      }
      const int tiles = g.tiles + (own + mla::kPrefixTile - 1) / mla::kPrefixTile;
      g.block_tiles[j] = tiles;
      n = tiles + mla::kSegmentTiles;
    }
    int64_t x = n;  // inclusive scan over the threads
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int64_t before = carry_s;
    for (int k = 0; k < warp; ++k) before += warp_sum[k];
    if (j < g.row_blocks) {
      mine = before + x - n;
      mine_n = (int)n;
      g.first_unit[j] = mine;
    }
    __syncthreads();
    if (threadIdx.x == kStageThreads - 1) carry_s = before + x;
    __syncthreads();
  }
  const mla::PrefixShares shares(carry_s, g.pairs);
  for (int j = threadIdx.x; j < g.row_blocks; j += kStageThreads) {
    // One batch of row blocks is still in registers.
    const bool here = g.row_blocks <= kStageThreads;
    const int64_t a = here ? mine : g.first_unit[j];
    const int tiles = here ? mine_n - mla::kSegmentTiles : g.block_tiles[j];
    // Tile t of the block is unit a + kSegmentTiles + t; a share that starts in
    // the units before starts at tile 0.
    const int first = shares.pair_of(a + mla::kSegmentTiles);
    const int last = shares.pair_of(a + mla::kSegmentTiles + tiles - 1);
    g.parts[j] = make_int2(first, last - first + 1);
    for (int i = last; i >= 0; --i) {
      const int64_t s = shares.start(i);
      if (s < a) break;
      g.pair_start[i] = make_int4(j, (int)max((int64_t)0, s - a - mla::kSegmentTiles), tiles, 0);
    }
  }
  // The end, and pairs past the last unit (own keys that the plan counted on).
  for (int i = (int)min((int64_t)g.pairs, carry_s) + threadIdx.x; i <= g.pairs; i += kStageThreads)
    g.pair_start[i] = make_int4(g.row_blocks, 0, 0, 0);
  // Contexts out of range, once per sequence.
  for (int b = threadIdx.x; b < g.batch; b += kStageThreads)
    if (g.seq_lens[b] < 0 || g.seq_lens[b] > g.max_ctx) atomicOr(g.status, MLA_DEVFLAG_CTX_RANGE);
}

// CTA 0: the partition.  Then one CTA per 32 rows: shared keys (with zeros up
// to the tile's end), query rows, own keys (row block by row block, sequence
// by sequence, then the zeros up to the last tile's end).  Bound by memory:
// 1152 or 576 B in and 1152 B out a row, 9 loads in flight a thread.  Flags go
// out as a byte for every row, not into words that something would have to
// clear first: a clearing kernel before this one cost 1 us, and 2 of host time.
//
// f16 loses bits below 2^-14 (an absolute 2^-25).  A bf16 row whose latent
// values are all below kLowLatent is staged once more, times a power of two that
// the attention undoes; any row is then off by at most 2^-17 of its largest
// latent value.  Ordinary rows pay for one vote.
__global__ void __launch_bounds__(kStageThreads) stage_kernel(StageParams p) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const mla::PrefixShape& g = p.g;
  if (blockIdx.x == 0) {
    partition(p);
    return;
  }
  int u = blockIdx.x - 1;
  // Rows [0, n) of this CTA go to `dst`; the first n_src of them come from
  // `src` or through a page table (from key `key0` of it), the rest are zero.
  int n = kChunk, n_src = 0, key0 = 0;
  const uint16_t* src = nullptr;
  const int32_t* table = nullptr;
  int64_t dst_row = 0;
  uint16_t* dst = p.k_out;
  if (u < p.prefix_chunks) {
    key0 = u * kChunk;
    dst_row = key0;
    n_src = min(kChunk, max(0, g.prefix_len - key0));
    table = p.prefix_table;
  } else if ((u -= p.prefix_chunks) < p.q_chunks) {
    const int r0 = u * kChunk;
    n = n_src = min(kChunk, g.rows - r0);
    src = p.q + (int64_t)r0 * MLA_D_QK;
    dst = p.q_out;
    dst_row = r0;
  } else {
    u -= p.q_chunks;
    const int per_block = g.block_seqs * p.own_chunks + kPadChunks;
    const int j = u / per_block, k = (u - j * per_block) / p.own_chunks;
    const int c = u - j * per_block - k * p.own_chunks;
    const int b0 = g.first_seq(j), b1 = g.last_seq(j);
    const bool pad = k >= g.block_seqs;
    const int b = b0 + k;
    const int first_key = c * kChunk;  // of the sequence's own
    int own = 0;
    if (!pad) {
      if (b > b1) return;
      own = g.own(b);
      if (first_key >= own) return;
    }
    // Own keys of the block's sequences before this one (pad: of all).
    __shared__ int sum_s;
    if (threadIdx.x == 0) sum_s = 0;
    __syncthreads();
    int part = 0;
    for (int i = b0 + threadIdx.x; i <= (pad ? b1 : b - 1); i += kStageThreads) part += g.own(i);
    if (part > 0) atomicAdd(&sum_s, part);
    __syncthreads();
    const int64_t region = (int64_t)g.tiles * mla::kPrefixTile + (int64_t)j * g.block_keys;
    if (pad) {
      const int end = (sum_s + mla::kPrefixTile - 1) / mla::kPrefixTile * mla::kPrefixTile;
      const int at = sum_s + (u - j * per_block - g.block_seqs * p.own_chunks) * kChunk;
      n = min(kChunk, end - at);
      if (n <= 0) return;
      dst_row = region + at;
    } else {
      n = n_src = min(kChunk, own - first_key);
      table = p.block_table + (int64_t)b * p.bt_stride;
      key0 = g.prefix_len + first_key;
      dst_row = region + sum_s + first_key;
    }
  }
  // Eight threads a row, nine pieces each: one page id and one division a row,
  // and every access of eight lanes is a whole 128-byte line.
  const int row = threadIdx.x >> 3, sub = threadIdx.x & 7;
  if (row >= n) return;
  uint4 v[kStageIters];
  bool fp8 = false, bad_page = false;
  uint32_t at_row = 0;  // below 2^31, as num_pages * page_size is
  if (row < n_src && src != nullptr) {
    const uint4* at = reinterpret_cast<const uint4*>(src + row * MLA_D_QK) + sub;
#pragma unroll
    for (int i = 0; i < kStageIters; ++i) v[i] = at[8 * i];
  } else if (row < n_src) {
    const uint32_t key = (uint32_t)(key0 + row), page_i = key / (uint32_t)p.page_size;
    int64_t page = table[page_i];
    bad_page = page < 0 || page >= p.num_pages;
    if (bad_page) page = 0;
    at_row = (uint32_t)(page * p.page_size + (key - page_i * (uint32_t)p.page_size));
    fp8 = p.fp8;
    if (fp8) {
      const uint2* at = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.cache) + (int64_t)at_row * MLA_D_QK) + sub;
#pragma unroll
      for (int i = 0; i < kStageIters; ++i) {
        const uint2 c = at[8 * i];
        v[i] = make_uint4(c.x, c.y, 0, 0);
      }
    } else {
      const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.cache) + (int64_t)at_row * MLA_D_QK) + sub;
#pragma unroll
      for (int i = 0; i < kStageIters; ++i) v[i] = at[8 * i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kStageIters; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  uint4* out = reinterpret_cast<uint4*>(dst + (dst_row + row) * MLA_D_QK) + sub;
  // Largest magnitudes of the latent values and of all; NaN if there is one.
  __half2 latent_top = __floats2half2_rn(0.f, 0.f), top;
#pragma unroll
  for (int i = 0; i < kStageIters; ++i) {
    const uint4 w = to_f16(v[i], fp8);
    out[8 * i] = w;
    const __half2 most = __hmax2_nan(__hmax2_nan(abs2(w.x), abs2(w.y)), __hmax2_nan(abs2(w.z), abs2(w.w)));
    if (i < kLatentIters) latent_top = __hmax2_nan(latent_top, most);
    else top = __hmax2_nan(latent_top, most);
  }
  const bool over = not_finite(*reinterpret_cast<const uint32_t*>(&top));
  const bool low = !fp8 && row < n_src && __hblt2(latent_top, __float2half2_rn(kLowLatent));
  const uint32_t row_lanes = 0xFFu << (threadIdx.x & 24);
  uint32_t note = 0;
  if (__any_sync(row_lanes, over || low))
    note = stage_again(src != nullptr ? src + row * MLA_D_QK
                                      : static_cast<const uint16_t*>(p.cache) + (int64_t)at_row * MLA_D_QK,
                       dst + (dst_row + row) * MLA_D_QK, over, low, src != nullptr);
  if (sub == 0)
    (src != nullptr ? g.row_flags : g.key_flags)[dst_row + row] = (uint8_t)(note | (bad_page ? mla::kStagedBadPage : 0));
}

struct MergeParams {
  mla::PrefixShape g;
  const float* pre_o;    // [row blocks + pairs, 128, 512]
  const float* pre_lse;  // [row blocks + pairs, 128]
  const float* own_o;    // [B, splits, rows, 512]
  const float* own_lse;  // [B, splits, rows]
  uint16_t* out;
  float* lse;
  int splits;            // of the own keys, where they are not folded in
};

// kWarps warps a row, eight warps a CTA; rows of blocks that one pair finished
// return at once.  Warp w of a row takes partials w, w + kWarps, ... under the
// row's maximum, 16 value dims a lane, and the warps' sums are added through
// shared memory.  A partial's row is loaded beside the log-sum-exps (its weight
// is needed only afterwards).  Bound by the round trips to L2, 2 KB a partial:
// a warp a row does best while there are few partials (batch 64 x 128 heads,
// two or three: 12 us, 17 with four warps sharing the dims), eight with many
// (512 rows of 18: 9 us, 13 with the dims shared).
template <int kWarps>
__global__ void __launch_bounds__(256) merge_kernel(MergeParams p) {
  const mla::PrefixShape& g = p.g;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % kWarps;
  const int r = blockIdx.x * (8 / kWarps) + (threadIdx.x >> 5) / kWarps;
  __shared__ float4 acc_s[kWarps][kWarps > 1 ? 128 : 1];
  __shared__ float sum_s[kWarps];
  ptx::grid_dependency_wait();
  if (r >= g.rows) return;  // with one row a CTA: never
  const int b = r / g.rows_per_seq, local = r - b * g.rows_per_seq, j = r / mla::kRowTile;
  int2 part = make_int2(0, 0);  // pairs that hold a part of the row's block
  if (g.tiles > 0) {
    part = g.parts[j];
    if (part.y == 1 && p.splits == 0) return;  // the same in all warps of a row
  }
  const int n = part.y + p.splits;
  if (n == 0 && lane == 0 && (g.seq_lens[b] < 0 || g.seq_lens[b] > g.max_ctx))
    atomicOr(g.status, MLA_DEVFLAG_CTX_RANGE);  // no other kernel has looked
  const size_t pre0 = (size_t)(part.x + j) * mla::kRowTile + r % mla::kRowTile;
  const size_t own0 = (size_t)b * p.splits * g.rows_per_seq + local;
  auto lse_of = [&](int s) -> float {
    return s < part.y ? p.pre_lse[pre0 + (size_t)s * mla::kRowTile]
                      : p.own_lse[own0 + (size_t)(s - part.y) * g.rows_per_seq];
  };
  float4 v[4];
  auto load = [&](int s) {
    if (s >= n) return;
    const float4* row = reinterpret_cast<const float4*>(
        s < part.y ? p.pre_o + (pre0 + (size_t)s * mla::kRowTile) * mla::kDV
                   : p.own_o + (own0 + (size_t)(s - part.y) * g.rows_per_seq) * mla::kDV);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = row[lane + 32 * i];
  };
  load(warp);
  float m = -INFINITY;
  for (int s = lane; s < n; s += 32) m = fmaxf(m, lse_of(s));
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float4 acc[4] = {};
  float sum = 0.f;
  for (int s = warp; s < n; s += kWarps) {
    const float x = lse_of(s);
    if (x != -INFINITY) {  // an empty part's row may hold anything
      const float w = expf(x - m);
      sum += w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i].x += w * v[i].x;
        acc[i].y += w * v[i].y;
        acc[i].z += w * v[i].z;
        acc[i].w += w * v[i].w;
      }
    }
    load(s + kWarps);
  }
  if (kWarps > 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc_s[warp][lane + 32 * i] = acc[i];
    if (lane == 0) sum_s[warp] = sum;
    __syncthreads();
    if (warp > 0) return;
    for (int k = 1; k < min(kWarps, n); ++k) {
      sum += sum_s[k];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = acc_s[k][lane + 32 * i];
        acc[i].x += x.x;
        acc[i].y += x.y;
        acc[i].z += x.z;
        acc[i].w += x.w;
      }
    }
  }
  float L = sum > 0.f ? m + logf(sum) : -INFINITY, inv = sum > 0.f ? 1.f / sum : 0.f;
  if (sum != sum) L = inv = NAN;  // a NaN partial
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[i].x * inv, acc[i].y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[i].z * inv, acc[i].w * inv);
    reinterpret_cast<uint2*>(p.out + (size_t)r * mla::kDV)[lane + 32 * i] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
  if (lane == 0) p.lse[r] = L;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align256(int64_t a) { return ceil_div(a, 256) * 256; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Most sequences with rows in one 128-row block: a block that starts at a
// sequence's last row still holds it.
int block_seqs(int64_t rows, int rows_per_seq) {
  const int64_t batch = rows / rows_per_seq;
  if (mla::kRowTile % rows_per_seq == 0) return (int)std::min<int64_t>(batch, mla::kRowTile / rows_per_seq);
  if (rows_per_seq % mla::kRowTile == 0) return 1;
  return (int)std::min<int64_t>(batch, (mla::kRowTile + rows_per_seq - 2) / rows_per_seq + 1);
}

bool room_to_fold(int64_t batch, int rows, int64_t own) {
  const int64_t blocks = ceil_div(batch * rows, mla::kRowTile);
  const int64_t keys = own * block_seqs(batch * rows, rows);
  return blocks * keys <= kMaxOwnRows &&
         blocks * ceil_div(keys, mla::kPrefixTile) * mla::kPrefixTile <= kMaxRegionRows;
}

// The decode kernels count keys in int32, up to the last chunk's end.
bool chunks_fit(const mla_decode_prefix_plan_t& p) {
  return p.own_splits == 0 ||
         (p.own_chunk > 0 && p.prefix_len + (int64_t)p.own_splits * p.own_chunk <= INT32_MAX);
}

// Staged rows of keys: the shared ones and each row block's own, in whole tiles.
int64_t staged_keys(const mla_decode_prefix_plan_t& p) {
  return (int64_t)p.prefix_tiles * mla::kPrefixTile + (int64_t)p.row_blocks * p.block_keys;
}

mla::PrefixShape shape_of(const mla_decode_prefix_plan_t& p, const int32_t* seq_lens, char* ws) {
  mla::PrefixShape g;
  std::memset(&g, 0, sizeof g);
  g.seq_lens = seq_lens;
  g.status = reinterpret_cast<int32_t*>(ws + p.ws_status_offset);
  g.key_flags = reinterpret_cast<uint8_t*>(g.status + 4);
  g.row_flags = g.key_flags + staged_keys(p);
  g.pair_start = reinterpret_cast<int4*>(ws + p.ws_partition_offset);
  g.first_unit = reinterpret_cast<int64_t*>(g.pair_start + p.pairs + 1);
  g.parts = reinterpret_cast<int2*>(g.first_unit + p.row_blocks);
  g.block_tiles = reinterpret_cast<int32_t*>(g.parts + p.row_blocks);
  g.own_off = g.block_tiles + p.row_blocks;
  g.rows = p.total_rows;
  g.rows_per_seq = p.rows;
  g.heads = p.num_heads;
  g.sq = p.sq;
  g.causal = p.causal;
  g.batch = p.batch;
  g.prefix_len = p.prefix_len;
  g.max_ctx = p.max_ctx;
  g.tiles = p.prefix_tiles;
  g.pairs = p.pairs;
  g.row_blocks = p.row_blocks;
  g.fold = p.own_folded;
  g.block_seqs = p.own_folded ? block_seqs(p.total_rows, p.rows) : 0;
  g.block_keys = p.block_keys;
  return g;
}

// Every size and offset that follows from the plan's choices (batch, heads,
// lengths, pairs, own_folded, own_chunk and own_splits).
void lay_out(mla_decode_prefix_plan_t* p) {
  p->rows = p->num_heads * p->sq;
  p->total_rows = p->batch * p->rows;
  p->row_blocks = (int32_t)ceil_div(p->total_rows, mla::kRowTile);
  p->prefix_tiles = (int32_t)ceil_div(p->prefix_len, mla::kPrefixTile);
  p->key_tile = mla_small_rows_fit(p->rows, p->kv_dtype) ? mla::kKeyTileSmall : mla::kKeyTile;
  const int seqs = block_seqs(p->total_rows, p->rows);
  const int64_t own = std::max(0, p->max_ctx - p->prefix_len);
  p->block_keys = p->own_folded ? (int32_t)(ceil_div(own * seqs, mla::kPrefixTile) * mla::kPrefixTile) : 0;
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = off;
    off = align256(off + bytes);
    return at;
  };
  const int64_t segments = p->prefix_tiles > 0 ? (int64_t)p->row_blocks + p->pairs : 0;
  const int64_t keys = staged_keys(*p);
  p->ws_status_offset = take(16 + (p->prefix_tiles > 0 ? keys + p->total_rows : 0));
  p->ws_partition_offset = take(20 * (int64_t)p->row_blocks + 16 * ((int64_t)p->pairs + 1) +
                                (p->own_folded ? 4ll * p->row_blocks * seqs : 0));
  p->ws_keys_offset = take(p->prefix_tiles > 0 ? keys * MLA_D_QK * 2 : 0);
  p->ws_q_offset = take(p->prefix_tiles > 0 ? (int64_t)p->total_rows * MLA_D_QK * 2 : 0);
  p->ws_prefix_o_offset = take(segments * mla::kRowTile * MLA_D_V * 4);
  p->ws_prefix_lse_offset = take(segments * mla::kRowTile * 4);
  p->ws_own_o_offset = take((int64_t)p->own_splits * p->total_rows * MLA_D_V * 4);
  p->ws_own_lse_offset = take((int64_t)p->own_splits * p->total_rows * 4);
  p->workspace_bytes = off;
}

int check_plan(const mla_decode_prefix_plan_t* p) {
  if (p == nullptr || p->version != MLA_DECODE_PREFIX_PLAN_VERSION) return MLA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->batch > 65535 || p->num_heads < 1 || p->num_heads > 128 || p->sq < 1 ||
      p->sq > 16 || p->num_heads * p->sq > mla::kMaxRows ||
      (int64_t)p->batch * p->num_heads * p->sq > MLA_PREFIX_MAX_ROWS)
    return MLA_ERR_INVALID_ARG;
  if (p->page_size < 1 || p->page_size > 4096 || p->prefix_len < 0 ||
      p->prefix_len > MLA_PREFIX_MAX_LEN || p->max_ctx < 0 || p->wait_limit_us < 0 ||
      p->causal < 0 || p->causal > 1)
    return MLA_ERR_INVALID_ARG;
  if (p->kv_dtype != MLA_KV_BF16 && p->kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID_ARG;
  if (p->own_folded < 0 || p->own_folded > 1 || p->own_splits < 0 ||
      p->own_splits > mla::kMaxSplits || p->own_chunk < 1 || p->own_chunk > (1 << 30))
    return MLA_ERR_INVALID_ARG;
  const int64_t own = std::max(0, p->max_ctx - p->prefix_len);
  if (p->own_folded ? p->prefix_len == 0 || p->own_splits != 0 ||
                          !room_to_fold(p->batch, p->num_heads * p->sq, own)
                    : (int64_t)p->own_splits * p->own_chunk < own || !chunks_fit(*p))
    return MLA_ERR_INVALID_ARG;
  // Everything else is what lay_out makes of these: a plan whose other fields
  // differ was edited.
  mla_decode_prefix_plan_t want = *p;
  lay_out(&want);
  if (std::memcmp(&want, p, sizeof want) != 0) return MLA_ERR_INVALID_ARG;
  if (p->prefix_tiles > 0 ? p->pairs < 1 || p->pairs > kMaxPairs : p->pairs != 0) return MLA_ERR_INVALID_ARG;
  if (p->own_chunk % p->key_tile != 0) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

}  // namespace

extern "C" int mla_decode_prefix_plan(const int32_t* seq_lens_host, int32_t batch,
                                      int32_t prefix_len, int32_t num_heads, int32_t sq,
                                      int32_t page_size, int32_t kv_dtype, int32_t causal,
                                      int32_t num_sms, mla_decode_prefix_plan_t* plan) {
  if (plan == nullptr || seq_lens_host == nullptr) return MLA_ERR_INVALID_ARG;
  if (batch < 1 || batch > 65535 || prefix_len < 0 || prefix_len > MLA_PREFIX_MAX_LEN)
    return MLA_ERR_INVALID_ARG;
  if (kv_dtype == MLA_KV_FP4_E2M1) return MLA_ERR_UNSUPPORTED;
  try {
    std::vector<int32_t> own(batch);
    int32_t max_ctx = 0;
    for (int b = 0; b < batch; ++b) {
      if (seq_lens_host[b] < 0) return MLA_ERR_INVALID_ARG;
      max_ctx = std::max(max_ctx, seq_lens_host[b]);
      own[b] = std::max(0, seq_lens_host[b] - prefix_len);
    }
    // The own keys as a decode of contexts ctx_b - P; that call checks the
    // other arguments.
    mla_decode_plan_t d;
    const int st = mla_decode_plan(own.data(), batch, num_heads, sq, page_size, kv_dtype, causal,
                                   num_sms, &d);
    if (st != MLA_OK) return st;
    const int64_t total_rows = (int64_t)batch * d.rows;
    if (total_rows > MLA_PREFIX_MAX_ROWS) return MLA_ERR_UNSUPPORTED;

    mla_decode_prefix_plan_t p;
    std::memset(&p, 0, sizeof p);
    p.version = MLA_DECODE_PREFIX_PLAN_VERSION;
    p.batch = batch;
    p.num_heads = num_heads;
    p.sq = sq;
    p.page_size = page_size;
    p.kv_dtype = kv_dtype;
    p.causal = causal;
    p.prefix_len = prefix_len;
    p.max_ctx = max_ctx;
    p.num_sms = d.num_sms;
    p.own_chunk = d.chunk_len;
    p.own_splits = d.max_ctx > 0 ? d.num_splits : 0;
    if (!chunks_fit(p)) return MLA_ERR_UNSUPPORTED;
    lay_out(&p);

    // Measured on GB300 (us): a 256-key tile on one pair, a segment's query
    // rows, first softmax, last values and output, and the merge of cut rows.
    constexpr double kTile = 2.4, kSegment = 4.7, kMergeFixed = 1.5, kMergeRow = 4096.0 / 4.0e6;
    const int pairs = std::min(std::max(1, d.num_sms / 2), kMaxPairs);
    std::vector<int64_t> first(p.row_blocks + 1, 0);  // tiles before each row block, own folded in
    double staged = 0.0;                              // own keys of all row blocks
    for (int j = 0; j < p.row_blocks; ++j) {
      const int b0 = (int)((int64_t)j * mla::kRowTile / p.rows);
      const int b1 = (int)((std::min<int64_t>((int64_t)(j + 1) * mla::kRowTile, total_rows) - 1) / p.rows);
      int64_t keys = 0;
      for (int b = b0; b <= b1; ++b) keys += own[b];
      staged += (double)keys;
      first[j + 1] = first[j] + p.prefix_tiles + ceil_div(keys, mla::kPrefixTile);
    }
    if (p.prefix_tiles > 0) {
      // Own keys as further tiles, unless they need too much room or cost more
      // than a launch of the decode kernels of their own: 10 us and 2.2 or 2.9
      // a key tile (of 64 or 128 keys) for each unit, all pairs at work, against
      // the tiles and the staging of what the cache is read for once.  Whole
      // calls, folded against apart (us, 1024 shared keys, bf16): 128 x 16 heads
      // with 250 own keys 33 / 43, 500: 53 / 54, 1000: 91 / 78, 2000: 163 / 114;
      // 128 x 128 heads, 1000: 117 / 124, 2000: 193 / 169; 32 x 16 heads, 2000:
      // 49 / 59.
      const double key_tile_us = p.key_tile == mla::kKeyTile ? 2.2 : 2.9;
      const double stage_key_us = kv_dtype == MLA_KV_BF16 ? 0.45e-3 : 0.36e-3;
      double separate = 0.0, longest = 0.0;
      for (int b = 0; b < batch; ++b) {
        const double unit = 10.0 + key_tile_us * (double)ceil_div(own[b], p.key_tile);
        separate += unit * d.row_blocks;
        longest = std::max(longest, unit);
      }
      separate = std::max(longest, separate / pairs) + kMergeFixed;
      const double folded =
          kTile * (double)(first[p.row_blocks] - (int64_t)p.row_blocks * p.prefix_tiles) / pairs + stage_key_us * staged;
      p.own_folded = max_ctx > prefix_len && folded <= separate &&
                     room_to_fold(batch, p.rows, max_ctx - prefix_len);
      if (p.own_folded) p.own_splits = 0;
      else for (int j = 0; j <= p.row_blocks; ++j) first[j] = (int64_t)j * p.prefix_tiles;
      // Pairs that share the tiles: the count with the smallest longest pair,
      // merge included.  With many row blocks all pairs are busy anyway.
      const int most = (int)std::min<int64_t>(pairs, first[p.row_blocks]);
      const int64_t total = first[p.row_blocks] + (int64_t)p.row_blocks * mla::kSegmentTiles;
      double best = 1e300;
      for (int n = p.row_blocks > 1024 ? most : 1; n <= most; ++n) {
        const mla::PrefixShares shares(total, n);
        double worst = 0.0;
        int64_t cut_parts = 0;
        int j = 0;  // row block of the unit where a share starts
        auto unit = [&](int k) { return first[k] + (int64_t)k * mla::kSegmentTiles; };
        auto tile_at = [&](int k, int64_t u) {  // tiles of row block k before unit u
          return std::min(std::max<int64_t>(0, u - unit(k) - mla::kSegmentTiles), first[k + 1] - first[k]);
        };
        for (int i = 0; i < n; ++i) {
          const int64_t a = shares.start(i), z = shares.start(i + 1);
          while (j + 1 < p.row_blocks && unit(j + 1) <= a) ++j;
          double cost = 0.0;
          for (int k = j; k < p.row_blocks && unit(k) < z; ++k) {
            const int64_t tiles = tile_at(k, z) - tile_at(k, a);
            if (tiles == 0) continue;
            cost += kTile * (double)tiles + kSegment;
            cut_parts += tiles < first[k + 1] - first[k];
          }
          worst = std::max(worst, cost);
        }
        if (cut_parts > 0) worst += kMergeFixed + kMergeRow * mla::kRowTile * (double)cut_parts;
        if (worst < best) {
          best = worst;
          p.pairs = n;
        }
      }
    }
    lay_out(&p);
    *plan = p;
  } catch (const std::bad_alloc&) {
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

extern "C" int mla_decode_prefix_fwd(const mla_decode_prefix_plan_t* plan, const void* q,
                                     const void* kv_cache, int64_t num_pages,
                                     const float* kv_scale, const int32_t* prefix_table,
                                     const int32_t* block_table, int64_t bt_stride,
                                     const int32_t* seq_lens, float softmax_scale, void* out,
                                     float* lse, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  const int st = check_plan(plan);
  if (st != MLA_OK) return st;
  if (workspace == nullptr || !aligned(workspace, 256) ||
      (int64_t)workspace_bytes < plan->workspace_bytes)
    return MLA_ERR_WORKSPACE;
  const bool owns = plan->own_folded || plan->own_splits > 0;
  if (!q || !kv_cache || !seq_lens || !out || !lse) return MLA_ERR_INVALID_ARG;
  if (plan->prefix_tiles > 0 && !prefix_table) return MLA_ERR_INVALID_ARG;
  if (owns && !block_table) return MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(prefix_table, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(kv_scale, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_pages < 1) return MLA_ERR_INVALID_ARG;
  if (num_pages * (int64_t)plan->page_size >= ((int64_t)1 << 31)) return MLA_ERR_UNSUPPORTED;
  if (owns && (bt_stride < 1 || bt_stride * (int64_t)plan->page_size < (int64_t)plan->max_ctx))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale >= 0.f && softmax_scale <= 3.0e38f)) return MLA_ERR_INVALID_ARG;

  char* ws = static_cast<char*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const mla::PrefixShape g = shape_of(*plan, seq_lens, ws);
  const bool fp8 = plan->kv_dtype == MLA_KV_FP8_E4M3;
  const uint64_t wait_ns =
      plan->wait_limit_us > 0 ? (uint64_t)plan->wait_limit_us * 1000ull : kDefaultWaitNs;
  cudaLaunchAttribute attr[1];  // of the launches that overlap the one before them
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;

  // The staging clears the status word.  Without shared keys the first launch is
  // a decode kernel, which flags contexts before its dependency wait, or the merge.
  if (plan->prefix_tiles == 0 && cudaMemsetAsync(g.status, 0, 16, s) != cudaSuccess) return MLA_ERR_CUDA;
  if (plan->prefix_tiles > 0) {
    StageParams t;
    t.g = g;
    t.cache = kv_cache;
    t.num_pages = num_pages;
    t.prefix_table = prefix_table;
    t.block_table = block_table;
    t.bt_stride = bt_stride;
    t.q = static_cast<const uint16_t*>(q);
    t.k_out = reinterpret_cast<uint16_t*>(ws + plan->ws_keys_offset);
    t.q_out = reinterpret_cast<uint16_t*>(ws + plan->ws_q_offset);
    t.page_size = plan->page_size;
    t.fp8 = fp8;
    t.prefix_chunks = plan->prefix_tiles * (mla::kPrefixTile / kChunk);
    t.q_chunks = (int)ceil_div(plan->total_rows, kChunk);
    t.own_chunks = plan->own_folded ? (int)ceil_div(plan->max_ctx - plan->prefix_len, kChunk) : 1;
    const int64_t ctas = 1 + (int64_t)t.prefix_chunks + t.q_chunks +
                         (plan->own_folded ? (int64_t)plan->row_blocks *
                                                 ((int64_t)g.block_seqs * t.own_chunks + kPadChunks)
                                           : 0);
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(kStageThreads, 1, 1);
    if (cudaLaunchKernelEx(&cfg, stage_kernel, t) != cudaSuccess) return MLA_ERR_CUDA;

    mla::PrefixParams p;
    p.g = g;
    p.kv_scale = fp8 ? kv_scale : nullptr;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.part_o = reinterpret_cast<float*>(ws + plan->ws_prefix_o_offset);
    p.part_lse = reinterpret_cast<float*>(ws + plan->ws_prefix_lse_offset);
    p.wait_ns = wait_ns;
    p.softmax_scale = softmax_scale;
    p.partials = plan->own_splits > 0;
    if (mla_launch_prefix_sm103(p, t.k_out, staged_keys(*plan), t.q_out, stream) != 0) return MLA_ERR_CUDA;
  }

  if (plan->own_splits > 0) {
    mla::FwdParams f;
    std::memset(&f, 0, sizeof f);
    f.q = static_cast<const uint16_t*>(q);
    f.cache = kv_cache;
    f.num_pages = num_pages;
    f.kv_scale = fp8 ? kv_scale : nullptr;
    f.bt = block_table;
    f.bt_stride = bt_stride;
    f.seq_lens = seq_lens;
    f.softmax_scale = softmax_scale;
    f.out = static_cast<uint16_t*>(out);
    f.lse = lse;
    f.part_o = reinterpret_cast<float*>(ws + plan->ws_own_o_offset);
    f.part_lse = reinterpret_cast<float*>(ws + plan->ws_own_lse_offset);
    f.status = g.status;
    f.wait_ns = wait_ns;
    f.key_tile = plan->key_tile;
    f.batch = plan->batch;
    f.heads = plan->num_heads;
    f.sq = plan->sq;
    f.rows = plan->rows;
    f.page_size = plan->page_size;
    f.kv_dtype = plan->kv_dtype;
    f.causal = plan->causal;
    f.chunk_len = plan->own_chunk;
    f.num_splits = plan->own_splits;
    f.max_ctx = plan->max_ctx;
    f.row_blocks = (int)ceil_div(plan->rows, mla::kRowTile);
    f.key_begin = plan->prefix_len;
    f.partials = 1;
    if (mla_launch_fwd(f, stream) != 0) return MLA_ERR_CUDA;
  }

  // Which row blocks were cut only the device knows (the merge's CTAs return
  // at once for the whole ones), unless there is one pair and one row block.
  if (plan->prefix_tiles > 0 && plan->own_splits == 0 && plan->row_blocks == 1 && plan->pairs == 1)
    return MLA_OK;
  MergeParams m;
  m.g = g;
  m.pre_o = reinterpret_cast<const float*>(ws + plan->ws_prefix_o_offset);
  m.pre_lse = reinterpret_cast<const float*>(ws + plan->ws_prefix_lse_offset);
  m.own_o = reinterpret_cast<const float*>(ws + plan->ws_own_o_offset);
  m.own_lse = reinterpret_cast<const float*>(ws + plan->ws_own_lse_offset);
  m.out = static_cast<uint16_t*>(out);
  m.lse = lse;
  m.splits = plan->own_splits;
  const int64_t parts = plan->pairs / plan->row_blocks + plan->own_splits;
  const bool many = parts >= kManyParts;
  cfg.gridDim = dim3((unsigned)ceil_div(plan->total_rows, many ? 1 : 8), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  if (cudaLaunchKernelEx(&cfg, many ? merge_kernel<8> : merge_kernel<1>, m) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

extern "C" int mla_decode_prefix_check(const mla_decode_prefix_plan_t* plan, const void* workspace,
                                       void* stream, int32_t* host_status) {
  const int st = check_plan(plan);
  if (st != MLA_OK) return st;
  if (workspace == nullptr || host_status == nullptr) return MLA_ERR_INVALID_ARG;
  int32_t v = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(&v, static_cast<const char*>(workspace) + plan->ws_status_offset, sizeof v,
                      cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return MLA_ERR_CUDA;
  *host_status = v;
  if (v & MLA_DEVFLAG_TIMEOUT) return MLA_ERR_TIMEOUT;
  return v != 0 ? MLA_ERR_DEVICE_CHECK : MLA_OK;
}
