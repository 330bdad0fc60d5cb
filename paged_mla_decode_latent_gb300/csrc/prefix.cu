// prefix.cu -- decode attention for a batch that shares a prefix: the plan,
// the staging of the shared keys, the merge and the entry points.
//
// With P shared keys, sequence b's query rows attend to the shared keys and to
// its own keys [P, ctx_b); one softmax over both is the log-sum-exp merge of
// the two parts' partials:
//   L = ln sum_s e^lse_s,   out = sum_s e^(lse_s - L) o_s.
//
// One call queues:
//   stage    shared keys (through prefix_table) and the query rows -> f16 rows
//            in the workspace
//   prefix   prefix_sm103.cu: all rows of the batch against the shared keys
//   own      the decode kernels over keys [P, ctx_b) of each sequence
//   merge    the partials of a row -> out, lse

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
constexpr int kStageThreads = 256;
constexpr int kMaxPairs = 256;
constexpr int kMaxParts = kMaxPairs + mla::kMaxSplits;  // partials of a row

struct StageParams {
  const void* cache;
  int64_t num_pages;
  const int32_t* table;
  const uint16_t* q;
  uint16_t* k_out;  // f16 [prefix_len, 576]
  uint16_t* q_out;  // f16 [rows, 576]
  int32_t* status;
  int prefix_len, rows, page_size, fp8;
};

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, bool& bad) {
  const float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xFFFF0000u);
  bad |= !(fabsf(lo) <= 65504.f) || !(fabsf(hi) <= 65504.f);
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One thread per 8-element piece: rows [0, prefix_len) are the shared keys,
// the rest the query rows.  Memory-bound (1152 or 576 B in, 1152 B out a row).
__global__ void __launch_bounds__(kStageThreads) stage_kernel(StageParams p) {
  const uint32_t i = blockIdx.x * kStageThreads + threadIdx.x;
  const uint32_t row = i / kPieces, piece = i % kPieces;
  if (row >= (uint32_t)p.prefix_len + (uint32_t)p.rows) return;
  bool bad = false;
  uint4 v;
  if (row < (uint32_t)p.prefix_len) {
    const uint32_t page_i = row / (uint32_t)p.page_size;
    int64_t page = p.table[page_i];
    if (page < 0 || page >= p.num_pages) {
      if (piece == 0) atomicOr(p.status, MLA_DEVFLAG_BAD_PAGE);
      page = 0;
    }
    const int64_t at = (page * p.page_size + (row - page_i * (uint32_t)p.page_size)) * MLA_D_QK + piece * 8;
    if (p.fp8) {
      const uint2 codes = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.cache) + at);
      const uint32_t cw[2] = {codes.x, codes.y};
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint16_t two = (uint16_t)(cw[e >> 1] >> (16 * (e & 1)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(w[e]) : "h"(two));
        bad |= (two & 0x7Fu) == 0x7Fu || (two & 0x7F00u) == 0x7F00u;  // NaN codes
      }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.cache) + at);
      v = make_uint4(bf16x2_to_f16x2(v.x, bad), bf16x2_to_f16x2(v.y, bad),
                     bf16x2_to_f16x2(v.z, bad), bf16x2_to_f16x2(v.w, bad));
    }
    if (bad) atomicOr(p.status, MLA_DEVFLAG_KV_RANGE);
    reinterpret_cast<uint4*>(p.k_out)[(size_t)row * kPieces + piece] = v;
  } else {
    const size_t at = (size_t)(row - (uint32_t)p.prefix_len) * kPieces + piece;
    v = reinterpret_cast<const uint4*>(p.q)[at];
    v = make_uint4(bf16x2_to_f16x2(v.x, bad), bf16x2_to_f16x2(v.y, bad), bf16x2_to_f16x2(v.z, bad),
                   bf16x2_to_f16x2(v.w, bad));
    if (bad) atomicOr(p.status, MLA_DEVFLAG_Q_RANGE);
    reinterpret_cast<uint4*>(p.q_out)[at] = v;
  }
}

struct MergeParams {
  const float* pre_o;    // [slots, total rows, 512]
  const float* pre_lse;  // [slots, total rows]
  const float* own_o;    // [B, splits, rows, 512]
  const float* own_lse;  // [B, splits, rows]
  uint16_t* out;
  float* lse;
  int64_t total_tiles;
  int total_rows, rows, splits, tiles, pairs;
};

// One 128-thread CTA per row, 4 value dims a thread (as combine.cu, whose
// partials have one layout; here a row's come from two).
__global__ void __launch_bounds__(128) merge_kernel(MergeParams p) {
  const int r = blockIdx.x;
  const int b = r / p.rows, local = r - b * p.rows;
  __shared__ float w_s[kMaxParts];
  __shared__ float red[4];
  __shared__ float L_s;
  ptx::grid_dependency_wait();
  int np = 0;  // partials over the shared keys
  if (p.tiles > 0) {
    const int64_t t0 = (int64_t)(r / mla::kRowTile) * p.tiles;
    np = mla::prefix_pair_of(p.total_tiles, p.pairs, t0 + p.tiles - 1) -
         mla::prefix_pair_of(p.total_tiles, p.pairs, t0) + 1;
  }
  const int n = np + p.splits;
  auto row_of = [&](int s) -> size_t {  // partial s of this row, in its own array
    return s < np ? (size_t)s * p.total_rows + r : ((size_t)b * p.splits + (s - np)) * p.rows + local;
  };
  float m = -INFINITY;
  for (int s = threadIdx.x; s < n; s += 128) {
    const float x = (s < np ? p.pre_lse : p.own_lse)[row_of(s)];
    w_s[s] = x;
    m = fmaxf(m, x);
  }
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  float sum = 0.f;
  for (int s = threadIdx.x; s < n; s += 128) {
    const float e = w_s[s] == -INFINITY ? 0.f : expf(w_s[s] - m);
    w_s[s] = e;
    sum += e;
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  const float tot = (red[0] + red[1]) + (red[2] + red[3]);
  if (threadIdx.x == 0) L_s = m == -INFINITY ? -INFINITY : m + logf(tot);
  __syncthreads();
  const float inv = m == -INFINITY ? 0.f : 1.f / tot;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < n; s0 += 4) {
    float4 v[4];
    float wt[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + u;
      wt[u] = s < n ? w_s[s] * inv : 0.f;
      // An empty part's row was never written: it is not read.
      v[u] = wt[u] != 0.f
                 ? reinterpret_cast<const float4*>((s < np ? p.pre_o : p.own_o) + row_of(s) * mla::kDV)[threadIdx.x]
                 : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      acc.x += wt[u] * v[u].x;
      acc.y += wt[u] * v[u].y;
      acc.z += wt[u] * v[u].z;
      acc.w += wt[u] * v[u].w;
    }
  }
  __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y);
  __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z, acc.w);
  uint2 packed;
  packed.x = *reinterpret_cast<uint32_t*>(&lo);
  packed.y = *reinterpret_cast<uint32_t*>(&hi);
  reinterpret_cast<uint2*>(p.out + (size_t)r * mla::kDV)[threadIdx.x] = packed;
  if (threadIdx.x == 0) p.lse[r] = L_s;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align256(int64_t a) { return ceil_div(a, 256) * 256; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_plan(const mla_decode_prefix_plan_t* p) {
  if (p == nullptr || p->version != MLA_DECODE_PREFIX_PLAN_VERSION) return MLA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->num_heads < 1 || p->num_heads > 128 || p->sq < 1 || p->sq > 16 ||
      p->rows != p->num_heads * p->sq || p->rows > mla::kMaxRows ||
      (int64_t)p->batch * p->rows != p->total_rows || p->total_rows > MLA_PREFIX_MAX_ROWS)
    return MLA_ERR_INVALID_ARG;
  if (p->page_size < 1 || p->page_size > 4096 || p->prefix_len < 0 ||
      p->prefix_len > MLA_PREFIX_MAX_LEN || p->max_ctx < 0 || p->wait_limit_us < 0)
    return MLA_ERR_INVALID_ARG;
  if (p->kv_dtype != MLA_KV_BF16 && p->kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID_ARG;
  if (p->prefix_tiles != (int32_t)ceil_div(p->prefix_len, mla::kPrefixTile) ||
      p->row_blocks != (int32_t)ceil_div(p->total_rows, mla::kRowTile))
    return MLA_ERR_INVALID_ARG;
  if (p->prefix_tiles > 0 &&
      (p->pairs < 1 || p->pairs > kMaxPairs || p->pairs > (int64_t)p->row_blocks * p->prefix_tiles || p->prefix_slots < 1 ||
       p->prefix_slots > p->pairs))
    return MLA_ERR_INVALID_ARG;
  if (p->own_splits < 0 || p->own_splits > mla::kMaxSplits || p->own_chunk < 1 ||
      p->prefix_slots + p->own_splits > kMaxParts)
    return MLA_ERR_INVALID_ARG;
  if (p->key_tile != (mla_small_rows_fit(p->rows, p->kv_dtype) ? mla::kKeyTileSmall : mla::kKeyTile) ||
      p->own_chunk % p->key_tile != 0)
    return MLA_ERR_INVALID_ARG;
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
  std::vector<int32_t> own;
  try {
    own.resize(batch);
  } catch (const std::bad_alloc&) {
    return MLA_ERR_CUDA;
  }
  int32_t max_ctx = 0;
  for (int b = 0; b < batch; ++b) {
    if (seq_lens_host[b] < 0) return MLA_ERR_INVALID_ARG;
    max_ctx = std::max(max_ctx, seq_lens_host[b]);
    own[b] = std::max(0, seq_lens_host[b] - prefix_len);
  }
  // The own keys are planned as a decode of contexts ctx_b - P; that call
  // checks the other arguments.
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
  p.rows = d.rows;
  p.total_rows = (int32_t)total_rows;
  p.prefix_len = prefix_len;
  p.max_ctx = max_ctx;
  p.num_sms = d.num_sms;
  p.row_blocks = (int32_t)ceil_div(total_rows, mla::kRowTile);
  p.prefix_tiles = (int32_t)ceil_div(prefix_len, mla::kPrefixTile);
  p.key_tile = d.key_tile;
  p.own_chunk = d.chunk_len;
  p.own_splits = d.max_ctx > 0 ? d.num_splits : 0;
  if (p.prefix_tiles > 0) {
    // Pairs that share the tiles.  A segment (row block, tile range) costs its
    // tiles and about kSegment more for its query rows, its exposed first
    // softmax and last values and the write of its partial; the count with the
    // smallest longest pair wins, fewer pairs (fewer partials) on a tie.
    const int64_t total = (int64_t)p.row_blocks * p.prefix_tiles;
    const int most = (int)std::min<int64_t>(std::min(std::max(1, d.num_sms / 2), kMaxPairs), total);
    constexpr double kSegment = 2.0;
    double best = 1e300;
    for (int n = 1; n <= most; ++n) {
      double longest = 0.0;
      for (int i = 0; i < n; ++i) {
        const int64_t a = mla::prefix_share(total, n, i), z = mla::prefix_share(total, n, i + 1);
        const int64_t segs = (z - 1) / p.prefix_tiles - a / p.prefix_tiles + 1;
        longest = std::max(longest, (double)(z - a) + kSegment * (double)segs);
      }
      if (longest < best) {
        best = longest;
        p.pairs = n;
      }
    }
    for (int j = 0; j < p.row_blocks; ++j) {
      const int64_t t0 = (int64_t)j * p.prefix_tiles;
      p.prefix_slots = std::max(
          p.prefix_slots, mla::prefix_pair_of(total, p.pairs, t0 + p.prefix_tiles - 1) -
                              mla::prefix_pair_of(total, p.pairs, t0) + 1);
    }
  }
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = off;
    off = align256(off + bytes);
    return at;
  };
  p.ws_status_offset = take(16);
  p.ws_keys_offset = take(p.prefix_tiles > 0 ? (int64_t)prefix_len * MLA_D_QK * 2 : 0);
  p.ws_q_offset = take(p.prefix_tiles > 0 ? total_rows * MLA_D_QK * 2 : 0);
  p.ws_prefix_o_offset = take(p.prefix_slots * total_rows * MLA_D_V * 4);
  p.ws_prefix_lse_offset = take(p.prefix_slots * total_rows * 4);
  p.ws_own_o_offset = take(p.own_splits * total_rows * MLA_D_V * 4);
  p.ws_own_lse_offset = take(p.own_splits * total_rows * 4);
  p.workspace_bytes = off;
  *plan = p;
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
  if (!q || !kv_cache || !seq_lens || !out || !lse) return MLA_ERR_INVALID_ARG;
  if (plan->prefix_tiles > 0 && !prefix_table) return MLA_ERR_INVALID_ARG;
  if (plan->own_splits > 0 && !block_table) return MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(prefix_table, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(kv_scale, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_pages < 1) return MLA_ERR_INVALID_ARG;
  if (num_pages * (int64_t)plan->page_size >= ((int64_t)1 << 31)) return MLA_ERR_UNSUPPORTED;
  if (plan->own_splits > 0 &&
      (bt_stride < 1 || bt_stride * (int64_t)plan->page_size < (int64_t)plan->max_ctx))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale >= 0.f && softmax_scale <= 3.0e38f)) return MLA_ERR_INVALID_ARG;

  char* ws = static_cast<char*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t* status = reinterpret_cast<int32_t*>(ws + plan->ws_status_offset);
  const bool fp8 = plan->kv_dtype == MLA_KV_FP8_E4M3;
  const uint64_t wait_ns =
      plan->wait_limit_us > 0 ? (uint64_t)plan->wait_limit_us * 1000ull : kDefaultWaitNs;
  float* pre_o = reinterpret_cast<float*>(ws + plan->ws_prefix_o_offset);
  float* pre_lse = reinterpret_cast<float*>(ws + plan->ws_prefix_lse_offset);
  float* own_o = reinterpret_cast<float*>(ws + plan->ws_own_o_offset);
  float* own_lse = reinterpret_cast<float*>(ws + plan->ws_own_lse_offset);
  if (cudaMemsetAsync(status, 0, sizeof(int32_t), s) != cudaSuccess) return MLA_ERR_CUDA;

  if (plan->prefix_tiles > 0) {
    StageParams g;
    g.cache = kv_cache;
    g.num_pages = num_pages;
    g.table = prefix_table;
    g.q = static_cast<const uint16_t*>(q);
    g.k_out = reinterpret_cast<uint16_t*>(ws + plan->ws_keys_offset);
    g.q_out = reinterpret_cast<uint16_t*>(ws + plan->ws_q_offset);
    g.status = status;
    g.prefix_len = plan->prefix_len;
    g.rows = plan->total_rows;
    g.page_size = plan->page_size;
    g.fp8 = fp8;
    const int64_t items = ((int64_t)plan->prefix_len + plan->total_rows) * kPieces;
    stage_kernel<<<(unsigned)ceil_div(items, kStageThreads), kStageThreads, 0, s>>>(g);
    if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;

    mla::PrefixParams p;
    p.kv_scale = fp8 ? kv_scale : nullptr;
    p.seq_lens = seq_lens;
    p.part_o = pre_o;
    p.part_lse = pre_lse;
    p.status = status;
    p.wait_ns = wait_ns;
    p.total_tiles = (int64_t)plan->row_blocks * plan->prefix_tiles;
    p.softmax_scale = softmax_scale;
    p.rows = plan->total_rows;
    p.rows_per_seq = plan->rows;
    p.heads = plan->num_heads;
    p.sq = plan->sq;
    p.causal = plan->causal;
    p.prefix_len = plan->prefix_len;
    p.max_ctx = plan->max_ctx;
    p.tiles = plan->prefix_tiles;
    p.pairs = plan->pairs;
    if (mla_launch_prefix_sm103(p, g.k_out, g.q_out, stream) != 0) return MLA_ERR_CUDA;
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
    f.part_o = own_o;
    f.part_lse = own_lse;
    f.status = status;
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

  MergeParams m;
  m.pre_o = pre_o;
  m.pre_lse = pre_lse;
  m.own_o = own_o;
  m.own_lse = own_lse;
  m.out = static_cast<uint16_t*>(out);
  m.lse = lse;
  m.total_tiles = (int64_t)plan->row_blocks * plan->prefix_tiles;
  m.total_rows = plan->total_rows;
  m.rows = plan->rows;
  m.splits = plan->own_splits;
  m.tiles = plan->prefix_tiles;
  m.pairs = plan->pairs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)plan->total_rows, 1, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, merge_kernel, m) != cudaSuccess) return MLA_ERR_CUDA;
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
