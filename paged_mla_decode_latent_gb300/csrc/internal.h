// internal.h -- constants and launch parameters shared by the library's
// translation units (not part of the public ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace mla {

constexpr int kDQK = 576;       // query/key row: 512 latent + 64 rope
constexpr int kDV = 512;        // value: first 512 dims of the same row
constexpr int kRowTile = 128;   // score rows per CTA pair (the MMA M)
constexpr int kKeyTile = 64;    // keys per pipeline stage (the QK^T MMA N)
constexpr int kKeyTileSmall = 128;  // the same for the few-row kernel
constexpr int kClusterSize = 2; // CTAs per work unit: each owns half the value dims
constexpr int kMaxRows = 1024;  // H * Sq limit
constexpr int kMaxSplits = 256; // split-count cap of the planner

// Everything a fwd kernel needs, resolved on the host from the plan and the
// caller's pointers.
struct FwdParams {
  const uint16_t* q;        // bf16 [B, Sq, H, 576]
  const void* cache;        // [num_pages, ps, 576] bf16 or e4m3
  int64_t num_pages;
  const float* kv_scale;    // device fp32[1] or nullptr
  const int32_t* bt;        // [B, bt_stride]
  int64_t bt_stride;
  const int32_t* seq_lens;  // [B]
  float softmax_scale;
  uint16_t* out;            // bf16 [B, Sq, H, 512]
  float* lse;               // [B, Sq, H]
  float* part_o;            // fp32 [B, S, rows, 512] (S > 1)
  float* part_lse;          // fp32 [B, S, rows]      (S > 1)
  int32_t* status;          // device status word
  uint64_t wait_ns;         // bound of every pipeline wait inside the kernel
  // Device-planned launches (nullptr otherwise): the unit list
  // {b, rb | chunk << 8, k0, k1}, its length, and per sequence
  // {clamped ctx, first partial slot, chunks, 0}.
  const int4* units;
  const int32_t* n_units;
  const int4* seq_info;
  const int32_t* bt_indptr;  // CSR row starts into bt (kv_indices), or nullptr
  int unit_capacity;         // device-planned: the grid's clusters (work-list capacity)
  int key_tile;              // 64: the 128-row kernel; 128: the few-row kernel
  int batch, heads, sq, rows, page_size, kv_dtype, causal;
  int chunk_len, num_splits, max_ctx, row_blocks;
  // Host-planned launches: the keys start at key_begin of every sequence (the
  // shared prefix before it is another launch's), and partials != 0 writes
  // partials even where there is one split (something else is merged in).
  int key_begin, partials;
};

// Raises a kernel's dynamic shared-memory limit to `bytes` on device `dev`,
// once per (device, kernel slot); thread-safe.  Slots name the library's
// kernels that need more than 48 KB (at most 32 of them).
cudaError_t opt_in_smem(const void* kernel, int bytes, int dev, int slot);

struct CombineParams {
  const float* part_o;
  const float* part_lse;
  uint16_t* out;
  float* lse;
  const int4* seq_info;  // device-planned: per sequence {ctx, first partial, count, 0}
  int batch, rows, num_splits;
};

// ---------------------------------------------------------- shared prefix ---

constexpr int kPrefixTile = 256;  // keys per tile

// A pair that meets a row block's start inside its share pays for one more
// segment (output of the one before, query rows, first softmax: 4.5 us, the
// time of two tiles, measured), so a row block of n tiles counts for n + 2.
constexpr int kSegmentTiles = 2;

// What the staging notes of a row, a byte each: the two marks, and in the bits
// from kStagedLift on the power of two that its values were multiplied by, in
// steps of kLiftStep binary orders.
constexpr uint32_t kStagedBadPage = 1;  // through a page id out of range
constexpr uint32_t kStagedRange = 2;    // holds a value that f16 cannot
constexpr int kStagedLift = 3, kLiftStep = 4, kMaxLift = 80;

// `total` such units dealt to pairs in contiguous shares that differ by at most
// one: pair i takes [start(i), start(i + 1)).
struct PrefixShares {
  int64_t q, r;
  // A 64-bit division takes about a thousand cycles on the device; few totals need one.
  __host__ __device__ static int64_t div(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
  }
  __host__ __device__ PrefixShares(int64_t total, int pairs)
      : q(div(total, pairs)), r(total - div(total, pairs) * pairs) {}
  __host__ __device__ int64_t start(int64_t i) const { return i * q + (i < r ? i : r); }
  __host__ __device__ int pair_of(int64_t x) const {  // the pair that holds unit x
    const int64_t big = r * (q + 1);  // the units of the longer shares
    return (int)(x < big ? div(x, q + 1) : r + div(x - big, q));
  }
};

// What the staging, the attention and the merge of a shared-prefix call know
// of its rows, keys and partition.
struct PrefixShape {
  const int32_t* seq_lens;  // [B]
  // [pairs + 1]: the row block and the tile of it at which a pair starts, and
  // the row block's tiles; the end
  int4* pair_start;
  int64_t* first_unit;      // [row blocks]: the units before each
  int32_t* block_tiles;     // [row blocks]
  int2* parts;              // [row blocks]: the first pair that holds a part of one, and their number
  int32_t* own_off;         // [row blocks, block_seqs]: a sequence's first own key in its block's
  int32_t* status;
  // The note of each staged key and query row, for the attention to act on and
  // to report.
  uint8_t *key_flags, *row_flags;
  int rows, rows_per_seq, heads, sq, causal, batch;
  int prefix_len, max_ctx;
  int tiles;       // of the shared keys
  int pairs, row_blocks;
  int fold;        // own keys are further tiles of each row block
  int block_seqs;  // most sequences with rows in one row block
  int block_keys;  // own keys that a row block's region holds (a multiple of the tile)

#ifdef __CUDACC__
  __device__ __forceinline__ int context(int b) const {
    const int ctx = seq_lens[b];
    return ctx < 0 ? 0 : min(ctx, max_ctx);
  }
  __device__ __forceinline__ int own(int b) const { return max(0, context(b) - prefix_len); }
  // Keys that row r (of sequence b) sees.
  __device__ __forceinline__ int visible(int r, int b) const {
    const int ctx = context(b);
    const int tok = (r - b * rows_per_seq) / heads;
    return causal ? max(0, min(ctx, ctx - sq + tok + 1)) : ctx;
  }
  __device__ __forceinline__ int first_seq(int block) const {
    return (int)((uint32_t)(block * kRowTile) / (uint32_t)rows_per_seq);
  }
  __device__ __forceinline__ int last_seq(int block) const {
    return (int)((uint32_t)(min((block + 1) * kRowTile, rows) - 1) / (uint32_t)rows_per_seq);
  }
#endif
};

struct PrefixParams {
  PrefixShape g;
  const float* kv_scale;  // device fp32[1], or nullptr (bf16 cache)
  uint16_t* out;          // bf16 [rows, 512] and [rows]: row blocks that one pair holds
  float* lse;
  float* part_o;          // fp32 [row blocks + pairs, 128, 512]: segment pair + row block
  float* part_lse;        // fp32 [row blocks + pairs, 128]
  uint64_t wait_ns;
  float softmax_scale;
  int partials;           // every row block writes partials (something else is merged in)
};

// Tensor maps with the 128-byte swizzle; false on failure.  _rows: a 2-D
// 16-bit map of `rows` rows of `cols` elements, in boxes of box_rows x 64.
// _groups: f16 rows of 576 as [9 groups][rows][64], in boxes of box_groups x
// 64 rows x 64.
bool tensor_map_rows(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t rows,
                     int cols, int box_rows);
bool tensor_map_groups(CUtensorMap* map, const void* base, int64_t rows, int box_groups);

}  // namespace mla

// keys: f16 [key_rows, 576], the shared keys' tiles, then each row block's own;
// rows: f16 [p.g.rows, 576].
int mla_launch_prefix_sm103(const mla::PrefixParams& p, const void* keys, int64_t key_rows,
                            const void* rows, void* stream);

// The few-row kernel (128-key tiles) takes problems of at most this many
// score rows per sequence: 64 with a bf16 cache, 16 with fp8.
bool mla_small_rows_fit(int rows, int kv_dtype);
int mla_launch_fwd_small_sm103(const mla::FwdParams& p, void* stream);

// Launchers (return a cudaError_t as int).
extern "C" int mla_decode_epilogue(const void* ql_nope, const void* q_pe, const void* kv_c,
                                   const void* k_pe, const int64_t* slot_mapping,
                                   int32_t num_tokens, int32_t num_heads, void* q_out,
                                   void* kv_cache, int64_t num_pages, int32_t page_size,
                                   int32_t kv_dtype, const float* kv_scale,
                                   int32_t cache_inputs_early, int32_t* status, void* stream);
int mla_launch_fwd(const mla::FwdParams& p, void* stream);
int mla_launch_combine(const mla::CombineParams& p, void* stream);
