// kv.h -- the cache types that the plans, the decode and the inserts take.
#pragma once

#include "../../include/mla_decode.h"
#include "internal.h"

namespace mla {

inline bool kv_dtype_known(int d) {
  return d == MLA_KV_BF16 || d == MLA_KV_FP8_E4M3 || d == MLA_KV_FP4_E2M1;
}

// Up to so many score rows a sequence a 4-bit cache has a kernel of its own, whose
// work units are single CTAs.  (64 rows in blocks of 32 take 187 us at batch
// 64 x 8192, by the kernel for more rows 111, which 48 rows take as well; 32 here 102.)
constexpr int kFewRowsFp4 = 32;

// Keys by which a plan cuts sequences: the decode kernel's tile.  The plan's key_tile
// tells the few-row kernels (128) from the others (64); the one for more rows of a
// 4-bit cache has tiles of 256.
inline int chunk_step(int kv_dtype, int key_tile) {
  return kv_dtype == MLA_KV_FP4_E2M1 && key_tile == kKeyTile ? 256 : key_tile;
}

}  // namespace mla

int mla_launch_fwd_fp4_sm103(const mla::FwdParams& p, void* stream);
int mla_launch_fwd_fp4_wide_sm103(const mla::FwdParams& p, void* stream);
