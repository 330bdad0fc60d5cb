// kv.h -- the cache types that the plans, the decode and the inserts take.
#pragma once

#include "../../include/mla_decode.h"
#include "internal.h"

namespace mla {

inline bool kv_dtype_known(int d) {
  return d == MLA_KV_BF16 || d == MLA_KV_FP8_E4M3 || d == MLA_KV_FP4_E2M1;
}

// Up to so many score rows a sequence a 4-bit cache has a kernel of its own, whose
// work units are single CTAs.  (In blocks of 32 it takes 64 rows in the time of the
// kernel for more rows, 187 against 180 us at batch 64 x 8192, and 128 twice that.)
constexpr int kFewRowsFp4 = 32;

}  // namespace mla

int mla_launch_fwd_fp4_sm103(const mla::FwdParams& p, void* stream);
int mla_launch_fwd_fp4_wide_sm103(const mla::FwdParams& p, void* stream);
