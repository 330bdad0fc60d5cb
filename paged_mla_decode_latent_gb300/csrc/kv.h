// kv.h -- the cache types that the plans, the decode and the inserts take.
#pragma once

#include "../../include/mla_decode.h"

namespace mla {

inline bool kv_dtype_known(int d) {
  return d == MLA_KV_BF16 || d == MLA_KV_FP8_E4M3 || d == MLA_KV_FP4_E2M1;
}

}  // namespace mla
