// api_util.h -- the C-ABI layer's per-device lookups and checks (api.cu),
// shared with the cache entry points (cache_api.cu).
#pragma once

#include "gqa_attn.h"

namespace gqa {
int* api_status_word();   // device status word of the current device, nullptr on error
int* api_check_line();    // debug builds: line of the first failed bounds check
int api_sm_count();       // SMs of the current device, 0 on error
attn_status api_check_arch();
attn_status api_check_heads(int Hq, int Hkv, int D);
}  // namespace gqa
