// serving_internal.h -- what the rotary and paged-cache translation units share
// with the rest of the library.
#pragma once

#include "../../include/relpos_attn.h"

namespace relpos {

// the device status word that kernels record errors in, and the number of SMs,
// of the current device (null and -1 on failure)
int* device_status();
int device_sms();

// whether two of n rows of d values, `stride` apart, share values
inline bool rows_overlap(int n, long long stride, int d) { return n > 1 && stride < d && stride > -d; }

// checks of a paged cache's sizes, types and pointers; a RELPOS_* code
int check_paged_cache(const RelposPagedCache* cache);

}  // namespace relpos
