// qmm_attn_tc.h -- the tensor-memory attention kernel for many rows
// (qmm_attn_tc.cu), as its launch sees it.
#pragma once

#include "qmm_attn.cuh"

namespace qmm {

constexpr int ATTN_TC_ROWS = 256;     // rows of a CTA
constexpr int ATTN_TC_RECORDS = 4;    // records of a step
constexpr int ATTN_TC_MAX_NB = 4;     // head sizes up to 128: O of two tiles is half of tensor memory

AttnKernel attn_tc_kernel(int NB);
int attn_tc_smem(int NB);
int attn_tc_threads();
unsigned attn_tc_wait_ns(unsigned long long limit_ns);  // the bound of a wait: 4 s at most

}  // namespace qmm
