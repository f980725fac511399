// The few-row form of kalm_merged_attention_cache (cache_rows_attention.cu), for its entry point.
#pragma once

#include <cuda_bf16.h>

#include "kalm_cache.cuh"
#include "kalm_internal.h"

namespace kalm {

struct CacheRowsParams {
  const __nv_bfloat16 *q, *k_self, *v_self;
  const uint8_t *k_codes, *v_codes, *k_scales, *v_scales;
  int64_t ldq, ld_self, ld_codes, ld_scales, ldo;
  CachePages pages;
  const int64_t *q_off, *in_off, *pool_off;
  int64_t total_in, total_q;  // rows of q and self K / V, of the output
  int32_t n_q, n_kv, G, max_q;
  float scale_log2;  // scale * log2(e)
  __nv_bfloat16* out;
  float* lse;
  uint32_t* err;
};

// Needs max_q * G <= KALM_CACHE_FEW_ROWS and arguments that kalm_merged_attention_cache has checked.
kalm_status launch_cache_rows_attention(const CacheRowsParams& p, int32_t n_docs, cudaStream_t stream);

}  // namespace kalm
