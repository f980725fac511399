// The 8-bit document cache's number format and page lookup, shared by the kernels that write it, read it back
// and attend over it.
//
// A cached row holds e4m3 codes and, for each 32 consecutive columns, one scale byte b that stands for
// 2^(b - 127).  kalm_cache_write keeps b in [7, 247], so that every stored value code * 2^(b - 127) is a bf16
// number: a code has four significant bits and is a multiple of 2^-9, and 2^-9 * 2^-120 is a multiple of bf16's
// least subnormal 2^-133; the largest, 240 * 2^120 and 448 * 2^119, lie below 2^128.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kalm.h"
#include "kalm_ptx.cuh"
#include "kalm_wide.cuh"

namespace kalm {

constexpr uint32_t kSiteCache = 8u << 8;  // device error word (see kalm_check_device_errors in kalm.h)
constexpr int kCacheGroup = KALM_CACHE_GROUP;  // columns that share a scale
constexpr int kCacheMinExp = -120;  // least scale exponent
constexpr int kCacheMaxExp = 120;   // greatest: bf16's largest value needs it

// Pages of a cache: document d's row i is row page_table[d * ld + i / rows] * rows + i % rows of the codes.
struct CachePages {
  const int32_t* table;
  int64_t ld;      // entries of a document in the table
  int64_t n_pages;
  int32_t shift;   // log2 of the rows of a page
};

// Page that holds row i of document d, -1 where the table has no such entry.
__device__ __forceinline__ int32_t cache_page(const CachePages& p, int d, int64_t i) {
  const int64_t at = i >> p.shift;
  return at < p.ld ? __ldg(p.table + d * p.ld + at) : -1;
}

// Cache row of row i of a document, given its page; -1 where that is no page of the cache.
__device__ __forceinline__ int64_t cache_row(const CachePages& p, int32_t page, int64_t i) {
  if (page < 0 || page >= p.n_pages) return -1;
  return (static_cast<int64_t>(page) << p.shift) + (i & ((int64_t{1} << p.shift) - 1));
}

// Two e4m3 codes (low byte first) as a bf16 pair; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// The bf16 pair (2^(b - 127), 2^(b - 127)) of a scale byte b in [1, 254].
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t b) { return b * 0x00800080u; }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r =
      __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Four codes of one word times their scale, as two bf16 pairs; exact (the scale is a power of two).
__device__ __forceinline__ uint2 e4m3x4_scaled(uint32_t word, uint32_t scale2) {
  return make_uint2(mul_bf16x2(e4m3x2_to_bf16x2(word & 0xffffu), scale2),
                    mul_bf16x2(e4m3x2_to_bf16x2(word >> 16), scale2));
}

// Sixteen codes times their scale, as eight bf16 pairs; exact.
__device__ __forceinline__ Words8 e4m3x16_scaled(const uint4& x, uint32_t scale2) {
  const uint2 a = e4m3x4_scaled(x.x, scale2), b = e4m3x4_scaled(x.y, scale2);
  const uint2 c = e4m3x4_scaled(x.z, scale2), d = e4m3x4_scaled(x.w, scale2);
  return Words8{{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y}};
}

}  // namespace kalm
