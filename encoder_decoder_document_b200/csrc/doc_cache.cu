// The 8-bit document cache: rows of bf16 vectors (pooled passage vectors, or their cross K/V) quantised into
// pages as they are written, and read back.  "KaLM-Reranker-V1-Nano - MLX (Apple Silicon)", "What this is": a
// passage's pooled vectors are computed once and cached for later queries; the pages name no storage type
// for them, e4m3 with power-of-two scales is this library's.
//
// For each 32 consecutive columns of a row, with t = max |v| over the finite values:
//   e = the least integer with t <= 448 * 2^e, at least -120      (448 = the largest e4m3 number)
//   code = v * 2^-e rounded to nearest even                       (at most 240 where e = 120)
// The product with 2^-e is exact, so a value is rounded once, by at most 2^-4 of itself (half a step of a
// 3-bit mantissa; 2^-10 * 2^e where it is below the normal range).
//
// Both kernels stream: bound by HBM, 3 + 1/32 bytes a value.  A lane takes 16 columns (32 bytes of bf16 in
// one access where the rows allow it, 16 bytes of codes), so a warp's loads and stores are runs of whole lines
// on both sides and two neighbouring lanes hold one scale group; kUnits such slices per lane are loaded before the
// first is used.  A warp's units are consecutive, so it searches the document of its first row once (128 offsets a
// round) and walks on from there.
#include <algorithm>

#include "kalm.h"
#include "kalm_cache.cuh"
#include "kalm_internal.h"
#include "kalm_ptx.cuh"

namespace kalm {
namespace {

// Measured (CUDA graph of calls over three sets of inputs): write of 14,854 x 9,216 values 64.7 us = 6.4 TB/s (0.98 of the
// copy bandwidth), of 60,752 x 640 24.7 us = 4.8 TB/s; read of 63,169 x 2,560 80.6 us = 6.1 TB/s (0.93); one row 2.8 us.
// Blocks of 256 threads took 68.7, 26.4 and 82.7 us (a block's last warp holds its registers), of 32 74.8, 27.5 and 90.6;
// 8 slices a lane in flight 81.8, 31.3 and 89.0, 2 slices 73.3, 27.7 and 91.7 (256 threads).
constexpr int kThreads = 128;
constexpr int kUnits = 4;    // 16-column slices a lane keeps in flight
constexpr int kUnitCols = 16;

// The document that holds packed row r: the largest d with off[d] <= r (0 if none).  A warp searches together.
__device__ __forceinline__ int find_doc_warp(const int64_t* __restrict__ off, int n_docs, int64_t r, int lane) {
  int lo = 0, hi = n_docs;  // off[lo] <= r < off[hi], taking off[0] <= r
  while (hi - lo > 1) {
    const int step = (hi - lo + 127) / 128;
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = lo + step * (32 * j + lane + 1);
      n += __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(off + at) <= r));
    }
    hi = min(hi, lo + step * (n + 1));
    lo += step * n;
  }
  return lo;
}

struct Rows {
  const int64_t* off;    // [n_docs + 1] packed rows of each document
  const int32_t* first;  // [n_docs] row of the document that its first packed row becomes, or NULL: 0
  int n_docs;
  int64_t total;         // packed rows in memory; those from off[n_docs] on belong to no document
  int upr;               // units of a row
};

// A lane's units: packed row (relative to the warp's first), column in units, and the cache row (-1: none).
struct Unit {
  int row, col;
  int64_t at;
};

// One thread of the launch flags documents whose packed rows are not all in memory; the others' are served.
__device__ __forceinline__ void check_rows(const Rows& rows, uint32_t* err) {
  if (blockIdx.x == 0 && threadIdx.x == kThreads - 1 &&
      (__ldg(rows.off) < 0 || __ldg(rows.off + rows.n_docs) > rows.total))
    record_error(err, kErrDeviceArg | kSiteCache);
}

// The warp's units and its first packed row.  Its rows are looked up once, a lane each: with units of 16 columns
// and rows of at least two units a warp's 128 units are 64 rows at most (two a lane, and only where a row has two
// units), and every unit takes its row's place from the lane that found it.
__device__ __forceinline__ int64_t locate(Unit (&u)[kUnits], const Rows& rows, const CachePages& pages,
                                          uint32_t* err) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int64_t base = warp * 32 * kUnits;
  const int64_t r0 = base >> 32 ? base / rows.upr : static_cast<uint32_t>(base) / static_cast<uint32_t>(rows.upr);
  int c = static_cast<int>(base - r0 * rows.upr) + lane;
  const int last = (c - lane + 32 * kUnits - 1) / rows.upr;  // the warp's last row, from r0
  int64_t mine[2] = {-1, -1};  // cache rows of packed rows r0 + lane and r0 + 32 + lane
  if (r0 < rows.total) {
    int d = find_doc_warp(rows.off, rows.n_docs, r0, lane);
    int64_t begin = __ldg(rows.off + d), end = __ldg(rows.off + d + 1);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t r = r0 + 32 * k + lane;
      if (32 * k + lane > last || r >= rows.total) continue;
      while (r >= end && d + 1 < rows.n_docs) {  // a later document's row (skips empty ones)
        ++d;
        begin = end;
        end = __ldg(rows.off + d + 1);
      }
      if (r < begin || r >= end) continue;  // of no document
      const int64_t i = r - begin + (rows.first ? __ldg(rows.first + d) : 0);
      if (i >= 0) mine[k] = cache_row(pages, cache_page(pages, d, i), i);
      if (mine[k] < 0) record_error(err, kErrDeviceArg | kSiteCache);
    }
  }
  __syncwarp();
  int r = 0;
#pragma unroll
  for (int i = 0; i < kUnits; ++i, c += 32) {
    while (c >= rows.upr) {
      c -= rows.upr;
      ++r;
    }
    u[i].row = r;
    u[i].col = c;
    u[i].at = __shfl_sync(0xffffffffu, mine[0], r & 31);
    if (last >= 32) {
      const int64_t far = __shfl_sync(0xffffffffu, mine[1], r & 31);
      if (r >= 32) u[i].at = far;
    }
  }
  return r0;
}

// Scale exponent of a group whose largest finite magnitude has these bf16 bits (without the sign).
__device__ __forceinline__ int group_exp(uint32_t top) {
  // top = 1.m * 2^k with k = (top >> 7) - 127; 448 = 1.75 * 2^8, and 1.75 is m = 0x60.  Zero and bf16's
  // subnormals come out below the least exponent.
  const int e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
  return max(e, kCacheMinExp);
}

// 16 values of a row; WIDE: the rows are 32-byte aligned.
template <bool WIDE>
__device__ __forceinline__ Words8 load16(const uint4* p) {
  if (WIDE) return ldg_words8(p);
  const uint4 a = __ldg(p), b = __ldg(p + 1);
  return Words8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
template <bool WIDE>
__device__ __forceinline__ void store16(uint4* p, const Words8& v) {
  if (WIDE) {
    stg_words8(p, v);
  } else {
    p[0] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    p[1] = make_uint4(v.w[4], v.w[5], v.w[6], v.w[7]);
  }
}

__device__ __forceinline__ uint32_t pair_max(uint32_t v) { return max(v, __shfl_xor_sync(0xffffffffu, v, 1)); }

// Magnitude bits of value k of 16.
__device__ __forceinline__ uint32_t magnitude(const Words8& x, int k) { return (x.w[k >> 1] >> (16 * (k & 1))) & 0x7fffu; }

__device__ __forceinline__ uint32_t e4m3x2(float2 f) { return __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3); }

template <bool WIDE>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const uint4* __restrict__ src, int64_t ld_src_v,
                                                               const Rows rows, const CachePages pages,
                                                               uint8_t* __restrict__ codes, int64_t ld_codes,
                                                               uint8_t* __restrict__ scales, int64_t ld_scales,
                                                               uint32_t* err) {
  pdl_launch_dependents();
  pdl_wait_predecessor();
  check_rows(rows, err);
  Unit u[kUnits];
  const uint4* const from = src + locate(u, rows, pages, err) * ld_src_v;
  Words8 x[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[i].w[k] = 0;
    if (u[i].at >= 0) x[i] = load16<WIDE>(from + u[i].row * ld_src_v + u[i].col * 2);
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const Words8& v = x[i];
    // largest magnitude: bf16 magnitudes order as their bits do
    constexpr uint32_t kMag = 0x7fff7fffu;
    uint32_t m2 = v.w[0] & kMag;
#pragma unroll
    for (int k = 1; k < 7; k += 2) m2 = __vimax3_u16x2(m2, v.w[k] & kMag, v.w[k + 1] & kMag);
    m2 = __vmaxu2(m2, v.w[7] & kMag);
    uint32_t top = pair_max(max(m2 & 0xffffu, m2 >> 16));
    const bool odd = top >= 0x7f80u;  // an infinity or NaN in the group: the scale is the finite values'
    if (__any_sync(0xffffffffu, odd)) {
      uint32_t fine = 0;
#pragma unroll
      for (int k = 0; k < 16; ++k) fine = max(fine, magnitude(v, k) < 0x7f80u ? magnitude(v, k) : 0u);
      fine = pair_max(fine);
      if (odd) top = fine;
    }
    const int e = group_exp(top);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    const F2 inv2 = pair2(inv, inv);
    uint32_t out[4];
    if (!odd && e < kCacheMaxExp) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        out[k] = e4m3x2(split2(mul2(unpack2(v.w[2 * k]), inv2))) |
                 e4m3x2(split2(mul2(unpack2(v.w[2 * k + 1]), inv2))) << 16;
    } else {
      const float lim = e >= kCacheMaxExp ? 240.f : 448.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        out[k] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // an infinity is stored as NaN: no finite code may stand for it
          const uint32_t m = magnitude(v, 4 * k + j);
          const uint32_t w = v.w[2 * k + (j >> 1)];
          const float f = __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16) * inv;
          const float g = m >= 0x7f80u ? __uint_as_float(0x7fffffffu) : fminf(fmaxf(f, -lim), lim);
          out[k] |= (e4m3x2(make_float2(g, 0.f)) & 0xffu) << (8 * j);
        }
      }
    }
    if (u[i].at >= 0) {
      *reinterpret_cast<uint4*>(codes + u[i].at * ld_codes + u[i].col * kUnitCols) =
          make_uint4(out[0], out[1], out[2], out[3]);
      if ((u[i].col & 1) == 0) scales[u[i].at * ld_scales + (u[i].col >> 1)] = static_cast<uint8_t>(e + 127);
    }
  }
}

template <bool WIDE>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const uint8_t* __restrict__ codes, int64_t ld_codes,
                                                              const uint8_t* __restrict__ scales, int64_t ld_scales,
                                                              const Rows rows, const CachePages pages,
                                                              uint4* __restrict__ dst, int64_t ld_dst_v,
                                                              uint32_t* err) {
  pdl_launch_dependents();
  pdl_wait_predecessor();
  check_rows(rows, err);
  Unit u[kUnits];
  uint4* const to = dst + locate(u, rows, pages, err) * ld_dst_v;
  uint4 x[kUnits];
  uint32_t s[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
    if (u[i].at >= 0) {
      x[i] = __ldg(reinterpret_cast<const uint4*>(codes + u[i].at * ld_codes + u[i].col * kUnitCols));
      s[i] = __ldg(scales + u[i].at * ld_scales + (u[i].col >> 1));
    }
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
    if (u[i].at >= 0)
      store16<WIDE>(to + u[i].row * ld_dst_v + u[i].col * 2, e4m3x16_scaled(x[i], scale_bf16x2(s[i])));
}

}  // namespace
}  // namespace kalm

using namespace kalm;

namespace {

// What the two calls check alike.  `bf` is the bf16 side.
kalm_status check_cache_args(const char* what, const void* bf, int64_t ld_bf, const int64_t* row_off, int32_t n_docs,
                             int64_t total_rows, int32_t width, const int32_t* page_table, int64_t ld_table,
                             int32_t page_rows, int64_t n_pages, const uint8_t* codes, int64_t ld_codes,
                             const uint8_t* scales, int64_t ld_scales) {
  if (n_docs < 0 || total_rows < 0 || width <= 0 || width % kCacheGroup)
    return fail(KALM_ERR_INVALID_ARG, "%s: n_docs=%d total_rows=%lld width=%d (a positive multiple of 32)", what,
                n_docs, (long long)total_rows, width);
  if (page_rows < KALM_CACHE_MIN_PAGE_ROWS || page_rows > KALM_CACHE_MAX_PAGE_ROWS || (page_rows & (page_rows - 1)))
    return fail(KALM_ERR_INVALID_ARG, "%s: page_rows=%d is not a power of two in [%d, %d]", what, page_rows,
                KALM_CACHE_MIN_PAGE_ROWS, KALM_CACHE_MAX_PAGE_ROWS);
  if (n_pages < 0 || n_pages > INT32_MAX || ld_table < 0)
    return fail(KALM_ERR_INVALID_ARG, "%s: n_pages=%lld ld_table=%lld", what, (long long)n_pages, (long long)ld_table);
  if (ld_bf % 8 || ld_bf < width || ld_codes % 16 || ld_codes < width || ld_scales < width / kCacheGroup)
    return fail(KALM_ERR_INVALID_ARG, "%s: row strides %lld (values), %lld (codes), %lld (scales) for width %d", what,
                (long long)ld_bf, (long long)ld_codes, (long long)ld_scales, width);
  if (n_docs == 0 || total_rows == 0) return KALM_OK;
  if (!bf || !row_off || !page_table || !codes || !scales)
    return fail(KALM_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if (!aligned16(bf) || !aligned16(codes))
    return fail(KALM_ERR_INVALID_ARG, "%s: values and codes must be 16-byte aligned", what);
  if (total_rows * static_cast<__int128>(width) / kUnitCols / (kThreads * kUnits) > INT32_MAX - 1)
    return fail(KALM_ERR_INVALID_ARG, "%s: too many values (%lld rows of %d)", what, (long long)total_rows, width);
  return KALM_OK;
}

Rows make_rows(const int64_t* row_off, const int32_t* first_row, int32_t n_docs, int64_t total_rows, int32_t width) {
  return Rows{row_off, first_row, n_docs, total_rows, width / kUnitCols};
}

CachePages make_pages(const int32_t* page_table, int64_t ld_table, int32_t page_rows, int64_t n_pages) {
  return CachePages{page_table, ld_table, n_pages, __builtin_ctz(static_cast<unsigned>(page_rows))};
}

bool rows_aligned32(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && ld % 16 == 0; }

dim3 cache_grid(int64_t total_rows, int32_t width) {
  const int64_t units = total_rows * (width / kUnitCols);
  return dim3(static_cast<unsigned>(std::max((units + kThreads * kUnits - 1) / (kThreads * kUnits), int64_t{1})));  // (1: the rows' check)
}

}  // namespace

extern "C" kalm_status kalm_cache_write(const kalm_bf16* src, int64_t ld_src, const int64_t* row_off, int32_t n_docs,
                                        int64_t total_rows, int32_t width, const int32_t* first_row,
                                        const int32_t* page_table, int64_t ld_table, int32_t page_rows,
                                        int64_t n_pages, uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                                        int64_t ld_scales, kalm_stream_t stream) {
  kalm_status st = check_cache_args("kalm_cache_write", src, ld_src, row_off, n_docs, total_rows, width, page_table,
                                    ld_table, page_rows, n_pages, codes, ld_codes, scales, ld_scales);
  if (st != KALM_OK) return st;
  if ((st = ensure_device(nullptr)) != KALM_OK) return st;
  if (n_docs == 0 || (total_rows == 0 && !row_off)) return KALM_OK;
  return check_cuda(launch_pdl(rows_aligned32(src, ld_src) ? cache_write_kernel<true> : cache_write_kernel<false>, cache_grid(total_rows, width), dim3(kThreads), 0,
                               static_cast<cudaStream_t>(stream), reinterpret_cast<const uint4*>(src), ld_src / 8,
                               make_rows(row_off, first_row, n_docs, total_rows, width),
                               make_pages(page_table, ld_table, page_rows, n_pages), codes, ld_codes, scales,
                               ld_scales, device_error_word()),
                    "launch cache_write_kernel");
}

extern "C" kalm_status kalm_cache_read(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales,
                                       int64_t ld_scales, const int64_t* row_off, int32_t n_docs, int64_t total_rows,
                                       int32_t width, const int32_t* first_row, const int32_t* page_table,
                                       int64_t ld_table, int32_t page_rows, int64_t n_pages, kalm_bf16* dst,
                                       int64_t ld_dst, kalm_stream_t stream) {
  kalm_status st = check_cache_args("kalm_cache_read", dst, ld_dst, row_off, n_docs, total_rows, width, page_table,
                                    ld_table, page_rows, n_pages, codes, ld_codes, scales, ld_scales);
  if (st != KALM_OK) return st;
  if ((st = ensure_device(nullptr)) != KALM_OK) return st;
  if (n_docs == 0 || (total_rows == 0 && !row_off)) return KALM_OK;
  return check_cuda(launch_pdl(rows_aligned32(dst, ld_dst) ? cache_read_kernel<true> : cache_read_kernel<false>, cache_grid(total_rows, width), dim3(kThreads), 0,
                               static_cast<cudaStream_t>(stream), codes, ld_codes, scales, ld_scales,
                               make_rows(row_off, first_row, n_docs, total_rows, width),
                               make_pages(page_table, ld_table, page_rows, n_pages), reinterpret_cast<uint4*>(dst),
                               ld_dst / 8, device_error_word()),
                    "launch cache_read_kernel");
}
