// Merged attention over an 8-bit cache for a few decoder rows: a document's decoder positions times the query
// heads of a KV head are at most KALM_CACHE_FEW_ROWS packed rows (one position with up to eight heads a KV head, as in
// a step that adds a token).  Same result as the tensor-core path of kalm_merged_attention_cache, one launch, no
// workspace: there is too little arithmetic for tensor-core tiles (4 or 8 rows of 128 would be real).
//
// Against the tensor-core path, this form / that one in us; one position per document, one KV head, documents of n / 16
// to n cached rows:
//   documents  rows    n = 64          256             512             1,024
//   1          1       4.1 / 11.8      7.2 / 12.8      10.8 / 15.4     18.0 / 19.6
//   1          4       6.1 / 11.8      10.8 / 13.0     16.4 / 15.4     27.1 / 20.0
//   1          8       10.3 / 11.8     20.0 / 13.3     32.8 / 15.4     56.8 / 19.8
//   100        1       4.6 / 14.4      8.7 / 18.0      14.3 / 24.2     25.1 / 39.7
//   100        4       7.8 / 14.8      13.5 / 18.5     21.5 / 24.6     37.6 / 40.4
//   100        8       12.4 / 14.9     25.6 / 18.5     44.3 / 24.9     82.5 / 40.4
//   1,000      1       23.1 / 63.2     45.1 / 112      67.2 / 163      113 / 275
//   1,000      4       40.9 / 64.6     76.5 / 113      111 / 164       179 / 279
//   1,000      8       41.4 / 65.1     91.5 / 113      147 / 165       261 / 277
// so it is the faster one but for long documents in small batches.  All calls of so few rows come here all the same:
// the two forms round differently, and a choice by the documents' lengths or number would make a document's result
// depend on its company.  Bound by the latency of the dependent loads (offsets, pages, codes) for few
// documents and by the fp32 pipe's instructions for many (100 documents of 4 rows: 6.9 MB in 13.3 us).
//
// One block per (document, KV head), eight warps (four of 8 rows each).  For each packed row r and visible key j
//   s = scale * q_r . k_j;   out_r = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
// A warp takes KEYS keys at a time (every eighth or fourth group of the document's), a lane 8 of the 256 columns of each:
//   * the codes become fp32 numbers; their power-of-two scale multiplies the finished partial sum, not each number;
//   * the KEYS x R partial dot products are summed over the lanes by halving: each exchange hands half of the sums
//     to the other half of the lanes, so KEYS x R sums cost KEYS x R - 1 shuffles instead of five each, and a
//     lane ends with the score of one (key, row);
//   * running maximum and sum per row in fp32 (base-2 exponentials), p fp32 as well: nothing is rounded before the
//     output;
//   * each p is broadcast to the lanes, which hold the row's output columns.
// The next group's codes are loaded before the present one is worked on.  The warps' partial results are joined
// through shared memory.
#include "cache_rows_attention.h"

#include "kalm.h"
#include "kalm_cache.cuh"
#include "kalm_internal.h"
#include "kalm_ptx.cuh"

namespace kalm {
namespace {

constexpr int kHeadDim = 256;

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, F2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = unpack2(w[k]);
}

__device__ __forceinline__ void unpack_e4m3x8(const uint2& v, F2 (&f)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t two = ((k & 2 ? v.y : v.x) >> (16 * (k & 1))) & 0xffffu;
    const float2 g = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3)));
    f[k] = pair2(g.x, g.y);
  }
}

constexpr int log2_of(int n) { return n <= 1 ? 0 : 1 + log2_of(n / 2); }

// R packed rows (1, 2, 4 or 8), KEYS keys at a time; R * KEYS <= 32.  (4 keys at a time: 9.2, 10.6, 13.3 us for 1, 2, 4 rows
// of 100 documents against 8.4, 9.6, 13.1 then.)  8 rows' state takes the registers of four warps, their sums 32 KB.
template <int R>
struct Few {
  static constexpr int KEYS = R <= 4 ? 8 : 4;
  static constexpr int WARPS = R <= 4 ? 8 : 4;
  static constexpr int N = R * KEYS;              // scores of a group of keys
  static constexpr int DUP = 5 - log2_of(N);      // the score of (key j, row r) is in lanes (j * R + r) << DUP and on
};

template <int R>
struct State {
  F2 q[R][4];    // this lane's 8 columns of each row, times scale * log2(e)
  F2 acc[R][4];  // sum of p * v, relative to the row's maximum
  float m, l;    // of this lane's row (lane >> DUP) % R: running maximum (base 2), this lane's keys' sum
};

// One group of keys: their 8 columns in this lane (k, v as fp32 numbers, times ks, vs), `seen`: whether this
// lane's (key, row) counts.  G > 0: self keys from position 0 on, row r (position r / G) sees key j if j * G <= r, and what it
// does not see is left out of its output altogether (0 * NaN would be NaN).
template <int R>
__device__ __forceinline__ void attend(State<R>& st, const F2 (&k)[Few<R>::KEYS][4], const float (&ks)[Few<R>::KEYS],
                                       const F2 (&v)[Few<R>::KEYS][4], const float (&vs)[Few<R>::KEYS], bool seen,
                                       int lane, int G = 0, int j0 = 0) {
  constexpr int KEYS = Few<R>::KEYS, N = Few<R>::N, DUP = Few<R>::DUP;
  float part[N];
#pragma unroll
  for (int j = 0; j < KEYS; ++j)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      F2 s = mul2(k[j][0], st.q[r][0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) s = fma2(k[j][e], st.q[r][e], s);
      const float2 both = split2(s);
      part[j * R + r] = (both.x + both.y) * ks[j];
    }
  // halve: after the step with mask b the lanes with that bit hold the upper half of the sums
  int b = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2, b /= 2) {
    const bool up = lane & b;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? part[i] : part[i + n];
      const float keep = up ? part[i + n] : part[i];
      part[i] = keep + __shfl_xor_sync(0xffffffffu, give, b);
    }
  }
  float s = part[0];
#pragma unroll
  for (int o = (1 << DUP) / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (!seen) s = -INFINITY;
  float top = s;
#pragma unroll
  for (int o = R << DUP; o < 32; o *= 2) {  // over the keys; NaN scores are left out here and come through p
    const float other = __shfl_xor_sync(0xffffffffu, top, o);
    top = fmaxf(top, other);
  }
  const float m = fmaxf(st.m, top);
  const float base = m == -INFINITY ? 0.f : m;  // a row that has seen nothing yet
  const float alpha = ex2_approx(st.m - base);
  const float p = ex2_approx(s - base);
  st.l = fmaf(st.l, alpha, p);
  const bool moved = st.m != m;
  st.m = m;
  if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float a = __shfl_sync(0xffffffffu, alpha, r << DUP);
#pragma unroll
      for (int e = 0; e < 4; ++e) st.acc[r][e] = mul2(st.acc[r][e], pair2(a, a));
    }
  }
#pragma unroll
  for (int j = 0; j < KEYS; ++j)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float pj = __shfl_sync(0xffffffffu, p, (j * R + r) << DUP) * vs[j];
      if ((j0 + j) * G > r) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) st.acc[r][e] = fma2(pair2(pj, pj), v[j][e], st.acc[r][e]);
    }
}

// A group of cached keys as loaded: codes and scale bytes of this lane's 8 columns.
template <int R>
struct Group {
  uint2 k[Few<R>::KEYS], v[Few<R>::KEYS];
  uint32_t ks[Few<R>::KEYS], vs[Few<R>::KEYS];
  int n;  // keys of the document in it
};

// Cache row (lane j: of key j of the group that starts at `first`), -1 past the document or without a page.
template <int R>
__device__ __forceinline__ int32_t group_page(const CacheRowsParams& p, int d, int64_t first, int64_t nc, int lane) {
  return lane < Few<R>::KEYS && first + lane < nc ? cache_page(p.pages, d, first + lane) : -1;
}

template <int R>
__device__ __forceinline__ void load_group(Group<R>& g, const CacheRowsParams& p, int head, int64_t first, int64_t nc,
                                           int32_t page, int lane) {
  constexpr int KEYS = Few<R>::KEYS;
  const int64_t left = nc - first;
  g.n = left < KEYS ? static_cast<int>(left > 0 ? left : 0) : KEYS;
  int64_t mine = -1;
  if (lane < g.n) {
    mine = cache_row(p.pages, page, first + lane);
    if (mine < 0) record_error(p.err, kErrDeviceArg | kSiteAttention);
  }
  const int64_t col = head * kHeadDim + lane * 8, sc = head * (kHeadDim / kCacheGroup) + (lane >> 2);
#pragma unroll
  for (int j = 0; j < KEYS; ++j) {
    const int64_t at = __shfl_sync(0xffffffffu, mine, j);
    g.k[j] = g.v[j] = make_uint2(0u, 0u);
    g.ks[j] = g.vs[j] = 0;
    if (at >= 0) {
      g.k[j] = __ldg(reinterpret_cast<const uint2*>(p.k_codes + at * p.ld_codes + col));
      g.v[j] = __ldg(reinterpret_cast<const uint2*>(p.v_codes + at * p.ld_codes + col));
      g.ks[j] = __ldg(p.k_scales + at * p.ld_scales + sc);
      g.vs[j] = __ldg(p.v_scales + at * p.ld_scales + sc);
    }
  }
}

template <int R>
__global__ void __launch_bounds__(Few<R>::WARPS * 32) cache_rows_attention_kernel(const CacheRowsParams p) {
  pdl_launch_dependents();
  pdl_wait_predecessor();
  constexpr int KEYS = Few<R>::KEYS, DUP = Few<R>::DUP, kWarps = Few<R>::WARPS;
  extern __shared__ float smem[];
  float* const acc_s = smem;                         // [kWarps][R][256]
  float* const m_s = smem + kWarps * R * kHeadDim;   // [kWarps][R]
  float* const l_s = m_s + kWarps * R;               // [kWarps][R]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d = blockIdx.x / p.n_kv, head = blockIdx.x - d * p.n_kv;
  const int64_t q0 = __ldg(p.q_off + d), c0 = __ldg(p.pool_off + d);
  int64_t lq = __ldg(p.q_off + d + 1) - q0;
  // Cached rows that the document claims, and those of them that its table has places for.  Only the latter are walked, so
  // that wild offsets end in a flag and not in a loop of their length; the others, which count as rows of zeros (score 0,
  // value 0), join the sums at the end.
  const int64_t claimed = __ldg(p.pool_off + d + 1) - c0, places = p.pages.ld << p.pages.shift;
  const int64_t nc = min(claimed, places);
  const int64_t in0 = p.in_off ? __ldg(p.in_off + d) : q0;
  if (lq == 0) return;
  // more rows than the call was sized for, or rows (of q and self K / V, or of the output) that do not exist
  if (lq < 0 || lq > p.max_q || in0 < 0 || in0 > p.total_in - lq || q0 < 0 || q0 > p.total_q - lq) {
    if (threadIdx.x == 0) record_error(p.err, kErrDeviceArg | kSiteAttention);
    return;
  }
  if ((claimed < 0 || claimed > places) && threadIdx.x == 0) record_error(p.err, kErrDeviceArg | kSiteAttention);
  const int rows = static_cast<int>(lq) * p.G;  // packed rows: position x head of the KV group

  // the first group's pages and codes go out before q is used
  const int64_t step = static_cast<int64_t>(kWarps) * KEYS;
  int64_t first = static_cast<int64_t>(warp) * KEYS;
  Group<R> next;
  load_group<R>(next, p, head, first, nc, group_page<R>(p, d, first, nc, lane), lane);
  int32_t page = group_page<R>(p, d, first + step, nc, lane);

  State<R> st;
  st.m = -INFINITY;
  st.l = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows)
      x = *reinterpret_cast<const uint4*>(p.q + (in0 + r / p.G) * p.ldq +
                                          static_cast<int64_t>(head * p.G + r % p.G) * kHeadDim + lane * 8);
    unpack_bf16x8(x, st.q[r]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      st.q[r][e] = mul2(st.q[r][e], pair2(p.scale_log2, p.scale_log2));
      st.acc[r][e] = 0;  // a pair of zeros
    }
  }
  const int my = lane >> DUP;             // this lane's (key, row) of a group
  const int my_key = my / R, my_row = my % R;

  // the last warp takes the self keys (at most R), the row's position and those before it
  if (warp == kWarps - 1) {
    for (int j0 = 0; j0 < (KEYS >= R ? 1 : static_cast<int>(lq)); j0 += KEYS) {  // (one group where KEYS >= R >= lq)
      F2 k[KEYS][4], v[KEYS][4];
      float one[KEYS];
#pragma unroll
      for (int j = 0; j < KEYS; ++j) {
        uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
        if (j0 + j < static_cast<int>(lq)) {
          const int64_t at = (in0 + j0 + j) * p.ld_self + static_cast<int64_t>(head) * kHeadDim + lane * 8;
          a = *reinterpret_cast<const uint4*>(p.k_self + at);
          b = *reinterpret_cast<const uint4*>(p.v_self + at);
        }
        unpack_bf16x8(a, k[j]);
        unpack_bf16x8(b, v[j]);
        one[j] = 1.f;
      }
      attend<R>(st, k, one, v, one, my_row < rows && (j0 + my_key) * p.G <= my_row, lane, p.G, j0);
    }
  }
  while (next.n > 0) {
    const Group<R> cur = next;
    first += step;
    load_group<R>(next, p, head, first, nc, page, lane);
    page = group_page<R>(p, d, first + step, nc, lane);
    F2 k[KEYS][4], v[KEYS][4];
    float ks[KEYS], vs[KEYS];
#pragma unroll
    for (int j = 0; j < KEYS; ++j) {
      unpack_e4m3x8(cur.k[j], k[j]);
      unpack_e4m3x8(cur.v[j], v[j]);
      ks[j] = __uint_as_float(cur.ks[j] << 23);
      vs[j] = __uint_as_float(cur.vs[j] << 23);
    }
    attend<R>(st, k, ks, v, vs, my_row < rows && my_key < cur.n, lane);
  }

  // the sum over this warp's keys: the lanes of a row that differ in their key (not in the copies of it)
  float l = st.l;
#pragma unroll
  for (int o = R << DUP; o < 32; o *= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
  if ((lane & ((1 << DUP) - 1)) == 0 && my_key == 0) {
    m_s[warp * R + my_row] = st.m;
    l_s[warp * R + my_row] = l;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float4* to = reinterpret_cast<float4*>(acc_s + (warp * R + r) * kHeadDim + lane * 8);
    const float2 a = split2(st.acc[r][0]), b = split2(st.acc[r][1]), c = split2(st.acc[r][2]), e = split2(st.acc[r][3]);
    to[0] = make_float4(a.x, a.y, b.x, b.y);
    to[1] = make_float4(c.x, c.y, e.x, e.y);
  }
  __syncthreads();
  // join the warps: thread t has columns 2 (t % 128), rows t / 128, + 2, ...
  const int c2 = (threadIdx.x & 127) * 2;
  for (int r = threadIdx.x >> 7; r < rows; r += kWarps / 4) {
    float m = claimed > places ? 0.f : -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, m_s[w * R + r]);
    float sum = claimed > places ? static_cast<float>(claimed - places) * ex2_approx(-m) : 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = m_s[w * R + r];
      const float a = mw == -INFINITY ? 0.f : ex2_approx(mw - m);  // a warp that saw no key
      const float2 o = *reinterpret_cast<const float2*>(acc_s + (w * R + r) * kHeadDim + c2);
      sum = fmaf(a, l_s[w * R + r], sum);
      x = fmaf(a, o.x, x);
      y = fmaf(a, o.y, y);
    }
    const float inv = 1.f / sum;
    const int64_t row = q0 + r / p.G;
    const int h = head * p.G + r % p.G;
    *reinterpret_cast<uint32_t*>(p.out + row * p.ldo + static_cast<int64_t>(h) * kHeadDim + c2) =
        pack_bf16x2(x * inv, y * inv);
    if (p.lse && c2 == 0) p.lse[row * p.n_q + h] = (m + log2f(sum)) * 0.69314718055994531f;
  }
}

template <int R>
constexpr int few_smem() {
  return (Few<R>::WARPS * R * kHeadDim + 2 * Few<R>::WARPS * R) * static_cast<int>(sizeof(float));
}

template <int R>
cudaError_t launch_rows(const CacheRowsParams& p, int n_docs, cudaStream_t s) {
  return launch_pdl(cache_rows_attention_kernel<R>, dim3(static_cast<unsigned>(n_docs * p.n_kv)), dim3(Few<R>::WARPS * 32),
                    few_smem<R>(), s, p);
}

}  // namespace

kalm_status launch_cache_rows_attention(const CacheRowsParams& p, int32_t n_docs, cudaStream_t stream) {
  const int rows = p.max_q * p.G;
  if (static_cast<int64_t>(n_docs) * p.n_kv > INT32_MAX)
    return fail(KALM_ERR_INVALID_ARG, "kalm_merged_attention_cache: too many work items");
  static_assert(KALM_CACHE_FEW_ROWS == 8 && few_smem<4>() <= 48 * 1024 && few_smem<8>() <= 48 * 1024, "row counts and shared memory");
  return check_cuda(rows <= 1   ? launch_rows<1>(p, n_docs, stream)
                    : rows <= 2 ? launch_rows<2>(p, n_docs, stream)
                    : rows <= 4 ? launch_rows<4>(p, n_docs, stream)
                                : launch_rows<8>(p, n_docs, stream),
                    "launch cache_rows_attention_kernel");
}

}  // namespace kalm
