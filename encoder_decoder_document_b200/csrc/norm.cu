// The norms around a decoder block: the RMS norm of a block's input, and, between two blocks, the RMS norm of the
// first one's output, its gate, the residual sum and the next one's input norm in one pass.
// "KaLM-Reranker-V1-Nano - MLX (Apple Silicon)", "Derivation": the decoder's layers are those of the base
// model's configuration; the pages do not spell its norms out.
//
// For a row, with norm(v, w) = v * rsqrt(mean(v^2) + eps) * (w + weight_offset):
//   t = residual_scale * x + gate * norm(y, w_post);   x_out = t;   h = norm(t, w_pre)
// Everything is held in fp32 from the loads to one rounding per output: h is the norm of t itself, not of the
// rounded x_out.
//
// Bound by memory (8 bytes a value: y, x, x_out, h).  A row lives in the registers of 8 lanes, a warp or a block,
// so each input is read once; the two sums of squares are shuffles (and one exchange through shared memory
// per sum in the block form).  Pairs of values share an instruction (f32x2), which halved the issue slots
// (121 -> 108 us at 26,077 x 2,560); a document's gate is asked for before the first sum, not after it (108 -> 90
// us: it comes from L2, and its latency stood behind the sum's).
// Measured (CUDA graph of calls over three sets of inputs; one gate for all / a gate per document): 12,800 x 640
// 15.1 / 16.9 us = 4.3 TB/s; 25,600 x 1,152 41.8 / 45.2 us = 5.6 TB/s; 26,077 x 2,560 85.6 / 95.4 us = 6.2 TB/s (0.95 of
// the copy bandwidth); 8,000 x 8,192 89.0 / 99.4 us = 5.9 TB/s; kalm_rms_norm of 26,077 x 2,560 42.4 us = 6.3 TB/s.  (From
// card to card these move by up to a tenth; the comparisons below are of one card each.)
#include <algorithm>
#include <cmath>

#include "kalm.h"
#include "kalm_internal.h"
#include "kalm_ptx.cuh"
#include "kalm_wide.cuh"

namespace kalm {
namespace {

constexpr int kWarpRowThreads = 128;  // block of the warp-per-row form (256: 12,800 x 640 in 14.9 us instead of 14.0 then)
constexpr int kMaxWidth = KALM_NORM_MAX_WIDTH;
constexpr uint32_t kSiteNorm = 9u << 8;  // device error word (see kalm_check_device_errors in kalm.h)
constexpr int kBlockRow = 448;                // threads of a block-per-row block, at most
constexpr int kWideRow = kMaxWidth / 8 / 4;   // and of the widest rows': four 8-column units each

struct NormParams {
  const uint4* y;       // block output (NULL: a norm of x alone)
  const uint4* x;       // residual stream
  const uint4* w_post;  // NULL: y enters as it is
  const uint4* gate;    // NULL: 1
  const uint4* w_pre;
  uint4* x_out;         // where y is
  uint4* h;             // NULL: not written (where y is)
  const int64_t* q_off; // rows of each document; NULL: all rows
  int64_t ldy, ldx, ld_gate, ldxo, ldh;  // in 16-byte units
  int64_t rows;
  int n_docs;
  int nv;               // 8-column units of a row
  float residual_scale, weight_offset, eps, inv_width;
  uint32_t* err;
};

__device__ __forceinline__ uint32_t pack2(F2 v) {
  const float2 f = split2(v);
  return pack_bf16x2(f.x, f.y);
}

// A row's sum over its threads: SPAN lanes of a warp (a power of two), or the whole block where SPAN is more than a warp
// (through `part`, one slot per warp).
template <int SPAN>
__device__ __forceinline__ float row_sum(F2 v2, float* part) {
  const float2 f = split2(v2);
  float v = f.x + f.y;
#pragma unroll
  for (int o = (SPAN <= 32 ? SPAN : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (SPAN > 32) {
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < warps; ++w) v += part[w];
  }
  return v;
}

// V: 8-column units a thread holds; unit i of thread t is i * (threads of the row) + t.  SPAN: lanes of a row, or the most
// threads of its block.  SUM: y is there (else a norm of x alone, whose fewer registers let more rows be in flight:
// 26,077 x 2,560 in 40.9 us instead of 44.8).
// Registers are bounded where that makes room for one more warp or block on an SM at (nearly) no spill; at a gate per
// document, without and with: five units a lane of a warp 44.0 and 41.9 us (25,600 x 1,152), four of a block 98 and 95
// (8,000 x 8,192), four of the widest rows' 141 and 106 (4,000 x 16,384; the next smaller form has one block an SM there).
template <int V, int SPAN, bool SUM>
__global__ void __launch_bounds__(SPAN <= 32 ? kWarpRowThreads : SPAN, SPAN == 32 && V == 5  ? 7
                                                                     : SPAN > 32 && V == 4 ? 2
                                                                                           : 0)
    norm_kernel(const NormParams p) {
  pdl_launch_dependents();
  pdl_wait_predecessor();
  // Documents whose rows are not all there are flagged by one thread; the rows that are get computed.  (In the last block,
  // which starts late in any case: 12,800 x 640 in 15.8 us, with the check beside the search 16.3, without one 15.7.)
  if (SUM && p.q_off && blockIdx.x == gridDim.x - 1 && threadIdx.x == 0 &&
      (__ldg(p.q_off) < 0 || __ldg(p.q_off + p.n_docs) > p.rows))
    record_error(p.err, kErrDeviceArg | kSiteNorm);
  __shared__ float part[2][SPAN <= 32 ? 1 : SPAN / 32];
  const int lane = threadIdx.x & 31;
  constexpr bool kLanes = SPAN <= 32;
  const int span = kLanes ? SPAN : blockDim.x;
  const int t = kLanes ? lane & (SPAN - 1) : threadIdx.x;
  const int64_t row = kLanes ? (static_cast<int64_t>(blockIdx.x) * kWarpRowThreads + threadIdx.x) / SPAN
                             : static_cast<int64_t>(blockIdx.x);
  // rows of no document, or past the last, are computed as zeros (their threads take part in the shuffles) and not written
  bool there = row < p.rows;
  // The row's document: up to 32 threads search together, four offsets each a round.  The first round's
  // offsets are asked for before x and y: loads come back in order, so that up to 128 documents cost the
  // latency of no load but the gate's own.
  constexpr int kWays = kLanes ? SPAN : 32;
  const int way = lane & (kWays - 1);
  const bool docs = SUM && p.q_off;
  int lo = 0, hi = docs ? p.n_docs : 0, step = max(1, (hi + 4 * kWays - 1) / (4 * kWays));
  int64_t o[4], o_first = 0, o_last = 0;
  if (docs) {
    o_first = __ldg(p.q_off);
    o_last = __ldg(p.q_off + p.n_docs);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = step * (j * kWays + way + 1);
      o[j] = at < hi ? __ldg(p.q_off + at) : INT64_MAX;
    }
  }
  uint4 xv[V], yv[SUM ? V : 1];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * span + t;
    xv[i] = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (SUM) yv[i] = xv[i];
    if (there && c < p.nv) {
      xv[i] = p.x[row * p.ldx + c];
      if constexpr (SUM) yv[i] = p.y[row * p.ldy + c];
    }
  }
  if (docs) {
    there = there && row >= o_first && row < o_last;
    while (true) {
      int n = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned below = __ballot_sync(0xffffffffu, o[j] <= row);
        n += __popc(kWays == 32 ? below : (below >> (lane & ~(kWays - 1))) & ((1u << (kWays & 31)) - 1u));
      }
      hi = min(hi, lo + step * (n + 1));
      lo += step * n;
      if (!__any_sync(0xffffffffu, hi - lo > 1)) break;
      step = max(1, (hi - lo + 4 * kWays - 1) / (4 * kWays));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = lo + step * (j * kWays + way + 1);
        o[j] = at < hi ? __ldg(p.q_off + at) : INT64_MAX;
      }
    }
    if (!kLanes && !there) return;  // the whole block's row
  }
  const int doc = lo;
  const F2 off = pair2(p.weight_offset, p.weight_offset);
  F2 r[V][4];
  if constexpr (SUM) {
    uint4 gv[V];  // asked for before the first sum: a document's gate comes from L2
#pragma unroll
    for (int i = 0; i < V; ++i) {
      gv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (p.gate) gv[i] = __ldg(p.gate + doc * p.ld_gate + min(i * span + t, p.nv - 1));
    }
    float rs = 1.f;
    if (p.w_post) {
      F2 ss = 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const F2 y = unpack2((&yv[i].x)[k]);
          ss = fma2(y, y, ss);
        }
      rs = rsqrtf(fmaf(row_sum<SPAN>(ss, part[0]), p.inv_width, p.eps));
    }
    const F2 rs2 = pair2(rs, rs), scale2 = pair2(p.residual_scale, p.residual_scale);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = min(i * span + t, p.nv - 1);  // (columns past the row are zeros, whatever their weight)
      uint4 wv = make_uint4(0u, 0u, 0u, 0u);
      if (p.w_post) wv = __ldg(p.w_post + c);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        F2 u = unpack2((&yv[i].x)[k]);
        if (p.w_post) u = mul2(mul2(u, rs2), add2(unpack2((&wv.x)[k]), off));
        const F2 x = unpack2((&xv[i].x)[k]);
        r[i][k] = p.gate ? fma2(u, unpack2((&gv[i].x)[k]), mul2(x, scale2)) : fma2(x, scale2, u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) r[i][k] = unpack2((&xv[i].x)[k]);
  }
  float rs = 0.f;
  if (!SUM || p.h) {
    F2 ss = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) ss = fma2(r[i][k], r[i][k], ss);
    rs = rsqrtf(fmaf(row_sum<SPAN>(ss, part[1]), p.inv_width, p.eps));
  }
  const F2 rs2 = pair2(rs, rs);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * span + t;
    if (!there || c >= p.nv) continue;
    if (SUM)
      p.x_out[row * p.ldxo + c] = make_uint4(pack2(r[i][0]), pack2(r[i][1]), pack2(r[i][2]), pack2(r[i][3]));
    if (!SUM || p.h) {
      const uint4 wv = __ldg(p.w_pre + c);
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = pack2(mul2(mul2(r[i][k], rs2), add2(unpack2((&wv.x)[k]), off)));
      p.h[row * p.ldh + c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <int SPAN, bool SUM>
cudaError_t launch_norm(int v, dim3 grid, dim3 block, cudaStream_t s, const NormParams& p) {
  if constexpr (SPAN == kWideRow) {
    return launch_pdl(norm_kernel<4, SPAN, SUM>, grid, block, 0, s, p);
  } else {
    if constexpr (SPAN <= 32) {  // (a block's threads have three units at least)
      if (v == 1) return launch_pdl(norm_kernel<1, SPAN, SUM>, grid, block, 0, s, p);
      if (v == 2) return launch_pdl(norm_kernel<2, SPAN, SUM>, grid, block, 0, s, p);
    }
    return v <= 3   ? launch_pdl(norm_kernel<3, SPAN, SUM>, grid, block, 0, s, p)
           : v == 4 ? launch_pdl(norm_kernel<4, SPAN, SUM>, grid, block, 0, s, p)
                    : launch_pdl(norm_kernel<5, SPAN, SUM>, grid, block, 0, s, p);
  }
}

template <bool SUM>
cudaError_t launch(const NormParams& p, cudaStream_t s) {
  // The fewest threads a row with at most five units each: 8 lanes, a warp, or whole warps (a block per row).  At
  // 26,077 x 2,560 (a gate per document) 64 threads x 5 units took 90 us, 96 x 4 100, 128 x 3 92, 160 x 2 94; at
  // 25,600 x 1,152 32 x 5 took 44 us, 64 x 3 47, 96 x 2 52; at 12,800 x 640 32 x 3 took 14 us, 16 x 5 16.  Wide rows have
  // four: their blocks are large, and with five fewer of them fit an SM (9,000 x 7,168: 224 x 4 89 us, 192 x 5 95;
  // 8,000 x 8,192: 256 x 4 96 us, 224 x 5 103, 352 x 3 96, 512 x 2 114; but 9,000 x 5,120: 128 x 5 68 us, 160 x 4 71).
  const int most = p.nv <= 800 ? 5 : 4;
  const int span = p.nv <= 8 ? 8 : 32 * ((p.nv + 32 * most - 1) / (32 * most));
  const int v = (p.nv + span - 1) / span;
  const int per_block = span <= 32 ? kWarpRowThreads / span : 1;
  const dim3 grid(static_cast<unsigned>(std::max((p.rows + per_block - 1) / per_block, int64_t{1})));  // (1: the offsets' check)
  return span == 8    ? launch_pdl(norm_kernel<1, 8, SUM>, grid, dim3(kWarpRowThreads), 0, s, p)
         : span == 32 ? launch_norm<32, SUM>(v, grid, dim3(kWarpRowThreads), s, p)
         : span <= kBlockRow ? launch_norm<kBlockRow, SUM>(v, grid, dim3(span), s, p)
                             : launch_norm<kWideRow, SUM>(v, grid, dim3(span), s, p);
}

bool bad_rows(const void* a, int64_t ld, int32_t width) { return !aligned16(a) || ld % 8 || ld < width; }

kalm_status check_norm_sizes(const char* what, int64_t rows, int32_t width, float eps, float weight_offset) {
  if (rows < 0 || rows > INT32_MAX - 1024 || width <= 0 || width % 8 || width > kMaxWidth)
    return fail(KALM_ERR_INVALID_ARG, "%s: rows=%lld width=%d (a multiple of 8 up to %d)", what, (long long)rows, width,
                kMaxWidth);
  if (!(eps > 0.f) || !std::isfinite(eps) || !std::isfinite(weight_offset))
    return fail(KALM_ERR_INVALID_ARG, "%s: eps must be positive, eps and weight_offset finite", what);
  return KALM_OK;
}

}  // namespace
}  // namespace kalm

using namespace kalm;

extern "C" kalm_status kalm_rms_norm(const kalm_bf16* x, int64_t ldx, const kalm_bf16* w, kalm_bf16* h, int64_t ldh,
                                     int64_t rows, int32_t width, float eps, float weight_offset,
                                     kalm_stream_t stream) {
  kalm_status st = check_norm_sizes("kalm_rms_norm", rows, width, eps, weight_offset);
  if (st != KALM_OK) return st;
  if (rows > 0) {
    if (!x || !w || !h) return fail(KALM_ERR_INVALID_ARG, "kalm_rms_norm: NULL pointer");
    if (bad_rows(x, ldx, width) || bad_rows(h, ldh, width) || !aligned16(w))
      return fail(KALM_ERR_INVALID_ARG, "kalm_rms_norm: bad alignment or stride (ldx=%lld ldh=%lld width=%d)",
                  (long long)ldx, (long long)ldh, width);
  }
  if ((st = ensure_device(nullptr)) != KALM_OK) return st;
  if (rows == 0) return KALM_OK;
  NormParams p{};
  p.x = reinterpret_cast<const uint4*>(x);
  p.ldx = ldx / 8;
  p.w_pre = reinterpret_cast<const uint4*>(w);
  p.h = reinterpret_cast<uint4*>(h);
  p.ldh = ldh / 8;
  p.rows = rows;
  p.nv = width / 8;
  p.weight_offset = weight_offset;
  p.eps = eps;
  p.inv_width = 1.f / static_cast<float>(width);
  return check_cuda(launch<false>(p, static_cast<cudaStream_t>(stream)), "launch norm_kernel (kalm_rms_norm)");
}

extern "C" kalm_status kalm_norm_residual(const kalm_bf16* y, int64_t ldy, const kalm_bf16* x, int64_t ldx,
                                          const kalm_bf16* w_post, const kalm_bf16* gate, int64_t ld_gate,
                                          const int64_t* q_off, int32_t n_docs, float residual_scale, kalm_bf16* x_out,
                                          int64_t ldxo, const kalm_bf16* w_pre, kalm_bf16* h, int64_t ldh, int64_t rows,
                                          int32_t width, float eps, float weight_offset, kalm_stream_t stream) {
  kalm_status st = check_norm_sizes("kalm_norm_residual", rows, width, eps, weight_offset);
  if (st != KALM_OK) return st;
  if (!std::isfinite(residual_scale)) return fail(KALM_ERR_INVALID_ARG, "kalm_norm_residual: residual_scale not finite");
  if (n_docs < 0 || ld_gate < 0) return fail(KALM_ERR_INVALID_ARG, "kalm_norm_residual: negative size");
  if (gate && ld_gate && !q_off)
    return fail(KALM_ERR_INVALID_ARG, "kalm_norm_residual: a gate per document needs q_off");
  if (rows > 0 && (h != nullptr) != (w_pre != nullptr))  // (without rows h may have no address)
    return fail(KALM_ERR_INVALID_ARG, "kalm_norm_residual: h and w_pre go together");
  const bool none = q_off ? n_docs == 0 : rows == 0;
  if (!none && rows > 0) {
    if (!y || !x || !x_out) return fail(KALM_ERR_INVALID_ARG, "kalm_norm_residual: NULL pointer");
    if (bad_rows(y, ldy, width) || bad_rows(x, ldx, width) || bad_rows(x_out, ldxo, width) ||
        (h && bad_rows(h, ldh, width)) || !aligned16(w_post) || !aligned16(w_pre) || !aligned16(gate) ||
        (gate && ld_gate && (ld_gate % 8 || ld_gate < width)))
      return fail(KALM_ERR_INVALID_ARG, "kalm_norm_residual: bad alignment or stride for width %d", width);
    if (h && h == x_out) return fail(KALM_ERR_INVALID_ARG, "kalm_norm_residual: h and x_out are the same memory");
  }
  if ((st = ensure_device(nullptr)) != KALM_OK) return st;
  if (none) return KALM_OK;
  if (rows == 0) w_post = gate = w_pre = h = nullptr;  // only the offsets' check is left to do
  NormParams p{};
  p.y = reinterpret_cast<const uint4*>(y);
  p.ldy = ldy / 8;
  p.x = reinterpret_cast<const uint4*>(x);
  p.ldx = ldx / 8;
  p.w_post = reinterpret_cast<const uint4*>(w_post);
  p.gate = reinterpret_cast<const uint4*>(gate);
  p.ld_gate = ld_gate / 8;
  p.q_off = q_off;
  p.n_docs = n_docs;
  p.err = device_error_word();
  p.residual_scale = residual_scale;
  p.x_out = reinterpret_cast<uint4*>(x_out);
  p.ldxo = ldxo / 8;
  p.w_pre = reinterpret_cast<const uint4*>(w_pre);
  p.h = reinterpret_cast<uint4*>(h);
  p.ldh = ldh / 8;
  p.rows = rows;
  p.nv = width / 8;
  p.weight_offset = weight_offset;
  p.eps = eps;
  p.inv_width = 1.f / static_cast<float>(width);
  return check_cuda(launch<true>(p, static_cast<cudaStream_t>(stream)), "launch norm_kernel (kalm_norm_residual)");
}
