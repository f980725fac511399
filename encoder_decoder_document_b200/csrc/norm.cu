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
// Bound by memory (8 bytes a value: y, x, x_out, h).  A row lives in the registers of one warp (up to 1,024
// columns) or one block, so each input is read once; the two sums of squares are shuffles (and one exchange
// through shared memory per sum in the block form).
#include <cmath>

#include "kalm.h"
#include "kalm_internal.h"
#include "kalm_ptx.cuh"

namespace kalm {
namespace {

constexpr int kWarpRowThreads = 256;  // block of the warp-per-row form
constexpr int kMaxWidth = KALM_NORM_MAX_WIDTH;

struct NormParams {
  const uint4* y;       // block output, or NULL: a norm of x alone
  const uint4* x;       // residual stream
  const uint4* w_post;  // NULL: y enters as it is
  const uint4* gate;    // NULL: 1
  const uint4* w_pre;
  uint4* x_out;         // NULL: not written
  uint4* h;             // NULL: not written
  const int64_t* q_off; // rows of each document; NULL: all rows
  int64_t ldy, ldx, ld_gate, ldxo, ldh;  // in 16-byte units
  int64_t rows;
  int n_docs;
  int nv;               // 8-column units of a row
  float residual_scale, weight_offset, eps, inv_width;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Sum over the row's threads: the warp, or the block (through `part`, one slot per warp).
template <bool BLOCK>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (BLOCK) {
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < warps; ++w) v += part[w];
  }
  return v;
}

// V: 8-column units a thread holds; unit i of thread t is i * (threads of the row) + t.
template <int V, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kMaxWidth / 32 : kWarpRowThreads) norm_kernel(const NormParams p) {
  pdl_launch_dependents();
  pdl_wait_predecessor();
  __shared__ float part[2][kMaxWidth / 1024];
  const int lane = threadIdx.x & 31;
  const int span = BLOCK ? blockDim.x : 32;
  const int t = BLOCK ? threadIdx.x : lane;
  const int64_t row = BLOCK ? static_cast<int64_t>(blockIdx.x)
                            : static_cast<int64_t>(blockIdx.x) * (kWarpRowThreads / 32) + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  uint4 xv[V], yv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * span + t;
    xv[i] = yv[i] = make_uint4(0u, 0u, 0u, 0u);
    if (c < p.nv) {
      xv[i] = p.x[row * p.ldx + c];
      if (p.y) yv[i] = p.y[row * p.ldy + c];
    }
  }
  int doc = 0;
  if (p.q_off) {  // the row's document; a row of none is left as it was
    int lo = 0, hi = p.n_docs;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = lo + step * (lane + 1);
      const int n = __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(p.q_off + at) <= row));
      hi = min(hi, lo + step * (n + 1));
      lo += step * n;
    }
    doc = lo;
    if (row < __ldg(p.q_off + doc) || row >= __ldg(p.q_off + doc + 1)) return;  // same for the whole row
  }
  float r[V][8];
  if (p.y) {
    float ss = 0.f;
    if (p.w_post) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float f[8];
        unpack8(yv[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(f[k], f[k], ss);
      }
      ss = row_sum<BLOCK>(ss, part[0]);
    }
    const float rs = p.w_post ? rsqrtf(fmaf(ss, p.inv_width, p.eps)) : 1.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * span + t;
      float x[8], y[8];
      unpack8(xv[i], x);
      unpack8(yv[i], y);
      if (p.w_post) {
        float w[8];
        unpack8(c < p.nv ? __ldg(p.w_post + c) : make_uint4(0u, 0u, 0u, 0u), w);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = y[k] * rs * (w[k] + p.weight_offset);
      }
      if (p.gate) {
        float g[8];
        unpack8(c < p.nv ? __ldg(p.gate + doc * p.ld_gate + c) : make_uint4(0u, 0u, 0u, 0u), g);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] *= g[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) r[i][k] = fmaf(p.residual_scale, x[k], y[k]);
      if (p.x_out && c < p.nv) xv[i] = pack8(r[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) unpack8(xv[i], r[i]);
  }
  if (p.h) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(r[i][k], r[i][k], ss);
    ss = row_sum<BLOCK>(ss, part[1]);
    const float rs = rsqrtf(fmaf(ss, p.inv_width, p.eps));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * span + t;
      if (c >= p.nv) continue;
      float w[8];
      unpack8(__ldg(p.w_pre + c), w);
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = r[i][k] * rs * (w[k] + p.weight_offset);
      p.h[row * p.ldh + c] = pack8(w);
    }
  }
  if (p.x_out) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * span + t;
      if (c < p.nv) p.x_out[row * p.ldxo + c] = xv[i];
    }
  }
}

template <bool BLOCK>
cudaError_t launch_norm(int v, dim3 grid, dim3 block, cudaStream_t s, const NormParams& p) {
  switch (v) {
    case 1: return launch_pdl(norm_kernel<1, BLOCK>, grid, block, 0, s, p);
    case 2: return launch_pdl(norm_kernel<2, BLOCK>, grid, block, 0, s, p);
    case 3: return launch_pdl(norm_kernel<3, BLOCK>, grid, block, 0, s, p);
    default: return launch_pdl(norm_kernel<4, BLOCK>, grid, block, 0, s, p);
  }
}

kalm_status run_norm(const char* what, const NormParams& p, cudaStream_t s) {
  cudaError_t e;
  if (p.nv <= 128) {  // a warp per row
    const int64_t blocks = (p.rows + kWarpRowThreads / 32 - 1) / (kWarpRowThreads / 32);
    e = launch_norm<false>((p.nv + 31) / 32, dim3(static_cast<unsigned>(blocks)), dim3(kWarpRowThreads), s, p);
  } else {  // a block per row, four units a thread
    const int threads = 32 * ((p.nv + 127) / 128);
    e = launch_norm<true>(4, dim3(static_cast<unsigned>(p.rows)), dim3(threads), s, p);
  }
  return check_cuda(e, what);
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
  return run_norm("launch norm_kernel (kalm_rms_norm)", p, static_cast<cudaStream_t>(stream));
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
  if ((h != nullptr) != (w_pre != nullptr))
    return fail(KALM_ERR_INVALID_ARG, "kalm_norm_residual: h and w_pre go together");
  const bool none = rows == 0 || (q_off && n_docs == 0);
  if (!none) {
    if (!y || !x || !x_out) return fail(KALM_ERR_INVALID_ARG, "kalm_norm_residual: NULL pointer");
    if (bad_rows(y, ldy, width) || bad_rows(x, ldx, width) || bad_rows(x_out, ldxo, width) ||
        (h && bad_rows(h, ldh, width)) || !aligned16(w_post) || !aligned16(w_pre) || !aligned16(gate) ||
        (gate && ld_gate && (ld_gate % 8 || ld_gate < width)))
      return fail(KALM_ERR_INVALID_ARG, "kalm_norm_residual: bad alignment or stride for width %d", width);
    if (h && h == x_out) return fail(KALM_ERR_INVALID_ARG, "kalm_norm_residual: h and x_out are the same memory");
  }
  if ((st = ensure_device(nullptr)) != KALM_OK) return st;
  if (none) return KALM_OK;
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
  return run_norm("launch norm_kernel (kalm_norm_residual)", p, static_cast<cudaStream_t>(stream));
}
