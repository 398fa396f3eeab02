// Per-token int8 quantization of many rows in natural order, for the many-token int8 operators: the decode
// quantizer's codes and scale (per-token absmax int8, technical summary §2.B-C), optionally of the
// RMS-normalised row (the final norm before the head).
//
// One CTA per token, eight consecutive values per thread and chunk, held in registers between the passes
// (sum of squares, absmax, codes), so each row is read once.  Rows of 2048 fp32 values, 2048 of them: 21 MB,
// bound by memory; a single row is bound by its latency (two block reductions).

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "rows.cuh"

namespace dfssm {
namespace {

constexpr int RQ_THREADS = 256;

// Part `part` of the scan (whole CTA).
__device__ __forceinline__ void scan_range(const RowsQuantArgs& a, int part) {
  __shared__ uint2 red[RQ_THREADS / 32];
  const int run = scan_run(a.V), per = RQ_THREADS / run;  // runs of the CTA at a time
  const long long runs = (a.V + run - 1) / run;
  uint32_t m = 0u, neg = 0u;
#pragma unroll 4
  for (long long r = part + (long long)kScanParts * (threadIdx.x / run); r < runs; r += (long long)kScanParts * per) {
    const long long v = r * run + threadIdx.x % run;
    const float s = v < a.V ? ld_f32(a.scan + v) : 0.0f;
    m = max(m, __float_as_uint(s) & 0x7FFFFFFFu);  // orders like |s|, a NaN above all
    neg |= s < 0.0f ? 1u : 0u;
  }
  m = __reduce_max_sync(0xffffffffu, m);
  neg = __reduce_or_sync(0xffffffffu, neg);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_uint2(m, neg);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < RQ_THREADS / 32; ++w) m = max(m, red[w].x), neg |= red[w].y;
    a.range[part] = make_uint2(m, neg);
  }
}

// CH: chunks of 2048 values a row may have.  SCAN: the last kScanParts CTAs look over a.scan.
template <typename T, int CH, bool SCAN>
__global__ void __launch_bounds__(RQ_THREADS) rows_quant_kernel(RowsQuantArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ double red_ss[RQ_THREADS / 32];
  __shared__ uint32_t red_m[RQ_THREADS / 32];
  __shared__ float red_rn;
  const int tok = blockIdx.x;
  if (SCAN && tok >= a.M) {
    scan_range(a, tok - a.M);
    return;
  }
  const T* xr = reinterpret_cast<const T*>(a.x) + (size_t)tok * a.ldx;
  float v[CH][8], nw[CH][8];  // the row, and the norm's weight with it
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (threadIdx.x + RQ_THREADS * c) * 8;
    if (i < a.d) {
      load8<T>(xr + i, v[c]);
      if (a.norm_w) load8<float>(a.norm_w + i, nw[c]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[c][k] = 0.0f;
    }
  }
  if (a.norm_w) {
    double ss = 0.0;  // exact squares in fp64
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fma((double)v[c][k], (double)v[c][k], ss);
    ss = warp_sum(ss);
    if (lane == 0) red_ss[warp] = ss;
    __syncthreads();
    if (warp == 0) {  // fp64 division and root once, not in every warp
      ss = warp_sum(lane < RQ_THREADS / 32 ? red_ss[lane] : 0.0);
      const float r = rms_factor(ss, a.d);
      if (lane == 0) {
        red_rn = r;
        if (a.rn) a.rn[tok] = r;
      }
    }
    __syncthreads();
    const float rn = red_rn;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (threadIdx.x + RQ_THREADS * c) * 8;
      if (i < a.d) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[c][k] = norm_value(v[c][k], rn, nw[c][k]);
      }
    }
  }
  // absmax as an unsigned pattern: infinities and NaN order above every finite value
  uint32_t mb = 0u;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) mb = max(mb, __float_as_uint(v[c][k]) & 0x7FFFFFFFu);
  mb = __reduce_max_sync(0xffffffffu, mb);
  if (lane == 0) red_m[warp] = mb;
  __syncthreads();
  mb = 0u;
#pragma unroll
  for (int w = 0; w < RQ_THREADS / 32; ++w) mb = max(mb, red_m[w]);
  const bool finite = mb < 0x7F800000u;
  // a token with a value that is not finite has the scale NaN (and zero codes): so are its outputs
  const float s0 = finite ? quant_scale(__uint_as_float(mb)) : __uint_as_float(0x7FC00000u);
  const float inv = finite ? quant_inv(s0) : 0.0f;
  if (threadIdx.x == 0) {
    a.s[tok] = (double)s0;
    if (a.dbg_s) a.dbg_s[tok] = s0;
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (threadIdx.x + RQ_THREADS * c) * 8;
    if (i >= a.d) continue;
    int cd[8];
    quant_codes<8>(v[c], s0, inv, cd);
    const uint2 o = finite ? pack_codes(cd) : make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(a.q + (size_t)tok * a.d + i) = o;
    if (a.dbg_q) *reinterpret_cast<uint2*>(a.dbg_q + (size_t)tok * a.d + i) = o;
  }
}

template <typename T, bool SCAN>
cudaError_t launch(const RowsQuantArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)a.M + (SCAN ? kScanParts : 0));
  if (a.d <= 8 * RQ_THREADS) return launch_pdl(rows_quant_kernel<T, 1, SCAN>, grid, dim3(RQ_THREADS), 0, st, a);
  if (a.d <= 16 * RQ_THREADS) return launch_pdl(rows_quant_kernel<T, 2, SCAN>, grid, dim3(RQ_THREADS), 0, st, a);
  return launch_pdl(rows_quant_kernel<T, 4, SCAN>, grid, dim3(RQ_THREADS), 0, st, a);
}

}  // namespace

cudaError_t launch_rows_quant(const RowsQuantArgs& a, cudaStream_t st) {
  if (a.scan) return a.x_type == DFSSM_BF16 ? launch<__nv_bfloat16, true>(a, st) : launch<float, true>(a, st);
  return a.x_type == DFSSM_BF16 ? launch<__nv_bfloat16, false>(a, st) : launch<float, false>(a, st);
}

}  // namespace dfssm
