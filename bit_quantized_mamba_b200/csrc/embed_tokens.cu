// Embedding of many tokens from the tied int8 matrix (technical summary §2.B: int8 embedding with per-row
// scaling), and its gradient (include/dfssm.h, dfssm_embed_tokens and dfssm_embed_tokens_backward).
//
// Forward: h[t][i] = fl32(W[tok_t][i] s_row[tok_t]) — a gather bound by memory (the output is four or two times
// the table rows read).  Four (fp32) or eight (bf16) values a thread, so that both the loads and the stores of
// a warp are contiguous.
//
// Gradient: dE[v][i] = sum over t with tok_t = v of dh[t][i] and ds_row[v] = sum_i W[v][i] dE[v][i], in an order
// fixed by the tokens alone:
//   1. sort the positions by token (stable).  Up to 16384 tokens one CTA sorts them in shared memory while the
//      other SMs write the zero rows of the dense gradient, whose stores are most of the traffic; more tokens
//      take a radix sort over the whole device.
//   2. the sorted positions are cut into windows of equal length, one CTA each, however often a token
//      repeats; a run of equal tokens inside a window is final, one that crosses windows leaves partial sums, which
//      the last of its CTAs to finish adds in order.
//
// 16384 tokens of 2048: forward (bf16) 18 us a call, 14.6 on the device alone (the 67 MB it writes at 4.6 TB/s); gradient of
// 50288 rows (bf16) 110 us for 490 MB read and written (4.5 TB/s).  500 tokens: 17 us, two launches in a row.

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "rows.cuh"

namespace dfssm {
namespace {

inline size_t al256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool al(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// ------------------------------------------------------------------------------------ forward

struct EmbedTokensArgs {
  const int8_t* W;
  const float* s_row;
  const int32_t* tokens;
  void* h;
  int64_t ldh;
  int* status;
  int V, d, n;
};

// WPT warps per token (8 or 1): a CTA for a token where there are few tokens, a warp where they fill the device, with
// the loads of four pieces of a row in flight.
template <typename T, int WPT>
__global__ void __launch_bounds__(256) embed_tokens_kernel(EmbedTokensArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int N = sizeof(T) == 4 ? 4 : 8, STEP = WPT * 32 * N, U = 4;  // values a thread handles at a time
  const int per_cta = 8 / WPT, sub = (threadIdx.x >> 5) / WPT, i0 = (threadIdx.x % (WPT * 32)) * N;
  for (int t = blockIdx.x * per_cta + sub; t < a.n; t += gridDim.x * per_cta) {
    const int tok = ld_s32(a.tokens + t);
    const bool ok = tok >= 0 && tok < a.V;
    if (!ok && i0 == 0) atomicExch(a.status, kBadTokenCode);
    const float sc = ok ? ld_f32(a.s_row + tok) : 0.0f;
    const int8_t* row = a.W + (size_t)(ok ? tok : 0) * a.d;
    T* h = reinterpret_cast<T*>(a.h) + (int64_t)t * a.ldh;
    for (int i = i0; i < a.d; i += U * STEP) {
      uint2 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = i + u * STEP;
        w[u] = make_uint2(0u, 0u);
        if (k < a.d) {
          if (N == 8) w[u] = __ldg(reinterpret_cast<const uint2*>(row + k));
          else w[u].x = __ldg(reinterpret_cast<const uint32_t*>(row + k));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = i + u * STEP;
        if (k >= a.d) continue;
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = ok ? fmul((float)(int8_t)(w[u].x >> (8 * j)), sc) : 0.0f;
          v[j + 4] = ok ? fmul((float)(int8_t)(w[u].y >> (8 * j)), sc) : 0.0f;
        }
        if constexpr (N == 8) store8<T>(h + k, v);
        else st_f4(h + k, make_float4(v[0], v[1], v[2], v[3]));
      }
    }
  }
}

template <typename T>
cudaError_t launch_embed_tokens(const EmbedTokensArgs& a, cudaStream_t st) {
  const int most = num_sms() * 8;  // CTAs resident at a time
  if (a.n <= most) return launch_pdl(embed_tokens_kernel<T, 8>, dim3(a.n), dim3(256), 0, st, a);
  const int ctas = a.n / 8 + (a.n % 8 != 0);
  return launch_pdl(embed_tokens_kernel<T, 1>, dim3(ctas < most ? ctas : most), dim3(256), 0, st, a);
}

// ------------------------------------------------------------------------------------ sort

constexpr int SORT_THREADS = 1024, SORT_WARPS = 32;
constexpr int SORT_MAX = 16384;  // tokens one CTA sorts: two copies of (id, position) beside the counts
constexpr size_t SORT_SMEM = (size_t)SORT_MAX * 2 * 4 + (size_t)SORT_MAX * 2 * 2 + 256 * SORT_WARPS * 4;

// Count of (digit, warp): digits in order, warps in order within one; rotated by the digit so that a warp's
// lanes, which share the warp index, fall into different banks.
__device__ __forceinline__ int at_count(int dg, int warp) { return dg * SORT_WARPS + ((warp + dg) & (SORT_WARPS - 1)); }

// Exclusive scan of the 256 x SORT_WARPS counts in place (8 entries per thread), whole CTA.
__device__ __forceinline__ void scan_counts(uint32_t* cnt, uint32_t* warp_tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t v[8], sum = 0u;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = cnt[at_count(threadIdx.x >> 2, (threadIdx.x & 3) * 8 + k)];
    sum += v[k];
  }
  uint32_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  uint32_t base = lane < warp ? warp_tot[lane] : 0u;
  base = __reduce_add_sync(0xffffffffu, base);
  uint32_t run = base + inc - sum;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    cnt[at_count(threadIdx.x >> 2, (threadIdx.x & 3) * 8 + k)] = run;
    run += v[k];
  }
  __syncthreads();
}

// One CTA: (ids, positions) of n <= SORT_MAX tokens sorted by id, stable, eight bits a pass.  Warp w owns a
// contiguous part of the sequence, so ranks within a warp, then warps in order, keep equal ids in order.  Ids out
// of range sort last, as V.
__device__ void sort_one_cta(const int32_t* tokens, int n, int V, int passes, int32_t* ids, int32_t* pos,
                             int* status, unsigned char* sm) {
  uint32_t* key[2] = {reinterpret_cast<uint32_t*>(sm), reinterpret_cast<uint32_t*>(sm) + SORT_MAX};
  uint16_t* at[2] = {reinterpret_cast<uint16_t*>(sm + (size_t)SORT_MAX * 8),
                     reinterpret_cast<uint16_t*>(sm + (size_t)SORT_MAX * 8) + SORT_MAX};
  uint32_t* cnt = reinterpret_cast<uint32_t*>(sm + (size_t)SORT_MAX * 12);  // [256][SORT_WARPS]
  __shared__ uint32_t warp_tot[SORT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < n; i += SORT_THREADS) {
    const int tok = tokens[i];
    const bool ok = tok >= 0 && tok < V;
    if (!ok) atomicExch(status, kBadTokenCode);
    key[0][i] = ok ? (uint32_t)tok : (uint32_t)V;
    at[0][i] = (uint16_t)i;
  }
  const int part = ((n + SORT_THREADS - 1) / SORT_THREADS) * 32;  // tokens per warp, a multiple of 32
  const int i0 = min(n, warp * part), i1 = min(n, i0 + part);
  for (int p = 0; p < passes; ++p) {
    const uint32_t* ks = key[p & 1];
    const uint16_t* as = at[p & 1];
    uint32_t* kd = key[(p & 1) ^ 1];
    uint16_t* ad = at[(p & 1) ^ 1];
    for (int i = threadIdx.x; i < 256 * SORT_WARPS; i += SORT_THREADS) cnt[i] = 0u;
    __syncthreads();
    // lanes with the same digit: the lowest of them counts for all
    for (int b = i0; b < i1; b += 32) {
      const int i = b + lane;
      const uint32_t dg = i < i1 ? (ks[i] >> (8 * p)) & 255u : 256u;
      const uint32_t same = __match_any_sync(0xffffffffu, dg);
      if (dg < 256u && lane == __ffs(same) - 1) cnt[at_count(dg, warp)] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    scan_counts(cnt, warp_tot);
    for (int b = i0; b < i1; b += 32) {
      const int i = b + lane;
      const bool in = i < i1;
      const uint32_t k = in ? ks[i] : 0u, dg = in ? (k >> (8 * p)) & 255u : 256u;
      const uint32_t same = __match_any_sync(0xffffffffu, dg);
      const uint32_t first = in ? cnt[at_count(dg, warp)] : 0u;
      __syncwarp();
      if (in) {
        const uint32_t dst = first + __popc(same & ((1u << lane) - 1u));
        kd[dst] = k;
        ad[dst] = as[i];
        if (lane == __ffs(same) - 1) cnt[at_count(dg, warp)] = first + __popc(same);
      }
      __syncwarp();
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n; i += SORT_THREADS) {
    ids[i] = (int32_t)key[passes & 1][i];
    pos[i] = (int32_t)at[passes & 1][i];
  }
}

struct SortFillArgs {
  const int32_t* tokens;
  int n, V, d, passes;
  int sort;         // 1: CTA 0 sorts (n <= SORT_MAX)
  int32_t* ids;     // [n] sorted
  int32_t* pos;     // [n] their positions
  unsigned* done;   // [windows] counters of the sums, zeroed here
  int windows;
  float* dE;        // dense gradient whose untouched rows are written zero, or NULL
  float* ds_row;    // likewise
  int* status;
};

// CTA 0 sorts; the others zero the rows of the dense gradient that no token of the batch touches (every CTA
// reads all tokens and marks its own rows).
__global__ void __launch_bounds__(SORT_THREADS, 1) sort_fill_kernel(SortFillArgs a) {
  extern __shared__ __align__(16) unsigned char sm[];
  pdl_launch_dependents();
  pdl_wait();
  if (a.sort && blockIdx.x == 0) {
    for (int i = threadIdx.x; i < a.windows; i += SORT_THREADS) a.done[i] = 0u;
    sort_one_cta(a.tokens, a.n, a.V, a.passes, a.ids, a.pos, a.status, sm);
    return;
  }
  const int b = blockIdx.x - a.sort, nb = gridDim.x - a.sort;
  const int v0 = (int)((long long)a.V * b / nb), v1 = (int)((long long)a.V * (b + 1) / nb);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int MARKS = 8192;  // rows marked at a time
  for (int r0 = v0; r0 < v1; r0 += MARKS) {
    const int nr = min(MARKS, v1 - r0);
    __syncthreads();
    for (int i = threadIdx.x; i < nr; i += SORT_THREADS) sm[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < a.n; i += SORT_THREADS) {
      const uint32_t r = (uint32_t)(ld_s32(a.tokens + i) - r0);
      if (r < (uint32_t)nr) sm[r] = 1;
    }
    __syncthreads();
    for (int r = warp; r < nr; r += SORT_WARPS) {
      if (sm[r]) continue;
      if (a.dE) {
        float* row = a.dE + (size_t)(r0 + r) * a.d;
        for (int i = lane * 4; i < a.d; i += 128) st_f4(row + i, make_float4(0.f, 0.f, 0.f, 0.f));
      }
      if (a.ds_row && lane == 0) a.ds_row[r0 + r] = 0.0f;
    }
  }
}

// Device-wide radix pass for more tokens: counts per tile, their scan, the stable scatter.  A tile is 4096 keys,
// 32 warps of 128.
constexpr int TILE = 4096, TILE_PART = TILE / SORT_WARPS;
struct RadixArgs {
  const int32_t* ids_in;   // pass 0: the tokens
  const int32_t* pos_in;   // pass 0: NULL
  int32_t* ids_out;
  int32_t* pos_out;
  uint32_t* cnt;           // [256][tiles]
  int n, V, tiles, shift;
  unsigned* done;          // [windows] counters of the sums, zeroed with pass 0
  int windows;
  int* status;
};
__device__ __forceinline__ uint32_t radix_key(const RadixArgs& a, int i) {
  const int k = a.ids_in[i];
  if (a.pos_in) return (uint32_t)k;
  return k >= 0 && k < a.V ? (uint32_t)k : (uint32_t)a.V;
}
__global__ void __launch_bounds__(SORT_THREADS) radix_count_kernel(RadixArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ uint32_t h[256];
  if (!a.pos_in)
    for (int i = blockIdx.x * SORT_THREADS + threadIdx.x; i < a.windows; i += gridDim.x * SORT_THREADS) a.done[i] = 0u;
  if (threadIdx.x < 256) h[threadIdx.x] = 0u;
  __syncthreads();
  for (int k = 0; k < TILE / SORT_THREADS; ++k) {
    const long long i = (long long)blockIdx.x * TILE + k * SORT_THREADS + threadIdx.x;
    if (i < a.n) {
      const uint32_t key = radix_key(a, (int)i);
      if (!a.pos_in && key == (uint32_t)a.V) atomicExch(a.status, kBadTokenCode);
      atomicAdd(&h[(key >> a.shift) & 255u], 1u);
    }
  }
  __syncthreads();
  if (threadIdx.x < 256) a.cnt[(size_t)threadIdx.x * a.tiles + blockIdx.x] = h[threadIdx.x];
}
// Exclusive scan of m counts in place, one CTA.
__global__ void __launch_bounds__(SORT_THREADS) radix_scan_kernel(uint32_t* cnt, long long m) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ uint32_t warp_tot[SORT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t carry = 0u;
  for (long long b = 0; b < m; b += SORT_THREADS) {
    const long long i = b + threadIdx.x;
    const uint32_t v = i < m ? cnt[i] : 0u;
    uint32_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    const uint32_t mine = warp_tot[lane];
    const uint32_t base = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0u);
    const uint32_t total = __reduce_add_sync(0xffffffffu, mine);
    if (i < m) cnt[i] = carry + base + inc - v;
    carry += total;
    __syncthreads();
  }
}
__global__ void __launch_bounds__(SORT_THREADS) radix_scatter_kernel(RadixArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ uint32_t cnt[256 * SORT_WARPS];
  __shared__ uint32_t warp_tot[SORT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < 256 * SORT_WARPS; i += SORT_THREADS) cnt[i] = 0u;
  __syncthreads();
  const long long w0 = (long long)blockIdx.x * TILE + warp * TILE_PART;
  uint32_t key[TILE_PART / 32], rank[TILE_PART / 32];
#pragma unroll
  for (int k = 0; k < TILE_PART / 32; ++k) {
    const long long i = w0 + 32 * k + lane;
    const bool in = i < a.n;
    key[k] = in ? radix_key(a, (int)i) : 0u;
    const uint32_t dg = in ? (key[k] >> a.shift) & 255u : 256u;
    const uint32_t same = __match_any_sync(0xffffffffu, dg);
    const uint32_t before = in ? cnt[at_count(dg, warp)] : 0u;
    __syncwarp();
    rank[k] = before + __popc(same & ((1u << lane) - 1u));
    if (in && lane == __ffs(same) - 1) cnt[at_count(dg, warp)] = before + __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // digit dg of warp w starts after the tile's earlier warps; the tile's own digits start at the global counts
  scan_counts(cnt, warp_tot);
#pragma unroll
  for (int k = 0; k < TILE_PART / 32; ++k) {
    const long long i = w0 + 32 * k + lane;
    if (i >= a.n) continue;
    const uint32_t dg = (key[k] >> a.shift) & 255u;
    const uint32_t in_tile = cnt[at_count(dg, warp)] - cnt[at_count(dg, 0)];
    const uint32_t dst = a.cnt[(size_t)dg * a.tiles + blockIdx.x] + in_tile + rank[k];
    a.ids_out[dst] = (int32_t)key[k];
    a.pos_out[dst] = a.pos_in ? a.pos_in[i] : (int32_t)i;
  }
}

// ------------------------------------------------------------------------------------ sums

struct SumArgs {
  const int32_t* ids;
  const int32_t* pos;
  const int8_t* W;      // for ds_row
  const void* dh;
  int64_t lddh;
  float* dE;            // or NULL
  float* ds_row;        // or NULL
  float* part;          // [windows][2][d] sums of the runs that cross a window's start (0) or only its end (1)
  float* dpart;         // [windows][2] their products with W's row
  unsigned* done;       // [windows] CTAs finished of the run that starts in the window and leaves it
  int n, V, d, window, accumulate;
};
constexpr int MAX_WINDOW = 64;

// Adds the partial sums of run v over windows w0 .. w1 in order (whole CTA).
template <int CH>
__device__ __forceinline__ void join_run(const SumArgs& a, int v, long long w0, long long w1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (a.ds_row && warp == 0) {
    float s = 0.0f;
    for (long long x = w0 + 1 + lane; x <= w1; x += 32) s += __ldcg(a.dpart + (size_t)x * 2);
    s = warp_sum(s);
    if (lane == 0) {
      s += __ldcg(a.dpart + (size_t)w0 * 2 + 1);
      a.ds_row[v] = a.accumulate ? a.ds_row[v] + s : s;
    }
  }
  if (!a.dE) return;
  constexpr int U = 4;  // partial rows in flight
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (threadIdx.x + 256 * c) * 8;
    if (i >= a.d) continue;
    const auto load = [&](size_t slot, float (&p)[8]) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part + slot * a.d + i));
      const float4 y = __ldcg(reinterpret_cast<const float4*>(a.part + slot * a.d + i) + 1);
      p[0] = x.x, p[1] = x.y, p[2] = x.z, p[3] = x.w;
      p[4] = y.x, p[5] = y.y, p[6] = y.z, p[7] = y.w;
    };
    float acc[8];
    load((size_t)w0 * 2 + 1, acc);
    for (long long x0 = w0 + 1; x0 <= w1; x0 += U) {
      float p[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (x0 + u <= w1) load((size_t)(x0 + u) * 2, p[u]);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (x0 + u <= w1) {
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] += p[u][j];
        }
    }
    float* e = a.dE + (size_t)v * a.d + i;
    if (a.accumulate) {
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += e[j];
    }
    store8<float>(e, acc);
  }
}

// A window of sorted positions: rows added in order, run by run.  A run is final when both its ends lie in the
// window; of a longer one the last CTA to finish joins the partial sums.
template <typename T, int CH>
__global__ void __launch_bounds__(256, CH == 1 ? 4 : CH == 2 ? 3 : 2) window_kernel(SumArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int32_t id[MAX_WINDOW + 2], ps[MAX_WINDOW];
  __shared__ float dots[MAX_WINDOW][8];
  __shared__ long long from, to;  // windows of the first run (where it starts) and of the last (where it ends)
  __shared__ int last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k0 = blockIdx.x * a.window, nk = min(a.window, a.n - k0);
  // id[0] and id[nk + 1]: the neighbours outside (-1 where there is none)
  for (int i = threadIdx.x; i < nk + 2; i += 256) {
    const int k = k0 + i - 1;
    id[i] = k >= 0 && k < a.n ? a.ids[k] : -1;
    if (i >= 1 && i <= nk) ps[i - 1] = a.pos[k];
  }
  __syncthreads();
  constexpr int U = CH == 1 ? 4 : CH == 2 ? 2 : 1;  // rows in flight
  float acc[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[c][j] = 0.0f;
  int start = 0;
  for (int r0 = 0; r0 < nk; r0 += U) {
    float x[U][CH][8];
    uint2 wr[U][CH];  // the rows of W where runs end, requested with the gradient's
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (threadIdx.x + 256 * c) * 8, r = r0 + u;
        wr[u][c] = make_uint2(0u, 0u);
        if (r < nk && i < a.d) {
          const int v = id[r + 1];
          if (a.ds_row && v < a.V && !(r + 1 < nk && id[r + 2] == v))
            wr[u][c] = __ldg(reinterpret_cast<const uint2*>(a.W + (size_t)v * a.d + i));
          load8<T>(reinterpret_cast<const T*>(a.dh) + (int64_t)ps[r0 + u] * a.lddh + i, x[u][c]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[u][c][j] = 0.0f;
        }
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u;
      if (r >= nk) break;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[c][j] += x[u][c][j];
      const int v = id[r + 1];
      if (r + 1 < nk && id[r + 2] == v) continue;  // the run goes on
      const bool before = start == 0 && id[0] == v, after = r + 1 == nk && id[nk + 1] == v;
      const bool whole = !before && !after;
      if (v < a.V) {
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int i = (threadIdx.x + 256 * c) * 8;
          if (i >= a.d) continue;
          if (a.ds_row) {
            const uint2 w = wr[u][c];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              dot = fmaf((float)(int8_t)(w.x >> (8 * j)), acc[c][j], dot);
              dot = fmaf((float)(int8_t)(w.y >> (8 * j)), acc[c][j + 4], dot);
            }
          }
          if (!whole) {
            store8<float>(a.part + ((size_t)blockIdx.x * 2 + (before ? 0 : 1)) * a.d + i, acc[c]);
          } else if (a.dE) {
            float* e = a.dE + (size_t)v * a.d + i;
            if (a.accumulate) {
              const float4 p = *reinterpret_cast<const float4*>(e), q = *reinterpret_cast<const float4*>(e + 4);
              acc[c][0] += p.x, acc[c][1] += p.y, acc[c][2] += p.z, acc[c][3] += p.w;
              acc[c][4] += q.x, acc[c][5] += q.y, acc[c][6] += q.z, acc[c][7] += q.w;
            }
            store8<float>(e, acc[c]);
          }
        }
        if (a.ds_row) {
          dot = warp_sum(dot);
          if (lane == 0) dots[r][warp] = dot;
        }
      }
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[c][j] = 0.0f;
      start = r + 1;
    }
  }
  __syncthreads();
  const int r = threadIdx.x;
  if (a.ds_row && r < nk) {
    const int v = id[r + 1];
    if (v < a.V && !(r + 1 < nk && id[r + 2] == v)) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += dots[r][w];
      int s0 = r;  // the run's first row in the window
      while (s0 > 0 && id[s0] == v) --s0;
      const bool before = s0 == 0 && id[0] == v, after = r + 1 == nk && id[nk + 1] == v;
      if (before || after) a.dpart[(size_t)blockIdx.x * 2 + (before ? 0 : 1)] = s;
      else a.ds_row[v] = a.accumulate ? a.ds_row[v] + s : s;
    }
  }
  // runs that cross the window's ends
  const bool lead = id[1] < a.V && id[0] == id[1], tail = id[nk] < a.V && id[nk + 1] == id[nk];
  if (!lead && !tail) return;
  const bool one = lead && tail && id[1] == id[nk];  // the window lies within one run
  const long long w = blockIdx.x;
  // windows the runs extend over, 32 boundaries between windows at a time: the one before window x lies within the run
  // if the ids on both sides are v
  if (warp == 0) {
    long long x = w;
    if (lead) {
      x = w - 1;
      while (true) {
        const long long k = (x - lane) * a.window;
        const bool in = k > 0 && a.ids[k - 1] == id[1] && a.ids[k] == id[1];
        const uint32_t out = ~__ballot_sync(0xffffffffu, in);
        x -= out ? __ffs(out) - 1 : 32;
        if (out) break;
      }
    }
    if (lane == 0) from = x;
  } else if (warp == 1) {
    long long x = w;
    if (tail) {
      while (true) {
        const long long k = (x + 1 + lane) * a.window;
        const bool in = k < a.n && a.ids[k - 1] == id[nk] && a.ids[k] == id[nk];
        const uint32_t out = ~__ballot_sync(0xffffffffu, in);
        x += out ? __ffs(out) - 1 : 32;
        if (out) break;
      }
    }
    if (lane == 0) to = x;
  }
#pragma unroll
  for (int side = 0; side < 2; ++side) {  // the first run, then the last
    if (side == 0 ? !lead : !tail || one) continue;
    __syncthreads();  // the partial sums are written, `from` and `to` set
    const long long w0 = side == 0 ? from : w, w1 = side == 0 && !one ? w : to;
    if (threadIdx.x == 0) {
      __threadfence();
      last = atomicAdd(a.done + w0, 1u) == (unsigned)(w1 - w0);
      __threadfence();
    }
    __syncthreads();
    if (last) join_run<CH>(a, side == 0 ? id[1] : id[nk], w0, w1);
  }
}

template <typename T>
cudaError_t launch_window(const SumArgs& a, int windows, cudaStream_t st) {
  if (a.d <= 2048) return launch_pdl(window_kernel<T, 1>, dim3(windows), dim3(256), 0, st, a);
  if (a.d <= 4096) return launch_pdl(window_kernel<T, 2>, dim3(windows), dim3(256), 0, st, a);
  return launch_pdl(window_kernel<T, 4>, dim3(windows), dim3(256), 0, st, a);
}

// Rows per window: about four CTAs per SM, within [4, 64].
int window_rows(int n) {
  const int r = (n + 4 * 148 - 1) / (4 * 148);
  return r < 4 ? 4 : r > MAX_WINDOW ? MAX_WINDOW : r;
}

struct BackwardWs {
  size_t ids, pos, ids2, pos2, cnt, done, part, dpart, total;
};
BackwardWs backward_ws(int n, int d) {
  const size_t list = al256(sizeof(int32_t) * (size_t)n);
  const size_t windows = ((size_t)n + window_rows(n) - 1) / window_rows(n);
  const bool big = n > SORT_MAX;
  BackwardWs w;
  w.ids = kStatusBytes;
  w.pos = w.ids + list;
  w.ids2 = w.pos + list;
  w.pos2 = w.ids2 + (big ? list : 0);
  w.cnt = w.pos2 + (big ? list : 0);
  w.done = w.cnt + (big ? al256(sizeof(uint32_t) * 256 * (((size_t)n + TILE - 1) / TILE)) : 0);
  w.part = w.done + al256(sizeof(unsigned) * windows);
  w.dpart = w.part + al256(sizeof(float) * 2 * windows * (size_t)d);
  w.total = w.dpart + al256(sizeof(float) * 2 * windows);
  return w;
}

}  // namespace

size_t embed_backward_workspace_bytes(int n, int d, int /*V*/) { return backward_ws(n, d).total; }

}  // namespace dfssm

extern "C" int dfssm_embed_tokens(const int8_t* W, const float* s_row, int V, int d, const int32_t* tokens, int n,
                                  void* h, int h_type, int64_t ldh, void* workspace, size_t ws_bytes,
                                  void* stream) {
  using namespace dfssm;
  int st = check_int8_matrix(W, V, d);
  if (st) return st;
  if (!s_row) return DFSSM_EINVAL;
  st = check_tokens(n);
  if (st) return st;
  if (n == 0) return DFSSM_OK;
  st = check_rows(h, h_type, ldh, d);
  if (st) return st;
  if (!tokens) return DFSSM_EINVAL;
  if (!al(s_row, 4) || !al(tokens, 4)) return DFSSM_EALIGN;
  if (!workspace || !al(workspace, 256) || ws_bytes < kStatusBytes) return DFSSM_EWORKSPACE;
  if (!device_ok()) return DFSSM_EDEVICE;
  const EmbedTokensArgs a{W, s_row, tokens, h, ldh, static_cast<int*>(workspace), V, d, n};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = h_type == DFSSM_F32 ? launch_embed_tokens<float>(a, s) : launch_embed_tokens<__nv_bfloat16>(a, s);
  return e == cudaSuccess ? DFSSM_OK : record_cuda_failure(e);
}

extern "C" int dfssm_embed_tokens_backward(const int8_t* W, int V, int d, const int32_t* tokens, int n,
                                           const void* dh, int dh_type, int64_t lddh, float* dE, float* ds_row,
                                           int accumulate, void* workspace, size_t ws_bytes, void* stream) {
  using namespace dfssm;
  int st = check_int8_matrix(W, V, d);
  if (st) return st;
  if (!dE && !ds_row) return DFSSM_EINVAL;
  st = check_tokens(n);
  if (st) return st;
  if (!al(dE, 16) || !al(ds_row, 4)) return DFSSM_EALIGN;
  if (n > 0) {
    st = check_rows(dh, dh_type, lddh, d);
    if (st) return st;
    if (!tokens) return DFSSM_EINVAL;
    if (!al(tokens, 4)) return DFSSM_EALIGN;
    if (!workspace || !al(workspace, 256) || ws_bytes < backward_ws(n, d).total) return DFSSM_EWORKSPACE;
  } else if (accumulate) {
    return DFSSM_OK;
  }
  if (!device_ok()) return DFSSM_EDEVICE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(workspace);
  int passes = 1;  // ids 0 .. V
  while (passes < 4 && ((unsigned)V >> (8 * passes))) ++passes;
  SortFillArgs f{};
  f.tokens = tokens;
  f.n = n;
  f.V = V;
  f.d = d;
  f.passes = passes;
  f.sort = n > 0 && n <= SORT_MAX ? 1 : 0;
  f.dE = dE;
  f.ds_row = ds_row;
  cudaError_t e = cudaSuccess;
  BackwardWs w{};
  if (n > 0) {
    w = backward_ws(n, d);
    f.ids = reinterpret_cast<int32_t*>(base + w.ids);
    f.pos = reinterpret_cast<int32_t*>(base + w.pos);
    f.done = reinterpret_cast<unsigned*>(base + w.done);
    f.windows = (int)(((long long)n + window_rows(n) - 1) / window_rows(n));
    f.status = reinterpret_cast<int*>(base);
  }
  if (f.sort || !accumulate) {
    const int fill = accumulate ? 0 : num_sms() - f.sort;
    e = set_max_dynamic_smem(reinterpret_cast<const void*>(sort_fill_kernel), (int)SORT_SMEM);
    if (e == cudaSuccess)
      e = launch_pdl(sort_fill_kernel, dim3(fill + f.sort), dim3(SORT_THREADS), SORT_SMEM, s, f);
    if (e != cudaSuccess) return record_cuda_failure(e);
  }
  if (n == 0) return DFSSM_OK;
  const int32_t* ids = f.ids;
  const int32_t* pos = f.pos;
  if (!f.sort) {
    int32_t* buf[2][2] = {{f.ids, f.pos},
                          {reinterpret_cast<int32_t*>(base + w.ids2), reinterpret_cast<int32_t*>(base + w.pos2)}};
    RadixArgs r{};
    r.ids_in = tokens;
    r.cnt = reinterpret_cast<uint32_t*>(base + w.cnt);
    r.n = n;
    r.V = V;
    r.tiles = (n + TILE - 1) / TILE;
    r.done = f.done;
    r.windows = f.windows;
    r.status = f.status;
    for (int p = 0; p < passes; ++p) {
      r.ids_out = buf[p & 1][0];
      r.pos_out = buf[p & 1][1];
      r.shift = 8 * p;
      e = launch_pdl(radix_count_kernel, dim3(r.tiles), dim3(SORT_THREADS), 0, s, r);
      if (e == cudaSuccess)
        e = launch_pdl(radix_scan_kernel, dim3(1), dim3(SORT_THREADS), 0, s, r.cnt, (long long)256 * r.tiles);
      if (e == cudaSuccess) e = launch_pdl(radix_scatter_kernel, dim3(r.tiles), dim3(SORT_THREADS), 0, s, r);
      if (e != cudaSuccess) return record_cuda_failure(e);
      ids = r.ids_in = r.ids_out;
      pos = r.pos_in = r.pos_out;
    }
  }
  SumArgs a{};
  a.ids = ids;
  a.pos = pos;
  a.W = W;
  a.dh = dh;
  a.lddh = lddh;
  a.dE = dE;
  a.ds_row = ds_row;
  a.part = reinterpret_cast<float*>(base + w.part);
  a.dpart = reinterpret_cast<float*>(base + w.dpart);
  a.n = n;
  a.V = V;
  a.d = d;
  a.window = window_rows(n);
  a.accumulate = accumulate;
  a.done = f.done;
  e = dh_type == DFSSM_BF16 ? launch_window<__nv_bfloat16>(a, f.windows, s) : launch_window<float>(a, f.windows, s);
  return e == cudaSuccess ? DFSSM_OK : record_cuda_failure(e);
}
