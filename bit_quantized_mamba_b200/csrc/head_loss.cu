// Softmax cross entropy of int8-head logits over the vocabulary, without keeping the logits, and its
// gradient (include/dfssm.h, dfssm_head_loss and dfssm_head_loss_backward).
//
// With l_v = acc_v s s_row_v the logits of a token (acc the exact int32 product of the int8 codes, as in the LM
// head), y its label, and the other rows' m = max_{v != y} l_v, S = sum_{v != y} exp(l_v - m):
//   z = m + log S - l_y,   loss = log(1 + exp z),   1 - p_y = 1 / (1 + exp(-z)),   p_v = exp(l_v - m) (1 - p_y) / S
// The label is kept out of m and S, so neither a loss near zero nor 1 - p_y is a difference of nearly equal
// numbers.
//
// Forward: the int8 product with tokens on the tensor memory's lanes and rows of W on its columns; a thread
// owns a token's logits of a tile and folds them into a running (max, sum), one pass, 8 bytes kept per
// token, tile and column half; a second kernel joins them.  (Up to 16 tokens: operands exchanged, one kernel.)
//
// Gradient with respect to the (dequantised) normalised token:  du = g [sum_{v != y} p_v s_row_v W_v -
// (1 - p_y) s_row_y W_y].  The coefficients c_v = exp(l_v - m) s_row_v / max|s_row| lie in [0, 1] (or [-1, 1] with
// negative scales) whatever the token.  They are written in fixed point, in steps of 2^-24 tau with
// tau = 2^-k ~ min(1, S / 32): below tau a coefficient is three base-256 digits, and at most 32 of a token's can
// be above it (they sum to at most S), whose further bits go into a list.  (A few rows whose scales are far above the
// others' are left out of the maximum; see scale_top().)  The sum over v is then three exact
// int8 products of digits with W, each at twice the rate of a bf16 product, free of bf16's rounding and of any
// order of summation, and a few listed rows of W.  Two kernels first quantize the tokens, look over the row scales and work
// out the tokens' factors; then the vocabulary is taken in pieces whose digits stay in L2:
//   1. the first product again, its epilogue turning logits into digits (and the row scales' gradient
//      into partial column sums);
//   2. the second product: digits x W, whose rows are its K dimension as they lie in memory ("MN-major" operand;
//      a transposed copy cost 40 us at 2048 tokens, 50288 rows), added to int32 accumulators in memory by
//      integer atomics (any order gives the same sum): rounds of whole (tile, digit) units, one per CTA pair, and
//      what is left split evenly along K.
//      Its epilogue's warps meanwhile take the column sums of W and join those of the row scales' gradient.
// At the end one kernel joins the digits, the listed rows and the label's row and applies the norm's backward.
// The digits are stored as signed bytes (digit - 128); the column sums of W give the 128s back.
//
// 2048 tokens x 50288 rows x 2048: loss 166 us (2530 TOPS), loss and gradients 886 us (2380 TOPS of five products).
// Bound by power: with operands that do not change the products alone run at 3270 TOPS under the same cap.  What the
// gradient takes beyond its products is the digits' epilogue (205 us for a product that alone takes 150).
// Measured and dropped: the digits of a piece in one kernel with the second product of the piece before, tiles of both in
// turn (1026 us where it took 962 apart); digits balanced around zero, which need no column sums but take a bit off the
// range (no gain); in the digits' epilogue the next columns fetched ahead, wider loads of the scales, the next
// tile's token data fetched into L1 (no gain each).

#include "gemm_i8.cuh"
#include "rows.cuh"

namespace dfssm {
namespace {

using namespace gemm_i8;

constexpr double kLog2e = 1.4426950408889634074;
constexpr double kLn2 = 0.69314718055994530942;
constexpr int kMaxRangeCtas = 160;  // workspaces are sized without asking the device:
constexpr int kSms = 148;           // the streaming multiprocessors of a B200

inline size_t al256(size_t x) { return (x + 255) & ~size_t(255); }
inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Row scale in units of log 2: the logits' base-2 exponents are then acc s scale2, and the one rounding that
// log2 e brings differs from row to row (in the token's scale it would be one factor on all its logits: losses
// 4.0e-8 off instead of 3.4e-8).
__device__ __forceinline__ float scale2(float s_row) { return __double2float_rn((double)s_row * kLog2e); }

// v[j] of an array in registers, N a power of two.
template <int N>
__device__ __forceinline__ uint32_t pick(const uint32_t (&v)[N], int j) {
  uint32_t x[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) x[i] = (j & (N / 2)) ? v[i + N / 2] : v[i];
#pragma unroll
  for (int n = N / 4; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = (j & n) ? x[i + n] : x[i];
  return x[0];
}

// ------------------------------------------------------------------------------------ forward

template <int CG_>
struct ForwardPolicy {
  static constexpr int CG = CG_;
  static constexpr bool W_EARLY = true, W_IS_A = false, A_MN = false, RESIDENT = false;
  static constexpr int EPI_WARPS = 8, EPI_COLS = BN_MAX / 2;  // columns of an epilogue warp
  struct Args {
    CUtensorMap map_a, map_b;  // codes, W
    RowArgs r;
    Common c;
    const double* s_tok;    // [M]
    const float* s_row;     // [V]
    const int32_t* labels;  // [M]
    int* label_acc;         // [M] the label's accumulator, in stats[2] until write_loss() takes it
    float2* part;           // [slots][M] (max, sum) in units of log 2
    int M, V;
  };
  static __device__ __forceinline__ bool tile(const Args& a, int j, Tile& t) { return row_tile<CG, false>(a.r, j, t); }
  static __device__ __forceinline__ uint32_t bytes(const Args& a, const Tile& t) { return row_bytes<CG>(a.r, t); }
  static __device__ __forceinline__ Boxes boxes_a(const Args& a, const Tile& t, int) {
    return row_boxes_a<CG>(a.r, &a.map_a, t);
  }
  static __device__ __forceinline__ Boxes boxes_b(const Args& a, const Tile& t, int rank) {
    return row_boxes_b<CG>(a.r, &a.map_b, t, rank);
  }
  static __device__ __forceinline__ uint64_t adesc(uint32_t addr) { return umma_desc_k_sw128(addr); }
  static __device__ __forceinline__ uint64_t bdesc(const Args&, uint32_t addr) { return umma_desc_k_sw128(addr); }
  static __device__ __forceinline__ uint64_t a_step() { return UMMA_K >> 4; }
  static __device__ __forceinline__ uint64_t b_step(const Args&) { return UMMA_K >> 4; }
  static constexpr int EPI_SMEM = EPI_WARPS * EPI_COLS * 4;
  struct Epilogue {
    int half, lane, row;  // row: lane of the tile
    float* sr;            // row scales of this warp's columns (chunks of 32: half, half + 2, ..), in units of log 2
    int tok = -1;         // the token whose running (m, S) this thread holds
    int slot = 0;
    float m = -INFINITY, S = 0.0f;
    float st;             // the token's scale and label
    int label;
    __device__ __forceinline__ Epilogue(const Args&, unsigned char* sm, int q, int half_, int lane_)
        : half(half_), lane(lane_), row(q * 32 + lane_),
          sr(reinterpret_cast<float*>(sm) + (half_ * 4 + q) * EPI_COLS) {}
    __device__ __forceinline__ void flush(const Args& a) {
      if (tok >= 0 && tok < a.M) a.part[(size_t)slot * a.M + tok] = make_float2(m, S);
      m = -INFINITY;
      S = 0.0f;
    }
    __device__ __forceinline__ void write_b(const Args&, unsigned char*, int) {}
    __device__ __forceinline__ void prepare(const Args& a, const Tile& t) {
      const int tk = t.a0 + row;
      const int sl = (a.r.mode == kGrid ? t.b0 / a.r.tile_b : (int)blockIdx.x / CG) * 2 + half;
      if (tk != tok || sl != slot) {
        flush(a);
        tok = tk;
        slot = sl;
      }
      st = tk < a.M ? (float)a.s_tok[tk] : 0.0f;
      label = tk < a.M ? a.labels[tk] : -1;
#pragma unroll
      for (int k = 0; k < EPI_COLS / 32; ++k) {
        const int c = k * 64 + half * 32 + lane;
        sr[k * 32 + lane] = c < t.nb ? scale2(ld_f32(a.s_row + t.b0 + c)) : 0.0f;
      }
      __syncwarp();
    }
    __device__ __forceinline__ void tile(const Args& a, const Tile& t, uint32_t taddr) {
      uint32_t v[32];
      const float* w1 = sr;
      if (half * 32 < t.nb) tmem_ld32(taddr + (uint32_t)(half * 32), v);
#pragma unroll 1  // four copies of the body would not stay in the instruction cache
      for (int c = half * 32; c < t.nb; c += 64, w1 += 32) {
        tmem_wait(v);
        const int v0 = t.b0 + c;
        const float4* w4 = reinterpret_cast<const float4*>(w1);
        // columns that do not count: past the tile's end, and the token's own label
        uint32_t skip = c + 32 > t.nb ? 0xFFFFFFFFu << (t.nb - c) : 0u;
        const uint32_t lc = (uint32_t)(label - v0);
        if (lc < 32u) skip |= 1u << lc;
        f2 x[16];
        const f2 st2 = pack2(st, st);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = mul2(pack2((float)(int)v[2 * j], (float)(int)v[2 * j + 1]), st2);
        if (lc < 32u && c + (int)lc < t.nb) {
          a.label_acc[tok] = (int)pick(v, (int)lc);
        }
        if (c + 64 < t.nb) tmem_ld32(taddr + (uint32_t)c + 64, v);  // the next chunk, while this one is summed
        float mx = m;
        if (!__any_sync(0xffffffffu, skip != 0u)) {
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const float4 w = w4[j / 2];
            float l0, l1, l2, l3;
            unpack2(mul2(x[j], pack2(w.x, w.y)), l0, l1);
            unpack2(mul2(x[j + 1], pack2(w.z, w.w)), l2, l3);
            mx = fmaxf(mx, fmaxf(fmaxf(l0, l1), fmaxf(l2, l3)));
          }
          const f2 mx2 = pack2(-mx, -mx);
          f2 s = pack2(S * ex2(m - mx), 0.0f);
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const float4 w = w4[j / 2];
            float l0, l1, l2, l3;
            unpack2(fma2(x[j], pack2(w.x, w.y), mx2), l0, l1);
            unpack2(fma2(x[j + 1], pack2(w.z, w.w), mx2), l2, l3);
            s = add2(s, add2(pack2(ex2(l0), ex2(l1)), pack2(ex2(l2), ex2(l3))));
          }
          float s0, s1;
          unpack2(s, s0, s1);
          S = s0 + s1;
        } else {
          float xs[32];
#pragma unroll
          for (int j = 0; j < 16; ++j) unpack2(x[j], xs[2 * j], xs[2 * j + 1]);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!((skip >> j) & 1u)) mx = fmaxf(mx, xs[j] * w1[j]);
          const float mz = mx == -INFINITY ? 0.0f : mx;  // nothing counted yet
          float s = S * ex2(m - mz);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!((skip >> j) & 1u)) s += ex2(fmaf(xs[j], w1[j], -mz));
          S = s;
        }
        m = mx;
      }
      __syncwarp();  // the scales are read: the next tile's may be written
    }
    __device__ __forceinline__ void finish(const Args& a) { flush(a); }
  };
};

// Loss and stats of token t from the other rows' (max, sum), its label y, and the scales of the token and of the label's
// row; stats[2][t] holds the label's accumulator, and 1 - p_y afterwards.  z is a difference of logits and wants fp64 (the
// label's logit too: rounded, it would be most of the error of a confident token's loss); exp z, with what fp32 leaves
// of z as a factor, and what follows keep fp32's relative precision without.
__device__ __forceinline__ void write_loss(int t, float m, double S, int y, double s, float s_label, int M, int V, float* stats,
                                           float* loss, int* status) {
  const bool bad = y >= V;
  if (bad) atomicExch(status, kBadTokenCode);
  float out = 0.0f, rest = 0.0f;
  if (y >= 0 && !bad) {
    const double l = dmul(dmul(int_to_f64(__ldcg(reinterpret_cast<const int*>(stats) + 2 * (size_t)M + t)), s), (double)s_label);
    if (S != 0.0) {
      const double z = ((double)m + log2(S)) * kLn2 - l;
      const float a = (float)fabs(z), e0 = expf(-a);
      const float e = a < 104.0f ? fmaf(e0, (float)((double)a - fabs(z)), e0) : e0;  // below 1; from there on 0
      rest = z > 0.0 ? 1.0f / (1.0f + e) : e / (1.0f + e);
      out = z > 0.0 ? (float)(z + (double)log1pf(e)) : log1pf(e);
    } else if (l != l) {  // no other row, but the token is not finite
      rest = out = (float)l;
    }
  }
  stats[t] = m;
  stats[(size_t)M + t] = (float)S;
  stats[2 * (size_t)M + t] = rest;
  loss[t] = out;
}

// Joins the partial (max, sum) of a token and forms its loss.  32 tokens per CTA, 32 slices of slots.
constexpr int LF_SLICES = 32;
__global__ void __launch_bounds__(32 * LF_SLICES) loss_finish_kernel(const float2* part, int slots, int M, int V,
                                                                     const int32_t* labels, const double* s_tok,
                                                                     const float* s_row, float* stats, float* loss,
                                                                     int* status) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float2 sm[LF_SLICES][33];
  const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int t = blockIdx.x * 32 + lane, tok = blockIdx.x * 32 + sl;  // summed by this lane, joined by this warp
  const int y = tok < M ? labels[tok] : -1;
  const double s_t = tok < M ? s_tok[tok] : 0.0;
  float m = -INFINITY, S = 0.0f;
  constexpr int U = 8;  // slots in flight
  for (int s0 = sl; s0 < slots; s0 += U * LF_SLICES) {
    float2 p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u * LF_SLICES;
      p[u] = t < M && s < slots ? part[(size_t)s * M + t] : make_float2(-INFINITY, 0.0f);
    }
    float mx = m;
#pragma unroll
    for (int u = 0; u < U; ++u) mx = fmaxf(mx, p[u].x);
    const float mz = mx == -INFINITY ? 0.0f : mx;
    S *= ex2(m - mz);
#pragma unroll
    for (int u = 0; u < U; ++u) S += p[u].y * ex2(p[u].x - mz);  // an empty part is (-inf, 0); a NaN sum stays one
    m = mx;
  }
  const float s_label = y >= 0 && y < V ? ld_f32(s_row + y) : 0.0f;  // (its address waits for y: after the slots)
  sm[sl][lane] = make_float2(m, S);
  __syncthreads();
  // warp sl joins token sl: lane i holds slice i
  const float2 p = sm[lane][sl];
  const float mx = warp_max(p.x), mz = mx == -INFINITY ? 0.0f : mx;
  const double sum = warp_sum((double)(p.y * ex2(p.x - mz)));
  if (lane == 0 && tok < M) write_loss(tok, mx, sum, y, s_t, s_label, M, V, stats, loss, status);
}

// ------------------------------------------------------------------------------------ forward, few tokens

// Up to 16 tokens: rows of W on the lanes, tokens on the columns, so that W streams through a deep ring of narrow
// stages.  A thread of the four epilogue warps that sum (all sixteen quantize) keeps a running (max, sum) over its rows
// for every token, lanes and warps are joined at the end, and the last CTA to finish joins the CTAs and writes the losses.
// What it takes grows with every token, the other form's time hardly (rows of 2048 and of 1040 values, 50288 / 20011:
// 5 tokens 24.7 / 14.9 us here, 32.2 / 17.2 there; 16 tokens 29.1 / 18.7 and 31.9 / 17.7; 32 tokens 34.4 / 24.2 and
// 32.8 / 17.4; 64 tokens 45.7 / 34.1 and 27.3 / 17.4).
constexpr int SMALL_TOKENS = 16;
template <bool RESIDENT_>
struct SmallForwardPolicy {
  static constexpr int CG = 1;
  static constexpr bool RESIDENT = RESIDENT_;
  static constexpr bool W_EARLY = true, W_IS_A = true, A_MN = false;
  static constexpr int EPI_WARPS = 16;
  static_assert(EPI_WARPS == RES_WARPS, "the epilogue's warps quantize");
  struct Args {
    CUtensorMap map_a, map_b;  // W, codes
    RowArgs r;
    Common c;
    ResidentArgs x;         // RESIDENT: the tokens, else
    const double* s_tok;    // [M] their scales
    const float* s_row;     // [V]
    const int32_t* labels;  // [M]
    float* stats;           // [3][M]
    float* loss;            // [M]
    float2* part;           // [CTAs][M]
    unsigned* done;         // CTAs finished: zero before and after
    int M, V;
  };
  static __device__ __forceinline__ bool tile(const Args& a, int j, Tile& t) { return row_tile<CG, true, false>(a.r, j, t); }
  static __device__ __forceinline__ uint32_t bytes(const Args& a, const Tile& t) { return row_bytes<CG, RESIDENT>(a.r, t); }
  static __device__ __forceinline__ Boxes boxes_a(const Args& a, const Tile& t, int) {
    return row_boxes_a<CG>(a.r, &a.map_a, t);
  }
  static __device__ __forceinline__ Boxes boxes_b(const Args& a, const Tile& t, int rank) {
    return row_boxes_b<CG>(a.r, &a.map_b, t, rank);
  }
  static __device__ __forceinline__ uint64_t adesc(uint32_t addr) { return umma_desc_k_sw128(addr); }
  static __device__ __forceinline__ uint64_t bdesc(const Args&, uint32_t addr) { return umma_desc_k_sw128(addr); }
  static __device__ __forceinline__ uint64_t a_step() { return UMMA_K >> 4; }
  static __device__ __forceinline__ uint64_t b_step(const Args&) { return UMMA_K >> 4; }
  struct Scratch {
    ResidentScratch res;
    float s[SMALL_TOKENS];
    int label[SMALL_TOKENS];
    float s_label[SMALL_TOKENS];  // the label's row scale
    float2 red[4][SMALL_TOKENS];
    int last;
  };
  static constexpr int EPI_SMEM = (int)((sizeof(Scratch) + 15) & ~size_t(15));
  struct Epilogue {
    Scratch* sc;
    int q, part, lane;
    float sw;
    float m[SMALL_TOKENS], S[SMALL_TOKENS];
    __device__ __forceinline__ Epilogue(const Args& a, unsigned char* sm, int q_, int part_, int lane_)
        : sc(reinterpret_cast<Scratch*>(sm)), q(q_), part(part_), lane(lane_) {
#pragma unroll
      for (int j = 0; j < SMALL_TOKENS; ++j) {
        m[j] = -INFINITY;
        S[j] = 0.0f;
      }
      // the four quadrants write the same values, and each reads its own
      const int t = lane;
      if (part == 0 && t < SMALL_TOKENS) {
        sc->label[t] = t < a.M ? ld_s32(a.labels + t) : -1;
        if (!RESIDENT) sc->s[t] = t < a.M ? (float)a.s_tok[t] : 0.0f;
      }
      __syncwarp();
    }
    __device__ __forceinline__ void write_b(const Args& a, unsigned char* b, int warp) {
      if (!RESIDENT) return;
      if (a.x.x_type == DFSSM_BF16) resident_quantize<__nv_bfloat16>(a.x, b, &sc->res, warp, lane);
      else resident_quantize<float>(a.x, b, &sc->res, warp, lane);
    }
    __device__ __forceinline__ float scale(int t) const { return RESIDENT ? sc->res.s[t & (RES_TOKENS - 1)] : sc->s[t]; }
    __device__ __forceinline__ void prepare(const Args& a, const Tile& t) {
      const int r = q * 32 + lane;
      sw = r < t.na ? scale2(ld_f32(a.s_row + t.a0 + r)) : 0.0f;
    }
    __device__ __forceinline__ void tile(const Args& a, const Tile& t, uint32_t taddr) {
      const int r = q * 32 + lane, row = t.a0 + r;
      if (part > 0) return;
      uint32_t v[SMALL_TOKENS];
      tmem_ld16(taddr, v);
      tmem_wait(v);
      if (r >= t.na) return;
#pragma unroll
      for (int j = 0; j < SMALL_TOKENS; ++j) {
        if (j >= a.M) break;
        const float st = scale(j), x = (float)(int)v[j] * st;
        if (row == sc->label[j]) {  // the label's own logit stays out of the sum
          reinterpret_cast<int*>(a.stats)[2 * (size_t)a.M + j] = (int)v[j];
        } else {
          const float mx = fmaxf(m[j], x * sw), mz = mx == -INFINITY ? 0.0f : mx;
          S[j] = S[j] * ex2(m[j] - mz) + ex2(fmaf(x, sw, -mz));
          m[j] = mx;
        }
      }
    }
    __device__ __forceinline__ void finish(const Args& a) {
      if (part == 0) {
        const int y = lane < a.M ? sc->label[lane] : -1;  // (a.M <= SMALL_TOKENS)
        const float s_label = y >= 0 && y < a.V ? ld_f32(a.s_row + y) : 0.0f;
#pragma unroll
        for (int j = 0; j < SMALL_TOKENS; ++j) {
          if (RESIDENT && j >= a.M) break;  // (1 token: 27 -> 26 us; with more the branches cost 2 us)
          const float mx = warp_max(m[j]), mz = mx == -INFINITY ? 0.0f : mx;
          const float s = warp_sum(S[j] * ex2(m[j] - mz));
          if (lane == j) sc->red[q][j] = make_float2(mx, s);
        }
        if (lane < a.M) sc->s_label[lane] = s_label;
      }
      epilogue_sync();
      const int tid = threadIdx.x - 64;
      if (tid < a.M) {
        float mx = -INFINITY, s = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, sc->red[i][tid].x);
        const float mz = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
        for (int i = 0; i < 4; ++i) s += sc->red[i][tid].y * ex2(sc->red[i][tid].x - mz);
        a.part[(size_t)blockIdx.x * a.M + tid] = make_float2(mx, s);
      }
      epilogue_sync();
      if (tid == 0) {
        __threadfence();
        sc->last = atomicAdd(a.done, 1u) == gridDim.x - 1;
        __threadfence();
      }
      epilogue_sync();
      if (!sc->last) return;
      if (tid == 0) *a.done = 0u;
      for (int t = tid >> 5; t < a.M; t += EPI_WARPS) {
        float mx = -INFINITY;
        for (int i = lane; i < (int)gridDim.x; i += 32) mx = fmaxf(mx, __ldcg(&a.part[(size_t)i * a.M + t].x));
        mx = warp_max(mx);
        const float mz = mx == -INFINITY ? 0.0f : mx;
        double s = 0.0;
        for (int i = lane; i < (int)gridDim.x; i += 32) {
          const float2 p = __ldcg(a.part + (size_t)i * a.M + t);
          s += (double)(p.y * ex2(p.x - mz));
        }
        s = warp_sum(s);
        if (lane == 0)
          write_loss(t, mx, s, sc->label[t], (double)scale(t), sc->s_label[t], a.M, a.V, a.stats, a.loss, a.c.err);
      }
    }
  };
};

// ------------------------------------------------------------------------------------ gradient

// Coefficients of a token that may need more than 24 bits: the more there may be, the finer the steps (11 tokens x
// 30000 rows: dx off by 9.5e-7 with 16, 5.0e-7 with 32, 3.1e-7 with 64; 2048 x 50288 x 2048: 882, 889, 897 us).
constexpr int kListed = 32;

// Per-token factors of the gradient.
constexpr int kPrepareCtas = 128, kPrepareThreads = 512;
struct TokenFactors {
  float4* tok;    // [M] {m', s, f s, w_y s}: m' = m - k, f = g p_max 2^-k, w_y = -g (1 - p_y)
  int* shift;     // [M] k
  double2* fac;   // [M] {f, w_y}
  uint2* srow;    // [kScanParts] {bits of max |s_row|, any negative} of the rows' parts
};

// The scale that coefficients are counted in.  It is the largest, unless that is far above the others': one such row would
// cost every token its precision (steps 10000 times as wide, dx off by 5e-4), also those that give the row no weight.
// "Far above" is beyond 8 times T, the least but an eighth of the parts' maxima; then it is the largest of the
// maxima up to 8 T, and the rows beyond it are looked at token by token (outliers()).  The whole warp works it out, from
// 128 numbers.
constexpr int kLowParts = kScanParts / 8;
struct ScaleTop {
  float top, most;  // the scale, and the largest there is
  bool outliers;    // rows beyond the top
  bool neg;         // negative scales
};
__device__ __forceinline__ ScaleTop scale_top(const uint2* srow, int V) {
  constexpr int N = kScanParts / 32;
  const int lane = threadIdx.x & 31, run = scan_run(V), runs = (V + run - 1) / run;
  const int parts = runs < kScanParts ? runs : kScanParts, low = parts * kLowParts / kScanParts;
  uint32_t m[N], most = 0u, neg = 0u;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint2 r = srow[k * 32 + lane];
    m[k] = k * 32 + lane < parts ? r.x : 0xFFFFFFFFu;
    most = max(most, r.x);
    neg |= r.y;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  ScaleTop t{__uint_as_float(most), __uint_as_float(most), false, __reduce_or_sync(0xffffffffu, neg) != 0u};
  // more than `low` parts stay below x
  const auto many_below = [&](uint32_t x) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) n += __popc(__ballot_sync(0xffffffffu, m[k] < x));
    return n > low;
  };
  if (most < 0x7F800000u && many_below(__float_as_uint(t.top * 0.125f))) {
    uint32_t x = 0u;  // the largest number that few parts stay below: the (low + 1)-th of the maxima
    for (uint32_t bit = 1u << 30; bit > 0u; bit >>= 1)
      if (!many_below(x | bit)) x |= bit;
    const uint32_t bound = __float_as_uint(__uint_as_float(x) * 8.0f);
    uint32_t top = 0u;
#pragma unroll
    for (int k = 0; k < N; ++k) top = max(top, m[k] <= bound ? m[k] : 0u);
    top = __reduce_max_sync(0xffffffffu, top);
    if (__uint_as_float(top) > 1e-30f && top < most) {
      t.top = __uint_as_float(top);
      t.outliers = true;
    }
  }
  return t;
}

struct PrepareArgs {
  const float* stats;
  const int32_t* labels;
  const float* dloss;
  const int8_t* q;  // [M][d] codes
  const double* s_tok;
  const int8_t* W;
  const float* s_row;
  int M, V, d;
  TokenFactors out;
  uint4* zero;      // to be zeroed
  size_t zeros;     // 16 bytes each
};
// Up to kOutliers rows whose scale is beyond `top`, in order (whole CTA); their number, or -1 if there are more.
// (2048 tokens x 50288 rows x 2048, loss and gradients: 755 us without such rows, 787 with one, 902 with 64, 1077 with 256.)
constexpr int kOutliers = 1024;
__device__ __forceinline__ int find_outliers(const PrepareArgs& a, float top, int* rows) {
  __shared__ int cnt[kPrepareThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n = 0;
  for (int v0 = 0; v0 < a.V; v0 += kPrepareThreads) {
    const int v = v0 + threadIdx.x;
    const bool out = v < a.V && fabsf(ld_f32(a.s_row + v)) > top;
    if (!__syncthreads_or(out)) continue;
    const uint32_t b = __ballot_sync(0xffffffffu, out);
    if (lane == 0) cnt[warp] = __popc(b);
    __syncthreads();
    int at = n;
    for (int w = 0; w < kPrepareThreads / 32; ++w) {
      if (w == warp) at = n + __popc(b & ((1u << lane) - 1u));
      n += cnt[w];
    }
    if (out && at < kOutliers) rows[at] = v;
    __syncthreads();
  }
  return n <= kOutliers ? n : -1;
}
// The largest and the sum of a token's coefficients exp(l - m) |s_row| in the outlying rows but its label's (whole warp).
__device__ __forceinline__ void outliers(const PrepareArgs& a, const int* rows, int n, int t, int y, float m, float& most,
                                         float& sum) {
  const int lane = threadIdx.x & 31;
  const float s = (float)a.s_tok[t];
  most = sum = 0.0f;
  for (int i = 0; i < n; ++i) {
    const int v = rows[i];
    const uint4* w = reinterpret_cast<const uint4*>(a.W + (size_t)v * a.d);
    const uint4* q = reinterpret_cast<const uint4*>(a.q + (size_t)t * a.d);
    int acc = 0;
    for (int c = lane; c < a.d / 16; c += 32) {
      const uint4 x = ld_u32x4(w + c), z = ld_u32x4(q + c);
      acc = dp4a_ss(x.x, z.x, acc);
      acc = dp4a_ss(x.y, z.y, acc);
      acc = dp4a_ss(x.z, z.z, acc);
      acc = dp4a_ss(x.w, z.w, acc);
    }
    acc = __reduce_add_sync(0xffffffffu, acc);
    const float r = ld_f32(a.s_row + v), c = ex2(fmaf((float)acc * s, scale2(r), -m)) * fabsf(r);
    if (v != y) {
      most = fmaxf(most, c);
      sum += c;
    }
  }
}
// The tokens' factors, and zeros in what the products add to.
__global__ void __launch_bounds__(kPrepareThreads) prepare_kernel(PrepareArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int rows[kOutliers];
  const int i = blockIdx.x * kPrepareThreads + threadIdx.x, n = kPrepareCtas * kPrepareThreads;
  const TokenFactors& o = a.out;
  struct Token {
    int y;
    float m, S, rest, g;  // rest: 1 - p_y
    double s;
  };
  const auto token = [&](int t) {
    return Token{a.labels[t], a.stats[t], a.stats[(size_t)a.M + t], a.stats[2 * (size_t)a.M + t], a.dloss[t], a.s_tok[t]};
  };
  Token c = token(min(i, a.M - 1));  // requested before the row scales are looked at
  for (size_t z = i; z < a.zeros; z += n) a.zero[z] = make_uint4(0u, 0u, 0u, 0u);
  const ScaleTop top = scale_top(o.srow, a.V);
  int outlying = 0;
  if (top.outliers) {
    outlying = find_outliers(a, top.top, rows);
    __syncthreads();
  }
  // a thread per token, or a warp (every lane the same) where there are outlying rows to look at
  const bool by_warp = outlying > 0;
  const int step = by_warp ? n >> 5 : n;
  for (int t = by_warp ? i >> 5 : i; t < a.M; t += step) {
    if (by_warp || t != i) c = token(t);
    float m = c.m;
    const float S = c.S;
    double f = 0.0, wy = 0.0;
    int k = 0;
    if (c.y >= 0 && c.y < a.V && (S != 0.0f || c.rest != 0.0f)) {
      const double g = (double)c.g, rest = (double)c.rest;
      f = g * rest / (double)S;
      wy = -g * rest;
      if (!top.outliers) {
        while (k < 4 && S * (float)(2 << k) <= (float)kListed) ++k;  // S 2^k <= kListed
      } else {
        // tau in units of the top: half of the list for the rows below it, which are all below 1, half for the others
        float most = top.most, sum = S * top.most;  // too many rows: what they may be at most
        if (by_warp) outliers(a, rows, outlying, t, c.y, m, most, sum);
        const float half = 2.0f / kListed;
        const float tau = fmaxf(fminf(1.0f, S * half), fminf(most, sum * half) / top.top);
        while (k < 4 && tau * (float)(2 << k) <= 1.0f) ++k;
        if (tau > 1.0f) k = tau < 1e37f ? -1 - ilogbf(tau) : -123;  // (a NaN leaves 0)
      }
      const float mk = k < 0 ? __fsub_ru(m, (float)k) : m - (float)k;
      f *= exp2((double)mk - (double)m);
      m = mk;
    }
    if (m == -INFINITY) m = 0.0f;  // no other row
    o.shift[t] = k;
    // a token that is ignored has no gradient whatever its values are
    o.tok[t] = f == 0.0 && wy == 0.0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                     : make_float4(m, (float)c.s, (float)(f * c.s), (float)(wy * c.s));
    o.fac[t] = make_double2(f, wy);
  }
}

// Fixed point: steps per unit of coefficient.  A number n is stored as n + offset, its low 24 bits as digits;
// numbers up to 2^24 tau need no more (2^23 with negative scales, which take the sign's bit).  The margin of 64
// steps takes up the rounding of exp(l - m) just above 1; where a number may be larger, with outlying rows, it cannot be
// cut off, and the margin is 2^-8.
struct FixedPoint {
  float unit;    // steps per unit of exp(l - m') scale2(s_row)
  int offset;    // 0, or 2^23 with negative scales
  int range;     // 2^24, or 2^23
  bool outliers;
  double step;   // what one step stands for, of exp(l - m') s_row
};
__device__ __forceinline__ FixedPoint fixed_point(const uint2* srow, int V) {  // (whole warps)
  const ScaleTop t = scale_top(srow, V);
  FixedPoint p;
  p.range = t.neg ? 1 << 23 : 1 << 24;
  // (with scales below 1e-30, nothing of du is left either)
  p.unit = t.top < 1e-30f ? 0.0f : (float)(p.range - (t.outliers ? p.range >> 8 : 64)) / scale2(t.top);
  p.offset = t.neg ? 1 << 23 : 0;
  p.outliers = t.outliers;
  p.step = p.unit == 0.0f ? 0.0 : 1.0 / ((double)p.unit * kLog2e);
  return p;
}

// Pseudo-random number in [1, 2) of an accumulator; less 3/2 it is added before the coefficient is rounded to whole steps:
// the rounding is then right on average for coefficients of any size.  (Rounded to nearest, the thousands of
// coefficients below half a step all become zero, which sums over tokens show: 4e-6 of the norm weight's
// gradient at 2048 tokens x 50288 rows.)
__device__ __forceinline__ float dither(uint32_t acc) {
  return __uint_as_float(((acc * 0x9E3779B1u) & 0x7FFFFFu) | 0x3F800000u);
}

// The first product of the gradient: digits of a piece, and the row scales' gradient per 32 tokens.
template <int CG_, bool DS>
struct DigitPolicy {
  static constexpr int CG = CG_;
  static constexpr bool W_EARLY = true, W_IS_A = false, A_MN = false, RESIDENT = false;
  static constexpr int EPI_WARPS = 16, PARTS = EPI_WARPS / 4, EPI_COLS = BN_MAX / PARTS;  // columns of a warp
  struct Args {
    CUtensorMap map_a, map_b;  // codes, W
    RowArgs r;
    Common c;
    const float4* tok;      // [M]
    const int32_t* labels;  // [M]
    const float* s_row;     // [V]
    const uint2* srow;
    const int* shift;       // [M]
    int* listed;            // [M] entries of a token's list, zero before the first piece
    int2* list;             // [M][kListed] {row of W, number / 2^24}
    unsigned char* digits;  // [3][M / tb][Vp / 16][tb][16]
    float* colpart;         // [ceil(M / 32)][Vp]
    int M, V, v0, Vp, tb;
    size_t plane;           // bytes of one digit's plane
  };
  static __device__ __forceinline__ bool tile(const Args& a, int j, Tile& t) { return row_tile<CG, false>(a.r, j, t); }
  static __device__ __forceinline__ uint32_t bytes(const Args& a, const Tile& t) { return row_bytes<CG>(a.r, t); }
  static __device__ __forceinline__ Boxes boxes_a(const Args& a, const Tile& t, int) {
    return row_boxes_a<CG>(a.r, &a.map_a, t);
  }
  static __device__ __forceinline__ Boxes boxes_b(const Args& a, const Tile& t, int rank) {
    return row_boxes_b<CG>(a.r, &a.map_b, t, rank);
  }
  static __device__ __forceinline__ uint64_t adesc(uint32_t addr) { return umma_desc_k_sw128(addr); }
  static __device__ __forceinline__ uint64_t bdesc(const Args&, uint32_t addr) { return umma_desc_k_sw128(addr); }
  static __device__ __forceinline__ uint64_t a_step() { return UMMA_K >> 4; }
  static __device__ __forceinline__ uint64_t b_step(const Args&) { return UMMA_K >> 4; }
  static constexpr int EPI_SMEM = EPI_WARPS * EPI_COLS * 8;
  struct Epilogue {
    int q, part, lane;
    float* sr;   // row scales of this warp's columns (chunks of 16: part, part + PARTS, ..), in units of log 2
    float* cu;   // the same times the steps per unit
    FixedPoint fp;
    float4 tf;
    int label, most;
    __device__ __forceinline__ Epilogue(const Args& a, unsigned char* sm, int q_, int part_, int lane_)
        : q(q_), part(part_), lane(lane_), sr(reinterpret_cast<float*>(sm) + (part_ * 4 + q_) * 2 * EPI_COLS),
          cu(sr + EPI_COLS), fp(fixed_point(a.srow, a.V)) {}
    __device__ __forceinline__ void write_b(const Args&, unsigned char*, int) {}
    __device__ __forceinline__ void prepare(const Args& a, const Tile& t) {
      const int tk = t.a0 + q * 32 + lane;
      const bool valid = tk < a.M;
      tf = valid ? a.tok[tk] : make_float4(0.f, 0.f, 0.f, 0.f);
      label = valid ? a.labels[tk] - a.v0 : -1;
      most = fp.outliers ? (1 << 30) - 1 : (fp.range << (valid ? a.shift[tk] : 0)) - 1 + fp.offset;
#pragma unroll
      for (int k = 0; k < EPI_COLS / 32; ++k) {
        const int i = k * 32 + lane, c = ((i >> 4) * PARTS + part) * 16 + (i & 15);
        const float w = c < t.nb ? scale2(ld_f32(a.s_row + a.v0 + t.b0 + c)) : 0.0f;
        sr[i] = w;
        cu[i] = w * fp.unit;
      }
      __syncwarp();
    }
    __device__ __forceinline__ void tile(const Args& a, const Tile& t, uint32_t taddr) {
      const int tk = t.a0 + q * 32 + lane;
      const bool valid = tk < a.M;
      unsigned char* dst = a.digits + (size_t)(tk / a.tb) * a.tb * a.Vp + (size_t)(tk % a.tb) * 16;
      uint32_t v[16];
      const float *w1 = sr, *u1 = cu;
      const f2 s2 = pack2(tf.y, tf.y), m2 = pack2(-tf.x, -tf.x), f_s = pack2(tf.z, tf.z);
      if (part * 16 < t.nb) tmem_ld16(taddr + (uint32_t)(part * 16), v);
#pragma unroll 1  // copies of the body would not stay in the instruction cache
      for (int c = part * 16; c < t.nb; c += 16 * PARTS, w1 += 16, u1 += 16) {
        tmem_wait(v);
        const int v0 = t.b0 + c;  // within the piece
        const uint32_t lc = (uint32_t)(label - v0);
        const bool any = __any_sync(0xffffffffu, lc < 16u);
        const float at_label = any ? (float)(int)pick(v, (int)(lc & 15u)) : 0.0f;
        f2 h[8];
        uint32_t high = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const f2 w = *reinterpret_cast<const f2*>(w1 + 2 * j), u = *reinterpret_cast<const f2*>(u1 + 2 * j);
          const f2 av = pack2((float)(int)v[2 * j], (float)(int)v[2 * j + 1]);
          float e0, e1, n0, n1;
          unpack2(fma2(mul2(av, s2), w, m2), e0, e1);
          const f2 e = pack2(ex2(e0), ex2(e1));
          if (DS) h[j] = mul2(mul2(e, av), f_s);
          unpack2(fma2(e, u, add2(pack2(dither(v[2 * j]), dither(v[2 * j + 1])), pack2(-1.5f, -1.5f))), n0, n1);
          v[2 * j] = (uint32_t)__viaddmin_s32(__float2int_rn(n0), fp.offset, most);
          v[2 * j + 1] = (uint32_t)__viaddmin_s32(__float2int_rn(n1), fp.offset, most);
          high |= v[2 * j] | v[2 * j + 1];
        }
        if (any && lc < 16u) {  // the label's own column: no digits, and its gradient of the row scale
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float h0 = 0.0f, h1 = 0.0f;
            if (DS) unpack2(h[j], h0, h1);
            if ((int)lc == 2 * j) v[2 * j] = (uint32_t)fp.offset, h0 = tf.w * at_label;
            if ((int)lc == 2 * j + 1) v[2 * j + 1] = (uint32_t)fp.offset, h1 = tf.w * at_label;
            if (DS) h[j] = pack2(h0, h1);
          }
        }
        if (valid && (high >> 24)) {
          // few: the order of a list does not matter, its sum is taken in integers
          uint32_t which = 0u;
#pragma unroll
          for (int j = 0; j < 16; ++j) which |= (v[j] >> 24 ? 1u : 0u) << j;
          if (c + 16 > t.nb) which &= ~(0xFFFFFFFFu << (t.nb - c));
          while (which) {
            const int j = __ffs(which) - 1, i = atomicAdd(a.listed + tk, 1);
            which &= which - 1u;
            if (i < kListed) a.list[(size_t)tk * kListed + i] = make_int2(a.v0 + v0 + j, (int)pick(v, j) >> 24);
          }
        }
        if (valid) {
          unsigned char* dp = dst + (size_t)(v0 >> 4) * a.tb * 16;
          uint32_t o[3][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t* x = v + 4 * i;
            const uint32_t p = __byte_perm(x[0], x[1], 0x5140), r = __byte_perm(x[2], x[3], 0x5140);
            const uint32_t u = __byte_perm(x[0], x[1], 0x0062), w = __byte_perm(x[2], x[3], 0x0062);
            o[0][i] = __byte_perm(p, r, 0x5410) ^ 0x80808080u;
            o[1][i] = __byte_perm(p, r, 0x7632) ^ 0x80808080u;
            o[2][i] = __byte_perm(u, w, 0x5410) ^ 0x80808080u;
          }
#pragma unroll
          for (int k = 0; k < 3; ++k)
            *reinterpret_cast<uint4*>(dp + k * a.plane) = make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
        }
        if (c + 16 * PARTS < t.nb) tmem_ld16(taddr + (uint32_t)(c + 16 * PARTS), v);  // the next chunk
        if (DS) {
          // column sums over the warp's 32 tokens: halves exchanged at every step, lanes 2 j and 2 j + 1 end with
          // column j
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) {
            const bool up = (lane & (4 * o)) != 0;
#pragma unroll
            for (int j = 0; j < o; ++j) {
              f2 give = up ? h[j] : h[j + o];
              const f2 keep = up ? h[j + o] : h[j];
              give.v = __shfl_xor_sync(0xffffffffu, give.v, 4 * o);
              h[j] = add2(keep, give);
            }
          }
          float h0, h1;
          unpack2(h[0], h0, h1);
          h0 = ((lane & 2) ? h1 : h0) + __shfl_xor_sync(0xffffffffu, (lane & 2) ? h0 : h1, 2);
          h0 += __shfl_xor_sync(0xffffffffu, h0, 1);
          if (!(lane & 1) && c + (lane >> 1) < t.nb) a.colpart[(size_t)(t.a0 / 32 + q) * a.Vp + v0 + (lane >> 1)] = h0;
        }
      }
      __syncwarp();  // the scales are read: the next tile's may be written
    }
    __device__ __forceinline__ void finish(const Args&) {}
  };
};

// The second product: accumulators [set][3][M][d] += digits x transposed W of a piece.  Lanes are columns of W
// (128 a CTA), columns are tokens (tb a CTA).  A unit is a (token tile, digit, column tile) over all of the piece; groups
// (CTAs or pairs) take whole units in rounds, so that all of them read the same rows of W and digits at a time, and
// the units of a last, incomplete round are cut into one even range of K steps per group.  (All of it cut evenly, with
// every group at another K: 958 us instead of 920 at 2048 tokens, 283 MB a piece from DRAM instead of 127.)
// (units of work, and rounds in which every group takes a whole one)
__host__ __device__ __forceinline__ long long grad_units(int M, int d, int lanes, int tokens) {
  return 3LL * ((d + lanes - 1) / lanes) * ((M + tokens - 1) / tokens);
}
__host__ __device__ __forceinline__ long long grad_rounds(long long units, int groups) {
  const long long whole = quotient(units, groups), rest = units - whole * groups;
  if (rest * 10 >= 9LL * groups) return whole + 1;
  return whole > 0 && rest > 0 && rest * 8 < groups ? whole - 1 : whole;
}
template <int CG_>
struct GradPolicy {
  static constexpr int CG = CG_;
  static constexpr bool W_EARLY = false, W_IS_A = true, A_MN = true, RESIDENT = false;
  static constexpr int EPI_WARPS = 16, PARTS = EPI_WARPS / 4, EPI_SMEM = EPI_WARPS * 32 * 8;
  struct Args {
    CUtensorMap map_a, map_b;  // W in boxes of 128 x 128, digits in blocks of 128 bytes
    Common c;
    int32_t* acc;  // this piece's set: [3][M][d]
    size_t plane;
    int M, d, Vp, tb, kblocks, v0, nv;
    const float* colpart;  // [M / 32][Vp] partial sums of the row scales' gradient, or NULL
    float* ds;             // [nv]
    const int8_t* W;
    int32_t* colsum;       // [d] += column sums of the piece
  };
  static __host__ __device__ __forceinline__ long long units(const Args& a) {
    return grad_units(a.M, a.d, BM * CG, a.tb * CG);
  }
  static __device__ __forceinline__ bool tile(const Args& a, int j, Tile& t) {
    const int group = blockIdx.x / CG, groups = gridDim.x / CG;
    const long long all = units(a), whole = grad_rounds(all, groups);
    long long u = (long long)j * groups + group;
    if (j < whole) {
      if (u >= all) return false;
      t.kb0 = 0;
      t.kb1 = a.kblocks;
    } else {
      const long long rest = (all - whole * groups) * a.kblocks;
      if (rest <= 0) return false;
      const long long s0 = quotient(rest * group, groups), s1 = quotient(rest * (group + 1), groups);
      u = quotient(s0, a.kblocks) + (j - whole);
      const long long first = u * a.kblocks;
      if (first >= s1 || s0 >= s1) return false;
      t.kb0 = (int)((s0 > first ? s0 : first) - first);
      t.kb1 = (int)((s1 < first + a.kblocks ? s1 : first + a.kblocks) - first);
      u += whole * groups;
    }
    const int nd = (a.d + BM * CG - 1) / (BM * CG), ui = (int)u;
    t.a0 = ui % nd * BM * CG;
    t.na = BM * CG;
    t.aux = ui / nd % 3;  // digit
    t.b0 = ui / nd / 3 * a.tb * CG;
    t.nb = a.tb * CG;
    return true;
  }
  static __device__ __forceinline__ uint32_t bytes(const Args& a, const Tile&) {
    return CG * (A_BYTES + (uint32_t)a.tb * BK);
  }
  // 128 rows x 128 columns of W as they are: zero past the vocabulary and past d
  static __device__ __forceinline__ Boxes boxes_a(const Args& a, const Tile& t, int) {
    return Boxes{&a.map_a, 1, BK, a.v0, 0, BK, t.a0};
  }
  // the digits were laid out as the product reads them: eight 16-byte K columns of all rows are contiguous
  static __device__ __forceinline__ Boxes boxes_b(const Args& a, const Tile& t, int rank) {
    return Boxes{&a.map_b, 1, a.tb, (int)((t.aux * a.plane + (size_t)(t.b0 + rank * a.tb) * a.Vp) / 128), 0, a.tb};
  }
  static __device__ __forceinline__ uint64_t adesc(uint32_t addr) { return umma_desc_mn_sw128(addr); }
  static __device__ __forceinline__ uint64_t bdesc(const Args& a, uint32_t addr) {
    return umma_desc_k_plain(addr, a.tb * 16);
  }
  static __device__ __forceinline__ uint64_t a_step() { return UMMA_K * 128 >> 4; }
  static __device__ __forceinline__ uint64_t b_step(const Args& a) { return (uint64_t)(2 * a.tb); }
  struct Epilogue {
    int q, part, lane;
    // While the first products accumulate: the column sums of the piece, and its part of ds_row, 32 rows of W per
    // CTA at a time, the partial sums of every 32 tokens in a slice per warp, joined in order.
    __device__ __forceinline__ Epilogue(const Args& a, unsigned char* sm, int q_, int part_, int lane_)
        : q(q_), part(part_), lane(lane_) {
      column_sums(a, reinterpret_cast<int*>(sm));
      if (!a.colpart) return;
      double* red = reinterpret_cast<double*>(sm);  // [EPI_WARPS][32]
      const int sl = part * 4 + q, parts = (a.M + 31) / 32;
      for (int b = blockIdx.x * 32; b < a.nv; b += gridDim.x * 32) {
        const int v = b + lane;
        double s = 0.0;
        if (v < a.nv) {
#pragma unroll 8
          for (int p = sl; p < parts; p += EPI_WARPS) s += (double)a.colpart[(size_t)p * a.Vp + v];
        }
        red[sl * 32 + lane] = s;
        sync();
        if (sl == 0 && v < a.nv) {
          for (int k = 1; k < EPI_WARPS; ++k) s += red[k * 32 + lane];
          a.ds[v] = (float)s;
        }
        sync();
      }
    }
    static __device__ __forceinline__ void sync() { asm volatile("bar.sync 1, %0;" ::"n"(EPI_WARPS * 32) : "memory"); }
    // Blocks of 128 rows x 512 columns in an even range per CTA, rows before columns; a warp takes eight rows, a lane
    // 16 columns, two sums of bytes + 128 per register (at most 8 x 255).
    __device__ __forceinline__ void column_sums(const Args& a, int* red) const {
      static_assert(EPI_WARPS * 8 == 128 && EPI_SMEM >= 512 * 4, "a block of columns");
      const int w = part * 4 + q, i = w * 32 + lane;
      const int nr = (a.nv + 127) / 128, total = nr * ((a.d + 511) / 512);
      const int u1 = (int)((long long)total * (blockIdx.x + 1) / gridDim.x);
      red[i] = 0;
      sync();
      for (int u = (int)((long long)total * blockIdx.x / gridDim.x); u < u1; ++u) {
        const int cb = u / nr, r0 = (u - cb * nr) * 128 + w * 8, col = cb * 512 + lane * 16;
        const int n = col < a.d ? min(8, a.nv - r0) : 0;
        uint4 x[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          x[r] = r < n ? ld_u32x4(a.W + (size_t)(a.v0 + r0 + r) * a.d + col) : make_uint4(0u, 0u, 0u, 0u);
        uint32_t even[4] = {0u, 0u, 0u, 0u}, odd[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const uint32_t y[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t b = y[k] ^ 0x80808080u;
            even[k] += b & 0x00FF00FFu;
            odd[k] += (b >> 8) & 0x00FF00FFu;
          }
        }
        if (n > 0) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint32_t h = (k & 1) ? odd[k >> 2] : even[k >> 2];
            atomicAdd_block(red + k * 32 + lane, (int)((k & 2) ? h >> 16 : h & 0xFFFFu) - 8 * 128);
          }
        }
        if (u + 1 == u1 || (u + 1) / nr != cb) {
          sync();
          const int c = cb * 512 + lane * 16 + w;
          if (c < a.d && red[i]) atomicAdd(a.colsum + c, red[i]);
          red[i] = 0;
          sync();
        }
      }
    }
    __device__ __forceinline__ void tile(const Args& a, const Tile& t, uint32_t taddr) {
      const int col = t.a0 + q * 32 + lane, n = min(t.nb, a.M - t.b0);
      const bool cv = col < a.d;
      int32_t* base = a.acc + ((size_t)t.aux * a.M + t.b0) * a.d + col;
      for (int c = part * 32; c < n; c += 32 * PARTS) {
        uint32_t v[32];
        tmem_ld32(taddr + (uint32_t)c, v);
        tmem_wait(v);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (cv && c + j < n) atomicAdd(base + (size_t)(c + j) * a.d, (int)v[j]);
      }
    }
    __device__ __forceinline__ void write_b(const Args&, unsigned char*, int) {}
    __device__ __forceinline__ void prepare(const Args&, const Tile&) {}
    __device__ __forceinline__ void finish(const Args&) {}
  };
};

struct GradFinishArgs {
  const int32_t* acc;     // [sets][3][M][d]
  const int32_t* colsum;  // [d]
  const uint2* srow;
  const double2* fac;     // [M]
  const int* listed;      // [M]
  const int2* list;       // [M][kListed]
  const int32_t* labels;
  const int8_t* W;
  const float* s_row;
  const void* x;
  const float* norm_w;
  const float* rn;
  void* dx;
  float* npart;           // [gridDim.x][d] or NULL
  int64_t ldx, lddx;
  int M, V, d, sets;
};

// Joins the digits of a token and the listed rows: du = f step (sum of digits base 256 + offsets + 2^24 listed) +
// w_y s_row_y W_y, integers and then fp64, rounded to fp32; then the norm's backward, dx = r (du w) - x r^3 / d sum(du w x).  One CTA per token at a time;
// the norm weight's gradient is summed over the CTA's tokens in registers.
template <typename T, int CH>
__global__ void __launch_bounds__(256) grad_finish_kernel(GradFinishArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ double red[2][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const FixedPoint fp = fixed_point(a.srow, a.V);
  // stored bytes are digit - 128 and the number itself is offset: both come back through W's column sums
  const long long back = 0x808080LL - (long long)fp.offset;
  float dn[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) dn[c][k] = 0.0f;
  int turn = 0;
  for (int t = blockIdx.x; t < a.M; t += gridDim.x, turn ^= 1) {
    const double2 fac = a.fac[t];
    const int y = a.labels[t];
    const bool kept = y >= 0 && y < a.V;
    const int nl = min(a.listed[t], kListed);
    const double f = fac.x * fp.step, wy = kept ? fac.y * (double)ld_f32(a.s_row + y) : 0.0;
    float du[CH][8], xv[CH][8];
    double dot = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (threadIdx.x + 256 * c) * 8;
#pragma unroll
      for (int k = 0; k < 8; ++k) du[c][k] = xv[c][k] = 0.0f;
      if (i >= a.d) continue;
      long long sum[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] = back * (long long)a.colsum[i + k];
      for (int s = 0; s < a.sets; ++s)
#pragma unroll
        for (int g = 0; g < 3; ++g) {
          const int4* p = reinterpret_cast<const int4*>(a.acc + (((size_t)s * 3 + g) * a.M + t) * a.d + i);
          const int4 u = p[0], w = p[1];
          const int n[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 8; ++k) sum[k] += (long long)n[k] << (8 * g);
        }
      for (int l = 0; l < nl; ++l) {
        const int2 e = a.list[(size_t)t * kListed + l];
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.W + (size_t)e.x * a.d + i));
#pragma unroll
        for (int k = 0; k < 8; ++k)
          sum[k] += (long long)(e.y * (int)(int8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3)))) << 24;
      }
      uint2 wr = make_uint2(0u, 0u);
      if (kept) wr = __ldg(reinterpret_cast<const uint2*>(a.W + (size_t)y * a.d + i));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int w = (int)(int8_t)((k < 4 ? wr.x : wr.y) >> (8 * (k & 3)));
        du[c][k] = kept ? (float)(f * (double)sum[k] + wy * (double)w) : 0.0f;
      }
      if (a.norm_w) {
        float nw[8];
        load8<float>(a.norm_w + i, nw);
        load8<T>(reinterpret_cast<const T*>(a.x) + (size_t)t * a.ldx + i, xv[c]);
        const float r = a.rn[t];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          dn[c][k] += kept ? du[c][k] * (xv[c][k] * r) : 0.0f;
          du[c][k] *= nw[k];
          dot += (double)du[c][k] * (double)xv[c][k];
        }
      }
    }
    if (a.norm_w) {
      dot = warp_sum(dot);
      if (lane == 0) red[turn][warp] = dot;
      __syncthreads();
      dot = 0.0;
#pragma unroll
      for (int w = 0; w < 8; ++w) dot += red[turn][w];
      const float r = a.rn[t];
      const float k3 = kept ? (float)((double)r * r * r * dot / (double)a.d) : 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) du[c][k] = kept ? fmaf(r, du[c][k], -xv[c][k] * k3) : 0.0f;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (threadIdx.x + 256 * c) * 8;
      if (i < a.d) store8<T>(reinterpret_cast<T*>(a.dx) + (size_t)t * a.lddx + i, du[c]);
    }
  }
  if (a.npart) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (threadIdx.x + 256 * c) * 8;
      if (i < a.d) store8<float>(a.npart + (size_t)blockIdx.x * a.d + i, dn[c]);
    }
  }
}

// 32 columns per CTA, 32 slices of the partial sums, joined in order.
__global__ void __launch_bounds__(1024) dnorm_finish_kernel(const float* npart, int parts, int d, float* dn) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (i < d) {
#pragma unroll 8
    for (int p = sl; p < parts; p += 32) s += npart[(size_t)p * d + i];
  }
  red[sl][lane] = s;
  __syncthreads();
  const double sum = warp_sum((double)red[lane][sl]);  // warp sl joins column sl
  const int c = blockIdx.x * 32 + sl;
  if (lane == 0 && c < d) dn[c] = (float)sum;
}

// ------------------------------------------------------------------------------------ host side

// Forward workspace: [status word][codes M x d][scales f64 M][partials float2 slots x M]
struct ForwardWs {
  size_t q, s, part, total;
};
// How tokens and columns are tiled: up to 128 tokens by single CTAs (the stream of W bounds the products), above
// by pairs.  (50288 x 2048, single against pairs: loss of 96 tokens 27.5 / 30.7 us, of 256 33.8 / 31.8; gradient of 96 101.7 /
// 101.8, of 192 135 / 124.  Over 8191 x 1040 it is the other way round by up to 12 %: 14.4 us of 96 tokens' loss in pairs, 13.8
// instead of 15.4 of 129's in single ones.)
struct Layout {
  int cg, tb;      // CTAs per tile; tokens of a block of digits
  size_t mp, dp;   // tokens and columns of W, padded to whole tiles
};
Layout layout(int M, int d) {
  Layout l;
  l.cg = M <= BM ? 1 : 2;
  const int tiles = ceil_div(M, BM * l.cg);  // blocks of equal size, a multiple of 16
  l.tb = (ceil_div(M, tiles * l.cg) + 15) & ~15;
  l.mp = (size_t)ceil_div(M, l.tb * l.cg) * l.tb * l.cg;
  l.dp = (size_t)ceil_div(d, BM * l.cg) * BM * l.cg;
  return l;
}

int forward_slots(int M, int d, int V) {
  const int cg = layout(M, d).cg, rows = ceil_div(M, BM * cg);
  const int grid = ceil_div(V, even_tile(rows, V, kSms / cg)), range = ceil_div(V, 32) < kMaxRangeCtas ? ceil_div(V, 32) : kMaxRangeCtas;
  return 2 * (M > BM * cg ? grid : range);
}
ForwardWs forward_ws(int M, int d, int V) {
  ForwardWs w;
  w.q = kStatusBytes;
  w.s = w.q + al256((size_t)M * d);
  w.part = w.s + al256(sizeof(double) * (size_t)M);
  w.total = w.part + al256(sizeof(float2) * (size_t)forward_slots(M, d, V) * M);
  return w;
}

// The vocabulary's pieces: rows per piece (a multiple of 256), and how many accumulator sets keep the int32 sums
// in range (|digit| <= 128, |W| <= 128: 2^14 rows-worth per row, so at most 131071 rows a set).
struct Pieces {
  int rows, n, per_set, sets;
};
// Bytes of digits and W of a piece at most.  Where the second product is one split along K, every CTA is at another K and
// the piece has to stay in the 126 MB L2 (333 tokens x 50288 x 2048: 80 MB 231 us, 120: 239, 220: 247).  Where CTAs
// take whole units they read the same K at a time, and fewer pieces are better (2048 tokens: 80 MB 920 us, 120: 880,
// 160: 868, 220: 861, 440: 860); 160 MB keep the workspace below half of what fp32 logits would take.
constexpr size_t kPieceBytes = 80u << 20, kSyncBytes = 160u << 20;
Pieces pieces(int M, int d, int V) {
  const Layout l = layout(M, d);
  const bool sync = grad_rounds(grad_units(M, d, BM * l.cg, l.tb * l.cg), kSms / l.cg) > 0;
  size_t t = (sync ? kSyncBytes : kPieceBytes) / (3 * l.mp + l.dp + l.mp / 8) / BN_MAX;  // tiles of 256 rows
  const int vt = ceil_div(V, BN_MAX), mt = ceil_div(M, BM * l.cg), groups = kSms / l.cg;
  const int most = (int)(t < 8 ? 8 : t > 256 ? 256 : t);
  // of the sizes up to that, the one with the least rounds of digit tiles, a piece counting as two more
  int best = 0;
  long long least = 0;
  for (int k = most < vt ? most : vt; k > 0 && k * 4 > most; --k) {
    const int full = vt / k, rest = vt % k;
    const long long cost = (long long)full * (ceil_div(mt * k, groups) + 2) + (rest ? ceil_div(mt * rest, groups) + 2 : 0);
    if (!best || cost < least) {
      best = k;
      least = cost;
    }
  }
  t = best ? best : vt;
  Pieces p;
  p.rows = (int)t * BN_MAX;
  p.n = ceil_div(V, p.rows);
  p.per_set = 131071 / p.rows;
  p.sets = ceil_div(p.n, p.per_set);
  return p;
}
constexpr int kNormParts = 4 * kSms;

struct BackwardWs {
  size_t q, s, rn, tok, fac, shift, list, srow, zero, listed, colsum, acc, zero_end, digits, colpart, npart, total;
};
BackwardWs backward_ws(int M, int d, int V) {
  const Pieces p = pieces(M, d, V);
  const Layout l = layout(M, d);
  BackwardWs w;
  w.q = kStatusBytes;
  w.s = w.q + al256((size_t)M * d);
  w.rn = w.s + al256(sizeof(double) * (size_t)M);
  w.tok = w.rn + al256(sizeof(float) * (size_t)M);
  w.fac = w.tok + al256(sizeof(float4) * (size_t)M);
  w.shift = w.fac + al256(sizeof(double2) * (size_t)M);
  w.list = w.shift + al256(sizeof(int) * (size_t)M);
  w.srow = w.list + al256(sizeof(int2) * kListed * (size_t)M);
  w.zero = w.srow + al256(sizeof(uint2) * kScanParts);
  w.listed = w.zero;
  w.colsum = w.listed + al256(sizeof(int) * (size_t)M);
  w.acc = w.colsum + al256(sizeof(int32_t) * (size_t)d);
  w.zero_end = w.acc + al256(sizeof(int32_t) * 3 * (size_t)p.sets * M * d);
  w.digits = w.zero_end;
  w.colpart = w.digits + al256(3 * l.mp * p.rows);
  w.npart = w.colpart + al256(sizeof(float) * 4 * l.cg * (size_t)ceil_div(M, BM * l.cg) * p.rows);
  w.total = w.npart + al256(sizeof(float) * (size_t)(M < kNormParts ? M : kNormParts) * d);
  return w;
}

// Token tiles on the lanes, rows of W on the columns: one tile of tokens streams W in balanced ranges, more take
// whole tiles.
template <class P>
int row_args(typename P::Args& a, int M, int rows, int first, int d, const int8_t* W, int V, const int8_t* q, int* err) {
  constexpr int CG = P::CG;
  a.r.rows_a = M;
  a.r.rows_b = rows;
  a.r.b_first = first;
  a.r.kblocks = ceil_div(d, BK);
  a.r.mode = M <= BM * CG ? kRangeB : kGrid;
  a.r.tile_b = a.r.mode == kRangeB ? BN_MAX : even_tile(ceil_div(M, BM * CG), rows, kSms / CG);
  a.r.box_a = BM;
  a.r.box_b = a.r.mode == kRangeB ? 32 / CG : a.r.tile_b / CG;
  a.c.b_tile = a.r.tile_b / CG;
  a.c.stages = ring_stages(a.c, P::EPI_SMEM);
  a.c.err = err;
  if (!encode_u8_map_sw128(&a.map_a, q, M, d, a.r.box_a) || !encode_u8_map_sw128(&a.map_b, W, V, d, a.r.box_b))
    return DFSSM_EUNSUPPORTED;
  return DFSSM_OK;
}
template <class P>
int row_groups(const RowArgs& r) {
  const long long most = max_groups<P>() < kMaxRangeCtas ? max_groups<P>() : kMaxRangeCtas;
  const long long units = r.mode == kGrid ? (long long)ceil_div(r.rows_a, BM * P::CG) * ceil_div(r.rows_b, r.tile_b)
                                          : ceil_div(r.rows_b, 32);
  return (int)(units < most ? units : most);
}

template <bool RESIDENT>
int forward_small(const int8_t* W, const float* s_row, int V, const RowsQuantArgs& qa, const int32_t* labels, float* loss,
                  float* stats, float2* part, int* err, cudaStream_t st) {
  using P = SmallForwardPolicy<RESIDENT>;
  const int M = qa.M, d = qa.d;
  typename P::Args a{};
  a.r.mode = kRangeA;
  a.r.rows_a = V;
  a.r.rows_b = M;
  a.r.tile_b = BN_MAX;
  a.r.kblocks = ceil_div(d, BK);
  a.r.box_a = 32;
  a.r.box_b = a.c.b_tile = RESIDENT ? RES_ROWS : (M + 15) & ~15;
  a.c.resident = RESIDENT ? resident_bytes(d) : 0;
  a.c.stages = ring_stages(a.c, P::EPI_SMEM);
  a.c.err = err;
  a.x = ResidentArgs{qa.x, qa.x_type, qa.ldx, M, d, qa.norm_w, nullptr, nullptr};
  a.s_tok = qa.s;
  a.s_row = s_row;
  a.labels = labels;
  a.stats = stats;
  a.loss = loss;
  a.part = part;
  a.done = reinterpret_cast<unsigned*>(err) + 16;  // beside the status word
  a.M = M;
  a.V = V;
  if (!encode_u8_map_sw128(&a.map_a, W, V, d, a.r.box_a)) return DFSSM_EUNSUPPORTED;
  cudaError_t e = cudaSuccess;
  if (!RESIDENT) {
    if (!encode_u8_map_sw128(&a.map_b, qa.q, M, d, a.r.box_b)) return DFSSM_EUNSUPPORTED;
    e = launch_rows_quant(qa, st);
  }
  const int most = max_groups<P>() < kMaxRangeCtas ? max_groups<P>() : kMaxRangeCtas, units = ceil_div(V, 32);
  if (e == cudaSuccess) e = launch<P>(a, units < most ? units : most, P::EPI_SMEM, st);
  return e == cudaSuccess ? DFSSM_OK : record_cuda_failure(e);
}

template <int CG>
int forward(const int8_t* W, const float* s_row, int V, const RowsQuantArgs& qa, const int32_t* labels, float* loss,
            float* stats, float2* part, int* err, cudaStream_t st) {
  using P = ForwardPolicy<CG>;
  const int M = qa.M, d = qa.d;
  typename P::Args a{};
  const int rc = row_args<P>(a, M, V, 0, d, W, V, qa.q, err);
  if (rc) return rc;
  a.s_tok = qa.s;
  a.s_row = s_row;
  a.labels = labels;
  a.label_acc = reinterpret_cast<int*>(stats + 2 * (size_t)M);
  a.part = part;
  a.M = M;
  a.V = V;
  const int groups = row_groups<P>(a.r);
  cudaError_t e = launch_rows_quant(qa, st);
  if (e == cudaSuccess) e = launch<P>(a, groups, P::EPI_SMEM, st);
  const int slots = 2 * (a.r.mode == kGrid ? ceil_div(V, a.r.tile_b) : groups);
  if (e == cudaSuccess)
    e = launch_pdl(loss_finish_kernel, dim3(ceil_div(M, 32)), dim3(32 * LF_SLICES), 0, st, (const float2*)part, slots, M, V,
                   labels, (const double*)qa.s, s_row, stats, loss, err);
  return e == cudaSuccess ? DFSSM_OK : record_cuda_failure(e);
}

// One piece of the vocabulary, rows [v0, v0 + nv): digits, the row scales' gradient, and their product with W.
struct Piece {
  const int8_t* W;
  const float* s_row;
  const int8_t* q;
  const int32_t* labels;
  TokenFactors tf;
  int* listed;
  int2* list;
  unsigned char* digits;
  float* colpart;
  int32_t* colsum;  // [d]
  int32_t* acc;     // the piece's set
  float* ds_row;    // [V] or NULL
  int* err;
  int V, d, M, v0, nv, Vp;
  Layout l;
};
// CGD and CG: CTAs per tile of the digits and of the second product.
template <int CGD, int CG, bool DS>
int piece_products(const Piece& p, cudaStream_t st) {
  using P = DigitPolicy<CGD, DS>;
  const size_t plane = p.l.mp * p.Vp;
  typename P::Args a{};
  const int rc = row_args<P>(a, p.M, p.nv, p.v0, p.d, p.W, p.V, p.q, p.err);
  if (rc) return rc;
  a.tok = p.tf.tok;
  a.shift = p.tf.shift;
  a.listed = p.listed;
  a.list = p.list;
  a.labels = p.labels;
  a.s_row = p.s_row;
  a.srow = p.tf.srow;
  a.digits = p.digits;
  a.colpart = p.colpart;
  a.M = p.M;
  a.V = p.V;
  a.v0 = p.v0;
  a.Vp = p.Vp;
  a.tb = p.l.tb;
  a.plane = plane;
  cudaError_t e = launch<P>(a, row_groups<P>(a.r), P::EPI_SMEM, st);
  if (e != cudaSuccess) return record_cuda_failure(e);
  using G = GradPolicy<CG>;
  typename G::Args g{};
  g.c.b_tile = p.l.tb;
  g.c.stages = ring_stages(g.c, G::EPI_SMEM);
  g.c.err = p.err;
  if (!encode_u8_map_sw128(&g.map_a, p.W, p.V, p.d, BK) ||
      !encode_blocks_map(&g.map_b, p.digits, (int64_t)(3 * plane / 128), p.l.tb))
    return DFSSM_EUNSUPPORTED;
  g.acc = p.acc;
  g.plane = plane;
  g.M = p.M;
  g.d = p.d;
  g.Vp = p.Vp;
  g.tb = p.l.tb;
  g.kblocks = ceil_div(p.nv, BK);
  g.colpart = DS ? p.colpart : nullptr;
  g.ds = DS ? p.ds_row + p.v0 : nullptr;
  g.v0 = p.v0;
  g.nv = p.nv;
  g.W = p.W;
  g.colsum = p.colsum;
  const long long steps = G::units(g) * g.kblocks;
  const int most = max_groups<G>();
  e = launch<G>(g, (int)(steps < most ? steps : most), G::EPI_SMEM, st);
  return e == cudaSuccess ? DFSSM_OK : record_cuda_failure(e);
}

template <typename T>
cudaError_t launch_grad_finish(const GradFinishArgs& a, int grid, cudaStream_t st) {
  if (a.d <= 2048) return launch_pdl(grad_finish_kernel<T, 1>, dim3(grid), dim3(256), 0, st, a);
  if (a.d <= 4096) return launch_pdl(grad_finish_kernel<T, 2>, dim3(grid), dim3(256), 0, st, a);
  return launch_pdl(grad_finish_kernel<T, 4>, dim3(grid), dim3(256), 0, st, a);
}

inline bool al(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

RowsQuantArgs quant_args(const void* x, int x_type, int64_t ldx, int M, int d, const float* norm_w, char* base,
                         size_t q, size_t s) {
  RowsQuantArgs a{};
  a.x = x;
  a.x_type = x_type;
  a.ldx = ldx;
  a.M = M;
  a.d = d;
  a.norm_w = norm_w;
  a.q = reinterpret_cast<int8_t*>(base + q);
  a.s = reinterpret_cast<double*>(base + s);
  return a;
}

}  // namespace

size_t head_loss_workspace_bytes(int M, int d, int V) { return forward_ws(M, d, V).total; }
size_t head_loss_backward_workspace_bytes(int M, int d, int V) { return backward_ws(M, d, V).total; }

}  // namespace dfssm

extern "C" int dfssm_head_loss(const int8_t* W, const float* s_row, int V, int d, const void* x, int x_type,
                               int64_t ldx, int M, const float* norm_w, const int32_t* labels, float* loss,
                               float* stats, void* workspace, size_t ws_bytes, void* stream) {
  using namespace dfssm;
  int st = check_int8_matrix(W, V, d);
  if (st) return st;
  if (!s_row) return DFSSM_EINVAL;
  st = check_tokens(M);
  if (st) return st;
  if (M == 0) return DFSSM_OK;
  st = check_rows(x, x_type, ldx, d);
  if (st) return st;
  if (!labels || !loss || !stats) return DFSSM_EINVAL;
  if (!al(s_row, 4) || !al(norm_w, 16) || !al(labels, 4) || !al(loss, 4) || !al(stats, 4)) return DFSSM_EALIGN;
  const ForwardWs w = forward_ws(M, d, V);
  if (!workspace || !al(workspace, 256) || ws_bytes < w.total) return DFSSM_EWORKSPACE;
  if (!device_ok()) return DFSSM_EDEVICE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(workspace);
  const RowsQuantArgs qa = quant_args(x, x_type, ldx, M, d, norm_w, base, w.q, w.s);
  const auto f = resident_supported(M, d)  ? forward_small<true>
                 : M <= SMALL_TOKENS       ? forward_small<false>
                 : layout(M, d).cg == 1    ? forward<1>
                                           : forward<2>;
  return f(W, s_row, V, qa, labels, loss, stats, reinterpret_cast<float2*>(base + w.part), reinterpret_cast<int*>(base), s);
}

extern "C" int dfssm_head_loss_backward(const int8_t* W, const float* s_row, int V, int d, const void* x,
                                        int x_type, int64_t ldx, int M, const float* norm_w,
                                        const int32_t* labels, const float* stats, const float* dloss, void* dx,
                                        int64_t lddx, float* ds_row, float* dnorm_w, void* workspace,
                                        size_t ws_bytes, void* stream) {
  using namespace dfssm;
  int st = check_int8_matrix(W, V, d);
  if (st) return st;
  if (!s_row || (dnorm_w && !norm_w)) return DFSSM_EINVAL;
  st = check_tokens(M);
  if (st) return st;
  if (V > 1 << 24) return DFSSM_EUNSUPPORTED;  // W's column sums are int32
  if (M == 0) {  // no tokens: the sums over them are zero
    if (!al(ds_row, 4) || !al(dnorm_w, 4)) return DFSSM_EALIGN;
    if ((ds_row || dnorm_w) && !device_ok()) return DFSSM_EDEVICE;
    cudaError_t e0 = cudaSuccess;
    if (ds_row) e0 = cudaMemsetAsync(ds_row, 0, sizeof(float) * (size_t)V, static_cast<cudaStream_t>(stream));
    if (e0 == cudaSuccess && dnorm_w)
      e0 = cudaMemsetAsync(dnorm_w, 0, sizeof(float) * (size_t)d, static_cast<cudaStream_t>(stream));
    return e0 == cudaSuccess ? DFSSM_OK : record_cuda_failure(e0);
  }
  st = check_rows(x, x_type, ldx, d);
  if (st) return st;
  st = check_rows(dx, x_type, lddx, d);
  if (st) return st;
  if (!labels || !stats || !dloss) return DFSSM_EINVAL;
  if (!al(s_row, 4) || !al(norm_w, 16) || !al(labels, 4) || !al(stats, 4) || !al(dloss, 4) || !al(ds_row, 4) ||
      !al(dnorm_w, 4))
    return DFSSM_EALIGN;
  const BackwardWs w = backward_ws(M, d, V);
  if (!workspace || !al(workspace, 256) || ws_bytes < w.total) return DFSSM_EWORKSPACE;
  if (!device_ok()) return DFSSM_EDEVICE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(workspace);
  RowsQuantArgs qa = quant_args(x, x_type, ldx, M, d, norm_w, base, w.q, w.s);
  qa.rn = reinterpret_cast<float*>(base + w.rn);
  qa.scan = s_row;
  qa.V = V;
  qa.range = reinterpret_cast<uint2*>(base + w.srow);
  cudaError_t e = launch_rows_quant(qa, s);
  if (e != cudaSuccess) return record_cuda_failure(e);
  TokenFactors tf{reinterpret_cast<float4*>(base + w.tok), reinterpret_cast<int*>(base + w.shift),
                  reinterpret_cast<double2*>(base + w.fac), qa.range};
  const PrepareArgs pa{stats, labels, dloss, qa.q, qa.s, W, s_row, M, V, d, tf, reinterpret_cast<uint4*>(base + w.zero),
                       (w.zero_end - w.zero) / 16};
  e = launch_pdl(prepare_kernel, dim3(kPrepareCtas), dim3(kPrepareThreads), 0, s, pa);
  if (e != cudaSuccess) return record_cuda_failure(e);

  const Pieces pc = pieces(M, d, V);
  int32_t* colsum = reinterpret_cast<int32_t*>(base + w.colsum);
  int32_t* acc = reinterpret_cast<int32_t*>(base + w.acc);
  Piece p{};
  p.W = W;
  p.s_row = s_row;
  p.q = qa.q;
  p.labels = labels;
  p.tf = tf;
  p.listed = reinterpret_cast<int*>(base + w.listed);
  p.list = reinterpret_cast<int2*>(base + w.list);
  p.digits = reinterpret_cast<unsigned char*>(base + w.digits);
  p.colpart = reinterpret_cast<float*>(base + w.colpart);
  p.colsum = colsum;
  p.ds_row = ds_row;
  p.err = reinterpret_cast<int*>(base);
  p.V = V;
  p.d = d;
  p.M = M;
  p.Vp = pc.rows;
  p.l = layout(M, d);
  // the digits are bound by their epilogue, which takes a tile's empty lanes as long as full ones: single CTAs where
  // pairs would have an eighth more lanes (gradient, single against pairs, 50288 x 2048, 20011 x 1040 and 8191 x 1040: 333
  // tokens, a third more lanes, 178 / 182, 64 / 68, 49 / 50 us; 850, a seventh more, 328 / 337, 110 / 113, 69 / 69; 1100, a
  // ninth, 423 / 425, 151 / 150, 78 / 78; 450, none, 217 / 215, 76 / 75, 54 / 53)
  const bool one = ceil_div(M, 2 * BM) * 2 * 8 >= ceil_div(M, BM) * 9;
  const auto products = p.l.cg == 1 ? (ds_row ? piece_products<1, 1, true> : piece_products<1, 1, false>)
                        : one       ? (ds_row ? piece_products<1, 2, true> : piece_products<1, 2, false>)
                                    : (ds_row ? piece_products<2, 2, true> : piece_products<2, 2, false>);
  for (int i = 0; i < pc.n; ++i) {
    p.v0 = i * pc.rows;
    p.nv = V - p.v0 < pc.rows ? V - p.v0 : pc.rows;
    p.acc = acc + (size_t)(i / pc.per_set) * 3 * M * d;
    st = products(p, s);
    if (st) return st;
  }
  GradFinishArgs fa{};
  fa.acc = acc;
  fa.colsum = colsum;
  fa.srow = tf.srow;
  fa.fac = tf.fac;
  fa.listed = p.listed;
  fa.list = p.list;
  fa.labels = labels;
  fa.W = W;
  fa.s_row = s_row;
  fa.x = x;
  fa.norm_w = norm_w;
  fa.rn = qa.rn;
  fa.dx = dx;
  fa.npart = dnorm_w ? reinterpret_cast<float*>(base + w.npart) : nullptr;
  fa.ldx = ldx;
  fa.lddx = lddx;
  fa.M = M;
  fa.V = V;
  fa.d = d;
  fa.sets = pc.sets;
  const int parts = M < kNormParts ? M : kNormParts;
  e = x_type == DFSSM_BF16 ? launch_grad_finish<__nv_bfloat16>(fa, parts, s) : launch_grad_finish<float>(fa, parts, s);
  if (e == cudaSuccess && dnorm_w)
    e = launch_pdl(dnorm_finish_kernel, dim3(ceil_div(d, 32)), dim3(1024), 0, s, (const float*)fa.npart, parts, d,
                   dnorm_w);
  return e == cudaSuccess ? DFSSM_OK : record_cuda_failure(e);
}
