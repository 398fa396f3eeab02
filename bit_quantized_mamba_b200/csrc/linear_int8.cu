// Many-token int8 linear (include/dfssm.h, dfssm_linear_int8): y[t][v] = fl32(acc[t][v] s[t] s_row[v]), the
// LM head's arithmetic (technical summary §2.B: int8 LM head with per-row scaling; §2.C: per-token int8
// activations) for any number of tokens.
//   1. rows_quant: codes and scale of every token (with the final RMSNorm when a weight is given); for up to
//      four tokens every CTA of the product does that itself;
//   2. the tcgen05 int8 product (gemm_i8.cuh) with the rows of W on the tensor memory's lanes and the tokens on
//      its columns: a warp's store of one token covers 32 consecutive outputs, and few tokens make a narrow
//      product (16 columns for one token), so that the stream of W alone bounds it.
// The outputs are the head's bit for bit: the accumulators are exact, and the epilogue gives the definition's
// value, an fp64 product rounded once to fp32 (bf16 outputs round that once more).
//
// W of 50288 x 2048: 1 token 21 us and 16 tokens 24.9 us (4.8 and 4.2 TB/s, the stream of W with a launch's
// latency before it), 2048 tokens 195 us (2170 TOPS; bound by power: the loss's product, which stores nothing, runs
// at 2550).

#include "gemm_i8.cuh"

#include <cuda_bf16.h>

namespace dfssm {
namespace {

using namespace gemm_i8;

// fl32(acc s w) of the definition, its fp64 product rounded once, in fp32: with x = acc exact (|acc| < 2^24), p = fl(x s)
// and e = x s - p, the product is y - r, y = fl(p w), r = (y - p w) - e w, where r alone is rounded, by less than
// 2^-47 |y|.  Where y - r rounds the same with r moved by 2^-46 |y| either way, that is the definition's value;
// otherwise (about one in 2^20) `sure` is cleared and the caller takes fp64.  (r is subtracted: for acc = 0 it is +0, so
// that the result keeps the sign of y, -0 under a negative w.)  (In fp64 throughout, the fp64 and
// conversion units bound the product: 2048 x 50288 x 2048 took 215 us of 133 us without an epilogue.)
// s and w in [2^-40, 2^40] (ordinary) keep every term normal; s = 0 gives acc = 0.
__device__ __forceinline__ bool ordinary(float s) { return fabsf(s) >= 0x1p-40f && fabsf(s) <= 0x1p40f; }
// Two at once; ns = -s and nw = -w spare the negations.
__device__ __forceinline__ void scaled(uint32_t acc0, uint32_t acc1, f2 s, f2 ns, f2 w, f2 nw, bool& sure, float& out0,
                                       float& out1) {
  const float x0 = (float)(int)acc0, x1 = (float)(int)acc1;
  const f2 x = pack2(x0, x1), t = pack2(0x1p-46f, 0x1p-46f), nt = pack2(-0x1p-46f, -0x1p-46f), minus = pack2(-1.0f, -1.0f);
  const f2 np = mul2(x, ns), e = fma2(x, s, np);
  const f2 y = mul2(np, nw), r = fma2(e, nw, fma2(np, w, y));
  const f2 lo = fma2(fma2(y, t, r), minus, y), hi = fma2(fma2(y, nt, r), minus, y);
  float hi0, hi1;
  unpack2(lo, out0, out1);
  unpack2(hi, hi0, hi1);
  sure = sure && out0 == hi0 && out1 == hi1 && fabsf(x0) < 0x1p24f && fabsf(x1) < 0x1p24f;
}

template <typename Y, int CG_, bool RESIDENT_ = false>
struct LinearPolicy {
  static constexpr int CG = CG_;
  static constexpr bool RESIDENT = RESIDENT_;  // one to four tokens, quantized here
  static constexpr bool W_EARLY = true, W_IS_A = true, A_MN = false;
  static constexpr int EPI_WARPS = 16, PARTS = EPI_WARPS / 4, EPI_COLS = BN_MAX / PARTS;  // columns of a warp
  struct Args {
    CUtensorMap map_a, map_b;  // W, codes
    RowArgs r;
    Common c;
    ResidentArgs x;       // RESIDENT: the tokens, else
    const double* s_tok;  // [M] their scales
    const float* s_row;   // [V]
    Y* y;
    int64_t ldy;
    int32_t* acc;         // [M][V] or NULL
    int V;
  };
  static __device__ __forceinline__ bool tile(const Args& a, int j, Tile& t) { return row_tile<CG, true, CG == 2>(a.r, j, t); }
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
  static constexpr int EPI_SMEM = EPI_WARPS * EPI_COLS * 8 + (int)sizeof(ResidentScratch);
  static_assert(EPI_WARPS == RES_WARPS, "the epilogue's warps quantize");
  struct Epilogue {
    ResidentScratch* res;  // RESIDENT: holds the tokens' scales
    int part, lane, r;  // r: lane of the tile
    float* s;           // scales of this warp's columns (chunks of 16: part, part + PARTS, ..), then negated
    float sw;
    bool plain;         // the warp's scales are of ordinary size
    __device__ __forceinline__ Epilogue(const Args&, unsigned char* sm, int q, int part_, int lane_)
        : res(reinterpret_cast<ResidentScratch*>(sm + EPI_WARPS * EPI_COLS * 8)), part(part_), lane(lane_), r(q * 32 + lane_),
          s(reinterpret_cast<float*>(sm) + (part_ * 4 + q) * 2 * EPI_COLS) {}
    __device__ __forceinline__ void write_b(const Args& a, unsigned char* b, int warp) {
      if (!RESIDENT) return;
      if (a.x.x_type == DFSSM_BF16) resident_quantize<__nv_bfloat16>(a.x, b, res, warp, lane);
      else resident_quantize<float>(a.x, b, res, warp, lane);
    }
    __device__ __forceinline__ void prepare(const Args& a, const Tile& t) {
      sw = r < t.na ? ld_f32(a.s_row + t.a0 + r) : 1.0f;
      bool ok = ordinary(sw);
#pragma unroll
      for (int k = 0; k < EPI_COLS / 32; ++k) {
        const int i = k * 32 + lane, c = ((i >> 4) * PARTS + part) * 16 + (i & 15);
        const float st = c < t.nb ? (RESIDENT ? res->s[c] : (float)a.s_tok[t.b0 + c]) : 1.0f;
        s[i] = st;
        s[EPI_COLS + i] = -st;
        ok = ok && (ordinary(st) || st == 0.0f);
      }
      plain = __all_sync(0xffffffffu, ok);
    }
    __device__ __forceinline__ void tile(const Args& a, const Tile& t, uint32_t taddr) {
      const int row = t.a0 + r;
      const bool rv = r < t.na;
      uint32_t v[16];
      const float* st = s;
      const f2 w2 = pack2(sw, sw), nw2 = pack2(-sw, -sw);
      Y* yp = a.y + (int64_t)(t.b0 + part * 16) * a.ldy + row;
      const uint32_t ld = (uint32_t)a.ldy;
      if (part * 16 < t.nb) tmem_ld16(taddr + (uint32_t)(part * 16), v);
#pragma unroll 1
      for (int c = part * 16; c < t.nb; c += 16 * PARTS, st += 16) {
        tmem_wait(v);
        const int n = min(16, t.nb - c);
        if (a.acc) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (rv && j < n) a.acc[(int64_t)(t.b0 + c + j) * a.V + row] = (int)v[j];
        }
        float out[16];
        bool sure = plain;
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 s4 = *reinterpret_cast<const float4*>(st + j), n4 = *reinterpret_cast<const float4*>(st + EPI_COLS + j);
          scaled(v[j], v[j + 1], pack2(s4.x, s4.y), pack2(n4.x, n4.y), w2, nw2, sure, out[j], out[j + 1]);
          scaled(v[j + 2], v[j + 3], pack2(s4.z, s4.w), pack2(n4.z, n4.w), w2, nw2, sure, out[j + 2], out[j + 3]);
        }
        if (!sure) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            out[j] = __double2float_rn(dmul(dmul(int_to_f64((int)v[j]), (double)st[j]), (double)sw));
        }
        if (c + 16 * PARTS < t.nb) tmem_ld16(taddr + (uint32_t)(c + 16 * PARTS), v);  // the next chunk, while this one is stored
        if (rv && n == 16) {
#pragma unroll
          for (int j = 0; j < 16; ++j) yp[(uint64_t)ld * j] = (Y)out[j];
        } else if (rv) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j < n) yp[(uint64_t)ld * j] = (Y)out[j];
        }
        yp += 16 * PARTS * a.ldy;
      }
      __syncwarp();  // the scales are read: the next tile's may be written
    }
    __device__ __forceinline__ void finish(const Args&) {}
  };
};

inline size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

template <typename Y, int CG, bool RESIDENT>
int launch_linear(const int8_t* W, const float* s_row, int V, const RowsQuantArgs& qa, void* y, int64_t ldy, int32_t* acc,
                  int* err, cudaStream_t st) {
  using P = LinearPolicy<Y, CG, RESIDENT>;
  const int M = qa.M, d = qa.d;
  typename P::Args a{};
  a.r.rows_a = V;
  a.r.rows_b = M;
  a.r.kblocks = (d + BK - 1) / BK;
  // one tile of tokens: W streams through once, in balanced ranges of rows.  More: whole tiles, the tokens' index
  // fastest.
  const bool range = M <= BN_MAX;
  a.r.mode = range ? kRangeA : kGrid;
  a.r.tile_b = range ? BN_MAX : even_tile((V + BM * CG - 1) / (BM * CG), M, max_groups<P>());
  a.r.box_a = range ? 32 : BM;
  const int bt = RESIDENT ? RES_ROWS : range ? (M + 16 * CG - 1) / (16 * CG) * 16 : a.r.tile_b / CG;  // a CTA's columns
  a.r.box_b = bt;
  a.c.b_tile = bt;
  a.c.resident = RESIDENT ? resident_bytes(d) : 0;
  a.c.stages = ring_stages(a.c, P::EPI_SMEM);
  a.c.err = err;
  a.x = ResidentArgs{qa.x, qa.x_type, qa.ldx, M, d, qa.norm_w, qa.dbg_q, qa.dbg_s};
  a.s_tok = qa.s;
  a.s_row = s_row;
  a.y = static_cast<Y*>(y);
  a.ldy = ldy;
  a.acc = acc;
  a.V = V;
  if (!encode_u8_map_sw128(&a.map_a, W, V, d, a.r.box_a)) return DFSSM_EUNSUPPORTED;
  cudaError_t e = cudaSuccess;
  if (!RESIDENT) {
    if (!encode_u8_map_sw128(&a.map_b, qa.q, M, d, bt)) return DFSSM_EUNSUPPORTED;
    e = launch_rows_quant(qa, st);
  }
  const long long units = range ? (V + 31) / 32
                                : (long long)((V + BM * CG - 1) / (BM * CG)) * ((M + a.r.tile_b - 1) / a.r.tile_b);
  const int most = max_groups<P>();
  if (e == cudaSuccess) e = launch<P>(a, (int)(units < most ? units : most), P::EPI_SMEM, st);
  return e == cudaSuccess ? DFSSM_OK : record_cuda_failure(e);
}

// One to four tokens: one kernel does it all; up to 128 the stream of W bounds the product and single CTAs keep more of it
// in flight; above, pairs halve the traffic of the tokens' codes.  (50288 x 2048, single against pairs: 65 tokens 25.5 / 26.3
// us, 128 28.6 / 28.8, 192 32.5 / 32.4, 256 37.9 / 35.7; 20011 x 1040: 65 13.9 / 15.7, 256 22.1 / 20.0.)
template <typename Y>
int launch_linear(const int8_t* W, const float* s_row, int V, const RowsQuantArgs& qa, void* y, int64_t ldy, int32_t* acc,
                  int* err, cudaStream_t st) {
  const auto f = resident_supported(qa.M, qa.d) ? launch_linear<Y, 1, true>
                 : qa.M <= 128                  ? launch_linear<Y, 1, false>
                                                : launch_linear<Y, 2, false>;
  return f(W, s_row, V, qa, y, ldy, acc, err, st);
}

}  // namespace

// [status word][codes M x d][scales f64 M]
size_t linear_int8_workspace_bytes(int M, int d) {
  return kStatusBytes + al256((size_t)M * d) + al256(sizeof(double) * (size_t)M);
}

}  // namespace dfssm

extern "C" int dfssm_linear_int8(const int8_t* W, const float* s_row, int V, int d, const void* x, int x_type,
                                 int64_t ldx, int M, const float* norm_w, void* y, int y_type, int64_t ldy,
                                 void* workspace, size_t ws_bytes, const dfssm_debug_t* dbg, void* stream) {
  using namespace dfssm;
  int st = check_int8_matrix(W, V, d);
  if (st) return st;
  if (!s_row || ldy < V || (y_type != DFSSM_F32 && y_type != DFSSM_BF16)) return DFSSM_EINVAL;
  st = check_tokens(M);
  if (st) return st;
  if (ldy > INT32_MAX) return DFSSM_EUNSUPPORTED;
  if (M == 0) return DFSSM_OK;
  st = check_rows(x, x_type, ldx, d);
  if (st) return st;
  if (!y) return DFSSM_EINVAL;
  const auto al = [](const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; };
  if (!al(s_row, 4) || !al(norm_w, 16) || !al(y, y_type == DFSSM_F32 ? 4 : 2)) return DFSSM_EALIGN;
  if (dbg && (!al(dbg->xq, 8) || !al(dbg->xscale, 4) || !al(dbg->acc, 4))) return DFSSM_EALIGN;
  if (!workspace || !al(workspace, 256) || ws_bytes < linear_int8_workspace_bytes(M, d)) return DFSSM_EWORKSPACE;
  if (!device_ok()) return DFSSM_EDEVICE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* p = static_cast<char*>(workspace);
  RowsQuantArgs qa{};
  qa.x = x;
  qa.x_type = x_type;
  qa.ldx = ldx;
  qa.M = M;
  qa.d = d;
  qa.norm_w = norm_w;
  qa.q = reinterpret_cast<int8_t*>(p + kStatusBytes);
  qa.s = reinterpret_cast<double*>(p + kStatusBytes + al256((size_t)M * d));
  if (dbg) {
    qa.dbg_q = dbg->xq;
    qa.dbg_s = dbg->xscale;
  }
  const auto f = y_type == DFSSM_F32 ? launch_linear<float> : launch_linear<__nv_bfloat16>;
  return f(W, s_row, V, qa, y, ldy, dbg ? dbg->acc : nullptr, reinterpret_cast<int*>(p), s);
}
