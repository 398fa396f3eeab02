// Int8 matrix product on the 5th-generation tensor cores, shared by the many-token operators: a
// persistent, warp-specialised main loop (TMA producer, MMA issuer, epilogue warps) around a policy P
// that says which tiles a CTA works on, how a K step is loaded and what becomes of the accumulators.
//
//   D[lanes][n columns] (int32, exact) = sum over K of A[lane][k] B[column][k]   (int8, both K-major)
//
// P::CG CTAs (1 or 2) work on a tile of 128 CG lanes x up to 256 columns: K steps of 128 bytes through a ring
// of shared-memory stages, two accumulators of 256 tensor-memory columns, so that a tile's epilogue runs while
// the next tile's products accumulate.  A pair (CG = 2, a cluster) splits both operands: each CTA loads and
// holds 128 lanes of A and half of B's columns, and one cta_group::2 product reads both halves.  What the
// product waits for at these sizes is the stream from L2: one CTA's 128 x 256 tile moves 48 KB a K step, at
// which it ran at 1350 TOPS (2048 x 50288 x 2048); a pair moves 32 KB per CTA.
//
// Every wait on an mbarrier is bounded: a wait that runs out of budget sets the status word, the CTA stops
// issuing work, waits (bounded) for its copies and products in flight, frees its tensor memory and returns.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "rows.cuh"
#include "umma.cuh"

namespace dfssm {
namespace gemm_i8 {

constexpr int BM = 128;      // lanes of a tile per CTA
constexpr int BN_MAX = 256;  // columns of a tile at most (the MMA's N)
constexpr int BK = 128;      // K bytes of a stage
constexpr int UMMA_K = 32;   // K bytes of one kind::i8 MMA
constexpr int A_BYTES = BM * BK;
constexpr int MAX_STAGES = 12;
constexpr int SMEM_LIMIT = 232448;  // 227 KB: the shared memory a CTA may have, all of it dynamic here
constexpr int BAR_BYTES = 256;
constexpr int TMEM_COLS = 2 * BN_MAX;

// Epilogue warps P::EPI_WARPS (8 or 16): `parts` of them share a quadrant of 32 lanes, part p taking the chunks p,
// p + parts, .. of a tile's columns.
template <class P>
constexpr int threads() { return (2 + P::EPI_WARPS) * 32; }

// One output tile: lanes a0 .. a0 + na, columns b0 .. b0 + nb, K steps kb0 .. kb1.  Policies give the whole
// tile (128 CG lanes); loads and epilogues see the CTA's own 128 lanes of it.
struct Tile {
  int a0, na, b0, nb;
  int kb0, kb1;
  int aux;  // the policy's own
};

// a / b of numbers that are short nearly always: every warp divides for every tile, and a 64-bit division is a hundred
// instructions.
__host__ __device__ __forceinline__ long long quotient(long long a, int b) {
  return (a >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Columns of the product: nb rounded up to what the instruction (16) and an even split over a pair (2 x 16) need.
template <int CG>
__device__ __forceinline__ int mma_n(int nb) { return (nb + 16 * CG - 1) & ~(16 * CG - 1); }

// kind::i8 instruction descriptor: D s32, A and B s8, B and (unless a_mn) A K-major, M = 128 CG, N = n.
template <int CG>
__device__ __forceinline__ uint32_t idesc(int n, bool a_mn) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)((BM * CG) >> 4) << 24);
}
template <int CG>
__device__ __forceinline__ void umma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t id,
                                     uint32_t accum) {
  if (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(id), "r"(accum)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(id), "r"(accum)
        : "memory");
}
// Arrival on the barrier (of both CTAs of a pair) when the products issued so far are complete.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if (CG == 1)
    umma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// The shared::cluster address of a barrier in the pair's first CTA.
template <int CG>
__device__ __forceinline__ uint32_t leader_bar(uint64_t* bar) {
  if (CG == 1) return smem_u32(bar);
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(bar)), "r"(0));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Copies into this CTA's shared memory, counted on the barrier at the shared::cluster address `bar` (of the pair's
// first CTA).
template <int CG>
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
// 32 lanes x 16 / 32 columns of tensor memory, one lane per thread (to be awaited with tmem_wait).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
      "%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Waits for the tensor-memory loads issued so far; the registers named are not used before.
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// The TMA copies of an operand's K step kb: n boxes of `box` rows of 128 bytes at (x + kb dx, y + kb dy + i box).
struct Boxes {
  const CUtensorMap* map;
  int n, box, y, dx, dy, x = 0;
};

// What every policy's arguments start with.
struct Common {
  int b_tile;   // columns a stage of one CTA has room for
  int resident; // bytes of B kept in shared memory for all of K instead (P::RESIDENT; a multiple of 1024)
  int stages;
  int* err;     // status word: kDeviceTimeout after a wait ran out of budget
};
__host__ __device__ inline int stage_bytes(const Common& c) {
  return A_BYTES + (c.resident ? 0 : c.b_tile * BK);
}
// Ring depth beside epi_bytes of epilogue scratch, and the shared memory it takes.
inline int ring_stages(const Common& c, int epi_bytes) {
  const int n = (SMEM_LIMIT - 1024 - BAR_BYTES - c.resident - epi_bytes) / stage_bytes(c);
  return n < MAX_STAGES ? n : MAX_STAGES;
}
inline size_t smem_bytes(const Common& c, int epi_bytes) {
  return 1024 + (size_t)c.resident + (size_t)c.stages * stage_bytes(c) + BAR_BYTES + epi_bytes;
}

// Position in the ring of stages: the stage, the parity of its phase, and how often the ring went round.
struct Ring {
  int s, stages, round;
  uint32_t phase;
  __device__ __forceinline__ explicit Ring(int n) : s(0), stages(n), round(0), phase(0u) {}
  __device__ __forceinline__ void next() {
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
      round = 1;
    }
  }
};

// What of a pair's tile belongs to this CTA of it.
template <int CG>
__device__ __forceinline__ Tile own_tile(Tile t, int rank) {
  if (CG == 2) {
    t.a0 += rank * BM;
    t.na = max(0, min(BM, t.na - rank * BM));
  }
  return t;
}

// (Converged warp; `leader` is one lane of it.)
template <int CG>
__device__ __forceinline__ void issue(const Boxes& o, int kb, unsigned char* dst, uint32_t bar, bool leader) {
  for (int i = 0; i < o.n; ++i)
    if (leader) tma_load<CG>(dst + i * o.box * BK, o.map, o.x + kb * o.dx, o.y + kb * o.dy + i * o.box, bar);
}

// With PDL the kernel may start while the one that writes the tokens' codes still runs: with W_EARLY the first round
// of W, whose codes are written before the call is enqueued, is requested without waiting for it.  Returns the number
// of K steps.  (Converged warp.)
template <class P>
__device__ __forceinline__ int request_w(const typename P::Args& ar, unsigned char* smem, uint64_t* full,
                                         uint32_t full_bar, int rank, bool leader) {
  if (!P::W_EARLY) return 0;
  constexpr int CG = P::CG;
  const int sbytes = stage_bytes(ar.c);
  int n = 0;
  Tile pt;
  for (int j = 0; n < ar.c.stages && P::tile(ar, j, pt); ++j) {
    const Tile t = own_tile<CG>(pt, rank);
    const uint32_t bytes = P::bytes(ar, pt);
    const Boxes w = P::W_IS_A ? P::boxes_a(ar, t, rank) : P::boxes_b(ar, t, rank);
    for (int kb = t.kb0; kb < t.kb1 && n < ar.c.stages; ++kb, ++n) {
      if (rank == 0 && leader) mbar_expect_tx(&full[n], bytes);
      issue<CG>(w, kb, smem + (size_t)n * sbytes + (P::W_IS_A ? 0 : A_BYTES), full_bar + 8 * n, leader);
    }
  }
  return n;
}

template <class P>
__global__ void __launch_bounds__(threads<P>(), 1) gemm_i8_kernel(const __grid_constant__ typename P::Args ar) {
  constexpr int CG = P::CG;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // aligned by an offset from the array itself, so that every access stays a shared-memory access
  unsigned char* resident = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* smem = resident + ar.c.resident;
  const int stages = ar.c.stages, sbytes = stage_bytes(ar.c);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + (size_t)stages * sbytes);  // [stages] TMA -> MMA
  uint64_t* empty = full + MAX_STAGES;      // [stages] MMA -> producer
  uint64_t* acc_full = empty + MAX_STAGES;  // [2] MMA -> epilogue
  uint64_t* acc_empty = acc_full + 2;       // [2] epilogue (of both CTAs) -> MMA
  uint64_t* mma_done = acc_empty + 2;       // every MMA of this CTA complete
  uint64_t* b_ready = mma_done + 1;         // a resident B is written: epilogue -> MMA
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(b_ready + 1);
  volatile int& abort_flag = *reinterpret_cast<volatile int*>(tmem_holder + 1);
  unsigned char* epi_smem = smem + (size_t)stages * sbytes + BAR_BYTES;
  static_assert((2 * MAX_STAGES + 6) * 8 + 8 <= BAR_BYTES, "barrier area");
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)(blockIdx.x & 1u) : 0;  // within the pair (a cluster of two consecutive CTAs)
  int early = 0;  // K steps whose W was requested ahead

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], P::EPI_WARPS * CG);
    }
    mbar_init(mma_done, 1);
    mbar_init(b_ready, P::EPI_WARPS);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    __syncwarp();
    if (CG == 1) early = request_w<P>(ar, smem, full, smem_u32(full), 0, elect_one());  // while tensor memory is allocated
  }
  if (warp == 1) {
    if (CG == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                   "r"(TMEM_COLS)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                   "r"(TMEM_COLS)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (CG == 2) cluster_sync();  // the other CTA's barriers are ready
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem_base = *tmem_holder;
  if (threadIdx.x == 0) pdl_launch_dependents();

  if (warp == 0) {
    // ---- producer: each tile's K steps through the stage ring (converged, like the MMA issuer)
    const bool leader = elect_one();
    const uint32_t full_bar = leader_bar<CG>(full);
    if (CG == 2) early = request_w<P>(ar, smem, full, full_bar, rank, leader);
    if (!P::RESIDENT) pdl_wait();  // with a resident B it loads W alone
    Ring ring(stages);
    bool ok = true;
    Tile pt;
    for (int j = 0; ok && P::tile(ar, j, pt); ++j) {
      const Tile t = own_tile<CG>(pt, rank);
      const uint32_t bytes = P::bytes(ar, pt);  // of the whole tile's K step, both CTAs'
      const Boxes a = P::boxes_a(ar, t, rank), b = P::boxes_b(ar, t, rank);
      for (int kb = t.kb0; kb < t.kb1; ++kb, ring.next()) {
        const int s = ring.s;
        if (ring.round > 0 && !mbar_wait_warp(&empty[s], ring.phase ^ 1u, &abort_flag)) {
          abort_flag = 1;
          ok = false;
          break;
        }
        const bool late = ring.round == 0 && s < early;  // its W is under way
        if (rank == 0 && leader && !late) mbar_expect_tx(&full[s], bytes);
        unsigned char* st = smem + (size_t)s * sbytes;
        if (!(late && P::W_IS_A)) issue<CG>(a, kb, st, full_bar + 8 * s, leader);
        if (!P::RESIDENT && !(late && !P::W_IS_A)) issue<CG>(b, kb, st + A_BYTES, full_bar + 8 * s, leader);
      }
    }
    // the last copies land before this CTA may exit (those of a pair's second CTA are counted by the first, which
    // the cluster barrier at the end waits for; after an abort they get a millisecond)
    __syncwarp();
    if (lane == 0 && rank == 0) {
      // the stage's last copy has the phase of the ring's current round, or of the one before
      for (int i = 0; i < stages; ++i) {
        if (i < ring.s) mbar_wait_drain(&full[i], ring.phase);
        else if (ring.round > 0) mbar_wait_drain(&full[i], ring.phase ^ 1u);
      }
    } else if (!ok) {
      const long long t0 = clock64();
      while (clock64() - t0 < 2000000LL) {
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---- MMA issuer: the warp stays converged and one lane issues, so that descriptors are formed in uniform
    // registers.  What a K step takes here has to stay below the product's 512 clocks, also while the epilogue
    // warps compete for issue slots: with divisions and per-thread operands it took up to 890.
    Ring ring(stages);
    int local = 0;
    bool ok = true, issued = false;
    Tile t;
    const bool leader = elect_one();
    const uint32_t smem0 = smem_u32(smem);
    const uint64_t a_desc = P::adesc(smem0), b_desc = P::bdesc(ar, P::RESIDENT ? smem_u32(resident) : smem0 + A_BYTES);
    const uint64_t a_step = P::a_step(), b_step = P::b_step(ar);  // 32 bytes of K on, in 16-byte units
    if (P::RESIDENT && !mbar_wait_warp(b_ready, 0, &abort_flag)) {
      abort_flag = 1;
      ok = false;
    }
    for (; ok && P::tile(ar, local, t); ++local) {
      const int buf = local & 1;
      if (local >= 2 && !mbar_wait_warp(&acc_empty[buf], ((local >> 1) - 1) & 1, &abort_flag)) {
        abort_flag = 1;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t d_tmem = tmem_base + (uint32_t)(buf * BN_MAX);
      const uint32_t id = idesc<CG>(mma_n<CG>(t.nb), P::A_MN);
      uint32_t accum = 0u;
      for (int kb = t.kb0; kb < t.kb1; ++kb, ring.next()) {
        if (!mbar_wait_warp(&full[ring.s], ring.phase, &abort_flag)) {
          abort_flag = 1;
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t off = (uint64_t)((uint32_t)(ring.s * sbytes) >> 4);
        const uint64_t ad = a_desc + off;
        const uint64_t bd = b_desc + (P::RESIDENT ? (uint64_t)((uint32_t)(kb * ar.c.b_tile * BK) >> 4) : off);
        if (leader) {
          umma<CG>(d_tmem, ad, bd, id, accum);
          umma<CG>(d_tmem, ad + a_step, bd + b_step, id, 1u);
          umma<CG>(d_tmem, ad + 2 * a_step, bd + 2 * b_step, id, 1u);
          umma<CG>(d_tmem, ad + 3 * a_step, bd + 3 * b_step, id, 1u);
          commit<CG>(&empty[ring.s]);
        }
        accum = 1u;
        issued = true;
      }
      if (!ok) break;
      if (leader) commit<CG>(&acc_full[buf]);
    }
    // every MMA this warp issued completes before the tensor memory is released
    if (issued) {
      if (leader) commit<CG>(mma_done);
      mbar_wait_drain(mma_done, 0);
    }
  } else if (warp >= 2) {
    // ---- epilogue: warp drains TMEM lanes [32 (warp % 4), +32)
    pdl_wait();
    typename P::Epilogue epi(ar, epi_smem, warp & 3, (warp - 2) >> 2, lane);
    if (P::RESIDENT) {
      epi.write_b(ar, resident, warp - 2);
      // written by the generic proxy, read by the tensor core through the async one
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b_ready)) : "memory");
      mbar_wait_warp(b_ready, 0, &abort_flag);  // every warp's part, as the epilogues read the scales
    }
    int local = 0;
    Tile t;
    for (; P::tile(ar, local, t); ++local) {
      const int buf = local & 1;
      const Tile own = own_tile<CG>(t, rank);
      epi.prepare(ar, own);  // what the tile needs from memory, fetched while its products run
      if (abort_flag || !mbar_wait(&acc_full[buf], (local >> 1) & 1, &abort_flag)) {
        abort_flag = 1;
        break;
      }
      __syncwarp();
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      epi.tile(ar, own, tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(buf * BN_MAX));
      // this warp's reads of the accumulator are complete
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      // (relaxed: the loads are complete, and a release would wait for this tile's stores as well)
      if (lane == 0)
        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         leader_bar<CG>(&acc_empty[buf]))
                     : "memory");
    }
    __syncwarp();
    epi.finish(ar);
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (CG == 2) cluster_sync();  // neither CTA's shared or tensor memory goes while the other may reach it
  if (abort_flag && threadIdx.x == 0) atomicExch(ar.c.err, kDeviceTimeout);
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (CG == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS) : "memory");
  }
}

// Launch of `groups` CTAs or pairs.
template <class P>
cudaError_t launch(const typename P::Args& a, int groups, int epi_smem, cudaStream_t st) {
  const auto k = gemm_i8_kernel<P>;
  const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(k), SMEM_LIMIT);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(P::CG, k, dim3(groups * P::CG), dim3(threads<P>()), smem_bytes(a.c, epi_smem), st, a);
}
// Groups that run at a time: one CTA per SM.
template <class P>
int max_groups() { return num_sms() / P::CG; }

// Columns of a tile for `cols` columns times `rows` tile rows on `groups` groups: of the widths 128 .. 256 the one whose
// fullest group has the fewest columns to do (with 32 for each tile's start and end), the widest of equals.
inline int even_tile(int rows, int cols, int groups) {
  int best = BN_MAX;
  long long least = -1;
  for (int w = BN_MAX; w >= 128; w -= 32) {
    const long long tiles = (long long)rows * ((cols + w - 1) / w), cost = (tiles + groups - 1) / groups * (w + 32);
    if (least < 0 || cost < least) {
      least = cost;
      best = w;
    }
  }
  return best;
}

// ------------------------------------------------------------------ row-major operands through TMA
// Both operands are row-major int8 matrices with K contiguous, loaded as 128-byte-swizzled boxes of 128 bytes
// of K (bytes past a row's end and rows past the last read as zero).  The rows of one operand are the
// tokens, of the other the matrix W.
enum Mode {
  kGrid = 0,    // whole tiles, strided over the groups, the token index fastest (W read once)
  kRangeA = 1,  // every group takes a balanced range of A rows (W) in units of 32, and all columns (one tile)
  kRangeB = 2   // every group takes a balanced range of B rows (W), and for it all tiles of A rows (tokens)
};
struct RowArgs {
  int mode;
  int rows_a, rows_b;
  int tile_b;        // columns of a whole tile
  int kblocks;
  int box_a, box_b;  // rows of one TMA box of each operand
  int b_first;       // first B row of the product (a piece of the vocabulary); rows_b counts from there
};

// W_IS_A: kRangeA, otherwise kRangeB, for the mode that is not kGrid; GRID = false leaves kGrid out (what a short
// kernel has to fetch of its own code counts: the loss of 7 tokens took 31 us with it, 28 without).
template <int CG, bool W_IS_A, bool GRID = true>
__device__ __forceinline__ bool row_tile(const RowArgs& r, int j, Tile& t) {
  constexpr int TA = BM * CG;
  const int group = blockIdx.x / CG, groups = gridDim.x / CG;
  t.kb0 = 0;
  t.kb1 = r.kblocks;
  const int ta = (r.rows_a + TA - 1) / TA;
  if (GRID && r.mode == kGrid) {
    const int tb = (r.rows_b + r.tile_b - 1) / r.tile_b;
    const long long i = group + (long long)j * groups;
    if (i >= (long long)ta * tb) return false;
    const int by = W_IS_A ? tb : ta, q = (int)quotient(i, by), m = (int)(i - (long long)q * by);
    const int ia = W_IS_A ? q : m;
    const int ib = W_IS_A ? m : q;
    t.a0 = ia * TA;
    t.b0 = ib * r.tile_b;
    t.na = min(TA, r.rows_a - t.a0);
    t.nb = min(r.tile_b, r.rows_b - t.b0);
    return true;
  }
  const int rows_w = W_IS_A ? r.rows_a : r.rows_b;
  const long long units = (rows_w + 31) / 32;
  const int w0 = (int)quotient(units * group, groups) * 32;
  const int w1 = min((int)quotient(units * (group + 1), groups) * 32, rows_w);
  if (W_IS_A) {
    t.a0 = w0 + TA * j;
    if (t.a0 >= w1) return false;
    t.na = min(TA, w1 - t.a0);
    t.b0 = 0;
    t.nb = r.rows_b;
    return true;
  }
  const int nt = (w1 - w0 + r.tile_b - 1) / r.tile_b;
  if (nt == 0 || j >= nt * ta) return false;
  t.a0 = (j / nt) * TA;
  t.na = min(TA, r.rows_a - t.a0);
  t.b0 = w0 + (j % nt) * r.tile_b;
  t.nb = min(r.tile_b, w1 - t.b0);
  return true;
}

// One K step: whole boxes of A up to the tile's last lane, and B's columns (half of them each in a pair).
template <int CG, bool RESIDENT = false>
__device__ __forceinline__ uint32_t row_bytes(const RowArgs& r, const Tile& t) {
  int n = mma_n<CG>(t.nb) / CG;
  n = RESIDENT ? 0 : (n + r.box_b - 1) / r.box_b * r.box_b * CG;
#pragma unroll
  for (int i = 0; i < CG; ++i) {
    const int na = max(0, min(BM, t.na - i * BM));
    n += (na + r.box_a - 1) / r.box_a * r.box_a;
  }
  return (uint32_t)n * BK;
}
template <int CG>
__device__ __forceinline__ Boxes row_boxes_a(const RowArgs& r, const CUtensorMap* map, const Tile& t) {
  return Boxes{map, (t.na + r.box_a - 1) / r.box_a, r.box_a, t.a0, BK, 0};
}
template <int CG>
__device__ __forceinline__ Boxes row_boxes_b(const RowArgs& r, const CUtensorMap* map, const Tile& t, int rank) {
  const int half = mma_n<CG>(t.nb) / CG;
  return Boxes{map, (half + r.box_b - 1) / r.box_b, r.box_b, r.b_first + t.b0 + rank * half, BK, 0};
}

// ------------------------------------------------------------------ few tokens, quantized by every CTA
// B is one to four tokens: every CTA quantizes them itself (as the single-token head does; codes and scales of
// rows_quant.cu) into the 128-byte swizzled layout the product reads, [K / 128][16 rows][128] bytes, while its first
// rows of W are on their way.  The epilogue's sixteen warps are split evenly over the tokens and keep their values in
// registers, which bounds M d.  (With a warp per token for 16 tokens this took longer than a launch: 47 us for 28.)
constexpr int RES_ROWS = 16, RES_TOKENS = 4, RES_WARPS = 16, RES_CHUNKS = 4;
inline bool resident_supported(int M, int d) {
  const int per = M == 1 ? 16 : M == 2 ? 8 : 4;  // warps per token
  return M <= RES_TOKENS && d <= per * 256 * RES_CHUNKS;
}
inline int resident_bytes(int d) { return (d + BK - 1) / BK * RES_ROWS * BK; }
struct ResidentArgs {
  const void* x;
  int x_type;
  int64_t ldx;
  int M, d;
  const float* norm_w;
  int8_t* dbg_q;  // optional taps, written by the first CTA
  float* dbg_s;
};
struct ResidentScratch {
  double ss[RES_WARPS];
  uint32_t m[RES_WARPS];
  float rn[RES_TOKENS], s[RES_TOKENS];  // s: the tokens' scales
};
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, %0;" ::"n"(RES_WARPS * 32) : "memory"); }
template <typename T>
__device__ __forceinline__ void resident_quantize(const ResidentArgs& r, unsigned char* res, ResidentScratch* sc, int w,
                                                  int lane) {
  const int per = r.M == 1 ? 16 : r.M == 2 ? 8 : 4, t = w / per, first = t * per;
  const bool on = t < r.M;
  const T* x = reinterpret_cast<const T*>(r.x) + (on ? t : 0) * r.ldx;
  const int i0 = ((w - first) * 32 + lane) * 8, step = per * 256;
  float v[RES_CHUNKS][8];
#pragma unroll
  for (int c = 0; c < RES_CHUNKS; ++c) {
    if (on && i0 + c * step < r.d) {
      load8<T>(x + i0 + c * step, v[c]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[c][k] = 0.0f;
    }
  }
  if (r.norm_w) {
    double ss = 0.0;  // exact squares in fp64
#pragma unroll
    for (int c = 0; c < RES_CHUNKS; ++c)
      if (c * step < r.d) {
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fma((double)v[c][k], (double)v[c][k], ss);
      }
    ss = warp_sum(ss);
    if (lane == 0) sc->ss[w] = ss;
    epilogue_sync();
    if (w == first) {
      ss = warp_sum(lane < per ? sc->ss[first + lane] : 0.0);
      if (lane == 0 && on) sc->rn[t] = rms_factor(ss, r.d);
    }
    epilogue_sync();
    if (on) {
      const float rn = sc->rn[t];
#pragma unroll
      for (int c = 0; c < RES_CHUNKS; ++c)
        if (i0 + c * step < r.d) {
          float nw[8];
          load8<float>(r.norm_w + i0 + c * step, nw);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[c][k] = norm_value(v[c][k], rn, nw[k]);
        }
    }
  }
  uint32_t mb = 0u;  // absmax as an unsigned pattern: infinities and NaN order above every finite value
#pragma unroll
  for (int c = 0; c < RES_CHUNKS; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) mb = max(mb, __float_as_uint(v[c][k]) & 0x7FFFFFFFu);
  mb = __reduce_max_sync(0xffffffffu, mb);
  if (lane == 0) sc->m[w] = mb;
  epilogue_sync();
  if (!on) return;
  mb = 0u;
  for (int k = 0; k < per; ++k) mb = max(mb, sc->m[first + k]);
  const bool finite = mb < 0x7F800000u;
  const float s0 = finite ? quant_scale(__uint_as_float(mb)) : __uint_as_float(0x7FC00000u);
  const float inv = finite ? quant_inv(s0) : 0.0f;
  if (w == first && lane == 0) {
    sc->s[t] = s0;
    if (r.dbg_s && blockIdx.x == 0) r.dbg_s[t] = s0;
  }
#pragma unroll
  for (int c = 0; c < RES_CHUNKS; ++c) {
    const int i = i0 + c * step;
    if (i >= r.d) continue;
    int cd[8];
    quant_codes<8>(v[c], s0, inv, cd);
    const uint2 o = finite ? pack_codes(cd) : make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(res + (i >> 7) * (RES_ROWS * BK) + t * BK + ((((i & 127) >> 4) ^ (t & 7)) << 4) + (i & 8)) = o;
    if (r.dbg_q && blockIdx.x == 0) *reinterpret_cast<uint2*>(r.dbg_q + (size_t)t * r.d + i) = o;
  }
}

}  // namespace gemm_i8
}  // namespace dfssm
