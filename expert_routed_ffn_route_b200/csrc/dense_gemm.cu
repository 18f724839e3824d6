// The dense gated feed-forward block on the tensor cores, forward and backward, for 16-bit
// weights and any number of rows:
//
//   forward    gate/up   g = Wg x, u = Wu x, h = act(g) u        one kernel; g, u kept in fp32
//                                                                when a backward pass follows
//              down      y = Wd h
//   backward   gate grad dh = Wd^T dy, dg = dh u act'(g), du = dh act(g), h again   one kernel
//              grads     dx = Wg^T dg + Wu^T du, dWg = dg x^T, dWu = du x^T, dWd = dy h^T
//                        one launch over the tiles of all four products
//
// h, dg and du are rounded to the block's 16-bit type because they are the next product's
// operands; dh never leaves the accumulators, and g and u are kept in fp32: rounding them too
// would add a second error of the same size to every gradient.
//
// One kernel, three epilogues. A pair of CTAs (a cluster of two, tcgen05 cta_group::2) computes
// D[256 x BN] tiles, K in steps of 64 (128 bytes, 128-byte swizzle): each CTA brings its own 128
// rows of A and half of B's columns by TMA, the leader's MMA warp issues tcgen05.mma kind::f16
// (M = 256, N = BN) over both, and each CTA's TMEM receives its 128 rows, in one of two
// accumulators while the epilogue warps empty the other. Why pairs: an SM takes in about 47
// bytes a cycle from L2 (measured at every tile width, at full clock), a 128 x 256 tile of one CTA would need 96
// at the MMA's full rate (it reached 967 TFLOP/s on a 4096 x 2560 x 10240 forward pass), a pair's
// 256 x 256 tile needs 64: at full clock the intake binds at 73 % of the tensor peak, where the
// measured library GEMM is too; under the power cap (1.6 GHz) the tensor pipe is 83 % busy.
// An operand is read as it lies in memory: with K contiguous (x, dy, h, dg, du and the forward
// weights) or with K as the slow dimension (the weights of dh and dx, and both operands of the
// weight gradients), as the MMA's "K-major" or "MN-major" operand; no transposed copies are
// made. In a gate/up tile one CTA brings gate rows and the other up rows, so the accumulator
// holds BN / 2 columns of each.
//
// Epilogue: results (and the kept g and u) move between registers and memory as 32-row blocks in
// TMA's swizzle, so that each byte crosses shared memory once each way; the MMA and the copies
// already use most of its 128 bytes a cycle (16 epilogue warps instead of 8, or blocks moved by
// the warps themselves, slowed the products: gate gradient 316 and 264 us against 214).
//
// Schedule: static, a tile at a time to each pair, longest products first. Tiles left over by
// the last full round are split along K over the idle pairs: each part leaves its fp32 sums in
// the workspace and the epilogue warp that arrives last (a counter per warp) adds the parts in
// order, so results do not depend on timing and no CTA waits for another.
//
// Roles (11 warps): warps 0 and 10 TMA of A and of B (one thread for both needed 500 cycles a step,
// the MMA 2 BN), warp 1 TMEM and (leader) MMA, warps 2..9 epilogue (two warps a TMEM lane
// quarter, each half of the columns). Every wait is bounded; one that gives up sets
// the status word and its site, and every role stops.
//
// Measured on one B200 (kernel time in graphs / in a steady loop under the power cap): forward of
// 4096 rows, 2560 x 10240, 422 / 490..500 us (1527 / 1300 TFLOP/s; 1631 and 1375 are the measured
// library peaks), training step 1.39 / 1.62..1.68 ms (1387 / 1170).
#include <cstring>

#include "dense.cuh"
#include "tc_common.cuh"

namespace moe {

namespace {

constexpr int kBM = 128, kBK = 64;    // rows of one CTA, K values of a step
constexpr int kPairM = 2 * kBM;
constexpr int kEpiWarps = 8, kWarpB = 2 + kEpiWarps;  // warp kWarpB: B's producer
constexpr int kGemmThreads = 32 * (kWarpB + 1);
constexpr int kMaxProblems = 4, kMaxPhases = 5;
constexpr int kMaxPairs = 74;         // CTA pairs of a launch (148 SMs)
constexpr int kGroupM = 16;           // row tiles walked together, for reuse in L2
constexpr int kSmemBytes = 227 * 1024;
static_assert(kFfnCounters == 2 * kMaxPairs * 2 * kEpiWarps, "a counter a warp of every cut tile");

enum Epi { EPI_STORE = 0, EPI_GATED = 1, EPI_GRAD = 2 };

// One product D[M][N] = sum over up to two K segments of A_s B_s.
struct GemmProblem {
  CUtensorMap a[2], b[2];  // per segment (EPI_GATED: b[0] gate, b[1] up, both of segment 0)
  int M, N;                // N: output columns (EPI_GATED: of h)
  int kt[2];               // K steps of each segment
  int a_mn, b_mn;          // operand stored with K as the slow dimension
  int b_early;             // B may be read before the kernel ahead has ended
  int tiles_m, tiles_n, first;
};

// A run of `count` tiles from `first` on, each cut into `splits` K parts, dealt out in turn to
// the pairs lo .. lo + n - 1. Cut tiles use the counters from `slot` on and the partial sums from
// `unit` on.
struct Phase {
  int first, count, splits, lo, n, slot, unit;
};

struct GemmArgs {
  GemmProblem p[kMaxProblems];
  Phase ph[kMaxPhases];
  int n, n_phases;
  CUtensorMap o[5];   // outputs by problem (EPI_STORE); h, g, u (EPI_GATED); g, u, h, dg, du
  float* partial;     // [unit][rank][BN * 128]
  int32_t* counters;  // [slot][rank][warp], zero between launches
  int keep;           // EPI_GATED: write g and u
  int hold;           // test control: the issuer gives up at its first wait
  int32_t* status;
};

template <int BN, int EPI> struct GemmCfg {
  static constexpr int A_BYTES = kBM * 128;
  static constexpr int B_BYTES = BN / 2 * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;  // one CTA's share
  // output columns of an epilogue warp, and of one of its blocks
  static constexpr int COLS = EPI == EPI_GATED ? BN / 4 : BN / 2;
  static constexpr int CH = EPI == EPI_GRAD ? 16 : EPI == EPI_GATED ? (COLS < 32 ? COLS : 32)
                                                                     : (COLS < 64 ? COLS : 64);
  // a warp's buffer: 32 rows of a block; the gate gradient's g and u (2048 bytes each) and
  // three outputs (1024 each)
  static constexpr int EPI_BYTES = EPI == EPI_GRAD ? 7168 : 4096;
  static constexpr int NS = (kSmemBytes - 2048 - kEpiWarps * EPI_BYTES) / STAGE;
  static constexpr int SMEM = NS * STAGE + kEpiWarps * EPI_BYTES + 2048;
  static_assert(NS >= 4 && STAGE % 1024 == 0 && EPI_BYTES % 1024 == 0 && SMEM <= kSmemBytes, "shared memory");
};

// The units of one pair, in order.
struct Unit {
  int p, mt, nt;       // problem, tile
  int k0, k1;          // K steps
  int splits, part;
  int slot, unit;      // partial sums: tile and unit
};

struct Walk {
  int ph, idx, pair;
  __device__ __forceinline__ explicit Walk(int pair_) : ph(0), idx(-1), pair(pair_) {}
  // The next unit; false after the last.
  __device__ __forceinline__ bool next(const GemmArgs& a, Unit* u) {
    while (ph < a.n_phases) {
      const Phase& f = a.ph[ph];
      const int mine = pair - f.lo;
      if (mine >= 0 && mine < f.n) {
        idx = idx < 0 ? mine : idx + f.n;
        if (idx < f.count * f.splits) break;
      }
      ++ph;
      idx = -1;
    }
    if (ph >= a.n_phases) return false;
    const Phase& f = a.ph[ph];
    const unsigned local = f.splits == 1 ? idx : (unsigned)idx / (unsigned)f.splits;
    const int t = f.first + (int)local;
    u->splits = f.splits;
    u->part = idx - (int)local * f.splits;
    u->slot = f.slot + (int)local;
    u->unit = f.unit + idx;
    u->p = 0;
#pragma unroll
    for (int i = 1; i < kMaxProblems; ++i)
      if (i < a.n && t >= a.p[i].first) u->p = i;
    const GemmProblem& q = a.p[u->p];
    const unsigned l = t - q.first;
    const unsigned b = l / (unsigned)(kGroupM * q.tiles_n), r = l - b * (kGroupM * q.tiles_n);
    const unsigned rows = min(kGroupM, q.tiles_m - (int)b * kGroupM);
    u->nt = r / rows;
    u->mt = b * kGroupM + (r - u->nt * rows);
    const int steps = q.kt[0] + q.kt[1];
    u->k0 = 0;
    u->k1 = steps;
    if (f.splits > 1) {
      u->k0 = (unsigned)(steps * u->part) / (unsigned)f.splits;
      u->k1 = (unsigned)(steps * (u->part + 1)) / (unsigned)f.splits;
    }
    return true;
  }
};

// Shared-memory descriptor of an operand stored with K as the slow dimension, 128-byte
// swizzle: blocks of 64 values along M or N (rows of 128 bytes, one a K value) 8192 bytes
// apart (the leading offset), groups of 8 K values 1024 bytes apart (the stride offset).
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(8192 >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;  // version
  d |= (uint64_t)2 << 61;  // SWIZZLE_128B
  return d;
}

// D[tmem] (+)= A B over both CTAs of the pair; issued by one elected lane of the leader.
__device__ __forceinline__ void umma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Commit of the issued MMAs to the same barrier of both CTAs.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void umma_commit_leader(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The leader's copy of a shared-memory address.
__device__ __forceinline__ uint32_t leader_addr(const void* p) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
// Relaxed: what it hands over are accumulator columns (ordered by the tcgen05 fence before it).
// A release at cluster scope would wait for the warp's global stores, 14,000 cycles a tile of
// the gate gradient (measured).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
// Tile load into this CTA's shared memory, counted on the leader's barrier.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// 16 TMEM columns of this thread's lane, without waiting for them.
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Eight fp32 values as 16 bytes of the 16-bit type.
template <bool F16> __device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack16x2<F16>(v[0], v[1]), pack16x2<F16>(v[2], v[3]), pack16x2<F16>(v[4], v[5]),
                    pack16x2<F16>(v[6], v[7]));
}

// 16-byte chunk c of row r in a block of 32 rows x 16 C bytes in shared memory, as TMA's swizzle
// of that row length lays it out; free of bank conflicts for a lane a row.
template <int C> __device__ __forceinline__ int block_at(int r, int c) {
  return (r * C + (c ^ ((r / (8 / C)) & (C - 1)))) * 16;
}
// A block to global memory by TMA (which leaves out what lies past the edges), and into it.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0,
                                             int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the last N groups of this thread's stores have read their source / are complete.
template <int N> __device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <int BN, int EPI, bool F16, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ GemmArgs a) {
  using C = GemmCfg<BN, EPI>;
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte alignment by the address inside the CTA's window, so that both CTAs of a pair
  // have the same layout
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* epi = smem + C::NS * C::STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + kEpiWarps * C::EPI_BYTES);  // [NS] (leader's)
  uint64_t* empty = full + C::NS;                                         // [NS]
  uint64_t* acc_full = empty + C::NS;                                     // [2]
  uint64_t* acc_empty = acc_full + 2;                                     // [2] (leader's used)
  uint64_t* pre_full = acc_empty + 2;                                     // [kEpiWarps]
  uint64_t* drain = pre_full + kEpiWarps;                                 // [1]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1;

  if (warp == 2 && lane < a.n) {  // the maps of the first copies
    prefetch_map(&a.p[lane].a[0]);
    prefetch_map(&a.p[lane].b[EPI == EPI_GATED ? rank : 0]);
  }
  if (warp == 3 && lane < (EPI == EPI_STORE ? a.n : EPI == EPI_GATED ? (a.keep ? 3 : 1) : 5))
    prefetch_map(&a.o[lane]);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    for (int w = 0; w < kEpiWarps; ++w) mbar_init(&pre_full[w], 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 2 * BN);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Launched before the kernel ahead has ended, whatever it is: nothing that another kernel may
  // write or read is touched before this wait. The next kernel may then set itself up on the SMs
  // that are free.
  // (B's producer waits at its first operand that the kernel ahead may write: a training step of 301
  // rows, 1032 x 2056, 55.0 us, 56.8 when it waits here.)
  if (warp != kWarpB) {
    pdl_wait();
    pdl_trigger();
  }
  auto fail = [&](int site) {
    set_timeout(a.status, site);
    *abort_flag = 1;
  };
  Walk walk(pair);
  Unit u;

  // The ring's stage and phase, counted along by the producers and the issuer.
  struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
      if (++s == C::NS) {
        s = 0;
        phase ^= 1;
      }
    }
  } ring;

  if (warp == 0 || warp == kWarpB) {
    // ------------------------------------------------------------ producers (both CTAs): A, B
    if (lane == 0) {
      const bool is_a = warp == 0;
      const uint32_t stage0 = smem_u32(smem) + (is_a ? 0 : C::A_BYTES);
      const uint32_t full0 = leader_addr(&full[0]);
      int it = 0;
      bool ok = true, waited = is_a;
      while (ok && !*abort_flag && walk.next(a, &u)) {
        const GemmProblem& q = a.p[u.p];
        // first row (column) of this CTA's share; gate/up: all gate rows in the leader, all up
        // rows in its peer
        const int m0 = is_a                 ? u.mt * kPairM + rank * kBM
                       : EPI == EPI_GATED   ? u.nt * (BN / 2)
                                            : u.nt * BN + rank * (BN / 2);
        const bool mn = is_a ? q.a_mn : EPI != EPI_GATED && q.b_mn;
        const int boxes = mn ? (is_a ? kBM : BN / 2) / 64 : 1;
        const int kt0 = q.kt[0];
        if (!waited && !q.b_early) {
          pdl_wait();
          waited = true;
        }
        for (int k = u.k0; k < u.k1; ++k, ++it, ring.next()) {
          if (!mbar_wait(&empty[ring.s], ring.phase ^ 1)) {  // (a new barrier passes parity 1)
            ok = false;
            break;
          }
          const int seg = k >= kt0;
          const int kk = (seg ? k - kt0 : k) * kBK;
          const CUtensorMap* map = is_a ? &q.a[seg] : &q.b[EPI == EPI_GATED ? rank : seg];
          const uint32_t dst = stage0 + ring.s * C::STAGE, bar = full0 + 8 * ring.s;
          if (is_a && rank == 0) mbar_arrive_expect_tx(&full[ring.s], 2 * C::STAGE);
          if (mn) {
            tma_load_pair(dst, map, m0, kk, bar);
            if (boxes > 1) tma_load_pair(dst + 8192, map, m0 + 64, kk, bar);
          } else {
            tma_load_pair(dst, map, kk, m0, bar);
          }
        }
      }
      if (!ok) fail(50);
      // every issued stage lands before the pair may exit (the leader waits for all shares; after a
      // timeout one may lack a share that another producer no longer brought: it uses the bound up,
      // the rest is only looked at)
      long long left = kWaitCycles;
      if (rank == 0 && is_a)
        for (int j = 0; j < min(it, C::NS); ++j, ring.next()) {
          // the last use of each stage, oldest first
          const bool wrapped = it > C::NS;
          const int s = wrapped ? ring.s : j;
          if (!mbar_wait_within(&full[s], wrapped ? ring.phase ^ 1 : 0, left)) left = 0;
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (rank == 0) {
      int tile = 0;
      bool aborted = a.hold != 0;
      const uint32_t stage0 = smem_u32(smem);
      for (; !aborted && walk.next(a, &u); ++tile) {
        const GemmProblem& q = a.p[u.p];
        // D fp32; A and B bf16 (1) or fp16 (0); majors; N; M
        const uint32_t idesc = (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) |
                               ((uint32_t)(q.a_mn != 0) << 15) | ((uint32_t)(q.b_mn != 0) << 16) |
                               ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(kPairM >> 4) << 24);
        const int b = tile & 1, buse = tile >> 1;
        if (buse > 0 && !mbar_wait(&acc_empty[b], (buse - 1) & 1)) aborted = true;
        aborted = __any_sync(0xffffffffu, aborted || *abort_flag);
        if (aborted) break;
        tc_fence_after();
        const uint32_t dacc = tmem + b * BN;
        const uint64_t astep = q.a_mn ? 2048 >> 4 : 32 >> 4, bstep = q.b_mn ? 2048 >> 4 : 32 >> 4;
        // descriptors of stage 0; a stage is STAGE / 16 further on
        const uint64_t ad0 = q.a_mn ? umma_desc_mn_sw128(stage0) : umma_desc_sw128(stage0);
        const uint64_t bd0 = q.b_mn ? umma_desc_mn_sw128(stage0 + C::A_BYTES)
                                    : umma_desc_sw128(stage0 + C::A_BYTES);
        for (int k = u.k0; k < u.k1; ++k, ring.next()) {
          const bool ok = mbar_wait(&full[ring.s], ring.phase);
          if (!__all_sync(0xffffffffu, ok)) {
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint64_t off = (uint64_t)(ring.s * (C::STAGE >> 4));
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            umma_f16_pair(dacc, ad0 + off + kk * astep, bd0 + off + kk * bstep, idesc,
                          (k > u.k0 || kk > 0) ? 1u : 0u);
          umma_commit_pair(&empty[ring.s]);
        }
        if (aborted) break;
        umma_commit_pair(&acc_full[b]);
      }
      if (aborted) fail(51);
      // all issued MMAs complete before TMEM and shared memory are released
      umma_commit_leader(drain);
      mbar_wait(drain, 0);
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..9)
    const int quarter = warp & 3;      // TMEM lanes 32 * quarter .. + 31
    const int half = (warp - 2) >> 2;  // which half of the columns
    constexpr int COLS = C::COLS, CH = C::CH;
    constexpr int ACC = BN / 2;        // accumulator columns a warp
    uint8_t* buf = epi + (warp - 2) * C::EPI_BYTES;
    const uint32_t acc_empty_leader[2] = {leader_addr(&acc_empty[0]), leader_addr(&acc_empty[1])};
    const auto first_row = [&](const Unit& v) {
      return v.mt * kPairM + rank * kBM + quarter * 32;
    };
    const auto first_col = [&](const Unit& v) {
      return v.nt * (EPI == EPI_GATED ? BN / 2 : BN) + half * COLS;
    };
    // The gate gradient's g and u of a block into the buffer (lane 0 issues).
    uint64_t* in_bar = &pre_full[warp - 2];
    uint32_t in_phase = 0;
    bool in_flight = false;
    auto fetch = [&](int m, int n) {
      if (lane == 0) {
        mbar_arrive_expect_tx(in_bar, 4096);
        tma_load_2d(buf, &a.o[0], n, m, in_bar);
        tma_load_2d(buf + 2048, &a.o[1], n, m, in_bar);
      }
      in_flight = true;
    };
    int tile = 0;
    Unit un;
    bool more = walk.next(a, &un);
    if (EPI == EPI_GRAD && more) fetch(first_row(un), first_col(un));
    // (whole warps go on or stop: the TMEM loads are warp-wide)
    for (; more && !__any_sync(0xffffffffu, *abort_flag); ++tile) {
      u = un;
      more = walk.next(a, &un);
      const GemmProblem& q = a.p[u.p];
      const int b = tile & 1;
      const int m0 = first_row(u), n0 = first_col(u);
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[b], (tile >> 1) & 1))) {
        fail(52);
        break;
      }
      tc_fence_after();
      const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16) + b * BN + half * COLS;
      // Accumulator column i (0..15) of chunk c of this warp: gate/up chunks are 16 gate columns,
      // then 16 up columns.
      auto acc_addr = [&](int c) -> uint32_t {
        if constexpr (EPI == EPI_GATED)
          return lane_addr + ((c & 16) ? BN / 2 : 0) + (c >> 5) * 16;
        else
          return lane_addr + c;
      };
      // A part of a split tile: this warp's sums into the workspace, 16 bytes a lane and row of
      // 512 bytes; the warp that brings the last part goes on with the sum of all.
      const float4* parts = nullptr;
      auto hand_back = [&]() {  // the accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty_leader[b]);
      };
      bool mine = m0 < q.M && n0 < q.N;  // (rows or columns past the edges: nothing to do)
      if (!mine) {
        hand_back();
      } else if (u.splits > 1) {
        const size_t unit_f4 = (size_t)2 * kEpiWarps * (ACC / 4) * 32;
        const size_t my = ((size_t)rank * kEpiWarps + (warp - 2)) * (ACC / 4) * 32 + lane;
        float4* base = reinterpret_cast<float4*>(a.partial);
        float4* dst = base + (size_t)u.unit * unit_f4 + my;
        constexpr int NC = ACC < 64 ? ACC / 16 : 4;  // chunks of 16 columns at a time
#pragma unroll 1
        for (int c = 0; c < ACC; c += 16 * NC) {
          uint32_t r[NC][16];
#pragma unroll
          for (int i = 0; i < NC; ++i) tmem_ld16_async(acc_addr(c + 16 * i), r[i]);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              __stcg(dst + (c / 4 + 4 * i + j) * 32,
                     make_float4(__uint_as_float(r[i][4 * j]), __uint_as_float(r[i][4 * j + 1]),
                                 __uint_as_float(r[i][4 * j + 2]),
                                 __uint_as_float(r[i][4 * j + 3])));
        }
        fence_acq_rel_gpu();
        __syncwarp();
        int last = 0;
        if (lane == 0) {
          int32_t* cnt = a.counters + ((size_t)u.slot * 2 + rank) * kEpiWarps + (warp - 2);
          last = atomicAdd(cnt, 1) == u.splits - 1;
          if (last) *cnt = 0;
          fence_acq_rel_gpu();
        }
        last = __shfl_sync(0xffffffffu, last, 0);
        __syncwarp();
        parts = base + (size_t)(u.unit - u.part) * unit_f4 + my;
        hand_back();
        mine = last;
      }
      if (!mine) {
        if (EPI == EPI_GRAD && more) {  // the block in the buffer is not this warp's to finish
          if (!__all_sync(0xffffffffu, mbar_wait(in_bar, in_phase))) {
            fail(53);
            break;
          }
          in_phase ^= 1;
          fetch(first_row(un), first_col(un));
        }
        continue;
      }
      // NC chunks of 16 accumulator columns from chunk column c on: from TMEM, or the sum of the
      // parts (all loads of a part in flight at once)
      auto load = [&](int c, auto& r) {
        constexpr int NC = sizeof(r) / 64;
        if (!parts) {
#pragma unroll
          for (int i = 0; i < NC; ++i) tmem_ld16_async(acc_addr(c + 16 * i), r[i]);
          tmem_wait_ld();
          return;
        }
        const size_t unit_f4 = (size_t)2 * kEpiWarps * (ACC / 4) * 32;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) r[i][j] = 0;  // 0.f
        for (int k = 0; k < u.splits; ++k) {
          float4 w[NC][4];
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[i][j] = __ldcg(parts + k * unit_f4 + (c / 4 + 4 * i + j) * 32);
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float v[4] = {w[i][j].x, w[i][j].y, w[i][j].z, w[i][j].w};
#pragma unroll
              for (int l = 0; l < 4; ++l)
                r[i][4 * j + l] = __float_as_uint(__uint_as_float(r[i][4 * j + l]) + v[l]);
            }
        }
      };
      // the accumulator is free once its last columns are read (a split tile's already is)
      auto release = [&]() {
        if (!parts) hand_back();
      };
      // The buffer's previous block has been read; then, after this lane's part is written, the
      // block may be stored.
      auto buffer_free = [&]() {
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
      };
      auto buffer_full = [&]() {
        fence_proxy_async();
        __syncwarp();
      };
      if constexpr (EPI == EPI_STORE) {
#pragma unroll 1
        for (int c = 0; c < COLS; c += CH) {
          uint32_t r[CH / 16][16];
          load(c, r);
          if (c + CH == COLS) release();
          buffer_free();
#pragma unroll
          for (int i = 0; i < CH / 8; ++i)
            *reinterpret_cast<uint4*>(buf + block_at<CH / 8>(lane, i)) =
                pack8<F16>(reinterpret_cast<const float*>(&r[i / 2][8 * (i & 1)]));
          buffer_full();
          if (lane == 0 && m0 < q.M && n0 + c < q.N) {
            tma_store_2d(&a.o[u.p], buf, n0 + c, m0);
            bulk_commit();
          }
        }
      } else if constexpr (EPI == EPI_GATED) {
#pragma unroll 1
        for (int c = 0; c < COLS; c += CH) {
          uint32_t r[CH / 8][16];  // 16 gate, 16 up columns, and so on
          load(2 * c, r);
          if (c + CH == COLS) release();
          const bool inside = m0 < q.M && n0 + c < q.N;
          if (a.keep) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              buffer_free();
#pragma unroll
              for (int i = 0; i < CH / 4; ++i) {
                const uint32_t* v = &r[2 * (i / 4) + k][4 * (i & 3)];
                *reinterpret_cast<uint4*>(buf + block_at<CH / 4>(lane, i)) =
                    make_uint4(v[0], v[1], v[2], v[3]);
              }
              buffer_full();
              if (lane == 0 && inside) {
                tma_store_2d(&a.o[1 + k], buf, n0 + c, m0);
                bulk_commit();
              }
            }
          }
          uint4 o4[CH / 8];
#pragma unroll
          for (int i = 0; i < CH / 8; ++i) {
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              o[j] = act_value<ACT>(__uint_as_float(r[2 * (i / 2)][8 * (i & 1) + j])) *
                     __uint_as_float(r[2 * (i / 2) + 1][8 * (i & 1) + j]);
            o4[i] = pack8<F16>(o);
          }
          buffer_free();
#pragma unroll
          for (int i = 0; i < CH / 8; ++i)
            *reinterpret_cast<uint4*>(buf + block_at<CH / 8>(lane, i)) = o4[i];
          buffer_full();
          if (lane == 0 && inside) {
            tma_store_2d(&a.o[0], buf, n0 + c, m0);
            bulk_commit();
          }
        }
      } else {
        // Blocks of 16 columns. The next block's g and u (of the next unit, at the end) are on
        // their way while this one is worked on.
        bool ok = true;
#pragma unroll 1
        for (int c = 0; c < COLS; c += 16) {
          uint32_t r[1][16];
          load(c, r);
          if (c + 16 == COLS) release();
          ok = __all_sync(0xffffffffu, mbar_wait(in_bar, in_phase));
          if (!ok) break;
          in_phase ^= 1;
          in_flight = false;
          float4 g4[4], u4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            g4[i] = *reinterpret_cast<const float4*>(buf + block_at<4>(lane, i));
            u4[i] = *reinterpret_cast<const float4*>(buf + 2048 + block_at<4>(lane, i));
          }
          // the reads above are done before the next block is written over them (__syncwarp
          // alone orders no asynchronous copy: the block then arrived too early now and then)
          fence_proxy_async();
          __syncwarp();
          if (c + 16 < COLS) fetch(m0, n0 + c + 16);
          else if (more) fetch(first_row(un), first_col(un));
          float o[3][16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float gv[4] = {g4[i].x, g4[i].y, g4[i].z, g4[i].w};
            const float uv[4] = {u4[i].x, u4[i].y, u4[i].z, u4[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float dh = __uint_as_float(r[0][4 * i + j]);
              float av, dav;
              act_grad<ACT>(gv[j], &av, &dav);
              o[0][4 * i + j] = av * uv[j];
              o[1][4 * i + j] = dh * uv[j] * dav;
              o[2][4 * i + j] = dh * av;
            }
          }
          buffer_free();
#pragma unroll
          for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              *reinterpret_cast<uint4*>(buf + 4096 + k * 1024 + block_at<2>(lane, i)) =
                  pack8<F16>(&o[k][8 * i]);
          buffer_full();
          if (lane == 0 && m0 < q.M && n0 + c < q.N) {
#pragma unroll
            for (int k = 0; k < 3; ++k)
              tma_store_2d(&a.o[2 + k], buf + 4096 + k * 1024, n0 + c, m0);
            bulk_commit();
          }
        }
        if (!ok) {
          fail(53);
          break;
        }
      }
    }
    // copies in flight end before the CTA may
    if (EPI == EPI_GRAD && in_flight) mbar_wait(in_bar, in_phase);
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * BN);
  }
}

// ------------------------------------------------------------------ host side

template <int BN, int EPI, bool F16, int ACT>
cudaError_t launch_kernel(const GemmArgs& a, int pairs, cudaStream_t st) {
  using C = GemmCfg<BN, EPI>;
  auto kern = ffn_gemm_kernel<BN, EPI, F16, ACT>;
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(kern), done);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int BN, int EPI>
cudaError_t launch_types(const GemmArgs& a, bool f16, int act, int pairs, cudaStream_t st) {
  constexpr int S = MOE_ACT_SILU, G = MOE_ACT_GELU;
  if (EPI == EPI_STORE || act == S)
    return f16 ? launch_kernel<BN, EPI, true, S>(a, pairs, st)
               : launch_kernel<BN, EPI, false, S>(a, pairs, st);
  if constexpr (EPI != EPI_STORE)
    return f16 ? launch_kernel<BN, EPI, true, G>(a, pairs, st)
               : launch_kernel<BN, EPI, false, G>(a, pairs, st);
  return cudaErrorInvalidValue;
}

struct Operand {
  const void* base;  // row-major [rows][cols]
  uint64_t rows, cols;
  bool mn;  // K is the rows
};

// One product on the host: up to two segments.
struct Product {
  Operand a[2], b[2];
  int K[2];
  int M, N;
  void* out;
  bool b_early;  // see GemmProblem
};

bool operand_map(CUtensorMap* m, const Operand& o, bool f16, int rows_k_major) {
  const CUtensorMapDataType dt =
      f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return make_map(m, dt, 2, o.base, o.cols, o.rows, 64, o.mn ? 64 : rows_k_major,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

// Blocks of 32 rows x ch columns of a row-major [rows][cols] array; type: 0 bf16, 1 fp16, 2 fp32.
bool block_map(CUtensorMap* m, const void* base, int rows, int cols, int ch, int type) {
  const int size = type == 2 ? 4 : 2;
  const int bytes = ch * size;
  return make_map(m,
                  type == 2   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                  : type == 1 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                              : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  size, base, cols, rows, ch, 32,
                  bytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                  : bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                : CU_TENSOR_MAP_SWIZZLE_32B);
}

// The schedule of a launch. Tile width and K splits by estimated cycles, from measured launches: an
// SM takes in about 46 bytes a cycle (a step of 64 K values brings it (128 + BN / 2) * 128, more
// than the MMA's 2 BN cycles allow for at every width), and 16 of those that come from DRAM (an
// operand is counted once for all tiles that share it; in forward launches alone, which is a fit
// and no model: counted for the gradients too, those of 64 rows of 2560 x 10240 take 94 us instead
// of 91). A tile takes 1500 more
// to start and drain, a split one 6000 + 20 BN for the fences and the count, 8 BN to write and
// 5.5 BN a part to read. With and without the terms 20 BN and DRAM: forward, 64 rows of 2560 x 10240
// 51.7 / 58.3 us, 301 rows of 4096 x 2048 30.7 / 35.2; gradients, 301 rows of 4096 x 2048 50.4 / 57.0,
// but slower: forward, 40 rows of 1024 x 4096 21.9 / 20.3; gradients, 64 rows of 4096 x 2048 44.8 / 42.1
// and 200 of 2560 x 10240 100 / 96.
struct GemmPlan {
  Phase ph[kMaxPhases];
  int n_phases, bn, units, slots, pairs;
  int order[kMaxProblems];  // products, longest K first
  double cost;
};

// Cycles of a step that brings a CTA `cold` bytes from DRAM.
double step_cycles(int bn, double cold) {
  return std::max(std::max(2.0 * bn, (128 + bn / 2) * 128 / 46.0), cold / 16);
}

// Cycles of a tile of `steps` K steps in s parts; `used`: the share of the tile's area that holds
// results (the rest is not exchanged).
double tile_cycles(int steps, int s, int bn, double used, double cold) {
  return (steps + s - 1) / s * step_cycles(bn, cold) + 1500 +
         (s > 1 ? 6000 + (20 + 8 * used + 5.5 * s) * bn : 0);
}

// Cycles of `r` tiles on R idle pairs, split the best way.
double split_cost(int r, int steps, int R, int bn, double used, double cold, int* splits) {
  double best = -1;
  for (int s = 1; s <= std::min(std::min(R / r, steps), 16); ++s) {
    const double c = tile_cycles(steps, s, bn, used, cold);
    if (best < 0 || c < best) {
      best = c;
      *splits = s;
    }
  }
  return best;
}

GemmPlan plan_width(const Product* pr, int n, bool gated, int R, int bn) {
  GemmPlan g;
  std::memset(&g, 0, sizeof(g));
  g.bn = bn;
  g.pairs = R;
  int steps[kMaxProblems];
  long long tiles[kMaxProblems];
  const int cols = gated ? bn / 2 : bn;
  for (int i = 0; i < n; ++i) {
    steps[i] = (pr[i].K[0] + kBK - 1) / kBK + (pr[i].K[1] + kBK - 1) / kBK;
    tiles[i] = (long long)((pr[i].M + kPairM - 1) / kPairM) * ((pr[i].N + cols - 1) / cols);
    g.order[i] = i;
  }
  for (int i = 1; i < n; ++i)  // longest first, equal ones in order
    for (int j = i; j > 0 && steps[g.order[j]] > steps[g.order[j - 1]]; --j)
      std::swap(g.order[j], g.order[j - 1]);
  double cold = 0;
  if (!pr[0].b[0].mn)  // a forward launch: one product
    cold = 128.0 * 128 / ((pr[0].N + cols - 1) / cols) +
           bn / 2 * 128.0 / ((pr[0].M + kPairM - 1) / kPairM);
  // at most two lengths: the input gradient's and the weight gradients'
  long long count[2] = {0, 0};
  double area[2] = {0, 0};
  int len[2] = {steps[g.order[0]], 0};
  for (int i = 0; i < n; ++i) {
    const int o = g.order[i];
    const int c = steps[o] == len[0] ? 0 : 1;
    if (c) len[1] = steps[o];
    count[c] += tiles[o];
    area[c] += (double)pr[o].M * pr[o].N;
  }
  double used[2];
  for (int c = 0; c < 2; ++c) used[c] = count[c] ? area[c] / (count[c] * 256.0 * cols) : 1;
  int first = 0;
  const auto add = [&](long long cnt, int splits, int lo, int np) {
    if (cnt <= 0) return;
    Phase& f = g.ph[g.n_phases++];
    f.first = first;
    f.count = (int)cnt;
    f.splits = splits;
    f.lo = lo;
    f.n = np;
    f.slot = g.slots;
    f.unit = g.units;
    if (splits > 1) {
      g.slots += (int)cnt;
      g.units += (int)cnt * splits;
    }
    first += (int)cnt;
  };
  // cnt tiles of length c over all pairs: whole rounds, then the rest split
  const auto rounds_cost = [&](long long cnt, int c, int* s) {
    const int rest = (int)(cnt % R);
    return cnt / R * tile_cycles(len[c], 1, bn, 1, cold) +
           (rest ? split_cost(rest, len[c], R, bn, used[c], cold, s) : 0);
  };
  const auto rounds = [&](long long cnt, int c) {
    int s = 1;
    g.cost += rounds_cost(cnt, c, &s);
    const long long rest = cnt % R;
    add(cnt - rest, 1, 0, R);
    add(rest, s, 0, (int)rest * s);
  };
  const int e = (int)(count[0] % R);
  if (!e || !count[1]) {
    rounds(count[0], 0);
    if (count[1]) rounds(count[1], 1);
    return g;
  }
  // The leftover long tiles (in parts or not) beside rounds of short tiles on the other pairs, or
  // split over all pairs before them. A step of 301 rows, 1032 x 2056 (10 long, 135 short tiles):
  // 59.6 us in parts beside, 63.5 over all pairs; 64 rows of 2560 x 1024: 49.8 and 55.5.
  int dummy = 1;
  double best = rounds_cost(e, 0, &dummy) + rounds_cost(count[1], 1, &dummy);
  int best_s = 0;
  long long best_beside = 0;
  const double small = tile_cycles(len[1], 1, bn, 1, cold);
  for (int s = 1; e * s < R && s <= std::min(len[0], 16); ++s) {
    const int others = R - e * s;
    const double t = tile_cycles(len[0], s, bn, used[0], cold);
    const long long want = std::max(1LL, (long long)(t / small + 0.5)) * others;
    const long long beside = std::min(want, count[1]);
    const double c = std::max(t, (beside + others - 1) / others * small) +
                     rounds_cost(count[1] - beside, 1, &dummy);
    if (c < best) {
      best = c;
      best_s = s;
      best_beside = beside;
    }
  }
  if (!best_s) {
    rounds(count[0], 0);
    rounds(count[1], 1);
    return g;
  }
  rounds(count[0] - e, 0);
  g.cost += best;
  add(e, best_s, 0, e * best_s);
  add(best_beside, 1, e * best_s, R - e * best_s);
  const double so_far = g.cost;
  rounds(count[1] - best_beside, 1);
  g.cost = so_far;
  return g;
}

// 64-column tiles need both operands with K contiguous: a pair's half of 32 columns is no whole
// 128-byte row of an operand that has K as the slow dimension.
GemmPlan plan_products(const Product* pr, int n, bool gated, int R) {
  bool mn = false;
  for (int i = 0; i < n; ++i) mn = mn || pr[i].b[0].mn;
  GemmPlan best = plan_width(pr, n, gated, R, 256);
  for (int bn = 128; bn >= (mn ? 128 : 64); bn /= 2) {
    const GemmPlan g = plan_width(pr, n, gated, R, bn);
    if (g.cost < best.cost) best = g;
  }
  return best;
}

size_t plan_bytes(const GemmPlan& g) { return (size_t)g.units * 2 * kBM * g.bn * sizeof(float); }

template <int EPI>
cudaError_t run_products(const Product* pr, int n, const FfnArgs& f, cudaStream_t st) {
  const int sms = device_sms();
  if (sms < 2) return cudaErrorInvalidDevice;
  const GemmPlan g = plan_products(pr, n, EPI == EPI_GATED, std::min(kMaxPairs, sms / 2));
  if (plan_bytes(g) > f.partial_bytes) return cudaErrorInvalidValue;
  const int bn = g.bn;
  GemmArgs a;
  std::memset(&a, 0, sizeof(a));
  a.n = n;
  int total = 0;
  for (int i = 0; i < n; ++i) {
    GemmProblem& q = a.p[i];
    const Product& s = pr[g.order[i]];
    q.M = s.M;
    q.N = s.N;
    q.a_mn = s.a[0].mn;
    q.b_mn = s.b[0].mn;
    q.b_early = s.b_early;
    const int segs = s.K[1] > 0 ? 2 : 1;
    for (int j = 0; j < segs; ++j) {
      q.kt[j] = (s.K[j] + kBK - 1) / kBK;
      if (!operand_map(&q.a[j], s.a[j], f.f16, kBM)) return cudaErrorInvalidValue;
    }
    const int n_b = EPI == EPI_GATED ? 2 : segs;
    for (int j = 0; j < n_b; ++j)
      if (!operand_map(&q.b[j], s.b[j], f.f16, bn / 2)) return cudaErrorInvalidValue;
    const int cols = EPI == EPI_GATED ? bn / 2 : bn;
    q.tiles_m = (s.M + kPairM - 1) / kPairM;
    q.tiles_n = (s.N + cols - 1) / cols;
    q.first = total;
    total += q.tiles_m * q.tiles_n;
  }
  std::memcpy(a.ph, g.ph, sizeof(a.ph));
  a.n_phases = g.n_phases;
  a.partial = f.partial;
  a.counters = f.counters;
  a.keep = f.pre != nullptr;
  a.hold = g_test_hold.hold;
  // outputs (and the gate gradient's inputs) by blocks of 32 rows
  const int cols = EPI == EPI_GATED ? bn / 4 : bn / 2;
  const int ch = EPI == EPI_GRAD ? 16 : std::min(cols, EPI == EPI_GATED ? 32 : 64);
  bool ok = true;
  if (EPI == EPI_STORE) {
    for (int i = 0; i < n; ++i) {
      const Product& s = pr[g.order[i]];
      ok = ok && block_map(&a.o[i], s.out, s.M, s.N, ch, f.f16 ? 1 : 0);
    }
  } else {
    const size_t rows_f = (size_t)f.T * f.f;
    const int in = EPI == EPI_GATED ? 1 : 0, first_out = EPI == EPI_GATED ? 0 : 2;
    if (f.pre)
      for (int k = 0; k < 2; ++k)
        ok = ok && block_map(&a.o[in + k], f.pre + k * rows_f, f.T, f.f, ch, 2);
    void* out[3] = {f.h, f.dg, f.du};
    for (int k = 0; k < (EPI == EPI_GATED ? 1 : 3); ++k)
      ok = ok && block_map(&a.o[first_out + k], out[k], f.T, f.f, ch, f.f16 ? 1 : 0);
  }
  if (!ok) return cudaErrorInvalidValue;
  a.status = f.status;
  int pairs = 0;
  for (int i = 0; i < g.n_phases; ++i)
    pairs = std::max(pairs, g.ph[i].lo + std::min(g.ph[i].n, g.ph[i].count * g.ph[i].splits));
  if (bn == 256) return launch_types<256, EPI>(a, f.f16, f.act, pairs, st);
  if (bn == 128) return launch_types<128, EPI>(a, f.f16, f.act, pairs, st);
  if constexpr (EPI != EPI_GRAD) return launch_types<64, EPI>(a, f.f16, f.act, pairs, st);
  return cudaErrorInvalidValue;
}

Operand k_major(const void* base, int rows, int cols) {
  return Operand{base, (uint64_t)rows, (uint64_t)cols, false};
}
Operand mn_major(const void* base, int rows, int cols) {
  return Operand{base, (uint64_t)rows, (uint64_t)cols, true};
}

Product gate_up_product(const FfnArgs& f) {
  Product p{};
  p.a[0] = k_major(f.x, f.T, f.d);
  p.b[0] = k_major(f.w_gate, f.f, f.d);
  p.b[1] = k_major(f.w_up, f.f, f.d);
  p.K[0] = f.d;
  p.M = f.T;
  p.N = f.f;
  return p;
}

Product down_product(const FfnArgs& f) {
  Product p{};
  p.a[0] = k_major(f.h, f.T, f.f);
  p.b[0] = k_major(f.w_down, f.d, f.f);
  p.K[0] = f.f;
  p.M = f.T;
  p.N = f.d;
  p.out = f.y;
  p.b_early = true;  // the kernel ahead is this block's gate/up kernel
  return p;
}

}  // namespace

size_t ffn_partial_bytes(bool backward) {
  return (size_t)(backward ? 2 : 1) * kMaxPairs * kPairM * 256 * sizeof(float);
}

cudaError_t launch_ffn_gate_up(const FfnArgs& f, cudaStream_t st) {
  const Product p = gate_up_product(f);
  return run_products<EPI_GATED>(&p, 1, f, st);
}

cudaError_t launch_ffn_down(const FfnArgs& f, cudaStream_t st) {
  const Product p = down_product(f);
  return run_products<EPI_STORE>(&p, 1, f, st);
}

cudaError_t launch_ffn_gate_grad(const FfnArgs& f, cudaStream_t st) {
  Product p{};
  p.a[0] = k_major(f.dy, f.T, f.d);
  p.b[0] = mn_major(f.w_down, f.d, f.f);
  p.K[0] = f.d;
  p.M = f.T;
  p.N = f.f;
  return run_products<EPI_GRAD>(&p, 1, f, st);
}

cudaError_t launch_ffn_grads(const FfnArgs& f, cudaStream_t st) {
  Product p[kMaxProblems] = {};
  int n = 0;
  if (f.dx) {
    Product& q = p[n++];
    q.a[0] = k_major(f.dg, f.T, f.f);
    q.a[1] = k_major(f.du, f.T, f.f);
    q.b[0] = mn_major(f.w_gate, f.f, f.d);
    q.b[1] = mn_major(f.w_up, f.f, f.d);
    q.K[0] = q.K[1] = f.f;
    q.M = f.T;
    q.N = f.d;
    q.out = f.dx;
    q.b_early = true;  // the kernel ahead is this block's gate-gradient kernel: it writes h, dg, du
  }
  const void* grad[3] = {f.dg, f.du, f.dy};
  void* out[3] = {f.dw_gate, f.dw_up, f.dw_down};
  for (int i = 0; i < 3; ++i) {
    if (!out[i]) continue;
    const int rows = i < 2 ? f.f : f.d, cols = i < 2 ? f.d : f.f;
    Product& q = p[n++];
    q.a[0] = mn_major(grad[i], f.T, rows);
    q.b[0] = mn_major(i < 2 ? f.x : f.h, f.T, cols);
    q.K[0] = f.T;
    q.M = rows;
    q.N = cols;
    q.out = out[i];
    q.b_early = i < 2;
  }
  return run_products<EPI_STORE>(p, n, f, st);
}

}  // namespace moe
