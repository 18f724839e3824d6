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
// One kernel, three epilogues. D[128 x BN] tiles, K in steps of 64 (128 bytes, 128-byte
// swizzle), both operands by TMA into a ring of stages, tcgen05.mma kind::f16 (M = 128,
// N = BN) issued by one warp into one of two TMEM accumulators while the epilogue warps empty
// the other. An operand is read as it lies in memory: with K contiguous (x, dy, h, dg, du and
// the forward weights) or with K as the slow dimension (the weights of dh and dx, and both
// operands of the weight gradients), as the MMA's "K-major" or "MN-major" operand; no
// transposed copies are made. Gate and up rows lie one behind the other in a stage, so a
// gate/up tile is one MMA whose accumulator holds BN / 2 gate and BN / 2 up columns.
//
// Roles (10 warps): warp 0 TMA, warp 1 TMEM and MMA, warps 2..9 epilogue (two warps a TMEM
// lane quarter, each half of the columns). Every wait is bounded; one that gives up sets the
// status word and its site, and every role stops.
#include <cstring>

#include "dense.cuh"
#include "tc_common.cuh"

namespace moe {

namespace {

constexpr int kBM = 128, kBK = 64;
constexpr int kGemmThreads = 320, kEpiWarps = 8;
constexpr int kMaxProblems = 4;
constexpr int kGroupM = 8;           // row tiles walked together, for reuse in L2
constexpr int kSmemBytes = 227 * 1024;

enum Epi { EPI_STORE = 0, EPI_GATED = 1, EPI_GRAD = 2 };

// One product D[M][N] = sum over up to two K segments of A_s B_s.
struct GemmProblem {
  CUtensorMap a[2], b[2];  // per segment (EPI_GATED: b[0] gate, b[1] up, both of segment 0)
  void* out;               // [M][N], 16-bit (EPI_STORE)
  int M, N;                // N: output columns (EPI_GATED: of h)
  int kt[2];               // K steps of each segment
  int a_mn, b_mn;          // operand stored with K as the slow dimension
  int tiles_m, tiles_n, first;
};

struct GemmArgs {
  GemmProblem p[kMaxProblems];
  int n, total;
  // gate/up and gate-gradient epilogues: rows of f elements
  float* pre;
  void* h;
  void* dg;
  void* du;
  int32_t* status;
};

template <int BN> struct GemmCfg {
  static constexpr int A_BYTES = kBM * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NS = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static_assert(NS * STAGE + 2048 <= kSmemBytes, "shared memory");
};

struct Tile {
  int p, m0, nt;
};

__device__ __forceinline__ Tile tile_at(const GemmArgs& a, int u) {
  Tile t;
  t.p = 0;
#pragma unroll
  for (int i = 1; i < kMaxProblems; ++i)
    if (i < a.n && u >= a.p[i].first) t.p = i;
  const GemmProblem& q = a.p[t.p];
  const int l = u - q.first;
  const int band = kGroupM * q.tiles_n;
  const int b = l / band, r = l - b * band;
  const int rows = min(kGroupM, q.tiles_m - b * kGroupM);
  t.nt = r / rows;
  t.m0 = (b * kGroupM + r % rows) * kBM;
  return t;
}

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

// D[tmem] (+)= A B, both operands in shared memory; issued by one elected lane.
__device__ __forceinline__ void umma_f16_warp(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
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

// 8 consecutive 16-bit results at `dst` (16-byte aligned).
template <bool F16> __device__ __forceinline__ void store8(void* dst, const float* v) {
  *static_cast<uint4*>(dst) = make_uint4(pack16x2<F16>(v[0], v[1]), pack16x2<F16>(v[2], v[3]),
                                         pack16x2<F16>(v[4], v[5]), pack16x2<F16>(v[6], v[7]));
}

template <int BN, int EPI, bool F16, int ACT>
__global__ void __launch_bounds__(kGemmThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ GemmArgs a) {
  using C = GemmCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::NS * C::STAGE);  // [NS]
  uint64_t* empty = full + C::NS;                                         // [NS]
  uint64_t* acc_full = empty + C::NS;                                     // [2]
  uint64_t* acc_empty = acc_full + 2;                                     // [2]
  uint64_t* drain = acc_empty + 2;                                        // [1]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 2 * BN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  auto fail = [&](int site) {
    set_timeout(a.status, site);
    *abort_flag = 1;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < a.total && ok && !*abort_flag; u += gridDim.x) {
        const Tile t = tile_at(a, u);
        const GemmProblem& q = a.p[t.p];
        for (int seg = 0; seg < 2 && ok; ++seg) {
          const int steps = q.kt[seg];
          for (int k = 0; k < steps; ++k, ++it) {
            const int s = it % C::NS, use = it / C::NS;
            if (use > 0 && !mbar_wait(&empty[s], (use - 1) & 1)) {
              ok = false;
              break;
            }
            uint8_t* as = smem + s * C::STAGE;
            uint8_t* bs = as + C::A_BYTES;
            mbar_arrive_expect_tx(&full[s], C::STAGE);
            if (q.a_mn) {
#pragma unroll
              for (int i = 0; i < kBM / 64; ++i)
                tma_load_2d(as + i * 8192, &q.a[seg], t.m0 + 64 * i, k * kBK, &full[s]);
            } else {
              tma_load_2d(as, &q.a[seg], k * kBK, t.m0, &full[s]);
            }
            if constexpr (EPI == EPI_GATED) {
              tma_load_2d(bs, &q.b[0], k * kBK, t.nt * (BN / 2), &full[s]);
              tma_load_2d(bs + BN / 2 * 128, &q.b[1], k * kBK, t.nt * (BN / 2), &full[s]);
            } else if (q.b_mn) {
#pragma unroll
              for (int i = 0; i < BN / 64; ++i)
                tma_load_2d(bs + i * 8192, &q.b[seg], t.nt * BN + 64 * i, k * kBK, &full[s]);
            } else {
              tma_load_2d(bs, &q.b[seg], k * kBK, t.nt * BN, &full[s]);
            }
          }
        }
      }
      if (!ok) fail(50);
      // every issued stage lands before the CTA may exit
      for (int j = (it > C::NS ? it - C::NS : 0); j < it; ++j)
        mbar_wait(&full[j % C::NS], (j / C::NS) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    int it = 0, tile = 0;
    bool aborted = false;
    for (int u = blockIdx.x; u < a.total && !aborted; u += gridDim.x, ++tile) {
      const Tile t = tile_at(a, u);
      const GemmProblem& q = a.p[t.p];
      const int steps = q.kt[0] + q.kt[1];
      // D fp32; A and B bf16 (1) or fp16 (0); majors; N; M
      const uint32_t idesc = (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) |
                             ((uint32_t)(q.a_mn != 0) << 15) | ((uint32_t)(q.b_mn != 0) << 16) |
                             ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
      const int b = tile & 1, buse = tile >> 1;
      if (buse > 0 && !mbar_wait(&acc_empty[b], (buse - 1) & 1)) aborted = true;
      aborted = __any_sync(0xffffffffu, aborted || *abort_flag);
      if (aborted) break;
      tc_fence_after();
      const uint32_t dacc = tmem + b * BN;
      const uint64_t astep = q.a_mn ? 2048 >> 4 : 32 >> 4, bstep = q.b_mn ? 2048 >> 4 : 32 >> 4;
      for (int k = 0; k < steps; ++k, ++it) {
        const int s = it % C::NS;
        const bool ok = mbar_wait(&full[s], (it / C::NS) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          aborted = true;
          break;
        }
        tc_fence_after();
        const uint32_t as = smem_u32(smem + s * C::STAGE), bs = as + C::A_BYTES;
        const uint64_t ad = q.a_mn ? umma_desc_mn_sw128(as) : umma_desc_sw128(as);
        const uint64_t bd = q.b_mn ? umma_desc_mn_sw128(bs) : umma_desc_sw128(bs);
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          umma_f16_warp(dacc, ad + kk * astep, bd + kk * bstep, idesc, (k > 0 || kk > 0) ? 1u : 0u);
        umma_commit_warp(&empty[s]);
      }
      if (aborted) break;
      umma_commit_warp(&acc_full[b]);
    }
    if (aborted) fail(51);
    // all issued MMAs complete before TMEM and shared memory are released
    umma_commit_warp(drain);
    mbar_wait(drain, 0);
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..9)
    const int quarter = warp & 3;      // TMEM lanes 32 * quarter .. + 31
    const int half = (warp - 2) >> 2;  // which half of the columns
    constexpr int COLS = EPI == EPI_GATED ? BN / 4 : BN / 2;  // output columns a warp
    int tile = 0;
    for (int u = blockIdx.x; u < a.total && !*abort_flag; u += gridDim.x, ++tile) {
      const Tile t = tile_at(a, u);
      const GemmProblem& q = a.p[t.p];
      const int b = tile & 1;
      if (!mbar_wait(&acc_full[b], (tile >> 1) & 1)) {
        fail(52);
        break;
      }
      tc_fence_after();
      __syncwarp();
      const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16) + b * BN + half * COLS;
      const int m = t.m0 + quarter * 32 + lane;
      const int n0 = t.nt * (EPI == EPI_GATED ? BN / 2 : BN) + half * COLS;
      const bool row_ok = m < q.M;
#pragma unroll 1
      for (int c = 0; c < COLS; c += 16) {
        const int n = n0 + c;
        const bool ok0 = row_ok && n < q.N, ok1 = row_ok && n + 8 < q.N;  // N is a multiple of 8
        const size_t at = (size_t)m * q.N + n;
        uint32_t r0[16];
        tmem_ld16_async(lane_addr + c, r0);
        float o[16];
        if constexpr (EPI == EPI_STORE) {
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = __uint_as_float(r0[j]);
          uint16_t* out = static_cast<uint16_t*>(q.out) + at;
          if (ok0) store8<F16>(out, o);
          if (ok1) store8<F16>(out + 8, o + 8);
        } else if constexpr (EPI == EPI_GATED) {
          uint32_t r1[16];
          tmem_ld16_async(lane_addr + BN / 2 + c, r1);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            o[j] = act_value<ACT>(__uint_as_float(r0[j])) * __uint_as_float(r1[j]);
          uint16_t* out = static_cast<uint16_t*>(a.h) + at;
          if (ok0) store8<F16>(out, o);
          if (ok1) store8<F16>(out + 8, o + 8);
          if (a.pre) {
            uint4* pg = reinterpret_cast<uint4*>(a.pre + at);
            uint4* pu = reinterpret_cast<uint4*>(a.pre + (size_t)q.M * q.N + at);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < 2 ? ok0 : ok1) {
                pg[j] = make_uint4(r0[4 * j], r0[4 * j + 1], r0[4 * j + 2], r0[4 * j + 3]);
                pu[j] = make_uint4(r1[4 * j], r1[4 * j + 1], r1[4 * j + 2], r1[4 * j + 3]);
              }
          }
        } else {
          const float4* pg = reinterpret_cast<const float4*>(a.pre + at);
          const float4* pu = reinterpret_cast<const float4*>(a.pre + (size_t)q.M * q.N + at);
          float4 g4[4], u4[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            g4[j] = u4[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j < 2 ? ok0 : ok1) {
              g4[j] = pg[j];
              u4[j] = pu[j];
            }
          }
          tmem_wait_ld();
          float dg[16], du[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float dh = __uint_as_float(r0[j]);
            const float g = reinterpret_cast<const float*>(g4)[j];
            const float uu = reinterpret_cast<const float*>(u4)[j];
            float av, dav;
            act_grad<ACT>(g, &av, &dav);
            o[j] = av * uu;
            dg[j] = dh * uu * dav;
            du[j] = dh * av;
          }
          if (ok0) {
            store8<F16>(static_cast<uint16_t*>(a.h) + at, o);
            store8<F16>(static_cast<uint16_t*>(a.dg) + at, dg);
            store8<F16>(static_cast<uint16_t*>(a.du) + at, du);
          }
          if (ok1) {
            store8<F16>(static_cast<uint16_t*>(a.h) + at + 8, o + 8);
            store8<F16>(static_cast<uint16_t*>(a.dg) + at + 8, dg + 8);
            store8<F16>(static_cast<uint16_t*>(a.du) + at + 8, du + 8);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * BN);
  }
  pdl_trigger();
}

// ------------------------------------------------------------------ host side

template <int BN, int EPI, bool F16, int ACT>
cudaError_t launch_kernel(const GemmArgs& a, int sms, cudaStream_t st, bool pdl) {
  using C = GemmCfg<BN>;
  auto kern = ffn_gemm_kernel<BN, EPI, F16, ACT>;
  static bool done[kMaxDevices] = {};
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(kern), done);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(std::min(sms, a.total));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = C::NS * C::STAGE + 2048;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int BN, int EPI>
cudaError_t launch_types(const GemmArgs& a, bool f16, int act, int sms, cudaStream_t st, bool pdl) {
  constexpr int S = MOE_ACT_SILU, G = MOE_ACT_GELU;
  if (EPI == EPI_STORE || act == S)
    return f16 ? launch_kernel<BN, EPI, true, S>(a, sms, st, pdl)
               : launch_kernel<BN, EPI, false, S>(a, sms, st, pdl);
  if constexpr (EPI != EPI_STORE)
    return f16 ? launch_kernel<BN, EPI, true, G>(a, sms, st, pdl)
               : launch_kernel<BN, EPI, false, G>(a, sms, st, pdl);
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
};

bool operand_map(CUtensorMap* m, const Operand& o, bool f16, int rows_k_major) {
  const CUtensorMapDataType dt =
      f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return make_map(m, dt, 2, o.base, o.cols, o.rows, 64, o.mn ? 64 : rows_k_major,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

// Tile width: the fewest cycles of the busiest CTA. A 128 x BN x 16 MMA takes BN / 2 cycles,
// at least the time its operands need from shared memory ((128 + BN) / 4), and a tile about
// 2000 cycles more to fill the ring and drain the accumulator.
template <int EPI>
int pick_bn(const Product* pr, int n, int sms) {
  int best = 256;
  double best_cost = -1;
  for (int bn = 256; bn >= 64; bn /= 2) {
    long long tiles = 0;
    double work = 0;
    for (int i = 0; i < n; ++i) {
      const int cols = EPI == EPI_GATED ? bn / 2 : bn;
      const long long t = (long long)((pr[i].M + kBM - 1) / kBM) * ((pr[i].N + cols - 1) / cols);
      const double step = std::max(bn / 2, (128 + bn) / 4);
      tiles += t;
      work += t * ((pr[i].K[0] + pr[i].K[1]) / 16.0 * step + 2000);
    }
    const double cost = work / tiles * ((tiles + sms - 1) / sms);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = bn;
    }
  }
  return best;
}

template <int EPI>
cudaError_t run_products(const Product* pr, int n, const FfnArgs& f, cudaStream_t st, bool pdl) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int bn = pick_bn<EPI>(pr, n, sms);
  GemmArgs a;
  std::memset(&a, 0, sizeof(a));
  a.n = n;
  for (int i = 0; i < n; ++i) {
    GemmProblem& q = a.p[i];
    const Product& s = pr[i];
    q.out = s.out;
    q.M = s.M;
    q.N = s.N;
    q.a_mn = s.a[0].mn;
    q.b_mn = s.b[0].mn;
    const int segs = s.K[1] > 0 ? 2 : 1;
    for (int j = 0; j < segs; ++j) {
      q.kt[j] = (s.K[j] + kBK - 1) / kBK;
      if (!operand_map(&q.a[j], s.a[j], f.f16, kBM)) return cudaErrorInvalidValue;
    }
    const int n_b = EPI == EPI_GATED ? 2 : segs;
    for (int j = 0; j < n_b; ++j)
      if (!operand_map(&q.b[j], s.b[j], f.f16, EPI == EPI_GATED ? bn / 2 : bn))
        return cudaErrorInvalidValue;
    const int cols = EPI == EPI_GATED ? bn / 2 : bn;
    q.tiles_m = (s.M + kBM - 1) / kBM;
    q.tiles_n = (s.N + cols - 1) / cols;
    q.first = a.total;
    a.total += q.tiles_m * q.tiles_n;
  }
  a.pre = f.pre;
  a.h = f.h;
  a.dg = f.dg;
  a.du = f.du;
  a.status = f.status;
  if (bn == 256) return launch_types<256, EPI>(a, f.f16, f.act, sms, st, pdl);
  if (bn == 128) return launch_types<128, EPI>(a, f.f16, f.act, sms, st, pdl);
  return launch_types<64, EPI>(a, f.f16, f.act, sms, st, pdl);
}

Operand k_major(const void* base, int rows, int cols) {
  return Operand{base, (uint64_t)rows, (uint64_t)cols, false};
}
Operand mn_major(const void* base, int rows, int cols) {
  return Operand{base, (uint64_t)rows, (uint64_t)cols, true};
}

}  // namespace

cudaError_t launch_ffn_gate_up(const FfnArgs& f, cudaStream_t st) {
  Product p{};
  p.a[0] = k_major(f.x, f.T, f.d);
  p.b[0] = k_major(f.w_gate, f.f, f.d);
  p.b[1] = k_major(f.w_up, f.f, f.d);
  p.K[0] = f.d;
  p.M = f.T;
  p.N = f.f;
  return run_products<EPI_GATED>(&p, 1, f, st, false);
}

cudaError_t launch_ffn_down(const FfnArgs& f, cudaStream_t st) {
  Product p{};
  p.a[0] = k_major(f.h, f.T, f.f);
  p.b[0] = k_major(f.w_down, f.d, f.f);
  p.K[0] = f.f;
  p.M = f.T;
  p.N = f.d;
  p.out = f.y;
  return run_products<EPI_STORE>(&p, 1, f, st, true);
}

cudaError_t launch_ffn_gate_grad(const FfnArgs& f, cudaStream_t st) {
  Product p{};
  p.a[0] = k_major(f.dy, f.T, f.d);
  p.b[0] = mn_major(f.w_down, f.d, f.f);
  p.K[0] = f.d;
  p.M = f.T;
  p.N = f.f;
  return run_products<EPI_GRAD>(&p, 1, f, st, false);
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
  }
  return run_products<EPI_STORE>(p, n, f, st, true);
}

}  // namespace moe
