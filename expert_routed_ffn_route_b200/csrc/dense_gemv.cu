// Products of a few activation rows with one weight matrix, for calls of up to 32 rows:
//
//   y[t][n] = sum_k W[n][k] x[t][k] (+ b[n])            (moe_matvec; the block's down product)
//   y[t][n] = act(Wg[n] . x[t]) * (Wu[n] . x[t])        (the block's gate/up product, gated)
//
// with W 16-bit, or int4 codes q with a bf16 scale s per group of 32, 64 or 128 values:
// W[n][k] = q[n][k] s[n][k / group].
//
// The weights are read once, so a call is bound by streaming them (0.52 bytes a weight for
// int4 in groups of 128). One CTA of 16 warps per SM. A warp takes 16 weight rows (gated: 8
// gate rows and the same 8 up rows, so that one lane ends with both sums of an output) and
// every KS-th slot of 128 (int4) or 32 (16-bit) K values; each lane copies 16 bytes of two
// rows a slot into its warp's own ring in shared memory (cp.async, kDepth slots deep, no
// barrier: a ring is private to its warp) and the copies run ahead across row tiles.
//
// Products: mma.sync m16n8k16, 8 activation rows wide. The int4 codes enter exactly, as the
// 16-bit values (136 + q) - 136 (bf16) or (1032 + q) - 1032 (fp16): one LOP3 and one packed
// subtraction for two codes. Subtracting before the product instead of correcting the sum
// keeps infinities in x infinite and costs only the FMA pipe, which is otherwise idle (the
// ALU pipe, 7 operations for 8 codes at half rate, is the busiest). A group's products are
// summed in fp32 by the tensor core, then acc += s * sum in fp32.
//
// The activation rows sit in shared memory in fragment order, staged once per CTA. Rows that
// do not fit (T K over about 70,000 values) are split into K parts over the CTAs; the parts
// of a row tile go to the workspace and the CTA that brings the last one adds them in part
// order, so the result does not depend on the order of arrival.
#include <cstring>

#include "dense.cuh"

namespace moe {

namespace {

constexpr int kWarps = 16;
constexpr int kDepth = 5;                        // ring slots a warp
constexpr int kRingBytes = kWarps * kDepth * 1024;
constexpr int kSmemMax = 227 * 1024;

struct GemvPlan {
  int slot_k;        // K values a slot
  int slots;         // slots of a row
  int parts;         // K parts
  int part_slots;    // slots a part
  int tiles;         // row tiles
  int rows;          // output rows a tile
  int ks;            // warps a tile
  int groups;        // CTAs a part
  int tc;            // 8-row column tiles
  int smem;
};

GemvPlan make_gemv_plan(const GemvArgs& a, int sms) {
  GemvPlan p;
  p.slot_k = a.fmt == 4 ? 128 : 32;
  p.slots = (a.K + p.slot_k - 1) / p.slot_k;
  p.tc = a.T <= 8 ? 1 : a.T <= 16 ? 2 : 4;
  p.rows = a.gated ? 8 : 16;
  p.tiles = (a.N + p.rows - 1) / p.rows;
  const int red = kWarps * p.tc * 512;
  const int slot_bytes = p.slot_k * 2 * a.T;
  const int fit = std::max(1, (kSmemMax - kRingBytes - red - 256) / slot_bytes);
  p.parts = (p.slots + fit - 1) / fit;
  p.part_slots = (p.slots + p.parts - 1) / p.parts;
  p.parts = (p.slots + p.part_slots - 1) / p.part_slots;
  const int ctas = std::max(1, sms / p.parts);
  // Warps a tile: the fewest slot steps of the busiest warp, a tile's reduction counted as
  // two (measured).
  long long best = -1;
  p.ks = kWarps;
  for (int ks = kWarps; ks >= 1; ks /= 2) {
    const int per = kWarps / ks;                       // tiles a CTA at a time
    const int g = std::min(ctas, (p.tiles + per - 1) / per);
    const long long rounds = (p.tiles + (long long)g * per - 1) / ((long long)g * per);
    const long long cost = rounds * ((p.part_slots + ks - 1) / ks + 2);
    if (best < 0 || cost < best) {
      best = cost;
      p.ks = ks;
    }
  }
  const int per = kWarps / p.ks;
  p.groups = std::min(ctas, (p.tiles + per - 1) / per);
  p.smem = kRingBytes + red + p.part_slots * slot_bytes + 256;
  return p;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// Nibbles 0 and 4 of w as an exact pair of 16-bit values: the code with its sign bit flipped
// in the mantissa of 128 (bf16) or 1024 (fp16), minus that offset plus 8.
template <bool F16> __device__ __forceinline__ uint32_t codes_pair(uint32_t w) {
  constexpr uint32_t kOff = F16 ? 0x64086408u : 0x43084308u;
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(w), "n"(0x000F000Fu), "r"(kOff));
  if constexpr (F16) {
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(kOff));
  } else {
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(kOff));
  }
  return r;
}

// Where word group i of lane t of an int4 slot lies (16-byte chunk, word in it), and the
// inverse for staging x: chunk c8 of 8 K values of a slot -> (i, t). Each MMA pair i of a slot
// multiplies one word (8 codes) of each of the quad's lanes, all of one group, so
//   group 128: lane t holds words 4t..4t+3;   64: words 8 (i/2) + 2t + i%2;   32: words 4i + t.
template <int GROUP> __device__ __forceinline__ int word_of(int i, int t) {
  return GROUP == 128 ? 4 * t + i : GROUP == 64 ? 8 * (i >> 1) + 2 * t + (i & 1) : 4 * i + t;
}
template <int GROUP> __device__ __forceinline__ void place_of(int w, int* i, int* t) {
  if constexpr (GROUP == 128) {
    *i = w & 3;
    *t = w >> 2;
  } else if constexpr (GROUP == 64) {
    *i = 2 * (w >> 3) + (w & 1);
    *t = (w & 7) >> 1;
  } else {
    *i = w >> 2;
    *t = w & 3;
  }
}

template <int FMT, int GROUP, bool F16, int TC, bool GATED>
__global__ void __launch_bounds__(kWarps * 32, 1)
    gemv_rows_kernel(const GemvArgs a, const GemvPlan p) {
  constexpr int XI = FMT == 4 ? 4 : 1;           // 16-byte fragment chunks a lane and slot
  constexpr int NSC = FMT == 4 ? 128 / GROUP : 1;  // scales a row and slot
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;
  float4* red = reinterpret_cast<float4*>(smem + kRingBytes);
  int* last_flag = reinterpret_cast<int*>(smem + kRingBytes + kWarps * TC * 512);
  uint4* xs = reinterpret_cast<uint4*>(smem + kRingBytes + kWarps * TC * 512 + 256);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int ks = warp % p.ks, tg = warp / p.ks, per = kWarps / p.ks;
  const int part = blockIdx.x % p.parts, grp = blockIdx.x / p.parts;
  const int begin = part * p.part_slots, end = min(p.slots, begin + p.part_slots);
  const int n_my = max(0, (end - begin - ks + p.ks - 1) / p.ks);
  const int tile0 = grp * per + tg, tstep = p.groups * per;
  const size_t row_bytes = FMT == 4 ? (size_t)a.K / 2 : (size_t)a.K * 2;
  const int chunks = (int)(row_bytes / 16);      // 16-byte chunks a row
  const int n_scales = FMT == 4 ? a.K / GROUP : 0;

  // this lane's two rows of a tile (past the end: the last row, never stored)
  auto row_of = [&](int tile, int half) -> int {
    const int r = GATED ? tile * 8 + g : tile * 16 + g + 8 * half;
    return min(r, a.N - 1);
  };
  const uint8_t* wbase[2] = {static_cast<const uint8_t*>(a.w[0]),
                             static_cast<const uint8_t*>(a.w[GATED ? 1 : 0])};
  const uint16_t* sbase[2] = {a.s[0], a.s[GATED ? 1 : 0]};

  // ---- the ring: the copy cursor runs kDepth - 1 items ahead of the products
  const uint32_t ring_base = smem_u32(ring) + warp * (kDepth * 1024);
  // chunk t4 of row g; with groups under 128 a quad exchanges words through the ring, and the
  // chunk position is rotated by the row so that its 4- and 8-byte reads spread over the banks
  const int cpos = (FMT == 4 && GROUP != 128) ? (t4 ^ ((g >> 1) & 3)) : t4;
  const uint32_t put = (FMT == 4 && GROUP != 128) ? g * 64 + cpos * 16 : lane * 16;
  int ct = tile0, ci = 0, cstage = 0;            // copy cursor: tile, item, stage
  const uint8_t* crow[2];
  auto set_copy_tile = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) crow[h] = wbase[h] + (size_t)row_of(ct, h) * row_bytes;
  };
  if (ct < p.tiles) set_copy_tile();
  auto copy_next = [&]() {
    if (ct < p.tiles && n_my > 0) {
      const int chunk = (begin + ks + ci * p.ks) * 4 + t4;
      const bool in = chunk < chunks;
      const uint32_t dst = ring_base + cstage * 1024 + put;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        cp_async16(dst + h * 512, crow[h] + (in ? (size_t)chunk * 16 : 0), in ? 16u : 0u);
      if (++ci == n_my) {
        ci = 0;
        ct += tstep;
        if (ct < p.tiles) set_copy_tile();
      }
    }
    cp_commit();
    if (++cstage == kDepth) cstage = 0;
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) copy_next();

  // scales run two items ahead, in registers
  int st = tile0, si = 0;
  auto load_scales = [&](uint32_t (&v)[2][NSC]) {
    if (FMT == 4 && st < p.tiles && n_my > 0) {
      const int first = (begin + ks + si * p.ks) * NSC;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint16_t* row = sbase[h] + (size_t)row_of(st, h) * n_scales;
#pragma unroll
        for (int j = 0; j < NSC; ++j) v[h][j] = __ldg(row + min(first + j, n_scales - 1));
      }
      if (++si == n_my) {
        si = 0;
        st += tstep;
      }
    }
  };
  uint32_t sc[3][2][NSC] = {};
  load_scales(sc[0]);
  load_scales(sc[1]);

  // ---- activation rows into shared memory, in fragment order (after the preceding kernel)
  pdl_wait();
  pdl_trigger();
  {
    const int per_slot = p.slot_k / 8;
    const int c0 = begin * per_slot, nc = (end - begin) * per_slot;
    const int total = nc * a.T;
    for (int i = threadIdx.x; i < total; i += kWarps * 32) {
      const int row = i / nc, c = i - row * nc;
      uint4 v = make_uint4(0, 0, 0, 0);
      if ((c0 + c) * 8 < a.K)
        v = *reinterpret_cast<const uint4*>(a.x + (size_t)row * a.ldx + (size_t)(c0 + c) * 8);
      int slot = c / per_slot, fi = 0, ft = c - slot * per_slot;
      if constexpr (FMT == 4) {
        place_of<GROUP>(c - slot * per_slot, &fi, &ft);
        const uint4 o = v;  // (0,1) (2,3) (4,5) (6,7) -> (0,4) (1,5) (2,6) (3,7)
        v.x = __byte_perm(o.x, o.z, 0x5410);
        v.y = __byte_perm(o.x, o.z, 0x7632);
        v.z = __byte_perm(o.y, o.w, 0x5410);
        v.w = __byte_perm(o.y, o.w, 0x7632);
      }
      xs[((size_t)(slot * XI + fi) * a.T + row) * 4 + ft] = v;
    }
  }
  __syncthreads();

  int stage = 0;
  for (int tile = tile0; tile < p.tiles; tile += tstep) {
    float acc[TC][4];
#pragma unroll
    for (int c = 0; c < TC; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[c][j] = 0.f;

    for (int it = 0; it < n_my; ++it) {
      copy_next();
      load_scales(sc[2]);
      cp_wait<kDepth - 1>();
      if constexpr (FMT == 4 && GROUP != 128) __syncwarp();
      const uint8_t* sp = ring + warp * (kDepth * 1024) + stage * 1024;
      if (++stage == kDepth) stage = 0;
      const int slot = ks + it * p.ks;
      if constexpr (FMT == 16) {
        const uint4 wa = *reinterpret_cast<const uint4*>(sp + lane * 16);
        const uint4 wb = *reinterpret_cast<const uint4*>(sp + 512 + lane * 16);
#pragma unroll
        for (int c = 0; c < TC; ++c) {
          uint4 b = make_uint4(0, 0, 0, 0);
          if (c * 8 + g < a.T) b = xs[((size_t)slot * a.T + c * 8 + g) * 4 + t4];
          mma16816<F16>(acc[c], wa.x, wb.x, wa.y, wb.y, b.x, b.y);
          mma16816<F16>(acc[c], wa.z, wb.z, wa.w, wb.w, b.z, b.w);
        }
      } else {
        uint32_t wa[4], wb[4];
        if constexpr (GROUP == 128) {
          const uint4 ua = *reinterpret_cast<const uint4*>(sp + lane * 16);
          const uint4 ub = *reinterpret_cast<const uint4*>(sp + 512 + lane * 16);
          wa[0] = ua.x, wa[1] = ua.y, wa[2] = ua.z, wa[3] = ua.w;
          wb[0] = ub.x, wb[1] = ub.y, wb[2] = ub.z, wb[3] = ub.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int w = word_of<GROUP>(i, t4);
            const int at = g * 64 + (((w >> 2) ^ ((g >> 1) & 3)) * 16) + (w & 3) * 4;
            wa[i] = *reinterpret_cast<const uint32_t*>(sp + at);
            wb[i] = *reinterpret_cast<const uint32_t*>(sp + 512 + at);
          }
        }
        float c[TC][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i % (GROUP / 32) == 0) {
#pragma unroll
            for (int n = 0; n < TC; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) c[n][j] = 0.f;
          }
          const uint32_t a0 = codes_pair<F16>(wa[i]), a1 = codes_pair<F16>(wb[i]);
          const uint32_t a2 = codes_pair<F16>(wa[i] >> 4), a3 = codes_pair<F16>(wb[i] >> 4);
          const uint32_t a4 = codes_pair<F16>(wa[i] >> 8), a5 = codes_pair<F16>(wb[i] >> 8);
          const uint32_t a6 = codes_pair<F16>(wa[i] >> 12), a7 = codes_pair<F16>(wb[i] >> 12);
#pragma unroll
          for (int n = 0; n < TC; ++n) {
            uint4 b = make_uint4(0, 0, 0, 0);
            if (n * 8 + g < a.T) b = xs[((size_t)(slot * XI + i) * a.T + n * 8 + g) * 4 + t4];
            mma16816<F16>(c[n], a0, a1, a2, a3, b.x, b.y);
            mma16816<F16>(c[n], a4, a5, a6, a7, b.z, b.w);
          }
          if ((i + 1) % (GROUP / 32) == 0) {
            const int j = i / (GROUP / 32);
            const float s0 = __uint_as_float(sc[0][0][j] << 16);
            const float s1 = __uint_as_float(sc[0][1][j] << 16);
#pragma unroll
            for (int n = 0; n < TC; ++n) {
              acc[n][0] = fmaf(s0, c[n][0], acc[n][0]);
              acc[n][1] = fmaf(s0, c[n][1], acc[n][1]);
              acc[n][2] = fmaf(s1, c[n][2], acc[n][2]);
              acc[n][3] = fmaf(s1, c[n][3], acc[n][3]);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < NSC; ++j) {
            sc[0][h][j] = sc[1][h][j];
            sc[1][h][j] = sc[2][h][j];
          }
        // every lane has read the slot before the quad's copies reuse it
        if constexpr (GROUP != 128) __syncwarp();
      }
    }

    // ---- the tile's warps add their sums in warp order, and the outputs are written
    const int nthr = p.ks * 32, id = ks * 32 + lane, bar = 1 + tg;
    auto tile_sync = [&]() {
      if (p.ks > 1) named_bar_sync(bar, nthr);
      else __syncwarp();
    };
    tile_sync();  // the previous tile's sums have been read
    float4* my = red + (size_t)tg * p.ks * TC * 32;
#pragma unroll
    for (int c = 0; c < TC; ++c)
      my[(ks * TC + c) * 32 + lane] = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
    tile_sync();
    bool write = true;
    if (p.parts > 1) {
      float4* dst = reinterpret_cast<float4*>(a.partial) + ((size_t)tile * p.parts + part) * TC * 32;
      for (int i = id; i < TC * 32; i += nthr) {
        float4 v = my[i];
        for (int k = 1; k < p.ks; ++k) {
          const float4 u = my[k * TC * 32 + i];
          v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        __stcg(dst + i, v);
      }
      __threadfence();
      tile_sync();
      if (id == 0) {
        const int old = atomicAdd(a.counters + tile, 1);
        if (old == p.parts - 1) a.counters[tile] = 0;
        last_flag[tg] = old == p.parts - 1;
        __threadfence();
      }
      tile_sync();
      write = last_flag[tg] != 0;
    }
    if (write) {
      for (int i = id; i < TC * 32; i += nthr) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.parts > 1) {
          const float4* src =
              reinterpret_cast<const float4*>(a.partial) + (size_t)tile * p.parts * TC * 32 + i;
          for (int c = 0; c < p.parts; ++c) {
            const float4 u = __ldcg(src + (size_t)c * TC * 32);
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
          }
        } else {
          for (int k = 0; k < p.ks; ++k) {
            const float4 u = my[k * TC * 32 + i];
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
          }
        }
        const int l = i & 31, col = (i >> 5) * 8 + 2 * (l & 3);
        const float o[4] = {v.x, v.y, v.z, v.w};  // (row, col) (row, col+1) (row+8, ...)
        if constexpr (GATED) {
          const int n = tile * 8 + (l >> 2);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (n < a.N && col + j < a.T) {
              const float act = a.act == MOE_ACT_SILU ? act_value<MOE_ACT_SILU>(o[j])
                                                      : act_value<MOE_ACT_GELU>(o[j]);
              static_cast<uint16_t*>(a.y)[(size_t)(col + j) * a.ldy + n] =
                  round16<F16>(act * o[2 + j]);
            }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int n = tile * 16 + (l >> 2) + 8 * (j >> 1), c = col + (j & 1);
            if (n < a.N && c < a.T) {
              const float r = o[j] + (a.bias ? __ldg(a.bias + n) : 0.f);
              const size_t at = (size_t)c * a.ldy + n;
              if (a.y32) static_cast<float*>(a.y)[at] = r;
              else static_cast<uint16_t*>(a.y)[at] = round16<F16>(r);
            }
          }
        }
      }
    }
  }
  cp_wait<0>();
}

template <int FMT, int GROUP, bool F16, int TC, bool GATED>
cudaError_t launch_one(const GemvArgs& a, const GemvPlan& p, cudaStream_t st, bool pdl) {
  auto kern = gemv_rows_kernel<FMT, GROUP, F16, TC, GATED>;
  static bool done[kMaxDevices] = {};
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(kern), done);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(p.groups * p.parts);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a, p);
}

template <int FMT, int GROUP, bool F16, bool GATED>
cudaError_t launch_tc(const GemvArgs& a, const GemvPlan& p, cudaStream_t st, bool pdl) {
  if (p.tc == 1) return launch_one<FMT, GROUP, F16, 1, GATED>(a, p, st, pdl);
  if (p.tc == 2) return launch_one<FMT, GROUP, F16, 2, GATED>(a, p, st, pdl);
  return launch_one<FMT, GROUP, F16, 4, GATED>(a, p, st, pdl);
}

template <bool F16>
cudaError_t launch_fmt(const GemvArgs& a, const GemvPlan& p, cudaStream_t st, bool pdl) {
  if (a.fmt == 16)
    return a.gated ? launch_tc<16, 128, F16, true>(a, p, st, pdl)
                   : launch_tc<16, 128, F16, false>(a, p, st, pdl);
  if (a.gated) {
    if constexpr (F16) return cudaErrorInvalidValue;  // int4 blocks take bf16 rows
    else return launch_tc<4, 128, F16, true>(a, p, st, pdl);
  }
  if (a.group == 128) return launch_tc<4, 128, F16, false>(a, p, st, pdl);
  if (a.group == 64) return launch_tc<4, 64, F16, false>(a, p, st, pdl);
  return launch_tc<4, 32, F16, false>(a, p, st, pdl);
}

}  // namespace

int device_sms() {
  static int sms[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  if (sms[dev] == 0) {  // racing threads store the same value
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    sms[dev] = n;
  }
  return sms[dev];
}

cudaError_t allow_smem(const void* kernel, bool* done) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (err == cudaSuccess) done[dev] = true;
  return err;
}

void gemv_scratch(const GemvArgs& a, size_t* partial_bytes, size_t* n_counters) {
  const GemvPlan p = make_gemv_plan(a, 148);  // parts and tiles do not depend on the SM count
  *partial_bytes = p.parts > 1 ? (size_t)p.tiles * p.parts * p.tc * 512 : 0;
  *n_counters = p.parts > 1 ? p.tiles : 0;
}

cudaError_t launch_gemv_rows(const GemvArgs& a, cudaStream_t st, bool pdl) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const GemvPlan p = make_gemv_plan(a, sms);
  if (p.smem > kSmemMax || p.parts > sms) return cudaErrorInvalidValue;
  return a.f16 ? launch_fmt<true>(a, p, st, pdl) : launch_fmt<false>(a, p, st, pdl);
}

}  // namespace moe
