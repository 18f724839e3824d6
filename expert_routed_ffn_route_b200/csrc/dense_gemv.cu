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
// gate rows and the same 8 up rows, so that one lane ends with both sums of an output) and a
// run of slots of 128 (int4) or 32 (16-bit) K values; each lane copies 16 bytes of two rows a
// slot into its warp's own ring in shared memory (cp.async, 4 or 8 slots deep, no barrier: a
// ring is private to its warp) and the copies run ahead across row tiles.
//
// Products: mma.sync m16n8k16, 8 activation rows wide. The int4 codes enter exactly, as the
// 16-bit values (136 + q) - 136 (bf16) or (1032 + q) - 1032 (fp16): one LOP3 and one packed
// subtraction for two codes. Subtracting before the product instead of correcting the sum
// keeps infinities in x infinite and costs only the FMA pipe, which is otherwise idle (the
// ALU pipe, 7 operations for 8 codes at half rate, is the busiest). A group's products are
// summed in fp32 by the tensor core, then acc += s * sum in fp32.
//
// The activation rows sit in shared memory in fragment order, staged once per CTA. Columns of
// the MMA beyond the last row repeat or hold anything: they are never stored. Rows that do not
// fit are split into K parts over the CTAs; the parts of a row tile go to the workspace and
// the CTA that brings the last one adds them in part order, so the result does not depend on
// the order of arrival.
#include <cstring>

#include "dense.cuh"

namespace moe {

namespace {

constexpr int kWarps = 16;
constexpr int kSmemMax = 227 * 1024;
constexpr int ring_bytes(int depth) { return kWarps * depth * 1024; }

struct GemvPlan {
  int slot_k;        // K values a slot
  int slots;         // slots of a row
  int parts;         // K parts
  int part_slots;    // slots a part
  int tiles;         // row tiles
  int rows;          // output rows a tile
  int ks;            // warps a tile
  int groups;        // CTAs a part
  int run;           // slots a warp
  int tc;            // 8-row column tiles
  int cols;          // activation rows staged (padded to whole column tiles above one)
  int wpr;           // log2 of the warps that stage one row
  int depth;         // ring slots a warp
  int smem;
};

GemvPlan make_gemv_plan(const GemvArgs& a, int sms) {
  GemvPlan p;
  p.slot_k = a.fmt == 4 ? 128 : 32;
  p.slots = (a.K + p.slot_k - 1) / p.slot_k;
  p.tc = a.T <= 8 ? 1 : a.T <= 16 ? 2 : a.T <= 24 ? 3 : 4;
  p.cols = p.tc == 1 ? a.T : 8 * p.tc;
  p.rows = a.gated ? 8 : 16;
  p.tiles = (a.N + p.rows - 1) / p.rows;
  const int red = kWarps * p.tc * 512;
  const int slot_bytes = p.slot_k * 2 * p.cols;
  const int room = kSmemMax - red - 256;
  // 8 slots deep where one part fits beside it: a call on one row then has 112 KB a SM on the way
  p.depth = p.tc == 1 && p.slots * slot_bytes <= room - ring_bytes(8) ? 8 : 4;
  const int fit = std::max(1, (room - ring_bytes(p.depth)) / slot_bytes);
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
  p.run = (p.part_slots + p.ks - 1) / p.ks;
  p.wpr = 0;
  while ((kWarps >> (p.wpr + 1)) >= a.T) ++p.wpr;
  p.smem = ring_bytes(p.depth) + red + p.part_slots * slot_bytes + 256;
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

// c (+)= a b; FIRST starts from zero.
template <bool F16, bool FIRST = false>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  const float i0 = FIRST ? 0.f : c[0], i1 = FIRST ? 0.f : c[1];
  const float i2 = FIRST ? 0.f : c[2], i3 = FIRST ? 0.f : c[3];
  if constexpr (F16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(i0), "f"(i1), "f"(i2),
          "f"(i3));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(i0), "f"(i1), "f"(i2),
          "f"(i3));
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

template <int FMT, int GROUP, bool F16, int TC, bool GATED, int DEPTH>
__global__ void __launch_bounds__(kWarps * 32, 1)
    gemv_rows_kernel(const GemvArgs a, const GemvPlan p) {
  constexpr int XI = FMT == 4 ? 4 : 1;             // 16-byte fragment chunks a lane and slot
  constexpr int NSC = FMT == 4 ? 128 / GROUP : 1;  // scales a row and slot
  constexpr int SLOT_CHUNKS = FMT == 4 ? 16 : 4;   // chunks of 8 K values a slot
  constexpr bool EXCHANGE = FMT == 4 && GROUP != 128;  // lanes read words other lanes copied
  constexpr int RING = ring_bytes(DEPTH);
  extern __shared__ __align__(1024) uint8_t smem[];
  float4* red = reinterpret_cast<float4*>(smem + RING);
  int* last_flag = reinterpret_cast<int*>(smem + RING + kWarps * TC * 512);
  uint4* xs = reinterpret_cast<uint4*>(smem + RING + kWarps * TC * 512 + 256);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int ks = warp % p.ks, tg = warp / p.ks, per = kWarps / p.ks;
  const int part = blockIdx.x % p.parts, grp = blockIdx.x / p.parts;
  const int begin = part * p.part_slots, end = min(p.slots, begin + p.part_slots);
  const int first = begin + ks * p.run;            // this warp's slots: first .. first + n_my - 1
  const int n_my = max(0, min(p.run, end - first));
  const int tile0 = grp * per + tg, tstep = p.groups * per;
  const size_t row_bytes = FMT == 4 ? (size_t)a.K / 2 : (size_t)a.K * 2;
  const int chunks = (int)(row_bytes / 16);        // 16-byte chunks a weight row
  const int n_scales = FMT == 4 ? a.K / GROUP : 0;

  // this lane's two rows of a tile (past the end: the last row, never stored)
  auto row_of = [&](int tile, int half) -> int {
    const int r = GATED ? tile * 8 + g : tile * 16 + g + 8 * half;
    return min(r, a.N - 1);
  };
  const uint8_t* wbase[2] = {static_cast<const uint8_t*>(a.w[0]),
                             static_cast<const uint8_t*>(a.w[GATED ? 1 : 0])};
  const uint16_t* sbase[2] = {a.s[0], a.s[GATED ? 1 : 0]};

  // ---- the ring: the copy cursor runs DEPTH - 1 slots ahead of the products
  uint8_t* ring = smem + warp * (DEPTH * 1024);
  // chunk t4 of row g; with groups under 128 a quad exchanges words through the ring, and the
  // chunk position is rotated by the row so that its 4-byte reads spread over the banks
  const uint32_t put = smem_u32(ring) +
                       (EXCHANGE ? g * 64 + (t4 ^ ((g >> 1) & 3)) * 16 : lane * 16);
  int ct = tile0, cleft = 0, cit = 0;              // copy cursor: tile, slots left in it, count
  const uint8_t* crow[2];
  auto copy_tile = [&]() {
    if (ct < p.tiles && n_my > 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        crow[h] = wbase[h] + (size_t)row_of(ct, h) * row_bytes + (size_t)first * 64 + t4 * 16;
      cleft = n_my;
    }
  };
  copy_tile();
  auto copy_next = [&]() {
    if (cleft > 0) {
      const uint32_t dst = put + (cit % DEPTH) * 1024;
      // a row may end inside the last slot of its K values (never for groups of 128)
      bool in = true;
      if constexpr (FMT != 4 || GROUP != 128) in = (first + n_my - cleft) * 4 + t4 < chunks;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        cp_async16(dst + h * 512, in ? crow[h] : wbase[h], in ? 16u : 0u);
        crow[h] += 64;
      }
      if (--cleft == 0) {
        ct += tstep;
        copy_tile();
      }
    }
    ++cit;
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) copy_next();

  // Scales of four slots at a time, slot 4 b + t4 of batch b in each lane of a quad; the next
  // batch (of the next tile, at the end) is loaded while one is used.
  const int batches = (n_my + 3) / 4;
  int st = tile0, sb = 0;
  float sc[2][NSC], sn[2][NSC];
  auto load_scales = [&]() {
    if (FMT == 4 && st < p.tiles) {
      const int at = (first + 4 * sb + t4) * NSC;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint16_t* row = sbase[h] + (size_t)row_of(st, h) * n_scales;
#pragma unroll
        for (int j = 0; j < NSC; ++j)
          sn[h][j] = bf16_to_f32(__ldg(row + min(at + j, n_scales - 1)));
      }
      if (++sb >= batches) {
        sb = 0;
        st += tstep;
      }
    }
  };
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < NSC; ++j) sn[h][j] = 0.f;
  if (n_my > 0) load_scales();

  // ---- activation rows into shared memory, in fragment order (after the preceding kernel);
  // 2^wpr warps a row, four chunks a lane on the way at a time
  pdl_wait();
  pdl_trigger();
  {
    const int c0 = begin * SLOT_CHUNKS, nc = (end - begin) * SLOT_CHUNKS, kc = a.K / 8;
    const int step = 32 << p.wpr;
    for (int row = warp >> p.wpr; row < a.T; row += kWarps >> p.wpr) {
      const uint4* src = reinterpret_cast<const uint4*>(a.x + (size_t)row * a.ldx) + c0;
      for (int c = lane + 32 * (warp & ((1 << p.wpr) - 1)); c < nc; c += 4 * step) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = make_uint4(0, 0, 0, 0);
          if (c + j * step < nc && c0 + c + j * step < kc) v[j] = src[c + j * step];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int cj = c + j * step;
          if (cj >= nc) break;
          int fi = 0, ft = cj % SLOT_CHUNKS;
          uint4 w = v[j];
          if constexpr (FMT == 4) {
            place_of<GROUP>(cj % SLOT_CHUNKS, &fi, &ft);
            // (0,1) (2,3) (4,5) (6,7) -> (0,4) (1,5) (2,6) (3,7)
            w.x = __byte_perm(v[j].x, v[j].z, 0x5410);
            w.y = __byte_perm(v[j].x, v[j].z, 0x7632);
            w.z = __byte_perm(v[j].y, v[j].w, 0x5410);
            w.w = __byte_perm(v[j].y, v[j].w, 0x7632);
          }
          xs[((cj / SLOT_CHUNKS * XI + fi) * p.cols + row) * 4 + ft] = w;
        }
      }
    }
  }
  __syncthreads();

  // this lane's column (beyond the last row of a single column tile: the last one again)
  const uint8_t* xlane =
      reinterpret_cast<const uint8_t*>(xs + (TC == 1 ? min(g, a.T - 1) : g) * 4 + t4) +
      (size_t)(first - begin) * XI * p.cols * 64;
  const int xstep = p.cols * 64;                   // bytes from one chunk i to the next
  int it = 0;
  for (int tile = tile0; tile < p.tiles; tile += tstep) {
    float acc[TC][4];
#pragma unroll
    for (int c = 0; c < TC; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[c][j] = 0.f;

    const uint8_t* xp = xlane;
    for (int b4 = 0; b4 < n_my; b4 += 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NSC; ++j) sc[h][j] = sn[h][j];
      load_scales();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (b4 + u >= n_my) break;
        copy_next();
        cp_wait<DEPTH - 1>();
        if constexpr (EXCHANGE) __syncwarp();
        const uint8_t* sp = ring + (it % DEPTH) * 1024;
        ++it;
        if constexpr (FMT == 16) {
          const uint4 wa = *reinterpret_cast<const uint4*>(sp + lane * 16);
          const uint4 wb = *reinterpret_cast<const uint4*>(sp + 512 + lane * 16);
#pragma unroll
          for (int n = 0; n < TC; ++n) {
            const uint4 x4 = *reinterpret_cast<const uint4*>(xp + n * 512);
            mma16816<F16>(acc[n], wa.x, wb.x, wa.y, wb.y, x4.x, x4.y);
            mma16816<F16>(acc[n], wa.z, wb.z, wa.w, wb.w, x4.z, x4.w);
          }
          xp += xstep;
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
            constexpr int kWords = GROUP / 32;  // words a group
            const uint32_t a0 = codes_pair<F16>(wa[i]), a1 = codes_pair<F16>(wb[i]);
            const uint32_t a2 = codes_pair<F16>(wa[i] >> 4), a3 = codes_pair<F16>(wb[i] >> 4);
            const uint32_t a4 = codes_pair<F16>(wa[i] >> 8), a5 = codes_pair<F16>(wb[i] >> 8);
            const uint32_t a6 = codes_pair<F16>(wa[i] >> 12), a7 = codes_pair<F16>(wb[i] >> 12);
#pragma unroll
            for (int n = 0; n < TC; ++n) {
              const uint4 x4 = *reinterpret_cast<const uint4*>(xp + n * 512);
              if (i % kWords == 0) mma16816<F16, true>(c[n], a0, a1, a2, a3, x4.x, x4.y);
              else mma16816<F16>(c[n], a0, a1, a2, a3, x4.x, x4.y);
              mma16816<F16>(c[n], a4, a5, a6, a7, x4.z, x4.w);
            }
            xp += xstep;
            if (i % kWords == kWords - 1) {
              const float s0 = __shfl_sync(0xffffffffu, sc[0][i / kWords], u, 4);
              const float s1 = __shfl_sync(0xffffffffu, sc[1][i / kWords], u, 4);
#pragma unroll
              for (int n = 0; n < TC; ++n) {
                acc[n][0] = fmaf(s0, c[n][0], acc[n][0]);
                acc[n][1] = fmaf(s0, c[n][1], acc[n][1]);
                acc[n][2] = fmaf(s1, c[n][2], acc[n][2]);
                acc[n][3] = fmaf(s1, c[n][3], acc[n][3]);
              }
            }
          }
          // every lane has read the slot before the quad's copies reuse it
          if constexpr (EXCHANGE) __syncwarp();
        }
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

template <int FMT, int GROUP, bool F16, int TC, bool GATED, int DEPTH>
cudaError_t launch_one(const GemvArgs& a, const GemvPlan& p, cudaStream_t st, bool pdl) {
  auto kern = gemv_rows_kernel<FMT, GROUP, F16, TC, GATED, DEPTH>;
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
  switch (p.tc) {
    case 1:
      return p.depth == 8 ? launch_one<FMT, GROUP, F16, 1, GATED, 8>(a, p, st, pdl)
                          : launch_one<FMT, GROUP, F16, 1, GATED, 4>(a, p, st, pdl);
    case 2: return launch_one<FMT, GROUP, F16, 2, GATED, 4>(a, p, st, pdl);
    case 3: return launch_one<FMT, GROUP, F16, 3, GATED, 4>(a, p, st, pdl);
    default: return launch_one<FMT, GROUP, F16, 4, GATED, 4>(a, p, st, pdl);
  }
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
