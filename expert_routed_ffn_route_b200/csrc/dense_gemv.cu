// Products of a few activation rows with one weight matrix, for calls of up to 32 rows:
//
//   y[t][n] = sum_k W[n][k] x[t][k] (+ b[n])            (moe_matvec; the block's down product)
//   y[t][n] = act(Wg[n] . x[t]) * (Wu[n] . x[t])        (the block's gate/up product, gated)
//
// with W 16-bit, or int4 codes q with a bf16 scale s per group of 32, 64 or 128 values:
// W[n][k] = q[n][k] s[n][k / group].
//
// The weights are read once, so a call is bound by streaming them (0.52 bytes a weight for
// int4 in groups of 128). One CTA of 16 warps per SM, a run of row tiles each: 16 weight rows
// (gated: 8 gate rows and the same 8 up rows, so that one lane ends with both sums of an
// output). The CTA's work, tiles x slots of 128 bytes of K (256 int4 or 64 16-bit values), is
// one line cut into 16 equal runs, one a warp, so that no warp waits for another inside the
// loop; a tile that several warps share is added up in warp order at the end. One lane brings
// a slot, 16 rows x 128 bytes, into its warp's own ring in shared memory by TMA (whole lines:
// boxes of 64 bytes reach 5.7 TB/s, of 128 bytes 6.5), 2 to 6 slots ahead of the products.
//
// Products: mma.sync m16n8k16, 8 activation rows wide, int4 codes exact in one of two forms.
//   masked  the nibbles of q + 8 as they lie in the word, at bits 0..3 or 4..7 of a 16-bit half:
//           as bf16 or fp16 bits that is (q + 8) or 16 (q + 8) times the smallest subnormal
//           (bits below 256 count it linearly in both types), so one LOP3 makes two codes and
//           one shift a word is left. bf16 rows are taken times 2^100, which keeps every
//           product a normal fp32 number. The sums start at -8 sum(x) of the group (computed
//           once a CTA by the same instructions), so they end at sum(q x).
//   offset  (136 + q) - 136 in bf16, (1032 + q) - 1032 in fp16: three shifts a word and a packed
//           subtraction for two codes, 48 instructions of 180 for 128 x 16 codes more. It has
//           no offset to cancel and no range, so a call whose rows hold infinities, NaN, or
//           bf16 magnitudes outside [2^-90, 2^26) takes it (each CTA sees that while it stages
//           the rows), and so do calls that it does not pay (kMaskedUnits).
// A group's products are summed in fp32 by the tensor core, then acc += s * sum in fp32.
//
// The activation rows sit in shared memory in fragment order, staged once per CTA. Columns of
// the MMA beyond the last row repeat or hold anything: they are never stored. Rows that do not
// fit are split into K parts over the CTAs; the parts of a row tile go to the workspace and
// the CTA that brings the last one adds them in part order, so the result does not depend on
// the order of arrival.
#include <cstring>
#include <type_traits>

#include "dense.cuh"
#include "tc_common.cuh"

namespace moe {

namespace {

constexpr int kWarps = 16, kWarpsLog2 = 4;
constexpr int kSmemMax = 227 * 1024;
constexpr int kSlotBytes = 2048;                 // 16 rows x 128 bytes
constexpr int kRingSlot = kWarps * kSlotBytes;   // one slot of every warp's ring
constexpr int kMaxDepth = 6;
constexpr int kSms = 148;
constexpr int kSiteGemvSlot = 60;
// The masked form from so many 16-row x 128-code units on. Its sums and its look at the rows cost
// a call 0.3 us: 1024 x 2560 (1280 units) 4.5 us against 4.2, 10240 x 2560 (12800) 8.8 against
// 9.3, 131072 x 2560 39.7 against 45.9. With groups of 32 four starts a unit cost more than they
// save (20480 x 4096 22.0 us against 21.1), with 16 rows likewise (10240 x 2560 12.1 against 11.5).
constexpr long long kMaskedUnits = 8192;

// K is counted in units of 64 bytes of a weight row (128 int4 or 32 16-bit values): what 8 (2)
// MMAs multiply. A slot holds two.
struct GemvPlan {
  int unit_k;        // K values a unit
  int units;         // units of a row
  int parts;         // K parts
  int part_units;    // units a part (even)
  int tiles;         // row tiles
  int rows;          // output rows a tile
  int groups;        // CTAs a part, each tiles_q tiles, the first tiles_r one more
  int tiles_q, tiles_r;
  int tc;            // 8-row column tiles
  int cols;          // activation rows staged (an even number; whole column tiles above one)
  int masked;        // the masked form where the rows allow it
  int sums;          // bytes of a unit's group sums
  int wpr;           // log2 of the warps that stage one row
  int depth;         // ring slots a warp
  int early;         // the kernel before writes no weights
  int drop;          // test control: warp 0 leaves its first copy out
  long long limit;   // cycles after which a wait gives up
  int smem;
};

GemvPlan make_gemv_plan(const GemvArgs& a, int sms) {
  GemvPlan p;
  p.unit_k = a.fmt == 4 ? 128 : 32;
  p.units = (a.K + p.unit_k - 1) / p.unit_k;
  p.tc = a.T <= 8 ? 1 : a.T <= 16 ? 2 : a.T <= 24 ? 3 : 4;
  p.cols = p.tc == 1 ? (a.T + 1) & ~1 : 8 * p.tc;
  p.rows = a.gated ? 8 : 16;
  p.tiles = (a.N + p.rows - 1) / p.rows;
  // a unit's rows, and (the masked form) its groups' sums
  p.masked = a.fmt == 4 && a.group == 128 && p.tc == 1 &&
             (long long)p.tiles * p.units >= kMaskedUnits;
  p.sums = p.masked ? 8 * 4 : 0;
  const int unit_bytes = p.unit_k * 2 * p.cols + p.sums;
  const int room = kSmemMax - 2048;                // beside the staged rows: two slots a warp
  const int fit = std::max(2, (room - 2 * kRingSlot) / unit_bytes & ~1);
  // K parts: at least so many that a part's rows fit; more where that is estimated shorter (cycles
  // of a CTA, from measured calls): its rows come in at 20 bytes a cycle while every SM fetches
  // the same ones, its slots go through 16 warps, and with parts the sums go through the
  // workspace. Measured with the number of parts forced: 16 rows on 2560 x 10240, groups of 32: 16.5 us
  // in two parts, 13.9 in four and in seven, 13.2 in eight (chosen); 32 rows on 10240 x 2560: 14.9 in one,
  // 14.5 in two (chosen), 16.6 in three; 7 rows on 5003 x 4096: 9.9 in one or two, 9.6 in four (chosen).
  // (The SM count is the B200's here: the workspace's size follows from it.)
  const int fewest = (p.units + fit - 1) / fit;
  double best = -1;
  for (int parts = fewest; parts <= std::max(fewest, 8); ++parts) {
    const int part_units = ((p.units + parts - 1) / parts + 1) & ~1;
    const int real = (p.units + part_units - 1) / part_units;
    const int groups = std::min(std::max(1, kSms / real), p.tiles);
    const double unit = a.fmt == 16 ? 250 : p.tc == 1 ? 1000 : p.tc == 2 ? 1100 : 1500;
    double cost = (double)part_units * unit_bytes / 20 +
                  (double)((p.tiles + groups - 1) / groups) * part_units / kWarps * unit;
    if (real > 1) cost += 2500 + (double)real * p.tiles * p.tc * 1024 / kSms / 20;
    if (best < 0 || cost < best) {
      best = cost;
      p.parts = real;
      p.part_units = part_units;
    }
  }
  const int xbytes = p.part_units * unit_bytes;
  p.depth = std::min(kMaxDepth, (room - xbytes) / kRingSlot);
  p.groups = std::min(std::max(1, sms / p.parts), p.tiles);
  p.tiles_q = p.tiles / p.groups;
  p.tiles_r = p.tiles % p.groups;
  p.wpr = 0;
  while ((kWarps >> (p.wpr + 1)) >= a.T) ++p.wpr;
  p.early = p.drop = 0;
  p.limit = kWaitCycles;
  p.smem = p.depth * kRingSlot + xbytes + 2048;
  return p;
}

struct GemvMaps {
  CUtensorMap w[2];  // weight rows in bytes, boxes of 128 bytes x 16 rows (gated: 8)
};

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

// The offset form. Nibbles 0 and 4 of w as an exact pair of 16-bit values: the code with its
// sign bit flipped in the mantissa of 128 (bf16) or 1024 (fp16), minus that offset plus 8.
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

// The masked form: nibbles (w & mask) with their sign bits flipped.
__device__ __forceinline__ uint32_t masked_codes(uint32_t w, uint32_t mask, uint32_t flip) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(w), "r"(mask), "r"(flip));  // (a & b) ^ c
  return r;
}
constexpr uint32_t kLow = 0x000F000Fu, kLow8 = 0x00080008u;    // bits 0..3: q + 8
constexpr uint32_t kHigh = 0x00F000F0u, kHigh8 = 0x00800080u;  // bits 4..7: 16 (q + 8)

// Range of the rows' magnitudes over packed 16-bit halves: the largest, and the smallest that
// is not zero, minus one.
struct Range16 {
  uint32_t hi = 0, lo = 0xffffffffu;
  __device__ __forceinline__ void add(uint32_t w) {
    const uint32_t m = w & 0x7fff7fffu;
    uint32_t d;
    asm("max.u16x2 %0, %0, %1;" : "+r"(hi) : "r"(m));
    asm("add.u16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(0xffffffffu));
    asm("min.u16x2 %0, %0, %1;" : "+r"(lo) : "r"(d));
  }
  // bf16: below 2^26 and at least 2^-90; fp16: finite.
  template <bool F16> __device__ __forceinline__ bool inside() const {
    const uint32_t h = max(hi & 0xffffu, hi >> 16), l = min(lo & 0xffffu, lo >> 16);
    return F16 ? h < 0x7C00u : h < 0x4C80u && l >= 0x1280u - 1;
  }
};

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

// MASKED: has the masked form too (a kernel of its own: the second loop costs small calls 0.5 us
// of instruction fetches).
template <int FMT, int GROUP, bool F16, int TC, bool GATED, bool MASKED>
__global__ void __launch_bounds__(kWarps * 32, 1)
    gemv_rows_kernel(const __grid_constant__ GemvMaps maps, const GemvArgs a, const GemvPlan p) {
  constexpr int XI = FMT == 4 ? 4 : 1;             // 16-byte fragment chunks a lane and unit
  constexpr int NSC = FMT == 4 ? 128 / GROUP : 1;  // scales a row and unit
  constexpr int UNIT_CHUNKS = FMT == 4 ? 16 : 4;   // chunks of 8 K values a unit
  constexpr int XB = TC == 1 ? 4 : 10;             // activation chunks a lane has on the way
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.depth * kRingSlot);  // [warp][kMaxDepth]
  uint4* xs = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(bars) + 1024);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < (GATED ? 2 : 1)) prefetch_map(&maps.w[threadIdx.x]);
  const int t4 = lane & 3;
  // the tile row of MMA row lane / 4: two rows that one phase of a 16-byte read covers lie four
  // apart, where the 128-byte swizzle gives them different banks
  const int g = ((lane >> 2 & 1) << 2) | (lane >> 3);
  const int part = blockIdx.x % p.parts, grp = blockIdx.x / p.parts;
  const int begin = part * p.part_units, n_units = min(p.part_units, p.units - begin);
  const int n_slots = (n_units + 1) / 2;
  // tiles of this CTA, and this warp's run of items (tile, slot)
  const int tb = grp * p.tiles_q + min(grp, p.tiles_r);
  const int items = (p.tiles_q + (grp < p.tiles_r)) * n_slots;
  auto run_start = [&](int w) -> int { return (int)((long long)items * w >> kWarpsLog2); };
  const int lo = run_start(warp), n_my = run_start(warp + 1) - lo;
  const int tile_off = (int)((unsigned)lo / (unsigned)n_slots);
  const int tile0 = tb + tile_off, slot0 = lo - tile_off * n_slots;

  // ---- the ring (lane 0 issues): `depth` slots ahead of the products
  uint8_t* ring = smem + warp * (p.depth * kSlotBytes);
  uint64_t* full = bars + warp * kMaxDepth;
  int ct = tile0, cs = slot0, cstage = 0, cleft = n_my;  // copy cursor
  auto copy_next = [&](bool drop = false) {
    if (cleft <= 0) return;
    --cleft;
    if (lane == 0 && !drop) {
      uint8_t* dst = ring + cstage * kSlotBytes;
      const int x = begin * 64 + cs * 128;
      mbar_arrive_expect_tx(&full[cstage], kSlotBytes);
      if constexpr (GATED) {
        tma_load_2d(dst, &maps.w[0], x, ct * 8, &full[cstage]);
        tma_load_2d(dst + kSlotBytes / 2, &maps.w[1], x, ct * 8, &full[cstage]);
      } else {
        tma_load_2d(dst, &maps.w[0], x, ct * 16, &full[cstage]);
      }
    }
    if (++cs == n_slots) {
      cs = 0;
      ++ct;
    }
    if (++cstage == p.depth) cstage = 0;
  };
  auto start_ring = [&]() {
    if (lane == 0) {
      for (int i = 0; i < p.depth; ++i) mbar_init(&full[i], 1);
      fence_barrier_init();
    }
    __syncwarp();
    for (int i = 0; i < p.depth; ++i) copy_next(p.drop && warp == 0 && i == 0);
  };

  // ---- scales: a slot ahead, in registers. A quad's lanes hold row half t4 / 2, unit t4 % 2.
  const int n_scales = FMT == 4 ? a.K / GROUP : 0;
  int st = tile0, ss = slot0, sleft = n_my;
  const uint16_t* srow = nullptr;
  auto scale_tile = [&]() {
    const int h = t4 >> 1;
    const int r = min(GATED ? st * 8 + g : st * 16 + g + 8 * h, a.N - 1);
    srow = (GATED && h ? a.s[1] : a.s[0]) + (size_t)r * n_scales;
  };
  uint32_t sn[NSC] = {};
  auto load_scales = [&]() {
    if (FMT != 4 || sleft <= 0) return;
    --sleft;
    const int at = (begin + 2 * ss + (t4 & 1)) * NSC;
#pragma unroll
    for (int j = 0; j < NSC; ++j) {
      // behind the last group (K need not fill a unit) the sum is zero, and so is the scale: the last
      // group's own may be infinite
      if (GROUP == 128) sn[j] = __ldg(srow + min(at + j, n_scales - 1));
      else sn[j] = at + j < n_scales ? __ldg(srow + at + j) : 0;
    }
    if (++ss == n_slots) {
      ss = 0;
      ++st;
      scale_tile();
    }
  };

  // ---- activation rows into shared memory, in fragment order; 2^wpr warps a row, XB chunks a
  // lane on the way at a time
  const int c0 = begin * UNIT_CHUNKS, nc = n_units * UNIT_CHUNKS, kc = a.K / 8;
  const int xstride = 32 << p.wpr;
  const int xstart = lane + 32 * (warp & ((1 << p.wpr) - 1));
  const int xwrap = (max(0, nc - xstart) + xstride - 1) & ~(xstride - 1);
  int xrow = 0, xc = 0;
  const uint4* xsrc = nullptr;
  auto x_start = [&]() {
    xrow = warp >> p.wpr;
    xc = xstart;
    xsrc = reinterpret_cast<const uint4*>(a.x + (size_t)xrow * a.ldx) + c0;
  };
  x_start();
  Range16 range;
  const size_t xrow_step = (size_t)(kWarps >> p.wpr) * (a.ldx / 8);
  uint4 xv[XB];
  int xat[XB];                                     // row in the upper half, chunk in the lower
  auto fetch_x = [&]() {
#pragma unroll
    for (int j = 0; j < XB; ++j) {
      if (xc >= nc) {                              // on to this warp's next row
        xc -= xwrap;
        xrow += kWarps >> p.wpr;
        xsrc += xrow_step;
      }
      const bool in = xrow < a.T && xc < nc;
      xat[j] = in ? xrow << 16 | xc : -1;
      xv[j] = make_uint4(0, 0, 0, 0);
      if (in && c0 + xc < kc) xv[j] = xsrc[xc];
      xc += xstride;
    }
  };
  auto put_x = [&](bool masked) {
#pragma unroll
    for (int j = 0; j < XB; ++j) {
      if (xat[j] < 0) continue;
      const int row = xat[j] >> 16, c = xat[j] & 0xffff;
      int fi = 0, ft = c % UNIT_CHUNKS;
      uint4 w = xv[j];
      if constexpr (FMT == 4) {
        place_of<GROUP>(c % UNIT_CHUNKS, &fi, &ft);
        // (0,1) (2,3) (4,5) (6,7) -> (0,4) (2,6) (1,5) (3,7)
        w.x = __byte_perm(xv[j].x, xv[j].z, 0x5410);
        w.y = __byte_perm(xv[j].y, xv[j].w, 0x5410);
        w.z = __byte_perm(xv[j].x, xv[j].z, 0x7632);
        w.w = __byte_perm(xv[j].y, xv[j].w, 0x7632);
        if (MASKED && masked) {
          range.add(w.x), range.add(w.y), range.add(w.z), range.add(w.w);
          if constexpr (!F16) {
            constexpr uint32_t k100 = 0x71807180u;  // 2^100
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w.x) : "r"(k100));
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w.y) : "r"(k100));
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w.z) : "r"(k100));
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w.w) : "r"(k100));
          }
        }
      }
      // neighbouring rows change places in odd chunk rows, halves of 64 bytes in chunks 2 and 3:
      // eight neighbouring chunks of a row then lie in different banks
      const int cr = c / UNIT_CHUNKS * XI + fi;
      xs[(cr * p.cols + (row ^ (cr & 1))) * 4 + (ft ^ (fi & 2))] = w;
    }
  };
  // Every launch is programmatic: the CTA sets itself up while the kernel ahead ends, and touches
  // nothing that this may write or read before pdl_wait (1 row of 1024 x 2560 3.5 us a call in a
  // row of calls, 4.2 without; 32 rows of 10240 x 2560 14.4 and 15.5). A block's down kernel follows
  // its gate/up kernel, which has waited for all before it when this one starts and writes no
  // weights, so there the copies of the weights come first of all; elsewhere the (shorter) rows'.
  if (FMT == 4 && n_my > 0) scale_tile();
  if (p.early) {
    start_ring();
    load_scales();
  }
  pdl_wait();
  pdl_trigger();
  if (!p.early) load_scales();
  fetch_x();
  if (!p.early) start_ring();
  put_x(MASKED);
  while (xrow < a.T) {
    fetch_x();
    put_x(MASKED);
  }
  bool masked = false;
  if constexpr (MASKED) {
    masked = !__syncthreads_or(!range.template inside<F16>());
    if (!masked) {                                 // (rare) the rows again, as they are
      x_start();
      while (xrow < a.T) {
        fetch_x();
        put_x(false);
      }
      __syncthreads();
    }
  } else {
    __syncthreads();
  }

  // this lane's column (beyond the last row of a single column tile: the last one again)
  const int col = TC == 1 ? min(lane >> 2, a.T - 1) : lane >> 2;
  const uint8_t* xlane = reinterpret_cast<const uint8_t*>(xs + col * 4 + t4);
  const int xflip = (col & 1) ? -64 : 64;          // to the row's place in odd chunk rows
  const int xswap = (t4 & 2) ? -32 : 32;           // to the swapped place of chunks 2 and 3
  const int xstep = p.cols * 64;                  // bytes from one chunk i to the next
  // 16 bytes of chunk c (0..7, units of 64 bytes side by side) of this lane's row, swizzled
  const uint32_t chunk_row = (uint32_t)g * 128;
  auto chunk_at = [&](int c) -> uint32_t { return chunk_row + ((c ^ g) << 4); };

  // ---- the masked form's start of a group: -8 sum(x), [unit][group][column], a warp a unit
  float* sums = reinterpret_cast<float*>(xs) + (size_t)p.part_units * XI * p.cols * 16;
  if (MASKED && masked) {
    for (int un = warp; un < n_units; un += kWarps) {
      float c[TC][2][4];
      const uint8_t* xp = xlane + un * XI * xstep;
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        constexpr int kWords = GROUP / 32;  // words a group
#pragma unroll
        for (int n = 0; n < TC; ++n) {
          const uint4 x4 = *reinterpret_cast<const uint4*>(
              xp + n * 512 + ((i & 1) ? xflip : 0) + ((i & 2) ? xswap : 0));
          if (i % kWords == 0) {
            mma16816<F16, true>(c[n][0], kLow8, kLow8, kLow8, kLow8, x4.x, x4.y);
            mma16816<F16, true>(c[n][1], kHigh8, kHigh8, kHigh8, kHigh8, x4.z, x4.w);
          } else {
            mma16816<F16>(c[n][0], kLow8, kLow8, kLow8, kLow8, x4.x, x4.y);
            mma16816<F16>(c[n][1], kHigh8, kHigh8, kHigh8, kHigh8, x4.z, x4.w);
          }
          if (i % kWords == kWords - 1 && lane < 4)
            *reinterpret_cast<float2*>(sums + ((un * NSC + i / kWords) * TC + n) * 8 + 2 * t4) =
                make_float2(-fmaf(0.0625f, c[n][1][0], c[n][0][0]),
                            -fmaf(0.0625f, c[n][1][1], c[n][0][1]));
        }
        xp += xstep;
      }
    }
    __syncthreads();
  }

  // ---- one tile's sums to the output
  const int esize = a.y32 ? 4 : 2;
  auto write_out = [&](int tile, const float (&v)[TC][4]) {
    const int n = GATED ? tile * 8 + g : tile * 16 + g;
    const size_t col_bytes = (size_t)a.ldy * esize;
    uint8_t* at = static_cast<uint8_t*>(a.y) + (size_t)n * esize + (2 * t4) * col_bytes;
    const bool ok0 = n < a.N, ok1 = !GATED && n + 8 < a.N;
    float b0 = 0.f, b1 = 0.f;
    if (!GATED && a.bias) {
      if (ok0) b0 = __ldg(a.bias + n);
      if (ok1) b1 = __ldg(a.bias + n + 8);
    }
#pragma unroll
    for (int c = 0; c < TC; ++c) {
      if (!GATED && TC == 1 && a.pairs) {  // columns 2 t4, 2 t4 + 1: the two rows of token t4
        if (2 * t4 < a.T) {
          uint8_t* to = static_cast<uint8_t*>(a.y) + (size_t)n * esize + t4 * col_bytes;
          if (ok0) *reinterpret_cast<uint16_t*>(to) = round16<F16>(v[c][0] + v[c][1]);
          if (ok1) *reinterpret_cast<uint16_t*>(to + 16) = round16<F16>(v[c][2] + v[c][3]);
        }
        continue;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (c * 8 + 2 * t4 + j < a.T) {
          uint8_t* to = at + j * col_bytes;
          if constexpr (GATED) {
            const float act = a.act == MOE_ACT_SILU ? act_value<MOE_ACT_SILU>(v[c][j])
                                                    : act_value<MOE_ACT_GELU>(v[c][j]);
            const float h = act * v[c][2 + j];
            const uint16_t r = round16<F16>(h);
            if (TC == 1 && a.pairs) {
              to = static_cast<uint8_t*>(a.y) + (size_t)n * 2 + 2 * (2 * t4 + j) * col_bytes;
              // (an infinite value has no rest)
              const float rest = h - value16<F16>(r);
              if (ok0)
                *reinterpret_cast<uint16_t*>(to + col_bytes) =
                    round16<F16>(isfinite(rest) ? rest : 0.f);
            }
            if (ok0) *reinterpret_cast<uint16_t*>(to) = r;
          } else if (a.y32) {
            if (ok0) *reinterpret_cast<float*>(to) = v[c][j] + b0;
            if (ok1) *reinterpret_cast<float*>(to + 32) = v[c][2 + j] + b1;
          } else {
            if (ok0) *reinterpret_cast<uint16_t*>(to) = round16<F16>(v[c][j] + b0);
            if (ok1) *reinterpret_cast<uint16_t*>(to + 16) = round16<F16>(v[c][2 + j] + b1);
          }
        }
      at += 8 * col_bytes;
    }
  };

  // ---- one tile's sums, complete over this CTA's K: to the output, or beside the other parts'
  float4* const partial = reinterpret_cast<float4*>(a.partial) + lane;
  auto finish = [&](int tile, const float (&v)[TC][4]) {
    if (p.parts == 1) {
      write_out(tile, v);
      return;
    }
    float4* dst = partial + ((size_t)tile * p.parts + part) * TC * 32;
#pragma unroll
    for (int c = 0; c < TC; ++c)
      __stcg(dst + c * 32, make_float4(v[c][0], v[c][1], v[c][2], v[c][3]));
  };

  // ---- the run
  bool ok = true;                                  // no wait has given up
  uint32_t phase = 0, bad_phase = 0;
  int stage = 0, bad_stage = 0, pending = 0, tile = tile0, slot = slot0;
  bool whole = slot0 == 0;                         // the tile's first slot is in this run
  float acc[TC][4], head[TC][4];
#pragma unroll
  for (int c = 0; c < TC; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[c][j] = head[c][j] = 0.f;
  const uint8_t* xp = xlane + slot0 * (2 * XI) * xstep;
  // 2^133 / 2^100 (bf16) or 2^24 (fp16): the masked form's unit. It goes into the group's sum, which
  // is in range with it; a scale of 2^95 (2^104) or more times it would be infinite.
  constexpr float unit = F16 ? 16777216.f : 8589934592.f;
  auto run = [&](auto fast) {
    constexpr bool FAST = decltype(fast)::value;
    for (int it = 0; it < n_my; ++it) {
      float sc[NSC];
#pragma unroll
      for (int j = 0; j < NSC; ++j) sc[j] = __uint_as_float(sn[j] << 16);
      load_scales();
      const uint8_t* sp = ring + stage * kSlotBytes;
      if (ok && !__all_sync(0xffffffffu, mbar_wait_within(&full[stage], phase, p.limit))) {
        set_timeout(a.status, kSiteGemvSlot);
        ok = false;                                // no more copies; those on the way are waited
        pending = n_my - cleft - it;               // for below
        bad_stage = stage;
        bad_phase = phase;
        cleft = 0;
      }
      const bool two = 2 * slot + 1 < n_units;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (u == 1 && !two) break;
        uint32_t wa[4], wb[4];
        if constexpr (FMT == 16 || GROUP == 128) {
          const uint32_t at = chunk_at(4 * u + t4);
          const uint4 ua = *reinterpret_cast<const uint4*>(sp + at);
          const uint4 ub = *reinterpret_cast<const uint4*>(sp + 1024 + at);
          wa[0] = ua.x, wa[1] = ua.y, wa[2] = ua.z, wa[3] = ua.w;
          wb[0] = ub.x, wb[1] = ub.y, wb[2] = ub.z, wb[3] = ub.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int w = word_of<GROUP>(i, t4);
            const uint32_t at = chunk_at(4 * u + (w >> 2)) + (w & 3) * 4;
            wa[i] = *reinterpret_cast<const uint32_t*>(sp + at);
            wb[i] = *reinterpret_cast<const uint32_t*>(sp + 1024 + at);
          }
        }
        // The slot is read (the fence: __syncwarp alone orders no asynchronous copy after the
        // reads): bring the next one.
        if (u == 1 || !two) {
          fence_proxy_async();
          __syncwarp();
          if (++stage == p.depth) {
            stage = 0;
            phase ^= 1;
          }
          copy_next();
        }
        if constexpr (FMT == 16) {
#pragma unroll
          for (int n = 0; n < TC; ++n) {
            const uint4 x4 = *reinterpret_cast<const uint4*>(xp + n * 512 + (u ? xflip : 0));
            mma16816<F16>(acc[n], wa[0], wb[0], wa[1], wb[1], x4.x, x4.y);
            mma16816<F16>(acc[n], wa[2], wb[2], wa[3], wb[3], x4.z, x4.w);
          }
          xp += xstep;
        } else {
          float c[TC][4], ch[FAST ? TC : 1][4];
          const float* start = sums + ((2 * slot + u) * NSC * TC) * 8 + 2 * t4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            constexpr int kWords = GROUP / 32;  // words a group
            uint32_t al[4], ah[4];              // codes 0, 4 | 2, 6 and 1, 5 | 3, 7 of both rows
            if constexpr (FAST) {
              const uint32_t va = wa[i] >> 8, vb = wb[i] >> 8;
              al[0] = masked_codes(wa[i], kLow, kLow8), al[1] = masked_codes(wb[i], kLow, kLow8);
              al[2] = masked_codes(va, kLow, kLow8), al[3] = masked_codes(vb, kLow, kLow8);
              ah[0] = masked_codes(wa[i], kHigh, kHigh8), ah[1] = masked_codes(wb[i], kHigh, kHigh8);
              ah[2] = masked_codes(va, kHigh, kHigh8), ah[3] = masked_codes(vb, kHigh, kHigh8);
            } else {
              al[0] = codes_pair<F16>(wa[i]), al[1] = codes_pair<F16>(wb[i]);
              al[2] = codes_pair<F16>(wa[i] >> 8), al[3] = codes_pair<F16>(wb[i] >> 8);
              ah[0] = codes_pair<F16>(wa[i] >> 4), ah[1] = codes_pair<F16>(wb[i] >> 4);
              ah[2] = codes_pair<F16>(wa[i] >> 12), ah[3] = codes_pair<F16>(wb[i] >> 12);
            }
#pragma unroll
            for (int n = 0; n < TC; ++n) {
              const uint4 x4 = *reinterpret_cast<const uint4*>(
                  xp + n * 512 + ((i & 1) ? xflip : 0) + ((i & 2) ? xswap : 0));
              if constexpr (FAST) {
                if (i % kWords == 0) {
                  const float2 s8 =
                      *reinterpret_cast<const float2*>(start + (i / kWords * TC + n) * 8);
                  c[n][0] = c[n][2] = s8.x;
                  c[n][1] = c[n][3] = s8.y;
                  mma16816<F16, true>(ch[n], ah[0], ah[1], ah[2], ah[3], x4.z, x4.w);
                } else {
                  mma16816<F16>(ch[n], ah[0], ah[1], ah[2], ah[3], x4.z, x4.w);
                }
                mma16816<F16>(c[n], al[0], al[1], al[2], al[3], x4.x, x4.y);
              } else {
                if (i % kWords == 0) mma16816<F16, true>(c[n], al[0], al[1], al[2], al[3], x4.x, x4.y);
                else mma16816<F16>(c[n], al[0], al[1], al[2], al[3], x4.x, x4.y);
                mma16816<F16>(c[n], ah[0], ah[1], ah[2], ah[3], x4.z, x4.w);
              }
            }
            xp += xstep;
            if (i % kWords == kWords - 1) {
              const float s0 = __shfl_sync(0xffffffffu, sc[i / kWords], u, 4);
              const float s1 = __shfl_sync(0xffffffffu, sc[i / kWords], 2 + u, 4);
#pragma unroll
              for (int n = 0; n < TC; ++n) {
                if constexpr (FAST)  // unit and unit / 16 are powers of two: one rounding
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    c[n][j] = fmaf(unit * 0.0625f, ch[n][j], unit * c[n][j]);
                acc[n][0] = fmaf(s0, c[n][0], acc[n][0]);
                acc[n][1] = fmaf(s0, c[n][1], acc[n][1]);
                acc[n][2] = fmaf(s1, c[n][2], acc[n][2]);
                acc[n][3] = fmaf(s1, c[n][3], acc[n][3]);
              }
            }
          }
        }
      }
      if (++slot == n_slots) {
        if (whole) {
          finish(tile, acc);
        } else {
#pragma unroll
          for (int c = 0; c < TC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) head[c][j] = acc[c][j];
        }
        slot = 0;
        ++tile;
        whole = true;
        xp = xlane;
#pragma unroll
        for (int c = 0; c < TC; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[c][j] = 0.f;
      }
    }
  };
  if (MASKED && masked) run(std::integral_constant<bool, MASKED>{});
  else run(std::false_type{});

  // after a timeout: the copies still on the way land (or their waits give up) before the ring is
  // written or the CTA ends (one that does not within the bound leaves none to the rest)
  long long left = kWaitCycles;
  for (; pending > 0; --pending) {
    if (!mbar_wait_within(&full[bad_stage], bad_phase, left)) left = 0;
    if (++bad_stage == p.depth) {
      bad_stage = 0;
      bad_phase ^= 1;
    }
  }

  // ---- tiles that several warps share: each leaves the sums of the tile it did not begin
  // ("head") in its ring, which nothing is on its way into any more; the warp that began a tile
  // adds the heads after it to its own, in warp order
  const bool open = n_my > 0 && slot != 0;         // the last tile goes on in the next warp
  float4* mine = reinterpret_cast<float4*>(ring) + lane;
  const bool inside = open && !whole;              // this run lies within one tile
#pragma unroll
  for (int c = 0; c < TC; ++c)                     // (zeros without a head)
    mine[c * 32] = inside ? make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3])
                          : make_float4(head[c][0], head[c][1], head[c][2], head[c][3]);
  __syncthreads();
  if (open && whole) {
    const int tile_end = (tile - tb + 1) * n_slots;
    // warps after this one that share the tile: run_start(w) < tile_end
    const int n = min(kWarps, (int)(((unsigned)tile_end * kWarps + items - 1) / (unsigned)items)) -
                  warp - 1;
    const uint8_t* theirs = smem + (warp + 1) * (p.depth * kSlotBytes) + lane * 16;
    for (int w = 0; w < n; w += 4) {
      float4 v[4][TC];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < TC; ++c) {
          v[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (w + i < n)
            v[i][c] = *reinterpret_cast<const float4*>(theirs + (w + i) * (p.depth * kSlotBytes) +
                                                       c * 512);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < TC; ++c) {
          acc[c][0] += v[i][c].x, acc[c][1] += v[i][c].y;
          acc[c][2] += v[i][c].z, acc[c][3] += v[i][c].w;
        }
    }
    finish(tile, acc);
  }

  // ---- K parts: this warp's tiles are a run too. One fence, one count a tile, then the sums of
  // the tiles whose last part this was.
  if (p.parts > 1) {
    const int from = tile0 + (slot0 != 0), to = tile + (open && whole);
    fence_acq_rel_gpu();
    __syncwarp();
    for (int t0 = from; t0 < to; t0 += 32) {
      bool last = false;
      if (t0 + lane < to) {
        last = atomicAdd(a.counters + t0 + lane, 1) == p.parts - 1;
        if (last) a.counters[t0 + lane] = 0;
      }
      uint32_t mask = __ballot_sync(0xffffffffu, last);
      if (mask) fence_acq_rel_gpu();
      while (mask) {
        const int t = t0 + __ffs(mask) - 1;
        mask &= mask - 1;
        const float4* src = partial + (size_t)t * p.parts * TC * 32;
#pragma unroll
        for (int c = 0; c < TC; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[c][j] = 0.f;
        for (int k = 0; k < p.parts; ++k)
#pragma unroll
          for (int c = 0; c < TC; ++c) {
            const float4 v = __ldcg(src + (k * TC + c) * 32);
            acc[c][0] += v.x, acc[c][1] += v.y, acc[c][2] += v.z, acc[c][3] += v.w;
          }
        write_out(t, acc);
      }
    }
  }
}

template <int FMT, int GROUP, bool F16, int TC, bool GATED, bool MASKED = false>
cudaError_t launch_one(const GemvArgs& a, const GemvPlan& p, cudaStream_t st) {
  auto kern = gemv_rows_kernel<FMT, GROUP, F16, TC, GATED, MASKED>;
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(kern), done);
  if (err != cudaSuccess) return err;
  GemvMaps maps;
  const uint64_t row_bytes = FMT == 4 ? (uint64_t)a.K / 2 : (uint64_t)a.K * 2;
  for (int i = 0; i < (GATED ? 2 : 1); ++i)
    if (!make_map(&maps.w[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.w[i], row_bytes, a.N, 128,
                  GATED ? 8 : 16, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
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
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, maps, a, p);
}

template <int FMT, int GROUP, bool F16, bool GATED>
cudaError_t launch_tc(const GemvArgs& a, const GemvPlan& p, cudaStream_t st) {
  switch (p.tc) {
    case 1:
      if constexpr (FMT == 4 && GROUP == 128)
        if (p.masked) return launch_one<FMT, GROUP, F16, 1, GATED, true>(a, p, st);
      return launch_one<FMT, GROUP, F16, 1, GATED>(a, p, st);
    case 2: return launch_one<FMT, GROUP, F16, 2, GATED>(a, p, st);
    case 3: return launch_one<FMT, GROUP, F16, 3, GATED>(a, p, st);
    default: return launch_one<FMT, GROUP, F16, 4, GATED>(a, p, st);
  }
}

template <bool F16>
cudaError_t launch_fmt(const GemvArgs& a, const GemvPlan& p, cudaStream_t st) {
  if (a.fmt == 16)
    return a.gated ? launch_tc<16, 128, F16, true>(a, p, st)
                   : launch_tc<16, 128, F16, false>(a, p, st);
  if (a.gated) {
    if constexpr (F16) return cudaErrorInvalidValue;  // int4 blocks take bf16 rows
    else return launch_tc<4, 128, F16, true>(a, p, st);
  }
  if (a.group == 128) return launch_tc<4, 128, F16, false>(a, p, st);
  if (a.group == 64) return launch_tc<4, 64, F16, false>(a, p, st);
  return launch_tc<4, 32, F16, false>(a, p, st);
}

}  // namespace

thread_local TestHold g_test_hold;

int device_sms() {
  static std::atomic<int> sms[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int n = sms[dev];
  if (n == 0) {  // racing threads store the same value
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    sms[dev] = n;
  }
  return n;
}

cudaError_t allow_smem(const void* kernel, std::atomic<bool>* done) {
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

cudaError_t launch_gemv_rows(const GemvArgs& a, cudaStream_t st, bool early) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  GemvPlan p = make_gemv_plan(a, sms);
  p.early = early;
  if (g_test_hold.hold) {
    p.drop = 1;
    if (g_test_hold.budget > 0) p.limit = g_test_hold.budget;
  }
  if (p.smem > kSmemMax || p.parts > sms) return cudaErrorInvalidValue;
  return a.f16 ? launch_fmt<true>(a, p, st) : launch_fmt<false>(a, p, st);
}

}  // namespace moe
