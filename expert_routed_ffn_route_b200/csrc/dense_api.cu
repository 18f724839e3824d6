// C entry points of the dense operators: host-side validation, workspace layout and kernel
// sequencing, in the manner of the layer's own entry points.
#include <cstring>

#include "dense.cuh"

using namespace moe;

namespace {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

#define MOE_TRY(expr)                           \
  do {                                          \
    cudaError_t _e = (expr);                    \
    if (_e != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)

// Whether [a, a + an) and [b, b + bn) share a byte.
inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && an && bn && x < y + bn && y < x + an;
}

struct Range {
  const void* p;
  size_t n;
};

// Whether one of the first n_out ranges (outputs) overlaps any other.
bool outputs_overlap(const Range* r, int n_out, int n) {
  for (int i = 0; i < n_out; ++i)
    for (int j = i + 1; j < n; ++j)
      if (overlap(r[i].p, r[i].n, r[j].p, r[j].n)) return true;
  return false;
}

// ------------------------------------------------------------------ matvec

// Whether a row of a (an bytes, rows as bytes apart) shares a byte with a row of b: both may be
// columns of one wider array, whose rows interleave without overlapping.
bool rows_overlap(const void* a, size_t an, size_t as, const void* b, size_t bn, size_t bs, int T) {
  if (!overlap(a, (T - 1) * as + an, b, (T - 1) * bs + bn)) return false;
  for (int i = 0; i < T; ++i)
    for (int j = 0; j < T; ++j)
      if (overlap(static_cast<const char*>(a) + i * as, an, static_cast<const char*>(b) + j * bs, bn))
        return true;
  return false;
}

inline size_t type_bytes(int t) { return t == MOE_T_FP32 ? 4 : 2; }

moe_status matvec_validate(const moe_matrix* M) {
  if (!M) return MOE_ERR_INVALID_ARG;
  if (M->T < 1 || M->N < 1 || M->K < 1) return MOE_ERR_INVALID_ARG;
  if (M->group != 32 && M->group != 64 && M->group != 128) return MOE_ERR_INVALID_ARG;
  if (M->K % M->group) return MOE_ERR_INVALID_ARG;
  if (M->x_type != MOE_T_BF16 && M->x_type != MOE_T_FP16) return MOE_ERR_INVALID_ARG;
  if (M->y_type != M->x_type && M->y_type != MOE_T_FP32) return MOE_ERR_INVALID_ARG;
  if (M->T > kGemvMaxRows || M->K > 32768 || M->N > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (M->ldx < M->K || M->ldx % 8 || M->ldy < M->N) return MOE_ERR_INVALID_ARG;
  if (M->ldx > (1LL << 40) || M->ldy > (1LL << 40)) return MOE_ERR_UNSUPPORTED;
  if (!M->w || !aligned(M->w, 16) || !M->s || !aligned(M->s, 2)) return MOE_ERR_INVALID_ARG;
  if (M->bias && !aligned(M->bias, 4)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

GemvArgs matvec_args(const moe_matrix* M) {
  GemvArgs a{};
  a.w[0] = M->w;
  a.s[0] = static_cast<const uint16_t*>(M->s);
  a.bias = M->bias;
  a.ldx = M->ldx;
  a.ldy = M->ldy;
  a.T = M->T;
  a.N = M->N;
  a.K = M->K;
  a.fmt = 4;
  a.group = M->group;
  a.f16 = M->x_type == MOE_T_FP16;
  a.y32 = M->y_type == MOE_T_FP32;
  return a;
}

// A workspace begins with a block of status words and kWsCounters counters, in the same place for
// every call, so that calls of any matrices and blocks can use one workspace in turn: what one
// leaves there (partial sums, h) never lies where the next expects its counters at zero. Then come
// the partial sums. A split product of more row tiles than that (over 131072 outputs) has its
// counters behind the others and clears them itself, before its kernel.
constexpr size_t kWsCounters = 8192;

struct GemvWs {
  size_t counters, partial, total;
  bool clear;
};
GemvWs gemv_ws(size_t partial_bytes, size_t n_counters) {
  GemvWs w;
  const size_t fixed = kAlign + 4 * kWsCounters;
  w.clear = n_counters > kWsCounters;
  w.counters = w.clear ? fixed : kAlign;
  w.partial = w.clear ? align_up(fixed + 4 * n_counters) : fixed;
  w.total = align_up(w.partial + partial_bytes);
  return w;
}
// A product that is not split uses the status words alone.
GemvWs matvec_ws(size_t partial_bytes, size_t n_counters) {
  GemvWs w = gemv_ws(partial_bytes, n_counters);
  if (n_counters == 0) w.total = kAlign;
  return w;
}

// ------------------------------------------------------------------ dense gated block

constexpr int kMaxWidth = 32768, kMaxFfnRows = 1 << 20;
static_assert(kMaxWidth / 8 <= kWsCounters && kFfnCounters <= kWsCounters, "counters");

inline bool is_16bit(const moe_ffn* F) {
  return F->bank.fmt == MOE_W_BF16 || F->bank.fmt == MOE_W_FP16;
}

moe_status ffn_validate(const moe_ffn* F) {
  if (!F) return MOE_ERR_INVALID_ARG;
  if (F->T < 1 || F->d < 1 || F->f < 1) return MOE_ERR_INVALID_ARG;
  if (F->act != MOE_ACT_SILU && F->act != MOE_ACT_GELU) return MOE_ERR_INVALID_ARG;
  const moe_bank& b = F->bank;
  if (b.n_exp != 1) return MOE_ERR_INVALID_ARG;
  if (!is_16bit(F) && b.fmt != MOE_W_INT4)
    return b.fmt == MOE_W_INT8 || b.fmt == MOE_W_NVFP4 ? MOE_ERR_UNSUPPORTED
                                                       : MOE_ERR_INVALID_ARG;
  const int step = is_16bit(F) ? 8 : 128;
  if (F->d % step || F->f % step) return MOE_ERR_INVALID_ARG;
  if (F->d > kMaxWidth || F->f > kMaxWidth || F->T > kMaxFfnRows) return MOE_ERR_UNSUPPORTED;
  for (const void* p : {b.w_gate, b.w_up, b.w_down})
    if (!p || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (b.fmt == MOE_W_INT4) {
    if (b.group != kGroup) return MOE_ERR_INVALID_ARG;
    for (const void* p : {b.s_gate, b.s_up, b.s_down})
      if (!p || !aligned(p, 2)) return MOE_ERR_INVALID_ARG;
    if (F->T > kGemvMaxRows) return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

// Up to 32 rows the weights are streamed through the GEMV kernels. bf16, us streamed / on the tensor
// cores (neither keeping g and u):
//             512 x 1024   1024 x 4096  2560 x 1024  4096 x 2048  4096 x 4096  2560 x 10240
//   8 rows    6.2 / 11.7   12.3 / 21.4  9.5 / 19.5   17.0 / 31.6  33.3 / 45.5  39.6 / 59.5
//   16        8.3 / 11.7   14.3 / 19.6  12.7 / 19.5  19.2 / 27.6  37.3 / 33.2  38.9 / 61.9
//   32        12.4 / 11.7  17.7 / 19.4  15.9 / 18.1  25.5 / 25.7  39.9 / 33.5  46.0 / 48.0
// So two of the six are better off on the tensor cores below the limit (512 x 1024 at 32 rows, by 6 %;
// 4096 x 4096 from 16 rows, by 8 to 19 %): the limit is one number for all widths, and a rule with the
// widths in it is not made. A call that keeps g and u for a backward pass takes the tensor-core
// kernels at any T (they write them).
inline bool streams(const moe_ffn* F, const void* pre) {
  return !is_16bit(F) || (F->T <= kGemvMaxRows && !pre);
}

// Product i of the streamed block: 0 gate/up, 1 down.
GemvArgs ffn_gemv(const moe_ffn* F, int i) {
  GemvArgs a{};
  const moe_bank& b = F->bank;
  a.w[0] = i ? b.w_down : b.w_gate;
  a.w[1] = i ? nullptr : b.w_up;
  a.s[0] = static_cast<const uint16_t*>(i ? b.s_down : b.s_gate);
  a.s[1] = static_cast<const uint16_t*>(i ? nullptr : b.s_up);
  a.T = F->T;
  a.N = i ? F->d : F->f;
  a.K = i ? F->f : F->d;
  a.ldx = a.K;
  a.ldy = a.N;
  a.fmt = is_16bit(F) ? 16 : 4;
  a.group = kGroup;
  a.f16 = b.fmt == MOE_W_FP16;
  a.gated = !i;
  a.act = F->act;
  a.pairs = F->T <= kPairRows;
  if (i && a.pairs) a.T = 2 * F->T;
  return a;
}

// Workspace of a block: the status words, the counters (at most 4096, see kMaxWidth) and partial
// sums of the streaming kernels or the tensor-core kernels (a call's products run one after the
// other and share them), h, and for the backward pass dg, du.
struct FfnWs {
  GemvWs g;
  size_t partial_bytes, h, dg, du, total;
};
FfnWs ffn_ws(const moe_ffn* F, bool backward) {
  FfnWs w;
  size_t part = 0;
  if (F->T <= kGemvMaxRows)
    for (int i = 0; i < 2; ++i) {
      size_t p, c;
      gemv_scratch(ffn_gemv(F, i), &p, &c);
      part = std::max(part, p);
    }
  if (is_16bit(F) && (backward || F->T > kGemvMaxRows))
    part = std::max(part, ffn_partial_bytes(backward));
  w.g = gemv_ws(part, kWsCounters);
  w.partial_bytes = part;
  const size_t rows = align_up((size_t)F->T * F->f * 2);
  w.h = w.g.total;
  w.dg = w.h + (F->T <= kPairRows ? align_up((size_t)F->T * F->f * 4) : rows);
  w.du = w.dg + (backward ? rows : 0);
  w.total = w.du + (backward ? rows : 0);
  return w;
}

moe_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  return ws && aligned(ws, kAlign) && ws_bytes >= need ? MOE_OK : MOE_ERR_WORKSPACE;
}

inline size_t weight_bytes(const moe_ffn* F) {
  const size_t n = (size_t)F->d * F->f;
  return is_16bit(F) ? 2 * n : n / 2;
}
// Scales of one int4 matrix (0 when the bank has none, whatever its pointers hold).
inline size_t scale_bytes(const moe_ffn* F) {
  return is_16bit(F) ? 0 : (size_t)F->d * F->f / kGroup * 2;
}

FfnArgs ffn_args(const moe_ffn* F, const FfnWs& w, void* ws) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  FfnArgs a{};
  a.T = F->T;
  a.d = F->d;
  a.f = F->f;
  a.act = F->act;
  a.f16 = F->bank.fmt == MOE_W_FP16;
  a.w_gate = F->bank.w_gate;
  a.w_up = F->bank.w_up;
  a.w_down = F->bank.w_down;
  a.h = base + w.h;
  a.dg = base + w.dg;
  a.du = base + w.du;
  a.status = reinterpret_cast<int32_t*>(base);
  a.counters = reinterpret_cast<int32_t*>(base + w.g.counters);
  a.partial = reinterpret_cast<float*>(base + w.g.partial);
  a.partial_bytes = w.partial_bytes;
  return a;
}

// Reads and clears the status and site words at the start of a workspace.
moe_status read_status(void* ws, int32_t* code, int32_t* site, cudaStream_t st) {
  int32_t words[kSiteWord + 1] = {};
  MOE_TRY(cudaMemcpyAsync(words, ws, sizeof(words), cudaMemcpyDeviceToHost, st));
  MOE_TRY(cudaStreamSynchronize(st));
  MOE_TRY(cudaMemsetAsync(ws, 0, sizeof(words), st));
  *code = words[0] == DEV_OK ? MOE_OK : words[0] == DEV_TIMEOUT ? MOE_ERR_TIMEOUT : MOE_ERR_DEVICE;
  *site = words[kSiteWord];
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_matvec_validate(const moe_matrix* M) { return matvec_validate(M); }

size_t moe_matvec_workspace_size(const moe_matrix* M) {
  if (matvec_validate(M) != MOE_OK) return 0;
  size_t part, cnt;
  gemv_scratch(matvec_args(M), &part, &cnt);
  return matvec_ws(part, cnt).total;
}

moe_status moe_matvec(const moe_matrix* M, const void* x, void* y, void* ws, size_t ws_bytes,
                      moe_stream_t stream) {
  moe_status s = matvec_validate(M);
  if (s != MOE_OK) return s;
  if (!x || !aligned(x, 16) || !y || !aligned(y, type_bytes(M->y_type))) return MOE_ERR_INVALID_ARG;
  const size_t T = M->T, N = M->N, K = M->K;
  const size_t ysize = type_bytes(M->y_type), yb = ((T - 1) * (size_t)M->ldy + N) * ysize;
  const Range y_r{y, yb}, x_r{x, ((T - 1) * (size_t)M->ldx + K) * 2}, w_r{M->w, N * K / 2},
      s_r{M->s, N * (K / M->group) * 2}, b_r{M->bias, N * 4};
  const Range out[] = {y_r, w_r, s_r, b_r};
  if (outputs_overlap(out, 1, 4) ||
      rows_overlap(y, N * ysize, M->ldy * ysize, x, K * 2, M->ldx * 2, M->T))
    return MOE_ERR_INVALID_ARG;
  GemvArgs a = matvec_args(M);
  size_t part, cnt;
  gemv_scratch(a, &part, &cnt);
  const GemvWs w = matvec_ws(part, cnt);
  if (!ws || !aligned(ws, kAlign) || ws_bytes < w.total) return MOE_ERR_WORKSPACE;
  // (the workspace holds partial sums and counters while inputs are still read)
  const Range held[] = {{ws, w.total}, y_r, x_r, w_r, s_r, b_r};
  if (outputs_overlap(held, 1, 6)) return MOE_ERR_INVALID_ARG;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.status = reinterpret_cast<int32_t*>(base);
  a.x = static_cast<const uint16_t*>(x);
  a.y = y;
  a.counters = reinterpret_cast<int32_t*>(base + w.counters);
  a.partial = reinterpret_cast<float*>(base + w.partial);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (w.clear) MOE_TRY(cudaMemsetAsync(a.counters, 0, 4 * cnt, st));
  MOE_TRY(launch_gemv_rows(a, st, false));
  return MOE_OK;
}

moe_status moe_matvec_device_status(const moe_matrix* M, void* ws, size_t ws_bytes, int32_t* code,
                                    int32_t* site, moe_stream_t stream) {
  moe_status s = matvec_validate(M);
  if (s != MOE_OK) return s;
  if (!code || !site) return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, kAlign) || ws_bytes < moe_matvec_workspace_size(M))
    return MOE_ERR_WORKSPACE;
  return read_status(ws, code, site, reinterpret_cast<cudaStream_t>(stream));
}

moe_status moe_test_inject_dense_hold(int32_t hold, int32_t budget_cycles) {
  if (budget_cycles < 0) return MOE_ERR_INVALID_ARG;
  g_test_hold.hold = hold != 0;
  g_test_hold.budget = budget_cycles;
  return MOE_OK;
}

moe_status moe_ffn_validate(const moe_ffn* F) { return ffn_validate(F); }

size_t moe_ffn_workspace_size(const moe_ffn* F, int32_t backward) {
  if (ffn_validate(F) != MOE_OK || (backward && !is_16bit(F))) return 0;
  return ffn_ws(F, backward != 0).total;
}

moe_status moe_ffn_forward(const moe_ffn* F, const void* x, void* y, float* pre, void* ws,
                           size_t ws_bytes, moe_stream_t stream) {
  moe_status s = ffn_validate(F);
  if (s != MOE_OK) return s;
  if (pre && !is_16bit(F)) return MOE_ERR_UNSUPPORTED;
  if (!x || !aligned(x, 16) || !y || !aligned(y, 16) || !aligned(pre, 16))
    return MOE_ERR_INVALID_ARG;
  const FfnWs w = ffn_ws(F, pre != nullptr);
  if ((s = check_ws(ws, ws_bytes, w.total)) != MOE_OK) return s;
  const size_t xb = (size_t)F->T * F->d * 2, wb = weight_bytes(F), sb = scale_bytes(F);
  const moe_bank& b = F->bank;
  const Range r[] = {{y, xb}, {pre, (size_t)F->T * F->f * 8}, {ws, w.total}, {x, xb},
                     {b.w_gate, wb}, {b.w_up, wb}, {b.w_down, wb}, {b.s_gate, sb}, {b.s_up, sb},
                     {b.s_down, sb}};
  if (outputs_overlap(r, 3, 10)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  FfnArgs a = ffn_args(F, w, ws);
  if (streams(F, pre)) {
    for (int i = 0; i < 2; ++i) {
      GemvArgs g = ffn_gemv(F, i);
      g.x = static_cast<const uint16_t*>(i ? a.h : x);
      g.y = i ? y : a.h;
      g.status = a.status;
      g.counters = a.counters;
      g.partial = a.partial;
      MOE_TRY(launch_gemv_rows(g, st, i == 1));
    }
    return MOE_OK;
  }
  a.x = x;
  a.y = y;
  a.pre = pre;
  MOE_TRY(launch_ffn_gate_up(a, st));
  MOE_TRY(launch_ffn_down(a, st));
  return MOE_OK;
}

moe_status moe_ffn_backward(const moe_ffn* F, const void* x, const void* dy, const float* pre,
                            void* dx, void* dw_gate, void* dw_up, void* dw_down, void* ws,
                            size_t ws_bytes, moe_stream_t stream) {
  moe_status s = ffn_validate(F);
  if (s != MOE_OK) return s;
  if (!is_16bit(F)) return MOE_ERR_UNSUPPORTED;
  for (const void* p : {x, dy, static_cast<const void*>(pre)})
    if (!p || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {dx, dw_gate, dw_up, dw_down})
    if (!aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (!dx && !dw_gate && !dw_up && !dw_down) return MOE_ERR_INVALID_ARG;
  const FfnWs w = ffn_ws(F, true);
  if ((s = check_ws(ws, ws_bytes, w.total)) != MOE_OK) return s;
  const size_t xb = (size_t)F->T * F->d * 2, wb = weight_bytes(F);
  const moe_bank& b = F->bank;
  const Range r[] = {{dx, xb}, {dw_gate, wb}, {dw_up, wb}, {dw_down, wb},
                     {ws, w.total}, {x, xb}, {dy, xb},
                     {pre, (size_t)F->T * F->f * 8}, {b.w_gate, wb}, {b.w_up, wb}, {b.w_down, wb}};
  if (outputs_overlap(r, 5, 11)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  FfnArgs a = ffn_args(F, w, ws);
  a.x = x;
  a.dy = dy;
  a.pre = const_cast<float*>(pre);
  a.dx = dx;
  a.dw_gate = dw_gate;
  a.dw_up = dw_up;
  a.dw_down = dw_down;
  MOE_TRY(launch_ffn_gate_grad(a, st));
  MOE_TRY(launch_ffn_grads(a, st));
  return MOE_OK;
}

moe_status moe_ffn_device_status(const moe_ffn* F, void* ws, size_t ws_bytes, int32_t* code,
                                 int32_t* site, moe_stream_t stream) {
  moe_status s = ffn_validate(F);
  if (s != MOE_OK) return s;
  if (!code || !site) return MOE_ERR_INVALID_ARG;
  if ((s = check_ws(ws, ws_bytes, ffn_ws(F, false).total)) != MOE_OK) return s;
  return read_status(ws, code, site, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
