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
  return a && b && x < y + bn && y < x + an;
}

// ------------------------------------------------------------------ matvec

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

// Workspace of one or two streaming products: a first block of 256 bytes (status words of the
// tensor-core kernels), the row tiles' counters, the partial sums.
struct GemvWs {
  size_t counters, partial, total;
};
GemvWs gemv_ws(size_t partial_bytes, size_t n_counters) {
  GemvWs w;
  w.counters = kAlign;
  w.partial = align_up(w.counters + 4 * n_counters);
  w.total = align_up(w.partial + partial_bytes);
  return w;
}

}  // namespace

extern "C" {

moe_status moe_matvec_validate(const moe_matrix* M) { return matvec_validate(M); }

size_t moe_matvec_workspace_size(const moe_matrix* M) {
  if (matvec_validate(M) != MOE_OK) return 0;
  size_t part, cnt;
  gemv_scratch(matvec_args(M), &part, &cnt);
  return gemv_ws(part, cnt).total;
}

moe_status moe_matvec(const moe_matrix* M, const void* x, void* y, void* ws, size_t ws_bytes,
                      moe_stream_t stream) {
  moe_status s = matvec_validate(M);
  if (s != MOE_OK) return s;
  if (!x || !aligned(x, 16) || !y || !aligned(y, type_bytes(M->y_type))) return MOE_ERR_INVALID_ARG;
  const size_t T = M->T, N = M->N, K = M->K;
  const size_t yb = ((T - 1) * (size_t)M->ldy + N) * type_bytes(M->y_type);
  if (overlap(y, yb, x, ((T - 1) * (size_t)M->ldx + K) * 2) || overlap(y, yb, M->w, N * K / 2) ||
      overlap(y, yb, M->s, N * (K / M->group) * 2) || overlap(y, yb, M->bias, N * 4))
    return MOE_ERR_INVALID_ARG;
  GemvArgs a = matvec_args(M);
  size_t part, cnt;
  gemv_scratch(a, &part, &cnt);
  const GemvWs w = gemv_ws(part, cnt);
  if (!ws || !aligned(ws, kAlign) || ws_bytes < w.total) return MOE_ERR_WORKSPACE;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.x = static_cast<const uint16_t*>(x);
  a.y = y;
  a.counters = reinterpret_cast<int32_t*>(base + w.counters);
  a.partial = reinterpret_cast<float*>(base + w.partial);
  MOE_TRY(launch_gemv_rows(a, reinterpret_cast<cudaStream_t>(stream), false));
  return MOE_OK;
}

}  // extern "C"
