// Internal interfaces of the dense operators (moe_matvec, moe_ffn_forward, moe_ffn_backward):
// the argument blocks of their kernels and the device helpers both kernel families share.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "pipeline.cuh"

namespace moe {

constexpr int kMaxDevices = 64;      // per-device caches
constexpr int kGemvMaxRows = 32;     // activation rows of the streaming kernels
// Up to so many rows a streamed block passes h on as two 16-bit rows, the rounded value and the
// rounded rest (together 16 bits or more): the down product has eight columns an instruction
// anyway, so the second row costs nothing and y is rounded once.
constexpr int kPairRows = 4;

// Multiprocessors of the current device (0 on error), cached per device.
int device_sms();
// Opts a kernel into the largest dynamic shared memory on the current device, once per device;
// `done` is the kernel's own array of kMaxDevices flags.
cudaError_t allow_smem(const void* kernel, std::atomic<bool>* done);

// Test control of the calling thread's launches (moe_test_inject_dense_hold). It is a kernel
// argument: a word in the workspace, as the layer's, cost ordinary calls 1 to 4 %.
struct TestHold {
  int hold = 0, budget = 0;
};
extern thread_local TestHold g_test_hold;

// mbar_wait with a bound of its own.
__device__ __forceinline__ bool mbar_wait_within(uint64_t* bar, uint32_t parity, long long limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > limit) return false;
  }
  return true;
}

// Starts the fetch of a tensor map (a kernel's first TMA copy waits for its map otherwise).
__device__ __forceinline__ void prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ------------------------------------------------------------------ activations

// Both activations are g sigma(k): silu with k = g, gelu in its tanh form with
// k = 2 sqrt(2 / pi) (g + 0.044715 g^3), since (1 + tanh z) / 2 = sigma(2 z). So one exponential
// and one reciprocal serve value and slope,
//   act = g s,  act' = s + g s (1 - s) k',   s = sigma(k),
// and no difference of near-equal numbers is taken where act is small. In fp32 with the
// approximate exponential and reciprocal instructions (a few units in the last place, far
// below the 16-bit rounding that follows; the IEEE reciprocal and tanhf made the gate-gradient
// epilogue issue 63 instructions a value). e^-k overflowing to infinity gives the limit s = 0.
__device__ __forceinline__ float sigmoid_approx(float k) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * k));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}

constexpr float kGelu1 = 1.5957691216057308f;              // 2 sqrt(2 / pi)
constexpr float kGelu3 = 1.5957691216057308f * 0.044715f;

template <int ACT> __device__ __forceinline__ float act_value(float g) {
  if constexpr (ACT == MOE_ACT_SILU) return g * sigmoid_approx(g);
  else return g * sigmoid_approx(g * fmaf(kGelu3, g * g, kGelu1));
}

// act(g) and act'(g). Gelu's k' takes |g| <= 16: beyond it s (1 - s) is 0 in fp32, while g^2
// could overflow and give 0 * inf.
template <int ACT> __device__ __forceinline__ void act_grad(float g, float* a, float* da) {
  if constexpr (ACT == MOE_ACT_SILU) {
    const float s = sigmoid_approx(g);
    *a = g * s;
    *da = fmaf(*a, 1.f - s, s);
  } else {
    const float s = sigmoid_approx(g * fmaf(kGelu3, g * g, kGelu1));
    const float c = fminf(fmaxf(g, -16.f), 16.f);
    *a = g * s;
    *da = fmaf(c * s * (1.f - s), fmaf(3.f * kGelu3, c * c, kGelu1), s);
  }
}

// Two fp32 values as a pair of the 16-bit type (bf16 or, F16, fp16), nearest even.
template <bool F16> __device__ __forceinline__ uint32_t pack16x2(float lo, float hi) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16x2(lo, hi);
  }
}
template <bool F16> __device__ __forceinline__ uint16_t round16(float v) {
  if constexpr (F16) {
    const __half h = __float2half_rn(v);
    return *reinterpret_cast<const uint16_t*>(&h);
  } else {
    return f32_to_bf16_rn(v);
  }
}

template <bool F16> __device__ __forceinline__ float value16(uint16_t b) {
  if constexpr (F16) return __half2float(__ushort_as_half(b));
  else return bf16_to_f32(b);
}

// ------------------------------------------------------------------ streaming kernels

// One product of up to 32 activation rows with a weight matrix (dense_gemv.cu).
struct GemvArgs {
  const void* w[2];        // int4 words or 16-bit values [N][K]; w[1]: the up matrix (gated)
  const uint16_t* s[2];    // bf16 scales [N][K / group] (int4)
  const float* bias;       // fp32 [N] or NULL (not gated)
  const uint16_t* x;       // 16-bit rows, ldx elements apart
  void* y;                 // 16-bit (the activations' type) or fp32 rows, ldy elements apart
  long long ldx, ldy;
  int T, N, K;
  int fmt, group;          // 4 (group 32, 64, 128) or 16
  bool f16, y32;           // activations (and 16-bit weights) fp16; output fp32
  int gated, act;          // y = act(w[0] x) * (w[1] x)
  int pairs;               // rows 2 t and 2 t + 1 (of y if gated, else of x) are the rounded value
                           // of token t and the rounded rest: see kPairRows
  float* partial;          // K parts: fp32 sums [tile][part][...]
  int32_t* counters;       // one per row tile, zero between calls
  int32_t* status;
};

// Bytes of partial sums and number of counters a call needs (0 when K is not split).
void gemv_scratch(const GemvArgs& a, size_t* partial_bytes, size_t* n_counters);
// early: the kernel before in the stream is one of these that writes no weights (their copies then
// start before it ends).
cudaError_t launch_gemv_rows(const GemvArgs& a, cudaStream_t st, bool early);

// ------------------------------------------------------------------ tensor-core kernels

// A dense gated block on the tensor cores (dense_gemm.cu). 16-bit operands of one type.
struct FfnArgs {
  const void* w_gate;  // [f][d]
  const void* w_up;    // [f][d]
  const void* w_down;  // [d][f]
  const void* x;       // [T][d]
  void* h;             // [T][f]
  float* pre;          // fp32 [2][T][f]: gate, then up, before the activation (or NULL)
  void* y;             // [T][d]
  const void* dy;      // [T][d]
  void* dg;            // [T][f]
  void* du;            // [T][f]
  void* dx;            // [T][d] or NULL
  void* dw_gate;       // [f][d] or NULL
  void* dw_up;         // [f][d] or NULL
  void* dw_down;       // [d][f] or NULL
  int T, d, f, act;
  bool f16;
  int32_t* status;
  float* partial;      // sums of tiles split along K
  size_t partial_bytes;
  int32_t* counters;   // kFfnCounters of them, zero between calls
};

// A launch cuts the leftover tiles of at most two rounds of 74 CTA pairs; a counter for each of the
// 16 epilogue warps of a pair.
constexpr size_t kFfnCounters = 2 * 74 * 16;

// Workspace of the tensor-core kernels, whatever the sizes: bytes of partial sums (a forward
// launch splits one leftover round of tiles, a backward launch at most two).
size_t ffn_partial_bytes(bool backward);

cudaError_t launch_ffn_gate_up(const FfnArgs& a, cudaStream_t st);          // x -> h (and pre)
cudaError_t launch_ffn_down(const FfnArgs& a, cudaStream_t st);             // h -> y
cudaError_t launch_ffn_gate_grad(const FfnArgs& a, cudaStream_t st);        // dy, pre -> dg, du, h
cudaError_t launch_ffn_grads(const FfnArgs& a, cudaStream_t st);            // -> dx and the weights'

}  // namespace moe
