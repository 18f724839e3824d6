// Internal interfaces of the dense operators (moe_matvec, moe_ffn_forward, moe_ffn_backward):
// the argument blocks of their kernels and the device helpers both kernel families share.
#pragma once

#include <cuda_fp16.h>

#include "pipeline.cuh"

namespace moe {

constexpr int kMaxDevices = 64;      // per-device caches
constexpr int kGemvMaxRows = 32;     // activation rows of the streaming kernels

// Multiprocessors of the current device (0 on error), cached per device.
int device_sms();
// Opts a kernel into the largest dynamic shared memory on the current device, once per device;
// `done` is the kernel's own array of kMaxDevices flags.
cudaError_t allow_smem(const void* kernel, bool* done);

// ------------------------------------------------------------------ activations

// act(g): silu g / (1 + e^-g), or gelu in its tanh form. In fp32; the fast exponential and
// division are off by a few units in the last place of fp32, far below the 16-bit rounding
// that follows (e^-g overflowing to infinity gives the limit 0).
template <int ACT> __device__ __forceinline__ float act_value(float g) {
  if constexpr (ACT == MOE_ACT_SILU) {
    return g * __frcp_rn(1.f + __expf(-g));
  } else {
    const float z = 0.7978845608028654f * (g + 0.044715f * g * g * g);
    return 0.5f * g * (1.f + tanhf(z));
  }
}

// act(g) and act'(g). The polynomial of gelu's derivative takes |g| <= 16: beyond it tanh is
// exactly +-1 and 1 - tanh^2 is 0, while g^2 could overflow and give 0 * inf.
template <int ACT> __device__ __forceinline__ void act_grad(float g, float* a, float* da) {
  if constexpr (ACT == MOE_ACT_SILU) {
    const float s = __frcp_rn(1.f + __expf(-g));
    *a = g * s;
    *da = fmaf(g * s, 1.f - s, s);
  } else {
    const float t = tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g));
    const float c = fminf(fmaxf(g, -16.f), 16.f);
    *a = 0.5f * g * (1.f + t);
    *da = 0.5f * (1.f + t) +
          0.5f * c * (1.f - t * t) * (0.7978845608028654f * (1.f + 0.134145f * c * c));
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
  float* partial;          // K parts: fp32 sums [tile][part][...]
  int32_t* counters;       // one per row tile, zero between calls
};

// Bytes of partial sums and number of counters a call needs (0 when K is not split).
void gemv_scratch(const GemvArgs& a, size_t* partial_bytes, size_t* n_counters);
cudaError_t launch_gemv_rows(const GemvArgs& a, cudaStream_t st, bool pdl);

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
  int32_t* counters;   // ffn_counters() of them, zero between calls
};

// Workspace of the tensor-core kernels: bytes of partial sums, number of counters.
size_t ffn_partial_bytes(const FfnArgs& a, bool backward);
size_t ffn_counters();

cudaError_t launch_ffn_gate_up(const FfnArgs& a, cudaStream_t st);          // x -> h (and pre)
cudaError_t launch_ffn_down(const FfnArgs& a, cudaStream_t st);             // h -> y
cudaError_t launch_ffn_gate_grad(const FfnArgs& a, cudaStream_t st);        // dy, pre -> dg, du, h
cudaError_t launch_ffn_grads(const FfnArgs& a, cudaStream_t st);            // -> dx and the weights'

}  // namespace moe
