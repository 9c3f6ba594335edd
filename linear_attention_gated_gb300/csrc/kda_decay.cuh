// kda_decay.cuh -- launch parameters shared by the kernels of the linear
// attention with a decay for each head (kda_decay_*.cu).
#pragma once

#include "kda_common.cuh"

namespace kda {

constexpr int kDecayChunk = 64;  // tokens of a chunk

// 2^x, 0 below 2^-126 (the hardware's approximation, 2 ulp)
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The token tensors of one call. Strides in elements; heads of q, k: Hqk, of v: Hv.
struct DecayProblem {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const void* g;           // log decay: BF16 [Ttot, Hv] (per token) or FP32 [Hv]
  const int64_t* cu;       // device cu_seqlens [N + 1], or null for sequences of T tokens
  int64_t qt, qh, kt, kh, vt, vh;
  int64_t N, T, Ttot;
  int Hqk, Hv, r;          // r = Hv / Hqk
  int per_token;
  float scale;
  int64_t seg;             // tokens of a segment, 0 for whole sequences (decay_segment_tokens)
  int64_t longest;         // tokens of the longest sequence
  const int64_t* cu_host;  // host offsets (packed layout), for the call only
  int32_t* status;         // bit 0: a bounded device wait gave up; bit 2: a device slot index out of the pool
};

// Where states come from and go to: [slots or N, Hv, 128, 128] value-first.
struct DecayStates {
  const void* in;          // null: zeros
  void* out;               // null: not written
  int bf16;
  const int32_t* slots;    // pool slot of each sequence, or null (slot n)
  int64_t num_slots;
};

struct DecayGrads {
  const __nv_bfloat16* d_o;  // [Ttot, Hv, 128]
  const float* d_hT;         // [N, Hv, 128, 128] or null (zeros)
  __nv_bfloat16* dq;         // [Ttot, Hqk, 128]
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;         // [Ttot, Hv, 128]
  __nv_bfloat16* dg;         // [Ttot, Hv] or null
  float* dh0;                // [N, Hv, 128, 128] or null
};

// First token and length of sequence n. The device offsets are held inside the tensors, so
// offsets that disagree with the checked host mirror never send a kernel outside its buffers.
struct DecaySpan {
  int64_t t0, len;
};
__device__ __forceinline__ DecaySpan decay_span(const DecayProblem& P, int64_t n) {
  if (!P.cu) return DecaySpan{n * P.T, P.T};
  int64_t a = P.cu[n], b = P.cu[n + 1];
  a = a < 0 ? 0 : (a > P.Ttot ? P.Ttot : a);
  b = b < a ? a : (b > P.Ttot ? P.Ttot : b);
  return DecaySpan{a, b - a};
}

// Log decay of one token in base 2. A decay of zero (log decay -inf, a reset of the state) becomes
// 2^-160, which is 0 in FP32 and leaves running sums finite; NaN stays NaN.
__device__ __forceinline__ float decay_log2(float g) {
  const float x = g * 1.4426950408889634f;
  return x < -160.f ? -160.f : x;
}
__device__ __forceinline__ float decay_g(const DecayProblem& P, int64_t tok, int h) {
  return P.per_token ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(P.g)[tok * P.Hv + h])
                     : reinterpret_cast<const float*>(P.g)[h];
}

// Tokens of the segments sequences are cut into, 0 for none. cu: host offsets or null.
int64_t decay_segment_tokens(const int64_t* cu, int64_t N, int64_t T, int64_t Hv);
// Workspace: the segments' states, then (training) what the backward needs.
size_t decay_workspace_bytes(int64_t N, int64_t Ttot, int64_t Hqk, int64_t Hv, int64_t seg, bool training, bool per_token);
// Blocks of the kernel that sums dq and dk over a group's heads.
int64_t decay_group_sum_blocks(const DecayProblem& P);
cudaError_t launch_decay_forward(const DecayProblem& P, const DecayStates& st, __nv_bfloat16* o, void* ws, cudaStream_t s);
cudaError_t launch_decay_backward(const DecayProblem& P, const float* h0, const float* hT, const DecayGrads& g, void* ws,
                                  cudaStream_t s);

}  // namespace kda
