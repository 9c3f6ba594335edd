// kda_decay.cuh -- launch parameters shared by the kernels of the linear
// attention with a decay for each head (kda_decay_*.cu).
#pragma once

#include "kda_common.cuh"
#include "tc.cuh"

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

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ uint32_t pack2(float2 x) { return pack2(x.x, x.y); }
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
// The factors 2^x that a state is multiplied by one after the other. Each rounded to FP32 by itself, a slow fixed decay's would
// be off by the same part of a step every time (states 6e-5 off after 1536 chunks). So what a rounding leaves goes
// into the next factor, and their product stays within a step of the exact one. |x| >= 1/2 is forgotten too soon for that.
struct StateFactor {
  float left = 0.f;
  __device__ __forceinline__ float next(float x) {
    if (!(fabsf(x) < 0.5f)) {
      left = 0.f;
      return fast_exp2(x);
    }
    const float m = expm1f(x * 0.6931471805599453f), e = 1.f + m;  // (2^-23 of m off: little where 2^x is next to 1)
    const float more = fmaf(left, e, m - (e - 1.f)), f = e + more;
    left = __fdividef(more - (f - e), f);
    return f;
  }
};
// x as BF16 pairs hi + lo: 16 mantissa bits together, for what feeds a state (products of two such operands leave out low x low, as
// small as what the pairs leave: states come out within 1e-5; a third part would take six products in place of three).
// x - hi by multiply-adds that take BF16 factors as they are, -1 hi + x: two
// instructions for two values where a subtraction takes three (8 x 1024 tokens of 96 heads of the gated delta rule 234 us, 246).
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack2(x);
  float a, b;
  asm("{\n .reg .b16 p, q, m;\n mov.b32 {p, q}, %2;\n mov.b16 m, 0xBF80;\n fma.rn.f32.bf16 %0, p, m, %3;\n fma.rn.f32.bf16 %1, q, m, %4;\n}\n"
      : "=f"(a), "=f"(b) : "r"(hi), "f"(x.x), "f"(x.y));
  lo = pack2(make_float2(a, b));
}

// Eight values of a state row, as they come from memory.
template <typename S>
struct StateVec;
template <>
struct StateVec<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* x) const { unpack_bf16x8(r, x); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* x) { store_bf16x8(p, x); }
};
template <>
struct StateVec<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

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
