// kda_delta.cuh -- launch parameters and the chunks' workspace shared by the kernels of the gated delta rule (kda_delta_*.cu).
//
// Per (sequence, value head), value first, with b the running sum of a chunk's log decays, D_ij = e^{b_i - b_j} (all
// exponents <= 0) and C = 64 tokens a chunk:
//   (1 + A) U = V - e^{b} K S^T,   A_ij = D_ij k_i . k_j beta_j  (j < i),   T = (1 + A)^-1
//   O  = s (e^{b} Q S^T + P (beta U)),   P_ij = D_ij q_i . k_j  (j <= i)
//   S <- e^{b_C} S + sum_j w_j beta_j u_j k_j^T,   w_j = e^{b_C - b_j}
// T and P are a chunk's own and are made for all chunks side by side; the pass over a sequence's chunks has three
// products in its chain (K S^T, T X, the state's update).
#pragma once

#include <cstddef>

#include "kda_decay.cuh"

namespace kda {

struct DeltaProblem : DecayProblem {  // (g may be null: no decay)
  const __nv_bfloat16* beta;          // [Ttot, Hv]
  int64_t slots;                      // places for chunks: Ttot / 64 + N
};

// What is made for each (chunk, head). T and P are BF16 tiles [64][64] in the 128-byte swizzle, in two parts hi + lo
// (16 mantissa bits). P's low part is for the backward alone, where it feeds an adjoint: o, which is rounded to BF16 itself, reads P in
// one part, since 8 KiB more a chunk leave no room for two stages of tiles (2.3e-3 from 64 bits with decays, 1.7e-3 of it o's own
// rounding).
constexpr uint32_t kPkT = 0, kPkTlo = 8192, kPkP = 16384, kPkAux = 24576, kPkPlo = 26624;
constexpr uint32_t kPkInfer = kPkPlo, kPkTrain = kPkPlo + 8192;
struct DeltaAux {
  float eb[64];    // e^{b_i}
  float w[64];     // e^{b_C - b_i}
  float beta[64];  // 0 past the sequence's end
  float whole;     // b_C in base 2
  float bound;     // log2 of a bound on what the chunk leaves of a state's norm: b_C + sum of max(0, log2 |1 - beta_i k_i . k_i|)
  float pad[62];
  float b[64];     // b_i in base 2
};
constexpr uint32_t kPkPass = kPkAux + 1024;  // what the forward's pass reads: up to `whole`
static_assert(sizeof(DeltaAux) <= kPkPlo - kPkAux && offsetof(DeltaAux, b) == 1024, "a chunk's numbers");

// The passes carry states and adjoints on in FP32; these are copies for the gradients within chunks, whose operands they are and no more.
constexpr uint32_t kStateTile = 32768, kUTile = 16384;  // a state in BF16 [2][128 rows][64], u [2][64 tokens][64], swizzled

// Place of a sequence's first chunk: leaves each sequence ceil(len / 64) places.
__host__ __device__ __forceinline__ int64_t delta_slot(int64_t t0, int64_t n) { return t0 / kDecayChunk + n; }

// The chunk of a place, as a kernel for all chunks side by side finds it: nt <= 0 where there is none. A warp looks for it, 32
// sequences at a time (one by one the loads take 2000 cycles).
struct DeltaChunk {
  int64_t t0;
  int nt;
};
__device__ __forceinline__ DeltaChunk delta_chunk(const DeltaProblem& P, int64_t slot) {
  int64_t lo = 0, hi = P.N;  // the last sequence whose first place is not behind this one
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 31) / 32, mid = lo + (threadIdx.x & 31) * step;
    const uint32_t b = __ballot_sync(0xffffffffu, mid < hi && delta_slot(decay_span(P, mid).t0, mid) <= slot);
    lo += b ? (31 - __clz(b)) * step : 0;
    hi = lo + step < hi ? lo + step : hi;
  }
  const DecaySpan sp = decay_span(P, lo);
  const int64_t c = slot - delta_slot(sp.t0, lo), left = sp.len - c * kDecayChunk;
  return DeltaChunk{sp.t0 + c * kDecayChunk, c < 0 || left <= 0 ? 0 : left < kDecayChunk ? (int)left : kDecayChunk};
}

// Workspace: packets; of the training pair, the places' chunks (first token, tokens), the states at the chunks' starts and u from
// the forward, the states' adjoints at the chunks' ends from the backward; where sequences are cut, what the segments make of zero and of the identity (and whether
// that is zero).
struct DeltaWs {
  size_t packet, chunks, states, u, adjoints, segments, through, none, total;
};
DeltaWs delta_workspace(const DeltaProblem& P, bool training);  // (goes by N, Ttot, Hv, slots and seg)

// Tokens of the segments that the forward cuts sequences into, 0 for none. cu: host offsets or null.
int64_t delta_segment_tokens(const int64_t* cu, int64_t N, int64_t T, int64_t Hv);

struct DeltaGrads {
  const __nv_bfloat16* d_o;  // [Ttot, Hv, 128]
  const float* d_hT;         // [N, Hv, 128, 128] or null (zeros)
  __nv_bfloat16* dq;         // [Ttot, Hqk, 128]
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;         // [Ttot, Hv, 128]
  __nv_bfloat16* dg;         // [Ttot, Hv] or null
  __nv_bfloat16* dbeta;      // [Ttot, Hv]
  float* dh0;                // [N, Hv, 128, 128] or null
};

cudaError_t launch_delta_prep(const DeltaProblem& P, bool training, void* ws, cudaStream_t s);
cudaError_t launch_delta_forward(const DeltaProblem& P, const DecayStates& st, __nv_bfloat16* o, bool training, void* ws,
                                 cudaStream_t s);
cudaError_t launch_delta_backward(const DeltaProblem& P, const DeltaGrads& g, void* ws, cudaStream_t s);
// The part of the backward within chunks (after the adjoints' pass).
cudaError_t launch_delta_grads(const DeltaProblem& P, const DeltaGrads& g, void* ws, cudaStream_t s);

}  // namespace kda
