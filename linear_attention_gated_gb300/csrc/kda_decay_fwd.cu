// kda_decay_fwd.cu -- chunked forward of the linear attention with a decay for
// each head, on sm_103a tensor cores.
//
// One CTA owns one (sequence, value head) unit, or one segment of it, and walks its
// tokens in chunks of C = 64. With b_i the sum of the chunk's log decays up to token i
// and S the FP32 state [value, key] at its start:
//   O^T = S Q^T diag(e^{b_i}) + V^T P^T,   P_ij = e^{b_i - b_j} q_i . k_j  (j <= i)
//   S  <- e^{b_C} S + V^T K~,              K~_j = e^{b_C - b_j} k_j
// All exponents are <= 0, so nothing overflows for any decay.
//
// Tensor cores (tcgen05.mma kind::f16, BF16 operands, FP32 accumulators in tensor memory):
//   group 1: scores Q K^T (M = 64: query i in lanes), and S Q^T (S as BF16 A operand in tensor memory)
//   group 2: O^T += V^T P^T, and U = V^T K~ with K~ in two BF16 parts (hi + lo, 16 mantissa bits), so
//            that the carried FP32 state, which lives in registers (64 of a row's 128 values
//            per thread), keeps FP32-level accuracy: S = e^{b_C} S + U.
// K~'s two parts are written over K and Q, which are dead after group 1. Q, K, V tiles come by tiled
// copies (128-byte swizzle), two stages; two CTAs share an SM, so that one's element-wise
// phases run beside the other's copies and products.
//
// Long axis, few units: each sequence is cut into segments. A first pass runs the state part alone
// over every segment but a sequence's last, a small kernel chains the segments' states, and
// the main pass starts every segment from its state.
#include "kda_decay.cuh"
#include "kda_layout.h"
#include "kda_tma.h"
#include "tc.cuh"

namespace kda {
namespace {

constexpr int kC = kDecayChunk;       // tokens of a chunk
constexpr int kThreads = 256;
constexpr uint32_t kTile = kC * kDim * 2;  // bytes of a Q, K or V tile
constexpr uint32_t kPanel = kC * 128;      // bytes of its 64-element half
constexpr uint32_t kTmemCols = 256;        // two CTAs share the 512 columns
constexpr uint32_t kColU = 0;              // U (128 columns); before group 2, the scores (64)
constexpr uint32_t kColS = 128;            // the state as BF16 A operand (64)
constexpr uint32_t kColO = 192;            // O^T (64)

struct Smem {
  unsigned char tile[2][3][kTile];  // stage: Q, K, V
  unsigned char P[kC * kC * 2];
  float b[2][kC];    // cumulative log2 decay of the chunk (by chunk parity)
  float eb[2][kC];   // s e^{b_i}
  float w[2][kC];    // e^{b_C - b_j}
  float lam[2];      // e^{b_C}
  unsigned long long full[2], g1, go, gu;
  uint32_t tmem;
};

struct Maps {
  CUtensorMap q, k, v;
};

struct Segments {
  int64_t len;       // tokens of a segment (a multiple of kC), 0: sequences are not cut
  int most;          // most segments of a sequence
  float* state;      // [slots, Hv, 128, 128]: the segments' own states, then their initial states
  float* decay;      // [slots, Hv]: log2 of a segment's decay
};
// Slot of a sequence's first segment: floor(t0 / len) + n leaves each sequence ceil(len_n / len) slots.
__device__ __forceinline__ int64_t seg_slot(const Segments& g, int64_t t0, int64_t n) { return t0 / g.len + n; }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}

__device__ __forceinline__ uint32_t pack2(float2 x) { return pack2(x.x, x.y); }
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
// w x of two BF16 values as BF16 pairs hi + lo: 16 mantissa bits together
__device__ __forceinline__ void scale_split2(uint32_t x, float2 w, uint32_t& hi, uint32_t& lo) {
  const float2 y = tc::mul2(unpack2(x), w);
  hi = pack2(y);
  lo = pack2(tc::sub2(y, unpack2(hi)));
}

// kState: the first pass over segments (states alone).
template <bool kState>
__global__ void __launch_bounds__(kThreads, 2)
kda_decay_fwd_kernel(const __grid_constant__ Maps maps, const DecayProblem P, const DecayStates st, const Segments sg,
                     __nv_bfloat16* o) {
  extern __shared__ unsigned char raw_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem + ((1024 - (tc::smem_u32(raw_smem) & 1023)) & 1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = (int)(blockIdx.x % P.Hv);
  const int64_t n = blockIdx.x / P.Hv;
  const int64_t seg = blockIdx.y;
  DecaySpan sp = decay_span(P, n);
  int64_t slot = st.slots ? st.slots[n] : n;
  bool last = true;
  int64_t sslot = 0;
  if (sg.len) {
    sslot = seg_slot(sg, sp.t0, n) + seg;
    const int64_t a = seg * sg.len;
    if (a >= sp.len && seg > 0) return;
    last = a + sg.len >= sp.len;
    if (kState && last) return;
    sp.t0 += a;
    sp.len = last ? sp.len - a : sg.len;
  }
  if (slot < 0 || slot >= st.num_slots) {
    // a device index outside the pool (it no longer matches the host mirror the call was checked
    // against, as in a replayed graph): flagged, and the pool is not touched
    if (tid == 0) atomicOr(P.status, 4);
    return;
  }
  const int qh = h / P.r;
  const int qd = warp & 3, half = warp >> 2;
  const int v = 32 * qd + lane;  // state row of this thread: keys 64 half .. 64 half + 63
  const int64_t nchunks = (sp.len + kC - 1) / kC;

  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&sm.tmem), kTmemCols);
  if (tid == 0) {
    tc::mbar_init(tc::smem_u32(&sm.full[0]), 1);
    tc::mbar_init(tc::smem_u32(&sm.full[1]), 1);
    tc::mbar_init(tc::smem_u32(&sm.g1), 1);
    tc::mbar_init(tc::smem_u32(&sm.go), 1);
    tc::mbar_init(tc::smem_u32(&sm.gu), 1);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = sm.tmem;
  const uint32_t tl = tbase + ((uint32_t)(32 * qd) << 16);

  auto load = [&](int64_t c) {  // one thread
    if (c >= nchunks) return;
    const int s = (int)(c & 1), t = (int)(sp.t0 + c * kC);
    const uint32_t bar = tc::smem_u32(&sm.full[s]);
    tc::mbar_arrive_expect_tx(bar, (kState ? 2 : 3) * kTile);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (!kState) tc::tma_load3(tc::smem_u32(sm.tile[s][0]) + p * kPanel, &maps.q, 64 * p, qh, t, bar);
      tc::tma_load3(tc::smem_u32(sm.tile[s][1]) + p * kPanel, &maps.k, 64 * p, qh, t, bar);
      tc::tma_load3(tc::smem_u32(sm.tile[s][2]) + p * kPanel, &maps.v, 64 * p, h, t, bar);
    }
  };
  if (tid == 0) {
    load(0);
    load(1);
  }

  // The decays of chunk c (warp 0, two tokens a lane): sums from both ends, so that the exponents that
  // matter most in each, the small ones, are sums of few terms.
  float total = 0.f;  // of the whole segment
  float g0 = 0.f, g1 = 0.f;
  auto fetch_decays = [&](int64_t c) {
    const int64_t j = c * kC + 2 * lane;
    g0 = j < sp.len ? decay_g(P, sp.t0 + j, h) : 0.f;
    g1 = j + 1 < sp.len ? decay_g(P, sp.t0 + j + 1, h) : 0.f;
  };
  auto decays = [&](int64_t c) {
    g0 = decay_log2(g0);
    g1 = decay_log2(g1);
    float pre = g0 + g1, suf = pre;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float a = __shfl_up_sync(0xffffffffu, pre, d), b = __shfl_down_sync(0xffffffffu, suf, d);
      if (lane >= d) pre += a;
      if (lane + d < 32) suf += b;
    }
    const float before = __shfl_up_sync(0xffffffffu, pre, 1), after = __shfl_down_sync(0xffffffffu, suf, 1);
    const float p0 = (lane ? before : 0.f) + g0, s1 = lane < 31 ? after : 0.f;
    const int s = (int)(c & 1);
    sm.b[s][2 * lane] = p0;
    sm.b[s][2 * lane + 1] = pre;
    sm.eb[s][2 * lane] = P.scale * exp2f(p0);
    sm.eb[s][2 * lane + 1] = P.scale * exp2f(pre);
    sm.w[s][2 * lane] = exp2f(s1 + g1);
    sm.w[s][2 * lane + 1] = exp2f(s1);
    if (lane == 31) sm.lam[s] = exp2f(pre);
    total += pre;  // lane 31's is the chunk's
  };

  // ---- the state: 64 values of row v
  float2 S[32];
  {
    const int64_t at = ((slot * P.Hv + h) * kDim + v) * kDim + 64 * half;
    if (kState || (!sg.len && !st.in)) {
#pragma unroll
      for (int j = 0; j < 32; ++j) S[j] = make_float2(0.f, 0.f);
    } else if (!sg.len && st.bf16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 x = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(st.in) + at)[j];
        S[4 * j] = unpack2(x.x); S[4 * j + 1] = unpack2(x.y); S[4 * j + 2] = unpack2(x.z); S[4 * j + 3] = unpack2(x.w);
      }
    } else {
      const float* src = !sg.len ? reinterpret_cast<const float*>(st.in) + at
                                 : sg.state + ((sslot * P.Hv + h) * kDim + v) * kDim + 64 * half;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float4 x = reinterpret_cast<const float4*>(src)[j];
        S[2 * j] = make_float2(x.x, x.y);
        S[2 * j + 1] = make_float2(x.z, x.w);
      }
    }
  }
  // the state as the next chunk's A operand
  auto put_state = [&] {
    if (kState) return;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      uint32_t x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = pack2(S[8 * m + e]);
      tc::tmem_st8(tl + kColS + 32 * half + 8 * m, x);
    }
  };
  put_state();
  tc::tmem_wait_st();
  if (warp == 0) {
    fetch_decays(0);
    decays(0);
  }

  bool ok = true;
  uint32_t ph = 0;  // parity of the group barriers
  int64_t c = 0;
  for (; c < nchunks; ++c, ph ^= 1) {
    const int s = (int)(c & 1);
    const int nt = (int)(sp.len - c * kC < kC ? sp.len - c * kC : kC);
    unsigned char* Qs = sm.tile[s][0];
    unsigned char* Ks = sm.tile[s][1];
    unsigned char* Vs = sm.tile[s][2];
    ok = ok && tc::mbar_wait_warp(tc::smem_u32(&sm.full[s]), (uint32_t)(c >> 1) & 1);
    if (nt < kC) {  // rows past the end hold other tokens: value rows are cleared (keys below)
      for (int i = tid; i < (kC - nt) * 16; i += kThreads)
        *reinterpret_cast<uint4*>(Vs + ((i >> 3) & 1) * kPanel + (nt + (i >> 4)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
      tc::fence_async_smem();
    }
    tc::fence_before();
    if (__syncthreads_or(!ok)) break;
    if (warp == 0) fetch_decays(c + 1);
    // ---- group 1
    if (!kState && warp == 0) {
      if (tc::elect_one()) {
        tc::fence_after();
        const uint64_t dq = tc::kmajor(tc::smem_u32(Qs)), dk = tc::kmajor(tc::smem_u32(Ks));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = (k >> 2) * (kPanel >> 4) + (k & 3) * 2;
          tc::mma_bf16_ss(tbase + kColU, dq + off, dk + off, tc::idesc_bf16(64, 64, false, false), k > 0);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = (k >> 2) * (kPanel >> 4) + (k & 3) * 2;
          tc::mma_bf16_ts(tbase + kColO, tbase + kColS + 8 * k, dq + off, tc::idesc_bf16(128, 64, false, false), k > 0);
        }
        tc::mma_commit(tc::smem_u32(&sm.g1));
      }
      __syncwarp();
    }
    // ---- K~ = e^{b_C - b_j} k_j in two parts: 16-byte chunks i, four a thread
    uint4 hi[4], lo[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int i = tid + kThreads * m, row = (i >> 3) & (kC - 1);
      const uint4 x = *reinterpret_cast<const uint4*>(Ks + 16 * i);
      const float w1 = sm.w[s][row];
      const float2 w = make_float2(w1, w1);
      scale_split2(x.x, w, hi[m].x, lo[m].x);
      scale_split2(x.y, w, hi[m].y, lo[m].y);
      scale_split2(x.z, w, hi[m].z, lo[m].z);
      scale_split2(x.w, w, hi[m].w, lo[m].w);
      if (row >= nt) hi[m] = lo[m] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (!kState) {
      ok = ok && tc::mbar_wait_warp(tc::smem_u32(&sm.g1), ph);
      tc::fence_after();
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      *reinterpret_cast<uint4*>(Ks + 16 * (tid + kThreads * m)) = hi[m];
      *reinterpret_cast<uint4*>(Qs + 16 * (tid + kThreads * m)) = lo[m];
    }
    if (!kState) {
      // ---- P: rows i = 16 qd + lane / 4 (+ 8), columns 32 half + 8 m + 2 (lane % 4) (+ 1)
      float x[32];
      tc::tmem_ld16x256(tl + kColU + 32 * half, x);
      tc::tmem_wait_ld(x);
      {
        const int i0 = 16 * qd + (lane >> 2), j0 = 32 * half + 2 * (lane & 3);
        const float b0 = sm.b[s][i0], b1 = sm.b[s][i0 + 8];
        const float2 scale = make_float2(P.scale, P.scale);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int j = j0 + 8 * m;
          const float2 bj = *reinterpret_cast<const float2*>(&sm.b[s][j]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int i = i0 + 8 * u;
            const float bi = u ? b1 : b0;
            const float2 e = make_float2(fast_exp2(bi - bj.x), fast_exp2(bi - bj.y));
            float2 y = tc::mul2(tc::mul2(make_float2(x[4 * m + 2 * u], x[4 * m + 2 * u + 1]), scale), e);
            y.x = j <= i && i < nt ? y.x : 0.f;  // (selected, not multiplied: rows past the end may hold anything)
            y.y = j < i && i < nt ? y.y : 0.f;
            *reinterpret_cast<uint32_t*>(sm.P + i * 128 + (((4 * half + m) ^ (i & 7)) << 4) + 4 * (lane & 3)) = pack2(y);
          }
        }
      }
      // ---- S Q^T scaled by s e^{b_i}: columns i
      tc::tmem_ld16_nowait(tl + kColO + 32 * half, x);
      tc::tmem_ld16_nowait(tl + kColO + 32 * half + 16, x + 16);
      tc::tmem_wait_ld2(x, x + 16);
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 e = *reinterpret_cast<const float4*>(&sm.eb[s][32 * half + j]);
        const float2 y = tc::mul2(make_float2(x[j], x[j + 1]), make_float2(e.x, e.y));
        const float2 z = tc::mul2(make_float2(x[j + 2], x[j + 3]), make_float2(e.z, e.w));
        x[j] = y.x; x[j + 1] = y.y; x[j + 2] = z.x; x[j + 3] = z.y;
      }
      tc::tmem_st16(tl + kColO + 32 * half, x);
      tc::tmem_st16(tl + kColO + 32 * half + 16, x + 16);
      tc::tmem_wait_st();
    }
    tc::fence_async_smem();
    tc::fence_before();
    if (__syncthreads_or(!ok)) break;
    // ---- group 2
    if (warp == 0) {
      if (tc::elect_one()) {
        tc::fence_after();
        const uint64_t dv = tc::mnmajor(tc::smem_u32(Vs), kPanel);
        if (!kState) {
          const uint64_t dp = tc::kmajor(tc::smem_u32(sm.P));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_bf16_ss(tbase + kColO, dv + 128 * k, dp + 2 * k, tc::idesc_bf16(128, 64, true, false), 1);
          tc::mma_commit(tc::smem_u32(&sm.go));
        }
        const uint64_t dh = tc::mnmajor(tc::smem_u32(Ks), kPanel), dl = tc::mnmajor(tc::smem_u32(Qs), kPanel);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc::mma_bf16_ss(tbase + kColU, dv + 128 * k, dh + 128 * k, tc::idesc_bf16(128, 128, true, true), k > 0);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc::mma_bf16_ss(tbase + kColU, dv + 128 * k, dl + 128 * k, tc::idesc_bf16(128, 128, true, true), 1);
        tc::mma_commit(tc::smem_u32(&sm.gu));
      }
      __syncwarp();
      decays(c + 1);
    }
    const float2 lam2 = make_float2(sm.lam[s], sm.lam[s]);
    if (!kState) {
      // ---- o: thread v, tokens 32 half .. + 31; neighbours exchange, so that each stores two values of a token
      ok = ok && tc::mbar_wait_warp(tc::smem_u32(&sm.go), ph);
      tc::fence_after();
      float x[32];
      tc::tmem_ld16_nowait(tl + kColO + 32 * half, x);
      tc::tmem_ld16_nowait(tl + kColO + 32 * half + 16, x + 16);
      tc::tmem_wait_ld2(x, x + 16);
      const int odd = lane & 1;
      const uint32_t pick = odd ? 0x3276u : 0x5410u;  // (own low, neighbour's low) or (neighbour's high, own high)
      __nv_bfloat16* dst = o + ((sp.t0 + c * kC + 32 * half + odd) * P.Hv + h) * kDim + (v & ~1);
      const int64_t step = 2 * (int64_t)P.Hv * kDim;
      const int left = nt - 32 * half - odd;
#pragma unroll
      for (int j = 0; j < 32; j += 2, dst += step) {
        const uint32_t mine = pack2(x[j], x[j + 1]);
        const uint32_t got = __shfl_xor_sync(0xffffffffu, mine, 1);
        if (j < left) *reinterpret_cast<uint32_t*>(dst) = __byte_perm(mine, got, pick);
      }
    }
    // ---- the state
    ok = ok && tc::mbar_wait_warp(tc::smem_u32(&sm.gu), ph);
    tc::fence_after();
    if (tid == 0 && ok) load(c + 2);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      float x[16];
      tc::tmem_ld16(tl + kColU + 64 * half + 16 * m, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) S[8 * m + j] = tc::fma2(lam2, S[8 * m + j], make_float2(x[2 * j], x[2 * j + 1]));
    }
    if (c + 1 < nchunks) {
      put_state();
      tc::tmem_wait_st();
    }
  }
  const bool aborted = c < nchunks;
  if (aborted && tid == 0) {
    // a wait gave up: flag it, and let this CTA's copies land before its memory is given back
    atomicOr(P.status, 1);
    for (int64_t k = c; k < c + 2 && k < nchunks; ++k) tc::mbar_wait(tc::smem_u32(&sm.full[k & 1]), (uint32_t)(k >> 1) & 1);
  }
  __syncthreads();
  if (!aborted) {
    if (kState) {
      float* dst = sg.state + ((sslot * P.Hv + h) * kDim + v) * kDim + 64 * half;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        reinterpret_cast<float4*>(dst)[j] = make_float4(S[2 * j].x, S[2 * j].y, S[2 * j + 1].x, S[2 * j + 1].y);
      if (tid == 31) sg.decay[sslot * P.Hv + h] = total;
    } else if (last && st.out) {
      const int64_t at = ((slot * P.Hv + h) * kDim + v) * kDim + 64 * half;
      if (st.bf16) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(st.out) + at)[j] =
              make_uint4(pack2(S[4 * j]), pack2(S[4 * j + 1]), pack2(S[4 * j + 2]), pack2(S[4 * j + 3]));
      } else {
        float* dst = reinterpret_cast<float*>(st.out) + at;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          reinterpret_cast<float4*>(dst)[j] = make_float4(S[2 * j].x, S[2 * j].y, S[2 * j + 1].x, S[2 * j + 1].y);
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after();
    tc::tmem_dealloc(tbase, kTmemCols);
  }
}

// Chains the segments of one (sequence, head): in, each segment's own state (from zero) but the last's;
// out, the state each segment starts from. A CTA takes 1024 of the state's values.
__global__ void __launch_bounds__(256) kda_decay_chain_kernel(const DecayProblem P, const DecayStates st, const Segments sg) {
  const int64_t n = blockIdx.x / P.Hv;
  const int h = (int)(blockIdx.x % P.Hv);
  const DecaySpan sp = decay_span(P, n);
  const int64_t slot = st.slots ? st.slots[n] : n;
  if (slot < 0 || slot >= st.num_slots) return;  // the main pass flags it
  const int at = 1024 * blockIdx.y + 4 * threadIdx.x;
  const int64_t from = (slot * P.Hv + h) * kDim * kDim + at;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (st.in && st.bf16) {
    const uint2 r = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(st.in) + from);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
    x = make_float4(a.x, a.y, b.x, b.y);
  } else if (st.in) {
    x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(st.in) + from);
  }
  const int64_t base = seg_slot(sg, sp.t0, n);
  const int64_t m = sp.len > sg.len ? (sp.len + sg.len - 1) / sg.len : 1;
  constexpr int kAhead = 8;  // loads in flight: none waits for the chain
  for (int64_t i = 0; i < m; i += kAhead) {
    float4 u[kAhead];
    float d[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i + j + 1 < m) {
        u[j] = *reinterpret_cast<const float4*>(sg.state + ((base + i + j) * P.Hv + h) * kDim * kDim + at);
        d[j] = sg.decay[(base + i + j) * P.Hv + h];
      }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j >= m) break;
      *reinterpret_cast<float4*>(sg.state + ((base + i + j) * P.Hv + h) * kDim * kDim + at) = x;
      if (i + j + 1 < m) {
        const float e = exp2f(d[j]);
        x.x = fmaf(e, x.x, u[j].x); x.y = fmaf(e, x.y, u[j].y);
        x.z = fmaf(e, x.z, u[j].z); x.w = fmaf(e, x.w, u[j].w);
      }
    }
  }
}

constexpr int64_t kResident = 2 * 152;  // CTAs that run at once

struct FwdWs {
  size_t state, decay, total;
};
FwdWs carve(int64_t N, int64_t Ttot, int64_t Hv, int64_t seg) {
  FwdWs w{0, 0, 0};
  if (!seg) return w;
  const size_t slots = (size_t)(Ttot / seg + N);
  w.decay = ctx_align_up(sizeof(float) * slots * Hv * kDim * kDim);
  w.total = ctx_align_up(w.decay + sizeof(float) * slots * Hv);
  return w;
}

template <bool kState>
cudaError_t run(const Maps& maps, const DecayProblem& P, const DecayStates& st, const Segments& sg, __nv_bfloat16* o,
                cudaStream_t s) {
  const int smem = (int)sizeof(Smem) + 1024;
  const cudaError_t e =
      cudaFuncSetAttribute(kda_decay_fwd_kernel<kState>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kda_decay_fwd_kernel<kState><<<dim3((unsigned)(P.N * P.Hv), (unsigned)sg.most), kThreads, smem, s>>>(maps, P, st, sg, o);
  return cudaGetLastError();
}

}  // namespace

int64_t decay_segment_tokens(const int64_t* cu, int64_t N, int64_t T, int64_t Hv) {
  auto len = [&](int64_t n) { return cu ? cu[n + 1] - cu[n] : T; };
  int64_t longest = 0, chunks = 0;
  for (int64_t n = 0; n < (cu ? N : 1); ++n) {
    const int64_t c = (len(n) + kC - 1) / kC;
    chunks += c;
    if (c > longest) longest = c;
  }
  if (!cu) chunks *= N;
  // an even share of the chunks for each CTA that can run at once, 8 chunks at least
  int64_t seg = (chunks * Hv + kResident - 1) / kResident;
  if (seg < 8) seg = 8;
  // cutting adds a pass over keys and values: only where the longest sequence takes over twice the share
  if (longest <= 2 * seg) return 0;
  if (N * Hv < kResident) {  // one wave
    for (;; ++seg) {
      int64_t ctas = 0;
      for (int64_t n = 0; n < (cu ? N : 1); ++n) {
        const int64_t c = (len(n) + kC - 1) / kC;
        ctas += c > seg ? (c + seg - 1) / seg : 1;
      }
      if (!cu) ctas *= N;
      if (ctas * Hv <= kResident) break;
    }
    if (longest <= 2 * seg) return 0;
  }
  return seg * kC;
}

size_t decay_forward_workspace(int64_t N, int64_t Ttot, int64_t Hv, int64_t seg) { return carve(N, Ttot, Hv, seg).total; }

cudaError_t launch_decay_forward(const DecayProblem& P, const DecayStates& st, __nv_bfloat16* o, void* ws,
                                 bool training, cudaStream_t s) {
  Maps maps{};
  cudaError_t e;
  if (P.Ttot) {
    if ((e = token_map(&maps.q, P.q, P.Hqk, P.Ttot, P.qh, P.qt, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.k, P.k, P.Hqk, P.Ttot, P.kh, P.kt, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.v, P.v, P.Hv, P.Ttot, P.vh, P.vt, kC)) != cudaSuccess) return e;
  }
  Segments sg{0, 1, nullptr, nullptr};
  if (P.seg) {
    const FwdWs w = carve(P.N, P.Ttot, P.Hv, P.seg);
    sg.len = P.seg;
    sg.most = (int)((P.longest + P.seg - 1) / P.seg);
    sg.state = reinterpret_cast<float*>(ws);
    sg.decay = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + w.decay);
    if ((e = run<true>(maps, P, st, sg, nullptr, s)) != cudaSuccess) return e;
    kda_decay_chain_kernel<<<dim3((unsigned)(P.N * P.Hv), 16), 256, 0, s>>>(P, st, sg);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = run<false>(maps, P, st, sg, o, s)) != cudaSuccess) return e;
  if (training)
    e = cudaMemcpyAsync(reinterpret_cast<char*>(ws) + decay_forward_workspace(P.N, P.Ttot, P.Hv, P.seg), st.out,
                        sizeof(float) * P.N * P.Hv * kDim * kDim, cudaMemcpyDeviceToDevice, s);
  return e;
}

}  // namespace kda
