// kda_delta_bwd.cu -- the states' adjoints of the gated delta rule, backwards over each sequence's chunks, on sm_103a tensor
// cores. From what the forward left of each chunk (T and P in two parts, its decays' numbers; kda_delta.cuh):
//   d_j = s sum_{i >= j} P_ij dO_i + w_j G k_j,   rho = T^T (beta d)  (= dv)
//   G  <- e^{b_C} G + s sum_i e^{b_i} dO_i q_i^T - sum_i e^{b_i} rho_i k_i^T
// with G the adjoint of the state at the chunk's end, value first; G in BF16 is left for kda_delta_grad.cu.
//
// The chain of a chunk, G K^T -> beta d -> T^T beta d -> e^b rho -> the update, goes in halves of its tokens and of G's
// columns as the forward's does (kda_delta_fwd.cu); T^T being upper triangular, the second half of the tokens leads. Bound: that
// chain; 4 x 2048 tokens of 32 heads, 128 units of 32 chunks on 152 SMs, 94 us.
#include <algorithm>

#include "kda_delta.cuh"
#include "kda_layout.h"
#include "kda_tma.h"
#include "tc.cuh"

namespace kda {
namespace {

constexpr int kC = kDecayChunk;
constexpr int kStages = 2;
constexpr int kWarpLoad = 0, kWarpMma = 1, kWarpOut = 4, kWarpChain = 12, kGroup = 8;
constexpr int kThreads = 32 * 20;
// Registers a thread of the control, out and chain warps (setmaxnreg): 128 x 48 + 256 x 72 + 256 x 144 = 61,440, all of the
// 640 x 96 = 61,440 the block is launched with (a split above that would wait for ever).
constexpr uint32_t kTile = kC * kDim * 2;  // bytes of a token tile
constexpr uint32_t kPanel = kC * 128;      // bytes of its 64-element half
// Tensor memory, columns. G as A operand: its columns 64 h + 16 m .. are in 64 h + 8 m .. (high parts) and 32 further
// (low parts).
constexpr uint32_t kColS = 0;    // 128: G
constexpr uint32_t kColX = 128;  // 64: G K^T, then T^T beta d
constexpr uint32_t kColA = 192;  // 32 + 32: beta d, then -e^b rho, as A operands
constexpr uint32_t kColD = 256;  // 64: dO^T P
constexpr uint32_t kColE = 320;  // 32 + 32: s e^b dO as A operand
constexpr uint32_t kColG = 384;  // 128: the update's sum

struct Smem {
  unsigned char tok[kStages][3][kTile];     // K, Q, dO
  unsigned char packet[kStages][kPkTrain];  // (kPkTrain is a multiple of 1024)
  unsigned char out[kTile];                 // dv on its way out,
  unsigned char G[kStateTile];              // and G in BF16
  unsigned long long full[kStages], empty[kStages], raw, eready, sready[2], gx, scopied, xready[2], gu[2], wready[2], gs[2], ofree;
  uint32_t tmem;
};
constexpr int kSmemBytes = (int)sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

constexpr int kOrder = 512;  // sequences whose order is passed (more run in index order)

struct PassArgs {
  DeltaProblem P;
  const float* d_hT;
  float* dh0;
  const unsigned char* packets;
  unsigned char* adjoints;
  __nv_bfloat16* dv;
  int ordered;
  uint16_t order[kOrder];  // longest sequence first
};
struct Maps {
  CUtensorMap q, k, d_o, dv;
};

__device__ __forceinline__ float* regs(uint32_t* x) { return reinterpret_cast<float*>(x); }

__global__ void __launch_bounds__(kThreads, 1) kda_delta_bwd_kernel(const __grid_constant__ Maps maps, const __grid_constant__ PassArgs a) {
  extern __shared__ unsigned char raw_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem + ((1024 - (tc::smem_u32(raw_smem) & 1023)) & 1023));
  const DeltaProblem& P = a.P;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [](unsigned long long& b) { return tc::smem_u32(&b); };

  int64_t n = blockIdx.x / P.Hv;
  const int h = (int)(blockIdx.x - n * P.Hv);
  if (a.ordered) n = a.order[n];
  const DecaySpan sp = decay_span(P, n);
  const int nchunks = (int)((sp.len + kC - 1) / kC);
  const int64_t place = delta_slot(sp.t0, n);
  auto tokens = [&](int ci) { return (int)(sp.len - (int64_t)ci * kC < kC ? sp.len - (int64_t)ci * kC : kC); };

  if (warp == kWarpMma) tc::tmem_alloc(tc::smem_u32(&sm.tmem), 512);
  if (tid == 0) {
    auto init = [&](unsigned long long& b, uint32_t count) { tc::mbar_init(bar(b), count); };
    for (int i = 0; i < 2; ++i) {
      init(sm.full[i], 1); init(sm.empty[i], 1 + 2 * kGroup);
      init(sm.sready[i], 4); init(sm.xready[i], 4); init(sm.wready[i], 4);
      init(sm.gu[i], 1); init(sm.gs[i], 1);
    }
    init(sm.raw, 1);
    init(sm.gx, 1);
    init(sm.eready, kGroup);
    init(sm.scopied, kGroup);
    init(sm.ofree, kGroup);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = sm.tmem;
  bool ok = true;  // false: a wait gave up; the warp leaves its loop
  auto wait = [&](unsigned long long& b, uint32_t parity) {
    if (ok) ok = tc::mbar_wait_lanes(bar(b), parity & 1);
    tc::fence_after();
    return ok;
  };
  auto arrive = [&](unsigned long long& b) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar(b));
  };

  if (warp < kWarpOut) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == kWarpLoad) {
      int c = 0;
      bool tail = false;
      for (; c < nchunks; ++c) {
        const int s = c % kStages, ci = nchunks - 1 - c;
        if (c >= kStages && !wait(sm.empty[s], c / kStages - 1)) break;
        if (lane == 0) {
          const int t = (int)(sp.t0 + (int64_t)ci * kC);
          const uint32_t f = tokens(ci) < kC ? bar(sm.raw) : bar(sm.full[s]);
          tc::mbar_arrive_expect_tx(f, 3 * kTile + kPkTrain);
          tc::bulk_g2s(tc::smem_u32(sm.packet[s]), a.packets + ((place + ci) * P.Hv + h) * (int64_t)kPkTrain, kPkTrain, f);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            tc::tma_load3(tc::smem_u32(sm.tok[s][0]) + p * kPanel, &maps.k, 64 * p, h / P.r, t, f);
            tc::tma_load3(tc::smem_u32(sm.tok[s][1]) + p * kPanel, &maps.q, 64 * p, h / P.r, t, f);
            tc::tma_load3(tc::smem_u32(sm.tok[s][2]) + p * kPanel, &maps.d_o, 64 * p, h, t, f);
          }
        }
        __syncwarp();
        const int nt = tokens(ci);
        if (nt < kC) {  // (the sequence's last chunk, the first turn) rows past the end hold other tokens
          tail = true;
          ok = tc::mbar_wait_lanes(bar(sm.raw), 0);
          for (int i = lane; ok && i < (kC - nt) * 48; i += 32) {
            const int row = nt + i / 48, x = i % 48;
            *reinterpret_cast<uint4*>(sm.tok[s][x >> 4] + ((x >> 3) & 1) * kPanel + row * 128 + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          tc::fence_async_smem();
          arrive(sm.full[s]);
        }
      }
      if (!ok) {  // flag it, and let this CTA's copies land before its memory is given back
        if (lane == 0) atomicOr(P.status, 1);
        if (tail) tc::mbar_wait_lanes(bar(sm.raw), 0, 1u << 16);
        for (int k = c > kStages ? c - kStages : 0; k < c; ++k) tc::mbar_wait_lanes(bar(sm.full[k % kStages]), (k / kStages) & 1, 1u << 16);
      }
    } else if (warp == kWarpMma) {
      constexpr uint32_t kN64 = tc::idesc_bf16(128, 64, false, false), kN32t = tc::idesc_bf16(128, 32, false, true);
      for (int c = 0; c < nchunks; ++c) {
        const int s = c % kStages;
        const uint32_t k = tc::smem_u32(sm.tok[s][0]), q = tc::smem_u32(sm.tok[s][1]), d = tc::smem_u32(sm.tok[s][2]);
        const uint32_t pk = tc::smem_u32(sm.packet[s]);
        const uint64_t kk = tc::kmajor(k), kn = tc::mnmajor(k, kPanel), qn = tc::mnmajor(q, kPanel);
        if (!wait(sm.full[s], c / kStages)) break;
        // dO^T P, once dO is prepared
        if (!wait(sm.eready, c)) break;
        if (tc::elect_one()) {
          const uint64_t dn = tc::mnmajor(d, kPanel), pn = tc::mnmajor(pk + kPkP, 8192), pl = tc::mnmajor(pk + kPkPlo, 8192);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tc::mma_bf16_ss(tbase + kColD, dn + 128 * i, pn + 128 * i, tc::idesc_bf16(128, 64, true, true), i > 0);
            tc::mma_bf16_ss(tbase + kColD, dn + 128 * i, pl + 128 * i, tc::idesc_bf16(128, 64, true, true), 1);
          }
        }
        __syncwarp();
        // G K^T, the columns of G as they come
        if (c && !wait(sm.ofree, c - 1)) break;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!wait(sm.sready[x], c)) break;
          if (tc::elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int part = 0; part < 2; ++part)
                tc::mma_bf16_ts(tbase + kColX, tbase + kColS + 64 * x + 8 * i + 32 * part, kk + x * (kPanel >> 4) + 2 * i, kN64, x + i + part > 0);
            if (x) tc::mma_commit(bar(sm.gx));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (tc::elect_one()) {
          // (s e^b dO)^T Q
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int part = 0; part < 2; ++part)
              tc::mma_bf16_ts(tbase + kColG, tbase + kColE + 8 * i + 32 * part, qn + 128 * i, tc::idesc_bf16(128, 128, false, true), i + part > 0);
        }
        __syncwarp();
        // with T^T: the last 32 tokens, the others
#pragma unroll
        for (int th = 1; th >= 0; --th) {
          if (!wait(sm.xready[th], c)) break;
          if (tc::elect_one()) {
            // rows of T are its inner index here; columns 32 th .. of it 64 bytes along
            const uint64_t hi = tc::mnmajor(pk + kPkT, 8192) + 4 * th, lo = tc::mnmajor(pk + kPkTlo, 8192) + 4 * th;
#pragma unroll
            for (int i = 2 * th; i < 4; ++i) {
              const uint32_t x = tbase + kColA + 8 * i;
              tc::mma_bf16_ts(tbase + kColX + 32 * th, x, hi + 128 * i, kN32t, i > 2 * th);
              tc::mma_bf16_ts(tbase + kColX + 32 * th, x, lo + 128 * i, kN32t, 1);
              tc::mma_bf16_ts(tbase + kColX + 32 * th, x + 32, hi + 128 * i, kN32t, 1);
            }
            tc::mma_commit(bar(sm.gu[th]));
          }
          __syncwarp();
        }
        if (!ok) break;
        // the update, the last of it for one half of the columns after the other
        if (!wait(sm.wready[1], c)) break;
        if (tc::elect_one())
#pragma unroll
          for (int i = 2; i < 4; ++i)
#pragma unroll
            for (int part = 0; part < 2; ++part)
              tc::mma_bf16_ts(tbase + kColG, tbase + kColA + 8 * i + 32 * part, kn + 128 * i, tc::idesc_bf16(128, 128, false, true), 1);
        __syncwarp();
        if (!wait(sm.wready[0], c)) break;
        if (tc::elect_one()) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int part = 0; part < 2; ++part)
                tc::mma_bf16_ts(tbase + kColG + 64 * x, tbase + kColA + 8 * i + 32 * part, kn + x * (kPanel >> 4) + 128 * i,
                                tc::idesc_bf16(128, 64, false, true), 1);
            tc::mma_commit(bar(sm.gs[x]));
          }
          tc::mma_commit(bar(sm.empty[s]));
        }
        __syncwarp();
      }
    }
  } else if (warp < kWarpChain) {
    // ================= dO as an operand, and dv on its way out
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int wq = (warp - kWarpOut) & 3, half = (warp - kWarpOut) >> 2;
    const uint32_t tl = tbase + ((uint32_t)(32 * wq) << 16);
    // The warps that fill a tile together leave together: a barrier among them is not bounded.
    auto agree = [&] {
      uint32_t all;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(all) : "r"((uint32_t)ok), "n"(32 * kGroup) : "memory");
      return ok = all != 0;
    };
    for (int c = 0; c < nchunks; ++c) {
      const int s = c % kStages, ci = nchunks - 1 - c, nt = tokens(ci);
      const int64_t t0 = sp.t0 + (int64_t)ci * kC;
      const DeltaAux& aux = *reinterpret_cast<const DeltaAux*>(sm.packet[s] + kPkAux);
      wait(sm.full[s], c / kStages);
      uint32_t hi[2][8], lo[2][8];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t r[8];  // [8 tokens][8 values] blocks, transposed: r[2 i + j] holds tokens 8 i + 2 (lane % 4) (+ 1) of value 8 j + lane / 4
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const int t = 32 * half + 8 * (i + (lane >> 4)) + (lane & 7), d = 32 * wq + 16 * q + 8 * ((lane >> 3) & 1);
          tc::ldmatrix4_trans(tc::smem_u32(sm.tok[s][2]) + (d >> 6) * kPanel + t * 128 + ((((d & 63) >> 3) ^ (t & 7)) << 4), r + 2 * i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 e = *reinterpret_cast<const float2*>(&aux.eb[32 * half + 8 * i + 2 * (lane & 3)]);
          const float2 f = make_float2(P.scale * e.x, P.scale * e.y);
          split2(tc::mul2(f, unpack2(r[2 * i])), hi[q][2 * i], lo[q][2 * i]);
          split2(tc::mul2(f, unpack2(r[2 * i + 1])), hi[q][2 * i + 1], lo[q][2 * i + 1]);
        }
      }
      // (gu of the last chunk was waited for below: the products with its operand are done)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        tc::tmem_st16x128(tl + (16u * q << 16) + kColE + 16 * half, regs(hi[q]));
        tc::tmem_st16x128(tl + (16u * q << 16) + kColE + 32 + 16 * half, regs(lo[q]));
      }
      tc::tmem_wait_st();
      tc::fence_before();
      arrive(sm.eready);
      // G's high parts
      wait(sm.sready[0], c);
      wait(sm.sready[1], c);
      if (warp == kWarpOut && lane == 0) tc::bulk_wait_read_but<1>();  // the last one has left
      if (!agree()) break;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float r[16];
        tc::tmem_ld16(tl + kColS + 64 * half + 16 * m, r);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<float4*>(sm.G + half * 16384 + (32 * wq + lane) * 128 + (((4 * m + q) ^ (lane & 7)) << 4)) =
              make_float4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
      }
      tc::fence_before();
      arrive(sm.scopied);
      tc::fence_async_smem();
      asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * kGroup) : "memory");
      if (warp == kWarpOut && lane == 0) {
        tc::bulk_s2g(a.adjoints + ((place + ci) * P.Hv + h) * (int64_t)kStateTile, tc::smem_u32(sm.G), kStateTile);
        tc::bulk_commit();
      }
      wait(sm.gu[1], c);
      wait(sm.gu[0], c);
      if (warp == kWarpOut && lane == 0) tc::bulk_wait_read_but<1>();  // the last dv has left
      if (!agree()) break;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float r[16];
        tc::tmem_ld16x256(tl + (16u * q << 16) + kColX + 32 * half, r);
        tc::tmem_wait_ld(r);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const int t = 32 * half + 8 * (i + (lane >> 4)) + (lane & 7), d = 32 * wq + 16 * q + 8 * ((lane >> 3) & 1);
          tc::stmatrix4_trans(tc::smem_u32(sm.out) + (d >> 6) * kPanel + t * 128 + ((((d & 63) >> 3) ^ (t & 7)) << 4),
                              pack2(r[4 * i], r[4 * i + 1]), pack2(r[4 * i + 2], r[4 * i + 3]), pack2(r[4 * i + 4], r[4 * i + 5]),
                              pack2(r[4 * i + 6], r[4 * i + 7]));
        }
      }
      tc::fence_before();
      arrive(sm.ofree);
      arrive(sm.empty[s]);
      tc::fence_async_smem();
      asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * kGroup) : "memory");
      if (nt == kC) {
        if (warp == kWarpOut && lane == 0) {
          tc::tma_store3(&maps.dv, tc::smem_u32(sm.out), 0, h, (int)t0);
          tc::tma_store3(&maps.dv, tc::smem_u32(sm.out) + kPanel, 64, h, (int)t0);
          tc::bulk_commit();
        }
      } else {  // (a whole tile would run into the next sequence)
        for (int i = tid - 32 * kWarpOut; i < nt * 16; i += 32 * kGroup) {
          const int t = i >> 4, k = i & 15;
          *reinterpret_cast<uint4*>(a.dv + ((t0 + t) * P.Hv + h) * kDim + 8 * k) =
              *reinterpret_cast<const uint4*>(sm.out + (k >> 3) * kPanel + t * 128 + (((k & 7) ^ (t & 7)) << 4));
        }
        // (the next chunk's tile is written after the barrier above it; an empty group, so that they are two a chunk)
        if (warp == kWarpOut && lane == 0) tc::bulk_commit();
      }
    }
    if (warp == kWarpOut && lane == 0) tc::bulk_wait();
    if (!ok && lane == 0) atomicOr(P.status, 1);
  } else {
    // ================= the chain of G
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int wq = (warp - kWarpChain) & 3, half = (warp - kWarpChain) >> 2;
    const int v = 32 * wq + lane;  // row of this thread, its columns 64 half .. + 63
    const uint32_t tl = tbase + ((uint32_t)(32 * wq) << 16);
    const int64_t at = (n * P.Hv + h) * kDim * kDim + v * kDim + 64 * half;
    float2 S[32];
    if (!a.d_hT) {
#pragma unroll
      for (int j = 0; j < 32; ++j) S[j] = make_float2(0.f, 0.f);
    } else {
      const float4* src = reinterpret_cast<const float4*>(a.d_hT + at);
#pragma unroll
      for (int j = 0; j < 16; ++j) reinterpret_cast<float4*>(S)[j] = src[j];
    }
    auto put_state = [&] {  // as the next turn's operand
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split2(S[8 * m + e], hi[e], lo[e]);
        tc::tmem_st8(tl + kColS + 64 * half + 8 * m, hi);
        tc::tmem_st8(tl + kColS + 64 * half + 32 + 8 * m, lo);
      }
      tc::tmem_wait_st();
      tc::fence_before();
      arrive(sm.sready[half]);
    };
    StateFactor factor;
    if (nchunks) put_state();
    for (int c = 0; c < nchunks; ++c) {
      const int s = c % kStages;
      const DeltaAux& aux = *reinterpret_cast<const DeltaAux*>(sm.packet[s] + kPkAux);
      if (!wait(sm.full[s], c / kStages)) break;
      const float lam1 = factor.next(aux.whole);
      const int j0 = 32 * half + 2 * (lane & 3);
      if (!wait(sm.gx, c)) break;
      // m = beta (s dO^T P + w (G k))
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float p[16], y[16];
        uint32_t hi[8], lo[8];
        tc::tmem_ld16x256(tl + (16u * q << 16) + kColX + 32 * half, p);
        tc::tmem_ld16x256(tl + (16u * q << 16) + kColD + 32 * half, y);
        tc::tmem_wait_ld2(p, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = j0 + 8 * i;
          const float2 e = *reinterpret_cast<const float2*>(&aux.w[t]), b = *reinterpret_cast<const float2*>(&aux.beta[t]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float2 x = tc::mul2(make_float2(P.scale, P.scale), make_float2(y[4 * i + 2 * j], y[4 * i + 2 * j + 1]));
            x = tc::mul2(b, tc::fma2(e, make_float2(p[4 * i + 2 * j], p[4 * i + 2 * j + 1]), x));
            split2(x, hi[2 * i + j], lo[2 * i + j]);
          }
        }
        tc::tmem_st16x128(tl + (16u * q << 16) + kColA + 16 * half, regs(hi));
        tc::tmem_st16x128(tl + (16u * q << 16) + kColA + 32 + 16 * half, regs(lo));
      }
      tc::tmem_wait_st();
      tc::fence_before();
      arrive(sm.xready[half]);
      if (!wait(sm.gu[half], c)) break;
      // -e^b rho
      uint32_t hi[2][8], lo[2][8];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float p[16];
        tc::tmem_ld16x256(tl + (16u * q << 16) + kColX + 32 * half, p);
        tc::tmem_wait_ld(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 e = *reinterpret_cast<const float2*>(&aux.eb[j0 + 8 * i]);
          e = make_float2(-e.x, -e.y);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            split2(tc::mul2(e, make_float2(p[4 * i + 2 * j], p[4 * i + 2 * j + 1])), hi[q][2 * i + j], lo[q][2 * i + j]);
        }
      }
      if (half == 1 && !wait(sm.gu[0], c)) break;  // (the first half's product reads m of both)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        tc::tmem_st16x128(tl + (16u * q << 16) + kColA + 16 * half, regs(hi[q]));
        tc::tmem_st16x128(tl + (16u * q << 16) + kColA + 32 + 16 * half, regs(lo[q]));
      }
      tc::tmem_wait_st();
      tc::fence_before();
      arrive(sm.wready[half]);
      arrive(sm.empty[s]);
      if (!wait(sm.gs[half], c)) break;
      const float2 lam = make_float2(lam1, lam1);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        float r[16];
        tc::tmem_ld16(tl + kColG + 64 * half + 16 * m, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) S[8 * m + j] = tc::fma2(lam, S[8 * m + j], make_float2(r[2 * j], r[2 * j + 1]));
      }
      if (c + 1 < nchunks) {
        if (!wait(sm.scopied, c)) break;
        put_state();
      }
    }
    if (!ok) {
      if (lane == 0) atomicOr(P.status, 1);
    } else if (a.dh0) {
      float4* dst = reinterpret_cast<float4*>(a.dh0 + at);
#pragma unroll
      for (int j = 0; j < 16; ++j) dst[j] = reinterpret_cast<const float4*>(S)[j];
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc::fence_after();
    tc::tmem_dealloc(tbase, 512);
  }
}

}  // namespace

cudaError_t launch_delta_backward(const DeltaProblem& P, const DeltaGrads& g, void* ws, cudaStream_t s) {
  Maps maps{};
  PassArgs a{};
  cudaError_t e;
  if (P.N * P.Hv == 0) return cudaSuccess;
  if (P.Ttot) {
    if ((e = token_map(&maps.q, P.q, P.Hqk, P.Ttot, P.qh, P.qt, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.k, P.k, P.Hqk, P.Ttot, P.kh, P.kt, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.d_o, g.d_o, P.Hv, P.Ttot, kDim, (int64_t)P.Hv * kDim, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.dv, g.dv, P.Hv, P.Ttot, kDim, (int64_t)P.Hv * kDim, kC)) != cudaSuccess) return e;
  }
  a.P = P;
  a.d_hT = g.d_hT;
  a.dh0 = g.dh0;
  const DeltaWs w = delta_workspace(P, true);
  unsigned char* base = reinterpret_cast<unsigned char*>(ws);
  a.packets = base + w.packet;
  a.adjoints = base + w.adjoints;
  a.dv = g.dv;
  if (P.cu_host && P.N > 1 && P.N <= kOrder) {
    a.ordered = 1;
    for (int64_t i = 0; i < P.N; ++i) a.order[i] = (uint16_t)i;
    auto len = [&](int64_t n) { return P.cu_host[n + 1] - P.cu_host[n]; };
    std::stable_sort(a.order, a.order + P.N, [&](uint16_t i, uint16_t j) { return len(i) > len(j); });
  }
  if ((e = cudaFuncSetAttribute(kda_delta_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes)) != cudaSuccess) return e;
  kda_delta_bwd_kernel<<<(unsigned)(P.N * P.Hv), kThreads, kSmemBytes, s>>>(maps, a);
  e = cudaGetLastError();
  return e != cudaSuccess || !P.Ttot ? e : launch_delta_grads(P, g, ws, s);
}

}  // namespace kda
