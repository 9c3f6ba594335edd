// kda_delta_pass.cu -- the passes of the gated delta rule over each sequence's chunks, on sm_103a tensor cores: the
// states forward in time (kda_delta.cuh has the formulas), and their adjoints backwards:
//   d_j = sum_{i >= j} P_ij dO_i + w_j G k_j,   rho = T^T (beta d)  (= dv)
//   G  <- e^{b_C} G + s sum_i e^{b_i} dO_i q_i^T - sum_i e^{b_i} rho_i k_i^T
// with G the adjoint of the state at the chunk's end, value first.
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
// Tensor memory, columns. The carried matrix S as A operand: its columns 64 h + 16 m .. are in 64 h + 8 m .. (high parts)
// and 32 further (low parts): a thread writes where it read the update from.
constexpr uint32_t kColS = 0;    // 128
constexpr uint32_t kColX = 128;  // 64: product with S, then with T
constexpr uint32_t kColA = 192;  // 96: the elements between them as A operands: high, low; forward: beta u too
// forward
constexpr uint32_t kColQ = 288;  // 64: S Q^T
constexpr uint32_t kColO = 352;  // 64: (beta U)^T P^T
// backward
constexpr uint32_t kColD = 256;  // 64: dO^T P
constexpr uint32_t kColE = 320;  // 32 + 32: s e^{b} dO as A operand: high, low
constexpr uint32_t kColG = 384;  // 128: the update's sum, which starts before S has been read (forward it takes S's place)

struct Smem {
  unsigned char tok[kStages][3][kTile];       // K, Q and V or dO
  unsigned char packet[kStages][kPkTrain];    // (kPkTrain is a multiple of 1024)
  unsigned char out[kTile];                   // o or dv on its way out
  unsigned char u[kUTile];                    // u on its way out (training)
  unsigned long long full[kStages], empty[kStages], sready, gx, xready, gu, wready, gs, go, ofree, ufree, eready;
  uint32_t tmem;
};
constexpr int kSmemBytes = (int)sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

constexpr int kOrder = 512;  // sequences whose order is passed (more run in index order)

struct PassArgs {
  DeltaProblem P;
  DecayStates st;
  const unsigned char* packets;
  unsigned char* states;   // BF16 states at the chunks' starts (training), or adjoints at their ends
  unsigned char* u;        // training
  __nv_bfloat16* y;        // o or dv
  int ordered;
  uint16_t order[kOrder];  // longest sequence first
};
struct Maps {
  CUtensorMap q, k, v, y;
};

__device__ __forceinline__ float* regs(uint32_t* x) { return reinterpret_cast<float*>(x); }

// 4 x 2 blocks [8 tokens][8 values] of a token tile, transposed, as tmem_ld16x256 gives a warp's 16 values (from
// `value`) of 32 tokens (from `token`): r[2 i + j] holds tokens token + 8 i + 2 (lane % 4) (+ 1) of value + 8 j + lane / 4.
__device__ __forceinline__ void load_block(uint32_t tile, uint32_t panel, int token, int value, int lane, uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const int t = token + 8 * (i + (lane >> 4)) + (lane & 7), d = value + 8 * ((lane >> 3) & 1);
    tc::ldmatrix4_trans(tile + (d >> 6) * panel + t * 128 + ((((d & 63) >> 3) ^ (t & 7)) << 4), r + 2 * i);
  }
}
// The reverse: into a token tile.
__device__ __forceinline__ void store_block(uint32_t tile, uint32_t panel, int token, int value, int lane, const uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const int t = token + 8 * (i + (lane >> 4)) + (lane & 7), d = value + 8 * ((lane >> 3) & 1);
    tc::stmatrix4_trans(tile + (d >> 6) * panel + t * 128 + ((((d & 63) >> 3) ^ (t & 7)) << 4), r[2 * i], r[2 * i + 1],
                        r[2 * i + 2], r[2 * i + 3]);
  }
}

// kRev: the adjoints, backwards. kTrain: the forward saves states and u.
template <bool kRev, bool kTrain>
__global__ void __launch_bounds__(kThreads, 1) kda_delta_pass_kernel(const __grid_constant__ Maps maps, const __grid_constant__ PassArgs a) {
  extern __shared__ unsigned char raw_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem + ((1024 - (tc::smem_u32(raw_smem) & 1023)) & 1023));
  const DeltaProblem& P = a.P;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [](unsigned long long& b) { return tc::smem_u32(&b); };
  constexpr uint32_t kPacket = kRev ? kPkTrain : kPkForward, kPacketStride = kRev || kTrain ? kPkTrain : kPkInfer;
  constexpr uint32_t kSum = kRev ? kColG : kColS;

  int64_t n = blockIdx.x / P.Hv;
  const int h = (int)(blockIdx.x - n * P.Hv);
  if (a.ordered) n = a.order[n];
  const DecaySpan sp = decay_span(P, n);
  const int64_t slot = a.st.slots ? a.st.slots[n] : n;
  if (slot < 0 || slot >= a.st.num_slots) {
    // a device slot index outside the pool (it no longer matches the host mirror the call was checked
    // against, as in a replayed graph): flagged, and the pool is not touched
    if (tid == 0) atomicOr(P.status, 4);
    return;
  }
  const int nchunks = (int)((sp.len + kC - 1) / kC);
  const int64_t place = delta_slot(sp.t0, n);
  auto chunk = [&](int c) { return kRev ? nchunks - 1 - c : c; };  // the chunk of turn c
  auto tokens = [&](int ci) { return (int)(sp.len - (int64_t)ci * kC < kC ? sp.len - (int64_t)ci * kC : kC); };

  if (warp == kWarpMma) tc::tmem_alloc(tc::smem_u32(&sm.tmem), 512);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) { tc::mbar_init(bar(sm.full[i]), 1); tc::mbar_init(bar(sm.empty[i]), 1 + 2 * kGroup); }
    for (unsigned long long* b : {&sm.sready, &sm.xready, &sm.wready, &sm.ofree, &sm.ufree, &sm.eready}) tc::mbar_init(bar(*b), kGroup);
    for (unsigned long long* b : {&sm.gx, &sm.gu, &sm.gs, &sm.go}) tc::mbar_init(bar(*b), 1);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = sm.tmem;
  bool ok = true;  // false: a wait gave up; the warp leaves its loop
  auto wait = [&](unsigned long long& b, uint32_t parity) {
    if (ok) ok = tc::mbar_wait_lanes(bar(b), parity);
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
      for (; c < nchunks; ++c) {
        const int s = c % kStages, ci = chunk(c);
        if (c >= kStages && !wait(sm.empty[s], (c / kStages - 1) & 1)) break;
        if (lane == 0) {
          const int t = (int)(sp.t0 + (int64_t)ci * kC);
          const uint32_t f = bar(sm.full[s]);
          tc::mbar_arrive_expect_tx(f, 3 * kTile + kPacket);
          tc::bulk_g2s(tc::smem_u32(sm.packet[s]), a.packets + ((place + ci) * P.Hv + h) * (int64_t)kPacketStride, kPacket, f);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            tc::tma_load3(tc::smem_u32(sm.tok[s][0]) + p * kPanel, &maps.k, 64 * p, h / P.r, t, f);
            tc::tma_load3(tc::smem_u32(sm.tok[s][1]) + p * kPanel, &maps.q, 64 * p, h / P.r, t, f);
            tc::tma_load3(tc::smem_u32(sm.tok[s][2]) + p * kPanel, &maps.v, 64 * p, h, t, f);
          }
        }
        __syncwarp();
      }
      if (!ok) {  // flag it, and let this CTA's copies land before its memory is given back
        if (lane == 0) atomicOr(P.status, 1);
        for (int k = c > kStages ? c - kStages : 0; k < c; ++k) tc::mbar_wait_lanes(bar(sm.full[k % kStages]), (k / kStages) & 1, 1u << 16);
      }
    } else if (warp == kWarpMma) {
      for (int c = 0; c < nchunks; ++c) {
        const int s = c % kStages;
        const uint32_t par = c & 1;
        const uint32_t k = tc::smem_u32(sm.tok[s][0]), q = tc::smem_u32(sm.tok[s][1]), v = tc::smem_u32(sm.tok[s][2]);
        const uint32_t pk = tc::smem_u32(sm.packet[s]);
        const uint64_t kk = tc::kmajor(k), kn = tc::mnmajor(k, kPanel), qk = tc::kmajor(q), qn = tc::mnmajor(q, kPanel);
        if (!wait(sm.full[s], (c / kStages) & 1)) break;
        if (kRev) {  // dO^T P, once dO is prepared
          if (!wait(sm.eready, par)) break;
          if (tc::elect_one()) {
            const uint64_t vn = tc::mnmajor(v, kPanel), pn = tc::mnmajor(pk + kPkP, 8192), pl = tc::mnmajor(pk + kPkPlo, 8192);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              tc::mma_bf16_ss(tbase + kColD, vn + 128 * i, pn + 128 * i, tc::idesc_bf16(128, 64, true, true), i > 0);
              tc::mma_bf16_ss(tbase + kColD, vn + 128 * i, pl + 128 * i, tc::idesc_bf16(128, 64, true, true), 1);
            }
          }
          __syncwarp();
        }
        // S K^T
        if (!wait(sm.sready, par)) break;
        if (kTrain && !kRev && c && !wait(sm.ufree, (c - 1) & 1)) break;
        if (kRev && c && !wait(sm.ofree, (c - 1) & 1)) break;
        if (tc::elect_one()) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t off = (i >> 2) * (kPanel >> 4) + (i & 3) * 2, col = tbase + kColS + 64 * (i >> 2) + 8 * (i & 3);
            tc::mma_bf16_ts(tbase + kColX, col, kk + off, tc::idesc_bf16(128, 64, false, false), i > 0);
            tc::mma_bf16_ts(tbase + kColX, col + 32, kk + off, tc::idesc_bf16(128, 64, false, false), 1);
          }
          tc::mma_commit(bar(sm.gx));
        }
        __syncwarp();
        if (!kRev) {  // S Q^T
          if (c && !wait(sm.ofree, (c - 1) & 1)) break;
          if (tc::elect_one()) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t off = (i >> 2) * (kPanel >> 4) + (i & 3) * 2, col = tbase + kColS + 64 * (i >> 2) + 8 * (i & 3);
              tc::mma_bf16_ts(tbase + kColQ, col, qk + off, tc::idesc_bf16(128, 64, false, false), i > 0);
              tc::mma_bf16_ts(tbase + kColQ, col + 32, qk + off, tc::idesc_bf16(128, 64, false, false), 1);
            }
          }
        } else if (tc::elect_one()) {  // (s e^b dO)^T Q
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tc::mma_bf16_ts(tbase + kSum, tbase + kColE + 8 * i, qn + 128 * i, tc::idesc_bf16(128, 128, false, true), i > 0);
            tc::mma_bf16_ts(tbase + kSum, tbase + kColE + 32 + 8 * i, qn + 128 * i, tc::idesc_bf16(128, 128, false, true), 1);
          }
        }
        __syncwarp();
        // with T
        if (!wait(sm.xready, par)) break;
        if (tc::elect_one()) {
          const uint64_t th = kRev ? tc::mnmajor(pk + kPkT, 8192) : tc::kmajor(pk + kPkT);
          const uint64_t tl = kRev ? tc::mnmajor(pk + kPkTlo, 8192) : tc::kmajor(pk + kPkTlo);
          constexpr uint32_t step = kRev ? 128 : 2;
          constexpr uint32_t id = tc::idesc_bf16(128, 64, false, kRev);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = tbase + kColA + 8 * i;
            tc::mma_bf16_ts(tbase + kColX, x, th + step * i, id, i > 0);
            tc::mma_bf16_ts(tbase + kColX, x, tl + step * i, id, 1);
            tc::mma_bf16_ts(tbase + kColX, x + 32, th + step * i, id, 1);
          }
          tc::mma_commit(bar(sm.gu));
        }
        __syncwarp();
        // the update of S, and what is left of the output
        if (!wait(sm.wready, par)) break;
        if (tc::elect_one()) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = tbase + kColA + 8 * i;
            tc::mma_bf16_ts(tbase + kSum, x, kn + 128 * i, tc::idesc_bf16(128, 128, false, true), kRev || i > 0);
            tc::mma_bf16_ts(tbase + kSum, x + 32, kn + 128 * i, tc::idesc_bf16(128, 128, false, true), 1);
          }
          tc::mma_commit(bar(sm.gs));
          if (!kRev) {
            const uint64_t p = tc::kmajor(pk + kPkP);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              tc::mma_bf16_ts(tbase + kColO, tbase + kColA + 64 + 8 * i, p + 2 * i, tc::idesc_bf16(128, 64, false, false), i > 0);
            tc::mma_commit(bar(sm.go));
          }
          tc::mma_commit(bar(sm.empty[s]));
        }
        __syncwarp();
      }
    }
  } else if (warp < kWarpChain) {
    // ================= what leaves: o and u, or dv; backward: dO as an operand
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
      const int s = c % kStages, ci = chunk(c), nt = tokens(ci);
      const uint32_t par = c & 1;
      const int64_t t0 = sp.t0 + (int64_t)ci * kC;
      const DeltaAux& aux = *reinterpret_cast<const DeltaAux*>(sm.packet[s] + kPkAux);
      wait(sm.full[s], (c / kStages) & 1);
      if (kRev) {
        if (ok && nt < kC)  // rows past the end hold other tokens
          for (int i = tid - 32 * kWarpOut; i < (kC - nt) * 48; i += 32 * kGroup) {
            const int row = nt + i / 48, x = i % 48;
            *reinterpret_cast<uint4*>(sm.tok[s][x >> 4] + ((x >> 3) & 1) * kPanel + row * 128 + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
        if (nt < kC) {
          tc::fence_async_smem();
          if (!agree()) break;
        }
        uint32_t hi[2][8], lo[2][8];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t r[8];
          load_block(tc::smem_u32(sm.tok[s][2]), kPanel, 32 * half, 32 * wq + 16 * q, lane, r);
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
      }
      if (kRev || kTrain) {
        wait(sm.gu, par);
        unsigned char* to = kRev ? sm.out : sm.u;
        if (warp == kWarpOut && lane == 0) {  // the last one has left
          if (kRev) tc::bulk_wait_read();
          else tc::bulk_wait_read1();
        }
        if (!agree()) break;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float r[16];
          tc::tmem_ld16x256(tl + (16u * q << 16) + kColX + 32 * half, r);
          tc::tmem_wait_ld(r);
          uint32_t z[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = pack2(r[2 * i], r[2 * i + 1]);
          store_block(tc::smem_u32(to), kPanel, 32 * half, 32 * wq + 16 * q, lane, z);
        }
        tc::fence_before();
        arrive(kRev ? sm.ofree : sm.ufree);
        tc::fence_async_smem();
        asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * kGroup) : "memory");
        if (!kRev && warp == kWarpOut && lane == 0) {
          tc::bulk_s2g(a.u + ((place + ci) * P.Hv + h) * (int64_t)kUTile, tc::smem_u32(sm.u), kUTile);
          tc::bulk_commit();
        }
      }
      if (!kRev) {
        wait(sm.go, par);
        if (warp == kWarpOut && lane == 0) {
          if (kTrain) tc::bulk_wait_read1();
          else tc::bulk_wait_read();
        }
        if (!agree()) break;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float r[16], y[16];
          tc::tmem_ld16x256(tl + (16u * q << 16) + kColQ + 32 * half, r);
          tc::tmem_ld16x256(tl + (16u * q << 16) + kColO + 32 * half, y);
          tc::tmem_wait_ld2(r, y);
          uint32_t z[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 e = *reinterpret_cast<const float2*>(&aux.eb[32 * half + 8 * i + 2 * (lane & 3)]);
            e = make_float2(P.scale * e.x, P.scale * e.y);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              z[2 * i + j] = pack2(tc::fma2(e, make_float2(r[4 * i + 2 * j], r[4 * i + 2 * j + 1]), make_float2(y[4 * i + 2 * j], y[4 * i + 2 * j + 1])));
          }
          store_block(tc::smem_u32(sm.out), kPanel, 32 * half, 32 * wq + 16 * q, lane, z);
        }
        tc::fence_before();
        arrive(sm.ofree);
        tc::fence_async_smem();
        asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * kGroup) : "memory");
      }
      arrive(sm.empty[s]);
      if (nt == kC) {
        if (warp == kWarpOut && lane == 0) {
          tc::tma_store3(&maps.y, tc::smem_u32(sm.out), 0, h, (int)t0);
          tc::tma_store3(&maps.y, tc::smem_u32(sm.out) + kPanel, 64, h, (int)t0);
          tc::bulk_commit();
        }
      } else {  // (a whole tile would run into the next sequence)
        for (int i = tid - 32 * kWarpOut; i < nt * 16; i += 32 * kGroup) {
          const int t = i >> 4, k = i & 15;
          *reinterpret_cast<uint4*>(a.y + ((t0 + t) * P.Hv + h) * kDim + 8 * k) =
              *reinterpret_cast<const uint4*>(sm.out + (k >> 3) * kPanel + t * 128 + (((k & 7) ^ (t & 7)) << 4));
        }
        // (the next chunk's tile is written after the barrier above it)
      }
    }
    if (warp == kWarpOut && lane == 0) tc::bulk_wait();
    if (!ok && lane == 0) atomicOr(P.status, 1);
  } else {
    // ================= the chain of the carried matrix
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int wq = (warp - kWarpChain) & 3, half = (warp - kWarpChain) >> 2;
    const int v = 32 * wq + lane;  // row of this thread, its columns 64 half .. + 63
    const uint32_t tl = tbase + ((uint32_t)(32 * wq) << 16);
    const int64_t at = (slot * P.Hv + h) * kDim * kDim + v * kDim + 64 * half;
    float2 S[32];
    if (!a.st.in) {
#pragma unroll
      for (int j = 0; j < 32; ++j) S[j] = make_float2(0.f, 0.f);
    } else if (!a.st.bf16) {
      const float4* src = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.st.in) + at);
#pragma unroll
      for (int j = 0; j < 16; ++j) reinterpret_cast<float4*>(S)[j] = src[j];
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.st.in) + at);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 r = src[j];
        S[4 * j] = unpack2(r.x); S[4 * j + 1] = unpack2(r.y); S[4 * j + 2] = unpack2(r.z); S[4 * j + 3] = unpack2(r.w);
      }
    }
    auto put_state = [&](int c) {  // as turn c's operand
      unsigned char* save = a.states + ((place + chunk(c)) * P.Hv + h) * (int64_t)kStateTile + half * 16384 + v * 128;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split2(S[8 * m + e], hi[e], lo[e]);
        tc::tmem_st8(tl + kColS + 64 * half + 8 * m, hi);
        tc::tmem_st8(tl + kColS + 64 * half + 32 + 8 * m, lo);
        if (kRev || kTrain) {
          *reinterpret_cast<uint4*>(save + (((2 * m) ^ (v & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(save + (((2 * m + 1) ^ (v & 7)) << 4)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
        }
      }
      tc::tmem_wait_st();
      tc::fence_before();
      arrive(sm.sready);
    };
    StateFactor factor;
    if (nchunks) put_state(0);
    for (int c = 0; c < nchunks; ++c) {
      const int s = c % kStages, nt = tokens(chunk(c));
      const uint32_t par = c & 1;
      const DeltaAux& aux = *reinterpret_cast<const DeltaAux*>(sm.packet[s] + kPkAux);
      if (!wait(sm.full[s], (c / kStages) & 1)) break;
      const float lam1 = factor.next(aux.whole);
      const int j0 = 32 * half + 2 * (lane & 3);
      if (!wait(sm.gx, par)) break;
      // x = v - e^b (S k), or m = beta (dO^T P + w (G k)); zero past the end
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float p[16], y[16];
        uint32_t r[8], hi[8], lo[8];
        tc::tmem_ld16x256(tl + (16u * q << 16) + kColX + 32 * half, p);
        if (kRev) {
          tc::tmem_ld16x256(tl + (16u * q << 16) + kColD + 32 * half, y);
          tc::tmem_wait_ld2(p, y);
        } else {
          load_block(tc::smem_u32(sm.tok[s][2]), kPanel, 32 * half, 32 * wq + 16 * q, lane, r);
          tc::tmem_wait_ld(p);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = j0 + 8 * i;
          float2 e = *reinterpret_cast<const float2*>(kRev ? &aux.w[t] : &aux.eb[t]);
          const float2 b = *reinterpret_cast<const float2*>(&aux.beta[t]);
          if (!kRev) e = make_float2(-e.x, -e.y);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 add = kRev ? make_float2(y[4 * i + 2 * j], y[4 * i + 2 * j + 1]) : unpack2(r[2 * i + j]);
            float2 x = tc::fma2(e, make_float2(p[4 * i + 2 * j], p[4 * i + 2 * j + 1]), add);
            if (kRev) x = tc::mul2(b, x);
            if (t >= nt) x.x = 0.f;
            if (t + 1 >= nt) x.y = 0.f;
            split2(x, hi[2 * i + j], lo[2 * i + j]);
          }
        }
        tc::tmem_st16x128(tl + (16u * q << 16) + kColA + 16 * half, regs(hi));
        tc::tmem_st16x128(tl + (16u * q << 16) + kColA + 32 + 16 * half, regs(lo));
      }
      if (!kRev && nt < kC) {  // K's rows past the end hold other tokens (its product with S is done)
        for (int i = tid - 32 * kWarpChain; i < (kC - nt) * 16; i += 32 * kGroup)
          *reinterpret_cast<uint4*>(sm.tok[s][0] + ((i >> 3) & 1) * kPanel + (nt + (i >> 4)) * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        tc::fence_async_smem();
      }
      tc::tmem_wait_st();
      tc::fence_before();
      arrive(sm.xready);
      if (!wait(sm.gu, par)) break;
      // w beta u, and beta u; or -e^b rho
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float p[16];
        uint32_t hi[8], lo[8], un[8];
        tc::tmem_ld16x256(tl + (16u * q << 16) + kColX + 32 * half, p);
        tc::tmem_wait_ld(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = j0 + 8 * i;
          const float2 e = *reinterpret_cast<const float2*>(kRev ? &aux.eb[t] : &aux.w[t]);
          const float2 b = kRev ? make_float2(-1.f, -1.f) : *reinterpret_cast<const float2*>(&aux.beta[t]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 x = tc::mul2(b, make_float2(p[4 * i + 2 * j], p[4 * i + 2 * j + 1]));
            split2(tc::mul2(e, x), hi[2 * i + j], lo[2 * i + j]);
            if (!kRev) un[2 * i + j] = pack2(x);
          }
        }
        tc::tmem_st16x128(tl + (16u * q << 16) + kColA + 16 * half, regs(hi));
        tc::tmem_st16x128(tl + (16u * q << 16) + kColA + 32 + 16 * half, regs(lo));
        if (!kRev) tc::tmem_st16x128(tl + (16u * q << 16) + kColA + 64 + 16 * half, regs(un));
      }
      tc::tmem_wait_st();
      tc::fence_before();
      arrive(sm.wready);
      arrive(sm.empty[s]);
      if (!wait(sm.gs, par)) break;
      const float2 lam = make_float2(lam1, lam1);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        float r[16];
        tc::tmem_ld16(tl + kSum + 64 * half + 16 * m, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) S[8 * m + j] = tc::fma2(lam, S[8 * m + j], make_float2(r[2 * j], r[2 * j + 1]));
      }
      if (c + 1 < nchunks) put_state(c + 1);
    }
    if (!ok) {
      if (lane == 0) atomicOr(P.status, 1);
    } else if (a.st.out && !a.st.bf16) {
      float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.st.out) + at);
#pragma unroll
      for (int j = 0; j < 16; ++j) dst[j] = reinterpret_cast<const float4*>(S)[j];
    } else if (a.st.out) {
      uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.st.out) + at);
#pragma unroll
      for (int j = 0; j < 8; ++j) dst[j] = make_uint4(pack2(S[4 * j]), pack2(S[4 * j + 1]), pack2(S[4 * j + 2]), pack2(S[4 * j + 3]));
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc::fence_after();
    tc::tmem_dealloc(tbase, 512);
  }
}

template <bool kRev, bool kTrain>
cudaError_t pass(const DeltaProblem& P, const DecayStates& st, const __nv_bfloat16* v, int64_t vt, int64_t vh, __nv_bfloat16* y,
                 unsigned char* ws, cudaStream_t s) {
  Maps maps{};
  PassArgs a{};
  cudaError_t e;
  if (P.N * P.Hv == 0) return cudaSuccess;
  if (P.Ttot) {
    if ((e = token_map(&maps.q, P.q, P.Hqk, P.Ttot, P.qh, P.qt, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.k, P.k, P.Hqk, P.Ttot, P.kh, P.kt, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.v, v, P.Hv, P.Ttot, vh, vt, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.y, y, P.Hv, P.Ttot, kDim, (int64_t)P.Hv * kDim, kC)) != cudaSuccess) return e;
  }
  a.P = P;
  a.st = st;
  const DeltaWs w = delta_workspace(P.slots, P.Hv, kRev || kTrain);
  a.packets = ws + w.packet;
  a.states = ws + (kRev ? w.adjoints : w.states);
  a.u = ws + w.u;
  a.y = y;
  if (P.cu_host && P.N > 1 && P.N <= kOrder) {
    a.ordered = 1;
    for (int64_t i = 0; i < P.N; ++i) a.order[i] = (uint16_t)i;
    auto len = [&](int64_t n) { return P.cu_host[n + 1] - P.cu_host[n]; };
    std::stable_sort(a.order, a.order + P.N, [&](uint16_t i, uint16_t j) { return len(i) > len(j); });
  }
  auto kern = kda_delta_pass_kernel<kRev, kTrain>;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes)) != cudaSuccess) return e;
  kern<<<(unsigned)(P.N * P.Hv), kThreads, kSmemBytes, s>>>(maps, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_forward(const DeltaProblem& P, const DecayStates& st, __nv_bfloat16* o, bool training, void* ws,
                                 cudaStream_t s) {
  const cudaError_t e = launch_delta_prep(P, training, ws, s);
  if (e != cudaSuccess) return e;
  unsigned char* w = reinterpret_cast<unsigned char*>(ws);
  return training ? pass<false, true>(P, st, P.v, P.vt, P.vh, o, w, s) : pass<false, false>(P, st, P.v, P.vt, P.vh, o, w, s);
}

cudaError_t launch_delta_backward(const DeltaProblem& P, const DeltaGrads& g, void* ws, cudaStream_t s) {
  unsigned char* w = reinterpret_cast<unsigned char*>(ws);
  const DecayStates st{g.d_hT, g.dh0, 0, nullptr, P.N};
  const cudaError_t e = pass<true, false>(P, st, g.d_o, (int64_t)P.Hv * kDim, kDim, g.dv, w, s);
  return e != cudaSuccess || !P.Ttot ? e : launch_delta_grads(P, g, ws, s);
}

}  // namespace kda
