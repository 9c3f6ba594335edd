// kda_delta_grad.cu -- the part of the gated delta rule's backward that lies within chunks, for all chunks side by side.
// From a chunk's start state S, the adjoint G of its end state, u and rho (= dv), with r a value head of the group:
//   A_ij = s D_ij beta_j dO_i . u_j  (j <= i),   R_ij = D_ij beta_j rho_i . u_j  (j < i)
//   dq_i = s e^{b_i} S^T dO_i + sum_j A_ij k_j
//   dk_j = w_j beta_j G^T u_j - e^{b_j} S^T rho_j + sum_i A_ij q_i - sum_i (R_ij + R_ji) k_i
// summed over the group's heads. The rest needs no product of its own: with E_ij = s D_ij (q_i . k_j)(dO_i . u_j) and
// F_ij = D_ij (k_i . k_j)(rho_i . u_j),
//   dbeta_j = sum_i E_ij - sum_i F_ij + w_j k_j . G^T u_j
// and, as a decay scales all that crosses its token,
//   dg_t = sum_{i >= t} e^{b_i} (s q_i . S^T dO_i - k_i . S^T rho_i) + sum_{j < t} w_j beta_j k_j . G^T u_j + e^{b_C} <G, S>
//        + sum_{i >= t > j} beta_j (E_ij - F_ij)
// whose last sum grows from t to t + 1 by the column t below the diagonal less the row t before it. (The shorter
// q_i . dq_i - v_i . dv_i summed from t on has the same value, but its terms cancel: 1.8e-2 off from operands in BF16, this 2.5e-3.)
// Nothing is carried on from these sums, so operands are in one BF16 part (S, G, u, rho = dv as it is returned, A, R): gradients are 2.4e-3
// to 3.0e-3 from 64 bits, 1.7e-3 of it their own rounding. Second parts of the tiles would be twice the bytes, and have no room.
#include "kda_delta.cuh"
#include "kda_layout.h"
#include "kda_tma.h"
#include "tc.cuh"

namespace kda {
namespace {

constexpr int kC = kDecayChunk;
constexpr int kThreads = 512;
constexpr int kWarpMma = 12;  // issues the products: all its scores lie above the diagonal, so it has time
// Tensor memory, columns (64 each)
constexpr uint32_t kColUU = 0;     // [dO; rho] u^T
constexpr uint32_t kColKK = 64;    // [Q; K] K^T
constexpr uint32_t kColQS = 128;   // S^T dO^T, and beside it
constexpr uint32_t kColKS = 192;   // S^T rho^T
constexpr uint32_t kColKG = 256;   // G^T u^T
constexpr uint32_t kColQA = 320;   // K^T A^T
constexpr uint32_t kColKA = 384;   // Q^T A - K^T (R + R^T)

struct Maps {
  CUtensorMap q, k, d_o, dv;
};

// A chunk's scalars, of two (chunk, value head) pairs in turn.
struct Numbers {
  float rowp[2][4][kC];       // rows of E beta and -F beta before the diagonal, by quarter of the columns
  float colp[4][kC];          // columns of E (two row halves), -F (two)
  float diag[kC];             // E_ii
  float dot[3][4][kC];        // q . S^T dO, k . G^T u, k . S^T rho, by lane quadrant
  float gs[kThreads / 32];       // <G, S> of each warp
};
struct Smem {
  unsigned char S[kStateTile], G[kStateTile];
  unsigned char qk[2][32768];  // [2 panels][64 rows of Q, 64 of K][64], of two units in turn; at last dq and dk on their way out
  unsigned char dr[32768];     // the same of dO and rho
  unsigned char u[kUTile];
  unsigned char A[8192], R[8192];
  DeltaAux aux[2];
  Numbers num[2];
  unsigned long long fullqk[2], full, g1, gs, g2;
  int2 next[2];                // chunks of units to come, of two in turn,
  uint32_t asked[2];           // and which they are
  uint32_t tmem;
};
constexpr int kSmemBytes = (int)sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

// 16 tokens (from `token`) and 16 values of a tile, transposed as tmem_ld16x256x2 gives a warp's: r[2 i + j] holds tokens
// token + 8 i + 2 (lane % 4) (+ 1) of value + 8 j + lane / 4. `at`: where this lane's matrix row is.
__device__ __forceinline__ uint32_t block_row(uint32_t tile, int token, int value, int lane) {
  const int t = token + 8 * (lane >> 4) + (lane & 7), d = value + 8 * ((lane >> 3) & 1);
  return tile + (d >> 6) * 16384 + t * 128 + ((((d & 63) >> 3) ^ (t & 7)) << 4);
}

// Sums over the eight lanes that share lane % 4 of four numbers, those of tokens 8 m + 2 (lane % 4) + e at 2 m + e: lane l
// < 16 gets that of token over_token(l).
__device__ __forceinline__ float over_rows(float (&x)[4], int lane) {
  const bool a = lane & 4, b = lane & 8;
  float y0 = (a ? x[2] : x[0]) + __shfl_xor_sync(0xffffffffu, a ? x[0] : x[2], 4);
  float y1 = (a ? x[3] : x[1]) + __shfl_xor_sync(0xffffffffu, a ? x[1] : x[3], 4);
  float y = (b ? y1 : y0) + __shfl_xor_sync(0xffffffffu, b ? y0 : y1, 8);
  return y + __shfl_xor_sync(0xffffffffu, y, 16);
}
__device__ __forceinline__ int over_token(int token, int lane) { return token + 8 * ((lane >> 2) & 1) + 2 * (lane & 3) + ((lane >> 3) & 1); }

// One CTA an SM goes through the (chunk, query/key head) units b, b + gridDim.x, ..., and in each through the group's value heads. The
// tiles of the next head are on their way once the first products of this one, their only readers, are done. Bound: a pair's
// chain of two products' groups and the elements between them, 16 warps (8000 cycles, of which the 144 KiB of tiles in and out take
// 70 %): 4 x 2048 tokens of 16 / 32 heads 135 us; a CTA for each unit, with nothing on its way, 236 us. Products are
// transposed, [128 values x 64 tokens], so that all have M = 128 and the tokens' factors are applied where the sums are read.
__global__ void __launch_bounds__(kThreads, 1)
kda_delta_grad_kernel(const __grid_constant__ Maps maps, const DeltaProblem P, const unsigned char* packets, const unsigned char* states,
                      const unsigned char* adjoints, const unsigned char* us, const int2* chunks, const DeltaGrads G) {
  extern __shared__ unsigned char raw_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem + ((1024 - (tc::smem_u32(raw_smem) & 1023)) & 1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wq = warp & 3, quarter = warp >> 2;
  auto bar = [](unsigned long long& b) { return tc::smem_u32(&b); };
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&sm.tmem), 512);
  if (tid == 0)
    for (unsigned long long* b : {&sm.fullqk[0], &sm.fullqk[1], &sm.full, &sm.g1, &sm.gs, &sm.g2}) tc::mbar_init(bar(*b), 1);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = sm.tmem, tl = tbase + ((uint32_t)(32 * wq) << 16) + 16 * quarter;
  const uint32_t dr = tc::smem_u32(sm.dr);
  bool ok = true;
  auto wait = [&](unsigned long long& b, uint32_t parity) {
    if (ok) ok = tc::mbar_wait_lanes(bar(b), parity & 1);
    tc::fence_after();
  };
  const uint32_t units = (uint32_t)(P.slots * P.Hqk);
  // the first unit from x on that has a chunk, from prep's list (looking for it took 2000 cycles, and a load behind all the tiles
  // on their way 5000: the usual one is asked for two units before)
  int2 ch{0, 0}, ch1{0, 0};
  // (held inside the tensors, whatever the workspace holds: tokens of none where it does not begin in one)
  auto held = [&](int2 c) {
    const uint32_t all = (uint32_t)P.Ttot, at = (uint32_t)c.x;
    return make_int2(c.x, at >= all ? 0 : min(c.y, (int)min(all - at, (uint32_t)kC)));
  };
  auto find = [&](uint32_t x, int2& c) {
    for (; x < units; x += gridDim.x) {
      c = held(chunks[x / (uint32_t)P.Hqk]);
      if (c.y > 0) break;
    }
    return x;
  };
  auto ask = [&](uint32_t x, uint32_t to) {
    if (tid) return;
    sm.asked[to] = x;
    if (x < units) tc::cp_async_small<8>(&sm.next[to], chunks + x / (uint32_t)P.Hqk, 8);
    tc::cp_async_commit();
  };
  // The tiles of one head (and, of a unit's first, of Q and K), by one lane of each of six warps. (One warp took 2000 cycles.)
  auto load = [&](int64_t slot, int hq, int64_t t, int r, uint32_t par, uint32_t ub) {
    if (warp > 5 || !tc::elect_one()) return;
    const int h = hq * P.r + r;
    const int64_t place = slot * P.Hv + h;
    const uint32_t f = bar(sm.full), fq = bar(sm.fullqk[ub]);
    if (warp == 0) {
      tc::mbar_arrive_expect_tx(f, 2 * kStateTile + 32768 + kUTile + sizeof(DeltaAux));
      tc::bulk_g2s(tc::smem_u32(sm.u), us + place * kUTile, kUTile, f);
    } else if (warp < 3) {
#pragma unroll
      for (int p = 0; p < 2; ++p) tc::tma_load3(dr + p * 16384 + 8192 * (warp - 1), warp == 1 ? &maps.d_o : &maps.dv, 64 * p, h, (int)t, f);
    } else if (warp == 3) {
      tc::bulk_g2s(tc::smem_u32(sm.S), states + place * kStateTile, kStateTile, f);
      tc::bulk_g2s(tc::smem_u32(&sm.aux[par]), packets + place * kPkTrain + kPkAux, sizeof(DeltaAux), f);
    } else if (warp == 4) {
      tc::bulk_g2s(tc::smem_u32(sm.G), adjoints + place * kStateTile, kStateTile, f);
    } else if (r == 0) {
      const uint32_t qk = tc::smem_u32(sm.qk[ub]);
      tc::mbar_arrive_expect_tx(fq, 32768);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        tc::tma_load3(qk + p * 16384, &maps.q, 64 * p, hq, (int)t, fq);
        tc::tma_load3(qk + p * 16384 + 8192, &maps.k, 64 * p, hq, (int)t, fq);
      }
    }
  };
  uint32_t unit = find(blockIdx.x, ch), unit1 = unit;
  int slot = (int)(unit / (uint32_t)P.Hqk), slot1 = slot, hq = (int)(unit - (uint32_t)slot * P.Hqk), hq1 = hq;
  if (unit < units) load(slot, hq, ch.x, 0, 0, 0);
  __syncwarp();
  const int tok0 = 16 * quarter + 2 * (lane & 3);  // this thread's tokens: tok0 + 8 m + e
  uint32_t n = 0;                                  // heads so far
  ask(unit + gridDim.x, 0);
  for (uint32_t un = 0; unit < units; ++un, unit = unit1, ch = ch1, slot = slot1, hq = hq1) {
    const uint32_t qk = tc::smem_u32(sm.qk[un & 1]);
    const int nt = ch.y;
    const int64_t t0 = ch.x;
    float sq[2][8], sk[2][8];  // dq, dk: values 32 wq + 16 q + 8 j + lane / 4 of tokens tok0 + 8 m + e, at 4 m + 2 j + e
#pragma unroll
    for (int i = 0; i < 16; ++i) sq[i >> 3][i & 7] = sk[i >> 3][i & 7] = 0.f;
    for (int r = 0; r < P.r; ++r, ++n) {
      const int h = hq * P.r + r;
      const uint32_t par = n & 1;
      const DeltaAux& aux = sm.aux[par];
      Numbers& num = sm.num[par];
      const bool last = r + 1 == P.r;
      if (last) ask(unit + 2 * gridDim.x, ~un & 1);
      if (r == 0) wait(sm.fullqk[un & 1], un >> 1);
      wait(sm.full, n);
      if (nt < kC) {  // rows past the end hold other tokens
        for (int i = tid; i < (kC - nt) * 64; i += kThreads) {
          const int row = nt + (i >> 6), x = i & 63;  // 16-byte pieces of a row: 16 of dO, rho, Q, K
          unsigned char* t = (x & 32 ? sm.qk[un & 1] : sm.dr) + ((x >> 3) & 1) * 16384 + ((x >> 4) & 1) * 8192;
          if (r == 0 || !(x & 32)) *reinterpret_cast<uint4*>(t + row * 128 + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        tc::fence_async_smem();
        __syncthreads();
      }
      constexpr uint32_t kn = tc::idesc_bf16(128, 64, false, false), tn = tc::idesc_bf16(128, 64, true, false), tt = tc::idesc_bf16(128, 64, true, true);
      if (warp == kWarpMma) {
        if (ok && tc::elect_one()) {
          const uint64_t u = tc::kmajor(tc::smem_u32(sm.u)), St = tc::mnmajor(tc::smem_u32(sm.S), 16384), Gt = tc::mnmajor(tc::smem_u32(sm.G), 16384);
          // (the scores first: their elements are worked on while the states' products run)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t off = (i >> 2) * (16384 >> 4) + (i & 3) * 2, off64 = (i >> 2) * (8192 >> 4) + (i & 3) * 2;
            tc::mma_bf16_ss(tbase + kColUU, tc::kmajor(dr) + off, u + off64, kn, i > 0);
            if (r == 0) tc::mma_bf16_ss(tbase + kColKK, tc::kmajor(qk) + off, tc::kmajor(qk + 8192) + off, kn, i > 0);
          }
          tc::mma_commit(bar(sm.g1));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t off = (i >> 2) * (16384 >> 4) + (i & 3) * 2, off64 = (i >> 2) * (8192 >> 4) + (i & 3) * 2;
            tc::mma_bf16_ss(tbase + kColQS, St + 128 * i, tc::kmajor(dr) + off, tc::idesc_bf16(128, 128, true, false), i > 0);
            tc::mma_bf16_ss(tbase + kColKG, Gt + 128 * i, u + off64, tn, i > 0);
          }
          tc::mma_commit(bar(sm.gs));
        }
        __syncwarp();
      }
      if (G.dg) {  // <G, S>: the tiles are laid out alike
        float x = 0.f;
#pragma unroll
        for (int j = 0; j < (int)kStateTile / 16 / kThreads; ++j) {
          const uint4 a = reinterpret_cast<const uint4*>(sm.S)[tid + kThreads * j], b = reinterpret_cast<const uint4*>(sm.G)[tid + kThreads * j];
          const float2 y = tc::fma2(unpack2(a.x), unpack2(b.x), tc::fma2(unpack2(a.y), unpack2(b.y), tc::fma2(unpack2(a.z), unpack2(b.z), tc::mul2(unpack2(a.w), unpack2(b.w)))));
          x += y.x + y.y;
        }
#pragma unroll
        for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
        if (lane == 0) num.gs[warp] = x;
      }
      wait(sm.g1, n);
      // the scores: rows i = 32 (wq % 2) + 16 q + 8 j + lane / 4 of dO and Q (wq < 2) or rho and K, columns tok0 + 8 m + e
      {
        const bool first = wq < 2;
        float col[4] = {0.f, 0.f, 0.f, 0.f};
        float2 beta[2], bt[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          beta[m] = *reinterpret_cast<const float2*>(&aux.beta[tok0 + 8 * m]);
          bt[m] = *reinterpret_cast<const float2*>(&aux.b[tok0 + 8 * m]);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          unsigned char* to = first ? sm.A : sm.R;
          const int block = 2 * (wq & 1) + q;  // of sixteen rows
          float uu[8], kk[8];
          if (quarter <= block) {
            tc::tmem_ld16x256x2(tl + (16u * q << 16) + kColUU, uu);
            tc::tmem_ld16x256x2(tl + (16u * q << 16) + kColKK, kk);
            tc::tmem_wait_ld8x2(uu, kk);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int i = 16 * block + 8 * j + (lane >> 2);
            const float bi = aux.b[i], f = first ? P.scale : -1.f;
            float row = 0.f;
            uint32_t packed[2] = {0u, 0u};
            if (quarter <= block) {
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                float z[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int t = tok0 + 8 * m + e;
                  const float be = e ? beta[m].y : beta[m].x, x = uu[4 * m + 2 * j + e];
                  const bool in = first ? t <= i : t < i;
                  const float d = in ? fast_exp2(bi - (e ? bt[m].y : bt[m].x)) * f * x : 0.f;
                  z[e] = d * be;
                  const float y = in ? d * kk[4 * m + 2 * j + e] : 0.f;
                  col[2 * m + e] += y;
                  if (t < i) row = fmaf(y, be, row);
                  if (first && t == i) num.diag[i] = y;
                }
                packed[m] = pack2(z[0], z[1]);
              }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
              *reinterpret_cast<uint32_t*>(to + i * 128 + (((2 * quarter + m) ^ (i & 7)) << 4) + 4 * (lane & 3)) = packed[m];
            row += __shfl_xor_sync(0xffffffffu, row, 1);
            row += __shfl_xor_sync(0xffffffffu, row, 2);
            if ((lane & 3) == 0) num.rowp[first ? 0 : 1][quarter][i] = row;
          }
        }
        const float c = over_rows(col, lane);
        if (lane < 16) num.colp[wq][over_token(16 * quarter, lane)] = c;
      }
      if (last && tid == 0) tc::cp_async_wait<1>();
      tc::fence_async_smem();
      tc::fence_before();
      __syncthreads();
      tc::fence_after();
      if (warp == kWarpMma) {
        if (ok && tc::elect_one()) {
          const uint64_t Qt = tc::mnmajor(qk, 16384), Kt = tc::mnmajor(qk + 8192, 16384);
          const uint32_t A = tc::smem_u32(sm.A), R = tc::smem_u32(sm.R);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tc::mma_bf16_ss(tbase + kColQA, Kt + 128 * i, tc::kmajor(A) + 2 * i, tn, i > 0);
            tc::mma_bf16_ss(tbase + kColKA, Qt + 128 * i, tc::mnmajor(A, 8192) + 128 * i, tt, i > 0);
            tc::mma_bf16_ss(tbase + kColKA, Kt + 128 * i, tc::kmajor(R) + 2 * i, tn, 1);
            tc::mma_bf16_ss(tbase + kColKA, Kt + 128 * i, tc::mnmajor(R, 8192) + 128 * i, tt, 1);
          }
          tc::mma_commit(bar(sm.g2));
        }
        __syncwarp();
      }
      wait(sm.gs, n);
      if (last) {
        unit1 = unit + gridDim.x;
        if (unit1 < units) {
          const bool here = sm.asked[un & 1] == unit1;
          if (here) ch1 = held(sm.next[un & 1]);
          if (!here || ch1.y <= 0) unit1 = find(here ? unit1 + gridDim.x : unit1, ch1);
        }
        slot1 = (int)(unit1 / (uint32_t)P.Hqk);
        hq1 = (int)(unit1 - (uint32_t)slot1 * P.Hqk);
      }
      if (ok) {  // the next head's tiles: the readers of this one's are done
        if (!last) load(slot, hq, t0, r + 1, par ^ 1, un & 1);
        else if (unit1 < units) load(slot1, hq1, ch1.x, 0, par ^ 1, (un + 1) & 1);
      }
      __syncwarp();
      // products with the states, and their dots with q and k
      auto part = [&](uint32_t col, uint32_t tile, float* dot, float2 f0, float2 f1, float (&sum)[2][8]) {
        float d[4] = {0.f, 0.f, 0.f, 0.f}, p[2][8];
        uint32_t x[2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          tc::tmem_ld16x256x2(tl + (16u * q << 16) + col, p[q]);
          tc::ldmatrix4_trans(block_row(tile, 16 * quarter, 32 * wq + 16 * q, lane), x[q]);
        }
        tc::tmem_wait_ld8x2(p[0], p[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const float2 f = m ? f1 : f0;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 y = unpack2(x[q][2 * m + j]);
              d[2 * m] = fmaf(y.x, p[q][4 * m + 2 * j], d[2 * m]);
              d[2 * m + 1] = fmaf(y.y, p[q][4 * m + 2 * j + 1], d[2 * m + 1]);
              sum[q][4 * m + 2 * j] = fmaf(f.x, p[q][4 * m + 2 * j], sum[q][4 * m + 2 * j]);
              sum[q][4 * m + 2 * j + 1] = fmaf(f.y, p[q][4 * m + 2 * j + 1], sum[q][4 * m + 2 * j + 1]);
            }
          }
        const float c = over_rows(d, lane);
        if (lane < 16) dot[wq * kC + over_token(16 * quarter, lane)] = c;
      };
      {
        float2 e[2], w[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          e[m] = *reinterpret_cast<const float2*>(&aux.eb[tok0 + 8 * m]);
          w[m] = tc::mul2(*reinterpret_cast<const float2*>(&aux.w[tok0 + 8 * m]), *reinterpret_cast<const float2*>(&aux.beta[tok0 + 8 * m]));
        }
        const float2 s2 = make_float2(P.scale, P.scale), minus = make_float2(-1.f, -1.f);
        part(kColQS, qk, num.dot[0][0], tc::mul2(s2, e[0]), tc::mul2(s2, e[1]), sq);
        part(kColKG, qk + 8192, num.dot[1][0], w[0], w[1], sk);
        part(kColKS, qk + 8192, num.dot[2][0], tc::mul2(minus, e[0]), tc::mul2(minus, e[1]), sk);
      }
      wait(sm.g2, n);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float a[8], b[8];
        tc::tmem_ld16x256x2(tl + (16u * q << 16) + kColQA, a);
        tc::tmem_ld16x256x2(tl + (16u * q << 16) + kColKA, b);
        tc::tmem_wait_ld8x2(a, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sq[q][i] += a[i];
          sk[q][i] += b[i];
        }
      }
      tc::fence_before();
      __syncthreads();
      tc::fence_after();
      if (warp == kThreads / 32 - 1) {
        // the tokens' scalars, two a lane, while the others go on
        float y[2], z[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 2 * lane + e;
          auto dots = [&](int x) { return (num.dot[x][0][t] + num.dot[x][1][t]) + (num.dot[x][2][t] + num.dot[x][3][t]); };
          auto rows = [&](int x) { return (num.rowp[x][0][t] + num.rowp[x][1][t]) + (num.rowp[x][2][t] + num.rowp[x][3][t]); };
          const float eb = aux.eb[t], in = aux.w[t] * dots(1);
          const float column = (num.colp[0][t] + num.colp[1][t]) + (num.colp[2][t] + num.colp[3][t]);
          if (t < nt) G.dbeta[(t0 + t) * P.Hv + h] = __float2bfloat16_rn(column + in);
          y[e] = t < nt ? eb * (P.scale * dots(0) - dots(2)) : 0.f;
          z[e] = t < nt ? aux.beta[t] * (column - num.diag[t] + in) - (rows(0) + rows(1)) : 0.f;
        }
        if (G.dg) {
          float after = y[0] + y[1], before = z[0] + z[1];
#pragma unroll
          for (int k = 1; k < 32; k <<= 1) {
            const float a = __shfl_down_sync(0xffffffffu, after, k), b = __shfl_up_sync(0xffffffffu, before, k);
            if (lane + k < 32) after += a;
            if (lane >= k) before += b;
          }
          before = __shfl_up_sync(0xffffffffu, before, 1);
          if (lane == 0) before = 0.f;
          float gs = 0.f;
#pragma unroll
          for (int k = 0; k < kThreads / 32; ++k) gs += num.gs[k];
          gs *= fast_exp2(aux.whole);
          const int t = 2 * lane;
          if (t < nt) G.dg[(t0 + t) * P.Hv + h] = __float2bfloat16_rn(after + before + gs);
          if (t + 1 < nt) G.dg[(t0 + t + 1) * P.Hv + h] = __float2bfloat16_rn(after - y[0] + before + z[0] + gs);
        }
      }
    }
    // dq and dk over the tiles of Q and K
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t at = block_row(qk, 16 * quarter, 32 * wq + 16 * q, lane);
      tc::stmatrix4_trans(at, pack2(sq[q][0], sq[q][1]), pack2(sq[q][2], sq[q][3]), pack2(sq[q][4], sq[q][5]), pack2(sq[q][6], sq[q][7]));
      tc::stmatrix4_trans(at + 8192, pack2(sk[q][0], sk[q][1]), pack2(sk[q][2], sk[q][3]), pack2(sk[q][4], sk[q][5]), pack2(sk[q][6], sk[q][7]));
    }
    __syncthreads();
    for (int i = tid; i < nt * 32; i += kThreads) {
      const int t = i >> 5, k = i & 15;
      __nv_bfloat16* dst = (i & 16 ? G.dk : G.dq) + ((t0 + t) * P.Hqk + hq) * kDim + 8 * k;
      *reinterpret_cast<uint4*>(dst) =
          *reinterpret_cast<const uint4*>(sm.qk[un & 1] + (k >> 3) * 16384 + (i & 16 ? 8192 : 0) + t * 128 + (((k & 7) ^ (t & 7)) << 4));
    }
    tc::fence_async_smem();  // (read before the next but one unit's copies)
  }
  if (tid == 0) tc::cp_async_wait_all();
  if (!ok) {  // flag it, and let the copies land before the memory is given back
    if (lane == 0) atomicOr(P.status, 1);
    for (uint32_t k = 0; k < 2; ++k) {
      tc::mbar_wait_lanes(bar(sm.full), k, 1u << 14);
      tc::mbar_wait_lanes(bar(sm.fullqk[0]), k, 1u << 14);
      tc::mbar_wait_lanes(bar(sm.fullqk[1]), k, 1u << 14);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after();
    tc::tmem_dealloc(tbase, 512);
  }
}

}  // namespace

cudaError_t launch_delta_grads(const DeltaProblem& P, const DeltaGrads& g, void* ws, cudaStream_t s) {
  Maps maps{};
  cudaError_t e;
  if ((e = token_map(&maps.q, P.q, P.Hqk, P.Ttot, P.qh, P.qt, kC)) != cudaSuccess) return e;
  if ((e = token_map(&maps.k, P.k, P.Hqk, P.Ttot, P.kh, P.kt, kC)) != cudaSuccess) return e;
  if ((e = token_map(&maps.d_o, g.d_o, P.Hv, P.Ttot, kDim, (int64_t)P.Hv * kDim, kC)) != cudaSuccess) return e;
  if ((e = token_map(&maps.dv, g.dv, P.Hv, P.Ttot, kDim, (int64_t)P.Hv * kDim, kC)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(kda_delta_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes)) != cudaSuccess) return e;
  const DeltaWs w = delta_workspace(P, true);
  unsigned char* b = reinterpret_cast<unsigned char*>(ws);
  const int64_t units = P.slots * P.Hqk;
  kda_delta_grad_kernel<<<(unsigned)(units < kSms ? units : kSms), kThreads, kSmemBytes, s>>>(maps, P, b + w.packet, b + w.states, b + w.adjoints, b + w.u, reinterpret_cast<const int2*>(b + w.chunks), g);
  return cudaGetLastError();
}

}  // namespace kda
