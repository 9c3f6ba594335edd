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
// q_i . dq_i - v_i . dv_i summed from t on has the same value, but its terms cancel: 1.8e-2 off from operands in BF16, this 2e-3.)
#include "kda_delta.cuh"
#include "kda_layout.h"
#include "kda_tma.h"
#include "tc.cuh"

namespace kda {
namespace {

constexpr int kC = kDecayChunk;
constexpr int kThreads = 256;
// Tensor memory, columns (64 each)
constexpr uint32_t kColUU = 0;     // [dO; rho] u^T
constexpr uint32_t kColKK = 64;    // [Q; K] K^T
constexpr uint32_t kColQS = 128;   // S^T dO^T
constexpr uint32_t kColKG = 192;   // G^T u^T
constexpr uint32_t kColKS = 256;   // S^T rho^T
constexpr uint32_t kColQA = 320;   // K^T A^T
constexpr uint32_t kColKA = 384;   // Q^T A - K^T (R + R^T)

struct Maps {
  CUtensorMap q, k, d_o, dv;
};

struct Smem {
  unsigned char S[kStateTile], G[kStateTile];
  unsigned char qk[32768];    // [2 panels][64 rows of Q, 64 of K][64]
  unsigned char dr[32768];    // the same of dO and rho; at last dq and dk on their way out
  unsigned char u[kUTile];
  unsigned char A[8192], R[8192];
  DeltaAux aux;
  float rowp[2][2][kC];       // rows of E beta and F beta before the diagonal, [half][i]
  float colp[4][kC];          // columns of E (two row halves), F (two)
  float diag[kC];             // E_ii
  float dot[3][4][kC];        // q . S^T dO, k . G^T u, k . S^T rho, by lane quadrant
  float gs[8];                // <G, S> of each warp
  unsigned long long fullqk, full, g1, g2;
  uint32_t tmem;
};
constexpr int kSmemBytes = (int)sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

__device__ __forceinline__ void load_block(uint32_t tile, int token, int value, int lane, uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const int t = token + 8 * (i + (lane >> 4)) + (lane & 7), d = value + 8 * ((lane >> 3) & 1);
    tc::ldmatrix4_trans(tile + (d >> 6) * 16384 + t * 128 + ((((d & 63) >> 3) ^ (t & 7)) << 4), r + 2 * i);
  }
}
__device__ __forceinline__ void store_block(uint32_t tile, int token, int value, int lane, const uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const int t = token + 8 * (i + (lane >> 4)) + (lane & 7), d = value + 8 * ((lane >> 3) & 1);
    tc::stmatrix4_trans(tile + (d >> 6) * 16384 + t * 128 + ((((d & 63) >> 3) ^ (t & 7)) << 4), r[2 * i], r[2 * i + 1],
                        r[2 * i + 2], r[2 * i + 3]);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
kda_delta_grad_kernel(const __grid_constant__ Maps maps, const DeltaProblem P, const unsigned char* packets, const unsigned char* states,
                      const unsigned char* adjoints, const unsigned char* us, const DeltaGrads G) {
  extern __shared__ unsigned char raw_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem + ((1024 - (tc::smem_u32(raw_smem) & 1023)) & 1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wq = warp & 3, half = warp >> 2;
  const int64_t slot = blockIdx.x / P.Hqk;
  const int hq = (int)(blockIdx.x - slot * P.Hqk);
  const DeltaChunk ch = delta_chunk(P, slot);
  if (ch.nt <= 0) return;  // a place without a chunk
  const int64_t t0 = ch.t0;
  const int nt = ch.nt;
  auto bar = [](unsigned long long& b) { return tc::smem_u32(&b); };
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&sm.tmem), 512);
  if (tid == 0)
    for (unsigned long long* b : {&sm.fullqk, &sm.full, &sm.g1, &sm.g2}) tc::mbar_init(bar(*b), 1);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = sm.tmem, tl = tbase + ((uint32_t)(32 * wq) << 16);
  const uint32_t qk = tc::smem_u32(sm.qk), dr = tc::smem_u32(sm.dr);
  bool ok = true;
  auto wait = [&](unsigned long long& b, uint32_t parity) {
    if (ok) ok = tc::mbar_wait_lanes(bar(b), parity);
    tc::fence_after();
  };
  if (tid == 0) {
    tc::mbar_arrive_expect_tx(bar(sm.fullqk), 32768);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      tc::tma_load3(qk + p * 16384, &maps.q, 64 * p, hq, (int)t0, bar(sm.fullqk));
      tc::tma_load3(qk + p * 16384 + 8192, &maps.k, 64 * p, hq, (int)t0, bar(sm.fullqk));
    }
  }
  float sq[2][16], sk[2][16];  // dq, dk: values 32 wq + 16 q + 8 j + lane / 4, tokens 32 half + 8 i + 2 (lane % 4) (+ 1)
#pragma unroll
  for (int i = 0; i < 32; ++i) sq[i >> 4][i & 15] = sk[i >> 4][i & 15] = 0.f;
  const int tok0 = 32 * half + 2 * (lane & 3);
  for (int r = 0; r < P.r; ++r) {
    const int h = hq * P.r + r;
    const uint32_t par = r & 1;
    const int64_t place = slot * P.Hv + h;
    if (tid == 0) {
      tc::mbar_arrive_expect_tx(bar(sm.full), 2 * kStateTile + 32768 + kUTile + sizeof(DeltaAux));
      tc::bulk_g2s(tc::smem_u32(sm.S), states + place * kStateTile, kStateTile, bar(sm.full));
      tc::bulk_g2s(tc::smem_u32(sm.G), adjoints + place * kStateTile, kStateTile, bar(sm.full));
      tc::bulk_g2s(tc::smem_u32(sm.u), us + place * kUTile, kUTile, bar(sm.full));
      tc::bulk_g2s(tc::smem_u32(&sm.aux), packets + place * kPkTrain + kPkAux, sizeof(DeltaAux), bar(sm.full));
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        tc::tma_load3(dr + p * 16384, &maps.d_o, 64 * p, h, (int)t0, bar(sm.full));
        tc::tma_load3(dr + p * 16384 + 8192, &maps.dv, 64 * p, h, (int)t0, bar(sm.full));
      }
    }
    if (r == 0) wait(sm.fullqk, 0);
    wait(sm.full, par);
    if (nt < kC) {  // rows past the end hold other tokens
      for (int i = tid; i < (kC - nt) * 64; i += kThreads) {
        const int row = nt + (i >> 6), x = i & 63;  // 16-byte pieces of a row: 16 of dO, rho, Q, K
        unsigned char* t = (x & 32 ? sm.qk : sm.dr) + ((x >> 3) & 1) * 16384 + ((x >> 4) & 1) * 8192;
        if (r == 0 || !(x & 32)) *reinterpret_cast<uint4*>(t + row * 128 + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      tc::fence_async_smem();
      __syncthreads();
    }
    if (warp == 0 && ok && tc::elect_one()) {
      const uint64_t un = tc::kmajor(tc::smem_u32(sm.u)), St = tc::mnmajor(tc::smem_u32(sm.S), 16384), Gt = tc::mnmajor(tc::smem_u32(sm.G), 16384);
      constexpr uint32_t kn = tc::idesc_bf16(128, 64, false, false), tn = tc::idesc_bf16(128, 64, true, false);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t off = (i >> 2) * (16384 >> 4) + (i & 3) * 2, off64 = (i >> 2) * (8192 >> 4) + (i & 3) * 2;
        tc::mma_bf16_ss(tbase + kColUU, tc::kmajor(dr) + off, un + off64, kn, i > 0);
        if (r == 0) tc::mma_bf16_ss(tbase + kColKK, tc::kmajor(qk) + off, tc::kmajor(qk + 8192) + off, kn, i > 0);
        tc::mma_bf16_ss(tbase + kColQS, St + 128 * i, tc::kmajor(dr) + off, tn, i > 0);
        tc::mma_bf16_ss(tbase + kColKG, Gt + 128 * i, un + off64, tn, i > 0);
        tc::mma_bf16_ss(tbase + kColKS, St + 128 * i, tc::kmajor(dr + 8192) + off, tn, i > 0);
      }
      tc::mma_commit(bar(sm.g1));
    }
    __syncwarp();
    if (G.dg) {  // <G, S>: the tiles are laid out alike
      float x = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 a = reinterpret_cast<const uint4*>(sm.S)[tid + kThreads * j], b = reinterpret_cast<const uint4*>(sm.G)[tid + kThreads * j];
        const float2 y = tc::fma2(unpack2(a.x), unpack2(b.x), tc::fma2(unpack2(a.y), unpack2(b.y), tc::fma2(unpack2(a.z), unpack2(b.z), tc::mul2(unpack2(a.w), unpack2(b.w)))));
        x += y.x + y.y;
      }
#pragma unroll
      for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
      if (lane == 0) sm.gs[warp] = x;
    }
    wait(sm.g1, par);
    // the scores: rows i = 32 (wq % 2) + 16 q + 8 j + lane / 4 of dO and Q (wq < 2) or rho and K, columns tok0 + 8 m + e
    {
      const bool first = wq < 2;
      float col[8];
#pragma unroll
      for (int m = 0; m < 8; ++m) col[m] = 0.f;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float uu[16], kk[16];
        tc::tmem_ld16x256(tl + (16u * q << 16) + kColUU + 32 * half, uu);
        tc::tmem_ld16x256(tl + (16u * q << 16) + kColKK + 32 * half, kk);
        tc::tmem_wait_ld2(uu, kk);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int i = 32 * (wq & 1) + 16 * q + 8 * j + (lane >> 2);
          const float bi = sm.aux.b[i];
          float row = 0.f;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            float z[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int t = tok0 + 8 * m + e;
              const float beta = sm.aux.beta[t], x = uu[4 * m + 2 * j + e];
              const bool in = first ? t <= i : t < i;
              const float d = in ? fast_exp2(bi - sm.aux.b[t]) * (first ? P.scale : 1.f) * x : 0.f;
              z[e] = d * beta;
              const float y = in ? d * kk[4 * m + 2 * j + e] : 0.f;
              col[2 * m + e] += y;
              if (t < i) row = fmaf(y, beta, row);
              if (first && t == i) sm.diag[i] = y;
            }
            const int chunk = 4 * half + m;
            if (first) {
              *reinterpret_cast<uint32_t*>(sm.A + i * 128 + ((chunk ^ (i & 7)) << 4) + 4 * (lane & 3)) = pack2(z[0], z[1]);
            } else {  // -(R + R^T): each element and its mirror
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int t = tok0 + 8 * m + e;
                const __nv_bfloat16 y = __float2bfloat16_rn(-z[e]);
                if (t <= i) *reinterpret_cast<__nv_bfloat16*>(sm.R + i * 128 + (((t >> 3) ^ (i & 7)) << 4) + 2 * (t & 7)) = y;
                if (t < i) *reinterpret_cast<__nv_bfloat16*>(sm.R + t * 128 + (((i >> 3) ^ (t & 7)) << 4) + 2 * (i & 7)) = y;
              }
            }
          }
          row += __shfl_xor_sync(0xffffffffu, row, 1);
          row += __shfl_xor_sync(0xffffffffu, row, 2);
          if ((lane & 3) == 0) sm.rowp[first ? 0 : 1][half][i] = row;
        }
      }
#pragma unroll
      for (int m = 0; m < 8; ++m) {
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) col[m] += __shfl_xor_sync(0xffffffffu, col[m], k);
        if (lane < 4) sm.colp[wq][tok0 + 8 * (m >> 1) + (m & 1)] = col[m];
      }
    }
    tc::fence_async_smem();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0 && ok && tc::elect_one()) {
      const uint64_t Qt = tc::mnmajor(qk, 16384), Kt = tc::mnmajor(qk + 8192, 16384);
      const uint64_t A = tc::kmajor(tc::smem_u32(sm.A)), An = tc::mnmajor(tc::smem_u32(sm.A), 8192), R = tc::kmajor(tc::smem_u32(sm.R));
      constexpr uint32_t tn = tc::idesc_bf16(128, 64, true, false), tt = tc::idesc_bf16(128, 64, true, true);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tc::mma_bf16_ss(tbase + kColQA, Kt + 128 * i, A + 2 * i, tn, i > 0);
        tc::mma_bf16_ss(tbase + kColKA, Qt + 128 * i, An + 128 * i, tt, i > 0);
        tc::mma_bf16_ss(tbase + kColKA, Kt + 128 * i, R + 2 * i, tn, 1);
      }
      tc::mma_commit(bar(sm.g2));
    }
    __syncwarp();
    // products with the states, and their dots with q and k
    auto part = [&](uint32_t col, uint32_t tile, float* dot, auto factor, float (&sum)[2][16]) {
      float d[8];
#pragma unroll
      for (int m = 0; m < 8; ++m) d[m] = 0.f;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float p[16];
        uint32_t x[8];
        tc::tmem_ld16x256(tl + (16u * q << 16) + col + 32 * half, p);
        load_block(tile, 32 * half, 32 * wq + 16 * q, lane, x);
        tc::tmem_wait_ld(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = factor(tok0 + 8 * i);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 y = unpack2(x[2 * i + j]);
            d[2 * i] = fmaf(y.x, p[4 * i + 2 * j], d[2 * i]);
            d[2 * i + 1] = fmaf(y.y, p[4 * i + 2 * j + 1], d[2 * i + 1]);
            sum[q][4 * i + 2 * j] = fmaf(f.x, p[4 * i + 2 * j], sum[q][4 * i + 2 * j]);
            sum[q][4 * i + 2 * j + 1] = fmaf(f.y, p[4 * i + 2 * j + 1], sum[q][4 * i + 2 * j + 1]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < 8; ++m) {
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) d[m] += __shfl_xor_sync(0xffffffffu, d[m], k);
        if (lane < 4) dot[wq * kC + tok0 + 8 * (m >> 1) + (m & 1)] = d[m];
      }
    };
    part(kColQS, qk, sm.dot[0][0], [&](int t) { return make_float2(P.scale * sm.aux.eb[t], P.scale * sm.aux.eb[t + 1]); }, sq);
    part(kColKG, qk + 8192, sm.dot[1][0],
         [&](int t) { return make_float2(sm.aux.w[t] * sm.aux.beta[t], sm.aux.w[t + 1] * sm.aux.beta[t + 1]); }, sk);
    part(kColKS, qk + 8192, sm.dot[2][0], [&](int t) { return make_float2(-sm.aux.eb[t], -sm.aux.eb[t + 1]); }, sk);
    wait(sm.g2, par);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float a[16], b[16];
      tc::tmem_ld16x256(tl + (16u * q << 16) + kColQA + 32 * half, a);
      tc::tmem_ld16x256(tl + (16u * q << 16) + kColKA + 32 * half, b);
      tc::tmem_wait_ld2(a, b);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        sq[q][i] += a[i];
        sk[q][i] += b[i];
      }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) {  // two tokens a lane
      float y[2], z[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = 2 * lane + e;
        auto dots = [&](int x) { return (sm.dot[x][0][t] + sm.dot[x][1][t]) + (sm.dot[x][2][t] + sm.dot[x][3][t]); };
        const float eb = sm.aux.eb[t], in = sm.aux.w[t] * dots(1);
        const float column = (sm.colp[0][t] + sm.colp[1][t]) - (sm.colp[2][t] + sm.colp[3][t]);
        const float row = (sm.rowp[0][0][t] + sm.rowp[0][1][t]) - (sm.rowp[1][0][t] + sm.rowp[1][1][t]);
        if (t < nt) G.dbeta[(t0 + t) * P.Hv + h] = __float2bfloat16_rn(column + in);
        y[e] = t < nt ? eb * (P.scale * dots(0) - dots(2)) : 0.f;
        z[e] = t < nt ? sm.aux.beta[t] * (column - sm.diag[t] + in) - row : 0.f;
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
        for (int k = 0; k < 8; ++k) gs += sm.gs[k];
        gs *= fast_exp2(sm.aux.whole);
        const int t = 2 * lane;
        if (t < nt) G.dg[(t0 + t) * P.Hv + h] = __float2bfloat16_rn(after + before + gs);
        if (t + 1 < nt) G.dg[(t0 + t + 1) * P.Hv + h] = __float2bfloat16_rn(after - y[0] + before + z[0] + gs);
      }
    }
    __syncthreads();  // the tiles and numbers are free
  }
  // dq and dk over the tiles of dO and rho
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = pack2(sq[q][2 * i], sq[q][2 * i + 1]);
    store_block(dr, 32 * half, 32 * wq + 16 * q, lane, z);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = pack2(sk[q][2 * i], sk[q][2 * i + 1]);
    store_block(dr + 8192, 32 * half, 32 * wq + 16 * q, lane, z);
  }
  __syncthreads();
  for (int i = tid; i < nt * 32; i += kThreads) {
    const int t = i >> 5, k = i & 15;
    __nv_bfloat16* dst = (i & 16 ? G.dk : G.dq) + ((t0 + t) * P.Hqk + hq) * kDim + 8 * k;
    *reinterpret_cast<uint4*>(dst) =
        *reinterpret_cast<const uint4*>(sm.dr + (k >> 3) * 16384 + (i & 16 ? 8192 : 0) + t * 128 + (((k & 7) ^ (t & 7)) << 4));
  }
  if (!ok) {  // flag it, and let the copies land before the memory is given back
    if (lane == 0) atomicOr(P.status, 1);
    tc::mbar_wait_lanes(bar(sm.fullqk), 0, 1u << 16);
    tc::mbar_wait_lanes(bar(sm.full), (P.r - 1) & 1, 1u << 16);
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
  const DeltaWs w = delta_workspace(P.slots, P.Hv, true);
  unsigned char* b = reinterpret_cast<unsigned char*>(ws);
  kda_delta_grad_kernel<<<(unsigned)(P.slots * P.Hqk), kThreads, kSmemBytes, s>>>(maps, P, b + w.packet, b + w.states, b + w.adjoints, b + w.u, g);
  return cudaGetLastError();
}

}  // namespace kda
