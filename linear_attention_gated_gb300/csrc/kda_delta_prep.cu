// kda_delta_prep.cu -- what a chunk of the gated delta rule has of its own, for all chunks side by side: the factors of its
// decays, P and T = (1 + A)^-1 (kda_delta.cuh).
#include "kda_delta.cuh"
#include "kda_layout.h"
#include "kda_tma.h"
#include "tc.cuh"

namespace kda {
namespace {

constexpr int kC = kDecayChunk;

struct Maps {
  CUtensorMap q, k;
};

struct Smem {
  unsigned char tile[32768];  // [2 panels][64 rows of K, 64 of Q][64]; then T, its low part, P, its low part
  float At[kC][kC];           // A transposed: At[j][i] = A_ij
  DeltaAux aux;
  unsigned long long full, done;
  uint32_t tmem;
};
constexpr int kSmemBytes = (int)sizeof(Smem) + 1024;

// One CTA a (chunk, head): 64 rows of K and of Q, scores [K; Q] K^T (M = 128, N = 64) on the tensor cores, then A and P
// element by element, and T by forward substitution, a column a thread: t_l -= A_li t_i for l > i once t_i is known, so
// that the products of a step are independent. All in FP32: powers of A (1 - A + A^2 ...) would lose
// everything where keys are alike.
template <bool kTrain>
__global__ void __launch_bounds__(128) kda_delta_prep_kernel(const __grid_constant__ Maps maps, const DeltaProblem P,
                                                             unsigned char* packets) {
  extern __shared__ unsigned char raw_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem + ((1024 - (tc::smem_u32(raw_smem) & 1023)) & 1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t slot = blockIdx.x / P.Hv;
  const int h = (int)(blockIdx.x - slot * P.Hv);
  int64_t lo = 0, hi = P.N;  // the last sequence whose first place is not behind this one
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (delta_slot(decay_span(P, mid).t0, mid) <= slot) lo = mid;
    else hi = mid;
  }
  const DecaySpan sp = decay_span(P, lo);
  const int64_t c = slot - delta_slot(sp.t0, lo);
  if (c < 0 || c * kC >= sp.len) return;  // a place without a chunk
  const int64_t t0 = sp.t0 + c * kC;
  const int nt = (int)(sp.len - c * kC < kC ? sp.len - c * kC : kC);
  const uint32_t full = tc::smem_u32(&sm.full), done = tc::smem_u32(&sm.done);
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&sm.tmem), 64);
  if (tid == 0) {
    tc::mbar_init(full, 1);
    tc::mbar_init(done, 1);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (tid == 0) {
    tc::mbar_arrive_expect_tx(full, 32768);
    const int hq = h / P.r;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      tc::tma_load3(tc::smem_u32(sm.tile) + p * 16384, &maps.k, 64 * p, hq, (int)t0, full);
      tc::tma_load3(tc::smem_u32(sm.tile) + p * 16384 + 8192, &maps.q, 64 * p, hq, (int)t0, full);
    }
  }
  if (warp == 1) {
    // Two tokens a lane. The sums are exact in 64-bit fixed point (units of 2^-40): D_ij is a difference of
    // sums that can be thousands of times larger.
    long long f[2];
    float be[2];
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = 2 * lane + e;
      float x = 0.f;
      be[e] = 0.f;
      if (j < nt) {
        if (P.g) x = decay_log2(__bfloat162float(reinterpret_cast<const __nv_bfloat16*>(P.g)[(t0 + j) * P.Hv + h]));
        be[e] = __bfloat162float(P.beta[(t0 + j) * P.Hv + h]);
      }
      if (!(x < 1048576.f)) { bad = true; x = 0.f; }  // NaN or infinite: so is the chunk
      f[e] = __float2ll_rn(x * 1099511627776.f);
    }
    bad = __any_sync(0xffffffffu, bad);
    long long sum = f[0] + f[1];
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, k);
      if (lane >= k) sum += y;
    }
    const long long whole = __shfl_sync(0xffffffffu, sum, 31);
    const float nan = bad ? __int_as_float(0x7fc00000) : 0.f;
    auto number = [&](long long x) { return (float)x * 9.094947017729282e-13f + nan; };
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = 2 * lane + e;
      const long long b = e ? sum : sum - f[1];
      sm.aux.eb[j] = fast_exp2(number(b));
      sm.aux.w[j] = fast_exp2(number(whole - b));
      sm.aux.beta[j] = be[e];
      sm.aux.bh[j] = (float)(b >> 32) * 0.00390625f + nan;
      sm.aux.bl[j] = (float)(b & 0xffffffffll) * 9.094947017729282e-13f;
    }
    if (lane == 0) sm.aux.whole = number(whole);
  }
  bool ok = tc::mbar_wait_lanes(full, 0);
  if (warp == 0 && ok && tc::elect_one()) {
    const uint64_t d = tc::kmajor(tc::smem_u32(sm.tile));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t off = (i >> 2) * (16384 >> 4) + (i & 3) * 2;
      tc::mma_bf16_ss(sm.tmem, d + off, d + off, tc::idesc_bf16(128, 64, false, false), i > 0);
    }
    tc::mma_commit(done);
  }
  __syncwarp();
  if (ok) ok = tc::mbar_wait_lanes(done, 0);
  tc::fence_after();
  __syncthreads();  // (the decays are there)
  const int i = tid & 63;
  const bool keys = warp < 2;
  const float bh = sm.aux.bh[i], bl = sm.aux.bl[i];
  const uint32_t tl = sm.tmem + ((uint32_t)(32 * warp) << 16);
  unsigned char* out = sm.tile + (keys ? 0 : 16384);
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    float r[16];
    tc::tmem_ld16(tl + 16 * m, r);
    uint32_t ph[8], pl[8];
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float2 y;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = 16 * m + e + x;
        const float d = fast_exp2((bh - sm.aux.bh[j]) + (bl - sm.aux.bl[j])) * (keys ? sm.aux.beta[j] : P.scale);
        // (selected, not multiplied: rows past the end may hold anything)
        const float v = (keys ? j < i : j <= i) && i < nt ? d * r[e + x] : 0.f;
        if (x) y.y = v;
        else y.x = v;
        if (keys) sm.At[j][i] = v;
      }
      if (!keys) split2(y, ph[e / 2], pl[e / 2]);
    }
    if (!keys) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t at = i * 128 + (((2 * m + x) ^ (i & 7)) << 4);
        *reinterpret_cast<uint4*>(out + at) = make_uint4(ph[4 * x], ph[4 * x + 1], ph[4 * x + 2], ph[4 * x + 3]);
        if (kTrain) *reinterpret_cast<uint4*>(out + 8192 + at) = make_uint4(pl[4 * x], pl[4 * x + 1], pl[4 * x + 2], pl[4 * x + 3]);
      }
    }
  }
  if (keys) {
    asm volatile("barrier.cta.sync 1, 64;" ::: "memory");
    float2 t[kC / 2];
#pragma unroll
    for (int l = 0; l < kC / 2; ++l) t[l] = make_float2(2 * l == i ? 1.f : 0.f, 2 * l + 1 == i ? 1.f : 0.f);
#pragma unroll
    for (int j = 0; j < kC - 1; ++j) {
      const float tj = -((j & 1) ? t[j / 2].y : t[j / 2].x);
#pragma unroll
      for (int l = (j + 1) / 4; l < kC / 4; ++l) {  // rows 4 l .. 4 l + 3 (A is zero on the diagonal and above)
        const float4 a = *reinterpret_cast<const float4*>(&sm.At[j][4 * l]);
        if (4 * l + 1 > j) t[2 * l] = tc::fma2(make_float2(a.x, a.y), make_float2(tj, tj), t[2 * l]);
        t[2 * l + 1] = tc::fma2(make_float2(a.z, a.w), make_float2(tj, tj), t[2 * l + 1]);
      }
    }
#pragma unroll
    for (int l = 0; l < kC / 2; ++l) {
      uint32_t th, tl2;
      split2(t[l], th, tl2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 2 * l + e;
        const uint32_t at = row * 128 + (((i >> 3) ^ (row & 7)) << 4) + 2 * (i & 7);
        *reinterpret_cast<uint16_t*>(sm.tile + at) = (uint16_t)(e ? th >> 16 : th & 0xffffu);
        *reinterpret_cast<uint16_t*>(sm.tile + 8192 + at) = (uint16_t)(e ? tl2 >> 16 : tl2 & 0xffffu);
      }
    }
  }
  tc::fence_async_smem();
  tc::fence_before();
  __syncthreads();
  if (tid == 0) {
    unsigned char* dst = packets + (slot * P.Hv + h) * (int64_t)(kTrain ? kPkTrain : kPkInfer);
    const uint32_t src = tc::smem_u32(sm.tile);
    tc::bulk_s2g(dst, src, kPkAux);
    tc::bulk_s2g(dst + kPkAux, tc::smem_u32(&sm.aux), sizeof(DeltaAux));
    if (kTrain) tc::bulk_s2g(dst + kPkPlo, src + 24576, 8192);
    tc::bulk_commit();
    tc::bulk_wait_read();
  }
  if (!ok) {  // flag it, and let the copies land before the memory is given back
    if (lane == 0) atomicOr(P.status, 1);
    tc::mbar_wait_lanes(full, 0, 1u << 16);
  }
  if (warp == 0) {
    tc::fence_after();
    tc::tmem_dealloc(sm.tmem, 64);
  }
}

template <bool kTrain>
cudaError_t launch(const Maps& maps, const DeltaProblem& P, void* ws, cudaStream_t s) {
  auto kern = kda_delta_prep_kernel<kTrain>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(P.slots * P.Hv), 128, kSmemBytes, s>>>(maps, P, reinterpret_cast<unsigned char*>(ws));
  return cudaGetLastError();
}

}  // namespace

DeltaWs delta_workspace(int64_t slots, int64_t Hv, bool training) {
  const size_t n = (size_t)slots * Hv;
  DeltaWs w{0, 0, 0, 0, 0};
  w.states = ctx_align_up(n * (training ? kPkTrain : kPkInfer));
  w.u = w.states + (training ? n * kStateTile : 0);
  w.adjoints = w.u + (training ? n * kUTile : 0);
  w.total = w.adjoints + (training ? n * kStateTile : 0);
  return w;
}

cudaError_t launch_delta_prep(const DeltaProblem& P, bool training, void* ws, cudaStream_t s) {
  if (!P.Ttot) return cudaSuccess;
  Maps maps{};
  cudaError_t e;
  if ((e = token_map(&maps.q, P.q, P.Hqk, P.Ttot, P.qh, P.qt, kC)) != cudaSuccess) return e;
  if ((e = token_map(&maps.k, P.k, P.Hqk, P.Ttot, P.kh, P.kt, kC)) != cudaSuccess) return e;
  return training ? launch<true>(maps, P, ws, s) : launch<false>(maps, P, ws, s);
}

}  // namespace kda
