// kda_delta_prep.cu -- what a chunk of the gated delta rule has of its own, for all chunks side by side: the factors of its
// decays, P and T = (1 + A)^-1 (kda_delta.cuh).
//
// CTAs of four warps, six an SM, go through the (chunk, head) pairs: scores [K; Q] K^T (M = 128, N = 64) on the tensor cores
// (tcgen05), once for heads that share them, then A (two warps) and P (the others) element by element, a row a thread. T comes
// from A's 16 x 16 blocks, by forward substitution in FP32 (a column a thread; powers of A would lose everything where keys are
// alike), joined to 32 x 32 and then 64 x 64 by T21 = -T22 (A21 T11): products of operands in two parts within a warp (mma.sync: a
// warp's first product comes out as the second's operand lies, so nothing is exchanged; a tcgen05 product of 16 or 32 rows would
// use a quarter of its lanes and take a round trip through tensor memory).
// Bound: memory where each head has its own keys (8 x 1024 tokens of 96 heads: 713 MB in 125 us, 5.7 TB/s; the pass reads what is
// written here, 26 KiB a chunk and head), issue slots (51 %) and the turn's chain where eight share them (24
// sequences, 8 / 64 heads: 289 us, of 46,000 pairs; 499 us with a CTA a pair, each with its own scores, where the loads of the
// decays took 5000 cycles behind all the tiles on their way and the search for the chunk 2000).
// Made inside the pass that uses them, a chunk ahead of it, T and P cost no traffic, but their chain of some 900 instructions a
// warp takes longer than a chunk's pass (7000 cycles against 4470), and 91 KiB of code of seven kinds of warps does not stay in the
// instruction cache: 8 x 1024 tokens of 96 heads 378 us so.
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

// A chunk's numbers, of two chunks in turn.
struct alignas(16) Numbers {       // (read 16 bytes at a time, and copied out)
  DeltaAux aux;
  // Where factors e^{-b_j} stay in range: with beta_j and without; else the tokens' decays, and nothing.
  float f[2][kC];
  bool range;
};
struct Next {
  int slot, t0;
  int h, nt;                      // nt 0: no more
  uint32_t left, unit;            // heads of the unit that come after; the unit after it
  bool first;                     // its scores are not there yet
};
// (Six CTAs an SM: T holds what makes it where it is empty so far. A21's parts lie in its upper right quarter, and A's blocks
// on the diagonal, FP32 and transposed, in the lower left one: those of a warp's 16 rows in 16 rows of T's high or low part.)
struct Smem {
  union {
    unsigned char kq[32768];      // [2 panels][64 rows of K, 64 of Q][64]
    struct {
      unsigned char T[2][8192];   // high, low part
      unsigned char P[2][8192];
    } o;
  };
  Numbers num[2];
  Next next[4];                   // of four chunks in turn
  unsigned long long full, done;
  float growth[2];                // of the rows of each of two warps: sum of max(0, log2 |1 - beta_i k_i . k_i|)
  uint32_t tmem;
};
constexpr int kSmemBytes = (int)sizeof(Smem) + 1024, kCtas = 6;
static_assert(offsetof(Smem, num) % 16 == 0 && sizeof(Numbers) % 16 == 0 && sizeof(DeltaAux) % 16 == 0 && offsetof(Numbers, f) % 16 == 0, "aligned copies");
static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of an SM");

// 2^x, half a step off where it is near 1: products of up to 63 of them are taken.
__device__ __forceinline__ float token_decay(float x) {
  return fabsf(x) < 0.5f ? 1.f + expm1f(x * 0.6931471805599453f) : fast_exp2(x);
}

// x = y where i == j (in C++ it becomes an indexed read of y's array, through local memory: 439 us instead of 130).
__device__ __forceinline__ void take_if(float& x, int i, int j, float y) {
  asm("{\n .reg .pred p;\n setp.eq.s32 p, %1, %2;\n @p mov.f32 %0, %3;\n}\n" : "+f"(x) : "r"(i), "r"(j), "f"(y));
}

// acc += A B for a 16 x 8 tile over 16 inner values, BF16 operands each in two parts (low x low left out: 2^-16 of a product at most).
__device__ __forceinline__ void mma_split(float* c, const uint32_t* ah, const uint32_t* al, const uint32_t* bh, const uint32_t* bl) {
  tc::mma_sync(c, ah, bl);
  tc::mma_sync(c, al, bh);
  tc::mma_sync(c, ah, bh);
}
// Byte of (row, 16-byte piece) in a tile of 128-byte rows, swizzled.
__device__ __forceinline__ uint32_t piece(int row, int c) { return row * 128 + ((c ^ (row & 7)) << 4); }

// kTrain: P's low part too.
template <bool kTrain>
__global__ void __launch_bounds__(128, kCtas) kda_delta_prep_kernel(const __grid_constant__ Maps maps, const DeltaProblem P, const int group,
                                                                    unsigned char* packets, int2* chunks) {
  extern __shared__ unsigned char raw_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem + ((1024 - (tc::smem_u32(raw_smem) & 1023)) & 1023));
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const uint32_t full = tc::smem_u32(&sm.full), done = tc::smem_u32(&sm.done);
  if (w == 1) tc::tmem_alloc(tc::smem_u32(&sm.tmem), 64);
  if (tid == 0) {
    tc::mbar_init(full, 1);
    tc::mbar_init(done, 1);
  }
  // What comes next but one (warp 3): looks for it and brings its numbers to the cache ... (What is known from turn to turn is in
  // shared memory: registers would be spilled, and wait for that.)
  auto advance = [&](const Next& now, Next& to) {
    int slot = now.slot, t0 = now.t0, h = now.h + 1, nt = now.nt;
    uint32_t left = now.left - 1, unit = now.unit;
    const bool first = now.left == 0;
    if (first) {
      const uint32_t groups = (uint32_t)(P.Hv / group), units = (uint32_t)P.slots * groups;
      for (nt = 0; unit < units && nt <= 0; unit += gridDim.x) {
        slot = (int)(unit / groups);
        const DeltaChunk ch = delta_chunk(P, slot);
        t0 = (int)ch.t0;
        nt = ch.nt;
        h = (int)(unit - (uint32_t)slot * groups) * group;
        if (kTrain && h == 0 && lane == 0) chunks[slot] = make_int2(t0, nt);
      }
      left = group - 1;
    }
    __syncwarp();
    if (lane == 0) to = Next{slot, t0, h, nt, left, unit, first};
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (lane + 32 * q < nt) {
        const int64_t at = (int64_t)(t0 + lane + 32 * q) * P.Hv + h;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(P.beta + at));
        if (P.g) asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const __nv_bfloat16*>(P.g) + at));
      }
  };
  // ... and, a turn later, warp 2 asks for them, two tokens a lane, before it waits for the scores (behind all the tiles that are on
  // their way this can take 5000 cycles; a load to a register is waited for at the next loop) ...
  // (A number in the upper half of a word comes with the two bytes before it, the tensor's own or not: in the same word, so
  // they can be read, and are not looked at.)
  auto ask = [&](const Next& of, Numbers& num) {  // to f: the 4-byte words that they are in
    const int64_t at = (int64_t)(of.t0 + 2 * lane) * P.Hv + of.h;
    auto copy = [](float* to, const void* p) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(p);
      tc::cp_async_small<4>(to, reinterpret_cast<const void*>(a & ~(uintptr_t)3), a & 2 ? 4u : 2u);
    };
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (2 * lane + q < of.nt) {
        copy(&num.f[0][2 * lane + q], P.beta + at + q * P.Hv);
        if (P.g) copy(&num.f[1][2 * lane + q], reinterpret_cast<const __nv_bfloat16*>(P.g) + at + q * P.Hv);
      }
    tc::cp_async_commit();
  };
  // ... and works them out.
  auto numbers = [&](const Next& of, Numbers& num) {
    tc::cp_async_wait_all();
    if (of.nt <= 0) return;
    const int64_t at = (int64_t)(of.t0 + 2 * lane) * P.Hv + of.h;
    auto value = [](float word, const void* p) {
      const uint32_t x = __float_as_uint(word);
      return __uint_as_float(reinterpret_cast<uintptr_t>(p) & 2 ? x & 0xffff0000u : x << 16);
    };
    // The sums are exact in 64-bit fixed point (units of 2^-40): factors are of differences of sums that can be thousands of
    // times larger.
    float x[2] = {0.f, 0.f}, beta[2] = {0.f, 0.f};
    bool bad = false;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (2 * lane + q < of.nt) {
        beta[q] = value(num.f[0][2 * lane + q], P.beta + at + q * P.Hv);
        if (P.g) x[q] = decay_log2(value(num.f[1][2 * lane + q], reinterpret_cast<const __nv_bfloat16*>(P.g) + at + q * P.Hv));
      }
      if (!(x[q] < 1048576.f)) { bad = true; x[q] = 0.f; }  // NaN or infinite: so is the chunk
    }
    bad = __any_sync(0xffffffffu, bad);
    const long long f1 = __float2ll_rn(x[1] * 1099511627776.f);
    long long sum = __float2ll_rn(x[0] * 1099511627776.f) + f1;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, k);
      if (lane >= k) sum += y;
    }
    const long long whole = __shfl_sync(0xffffffffu, sum, 31);
    const float nan = bad ? __int_as_float(0x7fc00000) : 0.f;
    auto number = [&](long long y) { return (float)y * 9.094947017729282e-13f + nan; };
    auto two = [&](float* to, float y0, float y1) { *reinterpret_cast<float2*>(to + 2 * lane) = make_float2(y0, y1); };
    const float b0 = number(sum - f1), b1 = number(sum), bC = number(whole);
    two(num.aux.eb, fast_exp2(b0), fast_exp2(b1));
    two(num.aux.w, fast_exp2(number(whole - sum + f1)), fast_exp2(number(whole - sum)));
    two(num.aux.beta, beta[0], beta[1]);
    two(num.aux.b, b0, b1);
    // (decays to 2^-100 over the chunk)
    const bool range = bC > -100.f && of.nt == kC;
    const float y0 = range ? fast_exp2(-b0) : token_decay(x[0]) + nan, y1 = range ? fast_exp2(-b1) : token_decay(x[1]) + nan;
    two(num.f[0], range ? y0 * beta[0] : y0, range ? y1 * beta[1] : y1);
    two(num.f[1], y0, y1);
    if (lane == 0) {
      num.aux.whole = bC;
      num.range = range;
    }
  };
  auto load = [&](const Next& x) {  // by one thread
    tc::mbar_arrive_expect_tx(full, 32768);
    const uint32_t kq = tc::smem_u32(sm.kq);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      tc::tma_load3(kq + p * 16384, &maps.k, 64 * p, x.h / P.r, (int)x.t0, full);
      tc::tma_load3(kq + p * 16384 + 8192, &maps.q, 64 * p, x.h / P.r, (int)x.t0, full);
    }
  };
  if (tid == 64) sm.next[3] = Next{0, 0, 0, 1, 0u, blockIdx.x, false};
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (w == 3)
#pragma unroll 1
    for (int k = 0; k < 2; ++k)
      if (sm.next[(k + 3) & 3].nt > 0) advance(sm.next[(k + 3) & 3], sm.next[k]);
  __syncthreads();
  if (w == 2) {
    ask(sm.next[0], sm.num[0]);
    numbers(sm.next[0], sm.num[0]);
  }
  __syncthreads();
  if (tid == 0 && sm.next[0].nt > 0) load(sm.next[0]);
  bool ok = true;
  // n's low bits count turns, its highest one the scores (a register less)
  for (uint32_t n = 0; sm.next[n & 3].nt > 0; ++n) {
    const Next& cur = sm.next[n & 3];
    Numbers& num = sm.num[n & 1];
    const int nt = cur.nt;
    if (w == 2) ask(sm.next[(n + 1) & 3], sm.num[(n + 1) & 1]);
    if (cur.first) {
      if (w == 1) {
        if (ok) ok = tc::mbar_wait_lanes(full, n >> 31);
        if (ok && tc::elect_one()) {
          const uint64_t d = tc::kmajor(tc::smem_u32(sm.kq));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t off = (i >> 2) * (16384 >> 4) + (i & 3) * 2;
            tc::mma_bf16_ss(sm.tmem, d + off, d + off, tc::idesc_bf16(128, 64, false, false), i > 0);
          }
          tc::mma_commit(done);
        }
        __syncwarp();
      }
      if (ok) ok = tc::mbar_wait_lanes(done, n >> 31);
      n ^= 1u << 31;
      tc::fence_after();
    }
    const int hw = w & 1, i = 32 * hw + lane;  // this thread's row, of K K^T (w < 2) or Q K^T
    const bool keys = w < 2;
    const uint32_t tl = sm.tmem + ((uint32_t)(32 * w) << 16);
    unsigned char* T = sm.o.T[0];
    unsigned char* mine = keys ? T : sm.o.P[0];
    // D_ij = e^{b_i} e^{-b_j} where both stay in range (decays to 2^-100 over the chunk); else, sixteen columns at a time from the
    // last, D_ij = D_i,j+1 a_j+1 from D_ii = 1.
    const bool range = num.range;
    const float bi = num.aux.eb[i];
    float d = 0.f, a1 = 0.f;
    float own = 0.f;  // beta_i k_i . k_i
#pragma unroll 1
    for (int m = 2 * hw + 1; m >= 0; --m) {
      float r[16];
      tc::tmem_ld16(tl + 16 * m, r);
      const int last = i < nt ? i - 16 * m - (keys ? 1 : 0) : -1;  // the columns up to it count
      if (range) {
        const float4* f = reinterpret_cast<const float4*>(&num.f[keys ? 0 : 1][16 * m]);
        const float2 b2 = make_float2(bi, bi);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 y = f[q];
          const float2 lo = tc::mul2(make_float2(r[4 * q], r[4 * q + 1]), tc::mul2(make_float2(y.x, y.y), b2));
          const float2 hi = tc::mul2(make_float2(r[4 * q + 2], r[4 * q + 3]), tc::mul2(make_float2(y.z, y.w), b2));
          r[4 * q] = lo.x; r[4 * q + 1] = lo.y; r[4 * q + 2] = hi.x; r[4 * q + 3] = hi.y;
        }
        if (P.seg && keys && (i >> 4) == m)
#pragma unroll
          for (int j = 0; j < 16; ++j) take_if(own, j, last + 1, r[j]);
        if (m >= 2 * hw)  // (the other half lies before all of its rows)
#pragma unroll
          for (int j = 0; j < 16; ++j) r[j] = j <= last ? r[j] : 0.f;
      } else {
#pragma unroll
        for (int q = 3; q >= 0; --q) {
          const float4 a4 = *reinterpret_cast<const float4*>(&num.f[0][16 * m + 4 * q]);
          const float4 b4 = keys ? *reinterpret_cast<const float4*>(&num.aux.beta[16 * m + 4 * q]) : make_float4(1.f, 1.f, 1.f, 1.f);
          const float av[4] = {a4.x, a4.y, a4.z, a4.w}, bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
          for (int e = 3; e >= 0; --e) {
            const int j = 4 * q + e;
            d = 16 * m + j == i ? 1.f : d * a1;
            a1 = av[e];
            // (selected, not multiplied: rows past the end may hold anything)
            r[j] *= bv[e] * d;
            take_if(own, 16 * m + j, i, r[j]);
            r[j] = j <= last ? r[j] : 0.f;
          }
        }
      }
      if (keys && (i >> 4) == m) {
#pragma unroll
        for (int j = 0; j < 16; ++j) *reinterpret_cast<float*>(T + 8192 * w + piece(32 + 16 * (m & 1) + j, (lane & 15) >> 2) + 4 * (lane & 3)) = r[j];
      } else {  // (above the diagonal: zeros)
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split2(make_float2(r[2 * e], r[2 * e + 1]), hi[e], lo[e]);
        const bool cross = keys && m < 2 * hw;  // a part of A21
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t at = piece(cross ? lane : i, 2 * m + q + (cross ? 4 : 0));
          *reinterpret_cast<uint4*>(mine + at) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
          if (keys || kTrain) *reinterpret_cast<uint4*>(mine + 8192 + at) = make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
        }
      }
    }
    if (!keys && !hw)
#pragma unroll
      for (int q = 4; q < 8; ++q) {
        *reinterpret_cast<uint4*>(mine + piece(i, q)) = make_uint4(0u, 0u, 0u, 0u);
        if (kTrain) *reinterpret_cast<uint4*>(mine + 8192 + piece(i, q)) = make_uint4(0u, 0u, 0u, 0u);
      }
    const uint32_t Ts = tc::smem_u32(T);
    const int r8 = lane & 7, q1 = (lane >> 3) & 1, q2 = lane >> 4;  // row and place of the 8 x 8 matrix whose address this lane gives
    if (keys) {
      if (P.seg) {  // (a little more, for the factors' roundings; NaN stays)
        float grown = i < nt ? __log2f(fabsf(1.f - own)) : 0.f;
        grown = grown < 0.f ? 1e-4f : grown + 1e-4f;
#pragma unroll
        for (int k = 16; k; k >>= 1) grown += __shfl_xor_sync(0xffffffffu, grown, k);
        if (lane == 0) sm.growth[w] = grown;
      }
      // the blocks on the diagonal, a column a thread: t_l -= A_lj t_j for l > j once t_j is known
      __syncwarp();
      const int blk = lane >> 4, col = lane & 15;
      float2 t[8];
#pragma unroll
      for (int l = 0; l < 8; ++l) t[l] = make_float2(2 * l == col ? 1.f : 0.f, 2 * l + 1 == col ? 1.f : 0.f);
#pragma unroll
      for (int j = 0; j < 15; ++j) {
        const float tj = -((j & 1) ? t[j / 2].y : t[j / 2].x);
#pragma unroll
        for (int l = (j + 1) / 4; l < 4; ++l) {  // rows 4 l .. 4 l + 3 (A is zero on the diagonal and above)
          const float4 y = *reinterpret_cast<const float4*>(T + 8192 * w + piece(32 + 16 * blk + j, l));
          if (4 * l + 1 > j) t[2 * l] = tc::fma2(make_float2(y.x, y.y), make_float2(tj, tj), t[2 * l]);
          t[2 * l + 1] = tc::fma2(make_float2(y.z, y.w), make_float2(tj, tj), t[2 * l + 1]);
        }
      }
#pragma unroll
      for (int l = 0; l < 8; ++l) {
        uint32_t th, tlo;
        split2(t[l], th, tlo);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t to = piece(32 * w + 16 * blk + 2 * l + e, i >> 3) + 2 * (i & 7);
          *reinterpret_cast<uint16_t*>(T + to) = (uint16_t)(e ? th >> 16 : th & 0xffffu);
          *reinterpret_cast<uint16_t*>(T + 8192 + to) = (uint16_t)(e ? tlo >> 16 : tlo & 0xffffu);
        }
      }
      __syncwarp();
      // joined: Y^T = T00^T A10^T (as its operands lie, Y is the next product's operand), T10 = -T11 Y
      uint32_t ah[4], al[4], bh[4], bl[4];
      const uint32_t t00 = Ts + piece(32 * w + 8 * q2 + r8, 4 * w + q1), a10 = Ts + piece(32 * w + 16 + 8 * q2 + r8, 4 * w + q1);
      const uint32_t t11 = Ts + piece(32 * w + 16 + 8 * q1 + r8, 4 * w + 2 + q2);
      tc::ldmatrix4_trans(t00, ah);
      tc::ldmatrix4_trans(t00 + 8192, al);
      tc::ldmatrix4(a10, bh);
      tc::ldmatrix4(a10 + 8192, bl);
      float y[2][4] = {};
      mma_split(y[0], ah, al, bh, bl);
      mma_split(y[1], ah, al, bh + 2, bl + 2);
      tc::ldmatrix4(t11, ah);
      tc::ldmatrix4(t11 + 8192, al);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        split2(make_float2(y[0][2 * n], y[0][2 * n + 1]), bh[0], bl[0]);
        split2(make_float2(y[1][2 * n], y[1][2 * n + 1]), bh[1], bl[1]);
        float z[4] = {};
        mma_split(z, ah, al, bh, bl);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t th, tlo;
          split2(make_float2(-z[2 * k], -z[2 * k + 1]), th, tlo);
          const uint32_t to = piece(32 * w + 16 + 8 * k + (lane >> 2), 4 * w + n) + 4 * (lane & 3);
          *reinterpret_cast<uint32_t*>(T + to) = th;
          *reinterpret_cast<uint32_t*>(T + 8192 + to) = tlo;
        }
      }
    } else if (w == 2) {
      numbers(sm.next[(n + 1) & 3], sm.num[(n + 1) & 1]);
    } else if (sm.next[(n + 1) & 3].nt > 0) {
      advance(sm.next[(n + 1) & 3], sm.next[(n + 2) & 3]);
    }
    __syncthreads();
    {
      // columns 16 hw .. of T21, as above over 32 inner values, by two warps
      uint32_t bh[2][4], bl[2][4];  // [8 columns][inner values in steps of 8]
      if (!keys) {
        float y[4][4] = {};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t ah[4], al[4];
          const uint32_t t11 = Ts + piece(16 * k + 8 * q2 + r8, 2 * hw + q1);
          tc::ldmatrix4_trans(t11, ah);
          tc::ldmatrix4_trans(t11 + 8192, al);
#pragma unroll
          for (int n = 0; n < 4; n += 2) {
            uint32_t ch[4], cl[4];
            const uint32_t a21 = Ts + piece(8 * n + 8 * q2 + r8, 4 + 2 * k + q1);
            tc::ldmatrix4(a21, ch);
            tc::ldmatrix4(a21 + 8192, cl);
            mma_split(y[n], ah, al, ch, cl);
            mma_split(y[n + 1], ah, al, ch + 2, cl + 2);
          }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) split2(make_float2(y[k][2 * n], y[k][2 * n + 1]), bh[n][k], bl[n][k]);
      }
      __syncthreads();  // A21 is read
      if (keys) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int x = tid + 64 * k;
          *reinterpret_cast<uint4*>(T + 8192 * (x >> 7) + piece((x >> 2) & 31, 4 + (x & 3))) = make_uint4(0u, 0u, 0u, 0u);
        }
      } else {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float z[2][4] = {};
#pragma unroll
          for (int k = 0; k <= m; ++k) {
            uint32_t ah[4], al[4];
            const uint32_t t22 = Ts + piece(32 + 16 * m + 8 * q1 + r8, 4 + 2 * k + q2);
            tc::ldmatrix4(t22, ah);
            tc::ldmatrix4(t22 + 8192, al);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma_split(z[n], ah, al, bh[n] + 2 * k, bl[n] + 2 * k);
          }
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t th, tlo;
              split2(make_float2(-z[n][2 * k], -z[n][2 * k + 1]), th, tlo);
              const uint32_t to = piece(32 + 16 * m + 8 * k + (lane >> 2), 2 * hw + n) + 4 * (lane & 3);
              *reinterpret_cast<uint32_t*>(T + to) = th;
              *reinterpret_cast<uint32_t*>(T + 8192 + to) = tlo;
            }
        }
      }
    }
    if (tid == 0) num.aux.bound = P.seg ? num.aux.whole + (sm.growth[0] + sm.growth[1]) : 0.f;
    tc::fence_async_smem();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (tid == 0 && ok) {
      unsigned char* dst = packets + ((int64_t)cur.slot * P.Hv + cur.h) * (int64_t)(kTrain ? kPkTrain : kPkInfer);
      tc::bulk_s2g(dst, Ts, kPkAux);
      tc::bulk_s2g(dst + kPkAux, tc::smem_u32(&num.aux), sizeof(DeltaAux));
      if (kTrain) tc::bulk_s2g(dst + kPkPlo, Ts + 24576, 8192);
      tc::bulk_commit();
      tc::bulk_wait_read();
      if (sm.next[(n + 1) & 3].nt > 0 && sm.next[(n + 1) & 3].first) load(sm.next[(n + 1) & 3]);
    }
    __syncthreads();  // the tiles have left
  }
  if (!ok) {  // flag it, and let the copies land before the memory is given back
    if (lane == 0) atomicOr(P.status, 1);
    tc::mbar_wait_lanes(full, 0, 1u << 14);
    tc::mbar_wait_lanes(full, 1, 1u << 14);
  }
  if (w == 1) {
    tc::fence_after();
    tc::tmem_dealloc(sm.tmem, 64);
  }
}

template <bool kTrain>
cudaError_t launch(const Maps& maps, const DeltaProblem& P, void* ws, cudaStream_t s) {
  auto kern = kda_delta_prep_kernel<kTrain>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  // A CTA takes heads that share their queries and keys one after another, so that their scores are made once, as many as leave
  // some eight turns for every CTA.
  const int64_t ctas = kCtas * kSms;
  int group = P.r;
  while (group > 1 && (P.r % group || P.slots * (P.Hv / group) < 8 * ctas)) --group;
  const int64_t units = P.slots * (P.Hv / group);
  kern<<<(unsigned)(units < ctas ? units : ctas), 128, kSmemBytes, s>>>(maps, P, group, reinterpret_cast<unsigned char*>(ws),
                                                                             reinterpret_cast<int2*>(reinterpret_cast<unsigned char*>(ws) + delta_workspace(P, kTrain).chunks));
  return cudaGetLastError();
}

}  // namespace

DeltaWs delta_workspace(const DeltaProblem& P, bool training) {
  const size_t n = (size_t)P.slots * P.Hv;
  DeltaWs w{};
  w.chunks = ctx_align_up(n * (training ? kPkTrain : kPkInfer));
  w.states = w.chunks + (training ? ctx_align_up((size_t)P.slots * sizeof(int2)) : 0);
  w.u = w.states + (training ? n * kStateTile : 0);
  w.adjoints = w.u + (training ? n * kUTile : 0);
  w.segments = w.adjoints + (training ? n * kStateTile : 0);
  const size_t cut = P.seg ? sizeof(float) * (size_t)(P.Ttot / P.seg + P.N) * P.Hv * kDim * kDim : 0;
  w.through = w.segments + cut;
  w.none = w.through + cut;
  w.total = w.none + ctx_align_up(cut / (kDim * kDim));
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
