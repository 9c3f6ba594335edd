// kda_qk_norm_rope.cu -- RMS norm of every query and key head and the rotation
// by position, in one pass, and their gradients.
//
// For a head row x[D] at position p, with weight w and pair (a, b) of the first
// R dimensions ((d, d + R/2), or (2d, 2d + 1) when interleaved):
//   r = 1 / sqrt(mean(x^2) + eps),   n = x r w,
//   y_a = n_a cos(p f_d) - n_b sin(p f_d),   y_b = n_b cos(p f_d) + n_a sin(p f_d)
// and the dimensions from R on pass through as n. Backward, dn = R(p)^T dy:
//   dw = sum over rows of dn x r,   dx = r (dn w - x r mean(dn w x r)).
//
// Memory bound: 10 to 20 flops per value moved. A row belongs to a group of
// G = 4, 8 or 16 lanes (the power of two at or above D / 16); each lane holds
// the two 8-value vectors whose elements rotate into each other, so the rotation
// needs no exchange and the norm log2(G) shuffles. A CTA takes an even run of one
// tensor's rows (queries or keys), keeps that tensor's weight in registers and
// computes the cosines and sines of a token once for all its heads in the run.
// Rows come by asynchronous 16-byte copies into a ring of 4 (backward 3) rows a
// group, each lane copying what it reads itself, so no barrier is needed.
//
// Measured: forward, 8191 tokens of 64 + 8 BF16 heads, 302 MB: 62 us, 4.9 TB/s,
// 73 % of the copy rate (57 us for the kernel alone); backward, 8192 tokens of
// 16 + 16 heads, 201 MB: 40 us, 5.0 TB/s, 75 % (the weights' last sum takes 5).
// Issue slots bound it next: 56 % of them busy, 229 instructions a warp for four
// rows of 128, and the waits of a row's chain (norm, then rotation). Earlier forms
// of the forward: the next row's loads into registers and tiles of whole tokens
// 69 us; that with 4 CTAs of 256 threads or 8 of 128 an SM (spills) 79; the ring,
// CTAs shared out by rows without the angles' cost, 65.
//
// Angles: p f is reduced modulo one turn in 64-bit fixed point, f / 2 pi scaled
// by 2^64 and multiplied by p with wrap-around, so a far position loses nothing
// (error p 2^-53 f turns); sincospif then sees half-turns in [-1, 1).
#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_host.h"
#include "tc.cuh"

#include <cuda_fp16.h>

#include <cmath>
#include <cstdio>

namespace kda {
namespace {

constexpr int kNrThreads = 128;

struct NrTensor {
  const void* x;
  const void* dy;   // backward
  void* y;          // forward: y; backward: dx
  const float* w;   // [D] or null
  int64_t xt, xh, dt, dh, yt, yh;  // token and head strides of x, dy and y (elements)
  int64_t x_step, x_wrap, d_step, d_wrap, y_step, y_wrap;  // from row to row of a group; more where the head wraps round
  int H;
  int rounds;       // for which angles are computed at a time
};

struct NrArgs {
  NrTensor t[2];         // queries, keys
  const int64_t* pos;    // [n]
  const double* freq;    // [R / 2]
  float* dw_part;        // backward: [CTAs, D], the queries' CTAs first
  int64_t n;
  int D, R;
  float eps;
  int ctas0;             // CTAs of the queries
  int tokens;            // most tokens whose angles are there
};

// 8 values of a row: raw as they come from memory, and as four FP32 pairs.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load_ring(const uint4* at) { r = *at; }
  __device__ __forceinline__ void get(float2* x) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(void* p, const float2* x) {
    uint4 v;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[i].x, x[i].y);
    *reinterpret_cast<uint4*>(p) = v;
  }
};
template <>
struct Vec8<__half> {
  uint4 r;
  __device__ __forceinline__ void load_ring(const uint4* at) { r = *at; }
  __device__ __forceinline__ void get(float2* x) const {
    const __half2* h = reinterpret_cast<const __half2*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __half22float2(h[i]);
  }
  static __device__ __forceinline__ void store(void* p, const float2* x) {
    uint4 v;
    __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[i].x, x[i].y);
    *reinterpret_cast<uint4*>(p) = v;
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void load_ring(const uint4* at) {  // pieces a thread's stride apart
    a = *reinterpret_cast<const float4*>(at);
    b = *reinterpret_cast<const float4*>(at + kNrThreads);
  }
  __device__ __forceinline__ void get(float2* x) const {
    x[0] = make_float2(a.x, a.y); x[1] = make_float2(a.z, a.w);
    x[2] = make_float2(b.x, b.y); x[3] = make_float2(b.z, b.w);
  }
  static __device__ __forceinline__ void store(void* p, const float2* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
  }
};

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// cos and sin of pos * f, f the fixed-point frequency (2^64 to the turn)
__device__ __forceinline__ float2 cos_sin(int64_t pos, uint64_t f) {
  const uint64_t a = (uint64_t)pos * f;
  const float half_turns = (float)(int32_t)(a >> 32) * 4.656612873077393e-10f;  // 2^-31
  float2 cs;
  sincospif(half_turns, &cs.y, &cs.x);
  return cs;
}

__device__ __forceinline__ uint64_t fixed_turns(double f) {
  double t = f * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return t >= 1.0 ? 0ull : (uint64_t)(t * 18446744073709551616.0);
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Rotates the lane's 8 pairs by c[d], s[d] (kBack: back), d = 0..7, two FP32 operations to an instruction. Half pairs: value d of a
// with value d of b. Interleaved: neighbours inside a (pairs 0..3) and b (pairs 4..7).
template <bool kInter, bool kBack>
__device__ __forceinline__ void rotate8(float2* a, float2* b, const float* c, const float* s) {
  if constexpr (kInter) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float2& x = e < 4 ? a[e] : b[e - 4];
      const float2 turned = kBack ? make_float2(s[e], -s[e]) : make_float2(-s[e], s[e]);
      x = tc::fma2(make_float2(x.y, x.x), turned, tc::mul2(x, both(c[e])));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 ce = make_float2(c[2 * e], c[2 * e + 1]), se = make_float2(s[2 * e], s[2 * e + 1]);
      const float2 x = a[e], y = b[e], minus = tc::mul2(kBack ? x : y, both(-1.f));  // (packed operands have no sign)
      a[e] = tc::fma2(kBack ? y : minus, se, tc::mul2(x, ce));
      b[e] = tc::fma2(kBack ? minus : x, se, tc::mul2(y, ce));
    }
  }
}

// CTAs an SM (what the registers allow) and rows of a group that are on their way: 72 KiB an SM, forward in BF16.
template <typename T, bool kBwd>
constexpr int kNrBlocks = sizeof(T) == 4 ? (kBwd ? 3 : 5) : (kBwd ? 4 : 6);
template <typename T, bool kBwd>
constexpr int kNrStages = kBwd ? 3 : 4;
template <typename T, bool kBwd>
constexpr int kNrPieces = (int)sizeof(T) * (kBwd ? 2 : 1);  // 16-byte pieces of a lane and row: x (and dy)

template <typename T, int G, bool kInter, bool kBwd>
__global__ void __launch_bounds__(kNrThreads, kNrBlocks<T, kBwd>) kda_qk_norm_rope_kernel(const NrArgs a) {
  extern __shared__ __align__(16) unsigned char nr_smem[];
  constexpr int kGroups = kNrThreads / G, kStages = kNrStages<T, kBwd>, kPieces = kNrPieces<T, kBwd>;
  const int which = (int)blockIdx.x >= a.ctas0;
  const NrTensor& t = a.t[which];
  const int64_t first = which ? (int64_t)blockIdx.x - a.ctas0 : blockIdx.x;
  const int64_t ctas = which ? (int64_t)gridDim.x - a.ctas0 : a.ctas0;
  const int tid = threadIdx.x, lane = tid % G, group = tid / G;
  const int R = a.R, half = R / 2, H = t.H;
  uint64_t* turns_of = reinterpret_cast<uint64_t*>(nr_smem);               // [R / 2] fixed-point frequencies
  float* cs = reinterpret_cast<float*>(nr_smem + half * sizeof(uint64_t));  // [tokens][cos, sin][R / 2]
  uint4* ring = reinterpret_cast<uint4*>(cs + a.tokens * R) + tid;          // [stages][pieces][threads]
  const bool active = lane < a.D / 16;
  const bool turns = active && 16 * lane < R;
  // the lane's two vectors: the halves of its pairs, or 16 neighbouring values
  int c0 = 16 * lane, c1 = 16 * lane + 8;
  if (!kInter && turns) {
    c0 = 8 * lane;
    c1 = 8 * lane + half;
  }
  // This CTA's rounds of kGroups rows, a row to a group each: rows (token, head) in order, shared out evenly.
  const int64_t rows = a.n * H, all = (rows + kGroups - 1) / kGroups;
  const int64_t u0 = all * first / ctas;
  const int rounds = (int)(all * (first + 1) / ctas - u0);
  const int64_t start = u0 * kGroups / H;  // the first row's token; the others count from it
  int head0 = (int)(u0 * kGroups - start * H), token0 = 0;  // the first row of the angles at hand
  const int64_t left = rows - u0 * kGroups - group;
  const int mine = left <= 0 ? 0 : left > (int64_t)rounds * kGroups ? rounds : (int)((left + kGroups - 1) / kGroups);  // rounds with a row
  // From row to row of a group, kGroups rows on, by additions alone: the row that is worked on (its output and its
  // angles) and the one whose copy starts next (its inputs).
  const int head_step = kGroups % H, token_step = kGroups / H;
  int head = (head0 + group) % H, next_head = head, row_angle = (head0 + group) / H * R;
  const int64_t token = start + (head0 + group) / H;
  const T* xs = reinterpret_cast<const T*>(t.x) + token * t.xt + head * t.xh;
  const T* ds = kBwd ? reinterpret_cast<const T*>(t.dy) + token * t.dt + head * t.dh : nullptr;
  T* ys = reinterpret_cast<T*>(t.y) + token * t.yt + head * t.yh;
  auto fetch = [&](int i) {  // round i's row; past the end: nothing
    if (active && i < mine) {
      uint4* to = ring + kNrThreads * kPieces * (i % kStages);
      constexpr int kEach = 16 / (int)sizeof(T);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {  // x's first vector, its second; dy's
        const int v = k * kEach / 8, off = k * kEach % 8;
        tc::cp_async16(to + kNrThreads * k, (v < 2 ? xs : ds) + (v & 1 ? c1 : c0) + off, 16);
      }
    }
    tc::cp_async_commit();
    next_head += head_step;
    xs += t.x_step;
    if (kBwd) ds += t.d_step;
    if (next_head >= H) {
      next_head -= H;
      xs += t.x_wrap;
      if (kBwd) ds += t.d_wrap;
    }
  };
  if (!active) {  // (their part of a row's sum)
#pragma unroll
    for (int k = 0; k < kStages * kPieces; ++k) ring[kNrThreads * k] = make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);
  for (int d = tid; d < half; d += kNrThreads) turns_of[d] = fixed_turns(a.freq[d]);
  float2 w0[4], w1[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w0[e] = w1[e] = both(1.f);
  if (active && t.w) {
    Vec8<float> v;
    v.load(t.w + c0); v.get(w0);
    v.load(t.w + c1); v.get(w1);
  }
  float2 g0[4], g1[4];  // backward: this lane's share of dw
#pragma unroll
  for (int e = 0; e < 4; ++e) g0[e] = g1[e] = both(0.f);
  const float inv_d = 1.f / (float)a.D;

  for (int i = 0; i < rounds;) {
    // angles of the tokens of the next rounds
    const int end = R && rounds - i > t.rounds ? i + t.rounds : rounds;
    if (R) {
      __syncthreads();  // the last ones are done with (and the frequencies are there)
      const int64_t left = a.n - start - token0;
      const int last = (head0 + (end - i) * kGroups - 1) / H + 1, ntok = last < left ? last : (int)left;
      for (int j = tid; j < ntok * half; j += kNrThreads) {
        const int tt = j / half, d = j - tt * half;
        const float2 v = cos_sin(a.pos[start + token0 + tt], turns_of[d]);
        cs[tt * R + d] = v.x;
        cs[tt * R + half + d] = v.y;
      }
      __syncthreads();
    }
    // all lanes of a warp make the same number of rounds: the shuffles are warp wide
    for (; i < end; ++i) {
      tc::cp_async_wait<kStages - 2>();
      const uint4* from = ring + kNrThreads * kPieces * (i % kStages);
      const bool live = active && i < mine;
      float2 p[4], q[4], u[4], v[4];
      {
        Vec8<T> x;
        constexpr int kVec = kNrThreads * (int)sizeof(T) / 2;  // from vector to vector
        x.load_ring(from); x.get(p);
        x.load_ring(from + kVec); x.get(q);
        if constexpr (kBwd) {
          x.load_ring(from + 2 * kVec); x.get(u);
          x.load_ring(from + 3 * kVec); x.get(v);
        }
      }
      fetch(i + kStages - 1);
      T* out = ys;
      const float* angle = cs + (live && turns ? row_angle + 8 * lane : 0);
      head += head_step;
      ys += t.y_step;
      row_angle += token_step * R;
      if (head >= H) {
        head -= H;
        ys += t.y_wrap;
        row_angle += R;
      }
      float2 s2 = tc::mul2(p[0], p[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) s2 = tc::fma2(p[e], p[e], s2);
#pragma unroll
      for (int e = 0; e < 4; ++e) s2 = tc::fma2(q[e], q[e], s2);
      const float r = rsqrtf(group_sum<G>(s2.x + s2.y) * inv_d + a.eps);
      float c[8], s[8];
      if (turns) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 x = *reinterpret_cast<const float4*>(angle + e), y = *reinterpret_cast<const float4*>(angle + half + e);
          c[e] = x.x; c[e + 1] = x.y; c[e + 2] = x.z; c[e + 3] = x.w;
          s[e] = y.x; s[e + 1] = y.y; s[e + 2] = y.z; s[e + 3] = y.w;
        }
      }
      const float2 rr = both(r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] = tc::mul2(p[e], rr);
        q[e] = tc::mul2(q[e], rr);
      }
      if constexpr (!kBwd) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = tc::mul2(p[e], w0[e]);
          q[e] = tc::mul2(q[e], w1[e]);
        }
        if (turns) rotate8<kInter, false>(p, q, c, s);
      } else {
        if (turns) rotate8<kInter, true>(u, v, c, s);
        if (live) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            g0[e] = tc::fma2(u[e], p[e], g0[e]);
            g1[e] = tc::fma2(v[e], q[e], g1[e]);
          }
        }
        float2 d2 = both(0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u[e] = tc::mul2(u[e], w0[e]);
          v[e] = tc::mul2(v[e], w1[e]);
          d2 = tc::fma2(u[e], p[e], d2);
          d2 = tc::fma2(v[e], q[e], d2);
        }
        const float2 minus = both(-group_sum<G>(d2.x + d2.y) * inv_d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = tc::mul2(rr, tc::fma2(p[e], minus, u[e]));
          q[e] = tc::mul2(rr, tc::fma2(q[e], minus, v[e]));
        }
      }
      if (live) {
        Vec8<T>::store(out + c0, p);
        Vec8<T>::store(out + c1, q);
      }
    }
    const int on = head0 + t.rounds * kGroups;
    token0 += on / H;
    row_angle -= on / H * R;
    head0 = on % H;
  }
  if (kBwd && a.dw_part) {  // (no weights, no workspace: nothing to sum)
    // the CTA's share of dw: the groups' sums in a fixed order
    float* acc = reinterpret_cast<float*>(nr_smem);  // [groups of a warp summed: warps][16 G]
    tc::cp_async_wait<0>();
    __syncthreads();
    float* f0 = reinterpret_cast<float*>(g0);
    float* f1 = reinterpret_cast<float*>(g1);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = G; o < 32; o <<= 1) {
        f0[e] += __shfl_xor_sync(0xffffffffu, f0[e], o);
        f1[e] += __shfl_xor_sync(0xffffffffu, f1[e], o);
      }
    }
    const int warp = tid >> 5;
    if ((tid & 31) < G && active) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc[warp * a.D + c0 + e] = f0[e];
        acc[warp * a.D + c1 + e] = f1[e];
      }
    }
    __syncthreads();
    for (int d = tid; d < a.D; d += kNrThreads) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kNrThreads / 32; ++k) s += acc[k * a.D + d];
      a.dw_part[(int64_t)blockIdx.x * a.D + d] = s;
    }
  }
}

// dw of queries (block y 0) and keys (1): 32 columns a CTA, 32 partial sums each.
__global__ void __launch_bounds__(1024) kda_norm_weight_grad_kernel(const float* part, int ctas0, int ctas, int D,
                                                                   float* dqw, float* dkw) {
  __shared__ float s[32][32];
  const int col = threadIdx.x & 31, lane = threadIdx.x >> 5, d = blockIdx.x * 32 + col;
  const int lo = blockIdx.y ? ctas0 : 0, hi = blockIdx.y ? ctas : ctas0;
  float* out = blockIdx.y ? dkw : dqw;
  float x = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (started while the last kernel ends)
  if (d < D && out) {
#pragma unroll 8
    for (int i = lo + lane; i < hi; i += 32) x += part[(int64_t)i * D + d];
  }
  s[lane][col] = x;
  __syncthreads();
  if (lane == 0 && d < D && out) {
#pragma unroll
    for (int k = 1; k < 32; ++k) x += s[k][col];
    out[d] = x;
  }
}

kda_status nfail(kda_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

constexpr int64_t kNrMaxCtas = kSms * 6;  // backward: most CTAs, rows of dw_part

// A strided [tokens, heads, D] view in bytes.
struct View {
  uintptr_t p;
  int64_t token, extent;  // token stride; bytes from the first to past the last value of one token
  int64_t n;
};

View view_of(const void* p, int64_t ts, int64_t hs, int64_t H, int64_t D, int64_t n, int64_t size) {
  return View{(uintptr_t)p, ts * size, ((H - 1) * hs + D) * size, n};
}

// False only where no value of one view is a value of the other: apart in memory, or rows of
// the same stride whose ranges within it are apart (queries and keys of one projection).
bool may_overlap(const View& a, const View& b) {
  if (!a.n || !b.n) return false;
  const uintptr_t a1 = a.p + (a.n - 1) * a.token + a.extent, b1 = b.p + (b.n - 1) * b.token + b.extent;
  if (a1 <= b.p || b1 <= a.p) return false;
  if (a.token != b.token || a.token <= 0) return true;
  const int64_t s = a.token;
  int64_t d = ((int64_t)(b.p - a.p)) % s;
  if (d < 0) d += s;
  return !(d >= a.extent && d + b.extent <= s);
}

// The two tensors of one call, checked: strides[4 i ..] = token and head strides of input i, etc.
struct NrCall {
  const void *q, *k, *dq, *dk;
  void *q_out, *k_out;
  int32_t dtype;
  const float *qw, *kw;
  float *dqw, *dkw;
  const int64_t* pos;
  const double* freq;
  int64_t n, Hq, Hk, D, R;
  float eps;
  int32_t inter;
  const int64_t* strides;
  float* part;
  bool bwd;
  cudaStream_t stream;
};

template <typename T, int G, bool kInter, bool kBwd>
cudaError_t nr_launch(const NrArgs& a, int64_t ctas, size_t smem, cudaStream_t s) {
  auto kern = kda_qk_norm_rope_kernel<T, G, kInter, kBwd>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<(unsigned)ctas, kNrThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int G>
cudaError_t nr_by_mode(const NrArgs& a, int64_t ctas, size_t smem, bool inter, bool bwd, cudaStream_t s) {
  if (inter) return bwd ? nr_launch<T, G, true, true>(a, ctas, smem, s) : nr_launch<T, G, true, false>(a, ctas, smem, s);
  return bwd ? nr_launch<T, G, false, true>(a, ctas, smem, s) : nr_launch<T, G, false, false>(a, ctas, smem, s);
}

template <typename T>
cudaError_t nr_by_group(const NrArgs& a, int64_t ctas, size_t smem, bool inter, bool bwd, cudaStream_t s) {
  if (a.D <= 64) return nr_by_mode<T, 4>(a, ctas, smem, inter, bwd, s);
  if (a.D <= 128) return nr_by_mode<T, 8>(a, ctas, smem, inter, bwd, s);
  return nr_by_mode<T, 16>(a, ctas, smem, inter, bwd, s);
}

kda_status nr_run(const NrCall& c) {
  if (c.dtype != KDA_DTYPE_BF16 && c.dtype != KDA_DTYPE_FP32 && c.dtype != KDA_DTYPE_FP16)
    return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: dtype must be KDA_DTYPE_BF16, KDA_DTYPE_FP32 or KDA_DTYPE_FP16");
  if (c.n < 0 || c.Hq < 1 || c.Hk < 1)
    return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: num_tokens must be >= 0, Hq and Hk >= 1");
  if (size_limit_violation(1, c.n ? c.n : 1, c.Hq, 0) || size_limit_violation(1, c.n ? c.n : 1, c.Hk, 0))
    return nfail(KDA_ERR_UNSUPPORTED, "qk_norm_rope: problem too large");
  if (c.Hq > 65536 || c.Hk > 65536) return nfail(KDA_ERR_UNSUPPORTED, "qk_norm_rope: more than 65536 heads");
  if (c.D < 16 || c.D > 256 || c.D % 16)
    return nfail(KDA_ERR_UNSUPPORTED, "qk_norm_rope: head_dim must be a multiple of 16 from 16 to 256");
  if (c.R < 0 || c.R > c.D || c.R % 16)
    return nfail(KDA_ERR_UNSUPPORTED, "qk_norm_rope: rotary_dim must be a multiple of 16 from 0 to head_dim");
  if (!(c.eps >= 0.f) || std::isinf(c.eps)) return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: eps must be finite and >= 0");
  if (c.inter != 0 && c.inter != 1) return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: interleaved must be 0 or 1");
  if (c.bwd && (c.dqw == nullptr) != (c.qw == nullptr))
    return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: dq_weight goes with q_weight");
  if (c.bwd && (c.dkw == nullptr) != (c.kw == nullptr))
    return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: dk_weight goes with k_weight");
  const int64_t size = c.dtype == KDA_DTYPE_FP32 ? 4 : 2;
  // (token stride, head stride) of q, k, q_out, k_out and, backward, dq, dk
  int64_t st[12];
  const int nst = c.bwd ? 12 : 8;
  const int64_t heads[6] = {c.Hq, c.Hk, c.Hq, c.Hk, c.Hq, c.Hk};
  for (int i = 0; i < nst; ++i)
    st[i] = c.strides ? c.strides[i] : (i & 1 ? c.D : heads[i / 2] * c.D);
  for (int i = 0; i < nst; i += 2) {
    bool too_large;
    if (!view_rows_apart(c.n, heads[i / 2], c.D, st[i], st[i + 1], &too_large))
      return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: heads or tokens of a tensor overlap (strides too small)");
    if (too_large || st[i] > (int64_t(1) << 40)) return nfail(KDA_ERR_UNSUPPORTED, "qk_norm_rope: strides too large");
    if ((st[i] * size) % 16 || (st[i + 1] * size) % 16)
      return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: token and head strides must be multiples of 16 bytes");
  }
  if (c.n) {
    const void* ptrs[] = {c.q, c.k, c.q_out, c.k_out, c.bwd ? c.dq : c.q, c.bwd ? c.dk : c.k};
    for (const void* p : ptrs) {
      if (!p) return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: null tensor pointer");
      if ((uintptr_t)p & 15u) return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: tensors must be 16-byte aligned");
    }
    if (c.R && (!c.pos || !c.freq))
      return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: a rotation needs positions and inv_freq");
    if (((uintptr_t)c.qw | (uintptr_t)c.kw) & 15u)
      return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: weights must be 16-byte aligned");
  }
  if (c.bwd && (c.dqw || c.dkw) && !c.part)
    return nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: the weights' gradients need the workspace");
  // an output may be the input of the same tensor (each row is read before it is written), else
  // nothing that is read or written may be written by another
  const View in[4] = {view_of(c.q, st[0], st[1], c.Hq, c.D, c.n, size), view_of(c.k, st[2], st[3], c.Hk, c.D, c.n, size),
                      c.bwd ? view_of(c.dq, st[8], st[9], c.Hq, c.D, c.n, size) : View{0, 0, 0, 0},
                      c.bwd ? view_of(c.dk, st[10], st[11], c.Hk, c.D, c.n, size) : View{0, 0, 0, 0}};
  const int64_t in_hs[4] = {st[1], st[3], c.bwd ? st[9] : 0, c.bwd ? st[11] : 0};
  const View out[2] = {view_of(c.q_out, st[4], st[5], c.Hq, c.D, c.n, size), view_of(c.k_out, st[6], st[7], c.Hk, c.D, c.n, size)};
  const int64_t out_hs[2] = {st[5], st[7]};
  auto span = [](const void* p, int64_t bytes) { return View{(uintptr_t)p, 0, bytes, p && bytes ? 1 : 0}; };
  const View flat[4] = {span(c.qw, 4 * c.D), span(c.kw, 4 * c.D), span(c.R ? c.pos : nullptr, 8 * c.n), span(c.R ? c.freq : nullptr, 4 * c.R)};
  for (int i = 0; i < 2; ++i) {
    for (int j = 0; j < 4; ++j) {
      const bool same = (j & 1) == i && in[j].p == out[i].p && in[j].token == out[i].token && in_hs[j] == out_hs[i];
      if (!same && may_overlap(in[j], out[i]))
        return nfail(KDA_ERR_ALIASING, "qk_norm_rope: an output overlaps an input that is not its own");
    }
    for (const View& f : flat)
      if (may_overlap(f, out[i])) return nfail(KDA_ERR_ALIASING, "qk_norm_rope: an output overlaps an input");
  }
  if (may_overlap(out[0], out[1])) return nfail(KDA_ERR_ALIASING, "qk_norm_rope: the outputs overlap");
  const View sums[3] = {span(c.dqw, 4 * c.D), span(c.dkw, 4 * c.D), span(c.part, kNrMaxCtas * 4 * c.D)};
  for (int i = 0; i < 3; ++i) {
    for (const View& x : in)
      if (may_overlap(x, sums[i])) return nfail(KDA_ERR_ALIASING, "qk_norm_rope: a weight's gradient or the workspace overlaps an input");
    for (const View& x : flat)
      if (may_overlap(x, sums[i])) return nfail(KDA_ERR_ALIASING, "qk_norm_rope: a weight's gradient or the workspace overlaps an input");
    for (const View& x : out)
      if (may_overlap(x, sums[i])) return nfail(KDA_ERR_ALIASING, "qk_norm_rope: a weight's gradient or the workspace overlaps an output");
    for (int j = 0; j < i; ++j)
      if (may_overlap(sums[j], sums[i])) return nfail(KDA_ERR_ALIASING, "qk_norm_rope: the weights' gradients or the workspace overlap");
  }

  int dev = -1, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e != cudaSuccess) return nfail(KDA_ERR_CUDA, cudaGetErrorString(e));
  if (major != 10 || minor != 3) return nfail(KDA_ERR_UNSUPPORTED, "qk_norm_rope: kernels are built for sm_103a");

  NrArgs a{};
  a.pos = c.pos;
  a.freq = c.freq;
  a.dw_part = c.part;
  a.n = c.n;
  a.D = (int)c.D;
  a.R = (int)c.R;
  a.eps = c.eps;
  const bool wide = c.dtype == KDA_DTYPE_FP32;
  const int64_t resident = kSms * (wide ? (c.bwd ? kNrBlocks<float, true> : kNrBlocks<float, false>)
                                       : (c.bwd ? kNrBlocks<__half, true> : kNrBlocks<__half, false>));
  const int groups = kNrThreads / (c.D <= 64 ? 4 : c.D <= 128 ? 8 : 16);
  int64_t ctas[2];
  for (int i = 0; i < 2; ++i) {
    NrTensor& t = a.t[i];
    t.x = i ? c.k : c.q;
    t.dy = i ? c.dk : c.dq;
    t.y = i ? c.k_out : c.q_out;
    t.w = i ? c.kw : c.qw;
    t.xt = st[2 * i]; t.xh = st[2 * i + 1];
    t.yt = st[4 + 2 * i]; t.yh = st[5 + 2 * i];
    t.dt = c.bwd ? st[8 + 2 * i] : 0; t.dh = c.bwd ? st[9 + 2 * i] : 0;
    t.H = (int)heads[i];
    auto steps = [&](int64_t ts, int64_t hs, int64_t& step, int64_t& wrap) {
      step = groups / t.H * ts + groups % t.H * hs;
      wrap = ts - t.H * hs;
    };
    steps(t.xt, t.xh, t.x_step, t.x_wrap);
    steps(t.dt, t.dh, t.d_step, t.d_wrap);
    steps(t.yt, t.yh, t.y_step, t.y_wrap);
    // the CTAs that run at once, shared out by work: a token's angles take about what two of its rows do
    const int64_t units = (c.n * t.H + groups - 1) / groups, angles = c.R ? 2 : 0;
    ctas[i] = resident * (t.H + angles) / (c.Hq + c.Hk + 2 * angles);
    if (ctas[i] < 1) ctas[i] = 1;
    if (ctas[i] > units) ctas[i] = units;
    // angles at a time: of up to 16 rounds, in 12 KiB (of one round's tokens at least)
    t.rounds = 16;
    auto tokens = [&] { return (int)((t.rounds * groups + t.H - 2) / t.H + 1); };  // (a round may start within a token)
    while (t.rounds > 1 && tokens() * c.R * sizeof(float) > 12 * 1024) --t.rounds;
    if (tokens() > a.tokens) a.tokens = tokens();
  }
  a.ctas0 = (int)ctas[0];
  const size_t stages = wide ? (c.bwd ? kNrStages<float, true> : kNrStages<float, false>)
                             : (c.bwd ? kNrStages<__half, true> : kNrStages<__half, false>);
  size_t smem = (size_t)(c.R / 2) * sizeof(uint64_t) + a.tokens * c.R * sizeof(float) +
                stages * 16 * kNrThreads * size * (c.bwd ? 2 : 1);
  const int64_t grid = ctas[0] + ctas[1];
  if (grid > 0) {
    if (c.dtype == KDA_DTYPE_BF16) e = nr_by_group<__nv_bfloat16>(a, grid, smem, c.inter, c.bwd, c.stream);
    else if (c.dtype == KDA_DTYPE_FP16) e = nr_by_group<__half>(a, grid, smem, c.inter, c.bwd, c.stream);
    else e = nr_by_group<float>(a, grid, smem, c.inter, c.bwd, c.stream);
    if (e != cudaSuccess) return nfail(KDA_ERR_CUDA, cudaGetErrorString(e));
  }
  if (c.bwd && (c.dqw || c.dkw)) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((c.D + 31) / 32), 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = c.stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    const float* part = c.part;
    e = cudaLaunchKernelEx(&cfg, kda_norm_weight_grad_kernel, part, (int)ctas[0], (int)grid, (int)c.D, c.dqw, c.dkw);
    if (e != cudaSuccess) return nfail(KDA_ERR_CUDA, cudaGetErrorString(e));
  }
  return KDA_OK;
}

}  // namespace
}  // namespace kda

extern "C" kda_status kda_qk_norm_rope_fwd(const void* q, const void* k, int32_t dtype, const float* q_weight,
                                           const float* k_weight, const int64_t* positions, const double* inv_freq,
                                           int64_t num_tokens, int64_t Hq, int64_t Hk, int64_t head_dim,
                                           int64_t rotary_dim, float eps, int32_t interleaved, const int64_t* strides,
                                           void* q_out, void* k_out, struct CUstream_st* stream) {
  return kda::guarded([&]() -> kda_status {
    kda::NrCall c{};
    c.q = q; c.k = k; c.q_out = q_out; c.k_out = k_out;
    c.dtype = dtype;
    c.qw = q_weight; c.kw = k_weight;
    c.pos = positions; c.freq = inv_freq;
    c.n = num_tokens; c.Hq = Hq; c.Hk = Hk; c.D = head_dim; c.R = rotary_dim;
    c.eps = eps; c.inter = interleaved; c.strides = strides;
    c.stream = stream;
    return kda::nr_run(c);
  });
}

extern "C" kda_status kda_qk_norm_rope_workspace_bytes(int64_t head_dim, size_t* bytes) {
  if (!bytes || head_dim < 16 || head_dim > 256 || head_dim % 16)
    return kda::nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: bytes is NULL or head_dim unsupported");
  *bytes = kda::kNrMaxCtas * (size_t)head_dim * sizeof(float);
  return KDA_OK;
}

extern "C" kda_status kda_qk_norm_rope_bwd(const void* dq, const void* dk, const void* q, const void* k, int32_t dtype,
                                           const float* q_weight, const float* k_weight, const int64_t* positions,
                                           const double* inv_freq, int64_t num_tokens, int64_t Hq, int64_t Hk,
                                           int64_t head_dim, int64_t rotary_dim, float eps, int32_t interleaved,
                                           const int64_t* strides, void* dq_out, void* dk_out, float* dq_weight,
                                           float* dk_weight, void* workspace, size_t workspace_bytes,
                                           struct CUstream_st* stream) {
  return kda::guarded([&]() -> kda_status {
    kda::NrCall c{};
    c.q = q; c.k = k; c.dq = dq; c.dk = dk; c.q_out = dq_out; c.k_out = dk_out;
    c.dtype = dtype;
    c.qw = q_weight; c.kw = k_weight; c.dqw = dq_weight; c.dkw = dk_weight;
    c.pos = positions; c.freq = inv_freq;
    c.n = num_tokens; c.Hq = Hq; c.Hk = Hk; c.D = head_dim; c.R = rotary_dim;
    c.eps = eps; c.inter = interleaved; c.strides = strides;
    c.part = reinterpret_cast<float*>(workspace);
    c.bwd = true;
    c.stream = stream;
    if (workspace && workspace_bytes < kda::kNrMaxCtas * (size_t)(head_dim > 0 ? head_dim : 0) * sizeof(float))
      return kda::nfail(KDA_ERR_WORKSPACE_TOO_SMALL, "qk_norm_rope: workspace below kda_qk_norm_rope_workspace_bytes()");
    if ((uintptr_t)workspace & 15u) return kda::nfail(KDA_ERR_INVALID_ARGUMENT, "qk_norm_rope: workspace must be 16-byte aligned");
    return kda::nr_run(c);
  });
}
