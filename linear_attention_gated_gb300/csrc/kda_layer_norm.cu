// kda_layer_norm.cu -- layer norm of rows and its gradients:
//   y = (x - m) r w + b,   m = mean(x),   r = 1 / sqrt(mean((x - m)^2) + eps)
//   dx = r (t - mean(t) - n mean(t n)),   t = dy w,   n = (x - m) r,   dw = sum dy n,   db = sum dy  (over rows)
//
// Bandwidth bounds both: x is read and y written, 16 flops a value at most. kG threads share a row and keep their part of it
// in registers, so it is read once, and the deviations are taken from the mean itself (a difference of squares
// would cancel). Rows are handed out so that a thread keeps the same columns: the weights stay in registers for all of its rows
// (a row's share of FP32 weights is twice its BF16 values), as do the sums of dw and db. Rows are on their way in a
// ring of asynchronous copies, each thread's part to its own place: nobody waits for anybody but in the rows' sums. Forward, the
// sum of the next row and the squares of this one are joined in one exchange.
// The CTAs' sums of dw and db are joined by a second small kernel in a fixed order.
// 8192 rows of 12288 BF16 forward 64 us, 6.3 TB/s (103 us with rows loaded when they are needed); 8192 rows of 4096 backward 39 us,
// 5.2 TB/s (64), and 3.6 for the join.
#include "../../include/kda.h"
#include "kda_decay_host.h"
#include "tc.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

namespace kda {
namespace {

constexpr int kThreads = 512;

struct NormArgs {
  const void* x;
  const void* dy;
  void* out;           // y or dx
  const float* w;      // null: 1
  const float* b;      // null: 0
  float* mean;         // written by the forward, read by the backward
  float* rstd;
  float* part;         // [gridDim.x][2][D]: the CTAs' dw and db
  int64_t rows, xs, dys;
  int D;
  float eps;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x) {
  if constexpr (std::is_same_v<T, float>) return x;
  else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

__device__ __forceinline__ float2 pair_of(uint32_t x, const __nv_bfloat16*) { return unpack2(x); }
__device__ __forceinline__ float2 pair_of(uint32_t x, const __half*) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }
__device__ __forceinline__ uint32_t of_pair(float2 x, const __nv_bfloat16*) { return pack2(x); }
__device__ __forceinline__ uint32_t of_pair(float2 x, const __half*) {
  const __half2 y = __floats2half2_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// A thread's part of a row: kPer pieces of 16 bytes, as pairs of values. Aligned rows: the pieces of a row's threads lie side by
// side and come through a ring of asynchronous copies; else a thread's values lie kG apart and are loaded one by one.
template <typename T, bool kAligned, int kG, int kPer>
struct Part {
  static constexpr int kE = 16 / (int)sizeof(T), kPairs = kPer * kE / 2;
  static constexpr int kStages = kPer > 3 ? 3 : 4, kRingBytes = kAligned ? kStages * kPer * kThreads * 16 : 0;
  uint32_t r[kPer * 4];
  static __device__ __forceinline__ int column(int pair, int e, int at) {
    return kAligned ? (2 * pair / kE * kG + at) * kE + 2 * pair % kE + e : (2 * pair + e) * kG + at;
  }
  static __device__ __forceinline__ uint4* place(uint4* ring, int stage, int i) { return ring + (stage * kPer + i) * kThreads + threadIdx.x; }
  // (aligned) starts the copy of a row's part, zeros where there is none
  static __device__ __forceinline__ void start(uint4* ring, int stage, const T* row, int at, int D, bool there) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = (i * kG + at) * kE;
      const bool in = there && c < D;
      tc::cp_async16(place(ring, stage, i), in ? row + c : row, in ? 16u : 0u);
    }
  }
  __device__ __forceinline__ void take(uint4* ring, int stage) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) *reinterpret_cast<uint4*>(r + 4 * i) = *place(ring, stage, i);
  }
  // (not aligned)
  __device__ __forceinline__ void load(const T* row, int at, int D, bool there) {
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      const int c0 = column(p, 0, at), c1 = column(p, 1, at);
      const T x0 = there && c0 < D ? row[c0] : from_float<T>(0.f), x1 = there && c1 < D ? row[c1] : from_float<T>(0.f);
      if constexpr (sizeof(T) == 4) {
        r[2 * p] = __float_as_uint(x0);
        r[2 * p + 1] = __float_as_uint(x1);
      } else {
        r[p] = (uint32_t) * reinterpret_cast<const uint16_t*>(&x0) | (uint32_t) * reinterpret_cast<const uint16_t*>(&x1) << 16;
      }
    }
  }
  __device__ __forceinline__ float2 get(int p) const {
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(r[2 * p]), __uint_as_float(r[2 * p + 1]));
    else return pair_of(r[p], (const T*)nullptr);
  }
  __device__ __forceinline__ void set(int p, float2 x) {
    if constexpr (sizeof(T) == 4) {
      r[2 * p] = __float_as_uint(x.x);
      r[2 * p + 1] = __float_as_uint(x.y);
    } else {
      r[p] = of_pair(x, (const T*)nullptr);
    }
  }
  __device__ __forceinline__ void store(T* row, int at, int D) const {
    if constexpr (kAligned) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int c = (i * kG + at) * kE;
        if (c < D) *reinterpret_cast<uint4*>(row + c) = *reinterpret_cast<const uint4*>(r + 4 * i);
      }
    } else {
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
        const int c0 = column(p, 0, at), c1 = column(p, 1, at);
        if constexpr (sizeof(T) == 4) {
          if (c0 < D) row[c0] = __uint_as_float(r[2 * p]);
          if (c1 < D) row[c1] = __uint_as_float(r[2 * p + 1]);
        } else {
          if (c0 < D) *reinterpret_cast<uint16_t*>(row + c0) = (uint16_t)r[p];
          if (c1 < D) *reinterpret_cast<uint16_t*>(row + c1) = (uint16_t)(r[p] >> 16);
        }
      }
    }
  }
};

// Sums of kN numbers over the kG threads of a row. The row's threads call it; `turn` picks one of two buffers, so that one barrier
// a call is enough: the row's own, so that a CTA's rows do not wait for each other.
template <int kG, int kN>
__device__ __forceinline__ void row_sums(float (&x)[kN], float* buf, int turn) {
#pragma unroll
  for (int k = (kG < 32 ? kG : 32) / 2; k; k >>= 1)
#pragma unroll
    for (int n = 0; n < kN; ++n) x[n] += __shfl_xor_sync(0xffffffffu, x[n], k);
  if constexpr (kG > 32) {
    constexpr int kWarps = kG / 32;
    float* at = buf + turn * kN * (kThreads / 32);
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int n = 0; n < kN; ++n) at[n * (kThreads / 32) + warp] = x[n];
    if constexpr (kG < kThreads) asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + threadIdx.x / kG), "n"(kG) : "memory");
    else __syncthreads();
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) s += at[n * (kThreads / 32) + (warp & ~(kWarps - 1)) + k];
      x[n] = s;
    }
  }
}

// FP32 vectors' values of this thread's columns, `none` where there is no vector.
template <typename P, int kPairs>
__device__ __forceinline__ void load_vector(float2 (&to)[kPairs], const float* v, float none, int at, int D) {
#pragma unroll
  for (int p = 0; p < kPairs; ++p) {
    const int c0 = P::column(p, 0, at), c1 = P::column(p, 1, at);
    to[p] = make_float2(v && c0 < D ? v[c0] : none, v && c1 < D ? v[c1] : none);
  }
}

template <typename T, bool kAligned, int kG, int kPer>
__global__ void __launch_bounds__(kThreads) kda_layer_norm_fwd_kernel(const NormArgs a) {
  using P = Part<T, kAligned, kG, kPer>;
  constexpr int kPairs = P::kPairs, kRows = kThreads / kG, kAhead = P::kStages - 1;
  extern __shared__ uint4 ring[];
  __shared__ float buf[4 * (kThreads / 32)];
  const int at = threadIdx.x % kG, group = threadIdx.x / kG, D = a.D;
  const T* x = reinterpret_cast<const T*>(a.x);
  const int64_t first = (int64_t)blockIdx.x * kRows + group, step = (int64_t)gridDim.x * kRows;
  // row k of this thread's group
  auto start = [&](int64_t k) {
    const int64_t row = first + k * step;
    P::start(ring, (int)(k % P::kStages), x + (row < a.rows ? row : 0) * a.xs, at, D, row < a.rows);
    tc::cp_async_commit();
  };
  auto fetch = [&](P& v, int64_t k) {
    const int64_t row = first + k * step;
    if constexpr (kAligned) {
      tc::cp_async_wait<kAhead - 1>();
      v.take(ring, (int)(k % P::kStages));
      start(k + kAhead);  // (to the place that was read last time)
    } else {
      v.load(x + (row < a.rows ? row : 0) * a.xs, at, D, row < a.rows);
    }
  };
  if constexpr (kAligned)
    for (int k = 0; k < kAhead; ++k) start(k);
  float2 w[kPairs], b[kPairs];
  load_vector<P>(w, a.w, 1.f, at, D);
  load_vector<P>(b, a.b, 0.f, at, D);
  const float inv = 1.f / (float)D;
  auto sum_of = [&](const P& v) {
    float2 s = make_float2(0.f, 0.f), t = s;
#pragma unroll
    for (int p = 0; p < kPairs; p += 2) {
      s = tc::add2(s, v.get(p));
      if (p + 1 < kPairs) t = tc::add2(t, v.get(p + 1));
    }
    s = tc::add2(s, t);
    return s.x + s.y;
  };
  P v;
  fetch(v, 0);
  float sums[1] = {sum_of(v)};
  row_sums<kG, 1>(sums, buf, 0);
  float mean = sums[0] * inv;
  int turn = 1;
  for (int64_t k = 0; first - group + k * step < a.rows; ++k, turn ^= 1) {
    const int64_t row = first + k * step;
    P next;
    fetch(next, k + 1);
    const float2 m2 = make_float2(-mean, -mean);
    float2 q = make_float2(0.f, 0.f), t = q;
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      float2 d = tc::add2(v.get(p), m2);
      if (P::column(p, 0, at) >= D) d.x = 0.f;
      if (P::column(p, 1, at) >= D) d.y = 0.f;
      if (p & 1) t = tc::fma2(d, d, t);
      else q = tc::fma2(d, d, q);
    }
    q = tc::add2(q, t);
    float s[2] = {q.x + q.y, sum_of(next)};
    row_sums<kG, 2>(s, buf, turn);
    const float rstd = rsqrtf(fmaf(s[0], inv, a.eps));
    if (row < a.rows) {
#pragma unroll
      for (int p = 0; p < kPairs; ++p)
        v.set(p, tc::fma2(tc::mul2(tc::add2(v.get(p), m2), make_float2(rstd, rstd)), w[p], b[p]));
      v.store(reinterpret_cast<T*>(a.out) + row * D, at, D);
      if (at == 0) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
      }
    }
    v = next;
    mean = s[1] * inv;
  }
  if constexpr (kAligned) tc::cp_async_wait_all();
}

template <typename T, bool kAligned, int kG, int kPer>
__global__ void __launch_bounds__(kThreads) kda_layer_norm_bwd_kernel(const NormArgs a) {
  using P = Part<T, kAligned, kG, kPer>;
  constexpr int kPairs = P::kPairs, kRows = kThreads / kG, kAhead = P::kStages - 1;
  extern __shared__ uint4 ring[];  // x, then dy; at last the groups' sums
  __shared__ float buf[4 * (kThreads / 32)];
  const int at = threadIdx.x % kG, group = threadIdx.x / kG, D = a.D;
  const T* x = reinterpret_cast<const T*>(a.x);
  const T* dy = reinterpret_cast<const T*>(a.dy);
  const int64_t first = (int64_t)blockIdx.x * kRows + group, step = (int64_t)gridDim.x * kRows;
  constexpr int kHalf = P::kStages * kPer * kThreads;
  auto start = [&](int64_t k) {
    const int64_t row = first + k * step, in = row < a.rows ? row : 0;
    P::start(ring, (int)(k % P::kStages), x + in * a.xs, at, D, row < a.rows);
    P::start(ring + kHalf, (int)(k % P::kStages), dy + in * a.dys, at, D, row < a.rows);
    tc::cp_async_commit();
  };
  if constexpr (kAligned)
    for (int k = 0; k < kAhead; ++k) start(k);
  float2 w[kPairs], dw[kPairs], db[kPairs];
  load_vector<P>(w, a.w, 1.f, at, D);
#pragma unroll
  for (int p = 0; p < kPairs; ++p) dw[p] = db[p] = make_float2(0.f, 0.f);
  const float inv = 1.f / (float)D;
  int turn = 0;
  float mean = first < a.rows ? a.mean[first] : 0.f, rstd = first < a.rows ? a.rstd[first] : 0.f;
  for (int64_t k = 0; first - group + k * step < a.rows; ++k, turn ^= 1) {
    const int64_t row = first + k * step;
    const bool there = row < a.rows, more = row + step < a.rows;
    P v, g;
    if constexpr (kAligned) {
      tc::cp_async_wait<kAhead - 1>();
      v.take(ring, (int)(k % P::kStages));
      g.take(ring + kHalf, (int)(k % P::kStages));
      start(k + kAhead);
    } else {
      v.load(x + (there ? row : 0) * a.xs, at, D, there);
      g.load(dy + (there ? row : 0) * a.dys, at, D, there);
    }
    const float mean1 = more ? a.mean[row + step] : 0.f, rstd1 = more ? a.rstd[row + step] : 0.f;
    const float2 m2 = make_float2(-mean, -mean), r2 = make_float2(rstd, rstd);
    float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {  // (columns past the end: dy is zero)
      const float2 d = g.get(p), n = tc::mul2(tc::add2(v.get(p), m2), r2), t = tc::mul2(d, w[p]);
      s0 = tc::add2(s0, t);
      s1 = tc::fma2(t, n, s1);
      dw[p] = tc::fma2(d, n, dw[p]);
      db[p] = tc::add2(db[p], d);
    }
    float s[2] = {s0.x + s0.y, s1.x + s1.y};
    row_sums<kG, 2>(s, buf, turn);
    if (there) {
      const float2 mt = make_float2(-s[0] * inv, -s[0] * inv), mn = make_float2(-s[1] * inv, -s[1] * inv);
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
        const float2 n = tc::mul2(tc::add2(v.get(p), m2), r2);
        v.set(p, tc::mul2(r2, tc::fma2(n, mn, tc::fma2(g.get(p), w[p], mt))));
      }
      v.store(reinterpret_cast<T*>(a.out) + row * D, at, D);
    }
    mean = mean1;
    rstd = rstd1;
  }
  if constexpr (kAligned) tc::cp_async_wait_all();
  if (!a.part) return;
  float* to = a.part + (int64_t)blockIdx.x * 2 * D;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int p = 0; p < kPairs; ++p)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = P::column(p, e, at);
        if (c < D) {
          to[c] = e ? dw[p].y : dw[p].x;
          to[D + c] = e ? db[p].y : db[p].x;
        }
      }
  } else {
    // the groups' sums, a few columns at a time
    float2* join = reinterpret_cast<float2*>(ring);
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      __syncthreads();
      join[threadIdx.x] = dw[p];
      join[kThreads + threadIdx.x] = db[p];
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * kG; i += kThreads) {
        const int k = i % kG, which = i / kG;
        float2 s = make_float2(0.f, 0.f);
        for (int r = 0; r < kRows; ++r) s = tc::add2(s, join[which * kThreads + r * kG + k]);
        const int c0 = P::column(p, 0, k), c1 = P::column(p, 1, k);
        if (c0 < D) to[(int64_t)which * D + c0] = s.x;
        if (c1 < D) to[(int64_t)which * D + c1] = s.y;
      }
    }
  }
}

// Rows wider than registers hold: a CTA a row, which it reads again (from L2) for each sum.
template <typename T>
__global__ void __launch_bounds__(kThreads) kda_layer_norm_wide_fwd_kernel(const NormArgs a) {
  __shared__ float buf[2 * (kThreads / 32)];
  const int64_t row = blockIdx.x;
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.xs;
  T* y = reinterpret_cast<T*>(a.out) + row * a.D;
  const float inv = 1.f / (float)a.D;
  float s[1] = {0.f};
  for (int c = threadIdx.x; c < a.D; c += kThreads) s[0] += to_float(x[c]);
  row_sums<kThreads, 1>(s, buf, 0);
  const float mean = s[0] * inv;
  s[0] = 0.f;
  for (int c = threadIdx.x; c < a.D; c += kThreads) {
    const float d = to_float(x[c]) - mean;
    s[0] = fmaf(d, d, s[0]);
  }
  row_sums<kThreads, 1>(s, buf, 1);
  const float rstd = rsqrtf(fmaf(s[0], inv, a.eps));
  for (int c = threadIdx.x; c < a.D; c += kThreads)
    y[c] = from_float<T>(fmaf((to_float(x[c]) - mean) * rstd, a.w ? a.w[c] : 1.f, a.b ? a.b[c] : 0.f));
  if (threadIdx.x == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
}
template <typename T>
__global__ void __launch_bounds__(kThreads) kda_layer_norm_wide_bwd_kernel(const NormArgs a) {
  __shared__ float buf[4 * (kThreads / 32)];
  const int64_t row = blockIdx.x;
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.xs;
  const T* dy = reinterpret_cast<const T*>(a.dy) + row * a.dys;
  T* dx = reinterpret_cast<T*>(a.out) + row * a.D;
  const float inv = 1.f / (float)a.D, mean = a.mean[row], rstd = a.rstd[row];
  float s[2] = {0.f, 0.f};
  for (int c = threadIdx.x; c < a.D; c += kThreads) {
    const float t = to_float(dy[c]) * (a.w ? a.w[c] : 1.f);
    s[0] += t;
    s[1] = fmaf(t, (to_float(x[c]) - mean) * rstd, s[1]);
  }
  row_sums<kThreads, 2>(s, buf, 0);
  const float mt = s[0] * inv, mn = s[1] * inv;
  for (int c = threadIdx.x; c < a.D; c += kThreads) {
    const float n = (to_float(x[c]) - mean) * rstd, t = to_float(dy[c]) * (a.w ? a.w[c] : 1.f);
    dx[c] = from_float<T>(rstd * (t - mt - n * mn));
  }
}
// dw and db of a share of the rows, a column a thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) kda_layer_norm_wide_sums_kernel(const NormArgs a) {
  const int c = blockIdx.y * kThreads + threadIdx.x;
  if (c >= a.D) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float d = to_float(reinterpret_cast<const T*>(a.dy)[row * a.dys + c]);
    dw = fmaf(d, (to_float(reinterpret_cast<const T*>(a.x)[row * a.xs + c]) - a.mean[row]) * a.rstd[row], dw);
    db += d;
  }
  a.part[((int64_t)blockIdx.x * 2) * a.D + c] = dw;
  a.part[((int64_t)blockIdx.x * 2 + 1) * a.D + c] = db;
}

// The sum of the CTAs' parts: 32 columns a CTA (of dw's and db's, one behind the other), 8 warps share the parts.
__global__ void __launch_bounds__(256) kda_layer_norm_join_kernel(const float* part, int parts, int D, float* dw, float* db) {
  __shared__ float s[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float x = 0.f;
  if (c < 2 * D)
    for (int p = warp; p < parts; p += 8) x += part[(int64_t)p * 2 * D + c];
  s[warp][lane] = x;
  __syncthreads();
  if (warp == 0 && c < 2 * D) {
    x = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) x += s[k][lane];
    if (c < D) { if (dw) dw[c] = x; }
    else if (db) db[c - D] = x;
  }
}

constexpr int kParts = kSms;  // most CTAs: one an SM; each of the backward leaves sums of its own

// Threads that share a row: the fewest (of 8, 32, 128, 256, 512) that keep it in 16 values each.
template <typename T, bool kAligned, bool kBwd>
cudaError_t launch_rows(const NormArgs& a, int* parts, cudaStream_t s) {
  constexpr int kE = 16 / (int)sizeof(T);
  auto go = [&](auto G, auto values) {
    constexpr int g = decltype(G)::value, n = decltype(values)::value / kE, rows = kThreads / g;
    using P = Part<T, kAligned, g, n>;
    constexpr int bytes = kBwd ? std::max(2 * P::kRingBytes, g < kThreads ? 16 * kThreads : 0) : P::kRingBytes;
    const int64_t need = (a.rows + rows - 1) / rows;
    const unsigned grid = (unsigned)std::min<int64_t>(need, kParts);
    *parts = (int)grid;
    auto kern = [] {
      if constexpr (kBwd) return kda_layer_norm_bwd_kernel<T, kAligned, g, n>;
      else return kda_layer_norm_fwd_kernel<T, kAligned, g, n>;
    }();
    if (bytes > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (e != cudaSuccess) return e;
    }
    kern<<<grid, kThreads, bytes, s>>>(a);
    return cudaGetLastError();
  };
  using std::integral_constant;
  constexpr integral_constant<int, 16> v16{};
  if (a.D <= 128) return go(integral_constant<int, 8>{}, v16);
  if (a.D <= 512) return go(integral_constant<int, 32>{}, v16);
  if (a.D <= 2048) return go(integral_constant<int, 128>{}, v16);
  if (a.D <= 4096) return go(integral_constant<int, 256>{}, v16);
  if (a.D <= 8192) return go(integral_constant<int, 512>{}, v16);
  if constexpr (sizeof(T) == 2)
    if (a.D <= 12288) return go(integral_constant<int, 512>{}, integral_constant<int, 24>{});
  if constexpr (!kBwd && sizeof(T) == 2)
    if (a.D <= 16384) return go(integral_constant<int, 512>{}, integral_constant<int, 32>{});
  if constexpr (kBwd) {
    kda_layer_norm_wide_bwd_kernel<T><<<(unsigned)a.rows, kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.part) return e;
    *parts = (int)std::min<int64_t>(a.rows, kParts);
    kda_layer_norm_wide_sums_kernel<T><<<dim3((unsigned)*parts, (unsigned)((a.D + kThreads - 1) / kThreads)), kThreads, 0, s>>>(a);
  } else {
    kda_layer_norm_wide_fwd_kernel<T><<<(unsigned)a.rows, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <bool kBwd>
cudaError_t launch_norm(const NormArgs& a, int32_t dtype, int* parts, cudaStream_t s) {
  auto of = [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    const int64_t e = 16 / (int64_t)sizeof(T);
    const bool aligned = a.D % e == 0 && (a.rows == 1 || (a.xs % e == 0 && a.dys % e == 0)) &&
                         (((uintptr_t)a.x | (uintptr_t)a.dy | (uintptr_t)a.out) & 15u) == 0;
    return aligned ? launch_rows<T, true, kBwd>(a, parts, s) : launch_rows<T, false, kBwd>(a, parts, s);
  };
  if (dtype == KDA_DTYPE_BF16) return of((__nv_bfloat16*)nullptr);
  if (dtype == KDA_DTYPE_FP16) return of((__half*)nullptr);
  return of((float*)nullptr);
}

using host::Span;
constexpr const char* kOp = "layer_norm";
kda_status fail(kda_status st, const char* what) { return host::fail(kOp, st, what); }

// The limits both directions have; the bytes of x (or dy) at this row stride.
kda_status check_rows(int32_t dtype, int64_t rows, int64_t D, int64_t stride, size_t* bytes) {
  if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_FP32 && dtype != KDA_DTYPE_FP16)
    return fail(KDA_ERR_INVALID_ARGUMENT, "dtype must be KDA_DTYPE_BF16, KDA_DTYPE_FP32 or KDA_DTYPE_FP16");
  if (rows < 0 || D < 1) return fail(KDA_ERR_INVALID_ARGUMENT, "rows must be >= 0 and the width >= 1");
  if (D > (1 << 24) || rows >= INT32_MAX || rows > (int64_t(1) << 40) / D) return fail(KDA_ERR_UNSUPPORTED, "problem too large (2^24 columns, 2^31 rows, 2^40 values)");
  if (stride < D) return fail(KDA_ERR_INVALID_ARGUMENT, "rows overlap");
  if (rows && stride > (int64_t(1) << 56) / rows) return fail(KDA_ERR_UNSUPPORTED, "strides too large");
  *bytes = rows ? (dtype == KDA_DTYPE_FP32 ? 4 : 2) * (size_t)((rows - 1) * stride + D) : 0;
  return KDA_OK;
}

}  // namespace
}  // namespace kda

using kda::fail;
using kda::host::Span;

extern "C" kda_status kda_layer_norm_fwd(const void* x, int32_t dtype, const float* weight, const float* bias, int64_t rows,
                                         int64_t width, int64_t row_stride, float eps, void* y, float* mean, float* rstd,
                                         struct CUstream_st* stream) {
  return kda::guarded([&]() -> kda_status {
    size_t xb = 0, yb = 0;
    kda_status st = kda::check_rows(dtype, rows, width, row_stride, &xb);
    if (st != KDA_OK || (st = kda::check_rows(dtype, rows, width, width, &yb)) != KDA_OK) return st;
    if (!(eps >= 0.f) || eps > 3.0e38f) return fail(KDA_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
    if (rows && (!x || !y || !mean || !rstd)) return fail(KDA_ERR_INVALID_ARGUMENT, "null tensor pointer");
    const size_t size = dtype == KDA_DTYPE_FP32 ? 4 : 2;
    if (kda::host::misaligned(x, size) || kda::host::misaligned(y, size) || kda::host::misaligned(weight, 4) || kda::host::misaligned(bias, 4) ||
        kda::host::misaligned(mean, 4) || kda::host::misaligned(rstd, 4))
      return fail(KDA_ERR_INVALID_ARGUMENT, kda::host::kMisaligned);
    const Span outs[] = {{y, yb}, {mean, 4 * (size_t)rows}, {rstd, 4 * (size_t)rows}};
    const Span own[] = {{weight, 4 * (size_t)width}, {bias, 4 * (size_t)width}, {x == y && row_stride == width ? nullptr : x, xb}};
    if (kda::host::aliasing(outs, own) || kda::host::overlap(Span{x, xb}, outs[1]) || kda::host::overlap(Span{x, xb}, outs[2]))
      return fail(KDA_ERR_ALIASING, "an output overlaps an input or another output");
    int32_t* unused = nullptr;
    int32_t word = 0;
    if ((st = kda::host::check_device(kda::kOp, &word, nullptr, &unused)) != KDA_OK) return st;
    if (!rows) return KDA_OK;
    kda::NormArgs a{};
    a.x = x; a.out = y; a.w = weight; a.b = bias; a.mean = mean; a.rstd = rstd;
    a.rows = rows; a.xs = row_stride; a.D = (int)width; a.eps = eps;
    int parts = 0;
    const cudaError_t e = kda::launch_norm<false>(a, dtype, &parts, stream);
    return e == cudaSuccess ? KDA_OK : fail(KDA_ERR_CUDA, cudaGetErrorString(e));
  });
}

extern "C" kda_status kda_layer_norm_workspace_bytes(int64_t rows, int64_t width, size_t* bytes) {
  return kda::guarded([&]() -> kda_status {
    if (!bytes) return fail(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    size_t xb = 0;
    const kda_status st = kda::check_rows(KDA_DTYPE_FP32, rows, width, width, &xb);
    if (st != KDA_OK) return st;
    *bytes = 8 * (size_t)std::min<int64_t>(rows, kda::kParts) * (size_t)width;
    return KDA_OK;
  });
}

extern "C" kda_status kda_layer_norm_bwd(const void* dy, const void* x, int32_t dtype, const float* weight, const float* mean,
                                         const float* rstd, int64_t rows, int64_t width, int64_t dy_stride, int64_t row_stride,
                                         void* dx, float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                                         struct CUstream_st* stream) {
  return kda::guarded([&]() -> kda_status {
    size_t xb = 0, gb = 0, ob = 0;
    kda_status st = kda::check_rows(dtype, rows, width, row_stride, &xb);
    if (st != KDA_OK || (st = kda::check_rows(dtype, rows, width, dy_stride, &gb)) != KDA_OK ||
        (st = kda::check_rows(dtype, rows, width, width, &ob)) != KDA_OK) return st;
    if (rows && (!x || !dy || !dx || !mean || !rstd)) return fail(KDA_ERR_INVALID_ARGUMENT, "null tensor pointer");
    const bool sums = dweight || dbias;
    const size_t need = sums ? 8 * (size_t)std::min<int64_t>(rows, kda::kParts) * (size_t)width : 0;
    if (need && (!workspace || workspace_bytes < need))
      return fail(KDA_ERR_WORKSPACE_TOO_SMALL, "workspace below kda_layer_norm_workspace_bytes()");
    const size_t size = dtype == KDA_DTYPE_FP32 ? 4 : 2;
    if (kda::host::misaligned(x, size) || kda::host::misaligned(dy, size) || kda::host::misaligned(dx, size) || kda::host::misaligned(weight, 4) ||
        kda::host::misaligned(mean, 4) || kda::host::misaligned(rstd, 4) || kda::host::misaligned(dweight, 4) || kda::host::misaligned(dbias, 4) ||
        kda::host::misaligned(workspace, 4))
      return fail(KDA_ERR_INVALID_ARGUMENT, kda::host::kMisaligned);
    // dx may take the place of dy or x (contiguous ones): a row is read before it is written. Rows wider than registers hold
    // are read again for the sums, so there it may not.
    const bool again = width > (dtype == KDA_DTYPE_FP32 ? 8192 : 12288);
    const size_t wb = 4 * (size_t)width, rb = 4 * (size_t)rows;
    const Span outs[] = {{dx, ob}, {dweight, wb}, {dbias, wb}, {workspace, workspace_bytes}};
    const Span ins[] = {{weight, wb}, {mean, rb}, {rstd, rb},
                        {!again && dx == x && row_stride == width ? nullptr : x, xb},
                        {!again && dx == dy && dy_stride == width ? nullptr : dy, gb}};
    bool clash = kda::host::aliasing(outs, ins);
    for (int i = 1; i < 4; ++i) clash = clash || kda::host::overlap(outs[i], Span{x, xb}) || kda::host::overlap(outs[i], Span{dy, gb});
    if (clash) return fail(KDA_ERR_ALIASING, "an output overlaps an input or another output");
    int32_t* unused = nullptr;
    int32_t word = 0;
    if ((st = kda::host::check_device(kda::kOp, &word, nullptr, &unused)) != KDA_OK) return st;
    kda::NormArgs a{};
    a.x = x; a.dy = dy; a.out = dx; a.w = weight;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.part = sums ? reinterpret_cast<float*>(workspace) : nullptr;
    a.rows = rows; a.xs = row_stride; a.dys = dy_stride; a.D = (int)width;
    int parts = 0;
    cudaError_t e = cudaSuccess;
    if (rows) e = kda::launch_norm<true>(a, dtype, &parts, stream);
    if (e == cudaSuccess && sums) {
      kda::kda_layer_norm_join_kernel<<<(unsigned)((2 * width + 31) / 32), 256, 0, stream>>>(a.part, parts, (int)width, dweight, dbias);
      e = cudaGetLastError();
    }
    return e == cudaSuccess ? KDA_OK : fail(KDA_ERR_CUDA, cudaGetErrorString(e));
  });
}
