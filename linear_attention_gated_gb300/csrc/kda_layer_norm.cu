// kda_layer_norm.cu -- layer norm of rows and its gradients:
//   y = (x - m) r w + b,   m = mean(x),   r = 1 / sqrt(mean((x - m)^2) + eps)
//   dx = r (t - mean(t) - n mean(t n)),   t = dy w,   n = (x - m) r,   dw = sum dy n,   db = sum dy  (over rows)
//
// Bandwidth bounds both: x is read and y written, 16 flops a value at most. kG threads share a row and keep their part of it
// in registers, so it is read once, and the deviations are taken from the mean itself (a difference of squares
// would cancel); rows are handed out so that a CTA keeps the same columns: the weights stay in registers for all of its rows,
// as do the sums of dw and db (a row's share of FP32 weights is twice its BF16 values).
// The CTAs' sums are joined by a second small kernel in a fixed order.
#include "../../include/kda.h"
#include "kda_decay_host.h"

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

// A thread's part of a row: kPer pieces of kE values. Aligned rows: a piece is 16 bytes, the pieces of a row's threads lie
// side by side; else a thread's values lie kG apart, one load each.
template <typename T, bool kAligned, int kG, int kPer>
struct Part {
  static constexpr int kE = 16 / (int)sizeof(T);
  static __device__ __forceinline__ int column(int i, int e, int at) { return kAligned ? (i * kG + at) * kE + e : (i * kE + e) * kG + at; }
  union Piece {
    uint4 v;
    T t[kE];
    __device__ __forceinline__ Piece() {}
  };
  Piece p[kPer];
  __device__ __forceinline__ void load(const T* row, int at, int D, bool there) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if constexpr (kAligned) {
        const int c = column(i, 0, at);
        p[i].v = there && c < D ? __ldcs(reinterpret_cast<const uint4*>(row + c)) : make_uint4(0u, 0u, 0u, 0u);
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const int c = column(i, e, at);
          p[i].t[e] = there && c < D ? row[c] : from_float<T>(0.f);
        }
      }
    }
  }
  __device__ __forceinline__ float get(int i, int e) const { return to_float(p[i].t[e]); }
  __device__ __forceinline__ void set(int i, int e, float x) { p[i].t[e] = from_float<T>(x); }
  __device__ __forceinline__ void store(T* row, int at, int D) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if constexpr (kAligned) {
        const int c = column(i, 0, at);
        if (c < D) *reinterpret_cast<uint4*>(row + c) = p[i].v;
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if (column(i, e, at) < D) row[column(i, e, at)] = p[i].t[e];
      }
    }
  }
};

// Sums of kN numbers over the kG threads of a row. The whole CTA calls it; `turn` picks one of two buffers, so that
// one barrier a call is enough.
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
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) s += at[n * (kThreads / 32) + (warp & ~(kWarps - 1)) + k];
      x[n] = s;
    }
  }
}

template <typename T, bool kAligned, int kG, int kPer>
__global__ void __launch_bounds__(kThreads) kda_layer_norm_fwd_kernel(const NormArgs a) {
  using P = Part<T, kAligned, kG, kPer>;
  constexpr int kE = P::kE, kRows = kThreads / kG;
  __shared__ float buf[2 * (kThreads / 32)];
  const int at = threadIdx.x % kG, group = threadIdx.x / kG, D = a.D;
  const T* x = reinterpret_cast<const T*>(a.x);
  float w[kPer][kE], b[kPer][kE];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int c = P::column(i, e, at);
      w[i][e] = a.w && c < D ? a.w[c] : 1.f;
      b[i][e] = a.b && c < D ? a.b[c] : 0.f;
    }
  const float inv = 1.f / (float)D;
  P next;
  int64_t row = (int64_t)blockIdx.x * kRows + group;
  next.load(x + row * a.xs, at, D, row < a.rows);
  for (; row - group < a.rows; row += (int64_t)gridDim.x * kRows) {
    P v = next;
    const int64_t after = row + (int64_t)gridDim.x * kRows;
    next.load(x + after * a.xs, at, D, after < a.rows);
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < kE; ++e) s[0] += v.get(i, e);
    row_sums<kG, 1>(s, buf, 0);
    const float mean = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float d = v.get(i, e) - mean;
        if (P::column(i, e, at) < D) s[0] = fmaf(d, d, s[0]);
      }
    row_sums<kG, 1>(s, buf, 1);
    const float rstd = rsqrtf(fmaf(s[0], inv, a.eps));
    if (row < a.rows) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int e = 0; e < kE; ++e) v.set(i, e, fmaf((v.get(i, e) - mean) * rstd, w[i][e], b[i][e]));
      v.store(reinterpret_cast<T*>(a.out) + row * D, at, D);
      if (at == 0) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
      }
    }
  }
}

template <typename T, bool kAligned, int kG, int kPer>
__global__ void __launch_bounds__(kThreads) kda_layer_norm_bwd_kernel(const NormArgs a) {
  using P = Part<T, kAligned, kG, kPer>;
  constexpr int kE = P::kE, kRows = kThreads / kG;
  __shared__ float buf[4 * (kThreads / 32)];
  __shared__ float join[kRows > 1 ? kThreads * kE : 1];
  const int at = threadIdx.x % kG, group = threadIdx.x / kG, D = a.D;
  const T* x = reinterpret_cast<const T*>(a.x);
  const T* dy = reinterpret_cast<const T*>(a.dy);
  float w[kPer][kE], dw[kPer][kE], db[kPer][kE];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int c = P::column(i, e, at);
      w[i][e] = a.w && c < D ? a.w[c] : 1.f;
      dw[i][e] = db[i][e] = 0.f;
    }
  const float inv = 1.f / (float)D;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRows + group; row - group < a.rows; row += (int64_t)gridDim.x * kRows, turn ^= 1) {
    const bool there = row < a.rows;
    P v, g;
    v.load(x + row * a.xs, at, D, there);
    g.load(dy + row * a.dys, at, D, there);
    const float mean = there ? a.mean[row] : 0.f, rstd = there ? a.rstd[row] : 0.f;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < kE; ++e) {  // (columns past the end: dy is zero)
        const float d = g.get(i, e), n = (v.get(i, e) - mean) * rstd, t = d * w[i][e];
        s[0] += t;
        s[1] = fmaf(t, n, s[1]);
        dw[i][e] = fmaf(d, n, dw[i][e]);
        db[i][e] += d;
      }
    row_sums<kG, 2>(s, buf, turn);
    if (there) {
      const float mt = s[0] * inv, mn = s[1] * inv;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const float n = (v.get(i, e) - mean) * rstd, t = g.get(i, e) * w[i][e];
          v.set(i, e, rstd * (t - mt - n * mn));
        }
      v.store(reinterpret_cast<T*>(a.out) + row * D, at, D);
    }
  }
  if (!a.part) return;
  float* to = a.part + (int64_t)blockIdx.x * 2 * D;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
#pragma unroll
    for (int x2 = 0; x2 < 2; ++x2) {
      if constexpr (kRows > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kE; ++e) join[e * kThreads + threadIdx.x] = x2 ? db[i][e] : dw[i][e];
        __syncthreads();
      }
      if (group == 0)
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          float s = x2 ? db[i][e] : dw[i][e];
          if constexpr (kRows > 1) {
            s = 0.f;
            for (int r = 0; r < kRows; ++r) s += join[e * kThreads + r * kG + at];
          }
          const int c = P::column(i, e, at);
          if (c < D) to[(int64_t)x2 * D + c] = s;
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

constexpr int kParts = kSms;  // most CTAs of the backward: each leaves sums of its own

// Threads that share a row: the fewest (of 8, 32, 128, 256, 512) that keep it in 16 values each.
template <typename T, bool kAligned, bool kBwd>
cudaError_t launch_rows(const NormArgs& a, int* parts, cudaStream_t s) {
  constexpr int kE = 16 / (int)sizeof(T), k16 = 16 / kE, kWide = kBwd ? (sizeof(T) == 2 ? 3 : 4) : 32 / kE;
  auto go = [&](auto G, auto per) {
    constexpr int g = decltype(G)::value, n = decltype(per)::value, rows = kThreads / g;
    const int64_t need = (a.rows + rows - 1) / rows;
    const unsigned grid = (unsigned)std::min<int64_t>(need, kBwd ? kParts : 2 * kSms);
    *parts = (int)grid;
    if constexpr (kBwd) kda_layer_norm_bwd_kernel<T, kAligned, g, n><<<grid, kThreads, 0, s>>>(a);
    else kda_layer_norm_fwd_kernel<T, kAligned, g, n><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  };
  using std::integral_constant;
  constexpr integral_constant<int, k16> per{};
  if (a.D <= 128) return go(integral_constant<int, 8>{}, per);
  if (a.D <= 512) return go(integral_constant<int, 32>{}, per);
  if (a.D <= 2048) return go(integral_constant<int, 128>{}, per);
  if (a.D <= 4096) return go(integral_constant<int, 256>{}, per);
  if (a.D <= 8192) return go(integral_constant<int, 512>{}, per);
  if constexpr (kWide > k16)
    if (a.D <= 512 * kE * kWide) return go(integral_constant<int, 512>{}, integral_constant<int, kWide>{});
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
bool misaligned(const void* p, size_t to) { return ((uintptr_t)p & (to - 1)) != 0; }

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
    if (kda::misaligned(x, size) || kda::misaligned(y, size) || kda::misaligned(weight, 4) || kda::misaligned(bias, 4) ||
        kda::misaligned(mean, 4) || kda::misaligned(rstd, 4))
      return fail(KDA_ERR_INVALID_ARGUMENT, "tensors must be aligned to their elements");
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
    if (kda::misaligned(x, size) || kda::misaligned(dy, size) || kda::misaligned(dx, size) || kda::misaligned(weight, 4) ||
        kda::misaligned(mean, 4) || kda::misaligned(rstd, 4) || kda::misaligned(dweight, 4) || kda::misaligned(dbias, 4) ||
        kda::misaligned(workspace, 4))
      return fail(KDA_ERR_INVALID_ARGUMENT, "tensors must be aligned to their elements");
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
