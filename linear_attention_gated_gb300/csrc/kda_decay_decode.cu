// kda_decay_decode.cu -- one token per sequence of the linear attention with a
// decay for each head, on a state pool, in place:
//   S <- e^{g} S + v k^T,   o = s S q
// for the state S [128 x 128] (value-first) of pool slot state_indices[n] and
// every value head.
//
// The step reads and writes each state once and does 6 flops per state value:
// HBM bandwidth bounds it (64 KiB there and 64 KiB back per FP32 state, against
// 1 KiB of vectors). The 128 rows of a state are independent, so a CTA takes
// kRows of them: few requests still spread over the whole GPU (32 heads of one
// request are 128 CTAs). A thread has all its rows' loads in flight before it
// touches the token's vectors; a half-warp owns a row, 8 keys a lane.
//
// Measured: 256 sequences x 96 heads, BF16 states, 1.64 GB: a call among others through the Python
// binding 255 us, 6.4 TB/s, 96 % of the copy rate (in a captured graph 251 us); 128 x 96 in FP32
// 235 us; one sequence of 32 heads 5.6 us on the GPU with nothing in its caches.
#include "../../include/kda.h"
#include "kda_decay.cuh"
#include "kda_host.h"

#include <cmath>
#include <type_traits>

namespace kda {
namespace {

constexpr int kDdThreads = 128;
constexpr int kDdPerPass = kDdThreads / 16;  // rows of one pass: a half-warp each

template <typename S>
struct DdVec;
template <>
struct DdVec<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* x) const { unpack_bf16x8(r, x); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* x) { store_bf16x8(p, x); }
};
template <>
struct DdVec<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

template <typename S, int kRows>
__global__ void __launch_bounds__(kDdThreads) kda_decay_decode_kernel(const DecayProblem P, S* pool, const int32_t* idx,
                                                                      int64_t num_slots, __nv_bfloat16* o) {
  constexpr int kParts = kDim / kRows, kPasses = kRows / kDdPerPass;
  const int part = blockIdx.x % kParts;
  const int64_t unit = blockIdx.x / kParts;
  const int64_t n = unit / P.Hv;
  const int h = (int)(unit - n * P.Hv);
  const int tid = threadIdx.x, hl = tid & 15, row0 = part * kRows + (tid >> 4);
  const int64_t slot = idx ? idx[n] : n;
  if (slot < 0 || slot >= num_slots) {
    // a device index outside the pool (it no longer matches the host mirror the call was checked
    // against, as in a replayed graph): no state is touched and these values of o read NaN
    if (tid < kRows) o[(n * P.Hv + h) * kDim + part * kRows + tid] = __ushort_as_bfloat16(0x7fc0);
    return;
  }
  S* s = pool + (slot * P.Hv + h) * (int64_t)(kDim * kDim) + row0 * kDim + 8 * hl;
  DdVec<S> raw[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) raw[p].load(s + p * kDdPerPass * kDim);
  float q[8], k[8], v[kPasses];
  const int hq = h / P.r;
  load_bf16x8(P.q + n * P.qt + hq * P.qh + 8 * hl, q);
  load_bf16x8(P.k + n * P.kt + hq * P.kh + 8 * hl, k);
  const __nv_bfloat16* vr = P.v + n * P.vt + h * P.vh + row0;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) v[p] = __bfloat162float(vr[p * kDdPerPass]);
  const float d = exp2f(decay_log2(decay_g(P, n, h)));
  __nv_bfloat16* out = o + (n * P.Hv + h) * kDim + row0;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    float x[8], y = 0.f;
    raw[p].get(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = fmaf(v[p], k[e], d * x[e]);
      y = fmaf(x[e], q[e], y);
    }
    DdVec<S>::store(s + p * kDdPerPass * kDim, x);
    y = row16_sum(y);
    if (hl == 0) out[p * kDdPerPass] = __float2bfloat16_rn(P.scale * y);
  }
}

kda_status dfail(kda_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

struct Span {
  const void* p;
  size_t bytes;
};

bool overlap(const Span& a, const Span& b) {
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a.p && b.p && a.bytes && b.bytes && a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

}  // namespace
}  // namespace kda

extern "C" kda_status kda_decay_attn_decode(const kda_bf16* q, const kda_bf16* k, const kda_bf16* v,
                                            const void* log_decay, int32_t decay_per_token, void* state,
                                            int32_t state_dtype, const int32_t* state_indices,
                                            const int32_t* state_indices_host, int64_t num_slots, int64_t N,
                                            int64_t Hqk, int64_t Hv, int64_t head_dim, float scale,
                                            const int64_t* strides, kda_bf16* o, struct CUstream_st* stream) {
  using kda::dfail;
  using kda::Span;
  return kda::guarded([&]() -> kda_status {
    if (N < 0 || Hqk < 1 || Hv < 1 || Hv % Hqk)
      return dfail(KDA_ERR_INVALID_ARGUMENT, "decay_attn decode: N must be >= 0 and Hv a positive multiple of Hqk");
    if (kda::size_limit_violation(1, N ? N : 1, Hv, 0) || N > INT32_MAX / 4 / Hv)
      return dfail(KDA_ERR_UNSUPPORTED, "decay_attn decode: too many (sequence, head) units");
    if (head_dim != kda::kDim) return dfail(KDA_ERR_UNSUPPORTED, "decay_attn decode: head_dim must be 128");
    if (num_slots < 0 || num_slots > (int64_t(1) << 31) || kda::pool_too_large(num_slots, Hv))
      return dfail(KDA_ERR_UNSUPPORTED, "decay_attn decode: more than 2^31 pool slots or 2^40 states");
    if (decay_per_token != 0 && decay_per_token != 1)
      return dfail(KDA_ERR_INVALID_ARGUMENT, "decay_attn decode: decay_per_token must be 0 or 1");
    if (std::isinf(scale)) return dfail(KDA_ERR_INVALID_ARGUMENT, "decay_attn decode: scale must be finite");
    if (state_dtype != KDA_STATE_BF16 && state_dtype != KDA_STATE_FP32)
      return dfail(KDA_ERR_INVALID_ARGUMENT, "decay_attn decode: state_dtype must be KDA_STATE_BF16 or KDA_STATE_FP32");
    if ((state_indices == nullptr) != (state_indices_host == nullptr))
      return dfail(KDA_ERR_INVALID_ARGUMENT, "decay_attn decode: state_indices needs its host mirror (and the reverse)");
    if (N && (!q || !k || !v || !log_decay || !state || !o))
      return dfail(KDA_ERR_INVALID_ARGUMENT, "decay_attn decode: null tensor pointer");
    if (state_indices_host) {
      const int fault = kda::slot_fault(state_indices_host, N, num_slots);
      if (fault == 1) return dfail(KDA_ERR_INVALID_ARGUMENT, "decay_attn decode: state index out of range");
      if (fault == 2) return dfail(KDA_ERR_INVALID_ARGUMENT, "decay_attn decode: two sequences share a state slot");
    } else if (num_slots < N) {
      return dfail(KDA_ERR_INVALID_ARGUMENT, "decay_attn decode: without state_indices the pool needs a slot per sequence");
    }
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)state | (uintptr_t)o) & 15u)
      return dfail(KDA_ERR_INVALID_ARGUMENT, "decay_attn decode: token and state tensors must be 16-byte aligned");
    const int64_t D = kda::kDim, heads[3] = {Hqk, Hqk, Hv};
    int64_t x[6] = {Hqk * D, D, Hqk * D, D, Hv * D, D};
    if (strides)
      for (int i = 0; i < 6; ++i) x[i] = strides[i];
    const void* ptrs[3] = {q, k, v};
    Span ins[5];
    for (int i = 0; i < 3; ++i) {
      const int64_t ts = x[2 * i], hs = x[2 * i + 1];
      bool too_large;
      if (!kda::view_rows_apart(N, heads[i], D, ts, hs, &too_large) || too_large || hs % 8 || ts % 8 || ts > (int64_t(1) << 38))
        return dfail(KDA_ERR_INVALID_ARGUMENT,
                     "decay_attn decode: token and head strides must be multiples of 8 elements and keep rows apart");
      ins[i] = Span{ptrs[i], N ? 2 * (size_t)((N - 1) * ts + (heads[i] - 1) * hs + D) : 0};
    }
    ins[3] = Span{log_decay, decay_per_token ? 2 * (size_t)N * Hv : 4 * (size_t)Hv};
    ins[4] = Span{state_indices, 4 * (size_t)N};
    const size_t esz = state_dtype == KDA_STATE_BF16 ? 2 : 4;
    const Span st{state, esz * (size_t)num_slots * Hv * D * D}, out{o, 2 * (size_t)N * Hv * D};
    for (const Span& in : ins)
      if (overlap(in, st) || overlap(in, out))
        return dfail(KDA_ERR_ALIASING, "decay_attn decode: an input overlaps the state or o");
    if (overlap(st, out)) return dfail(KDA_ERR_ALIASING, "decay_attn decode: o overlaps the state");

    int dev = -1, major = 0, minor = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e != cudaSuccess) return dfail(KDA_ERR_CUDA, cudaGetErrorString(e));
    if (major != 10 || minor != 3) return dfail(KDA_ERR_UNSUPPORTED, "decay_attn decode: kernels are built for sm_103a");
    if (N == 0) return KDA_OK;

    kda::DecayProblem P{};
    P.q = reinterpret_cast<const __nv_bfloat16*>(q);
    P.k = reinterpret_cast<const __nv_bfloat16*>(k);
    P.v = reinterpret_cast<const __nv_bfloat16*>(v);
    P.g = log_decay;
    P.qt = x[0]; P.qh = x[1]; P.kt = x[2]; P.kh = x[3]; P.vt = x[4]; P.vh = x[5];
    P.N = N;
    P.Hqk = (int)Hqk;
    P.Hv = (int)Hv;
    P.r = (int)(Hv / Hqk);
    P.per_token = decay_per_token;
    P.scale = std::isnan(scale) ? 1.0f / std::sqrt(128.0f) : scale;
    auto launch = [&](auto* pool, auto rows) {
      kda::kda_decay_decode_kernel<std::remove_pointer_t<decltype(pool)>, decltype(rows)::value>
          <<<(unsigned)(N * Hv * (kda::kDim / decltype(rows)::value)), kda::kDdThreads, 0, stream>>>(
              P, pool, state_indices, num_slots, reinterpret_cast<__nv_bfloat16*>(o));
    };
    // 16 KiB of state to a CTA, 32 rows in FP32 and 64 in BF16: fewer rows spread few requests over more SMs, more of them
    // have more loads in flight. us in a captured graph of calls on pools in turn, 600 MB together, with 16, 32, 64, 128 rows:
    //   BF16  1 x 32 heads 1.99, 2.04, 2.25, 2.60;  3 x 64 4.83, 4.82, 4.81, 5.46;  7 x 64 7.92, 7.70, 6.78, 7.04;
    //         16 x 64 14.5, 13.3, 13.0, 13.0;  64 x 96 76.5, 68.3, 65.2, 63.4;  256 x 96 297, 264, 251, 242
    //   FP32  1 x 32 3.04, 3.19, 3.62, 5.29;  3 x 64 5.94, 5.99, 6.86, 8.33;  4 x 64 7.30, 7.07, 8.08, 8.65;
    //         16 x 64 22.0, 22.4, 23.3, 24.8;  128 x 96 234, 235, 237, 239
    // One count serves all sizes: it is the best or within 8 % of it but for a single request, whose call takes
    // longer on the host (18 us) and would gain 0.4 us at most from another.
    if (state_dtype == KDA_STATE_BF16) launch(reinterpret_cast<__nv_bfloat16*>(state), std::integral_constant<int, 64>{});
    else launch(reinterpret_cast<float*>(state), std::integral_constant<int, 32>{});
    if ((e = cudaGetLastError()) != cudaSuccess) return dfail(KDA_ERR_CUDA, cudaGetErrorString(e));
    return KDA_OK;
  });
}
