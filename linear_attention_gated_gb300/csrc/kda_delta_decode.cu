// kda_delta_decode.cu -- one token per sequence of the gated delta rule, on a state pool, in place:
//   S' = e^{g} S,  u = v - S' k,  S <- S' + beta u k^T,   o = s S q
// for the state S [128 x 128] (value-first) of pool slot state_indices[n] and every value head.
//
// The step reads and writes each state once and does 10 flops per state value: HBM bandwidth bounds it (64 KiB there
// and 64 KiB back per FP32 state, against 1 KiB of vectors). The 128 rows of a state are independent, so a CTA takes
// kRows of them; a half-warp owns a row, 8 keys a lane, and all of a thread's rows are in flight before it touches the
// token's vectors. Both sums over the keys are taken of the old state, S k and S q, and o = s (e^g S q + beta u k . q): they do not
// follow one another. The sums of all of a half-warp's rows are exchanged together, each step halving what a lane holds:
// 15 and 8 shuffles for eight rows, where sums row by row take 64. 256 sequences of 96 heads, BF16: 264 us, 6.2 TB/s; the sums one
// after the other 323 us.
#include "kda_decay_host.h"
#include "kda_delta.cuh"

#include <type_traits>

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kPerPass = kThreads / 16;  // rows of one pass: a half-warp each

template <typename S, int kRows>
__global__ void __launch_bounds__(kThreads) kda_delta_decode_kernel(const DeltaProblem P, S* pool, const int32_t* idx,
                                                                    int64_t num_slots, __nv_bfloat16* o) {
  constexpr int kParts = kDim / kRows, kPasses = kRows / kPerPass;
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
  StateVec<S> raw[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) raw[p].load(s + p * kPerPass * kDim);
  float q[8], k[8];
  const int hq = h / P.r;
  load_bf16x8(P.q + n * P.qt + hq * P.qh + 8 * hl, q);
  load_bf16x8(P.k + n * P.kt + hq * P.kh + 8 * hl, k);
  // after the exchange lane hl holds number hl of 16 (S k of its 8 rows, then S q), or hl / 2 of 8
  constexpr int kSums = 2 * kPasses;
  static_assert(kSums == 16 || kSums == 8, "sums of a half-warp");
  const int mine = kSums == 16 ? hl & 7 : (hl >> 1) & 3, row = mine * kPerPass;  // its row
  const float v = __bfloat162float(P.v[n * P.vt + h * P.vh + row0 + row]);
  const float d = P.g ? exp2f(decay_log2(decay_g(P, n, h))) : 1.f;
  const float beta = __bfloat162float(P.beta[n * P.Hv + h]);
  float kq = 0.f, sum[kSums];
#pragma unroll
  for (int e = 0; e < 8; ++e) kq = fmaf(k[e], q[e], kq);
  kq = row16_sum(kq);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    float x[8], z = 0.f, y = 0.f;
    raw[p].get(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      z = fmaf(x[e], k[e], z);
      y = fmaf(x[e], q[e], y);
    }
    sum[p] = z;
    sum[kPasses + p] = y;
  }
  int m = kSums;
#pragma unroll
  for (int o = 8; o; o >>= 1) {
    if (m > 1) {
      m /= 2;
      const bool up = hl & o;
#pragma unroll
      for (int i = 0; i < kSums / 2; ++i)
        if (i < m) {
          const float got = __shfl_xor_sync(0xffffffffu, up ? sum[i] : sum[i + m], o);
          sum[i] = (up ? sum[i + m] : sum[i]) + got;
        }
    } else {
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
    }
  }
  const float own = d * sum[0];
  const float bu = beta * (v - own);  // (of the lanes that hold S k)
  const float there = __shfl_xor_sync(0xffffffffu, bu, 8);
  if ((hl & 8) && (kSums == 16 || !(hl & 1))) o[(n * P.Hv + h) * kDim + row0 + row] = __float2bfloat16_rn(P.scale * fmaf(there, kq, own));
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const float u = __shfl_sync(0xffffffffu, bu, (tid & 16) | (kSums == 16 ? p : 2 * p));
    float x[8];
    raw[p].get(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(u, k[e], d * x[e]);
    StateVec<S>::store(s + p * kPerPass * kDim, x);
  }
}

}  // namespace
}  // namespace kda

extern "C" kda_status kda_gated_delta_decode(const kda_bf16* q, const kda_bf16* k, const kda_bf16* v, const kda_bf16* log_decay,
                                             const kda_bf16* beta, void* state, int32_t state_dtype,
                                             const int32_t* state_indices, const int32_t* state_indices_host,
                                             int64_t num_slots, int64_t N, int64_t Hqk, int64_t Hv, int64_t head_dim,
                                             float scale, const int64_t* strides, kda_bf16* o, struct CUstream_st* stream) {
  using namespace kda::host;
  constexpr const char* op = "gated_delta decode";
  return kda::guarded([&]() -> kda_status {
    if (N < 0) return fail(op, KDA_ERR_INVALID_ARGUMENT, "N must be >= 0");
    kda::DeltaProblem P{};
    Span in[5];
    kda_status st = check_tokens(op, q, k, v, log_decay, false, 1, nullptr, nullptr, 0, N ? N : 1, N ? 1 : 0, Hqk, Hv, head_dim, scale,
                                 strides, &P, in);
    if (st != KDA_OK) return st;
    if (N > INT32_MAX / 4 / Hv) return fail(op, KDA_ERR_UNSUPPORTED, "too many (sequence, head) units");
    if (N && (!beta || !state || !o)) return fail(op, KDA_ERR_INVALID_ARGUMENT, "null tensor pointer");
    if (misaligned(beta, 2)) return fail(op, KDA_ERR_INVALID_ARGUMENT, kMisaligned);
    const kda::host::Pool pool{state, state_dtype, state_indices, state_indices_host, num_slots};
    if ((st = check_pool(op, pool, N, Hv)) != KDA_OK) return st;
    if ((uintptr_t)o & 15u) return fail(op, KDA_ERR_INVALID_ARGUMENT, "state and output tensors must be 16-byte aligned");
    const size_t gates = 2 * (size_t)N * Hv;
    const Span outs[] = {pool_span(pool, Hv), {o, gates * kda::kDim}};
    const Span ins[] = {in[0], in[1], in[2], {log_decay, gates}, {beta, gates}, {state_indices, 4 * (size_t)N}};
    if (aliasing(outs, ins)) return fail(op, KDA_ERR_ALIASING, "an output overlaps an input or another output");
    int32_t none = 0;  // (no status word: the kernel reports a bad slot in o)
    if ((st = check_device(op, &none, nullptr, &P.status)) != KDA_OK) return st;
    P.status = nullptr;
    if (N == 0) return KDA_OK;
    P.N = N;
    P.beta = reinterpret_cast<const __nv_bfloat16*>(beta);
    auto launch = [&](auto* states, auto rows) {
      kda::kda_delta_decode_kernel<std::remove_pointer_t<decltype(states)>, decltype(rows)::value>
          <<<(unsigned)(N * Hv * (kda::kDim / decltype(rows)::value)), kda::kThreads, 0, stream>>>(
              P, states, state_indices, num_slots, reinterpret_cast<__nv_bfloat16*>(o));
    };
    // 16 KiB of state to a CTA, as in the decay attention's step
    if (state_dtype == KDA_STATE_BF16) launch(reinterpret_cast<__nv_bfloat16*>(state), std::integral_constant<int, 64>{});
    else launch(reinterpret_cast<float*>(state), std::integral_constant<int, 32>{});
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? KDA_OK : fail(op, KDA_ERR_CUDA, cudaGetErrorString(e));
  });
}
