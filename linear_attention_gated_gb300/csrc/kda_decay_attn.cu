// kda_decay_attn.cu -- host side of the linear attention with a decay for each
// head: argument checks, workspace sizes and launches of kda_decay_attn_fwd,
// kda_decay_attn_bwd and kda_decay_attn_prefill. Nothing is allocated here.
#include "kda_decay_host.h"

namespace {

__device__ int32_t g_decay_status;

constexpr const char* kOp = "decay_attn";
using kda::host::aliasing;
using kda::host::check_shape;
using kda::host::Shape;
using kda::host::Span;

kda_status fail(kda_status st, const char* what) { return kda::host::fail(kOp, st, what); }

kda_status check_tokens(const void* q, const void* k, const void* v, const void* g, int32_t per_token,
                        const int64_t* cu_dev, const int64_t* cu_host, int64_t num_seqs, int64_t B, int64_t T,
                        int64_t Hqk, int64_t Hv, int64_t head_dim, float scale, const int64_t* strides,
                        kda::DecayProblem* P, Span (&spans)[5]) {
  const kda_status st = kda::host::check_tokens(kOp, q, k, v, g, true, per_token, cu_dev, cu_host, num_seqs, B, T, Hqk, Hv, head_dim,
                                                scale, strides, P, spans);
  if (st == KDA_OK) P->seg = kda::decay_segment_tokens(cu_host, P->N, T, Hv);
  return st;
}

kda_status check_workspace(const kda::DecayProblem& P, void* ws, size_t bytes, bool training) {
  const size_t need = kda::decay_workspace_bytes(P.N, P.Ttot, P.Hqk, P.Hv, P.seg, training, P.per_token);
  if (need && (!ws || bytes < need))
    return fail(KDA_ERR_WORKSPACE_TOO_SMALL, "workspace below kda_decay_attn_workspace_bytes()");
  if ((uintptr_t)ws & 255u) return fail(KDA_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
  return KDA_OK;
}

kda_status check_device(int32_t* device_status, int32_t** status) {
  return kda::host::check_device(kOp, device_status, &g_decay_status, status);
}

}  // namespace

extern "C" kda_status kda_decay_attn_workspace_bytes(int64_t B, int64_t T, int64_t Hqk, int64_t Hv,
                                                     const int64_t* cu_seqlens_host, int64_t num_seqs,
                                                     int32_t decay_per_token, int32_t training, size_t* bytes) {
  return kda::guarded([&]() -> kda_status {
    if (!bytes) return fail(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    Shape s{};
    const kda_status st = check_shape(kOp, B, T, Hqk, Hv, cu_seqlens_host, num_seqs, &s);
    if (st != KDA_OK) return st;
    *bytes = kda::decay_workspace_bytes(s.N, s.Ttot, Hqk, Hv, kda::decay_segment_tokens(cu_seqlens_host, s.N, T, Hv), training != 0, decay_per_token != 0);
    return KDA_OK;
  });
}

extern "C" kda_status kda_decay_attn_fwd(const kda_bf16* q, const kda_bf16* k, const kda_bf16* v, const void* log_decay,
                                         int32_t decay_per_token, const float* h0, const int64_t* cu_seqlens_dev,
                                         const int64_t* cu_seqlens_host, int64_t num_seqs, int64_t B, int64_t T,
                                         int64_t Hqk, int64_t Hv, int64_t head_dim, float scale,
                                         const int64_t* strides, kda_bf16* o, float* h_T, void* workspace,
                                         size_t workspace_bytes, int32_t* device_status, struct CUstream_st* stream) {
  return kda::guarded([&]() -> kda_status {
    kda::DecayProblem P{};
    Span in[5];
    kda_status st = check_tokens(q, k, v, log_decay, decay_per_token, cu_seqlens_dev, cu_seqlens_host, num_seqs, B, T,
                                 Hqk, Hv, head_dim, scale, strides, &P, in);
    if (st != KDA_OK) return st;
    if (!h_T || (P.Ttot && !o)) return fail(KDA_ERR_INVALID_ARGUMENT, "null output pointer");
    if (((uintptr_t)o | (uintptr_t)h0 | (uintptr_t)h_T) & 15u)
      return fail(KDA_ERR_INVALID_ARGUMENT, "state and output tensors must be 16-byte aligned");
    if ((st = check_workspace(P, workspace, workspace_bytes, true)) != KDA_OK) return st;
    const size_t states = 4 * (size_t)P.N * Hv * kda::kDim * kda::kDim;
    const Span outs[] = {{o, 2 * (size_t)P.Ttot * Hv * kda::kDim}, {h_T, states}, {workspace, workspace_bytes},
                         {device_status, 4}};
    const Span ins[] = {in[0], in[1], in[2], in[3], in[4], {h0, states}};
    if (aliasing(outs, ins)) return fail(KDA_ERR_ALIASING, "an output overlaps an input or another output");
    if ((st = check_device(device_status, &P.status)) != KDA_OK) return st;
    const kda::DecayStates S{h0, h_T, 0, nullptr, P.N};
    const cudaError_t e = kda::launch_decay_forward(P, S, reinterpret_cast<__nv_bfloat16*>(o), workspace, stream);
    return e == cudaSuccess ? KDA_OK : fail(KDA_ERR_CUDA, cudaGetErrorString(e));
  });
}

extern "C" kda_status kda_decay_attn_bwd(const kda_bf16* q, const kda_bf16* k, const kda_bf16* v, const void* log_decay,
                                         int32_t decay_per_token, const float* h0, const int64_t* cu_seqlens_dev,
                                         const int64_t* cu_seqlens_host, int64_t num_seqs, int64_t B, int64_t T,
                                         int64_t Hqk, int64_t Hv, int64_t head_dim, float scale,
                                         const int64_t* strides, const float* h_T, const kda_bf16* d_o,
                                         const float* d_hT, kda_bf16* dq,
                                         kda_bf16* dk, kda_bf16* dv, kda_bf16* dlog_decay, float* dh0, void* workspace,
                                         size_t workspace_bytes, int32_t* device_status, struct CUstream_st* stream) {
  return kda::guarded([&]() -> kda_status {
    kda::DecayProblem P{};
    Span in[5];
    kda_status st = check_tokens(q, k, v, log_decay, decay_per_token, cu_seqlens_dev, cu_seqlens_host, num_seqs, B, T,
                                 Hqk, Hv, head_dim, scale, strides, &P, in);
    if (st != KDA_OK) return st;
    if ((dlog_decay || P.r > 1) && kda::decay_group_sum_blocks(P) > INT32_MAX)
      return fail(KDA_ERR_UNSUPPORTED, "problem too large for the sums over heads (2^31 blocks)");
    if (P.Ttot && (!d_o || !dq || !dk || !dv)) return fail(KDA_ERR_INVALID_ARGUMENT, "null gradient pointer");
    if (dlog_decay && !decay_per_token)
      return fail(KDA_ERR_UNSUPPORTED, "a fixed decay for each head has no gradient: dlog_decay must be NULL");
    if (dlog_decay && d_hT && !h_T)
      return fail(KDA_ERR_INVALID_ARGUMENT, "the decays' gradient needs the forward's h_T where there is a d_hT");
    if (((uintptr_t)h_T | (uintptr_t)d_o | (uintptr_t)d_hT | (uintptr_t)dq | (uintptr_t)dk | (uintptr_t)dv | (uintptr_t)h0 | (uintptr_t)dh0) & 15u)
      return fail(KDA_ERR_INVALID_ARGUMENT, "state, adjoint and gradient tensors must be 16-byte aligned");
    if (kda::host::misaligned(dlog_decay, 2)) return fail(KDA_ERR_INVALID_ARGUMENT, kda::host::kMisaligned);
    if ((st = check_workspace(P, workspace, workspace_bytes, true)) != KDA_OK) return st;
    const size_t states = 4 * (size_t)P.N * Hv * kda::kDim * kda::kDim;
    const size_t tq = 2 * (size_t)P.Ttot * Hqk * kda::kDim, tv = 2 * (size_t)P.Ttot * Hv * kda::kDim;
    const Span outs[] = {{dq, tq}, {dk, tq}, {dv, tv}, {dlog_decay, 2 * (size_t)P.Ttot * Hv}, {dh0, states},
                         {workspace, workspace_bytes}, {device_status, 4}};
    const Span ins[] = {in[0], in[1], in[2], in[3], in[4], {h0, states}, {h_T, states}, {d_o, tv}, {d_hT, states}};
    if (aliasing(outs, ins)) return fail(KDA_ERR_ALIASING, "an output overlaps an input or another output");
    if ((st = check_device(device_status, &P.status)) != KDA_OK) return st;
    kda::DecayGrads G{};
    G.d_o = reinterpret_cast<const __nv_bfloat16*>(d_o);
    G.d_hT = d_hT;
    G.dq = reinterpret_cast<__nv_bfloat16*>(dq);
    G.dk = reinterpret_cast<__nv_bfloat16*>(dk);
    G.dv = reinterpret_cast<__nv_bfloat16*>(dv);
    G.dg = reinterpret_cast<__nv_bfloat16*>(dlog_decay);
    G.dh0 = dh0;
    const cudaError_t e = kda::launch_decay_backward(P, h0, h_T, G, workspace, stream);
    return e == cudaSuccess ? KDA_OK : fail(KDA_ERR_CUDA, cudaGetErrorString(e));
  });
}

extern "C" kda_status kda_decay_attn_prefill(const kda_bf16* q, const kda_bf16* k, const kda_bf16* v,
                                             const void* log_decay, int32_t decay_per_token,
                                             const int64_t* cu_seqlens_dev, const int64_t* cu_seqlens_host,
                                             int64_t num_seqs, int64_t B, int64_t T, int64_t Hqk, int64_t Hv,
                                             int64_t head_dim, float scale, const int64_t* strides, void* state,
                                             int32_t state_dtype, const int32_t* state_indices,
                                             const int32_t* state_indices_host, int64_t num_slots, kda_bf16* o,
                                             void* workspace, size_t workspace_bytes, int32_t* device_status,
                                             struct CUstream_st* stream) {
  return kda::guarded([&]() -> kda_status {
    kda::DecayProblem P{};
    Span in[5];
    kda_status st = check_tokens(q, k, v, log_decay, decay_per_token, cu_seqlens_dev, cu_seqlens_host, num_seqs, B, T,
                                 Hqk, Hv, head_dim, scale, strides, &P, in);
    if (st != KDA_OK) return st;
    if (state_dtype != KDA_STATE_BF16 && state_dtype != KDA_STATE_FP32)
      return fail(KDA_ERR_INVALID_ARGUMENT, "state_dtype must be KDA_STATE_BF16 or KDA_STATE_FP32");
    if (!state || (P.Ttot && !o)) return fail(KDA_ERR_INVALID_ARGUMENT, "null tensor pointer");
    if (((uintptr_t)o | (uintptr_t)state) & 15u)
      return fail(KDA_ERR_INVALID_ARGUMENT, "state and output tensors must be 16-byte aligned");
    if (kda::host::misaligned(state_indices, 4)) return fail(KDA_ERR_INVALID_ARGUMENT, kda::host::kMisaligned);
    if (num_slots < 1 || num_slots > (int64_t(1) << 31) || kda::pool_too_large(num_slots, Hv))
      return fail(KDA_ERR_UNSUPPORTED, "the pool needs 1 to 2^31 slots, and at most 2^40 states");
    if ((state_indices == nullptr) != (state_indices_host == nullptr))
      return fail(KDA_ERR_INVALID_ARGUMENT, "state_indices needs its host mirror (and the reverse)");
    if (state_indices_host) {
      const int fault = kda::slot_fault(state_indices_host, P.N, num_slots);
      if (fault == 1) return fail(KDA_ERR_INVALID_ARGUMENT, "state index out of range");
      if (fault == 2) return fail(KDA_ERR_INVALID_ARGUMENT, "two sequences share a state slot");
    } else if (num_slots < P.N) {
      return fail(KDA_ERR_INVALID_ARGUMENT, "without state_indices the pool needs a slot per sequence");
    }
    if ((st = check_workspace(P, workspace, workspace_bytes, false)) != KDA_OK) return st;
    const size_t esz = state_dtype == KDA_STATE_BF16 ? 2 : 4;
    const Span outs[] = {{state, esz * (size_t)num_slots * Hv * kda::kDim * kda::kDim},
                         {o, 2 * (size_t)P.Ttot * Hv * kda::kDim}, {workspace, workspace_bytes}, {device_status, 4}};
    const Span ins[] = {in[0], in[1], in[2], in[3], in[4], {state_indices, 4 * (size_t)P.N}};
    if (aliasing(outs, ins)) return fail(KDA_ERR_ALIASING, "an output overlaps an input or another output");
    if ((st = check_device(device_status, &P.status)) != KDA_OK) return st;
    const kda::DecayStates S{state, state, state_dtype == KDA_STATE_BF16, state_indices, num_slots};
    const cudaError_t e = kda::launch_decay_forward(P, S, reinterpret_cast<__nv_bfloat16*>(o), workspace, stream);
    return e == cudaSuccess ? KDA_OK : fail(KDA_ERR_CUDA, cudaGetErrorString(e));
  });
}
