// kda_delta_attn.cu -- host side of the gated delta rule: argument checks, workspace sizes and launches of
// kda_gated_delta_fwd, kda_gated_delta_bwd and kda_gated_delta_prefill. Nothing is allocated here.
#include "kda_decay_host.h"
#include "kda_delta.cuh"

namespace {

using namespace kda::host;

__device__ int32_t g_delta_status;

constexpr const char* kOp = "gated_delta";

kda_status fail(kda_status st, const char* what) { return kda::host::fail(kOp, st, what); }

kda_status set_slots(const Shape& s, int64_t Hv, int64_t* slots) {
  *slots = s.Ttot / kda::kDecayChunk + s.N;
  return *slots > INT32_MAX / Hv ? fail(KDA_ERR_UNSUPPORTED, "too many (chunk, head) pairs") : KDA_OK;
}

// What the three entry points share. spans: the bytes of q, k, v, the decays, the offsets and beta.
kda_status check(const void* q, const void* k, const void* v, const void* g, const void* beta, const int64_t* cu_dev,
                 const int64_t* cu_host, int64_t num_seqs, int64_t B, int64_t T, int64_t Hqk, int64_t Hv, int64_t head_dim,
                 float scale, const int64_t* strides, kda::DeltaProblem* P, Span (&spans)[6]) {
  Span in[5];
  const kda_status st = check_tokens(kOp, q, k, v, g, false, 1, cu_dev, cu_host, num_seqs, B, T, Hqk, Hv, head_dim, scale, strides, P, in);
  if (st != KDA_OK) return st;
  if (P->Ttot && !beta) return fail(KDA_ERR_INVALID_ARGUMENT, "null tensor pointer");
  if (misaligned(beta, 2)) return fail(KDA_ERR_INVALID_ARGUMENT, kMisaligned);
  for (int i = 0; i < 5; ++i) spans[i] = in[i];
  spans[5] = Span{beta, 2 * (size_t)P->Ttot * Hv};
  P->beta = reinterpret_cast<const __nv_bfloat16*>(beta);
  P->seg = kda::delta_segment_tokens(cu_host, P->N, T, Hv);
  return set_slots(Shape{P->N, P->Ttot, 0}, Hv, &P->slots);
}

kda_status check_workspace(const kda::DeltaProblem& P, void* ws, size_t bytes, bool training) {
  const size_t need = P.Ttot ? kda::delta_workspace(P, training).total : 0;
  if (need && (!ws || bytes < need))
    return fail(KDA_ERR_WORKSPACE_TOO_SMALL, "workspace below kda_gated_delta_workspace_bytes()");
  if ((uintptr_t)ws & 255u) return fail(KDA_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
  return KDA_OK;
}

}  // namespace

extern "C" kda_status kda_gated_delta_workspace_bytes(int64_t B, int64_t T, int64_t Hqk, int64_t Hv, const int64_t* cu_seqlens_host,
                                                      int64_t num_seqs, int32_t training, size_t* bytes) {
  return kda::guarded([&]() -> kda_status {
    if (!bytes) return fail(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    Shape s{};
    kda_status st = check_shape(kOp, B, T, Hqk, Hv, cu_seqlens_host, num_seqs, &s);
    kda::DeltaProblem P{};
    if (st != KDA_OK || (st = set_slots(s, Hv, &P.slots)) != KDA_OK) return st;
    P.N = s.N;
    P.Ttot = s.Ttot;
    P.Hv = (int)Hv;
    P.seg = kda::delta_segment_tokens(cu_seqlens_host, s.N, T, Hv);
    *bytes = s.Ttot ? kda::delta_workspace(P, training != 0).total : 0;
    return KDA_OK;
  });
}

extern "C" kda_status kda_gated_delta_fwd(const kda_bf16* q, const kda_bf16* k, const kda_bf16* v, const kda_bf16* log_decay,
                                          const kda_bf16* beta, const float* h0, const int64_t* cu_seqlens_dev,
                                          const int64_t* cu_seqlens_host, int64_t num_seqs, int64_t B, int64_t T, int64_t Hqk,
                                          int64_t Hv, int64_t head_dim, float scale, const int64_t* strides, kda_bf16* o,
                                          float* h_T, void* workspace, size_t workspace_bytes, int32_t* device_status,
                                          struct CUstream_st* stream) {
  return kda::guarded([&]() -> kda_status {
    kda::DeltaProblem P{};
    Span in[6];
    kda_status st = check(q, k, v, log_decay, beta, cu_seqlens_dev, cu_seqlens_host, num_seqs, B, T, Hqk, Hv, head_dim, scale, strides, &P, in);
    if (st != KDA_OK) return st;
    if (!h_T || (P.Ttot && !o)) return fail(KDA_ERR_INVALID_ARGUMENT, "null output pointer");
    if (((uintptr_t)o | (uintptr_t)h0 | (uintptr_t)h_T) & 15u)
      return fail(KDA_ERR_INVALID_ARGUMENT, "state and output tensors must be 16-byte aligned");
    if ((st = check_workspace(P, workspace, workspace_bytes, true)) != KDA_OK) return st;
    const size_t states = 4 * (size_t)P.N * Hv * kda::kDim * kda::kDim;
    const Span outs[] = {{o, 2 * (size_t)P.Ttot * Hv * kda::kDim}, {h_T, states}, {workspace, workspace_bytes}, {device_status, 4}};
    const Span ins[] = {in[0], in[1], in[2], in[3], in[4], in[5], {h0, states}};
    if (aliasing(outs, ins)) return fail(KDA_ERR_ALIASING, "an output overlaps an input or another output");
    if ((st = check_device(kOp, device_status, &g_delta_status, &P.status)) != KDA_OK) return st;
    const kda::DecayStates S{h0, h_T, 0, nullptr, P.N};
    const cudaError_t e = kda::launch_delta_forward(P, S, reinterpret_cast<__nv_bfloat16*>(o), true, workspace, stream);
    return e == cudaSuccess ? KDA_OK : fail(KDA_ERR_CUDA, cudaGetErrorString(e));
  });
}

extern "C" kda_status kda_gated_delta_bwd(const kda_bf16* q, const kda_bf16* k, const kda_bf16* v, const kda_bf16* log_decay,
                                          const kda_bf16* beta, const int64_t* cu_seqlens_dev, const int64_t* cu_seqlens_host,
                                          int64_t num_seqs, int64_t B, int64_t T, int64_t Hqk, int64_t Hv, int64_t head_dim,
                                          float scale, const int64_t* strides, const kda_bf16* d_o, const float* d_hT,
                                          kda_bf16* dq, kda_bf16* dk, kda_bf16* dv, kda_bf16* dlog_decay, kda_bf16* dbeta,
                                          float* dh0, void* workspace, size_t workspace_bytes, int32_t* device_status,
                                          struct CUstream_st* stream) {
  return kda::guarded([&]() -> kda_status {
    kda::DeltaProblem P{};
    Span in[6];
    kda_status st = check(q, k, v, log_decay, beta, cu_seqlens_dev, cu_seqlens_host, num_seqs, B, T, Hqk, Hv, head_dim, scale, strides, &P, in);
    if (st != KDA_OK) return st;
    if (P.Ttot && (!d_o || !dq || !dk || !dv || !dbeta)) return fail(KDA_ERR_INVALID_ARGUMENT, "null gradient pointer");
    if (dlog_decay && !log_decay) return fail(KDA_ERR_INVALID_ARGUMENT, "no log_decay: dlog_decay must be NULL");
    if (((uintptr_t)d_o | (uintptr_t)d_hT | (uintptr_t)dq | (uintptr_t)dk | (uintptr_t)dv | (uintptr_t)dh0) & 15u)
      return fail(KDA_ERR_INVALID_ARGUMENT, "state, adjoint and gradient tensors must be 16-byte aligned");
    if (misaligned(dlog_decay, 2) || misaligned(dbeta, 2)) return fail(KDA_ERR_INVALID_ARGUMENT, kMisaligned);
    if ((st = check_workspace(P, workspace, workspace_bytes, true)) != KDA_OK) return st;
    const size_t states = 4 * (size_t)P.N * Hv * kda::kDim * kda::kDim, gates = 2 * (size_t)P.Ttot * Hv;
    const size_t tq = 2 * (size_t)P.Ttot * Hqk * kda::kDim, tv = gates * kda::kDim;
    const Span outs[] = {{dq, tq}, {dk, tq}, {dv, tv}, {dlog_decay, gates}, {dbeta, gates}, {dh0, states},
                         {workspace, workspace_bytes}, {device_status, 4}};
    const Span ins[] = {in[0], in[1], in[2], in[3], in[4], in[5], {d_o, tv}, {d_hT, states}};
    if (aliasing(outs, ins)) return fail(KDA_ERR_ALIASING, "an output overlaps an input or another output");
    if ((st = check_device(kOp, device_status, &g_delta_status, &P.status)) != KDA_OK) return st;
    kda::DeltaGrads G{};
    G.d_o = reinterpret_cast<const __nv_bfloat16*>(d_o);
    G.d_hT = d_hT;
    G.dq = reinterpret_cast<__nv_bfloat16*>(dq);
    G.dk = reinterpret_cast<__nv_bfloat16*>(dk);
    G.dv = reinterpret_cast<__nv_bfloat16*>(dv);
    G.dg = reinterpret_cast<__nv_bfloat16*>(dlog_decay);
    G.dbeta = reinterpret_cast<__nv_bfloat16*>(dbeta);
    G.dh0 = dh0;
    const cudaError_t e = kda::launch_delta_backward(P, G, workspace, stream);
    return e == cudaSuccess ? KDA_OK : fail(KDA_ERR_CUDA, cudaGetErrorString(e));
  });
}

extern "C" kda_status kda_gated_delta_prefill(const kda_bf16* q, const kda_bf16* k, const kda_bf16* v, const kda_bf16* log_decay,
                                              const kda_bf16* beta, const int64_t* cu_seqlens_dev, const int64_t* cu_seqlens_host,
                                              int64_t num_seqs, int64_t B, int64_t T, int64_t Hqk, int64_t Hv, int64_t head_dim,
                                              float scale, const int64_t* strides, void* state, int32_t state_dtype,
                                              const int32_t* state_indices, const int32_t* state_indices_host, int64_t num_slots,
                                              kda_bf16* o, void* workspace, size_t workspace_bytes, int32_t* device_status,
                                              struct CUstream_st* stream) {
  return kda::guarded([&]() -> kda_status {
    kda::DeltaProblem P{};
    Span in[6];
    kda_status st = check(q, k, v, log_decay, beta, cu_seqlens_dev, cu_seqlens_host, num_seqs, B, T, Hqk, Hv, head_dim, scale, strides, &P, in);
    if (st != KDA_OK) return st;
    if (!state || (P.Ttot && !o)) return fail(KDA_ERR_INVALID_ARGUMENT, "null tensor pointer");
    if (num_slots < 1) return fail(KDA_ERR_UNSUPPORTED, "the pool needs 1 to 2^31 slots");
    const Pool pool{state, state_dtype, state_indices, state_indices_host, num_slots};
    if ((st = check_pool(kOp, pool, P.N, Hv)) != KDA_OK) return st;
    if ((uintptr_t)o & 15u) return fail(KDA_ERR_INVALID_ARGUMENT, "state and output tensors must be 16-byte aligned");
    if ((st = check_workspace(P, workspace, workspace_bytes, false)) != KDA_OK) return st;
    const Span outs[] = {pool_span(pool, Hv), {o, 2 * (size_t)P.Ttot * Hv * kda::kDim}, {workspace, workspace_bytes}, {device_status, 4}};
    const Span ins[] = {in[0], in[1], in[2], in[3], in[4], in[5], {state_indices, 4 * (size_t)P.N}};
    if (aliasing(outs, ins)) return fail(KDA_ERR_ALIASING, "an output overlaps an input or another output");
    if ((st = check_device(kOp, device_status, &g_delta_status, &P.status)) != KDA_OK) return st;
    const kda::DecayStates S{state, state, state_dtype == KDA_STATE_BF16, state_indices, num_slots};
    const cudaError_t e = kda::launch_delta_forward(P, S, reinterpret_cast<__nv_bfloat16*>(o), false, workspace, stream);
    return e == cudaSuccess ? KDA_OK : fail(KDA_ERR_CUDA, cudaGetErrorString(e));
  });
}
