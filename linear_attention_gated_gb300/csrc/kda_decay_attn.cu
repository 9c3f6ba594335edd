// kda_decay_attn.cu -- host side of the linear attention with a decay for each
// head: argument checks, workspace sizes and launches of kda_decay_attn_fwd,
// kda_decay_attn_bwd and kda_decay_attn_prefill. Nothing is allocated here.
#include "../../include/kda.h"
#include "kda_decay.cuh"
#include "kda_host.h"

#include <cmath>
#include <cstdio>

namespace {

__device__ int32_t g_decay_status;

kda_status fail(kda_status st, const char* what) {
  char buf[256];
  snprintf(buf, sizeof(buf), "decay_attn: %s", what);
  kda::set_last_error(buf);
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

template <size_t NO, size_t NI>
bool aliasing(const Span (&outs)[NO], const Span (&ins)[NI]) {
  for (size_t i = 0; i < NO; ++i) {
    for (const Span& in : ins)
      if (overlap(in, outs[i])) return true;
    for (size_t j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

struct Shape {
  int64_t N, Ttot, seg, longest;
};

kda_status check_shape(int64_t B, int64_t T, int64_t Hqk, int64_t Hv, const int64_t* cu, int64_t num_seqs, Shape* s) {
  if (B < 1 || T < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "B must be >= 1 and T >= 0");
  if (Hqk < 1 || Hv < 1 || Hv % Hqk) return fail(KDA_ERR_INVALID_ARGUMENT, "Hv must be a positive multiple of Hqk");
  if (kda::size_limit_violation(B, T ? T : 1, Hv, 0))
    return fail(KDA_ERR_UNSUPPORTED, "problem too large (over 2^40 tokens or token-heads, or 2^20 heads)");
  s->Ttot = B * T;
  s->N = B;
  if (cu) {
    if (B != 1) return fail(KDA_ERR_INVALID_ARGUMENT, "packed input needs a physical batch of one");
    if (num_seqs < 1) return fail(KDA_ERR_INVALID_ARGUMENT, "packed input needs num_seqs >= 1");
    if (cu[0] != 0 || cu[num_seqs] != T) return fail(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens must run from 0 to T");
    for (int64_t i = 0; i < num_seqs; ++i)
      if (cu[i + 1] < cu[i]) return fail(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens decreases");
    s->N = num_seqs;
  }
  if (s->N > INT32_MAX / Hv) return fail(KDA_ERR_UNSUPPORTED, "too many (sequence, head) units");
  if (s->Ttot >= INT32_MAX) return fail(KDA_ERR_UNSUPPORTED, "problem too large (2^31 tokens)");
  s->longest = cu ? 0 : T;
  for (int64_t i = 0; cu && i < s->N; ++i)
    if (cu[i + 1] - cu[i] > s->longest) s->longest = cu[i + 1] - cu[i];
  s->seg = kda::decay_segment_tokens(cu, s->N, T, Hv);
  return KDA_OK;
}

// Fills and checks what the three entry points share. strides: token and head strides (elements) of
// q, k, v, or null for contiguous tensors. spans: the bytes that q, k, v and the decays take.
kda_status check_tokens(const void* q, const void* k, const void* v, const void* g, int32_t per_token,
                        const int64_t* cu_dev, const int64_t* cu_host, int64_t num_seqs, int64_t B, int64_t T,
                        int64_t Hqk, int64_t Hv, int64_t head_dim, float scale, const int64_t* strides,
                        kda::DecayProblem* P, Span (&spans)[5]) {
  if ((cu_dev == nullptr) != (cu_host == nullptr))
    return fail(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens needs its host mirror (and the reverse)");
  Shape s{};
  const kda_status st = check_shape(B, T, Hqk, Hv, cu_host, num_seqs, &s);
  if (st != KDA_OK) return st;
  if (head_dim != kda::kDim) return fail(KDA_ERR_UNSUPPORTED, "head_dim must be 128");
  if (per_token != 0 && per_token != 1) return fail(KDA_ERR_INVALID_ARGUMENT, "decay_per_token must be 0 or 1");
  if (std::isinf(scale)) return fail(KDA_ERR_INVALID_ARGUMENT, "scale must be finite (NaN selects 1/sqrt(128))");
  if ((!g && (s.Ttot || !per_token)) || (s.Ttot && (!q || !k || !v))) return fail(KDA_ERR_INVALID_ARGUMENT, "null tensor pointer");
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v) & 15u)
    return fail(KDA_ERR_INVALID_ARGUMENT, "token tensors must be 16-byte aligned");
  const int64_t D = kda::kDim;
  int64_t x[6] = {Hqk * D, D, Hqk * D, D, Hv * D, D};
  if (strides)
    for (int i = 0; i < 6; ++i) x[i] = strides[i];
  const int64_t heads[3] = {Hqk, Hqk, Hv};
  const void* ptrs[3] = {q, k, v};
  for (int i = 0; i < 3; ++i) {
    const int64_t ts = x[2 * i], hs = x[2 * i + 1];
    bool too_large;
    if (!kda::view_rows_apart(s.Ttot, heads[i], D, ts, hs, &too_large) || hs % 8 || ts % 8)
      return fail(KDA_ERR_INVALID_ARGUMENT, "token and head strides must be multiples of 8 elements and keep rows apart");
    if (too_large || ts > (int64_t(1) << 38)) return fail(KDA_ERR_UNSUPPORTED, "strides too large");
    spans[i] = Span{ptrs[i], s.Ttot ? 2 * (size_t)((s.Ttot - 1) * ts + (heads[i] - 1) * hs + D) : 0};
  }
  spans[3] = Span{g, per_token ? 2 * (size_t)s.Ttot * Hv : 4 * (size_t)Hv};
  spans[4] = Span{cu_dev, cu_dev ? 8 * (size_t)(s.N + 1) : 0};
  P->q = reinterpret_cast<const __nv_bfloat16*>(q);
  P->k = reinterpret_cast<const __nv_bfloat16*>(k);
  P->v = reinterpret_cast<const __nv_bfloat16*>(v);
  P->g = g;
  P->cu = cu_dev;
  P->qt = x[0]; P->qh = x[1]; P->kt = x[2]; P->kh = x[3]; P->vt = x[4]; P->vh = x[5];
  P->N = s.N;
  P->T = T;
  P->Ttot = s.Ttot;
  P->Hqk = (int)Hqk;
  P->Hv = (int)Hv;
  P->r = (int)(Hv / Hqk);
  P->per_token = per_token;
  P->seg = s.seg;
  P->longest = s.longest;
  P->cu_host = cu_host;
  P->scale = std::isnan(scale) ? 1.0f / std::sqrt(128.0f) : scale;
  return KDA_OK;
}

kda_status check_workspace(const kda::DecayProblem& P, void* ws, size_t bytes, bool training) {
  const size_t need = kda::decay_workspace_bytes(P.N, P.Ttot, P.Hqk, P.Hv, P.seg, training, P.per_token);
  if (need && (!ws || bytes < need))
    return fail(KDA_ERR_WORKSPACE_TOO_SMALL, "workspace below kda_decay_attn_workspace_bytes()");
  if ((uintptr_t)ws & 255u) return fail(KDA_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
  return KDA_OK;
}

kda_status check_device(int32_t* device_status, int32_t** status) {
  int dev = -1, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e != cudaSuccess) return fail(KDA_ERR_CUDA, cudaGetErrorString(e));
  if (major != 10 || minor != 3) return fail(KDA_ERR_UNSUPPORTED, "kernels are built for sm_103a");
  *status = device_status;
  if (!device_status && (e = cudaGetSymbolAddress(reinterpret_cast<void**>(status), g_decay_status)) != cudaSuccess)
    return fail(KDA_ERR_CUDA, cudaGetErrorString(e));
  return KDA_OK;
}

}  // namespace

extern "C" kda_status kda_decay_attn_workspace_bytes(int64_t B, int64_t T, int64_t Hqk, int64_t Hv,
                                                     const int64_t* cu_seqlens_host, int64_t num_seqs,
                                                     int32_t decay_per_token, int32_t training, size_t* bytes) {
  return kda::guarded([&]() -> kda_status {
    if (!bytes) return fail(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    Shape s{};
    const kda_status st = check_shape(B, T, Hqk, Hv, cu_seqlens_host, num_seqs, &s);
    if (st != KDA_OK) return st;
    *bytes = kda::decay_workspace_bytes(s.N, s.Ttot, Hqk, Hv, s.seg, training != 0, decay_per_token != 0);
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
