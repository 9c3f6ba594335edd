// kda_decay_host.h -- host-side checks shared by the entry points of the linear attention with a decay for each head and of
// the gated delta rule. `op` names the operator in the messages.
#pragma once

#include <cmath>
#include <cstdio>

#include "../../include/kda.h"
#include "kda_decay.cuh"
#include "kda_host.h"

namespace kda {
namespace host {

inline kda_status fail(const char* op, kda_status st, const char* what) {
  char buf[256];
  snprintf(buf, sizeof(buf), "%s: %s", op, what);
  set_last_error(buf);
  return st;
}

// (device pointers: a kernel that reads through one that is not aligned to its elements faults)
inline bool misaligned(const void* p, size_t to) { return ((uintptr_t)p & (to - 1)) != 0; }
constexpr const char* kMisaligned = "tensors must be aligned to their elements";

struct Span {
  const void* p;
  size_t bytes;
};

inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a.p && b.p && a.bytes && b.bytes && a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

template <size_t NO, size_t NI>
inline bool aliasing(const Span (&outs)[NO], const Span (&ins)[NI]) {
  for (size_t i = 0; i < NO; ++i) {
    for (const Span& in : ins)
      if (overlap(in, outs[i])) return true;
    for (size_t j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

struct Shape {
  int64_t N, Ttot, longest;
};

inline kda_status check_shape(const char* op, int64_t B, int64_t T, int64_t Hqk, int64_t Hv, const int64_t* cu, int64_t num_seqs, Shape* s) {
  if (B < 1 || T < 0) return fail(op, KDA_ERR_INVALID_ARGUMENT, "B must be >= 1 and T >= 0");
  if (Hqk < 1 || Hv < 1 || Hv % Hqk) return fail(op, KDA_ERR_INVALID_ARGUMENT, "Hv must be a positive multiple of Hqk");
  if (size_limit_violation(B, T ? T : 1, Hv, 0))
    return fail(op, KDA_ERR_UNSUPPORTED, "problem too large (over 2^40 tokens or token-heads, or 2^20 heads)");
  s->Ttot = B * T;
  s->N = B;
  if (cu) {
    if (B != 1) return fail(op, KDA_ERR_INVALID_ARGUMENT, "packed input needs a physical batch of one");
    if (num_seqs < 1) return fail(op, KDA_ERR_INVALID_ARGUMENT, "packed input needs num_seqs >= 1");
    if (cu[0] != 0 || cu[num_seqs] != T) return fail(op, KDA_ERR_INVALID_ARGUMENT, "cu_seqlens must run from 0 to T");
    for (int64_t i = 0; i < num_seqs; ++i)
      if (cu[i + 1] < cu[i]) return fail(op, KDA_ERR_INVALID_ARGUMENT, "cu_seqlens decreases");
    s->N = num_seqs;
  }
  if (s->N > INT32_MAX / Hv) return fail(op, KDA_ERR_UNSUPPORTED, "too many (sequence, head) units");
  if (s->Ttot >= INT32_MAX) return fail(op, KDA_ERR_UNSUPPORTED, "problem too large (2^31 tokens)");
  s->longest = cu ? 0 : T;
  for (int64_t i = 0; cu && i < s->N; ++i)
    if (cu[i + 1] - cu[i] > s->longest) s->longest = cu[i + 1] - cu[i];
  return KDA_OK;
}

// Fills and checks what the entry points share (but P->seg). strides: token and head strides (elements) of q, k, v, or null
// for contiguous tensors. spans: the bytes that q, k, v, the decays and the offsets take. decays: null ones are refused.
inline kda_status check_tokens(const char* op, const void* q, const void* k, const void* v, const void* g, bool decays, int32_t per_token,
                               const int64_t* cu_dev, const int64_t* cu_host, int64_t num_seqs, int64_t B, int64_t T,
                               int64_t Hqk, int64_t Hv, int64_t head_dim, float scale, const int64_t* strides,
                               DecayProblem* P, Span (&spans)[5]) {
  if ((cu_dev == nullptr) != (cu_host == nullptr))
    return fail(op, KDA_ERR_INVALID_ARGUMENT, "cu_seqlens needs its host mirror (and the reverse)");
  Shape s{};
  const kda_status st = check_shape(op, B, T, Hqk, Hv, cu_host, num_seqs, &s);
  if (st != KDA_OK) return st;
  if (head_dim != kDim) return fail(op, KDA_ERR_UNSUPPORTED, "head_dim must be 128");
  if (per_token != 0 && per_token != 1) return fail(op, KDA_ERR_INVALID_ARGUMENT, "decay_per_token must be 0 or 1");
  if (std::isinf(scale)) return fail(op, KDA_ERR_INVALID_ARGUMENT, "scale must be finite (NaN selects 1/sqrt(128))");
  if ((decays && !g && (s.Ttot || !per_token)) || (s.Ttot && (!q || !k || !v))) return fail(op, KDA_ERR_INVALID_ARGUMENT, "null tensor pointer");
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v) & 15u)
    return fail(op, KDA_ERR_INVALID_ARGUMENT, "token tensors must be 16-byte aligned");
  if (misaligned(g, per_token ? 2 : 4) || misaligned(cu_dev, 8)) return fail(op, KDA_ERR_INVALID_ARGUMENT, kMisaligned);
  const int64_t D = kDim;
  int64_t x[6] = {Hqk * D, D, Hqk * D, D, Hv * D, D};
  if (strides)
    for (int i = 0; i < 6; ++i) x[i] = strides[i];
  const int64_t heads[3] = {Hqk, Hqk, Hv};
  const void* ptrs[3] = {q, k, v};
  for (int i = 0; i < 3; ++i) {
    const int64_t ts = x[2 * i], hs = x[2 * i + 1];
    bool too_large;
    if (!view_rows_apart(s.Ttot, heads[i], D, ts, hs, &too_large) || hs % 8 || ts % 8)
      return fail(op, KDA_ERR_INVALID_ARGUMENT, "token and head strides must be multiples of 8 elements and keep rows apart");
    if (too_large || ts > (int64_t(1) << 38)) return fail(op, KDA_ERR_UNSUPPORTED, "strides too large");
    spans[i] = Span{ptrs[i], s.Ttot ? 2 * (size_t)((s.Ttot - 1) * ts + (heads[i] - 1) * hs + D) : 0};
  }
  spans[3] = Span{g, !g ? 0 : per_token ? 2 * (size_t)s.Ttot * Hv : 4 * (size_t)Hv};
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
  P->longest = s.longest;
  P->cu_host = cu_host;
  P->scale = std::isnan(scale) ? 1.0f / std::sqrt(128.0f) : scale;
  return KDA_OK;
}

// A state pool of `num_slots` slots and the slots of N sequences (indices null: slot n).
struct Pool {
  const void* state;
  int32_t dtype;
  const int32_t* idx;
  const int32_t* idx_host;
  int64_t slots;
};
inline kda_status check_pool(const char* op, const Pool& p, int64_t N, int64_t Hv) {
  if (p.dtype != KDA_STATE_BF16 && p.dtype != KDA_STATE_FP32)
    return fail(op, KDA_ERR_INVALID_ARGUMENT, "state_dtype must be KDA_STATE_BF16 or KDA_STATE_FP32");
  if (p.slots < 0 || p.slots > (int64_t(1) << 31) || pool_too_large(p.slots, Hv))
    return fail(op, KDA_ERR_UNSUPPORTED, "more than 2^31 pool slots or 2^40 states");
  if ((uintptr_t)p.state & 15u) return fail(op, KDA_ERR_INVALID_ARGUMENT, "state and output tensors must be 16-byte aligned");
  if (misaligned(p.idx, 4)) return fail(op, KDA_ERR_INVALID_ARGUMENT, kMisaligned);
  if ((p.idx == nullptr) != (p.idx_host == nullptr))
    return fail(op, KDA_ERR_INVALID_ARGUMENT, "state_indices needs its host mirror (and the reverse)");
  if (p.idx_host) {
    const int fault = slot_fault(p.idx_host, N, p.slots);
    if (fault == 1) return fail(op, KDA_ERR_INVALID_ARGUMENT, "state index out of range");
    if (fault == 2) return fail(op, KDA_ERR_INVALID_ARGUMENT, "two sequences share a state slot");
  } else if (p.slots < N) {
    return fail(op, KDA_ERR_INVALID_ARGUMENT, "without state_indices the pool needs a slot per sequence");
  }
  return KDA_OK;
}
inline Span pool_span(const Pool& p, int64_t Hv) {
  return Span{p.state, (p.dtype == KDA_STATE_BF16 ? 2 : 4) * (size_t)p.slots * Hv * kDim * kDim};
}

// The device is one that the kernels are built for; *status: the caller's word, or the library's `own` one.
inline kda_status check_device(const char* op, int32_t* device_status, const void* own, int32_t** status) {
  if (misaligned(device_status, 4)) return fail(op, KDA_ERR_INVALID_ARGUMENT, kMisaligned);
  int dev = -1, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e != cudaSuccess) return fail(op, KDA_ERR_CUDA, cudaGetErrorString(e));
  if (major != 10 || minor != 3) return fail(op, KDA_ERR_UNSUPPORTED, "kernels are built for sm_103a");
  *status = device_status;
  if (!device_status && (e = cudaGetSymbolAddress(reinterpret_cast<void**>(status), own)) != cudaSuccess)
    return fail(op, KDA_ERR_CUDA, cudaGetErrorString(e));
  return KDA_OK;
}

}  // namespace host
}  // namespace kda
