// kda_decay_scan.cu -- the linear attention with a decay for each head as its
// recurrence, token by token, in FP32:
//   forward   S_t = e^{g_t} S_{t-1} + v_t k_t^T,       o_t  = s S_t q_t
//   backward  G_t = e^{g_{t+1}} G_{t+1} + s do_t q_t^T, dk_t = G_t^T v_t, dv_t = G_t k_t,
//             dq_t = s S_t^T do_t  (S as in the forward)
// Every one of the four is a scan y_t = c M_t x_t over M_t = e^{g} M + b_t a_t^T with a row
// (or column) of M in each of a CTA's 128 threads. The decay's gradient follows from the
// others: a decay scales all that crosses its token,
//   dg_t = sum_{i >= t} (q_i . dq_i - k_i . dk_i) + <S_T, dS_T>.
#include "kda_decay.cuh"
#include "kda_layout.h"

namespace kda {
namespace {

constexpr int kBatch = 8;  // tokens staged at once

struct Src {
  const __nv_bfloat16* p;
  int64_t t, h;
  int div;  // head of the source: h / div
};

struct ScanArgs {
  Src a, b, x;
  float b_scale, y_scale;
  const void* m0;       // initial states or null
  void* m1;             // final states or null
  float* m1_copy;       // a second, FP32 copy of the final states (by sequence), or null
  int bf16, transposed; // state type; 1: thread i holds column i of the value-first state
  const int32_t* slots;
  int64_t num_slots;
  __nv_bfloat16* y;     // [Ttot, Hv, 128] or null
  float* y32;           // the same in FP32, or null
};

template <bool kRev>
__global__ void __launch_bounds__(128) kda_decay_scan_kernel(const DecayProblem P, const ScanArgs s) {
  __shared__ float as[kBatch][kDim], xs[kBatch][kDim], ds[kBatch];
  const int i = threadIdx.x;
  const int64_t n = blockIdx.x / P.Hv;
  const int h = (int)(blockIdx.x % P.Hv);
  const DecaySpan sp = decay_span(P, n);
  const int64_t slot = s.slots ? s.slots[n] : n;
  if (slot < 0 || slot >= s.num_slots) {
    if (i == 0) atomicOr(P.status, 4);
    return;
  }
  const int64_t base = (slot * P.Hv + h) * kDim * kDim;
  const int64_t row = s.transposed ? 1 : kDim, col = s.transposed ? kDim : 1;
  float m[kDim];
#pragma unroll
  for (int j = 0; j < kDim; ++j) {
    const int64_t at = base + i * row + j * col;
    m[j] = !s.m0 ? 0.f : s.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(s.m0)[at])
                                : reinterpret_cast<const float*>(s.m0)[at];
  }
  for (int64_t c = 0; c < sp.len; c += kBatch) {
    const int nb = (int)(sp.len - c < kBatch ? sp.len - c : kBatch);
    __syncthreads();
    for (int u = 0; u < nb; ++u) {
      const int64_t tok = sp.t0 + (kRev ? sp.len - 1 - c - u : c + u);
      as[u][i] = __bfloat162float(s.a.p[tok * s.a.t + (h / s.a.div) * s.a.h + i]);
      xs[u][i] = __bfloat162float(s.x.p[tok * s.x.t + (h / s.x.div) * s.x.h + i]);
      if (i == 0) ds[u] = exp2f(decay_log2(decay_g(P, tok, h)));
    }
    __syncthreads();
    for (int u = 0; u < nb; ++u) {
      const int64_t tok = sp.t0 + (kRev ? sp.len - 1 - c - u : c + u);
      const float b = s.b_scale * __bfloat162float(s.b.p[tok * s.b.t + (h / s.b.div) * s.b.h + i]);
      const float d = ds[u];
      float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kDim; ++j) {
        m[j] = kRev ? fmaf(as[u][j], b, m[j]) : fmaf(as[u][j], b, d * m[j]);
        y[j & 3] = fmaf(m[j], xs[u][j], y[j & 3]);
        if (kRev) m[j] *= d;
      }
      const float out = s.y_scale * ((y[0] + y[1]) + (y[2] + y[3]));
      const int64_t at = (tok * P.Hv + h) * kDim + i;
      if (s.y) s.y[at] = __float2bfloat16_rn(out);
      if (s.y32) s.y32[at] = out;
    }
  }
#pragma unroll
  for (int j = 0; j < kDim; ++j) {
    const int64_t at = i * row + j * col;
    if (s.m1 && s.bf16) reinterpret_cast<__nv_bfloat16*>(s.m1)[base + at] = __float2bfloat16_rn(m[j]);
    if (s.m1 && !s.bf16) reinterpret_cast<float*>(s.m1)[base + at] = m[j];
    if (s.m1_copy) s.m1_copy[(n * P.Hv + h) * kDim * kDim + at] = m[j];
  }
}

// dg of one (sequence, head): a warp walks the tokens from the last; the sums cancel, so FP64.
__global__ void __launch_bounds__(32) kda_decay_gate_grad_kernel(const DecayProblem P, const float* dq, const float* dk,
                                                                const float* hT, const float* dhT, __nv_bfloat16* dg) {
  const int lane = threadIdx.x;
  const int64_t n = blockIdx.x / P.Hv;
  const int h = (int)(blockIdx.x % P.Hv);
  const DecaySpan sp = decay_span(P, n);
  auto total = [](double x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  };
  double acc = 0.0;
  if (dhT) {
    const int64_t base = (n * P.Hv + h) * kDim * kDim;
    for (int j = lane; j < kDim * kDim; j += 32) acc += (double)hT[base + j] * dhT[base + j];
    acc = total(acc);
  }
  for (int64_t t = sp.len - 1; t >= 0; --t) {
    const int64_t tok = sp.t0 + t, at = (tok * P.Hv + h) * kDim;
    double x = 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = lane + 32 * j;
      x += (double)__bfloat162float(P.q[tok * P.qt + (h / P.r) * P.qh + d]) * dq[at + d] -
           (double)__bfloat162float(P.k[tok * P.kt + (h / P.r) * P.kh + d]) * dk[at + d];
    }
    acc += total(x);
    if (lane == 0) dg[tok * P.Hv + h] = __float2bfloat16_rn((float)acc);
  }
}

// Sums of a query/key head's value heads, rounded once.
__global__ void kda_decay_group_sum_kernel(const float* x, __nv_bfloat16* y, int64_t rows, int r) {
  const int64_t at = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (at >= rows * kDim) return;
  const int64_t row = at / kDim, d = at % kDim;
  float s = 0.f;
  for (int j = 0; j < r; ++j) s += x[(row * r + j) * kDim + d];
  y[at] = __float2bfloat16_rn(s);
}

struct Ws {
  size_t hT, dq, dk, total;
};
Ws carve(int64_t N, int64_t Ttot, int64_t Hv) {
  Ws w;
  w.hT = 0;
  w.dq = ctx_align_up(sizeof(float) * (size_t)N * Hv * kDim * kDim);
  w.dk = ctx_align_up(w.dq + sizeof(float) * (size_t)Ttot * Hv * kDim);
  w.total = ctx_align_up(w.dk + sizeof(float) * (size_t)Ttot * Hv * kDim);
  return w;
}

template <bool kRev>
cudaError_t scan(const DecayProblem& P, const ScanArgs& a, cudaStream_t s) {
  if (P.N * P.Hv == 0) return cudaSuccess;
  kda_decay_scan_kernel<kRev><<<(unsigned)(P.N * P.Hv), 128, 0, s>>>(P, a);
  return cudaGetLastError();
}

}  // namespace

size_t decay_workspace_bytes(int64_t N, int64_t Ttot, int64_t, int64_t Hv, int64_t seg, bool training) {
  return decay_forward_workspace(N, Ttot, Hv, seg) + (training ? carve(N, Ttot, Hv).total : 0);
}

cudaError_t launch_decay_backward(const DecayProblem& P, const float* h0, const DecayGrads& g, void* ws,
                                  cudaStream_t s) {
  const Ws w = carve(P.N, P.Ttot, P.Hv);
  char* base = reinterpret_cast<char*>(ws) + decay_forward_workspace(P.N, P.Ttot, P.Hv, P.seg);
  float* hT = reinterpret_cast<float*>(base + w.hT);
  float* dq = reinterpret_cast<float*>(base + w.dq);
  float* dk = reinterpret_cast<float*>(base + w.dk);
  const Src q{P.q, P.qt, P.qh, P.r}, k{P.k, P.kt, P.kh, P.r}, v{P.v, P.vt, P.vh, 1};
  const Src d{g.d_o, (int64_t)P.Hv * kDim, kDim, 1};
  ScanArgs a{};
  a.num_slots = P.N;
  // dq: columns of S, forward
  a.a = v; a.b = k; a.x = d;
  a.b_scale = 1.f; a.y_scale = P.scale;
  a.m0 = h0; a.transposed = 1; a.y32 = dq;
  cudaError_t e = scan<false>(P, a, s);
  if (e != cudaSuccess) return e;
  // dk: columns of G, backwards in time
  a.a = d; a.b = q; a.x = v;
  a.b_scale = P.scale; a.y_scale = 1.f;
  a.m0 = g.d_hT; a.y32 = dk;
  if ((e = scan<true>(P, a, s)) != cudaSuccess) return e;
  // dv and dh0: rows of G
  a.a = q; a.b = d; a.x = k;
  a.transposed = 0; a.m1 = g.dh0; a.y32 = nullptr; a.y = g.dv;
  if ((e = scan<true>(P, a, s)) != cudaSuccess) return e;
  if (P.Ttot == 0) return cudaSuccess;
  if (g.dg) {
    kda_decay_gate_grad_kernel<<<(unsigned)(P.N * P.Hv), 32, 0, s>>>(P, dq, dk, hT, g.d_hT, g.dg);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const int64_t rows = P.Ttot * P.Hqk;
  const unsigned grid = (unsigned)((rows * kDim + 255) / 256);
  kda_decay_group_sum_kernel<<<grid, 256, 0, s>>>(dq, g.dq, rows, P.r);
  kda_decay_group_sum_kernel<<<grid, 256, 0, s>>>(dk, g.dk, rows, P.r);
  return cudaGetLastError();
}

}  // namespace kda
