// kda_decay_pass.cu -- the chunked pass of the linear attention with a decay for
// each head, on sm_103a tensor cores: one kernel for the forward and for the three
// passes of the backward.
//
// With roles Q, K, V (token tensors) and a state S [V dims, K dims] per (sequence, head), it computes
// for chunks of C = 64 tokens, b_i the sum of the chunk's log decays up to token i,
//   Y^T = S Q^T diag(e^{b_i}) + V^T P^T,   P_ij = e^{b_i - b_j} q_i . k_j  (j <= i)
//   S  <- e^{b_C} S + V^T K~,              K~_j = e^{b_C - b_j} k_j
// and backwards in time (last chunk first), where S is the adjoint of the state after the first token of the
// chunk done before, c_i the sum of the log decays from token i + 1 up to and with that token, and b_i the sum
// from the chunk's second token up to i,
//   Y^T = S Q^T diag(e^{c_i}) + V^T P^T,   P_ij = e^{b_j - b_i} q_i . k_j  (j >= i)
//   S  <- e^{c_1} S + V^T K~,              K~_j = e^{b_j} k_j
// All exponents are <= 0 and the largest factor in K~ is 1, so nothing overflows, and nothing that counts
// underflows, for any decay.
//   o :  Q = q,  K = k,  V = v     forward,   S = the state                      (value first)
//   dq:  Q = do, K = v,  V = k     forward,   S = the state, transposed
//   dk:  Q = v,  K = do, V = q     backwards, S = the state's adjoint, transposed
//   dv:  Q = k,  K = q,  V = do    backwards, S = the state's adjoint            (its end is dh0)
// Nothing is saved by the forward: what the backward needs of the states it carries again, from the 48 KiB of a
// chunk's three tiles, which a pass reads anyway. A state stored and read for every chunk would be 128 KiB more.
//
// One CTA an SM, 20 warps with roles, so that the copies, the products and the element-wise work of
// neighbouring chunks (and units) run side by side; only the state's update is a chain.
//   warp 0   copies: Q, K, V tiles by tiled copies (128-byte swizzle), three stages; the next unit's
//            number (cluster launch control: the grid has a CTA for each unit and a running CTA takes
//            over the next one that has not started)
//   warps 1, 3   products (tcgen05.mma kind::f16, BF16 operands, FP32 accumulators in tensor memory): scores and U;
//            S Q^T and V^T P^T. Starting a product takes as long as the tensor core is busy with the ones
//            before, so two warps start them: while one waits for an operand, the other's products run
//   warp 2   decays of each chunk: sums from both ends, so that the exponents that matter most in
//            each, the small ones, are sums of few terms
//   warps 4-11   K~ (over K and beside) and P
//   warps 12-19  the state, 64 of a row's 128 values a thread in registers, S = e^{b_C} S + U with U = V^T K~
//            from tensor memory, and as A operand back there; Y
// K~ is an operand in two BF16 parts, hi + lo, 16 mantissa bits: FP32 states are off by 2.4e-6 relative to 64 bits
// (FP32 arithmetic throughout: 2e-7), and by one FP32 rounding a chunk of what they were before (StateFactor). One part would
// leave 1.7e-3; a third would take 16 KiB of shared memory that is not there and a quarter more of the products' time.
// P and S, which feed Y alone, are rounded to BF16 once (as Y itself is) where Y is an output: o and dv (dq and dk too with
// fixed decays and no groups) are off by 2.4e-3 where one rounding of the exact value leaves 1.7e-3. Where Y is FP32 and summed further, over heads or, for the
// decays' gradient, over the sequence, so that errors of its terms would outlive a cancelling sum, they too are in two
// parts (kSplit); it costs 68 us against 56 in a pass over 4 x 2048 tokens of 32 heads.
// A unit is one (sequence, head), longest sequences first (24 sequences of 1 to 4000 tokens, 64 heads: 540 us, in
// index order 594), or one segment of it.
//
// What bounds it: shared memory's data pipe, which the products' operands (34 % of a chunk's some 3150 cycles), the
// element-wise loads and stores (39 %, and 7 % for the turns they lose to the others) and the copies (15 %) share.
// The tensor core is busy for a third, HBM would take half. Three stages of 48 KiB, two places of K~ and P and (one
// part) of S overlap the chains K~ -> U -> state -> S Q^T -> Y and scores -> P -> V^T P^T of neighbouring chunks.
// Measured: 1.6 us a chunk and SM. 8 x 1024 tokens of
// 96 heads (856 MB): 167 us, 5.1 TB/s, 77 % of the copy rate, of which the 8 units beyond 5 an SM take a tenth;
// 24 sequences, 45 k tokens of 64 heads: 481 us, 1.85 GB, 3.9 TB/s. Tried and slower: 24, 28 and 32 warps with other
// shares of the roles (195 to 232 us against 170 at the time), Y copied out by each warp for its part or by the copying
// warp (+5 %), tiles prefetched to L2 (+13 %).
//
// Long axis, few units: each sequence is cut into segments. A first pass runs the state part alone
// over every segment but the last in time, a small kernel chains the segments' states, and
// the main pass starts every segment from its state: 32771 tokens of 32 heads 99 + 11 + 176 us (whole: 763).
#include <algorithm>

#include "kda_decay.cuh"
#include "kda_layout.h"
#include "kda_tma.h"
#include "tc.cuh"

namespace kda {
namespace {

constexpr int kC = kDecayChunk;
constexpr int kTiles = 9, kStages = 4, kDecs = 8, kRing = 4;
constexpr int kWarpLoad = 0, kWarpMma = 1, kWarpDecay = 2, kWarpMma2 = 3, kWarpA = 4, kWarpB = 12;
constexpr int kGroup = 8;                  // warps of A and of B
constexpr int kThreads = 32 * 20;
// Registers a thread of the control, A and B warps (setmaxnreg): 128 x 48 + 256 x 72 + 256 x 144 (kSplit: 64 and 152) = 61,440, all of the
// 640 x 96 = 61,440 the block is launched with (a split above that would wait for ever).
constexpr uint32_t kTile = kC * kDim * 2;  // bytes of a Q, K or V tile
constexpr uint32_t kPanel = kC * 128;      // bytes of its 64-element half
constexpr uint32_t kColU = 0;              // U: 128 columns (in the pass over states alone, 128 more in the next one's place)
constexpr uint32_t kColS = 128;            // the state as A operand, 64 + 64: its high and low BF16 parts, or (one part)
                                           // that of two chunks
constexpr uint32_t kColO = 256;            // S Q^T, then V^T P^T: 64 + 64
constexpr uint32_t kColP = 384;            // scores (M = 64) of two chunks: 64 + 64

// One unit of work.
struct Unit {
  int64_t n, t0, len, nchunks, end;  // sequence, first token, tokens and chunks of the unit; the sequence's end
  int64_t slot, sslot;               // of its state, and of its segment's
  int h;
  bool run;   // there is something to do
  bool last;  // the last segment in time order of the pass
  bool none;  // no unit: the end
};

struct Smem {
  unsigned char tile[kTiles][kTile];      // stages of Q, K, V
  unsigned char lo[2][kTile];             // low parts of K~
  unsigned char P[2][kC * kC * 2];
  unsigned char extra[kTile];             // in two parts: the low parts of P (twice 8 KiB); else: Y on its way out
  float b[kDecs][kC];    // cumulative log2 decay of the chunk
  float eb[kDecs][kC];   // factor of S q_i
  float w[kDecs][kC];    // factor of k_j in K~
  float lam[kDecs];      // e^{b_C}
  uint4 clc;             // response: the next unit
  Unit ring[kRing];      // units to come
  // full, empty: a stage's tiles are there / read by all products; dec, decfree: a chunk's decays are there / read by the last who does; g0, gu, gy, gq: products done
  // (scores, U, Y, its S Q^T in two parts); kready, pready: K~, P are there; ufree, yfree: U, Y are read; sready: the state is there
  unsigned long long full[kStages], empty[kStages], dec[kDecs], decfree[kDecs], g0[2], gu[2], gy, gq, kready[2], pready[2], ufree[2], sready[2], yfree;
  unsigned long long clcbar, rfull[kRing], rempty[kRing];
  uint32_t tmem;
};
constexpr int kSmemBytes = (int)sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

struct Maps {
  CUtensorMap q, k, v, y;
};

struct Segments {
  int64_t len;       // tokens of a segment (a multiple of kC), 0: sequences are not cut
  int most;          // most segments of a sequence
  float* state;      // [slots, H, 128, 128]: the segments' own states, then their initial states
  float* decay;      // [slots, H]: log2 of a segment's decay
};
// Slot of a sequence's first segment: floor(t0 / len) + n leaves each sequence ceil(len_n / len) slots.
__device__ __forceinline__ int64_t seg_slot(const Segments& g, int64_t t0, int64_t n) { return t0 / g.len + n; }

constexpr int kOrder = 512;      // sequences whose order is passed (more run in index order, whole)
constexpr int kUnits = 2 * kSms;  // the units that a cut aims at: two for each SM, so no sequence has more segments

struct PassArgs {
  DecayProblem P;
  int qdiv, kdiv, vdiv;               // head of a role's tensor: h / div
  float s_inter, s_intra, s_w;        // scales of S q, of P and of K~
  DecayStates st;
  int transposed;                     // S is the stored state transposed
  Segments sg;
  __nv_bfloat16* y;                   // [Ttot, Hv, 128], or
  float* y32;
  int ordered;
  uint16_t order[kOrder];             // longest sequence first
  int32_t first[kUnits + 1];       // segments s of the sequences that have one: pairs first[s] .. first[s + 1] - 1
};

template <bool kRev, bool kState>
__device__ __forceinline__ Unit unit_of(const PassArgs& a, int u) {
  const DecayProblem& P = a.P;
  Unit x;
  const int64_t p = u / P.Hv;
  x.h = u - (int)(p * P.Hv);
  int64_t seg = 0;
  if (a.sg.len)
    while (seg + 1 < a.sg.most && p >= a.first[seg + 1]) ++seg;
  x.n = a.sg.len ? p - a.first[seg] : p;
  if (a.ordered) x.n = a.order[x.n];
  const DecaySpan sp = decay_span(P, x.n);
  x.t0 = sp.t0;
  x.len = sp.len;
  x.end = sp.t0 + sp.len;
  x.slot = a.st.slots ? a.st.slots[x.n] : x.n;
  x.sslot = 0;
  x.last = true;
  x.run = x.slot >= 0 && x.slot < a.st.num_slots;
  if (a.sg.len) {
    const int64_t from = seg * a.sg.len;
    x.sslot = seg_slot(a.sg, sp.t0, x.n) + seg;
    const bool tail = from + a.sg.len >= sp.len;
    x.last = kRev ? seg == 0 : tail;
    if ((seg > 0 && from >= sp.len) || (kState && x.last)) x.run = false;
    x.t0 += from;
    x.len = tail ? sp.len - from : a.sg.len;
  }
  x.nchunks = x.run ? (x.len + kC - 1) / kC : 0;
  x.none = false;
  return x;
}

// kRev: backwards in time. kState: the first pass over segments (states alone). kSplit: P and S in two
// BF16 parts and Y in FP32.
template <bool kRev, bool kState, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
kda_decay_pass_kernel(const __grid_constant__ Maps maps, const __grid_constant__ PassArgs a) {
  extern __shared__ unsigned char raw_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem + ((1024 - (tc::smem_u32(raw_smem) & 1023)) & 1023));
  const DecayProblem& P = a.P;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [](unsigned long long& b) { return tc::smem_u32(&b); };
  // Stages of copies, and a stage's tile of Q (0), K (1) or V (2). The pass over states alone has no Q and four stages:
  // it takes a stage in half the time.
  constexpr uint32_t kSt = kState ? 4 : 3;
  auto tile = [&](uint32_t s, int x) -> unsigned char* { return sm.tile[kState ? 2 * s + x - 1 : 3 * s + x]; };

  if (warp == kWarpMma) tc::tmem_alloc(tc::smem_u32(&sm.tmem), 512);
  if (tid == 0) {
    for (uint32_t i = 0; i < kSt; ++i) { tc::mbar_init(bar(sm.full[i]), 1); tc::mbar_init(bar(sm.empty[i]), kState ? 1 : 2); }
    for (int i = 0; i < kDecs; ++i) {
      tc::mbar_init(bar(sm.dec[i]), 1);
      tc::mbar_init(bar(sm.decfree[i]), kGroup);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(sm.g0[i]), 1);
      tc::mbar_init(bar(sm.gu[i]), 1);
      tc::mbar_init(bar(sm.ufree[i]), kGroup);
      tc::mbar_init(bar(sm.kready[i]), kGroup);
      tc::mbar_init(bar(sm.pready[i]), kGroup);
      tc::mbar_init(bar(sm.sready[i]), kGroup);
    }
    tc::mbar_init(bar(sm.gy), 1);
    tc::mbar_init(bar(sm.gq), 1);
    tc::mbar_init(bar(sm.yfree), kGroup);
    tc::mbar_init(bar(sm.clcbar), 1);
    for (int i = 0; i < kRing; ++i) { tc::mbar_init(bar(sm.rfull[i]), 1); tc::mbar_init(bar(sm.rempty[i]), (kState ? 2 : 3) + 2 * kGroup); }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = sm.tmem;
  bool ok = true;  // false: a wait gave up; the warp touches only its own CTA's memory and leaves

  // U of chunk k: its place (the pass over states alone has two, so that one is read while the other is summed) and parity
  auto uplace = [](uint32_t k) { return kState ? k & 1 : 0u; };
  auto uphase = [](uint32_t k) { return kState ? (k >> 1) & 1 : k & 1; };

  // The ring of units, as a consumer (a warp): its place, and the next unit (false: none).
  uint32_t ur = 0;
  auto next_unit = [&](Unit& x) {
    if (ok) ok = tc::mbar_wait_lanes(bar(sm.rfull[ur % kRing]), (ur / kRing) & 1);
    if (!ok) return false;
    x = sm.ring[ur % kRing];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar(sm.rempty[ur % kRing]));
    ++ur;
    return !x.none;
  };
  // A consumer that sees chunks alone: is there one more, `left` those of the unit at hand?
  auto any_chunk = [&](int64_t& left) {
    Unit x;
    while (left == 0) {
      if (!next_unit(x)) return false;
      left = x.nchunks;
    }
    return true;
  };
  auto arrive = [&](unsigned long long& b) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar(b));
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == kWarpLoad) {
      // ================= units and copies
      uint32_t g = 0;  // chunks so far
      uint32_t asked = 0;
      auto push = [&](const Unit& x) {
        if (ok && ur >= kRing) ok = tc::mbar_wait_lanes(bar(sm.rempty[ur % kRing]), (ur / kRing - 1) & 1);
        if (ok && lane == 0) {
          sm.ring[ur % kRing] = x;
          tc::mbar_arrive(bar(sm.rfull[ur % kRing]));
        }
        __syncwarp();
        ++ur;
      };
      auto ask = [&] {  // for the next unit
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(bar(sm.clcbar), 16);
          asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                       ::"r"(tc::smem_u32(&sm.clc)), "r"(bar(sm.clcbar)) : "memory");
        }
        __syncwarp();
      };
      Unit x = unit_of<kRev, kState>(a, (int)blockIdx.x), next;
      push(x);
      ask();
      for (;;) {
        next.none = true;
        for (int64_t c = 0;; ++c) {
          if (c == (x.nchunks < kSt ? x.nchunks : kSt)) {
            // the next unit, told to everybody while this one's first chunks are under way
            const bool came = tc::mbar_wait_lanes(bar(sm.clcbar), asked & 1);
            ++asked;
            ok = ok && came;
            uint32_t more = 0, nx = 0;
            if (came) {
              asm volatile(
                  "{\n .reg .b128 r;\n .reg .pred p;\n ld.shared.b128 r, [%2];\n"
                  " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
                  " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
                  : "=r"(more), "=r"(nx) : "r"(tc::smem_u32(&sm.clc)) : "memory");
              tc::fence_async_smem();  // read before the next response is written
            }
            __syncwarp();
            if (more) next = unit_of<kRev, kState>(a, (int)nx);
            push(next);
            if (ok && more) ask();
          }
          if (!ok || c == x.nchunks) break;
          const int s = g % kSt;
          if (g >= kSt) ok = tc::mbar_wait_lanes(bar(sm.empty[s]), (g / kSt - 1) & 1);
          if (!ok) break;
          if (lane == 0) {
            const int t = (int)(x.t0 + (kRev ? x.nchunks - 1 - c : c) * kC);
            tc::mbar_arrive_expect_tx(bar(sm.full[s]), (kState ? 2 : 3) * kTile);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              tc::tma_load3(tc::smem_u32(tile(s, 1)) + p * kPanel, &maps.k, 64 * p, x.h / a.kdiv, t, bar(sm.full[s]));
              if (!kState)
                tc::tma_load3(tc::smem_u32(tile(s, 0)) + p * kPanel, &maps.q, 64 * p, x.h / a.qdiv, t, bar(sm.full[s]));
              tc::tma_load3(tc::smem_u32(tile(s, 2)) + p * kPanel, &maps.v, 64 * p, x.h / a.vdiv, t, bar(sm.full[s]));
            }
          }
          __syncwarp();
          ++g;
        }
        if (!ok || next.none) break;
        x = next;
      }
      if (!ok) {
        // flag it, and let this CTA's copies (and a response) land before its memory is given back
        if (lane == 0) atomicOr(P.status, 1);
        tc::mbar_wait_lanes(bar(sm.clcbar), asked & 1, 1u << 16);
        for (uint32_t k = g > kSt ? g - kSt : 0; k < g; ++k)
          tc::mbar_wait_lanes(bar(sm.full[k % kSt]), (k / kSt) & 1);
      }
    } else if (warp == kWarpMma) {
      // ================= products that need no state: the scores and U
      uint32_t g = 0;
      auto tiles = [&](uint32_t k) {
        if (ok) ok = tc::mbar_wait_lanes(bar(sm.full[k % kSt]), (k / kSt) & 1);
        tc::fence_after();
      };
      auto scores = [&](uint32_t k) {
        tiles(k);
        if (ok && tc::elect_one()) {
          const uint64_t dq = tc::kmajor(tc::smem_u32(tile(k % kSt, 0)));
          const uint64_t dk = tc::kmajor(tc::smem_u32(tile(k % kSt, 1)));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t off = (i >> 2) * (kPanel >> 4) + (i & 3) * 2;
            tc::mma_bf16_ss(tbase + kColP + 64 * (k & 1), dq + off, dk + off, tc::idesc_bf16(64, 64, false, false), i > 0);
          }
          tc::mma_commit(bar(sm.g0[k & 1]));
        }
        __syncwarp();
      };
      // The scores run one chunk ahead of U. Only one unit is looked at while a U is still to come: the warps that wait
      // for that U hold the ring's places, and more empty units than it has places may follow.
      int64_t left = 0;
      bool end = false;
      for (uint32_t ahead = 0; !end || ahead > g;) {
        const bool due = ahead > g;
        if (left == 0 && !end) {
          Unit x;
          end = !next_unit(x);
          left = end ? 0 : x.nchunks;
        }
        if (left > 0) {
          --left;
          if (!kState) {
            // (the scores two chunks before have been read)
            if (ok && ahead > 1) ok = tc::mbar_wait_lanes(bar(sm.pready[ahead & 1]), ((ahead - 2) >> 1) & 1);
            scores(ahead);
          }
          ++ahead;
        }
        if (!due) continue;
        const int s = g % kSt;
        if (kState) tiles(g);
        // U, once K~ is there and the last U is read
        if (ok) ok = tc::mbar_wait_lanes(bar(sm.kready[g & 1]), (g >> 1) & 1);
        constexpr uint32_t kUs = kState ? 2 : 1;
        if (ok && g >= kUs) ok = tc::mbar_wait_lanes(bar(sm.ufree[uplace(g)]), uphase(g - kUs));
        tc::fence_after();
        if (ok && tc::elect_one()) {
          const uint64_t dv = tc::mnmajor(tc::smem_u32(tile(s, 2)), kPanel);
          const uint64_t dh = tc::mnmajor(tc::smem_u32(tile(s, 1)), kPanel);
          const uint64_t dl = tc::mnmajor(tc::smem_u32(sm.lo[g & 1]), kPanel);
          const uint32_t u = tbase + kColU + 128 * uplace(g);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            tc::mma_bf16_ss(u, dv + 128 * k, dh + 128 * k, tc::idesc_bf16(128, 128, true, true), k > 0);
            tc::mma_bf16_ss(u, dv + 128 * k, dl + 128 * k, tc::idesc_bf16(128, 128, true, true), 1);
          }
          tc::mma_commit(bar(sm.gu[uplace(g)]));
          tc::mma_commit(bar(sm.empty[s]));
        }
        __syncwarp();
        ++g;
      }
    } else if (warp == kWarpMma2) {
      // ================= products for Y, by a warp of their own: while one waits, the other's run
      if (!kState) {
        uint32_t g = 0;
        int64_t left = 0;
        for (; any_chunk(left); ++g, --left) {
          const int s = g % kSt;
          if (ok) ok = tc::mbar_wait_lanes(bar(sm.full[s]), (g / kSt) & 1);
          // once the state is there and the last Y is read
          if (ok) ok = tc::mbar_wait_lanes(bar(sm.sready[g & 1]), (g >> 1) & 1);
          if (ok && g > 0) ok = tc::mbar_wait_lanes(bar(sm.yfree), (g - 1) & 1);
          tc::fence_after();
          if (ok && tc::elect_one()) {
            const uint64_t dq = tc::kmajor(tc::smem_u32(tile(s, 0)));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t off = (i >> 2) * (kPanel >> 4) + (i & 3) * 2;
              tc::mma_bf16_ts(tbase + kColO, tbase + kColS + (kSplit ? 0 : 64 * (g & 1)) + 8 * i, dq + off,
                              tc::idesc_bf16(128, 64, false, false), i > 0);
              if (kSplit)
                tc::mma_bf16_ts(tbase + kColO, tbase + kColS + 64 + 8 * i, dq + off, tc::idesc_bf16(128, 64, false, false), 1);
            }
            if (kSplit) tc::mma_commit(bar(sm.gq));
          }
          __syncwarp();
          if (ok) ok = tc::mbar_wait_lanes(bar(sm.pready[g & 1]), (g >> 1) & 1);
          tc::fence_after();
          if (ok && tc::elect_one()) {
            const uint64_t dv = tc::mnmajor(tc::smem_u32(tile(s, 2)), kPanel);
            const uint64_t dp = tc::kmajor(tc::smem_u32(sm.P[g & 1])), dr = tc::kmajor(tc::smem_u32(sm.extra) + (g & 1) * (kTile / 2));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              tc::mma_bf16_ss(tbase + kColO + 64, dv + 128 * k, dp + 2 * k, tc::idesc_bf16(128, 64, true, false), k > 0);
              if (kSplit)
                tc::mma_bf16_ss(tbase + kColO + 64, dv + 128 * k, dr + 2 * k, tc::idesc_bf16(128, 64, true, false), 1);
            }
            tc::mma_commit(bar(sm.gy));
            tc::mma_commit(bar(sm.empty[s]));
          }
          __syncwarp();
        }
      }
    } else if (warp == kWarpDecay) {
      // ================= decays, two tokens a lane
      uint32_t g = 0;
      for (Unit x; next_unit(x);) {
        if (!kState && x.run && (a.sg.len || a.st.in)) {  // its initial state, on its way to L2
          const char* src = a.sg.len ? reinterpret_cast<const char*>(a.sg.state + (x.sslot * P.Hv + x.h) * kDim * kDim)
                                     : reinterpret_cast<const char*>(a.st.in) + (x.slot * P.Hv + x.h) * kDim * kDim * (a.st.bf16 ? 2 : 4);
          const int lines = kDim * kDim * (!a.sg.len && a.st.bf16 ? 2 : 4) / 128;
          for (int i = lane; i < lines; i += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 128 * i));
        }
        float total = 0.f;  // lane 31's: log2 of the unit's decay
        StateFactor factor;
        // two chunks ahead, as the bits that come (a conversion here would wait for the load)
        auto bits = [&](int64_t tok) -> uint32_t {
          return P.per_token ? reinterpret_cast<const uint16_t*>(P.g)[tok * P.Hv + x.h] : reinterpret_cast<const uint32_t*>(P.g)[x.h];
        };
        auto number = [&](uint32_t b) { return decay_log2(__uint_as_float(P.per_token ? b << 16 : b)); };
        auto fetch = [&](int64_t c) {
          const int64_t j = (kRev ? x.nchunks - 1 - c : c) * kC + 2 * lane;
          return make_uint2(c < x.nchunks && j < x.len ? bits(x.t0 + j) : 0u, c < x.nchunks && j + 1 < x.len ? bits(x.t0 + j + 1) : 0u);
        };
        uint2 next = fetch(0), next2 = fetch(1);
        // backwards: the decay of the token that follows the chunk
        float follow = kRev && x.nchunks && x.t0 + x.len < x.end ? decay_log2(decay_g(P, x.t0 + x.len, x.h)) : 0.f;
        float whole = 0.f;
        for (int64_t c = 0; c < x.nchunks; ++c, ++g) {
          const int d = g % kDecs;
          // of a fixed decay every whole chunk has the same numbers (but the state's factor), and the slot has them already
          const bool again = !P.per_token && c > kDecs && (kRev || (c + 1) * kC <= x.len);
          if (!again) {
            float g0 = number(next.x);
            const float g1 = number(next.y);
            next = next2;
            next2 = fetch(c + 2);
            const float lead = __shfl_sync(0xffffffffu, g0, 0);
            if (kRev && lane == 0) g0 = 0.f;
            float pre = g0 + g1, suf = pre;
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) {
              const float p = __shfl_up_sync(0xffffffffu, pre, k), q = __shfl_down_sync(0xffffffffu, suf, k);
              if (lane >= k) pre += p;
              if (lane + k < 32) suf += q;
            }
            const float before = __shfl_up_sync(0xffffffffu, pre, 1), after = __shfl_down_sync(0xffffffffu, suf, 1);
            const float p0 = (lane ? before : 0.f) + g0, s1 = (lane < 31 ? after : 0.f) + follow;
            const float2 up = make_float2(fast_exp2(p0), fast_exp2(pre)), down = make_float2(fast_exp2(s1 + g1), fast_exp2(s1));
            const float2 e = kRev ? down : up, w = kRev ? up : down;
            whole = pre + follow;
            const float lam = factor.next(whole);
            if (ok && g >= kDecs) ok = tc::mbar_wait_lanes(bar(sm.decfree[d]), (g / kDecs - 1) & 1);
            *reinterpret_cast<float2*>(&sm.b[d][2 * lane]) = make_float2(p0, pre);
            *reinterpret_cast<float2*>(&sm.eb[d][2 * lane]) = make_float2(a.s_inter * e.x, a.s_inter * e.y);
            *reinterpret_cast<float2*>(&sm.w[d][2 * lane]) = make_float2(a.s_w * w.x, a.s_w * w.y);
            if (lane == 31) sm.lam[d] = lam;
            if (kRev) follow = lead;
          } else {
            next = next2;
            next2 = fetch(c + 2);
            const float lam = factor.next(whole);
            if (ok) ok = tc::mbar_wait_lanes(bar(sm.decfree[d]), (g / kDecs - 1) & 1);
            if (lane == 31) sm.lam[d] = lam;
          }
          total += whole;
          arrive(sm.dec[d]);
        }
        if (kState && x.run && lane == 31) a.sg.decay[x.sslot * P.Hv + x.h] = total;
      }
    }
  } else if (warp < kWarpB) {
    // ================= K~ and P
    if (kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int at = tid - 32 * kWarpA, wq = (warp - kWarpA) & 3, half = (warp - kWarpA) >> 2;
    const uint32_t tl = tbase + ((uint32_t)(32 * wq) << 16);
    const float2 scale = make_float2(a.s_intra, a.s_intra);
    uint32_t g = 0;
    for (Unit x; next_unit(x);) {
      for (int64_t c = 0; c < x.nchunks; ++c, ++g) {
        const int s = g % kSt, d = g % kDecs;
        const int64_t left = x.len - (kRev ? x.nchunks - 1 - c : c) * kC;
        const int nt = (int)(left < kC ? left : kC);
        unsigned char* Ks = tile(s, 1);
        unsigned char* Ls = sm.lo[g & 1];
        if (ok) ok = tc::mbar_wait_lanes(bar(sm.dec[d]), (g / kDecs) & 1);
        if (kState) {
          if (ok) ok = tc::mbar_wait_lanes(bar(sm.full[s]), (g / kSt) & 1);
          if (ok && g >= 2) ok = tc::mbar_wait_lanes(bar(sm.empty[(g - 2) % kSt]), ((g - 2) / kSt) & 1);
        } else if (ok) {
          // K is free once its scores are done; they are started after chunk g - 2's U, which reads this parity's low parts
          ok = tc::mbar_wait_lanes(bar(sm.g0[g & 1]), (g >> 1) & 1);
        }
        tc::fence_after();
        uint4 r[4];  // (all loads first: a store could be to where the next load is from, for all the compiler knows)
        float w1[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int i = at + 32 * kGroup * m;
          r[m] = *reinterpret_cast<const uint4*>(Ks + 16 * i);
          w1[m] = sm.w[d][(i >> 3) & (kC - 1)];
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {  // 16-byte chunks i
          const int i = at + 32 * kGroup * m, row = (i >> 3) & (kC - 1);
          const float2 w = make_float2(w1[m], w1[m]);
          uint4 hi, lo;
          split2(tc::mul2(unpack2(r[m].x), w), hi.x, lo.x);
          split2(tc::mul2(unpack2(r[m].y), w), hi.y, lo.y);
          split2(tc::mul2(unpack2(r[m].z), w), hi.z, lo.z);
          split2(tc::mul2(unpack2(r[m].w), w), hi.w, lo.w);
          if (nt < kC && row >= nt) hi = lo = make_uint4(0u, 0u, 0u, 0u);  // rows past the end hold other tokens
          *reinterpret_cast<uint4*>(Ks + 16 * i) = hi;
          *reinterpret_cast<uint4*>(Ls + 16 * i) = lo;
        }
        if (nt < kC)
          for (int i = at; i < (kC - nt) * 16; i += 32 * kGroup)
            *reinterpret_cast<uint4*>(tile(s, 2) + ((i >> 3) & 1) * kPanel + (nt + (i >> 4)) * 128 + (i & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        tc::fence_async_smem();
        arrive(sm.kready[g & 1]);
        if (!kState) {
          // P's buffer is free once chunk g - 2's products are done
          if (ok && g >= 2) ok = tc::mbar_wait_lanes(bar(sm.empty[(g - 2) % kSt]), ((g - 2) / kSt) & 1);
          // rows i = 16 wq + lane / 4 (+ 8), columns 32 half + 8 m + 2 (lane % 4) (+ 1)
          const int i0 = 16 * wq + (lane >> 2), j0 = 32 * half + 2 * (lane & 3);
          unsigned char* Pt = sm.P[g & 1];
          unsigned char* Pl = sm.extra + (g & 1) * (kTile / 2);
          auto at_of = [&](int i, int m) { return i * 128 + (((4 * half + m) ^ (i & 7)) << 4) + 4 * (lane & 3); };
          if (kRev ? half == 0 && wq >= 2 : half == 1 && wq < 2) {  // all on the masked side
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              *reinterpret_cast<uint32_t*>(Pt + at_of(i0 + 8 * (m & 1), m >> 1)) = 0u;
              if (kSplit) *reinterpret_cast<uint32_t*>(Pl + at_of(i0 + 8 * (m & 1), m >> 1)) = 0u;
            }
          } else {
            const float b0 = sm.b[d][i0], b1 = sm.b[d][i0 + 8];
            float p[16];  // (nothing between the load and its wait, where a register could be moved too early)
            tc::tmem_ld16x256(tl + kColP + 64 * (g & 1) + 32 * half, p);
            tc::tmem_wait_ld(p);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const int j = j0 + 8 * m;
              const float2 bj = *reinterpret_cast<const float2*>(&sm.b[d][j]);
#pragma unroll
              for (int v = 0; v < 2; ++v) {
                const int i = i0 + 8 * v;
                const float bi = v ? b1 : b0;
                const float2 e = kRev ? make_float2(fast_exp2(bj.x - bi), fast_exp2(bj.y - bi))
                                      : make_float2(fast_exp2(bi - bj.x), fast_exp2(bi - bj.y));
                float2 y = tc::mul2(tc::mul2(make_float2(p[4 * m + 2 * v], p[4 * m + 2 * v + 1]), scale), e);
                // (selected, not multiplied: rows past the end may hold anything)
                y.x = (kRev ? (j < nt ? j : -1) >= i : j <= (i < nt ? i : -1)) ? y.x : 0.f;
                y.y = (kRev ? (j + 1 < nt ? j + 1 : -1) >= i : j < (i < nt ? i : -1)) ? y.y : 0.f;
                uint32_t hi, lo;
                split2(y, hi, lo);
                *reinterpret_cast<uint32_t*>(Pt + at_of(i, m)) = hi;
                if (kSplit) *reinterpret_cast<uint32_t*>(Pl + at_of(i, m)) = lo;
              }
            }
          }
          tc::fence_async_smem();
          tc::fence_before();
          arrive(sm.pready[g & 1]);
        }
      }
    }
  } else {
    // ================= the state and Y
    if (kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int wq = (warp - kWarpB) & 3, half = (warp - kWarpB) >> 2;
    const int v = 32 * wq + lane;  // state row of this thread, its columns 64 half .. + 63; value of Y, tokens 32 half .. + 31
    const uint32_t tl = tbase + ((uint32_t)(32 * wq) << 16);
    uint32_t g = 0;
    // 32 rows of four 16-byte pieces in the warp's part of `extra`; rows two apart keep out of each other's banks
    auto turn = [&](int row, int piece) {
      return reinterpret_cast<float4*>(sm.extra + 2048 * (warp - kWarpB) + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
    };
    // The warps that fill a tile of Y together leave together: a barrier among them is not bounded.
    auto agree = [&] {
      uint32_t all;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(all) : "r"((uint32_t)ok), "n"(32 * kGroup) : "memory");
      ok = all != 0;
    };
    for (Unit x;;) {
      const bool more = next_unit(x);
      if (!kState && !kSplit) agree();
      if (!ok || !more) break;
      if (!x.run) {
        // a device slot index outside the pool (it no longer matches the host mirror the call was checked
        // against, as in a replayed graph): flagged, and the pool is not touched
        if ((x.slot < 0 || x.slot >= a.st.num_slots) && warp == kWarpB && lane == 0) atomicOr(P.status, 4);
        continue;
      }
      float2 S[32];
      const int64_t at = (x.slot * P.Hv + x.h) * kDim * kDim;
      if (kState || (!a.sg.len && !a.st.in)) {
#pragma unroll
        for (int j = 0; j < 32; ++j) S[j] = make_float2(0.f, 0.f);
      } else if (a.transposed && !a.sg.len) {
        const float* src = reinterpret_cast<const float*>(a.st.in) + at + (int64_t)64 * half * kDim + v;
#pragma unroll
        for (int j = 0; j < 32; ++j) S[j] = make_float2(src[2 * j * kDim], src[(2 * j + 1) * kDim]);
      } else if (a.sg.len || !a.st.bf16) {  // (the segments' states are kept as S is)
        const float* src32 = a.sg.len ? a.sg.state + (x.sslot * P.Hv + x.h) * kDim * kDim : reinterpret_cast<const float*>(a.st.in) + at;
        float4* f = reinterpret_cast<float4*>(S);
        if (kSplit) {
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j] = reinterpret_cast<const float4*>(src32 + v * kDim + 64 * half)[j];
        } else {  // 16 columns at a time: four lanes to a row in memory, turned through the warp's part of `extra`
          const float4* src = reinterpret_cast<const float4*>(src32 + (32 * wq + (lane >> 2)) * kDim + 64 * half) + (lane & 3);
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j] = src[(j & 3) * 2 * kDim + 4 * (j >> 2)];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int j = 0; j < 4; ++j) *turn(8 * j + (lane >> 2), lane & 3) = f[4 * q + j];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) f[4 * q + j] = *turn(lane, j);
            __syncwarp();
          }
        }
      } else {  // BF16, 32 columns at a time
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.st.in) + at +
                                                          (32 * wq + (lane >> 2)) * kDim + 64 * half) + (lane & 3);
        uint4 f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = src[(j & 3) * kDim + 4 * (j >> 2)];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
          for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(turn(8 * j + (lane >> 2), lane & 3)) = f[4 * q + j];
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 r = *reinterpret_cast<const uint4*>(turn(lane, j));
            float2* z = S + 16 * q + 4 * j;
            z[0] = unpack2(r.x); z[1] = unpack2(r.y); z[2] = unpack2(r.z); z[3] = unpack2(r.w);
          }
          __syncwarp();
        }
      }
      auto put_state = [&](uint32_t k) {  // as chunk k's A operand
        const uint32_t col = tl + kColS + (kSplit ? 0 : 64 * (k & 1)) + 32 * half;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (kSplit) split2(S[8 * m + e], hi[e], lo[e]);
            else hi[e] = pack2(S[8 * m + e]);
          }
          tc::tmem_st8(col + 8 * m, hi);
          if (kSplit) tc::tmem_st8(col + 64 + 8 * m, lo);
        }
        tc::tmem_wait_st();
        tc::fence_before();
        arrive(sm.sready[k & 1]);
      };
      if (!kState && x.nchunks) put_state(g);
      for (int64_t c = 0; c < x.nchunks; ++c, ++g) {
        const int d = g % kDecs;
        const int64_t ci = kRev ? x.nchunks - 1 - c : c;
        const int nt = (int)(x.len - ci * kC < kC ? x.len - ci * kC : kC);
        if (ok) ok = tc::mbar_wait_lanes(bar(sm.dec[d]), (g / kDecs) & 1);
        const float2 lam = make_float2(sm.lam[d], sm.lam[d]);
        if (ok) ok = tc::mbar_wait_lanes(bar(sm.gu[uplace(g)]), uphase(g));
        tc::fence_after();
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          float r[16];
          tc::tmem_ld16(tl + kColU + 128 * uplace(g) + 64 * half + 16 * m, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) S[8 * m + j] = tc::fma2(lam, S[8 * m + j], make_float2(r[2 * j], r[2 * j + 1]));
        }
        tc::fence_before();
        arrive(sm.ufree[uplace(g)]);
        if (kState) {
          arrive(sm.decfree[d]);
          continue;
        }
        // in two parts, the columns are those of this chunk's S Q^T; in one, the last chunk's has left the others: its Y
        // was waited for
        if (kSplit && c + 1 < x.nchunks) {
          if (ok) ok = tc::mbar_wait_lanes(bar(sm.gq), g & 1);
          tc::fence_after();
        }
        if (c + 1 < x.nchunks) put_state(g + 1);
        if (ok) ok = tc::mbar_wait_lanes(bar(sm.gy), g & 1);
        tc::fence_after();
        if (kSplit) {  // FP32, straight from the registers: thread v holds one value of each token
          float2 z[16];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            float r[16], y[16];
            tc::tmem_ld16_nowait(tl + kColO + 32 * half + 16 * m, r);
            tc::tmem_ld16_nowait(tl + kColO + 64 + 32 * half + 16 * m, y);
            tc::tmem_wait_ld2(r, y);
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 e = *reinterpret_cast<const float4*>(&sm.eb[d][32 * half + 16 * m + j]);
              z[8 * m + j / 2] = tc::fma2(make_float2(e.x, e.y), make_float2(r[j], r[j + 1]), make_float2(y[j], y[j + 1]));
              z[8 * m + j / 2 + 1] = tc::fma2(make_float2(e.z, e.w), make_float2(r[j + 2], r[j + 3]), make_float2(y[j + 2], y[j + 3]));
            }
          }
          tc::fence_before();
          arrive(sm.yfree);
          arrive(sm.decfree[d]);
          float* dst = a.y32 + ((x.t0 + ci * kC + 32 * half) * P.Hv + x.h) * kDim + v;
          const int left = nt - 32 * half;
#pragma unroll
          for (int j = 0; j < 32; ++j, dst += (int64_t)P.Hv * kDim)
            if (j < left) *dst = j & 1 ? z[j / 2].y : z[j / 2].x;
        } else {
          // transposed by matrix stores into a tile of shared memory, copied out from there
          if (warp == kWarpB && lane == 0) tc::bulk_wait_read();  // the last one has left
          agree();
          const uint32_t out = tc::smem_u32(sm.extra);
#pragma unroll
          for (int q = 0; q < 2; ++q) {  // values 32 wq + 16 q + 8 j + lane / 4, tokens 32 half + 8 m + 2 (lane % 4) (+ 1)
            float r[16], y[16];
            tc::tmem_ld16x256(tl + (16u * q << 16) + kColO + 32 * half, r);
            tc::tmem_ld16x256(tl + (16u * q << 16) + kColO + 64 + 32 * half, y);
            tc::tmem_wait_ld2(r, y);
            uint32_t z[8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float2 e = *reinterpret_cast<const float2*>(&sm.eb[d][32 * half + 8 * m + 2 * (lane & 3)]);
#pragma unroll
              for (int j = 0; j < 2; ++j)
                z[2 * m + j] = pack2(tc::fma2(e, make_float2(r[4 * m + 2 * j], r[4 * m + 2 * j + 1]),
                                              make_float2(y[4 * m + 2 * j], y[4 * m + 2 * j + 1])));
            }
            // matrix (m, j): lanes 8 (2 (m & 1) + j) + i give token 32 half + 8 m + i
            const int col = 32 * wq + 16 * q + 8 * ((lane >> 3) & 1), chunk = (col & 63) >> 3;
#pragma unroll
            for (int m = 0; m < 4; m += 2) {
              const int t = 32 * half + 8 * (m + (lane >> 4)) + (lane & 7);
              tc::stmatrix4_trans(out + (col >> 6) * kPanel + t * 128 + ((chunk ^ (t & 7)) << 4), z[2 * m], z[2 * m + 1],
                                  z[2 * m + 2], z[2 * m + 3]);
            }
          }
          tc::fence_before();
          arrive(sm.yfree);
          arrive(sm.decfree[d]);
          tc::fence_async_smem();
          asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * kGroup) : "memory");
          const int64_t t0 = x.t0 + ci * kC;
          if (nt == kC) {
            if (warp == kWarpB && lane == 0) {
              tc::tma_store3(&maps.y, out, 0, x.h, (int)t0);
              tc::tma_store3(&maps.y, out + kPanel, 64, x.h, (int)t0);
              tc::bulk_commit();
            }
          } else {  // (a whole tile would run into the next sequence)
            for (int i = tid - 32 * kWarpB; i < nt * 16; i += 32 * kGroup) {
              const int t = i >> 4, k = i & 15;
              *reinterpret_cast<uint4*>(a.y + ((t0 + t) * P.Hv + x.h) * kDim + 8 * k) =
                  *reinterpret_cast<const uint4*>(sm.extra + (k >> 3) * kPanel + t * 128 + (((k & 7) ^ (t & 7)) << 4));
            }
          }
        }
      }
      if (!kState && !kSplit) {  // `extra` is the copy's until the last Y has left
        if (warp == kWarpB && lane == 0) tc::bulk_wait_read();
        agree();
      }
      if (!ok) break;
      if (kSplit) continue;  // (no final state is asked for)
      float* dst32 = kState ? a.sg.state + (x.sslot * P.Hv + x.h) * kDim * kDim
                     : x.last && a.st.out && !a.st.bf16 ? reinterpret_cast<float*>(a.st.out) + at : nullptr;  // (never transposed)
      if (kRev && !kState && x.last && x.nchunks) {  // the initial state's adjoint: through the first token's decay
        const float e = exp2f(decay_log2(decay_g(P, x.t0, x.h)));
#pragma unroll
        for (int j = 0; j < 32; ++j) S[j] = tc::mul2(S[j], make_float2(e, e));
      }
      if (dst32) {
        float4* dst = reinterpret_cast<float4*>(dst32 + (32 * wq + (lane >> 2)) * kDim + 64 * half) + (lane & 3);
        const float4* f = reinterpret_cast<const float4*>(S);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int j = 0; j < 4; ++j) *turn(lane, j) = f[4 * q + j];
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[j * 2 * kDim + 4 * q] = *turn(8 * j + (lane >> 2), lane & 3);
          __syncwarp();
        }
      } else if (!kState && x.last && a.st.out) {
        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.st.out) + at +
                                              (32 * wq + (lane >> 2)) * kDim + 64 * half) + (lane & 3);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2* z = S + 16 * q + 4 * j;
            *reinterpret_cast<uint4*>(turn(lane, j)) = make_uint4(pack2(z[0]), pack2(z[1]), pack2(z[2]), pack2(z[3]));
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[j * kDim + 4 * q] = *reinterpret_cast<const uint4*>(turn(8 * j + (lane >> 2), lane & 3));
          __syncwarp();
        }
      }
    }
    if (!kState && !kSplit && warp == kWarpB && lane == 0) tc::bulk_wait();
    if (!ok && lane == 0) atomicOr(P.status, 1);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc::fence_after();
    tc::tmem_dealloc(tbase, 512);
  }
}

// Chains the segments of one (sequence, head): in, each segment's own state (from zero) but the last's;
// out, the state each segment starts from. A CTA takes 1024 of the state's values (16 CTAs a head: few heads are cut).
// Latency bounds it, one load's and the launch's: 11 us for 9 segments of 32 heads (36 MB in L2).
template <bool kRev>
__global__ void __launch_bounds__(256) kda_decay_chain_kernel(const __grid_constant__ PassArgs a) {
  const DecayProblem& P = a.P;
  const Segments& sg = a.sg;
  const int64_t n = blockIdx.x / P.Hv;
  const int h = (int)(blockIdx.x % P.Hv);
  const DecaySpan sp = decay_span(P, n);
  const int64_t slot = a.st.slots ? a.st.slots[n] : n;
  if (slot < 0 || slot >= a.st.num_slots) return;  // the main pass flags it
  const int at = 1024 * blockIdx.y + 4 * threadIdx.x, row = at / kDim, col = at % kDim;
  const int64_t from = (slot * P.Hv + h) * kDim * kDim;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.st.in && a.transposed) {
    const float* src = reinterpret_cast<const float*>(a.st.in) + from + (int64_t)col * kDim + row;
    x = make_float4(src[0], src[kDim], src[2 * kDim], src[3 * kDim]);
  } else if (a.st.in && a.st.bf16) {
    const uint2 r = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(a.st.in) + from + at);
    const float2 p = unpack2(r.x), q = unpack2(r.y);
    x = make_float4(p.x, p.y, q.x, q.y);
  } else if (a.st.in) {
    x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.st.in) + from + at);
  }
  const int64_t base = seg_slot(sg, sp.t0, n);
  const int64_t m = sp.len > sg.len ? (sp.len + sg.len - 1) / sg.len : 1;
  auto slot_of = [&](int64_t i) { return (base + (kRev ? m - 1 - i : i)) * P.Hv + h; };
  StateFactor factor;
  constexpr int kAhead = 8;  // loads in flight: none waits for the chain
  for (int64_t i = 0; i < m; i += kAhead) {
    float4 u[kAhead];
    float d[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i + j + 1 < m) {
        u[j] = *reinterpret_cast<const float4*>(sg.state + slot_of(i + j) * kDim * kDim + at);
        d[j] = sg.decay[slot_of(i + j)];
      }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j >= m) break;
      *reinterpret_cast<float4*>(sg.state + slot_of(i + j) * kDim * kDim + at) = x;
      if (i + j + 1 < m) {
        const float e = factor.next(d[j]);
        x.x = fmaf(e, x.x, u[j].x); x.y = fmaf(e, x.y, u[j].y);
        x.z = fmaf(e, x.z, u[j].z); x.w = fmaf(e, x.w, u[j].w);
      }
    }
  }
}

// dq and dk from the value heads' FP32 parts: sums over a group's heads, rounded once; and, for the decays' gradient,
// what crosses each token in each value head, q . dq - k . dk. A warp takes four (token, value head) at a time: kHeads
// (1, 2, else 4) heads of 4 / kHeads tokens of a query/key head, all their loads in flight (one token and query/key
// head a warp, whatever the heads: 69 us against 57). Bandwidth bounds it, 1 KiB read for each token and value head:
// 8192 tokens of 16 and 32 heads, 336 MB, 57 us, 5.9 TB/s, 88 % of the copy rate.
template <bool kCross, int kHeads>
__global__ void __launch_bounds__(256) kda_decay_group_sum_kernel(const DecayProblem P, const float* dq32, const float* dk32,
                                                                  __nv_bfloat16* dq, __nv_bfloat16* dk, float* z) {
  constexpr int kTok = 4 / kHeads;
  // (a block takes consecutive tokens of a head, so that their z share sectors)
  const int hq = blockIdx.x % P.Hqk, lane = threadIdx.x & 31;
  const int64_t tok = ((int64_t)(blockIdx.x / P.Hqk) * 8 + (threadIdx.x >> 5)) * kTok;
  if (tok >= P.Ttot) return;
  float4 sq[kTok], sk[kTok];
#pragma unroll
  for (int t = 0; t < kTok; ++t) sq[t] = sk[t] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < P.r; j0 += kHeads) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = i / kHeads, j = j0 + i % kHeads;
      a[i] = b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < P.r && tok + t < P.Ttot) {
        const int64_t at = (((tok + t) * P.Hqk + hq) * P.r + j) * kDim + 4 * lane;
        a[i] = __ldcs(reinterpret_cast<const float4*>(dq32 + at));
        b[i] = __ldcs(reinterpret_cast<const float4*>(dk32 + at));
      }
    }
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = i / kHeads;
      sq[t].x += a[i].x; sq[t].y += a[i].y; sq[t].z += a[i].z; sq[t].w += a[i].w;
      sk[t].x += b[i].x; sk[t].y += b[i].y; sk[t].z += b[i].z; sk[t].w += b[i].w;
      if (kCross) {
        x[i] = 0.f;
        if (tok + t < P.Ttot) {
          const uint2 rq = *reinterpret_cast<const uint2*>(P.q + (tok + t) * P.qt + hq * P.qh + 4 * lane);
          const uint2 rk = *reinterpret_cast<const uint2*>(P.k + (tok + t) * P.kt + hq * P.kh + 4 * lane);
          const float2 q0 = unpack2(rq.x), q1 = unpack2(rq.y), k0 = unpack2(rk.x), k1 = unpack2(rk.y);
          x[i] = q0.x * a[i].x + q0.y * a[i].y + q1.x * a[i].z + q1.y * a[i].w -
                 (k0.x * b[i].x + k0.y * b[i].y + k1.x * b[i].z + k1.y * b[i].w);
        }
      }
    }
    if (kCross) {  // the four sums over the lanes at once: after two steps a lane holds one of them, i = 2 (lane / 16) + lane / 8 % 2
      const bool up = lane & 16, right = lane & 8;
      float y0 = (up ? x[2] : x[0]) + __shfl_xor_sync(0xffffffffu, up ? x[0] : x[2], 16);
      float y1 = (up ? x[3] : x[1]) + __shfl_xor_sync(0xffffffffu, up ? x[1] : x[3], 16);
      float y = (right ? y1 : y0) + __shfl_xor_sync(0xffffffffu, right ? y0 : y1, 8);
#pragma unroll
      for (int o = 4; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      const int i = lane >> 3, t = i / kHeads, j = j0 + i % kHeads;
      // heads first: the sums that follow run over tokens
      if ((lane & 7) == 0 && j < P.r && tok + t < P.Ttot) z[((int64_t)hq * P.r + j) * P.Ttot + tok + t] = y;
    }
  }
#pragma unroll
  for (int t = 0; t < kTok; ++t)
    if (tok + t < P.Ttot) {
      const int64_t at = ((tok + t) * P.Hqk + hq) * kDim + 4 * lane;
      *reinterpret_cast<uint2*>(dq + at) = make_uint2(pack2(sq[t].x, sq[t].y), pack2(sq[t].z, sq[t].w));
      *reinterpret_cast<uint2*>(dk + at) = make_uint2(pack2(sk[t].x, sk[t].y), pack2(sk[t].z, sk[t].w));
    }
}

// A sum in two FP32 numbers, 48 bits.
struct Sum2 {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, t = s - hi;
    lo += (hi - (s - t)) + (x - t);
    hi = s;
  }
  __device__ __forceinline__ void add(Sum2 x) {
    add(x.hi);
    lo += x.lo;
  }
  __device__ __forceinline__ Sum2 from(int lane_delta) const {
    return Sum2{__shfl_up_sync(0xffffffffu, hi, lane_delta), __shfl_up_sync(0xffffffffu, lo, lane_delta)};
  }
};

// dg of one (sequence, head): a decay scales all that crosses its token, so
//   dg_t = sum_{i >= t} (q_i . dq_i - k_i . dk_i) + <S_T, dS_T>.
// The sums cancel over long sequences: 48 bits. 512 threads, from the end in runs of 4096 tokens. Latency bounds it
// (scans over a block): 11 us for 4 x 2048 tokens of 32 heads, of 326 for the step.
constexpr int kGateThreads = 512, kGateEach = 8;
__global__ void __launch_bounds__(kGateThreads) kda_decay_gate_grad_kernel(const DecayProblem P, const float* z, const float* hT,
                                                                          const float* dhT, __nv_bfloat16* dg) {
  constexpr int kWarps = kGateThreads / 32;
  __shared__ Sum2 part[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t n = blockIdx.x / P.Hv;
  const int h = (int)(blockIdx.x % P.Hv);
  const DecaySpan sp = decay_span(P, n);
  z += (int64_t)h * P.Ttot + sp.t0;
  Sum2 acc{0.f, 0.f};  // of what lies behind the run
  if (dhT && sp.len) {
    const int64_t base = (n * P.Hv + h) * kDim * kDim;
    Sum2 x{0.f, 0.f};
#pragma unroll 8
    for (int j = 4 * tid; j < kDim * kDim; j += 4 * kGateThreads) {
      const float4 a = *reinterpret_cast<const float4*>(hT + base + j), b = *reinterpret_cast<const float4*>(dhT + base + j);
      x.add(a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sum2 p = x.from(d);
      if (lane >= d) x.add(p);
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kWarps; ++k) acc.add(part[k]);
    __syncthreads();
  }
  for (int64_t end = sp.len; end > 0; end -= kGateThreads * kGateEach) {
    const int64_t t = end - 1 - kGateEach * tid;  // this thread's tokens, the last first
    float v[kGateEach];
#pragma unroll
    for (int j = 0; j < kGateEach; ++j) v[j] = t - j >= 0 ? z[t - j] : 0.f;
    Sum2 run{0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kGateEach; ++j) run.add(v[j]);
    Sum2 pre = run;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sum2 p = pre.from(d);
      if (lane >= d) pre.add(p);
    }
    if (lane == 31) part[warp] = pre;
    Sum2 mine = pre.from(1);
    if (lane == 0) mine = Sum2{0.f, 0.f};
    __syncthreads();
    Sum2 before = acc;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) before.add(part[k]);
      acc.add(part[k]);
    }
    before.add(mine);
#pragma unroll
    for (int j = 0; j < kGateEach; ++j) {
      before.add(v[j]);
      if (t - j >= 0) dg[(sp.t0 + t - j) * P.Hv + h] = __float2bfloat16_rn(before.hi + before.lo);
    }
    __syncthreads();
  }
}

struct SegWs {
  size_t state, decay, total;
};
SegWs carve_segments(int64_t N, int64_t Ttot, int64_t Hv, int64_t seg) {
  SegWs w{0, 0, 0};
  if (!seg) return w;
  const size_t slots = (size_t)(Ttot / seg + N);
  w.decay = ctx_align_up(sizeof(float) * slots * Hv * kDim * kDim);
  w.total = ctx_align_up(w.decay + sizeof(float) * slots * Hv);
  return w;
}

// After the segments: FP32 dq and dk of each value head, and what crosses each token and head.
struct GradWs {
  size_t dq, dk, z, total;
};
GradWs carve_grads(int64_t Ttot, int64_t Hqk, int64_t Hv, bool per_token) {
  GradWs w{0, 0, 0, 0};
  if (!per_token && Hqk == Hv) return w;
  const size_t rows = (size_t)Ttot * Hv;
  w.dk = ctx_align_up(sizeof(float) * rows * kDim);
  w.z = ctx_align_up(w.dk + sizeof(float) * rows * kDim);
  w.total = ctx_align_up(w.z + (per_token ? sizeof(float) * rows : 0));
  return w;
}

template <bool kRev, bool kState, bool kSplit>
cudaError_t launch(const Maps& maps, const PassArgs& a, cudaStream_t s) {
  auto kern = kda_decay_pass_kernel<kRev, kState, kSplit>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  const int64_t units = (a.sg.len ? a.first[a.sg.most] : a.P.N) * a.P.Hv;
  kern<<<(unsigned)units, kThreads, kSmemBytes, s>>>(maps, a);
  return cudaGetLastError();
}

struct Role {
  const __nv_bfloat16* p;
  int64_t t, h;
  int heads;
};

// One pass with the given roles; ws: the segments' workspace.
template <bool kRev>
cudaError_t pass(const DecayProblem& P, const Role& q, const Role& k, const Role& v, float s_inter, float s_intra, float s_w,
                 const DecayStates& st, bool transposed, __nv_bfloat16* y, float* y32, void* ws, cudaStream_t s) {
  Maps maps{};
  PassArgs a{};
  cudaError_t e;
  if (P.N * P.Hv == 0) return cudaSuccess;
  if (P.Ttot) {
    if ((e = token_map(&maps.q, q.p, q.heads, P.Ttot, q.h, q.t, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.k, k.p, k.heads, P.Ttot, k.h, k.t, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.v, v.p, v.heads, P.Ttot, v.h, v.t, kC)) != cudaSuccess) return e;
    if (y && (e = token_map(&maps.y, y, P.Hv, P.Ttot, kDim, (int64_t)P.Hv * kDim, kC)) != cudaSuccess) return e;
  }
  a.P = P;
  a.qdiv = P.Hv / q.heads;
  a.kdiv = P.Hv / k.heads;
  a.vdiv = P.Hv / v.heads;
  a.s_inter = s_inter;
  a.s_intra = s_intra;
  a.s_w = s_w;
  a.st = st;
  a.transposed = transposed;
  a.y = y;
  a.y32 = y32;
  auto len = [&](int64_t n) { return P.cu_host ? P.cu_host[n + 1] - P.cu_host[n] : P.T; };
  if (P.cu_host && P.N > 1 && P.N <= kOrder) {
    a.ordered = 1;
    for (int64_t i = 0; i < P.N; ++i) a.order[i] = (uint16_t)i;
    std::stable_sort(a.order, a.order + P.N, [&](uint16_t i, uint16_t j) { return len(i) > len(j); });
  }
  a.sg.most = 1;
  if (P.seg) {
    const SegWs w = carve_segments(P.N, P.Ttot, P.Hv, P.seg);
    a.sg.len = P.seg;
    a.sg.most = (int)((P.longest + P.seg - 1) / P.seg);
    int64_t have = P.N;  // the sequences that have a segment s (longest first): all have the first
    for (int t = 0; t < a.sg.most; ++t) {
      while (t && have && len(a.ordered ? a.order[have - 1] : have - 1) <= t * P.seg) --have;
      a.first[t + 1] = a.first[t] + (int32_t)have;
    }
    a.sg.state = reinterpret_cast<float*>(ws);
    a.sg.decay = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + w.decay);
    if ((e = launch<kRev, true, false>(maps, a, s)) != cudaSuccess) return e;
    kda_decay_chain_kernel<kRev><<<dim3((unsigned)(P.N * P.Hv), 16), 256, 0, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (y32 && st.out) return cudaErrorInvalidValue;
  return y32 ? launch<kRev, false, true>(maps, a, s) : launch<kRev, false, false>(maps, a, s);
}

}  // namespace

int64_t decay_segment_tokens(const int64_t* cu, int64_t N, int64_t T, int64_t Hv) {
  if (N > kOrder) return 0;
  auto chunks_of = [&](int64_t n) { return ((cu ? cu[n + 1] - cu[n] : T) + kC - 1) / kC; };
  int64_t longest = 0, chunks = 0;
  for (int64_t n = 0; n < (cu ? N : 1); ++n) {
    chunks += chunks_of(n);
    longest = std::max(longest, chunks_of(n));
  }
  if (!cu) chunks *= N;
  // An even share of the chunks for each of kUnits units, 8 chunks at least. Cutting adds a pass over keys and values
  // (about 0.6 of the main pass) and the chain: only where the longest sequence takes well over an SM's share, two units.
  // Measured, cut against whole, one sequence of 8192 or 16384 tokens: 96 heads (3.2 shares) 269 us : 210 us and
  // 541 : 404, 64 heads (4.8 shares) 206 : 210 and 359 : 395, 48 heads (6.3) 158 : 207, 32 heads (9.5) 128 : 203;
  // 1600 tokens of 8 heads 55 : 54, 2048 of 8 heads 50 : 66, 20000 of one head 61 : 470. (The Python binding knows that
  // up to 24 chunks are never cut.)
  const int64_t share = (chunks * Hv + kUnits - 1) / kUnits;
  if (longest <= std::max<int64_t>(4 * share, 24)) return 0;
  int64_t seg = std::max<int64_t>(share, 8);
  // not a few units more than the SMs take in two turns (a third turn for them alone)
  for (int64_t tries = 0; N * Hv < kUnits && tries < 64; ++tries, ++seg) {
    int64_t units = 0;
    for (int64_t n = 0; n < (cu ? N : 1); ++n) units += std::max<int64_t>((chunks_of(n) + seg - 1) / seg, 1);
    if ((cu ? units : units * N) * Hv <= kUnits) break;
  }
  return longest <= seg ? 0 : seg * kC;
}

size_t decay_workspace_bytes(int64_t N, int64_t Ttot, int64_t Hqk, int64_t Hv, int64_t seg, bool training, bool per_token) {
  return carve_segments(N, Ttot, Hv, seg).total + (training ? carve_grads(Ttot, Hqk, Hv, per_token).total : 0);
}

// Heads that a warp of kda_decay_group_sum_kernel takes of each of its 4 / heads tokens.
static int group_sum_heads(const DecayProblem& P) { return P.r == 1 ? 1 : P.r == 2 ? 2 : 4; }
int64_t decay_group_sum_blocks(const DecayProblem& P) {
  const int64_t tokens = 8 * (4 / group_sum_heads(P));
  return (P.Ttot + tokens - 1) / tokens * P.Hqk;
}

cudaError_t launch_decay_forward(const DecayProblem& P, const DecayStates& st, __nv_bfloat16* o, void* ws, cudaStream_t s) {
  const Role q{P.q, P.qt, P.qh, P.Hqk}, k{P.k, P.kt, P.kh, P.Hqk}, v{P.v, P.vt, P.vh, P.Hv};
  return pass<false>(P, q, k, v, P.scale, P.scale, 1.f, st, false, o, nullptr, ws, s);
}

cudaError_t launch_decay_backward(const DecayProblem& P, const float* h0, const float* hT, const DecayGrads& g, void* ws,
                                  cudaStream_t s) {
  char* base = reinterpret_cast<char*>(ws) + carve_segments(P.N, P.Ttot, P.Hv, P.seg).total;
  const GradWs w = carve_grads(P.Ttot, P.Hqk, P.Hv, P.per_token);
  // summed over a group's heads, and in the decays' gradient over the whole sequence (differences of large numbers):
  // dq and dk stay FP32 until then
  const bool f32 = g.dg || P.r > 1;
  float* dq = f32 ? reinterpret_cast<float*>(base + w.dq) : nullptr;
  float* dk = f32 ? reinterpret_cast<float*>(base + w.dk) : nullptr;
  const Role q{P.q, P.qt, P.qh, P.Hqk}, k{P.k, P.kt, P.kh, P.Hqk}, v{P.v, P.vt, P.vh, P.Hv};
  const Role d{g.d_o, (int64_t)P.Hv * kDim, kDim, P.Hv};
  const float c = P.scale;
  cudaError_t e;
  const DecayStates none{g.d_hT, nullptr, 0, nullptr, P.N};
  if ((e = pass<true>(P, k, q, d, 1.f, c, c, DecayStates{g.d_hT, g.dh0, 0, nullptr, P.N}, false, g.dv, nullptr, ws,
                      s)) != cudaSuccess) return e;
  // (last what is summed over heads: some of it is still in L2 then)
  if ((e = pass<false>(P, d, v, k, c, c, 1.f, DecayStates{h0, nullptr, 0, nullptr, P.N}, true, f32 ? nullptr : g.dq, dq,
                       ws, s)) != cudaSuccess) return e;
  if ((e = pass<true>(P, v, d, q, 1.f, c, c, none, true, f32 ? nullptr : g.dk, dk, ws, s)) != cudaSuccess)
    return e;
  if (P.Ttot == 0 || !f32) return cudaSuccess;
  float* z = reinterpret_cast<float*>(base + w.z);
  const int heads = group_sum_heads(P);
  const unsigned blocks = (unsigned)decay_group_sum_blocks(P);  // (checked before the first launch)
  auto sum = [&](auto kern) { kern<<<blocks, 256, 0, s>>>(P, dq, dk, g.dq, g.dk, z); };
  if (!g.dg) heads == 2 ? sum(kda_decay_group_sum_kernel<false, 2>) : sum(kda_decay_group_sum_kernel<false, 4>);
  else if (heads == 1) sum(kda_decay_group_sum_kernel<true, 1>);
  else heads == 2 ? sum(kda_decay_group_sum_kernel<true, 2>) : sum(kda_decay_group_sum_kernel<true, 4>);
  if ((e = cudaGetLastError()) != cudaSuccess || !g.dg) return e;
  kda_decay_gate_grad_kernel<<<(unsigned)(P.N * P.Hv), kGateThreads, 0, s>>>(P, z, hT, g.d_hT, g.dg);
  return cudaGetLastError();
}

}  // namespace kda
