// kda_delta_fwd.cu -- the forward pass of the gated delta rule over each sequence's chunks, on sm_103a tensor cores
// (kda_delta.cuh has the formulas; what a chunk has of its own comes from kda_delta_prep.cu).
//
// One CTA an SM, 20 warps with roles:
//   warp 0   copies: K, Q and V tiles by tiled copies (128-byte swizzle), T, P and the decays' factors; the next unit's number
//            (cluster launch control: the grid has a CTA for each unit, one (sequence, head), longest first, and a running
//            CTA takes over the next one that has not started)
//   warps 1, 2   products (tcgen05.mma kind::f16, BF16 operands, FP32 accumulators in tensor memory): the chain's, and o's (a
//            warp that waits for room for o does not hold up the chain: 257 us from one warp, 249 from two)
//   warps 4-11   o (and u) on their way out
//   warps 12-19  the state, 64 of a row's 128 values a thread in registers, and the elements between the chain's products
// The chain of a chunk: S K^T -> x = v - e^b S k -> T x -> w beta u -> the state's update. Elements go in two halves of the
// tokens, T being lower triangular: the first half's u does not wait for the second's x. So does the update, in halves of
// the state's columns, and S K^T starts with the first of them. What is off the chain (S Q^T, beta u for the output) is put where
// the tensor core and the warps would wait.
// Bound: that chain, 4470 cycles a chunk (2.16 us): the turns of its three products (issue, tensor core, commit, wake: some 500 each) and the
// element-wise steps between them (430 to 700). 8 x 1024 tokens of 96 heads, 5.05 units an SM: 235 us, 1.1 GB moved; issue slots
// used to 40 %. When this took 249 us: with W = T e^b K made a chunk ahead the chain has two products and takes 301 us: the products a chunk ahead
// cost more issue time than that saves; waits that poll instead of being suspended, 277 us.
//
// Long axis, few units: each sequence is cut into segments. A pass over every segment but the last goes from a state of zero
// and, without values, from the identity (a chunk takes S to S M + N, whatever S is: so does a segment); a small kernel
// chains them, and the main pass starts every segment from its state. Where a segment's decays leave nothing of any state, the
// identity is not followed: with decays of 0.02 to 0.34 a token and head, seven of eight heads over 1728 tokens.
#include <algorithm>

#include "kda_delta.cuh"
#include "kda_layout.h"
#include "kda_tma.h"
#include "tc.cuh"

namespace kda {
namespace {

constexpr int kC = kDecayChunk;
constexpr int kWarpLoad = 0, kWarpMma = 1, kWarpMmaO = 2, kWarpOut = 4, kWarpChain = 12;
constexpr int kThreads = 32 * 20;
// Registers a thread of the control, out and chain warps (setmaxnreg): 128 x 48 + 256 x 72 + 256 x 144 = 61,440, all of the
// 640 x 96 = 61,440 the block is launched with (a split above that would wait for ever).
constexpr int kStages = 2, kRing = 4;
constexpr uint32_t kTile = kC * kDim * 2, kPanel = kC * 128;  // bytes of a token tile, of its 64-element half
// Tensor memory, columns. S as A operand: its columns 64 h + 16 m .. are in 64 h + 8 m .. (high parts) and 32 further
// (low parts): a thread writes where it read the update from.
constexpr uint32_t kColS = 0;    // 128: S, then the update's sum
constexpr uint32_t kColX = 128;  // 64: S K^T
constexpr uint32_t kColA = 192;  // x, then w beta u, as A operands: 32 high, 32 low; from 64 on beta u
constexpr uint32_t kColQ = 320;  // 64: S Q^T
constexpr uint32_t kColO = 384;  // 64: (beta U)^T P^T
constexpr uint32_t kColU = 448;  // 64: T x

struct Unit {
  int64_t n, t0, len;  // sequence; first token and tokens of the unit
  int64_t slot, sslot; // of its state, and of its segment's
  int64_t place;       // of its first chunk
  int nchunks, h;
  bool run, last;      // there is something to do (the slot is in the pool); the sequence's last segment
  bool identity;       // pass over segments: from the identity, without values
  bool none;           // no unit: the end
};

struct Smem {
  unsigned char tok[kStages][3][kTile];  // K, Q, V
  unsigned char packet[kStages][kPkPass];
  unsigned char out[kTile];              // o on its way out
  union {
    struct {
      unsigned char u[kUTile];           // training: u on its way out,
      unsigned char S[kStateTile];       // and the state in BF16
    };
    unsigned char state[4 * kDim * kDim];  // serving: the state that the next unit starts from, in boxes of 128 bytes of a row
  };
  uint4 clc;
  Unit ring[kRing];
  unsigned long long full[kStages], empty[kStages], raw, sfull, sempty, fready, ffree, sready[2], gx, xready[2], gu[2], gq, wready[2], gs[2], vready, go, ofree, ufree, scopied;
  unsigned long long clcbar, rfull[kRing], rempty[kRing];
  uint32_t tmem;
};
constexpr int kSmemBytes = (int)sizeof(Smem);
static_assert(kSmemBytes <= 227 * 1024 && kPkPass % 1024 == 0, "shared memory of a CTA");

constexpr int kOrder = 512;      // sequences whose order is passed (more run in index order, whole)
constexpr int kMost = 4 * kSms;  // most segments of a sequence

struct Segments {
  int64_t len;     // tokens of a segment (a multiple of kC), 0: sequences are not cut
  int most;        // most segments of a sequence
  float* state;    // [slots, Hv, 128, 128]: what a segment makes of zero, then the state it starts from
  __nv_bfloat16* through;  // [slots, Hv, 2, 128, 128]: what it makes of the identity, in two parts,
  int32_t* none;   // [slots, Hv]: 1 where that is zero and was not written
};
// Slot of a sequence's first segment: leaves each sequence ceil(len_n / len) slots.
__device__ __forceinline__ int64_t seg_slot(const Segments& g, int64_t t0, int64_t n) { return t0 / g.len + n; }

struct PassArgs {
  DeltaProblem P;
  DecayStates st;
  Segments sg;
  int32_t first[kMost + 1];  // segments s of the sequences that have one: pairs first[s] .. first[s + 1] - 1
  const unsigned char* packets;
  uint32_t stride;         // from packet to packet
  unsigned char* states;   // training: BF16 states at the chunks' starts
  unsigned char* u;
  __nv_bfloat16* o;
  int ordered;
  uint16_t order[kOrder];  // longest sequence first
};
struct Maps {
  CUtensorMap q, k, v, o, st;
};

__device__ __forceinline__ float* regs(uint32_t* x) { return reinterpret_cast<float*>(x); }

template <bool kState>
__device__ __forceinline__ Unit unit_of(const PassArgs& a, int u) {
  const DeltaProblem& P = a.P;
  Unit x;
  x.identity = kState && (u & 1);
  if (kState) u >>= 1;
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
  x.slot = a.st.slots ? a.st.slots[x.n] : x.n;
  x.run = x.slot >= 0 && x.slot < a.st.num_slots;
  x.place = delta_slot(sp.t0, x.n);
  x.sslot = 0;
  x.last = true;
  if (a.sg.len) {
    const int64_t from = seg * a.sg.len;
    x.sslot = seg_slot(a.sg, sp.t0, x.n) + seg;
    x.last = from + a.sg.len >= sp.len;
    if ((seg > 0 && from >= sp.len) || (kState && x.last)) x.run = false;
    x.t0 += from;
    x.len = x.last ? sp.len - from : a.sg.len;
    x.place += from / kC;
  }
  x.nchunks = x.run ? (int)((x.len + kC - 1) / kC) : 0;
  x.none = false;
  if (x.identity && x.run) {
    // Decays that leave less than FP32 holds of the identity (its smallest number is 2^-149): zero, whatever the tokens are.
    float bound = 0.f;
    for (int c = threadIdx.x & 31; c < x.nchunks; c += 32)
      bound += reinterpret_cast<const DeltaAux*>(a.packets + ((x.place + c) * P.Hv + x.h) * (int64_t)a.stride + kPkAux)->bound;
#pragma unroll
    for (int k = 16; k; k >>= 1) bound += __shfl_xor_sync(0xffffffffu, bound, k);
    const bool none = bound < -160.f;
    if ((threadIdx.x & 31) == 0) a.sg.none[x.sslot * P.Hv + x.h] = none;
    if (none) {
      x.run = false;
      x.nchunks = 0;
    }
  }
  return x;
}

// kTrain: states and u are saved. kState: the pass over segments (states alone).
template <bool kTrain, bool kState>
__global__ void __launch_bounds__(kThreads, 1) kda_delta_fwd_kernel(const __grid_constant__ Maps maps, const __grid_constant__ PassArgs a) {
  extern __shared__ __align__(1024) unsigned char raw_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem);
  const DeltaProblem& P = a.P;
  if (tc::smem_u32(raw_smem) & 1023) {  // (never: the tiles' swizzle needs the alignment that is asked for, and there is no room for more)
    if (threadIdx.x == 0) atomicOr(P.status, 1);
    return;
  }
  // Serving: a unit's start state comes by tiled copies, while the unit before it is worked on. (Loaded by the warps that need it,
  // behind the tiles that are on their way, it took two chunks' time.)
  const bool staged = !kTrain && !kState && (a.sg.len || a.st.in);
  const uint32_t state_bytes = a.sg.len || !a.st.bf16 ? 4 * kDim * kDim : 2 * kDim * kDim;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [](unsigned long long& b) { return tc::smem_u32(&b); };

  if (warp == kWarpMma) tc::tmem_alloc(tc::smem_u32(&sm.tmem), 512);
  if (tid == 0) {
    auto init = [&](unsigned long long& b, uint32_t n) { tc::mbar_init(bar(b), n); };
    for (int i = 0; i < 2; ++i) {
      init(sm.full[i], 1); init(sm.empty[i], kState ? 9 : 18);
      init(sm.sready[i], 4); init(sm.xready[i], 4); init(sm.wready[i], 4);
      init(sm.gu[i], 1); init(sm.gs[i], 1);
    }
    init(sm.raw, 1); init(sm.sfull, 1); init(sm.sempty, 8); init(sm.fready, 8); init(sm.ffree, 8); init(sm.gx, 1); init(sm.gq, 1); init(sm.vready, 8); init(sm.go, 1); init(sm.ofree, 8); init(sm.ufree, 8);
    init(sm.scopied, 8); init(sm.clcbar, 1);
    for (int i = 0; i < kRing; ++i) { init(sm.rfull[i], 1); init(sm.rempty[i], kState ? 17 : 18); }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = sm.tmem;
  bool ok = true;  // false: a wait gave up; the warp touches only its own CTA's memory and leaves
  auto wait = [&](unsigned long long& b, uint32_t parity) {
    if (ok) ok = tc::mbar_wait_lanes(bar(b), parity & 1);
    tc::fence_after();
    return ok;
  };
  auto arrive = [&](unsigned long long& b) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar(b));
  };
  // The ring of units, as a consumer (a warp): its place, and the next unit (false: none).
  uint32_t ur = 0;
  auto next_unit = [&](Unit& x) {
    if (!wait(sm.rfull[ur % kRing], ur / kRing)) return false;
    x = sm.ring[ur % kRing];
    arrive(sm.rempty[ur % kRing]);
    ++ur;
    return !x.none;
  };
  // A unit whose end state leaves by way of the warps that store o. (In training there are few units to an SM, and that would
  // come after the last one.)
  auto keeps = [&](const Unit& x) { return !kTrain && x.run && (kState || (x.last && a.st.out)); };
  // A consumer that sees chunks alone: is there one more, `left` those of the unit at hand? kept: end states before this unit's.
  uint32_t kept = 0;
  bool keep_this = false;
  auto any_chunk = [&](int& left) {
    Unit x;
    while (left == 0) {
      if (!next_unit(x)) return false;
      left = x.nchunks;
      kept += keep_this;
      keep_this = keeps(x);
    }
    return true;
  };

  if (warp < kWarpOut) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == kWarpLoad) {
      // ================= units and copies
      uint32_t g = 0, asked = 0, tails = 0;
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
      uint32_t loaded = 0;  // states
      auto load_state = [&](const Unit& x) {
        if (!staged || !x.run || !ok) return;
        if (loaded) ok = tc::mbar_wait_lanes(bar(sm.sempty), (loaded - 1) & 1);
        if (!ok) return;
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(bar(sm.sfull), state_bytes);
          const int each = state_bytes == 4 * kDim * kDim ? 32 : 64;
          for (int b = 0; b < kDim / each; ++b)
            tc::tma_load4(tc::smem_u32(sm.state) + b * 16384, &maps.st, b * each, 0, x.h, (int)(a.sg.len ? x.sslot : x.slot), bar(sm.sfull));
        }
        __syncwarp();
        ++loaded;
      };
      Unit x = unit_of<kState>(a, (int)blockIdx.x), next;
      load_state(x);
      push(x);
      ask();
      for (;;) {
        next.none = true;
        for (int c = 0;; ++c) {
          if (c == (x.nchunks < 2 ? x.nchunks : 2)) {
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
            if (more) next = unit_of<kState>(a, (int)nx);
            push(next);
            if (ok && more) {
              ask();
              load_state(next);
            }
          }
          if (!ok || c == x.nchunks) break;
          const uint32_t s = g % kStages;
          if (g >= kStages) ok = tc::mbar_wait_lanes(bar(sm.empty[s]), (g / kStages - 1) & 1);
          if (!ok) break;
          const int64_t left = x.len - (int64_t)c * kC;
          if (lane == 0) {
            const int t = (int)(x.t0 + (int64_t)c * kC);
            const uint32_t f = left < kC ? bar(sm.raw) : bar(sm.full[s]);
            tc::mbar_arrive_expect_tx(f, 3 * kTile + kPkPass);
#pragma unroll
            for (int p = 0; p < 2; ++p) tc::tma_load3(tc::smem_u32(sm.tok[s][0]) + p * kPanel, &maps.k, 64 * p, x.h / P.r, t, f);
            tc::bulk_g2s(tc::smem_u32(sm.packet[s]), a.packets + ((x.place + c) * P.Hv + x.h) * (int64_t)a.stride, kPkPass, f);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              tc::tma_load3(tc::smem_u32(sm.tok[s][2]) + p * kPanel, &maps.v, 64 * p, x.h, t, f);
              tc::tma_load3(tc::smem_u32(sm.tok[s][1]) + p * kPanel, &maps.q, 64 * p, x.h / P.r, t, f);
            }
          }
          __syncwarp();
          if (left < kC) {  // rows past the end hold other tokens
            ok = tc::mbar_wait_lanes(bar(sm.raw), tails & 1);
            ++tails;
            for (int i = lane; ok && i < (kC - (int)left) * 48; i += 32) {
              const int row = (int)left + i / 48, k = i % 48;
              *reinterpret_cast<uint4*>(sm.tok[s][k >> 4] + ((k >> 3) & 1) * kPanel + row * 128 + (k & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            tc::fence_async_smem();
            arrive(sm.full[s]);
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
        if (tails) tc::mbar_wait_lanes(bar(sm.raw), (tails - 1) & 1, 1u << 16);
        if (loaded) tc::mbar_wait_lanes(bar(sm.sfull), (loaded - 1) & 1, 1u << 16);
        for (uint32_t k = g > kStages ? g - kStages : 0; k < g; ++k) tc::mbar_wait_lanes(bar(sm.full[k % kStages]), (k / kStages) & 1, 1u << 16);
      }
    } else if (warp == kWarpMma) {
      // ================= the chain's products
      constexpr uint32_t kN32 = tc::idesc_bf16(128, 32, false, false), kN64 = tc::idesc_bf16(128, 64, false, false);
      uint32_t g = 0;
      int left = 0;
      for (; any_chunk(left); ++g, --left) {
        const uint32_t s = g % kStages;
        const uint32_t k = tc::smem_u32(sm.tok[s][0]), T = tc::smem_u32(sm.packet[s]) + kPkT;
        const uint64_t kk = tc::kmajor(k), kn = tc::mnmajor(k, kPanel);
        if (!wait(sm.full[s], g / kStages)) break;
        if (kTrain && g && !wait(sm.ufree, g - 1)) break;
        // S K^T, the columns of S as they come
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!wait(sm.sready[h], g)) break;
          if (tc::elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int part = 0; part < 2; ++part)
                tc::mma_bf16_ts(tbase + kColX, tbase + kColS + 64 * h + 8 * i + 32 * part, kk + h * (kPanel >> 4) + 2 * i, kN64, h + i + part > 0);
            if (h) tc::mma_commit(bar(sm.gx));
          }
          __syncwarp();
        }
        if (!ok) break;
        // T x: what the first 32 tokens give to all, what the others give to themselves (an end state in its place has been read)
        if (kept && !wait(sm.ffree, kept - 1)) break;
        const uint64_t th = tc::kmajor(T), tlo = tc::kmajor(T + 8192);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!wait(sm.xready[h], g)) break;
          if (tc::elect_one()) {
            const uint32_t to = tbase + kColU + 32 * h, id = h ? kN32 : kN64;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t x = tbase + kColA + 16 * h + 8 * i, at = 256 * h + 4 * h + 2 * i;
              tc::mma_bf16_ts(to, x, th + at, id, h + i > 0);
              tc::mma_bf16_ts(to, x, tlo + at, id, 1);
              tc::mma_bf16_ts(to, x + 32, th + at, id, 1);
            }
            tc::mma_commit(bar(sm.gu[h]));
          }
          __syncwarp();
        }
        if (!ok) break;
        // the state's update, in place of the operand (once that is read), the last of it for one half of the columns after the other
        if (!kState && !wait(sm.gq, g)) break;
        if (kTrain && !wait(sm.scopied, g)) break;
        if (!wait(sm.wready[0], g)) break;
        if (tc::elect_one())
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int part = 0; part < 2; ++part)
              tc::mma_bf16_ts(tbase + kColS, tbase + kColA + 8 * i + 32 * part, kn + 128 * i, tc::idesc_bf16(128, 128, false, true), i + part > 0);
        __syncwarp();
        if (!wait(sm.wready[1], g)) break;
        if (tc::elect_one())
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 2; i < 4; ++i)
#pragma unroll
              for (int part = 0; part < 2; ++part)
                tc::mma_bf16_ts(tbase + kColS + 64 * h, tbase + kColA + 8 * i + 32 * part, kn + h * (kPanel >> 4) + 128 * i,
                                tc::idesc_bf16(128, 64, false, true), 1);
            tc::mma_commit(bar(sm.gs[h]));
            if (h) tc::mma_commit(bar(sm.empty[s]));
          }
        __syncwarp();
      }
    } else if (!kState && warp == kWarpMmaO) {
      // ================= o's products: S Q^T behind S K^T, and P beta u
      constexpr uint32_t kN64 = tc::idesc_bf16(128, 64, false, false);
      uint32_t g = 0;
      int left = 0;
      for (; any_chunk(left); ++g, --left) {
        const uint32_t s = g % kStages;
        const uint64_t qk = tc::kmajor(tc::smem_u32(sm.tok[s][1])), p = tc::kmajor(tc::smem_u32(sm.packet[s]) + kPkP);
        if (!wait(sm.full[s], g / kStages)) break;
        if (g && !wait(sm.ofree, g - 1)) break;
        if (!wait(sm.gx, g)) break;
        // (both parts of S: with the high one alone o is 2.5e-3 from 64 bits without decays, so 1.9e-3, for 0.4 % of the time)
        if (tc::elect_one()) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int part = 0; part < 2; ++part)
              tc::mma_bf16_ts(tbase + kColQ, tbase + kColS + 64 * (i >> 2) + 8 * (i & 3) + 32 * part, qk + (i >> 2) * (kPanel >> 4) + (i & 3) * 2, kN64, i + part > 0);
          tc::mma_commit(bar(sm.gq));
        }
        __syncwarp();
        if (!wait(sm.vready, g)) break;
        if (tc::elect_one()) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tc::mma_bf16_ts(tbase + kColO, tbase + kColA + 64 + 8 * i, p + 2 * i, kN64, i > 0);
            tc::mma_bf16_ts(tbase + kColO, tbase + kColA + 96 + 8 * i, p + 2 * i, kN64, 1);
          }
          tc::mma_commit(bar(sm.go));
          tc::mma_commit(bar(sm.empty[s]));
        }
        __syncwarp();
      }
    }
  } else if (warp < kWarpChain) {
    // ================= what leaves: o (and u)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int wq = (warp - kWarpOut) & 3, half = (warp - kWarpOut) >> 2;
    const float2 scale = make_float2(P.scale, P.scale);
    const uint32_t tl = tbase + ((uint32_t)(32 * wq) << 16);
    // The warps that fill a tile together leave together: a barrier among them is not bounded.
    auto agree = [&] {
      uint32_t all;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(all) : "r"((uint32_t)ok) : "memory");
      return ok = all != 0;
    };
    // a block of 32 tokens and 16 values of a token tile, from the layout of tmem_ld16x256
    auto store_block = [&](uint32_t tile, int token, int value, const uint32_t* r) {
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const int t = token + 8 * (i + (lane >> 4)) + (lane & 7), d = value + 8 * ((lane >> 3) & 1);
        tc::stmatrix4_trans(tile + (d >> 6) * kPanel + t * 128 + ((((d & 63) >> 3) ^ (t & 7)) << 4), r[2 * i], r[2 * i + 1],
                            r[2 * i + 2], r[2 * i + 3]);
      }
    };
    uint32_t g = 0;
    for (Unit x;;) {
      const bool more = next_unit(x);
      if (!agree() || !more) break;
      for (int c = 0; !kState && c < x.nchunks; ++c, ++g) {
        const int nt = (int)(x.len - (int64_t)c * kC < kC ? x.len - (int64_t)c * kC : kC);
        const int64_t t0 = x.t0 + (int64_t)c * kC;
        const uint32_t s = g % kStages;
        const DeltaAux& aux = *reinterpret_cast<const DeltaAux*>(sm.packet[s] + kPkAux);
        wait(sm.full[s], g / kStages);
        if (kTrain) {
          // the state's high parts
          wait(sm.sready[0], g);
          wait(sm.sready[1], g);
          if (warp == kWarpOut && lane == 0) tc::bulk_wait_read_but<2>();  // the last one has left
          if (!agree()) break;
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            float r[16];
            tc::tmem_ld16(tl + kColS + 64 * half + 16 * m, r);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<float4*>(sm.S + half * 16384 + (32 * wq + lane) * 128 + (((4 * m + q) ^ (lane & 7)) << 4)) =
                  make_float4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
          }
          tc::fence_before();
          arrive(sm.scopied);
          tc::fence_async_smem();
          asm volatile("barrier.cta.sync 1, 256;" ::: "memory");
          if (warp == kWarpOut && lane == 0) {
            tc::bulk_s2g(a.states + ((x.place + c) * P.Hv + x.h) * (int64_t)kStateTile, tc::smem_u32(sm.S), kStateTile);
            tc::bulk_commit();
          }
          wait(sm.gu[0], g);
          wait(sm.gu[1], g);
          if (warp == kWarpOut && lane == 0) tc::bulk_wait_read_but<2>();  // the last u has left
          if (!agree()) break;
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            float r[16];
            tc::tmem_ld16x256(tl + (16u * m << 16) + kColU + 32 * half, r);
            tc::tmem_wait_ld(r);
            uint32_t z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = pack2(r[2 * i], r[2 * i + 1]);
            store_block(tc::smem_u32(sm.u), 32 * half, 32 * wq + 16 * m, z);
          }
          tc::fence_before();
          arrive(sm.ufree);
          tc::fence_async_smem();
          asm volatile("barrier.cta.sync 1, 256;" ::: "memory");
          if (warp == kWarpOut && lane == 0) {
            tc::bulk_s2g(a.u + ((x.place + c) * P.Hv + x.h) * (int64_t)kUTile, tc::smem_u32(sm.u), kUTile);
            tc::bulk_commit();
          }
        }
        wait(sm.go, g);
        if (warp == kWarpOut && lane == 0) {  // the last o has left
          if (kTrain) tc::bulk_wait_read_but<2>();
          else tc::bulk_wait_read();
        }
        if (!agree()) break;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float r[16], y[16];
          tc::tmem_ld16x256(tl + (16u * m << 16) + kColQ + 32 * half, r);
          tc::tmem_ld16x256(tl + (16u * m << 16) + kColO + 32 * half, y);
          tc::tmem_wait_ld2(r, y);
          uint32_t z[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 e = *reinterpret_cast<const float2*>(&aux.eb[32 * half + 8 * i + 2 * (lane & 3)]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              z[2 * i + j] = pack2(tc::mul2(scale, tc::fma2(e, make_float2(r[4 * i + 2 * j], r[4 * i + 2 * j + 1]),
                                                            make_float2(y[4 * i + 2 * j], y[4 * i + 2 * j + 1]))));
          }
          store_block(tc::smem_u32(sm.out), 32 * half, 32 * wq + 16 * m, z);
        }
        tc::fence_before();
        arrive(sm.ofree);
        arrive(sm.empty[s]);
        tc::fence_async_smem();
        asm volatile("barrier.cta.sync 1, 256;" ::: "memory");
        if (nt == kC) {
          if (warp == kWarpOut && lane == 0) {
            tc::tma_store3(&maps.o, tc::smem_u32(sm.out), 0, x.h, (int)t0);
            tc::tma_store3(&maps.o, tc::smem_u32(sm.out) + kPanel, 64, x.h, (int)t0);
            tc::bulk_commit();
          }
        } else {  // (a whole tile would run into the next sequence)
          for (int i = tid - 32 * kWarpOut; i < nt * 16; i += 256) {
            const int t = i >> 4, k = i & 15;
            *reinterpret_cast<uint4*>(a.o + ((t0 + t) * P.Hv + x.h) * kDim + 8 * k) =
                *reinterpret_cast<const uint4*>(sm.out + (k >> 3) * kPanel + t * 128 + (((k & 7) ^ (t & 7)) << 4));
          }
          // (an empty group, so that they are three a chunk)
          if (kTrain && warp == kWarpOut && lane == 0) tc::bulk_commit();
        }
      }
      if (!ok) break;
      if (!keeps(x)) continue;
      // the end state
      wait(sm.fready, kept);
      const int64_t to = ((kState ? x.sslot : x.slot) * P.Hv + x.h) * kDim * kDim;
      const int at = (32 * wq + lane) * kDim + 64 * half;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        float r[16];
        tc::tmem_ld16(tl + (half ? kColA + 64 : kColU) + 16 * m, r);
        if (m == 3) {
          tc::fence_before();
          arrive(sm.ffree);
        }
        if (!ok) break;
        uint32_t hi[8], lo[8];
        if (kState && x.identity) {
#pragma unroll
          for (int e = 0; e < 8; ++e) split2(make_float2(r[2 * e], r[2 * e + 1]), hi[e], lo[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) hi[e] = pack2(make_float2(r[2 * e], r[2 * e + 1]));
        }
        if (kState ? !x.identity : !a.st.bf16) {
          float4* dst = reinterpret_cast<float4*>((kState ? a.sg.state : reinterpret_cast<float*>(a.st.out)) + to + at + 16 * m);
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[j] = make_float4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
        } else {
          __nv_bfloat16* dst = kState ? a.sg.through + 2 * to + at + 16 * m : reinterpret_cast<__nv_bfloat16*>(a.st.out) + to + at + 16 * m;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            reinterpret_cast<uint4*>(dst)[j] = make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
            if (kState) reinterpret_cast<uint4*>(dst + kDim * kDim)[j] = make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
          }
        }
      }
      ++kept;
      if (!agree()) break;
    }
    if (warp == kWarpOut && lane == 0) tc::bulk_wait();
    if (!ok && lane == 0) atomicOr(P.status, 1);
  } else {
    // ================= the state
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int wq = (warp - kWarpChain) & 3, half = (warp - kWarpChain) >> 2;
    const int v = 32 * wq + lane;  // state row of this thread, its columns 64 half .. + 63
    const uint32_t tl = tbase + ((uint32_t)(32 * wq) << 16);
    const int j0 = 32 * half + 2 * (lane & 3);
    uint32_t g = 0, states = 0;
    for (Unit x; next_unit(x);) {
      if (!x.run) {
        if (kState) continue;
        // a device slot index outside the pool (it no longer matches the host mirror the call was checked
        // against, as in a replayed graph): flagged, and the pool is not touched
        if ((x.slot < 0 || x.slot >= a.st.num_slots) && warp == kWarpChain && lane == 0) atomicOr(P.status, 4);
        continue;
      }
      const int64_t at = (x.slot * P.Hv + x.h) * kDim * kDim + v * kDim + 64 * half;
      const int64_t sat = (x.sslot * P.Hv + x.h) * kDim * kDim + v * kDim + 64 * half;
      float2 S[32];
      if (kState) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          S[j] = make_float2(x.identity && v == 64 * half + 2 * j ? 1.f : 0.f, x.identity && v == 64 * half + 2 * j + 1 ? 1.f : 0.f);
      } else if (kTrain && a.sg.len) {
        const float4* src = reinterpret_cast<const float4*>(a.sg.state + sat);
#pragma unroll
        for (int j = 0; j < 16; ++j) reinterpret_cast<float4*>(S)[j] = src[j];
      } else if (!a.st.in && !a.sg.len) {
#pragma unroll
        for (int j = 0; j < 32; ++j) S[j] = make_float2(0.f, 0.f);
      } else if (kTrain) {  // (FP32 there)
        const float4* src = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.st.in) + at);
#pragma unroll
        for (int j = 0; j < 16; ++j) reinterpret_cast<float4*>(S)[j] = src[j];
      } else {
        if (!wait(sm.sfull, states)) break;
        ++states;
        const unsigned char* row = sm.state + v * 128;
        if (state_bytes == 4 * kDim * kDim) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            reinterpret_cast<float4*>(S)[j] = *reinterpret_cast<const float4*>(row + (2 * half + (j >> 3)) * 16384 + (((j & 7) ^ (v & 7)) << 4));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 r = *reinterpret_cast<const uint4*>(row + half * 16384 + ((j ^ (v & 7)) << 4));
            S[4 * j] = unpack2(r.x); S[4 * j + 1] = unpack2(r.y); S[4 * j + 2] = unpack2(r.z); S[4 * j + 3] = unpack2(r.w);
          }
        }
        arrive(sm.sempty);
      }
      StateFactor factor;
      for (int c = 0; c < x.nchunks; ++c, ++g) {
        // the state as an operand (here, not where it comes from: there are two such places, and code that runs once a unit
        // comes to the instruction cache anew each time)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) split2(S[8 * m + e], hi[e], lo[e]);
          tc::tmem_st8(tl + kColS + 64 * half + 8 * m, hi);
          tc::tmem_st8(tl + kColS + 64 * half + 32 + 8 * m, lo);
        }
        tc::tmem_wait_st();
        tc::fence_before();
        arrive(sm.sready[half]);
        const uint32_t s = g % kStages;
        const DeltaAux& aux = *reinterpret_cast<const DeltaAux*>(sm.packet[s] + kPkAux);
        if (!wait(sm.full[s], g / kStages)) break;
        const float lam1 = factor.next(aux.whole);
        // x = v - e^b (S k)
        uint32_t r[2][8];
        float2 e[4], f[4];
        const uint32_t keep = kState && x.identity ? 0u : 0xffffffffu;
        // 4 x 2 blocks [8 tokens][8 values], transposed: r[2 i + j] holds tokens j0 + 8 i (+ 1) of value 8 j + lane / 4
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const int t = 32 * half + 8 * (i + (lane >> 4)) + (lane & 7), d = 32 * wq + 16 * q + 8 * ((lane >> 3) & 1);
            tc::ldmatrix4_trans(tc::smem_u32(sm.tok[s][2]) + (d >> 6) * kPanel + t * 128 + ((((d & 63) >> 3) ^ (t & 7)) << 4), r[q] + 2 * i);
          }
        if (kState)
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i >> 3][i & 7] &= keep;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = *reinterpret_cast<const float2*>(&aux.eb[j0 + 8 * i]);
          e[i] = make_float2(-e[i].x, -e[i].y);
        }
        if (!wait(sm.gx, g)) break;
        {
          float p[2][16];
          tc::tmem_ld16x256(tl + kColX + 32 * half, p[0]);
          tc::tmem_ld16x256(tl + (16u << 16) + kColX + 32 * half, p[1]);
          tc::tmem_wait_ld2(p[0], p[1]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                split2(tc::fma2(e[i], make_float2(p[q][4 * i + 2 * j], p[q][4 * i + 2 * j + 1]), unpack2(r[q][2 * i + j])), hi[2 * i + j], lo[2 * i + j]);
            tc::tmem_st16x128(tl + (16u * q << 16) + kColA + 16 * half, regs(hi));
            tc::tmem_st16x128(tl + (16u * q << 16) + kColA + 32 + 16 * half, regs(lo));
          }
        }
        tc::tmem_wait_st();
        tc::fence_before();
        arrive(sm.xready[half]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = *reinterpret_cast<const float2*>(&aux.w[j0 + 8 * i]);
          f[i] = *reinterpret_cast<const float2*>(&aux.beta[j0 + 8 * i]);
        }
        if (!wait(sm.gu[half], g)) break;
        // w beta u, then (off the chain) beta u
        float2 y[2][8];
        {
          float p[2][16];
          tc::tmem_ld16x256(tl + kColU + 32 * half, p[0]);
          tc::tmem_ld16x256(tl + (16u << 16) + kColU + 32 * half, p[1]);
          tc::tmem_wait_ld2(p[0], p[1]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                y[q][2 * i + j] = tc::mul2(f[i], make_float2(p[q][4 * i + 2 * j], p[q][4 * i + 2 * j + 1]));
                split2(tc::mul2(e[i], y[q][2 * i + j]), hi[2 * i + j], lo[2 * i + j]);
              }
            const uint32_t col = tl + (16u * q << 16) + kColA + 16 * half;
            tc::tmem_st16x128(col, regs(hi));
            tc::tmem_st16x128(col + 32, regs(lo));
          }
        }
        tc::tmem_wait_st();
        tc::fence_before();
        arrive(sm.wready[half]);
        arrive(sm.empty[s]);
        if (!kState) {
          if (g && !wait(sm.go, g - 1)) break;  // (the last one is read, and so is an end state)
          if (kept && !wait(sm.ffree, kept - 1)) break;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) split2(y[q][i], hi[i], lo[i]);
            const uint32_t col = tl + (16u * q << 16) + kColA + 64 + 16 * half;
            tc::tmem_st16x128(col, regs(hi));
            tc::tmem_st16x128(col + 32, regs(lo));
          }
          tc::tmem_wait_st();
          tc::fence_before();
          arrive(sm.vready);
        }
        if (!wait(sm.gs[half], g)) break;
        const float2 lam = make_float2(lam1, lam1);
#pragma unroll
        for (int m = 0; m < 4; m += 2) {
          float r[16], z[16];
          tc::tmem_ld16_nowait(tl + kColS + 64 * half + 16 * m, r);
          tc::tmem_ld16_nowait(tl + kColS + 64 * half + 16 * m + 16, z);
          tc::tmem_wait_ld2(r, z);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            S[8 * m + j] = tc::fma2(lam, S[8 * m + j], make_float2(r[2 * j], r[2 * j + 1]));
            S[8 * m + 8 + j] = tc::fma2(lam, S[8 * m + 8 + j], make_float2(z[2 * j], z[2 * j + 1]));
          }
        }
      }
      if (!ok) break;
      if (kTrain && x.run && x.last) {
        float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.st.out) + at);
#pragma unroll
        for (int j = 0; j < 16; ++j) dst[j] = reinterpret_cast<const float4*>(S)[j];
      }
      if (!keeps(x)) continue;
      // By way of tensor memory, in u's place and beta u's. (Stored from here, behind the tiles that are on their way, it took a
      // chunk's time.)
      if (!kState && half == 1 && g && !wait(sm.go, g - 1)) break;
      if (kept && !wait(sm.ffree, kept - 1)) break;
#pragma unroll
      for (int m = 0; m < 8; ++m) tc::tmem_st8(tl + (half ? kColA + 64 : kColU) + 8 * m, reinterpret_cast<const uint32_t*>(S + 4 * m));
      tc::tmem_wait_st();
      tc::fence_before();
      arrive(sm.fready);
      ++kept;
    }
    if (!ok && lane == 0) atomicOr(P.status, 1);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc::fence_after();
    tc::tmem_dealloc(tbase, 512);
  }
}

// Chains the segments of one (sequence, head), x <- x M + N: in, each segment's N and M but the last's; out, the state each
// segment starts from, in N's place. A CTA takes 32 of the state's 128 rows (independent of each other), a warp 16 columns. x
// stays in FP32; for the product it and M are in two BF16 parts (mma.sync: the chain is short products one after the other, and x comes
// out where the next turn's N is loaded). M comes in parts of 32 rows through a ring of asynchronous copies.
constexpr int kChainRows = 32, kChainThreads = 256, kPart = 32, kParts = kDim / kPart, kChainStages = 6;
constexpr int kPartBytes = 2 * kPart * kDim * 2;
constexpr int kChainSmem = kChainStages * kPartBytes + 2 * kChainRows * kDim * 2;
// Byte of (row, 16-byte piece) in a tile of 256-byte rows.
__device__ __forceinline__ uint32_t chain_piece(int row, int c) { return row * 256 + ((c ^ (row & 7)) << 4); }

__global__ void __launch_bounds__(kChainThreads) kda_delta_chain_kernel(const __grid_constant__ PassArgs a) {
  extern __shared__ __align__(16) unsigned char chain_smem[];
  __shared__ uint32_t bad[2];  // bits of the rows that are not finite, of two segments in turn
  const uint32_t ring = tc::smem_u32(chain_smem), xs = ring + kChainStages * kPartBytes;  // xs: x in two parts, [2][32][128]
  const DeltaProblem& P = a.P;
  const Segments& sg = a.sg;
  const int64_t n = blockIdx.x / P.Hv;
  const int h = (int)(blockIdx.x % P.Hv);
  const DecaySpan sp = decay_span(P, n);
  const int64_t slot = a.st.slots ? a.st.slots[n] : n;
  if (slot < 0 || slot >= a.st.num_slots) return;  // the main pass flags it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // this thread's values, as products leave them: rows r0 + 8 j, columns c0 + 8 t (and the next)
  const int r0 = lane >> 2, c0 = 16 * warp + 2 * (lane & 3);
  const int64_t base = seg_slot(sg, sp.t0, n);
  const int64_t m = sp.len > sg.len ? (sp.len + sg.len - 1) / sg.len : 1;
  auto at = [&](int64_t i) { return ((base + i) * P.Hv + h) * kDim * kDim; };
  auto own = [&](int j, int t) { return (kChainRows * (int)blockIdx.y + r0 + 8 * j) * kDim + c0 + 8 * t; };
  auto none_of = [&](int64_t i) { return i + 1 < m && sg.none[(base + i) * P.Hv + h] != 0; };
  bool none = none_of(0), none1 = none_of(1), none2 = none_of(2);  // of segment i and the next two
  int64_t i = 0;
  auto fetch = [&](int64_t p) {  // part p of all
    const int64_t k = p / kParts;
    if (k + 1 < m && !(k == i ? none : k == i + 1 ? none1 : none2)) {
      const __nv_bfloat16* src = sg.through + 2 * at(k) + (p % kParts) * kPart * kDim;
      unsigned char* dst = chain_smem + (p % kChainStages) * kPartBytes;
#pragma unroll
      for (int x = tid; x < kPartBytes / 16; x += kChainThreads) {
        const int part = x >> 9, row = (x >> 4) & 31, c = x & 15;
        tc::cp_async16(dst + part * (kPartBytes / 2) + chain_piece(row, c), src + part * kDim * kDim + row * kDim + 8 * c, 16);
      }
    }
    tc::cp_async_commit();
  };
  for (int p = 0; p < kChainStages - 1; ++p) fetch(p);
  if (tid < 2) bad[tid] = 0u;
  __syncthreads();
  float2 x[4][2], y1[4][2];
  const int64_t from = (slot * P.Hv + h) * kDim * kDim;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t k = from + own(j, t);
      if (!a.st.in) x[j][t] = make_float2(0.f, 0.f);
      else if (a.st.bf16) x[j][t] = unpack2(*reinterpret_cast<const uint32_t*>(reinterpret_cast<const __nv_bfloat16*>(a.st.in) + k));
      else x[j][t] = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(a.st.in) + k);
    }
  auto load = [&](int64_t k) {  // N of segment k
    if (k + 1 < m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t) y1[j][t] = *reinterpret_cast<const float2*>(sg.state + at(k) + own(j, t));
  };
  load(0);
  for (; i < m; ++i) {
    float2 y[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        y[j][t] = y1[j][t];
        *reinterpret_cast<float2*>(sg.state + at(i) + own(j, t)) = x[j][t];
      }
    if (i + 1 == m) break;
    load(i + 1);
    if (none) {
      // M is zero: what is not finite gives NaN for its row, as a product would
      uint32_t found = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t) found |= isfinite(x[j][t].x) && isfinite(x[j][t].y) ? 0u : 1u << (r0 + 8 * j);
      if (found) atomicOr(&bad[i & 1], found);
      __syncthreads();
      const uint32_t rows = bad[i & 1];
      const float nan = __int_as_float(0x7fc00000);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (rows >> (r0 + 8 * j) & 1u) y[j][0] = y[j][1] = make_float2(nan, nan);
      for (int p = 0; p < kParts; ++p) fetch(i * kParts + p + kChainStages - 1);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t hi, lo;
          split2(x[j][t], hi, lo);
          const uint32_t to = xs + chain_piece(r0 + 8 * j, 2 * warp + t) + 4 * (lane & 3);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(hi) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + kChainRows * 256), "r"(lo) : "memory");
        }
      float acc[2][2][4] = {}, cross[2][2][4] = {};  // [16 rows][8 columns]: of the high parts, of a high and a low one
#pragma unroll 1
      for (int p = 0; p < kParts; ++p) {
        const int64_t at_part = i * kParts + p;
        tc::cp_async_wait<kChainStages - 2>();
        __syncthreads();  // the part is there for all (and xs); the one before is read
        fetch(at_part + kChainStages - 1);
        const uint32_t Mp = ring + (uint32_t)(at_part % kChainStages) * kPartBytes;
        const int lr = (lane & 7) + 8 * ((lane >> 3) & 1), lc = lane >> 4;  // row and piece this lane gives the address of
#pragma unroll
        for (int k = 0; k < kPart / 16; ++k) {
          uint32_t bh[4], bl[4], ah[2][4], al[2][4];
          const uint32_t b = Mp + chain_piece(16 * k + lr, 2 * warp + lc);
          tc::ldmatrix4_trans(b, bh);
          tc::ldmatrix4_trans(b + kPartBytes / 2, bl);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t ax = xs + chain_piece(16 * q + lr, 2 * (p * (kPart / 16) + k) + lc);
            tc::ldmatrix4(ax, ah[q]);
            tc::ldmatrix4(ax + kChainRows * 256, al[q]);
          }
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              tc::mma_sync(acc[q][t], ah[q], bh + 2 * t);
              tc::mma_sync(cross[q][t], ah[q], bl + 2 * t);
              tc::mma_sync(cross[q][t], al[q], bh + 2 * t);
            }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float* c = acc[j >> 1][t] + 2 * (j & 1);
          const float* d = cross[j >> 1][t] + 2 * (j & 1);
          y[j][t] = make_float2(y[j][t].x + (c[0] + d[0]), y[j][t].y + (c[1] + d[1]));
        }
      __syncthreads();  // xs is read
    }
    none = none1;
    none1 = none2;
    none2 = none_of(i + 3);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t) x[j][t] = y[j][t];
  }
  tc::cp_async_wait_all();
}

template <bool kTrain, bool kState>
cudaError_t launch(const Maps& maps, const PassArgs& a, cudaStream_t s) {
  auto kern = kda_delta_fwd_kernel<kTrain, kState>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  const int64_t units = (a.sg.len ? a.first[a.sg.most] : a.P.N) * a.P.Hv * (kState ? 2 : 1);
  kern<<<(unsigned)units, kThreads, kSmemBytes, s>>>(maps, a);
  return cudaGetLastError();
}

template <bool kTrain>
cudaError_t forward(const DeltaProblem& P, const DecayStates& st, __nv_bfloat16* o, unsigned char* ws, cudaStream_t s) {
  Maps maps{};
  PassArgs a{};
  cudaError_t e;
  if (P.N * P.Hv == 0) return cudaSuccess;
  if (P.Ttot) {
    if ((e = token_map(&maps.q, P.q, P.Hqk, P.Ttot, P.qh, P.qt, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.k, P.k, P.Hqk, P.Ttot, P.kh, P.kt, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.v, P.v, P.Hv, P.Ttot, P.vh, P.vt, kC)) != cudaSuccess) return e;
    if ((e = token_map(&maps.o, o, P.Hv, P.Ttot, kDim, (int64_t)P.Hv * kDim, kC)) != cudaSuccess) return e;
  }
  a.P = P;
  a.st = st;
  const DeltaWs w = delta_workspace(P, kTrain);
  a.packets = ws + w.packet;
  a.stride = kTrain ? kPkTrain : kPkInfer;
  a.states = ws + w.states;
  a.u = ws + w.u;
  a.o = o;
  auto len = [&](int64_t n) { return P.cu_host ? P.cu_host[n + 1] - P.cu_host[n] : P.T; };
  if (P.cu_host && P.N > 1 && P.N <= kOrder) {
    a.ordered = 1;
    for (int64_t i = 0; i < P.N; ++i) a.order[i] = (uint16_t)i;
    std::stable_sort(a.order, a.order + P.N, [&](uint16_t i, uint16_t j) { return len(i) > len(j); });
  }
  a.sg.most = 1;
  if (!kTrain && P.seg) {
    if ((e = state_map(&maps.st, ws + w.segments, false, P.Hv, P.Ttot / P.seg + P.N)) != cudaSuccess) return e;
  } else if (!kTrain && st.in) {
    if ((e = state_map(&maps.st, st.in, st.bf16, P.Hv, st.num_slots)) != cudaSuccess) return e;
  }
  if (P.seg) {
    a.sg.len = P.seg;
    a.sg.most = (int)((P.longest + P.seg - 1) / P.seg);
    int64_t have = P.N;  // the sequences that have a segment s (longest first): all have the first
    for (int t = 0; t < a.sg.most; ++t) {
      while (t && have && len(a.ordered ? a.order[have - 1] : have - 1) <= t * P.seg) --have;
      a.first[t + 1] = a.first[t] + (int32_t)have;
    }
    a.sg.state = reinterpret_cast<float*>(ws + w.segments);
    a.sg.through = reinterpret_cast<__nv_bfloat16*>(ws + w.through);
    a.sg.none = reinterpret_cast<int32_t*>(ws + w.none);
    if ((e = launch<false, true>(maps, a, s)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(kda_delta_chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kChainSmem)) != cudaSuccess) return e;
    kda_delta_chain_kernel<<<dim3((unsigned)(P.N * P.Hv), kDim / kChainRows), kChainThreads, kChainSmem, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return launch<kTrain, false>(maps, a, s);
}

}  // namespace

int64_t delta_segment_tokens(const int64_t* cu, int64_t N, int64_t T, int64_t Hv) {
  if (N > kOrder) return 0;
  auto chunks_of = [&](int64_t n) { return ((cu ? cu[n + 1] - cu[n] : T) + kC - 1) / kC; };
  int64_t longest = 0, chunks = 0;
  for (int64_t n = 0; n < (cu ? N : 1); ++n) {
    chunks += chunks_of(n);
    longest = std::max(longest, chunks_of(n));
  }
  if (!cu) chunks *= N;
  const int64_t share = (chunks * Hv + kSms - 1) / kSms;  // an SM's even share of the chunks
  // Whole, the longest sequence takes its chunks' time; cut, all take their share two to three times (with decays that leave
  // nothing over a segment, or none), and some 20 chunks' time goes into launches and the chain. One after the other, in us, whole
  // and cut (with decays; without): 1 head, 1024 tokens 57, 71 (71), 2048 tokens 91, 75 (75); 8 heads, 2048 tokens 92, 77 (77);
  // 32 heads, 4096 tokens 179, 168 (169), 16384 tokens 655, 470 (530); 64 heads, 16384 tokens 732, 816 (923), 32771 tokens 1445, 1466
  // (1730).
  if (longest <= 3 * share + 20) return 0;
  // a quarter of it, so that the last turn is short, 8 chunks at least (and no more segments than are passed)
  const int64_t seg = std::max({(share + 3) / 4, (int64_t)8, (longest + kMost - 1) / kMost});
  return seg * kC;
}

cudaError_t launch_delta_forward(const DeltaProblem& P, const DecayStates& st, __nv_bfloat16* o, bool training, void* ws,
                                 cudaStream_t s) {
  const cudaError_t e = launch_delta_prep(P, training, ws, s);
  if (e != cudaSuccess) return e;
  unsigned char* w = reinterpret_cast<unsigned char*>(ws);
  return training ? forward<true>(P, st, o, w, s) : forward<false>(P, st, o, w, s);
}

}  // namespace kda
