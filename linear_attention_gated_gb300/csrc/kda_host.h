// kda_host.h -- host-side helpers shared by the C entry points: problem-size
// limits and the exception barrier in front of every call that allocates host
// memory.
#pragma once

#include <cstdint>
#include <new>
#include <vector>

#include "../../include/kda.h"

namespace kda {

void set_last_error(const char* msg);

// Upper bounds on a problem, checked before anything is sized from it, so that no
// byte count or index product overflows 64 bits and no host table is built from an
// absurd count: at most 2^40 tokens, 2^40 token-heads and 2^20 value heads, and no
// more sequences than tokens. Expects B, T, Hv >= 1; num_seqs is 0 for the fixed
// layout. Returns a description of the first bound broken, or nullptr.
inline const char* size_limit_violation(int64_t B, int64_t T, int64_t Hv, int64_t num_seqs) {
  constexpr int64_t kMaxTokens = int64_t(1) << 40, kMaxHeads = int64_t(1) << 20;
  if (Hv > kMaxHeads) return "more than 2^20 value heads";
  if (T > kMaxTokens / B) return "more than 2^40 tokens";
  if (B * T > kMaxTokens / Hv) return "more than 2^40 token-heads";
  if (num_seqs > B * T) return "more sequences than tokens";
  return nullptr;
}

// Bounds on a strided [tokens, heads, D] view (token and head strides ts, hs in elements, hs >= D >= 1 checked here) and
// on a state pool, for the same reason: views of at most 2^56 elements, pools of 2^40 states.
inline bool view_rows_apart(int64_t tokens, int64_t heads, int64_t D, int64_t ts, int64_t hs, bool* too_large) {
  constexpr int64_t kMaxElements = int64_t(1) << 56;
  *too_large = hs > kMaxElements / heads || ts > kMaxElements / (tokens > 0 ? tokens : 1);
  return *too_large || (hs >= D && ts >= (heads - 1) * hs + D);
}
inline bool pool_too_large(int64_t slots, int64_t Hv) { return slots > (int64_t(1) << 40) / Hv; }

// The first fault of N slot indices of a pool of `slots`: 1 out of range, 2 a slot used twice, 0 none. (A bit for
// each slot in a buffer kept per thread; only the words touched are cleared again.)
inline int slot_fault(const int32_t* idx, int64_t N, int64_t slots) {
  static thread_local std::vector<uint64_t> seen;
  for (int64_t i = 0; i < N; ++i)
    if (idx[i] < 0 || idx[i] >= slots) return 1;
  if (N < 2) return 0;
  const size_t words = (size_t)(slots + 63) / 64;
  if (seen.size() < words) seen.resize(words, 0);
  int64_t n = 0;
  int fault = 0;
  for (; n < N; ++n) {
    uint64_t& w = seen[(size_t)idx[n] >> 6];
    const uint64_t bit = uint64_t(1) << (idx[n] & 63);
    if (w & bit) {
      fault = 2;
      break;
    }
    w |= bit;
  }
  for (int64_t i = 0; i < n; ++i) seen[(size_t)idx[i] >> 6] = 0;
  return fault;
}

// Runs the body of a C entry point. A host exception (std::bad_alloc while
// building the launch plan, say) becomes a status and a message instead of
// crossing the C ABI, where it would end the process.
template <typename F>
kda_status guarded(F&& body) {
  try {
    return body();
  } catch (const std::bad_alloc&) {
    set_last_error("host memory exhausted while validating or planning the call");
    return KDA_ERR_INVALID_ARGUMENT;
  } catch (...) {
    set_last_error("unexpected host-side exception");
    return KDA_ERR_INVALID_ARGUMENT;
  }
}

}  // namespace kda
