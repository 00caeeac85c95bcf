// packed.hpp -- sequences laid one behind the other: where they start, and which
// of them a range of tokens meets (device code shared by the packed scan and the
// short convolution).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssmq {

struct Seqs {
  const int32_t* offsets;   // (S + 1), or null: seqlen tokens each
  const int32_t* slot;      // (S) or null: s
  const uint8_t* resume;    // (S) or null: all
  int32_t tokens, S;
  int32_t seqlen;
  int32_t slots;
};

typedef const int32_t __attribute__((address_space(4)))* const_i32_ptr;

__device__ __forceinline__ int32_t in_tokens(const Seqs& q, int32_t v) {
  return v < 0 ? 0 : v > q.tokens ? q.tokens : v;
}

// First token of sequence i (wave-uniform); that of S is the end of the last one.
__device__ __forceinline__ int32_t seq_start(const Seqs& q, int32_t i) {
  return q.offsets ? in_tokens(q, ((const_i32_ptr)(q.offsets))[i]) : i * q.seqlen;
}

// How many sequences start before token t (whole waves call it).  The lanes sample
// the offsets 64 at a time, so up to 64 sequences cost one load, 4096 two.
__device__ __forceinline__ int32_t seqs_before(const Seqs& q, int32_t t) {
  if (!q.offsets) {
    if (t <= 0 || q.seqlen == 0) return t > 0 ? q.S : 0;
    const int32_t n = int32_t((uint32_t(t) + uint32_t(q.seqlen) - 1) / uint32_t(q.seqlen));   // (past 31 bits)
    return n < q.S ? n : q.S;
  }
  const int32_t lane = threadIdx.x & 63;
  int32_t lo = 0, n = q.S;   // below lo they start before t; from lo + n on they do not
  while (n > 0) {
    const int32_t step = (n + 63) >> 6;
    const bool below = lane * step < n && in_tokens(q, q.offsets[lo + lane * step]) < t;
    const int32_t c = __popcll(__builtin_amdgcn_ballot_w64(below));
    if (c == 0) break;
    const int32_t from = (c - 1) * step + 1, to = c * step < n ? c * step : n;
    lo += from;
    n = to - from;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// The slot of sequence s, or -1 where it has none (wave-uniform).
__device__ __forceinline__ int32_t seq_slot(const Seqs& q, int32_t s) {
  const int32_t v = q.slot ? ((const_i32_ptr)(q.slot))[s] : s;
  return v >= 0 && v < q.slots ? v : -1;
}

__device__ __forceinline__ bool seq_resumed(const Seqs& q, int32_t s) {
  return !q.resume || __builtin_amdgcn_readfirstlane(int32_t(q.resume[s])) != 0;
}

}  // namespace ssmq
