// Arithmetic of the gated delta rule's chunks that needs no device: their numbers,
// and how few long sequences are cut into parts.  Plain C++, so that a host
// compiler can build it alone.
#pragma once

#include "attn_plan.h"

namespace moe {

constexpr int kChunk = 64;       // tokens of a chunk

// The chunks of a sequence that begins at token t0 have the numbers from delta_chunk_base on (those of two sequences never
// meet: floor((t0 + n) / 64) + 1 - floor(t0 / 64) >= ceil(n / 64)).
MOE_HD int delta_chunk_base(int t0, int s) { return t0 / kChunk + s; }

// Few long sequences leave most SMs without work, as a state's chunks follow one another.  But a chunk, and so a part of a
// sequence, takes the state S before it to M S + N.  Pass 1 takes the first part through, and finds M and N of every other
// one but the last (M from the identity without V, N from zeros); joining them gives the states before the parts; pass 2 takes
// the other parts through.  That is at most three times the work in 2 / parts of the time.  (One sequence of 32 heads, us whole |
// in parts: 960 tokens 60 | 67, 1,280 74 | 78, 1,920 103 | 99, 3,840 197 | 168, 12,288 591 | 458; of 8 heads 57 | 61, 69 | 68,
// 93 | 82, 167 | 118, 508 | 206.)
constexpr int kCutChunks = 24;     // of a sequence at least
constexpr int kPartChunks = 5;     // of a part at least
struct DeltaParts {
  int parts, len;                 // parts of the n chunks of a sequence in this window, chunks of a part but the last
};
MOE_HD DeltaParts delta_parts(int n, int most) {
  int p = n / kPartChunks < most ? n / kPartChunks : most;
  if (n < kCutChunks) p = 1;
  const int len = (n + p - 1) / p;
  return DeltaParts{(n + len - 1) / len < 3 ? 1 : (n + len - 1) / len, (n + len - 1) / len < 3 ? n : len};
}
// blocks of a head in pass 1
MOE_HD int delta_pass1_blocks(int parts, int dk, int dv) { return 1 + (parts - 2) * (1 + (dk + dv - 1) / dv); }

// Parts of the sequences of a call (1: not cut): as many as pass 1 finds an SM for, and the part buffers hold `cuts` of.
MOE_HD int delta_cut(int n_seqs, int hv, int dk, int dv, int longest, int num_sms, int cuts, int most) {
  if (longest < kCutChunks) return 1;
  int parts = 2;
  while (parts < most && parts * kPartChunks < longest && (int64_t)n_seqs * (parts + 1) * hv <= cuts &&
         (int64_t)n_seqs * hv * delta_pass1_blocks(parts + 1, dk, dv) <= num_sms)
    ++parts;
  return parts < 3 ? 1 : parts;
}

}  // namespace moe
