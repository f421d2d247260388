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
// the other parts through.  The first part is `front` times as long as the others: where pass 1 takes the blocks for M and N
// in `front` waves, those of the first part go on beside them all the while.  (One sequence, us whole | in parts, as cut below:
// 32 heads of 128 x 128, 1,920 tokens 103 | 102, 3,840 197 | 158, 12,288 592 | 399, with equal parts 457; 64 heads, 3,840 tokens
// 237 | 232, 12,288 710 | 632; 8 heads, 1,536 tokens 79 | 68, 12,288 507 | 182.)
constexpr int kCutChunks = 24;     // of a sequence that is cut
constexpr int kPartChunks = 5;     // of a part at least
constexpr int kCutCost = 10;       // chunks that have to be saved: what joining and a second pass cost (64 heads, 2,560 tokens, where
                                   // cutting saves 10: 163 us whole, 168 in parts when this was chosen)
struct DeltaParts {
  int parts, first, len;          // parts of the n chunks of a sequence in this window, chunks of the first and of the others
};
MOE_HD DeltaParts delta_parts(int n, int most, int front) {
  if (n >= kCutChunks && most >= 3) {
    const int fits = n / kPartChunks - front + 1, p = fits < most ? fits : most;
    if (p >= 3) {
      const int len = (n + front + p - 2) / (front + p - 1), rest = n - front * len;
      const int parts = 1 + (rest + len - 1) / len;
      if (parts >= 3) return DeltaParts{parts, front * len, len};
    }
  }
  return DeltaParts{1, n, n};
}
// blocks of a head in pass 1
MOE_HD int delta_pass1_blocks(int parts, int dk, int dv) { return 1 + (parts - 2) * (1 + (dk + dv - 1) / dv); }

struct DeltaCut {
  int parts, front;               // parts 1: not cut
};
// How the sequences of a call are cut: for the fewest chunks one after another in both passes, with as many blocks at a time
// as there are SMs, and at most `most` parts and `cuts` heads' parts in all (what the buffers hold).
MOE_HD DeltaCut delta_cut(int n_seqs, int hv, int dk, int dv, int longest, int num_sms, int cuts, int most) {
  DeltaCut best{1, 1};
  const int64_t chains = (int64_t)n_seqs * hv;
  if (longest < kCutChunks || chains >= num_sms) return best;
  int64_t least = longest - kCutCost;
  for (int p = 3; p <= most && chains * p <= cuts; ++p) {
    const int64_t side = num_sms - chains, finds = chains * (delta_pass1_blocks(p, dk, dv) - 1);
    const int64_t front = (finds + side - 1) / side, waves = (chains * (p - 1) + num_sms - 1) / num_sms;
    const int64_t len = (longest + front + p - 2) / (front + p - 1);
    if (len < kPartChunks) break;
    if ((front + waves) * len < least) {
      least = (front + waves) * len;
      best = DeltaCut{p, (int)front};
    }
  }
  return best;
}

// Sequences of a call whose blocks start in the order of their lengths: nine prompts of 200 to 6,001 tokens, the longest last,
// 464 us as they come, 413 so (the longest first 413 either way).  More of them fill the SMs in any
// order, and where every block has an SM there is none to choose.
constexpr int kOrdered = 128;
MOE_HD bool delta_ordered(int n_seqs, int hv, int num_sms) { return n_seqs > 1 && n_seqs <= kOrdered && (int64_t)n_seqs * hv > num_sms; }

// Chunks that the work space holds at a time: K and Q of hk key heads, T's pairs and P of hv value heads, and their scalars.
// (544 MB are 420 chunks of 16 key and 32 value heads of 128 x 128; sequences go on alone in the next window: nine prompts of
// 16,900 tokens, the longest 6,000, 478 to 504 us with half as much, 413 us.)
constexpr int64_t kWorkBytes = 544ll << 20;
constexpr int kTPBytes = 3 * kChunk * 128;        // T's two halves and P of a value head: rows of 128 bytes
constexpr int kScalarBytes = (5 * kChunk + 16) * 4 + kChunk;
MOE_HD int64_t delta_chunk_bytes(int hk, int hv, int dk) {
  return (int64_t)hk * 2 * kChunk * dk * 2 + (int64_t)hv * (kTPBytes + kScalarBytes);
}
MOE_HD int delta_window(int hk, int hv, int dk) { return (int)(kWorkBytes / delta_chunk_bytes(hk, hv, dk)); }

// The order in which n chunks' copies go into a ring of stages: freed(stage, parity) waits until a stage may be overwritten
// (false: that wait gave up, so nothing more is copied, as the stage's last copy may still be under way), bring(i, stage)
// starts the copies of chunk i, landed(stage, parity) waits for the last ones of each stage.  These waits are made in any case: a
// block's shared memory is another block's when it has ended.
template <class Freed, class Bring, class Landed>
MOE_HD void delta_deliver(int n, int stages, Freed freed, Bring bring, Landed landed) {
  int i = 0;
  for (; i < n; ++i) {
    if (i >= stages && !freed(i % stages, (uint32_t)(i / stages - 1) & 1)) break;
    bring(i, i % stages);
  }
  for (int j = i > stages ? i - stages : 0; j < i; ++j) landed(j % stages, (uint32_t)(j / stages) & 1);
}

}  // namespace moe
