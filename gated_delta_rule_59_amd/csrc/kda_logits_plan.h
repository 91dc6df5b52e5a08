// Launch shapes of the adjusted logits, which depend on sizes only. Host only.
#pragma once

#include <cstdint>

namespace kda {

constexpr int kLogitsThreads = 256, kLogitsEach = 4;  // a thread takes kLogitsEach neighbouring tokens at a time

// How many times that is a block of a row.
//
// Blocks of 1,024 tokens while there are no more than six to a CU, else of 4,096: small ones take less time
// each, but every one goes through the whole history. (Histories of 2,000, one of 32,000 tokens: 9.7 us,
// with blocks of 4,096 15.9; 48 of them, the rule's last: 14.8, 17.5; 64: 18.8, 17.9; 128: 29.4, 22.6. Five
// rows of 131,072: 12.9, 15.8; 15 of them: 21.8, 17.0.)
inline int logits_steps(int N, int R, int V) {
  return (int64_t)N * R * (((int64_t)V + 1023) / 1024) <= 1536 ? 1 : 4;
}

inline int64_t logits_blocks(int V, int steps) {
  const int block = steps * kLogitsThreads * kLogitsEach;
  return ((int64_t)V + block - 1) / block;
}

// How many workgroups share the rows of a sequence.
//
// One row of a sequence to a workgroup while all rows' blocks fit the card's places at once, else all, which
// count the history once. (Five rows of 131,072 each, one sequence: 12.9 us, together 28.4; 8 sequences:
// 29.7, 34.2; 12, the rule's last: 35.6, 36.4; 16: 45.3, 37.0; 32: 81.0, 48.1.)
inline int logits_splits(int N, int R, int64_t blocks) { return (int64_t)N * R * blocks <= 2048 ? R : 1; }

}  // namespace kda
