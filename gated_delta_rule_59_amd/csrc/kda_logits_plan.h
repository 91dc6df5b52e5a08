// Launch shapes of the adjusted logits, which depend on sizes only. Host only.
#pragma once

#include <cstdint>

namespace kda {

constexpr int kLogitsThreads = 256, kLogitsEach = 4;  // a thread takes kLogitsEach neighbouring tokens at a time

// How many times that is a block of a row.
//
// Blocks of 1,024 tokens while there are no more than six to a CU, else of 4,096: small ones take less time
// each, but every one goes through the whole history. (Histories of 2,000, one of 32,000 tokens: 9.5 us,
// with blocks of 4,096 15.9; 48 of them, the rule's last: 15.3, 17.0; 64: 18.6, 17.4; 128: 29.3, 21.1. Five
// rows of 131,072: 13.8, 15.3; 15 of them: 22.9, 15.9.)
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
// count the history once. (Five rows of 131,072 each, one sequence: 13.8 us, together 29.6; 8 sequences:
// 27.4, 32.6; 12, the rule's last: 33.1, 33.2; 16: 41.5, 33.9; 32: 74.4, 45.6.)
inline int logits_splits(int N, int R, int64_t blocks) { return (int64_t)N * R * blocks <= 2048 ? R : 1; }

}  // namespace kda
