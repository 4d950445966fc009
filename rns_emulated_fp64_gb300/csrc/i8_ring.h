// The shared memory of k_i8few.cu: a ring of stages between the TMA warp and the
// warps that multiply.  Plain C++, so that its protocol can be followed without a GPU.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace os2i8 {

constexpr int kFewWarps = 8;              // of a group, 16 channels each
constexpr uint32_t kFewW = 128 * 128;     // a stage's weights: 128 channels x 128 terms

template <int NG>
struct Few {
  // Up to 16 tokens, two groups of warps take the stages in turn: 17.9 us against 19.1
  // for one token and 32000 x 2048 weights (before the ring was filled step by step), 8.3
  // against 8.8 for 4096 x 4096; above,
  // their exchange costs more than it gives (25.1 against 24.2 for 32 tokens).
  static constexpr int groups = NG <= 2 ? 2 : 1;
  static constexpr int all = kFewWarps * groups, threads = 32 * all + 32;
  static constexpr uint32_t block = NG * 8 * 128;       // 64 terms of the tokens
  static constexpr uint32_t stage = kFewW + 2 * block;
  static constexpr uint32_t part = all * NG * 32 * 16;  // a tile's sums, one side
  static constexpr int fit = (int)((227 * 1024 - 1024 - 512 - 2 * part) / stage);
  // A slot of the ring always belongs to one group, which then waits for each of the slot's
  // phases.  Were the number of slots no multiple of the groups', a group would meet every
  // second phase of a slot only; these have the same parity, so that its wait for one that
  // has not come could pass on the one before.
  static constexpr int stages = fit / groups * groups;
  static_assert(stages >= 2 * groups && stages % groups == 0, "slots of the ring");
  static constexpr size_t smem = 1024 + (size_t)stages * stage + 2 * part + 512;
};

}  // namespace os2i8
