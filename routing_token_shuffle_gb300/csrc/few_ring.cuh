// The stage ring of the few-token layer: how many stages fit, and which of its fp32 consumer
// groups takes which block. Plain C++, so that the rule below is checked on the host.
#pragma once

#include <stddef.h>

#ifdef __CUDACC__
#define SMOE_HD __host__ __device__ __forceinline__
#else
#define SMOE_HD inline
#endif

namespace smoe {

constexpr int kFewMaxCtas = 160;            // one per SM
constexpr int kFewMaxStages = 16;
constexpr int kFewSmem = 227 * 1024;
constexpr int kGateThreads = 320;           // warps 2-11 compute logits and select
constexpr int kFewStageA = 128 * 128;       // A tile: 128 rows x 128 bytes

// Floats between the rows of the exchange buffer: odd, or for 16-byte accesses an odd number
// of them.
SMOE_HD constexpr int few_xch(bool f32) { return f32 ? 20 : 17; }

// Shared memory beside the stages.
SMOE_HD constexpr size_t few_misc_bytes(bool f32, size_t E, size_t TK) {
  return 1024 + (2 * kFewMaxStages + 6) * 8 + 8 * E + 16 +
         4 * (kGateThreads + (size_t)(f32 ? 4 : 1) * 128 * few_xch(f32) + 192) + 4 * E + 8 * TK +
         (f32 ? 4 * (E + 1 + 2 * (kFewMaxCtas + 1)) : 0);
}

// fp32: the consumer group that takes the i-th block of a segment; the other steps over it.
SMOE_HD constexpr int few_group(int i) { return i & 1; }

// Stages that fit, nd rows of 128 bytes in a B tile. fp32: an even number, so that within a
// segment a stage belongs to one group, which has waited for the stage's last block when it
// waits for the next one (a barrier of both groups ends every segment). On an odd ring a group
// would wait on a stage whose last block was the other group's and may not have landed, and a
// barrier two phases behind passes for one that is done.
SMOE_HD constexpr int few_stages(bool f32, size_t E, size_t TK, int nd) {
  const size_t room = (kFewSmem - few_misc_bytes(f32, E, TK)) / (kFewStageA + (size_t)nd * 128);
  const int fit = room < kFewMaxStages ? (int)room : kFewMaxStages;
  return f32 ? fit & ~1 : fit;
}

}  // namespace smoe
