// What the launch rules share of the card.  Plain C++: tests compile it without CUDA.
#pragma once

#include <stddef.h>

namespace moe {

constexpr int kSms = 152;
constexpr size_t kSmemSm = 227 * 1024;             // shared memory of an SM that its blocks share
// Dynamic shared memory that a block may ask for: the limit that allow_smem sets and every rule plans with.  The rest is
// for a kernel's static arrays.
constexpr size_t kSmemBlock = kSmemSm - 2048;

// Blocks for n rows, `each` of them a block; n may be the largest int.
inline int blocks_of(int n, int each) { return n > 0 ? (n - 1) / each + 1 : 0; }

}  // namespace moe
