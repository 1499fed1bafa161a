// twq_check.h -- argument limits and checks shared by the C ABI sources.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace twq {

constexpr int64_t kMaxM = 131072;    // keeps 256 * 49 * m below 2^31 in the int32 accumulator
constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxN = int64_t(1) << 24;
constexpr int64_t kMaxRank = 256;

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool valid_m(int64_t m) { return m > 0 && m % 128 == 0 && m <= kMaxM; }
inline bool valid_b(int64_t b) { return b >= 0 && b <= kMaxTokens; }
inline bool valid_n(int64_t n) { return n >= 0 && n % 16 == 0 && n <= kMaxN; }
inline bool valid_r(int64_t r) { return r >= 0 && r % 16 == 0 && r <= kMaxRank; }
inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace twq
