// mq_kv.cuh -- what the append to the paged E4M3 cache and the attention over
// it share: the page scale's range and its powers of two.
#pragma once
#include <cstdint>

namespace mq {

// A page's scale is 2^e, e in this range: 448 * 2^119 is the largest bf16's
// binade, and 2^96 * (number of tokens) still fits binary32, which the
// attention's sums of 2^-e-weighted terms need.
constexpr int KV_E_MIN = -96, KV_E_MAX = 119;

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

}  // namespace mq
