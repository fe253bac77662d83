// fp8.h -- internal: what the 8-bit quantization (fp8_quantize.cu) and product (fp8_matmul.cu) share.
//
// Rows that belong to groups (experts) are named by offset[groups + 1] in device memory: group g holds rows
// [offset[g], offset[g + 1]). Along the rows (the inner dimension of a weight's gradient) a block of 128 never spans two
// groups: each group starts a block of its own, and the last block of a group is filled up with zeros.
#pragma once

#include <stdint.h>

#include "relay.h"

namespace relay {

constexpr int kBlock = 128;  // values that share a scale

inline int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// Reads and clears the product's fault word -- fp8_matmul.cu.
cudaError_t fp8_read_fault(unsigned* fault);

#ifdef __CUDACC__
// offset[i] as a row number, whatever is there: no access goes by a value outside [0, rows].
__device__ __forceinline__ int offset_at(const int32_t* offset, int i, int rows) { return min(max(offset[i], 0), rows); }
#endif

}  // namespace relay
