// int4_host.hpp -- sizes of 4-bit weights, as the host code of the product and
// of the expert layers needs them.
#pragma once

#include "host_common.hpp"

namespace fg {

// 32, 64 or a multiple of 128.
fg_status check_group(int group);

inline int int4_groups(int K, int group) { return (K + group - 1) / group; }
// Rows are padded to whole chunks of 128 codes.
inline int int4_row_bytes(int K) { return (K + 127) / 128 * 64; }

// The scales (zero points) of a chunk's groups are one aligned load: every row
// starts a whole number of chunks into arrays that are aligned to it.
inline bool int4_wide(int K, const void* s, const void* z) {
  return K % 128 == 0 && ((uintptr_t)s & 7) == 0 && ((uintptr_t)z & 3) == 0;
}

}  // namespace fg
