// int4_host.hpp -- sizes of 4-bit weights, as the host code of the product and
// of the expert layers needs them.
#pragma once

#include "host_common.hpp"
#include "weight_stream.hpp"

namespace fg {

// 32, 64 or a multiple of 128.
fg_status check_group(int group);

inline int int4_groups(int K, int group) { return K / group + (K % group != 0); }
// Rows are padded to whole chunks of 128 codes.
inline int int4_row_bytes(int K) { return (K + 127) / 128 * 64; }

// f.run<Format>() for the format of a call.
template <class F>
fg_status with_int4_format(int group, bool zeros, const F& f) {
  if (group == 32) return zeros ? f.template run<Int4Group<4, true>>() : f.template run<Int4Group<4, false>>();
  if (group == 64) return zeros ? f.template run<Int4Group<2, true>>() : f.template run<Int4Group<2, false>>();
  return zeros ? f.template run<Int4Group<1, true>>() : f.template run<Int4Group<1, false>>();
}

}  // namespace fg
