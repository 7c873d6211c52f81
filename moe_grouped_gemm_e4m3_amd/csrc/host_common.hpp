// host_common.hpp -- what the library's translation units share on the host:
// the thread's error text, the CU count and the launch helpers built on them.
// The definitions are in fp8gemm.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8gemm.h"

namespace fg {

// Clears the thread's error text (every entry point does this first).
void clear_error();
// Sets the thread's error text and returns st.
fg_status set_error(fg_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Compute units of the current device, at most fg_set_num_cus()'s cap; whether
// the cap took any.
fg_status usable_cus(int* cus, bool* capped = nullptr);
// The environment asks for a line on every launch (FG_PRINT_CONFIGS).
bool print_launches();
// FG_EINVAL / FG_EALIGN with the argument's name where a pointer or a row
// stride does not fit.
fg_status require_ptr(const void* p, uintptr_t align, const char* name);
fg_status require_ld(int64_t ld, int64_t row, int64_t mult, const char* name);

}  // namespace fg
