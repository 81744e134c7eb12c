// Declarations of distill.cu for the library's other translation units.
#pragma once

#include "tbe_internal.cuh"

namespace tbe {

// Self-test of the time limit of the slices' copies.
size_t distill_selftest_bytes();
tbe_status launch_distill_selftest(Launch &L, void *ws, int32_t *status);

}  // namespace tbe
