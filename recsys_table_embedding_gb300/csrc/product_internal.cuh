// Declarations of product.cu for the library's other translation units.
#pragma once

#include "tbe_internal.cuh"

namespace tbe {

// Self-test of the time limits of the products' waits.
size_t product_selftest_bytes();
tbe_status launch_product_selftest(Launch &L, void *ws, int32_t *status);

}  // namespace tbe
