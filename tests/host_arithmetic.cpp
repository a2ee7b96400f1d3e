// The library's host and plan arithmetic as C functions, for tests on the CPU.
#include "internal.h"

extern "C" {

int64_t cache_slice_rows(int rows) { return kda::cache_slice_rows(rows); }

}  // extern "C"
