// Launchers of the row kernels that rlk_api.hip builds, for the other
// translation units; internal to the library (not exported).  They only
// enqueue the launch on `st`; the caller checks hipGetLastError.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rlk {

// compact_rows: the rows t with y[t] != ignore_index, ascending, into idx
// (their y into yA unless NULL) and their number into n_act; zero0 .. zero2
// (each NULL or [T]) are set to 0 at the other rows.
__attribute__((visibility("hidden"))) void launch_compact_rows(hipStream_t st, const int32_t* y, int T,
                                                              int ignore_index, int32_t* idx, int32_t* yA,
                                                              int32_t* n_act, float* zero0, float* zero1,
                                                              float* zero2);

}  // namespace rlk
