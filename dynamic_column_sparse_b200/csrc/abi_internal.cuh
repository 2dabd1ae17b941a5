// abi_internal.cuh - helpers of the C ABI implementation shared between its
// translation units (api.cu defines them).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/chipmunk.h"

namespace cm {

// Records `msg` for chipmunk_last_error (this host thread) and returns st.
chipmunk_status record_error(chipmunk_status st, const char *msg);

// Records a formatted message and returns st.
chipmunk_status record_errorf(chipmunk_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));

// Checks that the current device is sm_100 and resolves its status word.
chipmunk_status device_ready(int **status_out);

// Tensor map of rank 2 or 3 (128-byte swizzle or none); dims, strides (from the
// second dimension on, in bytes) and box innermost first.
chipmunk_status encode_map(CUtensorMap *m, CUtensorMapDataType type, const void *base, int rank, const uint64_t *dims,
                           const uint64_t *strides, const uint32_t *box, bool swizzled, const char *what);

// chipmunk_mlp_delta with its delta scratch taken from get_scratch instead of
// a caller workspace. The arguments are checked first; a step that needs more
// than scratch_bytes is rejected with CHIPMUNK_ERR_WORKSPACE before anything
// else happens. get_scratch runs after the device checks, with the caller's
// device current.
chipmunk_status mlp_delta_fixed_scratch(const chipmunk_mlp_args *a, size_t scratch_bytes,
                                        chipmunk_status (*get_scratch)(void **), cudaStream_t s);

}  // namespace cm
