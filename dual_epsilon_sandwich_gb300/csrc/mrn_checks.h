// mrn_checks.h -- argument checks shared by the C entry points (mrn_api.cpp,
// mrn_train_api.cpp), and what both need of the launch state.  Host only; not
// part of the public ABI.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_runtime_api.h>

#include "mrn.h"

namespace mrn {

inline int elem_bytes(mrn_dtype dt) { return dt == MRN_F32 ? 4 : 2; }

struct Span {
    uintptr_t lo;
    uintptr_t hi;
};

inline Span span_of(const void *p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Span{lo, lo + static_cast<uintptr_t>(bytes)};
}

inline bool overlaps(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

// An output may coincide exactly with a row input or be disjoint from it.
inline bool output_vs_row_input_ok(Span out, Span in) { return !overlaps(out, in) || out.lo == in.lo; }

inline mrn_status check_common(int64_t rows, int64_t n, mrn_dtype dt, float eps1, float eps2) {
    if (dt != MRN_F32 && dt != MRN_BF16) return MRN_ERR_UNSUPPORTED_DTYPE;
    if (n < 1 || rows < 0) return MRN_ERR_INVALID_SIZE;
    const int64_t e = elem_bytes(dt);
    if (n > INT64_MAX / e) return MRN_ERR_INVALID_SIZE;
    if (rows > 0 && rows > INT64_MAX / (n * e)) return MRN_ERR_INVALID_SIZE;
    if (!(eps1 > 0.0f) || !std::isfinite(eps1)) return MRN_ERR_INVALID_EPS;
    if (!(eps2 > 0.0f) || !std::isfinite(eps2)) return MRN_ERR_INVALID_EPS;
    return MRN_OK;
}

inline bool aligned_to(const void *p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// SM count of the current device (GB300's where it cannot be asked).
int sm_count_of_current_device();
// The calling thread's launch option MRN_LAUNCH_PDL.
bool launch_pdl();
// ... and 16 with MRN_LAUNCH_TEST_WAIT_TIMEOUT, else 0.
uint32_t launch_stall_bytes();
// Counts a call's launches and turns its CUDA error into a status.
mrn_status launch_result(cudaError_t err, uint64_t launched);

}  // namespace mrn
