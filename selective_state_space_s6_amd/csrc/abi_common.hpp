// abi_common.hpp -- what the files of the extern "C" boundary share: the calling
// thread's error message, the status of a launch, and the argument checks.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ssm_scan.h"

namespace ssm {

// sets ssm_last_error()'s message and returns code
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// the status of a launch: SSM_OK (and an empty message) or SSM_ERR_HIP
int launched(const char *entry, hipError_t e, const char *kernel);

inline bool aligned16(const void *p) { return p == nullptr || ((uintptr_t)p & 15u) == 0; }

// elements of a tensor must stay addressable with 64-bit offsets and the grid
// with 32-bit block counts
inline bool too_big(int64_t a, int64_t b, int64_t c, int64_t d) {
    const double n = (double)a * (double)b * (double)c * (double)d;
    return n > 9.0e15;
}

}  // namespace ssm

#define REQUIRE_PTR(entry, p)                                                        \
    do {                                                                             \
        if ((p) == nullptr) return ssm::fail(SSM_ERR_INVALID_ARG, "%s: %s is NULL", entry, #p); \
    } while (0)
#define REQUIRE_POS(entry, v)                                                                  \
    do {                                                                                       \
        if ((v) <= 0) return ssm::fail(SSM_ERR_INVALID_ARG, "%s: %s must be > 0 (got %lld)", entry, \
                                       #v, (long long)(v));                                    \
    } while (0)
#define REQUIRE_ALIGN(entry, p)                                                                 \
    do {                                                                                        \
        if (!ssm::aligned16(p)) return ssm::fail(SSM_ERR_UNSUPPORTED, "%s: %s is not 16-byte aligned", \
                                                 entry, #p);                                    \
    } while (0)
