// la_check.h - argument checks shared by the C ABI's files.
#pragma once
#include <climits>
#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include "la.h"

namespace la {
namespace check {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Host-side fault injection for tests: LA_FAULT_INJECT=launch makes every
// compute entry point report a failed launch without enqueuing anything.
inline bool launch_fault_injected() {
    const char* e = std::getenv("LA_FAULT_INJECT");
    return e && std::strcmp(e, "launch") == 0;
}

inline bool fits_int(long long x) { return x >= 0 && x <= INT_MAX; }

inline la_status check_decay(const la_decay* decay, int* kind, const float** log_g) {
    *kind = LA_DECAY_NONE;
    *log_g = nullptr;
    if (!decay) return LA_OK;
    if (decay->kind < LA_DECAY_NONE || decay->kind > LA_DECAY_PER_STEP) return LA_ERR_INVALID_ARG;
    *kind = decay->kind;
    if (*kind != LA_DECAY_NONE) {
        if (!decay->log_g || !aligned4(decay->log_g)) return LA_ERR_INVALID_ARG;
        *log_g = decay->log_g;
    }
    return LA_OK;
}

inline size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace check
}  // namespace la
