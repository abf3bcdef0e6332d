// kda_api_util.hpp -- argument checks shared by the extern "C" layer's files.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <limits>

#include "../../include/kda.h"
#include "kda_internal.hpp"
#include "kda_linear.hpp"

namespace {

bool valid_dtype(int dt) { return dt == KDA_F32 || dt == KDA_BF16; }
int64_t esize(int dt) { return dt == KDA_F32 ? 4 : 2; }
bool supported_d(int32_t d) { return d == 64 || d == 128; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
Range range(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + static_cast<uintptr_t>(bytes > 0 ? bytes : 0)};
}
bool overlap(Range a, Range b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

kda_status from_hip(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

bool aligned16(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
    return true;
}
bool aligned4(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return false;
    return true;
}

// No output overlaps an input or another output.
bool disjoint(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range* a = outs.begin(); a != outs.end(); ++a) {
        for (const Range* b = a + 1; b != outs.end(); ++b)
            if (overlap(*a, *b)) return false;
        for (const Range& b : ins)
            if (overlap(*a, b)) return false;
    }
    return true;
}

// The debug check of g and cu_seqlens; KDA_OK with the check off.
int linear_debug(const float* g, const int32_t* cu, int32_t n_seqs, int64_t ntok, int32_t H, void* stream) {
    if (!kda::debug_validation_enabled() || ntok == 0) return KDA_OK;
    bool ok = true;
    if (kda::debug_validate_from(-std::numeric_limits<float>::infinity(), g, KDA_F32, H, cu, n_seqs, ntok,
                                 static_cast<hipStream_t>(stream), &ok) != hipSuccess)
        return KDA_ERR_HIP;
    return ok ? KDA_OK : KDA_ERR_INVALID_ARGUMENT;
}

}  // namespace
