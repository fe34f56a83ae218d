// Checks of arguments on the host, shared by the C entries of the
// sequence-layer operators (pn_seq_api.cpp, pn_ssm_api.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "pn_seq.hpp"

namespace pn {
namespace {

constexpr int64_t kMaxBlocks = (int64_t(1) << 31) - 1;
constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

int fail(int code, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return set_error(code, buf);
}

int launched(hipError_t e) {
    return e == hipSuccess ? PN_OK : fail(PN_EHIP, "launch failed: %s", hipGetErrorString(e));
}

int64_t elem_bytes(int64_t dtype) { return dtype == PN_F32 ? 4 : 2; }

// The bytes an array may touch.
struct Range {
    uintptr_t lo, hi;
};
Range range(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return p && bytes > 0 ? Range{a, a + static_cast<uintptr_t>(bytes)} : Range{0, 0};
}
Range range(const pn_tokens& x, int64_t B, int64_t T, int64_t heads, int64_t D, int64_t elem) {
    if (B <= 0 || T <= 0 || heads <= 0) return Range{0, 0};
    return range(x.p, elem * ((B - 1) * x.sb + (T - 1) * x.st + (heads - 1) * x.sh + D));
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// Products of sizes in int64 without overflow.
bool small_product(std::initializer_list<int64_t> v, int64_t limit) {
    int64_t p = 1;
    for (int64_t x : v) {
        if (x == 0) return true;
        if (p > limit / x) return false;
        p *= x;
    }
    return p <= limit;
}

constexpr int64_t kMaxStride = int64_t(1) << 40;
int check_tokens(const pn_tokens& x, const char* name, int64_t elem) {
    if (!x.p) return fail(PN_EINVAL, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(x.p) % elem) return fail(PN_EINVAL, "%s is not aligned to its type", name);
    for (int64_t s : {x.sb, x.st, x.sh})
        if (s < 0 || s > kMaxStride) return fail(PN_EINVAL, "a stride of %s is out of range", name);
    return PN_OK;
}

#define PN_TRY(call)                      \
    do {                                  \
        const int rc_ = (call);           \
        if (rc_ != PN_OK) return rc_;     \
    } while (0)

}  // namespace
}  // namespace pn
