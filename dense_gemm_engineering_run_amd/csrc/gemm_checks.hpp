// gemm_checks.hpp -- argument checks shared by the grouped and adapter entry
// points (host only; no HIP call).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "mi355_gemm.h"

namespace mg {

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxGroups = 65535;
constexpr uint64_t kMaxSpanBytes = (uint64_t)1 << 48;   // the GPU's virtual address range

inline int in_bytes(int dtype) { return dtype == GEMM_DTYPE_F32 ? 4 : 2; }
inline int out_bytes(int dtype) { return dtype == GEMM_DTYPE_BF16_BF16 || dtype == GEMM_DTYPE_F16_F16 ? 2 : 4; }

inline const char* dtype_name(int dtype)
{
    static const char* const names[GEMM_NUM_DTYPES] = {"f32", "f16_f32", "bf16_bf16", "f16_f16", "bf16_f32"};
    return names[dtype];
}

// One strided array of `count` matrices, each `outer` rows of `inner`
// contiguous elements of `es` bytes.
struct Operand {
    const void* p;
    int64_t outer, inner, ld, count, stride;
    int es;

    bool empty() const { return outer <= 0 || inner <= 0 || count <= 0; }
    // The leading dimension and the stride are usable: wide enough, and no
    // span over 2^48 bytes.
    bool lds_ok() const
    {
        const uint64_t lim = kMaxSpanBytes / (uint64_t)es;
        return ld >= std::max<int64_t>(1, inner) && stride >= 0 &&
               (uint64_t)ld <= lim / (uint64_t)std::max<int64_t>(1, outer) &&
               (uint64_t)stride <= lim / (uint64_t)std::max<int64_t>(1, count);
    }
    // Elements one matrix spans.
    uint64_t span() const { return empty() ? 0 : (uint64_t)(outer - 1) * ld + inner; }
    // Bytes read or written from p on; `round`: the last row up to 16 bytes.
    uint64_t bytes(bool round) const
    {
        if (empty()) return 0;
        const uint64_t last = (uint64_t)inner * es;
        return ((uint64_t)(count - 1) * stride + (uint64_t)(outer - 1) * ld) * es + (round ? (last + 15) / 16 * 16 : last);
    }
    bool aligned(int n) const
    {
        return ((uintptr_t)p % n) == 0 && (n <= es || ((ld * es) % n == 0 && (count <= 1 || (stride * es) % n == 0)));
    }
};

inline bool overlap(const void* p, uint64_t pn, const void* q, uint64_t qn)
{
    if (!p || !q || pn == 0 || qn == 0) return false;
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return a < b + qn && b < a + pn;
}

// MI355_GEMM_LOG (read once): a line on stderr per call that launches.
inline bool log_enabled()
{
    static const bool on = [] {
        const char* v = std::getenv("MI355_GEMM_LOG");
        return v && *v && std::strcmp(v, "0") != 0;
    }();
    return on;
}

}  // namespace mg
