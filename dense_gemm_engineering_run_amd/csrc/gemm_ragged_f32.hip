// Grouped-product kernels for dtype f32 (inputs F32, output F32).
#include "gemm_ragged.hpp"

namespace mg {

struct RaggedF32 {
    template <int BM, int BN, int ST, bool AK, bool BKM, By BY, bool EPI, bool VEC>
    static hipError_t go(const RaggedCall& c, hipStream_t s)
    {
        return launch_ragged<BY>(&gemm_ragged_f32_kernel<BM, BN, 32, 2, 2, ST, AK, BKM, BY, EPI, VEC>, c, BM, BN, 256, s);
    }
    template <bool AK, bool BKM, By BY, bool EPI, bool VEC>
    static hipError_t sized(const RaggedCall& c, hipStream_t s)
    {
        auto tiles = [&](int t) {
            const int64_t cols = (c.p.N + t - 1) / t;
            if (!c.by_rows) return cols * ((c.p.M + t - 1) / t) * c.r.groups;
            const int64_t avg = (c.r.rows + c.r.groups - 1) / c.r.groups;
            return cols * ((avg + t - 1) / t) * c.r.groups;
        };
        // RULE
        if (tiles(128) >= 192 && (!c.by_rows || c.r.rows > 48 * (int64_t)c.r.groups)) return go<128, 128, 2, AK, BKM, BY, EPI, VEC>(c, s);
        return go<64, 64, VEC ? 4 : 2, AK, BKM, BY, EPI, VEC>(c, s);
    }
    template <bool VEC>
    static hipError_t any(const RaggedCall& c, hipStream_t s)
    {
        if (c.by_rows)
            return c.b_kmajor ? sized<true, true, By::Rows, false, VEC>(c, s) : sized<true, false, By::Rows, false, VEC>(c, s);
        return c.p.epi ? sized<false, false, By::K, true, VEC>(c, s) : sized<false, false, By::K, false, VEC>(c, s);
    }
    static hipError_t launch(const RaggedCall& c, hipStream_t s) { return c.vec ? any<true>(c, s) : any<false>(c, s); }
};

hipError_t ragged_f32(const RaggedCall& c, hipStream_t s) { return RaggedF32::launch(c, s); }

}  // namespace mg
