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
        // Measured, us (K = 1024 by rows; 64x64 in three stages, 64x128 in two,
        // 128x128 in two):
        //   by rows   64 rows in  4 groups of 1024     24.2    41.9   66.9
        //           1024 rows in 16 groups of 2048     60.1    70.6  126
        //           4096 rows in 16 groups of 2048    178     165    196
        //          16384 rows in 16 groups of 2048    577     549    562
        //   by k (64x64 in two stages, 128x128 in two), 4096 k:
        //          16 groups of 512 x 512              28.1           43.4
        //           4 groups of 1024 x 1024            75.7           98.6
        //           4 groups of 4096 x 2048           550            503
        auto tiles = [&](int64_t rows, int bm, int bn) {
            return (rows + bm - 1) / bm * ((c.p.N + bn - 1) / bn) * c.r.groups;
        };
        if constexpr (BY == By::Rows && VEC) {
            const int64_t avg = (c.r.rows + c.r.groups - 1) / c.r.groups;
            if (tiles(avg, 64, 128) >= 1024) return go<64, 128, 2, AK, BKM, BY, EPI, VEC>(c, s);
            return go<64, 64, 3, AK, BKM, BY, EPI, VEC>(c, s);
        } else {
            if (BY == By::K && tiles(c.p.M, 128, 128) >= 512) return go<128, 128, 2, AK, BKM, BY, EPI, VEC>(c, s);
            return go<64, 64, 2, AK, BKM, BY, EPI, VEC>(c, s);
        }
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
