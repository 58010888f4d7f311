// Grouped-product kernels for dtype f32 (inputs F32, output F32).
#include "gemm_ragged.hpp"

namespace mg {

struct RaggedF32 {
    template <int BM, int BN, int ST, bool AK, bool BKM, By BY, bool EPI, bool VEC>
    static hipError_t go(const RaggedCall& c, hipStream_t s)
    {
        return launch_ragged<BY>(&gemm_ragged_f32_kernel<BM, BN, 32, 2, 2, ST, AK, BKM, BY, EPI, VEC>, c, BM, BN, 256, s);
    }
    template <int MT, int NT, int NW, int ST, bool BKM, bool VEC>
    static hipError_t skinny(const RaggedCall& c, hipStream_t s)
    {
        return launch_ragged<By::Rows>(&gemm_ragged_skinny_kernel<MT, NT, NW, ST, BKM, VEC>, c, MT * 16, NT * 16, NW * 64, s);
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
        const int64_t avg = (c.r.rows + c.r.groups - 1) / c.r.groups;
        if constexpr (BY == By::Rows) {
            // Few rows stream (16x32, 32x64 and 32x32 tiles; B k-major, n-major
            // in brackets), against 64x64, us:
            //        1 row  in 122 groups of  384 x 4224   86.7 [ 95.8]    95.1          94.9   157
            //       16 rows in   8 groups of 4096 x 4096  109   [121]     113           110     164
            //       22 rows in  14 groups of 7192 x 5264  569   [632]     455   [441]   505     611
            //       48 rows in  16 groups of 2048 x 2048   99.5 [107]      92.7          91.8   112
            //       64 rows in  16 groups of 2048 x 1024                   69.3          68.9    62.9
            //      300 rows in   1 group  of 1024 x 4096                   40.8          39.8    83.6
            // (Four waves that share a row's k-tiles also round less than one.)
            if (avg <= 16) return skinny<1, 2, 4, 3, BKM, VEC>(c, s);
            if (avg <= 48) return skinny<2, 4, 4, 2, BKM, VEC>(c, s);
            if (tiles(avg, 64, 64) <= 192) return skinny<2, 2, 4, 2, BKM, VEC>(c, s);
        }
        if constexpr (BY == By::Rows && VEC) {
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
