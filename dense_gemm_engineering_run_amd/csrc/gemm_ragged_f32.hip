// Grouped-product kernels for dtype f32 (inputs F32, output F32).
#include "gemm_ragged.hpp"

namespace mg {

struct RaggedF32 {
    template <RaggedTile T, bool AK, bool BKM, By BY, bool EPI, bool VEC>
    static hipError_t go(const RaggedCall& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T);
        return launch_ragged<BY>(&gemm_ragged_f32_kernel<t.bm, t.bn, t.bk, t.wm, t.wn, t.stages, AK, BKM, BY, EPI, VEC>, c, t, s);
    }
    template <RaggedTile T, bool BKM, bool VEC>
    static hipError_t stream(const RaggedCall& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T);
        return launch_ragged<By::Rows>(&gemm_ragged_skinny_kernel<t.wm, t.wn, t.extra, t.stages, BKM, VEC>, c, t, s);
    }
    template <bool BKM, bool VEC>
    static hipError_t rows(const RaggedCall& c, hipStream_t s)
    {
        const RaggedTile t = ragged_tile(shape_of(c, true));
        switch (t) {
        case RaggedTile::F32Stream16x32: return stream<RaggedTile::F32Stream16x32, BKM, VEC>(c, s);
        case RaggedTile::F32Stream32x64: return stream<RaggedTile::F32Stream32x64, BKM, VEC>(c, s);
        case RaggedTile::F32Stream32x32: return stream<RaggedTile::F32Stream32x32, BKM, VEC>(c, s);
        default: break;
        }
        if constexpr (VEC) {
            if (t == RaggedTile::F32Rows64x128) return go<RaggedTile::F32Rows64x128, true, BKM, By::Rows, false, true>(c, s);
            return go<RaggedTile::F32Rows64x64, true, BKM, By::Rows, false, true>(c, s);
        } else {
            return go<RaggedTile::F32Two64x64, true, BKM, By::Rows, false, false>(c, s);
        }
    }
    template <bool EPI, bool VEC>
    static hipError_t by_k(const RaggedCall& c, hipStream_t s)
    {
        if (ragged_tile(shape_of(c, true)) == RaggedTile::F32K128x128)
            return go<RaggedTile::F32K128x128, false, false, By::K, EPI, VEC>(c, s);
        return go<RaggedTile::F32Two64x64, false, false, By::K, EPI, VEC>(c, s);
    }
    template <bool VEC>
    static hipError_t any(const RaggedCall& c, hipStream_t s)
    {
        if (c.by_rows) return c.b_kmajor ? rows<true, VEC>(c, s) : rows<false, VEC>(c, s);
        return c.p.epi ? by_k<true, VEC>(c, s) : by_k<false, VEC>(c, s);
    }
    static hipError_t launch(const RaggedCall& c, hipStream_t s) { return c.vec ? any<true>(c, s) : any<false>(c, s); }
};

hipError_t ragged_f32(const RaggedCall& c, hipStream_t s) { return RaggedF32::launch(c, s); }

}  // namespace mg
