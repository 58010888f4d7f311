// gemm_i8.hpp -- products of 8-bit integers with a scale per row and column (gfx950).
//
//   C[m][n] = act(alpha * scale_a[m] scale_b[n] sum_k A[m][k] B[n][k] + beta * C_old[m][n] + bias[n])
//
// The sum is exact: 32-bit integers on the integer MFMAs, whose 16x16x64 and
// 32x32x32 forms take 16 consecutive k of a row a lane, the byte layout of the
// 16-bit forms.  So the tiles, rings and schedules of the 16-bit products
// (gemm_dma.hpp, gemm_ragged.hpp) hold here as they are, on pairs of 8-bit
// values (In::I8): Params::K, lda and ldb count pairs.  When the sums are
// done they are scaled in their registers and leave by the 16-bit products'
// stores.
#pragma once

#include "gemm_i8_tiles.hpp"
#include "gemm_quant.hpp"
#include "gemm_ragged.hpp"

namespace mg {

struct I8Scales {
    const float* a;       // per row of C, or null: 1
    const float* b;       // per column of C, or null: 1
};

// One output from its sum's bits: scaled in fp32 (the conversion and each
// product round once), then the elementwise epilogue.
template <Out TO>
__device__ __forceinline__ float i8_value(const Params& p, int m, int n, float bits, float sa, float sb)
{
    const float v = settled((float)__float_as_int(bits) * sa * sb);
    return p.epi && m < p.M && n < p.N ? epi_value<TO>(p, m, n, v) : v;
}

// The sums of an accumulator tile of KT (rows along its registers) to outputs.
template <class KT>
__device__ __forceinline__ void i8_finish(const Params& p, const I8Scales& s, int m0, int n0, typename KT::Acc& acc, int lane,
                                          int wave)
{
    constexpr int WN = KT::TILE_N / KT::WTN;
    const int wm = wave / WN, wn = wave % WN;
    float sb[KT::TN];
#pragma unroll
    for (int j = 0; j < KT::TN; ++j) {
        const int n = n0 + KT::col(wn, j, lane);
        sb[j] = s.b && n < p.N ? s.b[n] : 1.f;
    }
#pragma unroll
    for (int i = 0; i < KT::TM; ++i)
#pragma unroll
        for (int q = 0; q < KT::R; ++q) {
            const int m = m0 + KT::row(wm, i, q, lane);
            const float sa = s.a && m < p.M ? s.a[m] : 1.f;
#pragma unroll
            for (int j = 0; j < KT::TN; ++j)
                acc[i][j][q] = i8_value<KT::OUT>(p, m, n0 + KT::col(wn, j, lane), acc[i][j][q], sa, sb[j]);
        }
}

// ------------------------------------------------------------ 16-byte aligned operands

// The ring of gemm_dma.hpp.
template <Out TO, int BM, int BN, int BK, int WM, int WN, int MI, int STAGES>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_i8_dma_kernel(Params p, I8Scales sc)
{
    using KT = Dma16<In::I8, TO, BM, BN, BK, WM, WN, MI, STAGES, true, true>;
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm) * BM, n0 = __builtin_amdgcn_readfirstlane(tn) * BN;
    typename KT::OA oa;
    typename KT::OB ob;
    oa.init(wave, lane, p.lda);
    ob.init(wave, lane, p.ldb);
    typename KT::Acc acc;
    KT::zero(acc);
    KT::mainloop(p, smem, oa, ob, m0, n0, 0, (p.K + BK - 1) / BK, acc, tid, lane, wave);
    i8_finish<KT>(p, sc, m0, n0, acc, lane, wave);
    store_tile<KT, false>(p, smem, m0, n0, acc, tid, lane, wave);
}

// The ping-pong schedule (PingPong), whose accumulators run along C's rows.
template <Out TO, int BM, int BN, int BK, int WM, int WN, int MI>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_i8_pp_kernel(Params p, I8Scales sc)
{
    using PP = PingPong<In::I8, TO, BM, BN, BK, WM, WN, MI, true, true, true>;
    using KT = typename PP::KT;
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm) * BM, n0 = __builtin_amdgcn_readfirstlane(tn) * BN;
    typename KT::Acc acc;
    KT::zero(acc);
    PP::mainloop(p, smem, m0, n0, acc, tid, lane, wave);
    const int mb = m0 + wave / WN * KT::WTM + lane % MI, nb = n0 + wave % WN * KT::WTN + lane / MI * 4;
    float sa[KT::TM];
#pragma unroll
    for (int i = 0; i < KT::TM; ++i) sa[i] = sc.a && mb + i * MI < p.M ? sc.a[mb + i * MI] : 1.f;
#pragma unroll
    for (int j = 0; j < KT::TN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = nb + j * MI + e;
            const float sb = sc.b && n < p.N ? sc.b[n] : 1.f;
#pragma unroll
            for (int i = 0; i < KT::TM; ++i) acc[i][j][e] = i8_value<TO>(p, mb + i * MI, n, acc[i][j][e], sa[i], sb);
        }
    PP::store(p, smem, m0, n0, acc, lane, wave);
}

// Waves that hold sums of the same BM x BN tile, each over its own k: the sums of
// all of them, finished and stored.
template <Out TO, int BM, int BN, int NW>
__device__ __forceinline__ void i8_join(const Params& p, const I8Scales& sc, int* part, int m0, int n0,
                                        const f32x4 (&acc)[BM / 16][BN / 16], int tid, int lane, int wave)
{
    __syncthreads();
#pragma unroll
    for (int i = 0; i < BM / 16; ++i)
#pragma unroll
        for (int j = 0; j < BN / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                part[wave * BM * BN + (i * 16 + lane / 16 * 4 + e) * BN + j * 16 + lane % 16] = __float_as_int(acc[i][j][e]);
    __syncthreads();
    for (int x = tid; x < BM * BN; x += NW * 64) {
        const int m = m0 + x / BN, n = n0 + x % BN;
        if (m >= p.M || n >= p.N) continue;
        int v = part[x];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += part[w * BM * BN + x];
        store_out<TO>(p.C, (int64_t)m * p.ldc + n,
                      i8_value<TO>(p, m, n, __int_as_float(v), sc.a ? sc.a[m] : 1.f, sc.b ? sc.b[n] : 1.f));
    }
}

// Few rows: Skinny's streams, whose waves take the k-tiles in turn.
template <Out TO, int MT, int NT, int NW, int ST>
__global__ void __launch_bounds__(NW * 64)
gemm_i8_stream_kernel(Params p, I8Scales sc)
{
    using T = Skinny<In::I8, MT, NT, NW, ST, true, true>;
    static_assert(T::RING <= 160 * 1024 && NW * T::PART * 4 <= T::RING, "LDS budget");
    __shared__ __attribute__((aligned(1024))) char smem[T::RING];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm) * (MT * 16), n0 = __builtin_amdgcn_readfirstlane(tn) * (NT * 16);
    typename T::Acc acc;
    T::zero(acc);
    T::stream(p, smem, m0, n0, acc, lane, wave);
    i8_join<TO, T::PART / (NT * 16), NT * 16, NW>(p, sc, (int*)smem, m0, n0, acc, tid, lane, wave);
}

// ------------------------------------------------------------ operands at any byte

// Rows that start at any byte: as OddRows and OddChunk, whose elements are two
// bytes.  Words that hold an own byte are read, nothing else.
struct ByteRows {
    __amdgpu_buffer_rsrc_t r;

    __device__ __forceinline__ ByteRows(const char* base, uint64_t bytes)
        : r(make_rsrc(base - ((uint64_t)base & 3), bytes ? (bytes + ((uint64_t)base & 3) + 3) / 4 * 4 : 0))
    {
    }
};

// An operand's k-tiles of 2 * BK bytes a row, from memory through registers to
// the LDS layout of DmaOperand.  Neighbouring lanes hold neighbouring chunks: the
// word that a chunk needs of the next one comes from the next lane, and only a
// row's last chunk loads it (where all did, half of the accesses were for it: 2048
// x 4100 x 4096 took 83 us instead of 72).
template <int ROWS, int BK, int NW, int DEPTH>
struct ByteOperand {
    using LDS = DmaOperand<ROWS, BK, NW, true, 16>;
    static constexpr int CPR = LDS::CPR;
    static_assert(CPR <= 16 && 16 % CPR == 0, "a row's chunks lie in one row of 16 lanes");
    int voff[LDS::IPW];
    i32x4 words[DEPTH][LDS::IPW];
    int last[DEPTH][LDS::IPW];

    // ld in bytes.  (row0 is a multiple of 4 and k0 of 16, so every tile's
    // first byte lies in its word as the base's.)
    __device__ __forceinline__ void init(int wave, int lane, int64_t ld, const char* base)
    {
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j)
            voff[j] = (int)(((wave * LDS::IPW + j) * 64 + lane) / CPR * ld) + lane % CPR * 16 + (int)((uint64_t)base & 3);
    }
    __device__ __forceinline__ void load(int d, const char* base, uint64_t bytes, int64_t ld, int row0, int k0, int lane)
    {
        const int64_t origin = (int64_t)row0 * ld + k0;
        const ByteRows s(base + origin, (uint64_t)origin < bytes ? bytes - (uint64_t)origin : 0);
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) words[d][j] = buf_load16(s.r, voff[j] & ~3);
        if (lane % CPR == CPR - 1) {
#pragma unroll
            for (int j = 0; j < LDS::IPW; ++j) last[d][j] = __builtin_amdgcn_raw_buffer_load_b32(s.r, (voff[j] & ~3) + 16, 0, 0);
        }
    }
    // ... of the tile at k0; bytes from K on as zeros.
    __device__ __forceinline__ void store(int d, char* tile, int k0, int K, int wave, int lane) const
    {
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) {
            const int row = ((wave * LDS::IPW + j) * 64 + lane) / CPR, c = lane % CPR;
            const uint32_t sh = ((uint32_t)voff[j] & 3) * 8;
            const int next = __builtin_amdgcn_update_dpp(0, words[d][j][0], 0x101, 0xf, 0xf, false);   // of the lane above
            const int beyond = c == CPR - 1 ? last[d][j] : next;
            i32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = (int)__builtin_amdgcn_alignbit((uint32_t)(e < 3 ? words[d][j][e + 1] : beyond), (uint32_t)words[d][j][e], sh);
            if (k0 + 2 * BK > K) v = mask_bytes(v, K - k0 - c * 16);
            *(i32x4*)(tile + (row * CPR + swz_chunk<CPR, true>(row, c)) * 16) = v;
        }
    }
};

// Operands at any byte (p.K, lda, ldb and the extents in bytes): LDS in two
// stages, DEPTH tiles of loads in flight, one barrier a tile.
template <Out TO, int BM, int BN, int BK, int WM, int WN, int DEPTH>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_i8_odd_kernel(Params p, I8Scales sc)
{
    using KT = Dma16<In::I8, TO, BM, BN, BK, WM, WN, 16, 2, true, true>;
    static_assert(DEPTH % 2 == 0, "a tile's stage is known at compile time");
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_coords(p, tm, tn);
    tm = __builtin_amdgcn_readfirstlane(tm);
    tn = __builtin_amdgcn_readfirstlane(tn);
    const int m0 = tm * BM, n0 = tn * BN, wm = wave / WN, wn = wave % WN;
    constexpr int KB = 2 * BK;
    const int nkt = (p.K + KB - 1) / KB;
    typename KT::Acc acc;
    KT::zero(acc);
    ByteOperand<BM, BK, KT::NW, DEPTH> oa;
    ByteOperand<BN, BK, KT::NW, DEPTH> ob;
    oa.init(wave, lane, p.lda, p.A);
    ob.init(wave, lane, p.ldb, p.B);
    auto load = [&](int t, int d) {               // past the end: empty extents
        oa.load(d, p.A, t < nkt ? p.a_bytes : 0, p.lda, m0, t * KB, lane);
        ob.load(d, p.B, t < nkt ? p.b_bytes : 0, p.ldb, n0, t * KB, lane);
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(d, d);
    for (int t0 = 0; t0 < nkt; t0 += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int t = t0 + d;
            if (t >= nkt) break;
            char* const sa = smem + d % 2 * KT::STAGE;
            char* const sb = sa + KT::OA::BYTES;
            oa.store(d, sa, t * KB, p.K, wave, lane);
            ob.store(d, sb, t * KB, p.K, wave, lane);
            load(t + DEPTH, d);
            // The other stage is written after the next barrier, when every
            // wave has read it.
            __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
            bare_barrier();
#pragma unroll
            for (int g = 0; g < KT::NG; ++g) {
                i32x4 fa[KT::TM], fb[KT::TN];
#pragma unroll
                for (int i = 0; i < KT::TM; ++i) fa[i] = KT::OA::template frag<16>(sa, wm * KT::WTM + i * 16, g * 32, lane);
#pragma unroll
                for (int j = 0; j < KT::TN; ++j) fb[j] = KT::OB::template frag<16>(sb, wn * KT::WTN + j * 16, g * 32, lane);
#pragma unroll
                for (int i = 0; i < KT::TM; ++i)
#pragma unroll
                    for (int j = 0; j < KT::TN; ++j) mfma_step<In::I8, 16>(fa[i], fb[j], acc[i][j]);
            }
        }
    }
    i8_finish<KT>(p, sc, m0, n0, acc, lane, wave);
    store_tile<KT, false>(p, smem, m0, n0, acc, tid, lane, wave);
}

// Few of their tiles: the waves take the k-tiles in turn, each through LDS of its
// own with nothing to wait for but itself.
template <Out TO, int BM, int BN, int NW, int D>
__global__ void __launch_bounds__(NW * 64)
gemm_i8_odd_stream_kernel(Params p, I8Scales sc)
{
    constexpr int BK = 64, KB = 2 * BK;
    using KT = Dma16<In::I8, TO, BM, BN, BK, 1, 1, 16, 2, true, true>;
    constexpr int STAGE = KT::STAGE, PART = BM * BN * 4, SMEM = NW * (STAGE > PART ? STAGE : PART);
    static_assert(SMEM <= 160 * 1024, "LDS budget");
    __shared__ __attribute__((aligned(1024))) char smem[SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm) * BM, n0 = __builtin_amdgcn_readfirstlane(tn) * BN;
    const int nkt = (p.K + KB - 1) / KB;
    typename KT::Acc acc;
    KT::zero(acc);
    ByteOperand<BM, BK, 1, D> oa;
    ByteOperand<BN, BK, 1, D> ob;
    oa.init(0, lane, p.lda, p.A);
    ob.init(0, lane, p.ldb, p.B);
    auto load = [&](int t, int d) {               // past the end: empty extents
        oa.load(d, p.A, t < nkt ? p.a_bytes : 0, p.lda, m0, t * KB, lane);
        ob.load(d, p.B, t < nkt ? p.b_bytes : 0, p.ldb, n0, t * KB, lane);
    };
    char* const sa = smem + wave * STAGE;
    char* const sb = sa + KT::OA::BYTES;
#pragma unroll
    for (int d = 0; d < D; ++d) load(wave + d * NW, d);
    for (int t0 = wave; t0 < nkt; t0 += D * NW) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int t = t0 + d * NW;
            if (t >= nkt) break;
            oa.store(d, sa, t * KB, p.K, 0, lane);
            ob.store(d, sb, t * KB, p.K, 0, lane);
            load(t + D * NW, d);
            __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0): written
            asm volatile("" ::: "memory");
#pragma unroll
            for (int g = 0; g < KT::NG; ++g) {
                i32x4 fa[KT::TM], fb[KT::TN];
#pragma unroll
                for (int i = 0; i < KT::TM; ++i) fa[i] = KT::OA::template frag<16>(sa, i * 16, g * 32, lane);
#pragma unroll
                for (int j = 0; j < KT::TN; ++j) fb[j] = KT::OB::template frag<16>(sb, j * 16, g * 32, lane);
#pragma unroll
                for (int i = 0; i < KT::TM; ++i)
#pragma unroll
                    for (int j = 0; j < KT::TN; ++j) mfma_step<In::I8, 16>(fa[i], fb[j], acc[i][j]);
            }
            __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0): read, the next tile may be written
            asm volatile("" ::: "memory");
        }
    }
    i8_join<TO, BM, BN, NW>(p, sc, (int*)smem, m0, n0, acc, tid, lane, wave);
}

// ------------------------------------------------------------------ launchers

// What the host asks of an output type's launchers (gemm_i8_<type>.hip).
struct I8Call {
    Params p;             // sizes and leading dimensions of A and B in bytes
    I8Scales s;
    bool vec;             // operands allow 16-byte loads
};

inline I8Shape shape_of(const I8Call& c) { return {c.vec, c.p.M, c.p.N, c.p.K}; }

template <Out TO>
struct I8Inst {
    template <class Kernel>
    static hipError_t run(Kernel kernel, const I8Call& c, const Tile& t, hipStream_t s)
    {
        Params p = c.p;
        I8Scales sc = c.s;
        if (c.vec) {                  // pairs of values
            p.k_odd = p.K & 1;
            p.K = (p.K + 1) / 2;
            p.lda /= 2;
            p.ldb /= 2;
        }
        p.tiles_m = (int)ceil_div(p.M, t.bm);
        p.tiles_n = (int)ceil_div(p.N, t.bn);
        p.group_m = p.tiles_m < 8 ? p.tiles_m : 8;
        void* args[] = {&p, &sc};
        return hipLaunchKernel((const void*)kernel, dim3((unsigned)i8_grid(shape_of(c), t)), dim3(t.threads), args, 0, s);
    }
    template <I8Tile T>
    static hipError_t stream(const I8Call& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T);
        return run(&gemm_i8_stream_kernel<TO, t.wm, t.wn, t.extra, t.stages>, c, t, s);
    }
    template <I8Tile T>
    static hipError_t dma(const I8Call& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T);
        return run(&gemm_i8_dma_kernel<TO, t.bm, t.bn, t.bk, t.wm, t.wn, t.mi, t.stages>, c, t, s);
    }
    template <I8Tile T>
    static hipError_t odd(const I8Call& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T);
        return run(&gemm_i8_odd_kernel<TO, t.bm, t.bn, t.bk, t.wm, t.wn, t.stages>, c, t, s);
    }
    template <I8Tile T>
    static hipError_t odd_stream(const I8Call& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T);
        return run(&gemm_i8_odd_stream_kernel<TO, t.bm, t.bn, t.extra, t.stages>, c, t, s);
    }
    static hipError_t launch(const I8Call& c, hipStream_t s)
    {
        constexpr Tile pp = tile_of(I8Tile::PingPong);
        switch (i8_tile(shape_of(c))) {
        case I8Tile::Stream16x16: return stream<I8Tile::Stream16x16>(c, s);
        case I8Tile::Stream16x32: return stream<I8Tile::Stream16x32>(c, s);
        case I8Tile::Stream32x32: return stream<I8Tile::Stream32x32>(c, s);
        case I8Tile::Dma32x64: return dma<I8Tile::Dma32x64>(c, s);
        case I8Tile::Dma64x64: return dma<I8Tile::Dma64x64>(c, s);
        case I8Tile::Dma64x128: return dma<I8Tile::Dma64x128>(c, s);
        case I8Tile::Dma128x128: return dma<I8Tile::Dma128x128>(c, s);
        case I8Tile::Dma128x256: return dma<I8Tile::Dma128x256>(c, s);
        case I8Tile::PingPong: return run(&gemm_i8_pp_kernel<TO, pp.bm, pp.bn, pp.bk, pp.wm, pp.wn, pp.mi>, c, pp, s);
        case I8Tile::OddStream16x16: return odd_stream<I8Tile::OddStream16x16>(c, s);
        case I8Tile::OddStream32x32: return odd_stream<I8Tile::OddStream32x32>(c, s);
        case I8Tile::Odd32x32: return odd<I8Tile::Odd32x32>(c, s);
        case I8Tile::Odd64x64: return odd<I8Tile::Odd64x64>(c, s);
        case I8Tile::Odd128x128: return odd<I8Tile::Odd128x128>(c, s);
        case I8Tile::Odd128x256: return odd<I8Tile::Odd128x256>(c, s);
        default: return hipErrorInvalidValue;
        }
    }
};

hipError_t i8_f32(const I8Call& c, hipStream_t s);
hipError_t i8_f16(const I8Call& c, hipStream_t s);
hipError_t i8_bf16(const I8Call& c, hipStream_t s);

}  // namespace mg
