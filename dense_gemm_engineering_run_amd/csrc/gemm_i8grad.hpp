// gemm_i8grad.hpp -- products with 8-bit values whose scales lie along the
// summed index (gfx950): the gradients of a linear layer from 8-bit checkpoints.
//
//   C[m][n] (+)= sum_k A[m][k] scales[k] Q[n][k]
//
// Q is stored k by k (element (n, k) at n + k * ldq), A m- or k-contiguous.
// The scale cannot leave the sum, so it joins a factor before the matrix units
// take it:
//   16-bit C: the restored value scales[k] * Q[n][k], rounded to A's type, as
//     gemm_dequantize_rows gives it (off by half a step: 2^-8 of itself in bf16,
//     2^-11 in fp16, 2^-25 where that is more).
//   fp32 C: a product with the scale rounded to fp32, held whole by three bf16
//     terms of 8 bits each: scales[k] * Q[n][k] for bf16 A, scales[k] * A[m][k] for
//     fp16 and fp32 A (Q is exact in bf16).  Two terms (17 bits) made the result
//     2.5e-6 off (relative, 8192 k of normal values), where fp32 sums alone are off
//     by 5e-7.  For fp32 A three bf16 MFMAs take less than half the time of the
//     fp32 ones.
#pragma once

#include "gemm_quant.hpp"
#include "gemm_ragged.hpp"

namespace mg {

struct GradParams {
    Params p;             // B, ldb, b_bytes: Q, in bytes; lda in elements of A
    const float* scales;  // per k
};

// Terms that the kernels split each factor into, and the type they multiply in.
template <In TI, Out TO>
struct GradTypes {
    static constexpr bool SPLIT_A = TO == Out::F32 && TI != In::BF16;   // the scale joins A (else Q)
    static constexpr int TA = SPLIT_A ? 3 : 1;
    static constexpr int TQ = TO == Out::F32 && !SPLIT_A ? 3 : 1;
    static constexpr In MT = SPLIT_A ? In::BF16 : TI;
};

// Eight fp32 values as 16-bit ones.
template <In T>
__device__ __forceinline__ void split8(float (&v)[8], i32x4 (&t)[1])
{
#pragma unroll
    for (int d = 0; d < 4; ++d) t[0][d] = (int)((uint32_t)round16<T>(v[2 * d]) | ((uint32_t)round16<T>(v[2 * d + 1]) << 16));
}

// The same in three bf16 terms by cutting off: 8 of the 24 bits each, nothing
// is left.  An infinity stays one in the first term (NaN, whose cut-off bits
// may be an infinity's, leaves NaN behind).
template <In T>
__device__ __forceinline__ void split8(float (&v)[8], i32x4 (&t)[3])
{
    static_assert(T == In::BF16, "terms of 8 bits");
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if (s == 0) {
                v[2 * d] = settled(v[2 * d]);
                v[2 * d + 1] = settled(v[2 * d + 1]);
            }
            t[s][d] = (int)__builtin_amdgcn_perm((uint32_t)__float_as_int(v[2 * d + 1]), (uint32_t)__float_as_int(v[2 * d]),
                                                 0x07060302u);
            if (s < 2)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float& x = v[2 * d + e];
                    const float f = __int_as_float(__float_as_int(x) & (int)0xffff0000);
                    x = s == 0 && x == f ? 0.f : x - f;
                }
        }
}

// Eight bytes from any byte of a row: three words, shifted.
struct ByteChunk8 {
    int w0, w1, w2;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int off)     // off: from the first word
    {
        typedef int i32x3 __attribute__((ext_vector_type(3)));
        const i32x3 v = __builtin_amdgcn_raw_buffer_load_b96(r, off & ~3, 0, 0);
        w0 = v[0];
        w1 = v[1];
        w2 = v[2];
    }
    __device__ __forceinline__ void get(int off, int& lo, int& hi) const
    {
        const uint32_t sh = ((uint32_t)off & 3) * 8;
        lo = (int)__builtin_amdgcn_alignbit((uint32_t)w1, (uint32_t)w0, sh);
        hi = (int)__builtin_amdgcn_alignbit((uint32_t)w2, (uint32_t)w1, sh);
    }
};

// One operand's k-tile in LDS: TERMS tiles in DmaOperand's layout.

// Q: k rows of ROWS bytes to [BK][ROWS] values, exact or times scales[k].
template <In MT, int ROWS, int BK, int NW, int TERMS, bool SCALED>
struct QOperand {
    using LDS = DmaOperand<ROWS, BK, NW, false, 16>;
    int voff[LDS::IPW];
    ByteChunk8 q[LDS::IPW];
    float s[LDS::IPW];

    __device__ static __forceinline__ int slot(int wave, int lane, int j) { return (wave * LDS::IPW + j) * 64 + lane; }
    __device__ __forceinline__ void init(int wave, int lane, int64_t ld)
    {
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) {
            const int k = slot(wave, lane, j) / LDS::RCH, phys = slot(wave, lane, j) % LDS::RCH;
            voff[j] = (int)(k * ld) + (phys ^ LDS::mkey(k)) * 8;
        }
    }
    // Rows from K on lie past the extent and read as zeros, scale included.
    __device__ __forceinline__ void load(const GradParams& g, uint64_t bytes, int row0, int k0, int wave, int lane)
    {
        const int64_t origin = (int64_t)k0 * g.p.ldb + row0;
        const char* const at = g.p.B + origin;
        const int lead = (int)((uint64_t)at & 3);
        const uint64_t rem = (uint64_t)origin < bytes ? bytes - (uint64_t)origin : 0;
        const __amdgpu_buffer_rsrc_t r = make_rsrc(at - lead, rem ? (rem + lead + 3) / 4 * 4 : 0);
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) {
            q[j].load(r, voff[j] + lead);
            if constexpr (SCALED) {
                const int k = k0 + slot(wave, lane, j) / LDS::RCH;
                s[j] = k < g.p.K ? g.scales[k] : 0.f;
            }
        }
    }
    __device__ __forceinline__ void store(const GradParams& g, char* tile, int row0, int k0, int wave, int lane) const
    {
        const int lead = (int)((uint64_t)(g.p.B + (int64_t)k0 * g.p.ldb + row0) & 3);
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) {
            int w[2];
            q[j].get(voff[j] + lead, w[0], w[1]);
            // The words at the last row's end can hold bytes of what follows it: k from K on is zeros.
            const bool live = k0 + slot(wave, lane, j) / LDS::RCH < g.p.K;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = live ? byte_value(w[e / 4], e % 4) : 0.f;
                if constexpr (SCALED) v[e] *= s[j];
            }
            i32x4 t[TERMS];
            split8<MT>(v, t);
#pragma unroll
            for (int x = 0; x < TERMS; ++x) *(i32x4*)(tile + x * LDS::BYTES + slot(wave, lane, j) * 16) = t[x];
        }
    }
};

// 16-bit A as it is.
template <In TI, int ROWS, int BK, int NW, bool KMAJ, bool SPLIT>
struct AOperand {
    OddOperand<ROWS, BK, NW, KMAJ, 1> o;
    __device__ __forceinline__ void init(int wave, int lane, int64_t ld) { o.at.init(wave, lane, ld); }
    __device__ __forceinline__ void load(const GradParams& g, uint64_t bytes, int row0, int k0, int, int)
    {
        o.load(0, g.p.A, bytes, g.p.lda, row0, k0);
    }
    __device__ __forceinline__ void store(const GradParams& g, char* tile, int k0, int wave, int lane) const
    {
        o.store(0, tile, g.p.A, k0, g.p.K, wave, lane);
    }
};

// fp16 or fp32 A times scales[k], in three bf16 terms.
template <In TI, int ROWS, int BK, int NW, bool KMAJ>
struct AOperand<TI, ROWS, BK, NW, KMAJ, true> {
    using LDS = DmaOperand<ROWS, BK, NW, KMAJ, 16>;
    static constexpr bool WIDE = TI == In::F32;
    static constexpr int ES = WIDE ? 4 : 2;
    int voff[LDS::IPW];
    i32x4 wide[WIDE ? LDS::IPW : 1][2];
    OddChunk half[WIDE ? 1 : LDS::IPW];
    float s[LDS::IPW][KMAJ ? 8 : 1];

    // k of a slot's first value within the tile.
    __device__ static __forceinline__ int k_of(int slot)
    {
        return KMAJ ? swz_chunk<LDS::CPR, true>(slot / LDS::CPR, slot % LDS::CPR) * 8 : slot / LDS::RCH;
    }
    __device__ __forceinline__ void init(int wave, int lane, int64_t ld)
    {
        LDS o;
        o.init(wave, lane, 0);
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) {
            const int slot = (wave * LDS::IPW + j) * 64 + lane;
            voff[j] = (int)((KMAJ ? slot / LDS::CPR : slot / LDS::RCH) * ld * ES) + o.voff[j] * (ES / 2);
        }
    }
    __device__ __forceinline__ void load(const GradParams& g, uint64_t bytes, int row0, int k0, int wave, int lane)
    {
        const int64_t origin = (KMAJ ? (int64_t)row0 * g.p.lda + k0 : (int64_t)k0 * g.p.lda + row0) * ES;
        const uint64_t rem = (uint64_t)origin < bytes ? bytes - (uint64_t)origin : 0;
        const __amdgpu_buffer_rsrc_t r = make_rsrc(g.p.A + origin, rem);
        const OddRows odd(g.p.A + origin, rem);
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) {
            if constexpr (WIDE) {
                wide[j][0] = buf_load16(r, voff[j]);
                wide[j][1] = buf_load16(r, voff[j] + 16);
            } else {
                half[j].load(odd, voff[j]);
            }
            const int k = k0 + k_of((wave * LDS::IPW + j) * 64 + lane);
#pragma unroll
            for (int e = 0; e < (KMAJ ? 8 : 1); ++e) s[j][e] = k + e < g.p.K ? g.scales[k + e] : 0.f;
        }
    }
    __device__ __forceinline__ void store(const GradParams& g, char* tile, int k0, int wave, int lane) const
    {
        const int lead = (int)((uint64_t)g.p.A & 2);      // (every tile's first element lies in its word as A's)
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) {
            const int slot = (wave * LDS::IPW + j) * 64 + lane, k = k0 + k_of(slot);
            float v[8];
            if constexpr (WIDE) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __int_as_float(wide[j][e / 4][e % 4]);
            } else {
                QuantType<In::F16>::unpack(half[j].get(lead, voff[j]), v);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] *= s[j][KMAJ ? e : 0];
                if (k + (KMAJ ? e : 0) >= g.p.K) v[e] = 0.f;       // past K may stand anything
            }
            i32x4 t[3];
            split8<In::BF16>(v, t);
#pragma unroll
            for (int x = 0; x < 3; ++x) *(i32x4*)(tile + x * LDS::BYTES + slot * 16) = t[x];
        }
    }
};

// Operands at any element (Q: any byte) through registers: LDS in two stages,
// a tile of loads in flight, one barrier a tile.  EPI: added to C.
template <In TI, Out TO, int BM, int BN, int BK, int WM, int WN, bool AK, bool EPI>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_i8grad_odd_kernel(GradParams g)
{
    using GT = GradTypes<TI, TO>;
    constexpr In MT = GT::MT;
    constexpr int TA = GT::TA, TQ = GT::TQ, NW = WM * WN;
    using KT = Dma16<MT, TO, BM, BN, BK, WM, WN, 16, 2, AK, false>;
    using OA = AOperand<TI, BM, BK, NW, AK, GT::SPLIT_A>;
    using OQ = QOperand<MT, BN, BK, NW, TQ, !GT::SPLIT_A>;
    constexpr int STAGE = TA * KT::OA::BYTES + TQ * KT::OB::BYTES, SMEM = 2 * STAGE;
    static_assert(SMEM <= 160 * 1024 && SMEM >= KT::SMEM, "LDS budget");
    __shared__ __attribute__((aligned(1024))) char smem[SMEM];
    const Params& p = g.p;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_coords(p, tm, tn);
    tm = __builtin_amdgcn_readfirstlane(tm);
    tn = __builtin_amdgcn_readfirstlane(tn);
    const int m0 = tm * BM, n0 = tn * BN, wm = wave / WN, wn = wave % WN, nkt = (p.K + BK - 1) / BK;
    typename KT::Acc acc;
    KT::zero(acc);
    OA oa;
    OQ oq;
    oa.init(wave, lane, p.lda);
    oq.init(wave, lane, p.ldb);
    auto load = [&](int t) {                      // past the end: empty extents
        oa.load(g, t < nkt ? p.a_bytes : 0, m0, t * BK, wave, lane);
        oq.load(g, t < nkt ? p.b_bytes : 0, n0, t * BK, wave, lane);
    };
    load(0);
    for (int t = 0; t < nkt; ++t) {
        char* const sa = smem + t % 2 * STAGE;
        char* const sq = sa + TA * KT::OA::BYTES;
        oa.store(g, sa, t * BK, wave, lane);
        oq.store(g, sq, n0, t * BK, wave, lane);
        load(t + 1);
        // The other stage is written after the next barrier, when every wave
        // has read it.
        __builtin_amdgcn_s_waitcnt(0xc07f);       // lgkmcnt(0)
        bare_barrier();
#pragma unroll
        for (int x = 0; x < KT::NG; ++x) {
            i32x4 fa[TA][KT::TM], fq[TQ][KT::TN];
#pragma unroll
            for (int s = 0; s < TA; ++s)
#pragma unroll
                for (int i = 0; i < KT::TM; ++i)
                    fa[s][i] = KT::OA::template frag<16>(sa + s * KT::OA::BYTES, wm * KT::WTM + i * 16, x * 32, lane);
#pragma unroll
            for (int s = 0; s < TQ; ++s)
#pragma unroll
                for (int j = 0; j < KT::TN; ++j)
                    fq[s][j] = KT::OB::template frag<16>(sq + s * KT::OB::BYTES, wn * KT::WTN + j * 16, x * 32, lane);
            // Small terms first.
#pragma unroll
            for (int s = TA * TQ - 1; s >= 0; --s)
#pragma unroll
                for (int i = 0; i < KT::TM; ++i)
#pragma unroll
                    for (int j = 0; j < KT::TN; ++j) mfma_step<MT, 16>(fa[s / TQ][i], fq[s % TQ][j], acc[i][j]);
        }
    }
    store_tile<KT, EPI>(p, smem, m0, n0, acc, tid, lane, wave);
}

// ------------------------------------------------------------------ launchers

// What the host asks of a type's launchers (gemm_i8grad_<dtype>.hip).
struct GradCall {
    GradParams g;         // g.p.epi: add to C
    bool a_kmajor;
    bool vec;             // A and Q allow 16-byte loads
};

template <In TI, Out TO>
struct GradInst {
    template <class Kernel>
    static hipError_t run(Kernel kernel, GradParams g, int bm, int bn, int threads, hipStream_t s)
    {
        Params& p = g.p;
        p.tiles_m = (int)ceil_div(p.M, bm);
        p.tiles_n = (int)ceil_div(p.N, bn);
        p.group_m = p.tiles_m < 8 ? p.tiles_m : 8;
        void* args[] = {&g};
        return hipLaunchKernel((const void*)kernel, dim3((unsigned)(p.tiles_m * p.tiles_n)), dim3(threads), args, 0, s);
    }
    template <bool AK, bool EPI>
    static hipError_t go(const GradCall& c, hipStream_t s)
    {
        return run(&gemm_i8grad_odd_kernel<TI, TO, 64, 64, 32, 2, 2, AK, EPI>, c.g, 64, 64, 256, s);
    }
    static hipError_t launch(const GradCall& c, hipStream_t s)
    {
        if (c.a_kmajor) return c.g.p.epi ? go<true, true>(c, s) : go<true, false>(c, s);
        return c.g.p.epi ? go<false, true>(c, s) : go<false, false>(c, s);
    }
};

hipError_t i8grad_f32(const GradCall& c, hipStream_t s);
hipError_t i8grad_f16_f32(const GradCall& c, hipStream_t s);
hipError_t i8grad_bf16_bf16(const GradCall& c, hipStream_t s);
hipError_t i8grad_f16_f16(const GradCall& c, hipStream_t s);
hipError_t i8grad_bf16_f32(const GradCall& c, hipStream_t s);

}  // namespace mg
