// gemm_i8grad.hpp -- products with 8-bit values whose scales lie along the
// summed index (gfx950): the gradients of a linear layer from 8-bit checkpoints.
//
//   C[m][n] (+)= sum_k A[m][k] scales[k] Q[n][k]
//
// Q is stored k by k (element (n, k) at n + k * ldq), A m- or k-contiguous.
// The scale cannot leave the sum, so it joins a factor before the matrix units
// take it: A, as Q is exact in bf16 (bf16 A into fp32 C: Q, which is converted
// anyway).  The product scales[k] * A[m][k] (scales[k] * Q[n][k]), rounded to fp32,
// enters in bf16 terms:
//   fp32 C: three of 8 bits each, which hold it whole.  Two made the result 2.5e-6
//     off (relative, 8192 k of normal values), where fp32 sums alone are off by
//     5e-7.  For fp32 A three bf16 MFMAs take less than half the time of the fp32
//     ones.
//   16-bit C: two, off by 2^-16 of it at most, where C's own rounding is off by up
//     to 2^-9 (bf16) or 2^-12 (fp16).  With one (the restored value rounded to A's
//     type) results were 2.35e-3 off in bf16 and 2.9e-4 in fp16, where that rounding
//     alone is off by 1.66e-3 and 2.1e-4.
// The matrix units take bf16's subnormals as they are, whose step is 2^-133: bits of
// the product below that are cut off (rounded, of two terms).
#pragma once

#include "gemm_i8_tiles.hpp"
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
    static constexpr bool SPLIT_A = TO != Out::F32 || TI != In::BF16;   // the scale joins A (else Q)
    static constexpr int TERMS = TO == Out::F32 ? 3 : 2;
    static constexpr int TA = SPLIT_A ? TERMS : 1, TQ = SPLIT_A ? 1 : TERMS;
};

// Two fp32 values rounded to bf16, side by side.
__device__ __forceinline__ int pack_bf16(float lo, float hi)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(int, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}
// ... cut off to bf16.
__device__ __forceinline__ int cut_bf16(float lo, float hi)
{
    return (int)__builtin_amdgcn_perm((uint32_t)__float_as_int(hi), (uint32_t)__float_as_int(lo), 0x07060302u);
}
// What that leaves, exactly (of an infinity, NaN).
__device__ __forceinline__ float rest_bf16(float v) { return v - __int_as_float(__float_as_int(v) & (int)0xffff0000); }

// Eight integers of a byte each: bf16 holds them.
__device__ __forceinline__ void split8(float (&v)[8], i32x4 (&t)[1])
{
#pragma unroll
    for (int d = 0; d < 4; ++d) t[0][d] = pack_bf16(v[2 * d], v[2 * d + 1]);
}

// Eight fp32 values in two bf16 terms: the first 8 bits, and the rest rounded.  An
// infinity is all in the first, so that it stays one times Q.
__device__ __forceinline__ void split8(float (&v)[8], i32x4 (&t)[2])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = settled(v[e]);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        t[0][d] = cut_bf16(v[2 * d], v[2 * d + 1]);
        float r[2] = {rest_bf16(v[2 * d]), rest_bf16(v[2 * d + 1])};
        r[0] = r[0] == r[0] ? r[0] : 0.f;
        r[1] = r[1] == r[1] ? r[1] : 0.f;
        t[1][d] = pack_bf16(r[0], r[1]);
    }
}

// ... in three by cutting off: 8 of the 24 bits each, nothing is left (of an
// infinity, NaN).
__device__ __forceinline__ void split8(float (&v)[8], i32x4 (&t)[3])
{
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if (s == 0) {
                v[2 * d] = settled(v[2 * d]);
                v[2 * d + 1] = settled(v[2 * d + 1]);
            }
            t[s][d] = cut_bf16(v[2 * d], v[2 * d + 1]);
            if (s < 2) {
                v[2 * d] = rest_bf16(v[2 * d]);
                v[2 * d + 1] = rest_bf16(v[2 * d + 1]);
            }
        }
}

// An operand from one k-tile to the next: its resource begins at the tile and
// ends with the operand.  Scalar throughout (64-bit comparisons are not, and
// forming the resources anew from the tile's index took 150 cycles a tile).
// ALIGN: from the word that holds the first byte to the end of the last one;
// steps are multiples of 4 bytes.
template <bool ALIGN>
struct Walk {
    uint64_t at, left;
    int64_t step;
    __device__ __forceinline__ void init(const char* base, uint64_t bytes, int64_t origin, int64_t step_)
    {
        const uint64_t first = (uint64_t)base + (uint64_t)origin, lead = ALIGN ? first & 3 : 0;
        at = first - lead;
        left = bytes - (uint64_t)origin + lead;
        if (ALIGN) left = (left + 3) & ~(uint64_t)3;
        step = step_;
    }
    // Not live: nothing is left.
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t next(bool live)
    {
        uint32_t high = (uint32_t)(left >> 32);
        asm("" : "+s"(high));                     // (the compiler would make it one 64-bit comparison again)
        const uint32_t n = high != 0 ? 0xffffffffu : (uint32_t)left;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)at, (short)0, live ? (int)n : 0, kBufferFlags);
        at += (uint64_t)step;
        left -= (uint64_t)step;
        return r;
    }
};

// Eight bytes of a row: from any byte (three words, shifted), or of a 16-byte
// aligned one.
template <bool VEC>
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
template <>
struct ByteChunk8<true> {
    i32x2 w;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int off) { w = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0); }
    __device__ __forceinline__ void get(int, int& lo, int& hi) const
    {
        lo = w[0];
        hi = w[1];
    }
};
// Sixteen bytes of 16-bit values likewise.
template <bool VEC>
struct HalfChunk : OddChunk {
};
template <>
struct HalfChunk<true> {
    i32x4 v;
    __device__ __forceinline__ void load(const OddRows& s, int off) { v = buf_load16(s.r, off); }
    __device__ __forceinline__ i32x4 get(int, int) const { return v; }
};

// The operands: k-tiles from memory to registers, D tiles ahead, and from there
// to LDS as DmaOperand lays them out, a tile a term.

// Q: k rows of ROWS bytes to [BK][ROWS] bf16 values, exact or times scales[k].  A lane
// loads what makes one 16-byte chunk of values, or two, side by side (their XOR
// keys are even).
template <int ROWS, int BK, int NW, int TERMS, bool VEC, int D>
struct QOperand {
    using LDS = DmaOperand<ROWS, BK, NW, false, 16>;
    static constexpr bool SCALED = TERMS > 1, PAIR = VEC && LDS::IPW % 2 == 0;
    static constexpr int W = PAIR ? 2 : 1, UNITS = LDS::IPW / W, PER_ROW = LDS::RCH / W;
    int voff[UNITS];
    ByteChunk8<VEC> q[D][LDS::IPW];
    float s[D][UNITS];
    Walk<!VEC> walk;
    Walk<false> walk_s;

    __device__ static __forceinline__ int unit(int wave, int lane, int j) { return (wave * UNITS + j) * 64 + lane; }
    // From the tile at k0 on, `every` tiles at a time.
    __device__ __forceinline__ void init(int wave, int lane, const GradParams& g, int row0, int k0, int every)
    {
        const int64_t origin = (int64_t)k0 * g.p.ldb + row0;
        const int lead = VEC ? 0 : (int)((uint64_t)(g.p.B + origin) & 3);
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const int k = unit(wave, lane, j) / PER_ROW, phys = unit(wave, lane, j) % PER_ROW;
            voff[j] = (int)(k * g.p.ldb) + (phys * W ^ LDS::mkey(k)) * 8 + lead;
        }
        walk.init(g.p.B, g.p.b_bytes, origin, (int64_t)every * BK * g.p.ldb);
        walk_s.init((const char*)g.scales, (uint64_t)g.p.K * 4, (int64_t)k0 * 4, (int64_t)every * BK * 4);
    }
    // Rows from K on lie past the extent and read as zeros, scale included.
    __device__ __forceinline__ void load(int d, bool live, int wave, int lane)
    {
        const __amdgpu_buffer_rsrc_t r = walk.next(live), rs = walk_s.next(live);
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            if constexpr (PAIR) {
                const i32x4 v = buf_load16(r, voff[j]);
                q[d][2 * j].w = i32x2{v[0], v[1]};
                q[d][2 * j + 1].w = i32x2{v[2], v[3]};
            } else {
                q[d][j].load(r, voff[j]);
            }
            if constexpr (SCALED)
                s[d][j] = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, unit(wave, lane, j) / PER_ROW * 4, 0, 0));
        }
    }
    __device__ __forceinline__ void store(int d, const GradParams& g, char* tile, int k0, int wave, int lane) const
    {
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) {
            // Of a pair, lanes 4 to 7 of 8 write the second first: 8 lanes' writes then
            // lie on different banks of the 128 bytes that a cycle writes.
            const int u = j / W, swap = PAIR && (lane & 4) ? 1 : 0, chunk = unit(wave, lane, u) * W + (j % W ^ swap);
            int w[2];
            if constexpr (PAIR) {
                const i32x2 first = q[d][j].w, other = q[d][j ^ 1].w;
                w[0] = swap ? other[0] : first[0];
                w[1] = swap ? other[1] : first[1];
            } else {
                q[d][j].get(voff[u], w[0], w[1]);
            }
            if constexpr (!VEC) {
                // The words at the last row's end can hold bytes of what follows it.
                if (k0 + chunk / LDS::RCH >= g.p.K) w[0] = w[1] = 0;
            }
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = byte_value(w[e / 4], e % 4);
                if constexpr (SCALED) v[e] *= s[d][u];
            }
            i32x4 t[TERMS];
            split8(v, t);
#pragma unroll
            for (int x = 0; x < TERMS; ++x) *(i32x4*)(tile + x * LDS::BYTES + chunk * 16) = t[x];
        }
    }
};

// Physical 16-byte chunk of chunk c of a k-contiguous row in LDS.  As swz_chunk,
// but for rows of 4 chunks, where a read's lanes go by fours of rows in the order
// 0 3 1 2 with the next chunk in the latter two: XOR with 0 3 2 1 keeps those on
// different banks too (swz_chunk's 0 1 2 3 cost 6 % of the cycles of the
// k-major 256x256 tile).
template <int CPR>
__device__ __forceinline__ int grad_chunk(int row, int c)
{
    if constexpr (CPR == 4) return c ^ (-(row / 4) & 3);
    else return swz_chunk<CPR, true>(row, c);
}
template <class LDS, bool KMAJ>
__device__ __forceinline__ i32x4 a_frag(const char* t, int rbase, int kb, int lane)
{
    if constexpr (KMAJ) {
        const int row = rbase + lane % 16;
        return *(const i32x4*)(t + row * LDS::RB + grad_chunk<LDS::CPR>(row, kb / 8 + lane / 16) * 16);
    } else {
        return LDS::template frag<16>(t, rbase, kb, lane);
    }
}

// A: bf16 values as they are, or (SPLIT) times scales[k] in TERMS bf16 terms.
template <In TI, int ROWS, int BK, int NW, bool KMAJ, int TERMS, bool VEC, int D>
struct AOperand {
    using LDS = DmaOperand<ROWS, BK, NW, KMAJ, 16>;
    static constexpr bool WIDE = TI == In::F32, SPLIT = TERMS > 1;
    static constexpr int ES = WIDE ? 4 : 2, NS = !SPLIT ? 0 : KMAJ ? 8 : 1;
    int voff[LDS::IPW];
    i32x4 wide[WIDE ? D : 1][WIDE ? LDS::IPW : 1][2];
    HalfChunk<VEC> half[WIDE ? 1 : D][WIDE ? 1 : LDS::IPW];
    float s[SPLIT ? D : 1][LDS::IPW][NS ? NS : 1];
    Walk<!VEC && !WIDE> walk;
    Walk<false> walk_s;

    // k of a slot's first value within the tile.
    __device__ static __forceinline__ int k_of(int slot)
    {
        return KMAJ ? grad_chunk<LDS::CPR>(slot / LDS::CPR, slot % LDS::CPR) * 8 : slot / LDS::RCH;
    }
    // From the tile at k0 on, `every` tiles at a time.
    __device__ __forceinline__ void init(int wave, int lane, const GradParams& g, int row0, int k0, int every)
    {
        const int64_t ld = g.p.lda;
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) {
            const int slot = (wave * LDS::IPW + j) * 64 + lane, k = slot / LDS::RCH;
            voff[j] = KMAJ ? (int)(slot / LDS::CPR * ld * ES) + k_of(slot) * ES
                           : (int)(k * ld * ES) + (slot % LDS::RCH ^ LDS::mkey(k)) * 8 * ES;
        }
        walk.init(g.p.A, g.p.a_bytes, (KMAJ ? (int64_t)row0 * ld + k0 : (int64_t)k0 * ld + row0) * ES,
                  (int64_t)every * BK * (KMAJ ? 1 : ld) * ES);
        walk_s.init((const char*)g.scales, (uint64_t)g.p.K * 4, (int64_t)k0 * 4, (int64_t)every * BK * 4);
    }
    __device__ __forceinline__ void load(int d, const GradParams& g, bool live, int wave, int lane)
    {
        OddRows r;
        r.r = walk.next(live);
        r.lead = (int)((uint64_t)g.p.A & 2);              // (every tile's first element lies in its word as A's)
        const __amdgpu_buffer_rsrc_t rs = walk_s.next(live);
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) {
            if constexpr (WIDE) {
                wide[d][j][0] = buf_load16(r.r, voff[j]);
                wide[d][j][1] = buf_load16(r.r, voff[j] + 16);
            } else {
                half[d][j].load(r, voff[j]);
            }
            const int k = k_of((wave * LDS::IPW + j) * 64 + lane);
            if constexpr (NS == 1) {
                s[d][j][0] = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, k * 4, 0, 0));
            } else if constexpr (NS == 8) {       // (scales are 4-byte aligned: k is a multiple of 8)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const i32x4 v = buf_load16(rs, k * 4 + h * 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[d][j][h * 4 + e] = __int_as_float(v[e]);
                }
            }
        }
    }
    __device__ __forceinline__ void store(int d, const GradParams& g, char* tile, int k0, int wave, int lane) const
    {
        const int lead = (int)((uint64_t)g.p.A & 2);
        // What lies past K may be anything, but for whole rows past the extent.
        const bool part = (KMAJ || !VEC) && k0 + BK > g.p.K;
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) {
            const int slot = (wave * LDS::IPW + j) * 64 + lane, left = g.p.K - k0 - k_of(slot);
            if constexpr (!SPLIT) {
                i32x4 v = half[d][j].get(lead, voff[j]);
                if (part) {
                    asm volatile("");
                    if constexpr (KMAJ) v = mask_k<In::F16>(v, 0, left);
                    else v = left > 0 ? v : i32x4{0, 0, 0, 0};
                }
                *(i32x4*)(tile + slot * 16) = v;
            } else {
                float v[8];
                if constexpr (WIDE) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = __int_as_float(wide[d][j][e / 4][e % 4]);
                } else {
                    QuantType<TI>::unpack(half[d][j].get(lead, voff[j]), v);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= s[d][j][KMAJ ? e : 0];
                if (part) {
                    asm volatile("");
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if ((KMAJ ? e : 0) >= left) v[e] = 0.f;
                }
                i32x4 t[TERMS];
                split8(v, t);
#pragma unroll
                for (int x = 0; x < TERMS; ++x) *(i32x4*)(tile + x * LDS::BYTES + slot * 16) = t[x];
            }
        }
    }
};

// LDS in two stages, D tiles of loads in flight; while a tile is multiplied the
// next one is scaled, converted and written.  VEC: 16-byte aligned A and Q; else
// any element and byte.  EPI: added to C.
template <In TI, Out TO, int BM, int BN, int BK, int WM, int WN, int D, int OCC, bool AK, bool VEC, bool EPI>
__global__ void __launch_bounds__(WM * WN * 64, OCC)
gemm_i8grad_kernel(GradParams g)
{
    using GT = GradTypes<TI, TO>;
    constexpr int TA = GT::TA, TQ = GT::TQ, NW = WM * WN;
    using KT = Dma16<In::BF16, TO, BM, BN, BK, WM, WN, 16, 2, AK, false>;
    using OA = AOperand<TI, BM, BK, NW, AK, TA, VEC, D>;
    using OQ = QOperand<BN, BK, NW, TQ, VEC, D>;
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
    oa.init(wave, lane, g, m0, 0, 1);
    oq.init(wave, lane, g, n0, 0, 1);
    auto load = [&](int t, int d) {               // tile by tile; past the end: empty extents
        oa.load(d, g, t < nkt, wave, lane);
        oq.load(d, t < nkt, wave, lane);
    };
    auto store = [&](int t, int d, char* sa) {
        oa.store(d, g, sa, t * BK, wave, lane);
        oq.store(d, g, sa + TA * KT::OA::BYTES, t * BK, wave, lane);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, d);
    store(0, 0, smem);
    load(D, 0);
    __builtin_amdgcn_s_waitcnt(0xc07f);           // lgkmcnt(0)
    bare_barrier();
    // The loop twice: half the waves convert the next tile first and multiply
    // then, the others (which share the SIMDs with them) the other way round.
    auto loop = [&](auto early) {
        for (int t0 = 0; t0 < nkt; t0 += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int t = t0 + d;
                if (t >= nkt) break;
                const int stage = D == 1 ? t & 1 : d % 2;
                const char* const sa = smem + stage * STAGE;
                const char* const sq = sa + TA * KT::OA::BYTES;
                // The next k-group's fragments ahead, where registers hold both; where not
                // (the 256x256 tile), a term's are read behind the products of the other.
                constexpr bool AHEAD = KT::TM * KT::TN * 4 + 8 * (TA * KT::TM + TQ * KT::TN) <= 200;
                constexpr int F = AHEAD ? 2 : 1;
                static_assert(AHEAD || TQ == 1, "terms read one by one are A's");
                i32x4 fa[F][TA][KT::TM], fq[F][TQ][KT::TN];
                auto read_a = [&](int x, int s) {
#pragma unroll
                    for (int i = 0; i < KT::TM; ++i)
                        fa[x % F][s][i] = a_frag<typename KT::OA, AK>(sa + s * KT::OA::BYTES, wm * KT::WTM + i * 16, x * 32, lane);
                };
                auto read_q = [&](int x, int s) {
#pragma unroll
                    for (int j = 0; j < KT::TN; ++j)
                        fq[x % F][s][j] = KT::OB::template frag<16>(sq + s * KT::OB::BYTES, wn * KT::WTN + j * 16, x * 32, lane);
                };
                auto read = [&](int x) {
                    if constexpr (AHEAD) {
#pragma unroll
                        for (int s = 0; s < TA; ++s) read_a(x, s);
#pragma unroll
                        for (int s = 0; s < TQ; ++s) read_q(x, s);
                    } else {
                        read_a(x, TA - 1);
                        read_q(x, 0);
                    }
                };
                // The other stage: every wave has read it before the last barrier.
                auto next = [&]() {
                    store(t + 1, (d + 1) % D, smem + (1 - stage) * STAGE);
                    load(t + 1 + D, (d + 1) % D);
                };
                read(0);
                if constexpr (early) {
                    next();
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int x = 0; x < KT::NG; ++x) {
                    if (AHEAD && x + 1 < KT::NG) read(x + 1);
                    // Small terms first.
#pragma unroll
                    for (int s = TA * TQ - 1; s >= 0; --s) {
#pragma unroll
                        for (int i = 0; i < KT::TM; ++i)
#pragma unroll
                            for (int j = 0; j < KT::TN; ++j)
                                mfma_step<In::BF16, 16>(fa[x % F][s / TQ][i], fq[x % F][s % TQ][j], acc[i][j]);
                        if constexpr (!AHEAD) {
                            if (s > 0) read_a(x, s - 1);
                        }
                    }
                    if (!AHEAD && x + 1 < KT::NG) read(x + 1);
                }
                if constexpr (!early) {
                    __builtin_amdgcn_sched_barrier(0);
                    next();
                }
                __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
                bare_barrier();
            }
        }
    };
    if (wave < NW / 2) loop(std::true_type{});
    else loop(std::false_type{});
    store_tile<KT, EPI>(p, smem, m0, n0, acc, tid, lane, wave);
}

// Few tiles: NW waves take a tile's k-tiles in turn, each through LDS of its own
// with nothing to wait for but itself, and their sums meet at the end, in wave
// order.
template <In TI, Out TO, int BM, int BN, int BK, int NW, int D, bool AK, bool VEC>
__global__ void __launch_bounds__(NW * 64)
gemm_i8grad_stream_kernel(GradParams g)
{
    using GT = GradTypes<TI, TO>;
    constexpr int TA = GT::TA, TQ = GT::TQ;
    using KT = Dma16<In::BF16, TO, BM, BN, BK, 1, 1, 16, 2, AK, false>;
    using OA = AOperand<TI, BM, BK, 1, AK, TA, VEC, D>;
    using OQ = QOperand<BN, BK, 1, TQ, VEC, D>;
    constexpr int STAGE = TA * KT::OA::BYTES + TQ * KT::OB::BYTES, PART = BM * BN;
    constexpr int SMEM = NW * (STAGE > PART * 4 ? STAGE : PART * 4);
    static_assert(SMEM <= 160 * 1024, "LDS budget");
    __shared__ __attribute__((aligned(1024))) char smem[SMEM];
    const Params& p = g.p;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm) * BM, n0 = __builtin_amdgcn_readfirstlane(tn) * BN;
    const int nkt = (p.K + BK - 1) / BK;
    typename KT::Acc acc;
    KT::zero(acc);
    OA oa;
    OQ oq;
    oa.init(0, lane, g, m0, wave * BK, NW);
    oq.init(0, lane, g, n0, wave * BK, NW);
    auto load = [&](int t, int d) {               // tile by tile; past the end: empty extents
        oa.load(d, g, t < nkt, 0, lane);
        oq.load(d, t < nkt, 0, lane);
    };
    char* const sa = smem + wave * STAGE;
    char* const sq = sa + TA * KT::OA::BYTES;
#pragma unroll
    for (int d = 0; d < D; ++d) load(wave + d * NW, d);
    for (int t0 = wave; t0 < nkt; t0 += D * NW) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int t = t0 + d * NW;
            if (t >= nkt) break;
            oa.store(d, g, sa, t * BK, 0, lane);
            oq.store(d, g, sq, t * BK, 0, lane);
            load(t + D * NW, d);
            __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0): written
            asm volatile("" ::: "memory");
#pragma unroll
            for (int x = 0; x < KT::NG; ++x) {
                i32x4 fa[TA][KT::TM], fq[TQ][KT::TN];
#pragma unroll
                for (int s = 0; s < TA; ++s)
#pragma unroll
                    for (int i = 0; i < KT::TM; ++i)
                        fa[s][i] = a_frag<typename KT::OA, AK>(sa + s * KT::OA::BYTES, i * 16, x * 32, lane);
#pragma unroll
                for (int s = 0; s < TQ; ++s)
#pragma unroll
                    for (int j = 0; j < KT::TN; ++j)
                        fq[s][j] = KT::OB::template frag<16>(sq + s * KT::OB::BYTES, j * 16, x * 32, lane);
#pragma unroll
                for (int s = TA * TQ - 1; s >= 0; --s)            // small terms first
#pragma unroll
                    for (int i = 0; i < KT::TM; ++i)
#pragma unroll
                        for (int j = 0; j < KT::TN; ++j) mfma_step<In::BF16, 16>(fa[s / TQ][i], fq[s % TQ][j], acc[i][j]);
            }
            __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0): read, the next tile may be written
            asm volatile("" ::: "memory");
        }
    }
    __syncthreads();
    float* const part = (float*)smem;
#pragma unroll
    for (int i = 0; i < KT::TM; ++i)
#pragma unroll
        for (int j = 0; j < KT::TN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[wave * PART + KT::row(0, i, e, lane) * BN + KT::col(0, j, lane)] = acc[i][j][e];
    __syncthreads();
    for (int x = tid; x < PART; x += NW * 64) {
        const int m = m0 + x / BN, n = n0 + x % BN;
        if (m >= p.M || n >= p.N) continue;
        float v = part[x];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += part[w * PART + x];
        const int64_t at = (int64_t)m * p.ldc + n;
        store_out<TO>(p.C, at, p.epi ? v + load_out<TO>(p.C, at) : v);
    }
}

// ------------------------------------------------------------------ launchers

// What the host asks of a type's launchers (gemm_i8grad_<dtype>.hip).
struct GradCall {
    GradParams g;         // g.p.epi: add to C
    bool a_kmajor;
    bool vec;             // A and Q allow 16-byte loads
};

inline GradShape shape_of(const GradCall& c, bool wide, bool split_a) { return {c.vec, wide, split_a, c.g.p.M, c.g.p.N, c.g.p.K, c.a_kmajor}; }

template <In TI, Out TO>
struct GradInst {
    using GT = GradTypes<TI, TO>;
    static constexpr bool WIDE = TO == Out::F32;
    static hipError_t run(const void* kernel, const GradCall& c, const Tile& t, hipStream_t s)
    {
        GradParams g = c.g;
        Params& p = g.p;
        p.tiles_m = (int)ceil_div(p.M, t.bm);
        p.tiles_n = (int)ceil_div(p.N, t.bn);
        p.group_m = p.tiles_m < 8 ? p.tiles_m : 8;
        void* args[] = {&g};
        return hipLaunchKernel(kernel, dim3((unsigned)grad_grid(shape_of(c, WIDE, GT::SPLIT_A), t)), dim3(t.threads), args, 0, s);
    }
    template <GradTile T, bool AK, bool VEC>
    static hipError_t tile(const GradCall& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T, WIDE, GT::SPLIT_A, AK);
        if constexpr (!has_kernel(T, VEC, WIDE, GT::SPLIT_A, AK))
            return hipErrorInvalidValue;
        else if constexpr (T == GradTile::Stream32x32 || T == GradTile::Stream32x64)
            return run((const void*)&gemm_i8grad_stream_kernel<TI, TO, t.bm, t.bn, t.bk, t.extra, t.stages, AK, VEC>, c, t, s);
        else
            return run(c.g.p.epi ? (const void*)&gemm_i8grad_kernel<TI, TO, t.bm, t.bn, t.bk, t.wm, t.wn, t.stages, t.extra, AK, VEC, true>
                                 : (const void*)&gemm_i8grad_kernel<TI, TO, t.bm, t.bn, t.bk, t.wm, t.wn, t.stages, t.extra, AK, VEC, false>,
                       c, t, s);
    }
    template <bool AK, bool VEC>
    static hipError_t go(const GradCall& c, hipStream_t s)
    {
        switch (grad_tile(shape_of(c, WIDE, GT::SPLIT_A))) {
        case GradTile::Stream32x32: return tile<GradTile::Stream32x32, AK, VEC>(c, s);
        case GradTile::Stream32x64: return tile<GradTile::Stream32x64, AK, VEC>(c, s);
        case GradTile::T64x64: return tile<GradTile::T64x64, AK, VEC>(c, s);
        case GradTile::T64x128: return tile<GradTile::T64x128, AK, VEC>(c, s);
        case GradTile::T64x128Two: return tile<GradTile::T64x128Two, AK, VEC>(c, s);
        case GradTile::T128x128Deep: return tile<GradTile::T128x128Deep, AK, VEC>(c, s);
        case GradTile::T128x128: return tile<GradTile::T128x128, AK, VEC>(c, s);
        case GradTile::T256x256: return tile<GradTile::T256x256, AK, VEC>(c, s);
        case GradTile::Tall256x128: return tile<GradTile::Tall256x128, AK, VEC>(c, s);
        case GradTile::Wide128x256: return tile<GradTile::Wide128x256, AK, VEC>(c, s);
        default: return hipErrorInvalidValue;
        }
    }
    static hipError_t launch(const GradCall& c, hipStream_t s)
    {
        if (c.a_kmajor) return c.vec ? go<true, true>(c, s) : go<true, false>(c, s);
        return c.vec ? go<false, true>(c, s) : go<false, false>(c, s);
    }
};

hipError_t i8grad_f32(const GradCall& c, hipStream_t s);
hipError_t i8grad_f16_f32(const GradCall& c, hipStream_t s);
hipError_t i8grad_bf16_bf16(const GradCall& c, hipStream_t s);
hipError_t i8grad_f16_f16(const GradCall& c, hipStream_t s);
hipError_t i8grad_bf16_f32(const GradCall& c, hipStream_t s);

}  // namespace mg
