// gemm_lora.hpp -- a shared projection with a low-rank adapter per row (gfx950).
//
//   C[m][n] = sum_k A[m][k] B[n][k] + scale_i sum_r v[m][r] up_i[n][r],
//   v[m][r] = sum_k A[m][k] down_i[r][k],   i = ids[m]
//
// Two launches.  The first computes v, fp32, for every row that has an
// adapter.  The second is the shared product; after its main loop each wave
// adds scale_i v up_i^T to its accumulators, so C is rounded once and neither
// read nor written twice.  (Before the main loop the same code left the
// 256x256 tile's accumulators in registers that spilled all through it.)
//
// Rows of one tile may have different adapters.  A wave walks the distinct
// adapters of its rows: each is multiplied with all of them on the MFMA unit
// into a temporary, and a row takes the temporary only if the adapter is its
// own (a select, not a product with zero: an infinity or NaN in one adapter
// reaches no other request's rows).  The waste is small next to the shared
// product (rank against K), and adapters that no row of the tile has are not
// read.
#pragma once

#include "gemm_ragged.hpp"

namespace mg {

struct Lora {
    const char* down;     // slot l at down + l * s_down: R x K, k-contiguous
    const char* up;       // slot l at up + l * s_up: N x R, r-contiguous
    const int* ids;       // one per row; outside [0, slots): none
    const int* ranks;     // one per slot, or null: R
    const float* scales;  // one per slot, or null: 1
    float* v;             // [splits][M][pitch], fp32
    int64_t s_down, s_up;           // bytes
    int64_t ld_down, ld_up;         // elements
    int slots, R, pitch;            // pitch: R rounded up to 32
    int splits;                     // ranges of k whose partial sums of v add up
    int z;                          // workgroups sharing a row tile's adapters
    bool odd_up;          // up's rows are not 16-byte aligned (with any vec)
};

// R rounded up to whole MFMA steps of any input type.
constexpr int kRankStep = 32;
// Rows of v one workgroup computes, and its threads (64 rows where tiled).
constexpr int kShrinkRows = 16;
constexpr int kShrinkThreads = 256;

// The distinct adapters of up to 64 rows, one lane each.  A lane fetches its
// own row's rank and scale, so that the walk over the adapters waits for no
// memory.
struct Adapter {
    int id;               // -1: none
    int rank;
    float scale;
    uint64_t rows;        // the rows that have it
};
struct Distinct {
    int id, rank;         // of this lane's row; id -1: none
    float scale;
    uint64_t left;

    __device__ __forceinline__ Distinct(const Lora& q, int row, bool valid)
    {
        id = valid ? q.ids[row] : -1;
        if (id >= q.slots) id = -1;
        rank = id >= 0 && q.ranks ? min(max(q.ranks[id], 0), q.R) : q.R;
        scale = id >= 0 && q.scales ? q.scales[id] : 1.f;
        left = __builtin_amdgcn_ballot_w64(id >= 0);
    }
    __device__ __forceinline__ Adapter next()
    {
        if (!left) return {-1, 0, 0.f, 0};
        const int l = (int)__builtin_ctzll(left);
        Adapter a;
        a.id = __builtin_amdgcn_readlane(id, l);
        a.rank = __builtin_amdgcn_readlane(rank, l);
        a.scale = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale), l));
        a.rows = __builtin_amdgcn_ballot_w64(id == a.id);
        left &= ~a.rows;
        return a;
    }
};

// Chunks of rows from `base` on: of 16-byte aligned rows (VEC), fp32 rows, or
// 16-bit rows that start at any element.  kNowhere: an offset that reads zeros
// (also 20 bytes on).
constexpr int kNowhere = -4096;
template <int ES, bool VEC>
struct Rows {
    __amdgpu_buffer_rsrc_t r;
    Rows() = default;
    __device__ __forceinline__ Rows(const char* base, uint64_t bytes) : r(make_rsrc(base, bytes)) {}
    __device__ __forceinline__ i32x4 chunk(int off) const { return load_chunk<ES, VEC>(r, off); }
};
template <>
struct Rows<2, false> : OddRows {
    Rows() = default;
    using OddRows::OddRows;
    __device__ __forceinline__ i32x4 chunk(int off) const
    {
        OddChunk c;
        c.load(*this, off);
        return c.get(lead, off);
    }
};

// v: one workgroup per 16 rows, range of k and share of the rows' distinct
// adapters.  Its four waves take k-steps in turn (operands straight from
// memory into MFMA fragments: A's rows are read once per distinct adapter,
// nothing is reused enough to stage it) and add their sums in LDS in wave
// order.  Columns r >= the slot's rank are written as zeros up to the pitch.
template <In TI, bool VEC>
__global__ void __launch_bounds__(256)
lora_shrink_kernel(Params p, Lora q)
{
    constexpr int ES = TI == In::F32 ? 4 : 2, CE = 16 / ES, KS = 4 * CE;   // k per step
    constexpr int RJ = 2;                                                  // 16-column blocks at a time
    __shared__ float part[4][kShrinkRows][RJ * 16 + 4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m0 = blockIdx.x * kShrinkRows;
    const int split = blockIdx.y;
    const int steps = (p.K + KS - 1) / KS;
    const int s0 = (int)((int64_t)steps * split / q.splits), s1 = (int)((int64_t)steps * (split + 1) / q.splits);
    Distinct d(q, m0 + lane, lane < kShrinkRows && m0 + lane < p.M);
    const Rows<ES, VEC> ra(p.A + (int64_t)m0 * p.lda * ES,
                           rows_extent(min(p.M - m0, kShrinkRows), p.lda * ES, row_tail<ES, VEC>(p.K)));
    const int aoff = (int)((lane % 16) * p.lda * ES);
    float* const out = q.v + ((int64_t)split * p.M + m0) * q.pitch;
    for (int u = 0;;) {
        const Adapter a = d.next();
        if (a.id < 0) break;
        for (int r0 = 0; r0 < q.pitch; r0 += RJ * 16, ++u) {
            if (u % q.z != (int)blockIdx.z) continue;
            f32x4 acc[RJ];
#pragma unroll
            for (int j = 0; j < RJ; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
            const int left = max(0, min(a.rank - r0, RJ * 16));
            const Rows<ES, VEC> rd(q.down + a.id * q.s_down + (int64_t)r0 * q.ld_down * ES,
                                   rows_extent(left, q.ld_down * ES, row_tail<ES, VEC>(p.K)));
            const int doff = (int)((lane % 16) * q.ld_down * ES);
            const int nj = (left + 15) / 16;
            auto body = [&](auto NJ) {
                constexpr int n = decltype(NJ)::value;
                constexpr int UN = 4;                  // steps in flight
                // A wave's steps are neighbours: a row's 64 bytes per step share
                // cache lines with the next step's.
                for (int s = s0 + wave * UN; s < s1; s += 4 * UN) {
                    i32x4 fa[UN], fd[UN][n];
#pragma unroll
                    for (int t = 0; t < UN; ++t) {
                        const int k = (s + t) * KS + (lane / 16) * CE;
                        const bool in = s + t < s1 && k < p.K;
                        fa[t] = ra.chunk(in ? aoff + k * ES : kNowhere);       // past the extent: zeros
#pragma unroll
                        for (int j = 0; j < n; ++j)
                            fd[t][j] = rd.chunk(in ? doff + (int)(16 * j * q.ld_down * ES) + k * ES : kNowhere);
                    }
#pragma unroll
                    for (int t = 0; t < UN; ++t) {
                        const int k = (s + t) * KS + (lane / 16) * CE;
                        if (k + CE > p.K) {            // the chunk that holds K: zeros from K on
                            fa[t] = mask_k<TI>(fa[t], k, p.K);
#pragma unroll
                            for (int j = 0; j < n; ++j) fd[t][j] = mask_k<TI>(fd[t][j], k, p.K);
                        }
#pragma unroll
                        for (int j = 0; j < n; ++j) mfma_step<TI, 16>(fa[t], fd[t][j], acc[j]);
                    }
                }
            };
            if (nj == 1) body(std::integral_constant<int, 1>{});
            else if (nj > 1) body(std::integral_constant<int, RJ>{});
            __syncthreads();                           // the sums of the last adapter have been read
#pragma unroll
            for (int j = 0; j < RJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[wave][(lane / 16) * 4 + e][j * 16 + lane % 16] = acc[j][e];
            __syncthreads();
            for (int x = tid; x < kShrinkRows * RJ * 16; x += 256) {
                const int m = x / (RJ * 16), r = x % (RJ * 16);
                if (!(a.rows >> m & 1) || r0 + r >= q.pitch) continue;
                const float sum = ((part[0][m][r] + part[1][m][r]) + part[2][m][r]) + part[3][m][r];
                out[(int64_t)m * q.pitch + r0 + r] = r < left ? sum : 0.f;
            }
        }
    }
}

// The same for many rows: 64 rows and 64 columns of v per workgroup on the
// direct-to-LDS ring, so that each cache line of A and of the adapter is asked
// for whole and once per workgroup (the fragments straight from memory above
// ask for 64 bytes of 16 rows at a time: 41 us at 4096 rows, K = 4096, rank
// 64, where this form takes 13.6).
template <In TI>
using ShrinkTile = Dma16<TI, Out::F32, 64, 64, 64, 2, 2, 16, 4, true, true>;

template <In TI>
__global__ void __launch_bounds__(256)
lora_shrink_dma_kernel(Params p, Lora q)
{
    using KT = ShrinkTile<TI>;
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m0 = blockIdx.x * 64, split = blockIdx.y;
    const int nkt = (p.K + 63) / 64;
    const int kt0 = (int)((int64_t)nkt * split / q.splits), kt1 = (int)((int64_t)nkt * (split + 1) / q.splits);
    Distinct d(q, m0 + lane, m0 + lane < p.M);
    typename KT::OA oa;
    typename KT::OB ob;
    oa.init(wave, lane, p.lda);
    ob.init(wave, lane, q.ld_down);
    p.ldb = q.ld_down;
    float* const out = q.v + ((int64_t)split * p.M + m0) * q.pitch;
    for (int u = 0;; ++u) {
        const Adapter a = d.next();
        if (a.id < 0) break;
        if (u % q.z != (int)blockIdx.z) continue;
        for (int r0 = 0; r0 < q.pitch; r0 += 64) {
            const int left = max(0, min(a.rank - r0, 64));
            p.B = q.down + a.id * q.s_down + (int64_t)r0 * q.ld_down * 2;
            p.b_bytes = rows_extent(left, q.ld_down * 2, row_tail<2, true>(p.K));
            typename KT::Acc acc;
            KT::zero(acc);
            bare_barrier();               // no wave reads the ring any more
            if (left) KT::mainloop(p, smem, oa, ob, m0, 0, kt0, kt1, acc, tid, lane, wave);
#pragma unroll
            for (int i = 0; i < KT::TM; ++i)
#pragma unroll
                for (int j = 0; j < KT::TN; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int m = KT::row(wave / 2, i, e, lane), r = KT::col(wave % 2, j, lane);
                        if ((a.rows >> m & 1) && r0 + r < q.pitch) out[(int64_t)m * q.pitch + r0 + r] = r < left ? acc[i][j][e] : 0.f;
                    }
        }
    }
}

// Infinities and NaN among two values of a 16-bit type, at their sign bits:
// adding the exponent's lowest bit carries there where it is all ones.
template <In TI>
__device__ __forceinline__ uint32_t not_finite(int word)
{
    return (((uint32_t)word & 0x7fff7fffu) + (TI == In::F16 ? 0x04000400u : 0x00800080u)) & 0x80008000u;
}
// A chunk with zeros in their place.
template <In TI>
__device__ __forceinline__ i32x4 finite_part(i32x4 v)
{
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t over = not_finite<TI>(v[d]);
        v[d] = (int)((uint32_t)v[d] & ~((over << 1) - (over >> 15)));
    }
    return v;
}

// Terms of the input type that a value of v is split into, one MFMA each: the
// part that the type holds, then its rounding of the rest.  v is fp32: two
// terms are off by at most 2^-22 of it in fp16 and by 2^-16 in bf16, three in
// bf16 by 2^-24.  (One alone would be off by 2^-8 there.)  bf16 takes the third
// where the output is fp32 and would show it; a bf16 output is rounded to 2^-8.
// fp16's smallest step is 2^-24, so whoever splits v scales its rows first: to
// a largest value of 2^13 or more, which leaves half a step, 2^-38 of that
// largest, for the values far below it.
constexpr int terms_of_v(In ti, Out to)
{
    return ti == In::F32 ? 1 : ti == In::BF16 && to == Out::F32 ? 3 : 2;
}

// 8 (16-bit) or 4 (fp32) values of v as MFMA fragments.  APART: the first term
// meets infinities of the adapter, so it is zero for v = 0 only; the others, of
// either sign, meet finite values only.
template <In TI, int TERMS>
struct VFrag {
    i32x4 f[TERMS];

    template <bool APART = false>
    __device__ __forceinline__ void set(const float (&v)[TI == In::F32 ? 4 : 8])
    {
        if constexpr (TI == In::F32) {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[0][e] = __float_as_int(v[e]);
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                uint32_t w[TERMS] = {};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = v[2 * d + h];
                    const bool inf = __builtin_fabsf(x) == __builtin_inff();   // then the rest is inf - inf
#pragma unroll
                    for (int t = 0; t < TERMS; ++t) {
                        uint32_t a;
                        if constexpr (TI == In::BF16) {
                            // (Not past bf16's largest: that would be an infinity.)
                            const float most = 0x1.fep127f;
                            a = __builtin_bit_cast(uint16_t, (__bf16)(t > 0 || inf ? x : fminf(fmaxf(x, -most), most)));
                            x -= __int_as_float((int)(a << 16));
                        } else {
                            a = __builtin_bit_cast(uint16_t, (_Float16)x);
                            if (APART && t == 0 && x != 0.f && (a & 0x7fff) == 0) a |= 1;   // (the rest takes it back)
                            x -= (float)__builtin_bit_cast(_Float16, (uint16_t)a);
                        }
                        if (inf) x = 0.f;
                        w[t] |= a << (16 * h);
                    }
                }
#pragma unroll
                for (int t = 0; t < TERMS; ++t) f[t][d] = (int)w[t];
            }
        }
    }
};

// Add scale_i v up_i^T to the accumulators of one wave.  Its rows are m0 ..
// m0 + TM * MI - 1 (at most 64), its columns start at n0; MFMA tile (i, j)
// holds rows i * MI and columns j * MI on.  NB: adapters whose loads are
// in flight together.  Of the rows' distinct adapters, those with an index of
// `share` modulo `shares` are added (all: 0 of 1).
template <In TI, bool VEC, int TERMS, int NB, int MI, int TM, int TN, class AccT, class Col>
__device__ __forceinline__ void lora_add(const Params& p, const Lora& q, AccT (&acc)[TM][TN], int m0, int n0, int lane,
                                         float* tab, int share, int shares, Col col)
{
    constexpr int ES = TI == In::F32 ? 4 : 2, CE = 16 / ES, KS = 64 / MI * CE, R4 = MI == 32 ? 16 : 4;
    constexpr int CH = TI == In::F32 ? 32 : 64;          // columns of v held at a time
    constexpr int NK = CH / KS;
    static_assert(TM * MI <= 64, "one lane per row");
    if (q.slots == 0 || q.R == 0) return;
    const int fr = lane % MI, fk = lane / MI * CE;     // fragment row, first k
    const int up_row = (int)(q.ld_up * ES);            // (256 rows fit 32 bits)
    const int64_t vsplit = (int64_t)p.M * q.pitch * 4;
    const uint64_t vbytes = (uint64_t)max(0, min(p.M - m0, TM * MI)) * q.pitch * 4;
    auto load_v = [&](int i, int r, float (&v)[CE]) {
#pragma unroll
        for (int e = 0; e < CE; ++e) v[e] = 0.f;
        const int off = r + fk < q.pitch ? ((i * MI + fr) * q.pitch + r + fk) * 4 : kNowhere;
        for (int s = 0; s < q.splits; ++s) {
            const __amdgpu_buffer_rsrc_t rs = make_rsrc((const char*)(q.v + (int64_t)m0 * q.pitch) + s * vsplit, vbytes);
#pragma unroll
            for (int e = 0; e < CE; e += 4) {
                const i32x4 t = buf_load16(rs, off + e * 4);
#pragma unroll
                for (int x = 0; x < 4; ++x) v[e + x] += __int_as_float(t[x]);
            }
        }
    };
    Distinct d(q, m0 + lane, lane < TM * MI && m0 + lane < p.M);
    if (!d.left) return;
    const uint64_t all = d.left;
    // fp16: v is scaled by a power of two per row that brings its largest
    // finite value to 2^13 .. 2^14, so that neither part leaves fp16's range.
    // The factors stand in LDS (tab: 128 floats of this wave's own): 2^-e of
    // each row, then 2^e.
    if constexpr (TI == In::F16) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            float top = 0.f;
            for (int r = 0; r < q.pitch; r += KS) {
                float v[CE];
                load_v(i, r, v);
#pragma unroll
                for (int e = 0; e < CE; ++e) {
                    const float x = __builtin_fabsf(v[e]);
                    if (x < __builtin_inff()) top = fmaxf(top, x);
                }
            }
#pragma unroll
            for (int o = MI; o < 64; o *= 2) top = fmaxf(top, __shfl_xor(top, o));
            int e;
            __builtin_frexpf(top, &e);
            e = top > 0.f ? min(14 - e, 120) : 0;
            if (lane < MI) {
                tab[i * MI + lane] = __builtin_ldexpf(1.f, -e);
                tab[64 + i * MI + lane] = __builtin_ldexpf(1.f, e);
            }
        }
        __builtin_amdgcn_s_waitcnt(0xc07f);           // written; only this wave reads them
        asm volatile("" ::: "memory");
    }
    // All adapters of all rows.  APART: the rest of v meets finite values only;
    // `which` says what elements of acc are added to.
    auto pass = [&](auto apart, uint64_t which) {
        constexpr bool APART = decltype(apart)::value;
        for (int r0 = 0; r0 < q.pitch; r0 += CH) {
            VFrag<TI, TERMS> fv[TM][NK];
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    float v[CE];
                    load_v(i, r0 + k * KS, v);
                    if constexpr (TI == In::F16) {
                        const float up = tab[64 + i * MI + fr];
#pragma unroll
                        for (int e = 0; e < CE; ++e) v[e] *= up;
                    }
                    fv[i][k].template set<APART>(v);
                }
            d.left = all;
            int turn = 0;                                  // distinct adapters so far, modulo shares
            auto mine = [&]() {
                for (;;) {
                    const Adapter a = d.next();
                    const bool take = turn == share;
                    turn = turn + 1 == shares ? 0 : turn + 1;
                    if (a.id < 0 || take) return a;
                }
            };
            while (d.left) {
                Adapter a[NB];
                Rows<ES, VEC> ru[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    a[b] = mine();
                    ru[b] = Rows<ES, VEC>(q.up + max(a[b].id, 0) * q.s_up + (int64_t)n0 * q.ld_up * ES,
                                      a[b].id < 0 || n0 >= p.N ? 0 : rows_extent(min(p.N - n0, TN * MI), q.ld_up * ES, row_tail<ES, VEC>(q.R)));
                }
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    i32x4 fu[NB][NK];
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int k = 0; k < NK; ++k) {
                            const int r = r0 + k * KS + fk;
                            fu[b][k] = ru[b].chunk(r < a[b].rank ? col(j) * up_row + r * ES : kNowhere);
                        }
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        if (r0 >= a[b].rank) continue;
#pragma unroll
                        for (int k = 0; k < NK; ++k) {
                            const int r = r0 + k * KS + fk;
                            if (r + CE > a[b].rank) fu[b][k] = mask_k<TI>(fu[b][k], r, a[b].rank);
                        }
#pragma unroll
                        for (int i = 0; i < TM; ++i) {
                            AccT t = {};
#pragma unroll
                            for (int k = 0; k < NK; ++k) {
                                if (r0 + k * KS >= a[b].rank) continue;
#pragma unroll
                                for (int h = 0; h < TERMS; ++h)
                                    mfma_step<TI, MI>(fv[i][k].f[h], APART && h > 0 ? finite_part<TI>(fu[b][k]) : fu[b][k], t);
                            }
#pragma unroll
                            for (int x4 = 0; x4 < R4; x4 += 4) {
                                const int row4 = i * MI + (MI == 32 ? x4 / 4 * 8 + (lane / 32) * 4 : (lane / 16) * 4);
                                f32x4 f = {a[b].scale, a[b].scale, a[b].scale, a[b].scale};
                                if constexpr (TI == In::F16) {
                                    const f32x4 down = *(const f32x4*)(tab + row4);
#pragma unroll
                                    for (int x = 0; x < 4; ++x) f[x] *= down[x];
                                }
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    const float y = __builtin_fmaf(f[x], t[x4 + x], acc[i][j][x4 + x]);
                                    bool take = a[b].rows >> (row4 + x) & 1;
                                    if constexpr (APART) take = take && (which >> ((i * TN + j) * 4 + x) & 1);
                                    acc[i][j][x4 + x] = take ? y : acc[i][j][x4 + x];
                                }
                            }
                        }
                    }
                }
            }
        }
    };
    if constexpr (TI == In::F32) {
        pass(std::false_type{}, 0);
    } else {
        // An infinity of an adapter shows in the sums of its rows.  It is looked for
        // there, once before and once after all adapters: if the product alone has
        // one, everything is added the careful way; if adapters made one, only
        // those elements are, from zero (what was finite in them does not count).
        // (64 rows with an adapter each of rank 64, N = K = 4096, fp16, both
        // kernels: 36.5 us, 36.2 without; a look at every chunk of the adapters
        // 36.9, at every adapter's sums 37.6.)
        static_assert(R4 == 4 && TM * TN * 4 <= 64, "a bit for each accumulator");
        auto all_finite = [&]() {
            float zero = 0.f;                          // NaN if any is not
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x) zero = __builtin_fmaf(acc[i][j][x], 0.f, zero);
            return __builtin_amdgcn_ballot_w64(!(zero == 0.f)) == 0;
        };
        auto not_finite = [&]() {
            uint64_t m = 0;
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        m |= (uint64_t)!(__builtin_fabsf(acc[i][j][x]) < __builtin_inff()) << ((i * TN + j) * 4 + x);
            return m;
        };
        uint64_t which = ~(uint64_t)0;
        if (__builtin_expect(all_finite(), 1)) {
            pass(std::false_type{}, 0);
            if (__builtin_expect(all_finite(), 1)) return;
            which = not_finite();
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (which >> ((i * TN + j) * 4 + x) & 1) acc[i][j][x] = 0.f;
        }
        pass(std::true_type{}, which);
    }
}

// ... with the columns of MFMA tile j next to each other from j * MI on.
template <In TI, bool VEC, int TERMS, int NB, int MI, int TM, int TN, class AccT>
__device__ __forceinline__ void lora_add(const Params& p, const Lora& q, AccT (&acc)[TM][TN], int m0, int n0, int lane,
                                         float* tab, int share = 0, int shares = 1)
{
    const auto col = [&](int j) { return j * MI + lane % MI; };
    if (VEC && q.odd_up) lora_add<TI, false, TERMS, NB < 4 ? NB : 4, MI>(p, q, acc, m0, n0, lane, tab, share, shares, col);
    else lora_add<TI, VEC, TERMS, NB, MI>(p, q, acc, m0, n0, lane, tab, share, shares, col);
}

// The same for a whole workgroup on 16-bit inputs, through LDS (the ring, free
// after the main loop): v of the tile's rows, scaled and split, is put there
// once for all waves, and each adapter's rows for the tile's columns come in
// by direct loads, up to three adapters ahead of the one that is multiplied.  The MFMAs
// add straight into the accumulators (temporaries beside the 256x256 tile's
// accumulators spilled, as did any other use of them here); rows of other
// adapters enter them as zeros.  That keeps rows apart only while the adapter
// is finite, so infinities and NaN in it are replaced by finite values in LDS
// and reported: `repair` then adds their terms to the stored C, for the
// adapter's own rows.  Measured at 4096 rows, N = K =
// 4096, rank 64 in bf16: the product with its adapters 121 us by lora_add,
// whose every adapter waits for its own loads, 110 here (plain 97).
template <class KT, In TI>
struct SharedLora {
    static constexpr int BM = KT::TILE_M, BN = KT::TILE_N, NW = KT::NW, NT = KT::NT, MI = 16;
    static constexpr int TM = KT::TM, TN = KT::TN, WTM = KT::WTM, WTN = KT::WTN, WN = BN / WTN;
    static constexpr int TERMS = terms_of_v(TI, KT::OUT);
    // Columns of v at a time, in MFMA steps.  64, or 32 where three terms of them
    // leave no room for two adapters (256x256 tiles; 4096 rows, N = K = 4096,
    // bf16 into fp32, us: rank 64 124.0, 119.7 with 64 columns of two terms;
    // rank 16 114.0, 115.5).
    static constexpr int SMALL = BM * 16 + 16;         // tables
    static constexpr int CH = KT::SMEM - SMALL >= (TERMS * BM + 2 * BN) * 64 * 2 ? 64 : 32, NG = CH / 32, CPR = CH / 8;
    using OV = DmaOperand<BM, CH, NW, true, MI>;       // for its fragments
    using OU = DmaOperand<BN, CH, NW, true, MI>;
    static constexpr int V_BYTES = BM * CH * 2, U_BYTES = OU::BYTES;
    static constexpr int FIT = (KT::SMEM - TERMS * V_BYTES - SMALL) / U_BYTES, NU = FIT < 4 ? FIT : 4;   // adapters in LDS
    static constexpr int TAB = TERMS * V_BYTES + NU * U_BYTES, ROWS = TAB + BM * 8, BAD = ROWS + BM * 8;
    static_assert(NU >= 2 && (NU - 2) * OU::IPW < 64, "fits the ring; vmcnt range");
    static_assert(64 % WTM == 0, "a wave's rows in one mask");

    // True: an adapter held infinities or NaN (repair has work).
    __device__ static __forceinline__ bool add(const Params& p, const Lora& q, char* smem, typename KT::Acc& acc, int m0,
                                               int n0, int tid, int lane, int wave)
    {
        if (q.slots == 0 || q.R == 0) return false;
        const int wm = wave / WN, wn = wave % WN;
        char* const vt = smem;                         // the terms of v
        char* const ub = smem + TERMS * V_BYTES;       // NU buffers
        float* const tab = (float*)(smem + TAB);       // fp16: 2^e of each row, then 2^-e
        int* const row_id = (int*)(smem + ROWS);       // -1: none
        float* const row_scale = (float*)(row_id + BM);
        int* const bad = (int*)(smem + BAD);
        // Every wave walks the distinct adapters of all the tile's rows (NC
        // rows a lane), so that no wave waits for another to name the next.
        constexpr int NC = (BM + 63) / 64;
        int id[NC], rank[NC];
        uint64_t left_rows[NC];
        bare_barrier();                                // LDS is free
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int m = c * 64 + lane;
            const bool valid = m < BM && m0 + m < p.M;
            id[c] = valid ? q.ids[m0 + m] : -1;
            if (id[c] >= q.slots) id[c] = -1;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const bool has = id[c] >= 0;
            rank[c] = has && q.ranks ? min(max(q.ranks[id[c]], 0), q.R) : q.R;
            const float scale = has && q.scales ? q.scales[id[c]] : 1.f;
            if (wave == c % NW && c * 64 + lane < BM) {
                row_id[c * 64 + lane] = has ? id[c] : -1;
                row_scale[c * 64 + lane] = scale;
            }
        }
        if (tid == 0) *bad = 0;
        // The next adapter, its rank and this wave's rows of it.
        auto next = [&](int& rk, uint64_t& rows) {
            int a = -1;
            rk = 0;
#pragma unroll
            for (int c = NC - 1; c >= 0; --c)
                if (left_rows[c]) {
                    const int l = (int)__builtin_ctzll(left_rows[c]);
                    a = __builtin_amdgcn_readlane(id[c], l);
                    rk = __builtin_amdgcn_readlane(rank[c], l);
                }
            rows = 0;
            if (a < 0) return a;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const uint64_t m = __builtin_amdgcn_ballot_w64(id[c] == a);
                left_rows[c] &= ~m;
                if (wm * WTM / 64 == c) rows = m >> (wm * WTM % 64);
            }
            return a;
        };
        OU ou;
        ou.init(wave, lane, q.ld_up);
        auto issue = [&](int a, int left, int r0, char* dst) {
            if (q.odd_up) {       // through registers (rows of few columns: no loads ahead)
                const OddRows s(q.up + max(a, 0) * q.s_up + (int64_t)n0 * q.ld_up * 2 + r0 * 2,
                                a < 0 ? 0 : rows_extent(min(p.N - n0, BN), q.ld_up * 2, (q.R - r0) * 2));
#pragma unroll 1
                for (int slot = wave * OU::IPW * 64 + lane; slot < (wave + 1) * OU::IPW * 64; slot += 64) {
                    const int row = slot / OU::CPR, c = swz_chunk<OU::CPR, true>(row, slot % OU::CPR);
                    const int off = c * 8 < left ? (int)(row * q.ld_up * 2) + c * 16 : kNowhere;
                    OddChunk v;
                    v.load(s, off);
                    *(i32x4*)(dst + slot * 16) = v.get(s.lead, off);
                }
                return;
            }
            OU o;
#pragma unroll
            for (int j = 0; j < OU::IPW; ++j) {
                const int slot = (wave * OU::IPW + j) * 64 + lane;
                const int c = swz_chunk<OU::CPR, true>(slot / OU::CPR, slot % OU::CPR);
                o.voff[j] = c * 8 < left ? ou.voff[j] : kNowhere;          // past the rank: zeros
            }
            // Past the last adapter: an empty extent, zeros that nobody reads.
            o.issue(q.up + max(a, 0) * q.s_up + (int64_t)n0 * q.ld_up * 2 + r0 * 2,
                    a < 0 ? 0 : rows_extent(min(p.N - n0, BN), q.ld_up * 2, row_tail<2, true>(q.R - r0)), q.ld_up, 0, 0, dst, wave);
        };
        bool found = false, first = true;
        for (int r0 = 0; r0 < q.pitch; r0 += CH) {
#pragma unroll
            for (int c = 0; c < NC; ++c) left_rows[c] = __builtin_amdgcn_ballot_w64(id[c] >= 0);
            __syncthreads();                           // row_id is written; v and U have been read
            int a[NU - 1], rk[NU - 1];                 // the adapters in LDS or on their way
            uint64_t rows[NU - 1];
#pragma unroll
            for (int i = 0; i < NU - 1; ++i) {
                a[i] = next(rk[i], rows[i]);
                if (a[0] < 0) return false;
                issue(a[i], min(rk[i] - r0, CH), r0, ub + i * U_BYTES);
            }
            stage_v(p, q, vt, tab, row_id, row_scale, m0, r0, tid);
            for (int buf = 0; a[0] >= 0; buf = buf + 1 == NU ? 0 : buf + 1) {
                const int left = min(rk[0] - r0, CH);
                const uint64_t own = rows[0];
                char* const u = ub + buf * U_BYTES;
                wait_vmcnt<(NU - 2) * OU::IPW>();
                __builtin_amdgcn_s_waitcnt(0xc07f);
                bare_barrier();                        // this adapter has landed, the last one been read
                if (first) rescale(acc, tab, wm, lane);
                first = false;
#pragma unroll
                for (int i = 0; i + 1 < NU - 1; ++i) {
                    a[i] = a[i + 1];
                    rk[i] = rk[i + 1];
                    rows[i] = rows[i + 1];
                }
                a[NU - 2] = next(rk[NU - 2], rows[NU - 2]);
                issue(a[NU - 2], min(rk[NU - 2] - r0, CH), r0, ub + (buf == 0 ? NU - 1 : buf - 1) * U_BYTES);
                if (left > 0) {
                    clean(u, left, bad, tid);
                    __builtin_amdgcn_s_waitcnt(0xc07f);
                    bare_barrier();                    // (no fence: the next adapters are on their way)
                    if (own) multiply(acc, vt, u, own, left, wm, wn, lane);
                }
            }
            wait_vmcnt<0>();                           // the empty loads have landed
            __syncthreads();
            found = found || *bad;
        }
        rescale(acc, tab + BM, wm, lane);
        return found;
    }

    // fp16: the accumulators' rows by the power of two of each row of v (2^64
    // at most: no product of fp16 values over 2^30 terms leaves fp32 by it).
    __device__ static __forceinline__ void rescale(typename KT::Acc& acc, const float* tab, int wm, int lane)
    {
        if constexpr (TI == In::F16) {
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const f32x4 f = *(const f32x4*)(tab + wm * WTM + i * MI + lane / 16 * 4);
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x) acc[i][j][x] *= f[x];
            }
        }
    }

    // Zeros from the rank on in the chunk that holds it, and values of one to two
    // with their signs in the place of the adapter's infinities and NaN (*bad:
    // there were some).  What finite values of v make of them does not count
    // beside the terms that `repair` adds; an infinite one makes the same
    // infinity, where zeros would make NaN.
    __device__ static __forceinline__ void clean(char* u, int left, int* bad, int tid)
    {
        for (int x = tid; x < BN * CPR; x += NT) {
            const int row = x / CPR, c = x % CPR;
            if (c * 8 >= left) continue;
            i32x4* const at = (i32x4*)(u + row * (CH * 2) + swz_chunk<CPR, true>(row, c) * 16);
            i32x4 v = *at;
            const bool cut = c * 8 + 8 > left;
            if (cut) v = mask_k<TI>(v, c * 8, left);
            uint32_t any = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t over = not_finite<TI>(v[w]);
                any |= over;
                v[w] = (int)((uint32_t)v[w] & ~(over >> 1));               // the exponent's highest bit
            }
            if (any || cut) *at = v;
            if (any) *bad = 1;
        }
    }

    // Add the terms of infinite and NaN adapter values to C, which holds the
    // rest.  Rare, and only for the rows of such an adapter: column by column,
    // straight from memory.  A rest that C's type holds as an infinity of the
    // other sign may have been finite before it was rounded: such an element is
    // summed again from its definition.
    template <bool BKM>
    __device__ static __forceinline__ void repair(const Params& p, const Lora& q, int m0, int n0, int tid)
    {
        constexpr int EO = KT::OUT == Out::F32 ? 4 : 2;
        constexpr uint32_t EXP = TI == In::F16 ? 0x7c00u : 0x7f80u;
        const auto value = [](uint16_t h) {
            return TI == In::F16 ? (float)__builtin_bit_cast(_Float16, h) : __int_as_float((int)((uint32_t)h << 16));
        };
        __builtin_amdgcn_s_waitcnt(0);                 // the tile is stored
        __syncthreads();
        for (int n = n0 + tid; n < min(n0 + BN, p.N); n += NT) {
            int last = -1, rank = 0;
            bool harm = false;
            for (int m = m0; m < min(m0 + BM, p.M); ++m) {
                const int id = q.ids[m];
                if (id < 0 || id >= q.slots) continue;
                const uint16_t* u = (const uint16_t*)(q.up + id * q.s_up) + (int64_t)n * q.ld_up;
                if (id != last) {
                    last = id;
                    rank = q.ranks ? min(max(q.ranks[id], 0), q.R) : q.R;
                    harm = false;
                    for (int r = 0; r < rank; ++r) harm = harm || (u[r] & EXP) == EXP;
                }
                if (!harm) continue;
                const float scale = q.scales ? q.scales[id] : 1.f;
                // scale v up_i^T over the terms whose up is not finite, or over all
                auto terms = [&](bool all) {
                    float sum = 0.f;
                    for (int r = 0; r < rank; ++r) {
                        if (!all && (u[r] & EXP) != EXP) continue;
                        float v = 0.f;
                        for (int s = 0; s < q.splits; ++s) v += q.v[((int64_t)s * p.M + m) * q.pitch + r];
                        sum += scale * v * value(u[r]);
                    }
                    return sum;
                };
                const float sum = terms(false);
                // past this CU's cache: other lanes stored this element
                const __amdgpu_buffer_rsrc_t rc = make_rsrc(p.C + ((int64_t)m * p.ldc + n) * EO, EO);
                float c;
                if constexpr (EO == 4) {
                    c = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(rc, 0, 0, kDeviceCoherent));
                } else {
                    const uint16_t h = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rc, 0, 0, kDeviceCoherent);
                    c = load_out<KT::OUT>((const char*)&h, 0);
                }
                float y = c + sum;
                if (EO == 2 && c == -sum) {            // infinities
                    const uint16_t* const a = (const uint16_t*)p.A + (int64_t)m * p.lda;
                    y = 0.f;
                    for (int k = 0; k < p.K; ++k)
                        y += value(a[k]) * value(((const uint16_t*)p.B)[BKM ? (int64_t)n * p.ldb + k : (int64_t)k * p.ldb + n]);
                    y += terms(true);
                }
                store_out<KT::OUT>(p.C, (int64_t)m * p.ldc + n, y);
            }
        }
    }

    // scale * v of the tile's rows, CH columns from r0 on, as terms of the input
    // type in LDS.  fp16 rows are brought to a largest value of 2^13 ..
    // 2^14 by a power of two (at most 2^64), so that neither term leaves
    // fp16's range; tab: that power and its inverse.
    __device__ static __forceinline__ void stage_v(const Params& p, const Lora& q, char* vt, float* tab,
                                                   const int* row_id, const float* row_scale, int m0, int r0, int tid)
    {
        constexpr int TPR = CH / 4, STEP = NT / TPR, IT = BM / STEP;      // threads per row, rows at a time
        constexpr int MOST = (TI == In::F16 || TERMS > 2) && TM * TN >= 32 ? 2 : 4, BATCH = IT < MOST ? IT : MOST;
        static_assert(IT % BATCH == 0, "whole batches");
        const int c4 = tid % TPR * 4;                  // this thread's 4 columns
        const int64_t split = (int64_t)p.M * q.pitch;
        // The rows of a batch: all their loads before the first is waited for.
        auto load = [&](int mb, int r, f32x4 (&v)[BATCH]) {
            const float* src[BATCH];
            bool has[BATCH];
#pragma unroll
            for (int x = 0; x < BATCH; ++x) {
                const int m = mb + x * STEP;
                has[x] = r < q.pitch && row_id[m] >= 0;
                src[x] = q.v + (int64_t)(m0 + m) * q.pitch + r;
                v[x] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            int s = 0;
            for (; s + 1 < q.splits; s += 2) {
                f32x4 t[2][BATCH];
#pragma unroll
                for (int x = 0; x < BATCH; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        t[y][x] = has[x] ? *(const f32x4*)(src[x] + (s + y) * split) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int x = 0; x < BATCH; ++x) v[x] = v[x] + t[0][x] + t[1][x];
            }
            if (s < q.splits) {
#pragma unroll
                for (int x = 0; x < BATCH; ++x)
                    if (has[x]) v[x] += *(const f32x4*)(src[x] + s * split);
            }
#pragma unroll
            for (int x = 0; x < BATCH; ++x) v[x] *= row_scale[mb + x * STEP];
        };
#pragma unroll 1
        for (int mb = tid / TPR; mb < BM; mb += BATCH * STEP) {
            f32x4 v[BATCH];
            load(mb, r0 + c4, v);
            if constexpr (TI == In::F16) {
                float top[BATCH];
                auto up_to = [&](const f32x4 (&x)[BATCH]) {
#pragma unroll
                    for (int y = 0; y < BATCH; ++y)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = __builtin_fabsf(x[y][e]);
                            if (a < __builtin_inff()) top[y] = fmaxf(top[y], a);
                        }
                };
#pragma unroll
                for (int y = 0; y < BATCH; ++y) top[y] = 0.f;
                if (q.pitch <= CH) {
                    up_to(v);
                } else {
                    for (int r = c4; r < q.pitch; r += CH) {
                        f32x4 w[BATCH];
                        load(mb, r, w);
                        up_to(w);
                    }
                }
#pragma unroll
                for (int y = 0; y < BATCH; ++y) {
#pragma unroll
                    for (int o = 1; o < TPR; o *= 2) top[y] = fmaxf(top[y], __shfl_xor(top[y], o));
                    int e;
                    __builtin_frexpf(top[y], &e);
                    e = top[y] > 0.f ? min(14 - e, 64) : 0;
                    if (c4 == 0) {
                        tab[mb + y * STEP] = __builtin_ldexpf(1.f, e);
                        tab[BM + mb + y * STEP] = __builtin_ldexpf(1.f, -e);
                    }
                    v[y] *= __builtin_ldexpf(1.f, e);
                }
            }
#pragma unroll
            for (int y = 0; y < BATCH; ++y) {
                const int m = mb + y * STEP;
                VFrag<TI, TERMS> f;
                const float x[8] = {v[y][0], v[y][1], v[y][2], v[y][3], 0.f, 0.f, 0.f, 0.f};
                f.set(x);
                const int off = m * (CH * 2) + swz_chunk<CPR, true>(m, c4 / 8) * 16 + c4 % 8 * 2;
                typedef int i32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
                for (int t = 0; t < TERMS; ++t) *(i32x2*)(vt + t * V_BYTES + off) = i32x2{f.f[t][0], f.f[t][1]};
            }
        }
    }

    __device__ static __forceinline__ void multiply(typename KT::Acc& acc, const char* vt, const char* u,
                                                    uint64_t rows, int left, int wm, int wn, int lane)
    {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g * 32 >= left) break;
            i32x4 fv[TERMS][TM];
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const bool own = rows >> (i * MI + lane % MI) & 1;
                const i32x4 zero = {0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < TERMS; ++t) {
                    fv[t][i] = OV::template frag<MI>(vt + t * V_BYTES, wm * WTM + i * MI, g * 32, lane);
                    fv[t][i] = own ? fv[t][i] : zero;
                }
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                __builtin_amdgcn_sched_barrier(0);
                const i32x4 f = OU::template frag<MI>(u, wn * WTN + j * MI, g * 32, lane);
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
#pragma unroll
                    for (int i = 0; i < TM; ++i) mfma_step<TI, MI>(fv[t][i], f, acc[i][j]);
            }
        }
    }
};

// The shared product, for 16-bit operands that are not 16-byte aligned.
template <In TI, Out TO, int BM, int BN, int BK, int WM, int WN, int DEPTH, bool BKM>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_lora_odd_kernel(Params p, Lora q)
{
    using T = OddTile<TI, TO, BM, BN, BK, WM, WN, DEPTH, true, BKM>;
    using KT = typename T::KT;
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm * BM), n0 = __builtin_amdgcn_readfirstlane(tn * BN);
    typename KT::Acc acc;
    KT::zero(acc);
    T::mainloop(p, smem, m0, n0, acc, lane, wave);
    bare_barrier();       // no wave reads the tiles any more
    lora_add<TI, false, terms_of_v(TI, TO), 1, 16, KT::TM, KT::TN>(p, q, acc, m0 + wave / WN * KT::WTM, n0 + wave % WN * KT::WTN,
                                                                   lane, (float*)smem + 128 * wave);
    store_tile<KT, false>(p, smem, m0, n0, acc, tid, lane, wave);
}

// ... on the direct-to-LDS ring (16-bit inputs).  NB: adapters at a time in
// lora_add; 0: SharedLora.
template <In TI, Out TO, int BM, int BN, int BK, int WM, int WN, int STAGES, int NB, bool BKM>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_lora_dma_kernel(Params p, Lora q)
{
    constexpr int MI = 16;
    using KT = Dma16<TI, TO, BM, BN, BK, WM, WN, MI, STAGES, true, BKM>;
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm * BM), n0 = __builtin_amdgcn_readfirstlane(tn * BN);
    typename KT::OA oa;
    typename KT::OB ob;
    typename KT::Acc acc;
    KT::zero(acc);
    oa.init(wave, lane, p.lda);
    ob.init(wave, lane, p.ldb);
    KT::mainloop(p, smem, oa, ob, m0, n0, 0, (p.K + BK - 1) / BK, acc, tid, lane, wave);
    bool bad = false;
    if constexpr (NB > 0) {
        bare_barrier();   // no wave reads the ring any more
        lora_add<TI, true, terms_of_v(TI, TO), NB, MI, KT::TM, KT::TN>(p, q, acc, m0 + wave / WN * KT::WTM,
                                                                       n0 + wave % WN * KT::WTN, lane, (float*)smem + 128 * wave);
    } else {
        bad = SharedLora<KT, TI>::add(p, q, smem, acc, m0, n0, tid, lane, wave);
    }
    store_tile<KT, false>(p, smem, m0, n0, acc, tid, lane, wave);
    if constexpr (NB == 0)
        if (bad) SharedLora<KT, TI>::template repair<BKM>(p, q, m0, n0, tid);
}

// ... on the fp32 ring of gemm_f32dma.hpp (VEC = false: 4-byte loads).
template <int BM, int BN, int STAGES, bool BKM, bool VEC>
__global__ void __launch_bounds__(256)
gemm_lora_f32_kernel(Params p, Lora q)
{
    constexpr int BK = 32, WN = 2;
    using KT = F32Dma<Out::F32, BM, BN, BK, 2, WN, STAGES, true, BKM, VEC>;
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm * BM), n0 = __builtin_amdgcn_readfirstlane(tn * BN);
    typename KT::OA oa;
    typename KT::OB ob;
    oa.init(wave, lane, p.lda);
    ob.init(wave, lane, p.ldb);
    typename KT::Acc acc;
    KT::zero(acc);
    KT::mainloop(p, smem, oa, ob, m0, n0, 0, (p.K + BK - 1) / BK, acc, tid, lane, wave);
    const auto col = [&](int j) { return KT::UB::row(j, lane % 32); };
    const int rm0 = m0 + wave / WN * KT::WTM, cn0 = n0 + wave % WN * KT::WTN;
    if (VEC && q.odd_up) lora_add<In::F32, false, 1, 2, 32>(p, q, acc, rm0, cn0, lane, nullptr, 0, 1, col);
    else lora_add<In::F32, VEC, 1, 2, 32>(p, q, acc, rm0, cn0, lane, nullptr, 0, 1, col);
    KT::template store<false, false>(p, m0, n0, acc, lane, wave, smem);
}

// Few rows (a decoding step), on the streaming tile: NL more waves share out
// the rows' adapters, so that the chain of loads they wait for (ids, then
// slots, then the adapters) runs beside the stream.
template <In TI, Out TO, int MT, int NT, int NW, int ST, int NL, bool BKM = true, bool VEC = true>
__global__ void __launch_bounds__((NW + NL) * 64)
gemm_lora_skinny_kernel(Params p, Lora q)
{
    using T = Skinny<TI, MT, NT, NW, ST, BKM, VEC>;
    constexpr int NB = (MT * 16 + NL - 1) / NL > 8 ? 8 : (MT * 16 + NL - 1) / NL;   // adapters at a time
    static_assert((NW + NL) * T::PART * 4 <= T::RING && T::RING + NL * 512 <= 160 * 1024, "sums fit the ring; LDS budget");
    __shared__ __attribute__((aligned(1024))) char smem[T::RING + NL * 512];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // The row tiles of one column tile sit on one XCD, so that its L2 gives
    // them the same rows of B.
    const int rt = p.tiles_m;
    const int chunk = blockIdx.x / (8 * rt), in = blockIdx.x % (8 * rt);
    const int tn = chunk * 8 + in % 8;
    if (tn >= p.tiles_n) return;
    const int m0 = in / 8 * (MT * 16), n0 = tn * (NT * 16);
    typename T::Acc acc;
    T::zero(acc);
    if (wave >= NW)
        lora_add<TI, VEC, terms_of_v(TI, TO), NB, 16, MT, NT>(p, q, acc, m0, n0, lane, (float*)(smem + T::RING) + 128 * (wave - NW),
                                                              wave - NW, NL);
    else
        T::stream(p, smem, m0, n0, acc, lane, wave);
    T::template join<TO, NW + NL>(p, smem, m0, n0, acc, tid, lane, wave);
}

// ... on the ping-pong schedule (16-bit inputs, 256x256 tiles).
template <In TI, Out TO, bool BKM>
__global__ void __launch_bounds__(512)
gemm_lora_pp_kernel(Params p, Lora q)
{
    constexpr int BM = 256, BN = 256, WN = 2, MI = 16;
    using PP = PingPong<TI, TO, BM, BN, 64, 4, WN, MI, true, BKM, false>;
    using KT = typename PP::KT;
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm * BM), n0 = __builtin_amdgcn_readfirstlane(tn * BN);
    typename KT::Acc acc;
    KT::zero(acc);
    PP::mainloop(p, smem, m0, n0, acc, tid, lane, wave);
    const bool bad = SharedLora<KT, TI>::add(p, q, smem, acc, m0, n0, tid, lane, wave);
    store_tile<KT, false>(p, smem, m0, n0, acc, tid, lane, wave);
    if (bad) SharedLora<KT, TI>::template repair<BKM>(p, q, m0, n0, tid);
}

// ------------------------------------------------------------------ launchers

struct LoraCall {
    Params p;
    Lora q;
    bool b_kmajor;
    bool vec;             // A, B and the adapters allow 16-byte loads
    int shrink_rows;      // ShrinkPlan::rows
};

// How v is computed: rows per workgroup, ranges of k (their partial sums add
// up where v is used) and workgroups sharing a row tile's adapters.  From 128
// rows up the 64-row tile; below, the 16-row one, with a workgroup per adapter
// and enough ranges of k, at least 256 long, to fill the chip.
struct ShrinkPlan {
    int rows, splits, z;
};
inline ShrinkPlan shrink_plan(int64_t M, int64_t K, bool tiled, int pitch = 32)
{
    ShrinkPlan s;
    tiled = tiled && M >= 128;
    s.rows = tiled ? 64 : kShrinkRows;
    const int64_t tiles = (M + s.rows - 1) / s.rows;
    int64_t n;
    if (tiled) {
        n = 256 / tiles;
    } else {
        s.z = (int)(tiles >= 64 ? 1 : M < kShrinkRows ? M : kShrinkRows);
        n = 512 / (tiles * s.z);
    }
    if (n > 8) n = 8;
    if (n > K / 256) n = K / 256;
    s.splits = (int)(n < 1 ? 1 : n);
    if (tiled) {
        n = 512 / (tiles * s.splits);
        s.z = (int)(n < 2 ? 2 : n > 16 ? 16 : n);
    } else {
        n = 512 / (tiles * s.splits * s.z);
        const int blocks = (pitch + 31) / 32;
        s.z *= (int)(n < 1 ? 1 : n > blocks ? blocks : n);
    }
    return s;
}

// The 64-row tile is for 16-bit operands that allow 16-byte loads.  (In fp32
// on 32x32 MFMAs it took 110 us against 97 at 256 rows, N = K = 4096, rank 16,
// both kernels together, and 1261 against 1333 at 4096 rows of rank 128.)
inline bool shrink_tiled(int in_bytes, bool vec) { return in_bytes == 2 && vec; }

inline LoraShape shape_of(const LoraCall& c, bool f32) { return {f32, c.vec, c.b_kmajor, c.p.M, c.p.N}; }

template <class Kernel>
hipError_t launch_lora(Kernel kernel, const LoraCall& c, const Tile& t, hipStream_t s)
{
    Params p = c.p;
    Lora q = c.q;
    p.tiles_m = (int)ceil_div(p.M, t.bm);
    p.tiles_n = (int)ceil_div(p.N, t.bn);
    p.group_m = p.tiles_m < 8 ? p.tiles_m : 8;
    void* args[] = {&p, &q};
    return hipLaunchKernel((const void*)kernel, dim3((unsigned)lora_grid(shape_of(c, false), t)), dim3(t.threads), args, 0, s);
}

template <In TI>
hipError_t launch_shrink(const LoraCall& c, hipStream_t s)
{
    Params p = c.p;
    Lora q = c.q;
    void* args[] = {&p, &q};
    const int rows = c.shrink_rows;
    const dim3 grid((unsigned)((p.M + rows - 1) / rows), (unsigned)q.splits, (unsigned)q.z);
    if constexpr (TI != In::F32)
        if (rows == 64) return hipLaunchKernel((const void*)&lora_shrink_dma_kernel<TI>, grid, dim3(kShrinkThreads), args, 0, s);
    const void* kernel = c.vec ? (const void*)&lora_shrink_kernel<TI, true> : (const void*)&lora_shrink_kernel<TI, false>;
    return hipLaunchKernel(kernel, grid, dim3(kShrinkThreads), args, 0, s);
}

template <In TI, Out TO>
struct LoraInst {
    template <LoraTile T, bool BKM, bool VEC>
    static hipError_t stream(const LoraCall& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T);
        return launch_lora(&gemm_lora_skinny_kernel<TI, TO, t.wm, t.wn, t.extra, t.stages, t.threads / 64 - t.extra, BKM, VEC>, c, t, s);
    }
    template <LoraTile T, bool BKM>
    static hipError_t dma(const LoraCall& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T);
        return launch_lora(&gemm_lora_dma_kernel<TI, TO, t.bm, t.bn, t.bk, t.wm, t.wn, t.stages, t.extra, BKM>, c, t, s);
    }
    template <LoraTile T, bool BKM>
    static hipError_t odd(const LoraCall& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T);
        return launch_lora(&gemm_lora_odd_kernel<TI, TO, t.bm, t.bn, t.bk, t.wm, t.wn, t.stages, BKM>, c, t, s);
    }
    template <LoraTile T, bool BKM, bool VEC>
    static hipError_t f32(const LoraCall& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T);
        return launch_lora(&gemm_lora_f32_kernel<t.bm, t.bn, t.stages, BKM, VEC>, c, t, s);
    }
    template <bool BKM, bool VEC>
    static hipError_t product(const LoraCall& c, hipStream_t s)
    {
        const LoraTile t = lora_tile(shape_of(c, TI == In::F32));
        if constexpr (TI == In::F32 || (BKM && VEC)) {
            if (t == LoraTile::Stream16x16) return stream<LoraTile::Stream16x16, BKM, VEC>(c, s);
            if (t == LoraTile::Stream16x32) return stream<LoraTile::Stream16x32, BKM, VEC>(c, s);
        }
        if constexpr (TI == In::F32) {
            if (t == LoraTile::Stream32x32) return stream<LoraTile::Stream32x32, BKM, VEC>(c, s);
            if constexpr (VEC) {
                if (t == LoraTile::F32Rows64x128) return f32<LoraTile::F32Rows64x128, BKM, true>(c, s);
                return f32<LoraTile::F32Rows64x64, BKM, true>(c, s);
            } else {
                return f32<LoraTile::F32Odd64x64, BKM, false>(c, s);
            }
        } else if constexpr (!VEC) {
            switch (t) {
            case LoraTile::Odd32x32: return odd<LoraTile::Odd32x32, BKM>(c, s);
            case LoraTile::Odd64x64: return odd<LoraTile::Odd64x64, BKM>(c, s);
            case LoraTile::Odd128x128: return odd<LoraTile::Odd128x128, BKM>(c, s);
            case LoraTile::Odd256x128: return odd<LoraTile::Odd256x128, BKM>(c, s);
            default: return hipErrorInvalidValue;
            }
        } else {
            if constexpr (!BKM)
                if (t == LoraTile::Few16x32) return dma<LoraTile::Few16x32, BKM>(c, s);
            switch (t) {
            case LoraTile::Few32x32: return dma<LoraTile::Few32x32, BKM>(c, s);
            case LoraTile::Shared32x32: return dma<LoraTile::Shared32x32, BKM>(c, s);
            case LoraTile::Shared64x64: return dma<LoraTile::Shared64x64, BKM>(c, s);
            case LoraTile::Shared64x64Four: return dma<LoraTile::Shared64x64Four, BKM>(c, s);
            case LoraTile::Shared128x128: return dma<LoraTile::Shared128x128, BKM>(c, s);
            case LoraTile::PingPong: return launch_lora(&gemm_lora_pp_kernel<TI, TO, BKM>, c, tile_of(LoraTile::PingPong), s);
            default: return hipErrorInvalidValue;
            }
        }
    }
    static hipError_t launch(const LoraCall& c, hipStream_t s)
    {
        if (c.q.slots > 0 && c.q.R > 0) {
            const hipError_t e = launch_shrink<TI>(c, s);
            if (e != hipSuccess) return e;
        }
        if (c.vec) return c.b_kmajor ? product<true, true>(c, s) : product<false, true>(c, s);
        return c.b_kmajor ? product<true, false>(c, s) : product<false, false>(c, s);
    }
};

hipError_t lora_f32(const LoraCall& c, hipStream_t s);
hipError_t lora_f16_f32(const LoraCall& c, hipStream_t s);
hipError_t lora_bf16_bf16(const LoraCall& c, hipStream_t s);
hipError_t lora_f16_f16(const LoraCall& c, hipStream_t s);
hipError_t lora_bf16_f32(const LoraCall& c, hipStream_t s);

}  // namespace mg
