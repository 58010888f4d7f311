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
};

// R rounded up to whole MFMA steps of any input type.
constexpr int kRankStep = 32;
// Rows of v one workgroup computes.
constexpr int kShrinkRows = 16;

__device__ __forceinline__ int lora_rank(const Lora& q, int a)
{
    return q.ranks ? min(max(q.ranks[a], 0), q.R) : q.R;
}

// The distinct adapters of up to 64 rows, one lane each: `next` gives an
// adapter and the rows (bits) that have it.
struct Distinct {
    int id;               // this lane's row's adapter, or -1
    uint64_t left;

    __device__ __forceinline__ Distinct(const Lora& q, int row, bool valid)
    {
        id = valid ? q.ids[row] : -1;
        if (id >= q.slots) id = -1;
        left = __builtin_amdgcn_ballot_w64(id >= 0);
    }
    __device__ __forceinline__ int next(uint64_t& rows)
    {
        if (!left) { rows = 0; return -1; }
        const int a = __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(left));
        rows = __builtin_amdgcn_ballot_w64(id == a);
        left &= ~rows;
        return a;
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
    constexpr int RJ = 4;                                                  // 16-column blocks at a time
    __shared__ float part[4][kShrinkRows][RJ * 16 + 4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m0 = blockIdx.x * kShrinkRows;
    const int split = blockIdx.y;
    const int steps = (p.K + KS - 1) / KS;
    const int s0 = (int)((int64_t)steps * split / q.splits), s1 = (int)((int64_t)steps * (split + 1) / q.splits);
    Distinct d(q, m0 + lane, lane < kShrinkRows && m0 + lane < p.M);
    const __amdgpu_buffer_rsrc_t ra =
        make_rsrc(p.A + (int64_t)m0 * p.lda * ES, rows_extent(min(p.M - m0, kShrinkRows), p.lda * ES, row_tail<ES, VEC>(p.K)));
    const int aoff = (int)((lane % 16) * p.lda * ES);
    float* const out = q.v + ((int64_t)split * p.M + m0) * q.pitch;
    for (int u = 0;; ++u) {
        uint64_t rows;
        const int a = d.next(rows);
        if (a < 0) break;
        if (u % q.z != (int)blockIdx.z) continue;
        const int rank = lora_rank(q, a);
        for (int r0 = 0; r0 < q.pitch; r0 += RJ * 16) {
            f32x4 acc[RJ];
#pragma unroll
            for (int j = 0; j < RJ; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
            const int left = max(0, min(rank - r0, RJ * 16));
            const __amdgpu_buffer_rsrc_t rd = make_rsrc(q.down + a * q.s_down + (int64_t)r0 * q.ld_down * ES,
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
                        fa[t] = load_chunk<ES, VEC>(ra, in ? aoff + k * ES : -16);       // past the extent: zeros
#pragma unroll
                        for (int j = 0; j < n; ++j)
                            fd[t][j] = load_chunk<ES, VEC>(rd, in ? doff + (int)(16 * j * q.ld_down * ES) + k * ES : -16);
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
            else if (nj == 2) body(std::integral_constant<int, 2>{});
            else if (nj > 0) body(std::integral_constant<int, RJ>{});
            __syncthreads();                           // the sums of the last adapter have been read
#pragma unroll
            for (int j = 0; j < RJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[wave][(lane / 16) * 4 + e][j * 16 + lane % 16] = acc[j][e];
            __syncthreads();
            for (int x = tid; x < kShrinkRows * RJ * 16; x += 256) {
                const int m = x / (RJ * 16), r = x % (RJ * 16);
                if (!(rows >> m & 1) || r0 + r >= q.pitch) continue;
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
// 64, where this form takes SHRINK_US).
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
        uint64_t rows;
        const int a = d.next(rows);
        if (a < 0) break;
        if (u % q.z != (int)blockIdx.z) continue;
        const int rank = lora_rank(q, a);
        for (int r0 = 0; r0 < q.pitch; r0 += 64) {
            const int left = max(0, min(rank - r0, 64));
            p.B = q.down + a * q.s_down + (int64_t)r0 * q.ld_down * 2;
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
                        if ((rows >> m & 1) && r0 + r < q.pitch) out[(int64_t)m * q.pitch + r0 + r] = r < left ? acc[i][j][e] : 0.f;
                    }
        }
    }
}

// 8 (16-bit) or 4 (fp32) values of v as MFMA fragments.  v is fp32 and the
// adapters are 16-bit, so v is split into the part that the type holds and
// the type's rounding of the rest, one MFMA each: fp16 keeps 22 bits, bf16 16
// (truncated, so that the first part cannot round up to an infinity).
template <In TI>
struct VFrag {
    static constexpr int N = TI == In::F32 ? 1 : 2;
    i32x4 f[N];

    __device__ __forceinline__ void set(const float (&v)[TI == In::F32 ? 4 : 8])
    {
        if constexpr (TI == In::F32) {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[0][e] = __float_as_int(v[e]);
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                uint32_t hi = 0, lo = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float x = v[2 * d + h];
                    const bool inf = __builtin_fabsf(x) == __builtin_inff();   // then the rest is inf - inf
                    uint32_t a, b;
                    if constexpr (TI == In::BF16) {
                        a = (uint32_t)__float_as_int(x) >> 16;
                        if (x != x) a |= 0x40;                                  // a NaN must stay one
                        const float rest = x - __int_as_float((int)(a << 16));
                        b = __builtin_bit_cast(uint16_t, (__bf16)(inf ? 0.f : rest));
                    } else {
                        const _Float16 t = (_Float16)x;
                        a = __builtin_bit_cast(uint16_t, t);
                        b = __builtin_bit_cast(uint16_t, (_Float16)(inf ? 0.f : x - (float)t));
                    }
                    hi |= a << (16 * h);
                    lo |= b << (16 * h);
                }
                f[0][d] = (int)hi;
                f[1][d] = (int)lo;
            }
        }
    }
};

// Add scale_i v up_i^T to the accumulators of one wave.  Its rows are m0 ..
// m0 + TM * MI - 1 (at most 64), its columns start at n0; MFMA tile (i, j)
// holds rows i * MI and columns j * MI on.  NB: adapters whose loads are
// in flight together.
template <In TI, bool VEC, int NB, int MI, int TM, int TN, class AccT>
__device__ __forceinline__ void lora_add(const Params& p, const Lora& q, AccT (&acc)[TM][TN], int m0, int n0, int lane,
                                         float* tab = nullptr)
{
    constexpr int ES = TI == In::F32 ? 4 : 2, CE = 16 / ES, KS = 64 / MI * CE, R4 = MI == 32 ? 16 : 4;
    constexpr bool BIG = TM * TN * R4 >= 128;          // accumulators that leave few registers
    constexpr int CH = TI == In::F32 || BIG ? 32 : 64;   // columns of v held at a time
    constexpr int NK = CH / KS;
    static_assert(TM * MI <= 64, "one lane per row");
    if (q.slots == 0 || q.R == 0) return;
    Distinct d(q, m0 + lane, lane < TM * MI && m0 + lane < p.M);
    if (!d.left) return;
    const uint64_t all = d.left;
    const int fr = lane % MI, fk = lane / MI * CE;     // fragment row, first k
    const int up_row = (int)(q.ld_up * ES);            // (256 rows fit 32 bits)
    const int64_t vsplit = (int64_t)p.M * q.pitch * 4;
    auto load_v = [&](int i, int r, float (&v)[CE]) {
#pragma unroll
        for (int e = 0; e < CE; ++e) v[e] = 0.f;
        const int off = r + fk < q.pitch ? ((i * MI + fr) * q.pitch + r + fk) * 4 : -16;
        for (int s = 0; s < q.splits; ++s) {
            const __amdgpu_buffer_rsrc_t rs = make_rsrc((const char*)(q.v + (int64_t)m0 * q.pitch) + s * vsplit,
                                                        (uint64_t)min(p.M - m0, TM * MI) * q.pitch * 4);
#pragma unroll
            for (int e = 0; e < CE; e += 4) {
                const i32x4 t = buf_load16(rs, off + e * 4);
#pragma unroll
                for (int x = 0; x < 4; ++x) v[e + x] += __int_as_float(t[x]);
            }
        }
    };
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
    for (int r0 = 0; r0 < q.pitch; r0 += CH) {
        VFrag<TI> fv[TM][NK];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                if constexpr (BIG) __builtin_amdgcn_sched_barrier(0);
                float v[CE];
                load_v(i, r0 + k * KS, v);
                if constexpr (TI == In::F16) {
                    const float up = tab[64 + i * MI + fr];
#pragma unroll
                    for (int e = 0; e < CE; ++e) v[e] *= up;
                }
                fv[i][k].set(v);
            }
        d.left = all;
        while (d.left) {
            uint64_t rows[NB];
            int rank[NB];
            float scale[NB];
            __amdgpu_buffer_rsrc_t ru[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int a = d.next(rows[b]);
                rank[b] = a < 0 ? 0 : lora_rank(q, a);
                scale[b] = a < 0 ? 0.f : q.scales ? q.scales[a] : 1.f;
                ru[b] = make_rsrc(q.up + max(a, 0) * q.s_up + (int64_t)n0 * q.ld_up * ES,
                                  a < 0 || n0 >= p.N ? 0 : rows_extent(min(p.N - n0, TN * MI), q.ld_up * ES, row_tail<ES, VEC>(q.R)));
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                if constexpr (BIG) __builtin_amdgcn_sched_barrier(0);
                i32x4 fu[NB][NK];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int k = 0; k < NK; ++k) {
                        const int r = r0 + k * KS + fk;
                        fu[b][k] = load_chunk<ES, VEC>(ru[b], r < rank[b] ? fr * up_row + r * ES + j * MI * up_row : -16);
                    }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if (r0 >= rank[b]) continue;
#pragma unroll
                    for (int k = 0; k < NK; ++k) {
                        const int r = r0 + k * KS + fk;
                        if (r + CE > rank[b]) fu[b][k] = mask_k<TI>(fu[b][k], r, rank[b]);
                    }
#pragma unroll
                    for (int i = 0; i < TM; ++i) {
                        AccT t = {};
#pragma unroll
                        for (int k = 0; k < NK; ++k) {
                            if (r0 + k * KS >= rank[b]) continue;
#pragma unroll
                            for (int h = 0; h < VFrag<TI>::N; ++h) mfma_step<TI, MI>(fv[i][k].f[h], fu[b][k], t);
                        }
#pragma unroll
                        for (int x4 = 0; x4 < R4; x4 += 4) {
                            const int row4 = i * MI + (MI == 32 ? x4 / 4 * 8 + (lane / 32) * 4 : (lane / 16) * 4);
                            f32x4 f = {scale[b], scale[b], scale[b], scale[b]};
                            if constexpr (TI == In::F16) {
                                const f32x4 down = *(const f32x4*)(tab + row4);
#pragma unroll
                                for (int x = 0; x < 4; ++x) f[x] *= down[x];
                            }
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const float y = __builtin_fmaf(f[x], t[x4 + x], acc[i][j][x4 + x]);
                                acc[i][j][x4 + x] = rows[b] >> (row4 + x) & 1 ? y : acc[i][j][x4 + x];
                            }
                        }
                    }
                }
            }
        }
    }
}

// The shared product on the register-staged tile: any type and alignment.
template <In TI, Out TO, int BM, int BN, int BK, int WM, int WN, bool BKM, bool VEC>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_lora_kernel(Params p, Lora q)
{
    constexpr int MI = 16;
    using T = GemmTile<TI, TO, BM, BN, BK, WM, WN, MI, true, BKM, true, VEC>;
    __shared__ __attribute__((aligned(16))) char smem[2 * T::STAGE];
    T t;
    t.tid = threadIdx.x;
    const int lane = t.tid & 63, wave = __builtin_amdgcn_readfirstlane(t.tid >> 6);
    t.wm = wave / WN;
    t.wn = wave % WN;
    t.frow = lane % MI;
    t.fq = lane / MI;
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    t.la.init(t.tid, p.lda);
    t.lb.init(t.tid, p.ldb);
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j) t.acc[i][j] = typename T::Acc{};
    staged_mainloop<T, BK>(t, smem, p, m0, n0);
    __syncthreads();      // no wave reads the tiles any more
    lora_add<TI, VEC, 1, MI, T::TM, T::TN>(p, q, t.acc, m0 + t.wm * T::WTM, n0 + t.wn * T::WTN, lane,
                                           (float*)smem + 128 * wave);
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int m = m0 + t.wm * T::WTM + i * MI + (lane / 16) * 4 + e;
                const int n = n0 + t.wn * T::WTN + j * MI + lane % 16;
                if (m < p.M && n < p.N) store_out<TO>(p.C, (int64_t)m * p.ldc + n, t.acc[i][j][e]);
            }
}

// ... on the direct-to-LDS ring (16-bit inputs).
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
    bare_barrier();       // no wave reads the ring any more
    lora_add<TI, true, NB, MI, KT::TM, KT::TN>(p, q, acc, m0 + wave / WN * KT::WTM, n0 + wave % WN * KT::WTN, lane,
                                               (float*)smem + 128 * wave);
    store_tile<KT, false>(p, smem, m0, n0, acc, tid, lane, wave);
}

// ... on the ping-pong schedule (16-bit inputs, 256x256 tiles).
template <In TI, Out TO, bool BKM>
__global__ void __launch_bounds__(512)
gemm_lora_pp_kernel(Params p, Lora q)
{
    constexpr int BM = 256, BN = 256, WN = 2, MI = 16;
    using PP = PingPong<TI, TO, BM, BN, 64, 4, WN, MI, true, BKM>;
    using KT = typename PP::KT;
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm * BM), n0 = __builtin_amdgcn_readfirstlane(tn * BN);
    typename KT::Acc acc;
    KT::zero(acc);
    PP::mainloop(p, smem, m0, n0, acc, tid, lane, wave);
    bare_barrier();       // no wave reads the ring any more
    lora_add<TI, true, 1, MI, KT::TM, KT::TN>(p, q, acc, m0 + wave / WN * KT::WTM, n0 + wave % WN * KT::WTN, lane,
                                               (float*)smem + 128 * wave);
    store_tile<KT, false>(p, smem, m0, n0, acc, tid, lane, wave);
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
inline ShrinkPlan shrink_plan(int64_t M, int64_t K, bool tiled)
{
    ShrinkPlan s;
    tiled = tiled && M >= 128;
    s.rows = tiled ? 64 : kShrinkRows;
    const int64_t tiles = (M + s.rows - 1) / s.rows;
    int64_t n;
    if (tiled) {
        s.z = 2;
        n = 256 / tiles;
    } else {
        s.z = (int)(tiles >= 64 ? 1 : M < kShrinkRows ? M : kShrinkRows);
        n = 512 / (tiles * s.z);
    }
    if (n > 8) n = 8;
    if (n > K / 256) n = K / 256;
    s.splits = (int)(n < 1 ? 1 : n);
    return s;
}
// The 64-row tile is for 16-bit operands that allow 16-byte loads.
inline bool shrink_tiled(int in_bytes, bool vec) { return in_bytes == 2 && vec; }

template <class Kernel>
hipError_t launch_lora(Kernel kernel, const LoraCall& c, int BM, int BN, int threads, hipStream_t s)
{
    Params p = c.p;
    Lora q = c.q;
    p.tiles_m = (p.M + BM - 1) / BM;
    p.tiles_n = (p.N + BN - 1) / BN;
    p.group_m = p.tiles_m < 8 ? p.tiles_m : 8;
    void* args[] = {&p, &q};
    return hipLaunchKernel((const void*)kernel, dim3((unsigned)((int64_t)p.tiles_m * p.tiles_n)), dim3(threads), args, 0, s);
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
        if (rows == 64) return hipLaunchKernel((const void*)&lora_shrink_dma_kernel<TI>, grid, dim3(256), args, 0, s);
    const void* kernel = c.vec ? (const void*)&lora_shrink_kernel<TI, true> : (const void*)&lora_shrink_kernel<TI, false>;
    return hipLaunchKernel(kernel, grid, dim3(256), args, 0, s);
}

template <In TI, Out TO>
struct LoraInst {
    template <bool BKM, bool VEC>
    static hipError_t staged(const LoraCall& c, hipStream_t s)
    {
        return launch_lora(&gemm_lora_kernel<TI, TO, 64, 64, TI == In::F32 ? 32 : 64, 2, 2, BKM, VEC>, c, 64, 64, 256, s);
    }
    template <int BM, int BN, int BK, int WM, int WN, int ST, int NB, bool BKM>
    static hipError_t dma(const LoraCall& c, hipStream_t s)
    {
        return launch_lora(&gemm_lora_dma_kernel<TI, TO, BM, BN, BK, WM, WN, ST, NB, BKM>, c, BM, BN, WM * WN * 64, s);
    }
    template <bool BKM>
    static hipError_t product(const LoraCall& c, hipStream_t s)
    {
        if (!c.vec) return staged<BKM, false>(c, s);
        if constexpr (TI == In::F32) {
            return staged<BKM, true>(c, s);
        } else {
            auto tiles = [&](int t) { return ((int64_t)c.p.M + t - 1) / t * ((c.p.N + t - 1) / t); };
            if (c.p.M <= 32) return dma<16, 32, 256, 1, 2, 4, 4, BKM>(c, s);
            if (c.p.M <= 96) return dma<32, 32, 128, 2, 2, 4, 4, BKM>(c, s);
            if (tiles(256) >= 100) return launch_lora(&gemm_lora_pp_kernel<TI, TO, BKM>, c, 256, 256, 512, s);
            if (tiles(128) >= 96) return dma<128, 128, 64, 2, 2, 4, 1, BKM>(c, s);
            return dma<64, 64, 64, 2, 2, 4, 1, BKM>(c, s);
        }
    }
    static hipError_t launch(const LoraCall& c, hipStream_t s)
    {
        if (c.q.slots > 0 && c.q.R > 0) {
            const hipError_t e = launch_shrink<TI>(c, s);
            if (e != hipSuccess) return e;
        }
        return c.b_kmajor ? product<true>(c, s) : product<false>(c, s);
    }
};

hipError_t lora_f32(const LoraCall& c, hipStream_t s);
hipError_t lora_f16_f32(const LoraCall& c, hipStream_t s);
hipError_t lora_bf16_bf16(const LoraCall& c, hipStream_t s);
hipError_t lora_f16_f16(const LoraCall& c, hipStream_t s);
hipError_t lora_bf16_f32(const LoraCall& c, hipStream_t s);

}  // namespace mg
