// gemm_ragged.hpp -- grouped products with ragged sizes (gfx950).
//
//   by rows:  C[m][n] = sum_k A[m][k] B_g[n][k]      for the rows m of group g
//   by k:     C_g[m][n] = sum_{k in group g} A[m][k] B[n][k]
//
// The groups are consecutive ranges of the rows (or of k) whose ends the GPU
// holds, so the host never learns them: the grid covers the most tiles that
// any ends could need, and every workgroup finds its own group and tile.
//
// What the ends may hold: group g covers [s_g, e_g), e_g = max over h <= g of
// ends[h] clamped to [0, rows], s_g = e_{g-1} (0 for the first).  For
// ascending ends that is [ends[g-1], ends[g]); any other content gives groups
// that still do not overlap and stay inside A, B and C.
#pragma once

#include "gemm_f32dma.hpp"
#include "gemm_tiles.hpp"

namespace mg {

struct Ragged {
    const int* ends;      // device, one per group
    int groups;
    int rows;             // rows of A and C (by rows), or the k of A and B (by k)
    int64_t stride;       // bytes between B_g's (by rows) or C_g's (by k)
};

// Inclusive scans over the 64 lanes of a wave.
__device__ __forceinline__ int wave_scan_max(int v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v = max(v, u);
    }
    return v;
}
__device__ __forceinline__ int wave_scan_add(int v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v += u;
    }
    return v;
}

__device__ __forceinline__ int group_end(const Ragged& r, int g)
{
    return g < r.groups ? min(max(r.ends[g], 0), r.rows) : 0;
}

// By rows: the workgroup's group g with its rows [start, start + len), and its
// tile L of that group's ceil(len / bm) * tiles_n.  False when the grid's
// upper bound has more workgroups than there are tiles.  Every wave does the
// same search: 64 groups at a time, one lane each, a running maximum for the
// starts and a running sum for the tiles.  The tiles of all groups form one
// list, which the XCDs share out in contiguous ranges (as in tile_coords), so
// that an L2 sees few groups' matrices.
__device__ __forceinline__ bool find_row_group(const Ragged& r, int bm, int tiles_n, int lane, int& g, int& start,
                                               int& len, int& L)
{
    int total = 0, prev = 0, st = 0, ln = 0, inc = 0;
    for (int g0 = 0; g0 < r.groups; g0 += 64) {
        const int m = max(wave_scan_max(group_end(r, g0 + lane), lane), prev);
        st = __shfl_up(m, 1);
        if (lane == 0) st = prev;
        ln = m - st;
        inc = wave_scan_add((ln + bm - 1) / bm * tiles_n, lane);
        prev = __builtin_amdgcn_readlane(m, 63);
        total += __builtin_amdgcn_readlane(inc, 63);
    }
    const int w = blockIdx.x;
    if (w >= total) return false;
    const int per = total / 8, rem = total % 8, x = w % 8;
    int t = x * per + (x < rem ? x : rem) + w / 8;
    int g0 = 0;
    if (r.groups > 64) {      // the search proper: the 64 groups that hold tile t
        prev = 0;
        for (;; g0 += 64) {
            const int m = max(wave_scan_max(group_end(r, g0 + lane), lane), prev);
            st = __shfl_up(m, 1);
            if (lane == 0) st = prev;
            ln = m - st;
            inc = wave_scan_add((ln + bm - 1) / bm * tiles_n, lane);
            prev = __builtin_amdgcn_readlane(m, 63);
            const int here = __builtin_amdgcn_readlane(inc, 63);
            if (t < here || g0 + 64 >= r.groups) break;
            t -= here;
        }
    }
    const int l = (int)__builtin_ctzll(__builtin_amdgcn_ballot_w64(inc > t));   // first lane past t
    g = g0 + l;
    start = __builtin_amdgcn_readlane(st, l);
    len = __builtin_amdgcn_readlane(ln, l);
    L = t - (l ? __builtin_amdgcn_readlane(inc, l - 1) : 0);
    return true;
}

// By k: the k-range [start, start + len) of group g.
__device__ __forceinline__ void k_group(const Ragged& r, int g, int lane, int& start, int& len)
{
    int s = 0;
    for (int h = lane; h < g; h += 64) s = max(s, group_end(r, h));
#pragma unroll
    for (int d = 32; d >= 1; d /= 2) s = max(s, __shfl_xor(s, d));
    start = __builtin_amdgcn_readfirstlane(s);
    len = max(__builtin_amdgcn_readfirstlane(group_end(r, g)) - start, 0);
}

// Bytes from an operand's first row to the end of its last one's readable
// part: `tail` is that part (inner extent, rounded up to 16 bytes where the
// loads are 16 bytes wide).
__device__ __forceinline__ uint64_t rows_extent(int rows, int64_t ld_bytes, int64_t tail)
{
    return rows > 0 ? (uint64_t)(rows - 1) * (uint64_t)ld_bytes + (uint64_t)tail : 0;
}

template <int ES, bool VEC>
__device__ __forceinline__ int64_t row_tail(int inner)
{
    return VEC ? ((int64_t)inner * ES + 15) / 16 * 16 : (int64_t)inner * ES;
}

// Which index of the canonical product C = A * B^T the groups divide.
//  Rows: the rows of A and C; each group has a matrix of its own in B.
//  K:    the summed index; each group has a C of its own.
enum class By : int { Rows = 0, K = 1 };

// Point p at the workgroup's group; false: no tile for this workgroup.
// By rows p.M becomes the group's rows, A and C start at its first row, B at
// its matrix.  By k p.K is the
// group's k-range, A and B (both with k as the outer index) start at its first
// k, C at the group's matrix; a group without any k writes zeros, or nothing
// where C is added to.
// tm, tn: the tile within the group.
template <In TI, Out TO, int BM, int BN, By BY, bool VEC>
__device__ __forceinline__ bool select_group(Params& p, const Ragged& r, int lane, int& tm, int& tn)
{
    constexpr int ES = TI == In::F32 ? 4 : 2, EO = TO == Out::F32 ? 4 : 2;
    int g, start, len;
    if constexpr (BY == By::Rows) {
        int L;
        p.tiles_n = (p.N + BN - 1) / BN;
        if (!find_row_group(r, BM, p.tiles_n, lane, g, start, len, L)) return false;
        p.tiles_m = (len + BM - 1) / BM;
        p.group_m = min(8, p.tiles_m);
        raster(p, L, tm, tn);
        p.M = len;
        p.A += (int64_t)start * p.lda * ES;
        p.C += (int64_t)start * p.ldc * EO;
        p.B += (int64_t)g * r.stride;
        p.a_bytes = p.K > 0 ? rows_extent(len, p.lda * ES, row_tail<ES, VEC>(p.K)) : 0;
    } else {
        g = blockIdx.y;
        tile_coords(p, tm, tn);
        k_group(r, g, lane, start, len);
        if (len == 0 && p.epi) return false;
        p.K = len;
        p.A += (int64_t)start * p.lda * ES;
        p.B += (int64_t)start * p.ldb * ES;
        p.C += (int64_t)g * r.stride;
        p.a_bytes = rows_extent(len, p.lda * ES, row_tail<ES, VEC>(p.M));
        p.b_bytes = rows_extent(len, p.ldb * ES, row_tail<ES, VEC>(p.N));
    }
    // Wave-uniform, but divisions run on the vector unit: back into scalar
    // registers, which the main loop's addresses are made of.
    tm = __builtin_amdgcn_readfirstlane(tm);
    tn = __builtin_amdgcn_readfirstlane(tn);
    return true;
}

// ------------------------------------------------------- direct-to-LDS kernels

// Rows of C from LDS, where a wave has put KT::RPP of them, to memory in
// 16-byte chunks.  The stores are non-temporal: nothing here reads C again, and
// what the caches would keep of it is room for the operands (256x256 tiles, us,
// with plain stores in brackets: 8192 k in 16 and 32 groups of 4096 x 2048 into
// fp32 188 (211) and 284 (323), into bf16 in 32 groups 201 (245); 8192 rows in
// 16 groups, 4096 x 2048, 144 (151)).
template <class KT>
__device__ __forceinline__ void copy_rows(const Params& p, const char* w, int m0, int n0, int lane)
{
    constexpr int EO = KT::OBY, EPC = 16 / EO, RPI = 64 / KT::SCPR;
    if (!p.c_vec) {               // rows that start at any element: one element a lane (4095 for 4096: 156 us)
        using E = std::conditional_t<EO == 4, int, uint16_t>;
        constexpr int AT = 64 / KT::WTN > 0 ? 64 / KT::WTN : 1, STEP = KT::WTN < 64 ? KT::WTN : 64;
        static_assert(STEP * AT == 64 && KT::RPP % AT == 0 && KT::WTN % STEP == 0, "64 elements at a time");
        const int r1 = lane / STEP, c1 = lane % STEP;
        E* const dst = (E*)p.C + (int64_t)(m0 + r1) * p.ldc + n0 + c1;
#pragma unroll 8
        for (int r0 = 0; r0 < KT::RPP; r0 += AT)
#pragma unroll
            for (int c0 = 0; c0 < KT::WTN; c0 += STEP) {
                const E v = ((const E*)(w + (r0 + r1) * KT::SPITCH))[c0 + c1];
                if (m0 + r0 + r1 < p.M && n0 + c0 + c1 < p.N) __builtin_nontemporal_store(v, dst + (int64_t)r0 * p.ldc + c0);
            }
        return;
    }
#pragma unroll
    for (int r0 = 0; r0 < KT::RPP; r0 += RPI) {
        const int r = r0 + lane / KT::SCPR, ch = lane % KT::SCPR;
        const i32x4 v = *(const i32x4*)(w + r * KT::SPITCH + ch * 16);
        const int m = m0 + r, n = n0 + ch * EPC;
        if (m >= p.M) continue;
        char* dst = p.C + ((int64_t)m * p.ldc + n) * EO;
        if (n + EPC <= p.N) {
            __builtin_nontemporal_store(v, (i32x4*)dst);
        } else {
#pragma unroll
            for (int e = 0; e < EPC; ++e)
                if (n + e < p.N) {
                    if constexpr (EO == 4) ((int*)dst)[e] = v[e];
                    else ((uint16_t*)dst)[e] = (uint16_t)((uint32_t)v[e / 2] >> (16 * (e % 2)));
                }
        }
    }
}

// Store a tile held by a Dma16 engine: through the elementwise epilogue (EPI),
// as whole rows through LDS, or element by element.
template <class KT, bool EPI>
__device__ __forceinline__ void store_tile(const Params& p, char* smem, int m0, int n0, const typename KT::Acc& acc,
                                           int tid, int lane, int wave)
{
    if constexpr (EPI) {
        KT::store_staged(p, smem, m0, n0, acc, tid, lane, wave);
    } else {
        if (KT::ROWS_OK && p.c_vec) {
            if constexpr (KT::ROWS_OK) {
                bare_barrier();   // every wave's loads have landed and its ring reads are done
                constexpr int WN = KT::TILE_N / KT::WTN, MI = KT::WTM / KT::TM;
                char* const w = smem + wave * KT::SHARE;
#pragma unroll
                for (int pass = 0; pass < KT::WTM / KT::RPP; ++pass) {
#pragma unroll
                    for (int i = pass * KT::RPP / MI; i < (pass + 1) * KT::RPP / MI; ++i)
#pragma unroll
                        for (int j = 0; j < KT::TN; ++j)
#pragma unroll
                            for (int q = 0; q < KT::R; ++q)
                                store_out<KT::OUT>(w + (KT::row(0, i, q, lane) - pass * KT::RPP) * KT::SPITCH,
                                                   KT::col(0, j, lane), acc[i][j][q]);
                    copy_rows<KT>(p, w, m0 + wave / WN * KT::WTM + pass * KT::RPP, n0 + wave % WN * KT::WTN, lane);
                }
            }
        } else {
            KT::store_direct(p, m0, n0, acc, lane, wave);
        }
    }
}

// 16-bit operands whose rows start at any element.  A 16-byte chunk of one is
// the 20 bytes from the 4-byte word that holds its first element, shifted into
// place: two loads that are aligned as the hardware wants them, where loads
// element by element are eight.  The words at either end may hold a neighbour's
// element: they are words that the operand's own elements share, so nothing
// outside its memory is touched, and what lies past an inner extent is masked
// by whoever uses it.
struct OddRows {
    __amdgpu_buffer_rsrc_t r;
    int lead;             // bytes from the first word to the first element: 0 or 2

    OddRows() = default;
    __device__ __forceinline__ OddRows(const char* base, uint64_t bytes)
        : r(make_rsrc(base - ((uint64_t)base & 2), bytes ? (bytes + ((uint64_t)base & 2) + 3) / 4 * 4 : 0)),
          lead((int)((uint64_t)base & 2))
    {
    }
};
struct OddChunk {
    i32x4 words;
    int last;
    // The chunk at `off` bytes from the rows' base (multiple of 2; far below 0: zeros).
    __device__ __forceinline__ void load(const OddRows& s, int off)
    {
        const int at = (off + s.lead) & ~3;
        words = buf_load16(s.r, at);
        last = __builtin_amdgcn_raw_buffer_load_b32(s.r, at + 16, 0, 0);
    }
    __device__ __forceinline__ i32x4 get(int lead, int off) const
    {
        const uint32_t sh = ((uint32_t)(off + lead) & 2) * 8;
        i32x4 v;
#pragma unroll
        for (int d = 0; d < 4; ++d)
            v[d] = (int)__builtin_amdgcn_alignbit((uint32_t)(d < 3 ? words[d + 1] : last), (uint32_t)words[d], sh);
        return v;
    }
};

// One such operand's k-tiles, from memory to registers (DEPTH tiles ahead) to
// the LDS layout of DmaOperand.
template <int ROWS, int BK, int NW, bool KMAJ, int DEPTH>
struct OddOperand {
    using LDS = DmaOperand<ROWS, BK, NW, KMAJ, 16>;
    LDS at;
    OddChunk q[DEPTH][LDS::IPW];

    __device__ __forceinline__ void load(int d, const char* base, uint64_t bytes, int64_t ld, int row0, int k0)
    {
        const int64_t origin = (KMAJ ? (int64_t)row0 * ld + k0 : (int64_t)k0 * ld + row0) * 2;
        const OddRows s(base + origin, (uint64_t)origin < bytes ? bytes - (uint64_t)origin : 0);
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) q[d][j].load(s, at.voff[j]);
    }
    // ... of the tile at k0; elements from K on as zeros.  (row0 * ld and k0
    // are even, so every tile's first element lies in its word as the base's.)
    __device__ __forceinline__ void store(int d, char* tile, const char* base, int k0, int K, int wave, int lane) const
    {
#pragma unroll
        for (int j = 0; j < LDS::IPW; ++j) {
            const int slot = (wave * LDS::IPW + j) * 64 + lane;
            i32x4 v = q[d][j].get((int)((uint64_t)base & 2), at.voff[j]);
            if (k0 + BK > K) {
                if constexpr (KMAJ) {
                    v = mask_k<In::F16>(v, k0 + swz_chunk<LDS::CPR, true>(slot / LDS::CPR, slot % LDS::CPR) * 8, K);
                } else {
                    const i32x4 zero = {0, 0, 0, 0};
                    v = k0 + slot / LDS::RCH < K ? v : zero;
                }
            }
            *(i32x4*)(tile + slot * 16) = v;
        }
    }
};

// A tile of such operands: LDS in two stages, DEPTH tiles of loads in flight.
template <In TI, Out TO, int BM, int BN, int BK, int WM, int WN, int DEPTH, bool AK, bool BKM>
struct OddTile {
    using KT = Dma16<TI, TO, BM, BN, BK, WM, WN, 16, 2, AK, BKM>;
    static_assert(DEPTH % 2 == 0, "a tile's stage is known at compile time");
    // Adds all of p.K to acc.
    __device__ static __forceinline__ void mainloop(const Params& p, char* smem, int m0, int n0, typename KT::Acc& acc,
                                                    int lane, int wave)
    {
        const int wm = wave / WN, wn = wave % WN, nkt = (p.K + BK - 1) / BK;
        OddOperand<BM, BK, KT::NW, AK, DEPTH> oa;
        OddOperand<BN, BK, KT::NW, BKM, DEPTH> ob;
        oa.at.init(wave, lane, p.lda);
        ob.at.init(wave, lane, p.ldb);
        auto load = [&](int t, int d) {               // past the end: empty extents
            oa.load(d, p.A, t < nkt ? p.a_bytes : 0, p.lda, m0, t * BK);
            ob.load(d, p.B, t < nkt ? p.b_bytes : 0, p.ldb, n0, t * BK);
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
                oa.store(d, sa, p.A, t * BK, p.K, wave, lane);
                ob.store(d, sb, p.B, t * BK, p.K, wave, lane);
                load(t + DEPTH, d);
                // One barrier a tile: the other stage is written after the
                // next one, when every wave has read it.
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
                        for (int j = 0; j < KT::TN; ++j) mfma_step<TI, 16>(fa[i], fb[j], acc[i][j]);
                }
            }
        }
    }
};

template <In TI, Out TO, int BM, int BN, int BK, int WM, int WN, int DEPTH, bool AK, bool BKM, By BY, bool EPI>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_ragged_odd_kernel(Params p, Ragged r)
{
    using T = OddTile<TI, TO, BM, BN, BK, WM, WN, DEPTH, AK, BKM>;
    using KT = typename T::KT;
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    if (!select_group<TI, TO, BM, BN, BY, false>(p, r, lane, tm, tn)) return;
    const int m0 = tm * BM, n0 = tn * BN;
    typename KT::Acc acc;
    KT::zero(acc);
    T::mainloop(p, smem, m0, n0, acc, lane, wave);
    store_tile<KT, EPI>(p, smem, m0, n0, acc, tid, lane, wave);
}

// 16-bit inputs on the direct-to-LDS ring of gemm_dma.hpp.
template <In TI, Out TO, int BM, int BN, int BK, int WM, int WN, int MI, int STAGES, bool AK, bool BKM, By BY, bool EPI>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_ragged_dma_kernel(Params p, Ragged r)
{
    using KT = Dma16<TI, TO, BM, BN, BK, WM, WN, MI, STAGES, AK, BKM>;
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    if (!select_group<TI, TO, BM, BN, BY, true>(p, r, lane, tm, tn)) return;
    const int m0 = tm * BM, n0 = tn * BN;
    typename KT::OA oa;
    typename KT::OB ob;
    oa.init(wave, lane, p.lda);
    ob.init(wave, lane, p.ldb);
    typename KT::Acc acc;
    KT::zero(acc);
    KT::mainloop(p, smem, oa, ob, m0, n0, 0, (p.K + BK - 1) / BK, acc, tid, lane, wave);
    store_tile<KT, EPI>(p, smem, m0, n0, acc, tid, lane, wave);
}

// The ping-pong schedule of gemm_pp_kernel (gemm_dma.hpp, which explains it)
// over all of p.K, adding to acc: two groups of four waves, one multiplying a
// k-tile out of registers while the other issues its loads and reads the next
// fragments.  All loads have landed on return.
// SWAP: the operands are exchanged at the MFMA, which makes C's tile transposed
// in the accumulators: a lane holds 4 consecutive columns of one row.
template <In TI, Out TO, int BM, int BN, int BK, int WM, int WN, int MI, bool AK, bool BKM, bool SWAP>
struct PingPong {
    using KT = Dma16<TI, TO, BM, BN, BK, WM, WN, MI, 3, AK, BKM, 2>;
    using LA = DmaOperand<BM, BK, 4, AK, MI>;     // loaded by group 1
    using LB = DmaOperand<BN, BK, 4, BKM, MI>;    // loaded by group 0
    static constexpr int NG = KT::NG, KG = KT::KG, TM = KT::TM, TN = KT::TN, NT = KT::NT;
    static constexpr int WTM = KT::WTM, WTN = KT::WTN, IA = LA::IPW, IB = LB::IPW;
    static_assert(WM * WN == 8, "two groups of four waves");
    static_assert(IA == IB, "one offset set for either operand");

    __device__ static __forceinline__ void mainloop(const Params& p, char* smem, int m0, int n0, typename KT::Acc& acc,
                                                    int tid, int lane, int wave)
    {
        const int grp = wave >> 2, gw = wave & 3, wm = wave / WN, wn = wave % WN;
        // The loop runs the whole k-tiles.  (A k-contiguous operand's partial
        // last tile needs zeros past K, written in LDS: inside the loop that
        // code's registers spill, and each reload waits for every load in
        // flight -- measured 1.7x on the gradient of the tokens.  An
        // m-contiguous operand reads zeros there, so if both are it is a tile
        // like the others.)
        constexpr bool TAIL = AK || BKM;
        const int nkt = TAIL ? p.K / BK : (p.K + BK - 1) / BK;
        // A wave loads one operand only; its per-lane offsets pass through an
        // empty asm so that each takes one register (the 64-bit product they
        // come from would keep two, and a spilled offset's reload waits for
        // every load in flight).
        int voff[IA];
        if (grp) {
            LA o;
            o.init(gw, lane, p.lda);
#pragma unroll
            for (int j = 0; j < IA; ++j) voff[j] = o.voff[j];
        } else {
            LB o;
            o.init(gw, lane, p.ldb);
#pragma unroll
            for (int j = 0; j < IB; ++j) voff[j] = o.voff[j];
        }
#pragma unroll
        for (int j = 0; j < IA; ++j) asm volatile("" : "+v"(voff[j]));
        auto issue_a = [&](int t, int stage, uint64_t bytes) {
            LA o;
#pragma unroll
            for (int j = 0; j < IA; ++j) o.voff[j] = voff[j];
            o.issue(p.A, bytes, p.lda, m0, t * BK, KT::a_stage(smem, stage), gw);
        };
        auto issue_b = [&](int t, int stage, uint64_t bytes) {
            LB o;
#pragma unroll
            for (int j = 0; j < IB; ++j) o.voff[j] = voff[j];
            o.issue(p.B, bytes, p.ldb, n0, t * BK, KT::b_stage(smem, stage), gw);
        };
        // Loads past the last tile get an empty extent: zeros into a free slot.
        auto next_a = [&](int t) { issue_a(t, t, t < nkt ? p.a_bytes : 0); };
        auto next_b = [&](int t) { issue_b(t, t, t < nkt ? p.b_bytes : 0); };
        i32x4 fa[NG][TM], fb[NG][TN];
        auto read_all = [&](int s) {
            const char* sa = KT::a_stage(smem, s);
            const char* sb = KT::b_stage(smem, s);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
#pragma unroll
                for (int i = 0; i < TM; ++i) fa[g][i] = LA::template frag<MI>(sa, wm * WTM + i * MI, g * KG, lane);
#pragma unroll
                for (int j = 0; j < TN; ++j) fb[g][j] = LB::template frag<MI>(sb, wn * WTN + j * MI, g * KG, lane);
            }
        };
        auto mfma_all = [&]() {
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) mfma_step<TI, MI>(SWAP ? fb[g][j] : fa[g][i], SWAP ? fa[g][i] : fb[g][j], acc[i][j]);
        };
        if (grp) {
            next_a(0);
            next_a(1);
            wait_vmcnt<IA>();
        } else {
            next_b(0);
            next_b(1);
            wait_vmcnt<IB>();
        }
        bare_barrier();
        if (!grp) {
            read_all(0);
            __builtin_amdgcn_s_waitcnt(0xc07f);
            for (int t = 0; t < nkt; ++t) {
                __builtin_amdgcn_sched_barrier(0);
                mfma_all();                       // phase A: tile t
                __builtin_amdgcn_sched_barrier(0);
                wait_vmcnt<0>();                  // B of tile t + 1
                bare_barrier();
                __builtin_amdgcn_sched_barrier(0);
                next_b(t + 2);                   // phase B: into tile t's B slot
                if (t + 1 < nkt) read_all(t + 1);
                __builtin_amdgcn_s_waitcnt(0xc07f);
                __builtin_amdgcn_sched_barrier(0);
                bare_barrier();
            }
        } else {
            for (int t = 0; t < nkt; ++t) {
                __builtin_amdgcn_sched_barrier(0);
                next_a(t + 2);                   // phase A: into tile t-1's A slot
                read_all(t);
                __builtin_amdgcn_s_waitcnt(0xc07f);
                wait_vmcnt<IA>();                 // A of tile t + 1
                __builtin_amdgcn_sched_barrier(0);
                bare_barrier();
                __builtin_amdgcn_sched_barrier(0);
                mfma_all();                       // phase B: tile t
                __builtin_amdgcn_sched_barrier(0);
                bare_barrier();
            }
        }
        wait_vmcnt<0>();
        if constexpr (TAIL) {
            const int left = p.K - nkt * BK;
            if (left == 0) return;
            bare_barrier();                       // no empty load into the ring is still to land
            if (grp) issue_a(nkt, 0, p.a_bytes);
            else issue_b(nkt, 0, p.b_bytes);
            wait_vmcnt<0>();
            bare_barrier();
            LA::template zero_tail<NT>(KT::a_stage(smem, 0), left, tid);
            LB::template zero_tail<NT>(KT::b_stage(smem, 0), left, tid);
            __syncthreads();
#pragma unroll 1
            for (int g = 0; g * KG < left; ++g) {    // rolled: the accumulators stay where they are
                i32x4 ta[TM], tb[TN];
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    ta[i] = LA::template frag<MI>(KT::a_stage(smem, 0), wm * WTM + i * MI, g * KG, lane);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    tb[j] = LB::template frag<MI>(KT::b_stage(smem, 0), wn * WTN + j * MI, g * KG, lane);
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) mfma_step<TI, MI>(SWAP ? tb[j] : ta[i], SWAP ? ta[i] : tb[j], acc[i][j]);
            }
        }
    }

    // Add C's old values, in fp32.
    __device__ static __forceinline__ void add_c(const Params& p, int m0, int n0, typename KT::Acc& acc, int lane, int wave)
    {
        static_assert(SWAP, "a lane's accumulators run along a row");
        const int wm = wave / WN, wn = wave % WN;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int m = m0 + wm * WTM + i * MI + lane % MI;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int n = n0 + wn * WTN + j * MI + lane / MI * 4;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m < p.M && n + e < p.N) acc[i][j][e] += load_out<TO>(p.C, (int64_t)m * p.ldc + n + e);
            }
        }
    }

    // Through LDS as Dma16::store_rows, each wave on its own, with a vector of 4
    // columns to an LDS write.  C is written in
    // row pieces of WTN elements: straight from the accumulators, 16 or 8
    // bytes of 16 rows to a store, the product below took 185 us.
    // Measured on 8192 rows in 16 groups, N = 4096, K = 2048, bf16: 146 us; by
    // k, 32 groups of 256 k, 4096 x 2048 in bf16: 233 us (249 with an LDS write
    // per element).
    __device__ static __forceinline__ void store(const Params& p, char* smem, int m0, int n0, const typename KT::Acc& acc,
                                                 int lane, int wave)
    {
        static_assert(SWAP, "a lane's accumulators run along a row");
        constexpr int EO = KT::OBY;
        const int wm = wave / WN, wn = wave % WN;
        char* const w = smem + wave * KT::SHARE;
        const int mb = m0 + wm * WTM, nb = n0 + wn * WTN;
        bare_barrier();               // every wave's loads have landed and its ring reads are done
#pragma unroll
        for (int pass = 0; pass < WTM / KT::RPP; ++pass) {
#pragma unroll
            for (int i = pass * KT::RPP / MI; i < (pass + 1) * KT::RPP / MI; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    char* d = w + (i * MI - pass * KT::RPP + lane % MI) * KT::SPITCH + (j * MI + lane / MI * 4) * EO;
                    if constexpr (EO == 4) {
                        *(f32x4*)d = acc[i][j];
                    } else {
                        typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
                        uint16_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            h[e] = TO == Out::F16 ? __builtin_bit_cast(uint16_t, (_Float16)acc[i][j][e])
                                                  : __builtin_bit_cast(uint16_t, (__bf16)acc[i][j][e]);
                        *(u32x2*)d = u32x2{(unsigned)h[0] | ((unsigned)h[1] << 16), (unsigned)h[2] | ((unsigned)h[3] << 16)};
                    }
                }
            copy_rows<KT>(p, w, mb + pass * KT::RPP, nb, lane);
        }
    }
};

template <In TI, Out TO, int BM, int BN, int BK, int WM, int WN, int MI, bool AK, bool BKM, By BY, bool EPI>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_ragged_pp_kernel(Params p, Ragged r)
{
    using PP = PingPong<TI, TO, BM, BN, BK, WM, WN, MI, AK, BKM, true>;
    using KT = typename PP::KT;
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    if (!select_group<TI, TO, BM, BN, BY, true>(p, r, lane, tm, tn)) return;
    const int m0 = tm * BM, n0 = tn * BN;
    typename KT::Acc acc;
    KT::zero(acc);
    PP::mainloop(p, smem, m0, n0, acc, tid, lane, wave);
    if constexpr (EPI) PP::add_c(p, m0, n0, acc, lane, wave);
    PP::store(p, smem, m0, n0, acc, lane, wave);
}

// fp32 on the direct-to-LDS engine of gemm_f32dma.hpp (VEC = false: 4-byte
// loads of element-aligned operands).
template <int BM, int BN, int BK, int WM, int WN, int STAGES, bool AK, bool BKM, By BY, bool EPI, bool VEC>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_ragged_f32_kernel(Params p, Ragged r)
{
    using KT = F32Dma<Out::F32, BM, BN, BK, WM, WN, STAGES, AK, BKM, VEC>;
    __shared__ __attribute__((aligned(1024))) char smem[KT::SMEM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    if (!select_group<In::F32, Out::F32, BM, BN, BY, VEC>(p, r, lane, tm, tn)) return;
    const int m0 = tm * BM, n0 = tn * BN;
    typename KT::OA oa;
    typename KT::OB ob;
    oa.init(wave, lane, p.lda);
    ob.init(wave, lane, p.ldb);
    typename KT::Acc acc;
    KT::zero(acc);
    KT::mainloop(p, smem, oa, ob, m0, n0, 0, (p.K + BK - 1) / BK, acc, tid, lane, wave);
    KT::template store<false, EPI>(p, m0, n0, acc, lane, wave, smem);
}

// Few rows: the product streams B once and is bound by how many of its bytes
// are in flight.  A workgroup has 16 MT rows and 16 NT columns.  NW waves take
// the k-tiles in turn, each with a ring of ST tiles of its own in LDS: nothing
// waits for another wave until the sums meet at the end, in wave order.  A
// tile's slot is loaded again as soon as its fragments are in registers.
template <In TI, int MT, int NT, int NW, int ST, bool BKM, bool VEC>
struct Skinny {
    // A k-tile is 128 bytes of a row: 64 or 32 of k.
    static constexpr bool F32 = TI == In::F32;
    static constexpr int ES = F32 ? 4 : 2, BK = 128 / ES, MI = 16, NG = 2;
    using OA = std::conditional_t<F32, F32Operand<MT * 16, BK, 1, true, VEC>, DmaOperand<MT * 16, BK, 1, true, MI>>;
    using OB = std::conditional_t<F32, F32Operand<NT * 16, BK, 1, BKM, VEC>, DmaOperand<NT * 16, BK, 1, true, MI>>;
    static_assert(F32 || (BKM && VEC), "16-bit operands: k-major, 16-byte loads");
    static constexpr int STAGE = OA::BYTES + OB::BYTES, L = (OA::IPW + OB::IPW) * (VEC ? 1 : 4);
    static constexpr int PART = MT * 16 * NT * 16;            // sums of a wave
    static constexpr int RING = NW * ST * STAGE;
    static_assert((ST - 1) * L < 64, "vmcnt range");
    typedef f32x4 Acc[MT][NT];

    __device__ static __forceinline__ void zero(Acc& acc)
    {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // This wave's k-tiles.
    __device__ static __forceinline__ void stream(const Params& p, char* smem, int m0, int n0, Acc& acc, int lane, int wave)
    {
        const int nkt = (p.K + BK - 1) / BK, left = p.K - (nkt - 1) * BK;
        OA oa;
        OB ob;
        oa.init(0, lane, p.lda);
        ob.init(0, lane, p.ldb);
        char* const ring = smem + wave * ST * STAGE;
        auto issue = [&](int t, int slot) {            // past the end: an empty extent, zeros
            char* s = ring + slot * STAGE;
            oa.issue(p.A, t < nkt ? p.a_bytes : 0, p.lda, m0, t * BK, s, 0);
            ob.issue(p.B, t < nkt ? p.b_bytes : 0, p.ldb, n0, t * BK, s + OA::BYTES, 0);
        };
#pragma unroll
        for (int i = 0; i < ST; ++i) issue(wave + i * NW, i);
        int slot = 0;
        for (int t = wave; t < nkt; t += NW) {
            wait_vmcnt<(ST - 1) * L>();
            char* s = ring + slot * STAGE;
            if (t == nkt - 1 && left != BK) {
                oa.template zero_tail<64>(s, left, lane);
                if constexpr (BKM) ob.template zero_tail<64>(s + OA::BYTES, left, lane);
                __builtin_amdgcn_s_waitcnt(0xc07f);
            }
            asm volatile("" ::: "memory");
            // Fragment g: the 16 bytes of k-chunk 4 g + lane / 16 of a row.  A
            // chunk of an n-major B is four values of one column.
            auto chunk = [&](const char* tile, int row, int g) {
                return *(const i32x4*)(tile + row * 128 + swz_chunk<8, true>(row, g * 4 + lane / 16) * 16);
            };
            i32x4 fa[NG][MT], fb[NG][NT];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
#pragma unroll
                for (int i = 0; i < MT; ++i) fa[g][i] = chunk(s, i * MI + lane % MI, g);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int n = j * MI + lane % MI;
                    if constexpr (BKM) {
                        fb[g][j] = chunk(s + OA::BYTES, n, g);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            fb[g][j][e] = ((const int*)(s + OA::BYTES))[(g * 16 + lane / 16 * 4 + e) * (NT * MI) + n];
                    }
                }
            }
            __builtin_amdgcn_s_waitcnt(0xc07f);        // lgkmcnt(0): the slot has been read
            __builtin_amdgcn_sched_barrier(0);
            issue(t + ST * NW, slot);
            slot = slot + 1 == ST ? 0 : slot + 1;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) mfma_step<TI, MI>(fa[g][i], fb[g][j], acc[i][j]);
        }
        wait_vmcnt<0>();                               // the empty loads have landed
    }

    // The sums of all WAVES waves, stored.
    template <Out TO, int WAVES>
    __device__ static __forceinline__ void join(const Params& p, char* smem, int m0, int n0, const Acc& acc, int tid, int lane,
                                                int wave)
    {
        static_assert(WAVES * PART * 4 <= RING, "sums fit the ring");
        __syncthreads();
        float* const part = (float*)smem;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    part[wave * PART + (i * 16 + lane / 16 * 4 + e) * (NT * 16) + j * 16 + lane % 16] = acc[i][j][e];
        __syncthreads();
        for (int x = tid; x < PART; x += WAVES * 64) {
            const int m = m0 + x / (NT * 16), n = n0 + x % (NT * 16);
            if (m >= p.M || n >= p.N) continue;
            float v = part[x];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v += part[w * PART + x];
            store_out<TO>(p.C, (int64_t)m * p.ldc + n, v);
        }
    }
};

template <int MT, int NT, int NW, int ST, bool BKM, bool VEC>
__global__ void __launch_bounds__(NW * 64)
gemm_ragged_skinny_kernel(Params p, Ragged r)
{
    using T = Skinny<In::F32, MT, NT, NW, ST, BKM, VEC>;
    static_assert(T::RING <= 160 * 1024, "LDS budget");
    __shared__ __attribute__((aligned(1024))) char smem[T::RING];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    if (!select_group<In::F32, Out::F32, MT * 16, NT * 16, By::Rows, VEC>(p, r, lane, tm, tn)) return;
    typename T::Acc acc;
    T::zero(acc);
    T::stream(p, smem, tm * (MT * 16), tn * (NT * 16), acc, lane, wave);
    T::template join<Out::F32, NW>(p, smem, tm * (MT * 16), tn * (NT * 16), acc, tid, lane, wave);
}

// ------------------------------------------------------------------ launchers

// What the host asks of a dtype's launchers (gemm_ragged_<dtype>.hip).
struct RaggedCall {
    Params p;             // p.epi: add to C (by k only)
    Ragged r;
    bool by_rows;
    bool b_kmajor;        // by rows: B_g k-major (else n-major)
    bool vec;             // operands allow 16-byte loads
};

inline RaggedShape shape_of(const RaggedCall& c, bool f32)
{
    return {f32, c.by_rows, c.vec, c.b_kmajor, c.by_rows ? c.r.rows : c.p.M, c.p.N, c.r.groups};
}

template <By BY, class Kernel>
hipError_t launch_ragged(Kernel kernel, const RaggedCall& c, const Tile& t, hipStream_t s)
{
    Params p = c.p;
    Ragged r = c.r;
    p.tiles_m = (int)ceil_div(p.M, t.bm);
    p.tiles_n = (int)ceil_div(p.N, t.bn);
    // By k an XCD has 16 tiles of 4096 x 2048 outputs: 4 x 4 of them read fewer
    // rows of A and B than 8 x 2 (8192 k in 16 groups into fp32 187 us against
    // 192, in 32 groups 270 against 288).
    const int high = BY == By::K ? 4 : 8;
    p.group_m = p.tiles_m < high ? p.tiles_m : high;
    const dim3 grid((unsigned)ragged_grid(shape_of(c, false), t), BY == By::K ? (unsigned)r.groups : 1u);
    void* args[] = {&p, &r};
    return hipLaunchKernel((const void*)kernel, grid, dim3(t.threads), args, 0, s);
}

template <In TI, Out TO>
struct RaggedInst {
    template <RaggedTile T, bool AK, bool BKM, By BY, bool EPI>
    static hipError_t odd(const RaggedCall& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T);
        return launch_ragged<BY>(&gemm_ragged_odd_kernel<TI, TO, t.bm, t.bn, t.bk, t.wm, t.wn, t.stages, AK, BKM, BY, EPI>, c, t, s);
    }
    template <RaggedTile T, bool AK, bool BKM, By BY, bool EPI>
    static hipError_t dma(const RaggedCall& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(T);
        return launch_ragged<BY>(&gemm_ragged_dma_kernel<TI, TO, t.bm, t.bn, t.bk, t.wm, t.wn, t.mi, t.stages, AK, BKM, BY, EPI>, c, t, s);
    }
    template <bool AK, bool BKM, By BY, bool EPI>
    static hipError_t pp(const RaggedCall& c, hipStream_t s)
    {
        constexpr Tile t = tile_of(RaggedTile::PingPong);
        return launch_ragged<BY>(&gemm_ragged_pp_kernel<TI, TO, t.bm, t.bn, t.bk, t.wm, t.wn, t.mi, AK, BKM, BY, EPI>, c, t, s);
    }
    template <bool BKM>
    static hipError_t rows(const RaggedCall& c, hipStream_t s)
    {
        switch (ragged_tile(shape_of(c, false))) {
        case RaggedTile::Rows32x64: return dma<RaggedTile::Rows32x64, true, BKM, By::Rows, false>(c, s);
        case RaggedTile::Rows64x128: return dma<RaggedTile::Rows64x128, true, BKM, By::Rows, false>(c, s);
        case RaggedTile::Rows128x64: return dma<RaggedTile::Rows128x64, true, BKM, By::Rows, false>(c, s);
        case RaggedTile::Rows128x128: return dma<RaggedTile::Rows128x128, true, BKM, By::Rows, false>(c, s);
        case RaggedTile::Rows128x128Two: return dma<RaggedTile::Rows128x128Two, true, BKM, By::Rows, false>(c, s);
        case RaggedTile::Rows128x256: return dma<RaggedTile::Rows128x256, true, BKM, By::Rows, false>(c, s);
        case RaggedTile::PingPong: return pp<true, BKM, By::Rows, false>(c, s);
        case RaggedTile::Odd32x64: return odd<RaggedTile::Odd32x64, true, BKM, By::Rows, false>(c, s);
        case RaggedTile::Odd64x128: return odd<RaggedTile::Odd64x128, true, BKM, By::Rows, false>(c, s);
        case RaggedTile::Odd128x128: return odd<RaggedTile::Odd128x128, true, BKM, By::Rows, false>(c, s);
        default: return hipErrorInvalidValue;
        }
    }
    template <bool EPI>
    static hipError_t by_k(const RaggedCall& c, hipStream_t s)
    {
        switch (ragged_tile(shape_of(c, false))) {
        case RaggedTile::K64x64: return dma<RaggedTile::K64x64, false, false, By::K, EPI>(c, s);
        case RaggedTile::K128x128: return dma<RaggedTile::K128x128, false, false, By::K, EPI>(c, s);
        case RaggedTile::K128x128Two: return dma<RaggedTile::K128x128Two, false, false, By::K, EPI>(c, s);
        case RaggedTile::PingPong: return pp<false, false, By::K, EPI>(c, s);
        case RaggedTile::OddK64x64: return odd<RaggedTile::OddK64x64, false, false, By::K, EPI>(c, s);
        case RaggedTile::OddK128x128: return odd<RaggedTile::OddK128x128, false, false, By::K, EPI>(c, s);
        default: return hipErrorInvalidValue;
        }
    }
    static hipError_t launch(const RaggedCall& c, hipStream_t s)
    {
        if (c.by_rows) return c.b_kmajor ? rows<true>(c, s) : rows<false>(c, s);
        return c.p.epi ? by_k<true>(c, s) : by_k<false>(c, s);
    }
};

hipError_t ragged_f32(const RaggedCall& c, hipStream_t s);
hipError_t ragged_f16_f32(const RaggedCall& c, hipStream_t s);
hipError_t ragged_bf16_bf16(const RaggedCall& c, hipStream_t s);
hipError_t ragged_f16_f16(const RaggedCall& c, hipStream_t s);
hipError_t ragged_bf16_f32(const RaggedCall& c, hipStream_t s);

}  // namespace mg
