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

// Point p at the workgroup's group; false: no tile for this workgroup.
// ROWS (by rows): p.M is the group's rows, A and C start at its first row, B
// at its matrix.  Otherwise p.K is the group's k-range, A and B (both with k
// as the outer index) start at its first k, C at the group's matrix; a group
// without any k writes zeros, or nothing where C is added to.
// tm, tn: the tile within the group.
template <In TI, Out TO, int BM, int BN, bool ROWS, bool VEC>
__device__ __forceinline__ bool select_group(Params& p, const Ragged& r, int lane, int& tm, int& tn)
{
    constexpr int ES = TI == In::F32 ? 4 : 2, EO = TO == Out::F32 ? 4 : 2;
    int g, start, len;
    if constexpr (ROWS) {
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
    return true;
}

// The grouped product on the register-staged tile of gemm_kernel.hpp: right
// for every type, layout and alignment (VEC = false: element-aligned operands).
template <In TI, Out TO, int BM, int BN, int BK, int WM, int WN, int MI, bool AK, bool BKM, bool ROWS, bool EPI, bool VEC>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_ragged_kernel(Params p, Ragged r)
{
    using T = GemmTile<TI, TO, BM, BN, BK, WM, WN, MI, AK, BKM, true, VEC>;
    static_assert(MI == 16, "accumulator layout of the store below");
    __shared__ __attribute__((aligned(16))) char smem[2 * T::STAGE];
    T t;
    t.tid = threadIdx.x;
    const int lane = t.tid & 63, wave = t.tid >> 6;
    t.wm = wave / WN;
    t.wn = wave % WN;
    t.frow = lane % MI;
    t.fq = lane / MI;
    int tm, tn;
    if (!select_group<TI, TO, BM, BN, ROWS, VEC>(p, r, lane, tm, tn)) return;
    const int m0 = tm * BM, n0 = tn * BN;
    t.la.init(t.tid, p.lda);
    t.lb.init(t.tid, p.ldb);
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j) t.acc[i][j] = typename T::Acc{};

    // k-tile kt is multiplied out of LDS while kt + 1 goes from registers to
    // the other LDS stage and kt + 2 from memory to registers.
    const int nkt = (p.K + BK - 1) / BK;
    const bool ragged = p.K % BK != 0;
    auto load = [&](int kt) {
        t.la.load(p.A, p.a_bytes, p.lda, m0, kt * BK, t.tid);
        t.lb.load(p.B, p.b_bytes, p.ldb, n0, kt * BK, t.tid);
    };
    auto mask = [&](int kt) {
        if (!ragged || kt != nkt - 1) return;
        t.la.mask(kt * BK, p.K, t.tid);
        t.lb.mask(kt * BK, p.K, t.tid);
    };
    if (nkt > 0) {
        load(0);
        mask(0);
        t.la.store(smem, t.tid);
        t.lb.store(smem + T::A_BYTES, t.tid);
        if (nkt > 1) load(1);
        __syncthreads();
        t.read_frags(smem, 0, 0);
        int kt = 0;
        for (; kt + 2 < nkt; ++kt) t.template tile<true, true, true>(smem, kt & 1, p, m0, n0, (kt + 2) * BK);
        if (kt + 1 < nkt) {
            mask(kt + 1);
            t.template tile<true, false, true>(smem, kt & 1, p, m0, n0, 0);
            ++kt;
        }
        t.template tile<false, false, false>(smem, kt & 1, p, m0, n0, 0);
    }
    if constexpr (EPI) {
        store_tile_via_lds<TO, BM, BN, T::NT, T::TM * T::TN * 4, 2 * T::STAGE>(
            p, smem, m0, n0, t.tid, [&](int v) { return t.acc[v / (T::TN * 4)][(v / 4) % T::TN][v % 4]; },
            [&](int v, int& row, int& col) {
                const int i = v / (T::TN * 4), j = (v / 4) % T::TN, q = v % 4;
                row = t.wm * T::WTM + i * MI + (lane / 16) * 4 + q;
                col = t.wn * T::WTN + j * MI + lane % 16;
            });
    } else {
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
#pragma unroll
            for (int j = 0; j < T::TN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int m = m0 + t.wm * T::WTM + i * MI + (lane / 16) * 4 + q;
                    const int n = n0 + t.wn * T::WTN + j * MI + lane % 16;
                    if (m < p.M && n < p.N) store_out<TO>(p.C, (int64_t)m * p.ldc + n, t.acc[i][j][q]);
                }
    }
}

// What the host asks of a dtype's launchers (gemm_grouped_<dtype>.hip).
struct RaggedCall {
    Params p;             // p.epi: add to C (by k only)
    Ragged r;
    bool by_rows;
    bool b_kmajor;        // by rows: B_g k-major (else n-major)
    bool vec;             // operands allow 16-byte loads
};

// Tiles of the grid's upper bound: by rows, ceil(len_g / BM) summed over the
// groups is at most (rows + groups * (BM - 1)) / BM.
template <class Kernel>
hipError_t launch_ragged(Kernel kernel, const RaggedCall& c, int BM, int BN, int threads, hipStream_t s)
{
    Params p = c.p;
    Ragged r = c.r;
    p.tiles_m = (p.M + BM - 1) / BM;
    p.tiles_n = (p.N + BN - 1) / BN;
    p.group_m = p.tiles_m < 8 ? p.tiles_m : 8;
    dim3 grid;
    if (c.by_rows) {
        int64_t tm = ((int64_t)r.rows + (int64_t)r.groups * (BM - 1)) / BM;
        if (tm > r.rows) tm = r.rows;
        grid = dim3((unsigned)(tm * p.tiles_n));
    } else {
        grid = dim3((unsigned)(p.tiles_m * p.tiles_n), (unsigned)r.groups);
    }
    void* args[] = {&p, &r};
    return hipLaunchKernel((const void*)kernel, grid, dim3(threads), args, 0, s);
}

template <In TI, Out TO>
struct RaggedInst {
    static constexpr int BK = TI == In::F32 ? 32 : 64;
    template <bool AK, bool BKM, bool ROWS, bool EPI, bool VEC>
    static hipError_t generic(const RaggedCall& c, hipStream_t s)
    {
        return launch_ragged(&gemm_ragged_kernel<TI, TO, 64, 64, BK, 2, 2, 16, AK, BKM, ROWS, EPI, VEC>, c, 64, 64, 256, s);
    }
    template <bool VEC>
    static hipError_t any(const RaggedCall& c, hipStream_t s)
    {
        if (c.by_rows)
            return c.b_kmajor ? generic<true, true, true, false, VEC>(c, s) : generic<true, false, true, false, VEC>(c, s);
        return c.p.epi ? generic<false, false, false, true, VEC>(c, s) : generic<false, false, false, false, VEC>(c, s);
    }
    static hipError_t launch(const RaggedCall& c, hipStream_t s) { return c.vec ? any<true>(c, s) : any<false>(c, s); }
};

hipError_t ragged_f32(const RaggedCall& c, hipStream_t s);
hipError_t ragged_f16_f32(const RaggedCall& c, hipStream_t s);
hipError_t ragged_bf16_bf16(const RaggedCall& c, hipStream_t s);
hipError_t ragged_f16_f16(const RaggedCall& c, hipStream_t s);
hipError_t ragged_bf16_f32(const RaggedCall& c, hipStream_t s);

}  // namespace mg
