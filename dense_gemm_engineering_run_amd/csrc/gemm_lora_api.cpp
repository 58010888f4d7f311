// gemm_lora_api.cpp -- the adapter entry points of include/mi355_gemm.h:
// argument checks (all before any HIP call), the workspace and the launch.
#include <hip/hip_runtime.h>

#include <cctype>

#include "gemm_checks.hpp"
#include "gemm_lora.hpp"

namespace {

using mg::Operand;

constexpr int64_t kMaxSlots = (int64_t)1 << 20;
constexpr int64_t kMaxRank = 4096;
constexpr int64_t kTileRows = 256;     // rows a tile of any kernel here spans

typedef hipError_t (*Launcher)(const mg::LoraCall&, hipStream_t);
const Launcher kLaunch[GEMM_NUM_DTYPES] = {mg::lora_f32, mg::lora_f16_f32, mg::lora_bf16_bf16, mg::lora_f16_f16,
                                           mg::lora_bf16_f32};

bool offsets_fit(const Operand& o) { return (kTileRows * o.ld + kTileRows) * o.es < ((int64_t)1 << 31); }

int64_t pitch(int64_t rank) { return (rank + mg::kRankStep - 1) / mg::kRankStep * mg::kRankStep; }

bool bad_shape(int64_t M, int64_t N, int64_t K, int64_t rank)
{
    return M < 0 || N < 0 || K < 0 || rank < 0 || M > mg::kMaxDim || N > mg::kMaxDim || K > mg::kMaxDim || rank > kMaxRank;
}

uint64_t workspace(int64_t M, int64_t N, int64_t K, int64_t rank, bool tiled)
{
    if (M == 0 || N == 0 || K == 0 || rank == 0) return 0;
    return (uint64_t)mg::shrink_plan(M, K, tiled).splits * M * pitch(rank) * 4;
}

// The most that any call of at most M rows needs, whatever its alignment: the
// ranges of k grow fewer as the tiles of rows grow more, so fewer rows can
// need more.
uint64_t workspace_up_to(int64_t M, int64_t N, int64_t K, int dtype, int64_t rank)
{
    uint64_t most = 0;
    for (int tiled = 0; tiled <= mg::shrink_tiled(mg::in_bytes(dtype), true); ++tiled) {
        most = std::max(most, workspace(M, N, K, rank, tiled));
        for (int64_t m = mg::kShrinkRows; m < std::min<int64_t>(M, 1 << 14); m += mg::kShrinkRows)
            most = std::max(most, std::max(workspace(m - 1, N, K, rank, tiled), workspace(m, N, K, rank, tiled)));
    }
    return most;
}

int run(int64_t M, int64_t N, int64_t K, char a, char b, char c, int dtype, const void* A, const void* B, void* C,
        int64_t lda, int64_t ldb, int64_t ldc, const gemm_lora_t* lora, void* ws, size_t ws_bytes, void* stream)
{
    static const gemm_lora_t none = {};
    const gemm_lora_t& l = lora ? *lora : none;
    if (bad_shape(M, N, K, l.rank) || l.adapters < 0 || l.adapters > kMaxSlots) return GEMM_ERR_BAD_SHAPE;
    a = (char)std::tolower((unsigned char)a);
    b = (char)std::tolower((unsigned char)b);
    c = (char)std::tolower((unsigned char)c);
    if (a != 'k' || (b != 'k' && b != 'n') || c != 'n') return GEMM_ERR_BAD_MAJOR;
    if (dtype < 0 || dtype >= GEMM_NUM_DTYPES) return GEMM_ERR_BAD_DTYPE;
    const int es = mg::in_bytes(dtype), eo = mg::out_bytes(dtype);

    const bool adapted = l.adapters > 0 && l.rank > 0;
    const Operand oa = {A, M, K, lda, 1, 0, es};
    const Operand ob = b == 'k' ? Operand{B, N, K, ldb, 1, 0, es} : Operand{B, K, N, ldb, 1, 0, es};
    const Operand oc = {C, M, N, ldc, 1, 0, eo};
    const Operand od = {l.down, l.rank, K, l.ld_down, l.adapters, l.stride_down, es};
    const Operand ou = {l.up, N, l.rank, l.ld_up, l.adapters, l.stride_up, es};
    if (!oa.lds_ok() || !ob.lds_ok() || !oc.lds_ok()) return GEMM_ERR_BAD_LD;
    if (adapted && (!od.lds_ok() || !ou.lds_ok())) return GEMM_ERR_BAD_LD;

    if (M == 0 || N == 0) return GEMM_OK;
    const bool reads = K > 0, with = adapted && reads;
    if ((reads && (!A || !B)) || !C) return GEMM_ERR_NULL_PTR;
    if (with && (!l.down || !l.up || !l.ids)) return GEMM_ERR_NULL_PTR;
    if ((reads && (!oa.aligned(es) || !ob.aligned(es))) || !oc.aligned(eo) || (ws && ((uintptr_t)ws & 15)))
        return GEMM_ERR_MISALIGNED;
    if (with && (!od.aligned(es) || !ou.aligned(es) ||
                 (((uintptr_t)l.ids | (uintptr_t)l.ranks | (uintptr_t)l.scales) & 3)))
        return GEMM_ERR_MISALIGNED;
    const bool vec = !reads || (oa.aligned(16) && ob.aligned(16) && (!with || od.aligned(16)));
    const bool odd_up = with && !ou.aligned(16);
    const uint64_t cn = oc.bytes(false), need = with ? workspace(M, N, K, l.rank, mg::shrink_tiled(es, vec)) : 0;
    // What is read, against what is written: C and the part of the workspace in use.
    const struct { const void* p; uint64_t n; } in[] = {
        {A, reads ? oa.bytes(vec) : 0}, {B, reads ? ob.bytes(vec) : 0},
        {l.down, with ? od.bytes(vec) : 0}, {l.up, with ? ou.bytes(vec && !odd_up) : 0}, {l.ids, with ? (uint64_t)M * 4 : 0},
        {l.ranks, with ? (uint64_t)l.adapters * 4 : 0}, {l.scales, with ? (uint64_t)l.adapters * 4 : 0}};
    for (const auto& x : in)
        if (mg::overlap(C, cn, x.p, x.n) || mg::overlap(ws, need, x.p, x.n)) return GEMM_ERR_ALIAS;
    if (mg::overlap(C, cn, ws, need)) return GEMM_ERR_ALIAS;
    if ((reads && (!offsets_fit(oa) || !offsets_fit(ob))) || (with && (!offsets_fit(od) || !offsets_fit(ou))))
        return GEMM_ERR_BAD_SHAPE;
    if (with && (!ws || ws_bytes < need)) return GEMM_ERR_WORKSPACE;

    mg::LoraCall q = {};
    mg::Params& p = q.p;
    p.A = (const char*)A;
    p.B = (const char*)B;
    p.C = (char*)C;
    p.M = (int)M; p.N = (int)N; p.K = (int)K;
    p.lda = lda; p.ldb = ldb; p.ldc = ldc;
    p.batch = 1;
    p.split = 1;
    p.alpha = 1.f;
    p.a_bytes = reads ? oa.bytes(vec) : 0;
    p.b_bytes = reads ? ob.bytes(vec) : 0;
    p.c_vec = oc.aligned(16);
    if (with) {
        const mg::ShrinkPlan s = mg::shrink_plan(M, K, mg::shrink_tiled(es, vec), pitch(l.rank));
        q.shrink_rows = s.rows;
        q.q = mg::Lora{(const char*)l.down, (const char*)l.up, l.ids, l.ranks, l.scales, (float*)ws,
                       l.stride_down * es, l.stride_up * es, l.ld_down, l.ld_up,
                       (int)l.adapters, (int)l.rank, (int)pitch(l.rank), s.splits, s.z, odd_up};
    }
    q.b_kmajor = b == 'k';
    q.vec = vec;
    const mg::LoraShape shape = mg::shape_of(q, es == 4);
    const mg::Tile& tile = mg::kLoraTiles[(int)mg::lora_tile(shape)];
    if (mg::lora_grid(shape, tile) > mg::kMaxGridThreads / tile.threads) return GEMM_ERR_BAD_SHAPE;
    if (with && mg::ceil_div(M, q.shrink_rows) > mg::kMaxGridThreads / mg::kShrinkThreads) return GEMM_ERR_BAD_SHAPE;
    const int st = kLaunch[dtype](q, (hipStream_t)stream) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
    if (mg::log_enabled())
        std::fprintf(stderr, "mi355_gemm: lora %s M=%lld N=%lld K=%lld a=%c b=%c c=%c adapters=%lld rank=%lld %s\n",
                     mg::dtype_name(dtype), (long long)M, (long long)N, (long long)K, a, b, c, (long long)l.adapters,
                     (long long)l.rank, gemm_status_str(st));
    return st;
}

}  // namespace

extern "C" {

int gemm_run_lora(int64_t M, int64_t N, int64_t K, char a_major, char b_major, char c_major, int dtype, const void* A,
                  const void* B, void* C, int64_t lda, int64_t ldb, int64_t ldc, const gemm_lora_t* lora,
                  void* workspace, size_t workspace_bytes, void* stream)
{
    return run(M, N, K, a_major, b_major, c_major, dtype, A, B, C, lda, ldb, ldc, lora, workspace, workspace_bytes,
               stream);
}

int gemm_lora_workspace_size(int64_t M, int64_t N, int64_t K, int dtype, int64_t rank, size_t* bytes)
{
    if (!bytes) return GEMM_ERR_NULL_PTR;
    *bytes = 0;
    if (bad_shape(M, N, K, rank)) return GEMM_ERR_BAD_SHAPE;
    if (dtype < 0 || dtype >= GEMM_NUM_DTYPES) return GEMM_ERR_BAD_DTYPE;
    *bytes = (size_t)workspace_up_to(M, N, K, dtype, rank);
    return GEMM_OK;
}

}  // extern "C"
