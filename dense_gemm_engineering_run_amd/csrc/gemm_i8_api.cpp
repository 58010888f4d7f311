// gemm_i8_api.cpp -- the products of 8-bit integers of include/mi355_gemm.h:
// argument checks (all before any HIP call) and the launch.
#include <hip/hip_runtime.h>

#include <cctype>

#include "gemm_checks.hpp"
#include "gemm_i8.hpp"
#include "gemm_i8grad.hpp"

namespace {

using mg::Operand;

constexpr int64_t kTileRows = 256;     // rows a tile of any kernel here spans

// The longest sum of products of two 8-bit integers (at most 2^14 each) that
// 32 bits always hold.
constexpr int64_t kMaxSum = ((int64_t)1 << 17) - 1;

const char* const kTypeNames[GEMM_NUM_TYPES] = {"f32", "f16", "bf16"};

typedef hipError_t (*Launcher)(const mg::I8Call&, hipStream_t);
const Launcher kLaunch[GEMM_NUM_TYPES] = {mg::i8_f32, mg::i8_f16, mg::i8_bf16};
typedef hipError_t (*GradLauncher)(const mg::GradCall&, hipStream_t);
const GradLauncher kGradLaunch[GEMM_NUM_DTYPES] = {mg::i8grad_f32, mg::i8grad_f16_f32, mg::i8grad_bf16_bf16,
                                                   mg::i8grad_f16_f16, mg::i8grad_bf16_f32};

bool offsets_fit(const Operand& o) { return (kTileRows * o.ld + kTileRows) * o.es < ((int64_t)1 << 31); }

bool bad_shape(int64_t M, int64_t N, int64_t K)
{
    return M < 0 || N < 0 || K < 0 || M > mg::kMaxDim || N > mg::kMaxDim || K > mg::kMaxDim;
}

mg::Params params(int64_t M, int64_t N, int64_t K, const void* A, const void* B, void* C, int64_t lda, int64_t ldb,
                  int64_t ldc, bool c_vec)
{
    mg::Params p = {};
    p.A = (const char*)A;
    p.B = (const char*)B;
    p.C = (char*)C;
    p.M = (int)M; p.N = (int)N; p.K = (int)K;
    p.lda = lda; p.ldb = ldb; p.ldc = ldc;
    p.batch = 1;
    p.split = 1;
    p.alpha = 1.f;
    p.c_vec = c_vec;
    return p;
}

// Launches a product, its thin last rows and columns (i8_edges) after the rest.
hipError_t launch_parts(mg::I8Call q, int type, int eo, hipStream_t s)
{
    const mg::I8Edges edges = mg::i8_edges(mg::shape_of(q));
    // The last `left` rows or columns, which q loses.
    auto cut = [&](bool rows, int64_t left) {
        mg::I8Call rest = q;
        mg::Params& p = rest.p;
        const int64_t at = (rows ? p.M : p.N) - left;
        (rows ? q.p.M : q.p.N) = (int)at;
        (rows ? p.M : p.N) = (int)left;
        if (rows) {
            p.A += at * p.lda;
            p.a_bytes -= (uint64_t)(at * p.lda);
            if (rest.s.a) rest.s.a += at;
        } else {
            p.B += at * p.ldb;
            p.b_bytes -= (uint64_t)(at * p.ldb);
            if (rest.s.b) rest.s.b += at;
            if (p.bias) p.bias += at;
        }
        p.C += (rows ? at * p.ldc : at) * eo;
        p.c_vec = p.c_vec && (uintptr_t)p.C % 16 == 0;
        return rest;
    };
    mg::I8Call parts[2];
    int n = 0;
    if (edges.rows) parts[n++] = cut(true, edges.rows);
    if (edges.cols) parts[n++] = cut(false, edges.cols);
    hipError_t e = kLaunch[type](q, s);
    for (int i = 0; i < n && e == hipSuccess; ++i) e = kLaunch[type](parts[i], s);
    return e;
}

int run(int64_t M, int64_t N, int64_t K, char a, char b, char c, int type, const int8_t* A, const int8_t* B, void* C,
        int64_t lda, int64_t ldb, int64_t ldc, const float* scale_a, const float* scale_b, const gemm_epilogue_t* epi,
        void* stream)
{
    if (bad_shape(M, N, K) || K > kMaxSum) return GEMM_ERR_BAD_SHAPE;
    a = (char)std::tolower((unsigned char)a);
    b = (char)std::tolower((unsigned char)b);
    c = (char)std::tolower((unsigned char)c);
    if (a != 'k' || b != 'k' || c != 'n') return GEMM_ERR_BAD_MAJOR;
    if (type < 0 || type >= GEMM_NUM_TYPES) return GEMM_ERR_BAD_DTYPE;
    const int eo = type == GEMM_TYPE_F32 ? 4 : 2;
    const Operand oa = {A, M, K, lda, 1, 0, 1}, ob = {B, N, K, ldb, 1, 0, 1}, oc = {C, M, N, ldc, 1, 0, eo};
    if (!oa.lds_ok() || !ob.lds_ok() || !oc.lds_ok()) return GEMM_ERR_BAD_LD;

    if (M == 0 || N == 0) return GEMM_OK;
    const bool reads = K > 0;
    const float* const bias = epi ? epi->bias : nullptr;
    if ((reads && (!A || !B)) || !C) return GEMM_ERR_NULL_PTR;
    if (!oc.aligned(eo) || (((uintptr_t)scale_a | (uintptr_t)scale_b | (uintptr_t)bias) & 3)) return GEMM_ERR_MISALIGNED;
    const bool vec = reads && oa.aligned(16) && ob.aligned(16);
    const uint64_t cn = oc.bytes(false);
    const struct { const void* p; uint64_t n; } in[] = {
        {A, reads ? oa.bytes(vec) : 0}, {B, reads ? ob.bytes(vec) : 0}, {scale_a, (uint64_t)M * 4},
        {scale_b, (uint64_t)N * 4}, {bias, (uint64_t)N * 4}};
    for (const auto& x : in)
        if (mg::overlap(C, cn, x.p, x.n)) return GEMM_ERR_ALIAS;
    if (reads && (!offsets_fit(oa) || !offsets_fit(ob))) return GEMM_ERR_BAD_SHAPE;
    if (epi && (epi->activation < GEMM_ACT_NONE || epi->activation > GEMM_ACT_GELU)) return GEMM_ERR_BAD_EPILOGUE;

    mg::I8Call q = {};
    q.p = params(M, N, K, A, B, C, lda, ldb, ldc, oc.aligned(16));
    q.p.a_bytes = reads ? oa.bytes(vec) : 0;
    q.p.b_bytes = reads ? ob.bytes(vec) : 0;
    if (epi) {
        q.p.epi = epi->alpha != 1.f || epi->beta != 0.f || bias || epi->activation != GEMM_ACT_NONE;
        q.p.alpha = epi->alpha;
        q.p.beta = epi->beta;
        q.p.bias = bias;
        q.p.act = epi->activation;
    }
    q.s = mg::I8Scales{scale_a, scale_b};
    q.vec = vec;
    if (!mg::i8_fits(mg::shape_of(q))) return GEMM_ERR_BAD_SHAPE;
    hipError_t e = launch_parts(q, type, eo, (hipStream_t)stream);
    const int st = e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
    if (mg::log_enabled())
        std::fprintf(stderr, "mi355_gemm: i8 %s M=%lld N=%lld K=%lld %s\n", kTypeNames[type], (long long)M, (long long)N,
                     (long long)K, gemm_status_str(st));
    return st;
}

int run_grad(int64_t M, int64_t N, int64_t K, char a, char b, char c, int dtype, const void* A, const int8_t* Q, void* C,
             int64_t lda, int64_t ldq, int64_t ldc, const float* scales, int accumulate, void* stream)
{
    if (bad_shape(M, N, K)) return GEMM_ERR_BAD_SHAPE;
    a = (char)std::tolower((unsigned char)a);
    b = (char)std::tolower((unsigned char)b);
    c = (char)std::tolower((unsigned char)c);
    if ((a != 'k' && a != 'm') || b != 'n' || c != 'n') return GEMM_ERR_BAD_MAJOR;
    if (dtype < 0 || dtype >= GEMM_NUM_DTYPES) return GEMM_ERR_BAD_DTYPE;
    const int es = mg::in_bytes(dtype), eo = mg::out_bytes(dtype);
    const Operand oa = a == 'k' ? Operand{A, M, K, lda, 1, 0, es} : Operand{A, K, M, lda, 1, 0, es};
    const Operand oq = {Q, K, N, ldq, 1, 0, 1}, oc = {C, M, N, ldc, 1, 0, eo};
    if (!oa.lds_ok() || !oq.lds_ok() || !oc.lds_ok()) return GEMM_ERR_BAD_LD;

    if (M == 0 || N == 0) return GEMM_OK;
    const bool reads = K > 0;
    if ((reads && (!A || !Q || !scales)) || !C) return GEMM_ERR_NULL_PTR;
    if ((reads && (!oa.aligned(es) || ((uintptr_t)scales & 3))) || !oc.aligned(eo)) return GEMM_ERR_MISALIGNED;
    const bool vec = reads && oa.aligned(16) && oq.aligned(16);
    const uint64_t cn = oc.bytes(false);
    if (reads && (mg::overlap(C, cn, A, oa.bytes(vec)) || mg::overlap(C, cn, Q, oq.bytes(vec)) ||
                  mg::overlap(C, cn, scales, (uint64_t)K * 4)))
        return GEMM_ERR_ALIAS;
    if (reads && (!offsets_fit(oa) || !offsets_fit(oq))) return GEMM_ERR_BAD_SHAPE;
    if (!reads && accumulate) return GEMM_OK;                       // nothing to add

    mg::GradCall q = {};
    q.g.p = params(M, N, K, A, Q, C, lda, ldq, ldc, oc.aligned(16));
    q.g.p.a_bytes = reads ? oa.bytes(vec) : 0;
    q.g.p.b_bytes = reads ? oq.bytes(vec) : 0;
    q.g.p.epi = accumulate != 0;
    q.g.p.beta = accumulate ? 1.f : 0.f;
    q.g.scales = scales;
    q.a_kmajor = a == 'k';
    q.vec = vec;
    const mg::GradShape shape = mg::shape_of(q, eo == 4, dtype != GEMM_DTYPE_BF16_F32);
    const mg::Tile tile = mg::tile_of(mg::grad_tile(shape), shape.wide, shape.split_a, shape.a_kmajor);
    if (mg::grad_grid(shape, tile) > mg::kMaxGridThreads / tile.threads) return GEMM_ERR_BAD_SHAPE;
    const int st = kGradLaunch[dtype](q, (hipStream_t)stream) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
    if (mg::log_enabled())
        std::fprintf(stderr, "mi355_gemm: i8_grad %s M=%lld N=%lld K=%lld a=%c %s\n", mg::dtype_name(dtype), (long long)M,
                     (long long)N, (long long)K, a, gemm_status_str(st));
    return st;
}

}  // namespace

extern "C" {

int gemm_run_i8(int64_t M, int64_t N, int64_t K, char a_major, char b_major, char c_major, int type, const int8_t* A,
                const int8_t* B, void* C, int64_t lda, int64_t ldb, int64_t ldc, const float* scale_a,
                const float* scale_b, const gemm_epilogue_t* epilogue, void* stream)
{
    return run(M, N, K, a_major, b_major, c_major, type, A, B, C, lda, ldb, ldc, scale_a, scale_b, epilogue, stream);
}

int gemm_run_i8_grad(int64_t M, int64_t N, int64_t K, char a_major, char b_major, char c_major, int dtype, const void* A,
                     const int8_t* Q, void* C, int64_t lda, int64_t ldq, int64_t ldc, const float* scales, int accumulate,
                     void* stream)
{
    return run_grad(M, N, K, a_major, b_major, c_major, dtype, A, Q, C, lda, ldq, ldc, scales, accumulate, stream);
}

}  // extern "C"
