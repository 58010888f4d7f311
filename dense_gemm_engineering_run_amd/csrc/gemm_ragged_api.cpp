// gemm_ragged_api.cpp -- the grouped entry points of include/mi355_gemm.h:
// argument checks (all before any HIP call) and the launch.
#include <hip/hip_runtime.h>

#include <cctype>

#include "gemm_checks.hpp"
#include "gemm_ragged.hpp"

namespace {

using mg::Operand;

// Rows a tile of any kernel here spans along an operand's outer index, for the
// bound on its 32-bit byte offsets.
constexpr int64_t kTileRows = 256;

typedef hipError_t (*Launcher)(const mg::RaggedCall&, hipStream_t);
const Launcher kLaunch[GEMM_NUM_DTYPES] = {mg::ragged_f32, mg::ragged_f16_f32, mg::ragged_bf16_bf16,
                                           mg::ragged_f16_f16, mg::ragged_bf16_f32};

bool offsets_fit(const Operand& o) { return (kTileRows * o.ld + kTileRows) * o.es < ((int64_t)1 << 31); }

// by_rows: C[m][:] = A[m][:] * B_g^T; else C_g = (A * B^T over the k of g).
int run(bool by_rows, int64_t M, int64_t N, int64_t K, char a, char b, char c, int dtype, const void* A, const void* B,
        void* C, int64_t lda, int64_t ldb, int64_t ldc, int64_t groups, int64_t stride, const int32_t* ends,
        int accumulate, void* stream)
{
    if (M < 0 || N < 0 || K < 0 || M > mg::kMaxDim || N > mg::kMaxDim || K > mg::kMaxDim) return GEMM_ERR_BAD_SHAPE;
    if (groups < 0 || groups > mg::kMaxGroups) return GEMM_ERR_BAD_SHAPE;
    a = (char)std::tolower((unsigned char)a);
    b = (char)std::tolower((unsigned char)b);
    c = (char)std::tolower((unsigned char)c);
    if (by_rows ? (a != 'k' || (b != 'k' && b != 'n') || c != 'n') : (a != 'm' || b != 'n' || (c != 'n' && c != 'm')))
        return GEMM_ERR_BAD_MAJOR;
    if (dtype < 0 || dtype >= GEMM_NUM_DTYPES) return GEMM_ERR_BAD_DTYPE;
    const int es = mg::in_bytes(dtype), eo = mg::out_bytes(dtype);

    const Operand oa = a == 'k' ? Operand{A, M, K, lda, 1, 0, es} : Operand{A, K, M, lda, 1, 0, es};
    const int64_t nb = by_rows ? groups : 1, nc = by_rows ? 1 : groups;
    const Operand ob = b == 'k' ? Operand{B, N, K, ldb, nb, by_rows ? stride : 0, es}
                                : Operand{B, K, N, ldb, nb, by_rows ? stride : 0, es};
    const Operand oc = c == 'n' ? Operand{C, M, N, ldc, nc, by_rows ? 0 : stride, eo}
                                : Operand{C, N, M, ldc, nc, by_rows ? 0 : stride, eo};
    if (!oa.lds_ok() || !ob.lds_ok() || !oc.lds_ok()) return GEMM_ERR_BAD_LD;
    if (!by_rows && groups > 1 && (uint64_t)stride < oc.span()) return GEMM_ERR_BAD_LD;   // C_g may not overlap

    if (M == 0 || N == 0 || groups == 0) return GEMM_OK;
    const bool reads = K > 0;
    if ((reads && (!A || !B)) || !C || !ends) return GEMM_ERR_NULL_PTR;
    if ((reads && (!oa.aligned(es) || !ob.aligned(es))) || !oc.aligned(eo) || ((uintptr_t)ends & 3))
        return GEMM_ERR_MISALIGNED;
    const bool vec = !reads || (oa.aligned(16) && ob.aligned(16));
    const uint64_t cn = oc.bytes(false);
    if (mg::overlap(C, cn, ends, (uint64_t)groups * 4) ||
        (reads && (mg::overlap(C, cn, A, oa.bytes(vec)) || mg::overlap(C, cn, B, ob.bytes(vec)))))
        return GEMM_ERR_ALIAS;
    if (reads && (!offsets_fit(oa) || !offsets_fit(ob))) return GEMM_ERR_BAD_SHAPE;
    if (!reads && accumulate) return GEMM_OK;                       // nothing to add

    mg::RaggedCall q = {};
    mg::Params& p = q.p;
    p.A = (const char*)A;
    p.B = (const char*)B;
    p.C = (char*)C;
    p.M = (int)M; p.N = (int)N; p.K = (int)K;
    p.lda = lda; p.ldb = ldb; p.ldc = ldc;
    p.batch = 1;
    p.split = 1;
    p.alpha = 1.f;
    if (!by_rows && c == 'm') {      // C_g^T = B A^T
        std::swap(p.A, p.B);
        std::swap(p.M, p.N);
        std::swap(p.lda, p.ldb);
    }
    p.epi = !by_rows && accumulate;
    p.beta = p.epi ? 1.f : 0.f;
    p.c_vec = oc.aligned(16);
    // One matrix B_g (the kernel sets what else depends on the group).
    if (by_rows && reads) p.b_bytes = Operand{B, ob.outer, ob.inner, ldb, 1, 0, es}.bytes(vec);
    q.r = mg::Ragged{ends, (int)groups, (int)(by_rows ? M : K), stride * (by_rows ? es : eo)};
    q.by_rows = by_rows;
    q.b_kmajor = b == 'k';
    q.vec = vec;
    const mg::RaggedShape shape = mg::shape_of(q, es == 4);
    const mg::Tile& tile = mg::kRaggedTiles[(int)mg::ragged_tile(shape)];
    if (mg::ragged_grid(shape, tile) > mg::kMaxGridThreads / tile.threads) return GEMM_ERR_BAD_SHAPE;
    const int st = kLaunch[dtype](q, (hipStream_t)stream) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
    if (mg::log_enabled())
        std::fprintf(stderr, "mi355_gemm: %s %s M=%lld N=%lld K=%lld a=%c b=%c c=%c groups=%lld %s\n",
                     by_rows ? "grouped" : "grouped_k", mg::dtype_name(dtype), (long long)M, (long long)N, (long long)K,
                     a, b, c, (long long)groups, gemm_status_str(st));
    return st;
}

}  // namespace

extern "C" {

int gemm_run_grouped(int64_t M, int64_t N, int64_t K, char a_major, char b_major, char c_major, int dtype,
                     const void* A, const void* B, void* C, int64_t lda, int64_t ldb, int64_t ldc, int64_t groups,
                     int64_t stride_b, const int32_t* ends, void* stream)
{
    return run(true, M, N, K, a_major, b_major, c_major, dtype, A, B, C, lda, ldb, ldc, groups, stride_b, ends, 0,
               stream);
}

int gemm_run_grouped_k(int64_t M, int64_t N, int64_t K, char a_major, char b_major, char c_major, int dtype,
                       const void* A, const void* B, void* C, int64_t lda, int64_t ldb, int64_t ldc, int64_t groups,
                       int64_t stride_c, const int32_t* ends, int accumulate, void* stream)
{
    return run(false, M, N, K, a_major, b_major, c_major, dtype, A, B, C, lda, ldb, ldc, groups, stride_c, ends,
               accumulate, stream);
}

}  // extern "C"
