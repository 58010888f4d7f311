// gemm_quant.hip -- gemm_quantize_rows and gemm_dequantize_rows: argument
// checks (all before any HIP call) and the launches.
#include <hip/hip_runtime.h>

#include "gemm_checks.hpp"
#include "gemm_quant.hpp"
#include "gemm_tiles.hpp"

namespace {

using mg::In;
using mg::Operand;
using mg::Quant;

template <class Kernel, class... More>
hipError_t launch(Kernel kernel, int64_t groups, int threads, hipStream_t s, Quant p, More... more)
{
    void* args[] = {&p, &more...};
    return hipLaunchKernel((const void*)kernel, dim3((unsigned)groups), dim3(threads), args, 0, s);
}

// How a call runs: waves a row and chunks a lane (0 waves: rows longer than
// registers hold).
struct QuantPlan {
    int waves, chunks;
    int64_t groups;
};
QuantPlan plan(int64_t M, int64_t K, int es)
{
    const int64_t lane_chunks = mg::ceil_div(K * es, 16 * 64);      // by one wave
    if (lane_chunks > 64) return {0, 0, M};
    if (M > 2048 && lane_chunks <= 8) return {1, lane_chunks <= 2 ? 2 : lane_chunks <= 4 ? 4 : 8, mg::ceil_div(M, 4)};
    const int64_t c = mg::ceil_div(lane_chunks, 4);
    return {4, c <= 2 ? 2 : c <= 4 ? 4 : c <= 8 ? 8 : 16, M};
}

template <In T>
hipError_t quantize(const Quant& p, const QuantPlan& q, hipStream_t s)
{
    using mg::quantize_kernel;
    switch (q.waves * 100 + q.chunks) {
    case 102: return launch(&quantize_kernel<T, 1, 2>, q.groups, 256, s, p);
    case 104: return launch(&quantize_kernel<T, 1, 4>, q.groups, 256, s, p);
    case 108: return launch(&quantize_kernel<T, 1, 8>, q.groups, 256, s, p);
    case 402: return launch(&quantize_kernel<T, 4, 2>, q.groups, 256, s, p);
    case 404: return launch(&quantize_kernel<T, 4, 4>, q.groups, 256, s, p);
    case 408: return launch(&quantize_kernel<T, 4, 8>, q.groups, 256, s, p);
    case 416: return launch(&quantize_kernel<T, 4, 16>, q.groups, 256, s, p);
    default: return launch(&mg::quantize_long_kernel<T>, q.groups, 256, s, p);
    }
}

struct RestorePlan {
    int spans;
    int64_t groups;
};
RestorePlan restore_plan(int64_t M, int64_t K, int es)
{
    const int64_t spans = mg::ceil_div(K, 64 * mg::kRestoreSteps * (16 / es));
    return {(int)spans, mg::ceil_div(M * spans, 4)};
}

template <In T>
hipError_t dequantize(const Quant& p, const RestorePlan& q, hipStream_t s)
{
    return launch(&mg::dequantize_kernel<T>, q.groups, 256, s, p, q.spans);
}

void log_call(const char* what, int64_t M, int64_t K, int type, int st)
{
    static const char* const names[] = {"f32", "f16", "bf16"};
    if (mg::log_enabled())
        std::fprintf(stderr, "mi355_gemm: %s %s M=%lld K=%lld %s\n", what, names[type], (long long)M, (long long)K,
                     gemm_status_str(st));
}

int run(bool to8, int64_t M, int64_t K, int type, const void* X, void* Y, float* scales, int64_t ldx, int64_t ldy,
        void* stream)
{
    if (M < 0 || K < 0 || M > mg::kMaxDim || K > mg::kMaxDim) return GEMM_ERR_BAD_SHAPE;
    if (type < 0 || type >= GEMM_NUM_TYPES) return GEMM_ERR_BAD_DTYPE;
    const int es = type == GEMM_TYPE_F32 ? 4 : 2;
    const Operand ox = {X, M, K, ldx, 1, 0, to8 ? es : 1};
    const Operand oy = {Y, M, K, ldy, 1, 0, to8 ? 1 : es};
    if (!ox.lds_ok() || !oy.lds_ok()) return GEMM_ERR_BAD_LD;
    if (M == 0 || (!to8 && K == 0)) return GEMM_OK;
    if ((K > 0 && (!X || !Y)) || !scales) return GEMM_ERR_NULL_PTR;
    if ((K > 0 && (!ox.aligned(ox.es) || !oy.aligned(oy.es))) || ((uintptr_t)scales & 3)) return GEMM_ERR_MISALIGNED;
    const uint64_t nx = ox.bytes(false), ny = oy.bytes(false), ns = (uint64_t)M * 4;
    if (mg::overlap(X, nx, Y, ny) || mg::overlap(scales, ns, Y, ny) || (to8 && mg::overlap(scales, ns, X, nx)))
        return GEMM_ERR_ALIAS;
    const Quant p = {(const char*)X, (char*)Y, scales, M, ldx, ldy, (int)K};
    hipError_t e;
    if (to8) {
        const QuantPlan q = plan(M, K, es);
        if (q.groups > mg::kMaxGridThreads / mg::kQuantThreads) return GEMM_ERR_BAD_SHAPE;
        e = type == GEMM_TYPE_F32 ? quantize<In::F32>(p, q, (hipStream_t)stream)
            : type == GEMM_TYPE_F16 ? quantize<In::F16>(p, q, (hipStream_t)stream)
                                    : quantize<In::BF16>(p, q, (hipStream_t)stream);
    } else {
        const RestorePlan q = restore_plan(M, K, es);
        if (q.groups > mg::kMaxGridThreads / mg::kQuantThreads) return GEMM_ERR_BAD_SHAPE;
        e = type == GEMM_TYPE_F32 ? dequantize<In::F32>(p, q, (hipStream_t)stream)
            : type == GEMM_TYPE_F16 ? dequantize<In::F16>(p, q, (hipStream_t)stream)
                                    : dequantize<In::BF16>(p, q, (hipStream_t)stream);
    }
    const int st = e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
    log_call(to8 ? "quantize_rows" : "dequantize_rows", M, K, type, st);
    return st;
}

}  // namespace

extern "C" {

int gemm_quantize_rows(int64_t M, int64_t K, int type, const void* X, int8_t* Q, float* scales, int64_t ldx, int64_t ldq,
                       void* stream)
{
    return run(true, M, K, type, X, Q, scales, ldx, ldq, stream);
}

int gemm_dequantize_rows(int64_t M, int64_t K, int type, const int8_t* Q, const float* scales, void* X, int64_t ldq,
                         int64_t ldx, void* stream)
{
    return run(false, M, K, type, Q, X, (float*)scales, ldq, ldx, stream);
}

}  // extern "C"
