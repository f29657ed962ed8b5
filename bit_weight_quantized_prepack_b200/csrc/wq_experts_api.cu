// C ABI of the expert operators (declared in include/wq.h): argument checks and launches.
#include <cuda_runtime.h>
#include <cstdint>
#include <cstring>

#include "wq.h"
#include "wq_experts.h"

namespace {

using namespace wq;

constexpr long long kMaxTokens = 1ll << 24;
constexpr long long kMaxPairs = 1ll << 28;
constexpr int kMaxN = 0x7FFFFFFF - 255;  // columns rounded up to those of a tile must be an int

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int status_of(cudaError_t e) {
    if (e == cudaSuccess) return WQ_OK;
    cudaGetLastError();
    return WQ_ERR_CUDA;
}

// top_k may pass E here: of the experts that a token takes only some may be this device's. Only the
// routing, which chooses among E, wants top_k <= E.
int check_counts(int T, int E, int top_k) {
    if (T < 0 || E <= 0 || top_k <= 0) return WQ_ERR_INVALID_ARG;
    if (E > kExMaxExperts || top_k > kExMaxTopK || T > kMaxTokens || static_cast<long long>(T) * top_k > kMaxPairs)
        return WQ_ERR_UNSUPPORTED_SHAPE;
    return WQ_OK;
}

int check_weight(int E, int K, int N, int g, int gated) {
    if (E <= 0 || K <= 0 || N <= 0 || (gated != 0 && gated != 1)) return WQ_ERR_INVALID_ARG;
    if (E > kExMaxExperts || !shape_ok(K, N) || (gated && N % 16) || N > kMaxN) return WQ_ERR_UNSUPPORTED_SHAPE;
    if (scale_slots(K, g) < 0) return WQ_ERR_INVALID_ARG;
    return WQ_OK;
}

int check_lists(const int32_t* offsets, const int32_t* rows) {
    if (!offsets || !rows) return WQ_ERR_INVALID_ARG;
    if (!aligned(offsets, 4) || !aligned(rows, 4)) return WQ_ERR_MISALIGNED;
    return WQ_OK;
}

ExpertArgs product_args(const uint16_t* A, const void* Wp, const int32_t* offsets, const int32_t* rows, uint16_t* Y,
                        int T, int E, int top_k, int a_div, int N, int K, int g, int gated, const DeviceInfo& d) {
    ExpertArgs a;
    std::memset(&a, 0, sizeof(a));
    a.a = A;
    a.wp = static_cast<const uint8_t*>(Wp);
    a.offsets = offsets;
    a.rows = rows;
    a.y = Y;
    a.status = d.status;
    a.expert_stride = ex_expert_stride(K, N, g);
    a.scale_offset = ex_scale_offset(K, N);
    a.pairs = T * top_k;
    a.a_div = a_div;
    a.a_mul = static_cast<unsigned>(((1ull << 32) + a_div - 1) / a_div);  // unused for a_div == 1
    a.E = E;
    a.N = N;
    a.K = K;
    a.g = g;
    a.gated = gated;
    return a;
}

}  // namespace

extern "C" {

int wq_route_experts(const void* logits, int logits_fp32, const float* bias, int T, int E, int top_k, int score,
                     int groups, int top_groups, int group_top, int renorm, double scale, int32_t* idx, float* w,
                     int32_t* offsets, int32_t* rows, void* stream) {
    if (E > 0 && top_k > E) return WQ_ERR_INVALID_ARG;
    int rc = check_counts(T, E, top_k);
    if (rc) return rc;
    if (logits_fp32 < 0 || logits_fp32 > 1 || score < 0 || score > 1 || renorm < 0 || renorm > 1 || group_top < 1 ||
        group_top > 2 || groups < 1 || E % groups || top_groups < 1 || top_groups > groups)
        return WQ_ERR_INVALID_ARG;
    if (static_cast<long long>(top_groups) * (E / groups) < top_k) return WQ_ERR_INVALID_ARG;
    if (groups > kExMaxGroups) return WQ_ERR_UNSUPPORTED_SHAPE;
    if ((rows && !offsets) || (T > 0 && offsets && !rows)) return WQ_ERR_INVALID_ARG;
    if (T > 0 && (!logits || !idx || !w)) return WQ_ERR_INVALID_ARG;
    if (!aligned(logits, logits_fp32 ? 4 : 2) || !aligned(bias, 4) || !aligned(idx, 4) || !aligned(w, 4) ||
        !aligned(offsets, 4) || !aligned(rows, 4))
        return WQ_ERR_MISALIGNED;
    if (T == 0 && !offsets) return WQ_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    DeviceInfo d;
    rc = acquire_device(st, &d);
    if (rc) return rc;
    if (T > 0) {
        RouteArgs a;
        std::memset(&a, 0, sizeof(a));
        a.logits = logits;
        a.bias = bias;
        a.idx = idx;
        a.w = w;
        a.T = T;
        a.E = E;
        a.top_k = top_k;
        a.fp32 = logits_fp32;
        a.sigmoid = score;
        a.groups = groups;
        a.top_groups = top_groups;
        a.group_top = group_top;
        a.renorm = renorm;
        a.scale = scale;
        return status_of(launch_route(a, offsets, rows, st));
    }
    return status_of(launch_expert_lists(idx, 0, E, offsets, rows, st));
}

int wq_expert_lists(const int32_t* idx, int T, int E, int top_k, int32_t* offsets, int32_t* rows, void* stream) {
    int rc = check_counts(T, E, top_k);
    if (rc) return rc;
    if (!offsets || (T > 0 && (!idx || !rows))) return WQ_ERR_INVALID_ARG;
    if (!aligned(idx, 4) || !aligned(offsets, 4) || !aligned(rows, 4)) return WQ_ERR_MISALIGNED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    DeviceInfo d;
    rc = acquire_device(st, &d);
    if (rc) return rc;
    return status_of(launch_expert_lists(idx, T * top_k, E, offsets, rows, st));
}

size_t wq_prepacked_bytes_experts(int E, int K, int N, int g) {
    if (check_weight(E, K, N, g, 0) != WQ_OK) return 0;
    return static_cast<size_t>(E) * ex_expert_stride(K, N, g);
}

int wq_prepack_experts(const int32_t* Q, const uint16_t* s, int E, int K, int N, int g, int gated, void* Wp,
                       void* stream) {
    int rc = check_weight(E, K, N, g, gated);
    if (rc) return rc;
    if (!Q || !s || !Wp) return WQ_ERR_INVALID_ARG;
    if (!aligned(Q, 16) || !aligned(s, 16) || !aligned(Wp, 16)) return WQ_ERR_MISALIGNED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    DeviceInfo d;
    rc = acquire_device(st, &d);
    if (rc) return rc;
    return status_of(launch_prepack_experts(Q, s, E, K, N, g, gated, Wp, st));
}

int wq_unpack_experts(const void* Wp, int E, int K, int N, int g, int gated, int32_t* Q_out, uint16_t* s_out,
                      void* stream) {
    int rc = check_weight(E, K, N, g, gated);
    if (rc) return rc;
    if (!Wp || !Q_out || !s_out) return WQ_ERR_INVALID_ARG;
    if (!aligned(Wp, 16) || !aligned(Q_out, 16) || !aligned(s_out, 16)) return WQ_ERR_MISALIGNED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    DeviceInfo d;
    rc = acquire_device(st, &d);
    if (rc) return rc;
    return status_of(launch_unpack_experts(Wp, E, K, N, g, gated, Q_out, s_out, st));
}

int wq_gemm_w4a16_experts(const uint16_t* A, const void* Wp, const int32_t* offsets, const int32_t* rows, uint16_t* Y,
                          int T, int E, int top_k, int N, int K, int g, int gated, void* stream) {
    int rc = check_counts(T, E, top_k);
    if (rc == WQ_OK) rc = check_weight(E, K, N, g, gated);
    if (rc) return rc;
    if (!Wp) return WQ_ERR_INVALID_ARG;
    if (!aligned(Wp, 16)) return WQ_ERR_MISALIGNED;
    if (T == 0) return WQ_OK;
    if (!A || !Y) return WQ_ERR_INVALID_ARG;
    rc = check_lists(offsets, rows);
    if (rc) return rc;
    if (!aligned(A, 16) || !aligned(Y, 16)) return WQ_ERR_MISALIGNED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    DeviceInfo d;
    rc = acquire_device(st, &d);
    if (rc) return rc;
    return status_of(launch_experts(product_args(A, Wp, offsets, rows, Y, T, E, top_k, top_k, N, K, g, gated, d), d, st));
}

size_t wq_experts_scratch_bytes(int T, int E, int top_k, int N) {
    if (check_counts(T, E, top_k) != WQ_OK || N <= 0 || N % 8 || experts_token_form(T * top_k, E)) return 0;
    return static_cast<size_t>(T) * top_k * N * sizeof(float);
}

int wq_gemm_w4a16_experts_combine(const uint16_t* H, const void* Wp, const int32_t* idx, const float* w,
                                  const int32_t* offsets, const int32_t* rows, uint16_t* Y, void* scratch,
                                  size_t scratch_bytes, int T, int E, int top_k, int N, int K, int g, void* stream) {
    int rc = check_counts(T, E, top_k);
    if (rc == WQ_OK) rc = check_weight(E, K, N, g, 0);
    if (rc) return rc;
    if (!Wp) return WQ_ERR_INVALID_ARG;
    if (!aligned(Wp, 16)) return WQ_ERR_MISALIGNED;
    if (T == 0) return WQ_OK;
    const size_t need = wq_experts_scratch_bytes(T, E, top_k, N);
    if (!H || !Y || !idx || !w || (need && !scratch)) return WQ_ERR_INVALID_ARG;
    rc = check_lists(offsets, rows);
    if (rc) return rc;
    if (!aligned(H, 16) || !aligned(Y, 16) || !aligned(scratch, 16) || !aligned(idx, 4) || !aligned(w, 4))
        return WQ_ERR_MISALIGNED;
    if (scratch_bytes < need) return WQ_ERR_INVALID_ARG;
    // one thread of the summing kernel per 4 columns of a token
    if (static_cast<long long>(T) * (N / 4) >= (1ll << 31) * 128) return WQ_ERR_UNSUPPORTED_SHAPE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    DeviceInfo d;
    rc = acquire_device(st, &d);
    if (rc) return rc;
    if (experts_token_form(T * top_k, E))
        return status_of(launch_experts_token(product_args(H, Wp, offsets, rows, Y, T, E, top_k, 1, N, K, g, 0, d), idx, w,
                                              top_k, d.num_sms, st));
    ExpertArgs a = product_args(H, Wp, offsets, rows, nullptr, T, E, top_k, 1, N, K, g, 0, d);
    a.y32 = static_cast<float*>(scratch);
    rc = status_of(launch_experts(a, d, st));
    if (rc) return rc;
    return status_of(launch_combine_experts(a.y32, idx, w, T, top_k, E, N, Y, st));
}

}  // extern "C"
