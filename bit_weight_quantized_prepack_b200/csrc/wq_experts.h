// Geometry, prepacked layout and launch declarations of the expert operators (routing, lists,
// the experts' 4-bit products). Host and device.
//
// Prepacked expert weights: E buffers of `expert_stride` bytes, one per expert, each
//   codes:  unit (u, kb), u < NU = ceil(N/32), kb < K/128, at byte (u*(K/128) + kb) * 2048:
//     word ((rt*2 + h)*32 + 4*gc + q)*4 + c  (rt, h < 2, gc < 8, q, c < 4) holds the 8 codes of
//     column v = 32u + 16rt + 8h + gc, rows 128kb + 32c + 8i + 2q + b (i < 4, b < 2), code
//     2i + b at nibble (0, 4, 1, 5, 2, 6, 3, 7)[2i + b]: one mask gives the fp16 pair of two
//     consecutive rows;
//   scales: after the codes, [NU][K/g groups (1 for g == K)][32] fp16; column v of the unit at
//     position 4*gc + 2*rt + h.
//   The buffer is padded to 128 bytes. Columns past N hold code 8 and scale 0 (zero weights).
// Why this order: lane 4*gc + q of a warp takes the four words c = 0..3 of one (rt, h) with one
// 16-byte load, a warp's load is 512 contiguous bytes, and the pairs i of the words (h = 0, 1) are
// what that lane holds of the weight both as the 16-row operand of the warp's m16n8k16 (rows 2q,
// 2q + 1, 2q + 8, 2q + 9 of each 16) and of a 16-lane x 128-bit store to tensor memory (32-bit
// columns q, 4 + q, ...): K keeps its order, and the activations need no permutation. A lane's
// scales of its four columns are 8 contiguous bytes.
// Gated weights ([gate | up], N = 2I): column v is gate column 8(v/16) + v%8 when h = 0, up column
// the same when h = 1: a lane's two accumulator rows (gc and gc + 8) are the pair that
// silu(gate) * up needs.
#pragma once
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "wq_layout.h"

namespace wq {

constexpr int kExUnitN = 32;                             // columns of a unit
constexpr int kExUnitBytes = kExUnitN * kTileK / 2;      // 2048 bytes of codes
constexpr int kExMaxExperts = 1024;
constexpr int kExMaxTopK = 32;
constexpr int kExMaxGroups = 64;

__host__ __device__ inline int ex_units(int N) { return (N + kExUnitN - 1) / kExUnitN; }

inline size_t ex_scale_offset(int K, int N) {
    return static_cast<size_t>(ex_units(N)) * (K / kTileK) * kExUnitBytes;
}

inline size_t ex_expert_stride(int K, int N, int g) {
    const size_t b = ex_scale_offset(K, N) + static_cast<size_t>(ex_units(N)) * (K / g) * kExUnitN * 2;
    return (b + 127) / 128 * 128;
}

// What a call needs of the current device (wq_api.cu keeps it per device). WQ_OK or an error.
struct DeviceInfo {
    int num_sms;
    int* status;                    // device status word
    unsigned long long timeout_ns;  // limit of every device-side wait
};
int acquire_device(cudaStream_t stream, DeviceInfo* info);

struct RouteArgs {
    const void* logits;
    const float* bias;     // nullable
    int32_t* idx;
    float* w;
    int T, E, top_k;
    int fp32;              // logits type
    int sigmoid;
    int groups, top_groups, group_top;
    int renorm;
    double scale;
};

struct ExpertArgs {
    const uint16_t* a;         // activations [a_rows, K]
    const uint8_t* wp;
    const int32_t* offsets;    // [E + 1]
    const int32_t* rows;       // [pairs]
    uint16_t* y;               // [pairs, n_out]
    float* y32;                // not null: the products go here instead, not rounded to fp16 (gated 0)
    int* status;               // device status word
    size_t expert_stride, scale_offset;
    int pairs, a_div;          // pair p reads row p / a_div of a
    unsigned a_mul;            // ceil(2^32 / a_div): the division as a product (row_of_pair)
    int E, N, K, g;
    int gated;
};

cudaError_t configure_route();
// offsets and rows: null, or the lists of the choices too
cudaError_t launch_route(const RouteArgs& a, int32_t* offsets, int32_t* rows, cudaStream_t st);
cudaError_t launch_expert_lists(const int32_t* idx, int pairs, int E, int32_t* offsets, int32_t* rows,
                                cudaStream_t st);
cudaError_t launch_prepack_experts(const int32_t* Q, const uint16_t* s, int E, int K, int N, int g, int gated, void* Wp,
                                   cudaStream_t st);
cudaError_t launch_unpack_experts(const void* Wp, int E, int K, int N, int g, int gated, int32_t* Q, uint16_t* s,
                                  cudaStream_t st);
cudaError_t configure_expert_kernels();
cudaError_t configure_experts_large();
cudaError_t launch_experts(const ExpertArgs& a, const DeviceInfo& d, cudaStream_t st);
cudaError_t launch_experts_large(const ExpertArgs& a, const DeviceInfo& d, cudaStream_t st);
// Whether the combined product of so few pairs takes the form without lists and scratch.
bool experts_token_form(int pairs, int E);
// Y of args: [tokens, N]; a_div 1.
cudaError_t launch_experts_token(const ExpertArgs& a, const int32_t* idx, const float* w, int top_k, int num_sms,
                                 cudaStream_t st);
cudaError_t launch_combine_experts(const float* yp, const int32_t* idx, const float* w, int T, int top_k, int E,
                                   int N, uint16_t* Y, cudaStream_t st);

}  // namespace wq
