// Layout pass of the expert weights and its inverse (a test aid); the layout is in wq_experts.h.
// One thread per code word or scale, grid-strided. Run once per weight, and kept simple: 128 experts of 2048 x
// 1536 in 387 us, 1.1 TB/s of what is read and written, bound by its scattered accesses (a word written 64
// bytes from the next lane's, each source word read by four threads).
#include <cuda_runtime.h>
#include <cstdint>

#include "wq_experts.h"

namespace wq {

namespace {

constexpr int kThreads = 256;

// Column of the checkpoint's [K, N] weight that layout column v holds, or -1 for padding.
__device__ __forceinline__ int source_column(int v, int N, int gated) {
    if (v >= N) return -1;
    if (!gated) return v;
    return (v / 16) * 8 + (v & 7) + ((v & 8) ? N / 2 : 0);
}

__device__ __forceinline__ int nibble_of(int j) { return (j >> 1) + 4 * (j & 1); }  // (0,4,1,5,2,6,3,7)[j]

template <bool kUnpack>
__global__ void __launch_bounds__(kThreads) codes_kernel(uint32_t* __restrict__ Q, uint8_t* __restrict__ wp, int K, int N,
                                                         int gated, size_t stride, long long words_per_expert,
                                                         long long total) {
    const int KT = K / kTileK;
    for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < total;
         i += gridDim.x * static_cast<long long>(kThreads)) {
        const long long e = i / words_per_expert;
        const long long local = i % words_per_expert;
        // consecutive threads take consecutive columns: Q is read coalesced
        const int col = static_cast<int>(local % kExUnitN);
        const int cq = static_cast<int>((local / kExUnitN) % 16);
        const long long unit = local / (kExUnitN * 16);
        const int kb = static_cast<int>(unit % KT);
        const int u = static_cast<int>(unit / KT);
        const int c = cq >> 2, q = cq & 3;
        const int n = source_column(u * kExUnitN + col, N, gated);
        // the block's four words of Q for this column: rows 32c + 8i .. + 7, two of them each
        uint32_t* src = Q + (e * (K / 8) + static_cast<long long>(kb) * 16 + c * 4) * N + (n < 0 ? 0 : n);
        uint32_t* word = reinterpret_cast<uint32_t*>(wp + e * stride + unit * kExUnitBytes) +
                         (((col >> 3) * 32 + (col & 7) * 4 + q) * 4 + c);
        if (kUnpack) {
            if (n < 0) continue;
            // this thread writes Q's word i = q, whose codes lie in the words of all four q
            uint32_t out = 0;
            const uint32_t* first = word - q * 4;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                out |= ((first[(j >> 1) * 4] >> (4 * nibble_of(2 * q + (j & 1)))) & 0xFu) << (4 * j);
            src[static_cast<size_t>(q) * N] = out;
        } else {
            uint32_t out = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t in = n < 0 ? 0x88888888u : src[static_cast<size_t>(i) * N];
#pragma unroll
                for (int b = 0; b < 2; ++b) out |= ((in >> (4 * (2 * q + b))) & 0xFu) << (4 * nibble_of(2 * i + b));
            }
            *word = out;
        }
    }
}

template <bool kUnpack>
__global__ void __launch_bounds__(kThreads) scales_kernel(uint16_t* __restrict__ s, uint8_t* __restrict__ wp, int N,
                                                          int groups, int gated, size_t stride, size_t scale_offset,
                                                          long long per_expert, long long total) {
    for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < total;
         i += gridDim.x * static_cast<long long>(kThreads)) {
        const long long e = i / per_expert;
        const long long local = i % per_expert;
        const int col = static_cast<int>(local % kExUnitN);
        const long long ug = local / kExUnitN;
        const int grp = static_cast<int>(ug % groups);
        const int u = static_cast<int>(ug / groups);
        const int n = source_column(u * kExUnitN + col, N, gated);
        uint16_t* dst = reinterpret_cast<uint16_t*>(wp + e * stride + scale_offset) + ug * kExUnitN +
                        ((col & 7) * 4 + (col >> 4) * 2 + ((col >> 3) & 1));
        uint16_t* src = s + (e * groups + grp) * N + (n < 0 ? 0 : n);
        if (kUnpack) {
            if (n >= 0) *src = *dst;
        } else {
            *dst = n < 0 ? static_cast<uint16_t>(0) : *src;
        }
    }
}

template <bool kUnpack>
cudaError_t run(uint32_t* Q, uint16_t* s, int E, int K, int N, int g, int gated, uint8_t* wp, cudaStream_t st) {
    const size_t stride = ex_expert_stride(K, N, g);
    const long long words = static_cast<long long>(ex_units(N)) * (K / kTileK) * (kExUnitBytes / 4);
    const long long scales = static_cast<long long>(ex_units(N)) * (K / g) * kExUnitN;
    const long long most = 1 << 20;  // blocks; the kernels stride over the rest
    auto blocks = [&](long long n) {
        const long long b = (n + kThreads - 1) / kThreads;
        return static_cast<unsigned>(b < most ? b : most);
    };
    codes_kernel<kUnpack><<<blocks(words * E), kThreads, 0, st>>>(Q, wp, K, N, gated, stride, words, words * E);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    scales_kernel<kUnpack><<<blocks(scales * E), kThreads, 0, st>>>(s, wp, N, K / g, gated, stride,
                                                                   ex_scale_offset(K, N), scales, scales * E);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prepack_experts(const int32_t* Q, const uint16_t* s, int E, int K, int N, int g, int gated, void* Wp,
                                   cudaStream_t st) {
    return run<false>(const_cast<uint32_t*>(reinterpret_cast<const uint32_t*>(Q)), const_cast<uint16_t*>(s), E, K, N, g,
                      gated, static_cast<uint8_t*>(Wp), st);
}

cudaError_t launch_unpack_experts(const void* Wp, int E, int K, int N, int g, int gated, int32_t* Q, uint16_t* s,
                                  cudaStream_t st) {
    return run<true>(reinterpret_cast<uint32_t*>(Q), s, E, K, N, g, gated,
                     const_cast<uint8_t*>(static_cast<const uint8_t*>(Wp)), st);
}

}  // namespace wq
