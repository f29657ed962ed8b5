// The experts' 4-bit products: y[p] = a[p / a_div] . W[e(p)] for every pair p of the lists,
// W = (q - 8) * s, fp32 sums, one rounding to fp16; gated: silu(gate) * up in the epilogue.
// And the weighted sum of a token's pairs after the down product.
//
// experts_kernel (few rows per expert). Tile: 32 columns of one expert x up to 8*NB of its rows,
// all of K. Eight warps take the tile's 128-row k-blocks in turn; a warp needs nothing from the
// others until the sums are added, in the order of the warps, at the end. Every lane copies with
// cp.async the codes and scales that it will itself multiply and its share of the activations (four
// 16-byte chunks of codes, 4*NB of activations per k-block) into its warp's ring in shared memory,
// so that the ring needs no barrier beyond the warp's. The weight is the 16-row operand of m16n8k16 (exact fp16
// q - 8), the tokens are its 8 columns; each group's fp32 partial is scaled in fp32, so no weight
// is rounded.
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "wq_experts.h"
#include "wq_experts_dev.cuh"
#include "wq_ptx.cuh"

namespace wq {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four 8 x 8 fp16 matrices: lane l gives the address of row l % 8 of matrix l / 8 and receives
// elements (l / 4, 2 (l % 4)) and the next of each.
__device__ __forceinline__ uint4 ldmatrix4(const void* row) {
    uint4 v;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(smem_addr(row))
                 : "memory");
    return v;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// SL: scales per k-block and column (1, 2 or 4 groups of a k-block; 0: per-column, g == K)
template <int NB, int SL>
__global__ void __launch_bounds__(kThreads) experts_kernel(ExpertArgs a, int stages) {
    extern __shared__ uint8_t smem_raw[];
    constexpr int kStage = (4 + 4 * NB) * 512 + (SL ? SL : 1) * 256;
    constexpr int kRows = 8 * NB;
    __shared__ int s_start[kExMaxExperts + 1], s_tiles[kExMaxExperts + 1], s_scratch[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q = lane & 3, gc = lane >> 2;
    uint8_t* ring = smem_raw + static_cast<size_t>(warp) * stages * kStage;
    float* red = reinterpret_cast<float*>(smem_raw + static_cast<size_t>(kWarps) * stages * kStage);
    expert_table<kThreads>(a.offsets, a.E, a.pairs, kRows, s_start, s_tiles, s_scratch);

    const int KT = a.K / kTileK, NU = ex_units(a.N);
    const long long tiles = static_cast<long long>(s_tiles[a.E]) * NU;
    const int n_out = a.gated ? a.N / 2 : a.N;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        // expert of the tile: the last e with s_tiles[e] * NU <= tile
        const int rt_all = static_cast<int>(tile / NU);
        int lo = 0, hi = a.E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_tiles[mid] <= rt_all) lo = mid; else hi = mid;
        }
        const int e = lo;
        const int ert = s_tiles[e + 1] - s_tiles[e];
        const long long local = tile - static_cast<long long>(s_tiles[e]) * NU;
        const int u = static_cast<int>(local / ert), rt = static_cast<int>(local % ert);
        const int row0 = s_start[e] + rt * kRows;
        const int nrows = min(kRows, s_start[e + 1] - row0);
        const uint8_t* we = a.wp + static_cast<size_t>(e) * a.expert_stride;
        const uint8_t* codes = we + static_cast<size_t>(u) * KT * kExUnitBytes + lane * 16;
        const uint8_t* scales = we + a.scale_offset + static_cast<size_t>(u) * (a.K / a.g) * (kExUnitN * 2) + gc * 8;
        const uint16_t* arow[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int r = b * 8 + gc;
            arow[b] = nullptr;
            if (r < nrows) {
                const int p = __ldg(a.rows + row0 + r);
                if (static_cast<unsigned>(p) < static_cast<unsigned>(a.pairs))
                    arow[b] = a.a + static_cast<size_t>(row_of_pair(p, a)) * a.K + q * 8;
                else
                    atomicCAS(a.status, 0, 1 /* WQ_ERR_INVALID_ARG */);
            }
        }
        auto issue = [&](int kb, int slot) {
            if (kb < KT) {
                uint8_t* st = ring + slot * kStage;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    cp_async16(st + i * 512 + lane * 16, codes + static_cast<size_t>(kb) * kExUnitBytes + i * 512);
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    if (arow[b]) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            cp_async16(st + (4 + b * 4 + c) * 512 + q * 128 + gc * 16, arow[b] + kb * kTileK + c * 32);
                    }
                if (SL) {
#pragma unroll
                    for (int i = 0; i < SL; ++i) {
                        const int grp = SL == 1 ? kb * kTileK / a.g : kb * SL + i;
                        cp_async8(st + (4 + 4 * NB) * 512 + i * 256 + lane * 8, scales + static_cast<size_t>(grp) * (kExUnitN * 2));
                    }
                }
            }
            cp_async_commit();
        };
        float acc[2][NB][4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][b][i] = 0.f;
        int kb_issue = warp;
        for (int s = 0; s < stages - 1; ++s, kb_issue += kWarps) issue(kb_issue, s);
        int slot = 0;
        for (int kb = warp; kb < KT; kb += kWarps) {
            issue(kb_issue, slot == 0 ? stages - 1 : slot - 1);
            kb_issue += kWarps;
            // all groups but the newest stages - 1 have arrived
            if (stages == 2) cp_async_wait<1>(); else if (stages == 3) cp_async_wait<2>(); else cp_async_wait<3>();
            __syncwarp();
            const uint8_t* st = ring + slot * kStage;
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4*>(st + i * 512 + lane * 16);
            float d[2][NB][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (SL && c % (4 / (SL ? SL : 1)) == 0) {
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i) d[r][b][i] = 0.f;
                }
                uint4 x[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    // rows behind the tile's last are not copied: what lies there meets no stored sum
                    x[b] = ldmatrix4(st + (4 + b * 4 + c) * 512 + lane * 16);
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t p0[4], p1[4];
                    const uint4 w0 = w[2 * r], w1 = w[2 * r + 1];
                    dequant8(c == 0 ? w0.x : c == 1 ? w0.y : c == 2 ? w0.z : w0.w, p0);
                    dequant8(c == 0 ? w1.x : c == 1 ? w1.y : c == 2 ? w1.z : w1.w, p1);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        float (&t)[4] = SL ? d[r][b] : acc[r][b];
                        mma_16816(t, p0[0], p1[0], p0[1], p1[1], x[b].x, x[b].y);
                        mma_16816(t, p0[2], p1[2], p0[3], p1[3], x[b].z, x[b].w);
                    }
                }
                if (SL && c % (4 / (SL ? SL : 1)) == 4 / (SL ? SL : 1) - 1) {
                    const uint2 sv = *reinterpret_cast<const uint2*>(st + (4 + 4 * NB) * 512 +
                                                                     (c / (4 / (SL ? SL : 1))) * 256 + lane * 8);
                    const float2 s0 = __half22float2(*reinterpret_cast<const __half2*>(&sv.x));
                    const float2 s1 = __half22float2(*reinterpret_cast<const __half2*>(&sv.y));
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        acc[0][b][0] += s0.x * d[0][b][0];
                        acc[0][b][1] += s0.x * d[0][b][1];
                        acc[0][b][2] += s0.y * d[0][b][2];
                        acc[0][b][3] += s0.y * d[0][b][3];
                        acc[1][b][0] += s1.x * d[1][b][0];
                        acc[1][b][1] += s1.x * d[1][b][1];
                        acc[1][b][2] += s1.y * d[1][b][2];
                        acc[1][b][3] += s1.y * d[1][b][3];
                    }
                }
            }
            slot = slot + 1 == stages ? 0 : slot + 1;
        }
        cp_async_wait<0>();
        // sums of the warps: red[warp][token][column]
        float* mine = red + warp * (kRows * 33);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mine[(b * 8 + 2 * q + (i & 1)) * 33 + r * 16 + (i >> 1) * 8 + gc] = acc[r][b][i];
        __syncthreads();
        const int out_cols = a.gated ? 16 : 32;
        for (int i = tid; i < nrows * out_cols; i += kThreads) {
            const int m = i / out_cols, col = i % out_cols;
            const int p = __ldg(a.rows + row0 + m);
            const int v0 = a.gated ? (col >> 3) * 16 + (col & 7) : col;
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s0 += red[w * (kRows * 33) + m * 33 + v0];
            if (a.gated) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s1 += red[w * (kRows * 33) + m * 33 + v0 + 8];
            }
            if (!SL) {
                const __half* cs = reinterpret_cast<const __half*>(we + a.scale_offset) + static_cast<size_t>(u) * kExUnitN;
                const int at = (v0 & 7) * 4 + (v0 >> 4) * 2 + ((v0 >> 3) & 1);
                s0 *= __half2float(cs[at]);
                if (a.gated) s1 *= __half2float(cs[at + 1]);
            }
            const float out = a.gated ? silu_mul(s0, s1) : s0;
            const int n = u * out_cols + col;
            if (n < n_out && static_cast<unsigned>(p) < static_cast<unsigned>(a.pairs))
                a.y[static_cast<size_t>(p) * n_out + n] = __half_as_ushort(__float2half_rn(out));
        }
        __syncthreads();
    }
}

// Y[t] = sum over j of w[t, j] * yp[t * top_k + j], in the order of j, fp32; a choice outside
// [0, E) adds nothing. One thread per 8 columns of a token.
__global__ void __launch_bounds__(256) combine_kernel(const uint16_t* __restrict__ yp, const int32_t* __restrict__ idx,
                                                      const float* __restrict__ w, int top_k, int E, int N,
                                                      uint16_t* __restrict__ Y, long long total) {
    const long long i = blockIdx.x * 256ll + threadIdx.x;
    if (i >= total) return;
    const int per_row = N / 8;
    const long long t = i / per_row;
    const int n = static_cast<int>(i % per_row) * 8;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < top_k; ++j) {
        const long long p = t * top_k + j;
        if (static_cast<unsigned>(__ldg(idx + p)) >= static_cast<unsigned>(E)) continue;
        const float wj = __ldg(w + p);
        const uint4 v = *reinterpret_cast<const uint4*>(yp + p * N + n);
        const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = __half22float2(h[k]);
            acc[2 * k] += wj * f.x;
            acc[2 * k + 1] += wj * f.y;
        }
    }
    uint4 out;
    __half2* o = reinterpret_cast<__half2*>(&out);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = __floats2half2_rn(acc[2 * k], acc[2 * k + 1]);
    *reinterpret_cast<uint4*>(Y + t * N + n) = out;
}

template <int NB, int SL>
struct Small {
    static constexpr int kStage = (4 + 4 * NB) * 512 + (SL ? SL : 1) * 256;
    static constexpr int kStages = NB == 1 ? 3 : 2;
    static constexpr int kSmem = kWarps * kStages * kStage + kWarps * 8 * NB * 33 * 4;
    static cudaError_t configure() {
        return cudaFuncSetAttribute(experts_kernel<NB, SL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    }
    static cudaError_t launch(const ExpertArgs& a, int num_sms, cudaStream_t st) {
        // at most every pair a tile of its own; CTAs past the last tile return at once
        const long long most = static_cast<long long>(a.pairs) * ex_units(a.N);
        const int want = num_sms * (kSmem <= 110 * 1024 ? 2 : 1);
        experts_kernel<NB, SL><<<static_cast<unsigned>(most < want ? most : want), kThreads, kSmem, st>>>(a, kStages);
        return cudaGetLastError();
    }
};

template <int NB>
cudaError_t configure_nb() {
    cudaError_t e = Small<NB, 0>::configure();
    if (e == cudaSuccess) e = Small<NB, 1>::configure();
    if (e == cudaSuccess) e = Small<NB, 2>::configure();
    if (e == cudaSuccess) e = Small<NB, 4>::configure();
    return e;
}

template <int NB>
cudaError_t launch_nb(const ExpertArgs& a, int num_sms, cudaStream_t st) {
    if (a.g == a.K) return Small<NB, 0>::launch(a, num_sms, st);
    if (a.g == 64) return Small<NB, 2>::launch(a, num_sms, st);
    if (a.g == 32) return Small<NB, 4>::launch(a, num_sms, st);
    return Small<NB, 1>::launch(a, num_sms, st);
}

}  // namespace

cudaError_t configure_expert_kernels() {
    cudaError_t e = configure_nb<1>();
    if (e == cudaSuccess) e = configure_nb<2>();
    if (e == cudaSuccess) e = configure_nb<4>();
    if (e == cudaSuccess) e = configure_experts_large();
    return e;
}

cudaError_t launch_experts(const ExpertArgs& a, const DeviceInfo& d, cudaStream_t st) {
    const long long per_expert = (static_cast<long long>(a.pairs) + a.E - 1) / a.E;
    const int num_sms = d.num_sms;
    if (per_expert > 16) return launch_experts_large(a, d, st);
    if (per_expert <= 4) return launch_nb<1>(a, num_sms, st);
    if (per_expert <= 8) return launch_nb<2>(a, num_sms, st);
    return launch_nb<4>(a, num_sms, st);
}

cudaError_t launch_combine_experts(const uint16_t* yp, const int32_t* idx, const float* w, int T, int top_k, int E,
                                   int N, uint16_t* Y, cudaStream_t st) {
    const long long total = static_cast<long long>(T) * (N / 8);
    combine_kernel<<<static_cast<unsigned>((total + 255) / 256), 256, 0, st>>>(yp, idx, w, top_k, E, N, Y, total);
    return cudaGetLastError();
}

}  // namespace wq
