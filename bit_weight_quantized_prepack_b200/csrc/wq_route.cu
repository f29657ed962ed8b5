// Routing of tokens to experts, and the lists of (token, choice) pairs by expert.
//
// route_kernel: one warp per token; lane l holds experts l, l + 32, ... With p the scores
// (softmax or sigmoid of the logits) and c = p + bias, the groups' values and the choice go by c
// in 64 bits: two experts' scores may lie closer than 32 bits hold, and a choice is a whole
// number that a rounding must not decide. Without a bias the choice goes by the logits
// themselves, whose order is that of the scores. Keys are mapped to unsigned integers of the
// same order, so that a warp's maximum is one reduction instruction per 32 bits; among equal keys
// the lowest expert wins. An expert whose logit or bias is not finite has key 0, below every
// finite one, and is never chosen.
//
// lists_kernel: one CTA per expert. Its warps own consecutive runs of the pairs: a first pass
// counts the pairs of lower experts (the expert's place in `rows`) and each warp's own pairs, a
// second writes them in order. No atomics: the lists are the same every time.
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "wq_experts.h"

namespace wq {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kRouteWarps = 4;
constexpr int kListThreads = 512;

__device__ __forceinline__ unsigned long long key_of(double v) {
    const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(v + 0.0));  // -0 -> +0
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// Lane with the largest 64-bit key, lowest `index` among equals. All lanes return the same.
__device__ __forceinline__ void warp_best(unsigned long long key, int index, unsigned long long* best, int* best_index) {
    const unsigned hi = static_cast<unsigned>(key >> 32), lo = static_cast<unsigned>(key);
    const unsigned mh = __reduce_max_sync(kFull, hi);
    const unsigned ml = __reduce_max_sync(kFull, hi == mh ? lo : 0u);
    const unsigned mi = __reduce_min_sync(kFull, (hi == mh && lo == ml) ? static_cast<unsigned>(index) : kFull);
    *best = (static_cast<unsigned long long>(mh) << 32) | ml;
    *best_index = static_cast<int>(mi);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

template <int VPL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a) {
    extern __shared__ double smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    const int E = a.E;
    const bool grouped = a.top_groups < a.groups;
    float x[VPL];
    unsigned ok = 0;  // bit i: expert i*32 + lane may be chosen
    unsigned fin = 0; // bit i: its logit is finite
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 32 + lane;
        x[i] = -INFINITY;
        if (e < E) {
            const size_t at = static_cast<size_t>(t) * E + e;
            x[i] = a.fp32 ? static_cast<const float*>(a.logits)[at] : __half2float(static_cast<const __half*>(a.logits)[at]);
            const bool f = isfinite(x[i]);
            fin |= static_cast<unsigned>(f) << i;
            ok |= static_cast<unsigned>(f && (!a.bias || isfinite(a.bias[e]))) << i;
        }
    }
    // softmax: the largest logit and the sum of exp(x - largest)
    double top = 0.0, denom = 1.0;
    const bool need_scores = a.bias || grouped;
    if (!a.sigmoid) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if ((fin >> i) & 1) m = fmaxf(m, x[i]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        top = static_cast<double>(m);
        if (need_scores || !a.renorm) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if ((fin >> i) & 1) s += exp(static_cast<double>(x[i]) - top);
            denom = warp_sum(s);
        }
    }
    auto score = [&](float v) {
        return a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(v))) : exp(static_cast<double>(v) - top) / denom;
    };
    unsigned long long key[VPL];
    double* c_row = smem + static_cast<size_t>(warp) * E;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 32 + lane;
        double c = 0.0;
        if (need_scores && ((ok >> i) & 1)) c = score(x[i]) + (a.bias ? static_cast<double>(a.bias[e]) : 0.0);
        key[i] = ((ok >> i) & 1) ? key_of(a.bias ? c : static_cast<double>(x[i])) : 0ull;
        if (grouped && e < E) c_row[e] = ((ok >> i) & 1) ? c : -INFINITY;
    }
    if (grouped) {
        __syncwarp();
        const int size = E / a.groups;
        unsigned long long gkey[2] = {0ull, 0ull};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int gi = r * 32 + lane;
            if (gi >= a.groups) continue;
            double b0 = -INFINITY, b1 = -INFINITY;
            for (int j = 0; j < size; ++j) {
                const double c = c_row[gi * size + j];
                if (c > b0) {
                    b1 = b0;
                    b0 = c;
                } else if (c > b1) {
                    b1 = c;
                }
            }
            // a group counts the members it has; one without any is never chosen
            if (b0 > -INFINITY) gkey[r] = key_of(a.group_top == 2 && b1 > -INFINITY ? b0 + b1 : b0);
        }
        unsigned stay[2] = {0u, 0u};  // group numbers that stay
        for (int n = 0; n < a.top_groups; ++n) {
            unsigned long long best;
            int bi;
            const bool second = gkey[1] > gkey[0];
            warp_best(second ? gkey[1] : gkey[0], second ? lane + 32 : lane, &best, &bi);
            if (best == 0ull) break;
            stay[bi >> 5] |= 1u << (bi & 31);
            if ((bi & 31) == lane) gkey[bi >> 5] = 0ull;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = i * 32 + lane;
            const int gi = e < E ? e / size : 0;
            if (!((stay[gi >> 5] >> (gi & 31)) & 1)) key[i] = 0ull;
        }
    }
    // top_k times the largest key; lane j keeps the j-th choice
    int mine = -1;
    float mine_x = 0.f;
    for (int j = 0; j < a.top_k; ++j) {
        unsigned long long lk = 0ull;
        int li = 0;
        float lx = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i] > lk) {
                lk = key[i];
                li = i;
                lx = x[i];
            }
        unsigned long long best;
        int e;
        warp_best(lk, li * 32 + lane, &best, &e);
        if (best == 0ull) break;
        const float ex = __shfl_sync(kFull, lx, e & 31);
        if (lane == j) {
            mine = e;
            mine_x = ex;
        }
        if ((e & 31) == lane) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i == (e >> 5)) key[i] = 0ull;
        }
    }
    // weights in 64 bits, rounded once
    double p = 0.0;
    if (mine >= 0) p = score(mine_x);
    if (a.renorm) {
        const double s = warp_sum(p);
        p = s > 0.0 ? p / s : 0.0;
    }
    if (lane < a.top_k) {
        const size_t at = static_cast<size_t>(t) * a.top_k + lane;
        a.idx[at] = mine;
        a.w[at] = static_cast<float>(p * static_cast<double>(a.scale));
    }
}

__global__ void __launch_bounds__(kListThreads) lists_kernel(const int32_t* __restrict__ idx, int pairs, int E,
                                                             int32_t* __restrict__ offsets, int32_t* __restrict__ rows) {
    constexpr int kWarps = kListThreads / 32;
    __shared__ int s_less[kWarps], s_same[kWarps];
    const int e = blockIdx.x;  // E: only the last offset
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_warp = ((pairs + kWarps - 1) / kWarps + 31) / 32 * 32;
    const long long beg = static_cast<long long>(warp) * per_warp;
    const int first = beg < pairs ? static_cast<int>(beg) : pairs;
    const int last = beg + per_warp < pairs ? static_cast<int>(beg + per_warp) : pairs;
    int less = 0, same = 0;
    for (int i = first + lane; i < last; i += 32) {
        const int v = __ldg(idx + i);
        less += (v >= 0 && v < e) ? 1 : 0;
        same += v == e ? 1 : 0;
    }
    less = __reduce_add_sync(kFull, less);
    same = __reduce_add_sync(kFull, same);
    if (lane == 0) {
        s_less[warp] = less;
        s_same[warp] = same;
    }
    __syncthreads();
    int at = 0;
    for (int i = 0; i < kWarps; ++i) at += s_less[i] + (i < warp ? s_same[i] : 0);
    if (threadIdx.x == 0) offsets[e] = at;
    if (e == E) return;
    for (int i0 = first; i0 < last; i0 += 32) {
        const int i = i0 + lane;
        const bool hit = i < last && __ldg(idx + i) == e;
        const unsigned m = __ballot_sync(kFull, hit);
        if (hit) rows[at + __popc(m & ((1u << lane) - 1u))] = i;
        at += __popc(m);
    }
}

template <int VPL>
cudaError_t route_vpl(const RouteArgs& a, cudaStream_t st) {
    const size_t smem = a.top_groups < a.groups ? static_cast<size_t>(kRouteWarps) * a.E * sizeof(double) : 0;
    route_kernel<VPL><<<(a.T + kRouteWarps - 1) / kRouteWarps, kRouteWarps * 32, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t st) {
    if (a.E <= 32) return route_vpl<1>(a, st);
    if (a.E <= 64) return route_vpl<2>(a, st);
    if (a.E <= 128) return route_vpl<4>(a, st);
    if (a.E <= 256) return route_vpl<8>(a, st);
    if (a.E <= 512) return route_vpl<16>(a, st);
    return route_vpl<32>(a, st);
}

cudaError_t launch_expert_lists(const int32_t* idx, int pairs, int E, int32_t* offsets, int32_t* rows,
                                cudaStream_t st) {
    lists_kernel<<<E + 1, kListThreads, 0, st>>>(idx, pairs, E, offsets, rows);
    return cudaGetLastError();
}

}  // namespace wq
