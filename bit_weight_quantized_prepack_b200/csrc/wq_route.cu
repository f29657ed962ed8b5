// Routing of tokens to experts, and the lists of (token, choice) pairs by expert.
//
// route_token: one warp per token; lane l holds experts l, l + 32, ... With p the scores (softmax or
// sigmoid of the logits) and c = p + bias, the groups' values and the choice are those of c in 64
// bits: two experts' scores may lie closer than 32 bits hold, and a choice is a whole number that a
// rounding must not decide. Without a bias the choice goes by the logits themselves, whose order is
// that of the scores. The scores are first computed in 32 bits, with a bound on what that may be
// off; where every comparison that decides something clears the bound, its outcome is that of 64
// bits, and only the other tokens (one in some hundred for random scores) are done again in 64.
// Keys are mapped to unsigned integers of the same order, so that a warp's maximum is one reduction
// instruction per 32 bits; among equal keys the lowest expert wins. An expert whose logit or bias is
// not finite has key 0, below every finite one, and is never chosen. Bound by the integer pipe (68 % at
// 8192 tokens of 256 experts with groups, 74 % of the issue slots: 20 us for 8.4 MB of logits).
//
// lists_kernel: one CTA per two experts. Every CTA reads all choices: a thread counts those of lower
// experts (the place in `rows` where its experts begin) and notes, a bit per choice and expert, which
// are its experts' own; the pairs are then written from the notes, in order, the places of up to
// eight steps from one sum over the lanes where an expert is in many of them (one step after
// another, the lists of 65536 choices over 256 experts took 16 us, now 11). No
// atomics and no scratch: the lists are the same every time. Bound by the count and notes of every
// choice in every CTA, hence two experts to each. Up to kFuseTokens tokens the routing and the lists
// are one launch of one CTA, with a thread per expert.
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "wq_experts.h"

namespace wq {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kRouteWarps = 4;
constexpr int kFuseWarps = 16, kFuseTokens = 16, kFusePairs = 128;
constexpr int kListThreads = 1024, kListExperts = 2;
constexpr int kNotes = 64;   // choices a thread notes at a time
// What c in 32 bits may be off. __expf is within 2 + 1.173 |x| units in the last place. Sigmoid: that
// error times p (1 - p), below 0.6 * 2^-23, the rounding of 1 + e and the rounded reciprocal: below
// 2e-7. Softmax: p off by the same of its own term, below 2^-22 = 2.4e-7; by the sum's share, below p
// times 2^-23 (2 + 1.7 ln E) + 37 * 2^-24, for up to 1024 terms 1.65e-6 + 2.21e-6; by the quotient's 2
// units and the product's rounding, p times 2^-22 + 2^-24 = 3.0e-7: below 4.5e-6 together. The sum with
// the bias, and of two such, is rounded: 2^-23 of the magnitude covers one rounding twice over.
constexpr float kSigmoidErr = 2.5e-7f, kSoftmaxErr = 4.5e-6f, kRoundErr = 1.2e-7f;

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

__device__ __forceinline__ unsigned key_of(float v) {
    const unsigned b = __float_as_uint(v + 0.0f);  // -0 -> +0
    return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned key) {
    return __uint_as_float((key >> 31) ? (key & 0x7FFFFFFFu) : ~key);
}

// Largest key of the warp and the lowest index among its holders.
__device__ __forceinline__ void warp_best(unsigned key, int index, unsigned* best, int* best_index) {
    *best = __reduce_max_sync(kFull, key);
    *best_index = static_cast<int>(__reduce_min_sync(kFull, key == *best ? static_cast<unsigned>(index) : kFull));
}

// Whether two values of c in 32 bits may stand in the other order. Also where both passed the range of 32 bits
// (sums of two biases near the type's lowest value): their difference is no number.
__device__ __forceinline__ bool too_close(float hi, float lo, float terms, float err) {
    return !(hi - lo > 2.0f * terms * err + (fabsf(hi) + fabsf(lo)) * terms * kRoundErr);
}

__device__ __forceinline__ float logit(const RouteArgs& a, int t, int e) {
    const size_t at = static_cast<size_t>(t) * a.E + e;
    return a.fp32 ? __ldg(static_cast<const float*>(a.logits) + at)
                  : __half2float(__ldg(static_cast<const __half*>(a.logits) + at));
}

// A row's logits, and which experts may be chosen.
template <int VPL>
struct Row {
    float x[VPL], b[VPL];  // logits, bias (0 without one)
    unsigned ok, fin;      // bit i: expert i*32 + lane may be chosen / has a finite logit
};

// The 64-bit path reads the logits again, in loops: it is rare, and its arrays would push those of
// the 32-bit path out of registers.
__device__ __forceinline__ double denominator64(const RouteArgs& a, int t, double top) {
    double s = 0.0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < a.E; e += 32) {
        const float v = logit(a, t, e);
        if (isfinite(v)) s += exp(static_cast<double>(v) - top);
    }
    return warp_sum(s);
}

__device__ __forceinline__ double score64(bool sigmoid, float v, double top, double denom) {
    return sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(v))) : exp(static_cast<double>(v) - top) / denom;
}

// Scores, groups and choice in 64 bits. c_row: E doubles of shared memory of this warp. Lane j returns
// the j-th choice.
__device__ __noinline__ int route64(const RouteArgs a, int t, double top, double* c_row) {
    const int lane = threadIdx.x & 31, E = a.E;
    const double denom = a.sigmoid ? 1.0 : denominator64(a, t, top);
#pragma unroll 1
    for (int e = lane; e < E; e += 32) {
        const float v = logit(a, t, e);
        const double b = a.bias ? static_cast<double>(a.bias[e]) : 0.0;
        c_row[e] = isfinite(v) && isfinite(b) ? score64(a.sigmoid, v, top, denom) + b : -INFINITY;
    }
    __syncwarp();
    if (a.top_groups < a.groups) {
        const int size = E / a.groups;
        unsigned long long gkey[2] = {0ull, 0ull};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int gi = h * 32 + lane;
            if (gi >= a.groups) continue;
            double b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll 1
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
            if (b0 > -INFINITY) gkey[h] = key_of(a.group_top == 2 && b1 > -INFINITY ? b0 + b1 : b0);
        }
        unsigned long long stay = 0ull;  // group numbers that stay
#pragma unroll 1
        for (int n = 0; n < a.top_groups; ++n) {
            unsigned long long best;
            int bi;
            const bool second = gkey[1] > gkey[0];
            warp_best(second ? gkey[1] : gkey[0], second ? lane + 32 : lane, &best, &bi);
            if (best == 0ull) break;
            stay |= 1ull << bi;
            if (bi == lane) gkey[0] = 0ull;
            if (bi == lane + 32) gkey[1] = 0ull;
        }
        __syncwarp();
#pragma unroll 1
        for (int e = lane; e < E; e += 32)
            if (!((stay >> (e / size)) & 1)) c_row[e] = -INFINITY;
    }
    if (!a.bias) {
#pragma unroll 1
        for (int e = lane; e < E; e += 32)
            if (c_row[e] > -INFINITY) c_row[e] = static_cast<double>(logit(a, t, e));
    }
    int mine = -1;
#pragma unroll 1
    for (int j = 0; j < a.top_k; ++j) {
        double lc = -INFINITY;
        int le = lane;
#pragma unroll 1
        for (int e = lane; e < E; e += 32)
            if (c_row[e] > lc) {
                lc = c_row[e];
                le = e;
            }
        unsigned long long best;
        int e;
        warp_best(lc > -INFINITY ? key_of(lc) : 0ull, le, &best, &e);
        if (best == 0ull) break;
        if (lane == j) mine = e;
        if ((e & 31) == lane) c_row[e] = -INFINITY;
    }
    __syncwarp();
    return mine;
}

// The choice by 32-bit keys, those of the experts that stay: one expert after another, the lowest index
// first among equal keys.
template <int VPL>
__device__ __forceinline__ int choose_each(const unsigned (&keys)[VPL], int top_k, int steps, unsigned* place) {
    const int lane = threadIdx.x & 31;
    unsigned key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = keys[i];
    int mine = -1;
    *place = 0;
#pragma unroll 1
    for (int j = 0; j < steps; ++j) {
        unsigned lk = key[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) lk = max(lk, key[i]);
        int li = 0;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i) li = key[i] == lk ? i : li;
        unsigned best;
        int e;
        warp_best(lk, li * 32 + lane, &best, &e);
        if (best == 0u) break;
        if (lane == j) {
            *place = best;
            if (j < top_k) mine = e;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (i * 32 + lane == e) key[i] = 0u;
    }
    return mine;
}

template <int VPL>
__device__ __noinline__ int choose_ties(const unsigned (&keys)[VPL], int top_k, int steps, unsigned* place) {
    return choose_each<VPL>(keys, top_k, steps, place);
}

// The choice by 32-bit keys. Lane j returns the j-th choice; *place its key, lane top_k the key
// behind the last choice, where `next` asks for it. With 8 keys a lane or more, every lane sorts its keys once, so that a
// choice is the largest of the lanes' first keys and a step of one lane's list; the index is looked
// up at the end, by all lanes at once. Two equal keys, which this way come out one after the other
// (the last one's equal as the key behind it, or, with 32 choices, in another lane or next in the
// list), are left to the loop above. 8192 tokens of 256 experts: 30.6 us with the lists against 32.8;
// with 2 or 4 keys a lane the loop is as fast or faster (1000 tokens of 60 experts 6.9 us, sorted 7.2).
template <int VPL>
__device__ __forceinline__ int choose32(const unsigned (&key)[VPL], int top_k, bool next, unsigned* place) {
    const int lane = threadIdx.x & 31;
    const int steps = top_k < 32 ? top_k + 1 : top_k;
    if constexpr (VPL < 8) return choose_each<VPL>(key, top_k, next ? steps : top_k, place);
    unsigned s[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = key[i];
#pragma unroll
    for (int size = 2; size <= VPL; size *= 2)  // bitonic, descending
#pragma unroll
        for (int stride = size / 2; stride; stride /= 2)
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if ((i & stride) == 0) {
                    const unsigned x = s[i], y = s[i + stride];
                    const bool down = (i & size) == 0;
                    s[i] = down ? max(x, y) : min(x, y);
                    s[i + stride] = down ? min(x, y) : max(x, y);
                }
    unsigned last = 0u;
    int who = 0;
    bool tie = false;
    *place = 0;
#pragma unroll 1
    for (int j = 0; j < steps; ++j) {
        const unsigned best = __reduce_max_sync(kFull, s[0]);
        if (best == 0u) break;
        tie |= best == last;
        last = best;
        const unsigned holders = __ballot_sync(kFull, s[0] == best);
        const int w = __ffs(holders) - 1;
        tie |= j == 31 && (holders & (holders - 1u)) != 0u;
        if (lane == j) {
            *place = best;
            who = w;
        }
        if (lane == w) {
#pragma unroll
            for (int i = 0; i + 1 < VPL; ++i) s[i] = s[i + 1];
            s[VPL - 1] = 0u;
        }
    }
    if (top_k == 32) tie |= __any_sync(kFull, last != 0u && s[0] == last);
    if (tie) return choose_ties<VPL>(key, top_k, steps, place);
    int mine = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (__shfl_sync(kFull, key[i], who) == *place) mine = i * 32 + who;
    return lane < top_k && *place ? mine : -1;
}

// The 32-bit choice may hold the right experts in the wrong order, or miss one by a hair: all experts
// within reach of the last choice, one per lane, are ordered by their c in 64 bits. Returns false
// for more than 32 of them.
template <int VPL>
__device__ __noinline__ bool resolve64(const RouteArgs a, int t, double top, unsigned within, double* scratch, int* mine) {
    const int lane = threadIdx.x & 31;
    const unsigned below = (1u << lane) - 1u;
    int* list = reinterpret_cast<int*>(scratch);
    int n = 0;
#pragma unroll 1
    for (int i = 0; i < VPL; ++i) {
        const bool in = (within >> i) & 1;
        const unsigned m = __ballot_sync(kFull, in);
        const int at = n + __popc(m & below);
        if (in && at < 32) list[at] = i * 32 + lane;
        n += __popc(m);
    }
    if (n > 32) return false;
    const double denom = a.sigmoid ? 1.0 : denominator64(a, t, top);
    __syncwarp();
    const int e = lane < n ? list[lane] : 0;
    const unsigned long long key =
        lane < n ? key_of(score64(a.sigmoid, logit(a, t, e), top, denom) + (a.bias ? static_cast<double>(a.bias[e]) : 0.0))
                 : 0ull;
    int rank = 0;  // experts lie in the list by rising number within a lane only: ties by the number
#pragma unroll 4
    for (int o = 0; o < n; ++o) {
        const unsigned long long ok = __shfl_sync(kFull, key, o);
        const int oe = __shfl_sync(kFull, e, o);
        rank += ok > key || (ok == key && oe < e) ? 1 : 0;
    }
    __syncwarp();
    if (lane < n) list[rank] = e;
    __syncwarp();
    *mine = lane < a.top_k && lane < n ? list[lane] : -1;
    __syncwarp();
    return true;
}

// The same in 32 bits; false where a comparison of groups came too close.
template <int VPL>
__device__ __forceinline__ bool route32(const RouteArgs& a, int t, const Row<VPL>& r, float top, double* scratch, int* mine) {
    float* c_row = reinterpret_cast<float*>(scratch);
    const int lane = threadIdx.x & 31, E = a.E;
    const bool grouped = a.top_groups < a.groups;
    unsigned key[VPL];
    if (!a.bias && !grouped) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = ((r.ok >> i) & 1) ? key_of(r.x[i]) : 0u;
        unsigned unused;
        *mine = choose32<VPL>(key, a.top_k, false, &unused);
        return true;
    }
    const float err = a.sigmoid ? kSigmoidErr : kSoftmaxErr;
    float inv = 1.f;
    // the groups' shape; e / size as a product, exact for e < 1024
    const int size = E / a.groups;
    const unsigned size_mul = ((1u << 20) + size - 1) / size;
    int part_log = 5;
    while (part_log > 0 && (a.groups << part_log) > 32) --part_log;
    const int part = 1 << part_log;
    const int pad = size >= 32 ? part : 0;  // so that the groups' lanes read different banks
    float p[VPL];
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) p[i] = __frcp_rn(1.0f + __expf(-r.x[i]));
    } else {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            p[i] = ((r.fin >> i) & 1) ? __expf(r.x[i] - top) : 0.f;
            s += p[i];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
        inv = __fdividef(1.0f, s);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 32 + lane;
        const float c = ((r.ok >> i) & 1) ? p[i] * inv + r.b[i] : 0.f;
        key[i] = ((r.ok >> i) & 1) ? key_of(c) : 0u;
        if (grouped && e < E) c_row[e + pad * static_cast<int>((e * size_mul) >> 20)] = __uint_as_float(key[i]);
    }
    bool close = false;
    if (grouped) {
        __syncwarp();
        // The two largest of every group: `part` lanes share a group, lane g * part + i its members i,
        // i + part, ...; 64 groups in two rounds. Lane g then keeps group g (and g + 32).
        unsigned gkey[2] = {0u, 0u};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h * 32 >= a.groups) break;
            const int gi = h * 32 + (lane >> part_log);
            unsigned b0 = 0u, b1 = 0u;
            if (gi < a.groups)
                for (int j = lane & (part - 1); j < size; j += part) {
                    const unsigned k = __float_as_uint(c_row[gi * (size + pad) + j]);
                    b1 = max(b1, min(b0, k));
                    b0 = max(b0, k);
                }
            for (int o = part >> 1; o; o >>= 1) {
                const unsigned o0 = __shfl_xor_sync(kFull, b0, o), o1 = __shfl_xor_sync(kFull, b1, o);
                b1 = max(min(b0, o0), max(b1, o1));
                b0 = max(b0, o0);
            }
            // a group counts the members it has; one without any is never chosen
            const float v = value_of(b0) + (a.group_top == 2 && b1 ? value_of(b1) : 0.f);
            const unsigned k = b0 ? key_of(v) : 0u;
            gkey[h] = __shfl_sync(kFull, k, (lane * part) & 31);
            if (h * 32 + lane >= a.groups) gkey[h] = 0u;
        }
        unsigned long long stay = 0ull;
        float last = 0.f;
        for (int n = 0; n <= a.top_groups; ++n) {
            unsigned best;
            int bi;
            const bool second = gkey[1] > gkey[0];
            warp_best(second ? gkey[1] : gkey[0], second ? lane + 32 : lane, &best, &bi);
            if (best == 0u) break;
            const float v = value_of(best);
            if (n == a.top_groups) {
                close = too_close(last, v, 2.0f, err);
                break;
            }
            last = v;
            stay |= 1ull << bi;
            if (bi == lane) gkey[0] = 0u;
            if (bi == lane + 32) gkey[1] = 0u;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = i * 32 + lane;
            const int gi = e < E ? static_cast<int>((e * size_mul) >> 20) : 0;
            if (!((stay >> gi) & 1)) key[i] = 0u;
            else if (!a.bias) key[i] = ((r.ok >> i) & 1) ? key_of(r.x[i]) : 0u;
        }
        __syncwarp();
    }
    if (close) return false;
    unsigned mk;
    *mine = choose32<VPL>(key, a.top_k, a.bias != nullptr, &mk);
    if (!a.bias) return true;
    const unsigned after = __shfl_down_sync(kFull, mk, 1);
    // the place behind 32 choices is not looked at: call it close
    close = a.top_k == 32 || (lane < a.top_k && mk && after && too_close(value_of(mk), value_of(after), 1.0f, err));
    if (!__any_sync(kFull, close)) return true;
    // experts that may stand before the last choice
    const unsigned chosen = __ballot_sync(kFull, lane < a.top_k && mk);
    const float last = value_of(__shfl_sync(kFull, mk, 31 - __clz(chosen)));
    unsigned within = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (key[i] && too_close(last, value_of(key[i]), 1.0f, err)) within |= 1u << i;
    return resolve64<VPL>(a, t, static_cast<double>(top), within, scratch, mine);
}

// Route token t: writes its choices and weights; lane j returns choice j.
template <int VPL>
__device__ __forceinline__ int route_token(const RouteArgs& a, int t, double* scratch) {
    const int lane = threadIdx.x & 31, E = a.E;
    Row<VPL> r;
    r.ok = r.fin = 0;
    float top = 0.f;  // softmax: the largest finite logit
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 32 + lane;
        r.x[i] = e < E ? logit(a, t, e) : -INFINITY;
        r.b[i] = e < E && a.bias ? __ldg(a.bias + e) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const bool f = isfinite(r.x[i]);
        r.fin |= static_cast<unsigned>(f) << i;
        r.ok |= static_cast<unsigned>(f && isfinite(r.b[i])) << i;
    }
    if (!a.sigmoid) {
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if ((r.fin >> i) & 1) top = fmaxf(top, r.x[i]);
        top = value_of(__reduce_max_sync(kFull, key_of(top)));
    }
    int mine;
    if (!route32<VPL>(a, t, r, top, scratch, &mine)) mine = route64(a, t, top, scratch);
    const float mine_x = mine >= 0 ? logit(a, t, mine) : 0.f;
    // weights in 64 bits, rounded once
    const double denom = a.sigmoid || a.renorm ? 1.0 : denominator64(a, t, top);  // renormalised: it cancels
    double p = 0.0;
    if (mine >= 0) p = score64(a.sigmoid, mine_x, top, denom);
    if (a.renorm) {
        const double s = warp_sum(p);
        p = s > 0.0 ? p / s : 0.0;
    }
    if (lane < a.top_k) {
        const size_t at = static_cast<size_t>(t) * a.top_k + lane;
        a.idx[at] = mine;
        a.w[at] = static_cast<float>(p * a.scale);
    }
    return mine;
}

// Bytes of a warp's scratch: c of a row, where groups are chosen or 64 bits may be needed.
__host__ __device__ inline size_t route_scratch(const RouteArgs& a) {
    return a.bias || a.top_groups < a.groups ? static_cast<size_t>(a.E) * sizeof(double) : 0;
}

template <int VPL>
__global__ void __launch_bounds__(kRouteWarps * 32, VPL <= 8 ? 12 : 1) route_kernel(RouteArgs a) {
    extern __shared__ double smem[];
    const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    route_token<VPL>(a, t, smem + (threadIdx.x >> 5) * (route_scratch(a) / sizeof(double)));
}

// Exclusive sum over the block's threads; *all: over all of them. `scan`: one int per warp.
template <int W>
__device__ __forceinline__ int block_exclusive(int own, int* scan, int* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = v;
    __syncthreads();
    int before = 0, sum = 0;
    for (int w = 0; w < W; ++w) {
        before += w < warp ? scan[w] : 0;
        sum += scan[w];
    }
    *all = sum;
    return before + v - own;
}

// A few tokens: a warp each, then the lists with a thread per expert. Dynamic shared memory: the
// warps' scratch for routing.
template <int VPL>
__global__ void __launch_bounds__(kFuseWarps * 32) route_lists_kernel(RouteArgs a, int32_t* __restrict__ offsets,
                                                                      int32_t* __restrict__ rows) {
    extern __shared__ double smem[];
    __shared__ int s_idx[kFusePairs], s_scan[kFuseWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pairs = a.T * a.top_k;
    if (warp < a.T) {
        const int e = route_token<VPL>(a, warp, smem + warp * (route_scratch(a) / sizeof(double)));
        if (lane < a.top_k) s_idx[warp * a.top_k + lane] = e;
    }
    __syncthreads();
    int carry = 0;
    for (int base = 0; base < a.E; base += kFuseWarps * 32) {
        const int e = base + tid;
        int n = 0;
        for (int p = 0; p < pairs; ++p) n += s_idx[p] == e ? 1 : 0;
        if (e >= a.E) n = 0;
        int all;
        int place = carry + block_exclusive<kFuseWarps>(n, s_scan, &all);
        carry += all;
        if (e < a.E) {
            offsets[e] = place;
            if (n)
                for (int p = 0; p < pairs; ++p)
                    if (s_idx[p] == e) rows[place++] = p;
        }
    }
    if (tid == 0) offsets[a.E] = carry;
}

__global__ void __launch_bounds__(kListThreads) lists_kernel(const int32_t* __restrict__ idx, int pairs, int E,
                                                             int32_t* __restrict__ offsets, int32_t* __restrict__ rows) {
    constexpr int W = kListThreads / 32;
    constexpr int X = kListExperts;
    __shared__ int s_less[W], s_same[X][W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int e0 = blockIdx.x * X;
    const bool vec = (reinterpret_cast<uintptr_t>(idx) & 15) == 0;
    // Block by block of choices, at most kListThreads * kNotes; every warp has an equal run of a block,
    // in steps of 128 consecutive choices, four to a lane.
    const int run = static_cast<int>(min((static_cast<long long>(pairs) + W * 128 - 1) / (W * 128), kNotes / 4ll)) * 128;
    const long long block = static_cast<long long>(W) * run;
    const int blocks = pairs ? static_cast<int>((pairs + block - 1) / block) : 0;
    int less = 0, same[X] = {};
    unsigned note[X][kNotes / 32];  // bit 4s + j of word g: choice j of step 8g + s is the expert's
    auto look = [&](int v, int g, int bit) {
        less += static_cast<unsigned>(v) < static_cast<unsigned>(e0) ? 1 : 0;
#pragma unroll
        for (int x = 0; x < X; ++x)
            if (v == e0 + x && e0 + x < E) note[x][g] |= 1u << bit;
    };
    auto read_block = [&](int b) {
        const long long at = b * block + static_cast<long long>(warp) * run;
#pragma unroll
        for (int g = 0; g < kNotes / 32; ++g) {
#pragma unroll
            for (int x = 0; x < X; ++x) note[x][g] = 0u;
            if (vec && (g + 1) * 1024 <= run && at + (g + 1) * 1024 <= pairs) {
                int4 q[8];  // eight loads under way at a time
#pragma unroll
                for (int s = 0; s < 8; ++s) q[s] = __ldg(reinterpret_cast<const int4*>(idx + at + (g * 8 + s) * 128) + lane);
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    look(q[s].x, g, s * 4);
                    look(q[s].y, g, s * 4 + 1);
                    look(q[s].z, g, s * 4 + 2);
                    look(q[s].w, g, s * 4 + 3);
                }
            } else {
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const int step = (g * 8 + s) * 128;
                    if (step >= run || at + step >= pairs) break;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const long long i = at + step + lane * 4 + j;
                        look(i < pairs ? __ldg(idx + i) : -1, g, s * 4 + j);
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < X; ++x) same[x] += __popc(note[x][g]);
        }
    };
    for (int b = 0; b < blocks; ++b) read_block(b);
    less = __reduce_add_sync(kFull, less);
    if (lane == 0) s_less[warp] = less;
#pragma unroll
    for (int x = 0; x < X; ++x) {
        same[x] = __reduce_add_sync(kFull, same[x]);
        if (lane == 0) s_same[x][warp] = same[x];
    }
    __syncthreads();
    // every warp adds up the warps' counts: W = 32 of them, one per lane
    int start[X];
    start[0] = __reduce_add_sync(kFull, s_less[lane]);
#pragma unroll
    for (int x = 1; x < X; ++x) start[x] = start[x - 1] + __reduce_add_sync(kFull, s_same[x - 1][lane]);
    if (tid == 0) {
#pragma unroll
        for (int x = 0; x < X; ++x)
            if (e0 + x <= E) offsets[e0 + x] = start[x];
    }
    if (e0 + X == E) {
        const int last = start[X - 1] + __reduce_add_sync(kFull, s_same[X - 1][lane]);
        if (tid == 0) offsets[E] = last;
    }
    const unsigned below = (1u << lane) - 1u;
    for (int b = 0; b < blocks; ++b) {
        if (blocks > 1) {  // one block: its notes and counts are still here
#pragma unroll
            for (int x = 0; x < X; ++x) same[x] = 0;
            read_block(b);
            __syncthreads();
#pragma unroll
            for (int x = 0; x < X; ++x) {
                same[x] = __reduce_add_sync(kFull, same[x]);
                if (lane == 0) s_same[x][warp] = same[x];
            }
            __syncthreads();
        }
        const int first = static_cast<int>(b * block) + warp * run + lane * 4;
#pragma unroll
        for (int x = 0; x < X; ++x) {
            const int n = s_same[x][lane];
            int at = start[x] + __reduce_add_sync(kFull, lane < warp ? n : 0);
            start[x] += __reduce_add_sync(kFull, n);
            if (same[x] == 0) continue;
#pragma unroll
            for (int g = 0; g < kNotes / 32; ++g) {
                unsigned hits = __reduce_or_sync(kFull, note[x][g]);
                const unsigned steps = (hits | hits >> 1 | hits >> 2 | hits >> 3) & 0x11111111u;
                if (__popc(steps) <= 3) {  // one step after another
                    while (hits) {
                        const int s = (__ffs(hits) - 1) >> 2;
                        hits &= ~(15u << (s * 4));
                        const unsigned bits = (note[x][g] >> (s * 4)) & 15u;
                        int before = 0, all = 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const unsigned m = __ballot_sync(kFull, (bits >> j) & 1u);
                            before += __popc(m & below);
                            all += __popc(m);
                        }
                        int p = at + before;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if ((bits >> j) & 1u) rows[p++] = first + (g * 8 + s) * 128 + j;
                        at += all;
                    }
                    continue;
                }
                // All at once: a lane's count in each of the 8 steps, a byte each (even steps, odd steps), and the
                // sums over the lanes before it: at most 128.
                unsigned n4 = note[x][g] - ((note[x][g] >> 1) & 0x55555555u);
                n4 = (n4 & 0x33333333u) + ((n4 >> 2) & 0x33333333u);
                const unsigned own[2] = {n4 & 0x0F0F0F0Fu, (n4 >> 4) & 0x0F0F0F0Fu};
                unsigned before[2] = {own[0], own[1]}, all[2];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const unsigned u = __shfl_up_sync(kFull, before[h], o);
                        before[h] += lane >= o ? u : 0u;
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    all[h] = __shfl_sync(kFull, before[h], 31);
                    before[h] -= own[h];
                }
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    if (!((hits >> (4 * s)) & 15u)) continue;
                    const int byte = s / 2 * 8;
                    int p = at + static_cast<int>((before[s & 1] >> byte) & 255u);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if ((note[x][g] >> (4 * s + j)) & 1u) rows[p++] = first + (g * 8 + s) * 128 + j;
                    at += static_cast<int>((all[s & 1] >> byte) & 255u);
                }
            }
        }
    }
}

template <int VPL>
cudaError_t configure_vpl() {
    const size_t most = static_cast<size_t>(kFuseWarps) * VPL * 32 * sizeof(double);
    return cudaFuncSetAttribute(route_lists_kernel<VPL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(most));
}

template <int VPL>
cudaError_t route_vpl(const RouteArgs& a, int32_t* offsets, int32_t* rows, cudaStream_t st) {
    const size_t scratch = route_scratch(a);
    if (offsets && a.T <= kFuseTokens && a.T * a.top_k <= kFusePairs) {
        route_lists_kernel<VPL><<<1, kFuseWarps * 32, a.T * scratch, st>>>(a, offsets, rows);
        return cudaGetLastError();
    }
    route_kernel<VPL><<<(a.T + kRouteWarps - 1) / kRouteWarps, kRouteWarps * 32, kRouteWarps * scratch, st>>>(a);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || !offsets) return err;
    return launch_expert_lists(a.idx, a.T * a.top_k, a.E, offsets, rows, st);
}

}  // namespace

cudaError_t configure_route() {
    cudaError_t e = configure_vpl<1>();
    if (e == cudaSuccess) e = configure_vpl<2>();
    if (e == cudaSuccess) e = configure_vpl<4>();
    if (e == cudaSuccess) e = configure_vpl<8>();
    if (e == cudaSuccess) e = configure_vpl<16>();
    if (e == cudaSuccess) e = configure_vpl<32>();
    return e;
}

cudaError_t launch_route(const RouteArgs& a, int32_t* offsets, int32_t* rows, cudaStream_t st) {
    if (a.E <= 32) return route_vpl<1>(a, offsets, rows, st);
    if (a.E <= 64) return route_vpl<2>(a, offsets, rows, st);
    if (a.E <= 128) return route_vpl<4>(a, offsets, rows, st);
    if (a.E <= 256) return route_vpl<8>(a, offsets, rows, st);
    if (a.E <= 512) return route_vpl<16>(a, offsets, rows, st);
    return route_vpl<32>(a, offsets, rows, st);
}

cudaError_t launch_expert_lists(const int32_t* idx, int pairs, int E, int32_t* offsets, int32_t* rows,
                                cudaStream_t st) {
    lists_kernel<<<(E + kListExperts - 1) / kListExperts, kListThreads, 0, st>>>(idx, pairs, E, offsets, rows);
    return cudaGetLastError();
}

}  // namespace wq
