// The experts' 4-bit products: y[p] = a[p / a_div] . W[e(p)] for every pair p of the lists,
// W = (q - 8) * s, fp32 sums, one rounding to fp16; gated: silu(gate) * up in the epilogue.
// And the weighted sum of a token's pairs after the down product.
//
// experts_kernel (few rows per expert). Tile: 32 columns of one expert x up to 8*NB of its rows, all
// of K. A group of WK warps shares a tile, its 128-row k-blocks dealt in turn; the groups' tiles
// follow one another without a break: a warp loads the codes of its next k-blocks, of this tile or
// the next, into registers (16 bytes a lane, a whole fragment of the weight) and its activations
// with cp.async into its own ring, and needs nothing from other warps until its group adds the
// tile's sums, in the order of the warps, behind one barrier. The weight is the 16-row operand of
// m16n8k16 (exact fp16 q - 8), the tokens are its 8 columns; each group's fp32 partial is scaled in
// fp32, so no weight is rounded. Bound by HBM: a k-block of a tile is 2 KiB of codes.
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "wq_experts.h"
#include "wq_experts_dev.cuh"
#include "wq_ptx.cuh"

namespace wq {

namespace {

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    // through L1: the warps of a CTA want the same rows at about the same time
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
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

// NB: blocks of 8 rows. SL: scales per k-block and column (1, 2 or 4 groups of a k-block; 0:
// per-column, g == K). W: warps. D: k-blocks in flight per warp.
template <int NB_, int SL_>
struct Small {
    static constexpr int NB = NB_, SL = SL_;
    static constexpr int W = NB == 4 ? 8 : 16;
    static constexpr int D = NB == 1 && SL < 4 ? 3 : 2;
    static constexpr int kRows = 8 * NB;
    static constexpr int kRing = D * NB * 2048;            // bytes of a warp's ring
    static constexpr int kRedRow = 36;                     // floats of a row of sums, with padding
    static constexpr int kRed = kRows * kRedRow * 4;       // bytes of a warp's sums
    // tiles that are open at a time: summed, D loaded, and the one after whose rows are known
    static constexpr int kQueue = D + 2;
    static constexpr int kSmem = W * (kRing + 2 * kRed);
};

template <class C>
__global__ void __launch_bounds__(C::W * 32, 1) experts_kernel(ExpertArgs a, int WK) {
    constexpr int NB = C::NB, SL = C::SL, D = C::D, kS = SL ? SL : 1, kRows = C::kRows;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ int s_start[kExMaxExperts + 1], s_tiles[kExMaxExperts + 1], s_each[kExMaxExperts], s_scratch[C::W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q = lane & 3, gc = lane >> 2;
    const int group = warp / WK, ks = warp % WK, groups = C::W / WK;
    uint8_t* ring = smem_raw + warp * C::kRing;
    float* red = reinterpret_cast<float*>(smem_raw + C::W * C::kRing) + group * WK * (C::kRed / 4);
    expert_table<C::W * 32>(a.offsets, a.E, a.pairs, kRows, s_start, s_tiles, s_scratch);
    rows_per_tile<C::W * 32>(a.E, 8, s_start, s_tiles, s_each);
    __syncthreads();

    const int KT = a.K / kTileK, NU = ex_units(a.N);
    const int n_out = a.gated ? a.N / 2 : a.N;
    const int kb_per_group = SL == 1 ? a.g / kTileK : 1;

    // A warp's tiles between the loads that open them and the sums that end them.
    struct Entry {
        int e, ct, nrows;   // nrows 0: no tile left
        int pair[kRows];    // -1: an entry of the lists that names no pair
    };
    __shared__ Entry s_queue[C::W][C::kQueue];
    Walk next(NU, a.E, blockIdx.x * groups + group, gridDim.x * groups, s_start, s_tiles, s_each);  // to be opened
    int place[NB];  // its rows' entries of the lists
    auto read_rows = [&]() {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int r = b * 8 + gc;
            place[b] = !next.done() && r < next.nrows ? __ldg(a.rows + next.row0 + r) : -1;
        }
    };
    read_rows();

    uint4 w[D][4];    // codes [(rt, h)]
    uint2 sc[D][kS];  // scales of the columns (rt, h) as fp16
    const uint8_t* f_codes = nullptr;
    const uint8_t* f_scales = nullptr;
    const uint16_t* arow[NB];
    int f_kb = ks, f_at = 0;
    bool f_valid = false;
    auto open_tile = [&]() {
        Entry& q_entry = s_queue[warp][f_at];
        f_at = f_at + 1 == C::kQueue ? 0 : f_at + 1;
        f_valid = !next.done();
        if (!f_valid) {
            if (lane == 0) q_entry.nrows = 0;
            return;
        }
        const uint8_t* we = a.wp + static_cast<size_t>(next.e) * a.expert_stride;
        f_codes = we + (static_cast<size_t>(next.ct) * KT + f_kb) * kExUnitBytes + lane * 16;
        f_scales = we + a.scale_offset + static_cast<size_t>(next.ct) * (a.K / a.g) * (kExUnitN * 2) + gc * 8;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const bool in = b * 8 + gc < next.nrows;
            const bool good = static_cast<unsigned>(place[b]) < static_cast<unsigned>(a.pairs);
            arow[b] = in && good ? a.a + static_cast<size_t>(row_of_pair(place[b], a)) * a.K + q * 8 : nullptr;
            if (in && !good) atomicCAS(a.status, 0, 1 /* WQ_ERR_INVALID_ARG */);
            if (q == 0) q_entry.pair[b * 8 + gc] = in && good ? place[b] : -1;
        }
        if (lane == 0) {
            q_entry.e = next.e;
            q_entry.ct = next.ct;
            q_entry.nrows = next.nrows;
        }
        next.next();
        read_rows();
    };
    // load this warp's next k-block into slot d (compile-time): codes, scales, activations
    auto fetch = [&](int d) {
        if (f_valid) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[d][i] = ldg_stream16(f_codes + i * 512);
            f_codes += WK * kExUnitBytes;
            if (SL) {
#pragma unroll
                for (int i = 0; i < kS; ++i) {
                    const int grp = SL == 1 ? (kb_per_group == 1 ? f_kb : f_kb / kb_per_group) : f_kb * SL + i;
                    sc[d][i] = __ldg(reinterpret_cast<const uint2*>(f_scales + static_cast<size_t>(grp) * (kExUnitN * 2)));
                }
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
                if (arow[b]) {
                    // rows behind the tile's last are not copied: what lies there meets no stored sum
                    uint8_t* dst = ring + (d * NB + b) * 2048 + q * 128 + gc * 16;
#pragma unroll
                    for (int c = 0; c < 4; ++c) cp_async16(dst + c * 512, arow[b] + f_kb * kTileK + c * 32);
                }
            f_kb += WK;
            if (f_kb >= KT) {
                f_kb = ks;
                open_tile();
            }
        }
        cp_async_commit();
    };
    open_tile();
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d);

    float acc[2][NB][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][b][i] = 0.f;
    int kb = ks, at = 0, turn = 0;
    __syncwarp();
    const Entry* t = &s_queue[warp][0];  // the tile that is summed
    int nrows = t->nrows;
    float cs0 = 1.f, cs1 = 1.f;  // column scales of this lane's output, g == K
    auto column_scales = [&]() {
        if (SL == 0 && nrows) {
            const uint8_t* we = a.wp + static_cast<size_t>(t->e) * a.expert_stride;
            const __half* cs = reinterpret_cast<const __half*>(we + a.scale_offset) + static_cast<size_t>(t->ct) * kExUnitN;
            const int v0 = a.gated ? ((lane >> 3) & 1) * 16 + (lane & 7) : lane;
            const int place = (v0 & 7) * 4 + (v0 >> 4) * 2 + ((v0 >> 3) & 1);
            cs0 = __half2float(cs[place]);
            if (a.gated) cs1 = __half2float(cs[place + 1]);
        }
    };
    column_scales();
    while (nrows) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (!nrows) break;
            cp_async_wait<D - 1>();
            __syncwarp();
            const uint8_t* st = ring + d * NB * 2048 + lane * 16;
            float s[2][NB][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                constexpr int kPer = SL ? 4 / kS : 4;  // 32-row blocks of a scale
                if (SL && c % kPer == 0) {
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i) s[r][b][i] = 0.f;
                }
                uint4 x[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    if (b == 0 || b * 8 < nrows) x[b] = ldmatrix4(st + b * 2048 + c * 512);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t p0[4], p1[4];
                    const uint4 w0 = w[d][2 * r], w1 = w[d][2 * r + 1];
                    dequant8(c == 0 ? w0.x : c == 1 ? w0.y : c == 2 ? w0.z : w0.w, p0);
                    dequant8(c == 0 ? w1.x : c == 1 ? w1.y : c == 2 ? w1.z : w1.w, p1);
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        if (b == 0 || b * 8 < nrows) {
                            float(&u)[4] = SL ? s[r][b] : acc[r][b];
                            mma_16816(u, p0[0], p1[0], p0[1], p1[1], x[b].x, x[b].y);
                            mma_16816(u, p0[2], p1[2], p0[3], p1[3], x[b].z, x[b].w);
                        }
                }
                if (SL && c % kPer == kPer - 1) {
                    const uint2 sv = sc[d][c / kPer];
                    const float2 s0 = __half22float2(*reinterpret_cast<const __half2*>(&sv.x));
                    const float2 s1 = __half22float2(*reinterpret_cast<const __half2*>(&sv.y));
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        if (b == 0 || b * 8 < nrows) {
                            acc[0][b][0] += s0.x * s[0][b][0];
                            acc[0][b][1] += s0.x * s[0][b][1];
                            acc[0][b][2] += s0.y * s[0][b][2];
                            acc[0][b][3] += s0.y * s[0][b][3];
                            acc[1][b][0] += s1.x * s[1][b][0];
                            acc[1][b][1] += s1.x * s[1][b][1];
                            acc[1][b][2] += s1.y * s[1][b][2];
                            acc[1][b][3] += s1.y * s[1][b][3];
                        }
                }
            }
            fetch(d);
            kb += WK;
            if (kb < KT) continue;

            // the tile's end: sums of the group's warps, [warp][row][column]
            float* sums = red + turn * (C::W * C::kRed / 4);
            turn ^= 1;
            float* mine = sums + ks * (C::kRed / 4);
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mine[(b * 8 + 2 * q + (i & 1)) * C::kRedRow + r * 16 + (i >> 1) * 8 + gc] = acc[r][b][i];
                        acc[r][b][i] = 0.f;
                    }
            // one barrier a tile: the sums of the next one go to the other buffer
            if (WK > 1) named_barrier_sync(1 + group, WK * 32); else __syncwarp();
            if (a.gated) {
                const int col = lane & 15, v0 = (col >> 3) * 16 + (col & 7), n = t->ct * 16 + col;
                for (int m = ks * 2 + (lane >> 4); m < nrows; m += WK * 2) {
                    float gate = 0.f, up = 0.f;
                    for (int k = 0; k < WK; ++k) {
                        gate += sums[k * (C::kRed / 4) + m * C::kRedRow + v0];
                        up += sums[k * (C::kRed / 4) + m * C::kRedRow + v0 + 8];
                    }
                    const int p = t->pair[m];
                    const float out = silu_mul(gate * cs0, up * cs1);
                    if (n < n_out && p >= 0) a.y[static_cast<size_t>(p) * n_out + n] = __half_as_ushort(__float2half_rn(out));
                }
            } else {
                const int n = t->ct * 32 + lane;
                for (int m = ks; m < nrows; m += WK) {
                    float out = 0.f;
                    for (int k = 0; k < WK; ++k) out += sums[k * (C::kRed / 4) + m * C::kRedRow + lane];
                    const int p = t->pair[m];
                    if (n < n_out && p >= 0) a.y[static_cast<size_t>(p) * n_out + n] = __half_as_ushort(__float2half_rn(out * cs0));
                }
            }
            kb = ks;
            at = at + 1 == C::kQueue ? 0 : at + 1;
            __syncwarp();
            t = &s_queue[warp][at];
            nrows = t->nrows;
            column_scales();
        }
    }
    cp_async_wait<0>();
}

// The combined down product of a few tokens, without lists: a tile is 32 columns of one token's sum
// over its experts, top_k * K long, whose 128-row k-blocks a group of WK warps takes in turn. A
// weight's k-block is scaled by its group scale and the choice's weight together, in fp32. Experts
// that two tokens share are read twice (the second time from L2), which is what limits this form to
// few pairs; what it saves is a launch, the pairs' sums through memory and a rounding of each.
template <int SL>
__global__ void __launch_bounds__(512, 1) experts_token_kernel(ExpertArgs a, const int32_t* __restrict__ idx,
                                                               const float* __restrict__ wt, int top_k, int WK) {
    constexpr int W = 16, D = SL == 4 ? 2 : 3;
    __shared__ __align__(16) uint8_t s_ring[W][D][256];  // the token's row of a k-block
    __shared__ float s_sums[2][W][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int q = lane & 3, gc = lane >> 2;
    const int group = warp / WK, ks = warp % WK, groups = W / WK;
    const int KT = a.K / kTileK, NU = ex_units(a.N);
    const int units = top_k * KT;
    const int G = a.K / a.g;                                     // groups along K (1: per-column scales)
    const int kb_per_group = SL == 1 && G > 1 ? a.g / kTileK : KT;
    const unsigned tokens = a.pairs / top_k;
    const unsigned step = gridDim.x * groups, step_t = step / NU, step_u = step % NU;

    uint4 w[D][4];
    uint2 sc[D][SL];
    float wj[D];
    unsigned good = 0;  // bit d: slot d holds a k-block of an expert
    // the tile that is loaded; lane j has its j-th choice
    unsigned f_t = (blockIdx.x * groups + group) / NU, f_u = (blockIdx.x * groups + group) % NU;
    int f_unit = ks, my_e = -1;
    float my_w = 0.f;
    auto open_tile = [&]() {
        if (f_t < tokens && lane < top_k) {
            const size_t p = static_cast<size_t>(f_t) * top_k + lane;
            my_e = __ldg(idx + p);
            my_w = __ldg(wt + p);
        }
    };
    auto fetch = [&](int d) {
        if (f_t < tokens) {
            const int j = f_unit / KT, kb = f_unit - j * KT;
            const int e = __shfl_sync(kFull, my_e, j);
            wj[d] = __shfl_sync(kFull, my_w, j);
            good &= ~(1u << d);
            if (static_cast<unsigned>(e) < static_cast<unsigned>(a.E)) {  // else the choice adds nothing
                good |= 1u << d;
                const uint8_t* we = a.wp + static_cast<size_t>(e) * a.expert_stride;
                const uint8_t* codes = we + (static_cast<size_t>(f_u) * KT + kb) * kExUnitBytes + lane * 16;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[d][i] = ldg_stream16(codes + i * 512);
#pragma unroll
                for (int i = 0; i < SL; ++i) {
                    const int grp = SL == 1 ? kb / kb_per_group : kb * SL + i;
                    sc[d][i] = __ldg(reinterpret_cast<const uint2*>(
                        we + a.scale_offset + (static_cast<size_t>(f_u) * G + grp) * (kExUnitN * 2) + gc * 8));
                }
                if (lane < 16)
                    cp_async16(&s_ring[warp][d][lane * 16],
                               a.a + (static_cast<size_t>(f_t) * top_k + j) * a.K + kb * kTileK + lane * 8);
            }
            f_unit += WK;
            if (f_unit >= units) {
                f_unit = ks;
                f_t += step_t;
                f_u += step_u;
                if (f_u >= static_cast<unsigned>(NU)) {
                    f_u -= NU;
                    ++f_t;
                }
                open_tile();
            }
        }
        cp_async_commit();
    };
    unsigned t = f_t, u = f_u;  // the tile that is summed
    open_tile();
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d);
    float acc[2][2] = {};  // columns (rt, h) of lane gc; every quad lane holds the same
    int unit = ks, turn = 0;
    while (t < tokens) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (t >= tokens) break;
            cp_async_wait<D - 1>();
            __syncwarp();
            if ((good >> d) & 1u) {
                // all eight rows of the activation operand are the token's
                const uint8_t* st = &s_ring[warp][d][(lane >> 3) * 16];
                float s[2][4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    constexpr int kPer = 4 / SL;
                    if (c % kPer == 0) {
#pragma unroll
                        for (int r = 0; r < 2; ++r)
#pragma unroll
                            for (int i = 0; i < 4; ++i) s[r][i] = 0.f;
                    }
                    const uint4 x = ldmatrix4(st + c * 64);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        uint32_t p0[4], p1[4];
                        const uint4 w0 = w[d][2 * r], w1 = w[d][2 * r + 1];
                        dequant8(c == 0 ? w0.x : c == 1 ? w0.y : c == 2 ? w0.z : w0.w, p0);
                        dequant8(c == 0 ? w1.x : c == 1 ? w1.y : c == 2 ? w1.z : w1.w, p1);
                        mma_16816(s[r], p0[0], p1[0], p0[1], p1[1], x.x, x.y);
                        mma_16816(s[r], p0[2], p1[2], p0[3], p1[3], x.z, x.w);
                    }
                    if (c % kPer == kPer - 1) {
                        const uint2 sv = sc[d][c / kPer];
                        const float2 s0 = __half22float2(*reinterpret_cast<const __half2*>(&sv.x));
                        const float2 s1 = __half22float2(*reinterpret_cast<const __half2*>(&sv.y));
                        acc[0][0] += s0.x * wj[d] * s[0][0];
                        acc[0][1] += s0.y * wj[d] * s[0][2];
                        acc[1][0] += s1.x * wj[d] * s[1][0];
                        acc[1][1] += s1.y * wj[d] * s[1][2];
                    }
                }
            }
            fetch(d);
            unit += WK;
            if (unit < units) continue;
            // the tile's end: the group's sums, in the order of its warps
            float(*sums)[32] = s_sums[turn] + group * WK;
            turn ^= 1;
            if (q == 0) {
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h) sums[ks][r * 16 + h * 8 + gc] = acc[r][h];
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) acc[r][0] = acc[r][1] = 0.f;
            if (WK > 1) named_barrier_sync(1 + group, WK * 32); else __syncwarp();
            if (ks == 0) {
                float out = 0.f;
                for (int k = 0; k < WK; ++k) out += sums[k][lane];
                const int n = u * kExUnitN + lane;
                if (n < a.N) a.y[static_cast<size_t>(t) * a.N + n] = __half_as_ushort(__float2half_rn(out));
            }
            unit = ks;
            t += step_t;
            u += step_u;
            if (u >= static_cast<unsigned>(NU)) {
                u -= NU;
                ++t;
            }
        }
    }
    cp_async_wait<0>();
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
cudaError_t configure_small() {
    using C = Small<NB, SL>;
    return cudaFuncSetAttribute(experts_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
}

// Warps per tile: the count that gives the busiest warp the fewest k-blocks, a tile's end counted as one.
int warps_per_tile(long long tiles, int k_blocks, int warps, int num_sms) {
    int best = 1;
    long long best_cost = -1;
    for (int wk = 1; wk <= warps && wk <= k_blocks; wk *= 2) {
        const long long workers = static_cast<long long>(num_sms) * (warps / wk);
        const long long cost = (tiles + workers - 1) / workers * ((k_blocks + wk - 1) / wk + 1);
        if (best_cost < 0 || cost < best_cost) {
            best = wk;
            best_cost = cost;
        }
    }
    return best;
}

template <int NB, int SL>
cudaError_t launch_small(const ExpertArgs& a, int num_sms, cudaStream_t st) {
    using C = Small<NB, SL>;
    // the lists are on the device: taken to be spread over as many experts as there are pairs
    const long long experts = a.pairs < a.E ? a.pairs : a.E;
    const long long per = (a.pairs + experts - 1) / experts;
    const long long tiles = experts * ((per + C::kRows - 1) / C::kRows) * ex_units(a.N);
    const int best = warps_per_tile(tiles, a.K / kTileK, C::W, num_sms);
    experts_kernel<C><<<num_sms, C::W * 32, C::kSmem, st>>>(a, best);
    return cudaGetLastError();
}

template <int NB>
cudaError_t configure_nb() {
    cudaError_t e = configure_small<NB, 0>();
    if (e == cudaSuccess) e = configure_small<NB, 1>();
    if (e == cudaSuccess) e = configure_small<NB, 2>();
    if (e == cudaSuccess) e = configure_small<NB, 4>();
    return e;
}

template <int NB>
cudaError_t launch_nb(const ExpertArgs& a, int num_sms, cudaStream_t st) {
    if (a.g == a.K) return launch_small<NB, 0>(a, num_sms, st);
    if (a.g == 64) return launch_small<NB, 2>(a, num_sms, st);
    if (a.g == 32) return launch_small<NB, 4>(a, num_sms, st);
    return launch_small<NB, 1>(a, num_sms, st);
}

}  // namespace

cudaError_t configure_expert_kernels() {
    cudaError_t e = configure_nb<1>();
    if (e == cudaSuccess) e = configure_nb<2>();
    if (e == cudaSuccess) e = configure_nb<4>();
    if (e == cudaSuccess) e = configure_experts_large();
    if (e == cudaSuccess) e = configure_route();
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

bool experts_token_form(int pairs, int E) { return pairs <= E / 4; }

cudaError_t launch_experts_token(const ExpertArgs& a, const int32_t* idx, const float* w, int top_k, int num_sms,
                                 cudaStream_t st) {
    const long long tiles = static_cast<long long>(a.pairs / top_k) * ex_units(a.N);
    const int wk = warps_per_tile(tiles, top_k * (a.K / kTileK), 16, num_sms);
    const long long ctas = (tiles + 16 / wk - 1) / (16 / wk);
    const unsigned grid = static_cast<unsigned>(ctas < num_sms ? ctas : num_sms);
    if (a.g == 64) experts_token_kernel<2><<<grid, 512, 0, st>>>(a, idx, w, top_k, wk);
    else if (a.g == 32) experts_token_kernel<4><<<grid, 512, 0, st>>>(a, idx, w, top_k, wk);
    else experts_token_kernel<1><<<grid, 512, 0, st>>>(a, idx, w, top_k, wk);
    return cudaGetLastError();
}

cudaError_t launch_combine_experts(const uint16_t* yp, const int32_t* idx, const float* w, int T, int top_k, int E,
                                   int N, uint16_t* Y, cudaStream_t st) {
    const long long total = static_cast<long long>(T) * (N / 8);
    combine_kernel<<<static_cast<unsigned>((total + 255) / 256), 256, 0, st>>>(yp, idx, w, top_k, E, N, Y, total);
    return cudaGetLastError();
}

}  // namespace wq
