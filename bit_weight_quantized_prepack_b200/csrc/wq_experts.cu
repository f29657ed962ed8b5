// The experts' 4-bit products: y[p] = a[p / a_div] . W[e(p)] for every pair p of the lists,
// W = (q - 8) * s, fp32 sums, one rounding to fp16; gated: silu(gate) * up in the epilogue.
// And the weighted sum of a token's pairs after the down product.
//
// experts_kernel (few rows per expert). Tile: 32 columns of one expert x up to 8 of its rows, all of
// K. A CTA has an equal run of all tiles, as segments of one row tile each, whose rows it keeps
// in shared memory. Each of its 24 warps (16 where the rows are long) has an equal run of a segment's
// k-blocks (tile after tile, 2 KiB of codes each, contiguous in memory) and streams them, across
// segments, into registers: 16 bytes a lane, a whole fragment of the weight. The weight is the 16-row
// operand of m16n8k16 (exact fp16 q - 8), the tokens are its 8 columns; each scale multiplies its
// fp32 partial, so no weight is rounded. A tile whose k-blocks lie with several warps is summed by the
// one that has the first, in the order of the warps. The rows stay in shared memory because every SM
// wants the same few at the same time: through a ring per warp 16 tokens over 2 of 8 experts of 4096 x
// 22016 took 148 us, with the ring filled through L1 85. Now 72.4 us, 357 MB at 4.9 TB/s; 24 tokens
// over 6 of 60 of 4096 x 1400, g = 64: 42 us, 167 MB at 4.0 TB/s. Without rows and MMAs the streams
// reach 0.80 to 0.89 of the copy rate; the rest is the dequantisation's instructions, which grow with
// the scales of a k-block.
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "wq_experts.h"
#include "wq_experts_dev.cuh"
#include "wq_ptx.cuh"

namespace wq {

namespace {

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    // through L1: neighbouring tiles want the same rows
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

// SL: scales per k-block and column (1, 2 or 4 groups of a k-block; 0: per-column, g == K). W: warps.
// With one k-block ahead of the one in hand, 24 warps of 80 registers hide more than 16 of 128 with
// three (16 tokens, 2 of 8 experts of 4096 x 22016: 72.6 us against 84.4; 28 warps 74.6, 32 76.5).
template <int SL_, int W_>
struct Small {
    static constexpr int SL = SL_, W = W_;
    static constexpr int kRows = 8;
    static constexpr int kSumRow = 36;                     // floats of a row of sums, with padding
    static constexpr int kSums = kRows * kSumRow;          // floats of a tile's sums
    static constexpr size_t rows_bytes(int K) { return static_cast<size_t>(kRows) * K * 2; }
    static constexpr size_t kFixed = static_cast<size_t>(W) * 2 * kSums * 4;
    // shared memory with one or two places for the rows, and whether it fits
    static constexpr size_t kMost = 232448 - 16384;        // less than the tables' static part
    static size_t smem(int K, int places) { return kFixed + places * rows_bytes(K); }
    static int places(int K) { return smem(K, 2) <= kMost ? 2 : smem(K, 1) <= kMost ? 1 : 0; }
};

// kPairs: the products go to y32, unrounded (not gated); as a branch on the argument it cost the other form
// 1.5 to 2 % (24 warps use every register that they may).
template <class C, bool kPairs>
__global__ void __launch_bounds__(C::W * 32, 1) experts_kernel(ExpertArgs a, int places) {
    constexpr int SL = C::SL, W = C::W, kS = SL ? SL : 1, kRows = C::kRows;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ int s_start[kExMaxExperts + 1], s_tiles[kExMaxExperts + 1], s_each[kExMaxExperts], s_scratch[W];
    __shared__ int s_pair[2][kRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q = lane & 3, gc = lane >> 2;
    float* sums = reinterpret_cast<float*>(smem_raw);          // [W][2][kSums]
    uint8_t* s_rows = smem_raw + C::kFixed;
    const size_t rows_bytes = C::rows_bytes(a.K);
    expert_table<W * 32>(a.offsets, a.E, a.pairs, kRows, s_start, s_tiles, s_scratch);
    rows_per_tile<W * 32>(a.E, 8, s_start, s_tiles, s_each);
    __syncthreads();

    const int KT = a.K / kTileK, NU = ex_units(a.N), G = a.K / a.g;
    const int n_out = a.gated ? a.N / 2 : a.N;
    const int kb_per_group = SL == 1 ? a.g / kTileK : 1;
    const long long tiles = static_cast<long long>(s_tiles[a.E]) * NU;
    const long long tile0 = tiles * blockIdx.x / gridDim.x, tile1 = tiles * (blockIdx.x + 1ll) / gridDim.x;

    // A segment: the column tiles u0 .. u1 - 1 of one row tile; the CTA's tiles are a run of segments.
    struct Segment {
        int e, rt, u0, u1, row0, nrows;  // nrows 0: none left
    };
    auto segment_at = [&](long long tile, int e) {
        Segment s{e, 0, 0, 0, 0, 0};
        if (tile >= tile1) return s;
        s.rt = static_cast<int>(tile / NU);
        s.u0 = static_cast<int>(tile - static_cast<long long>(s.rt) * NU);
        s.u1 = static_cast<int>(min(static_cast<long long>(NU), s.u0 + (tile1 - tile)));
        int lo = e, hi = a.E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_tiles[mid] <= s.rt) lo = mid; else hi = mid;
        }
        s.e = lo;
        const int first = (s.rt - s_tiles[lo]) * s_each[lo];
        s.row0 = s_start[lo] + first;
        s.nrows = min(s_each[lo], s_start[lo + 1] - s.row0);
        return s;
    };
    auto after = [&](const Segment& s) { return segment_at(static_cast<long long>(s.rt) * NU + s.u1, s.e); };
    // this warp's run of a segment's k-blocks, the segment's tiles one after another
    auto run_of = [&](const Segment& s, int w, int* beg, int* end) {
        const int units = (s.u1 - s.u0) * KT, per = (units + W - 1) / W;
        *beg = min(w * per, units);
        *end = min((w + 1) * per, units);
    };

    // ---- loads of the weights, across segments
    uint4 w[4];    // codes [(rt, h)] of the next k-block
    uint2 sc[kS];  // scales of the columns (rt, h) as fp16
    Segment f = segment_at(tile0, 0);
    int f_left = 0, f_kb = 0;
    const uint8_t* f_codes = nullptr;
    const uint8_t* f_scales = nullptr;
    auto open_run = [&]() {  // the first segment from f on in which this warp has k-blocks
        while (f.nrows) {
            int beg, end;
            run_of(f, warp, &beg, &end);
            f_left = end - beg;
            if (f_left > 0) {
                const uint8_t* we = a.wp + static_cast<size_t>(f.e) * a.expert_stride;
                const int u = f.u0 + beg / KT;
                f_kb = beg % KT;
                f_codes = we + (static_cast<size_t>(u) * KT + f_kb) * kExUnitBytes + lane * 16;
                f_scales = we + a.scale_offset + static_cast<size_t>(u) * G * (kExUnitN * 2) + gc * 8;
                return;
            }
            f = after(f);
        }
        f_left = 0;
    };
    auto fetch = [&]() {
        if (f_left == 0) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = ldg_stream16(f_codes + i * 512);
        f_codes += kExUnitBytes;
        if (SL) {
#pragma unroll
            for (int i = 0; i < kS; ++i) {
                const int grp = SL == 1 ? (kb_per_group == 1 ? f_kb : f_kb / kb_per_group) : f_kb * SL + i;
                sc[i] = __ldg(reinterpret_cast<const uint2*>(f_scales + static_cast<size_t>(grp) * (kExUnitN * 2)));
            }
        }
        if (++f_kb == KT) {
            f_kb = 0;
            f_scales += static_cast<size_t>(G) * (kExUnitN * 2);
        }
        if (--f_left == 0) {
            f = after(f);
            open_run();
        }
    };

    // ---- the rows of a segment, in the order in which ldmatrix takes them: [K / 8][8 rows] 16 bytes
    auto load_rows = [&](const Segment& s, int place) {
        if (s.nrows == 0) return;
        uint8_t* dst = s_rows + (places == 2 ? place : 0) * rows_bytes;
        const int row = lane & 7, piece = lane >> 3;  // four pieces of a row, eight rows
        if (row >= s.nrows) return;  // what lies there meets no stored sum
        const int p = __ldg(a.rows + s.row0 + row);
        const bool good = static_cast<unsigned>(p) < static_cast<unsigned>(a.pairs);
        if (!good) atomicCAS(a.status, 0, 1 /* WQ_ERR_INVALID_ARG */);
        if (warp == 0 && piece == 0) s_pair[place][row] = good ? p : -1;
        const uint16_t* src = a.a + static_cast<size_t>(good ? row_of_pair(p, a) : 0) * a.K;
        for (int c = warp * 4 + piece; c < a.K / 8; c += W * 4)
            cp_async16(dst + static_cast<size_t>(c) * 128 + row * 16, src + c * 8);
    };

    open_run();
    Segment s = segment_at(tile0, 0);
    if (s.nrows == 0) return;
    fetch();
    load_rows(s, 0);
    cp_async_commit();
    int place = 0;
    float* mine = sums + warp * 2 * C::kSums;

    // Columns of lane's output in column tile u: value of a row from sums already added up.
    auto store_rows = [&](int u, const Segment& g, auto&& value) {
        const uint8_t* we = a.wp + static_cast<size_t>(g.e) * a.expert_stride;
        const __half* cs = reinterpret_cast<const __half*>(we + a.scale_offset) + static_cast<size_t>(u) * kExUnitN;
        if (!kPairs && a.gated) {
            const int col = lane & 15, v0 = (col >> 3) * 16 + (col & 7), n = u * 16 + col;
            float c0 = 1.f, c1 = 1.f;
            if (SL == 0) {
                const int at = (v0 & 7) * 4 + (v0 >> 4) * 2;
                c0 = __half2float(cs[at]);
                c1 = __half2float(cs[at + 1]);
            }
            for (int m = lane >> 4; m < g.nrows; m += 2) {
                const float out = silu_mul(value(m, v0) * c0, value(m, v0 + 8) * c1);
                const int p = s_pair[place][m];
                if (n < n_out && p >= 0) a.y[static_cast<size_t>(p) * n_out + n] = __half_as_ushort(__float2half_rn(out));
            }
        } else {
            const int n = u * kExUnitN + lane;
            float c0 = 1.f;
            if (SL == 0) c0 = __half2float(cs[(lane & 7) * 4 + (lane >> 4) * 2 + ((lane >> 3) & 1)]);
            for (int m = 0; m < g.nrows; ++m) {
                const float out = value(m, lane) * c0;
                const int p = s_pair[place][m];
                if (n < n_out && p >= 0) {
                    if (kPairs) a.y32[static_cast<size_t>(p) * n_out + n] = out;
                    else a.y[static_cast<size_t>(p) * n_out + n] = __half_as_ushort(__float2half_rn(out));
                }
            }
        }
    };

    float acc[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][i] = 0.f;
    while (s.nrows) {
        const Segment next = after(s);
        cp_async_wait<0>();
        __syncthreads();  // this segment's rows are there, and the last one's sums and pairs are read
        if (places == 2) load_rows(next, place ^ 1);
        cp_async_commit();
        int beg, end;
        run_of(s, warp, &beg, &end);
        const uint8_t* rows0 = s_rows + (places == 2 ? place : 0) * rows_bytes + lane * 16;
        int kb = beg % KT, u = s.u0 + beg / KT;
        bool whole = kb == 0, first = true;  // the piece of tile u that this warp is on
        for (int unit = beg; unit < end;) {
            const uint8_t* st = rows0 + static_cast<size_t>(kb) * 2048;
            float t[2][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                constexpr int kPer = SL ? 4 / kS : 4;  // 32-row blocks of a scale
                if (SL && c % kPer == 0) {
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int i = 0; i < 4; ++i) t[r][i] = 0.f;
                }
                const uint4 x = ldmatrix4(st + c * 512);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t p0[4], p1[4];
                    const uint4 w0 = w[2 * r], w1 = w[2 * r + 1];
                    dequant8(c == 0 ? w0.x : c == 1 ? w0.y : c == 2 ? w0.z : w0.w, p0);
                    dequant8(c == 0 ? w1.x : c == 1 ? w1.y : c == 2 ? w1.z : w1.w, p1);
                    float(&v)[4] = SL ? t[r] : acc[r];
                    mma_16816(v, p0[0], p1[0], p0[1], p1[1], x.x, x.y);
                    mma_16816(v, p0[2], p1[2], p0[3], p1[3], x.z, x.w);
                }
                if (SL && c % kPer == kPer - 1) {
                    const uint2 sv = sc[c / kPer];
                    const float2 s0 = __half22float2(*reinterpret_cast<const __half2*>(&sv.x));
                    const float2 s1 = __half22float2(*reinterpret_cast<const __half2*>(&sv.y));
                    acc[0][0] += s0.x * t[0][0];
                    acc[0][1] += s0.x * t[0][1];
                    acc[0][2] += s0.y * t[0][2];
                    acc[0][3] += s0.y * t[0][3];
                    acc[1][0] += s1.x * t[1][0];
                    acc[1][1] += s1.x * t[1][1];
                    acc[1][2] += s1.y * t[1][2];
                    acc[1][3] += s1.y * t[1][3];
                }
            }
            fetch();
            ++unit;
            if (++kb < KT && unit < end) continue;
            // the piece's end: a whole tile is stored, a part is left for the tile's first warp
            const bool done = whole && kb == KT;
            float* part = mine + (first && !done ? 0 : C::kSums);
            __syncwarp();
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    part[(2 * q + (i & 1)) * C::kSumRow + r * 16 + (i >> 1) * 8 + gc] = acc[r][i];
                    acc[r][i] = 0.f;
                }
            __syncwarp();
            if (done) store_rows(u, s, [&](int m, int v) { return part[m * C::kSumRow + v]; });
            first = false;
            whole = true;
            kb = 0;
            ++u;
        }
        __syncthreads();  // all parts are there, the rows have been read
        if (places == 1) load_rows(next, place ^ 1);
        cp_async_commit();
        if (beg < end) {
            // a tile that begins in this warp's run and ends behind it
            const int per = ((s.u1 - s.u0) * KT + W - 1) / W;
            const int ut = (end - 1) / KT, tile_beg = ut * KT, tile_end = tile_beg + KT;
            if (tile_beg >= beg && tile_end > end) {
                const float* own = mine + (tile_beg == beg ? 0 : C::kSums);
                const int last = (tile_end - 1) / per;  // warp with its last k-block
                store_rows(s.u0 + ut, s, [&](int m, int v) {
                    float sum = own[m * C::kSumRow + v];
                    for (int k = warp + 1; k <= last; ++k) sum += sums[k * 2 * C::kSums + m * C::kSumRow + v];
                    return sum;
                });
            }
        }
        s = next;
        place ^= 1;
    }
    cp_async_wait<0>();
}

// Few pairs: one row at a time, without a table of tiles. A tile is 32 columns of one row's product,
// whose 128-row k-blocks a group of WK warps takes in turn, loading three ahead, across tiles.
// kSum: the combined down product of a few tokens, without lists: the tile is a token's sum over its
// experts, top_k * K long; a k-block is scaled by its group scale and the choice's weight together,
// in fp32. It saves a launch, the pairs' sums through memory and a rounding of each. Otherwise row i
// is place i of the lists; its expert ends at the first offset above i.
// An expert that two rows share is read twice (the second time from L2), which is what limits this
// form to few pairs. Bound by latency: one token over 8 of 128 experts, gated 2048 x 1536: 8.1 us for
// 13 MB, combined 768 x 2048: 6.6 us for 6.5 MB, of which an empty kernel takes 2.5; the 8-row tiles
// with their table took 12 and 10.8.
template <int SL, bool kSum>
__global__ void __launch_bounds__(512, 1) experts_token_kernel(ExpertArgs a, const int32_t* __restrict__ idx,
                                                               const float* __restrict__ wt, int top_k, int WK) {
    constexpr int W = 16, D = SL == 4 ? 2 : 3;
    __shared__ __align__(16) uint8_t s_ring[W][D][256];  // the token's row of a k-block
    __shared__ float s_sums[2][W][32];
    __shared__ int s_out[W][D + 2];  // rows of Y of the open tiles, -1: none
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int q = lane & 3, gc = lane >> 2;
    const int group = warp / WK, ks = warp % WK, groups = W / WK;
    const int KT = a.K / kTileK, NU = ex_units(a.N);
    const int n_out = a.gated ? a.N / 2 : a.N;
    const int units = kSum ? top_k * KT : KT;
    const int G = a.K / a.g;                                     // groups along K (1: per-column scales)
    const int kb_per_group = SL == 1 && G > 1 ? a.g / kTileK : KT;
    const unsigned tokens = kSum ? a.pairs / top_k : a.pairs;  // rows of the product
    const unsigned step = gridDim.x * groups, step_t = step / NU, step_u = step % NU;

    uint4 w[D][4];
    uint2 sc[D][SL];
    float wj[D];
    unsigned good = 0;  // bit d: slot d holds a k-block of an expert
    // the tile that is loaded; lane j has its j-th choice
    unsigned f_t = (blockIdx.x * groups + group) / NU, f_u = (blockIdx.x * groups + group) % NU;
    int f_unit = ks, f_at = 0, my_e = -1;
    float my_w = 1.f;
    const uint16_t* f_row = a.a;
    auto open_tile = [&]() {
        if (f_t >= tokens) return;
        int out = static_cast<int>(f_t);
        if (kSum) {
            if (lane < top_k) {
                const size_t p = static_cast<size_t>(f_t) * top_k + lane;
                my_e = __ldg(idx + p);
                my_w = __ldg(wt + p);
            }
            f_row = a.a + static_cast<size_t>(f_t) * top_k * a.K;
        } else {
            const int p = __ldg(a.rows + f_t);
            // the first offset above the row's place ends its expert; none, or the very first: no expert
            unsigned ends = a.E + 1;
#pragma unroll 4
            for (int e = lane; e <= a.E; e += 32)
                if (__ldg(a.offsets + e) > static_cast<int>(f_t)) ends = min(ends, static_cast<unsigned>(e));
            ends = __reduce_min_sync(kFull, ends);
            my_e = ends == 0 ? a.E : static_cast<int>(ends) - 1;
            out = -1;
            if (static_cast<unsigned>(p) < static_cast<unsigned>(a.pairs)) {
                out = my_e < a.E ? p : -1;
                f_row = a.a + static_cast<size_t>(row_of_pair(p, a)) * a.K;
            } else if (my_e < a.E) {
                atomicCAS(a.status, 0, 1 /* WQ_ERR_INVALID_ARG */);
                my_e = a.E;
            }
        }
        if (lane == 0) s_out[warp][f_at] = out;
        f_at = f_at + 1 == D + 2 ? 0 : f_at + 1;
    };
    auto fetch = [&](int d) {
        if (f_t < tokens) {
            const int j = kSum ? f_unit / KT : 0, kb = f_unit - j * KT;
            const int e = kSum ? __shfl_sync(kFull, my_e, j) : my_e;
            wj[d] = kSum ? __shfl_sync(kFull, my_w, j) : 1.f;
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
                    cp_async16(&s_ring[warp][d][lane * 16], f_row + static_cast<size_t>(j) * a.K + kb * kTileK + lane * 8);
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
    int unit = ks, turn = 0, at = 0;
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
            const int row = s_out[warp][at];
            at = at + 1 == D + 2 ? 0 : at + 1;
            if (ks == 0 && row >= 0) {
                float out = 0.f;
                for (int k = 0; k < WK; ++k) out += sums[k][lane];
                int n = u * kExUnitN + lane;
                bool here = true;
                if (!kSum && a.gated) {  // gate lanes take the up lane's sum
                    out = silu_mul(out, __shfl_down_sync(kFull, out, 8));
                    here = !(lane & 8);
                    n = u * 16 + (lane >> 4) * 8 + (lane & 7);
                }
                if (here && n < n_out) a.y[static_cast<size_t>(row) * n_out + n] = __half_as_ushort(__float2half_rn(out));
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
// [0, E) adds nothing and its row is not read. The pairs' products come unrounded: a rounding of each
// to fp16 would add to the output's own (1.4 times as far from the exact sum), and a product beyond
// 65504 would be lost although its weighted sum is finite. One thread per 4 columns of a token, four
// choices' rows under way at a time. Bound by the pairs' bytes: 4096 tokens, 8 choices of 2048 columns,
// 268 MB read and 17 MB written in 46 us, 6.2 TB/s.
__global__ void __launch_bounds__(256) combine_kernel(const float* __restrict__ yp, const int32_t* __restrict__ idx,
                                                      const float* __restrict__ w, int top_k, int E, int N,
                                                      uint16_t* __restrict__ Y, long long total) {
    const long long i = blockIdx.x * 256ll + threadIdx.x;
    if (i >= total) return;
    const int per_row = N / 4;
    const long long t = i / per_row;
    const int n = static_cast<int>(i - t * per_row) * 4;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < top_k; j0 += 4) {
        uint4 v[4];
        float wj[4];
        bool in[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long p = t * top_k + j0 + j;
            in[j] = j0 + j < top_k && static_cast<unsigned>(__ldg(idx + p)) < static_cast<unsigned>(E);
            wj[j] = in[j] ? __ldg(w + p) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (in[j]) v[j] = ldg_stream16(yp + (t * top_k + j0 + j) * N + n);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!in[j]) continue;
            acc[0] += wj[j] * __uint_as_float(v[j].x);
            acc[1] += wj[j] * __uint_as_float(v[j].y);
            acc[2] += wj[j] * __uint_as_float(v[j].z);
            acc[3] += wj[j] * __uint_as_float(v[j].w);
        }
    }
    uint2 out;
    __half2* o = reinterpret_cast<__half2*>(&out);
    o[0] = __floats2half2_rn(acc[0], acc[1]);
    o[1] = __floats2half2_rn(acc[2], acc[3]);
    *reinterpret_cast<uint2*>(Y + t * N + n) = out;
}

static_assert(Small<0, 24>::kFixed + Small<0, 24>::rows_bytes(9984) <= Small<0, 24>::kMost &&
                  Small<0, 24>::kFixed + Small<0, 24>::rows_bytes(9984 + kTileK) > Small<0, 24>::kMost &&
                  Small<0, 16>::kFixed + Small<0, 16>::rows_bytes(11136) <= Small<0, 16>::kMost &&
                  Small<0, 16>::kFixed + Small<0, 16>::rows_bytes(11136 + kTileK) > Small<0, 16>::kMost,
              "the longest rows that launch_experts names");

template <class C>
cudaError_t configure_small() {
    const cudaError_t e = cudaFuncSetAttribute(experts_kernel<C, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(C::kMost));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(experts_kernel<C, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(C::kMost));
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

template <class C>
cudaError_t launch_small(const ExpertArgs& a, int num_sms, cudaStream_t st) {
    const int places = C::places(a.K);
    if (a.y32) experts_kernel<C, true><<<num_sms, C::W * 32, C::smem(a.K, places), st>>>(a, places);
    else experts_kernel<C, false><<<num_sms, C::W * 32, C::smem(a.K, places), st>>>(a, places);
    return cudaGetLastError();
}

template <int W>
cudaError_t configure_w() {
    cudaError_t e = configure_small<Small<0, W>>();
    if (e == cudaSuccess) e = configure_small<Small<1, W>>();
    if (e == cudaSuccess) e = configure_small<Small<2, W>>();
    if (e == cudaSuccess) e = configure_small<Small<4, W>>();
    return e;
}

template <int W>
cudaError_t launch_w(const ExpertArgs& a, int num_sms, cudaStream_t st) {
    if (a.g == a.K) return launch_small<Small<0, W>>(a, num_sms, st);
    if (a.g == 64) return launch_small<Small<2, W>>(a, num_sms, st);
    if (a.g == 32) return launch_small<Small<4, W>>(a, num_sms, st);
    return launch_small<Small<1, W>>(a, num_sms, st);
}

template <bool kSum>
cudaError_t launch_token(const ExpertArgs& a, const int32_t* idx, const float* w, int top_k, int num_sms,
                         cudaStream_t st) {
    const long long tiles = static_cast<long long>(kSum ? a.pairs / top_k : a.pairs) * ex_units(a.N);
    const int wk = warps_per_tile(tiles, (kSum ? top_k : 1) * (a.K / kTileK), 16, num_sms);
    const long long ctas = (tiles + 16 / wk - 1) / (16 / wk);
    const unsigned grid = static_cast<unsigned>(ctas < num_sms ? ctas : num_sms);
    if (a.g == 64) experts_token_kernel<2, kSum><<<grid, 512, 0, st>>>(a, idx, w, top_k, wk);
    else if (a.g == 32) experts_token_kernel<4, kSum><<<grid, 512, 0, st>>>(a, idx, w, top_k, wk);
    else experts_token_kernel<1, kSum><<<grid, 512, 0, st>>>(a, idx, w, top_k, wk);
    return cudaGetLastError();
}

}  // namespace

bool experts_token_form(int pairs, int E) { return pairs <= E / 4; }

cudaError_t launch_experts_token(const ExpertArgs& a, const int32_t* idx, const float* w, int top_k, int num_sms,
                                 cudaStream_t st) {
    return launch_token<true>(a, idx, w, top_k, num_sms, st);
}

cudaError_t configure_expert_kernels() {
    cudaError_t e = configure_w<24>();
    if (e == cudaSuccess) e = configure_w<16>();
    if (e == cudaSuccess) e = configure_experts_large();
    if (e == cudaSuccess) e = configure_route();
    return e;
}

// Rows per expert, were the pairs spread evenly over all E, up to which mma.sync tiles of 8 rows beat the
// tcgen05 tiles, whose time is that of the dequantised weight and of each group's sums up to some hundred
// rows. Pairs of other devices' experts and padded places count here, since only the device knows them.
// Measured from a cold L2 (tiles of 8 rows against tcgen05 tiles): g = 128, 64 experts of 2048 x 2048: 16 rows
// 67.5 us against 67.5; 8 of 4096 x 8192: 16 rows 66.8 / 72.3, 20 rows 88.2 / 73.2; g = K, 32 of 2048 x
// 2048: 12 rows 38.1 / 38.0, 16 rows 39.6 / 38.5, 20 rows 50.3 / 38.8. g = 64, 128 of 1024 x 1536: 24 rows 82.8
// / 93.2, 28 rows 104 / 94. g = 32, 32 of 2048 x 2048: 48 rows 103 / 121, 64 rows 129 / 128; 128 of 1024 x
// 1536: 48 rows 160 / 167, 56 rows 182 / 179.
int few_rows(const ExpertArgs& a) { return a.g == 32 ? 48 : a.g == 64 ? 24 : 16; }

cudaError_t launch_experts(const ExpertArgs& a, const DeviceInfo& d, cudaStream_t st) {
    const long long per_expert = (static_cast<long long>(a.pairs) + a.E - 1) / a.E;
    if (experts_token_form(a.pairs, a.E)) return launch_token<false>(a, nullptr, nullptr, 1, d.num_sms, st);
    // rows of 16 warps' places reach further than those of 24: K up to 11136 against 9984
    if (per_expert > few_rows(a) || Small<0, 16>::places(a.K) == 0) return launch_experts_large(a, d, st);
    if (Small<0, 24>::places(a.K)) return launch_w<24>(a, d.num_sms, st);
    return launch_w<16>(a, d.num_sms, st);
}

cudaError_t launch_combine_experts(const float* yp, const int32_t* idx, const float* w, int T, int top_k, int E,
                                   int N, uint16_t* Y, cudaStream_t st) {
    const long long total = static_cast<long long>(T) * (N / 4);
    combine_kernel<<<static_cast<unsigned>((total + 255) / 256), 256, 0, st>>>(yp, idx, w, top_k, E, N, Y, total);
    return cudaGetLastError();
}

}  // namespace wq
