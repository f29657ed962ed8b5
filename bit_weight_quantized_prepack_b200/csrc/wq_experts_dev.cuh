// Device code that the expert products share: dequantisation, the table of tiles, the gate.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "wq_experts.h"
#include "wq_ptx.cuh"

namespace wq {

constexpr unsigned kFull = 0xFFFFFFFFu;

// The four fp16 pairs (rows 0..7) of one code word as exact q - 8: a nibble under the exponent of
// 1024 is 1024 + q (low) or 1024 + 16q (high).
__device__ __forceinline__ void dequant8(uint32_t w, uint32_t (&p)[4]) {
    const __half2 low = __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));    // 1032
    const __half2 mul = __halves2half2(__ushort_as_half(0x2C00), __ushort_as_half(0x2C00));    // 1/16
    const __half2 off = __halves2half2(__ushort_as_half(0xD480), __ushort_as_half(0xD480));    // -72
    const uint32_t w8 = w >> 8;
    uint32_t t[4] = {lop3_and_or(w, 0x000F000Fu, 0x64006400u), lop3_and_or(w, 0x00F000F0u, 0x64006400u),
                     lop3_and_or(w8, 0x000F000Fu, 0x64006400u), lop3_and_or(w8, 0x00F000F0u, 0x64006400u)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __half2 h = *reinterpret_cast<__half2*>(&t[i]);
        h = (i & 1) ? __hfma2(h, mul, off) : __hsub2(h, low);
        p[i] = *reinterpret_cast<uint32_t*>(&h);
    }
}

// Rows of each expert from the offsets, clamped into [0, pairs] and made non-decreasing, so that
// no content of the lists leads outside them: s_start[e] first place, s_tiles[e] tiles before e.
template <int kBlock>
__device__ void expert_table(const int32_t* offsets, int E, int pairs, int tile_rows, int* s_start, int* s_tiles,
                             int* s_scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kW = kBlock / 32;
    int carry = 0;  // largest offset so far
    for (int base = 0; base <= E; base += kBlock) {
        const int e = base + tid;
        int v = e <= E ? min(max(__ldg(offsets + e), 0), pairs) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kFull, v, o);
            if (lane >= o) v = max(v, u);
        }
        if (lane == 31) s_scratch[warp] = v;
        __syncthreads();
        for (int i = 0; i < warp; ++i) v = max(v, s_scratch[i]);
        v = max(v, carry);
        if (e <= E) s_start[e] = v;
        for (int i = 0; i < kW; ++i) carry = max(carry, s_scratch[i]);
        __syncthreads();
    }
    int sum = 0;  // tiles before this block's first expert
    for (int base = 0; base < E; base += kBlock) {
        const int e = base + tid;
        const int own = e < E ? (s_start[e + 1] - s_start[e] + tile_rows - 1) / tile_rows : 0;
        int v = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kFull, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) s_scratch[warp] = v;
        __syncthreads();
        int before = sum;
        for (int i = 0; i < kW; ++i) {
            if (i < warp) before += s_scratch[i];
            sum += s_scratch[i];
        }
        if (e < E) s_tiles[e] = before + v - own;
        __syncthreads();
    }
    if (tid == 0) s_tiles[E] = sum;
    __syncthreads();
}

// p / a_div for 0 <= p < 2^28, a_div <= 32. With m = ceil(2^32 / d) the product's high word is at
// most one above the quotient (p * m / 2^32 < p / d + 2^-4), which the second term takes back.
__device__ __forceinline__ int row_of_pair(int p, const ExpertArgs& a) {
    const int r = static_cast<int>(__umulhi(static_cast<unsigned>(p), a.a_mul));
    return a.a_div == 1 ? p : r - (r * a.a_div > p);
}

// silu(gate) * up, off by less than (8 + 1.18 |gate|) 2^-23 of itself: exp's 2 + 1.173 |gate| units in the last
// place, the quotient's 2, three roundings. At gate = -104, where exp passes the range, that is 2^-16, a
// thirtieth of the output's rounding; from there on the value is 0 (fp32 itself leaves 2^-147 of up).
__device__ __forceinline__ float silu_mul(float gate, float up) { return __fdividef(gate, 1.0f + __expf(-gate)) * up; }

// Rows of each of an expert's row tiles: even shares, rounded up to `unit` rows.
template <int kBlock>
__device__ void rows_per_tile(int E, int unit, const int* s_start, const int* s_tiles, int* s_each) {
    for (int e = threadIdx.x; e < E; e += kBlock) {
        const int n = s_start[e + 1] - s_start[e], share = s_tiles[e + 1] - s_tiles[e];
        s_each[e] = share ? ((n + share - 1) / share + unit - 1) / unit * unit : 0;
    }
}

// Walk of worker `first` of `workers` over the tiles: row tile rt_all of all experts' row tiles, column
// tile ct of CT; the column tiles of one row tile are neighbours. next() is for whole warps: its search
// looks at 32 experts at a time.
struct Walk {
    int rt_all, ct, e;       // position
    int row0, nrows;         // rows of the tile: places row0 .. of the lists
    int CT, E, step_rt, step_ct;
    const int* start;
    const int* tiles;
    const int* each;

    __device__ __forceinline__ Walk(int CT_, int E_, unsigned first, unsigned workers, const int* s_start,
                                    const int* s_tiles, const int* s_each)
        : e(0), row0(0), nrows(0), CT(CT_), E(E_), start(s_start), tiles(s_tiles), each(s_each) {
        step_rt = workers / CT;
        step_ct = workers % CT;
        rt_all = first / CT;
        ct = first % CT;
        locate();
    }
    // tiles of this worker from here on
    __device__ __forceinline__ int left(int workers) const {
        const long long n = static_cast<long long>(tiles[E]) * CT - (static_cast<long long>(rt_all) * CT + ct);
        return n <= 0 ? 0 : static_cast<int>((n + workers - 1) / workers);
    }
    __device__ __forceinline__ bool done() const { return rt_all >= tiles[E]; }
    __device__ __forceinline__ void next() {
        rt_all += step_rt;
        ct += step_ct;
        if (ct >= CT) {
            ct -= CT;
            ++rt_all;
        }
        locate();
    }
    __device__ __forceinline__ void locate() {
        if (done()) return;
        for (int n = 32; n == 32; e += n) {
            const int i = e + 1 + (threadIdx.x & 31);
            n = __popc(__ballot_sync(kFull, i < E && tiles[i] <= rt_all));
        }
        row0 = start[e] + (rt_all - tiles[e]) * each[e];
        nrows = min(each[e], start[e + 1] - row0);
    }
};

// 16 bytes that are read once: past L1.
__device__ __forceinline__ uint4 ldg_stream16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

}  // namespace wq
