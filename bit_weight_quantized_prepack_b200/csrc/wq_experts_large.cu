// The experts' 4-bit products for many rows per expert: tcgen05 tiles over the lists.
//
// Tile: 128 columns of one expert's weight (the MMA's M) x up to 256 of its rows (the MMA's N),
// all of K in chunks of 64 rows. One persistent CTA per SM, warp-specialised:
//   warp 0       gathers the rows' 128-byte pieces with TMA gather4 (the lists give the rows);
//   warp 1       issues the MMAs: both operands from shared memory (128-byte swizzle), fp32
//                accumulators in tensor memory, two of 256 columns used in turn;
//   warps 4..7   epilogue of the tile before, while the next one is multiplied;
//   warps 8..15  dequantise: each owns 16 columns, loads its codes straight from global memory
//                several k-blocks ahead (across tiles) and writes fp16 weights (q - 8) * s,
//                rounded once, into the weight operand's place.
// An expert's rows are split evenly over its row tiles. Tiles of the same rows are neighbours, so
// that the rows are gathered from L2 after the first time.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <cstring>

#include "wq_experts.h"
#include "wq_experts_dev.cuh"
#include "wq_ptx.cuh"

namespace wq {

namespace {

constexpr int kLThreads = 512;
constexpr int kRowsMax = 256;                      // rows of a tile
constexpr int kColsL = 128;                        // columns of a tile
constexpr int kChunkK = 64;                        // weight rows of a stage: one 128-byte swizzle span
constexpr int kABytes = kColsL * kChunkK * 2;      // 16 KiB
constexpr int kBBytes = kRowsMax * kChunkK * 2;    // 32 KiB
constexpr int kStageL = kABytes + kBBytes;
constexpr int kStagesL = 4;
constexpr int kSmemL = kStagesL * kStageL + 1024;  // + alignment of the first stage
constexpr int kDqWarp0 = 8, kDqWarpsL = 8;
constexpr int kDepth = 4;                          // k-blocks of codes in flight per dequant warp

struct Bars {
    uint64_t full_a[kStagesL], full_b[kStagesL], empty[kStagesL];
    uint64_t acc_full[2], acc_empty[2], drain;
};

struct LargeArgs {
    ExpertArgs e;
    unsigned long long timeout_ns;
};

struct Ctl {
    volatile int* stop;
    int* status;
    unsigned long long timeout_ns;
};

// Bounded wait for a phase; false when it expired or another role gave up.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, const Ctl& c, bool honour_stop = true) {
    if (mbar_test_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait_sleep(bar, parity, 20000)) return true;
        if (honour_stop && *c.stop) return false;
        if (global_timer_ns() - t0 > c.timeout_ns) {
            *c.stop = 1;
            atomicCAS(c.status, 0, 6 /* WQ_ERR_TIMEOUT */);
            return false;
        }
    }
}

// Four rows (any rows of the matrix) x 64 columns, 128 bytes each, to 512 bytes of shared memory.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, int x, int4 r, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(smem_addr(bar))
        : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]; fp16 inputs, fp32 accumulator.
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ uint4 ldg_stream16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

struct TileL {
    int e, ct, row0, nrows;
};

// Tile number -> expert, column tile and rows. s_tiles counts row tiles of kRowsMax.
__device__ __forceinline__ TileL locate(long long tile, int CT, int E, const int* s_start, const int* s_tiles) {
    const int rt_all = static_cast<int>(tile / CT);
    TileL t;
    t.ct = static_cast<int>(tile % CT);
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tiles[mid] <= rt_all) lo = mid; else hi = mid;
    }
    t.e = lo;
    const int n = s_start[lo + 1] - s_start[lo];
    const int tiles = s_tiles[lo + 1] - s_tiles[lo];
    const int each = ((n + tiles - 1) / tiles + 15) / 16 * 16;  // even shares, at most kRowsMax
    const int first = (rt_all - s_tiles[lo]) * each;
    t.row0 = s_start[lo] + first;
    t.nrows = min(each, n - first);
    return t;
}

// SL as in the small kernel: scales per k-block and column; 0: per-column, applied in the epilogue.
template <int SL>
__global__ void __launch_bounds__(kLThreads, 1) experts_large_kernel(const __grid_constant__ CUtensorMap map, LargeArgs args) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars;
    __shared__ int s_start[kExMaxExperts + 1], s_tiles[kExMaxExperts + 1], s_scratch[kLThreads / 32];
    __shared__ uint32_t s_tmem;
    __shared__ int s_stop;
    const ExpertArgs& a = args.e;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);

    if (tid == 0) {
        for (int i = 0; i < kStagesL; ++i) {
            mbar_init(&bars.full_a[i], kDqWarpsL);
            mbar_init(&bars.full_b[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], 4);
        }
        mbar_init(&bars.drain, 1);
        s_stop = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    expert_table<kLThreads>(a.offsets, a.E, a.pairs, kRowsMax, s_start, s_tiles, s_scratch);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const Ctl ctl{&s_stop, a.status, args.timeout_ns};
    const int KT = a.K / kTileK, chunks = a.K / kChunkK;
    const int CT = (a.N + kColsL - 1) / kColsL, NU = ex_units(a.N);
    const long long tiles = static_cast<long long>(s_tiles[a.E]) * CT;

    if (warp == 0) {
        // ---------------------------------------------------------------- rows of the activations
        int s = 0;
        uint32_t ph = 1;  // empty barriers: the first pass over the ring waits for nothing
        long long issued = 0;
        bool ok = true;
        for (long long tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
            const TileL t = locate(tile, CT, a.E, s_start, s_tiles);
            const int n_mma = (t.nrows + 15) / 16 * 16;
            int r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // rows behind the tile's last repeat it: their sums are never stored
                const int at = min((i >> 2) * 128 + lane * 4 + (i & 3), t.nrows - 1);
                const int p = __ldg(a.rows + t.row0 + at);
                const bool good = static_cast<unsigned>(p) < static_cast<unsigned>(a.pairs);
                if (!good) atomicCAS(a.status, 0, 1 /* WQ_ERR_INVALID_ARG */);
                r[i] = good ? p / a.a_div : 0;
            }
            for (int c = 0; c < chunks; ++c) {
                ok = __all_sync(kFull, wait_phase(&bars.empty[s], ph, ctl));
                if (!ok) break;
                uint8_t* b = ring + s * kStageL + kABytes;
                if (lane == 0) mbar_arrive_expect_tx(&bars.full_b[s], n_mma * kChunkK * 2);
                __syncwarp();
                if (lane * 4 < n_mma)
                    tma_gather4(b + lane * 512, &map, c * kChunkK, make_int4(r[0], r[1], r[2], r[3]), &bars.full_b[s]);
                if (128 + lane * 4 < n_mma)
                    tma_gather4(b + (32 + lane) * 512, &map, c * kChunkK, make_int4(r[4], r[5], r[6], r[7]),
                                &bars.full_b[s]);
                ++issued;
                if (++s == kStagesL) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (!ok) {
            // given up: the copies still in flight must land before the CTA leaves
            for (long long i = issued > kStagesL ? issued - kStagesL : 0; i < issued; ++i)
                wait_phase(&bars.full_b[i % kStagesL], static_cast<uint32_t>((i / kStagesL) & 1), ctl, false);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMAs
        if (lane == 0) {
            int s = 0, buf = 0;
            uint32_t ph = 0, aph = 1;
            bool ok = true;
            for (long long tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
                const TileL t = locate(tile, CT, a.E, s_start, s_tiles);
                const uint32_t idesc = idesc_f16_f32(kColsL, (t.nrows + 15) / 16 * 16);
                ok = wait_phase(&bars.acc_empty[buf], aph, ctl);
                tc_fence_after();
                for (int c = 0; c < chunks && ok; ++c) {
                    ok = wait_phase(&bars.full_a[s], ph, ctl) && wait_phase(&bars.full_b[s], ph, ctl);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t base = smem_addr(ring + s * kStageL);
                    uint64_t da = smem_desc_sw128(base), db = smem_desc_sw128(base + kABytes);
#pragma unroll
                    for (int k = 0; k < kChunkK / 16; ++k) {
                        mma_f16_ss(tmem + buf * kRowsMax, da, db, idesc, (c | k) ? 1u : 0u);
                        da = smem_desc_advance(da, 32);
                        db = smem_desc_advance(db, 32);
                    }
                    tc_commit(&bars.empty[s]);
                    if (++s == kStagesL) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                if (ok) tc_commit(&bars.acc_full[buf]);
                buf ^= 1;
                if (buf == 0) aph ^= 1;
            }
            // every MMA done before the CTA frees its tensor memory
            tc_commit(&bars.drain);
            wait_phase(&bars.drain, 0, ctl, false);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ---------------------------------------------------------------- epilogue
        const int quarter = warp & 3;
        const int n_out = a.gated ? a.N / 2 : a.N;
        int buf = 0;
        uint32_t ph = 0;
        for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const TileL t = locate(tile, CT, a.E, s_start, s_tiles);
            const int v = t.ct * kColsL + quarter * 32 + lane;  // layout column of this lane
            float cs = 1.f;
            if (SL == 0 && v < a.N) {
                const __half* sp = reinterpret_cast<const __half*>(a.wp + static_cast<size_t>(t.e) * a.expert_stride +
                                                                   a.scale_offset) + static_cast<size_t>(v / 32) * kExUnitN;
                cs = __half2float(sp[(v & 7) * 4 + ((v >> 4) & 1) * 2 + ((v >> 3) & 1)]);
            }
            // lane l of each 32 rows keeps row l's pair; the next 32 are read while these are stored
            int pair_next = lane < t.nrows ? __ldg(a.rows + t.row0 + lane) : -1;
            if (!__all_sync(kFull, wait_phase(&bars.acc_full[buf], ph, ctl))) break;
            tc_fence_after();
            const uint32_t taddr = tmem + buf * kRowsMax + (static_cast<uint32_t>(quarter * 32) << 16);
            for (int m0 = 0; m0 < t.nrows; m0 += 32) {
                uint32_t d[32];
                tmem_ld_x32(taddr + m0, d);
                const int pair = static_cast<unsigned>(pair_next) < static_cast<unsigned>(a.pairs) ? pair_next : -1;
                pair_next = m0 + 32 + lane < t.nrows ? __ldg(a.rows + t.row0 + m0 + 32 + lane) : -1;
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float x0 = __uint_as_float(d[i]), x1 = __uint_as_float(d[i + 1]);
                    if (SL == 0) {
                        x0 *= cs;
                        x1 *= cs;
                    }
                    if (a.gated) {
                        // gate lanes take row i, up lanes row i + 1
                        const bool up = lane & 8;
                        const float other = __shfl_xor_sync(kFull, up ? x0 : x1, 8);
                        const float h = up ? silu_mul(other, x1) : silu_mul(x0, other);
                        const int p = __shfl_sync(kFull, pair, i + (up ? 1 : 0));
                        const int n = (v >> 4) * 8 + (v & 7);
                        if (p >= 0 && v < a.N) a.y[static_cast<size_t>(p) * n_out + n] = __half_as_ushort(__float2half_rn(h));
                    } else {
                        // even lanes take row i of two neighbouring columns, odd lanes row i + 1
                        const bool odd = lane & 1;
                        const float other = __shfl_xor_sync(kFull, odd ? x0 : x1, 1);
                        const __half2 h = odd ? __floats2half2_rn(other, x1) : __floats2half2_rn(x0, other);
                        const int p = __shfl_sync(kFull, pair, i + (odd ? 1 : 0));
                        const int n = v & ~1;
                        if (p >= 0 && n < a.N) *reinterpret_cast<__half2*>(a.y + static_cast<size_t>(p) * n_out + n) = h;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.acc_empty[buf]);
            buf ^= 1;
            if (buf == 0) ph ^= 1;
        }
    } else if (warp >= kDqWarp0) {
        // ---------------------------------------------------------------- weights
        const int dw = warp - kDqWarp0;
        const int q = lane & 3, gc = lane >> 2;
        constexpr int kS = SL ? SL : 1;
        uint4 w[kDepth][2];
        uint32_t sc[kDepth][kS];
        uint32_t valid = 0, live = 0;  // bit d: slot d holds a k-block / one inside the weight
        long long f_tile = blockIdx.x;
        int f_kb = 0;
        bool f_live = false;
        const uint8_t* f_codes = a.wp;
        const uint8_t* f_scales = a.wp;
        auto open_tile = [&]() {
            if (f_tile >= tiles) return;
            const TileL t = locate(f_tile, CT, a.E, s_start, s_tiles);
            const int u = t.ct * 4 + (dw >> 1);
            f_live = u < NU;
            const uint8_t* we = a.wp + static_cast<size_t>(t.e) * a.expert_stride;
            f_codes = we + static_cast<size_t>(u) * KT * kExUnitBytes + (dw & 1) * 1024 + lane * 16;
            f_scales = we + a.scale_offset + static_cast<size_t>(u) * (a.K / a.g) * (kExUnitN * 2) + gc * 8 + (dw & 1) * 4;
        };
        open_tile();
        int s = 0;
        uint32_t ph = 1;
        bool ok = true;
        auto fetch = [&](int d) {
            if (f_tile >= tiles) {
                valid &= ~(1u << d);
                return;
            }
            valid |= 1u << d;
            live = f_live ? live | (1u << d) : live & ~(1u << d);
            if (f_live) {
                w[d][0] = ldg_stream16(f_codes + static_cast<size_t>(f_kb) * kExUnitBytes);
                w[d][1] = ldg_stream16(f_codes + static_cast<size_t>(f_kb) * kExUnitBytes + 512);
                if (SL) {
#pragma unroll
                    for (int i = 0; i < kS; ++i) {
                        const int grp = SL == 1 ? f_kb * kTileK / a.g : f_kb * SL + i;
                        sc[d][i] = __ldg(reinterpret_cast<const uint32_t*>(f_scales + static_cast<size_t>(grp) * (kExUnitN * 2)));
                    }
                }
            }
            if (++f_kb == KT) {
                f_kb = 0;
                f_tile += gridDim.x;
                open_tile();
            }
        };
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            w[d][0] = w[d][1] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < kS; ++i) sc[d][i] = 0;
            fetch(d);
        }
        while (ok && (valid & 1u)) {
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                if (!ok || !((valid >> d) & 1u)) break;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    ok = __all_sync(kFull, wait_phase(&bars.empty[s], ph, ctl));
                    if (!ok) break;
                    if ((live >> d) & 1u) {
                        uint8_t* row = ring + s * kStageL + (dw * 16 + gc) * 128;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            // lanes of odd gc take the two 32-row blocks in the other order: a store's
                            // eight lanes then cover all banks
                            const uint32_t wa = half ? w[d][h].z : w[d][h].x, wb = half ? w[d][h].w : w[d][h].y;
                            const bool swap = gc & 1;
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint32_t word = (j == 0) != swap ? wa : wb;
                                const int c = (j == 0) != swap ? 0 : 1;  // 32-row block of the chunk
                                uint32_t p[4];
                                dequant8(word, p);
                                if (SL) {
                                    // scale of the block's group: slot (2*half + c) * SL / 4
                                    uint32_t sv;
                                    if (SL == 4) sv = ((j == 0) != swap) ? sc[d][(2 * half) % kS] : sc[d][(2 * half + 1) % kS];
                                    else if (SL == 2) sv = sc[d][half % kS];
                                    else sv = sc[d][0];
                                    const __half2 s2 = *reinterpret_cast<const __half2*>(&sv);
                                    const __half2 sb = h ? __high2half2(s2) : __low2half2(s2);
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const __half2 m = __hmul2(*reinterpret_cast<__half2*>(&p[i]), sb);
                                        p[i] = *reinterpret_cast<const uint32_t*>(&m);
                                    }
                                }
                                *reinterpret_cast<uint4*>(row + h * 8 * 128 + (((c * 4 + q) ^ gc) << 4)) =
                                    make_uint4(p[0], p[1], p[2], p[3]);
                            }
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.full_a[s]);
                    if (++s == kStagesL) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                if (ok) fetch(d);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

template <int SL>
cudaError_t launch_sl(const CUtensorMap& map, const LargeArgs& a, int num_sms, cudaStream_t st) {
    experts_large_kernel<SL><<<num_sms, kLThreads, kSmemL, st>>>(map, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t configure_experts_large() {
    cudaError_t e = cudaFuncSetAttribute(experts_large_kernel<0>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemL);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(experts_large_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemL);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(experts_large_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemL);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(experts_large_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemL);
    return e;
}

cudaError_t launch_experts_large(const ExpertArgs& a, const DeviceInfo& d, cudaStream_t st) {
    // the activations as [rows, K] with boxes of one row x 64 elements: gather4 takes any four rows
    const long long a_rows = static_cast<long long>(a.pairs) / a.a_div;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a_rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.K) * 2};
    const cuuint32_t box[2] = {kChunkK, 1}, estr[2] = {1, 1};
    CUtensorMap map;
    std::memset(&map, 0, sizeof(map));
    if (reinterpret_cast<EncodeTiledFn>(d.encode)(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<uint16_t*>(a.a),
                                                  dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    LargeArgs l;
    l.e = a;
    l.timeout_ns = d.timeout_ns;
    if (a.g == a.K) return launch_sl<0>(map, l, d.num_sms, st);
    if (a.g == 64) return launch_sl<2>(map, l, d.num_sms, st);
    if (a.g == 32) return launch_sl<4>(map, l, d.num_sms, st);
    return launch_sl<1>(map, l, d.num_sms, st);
}

}  // namespace wq
