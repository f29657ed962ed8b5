// The experts' 4-bit products for many rows per expert: tcgen05 tiles over the lists.
//
// Tile: 256 columns of one expert's weight (the MMA's M, 128 for each CTA of a pair) x up to 128 of its
// rows (the MMA's N), all of K in k-blocks of 128 rows. One persistent CTA per SM, warp-specialised:
//   warps 0..2    gather the rows' 128-byte pieces with cp.async into a ring of 8 k-blocks, each warp
//                 every third k-block;
//   warp 3        one elected thread issues the pair's MMAs: weights from tensor memory, rows from
//                 shared memory (128-byte swizzle), the sums of one scale group to tensor memory;
//   warps 4..19   add the groups' sums up: warp 4 + w takes columns 32 (w % 4) .. + 31 and every fourth
//                 16 rows, reads a group's sums while the next group is multiplied, and adds scale
//                 times sum in its registers, fp32; at the tile's end it stores its rows;
//   warps 20..27  dequantise: warp 20 + w takes columns 32 (w % 4) .. + 31 of every second k-block,
//                 loads its codes straight from global memory a turn ahead (across tiles) and
//                 stores exact fp16 q - 8 into one of four slots in tensor memory.
// An expert's rows are split evenly over its row tiles. Tiles of the same rows are neighbours, so
// that the rows are gathered from L2 after the first time.
// Why so: the weights stay exact. With (q - 8) * s rounded to fp16 in the dequantisation the outputs
// were 1.6 times as far from the exact product as the fp16 rounding of the output alone. The weight
// operand in tensor memory saves the ~32 cycles that each MMA spends on loading it from shared memory
// (probe, 128 x 256 x 16: 137 cycles against 168). TMA gather4 in place of cp.async moves a row of 128
// bytes per 14 cycles and set the pace at a quarter of this kernel's rate. The pair halves the rows'
// way from L2, which one CTA alone loaded to two thirds.
// Measured: 4096 tokens over 8 of 128 experts, g = 128: gated 2048 x 1536 283 us (730 TFLOP/s, 0.44 of
// the dense rate), 768 x 2048 with the sum of pairs 222 us; 300 tokens over 2 of 8 of 11008 x 4096 120
// us. No unit is full (2048 x 1536 / 768 x 2048): 74 / 65 % of the issue slots, 52 / 45 % of the integer pipe, 37 /
// 28 % of the tensor pipe, 20 / 22 % of L2. The groups' sums are ready when the adding warps come to them:
// the pace is that of the chains of load, wait and arithmetic in the adding and dequantising warps.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "wq_experts.h"
#include "wq_experts_dev.cuh"
#include "wq_ptx.cuh"

namespace wq {

namespace {

constexpr int kLThreads = 28 * 32;
constexpr int kRowsMax = 128;                      // rows of a tile
// Rows of a tile are rounded up to this: the pair's MMA (M = 256, weights in tensor memory) takes its N
// in steps of 32. The places behind a tile's last row hold whatever was there; their sums are not stored.
constexpr int kRowStep = 32;
static_assert(kRowStep % 32 == 0 && kRowsMax % kRowStep == 0 && kRowsMax <= 256, "N of the pair's MMA");
constexpr int kColsL = 128;                        // columns of a tile per CTA
constexpr int kChunkK = 64;                        // weight rows of a chunk: one 128-byte swizzle span
constexpr int kHalfRows = kRowsMax / 2;            // rows of a tile that one CTA of the pair holds
constexpr int kChunkBytes = kHalfRows * kChunkK * 2;  // 8 KiB
constexpr int kStageBytes = 2 * kChunkBytes;       // a k-block: two chunks
constexpr int kStages = 8;                         // k-blocks of rows in shared memory
constexpr int kSlotsA = 4;                         // k-blocks of weights in tensor memory
constexpr int kTmemA = 2 * kRowsMax;               // their first column, behind two groups' sums
constexpr int kSmemL = kStages * kStageBytes + 1024;  // + alignment of the first stage
constexpr int kGatherWarps = 3, kMmaWarp = 3, kAddWarp0 = 4, kAddWarps = 16, kDqWarp0 = 20, kDqTurns = 2;
constexpr int kQuads = kHalfRows / 4;              // a warp's copy instruction takes four rows
constexpr int kYRow = 80, kYRowGated = 48;         // bytes of an output row on its way out, with padding
constexpr int kYBytes = 16 * kYRow;

struct Bars {
    uint64_t full[kStages], empty[kStages];
    uint64_t sum_full[2], sum_empty[2], drain;
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

// Arrive on the leader's barrier that lies where `bar` lies in this CTA, for what lies in tensor memory:
// weights stored there, sums read from there. Those are ordered by the tcgen05 fences of both sides around
// the barrier, which want no more of it than that one thread's step comes after the other's; nothing
// else is handed over with these arrivals. (Released at cluster scope all the same, they cost their
// threads some hundred cycles each: 4096 tokens, 128 experts of 2048 x 1536, 334 us with the weights', 447
// with the sums' too, against 284.)
__device__ __forceinline__ void mbar_arrive_leader(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .b32 remote;\n\t"
        "mapa.shared::cluster.u32 remote, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [remote];\n\t}" ::"r"(smem_addr(bar))
        : "memory");
}
// The same for rows in shared memory: what this thread wrote, or has seen written, is released at cluster
// scope to the leader's thread, whose wait acquires it there (2 us of 282).
__device__ __forceinline__ void mbar_arrive_leader_release(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .b32 remote;\n\t"
        "mapa.shared::cluster.u32 remote, %0, 0;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [remote];\n\t}" ::"r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ bool mbar_test_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ bool mbar_try_wait_sleep_cluster(uint64_t* bar, uint32_t parity, uint32_t suspend_ns) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(suspend_ns)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Bounded wait for a phase; false when it expired or another role gave up. kCluster: what the arrivals of
// both CTAs released is acquired.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, const Ctl& c, bool honour_stop = true) {
    const auto tried = [&] {
        return kCluster ? mbar_try_wait_sleep_cluster(bar, parity, 20000) : mbar_try_wait_sleep(bar, parity, 20000);
    };
    if (kCluster ? mbar_test_wait_cluster(bar, parity) : mbar_test_wait(bar, parity)) return true;
    if (tried()) return true;  // the timer is read only by long waits
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (tried()) return true;
        if (honour_stop && *c.stop) return false;
        if (global_timer_ns() - t0 > c.timeout_ns) {
            *c.stop = 1;
            atomicCAS(c.status, 0, 6 /* WQ_ERR_TIMEOUT */);
            return false;
        }
    }
}

// Tensor memory, MMA and commit of a CTA pair: the leader's thread multiplies for both CTAs, each
// with its own 128 weight columns in its tensor memory and half of the rows in its shared memory.
__device__ __forceinline__ void tmem_alloc2(uint32_t* smem_result, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(smem_result)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma2_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on this barrier of both CTAs when every MMA issued before has completed.
__device__ __forceinline__ void tc_commit2(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// 16 lanes x 32 columns of 32 bits: lane 4g + q of the warp writes rows g (even registers) and g + 8
// (odd ones) of columns q, 4 + q, ... 28 + q.
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

// SL: scales per k-block and column (1, 2 or 4); 0: per-column, g == K. kPairs: the products go to y32,
// unrounded (not gated).
template <int SL, bool kPairs>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLThreads, 1) experts_large_kernel(LargeArgs args) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars;
    __shared__ int s_start[kExMaxExperts + 1], s_tiles[kExMaxExperts + 1], s_each[kExMaxExperts], s_scratch[kLThreads / 32];
    __shared__ __align__(16) uint8_t stage_y[kAddWarps * kYBytes];
    __shared__ uint32_t s_tmem;
    __shared__ int s_stop, s_rows_of[kStages];  // rows of the tile that a k-block belongs to
    const ExpertArgs& a = args.e;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();  // 0: the leader, whose thread issues the pair's MMAs
    uint8_t* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars.full[i], 2 + 8);  // a gather warp and four dequant warps of each CTA
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.sum_full[i], 1);
            mbar_init(&bars.sum_empty[i], 2 * kAddWarps);
        }
        mbar_init(&bars.drain, 1);
        s_stop = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc2(&s_tmem, 512);
    expert_table<kLThreads>(a.offsets, a.E, a.pairs, kRowsMax, s_start, s_tiles, s_scratch);
    rows_per_tile<kLThreads>(a.E, kRowStep, s_start, s_tiles, s_each);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the barriers of both CTAs stand
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const Ctl ctl{&s_stop, a.status, args.timeout_ns};
    const int KT = a.K / kTileK;
    const int kb_per_group = SL == 0 ? KT : SL == 1 ? a.g / kTileK : 1;  // k-blocks summed in tensor memory
    const int CT = (a.N + 2 * kColsL - 1) / (2 * kColsL), NU = ex_units(a.N);
    // column tiles of the same rows are neighbours; pair b takes tiles b, b + pairs, ...
    Walk t(CT, a.E, blockIdx.x / 2, gridDim.x / 2, s_start, s_tiles, s_each);

    if (warp < kGatherWarps) {
        // ---------------------------------------------------------------- rows of the activations
        // Warp w copies k-blocks w, w + 3, ... whole: lane l the 16-byte piece l % 8 of rows 4j + l / 8 of
        // both chunks. It signals a k-block when the next of its own is under way.
        const int piece = lane & 7, sub = lane >> 3;
        // place of the piece in the swizzled row, for even and odd quads
        const uint32_t base = smem_addr(ring) + sub * 128;
        const uint32_t dst_even = base + ((piece ^ sub) << 4), dst_odd = base + ((piece ^ (4 + sub)) << 4);
        const unsigned row_bytes = static_cast<unsigned>(a.K) * 2;
        unsigned n = 0;     // k-block
        bool ok = true, pending = false;
        unsigned last = 0;  // stage of the pending one
        auto signal = [&]() {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive_leader_release(&bars.full[last]);
        };
        // Entries of the lists of the next tile, read while this one is copied: lane l the rows l, l +
        // 32, .. of this CTA's half; places behind its last row repeat that row.
        int place[kHalfRows / 32];
        int have = 0;       // rows of that tile that this CTA holds
        auto read_rows = [&]() {
            const int half = t.done() ? 0 : (t.nrows + kRowStep - 1) / kRowStep * (kRowStep / 2), first = rank * half;
            have = t.done() ? 0 : max(0, min(half, t.nrows - first));
#pragma unroll
            for (int j = 0; j < kHalfRows / 32; ++j)
                place[j] = have > 0 ? __ldg(a.rows + t.row0 + first + min(j * 32 + lane, have - 1)) : 0;
        };
        read_rows();
        bool more = !t.done();
        while (ok && more) {
            const int quads = (have + 3) / 4;
            int row[kQuads];
#pragma unroll
            for (int j = 0; j < kHalfRows / 32; ++j) {
                // an entry that names no pair takes row 0: its sums are never stored
                const bool good = static_cast<unsigned>(place[j]) < static_cast<unsigned>(a.pairs);
                if (!good) atomicCAS(a.status, 0, 1 /* WQ_ERR_INVALID_ARG */);
                const int mine = good ? row_of_pair(place[j], a) : 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) row[j * 8 + i] = __shfl_sync(kFull, mine, i * 4 + sub);
            }
            const unsigned tile_n = n;
            const int nrows = t.nrows;
            t.next();
            more = !t.done();
            bool read = false;
            // this warp's first k-block of the tile
            for (int c = (warp + kGatherWarps - tile_n % kGatherWarps) % kGatherWarps; c < KT; c += kGatherWarps) {
                n = tile_n + c;
                const unsigned stage = n % kStages;
                ok = __all_sync(kFull, wait_phase(&bars.empty[stage], ((n / kStages) & 1) ^ 1, ctl));
                if (!ok) break;
                if (lane == 0) s_rows_of[stage] = nrows;
                const uint8_t* src = reinterpret_cast<const uint8_t*>(a.a + c * kTileK + piece * 8);
#pragma unroll
                for (int j = 0; j < kQuads; ++j)
                    if (j < quads) {
                        const uint32_t dst = ((j & 1) ? dst_odd : dst_even) + stage * kStageBytes + j * 512;
                        const uint8_t* from = src + static_cast<unsigned long long>(static_cast<unsigned>(row[j])) * row_bytes;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(from) : "memory");
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + kChunkBytes), "l"(from + kChunkK * 2)
                                     : "memory");
                    }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (pending) {
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                    signal();
                }
                pending = true;
                last = stage;
                if (!read) {
                    read_rows();
                    read = true;
                }
            }
            if (!read) read_rows();
            n = tile_n + KT;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (pending) signal();
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- MMAs
        // One elected thread runs the whole loop: inside its branch the operands stay uniform (174
        // cycles per MMA from a thread picked by its number, 40 from an elected one).
        if (rank == 0 && elect_one()) {
            // The thread's own instructions set the pace of small steps (a wait and a commit cost it about
            // 250 cycles, an MMA 15; probe): a wait per k-block, looked at while the one before is issued.
            // A tile's rows come with its first k-block: to search the table cost one thread 2100 cycles a
            // tile (4096 tokens, 8 of 128 experts: 2048 x 1536 281 us against 275, 768 x 2048 207 against 197).
            uint32_t stage = 0, ph = 0;
            unsigned m = 0;  // groups so far: sums m & 1
            bool ok = true;
            const uint64_t desc0 = smem_desc_sw128(smem_addr(ring));
            bool ready = mbar_test_wait_cluster(&bars.full[0], 0);
            for (int left = t.left(gridDim.x / 2); ok && left > 0; --left) {
                uint32_t idesc = 0;
                int in_group = 0;  // k-blocks of the group that have been issued
                for (int kb = 0; kb < KT; ++kb) {
                    if (SL < 2 && in_group == 0) ok = wait_phase(&bars.sum_empty[m & 1], ((m >> 1) & 1) ^ 1, ctl);
                    if (ok && !ready) ok = wait_phase<true>(&bars.full[stage], ph, ctl);
                    if (!ok) break;
                    tc_fence_after();
                    if (kb == 0)
                        idesc = idesc_f16_f32(2 * kColsL,
                                              (*(volatile int*)&s_rows_of[stage] + kRowStep - 1) / kRowStep * kRowStep);
                    const uint64_t db = smem_desc_advance(desc0, stage * kStageBytes);
                    const uint32_t wa = tmem + kTmemA + (stage % kSlotsA) * kChunkK;
                    constexpr int kGroups = SL < 2 ? 1 : SL;  // groups of a k-block
#pragma unroll
                    for (int q = 0; q < kGroups; ++q) {
                        if (SL >= 2) {
                            ok = wait_phase(&bars.sum_empty[m & 1], ((m >> 1) & 1) ^ 1, ctl);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        const uint32_t d = tmem + (m & 1) * kRowsMax;
#pragma unroll
                        for (int k = q * (8 / kGroups); k < (q + 1) * (8 / kGroups); ++k)
                            mma2_f16_ts(d, wa + k * 8, smem_desc_advance(db, (k >> 2) * kChunkBytes + (k & 3) * 32), idesc,
                                        (k > q * (8 / kGroups) || in_group > 0) ? 1u : 0u);
                        if (SL >= 2) {
                            tc_commit2(&bars.sum_full[m & 1]);
                            ++m;
                        }
                    }
                    if (!ok) break;
                    tc_commit2(&bars.empty[stage]);
                    if (SL < 2 && ++in_group == kb_per_group) {
                        tc_commit2(&bars.sum_full[m & 1]);
                        ++m;
                        in_group = 0;
                    }
                    stage = (stage + 1) % kStages;
                    ph ^= stage == 0;
                    ready = mbar_test_wait_cluster(&bars.full[stage], ph);
                }
            }
            tc_commit2(&bars.drain);
        }
        __syncwarp();
    } else if (warp >= kDqWarp0) {
        // ---------------------------------------------------------------- weights
        const int quarter = warp & 3, turn = (warp - kDqWarp0) >> 2;
        constexpr int kDepth = 1;  // k-blocks of codes in flight
        uint4 w[kDepth][4];        // codes [(rt, h)]
        uint32_t valid = 0, inside = 0;  // bit d: slot d holds a k-block / one inside the weight
        bool live = false;
        int f_kb = turn;
        const uint8_t* f_at = a.wp;
        auto open_tile = [&]() {  // step over the tiles until f_kb lies in one
            while (!t.done() && f_kb >= KT) {
                f_kb -= KT;
                t.next();
            }
            if (t.done()) return;
            const int u = (t.ct * 2 + rank) * 4 + quarter;
            live = u < NU;
            f_at = a.wp + static_cast<size_t>(t.e) * a.expert_stride + (static_cast<size_t>(u) * KT + f_kb) * kExUnitBytes +
                   lane * 16;
        };
        auto fetch = [&](int d) {
            valid &= ~(1u << d);
            if (t.done()) return;
            valid |= 1u << d;
            inside = live ? inside | (1u << d) : inside & ~(1u << d);
            if (live) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[d][i] = ldg_stream16(f_at + i * 512);
                f_at += kDqTurns * kExUnitBytes;
            }
            f_kb += kDqTurns;
            if (f_kb >= KT) open_tile();
        };
        open_tile();
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[d][i] = make_uint4(0, 0, 0, 0);
            fetch(d);
        }
        const uint32_t tbase = tmem + kTmemA + (static_cast<uint32_t>(quarter * 32) << 16);
        unsigned n = turn;  // k-block
        bool ok = true;
        while (ok && (valid & 1u)) {
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                if (!ok || !((valid >> d) & 1u)) break;
                const bool store = (inside >> d) & 1u;
                const uint32_t slot = tbase + (n % kSlotsA) * kChunkK;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t v[2][16];
#pragma unroll
                    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint4 q4 = w[d][rt * 2 + h];
                                uint32_t p[4];
                                dequant8(half ? (b ? q4.w : q4.z) : (b ? q4.y : q4.x), p);
#pragma unroll
                                for (int i = 0; i < 4; ++i) v[rt][2 * (4 * b + i) + h] = p[i];
                            }
                    if (half == 1) fetch(d);
                    // the k-block four before has left the slot; the first four find it empty
                    if (half == 0 && n >= kSlotsA) {
                        const unsigned before = n - kSlotsA;
                        ok = __all_sync(kFull, wait_phase(&bars.empty[before % kStages], (before / kStages) & 1, ctl));
                        if (!ok) break;
                        tc_fence_after();
                    }
                    if (store) {
                        tmem_st_16x128b_x8(slot + half * (kChunkK / 2), v[0]);
                        tmem_st_16x128b_x8(slot + half * (kChunkK / 2) + (16u << 16), v[1]);
                    }
                }
                if (!ok) break;
                if (store) {
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_leader(&bars.full[n % kStages]);
                n += kDqTurns;
            }
        }
    } else {
        // ---------------------------------------------------------------- the groups' sums, the output
        const int quarter = warp & 3, part = (warp - kAddWarp0) >> 2;  // 16-row pieces 4i + part
        const int n_out = a.gated ? a.N / 2 : a.N;
        const int groups = SL == 0 ? 1 : a.K / a.g;
        const uint32_t tbase = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        uint8_t* out = stage_y + (warp - kAddWarp0) * kYBytes;
        unsigned m = 0;  // groups so far
        bool ok = true;
        for (; ok && !t.done(); t.next()) {
            const int ct = t.ct * 2 + rank;
            const int u = ct * 4 + quarter;  // this warp's 32 columns
            const bool live = u < NU;
            const int pieces = (t.nrows + 15) / 16;
            const __half* sp = reinterpret_cast<const __half*>(a.wp + static_cast<size_t>(t.e) * a.expert_stride +
                                                               a.scale_offset) +
                               static_cast<size_t>(live ? u : 0) * groups * kExUnitN +
                               (lane & 7) * 4 + (lane >> 4) * 2 + ((lane >> 3) & 1);
            // lane l % 16 keeps the pair of that row of each piece
            int pair[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = (4 * i + part) * 16 + (lane & 15);
                pair[i] = r < t.nrows ? __ldg(a.rows + t.row0 + r) : -1;
            }
            float acc[2][16];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
            __half next = __ldg(sp);
            for (int g = 0; g < groups; ++g, ++m) {
                const float scale = __half2float(next);
                sp += kExUnitN;
                if (g + 1 < groups) next = __ldg(sp);
                ok = __all_sync(kFull, wait_phase(&bars.sum_full[m & 1], (m >> 1) & 1, ctl));
                if (!ok) break;
                tc_fence_after();
                const uint32_t from = tbase + (m & 1) * kRowsMax;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (4 * i + part < pieces) {
                        uint32_t d[16];
                        tmem_ld_x16(from + (4 * i + part) * 16, d);
                        tmem_ld_wait();
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[i][r] += scale * __uint_as_float(d[r]);
                    }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_leader(&bars.sum_empty[m & 1]);
            }
            if (!ok) break;
            // 16 rows x 32 columns at a time turned round in shared memory: rows of 64 (gated: 32)
            // bytes, so that a row leaves in 16-byte stores
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (4 * i + part >= pieces) continue;
                const int p_row = static_cast<unsigned>(pair[i]) < static_cast<unsigned>(a.pairs) ? pair[i] : -1;
                __syncwarp();
                if (!kPairs && a.gated) {
                    // gate lanes take the first 8 rows, up lanes the others
                    const bool up = lane & 8;
                    uint16_t* col = reinterpret_cast<uint16_t*>(out) + ((lane >> 4) * 8 + (lane & 7)) + (up ? 8 * (kYRowGated / 2) : 0);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float other = __shfl_xor_sync(kFull, up ? acc[i][r] : acc[i][r + 8], 8);
                        const float h = up ? silu_mul(other, acc[i][r + 8]) : silu_mul(acc[i][r], other);
                        col[r * (kYRowGated / 2)] = __half_as_ushort(__float2half_rn(h));
                    }
                    __syncwarp();
                    const int p = __shfl_sync(kFull, p_row, lane >> 1);
                    const int n = ct * (kColsL / 2) + quarter * 16 + (lane & 1) * 8;
                    const uint4 v4 = *reinterpret_cast<const uint4*>(out + (lane >> 1) * kYRowGated + (lane & 1) * 16);
                    if (p >= 0 && n < n_out) *reinterpret_cast<uint4*>(a.y + static_cast<size_t>(p) * n_out + n) = v4;
                } else if (kPairs) {
                    // 8 rows x 32 columns at a time, a row of 128 bytes
                    float* col = reinterpret_cast<float*>(out) + lane;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (k) __syncwarp();
#pragma unroll
                        for (int r = 0; r < 8; ++r) col[r * 32] = acc[i][k * 8 + r];
                        __syncwarp();
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int row = q * 4 + (lane >> 3);
                            const int p = __shfl_sync(kFull, p_row, k * 8 + row);
                            const int n = ct * kColsL + quarter * 32 + (lane & 7) * 4;
                            const uint4 v4 = *reinterpret_cast<const uint4*>(out + row * 128 + (lane & 7) * 16);
                            if (p >= 0 && n < n_out) *reinterpret_cast<uint4*>(a.y32 + static_cast<size_t>(p) * n_out + n) = v4;
                        }
                    }
                } else {
                    uint16_t* col = reinterpret_cast<uint16_t*>(out) + lane;
#pragma unroll
                    for (int r = 0; r < 16; ++r) col[r * (kYRow / 2)] = __half_as_ushort(__float2half_rn(acc[i][r]));
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int row = k * 8 + (lane >> 2);
                        const int p = __shfl_sync(kFull, p_row, row);
                        const int n = ct * kColsL + quarter * 32 + (lane & 3) * 8;
                        const uint4 v4 = *reinterpret_cast<const uint4*>(out + row * kYRow + (lane & 3) * 16);
                        if (p >= 0 && n < n_out) *reinterpret_cast<uint4*>(a.y + static_cast<size_t>(p) * n_out + n) = v4;
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // Both CTAs wait for every commit that nobody has waited for yet: the last k-block's of each stage, and
    // the drain, which a leader that gave up sends too. No MMA may run on freed tensor memory and no
    // arrival reach a CTA that has left. Only now, with the CTA's roles at their end: the limit is on
    // a wait, not on a call.
    if (warp == kMmaWarp) {
        const unsigned pairs = gridDim.x / 2;
        const long long tiles = static_cast<long long>(s_tiles[a.E]) * ((a.N + 2 * kColsL - 1) / (2 * kColsL));
        const unsigned blocks = static_cast<unsigned>((tiles + pairs - 1 - blockIdx.x / 2) / pairs) * (a.K / kTileK);
        if (lane < kStages && lane < blocks) wait_phase(&bars.empty[lane], ((blocks - lane - 1) / kStages) & 1, ctl);
        if (lane == kStages) wait_phase(&bars.drain, 0, ctl, false);
        __syncwarp();
    }
    cluster_sync();  // neither CTA leaves, or frees tensor memory, before both are done
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc2(tmem, 512);
    }
}

template <int SL>
cudaError_t configure_sl() {
    const cudaError_t e = cudaFuncSetAttribute(experts_large_kernel<SL, false>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemL);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(experts_large_kernel<SL, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemL);
}

template <int SL>
cudaError_t launch_sl(const LargeArgs& l, int grid, cudaStream_t st) {
    if (l.e.y32) experts_large_kernel<SL, true><<<grid, kLThreads, kSmemL, st>>>(l);
    else experts_large_kernel<SL, false><<<grid, kLThreads, kSmemL, st>>>(l);
    return cudaGetLastError();
}

}  // namespace

cudaError_t configure_experts_large() {
    cudaError_t e = configure_sl<0>();
    if (e == cudaSuccess) e = configure_sl<1>();
    if (e == cudaSuccess) e = configure_sl<2>();
    if (e == cudaSuccess) e = configure_sl<4>();
    return e;
}

cudaError_t launch_experts_large(const ExpertArgs& a, const DeviceInfo& d, cudaStream_t st) {
    const LargeArgs l{a, d.timeout_ns};
    const int grid = d.num_sms & ~1;
    if (a.g == a.K) return launch_sl<0>(l, grid, st);
    if (a.g == 64) return launch_sl<2>(l, grid, st);
    if (a.g == 32) return launch_sl<4>(l, grid, st);
    return launch_sl<1>(l, grid, st);
}

}  // namespace wq
