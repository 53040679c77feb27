// The dense products on the 5th-generation tensor cores (contract: lora_linear and lora_expert_linear in
// lora_delta.h): bf16 operands, fp32 sums in tensor memory.
//
// W's rows are the MMA's M side: a pair of blocks (cta_group::2) takes 256 features, each block loading its own 128; the
// rows of x are the N side, any multiple of 32 up to 256, each block loading half.  So a decode batch reads W once and
// computes no more than it must, a group of an expert's rows wastes at most 31 of a tile, and many rows get 256 x 256
// or 512 x 128 tiles (MT = 2: two feature blocks on one x tile: the gate's and the up projection's columns of a gated product,
// which then meet in one thread, or twice the features), 64 to 80 bytes of operands a clock and SM at the tensor cores' full rate.
//
// One persistent kernel for all sizes.  Tile t of cluster c: t = c, c + clusters, ....  Few tiles: a cluster is S pairs that
// split k, each cluster has one tile, and its blocks add their sums, in rank order, through distributed shared memory.
//
// Warp 0 copies W's boxes (and x's, plain product) by TMA; warp 1 of the first block of a pair issues the MMAs; eight warps
// read the accumulators (lane = feature, column = row of x), apply the epilogue and store, while the next tile's products go
// into the other accumulator.  Experts (GATHERED): four more warps copy the group's rows of x, wherever they lie, with
// cp.async into the same swizzle, 16 bytes a lane (gather4 copies of four rows x 128 bytes would be 32 a stage; a TMA copy
// costs its warp 40-60 ns); they count on the block's own barrier, from which one more warp of each block passes the word
// on to the first one's warp 1.
//
// Bound.  Few rows: HBM behind about 4 us that any call takes (1 x 4096 x 4096 9.4 us; 16 x 8192 x 28672 73.6 us = 6.4 TB/s;
// 8 experts of 4096 x 2 x 14336, 64 tokens, 290 us = 6.5 TB/s, 99 % of the measured copy rate).  Many rows: the tensor cores
// (8192 x 4096 x 2 x 14336 1190 us = 1620 TFLOP/s in a short burst, 1417 at the power cap; the issuing warp waits for no
// operands: 513 clocks a step of 512).  Between, 100 to 1000 rows: the operands' way into shared memory, about 64 bytes a
// clock and SM, and the exchange (257 x 14336 x 4096 34.7 us, its floor 19.7).  Many rows, few columns: the epilogue's latencies
// (4126 x 128 x 13536 74 us, 1.6 TB/s).  Many small experts (8192 tokens, 4 of 64, 2048 x
// 2 x 1024: 240 us): 630 clocks a step where dense rows take 513, at 1.35 GHz under the power cap.
//
// Measured and dropped: 16-bit accesses of y and the operands straight from tensor memory's layout (see the epilogue); one accumulator
// of 512 x 256 (8192 x 4096 x 2 x 14336 1380 us); W prefetched to L2 eight steps ahead (experts 262 -> 268, decode 291 -> 430);
// x in a deeper ring of its own (experts: no gain); the next 16 columns of tensor memory asked for ahead (4126 x 128 x 13536 72 -> 76).
#include "linear.cuh"
#include "pipe.cuh"

#include <algorithm>
#include <cstdlib>
#include <mutex>

namespace lora {

namespace {

constexpr int PAIR_STAGES = 12;
constexpr int PAIR_ROWS = 256;    // widest tile of x rows
constexpr int MAX_S = 4;          // most pairs that split k: clusters of eight blocks
// How a kernel's operands come: W and x by TMA; the experts' W by TMA, their rows of x by cp.async; both through registers
// (rows off 16-byte steps, with or without experts).
enum { PLAIN = 0, GATHERED = 1, LOADED = 2 };
constexpr int EPI_WARPS = 8;
constexpr uint32_t EPI_BYTES = 2048;   // of shared memory a warp of the epilogue
template <int MODE>
constexpr int load_warps() { return MODE == PLAIN ? 0 : MODE == GATHERED ? 4 : 8; }
template <int MODE>
constexpr int pair_threads() { return 32 * (2 + EPI_WARPS + load_warps<MODE>() + (MODE == GATHERED)); }
constexpr size_t PAIR_SMEM = 226 * 1024;   // all of the shared memory: one block an SM, as its tensor memory asks for
enum { STALL_MMA = 1, STALL_ROWS = 2, STALL_COPY = 3, STALL_SUMS = 4, STALL_COPY_FIRST = 5 };   // LORA_DEBUG_STALL

struct PairArgs {
    CUtensorMap tmW, tmX;
    LinArgs l;
    int gated;
    int up;              // rows of W between a tile's two feature blocks
    int bn;              // rows of a tile
    int m_tiles, n_tiles;   // tiles along the features; along x (plain product)
    int n_k;             // ring slots of k (KT steps of 64 columns each)
    int stages;          // ring slots
    int S;               // pairs that split k
    int own_red;         // the partial sums' place is behind the ring
    uint32_t epi_at;     // the epilogue's, behind both
    uint32_t table_at;   // experts: row tiles and slots before each, behind that
    int step;            // elements of an access to y, addend, residual and bias: 8, 2 or 1
    unsigned limit;
    int stall;
};

// Instruction descriptor: as idesc_bf16, with N known at run time
__device__ __forceinline__ uint32_t pair_idesc(int N) { return idesc_bf16(256, 8) - (1u << 17) + ((uint32_t)(N >> 3) << 17); }
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// 16 bytes, or zeros where bytes is 0
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrival on a barrier of another block of the cluster.  The rows it speaks for are read by the tensor core of this thread's
// own SM, for which its proxy fence has made them visible.  (A release and an acquire of the cluster's scope took 1.2 us a stage.)
__device__ __forceinline__ void mbar_arrive_peer(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

// A tile: its features from m0 (MT blocks of 256), its rows q0 .. q0 + cnt - 1 of expert e, n = rows of the MMA.
struct Tile {
    int m0, e, q0, cnt, n;
};

// What the epilogue adds to a thread's eight columns of a row (of MT feature blocks), and where the row lies.
template <int MT>
struct Operands {
    uint4 add[MT], res[MT];
    int64_t row;
};
// n (0 to 8) elements at p; step: elements of an access, 8, 2 or 1, of which n is a multiple.  At step 1 eight elements
// go as words all the same: four, or three between two halves where p is off a word.
__device__ __forceinline__ bool off_word(const void *p) { return reinterpret_cast<uintptr_t>(p) & 2; }
__device__ __forceinline__ uint4 load_cols(const __nv_bfloat16 *p, int n, int step) {
    if (step == 8) return n > 0 ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
    uint32_t w[4];
    if (step == 2 || (n == 8 && !off_word(p))) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = 2 * i < n ? *reinterpret_cast<const uint32_t *>(p + 2 * i) : 0u;
    } else if (n == 8) {
        uint32_t m[5];
        m[0] = (uint32_t)__bfloat16_as_ushort(p[0]) << 16;
#pragma unroll
        for (int i = 0; i < 3; ++i) m[i + 1] = *reinterpret_cast<const uint32_t *>(p + 1 + 2 * i);
        m[4] = __bfloat16_as_ushort(p[7]);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(m[i], m[i + 1], 16);
    } else {
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = i < n ? __bfloat16_as_ushort(p[i]) : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = h[2 * i] | h[2 * i + 1] << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_cols(__nv_bfloat16 *p, const uint4 &u, int n, int step) {
    if (step == 8) {
        if (n > 0) *reinterpret_cast<uint4 *>(p) = u;
        return;
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if (step == 2 || (n == 8 && !off_word(p))) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (2 * i < n) *reinterpret_cast<uint32_t *>(p + 2 * i) = w[i];
    } else if (n == 8) {
        p[0] = __ushort_as_bfloat16((unsigned short)w[0]);
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t *>(p + 1 + 2 * i) = __funnelshift_r(w[i], w[i + 1], 16);
        p[7] = __ushort_as_bfloat16((unsigned short)(w[3] >> 16));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = __ushort_as_bfloat16((unsigned short)(w[i >> 1] >> (16 * (i & 1))));
    }
}

// Rows of a block in the exchange of partial sums: a power of two up to 16, or a multiple of 16, so that 16 rows' owners
// follow from shifts or are one.
__host__ __device__ __forceinline__ int own_rows(int rows, int S) {
    const int fair = (rows + S - 1) / S;
    if (fair > 16) return (fair + 15) & ~15;
    int own = 1;
    while (own < fair) own *= 2;
    return own;
}

// 16 bytes from byte o (even) of 32: a, then b
__device__ __forceinline__ uint4 shift_bytes(const uint4 &a, const uint4 &b, uint32_t o) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = o & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = o & 4 ? w[i + 1] : w[i];
    const uint32_t s = (o & 2) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s),
                      __funnelshift_r(w[3], w[4], s));
}
__device__ __forceinline__ uint4 shfl4(const uint4 &v, int from) {
    return make_uint4(__shfl_sync(FULL, v.x, from), __shfl_sync(FULL, v.y, from), __shfl_sync(FULL, v.z, from),
                      __shfl_sync(FULL, v.w, from));
}

// uniform_wait for two barriers at once: each costs 100 clocks where it is complete already
__device__ __forceinline__ bool uniform_wait2(uint32_t a, uint32_t b, unsigned parity, const Bound &w, bool &failed) {
    for (unsigned it = 0; it < w.limit; ++it) {
        const bool x = mbar_try<false>(a, parity), y = mbar_try<false>(b, parity);
        if (__all_sync(FULL, x && y)) return true;
        if (__any_sync(FULL, stopped(w.stop))) break;
    }
    failed = true;
    return false;
}

template <int MODE, int MT, int KT>
__global__ void __launch_bounds__(pair_threads<MODE>(), 1) linear_pair_kernel(const __grid_constant__ PairArgs a) {
    extern __shared__ __align__(1024) unsigned char lin_sm[];
    __shared__ uint32_t tmem_sm;
    __shared__ __align__(8) uint64_t bars[4 * PAIR_STAGES + 6];
    __shared__ uint32_t stop_sm, used_sm;   // used_sm: ring uses that this block's copies have begun
    __shared__ int part[32];
    constexpr int FIRST_EPI = 2 + load_warps<MODE>();
    const bool grouped = MODE == GATHERED || (MODE == LOADED && a.l.perm);
    const int warp = __shfl_sync(FULL, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t w_bytes = 16384u * MT * KT, x_bytes = 64u * (uint32_t)a.bn, slot_bytes = w_bytes + x_bytes * KT;
    const uint32_t base = (smem_u32(lin_sm) + 1023u) & ~1023u, red = base + (a.own_red ? (uint32_t)a.stages * slot_bytes : 0u);
    const int rank = (int)cluster_rank(), S = a.S;
    const uint32_t half = rank & 1, first = rank & ~1;   // this block of the pair; the pair's first block
    const int cluster = (int)blockIdx.x / (2 * S), clusters = (int)gridDim.x / (2 * S);
    const int k_lo = a.n_k * (rank >> 1) / S, k_hi = a.n_k * ((rank >> 1) + 1) / S;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    auto full = [&](int s) { return bar(s); };                       // the first block's counts both blocks' TMA bytes
    auto empty = [&](int s) { return bar(PAIR_STAGES + s); };
    auto rows_in = [&](int s) { return bar(2 * PAIR_STAGES + s); };       // this block's gathered rows
    auto rows_ready = [&](int s) { return bar(3 * PAIR_STAGES + s); };    // the first block's: both blocks' rows (W's too, LOADED)
    auto acc_full = [&](int b) { return bar(4 * PAIR_STAGES + b); };
    auto acc_empty = [&](int b) { return bar(4 * PAIR_STAGES + 2 + b); };   // the first block's: eight warps of each block
    const uint32_t ready = bar(4 * PAIR_STAGES + 5);   // the first block's: the second has its tensor memory
    const uint32_t rest = bar(4 * PAIR_STAGES + 4);   // completes in the teardown after a wait that ran out, else never
    const Bound bound{smem_u32(&stop_sm), a.limit, a.l.status};
    bool failed = false;

    if (warp == 0) {
        for (int i = lane; i < 4 * PAIR_STAGES + 6; i += 32) {
            const int kind = i / PAIR_STAGES;   // 2: rows_in, 3: rows_ready
            const bool drained = i >= 4 * PAIR_STAGES + 2 && i < 4 * PAIR_STAGES + 4;
            mbar_init(bar(i), kind == 2 ? 32 * max(1, load_warps<MODE>()) : kind == 3 ? (MODE == LOADED ? 2 * load_warps<MODE>() : 2)
                                                                          : drained ? 2 * EPI_WARPS : 1);
        }
        if (lane == 0) {
            stop_sm = 0, used_sm = 0;
            if (MODE != LOADED) prefetch_tmap(&a.tmW);
            if (MODE == PLAIN) prefetch_tmap(&a.tmX);
        }
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    // The warps that copy need no more than the barriers of the cluster's blocks; tensor memory is got meanwhile.
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&tmem_sm)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
    }
    pdl_next();
    pdl_wait();   // all warps: none of the bounded waits below runs while the kernel before this one does
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    uint32_t tmem = 0;
    const bool sums = warp >= FIRST_EPI && warp < FIRST_EPI + EPI_WARPS;   // the warps of the epilogue
    if (warp == 1 || sums) {
        tc_fence_before();
        asm volatile("bar.sync 1, %0;\n" ::"n"(32 * (1 + EPI_WARPS)) : "memory");
        tc_fence_after();
        tmem = __shfl_sync(FULL, tmem_sm, 0);
        if (warp == 1 && half == 1 && elect_one()) mbar_arrive_peer(map_rank(ready, first));
    }
    int *const pre = reinterpret_cast<int *>(lin_sm + (base - smem_u32(lin_sm)) + a.table_at), *const start = pre + a.l.N + 1;
    int tiles = a.m_tiles * a.n_tiles;
    if (grouped) {
        count_tiles(a.l.seg_start, a.l.N, a.bn, pre, start, part);
        tiles = a.m_tiles * pre[a.l.N];
    }

    // Tiles run along x first: pairs at work at the same time share W's rows (and, in bands of 16 tiles of x, few enough
    // rows of x to find both in L2).
    int e_from = 0;   // a warp's tiles go up, and their experts
    auto place = [&](int t) {
        Tile p;
        int mi, rows;
        if (grouped) {
            p.e = e_from = expert_of(pre, a.l.N, (int)((unsigned)t / (unsigned)a.m_tiles), e_from);
            const int n = pre[p.e + 1] - pre[p.e], left = t - pre[p.e] * a.m_tiles;
            mi = (int)((unsigned)left / (unsigned)n);
            p.q0 = start[p.e] + (left - mi * n) * a.bn;
            rows = start[p.e + 1];
        } else {
            constexpr int BAND = 16;
            const int per = BAND * a.m_tiles, band = t / per, left = t - band * per, high = min(BAND, a.n_tiles - band * BAND);
            mi = left / high;
            p.e = 0;
            p.q0 = (band * BAND + left - mi * high) * a.bn;
            rows = a.l.T;
        }
        p.cnt = min(a.bn, rows - p.q0);
        p.n = (p.cnt + 31) & ~31;
        p.m0 = mi * (a.gated ? 256 : 256 * MT);
        return p;
    };
    const uint32_t tx = 2u * (MODE == GATHERED ? w_bytes : slot_bytes);

    if (MODE != LOADED && warp == 0) {
        Ring ring(a.stages);
        if (a.stall == (half ? STALL_COPY : STALL_COPY_FIRST)) uniform_wait(rest, 0, bound, failed);
        for (int t = cluster; t < tiles && !failed; t += clusters) {
            const Tile p = place(t);
            const int w0 = p.e * a.l.n_w + p.m0 + 128 * (int)half, x0 = p.q0 + (int)half * (p.n >> 1);
            for (int k = k_lo; k < k_hi; ++k, ring.next()) {
                if (ring.reused() && !uniform_wait(empty(ring.slot), ring.parity ^ 1u, bound, failed)) break;
                const uint32_t slot = base + (uint32_t)ring.slot * slot_bytes, b = map_rank(full(ring.slot), first);
                if (elect_one()) {
                    if (half == 0) mbar_expect_tx(full(ring.slot), tx);
#pragma unroll
                    for (int u = 0; u < MT; ++u)
#pragma unroll
                        for (int i = 0; i < KT; ++i) tma_2d_pair(slot + 16384u * (u + MT * i), &a.tmW, 64 * (k * KT + i), w0 + u * a.up, b);
                    if (MODE == PLAIN)
#pragma unroll
                        for (int i = 0; i < KT; ++i) tma_2d_pair(slot + w_bytes + x_bytes * i, &a.tmX, 64 * (k * KT + i), x0, b);
                }
            }
        }
        if (elect_one()) used_sm = ring.uses;
    } else if (warp == 1) {
        if (half == 0) {
            Ring ring(a.stages);
            int n = 0;
            uniform_wait(a.stall == STALL_MMA ? rest : ready, 0, bound, failed);
            for (int t = cluster; t < tiles && !failed; t += clusters, ++n) {
                const Tile p = place(t);
                const int b = n & 1, uses = n >> 1;   // accumulator buffer, its earlier uses
                if (uses > 0 && !uniform_wait(acc_empty(b), (unsigned)(uses - 1) & 1u, bound, failed)) break;
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(b * MT * a.bn), idesc = pair_idesc(p.n);
                for (int k = k_lo; k < k_hi; ++k, ring.next()) {
                    const int s = ring.slot;
                    if (!(MODE == GATHERED ? uniform_wait2(full(s), rows_ready(s), ring.parity, bound, failed)
                                           : uniform_wait(MODE == PLAIN ? full(s) : rows_ready(s), ring.parity, bound, failed)))
                        break;
                    tc_fence_after();
                    const uint32_t slot = base + (uint32_t)s * slot_bytes;
                    if (elect_one()) {
#pragma unroll
                        for (int x = 0; x < KT; ++x) {
                            const uint64_t dx = desc_sw128(slot + w_bytes + x_bytes * x);
#pragma unroll
                            for (int u = 0; u < MT; ++u) {
                                const uint64_t dw = desc_sw128(slot + 16384u * (u + MT * x));
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    pair_mma(d + (uint32_t)(u * a.bn), dw + 2 * i, dx + 2 * i, idesc, k == k_lo && x == 0 && i == 0 ? 0u : 1u);
                            }
                        }
                        tc_commit_pair(empty(s), first);
                    }
                }
                if (elect_one()) tc_commit_pair(acc_full(b), first);
            }
        }
    } else if (MODE == GATHERED && warp == FIRST_EPI + EPI_WARPS) {
        // Rows that came by cp.async (generic proxy) are made visible to the MMA, which reads them as operands; the word goes to the
        // first block's warp 1 from here, for which a fence of its own each step was too much.
        Ring ring(a.stages);
        for (int t = cluster; t < tiles && !failed; t += clusters)
            for (int k = k_lo; k < k_hi; ++k, ring.next()) {
                if (!uniform_wait(rows_in(ring.slot), ring.parity, bound, failed)) break;
                if (elect_one()) {
                    fence_proxy_async();
                    mbar_arrive_peer(map_rank(rows_ready(ring.slot), first));
                }
            }
    } else if (MODE == GATHERED && warp >= 2 && warp < FIRST_EPI) {
        // Lane l of warp w copies columns 8 (l % 8) .. of rows 16 i + 4 (w - 2) + l / 8 of this block's half.  Rows past the
        // group's last are not read: what the slot holds there only enters columns of the accumulator that no one stores.
        const int r0 = 4 * (warp - 2) + (lane >> 3), col = 8 * (lane & 7);
        const uint32_t at = (uint32_t)r0 * 128u + (uint32_t)(((lane & 7) ^ (r0 & 7)) << 4);
        Ring ring(a.stages);
        if (a.stall == STALL_ROWS && half && warp == 2) uniform_wait(rest, 0, bound, failed);
        // The slots of the next tile are asked for while this one's rows are copied.
        int slots[PAIR_ROWS / 32];
        auto ask = [&](int t) {
            const Tile p = place(t);
            const int own = p.n >> 1, in = min(own, p.cnt - (int)half * own);   // rows of this half, of them there
#pragma unroll
            for (int i = 0; i < PAIR_ROWS / 32; ++i) slots[i] = 16 * i + r0 < in ? a.l.perm[p.q0 + (int)half * own + 16 * i + r0] : -1;
        };
        if (cluster < tiles) ask(cluster);
        const float per = 1.f / (float)a.l.x_div;   // slots are below 2^17: (slot + 1/2) / x_div is off a whole number by far more than fp32's error
        for (int t = cluster; t < tiles && !failed; t += clusters) {
            const __nv_bfloat16 *src[PAIR_ROWS / 32];
#pragma unroll
            for (int i = 0; i < PAIR_ROWS / 32; ++i)
                src[i] = slots[i] < 0 ? nullptr
                                      : static_cast<const __nv_bfloat16 *>(a.l.x) + (int64_t)(int)(((float)slots[i] + 0.5f) * per) * a.l.ld_x + col;
            if (t + clusters < tiles) ask(t + clusters);
            for (int k = k_lo; k < k_hi; ++k, ring.next()) {
                if (ring.reused() && !uniform_wait(empty(ring.slot), ring.parity ^ 1u, bound, failed)) break;
                const uint32_t to = base + (uint32_t)ring.slot * slot_bytes + w_bytes + at;
#pragma unroll
                for (int x = 0; x < KT; ++x) {
                    const int at_k = 64 * (k * KT + x);
                    const uint32_t bytes = at_k + col < a.l.d_in ? 16u : 0u;   // d_in is a multiple of 8
#pragma unroll
                    for (int i = 0; i < PAIR_ROWS / 32; ++i)
                        if (src[i]) cp_async16z(to + x_bytes * x + 2048u * i, src[i] + (bytes ? at_k : 0), bytes);
                }
                cp_async_arrive(rows_in(ring.slot));
            }
        }
        asm volatile("cp.async.wait_all;\n" ::: "memory");
    } else if (MODE == LOADED && warp >= 2 && warp < FIRST_EPI) {
        // Rows at any (even) address: eight lanes read the aligned 16-byte pieces around 64 columns of a row, a ninth piece comes
        // from a load that a warp makes once for all its rows, and each lane shifts two neighbouring pieces into the 16 bytes
        // that the operand's swizzle wants.  Pieces that hold no column of the row are not read; of those at a row's ends up to
        // 14 bytes are not the row's.  They share 16 aligned bytes, so a page, with bytes that are, and are dropped.  (By halves
        // where a row ends: 64 x 4095 x 28672 162 -> 179 us, 33 x 129 x 2 x 4099 10.7 -> 19.3; only where x or w ends: 171, 18.6.)
        // Loads go out ahead of the wait for the slot; a slot's 32 KB in flight bound it, about 1 us a step (8192 x 4095 x 4096
        // 717 us = 383 TFLOP/s, where 4096 columns take 196).
        constexpr int W_IT = 4 * MT, X_IT = PAIR_ROWS / MT / 2 / 32, ITS = W_IT + X_IT, EXTRA = (ITS + 7) / 8;
        const int lw = warp - 2, lr = lane >> 3, c = lane & 7;   // rows 4 (lw + 8 i) + lr of W's, then of x's
        Ring ring(a.stages);
        if (a.stall == STALL_ROWS && half && warp == 2) uniform_wait(rest, 0, bound, failed);
        for (int t = cluster; t < tiles && !failed; t += clusters) {
            const Tile p = place(t);
            const int own = p.n >> 1, in = min(own, p.cnt - (int)half * own);   // rows of this half, of them there
            const char *src[ITS];   // rows' first bytes; what is not there reads a row that is
#pragma unroll
            for (int i = 0; i < ITS; ++i) {
                if (i < W_IT) {
                    const int f = 4 * (lw + 8 * (i & 3)) + lr;
                    const int64_t row = (int64_t)p.e * a.l.n_w + p.m0 + 128 * (int)half + f + (i >> 2) * a.up;
                    src[i] = reinterpret_cast<const char *>(static_cast<const __nv_bfloat16 *>(a.l.w) +
                                                            min(row, (int64_t)a.l.N * a.l.n_w - 1) * a.l.ld_w);
                } else {
                    const int r = 4 * (lw + 8 * (i - W_IT)) + lr, q = p.q0 + (in > 0 ? (int)half * own + min(r, in - 1) : 0);
                    src[i] = reinterpret_cast<const char *>(static_cast<const __nv_bfloat16 *>(a.l.x) +
                                                            (int64_t)(grouped ? a.l.perm[q] / a.l.x_div : q) * a.l.ld_x);
                }
            }
            const char *more[EXTRA];   // lane 4 i + r: row r of turn i (then i + 8)
#pragma unroll
            for (int x = 0; x < EXTRA; ++x) {
                more[x] = nullptr;
#pragma unroll
                for (int i = 8 * x; i < (ITS < 8 * x + 8 ? ITS : 8 * x + 8); ++i) {
                    const uint64_t got = __shfl_sync(FULL, reinterpret_cast<uint64_t>(src[i]), 8 * (lane & 3));
                    if (lane >> 2 == (i & 7)) more[x] = reinterpret_cast<const char *>(got);
                }
            }
            const int64_t row_bytes = 2 * (int64_t)a.l.d_in;
            auto piece = [&](const char *row, int64_t at) {   // the aligned 16 bytes around byte `at` of a row
                const char *s = reinterpret_cast<const char *>(reinterpret_cast<uint64_t>(row + at) & ~15ull);
                return row && s < row + row_bytes ? *reinterpret_cast<const uint4 *>(s) : make_uint4(0, 0, 0, 0);
            };
            for (int k = k_lo; k < k_hi; ++k, ring.next()) {
                uint4 v[ITS], ninth[EXTRA];
#pragma unroll
                for (int i = 0; i < ITS; ++i)
                    if (i < W_IT || 32 * (i - W_IT) < own) v[i] = piece(src[i], 128 * (int64_t)k + 16 * c);
#pragma unroll
                for (int x = 0; x < EXTRA; ++x) ninth[x] = piece(more[x], 128 * (int64_t)k + 128);
                if (ring.reused() && !uniform_wait(empty(ring.slot), ring.parity ^ 1u, bound, failed)) break;
                const uint32_t slot = base + (uint32_t)ring.slot * slot_bytes;
                const int keep = max(0, min(8, a.l.d_in - 64 * k - 8 * c));   // columns past d_in: zeros on both sides
#pragma unroll
                for (int i = 0; i < ITS; ++i)
                    if (i < W_IT || 32 * (i - W_IT) < own) {
                        const uint4 up = shfl4(v[i], (lane + 1) & 31), last = shfl4(ninth[i >> 3], 4 * (i & 7) + lr);
                        const uint4 out = keep8(shift_bytes(v[i], c == 7 ? last : up, (uint32_t)reinterpret_cast<uint64_t>(src[i]) & 15u), keep);
                        const int r = 4 * (lw + 8 * (i < W_IT ? i & 3 : i - W_IT)) + lr;
                        const uint32_t at = slot + (i < W_IT ? 16384u * (i >> 2) : w_bytes) + 128u * (uint32_t)r;
                        if (i < W_IT || r < own) sts128(at + (uint32_t)((c ^ (r & 7)) << 4), out);
                    }
                fence_proxy_async();   // the MMA reads what these stores wrote
                __syncwarp();
                if (elect_one()) mbar_arrive_peer(map_rank(rows_ready(ring.slot), first));
            }
        }
    } else if (sums) {
        // A warp reads 32 lanes of tensor memory: features f, a row of x in each column.  Through shared memory of its own, eight
        // or 16 rows at a time, a thread gets eight columns of one row, four neighbours the warp's 32: one 16-byte access of each
        // operand and of y where there were eight of two bytes, each with its address.  (As they lie in tensor memory: 256 rows
        // 5.5 us for 256 features, and a chunk's operands, loaded one after the other, up to 0.5 us a row; 8192 x 1024 x 4096
        // with a residual: eight rows at a time 110 us, 16 79.)
        const int q = warp & 3, f = 32 * q + lane;
        const int side = warp >= FIRST_EPI + 4;             // which of the two warps of these lanes
        const int l_row = lane >> 2, l_col = 32 * q + 8 * (lane & 3);   // this thread's row of eight and columns
        const uint32_t buf = base + a.epi_at + (uint32_t)(warp - FIRST_EPI) * EPI_BYTES;
        const LinArgs &l = a.l;
        __nv_bfloat16 *const y = static_cast<__nv_bfloat16 *>(l.y);
        const __nv_bfloat16 *const add = static_cast<const __nv_bfloat16 *>(l.addend);
        const __nv_bfloat16 *const res = static_cast<const __nv_bfloat16 *>(l.residual);
        const __nv_bfloat16 *const bias = static_cast<const __nv_bfloat16 *>(l.bias);
        const int step = a.step;
        int n = 0;
        for (int t = cluster; t < tiles && !failed; t += clusters, ++n) {
            const Tile p = place(t);
            const int b = n & 1, uses = n >> 1;   // accumulator buffer, its earlier uses
            const int m = p.m0 + 128 * (int)half + l_col;   // this thread's columns of y; the second block's are m + up
            const int n0 = min(8, max(0, l.d_out - m)), n1 = MT == 1 ? 0 : a.gated ? n0 : min(8, max(0, l.d_out - m - a.up));
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(b * MT * a.bn);
            uint4 bz[MT];
#pragma unroll
            for (int u = 0; u < MT; ++u)
                bz[u] = bias ? load_cols(bias + (int64_t)p.e * l.n_w + m + u * a.up, u ? n1 : n0, step) : make_uint4(0, 0, 0, 0);

            auto fetch = [&](Operands<MT> &o, int r) {   // for tile row r (past the last: the last one again)
                const int at = p.q0 + min(r, p.cnt - 1);
                o.row = grouped ? l.perm[at] : at;
                if (add) {
                    o.add[0] = load_cols(add + o.row * l.ld_a + m, n0, step);
                    if (MT == 2) o.add[MT - 1] = load_cols(add + o.row * l.ld_a + m + a.up, n1, step);
                }
                if (res) {
                    o.res[0] = load_cols(res + o.row * l.ld_r + m, n0, step);
                    if (MT == 2 && !a.gated) o.res[MT - 1] = load_cols(res + o.row * l.ld_r + m + a.up, n1, step);
                }
            };
            auto plus = [](float *z, const uint4 &u) {
                float v[8];
                raw_values(u, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] += v[i];
            };
            auto finish = [&](float (&z)[MT][8], const Operands<MT> &o, bool there) {   // sums of eight columns to y
#pragma unroll
                for (int u = 0; u < MT; ++u) {
                    if (bias) plus(z[u], bz[u]);
                    if (add) plus(z[u], o.add[u]);
                }
                activate<true, 8>(l.act, z[0]);
                uint4 out;
                __nv_bfloat16 *to = y + o.row * l.ld_y + m;
                if (MT == 2) {
                    if (a.gated) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) z[0][i] *= z[MT - 1][i];
                    } else {
                        activate<true, 8>(l.act, z[MT - 1]);
                        if (res) plus(z[MT - 1], o.res[MT - 1]);
                        raw_round(z[MT - 1], out);
                        if (there) store_cols(to + a.up, out, n1, step);
                    }
                }
                if (res) plus(z[0], o.res[0]);
                raw_round(z[0], out);
                if (there) store_cols(to, out, n0, step);
            };
            // eight floats of a row of 128 bytes (buf) or 512 (partial sums); odd rows take their halves the other way round, so
            // that eight threads meet no bank twice
            auto load_row = [&](float *z, uint32_t at) {
                const float4 x = lds128f(at + 16u * (l_row & 1)), w = lds128f(at + 16u * (~l_row & 1));
                const float4 lo = l_row & 1 ? w : x, hi = l_row & 1 ? x : w;
                z[0] = lo.x, z[1] = lo.y, z[2] = lo.z, z[3] = lo.w, z[4] = hi.x, z[5] = hi.y, z[6] = hi.z, z[7] = hi.w;
            };
            auto drained = [&] {   // this warp's part of the accumulator is in registers
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_rank(acc_empty(b), first));
            };
            // the two warps of the same lanes take half of the columns each; after an exchange, every other eight rows of the
            // block's own.  Operands are fetched 16 rows ahead (8: 8192 x 1024 x 4096 with a residual 81 us, without 68), the first before
            // the sums are there.
            const int own = own_rows(p.cnt, S), mine = rank >> 1, r_lo = mine * own, rows = min(own, p.cnt - r_lo);
            const int c_lo = side * (p.n >> 1), c_hi = min(c_lo + (p.n >> 1), p.cnt);
            Operands<MT> o[2];
            fetch(o[0], S > 1 ? r_lo + 8 * side + l_row : c_lo + l_row);
            if (S == 1) fetch(o[1], c_lo + 8 + l_row);
            // S > 1: on to the exchange all the same, which every block of the cluster takes part in
            const bool stall = a.stall == STALL_SUMS && half == 1 && warp == FIRST_EPI;
            if (!lanes_wait(stall ? rest : acc_full(b), (unsigned)uses & 1u, bound, failed) && S == 1) break;
            tc_fence_after();
            if (S == 1) {
                for (int c = c_lo; c < c_hi; c += 16) {
                    float v[MT][16];
#pragma unroll
                    for (int u = 0; u < MT; ++u) tc_ld16(acc + (uint32_t)(u * a.bn + c), v[u]);
                    tc_wait_ld();
                    if (c + 16 >= c_hi) drained();
                    // 16 rows of one feature block at a time, or eight of two
#pragma unroll
                    for (int h = 0; h < 16; h += 16 / MT)
                        if (c + h < c_hi) {
                            __syncwarp();
#pragma unroll
                            for (int u = 0; u < MT; ++u)
#pragma unroll
                                for (int j = 0; j < 16 / MT; ++j) sts32(buf + 1024u * u + 128u * j + 4u * lane, __float_as_uint(v[u][h + j]));
                            __syncwarp();
                            float z[2 / MT][MT][8];
#pragma unroll
                            for (int g = 0; g < 2 / MT; ++g)
#pragma unroll
                                for (int u = 0; u < MT; ++u) load_row(z[g][u], buf + 1024u * (g + u) + 128u * (uint32_t)l_row + 32u * (lane & 3));
#pragma unroll
                            for (int g = 0; g < 2 / MT; ++g) {
                                const int at = h / 8 + g;   // eight rows from c + 8 at
                                const Operands<MT> now = o[at];
                                if (c + 8 * at + 16 < c_hi) fetch(o[at], c + 8 * at + 16 + l_row);
                                finish(z[g], now, c + 8 * at + l_row < c_hi);
                            }
                        }
                }
                if (c_lo >= c_hi) drained();
            } else {
                const int own_log2 = 31 - __clz(own);
                // [feature block][source][row of own][128 features], in each owner's shared memory
                const uint32_t part_bytes = 512u * (uint32_t)own, block_bytes = part_bytes * (uint32_t)S;
                const uint32_t to0 = red + (uint32_t)mine * part_bytes + 4u * (uint32_t)f;
                if (!a.own_red) cluster_sync_all();   // every block's products are done with its ring
                for (int c = 16 * side; c < p.cnt; c += 32) {
                    float z[MT][16];
#pragma unroll
                    for (int u = 0; u < MT; ++u) tc_ld16(acc + (uint32_t)(u * a.bn + c), z[u]);
                    tc_wait_ld();
                    // 16 rows have one owner, or owners that follow from shifts
                    if (own >= 16) {
                        const int owner = c / own;
                        const uint32_t at = map_rank(to0, 2u * (uint32_t)owner + half) + 512u * (uint32_t)(c - owner * own);
#pragma unroll
                        for (int u = 0; u < MT; ++u)
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (c + j < p.cnt) st_cluster(at + (uint32_t)u * block_bytes + 512u * j, z[u][j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const uint32_t at = map_rank(to0, 2u * ((uint32_t)(c + j) >> own_log2) + half) + 512u * ((c + j) & (own - 1));
                            if (c + j < p.cnt)
#pragma unroll
                                for (int u = 0; u < MT; ++u) st_cluster(at + (uint32_t)u * block_bytes, z[u][j]);
                        }
                    }
                }
                cluster_sync_all();
                for (int r = 8 * side; r < rows; r += 16) {
                    const uint32_t at = red + 512u * (uint32_t)min(r + l_row, rows - 1) + 4u * (uint32_t)l_col;
                    float z[MT][8];
#pragma unroll
                    for (int u = 0; u < MT; ++u) load_row(z[u], at + (uint32_t)u * block_bytes);
                    for (int s = 1; s < S; ++s)
#pragma unroll
                        for (int u = 0; u < MT; ++u) {
                            float v[8];
                            load_row(v, at + (uint32_t)u * block_bytes + (uint32_t)s * part_bytes);
#pragma unroll
                            for (int i = 0; i < 8; ++i) z[u][i] += v[i];
                        }
                    const Operands<MT> now = o[0];
                    if (r + 16 < rows) fetch(o[0], r_lo + r + 16 + l_row);
                    finish(z, now, r + l_row < rows);
                }
                drained();
            }
        }
    }
    // ---------------------------------------------------------------- teardown
    __syncwarp();
    leave<true>(bound, failed, first);
    if (S > 1 && !sums && cluster < tiles) {   // the barriers of the exchange, for the warps that take no part in it
        if (!a.own_red) cluster_sync_all();
        cluster_sync_all();
    }
    tc_fence_before();
    cluster_sync_all();
    if (stop_sm) {   // a wait ran out: in both blocks of the pair, which stopped where they were
        if (warp == 0 && half == 0) {
            // The first block's barriers count both blocks' bytes.  The uses that one block has begun and the other not (at
            // most one a slot) complete with the bytes of that one.
            Ring r(a.stages, used_sm);
            uint32_t other;
            asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(other) : "r"(map_rank(smem_u32(&used_sm), first + 1)) : "memory");
            for (uint32_t k = other; k < r.uses; ++k)
                if (elect_one()) mbar_complete_tx(full((int)(k % (unsigned)a.stages)), tx / 2);
            for (; r.uses < other; r.next())
                if (elect_one()) mbar_expect_tx(full(r.slot), tx / 2);
            drain_ring(r, full(0));
        } else if (warp == 1) {   // the products read both blocks' memory and tensor memory
            if (half == 0 && elect_one()) tc_commit_pair(rest, first);
            rest_wait(rest, 0);
        }
    }
    if (stop_sm) cluster_sync_all();   // of those that are still here: both blocks of the pair
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
    }
}

// A shape of the tiles and what the call would take with it.
struct PairPlan {
    int mt = 0, bn = 0, kt = 0, S = 1, clusters = 1;
    int64_t ns = 0;
};

// clusters resident at once, of 1 to 4 pairs: a property of the device and the kernel, asked for once
template <int MODE, int MT, int KT>
int pair_fit(int dev, const int **fit) {
    static std::mutex mu;
    static int table[64][MAX_S] = {};
    std::lock_guard<std::mutex> lock(mu);
    int *f = table[dev & 63];
    auto kernel = linear_pair_kernel<MODE, MT, KT>;
    if (!f[0]) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PAIR_SMEM);
        for (int i = MAX_S - 1; i >= 0 && e == cudaSuccess; --i) {   // f[0] last: it marks the table as filled
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(2u * (i + 1));
            cfg.blockDim = dim3(pair_threads<MODE>());
            cfg.dynamicSmemBytes = PAIR_SMEM;
            cudaLaunchAttribute attr{};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = 2u * (i + 1);
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            if (e == cudaSuccess) f[i] = i ? n : std::max(1, n);
        }
        if (e != cudaSuccess) return cuda_rc(e);
    }
    *fit = f;
    return LORA_OK;
}

int m_tiles_of(const LinArgs &l, bool gated, int mt) { return (l.d_out + (gated ? 256 : 256 * mt) - 1) / (gated ? 256 : 256 * mt); }

// Two 64-column steps to a ring slot while three slots fit: half the waits (257 x 14336 x 4096, 96-row tiles: 55.3 -> 50.1 us).
bool two_steps(int mt, int bn) { return mt == 1 ? bn <= 160 : bn <= 32; }

// The best split of k for tiles of bn rows; row_tiles: as many as there may be, likely: as many as are expected.  The times
// are those of the cases below, whose plan was the best of all within 7 % (us; MT, rows of a tile, S): 1 x 4096 x 4096 9.3 (1, 32, 3), S = 2
// 10.0; 64 x 4096 x 4096 10.8 (1, 32, 2); 128 x 14336 x 4096 26.9 (1, 128, 3), S = 1 50; 257 x 14336 x 4096 34.7 (1, 160, 2), S = 1 58,
// (1, 96, 1) 42.6; 512 x 14336 x 4096 49.4 (1, 256, 2); 1024 x 4096 x 4096 29.3 (1, 256, 1); 4096 x 4096 x 4096 97 (2, 128, 1),
// (1, 256, 1) 100.  8 % off: 512 x 4096 x 4096 21.0 for 18.9 (1, 128, 1), 1024 x 14336 x 4096 93 for 85 (1, 256, 1).
template <int MODE, int MT, int KT>
int consider(const LinArgs &l, bool gated, int bn, int64_t row_tiles, int64_t likely, int dev, PairPlan *best) {
    const int *fit = nullptr;
    const int rc = pair_fit<MODE, MT, KT>(dev, &fit);
    if (rc != LORA_OK) return rc;
    const int64_t m = m_tiles_of(l, gated, MT), n_k = (l.d_in + 64 * KT - 1) / (64 * KT);
    // a 64-column step: its products, its copies into shared memory, or what a step takes at least (ns); rows off 16-byte steps: 1000
    // whatever the tile, which chose the best plan of all at 8192 x 4095 x 4096, 2048 x 2047 x 2 x 2048, 257 x 14335 x 4096, 700 x 1001 x 600, 64 x
    // 4095 x 28672 and 64 x 4095 x 2 x 4096, but (2, 32, 4), 42 us, for (1, 32, 3), 28, at 1 x 4095 x 4096
    const int64_t step = std::max<int64_t>({(int64_t)MT * bn * 8 / 7, (16384 * MT + 64 * bn) / 112, MODE == LOADED ? 1000 : 90});
    const int64_t sums = 500 + 25 * bn * MT;   // a tile's epilogue, beside the next tile's products
    const int64_t hbm = ((int64_t)std::min<int64_t>(l.N, likely) * l.n_w * l.d_in + (int64_t)l.T * (l.d_in + l.d_out)) * 2 / 6400;
    const int rows = std::min(bn, l.T);
    for (int s = 1; s <= MAX_S && s <= n_k; ++s) {
        const int64_t tiles = m * row_tiles, expect = m * likely;
        if (s > 1 && tiles > fit[s - 1]) break;   // a cluster that splits k has one tile
        if (s > 1 && bn > 32 && (size_t)own_rows(rows, s) * s * 512 * MT > PAIR_SMEM - 1024) continue;
        const int64_t clusters = std::min<int64_t>(tiles, fit[s - 1]);
        const int64_t rounds = (expect + clusters - 1) / clusters;
        const int64_t k_ns = (n_k + s - 1) / s * KT * step;
        const int64_t ns = 3500 + std::max(hbm, rounds * std::max(k_ns, sums)) + 14 * rows * MT + (s > 1 ? 500 + 8 * rows * MT : 0);
        if (!best->mt || ns < best->ns) best->mt = MT, best->kt = KT, best->bn = bn, best->S = s, best->clusters = (int)clusters, best->ns = ns;
    }
    return LORA_OK;
}

template <int MODE, int MT, int KT>
int launch_pair(PairArgs &a, const PairPlan &plan, cudaStream_t st) {
    a.bn = plan.bn, a.S = plan.S;
    a.up = a.gated ? a.l.d_out : 256;
    a.m_tiles = m_tiles_of(a.l, a.gated, MT);
    a.own_red = plan.S > 1 && plan.bn <= 32;
    a.n_k = (a.l.d_in + 64 * KT - 1) / (64 * KT);
    a.step = a.l.d_out % 8 == 0 ? 8 : a.l.d_out % 2 == 0 ? 2 : 1;
    auto allow = [&](const void *p, int64_t ld) {   // rows of ld elements at p
        while (p && a.step > 1 && (!mx_aligned(p, 2 * a.step) || ld % a.step)) a.step = a.step == 8 ? 2 : 1;
    };
    allow(a.l.y, a.l.ld_y), allow(a.l.addend, a.l.ld_a), allow(a.l.residual, a.l.ld_r), allow(a.l.bias, 0);
    const size_t slot = (16384u * MT + 64u * (size_t)plan.bn) * KT, red = a.own_red ? (size_t)own_rows(plan.bn, plan.S) * 512 * MT * plan.S : 0;
    const size_t table = a.l.perm ? 8 * (size_t)(a.l.N + 1) : 0;
    const size_t epi = plan.S > 1 ? 0 : EPI_WARPS * EPI_BYTES;   // sums of an exchange lie as the epilogue wants them
    a.stages = (int)std::min<size_t>(PAIR_STAGES, (PAIR_SMEM - 1024 - epi - table - red) / slot);
    a.epi_at = (uint32_t)(a.stages * slot + red);
    a.table_at = (uint32_t)(a.epi_at + epi);
    return launch_after(linear_pair_kernel<MODE, MT, KT>, dim3((unsigned)(plan.clusters * 2 * plan.S)), pair_threads<MODE>(),
                        PAIR_SMEM, 2u * plan.S, st, a);
}

template <int MODE>
int consider_mt(int mt, const LinArgs &l, bool gated, int bn, int64_t row_tiles, int64_t likely, int dev, PairPlan *best) {
    if constexpr (MODE == LOADED) {
        return mt == 1 ? consider<MODE, 1, 1>(l, gated, bn, row_tiles, likely, dev, best)
                       : consider<MODE, 2, 1>(l, gated, bn, row_tiles, likely, dev, best);
    } else {
        if (mt == 1)
            return two_steps(1, bn) ? consider<MODE, 1, 2>(l, gated, bn, row_tiles, likely, dev, best)
                                    : consider<MODE, 1, 1>(l, gated, bn, row_tiles, likely, dev, best);
        return two_steps(2, bn) ? consider<MODE, 2, 2>(l, gated, bn, row_tiles, likely, dev, best)
                                : consider<MODE, 2, 1>(l, gated, bn, row_tiles, likely, dev, best);
    }
}
template <int MODE>
int launch_plan(PairArgs &a, const PairPlan &p, cudaStream_t st) {
    if constexpr (MODE == LOADED) {
        return p.mt == 1 ? launch_pair<MODE, 1, 1>(a, p, st) : launch_pair<MODE, 2, 1>(a, p, st);
    } else {
        if (p.mt == 1) return p.kt == 1 ? launch_pair<MODE, 1, 1>(a, p, st) : launch_pair<MODE, 1, 2>(a, p, st);
        return p.kt == 1 ? launch_pair<MODE, 2, 1>(a, p, st) : launch_pair<MODE, 2, 2>(a, p, st);
    }
}

int round32(int64_t n) { return (int)((n + 31) / 32 * 32); }

// Rows of x and W in the 16-byte steps that TMA and 16-byte copies take.
bool whole_steps(const LinArgs &a, int64_t x_rows) {
    return (a.d_in & 7) == 0 && (x_rows <= 1 || (a.ld_x & 7) == 0) && (a.ld_w & 7) == 0 && mx_aligned(a.x, 16) && mx_aligned(a.w, 16);
}

}  // namespace

int launch_linear_tc(const LinArgs &l, int64_t x_rows, bool gated, int dev, cudaStream_t st) {
    PairArgs a{};
    a.l = l;
    a.gated = gated;
    const char *stall = std::getenv("LORA_DEBUG_STALL");   // test hook: the waits of one role run out, after a short while
    a.stall = stall ? std::atoi(stall) : 0;
    a.limit = a.stall ? 64 : WAIT_LIMIT;
    PairPlan best;
    int rc = LORA_OK;
    const bool gather = l.perm != nullptr;
    const int mode = !whole_steps(l, x_rows) ? LOADED : gather ? GATHERED : PLAIN;
    auto consider_tiles = [&](int mt, int bn, int64_t tiles, int64_t likely) {
        if (mode == LOADED) return consider_mt<LOADED>(mt, l, gated, bn, tiles, likely, dev, &best);
        return mode == GATHERED ? consider_mt<GATHERED>(mt, l, gated, bn, tiles, likely, dev, &best)
                                : consider_mt<PLAIN>(mt, l, gated, bn, tiles, likely, dev, &best);
    };
    for (int mt = gated ? 2 : 1; mt <= 2 && rc == LORA_OK; ++mt) {
        // rows that two accumulator buffers hold: with one (MT = 2, 256 rows) 8192 x 4096 x 2 x 14336 took 1380 us for 1200
        const int most = PAIR_ROWS / mt;
        if (gather) {   // tiles that most groups fit in
            const int64_t groups = std::min(l.N, l.T), mean = (l.T + groups - 1) / groups;
            const int bn = std::min(most, round32(mean + mean / 2));
            rc = consider_tiles(mt, bn, l.T / bn + groups, std::max<int64_t>(groups, l.T / bn + groups / 2));
            continue;
        }
        const int least = (l.T + most - 1) / most;
        for (int nt = least; nt <= least + 2 && rc == LORA_OK; ++nt) {   // the fewest row tiles, or a little more that fill the SMs better
            const int bn = round32((l.T + nt - 1) / nt), n = (l.T + bn - 1) / bn;
            rc = consider_tiles(mt, bn, n, n);
            if (bn == 32) break;
        }
    }
    if (rc != LORA_OK) return rc;
    if (mode != LOADED) rc = tensor_map_rows(&a.tmW, l.w, (uint64_t)l.d_in, (uint64_t)l.N * l.n_w, (uint64_t)l.ld_w, 128);
    if (rc == LORA_OK && mode == PLAIN)   // one row's stride is of no use, and need not be one that a map takes
        rc = tensor_map_rows(&a.tmX, l.x, (uint64_t)l.d_in, (uint64_t)l.T, (uint64_t)(l.T > 1 ? l.ld_x : l.d_in), (uint32_t)best.bn / 2);
    if (rc != LORA_OK) return rc;
    a.n_tiles = gather ? 0 : (l.T + best.bn - 1) / best.bn;
    if (mode == LOADED) return launch_plan<LOADED>(a, best, st);
    return mode == GATHERED ? launch_plan<GATHERED>(a, best, st) : launch_plan<PLAIN>(a, best, st);
}

}  // namespace lora
