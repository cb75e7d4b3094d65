// Products of MXFP4 experts with many rows each (tcgen05 kernel).
//
// y[s][n] = sum_k w[n][k] x[s][k] with the weights as operand A (256 rows of
// a tcgen05.mma over a pair of SMs, from tensor memory) and up to 160
// rows of x as operand B (half in each SM's shared memory).  Both are halves: a
// code times its scale relative to the row's largest, times 2^13, is one
// exactly (a row with a scale below 2^-27 is marked, and computed at the end); fp16 rows are what they are;
// bf16 rows go by a power of two that brings the row's largest finite element
// to [2^14, 2^15), which keeps every element to 2^-39 of it (all eight bits of
// those within 2^-31), fp32 rows as two such terms, in a pass of its own.  (As
// bf16 numbers the weights take 19 instructions a word instead of 8, and
// bound the kernel: 1240 clocks a step of 660.)  The codes go from the pack's words
// to tensor memory as fragments (16x256b): that operand costs no
// shared-memory bandwidth, and the pair halves what the other one costs.
// Sums are the tensor core's, in fp32 (of fp32 rows, those of 256 values each); the epilogue multiplies by the powers of two.
//
// In each CTA of a pair 12 warps convert weights (32 rows of tensor memory
// each, every third step), 3 gather rows of x by asynchronous copies into
// 128-byte-swizzled shared memory (TMA's gather of four rows takes twice as long), 4 write
// results while the next item's products run (two accumulators); one thread
// of the first CTA issues the products for both.  256 rows of weights (128 of gate and of up,
// 16 by 16, so that a warp has both of a row) by one row tile is an item;
// items go round-robin over pairs, row tiles of an expert are of even size, N
// is the row tile's count rounded up to 32.
//
// Bound by the tensor pipe where K is long: 4096 tokens of 6 of 64 experts, gate
// and up of 1408 x 5120, 709 GFLOP in 429 us, 1.65 PFLOP/s (call after call, under the power cap,
// 490 us, 1.45).  Where K is short the results
// take as long (down of 5120 x 1408: 11 steps an item, 379 us with the pass over h and the sum).  A
// product of 16 values of K takes 75 clocks for any N up to 160, that of its 256 rows
// of weights: 64 experts of 12 rows take 126 us for their 490 MB.
#pragma once

#include "mx_gemm.cuh"
#include "mx_row_tile.cuh"

namespace qgemv {

constexpr int MXT_CONVERT = 12, MXT_EPI = 4, MXT_EPI_WARP = 12, MXT_MMA_WARP = 16, MXT_LOAD_WARP = 17, MXT_LOAD = 3;
constexpr int MXT_THREADS = (MXT_LOAD_WARP + MXT_LOAD) * 32;
// Rows of x an item: two accumulators of that many columns, and for fp32 rows their sums.
template <int TERMS>
constexpr int MXT_ROWS = TERMS == 1 ? 160 : 96;
// Steps of fp32 rows that an accumulator takes.  The tensor core cuts what does not fit its sum's 24
// bits, always towards zero, by up to 2^-23 for a product of 16 values: 5120 values of one sign in one accumulator
// come out 9e-6 too small, 32768 (the longest) 1.2e-4.  16-bit rows are summed so: their outputs'
// half steps are 4.9e-4 and 3.9e-3, and sums apart would leave tensor memory for 96 rows an item
// in place of 160.  Of fp32 rows every two steps (256 values) are added up by the
// results' warps, rounding to nearest, in tensor memory: 3e-7 off, and 64 experts of 768 x 2048,
// gate and up, 16 rows each, take 53 us for 50, 32 rows 60 for 53.
constexpr int MXT_CHUNK = 2;
static_assert(MXT_ROWS<1> % MXT_N_STEP == 0 && MXT_ROWS<2> % MXT_N_STEP == 0, "whole products");
constexpr int MXT_A_STAGES = 3;  // of two units, 64 columns each: what hides a round trip between the roles
static_assert(MXT_CONVERT == 4 * MXT_A_STAGES, "a warpgroup a stage");
// Registers a thread: 640 of 96 at launch, of which the results' warpgroup gets 24 each of the last one's.
constexpr int MXT_REGS = 96, MXT_EPI_REGS = 120, MXT_REST_REGS = 72;
static_assert(MXT_THREADS == 640 && MXT_CONVERT * MXT_REGS + MXT_EPI * MXT_EPI_REGS + 4 * MXT_REST_REGS == 20 * MXT_REGS, "register shares");
constexpr uint32_t MXT_A_COL = 320;
static_assert(2 * MXT_ROWS<1> <= MXT_A_COL && 3 * MXT_ROWS<2> <= MXT_A_COL, "accumulators");
static_assert(MXT_A_COL + MXT_A_STAGES * 64 <= 512, "tensor memory");
constexpr long long MXT_WAIT_CLOCKS = 2000000000;  // about a second
constexpr int MXT_SHIFT = 13;                      // the scales in A are 2^13 times what they are

// Items whose slots and powers of two are in shared memory: a warp that writes results may be
// ahead of another by two (an accumulator that is free again takes all of them).
constexpr int MXT_SETS = 3;
constexpr int MXT_EPI_BYTES = 2 * 16 * 128 * 4;  // two halves of 16 columns of results

// For rows of x of so many terms: the ring for them, batches of steps, a step
// being half a row tile of two units of 64 values (a batch is announced and given
// back as one), and the steps of a converting warp's own ring of codes.
template <int TERMS>
struct MxtShape {
    static constexpr int BATCH = TERMS == 1 ? 2 : 1, BATCHES = 3, AHEAD = 2;
};

struct MxtRows {
    const __half* x;  // row r of term i at x + i * plane + r * ld, 16-byte aligned
    int64_t ld, plane;
    int values;          // of a row that are there
    const float* scale;  // what a row's products are to be multiplied by, as mxt_power has it (fp16 rows: null, by nothing)
    int drop;            // test only: the first CTA does not announce its first rows
};

template <int TERMS>
constexpr size_t mxt_smem(int experts)
{
    using S = MxtShape<TERMS>;
    return 1024 + (size_t)S::BATCHES * S::BATCH * 2 * TERMS * (MXT_ROWS<TERMS> / 2) * 128 +
           (size_t)MXT_CONVERT * S::AHEAD * 4 * MX_UNIT_BYTES + MXT_EPI_BYTES + (2 * S::BATCHES + 2 * MXT_A_STAGES + 5) * sizeof(uint64_t) +
           8 + MXT_SETS * MXT_ROWS<TERMS> * (sizeof(int) + sizeof(float)) + (size_t)(2 * (experts + 1) + 32 + 4) * sizeof(int);
}

// Where the row tiles' table lies in shared memory: after the rings, the results' buffer, 8-byte
// barriers (and what aligns what follows to 16), the items' slots and powers.
template <int TERMS>
__device__ __forceinline__ int* mxt_before(uint8_t* sm_raw)
{
    using S = MxtShape<TERMS>;
    constexpr size_t BARRIERS = (2 * S::BATCHES + 2 * MXT_A_STAGES + 5) * sizeof(uint64_t);
    constexpr size_t AT = (size_t)S::BATCHES * S::BATCH * 2 * TERMS * (MXT_ROWS<TERMS> / 2) * 128 +
                          (size_t)MXT_CONVERT * S::AHEAD * 4 * MX_UNIT_BYTES + MXT_EPI_BYTES + BARRIERS;
    return reinterpret_cast<int*>(sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u) + AT + AT % 16 +
                                  MXT_SETS * MXT_ROWS<TERMS> * (sizeof(int) + sizeof(float)));
}

// ---- tcgen05, clusters --------------------------------------------------------

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// The warp's one thread that issues for it (the others run along, which keeps
// the operands in uniform registers).
__device__ __forceinline__ bool elected()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// Arrives at the barrier of both CTAs once what this thread has issued is done.
__device__ __forceinline__ void tc_commit_both(uint32_t bar, bool on)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"((uint16_t)3), "r"((uint32_t)on)
        : "memory");
}

__device__ __forceinline__ void tc_mma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, bool on)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"((uint32_t)on)
        : "memory");
}

// 16 rows x 32 columns (32-bit) of tensor memory from the fragments of a warp.
__device__ __forceinline__ void tc_st_16x256b_x4(uint32_t at, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 columns of the warp's 32 rows, a row a lane.
__device__ __forceinline__ void tc_ld_32x32b_x16(uint32_t at, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tc_st_32x32b_x16(uint32_t at, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void add_sums(uint32_t (&v)[16], const uint32_t (&s)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(s[i]));
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// K-major operand in shared memory, rows of 128 bytes, 8 rows a 1024-byte
// swizzle atom: start address, 1024 bytes from eight rows to the next.
__device__ __forceinline__ uint64_t tc_desc(uint32_t smem)
{
    return (uint64_t)((smem & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

// D fp32, A and B fp16, both K-major, 256 x n (n in steps of MXT_N_STEP).
__device__ __forceinline__ uint32_t tc_idesc(int n) { return 1u << 4 | (uint32_t)(n >> 3) << 17 | 16u << 24; }

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ bool mbar_try_wait_at(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
// One arrival at that barrier of the pair's first CTA.
__device__ __forceinline__ void arrive_first(uint64_t* bar)
{
    asm volatile(
        "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [r];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
// A word's eight codes, times a scale (in both halves), as four pairs of halves.
__device__ __forceinline__ void e2m1_scaled(uint32_t w, uint32_t scale, uint32_t& p0, uint32_t& p1, uint32_t& p2, uint32_t& p3)
{
    uint32_t h[4];
    e2m1_halves(w, h);
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(p0) : "r"(h[0]), "r"(scale));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(p1) : "r"(h[1]), "r"(scale));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(p2) : "r"(h[2]), "r"(scale));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(p3) : "r"(h[3]), "r"(scale));
}

// ---- rows of x as halves ------------------------------------------------------------

// A row's power of two as the products read it: the number 2^e, or e itself (below
// zero) where that is none of fp32's normal ones.
__device__ __forceinline__ float mxt_power(int e) { return e < -126 ? (float)e : __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ int mxt_exponent(float power)
{
    return power < 0.0f ? (int)power : (int)(__float_as_uint(power) >> 23) - 127;
}

// x [rows][K] -> planes [term][rows][padded], zeros behind a row, and each
// row's power of two.  WARPS warps a row, eight values a lane at a time, the first
// 2048 WARPS (fp32: 1024) of a row kept in registers between its maximum and its conversion (a longer
// row's rest is read twice); bound by memory, or by latency where rows are few.
constexpr int MXT_ROW_THREADS = 128;

template <typename T, int WARPS>
__global__ void __launch_bounds__(MXT_ROW_THREADS, 8) mxt_rows_kernel(const T* x, int64_t ld, __half* planes, float* scale,
                                                                   int64_t rows, int K, int padded, bool wide,
                                                                   unsigned int* status)
{
    constexpr int TERMS = MX_TERMS<T>, ROWS = MXT_ROW_THREADS / 32 / WARPS, STEP = 256 * WARPS, KEEP = 16 / sizeof(T);
    constexpr bool SCALED = !std::is_same<T, __half>::value;
    __shared__ uint32_t tops[MXT_ROW_THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int k0 = (threadIdx.x % (32 * WARPS)) * 8;
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t first = (int64_t)blockIdx.x * ROWS; first < rows; first += (int64_t)gridDim.x * ROWS) {
        const int64_t row = first + warp / WARPS;
        const bool there = row < rows;
        const T* from = x + row * ld;
        Raw<T> v[KEEP];
        uint32_t top = 0;
        auto values = [](const Raw<T>& r, float (&f)[8]) {
            float a[4], b[4];
            values4<T>(r.w, a);
            values4<T>(r.w + sizeof(T), b);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[j] = a[j];
                f[4 + j] = b[j];
            }
        };
        auto take = [&](const float (&f)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t m = __float_as_uint(f[j]) & 0x7FFFFFFFu;
                top = max(top, m < 0x7F800000u ? m : 0u);
            }
        };
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int k = k0 + i * STEP;
            if (there && k < K) v[i] = load_raw(from + k, wide);  // (K is a multiple of 32)
            else v[i] = Raw<T>{};
        }
        if constexpr (SCALED) {
#pragma unroll
            for (int i = 0; i < KEEP; ++i) {
                float f[8];
                values(v[i], f);
                take(f);
            }
            for (int k = k0 + KEEP * STEP; k < K && there; k += STEP) {
                float f[8];
                mx_load8(from + k, wide, K - k, f);
                take(f);
            }
            top = __reduce_max_sync(~0u, top);
            if constexpr (WARPS > 1) {
                __syncthreads();  // (the row before is done with)
                if (lane == 0) tops[warp] = top;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < WARPS; ++i) top = max(top, tops[warp / WARPS * WARPS + i]);
            }
        }
        const int e = SCALED ? mx_row_exponent(top) : 0;
        if (SCALED && there && k0 == 0) scale[row] = mxt_power(e);
        const MxRowFactor f(e);
        auto put = [&](int k, const float (&z)[8]) {
            __half h[8], l[8];
            mx_row_halves<T>(z, f, h, l);
            if (!QG_OK(qg_in(row * padded + k, 8, rows * padded), status, 330)) return;
            __half* to = planes + row * padded + k;
            *reinterpret_cast<uint4*>(to) =
                make_uint4(mx_halves(h[0], h[1]), mx_halves(h[2], h[3]), mx_halves(h[4], h[5]), mx_halves(h[6], h[7]));
            if constexpr (TERMS == 2)
                *reinterpret_cast<uint4*>(to + rows * padded) =
                    make_uint4(mx_halves(l[0], l[1]), mx_halves(l[2], l[3]), mx_halves(l[4], l[5]), mx_halves(l[6], l[7]));
        };
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if (there && k0 + i * STEP < padded) {
                float z[8];
                values(v[i], z);
                put(k0 + i * STEP, z);
            }
        for (int k = k0 + KEEP * STEP; k < padded && there; k += STEP) {
            float z[8];
            mx_load8(from + k, wide, max(0, K - k), z);
            put(k, z);
        }
    }
}

// ---- the kernel -------------------------------------------------------------------

// An item: a row tile and a group of weight tiles.  Every role walks the same ones.
template <int ROWS>
struct MxtWalk {
    const int *before, *start;
    int groups;
    int64_t item, items;
    int step;
    int e, g, s0, cnt, n;  // expert, group, first place, rows, the product's N
    __device__ bool find()
    {
        if (item >= items) return false;
        const int rt = (int)(item / groups);
        g = (int)(item - (int64_t)rt * groups);
        while (rt >= before[e + 1]) ++e;
        const int first = start[e], all = start[e + 1] - first;
        const int tiles = before[e + 1] - before[e];
        const MxRowTile t = mxt_row_tile(all, tiles, rt - before[e], ROWS);
        s0 = first + t.first;
        cnt = t.cnt;
        n = t.n;
        return true;
    }
    __device__ bool next()
    {
        item += step;
        return find();
    }
};

// A place in a ring of N stages; `phase` is the parity that a wait for its data wants.
template <int N>
struct MxtStage {
    int i = 0;
    uint32_t phase = 0;
    __device__ void next()
    {
        if (++i == N) {
            i = 0;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ int mxt_slot(const MxArgs& a, int place)
{
    const int s = a.order ? a.order[place] : place;
    return s < 0 || s >= a.slots ? -1 : s;
}

// Rows of x as halves, from place s0 on, for mx_marked_row: take() goes to one, and returns its slot.
template <int TERMS>
struct MxtPlaceRows {
    const MxArgs& a;
    const MxtRows& x;
    int s0;
    const __half* row = nullptr;
    int exponent = 0;
    __device__ int take(int c)
    {
        const int s = mxt_slot(a, s0 + c);
        if (s < 0) return s;
        row = x.x + (int64_t)(s / a.x_div) * x.ld;
        if (x.scale) exponent = mxt_exponent(x.scale[s / a.x_div]);
        return s;
    }
    __device__ void values(int b, int t, float (&v)[8]) const
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint2 q[TERMS];
#pragma unroll
            for (int i = 0; i < TERMS; ++i)
                q[i] = 32 * b < x.values ? *reinterpret_cast<const uint2*>(row + i * x.plane + 32 * b + 4 * t + 16 * h) : make_uint2(0, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float f = 0.0f;
#pragma unroll
                for (int i = 0; i < TERMS; ++i) f += __half2float(__ushort_as_half((unsigned short)((k < 2 ? q[i].x : q[i].y) >> 16 * (k & 1))));
                v[4 * h + k] = f;
            }
        }
    }
};

// The marked rows of the items of this CTA, if it has met any.  By the converting warps.
template <typename T, int MODE>
__device__ __forceinline__ void mxt_marked_rows(const MxArgs& a, const MxtRows& x, const int* before, unsigned int* status)
{
    using O = typename std::conditional<MODE == MX_DOWN, float, T>::type;
    constexpr int GROUP_TILES = MODE == MX_GATE_UP ? 8 : 16;
    const int* start = before + a.L.experts + 1;
    const volatile int* sums = start + a.L.experts + 1;
    if (sums[32] || !sums[34]) return;  // (gave up; marks seen)
    MxtWalk<MXT_ROWS<MX_TERMS<T>>> walk;
    walk.before = before;
    walk.start = start;
    walk.groups = (a.L.tiles() + GROUP_TILES - 1) / GROUP_TILES;
    walk.items = (int64_t)before[a.L.experts] * walk.groups;
    walk.item = blockIdx.x / 2;
    walk.step = gridDim.x / 2;
    walk.e = 0;
    const int tile = (int)cluster_rank() * (GROUP_TILES / 2);
    for (bool more = walk.find(); more; more = walk.next()) {
        MxtPlaceRows<MX_TERMS<T>> rows{a, x, walk.s0};
        for (int i = (threadIdx.x >> 5) - MXT_LOAD_WARP; i < GROUP_TILES / 2 * MX_TILE_N; i += MXT_LOAD)
            mx_marked_row<T, MODE>(a, static_cast<O*>(a.y), walk.e, walk.g * GROUP_TILES + tile + i / MX_TILE_N, i % MX_TILE_N, walk.s0,
                                   walk.cnt, rows, status);
    }
}

template <typename T, int MODE>
__global__ void __launch_bounds__(MXT_THREADS, 1)
    mxt_kernel(MxArgs a, MxtRows x, unsigned int* status)
{
    constexpr int TERMS = MX_TERMS<T>;
    using S = MxtShape<TERMS>;
    using O = typename std::conditional<MODE == MX_DOWN, float, T>::type;
    constexpr int BATCH = S::BATCH, BATCHES = S::BATCHES;
    constexpr int ROWS = MXT_ROWS<TERMS>, TERM_BYTES = ROWS / 2 * 128, UNIT_BYTES = TERMS * TERM_BYTES, STEP_BYTES = 2 * UNIT_BYTES;
    extern __shared__ uint8_t sm_raw[];
    uint8_t* sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
    uint64_t* full_b = reinterpret_cast<uint64_t*>(sm + BATCHES * BATCH * STEP_BYTES + MXT_CONVERT * S::AHEAD * 4 * MX_UNIT_BYTES + MXT_EPI_BYTES);
    uint8_t* epi_stage = reinterpret_cast<uint8_t*>(full_b) - MXT_EPI_BYTES;
    uint64_t *empty_b = full_b + BATCHES, *full_a = empty_b + BATCHES;
    uint64_t *empty_a = full_a + MXT_A_STAGES, *acc_full = empty_a + MXT_A_STAGES, *acc_empty = acc_full + 2;
    uint64_t* all_done = acc_empty + 2;
    int* epi_slots = reinterpret_cast<int*>(all_done + 1 + (reinterpret_cast<uintptr_t>(all_done + 1) & 8) / 8);
    float* epi_scale = reinterpret_cast<float*>(epi_slots + MXT_SETS * ROWS);
    int* before = mxt_before<TERMS>(sm_raw);
    int* start = before + a.L.experts + 1;
    int* sums = start + a.L.experts + 1;
    volatile int* gave_up = sums + 32;
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(sums + 33);
    volatile int* marks = sums + 34;  // this CTA's weights have rows marked by 255

    const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
    const uint32_t rank = cluster_rank();
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < BATCHES; ++i) {
            mbar_init(full_b + i, MXT_LOAD);
            mbar_init(empty_b + i, 1);
        }
        for (int i = 0; i < MXT_A_STAGES; ++i) {
            mbar_init(full_a + i, 8);  // four warps of each CTA
            mbar_init(empty_a + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, 2 * MXT_EPI);
        }
        mbar_init(all_done, 1);
        fence_barrier_init();
        *gave_up = 0;
        *marks = 0;
    }
    if (warp == MXT_MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_at)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    pdl_wait();
    const int n_rt = mx_row_tiles<MXT_THREADS>(a, ROWS, before, start, sums);
    cluster_barrier();  // both CTAs' barriers and tensor memory are there
    tc_fence_after();
    const uint32_t tmem = *tmem_at;
    mx_rest<MODE>(a, static_cast<O*>(a.y), start, status);

    constexpr int GROUP_TILES = MODE == MX_GATE_UP ? 8 : 16;  // of a pair
    const int units = a.L.units(), steps = (units + 1) / 2, tiles = a.L.tiles();
    MxtWalk<ROWS> walk;
    walk.before = before;
    walk.start = start;
    walk.groups = (tiles + GROUP_TILES - 1) / GROUP_TILES;
    walk.items = (int64_t)n_rt * walk.groups;
    walk.item = blockIdx.x / 2;
    walk.step = gridDim.x / 2;
    walk.e = 0;

    // A bounded wait (by the SM's clock: the wall clock's register takes longer
    // to read than most waits); where one runs out, all roles of the CTA stop,
    // and with them the other CTA's, whose waits run out then.
    auto wait_at = [&](uint32_t bar, uint32_t parity) -> bool {
        bool ok = mbar_try_wait_at(bar, parity);
        if (!ok) {
            const long long t0 = clock64();
            while (!(ok = mbar_try_wait_at(bar, parity))) {
                if (*gave_up) break;
                if (clock64() - t0 > MXT_WAIT_CLOCKS) {
                    *gave_up = 1;
                    if (lane == 0) atomicAdd_system(status, 1u);
                    break;
                }
            }
        }
        return __all_sync(~0u, ok);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return wait_at(smem_u32(bar), parity); };
    // The 16-row tile of this CTA's rows 32 quad + 16 i, and its place in the weight's tiles.
    auto weight = [&](int i) { return MODE == MX_GATE_UP && i ? a.w2 : a.w; };
    auto tile_of = [&](int quad, int i) {
        return walk.g * GROUP_TILES + (int)rank * (GROUP_TILES / 2) + (MODE == MX_GATE_UP ? quad : 2 * quad + i);
    };

    if (warp >= MXT_MMA_WARP) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(MXT_REST_REGS));
    else if (warp >= MXT_EPI_WARP) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(MXT_EPI_REGS));

    if (warp < MXT_CONVERT) {
        // ---- weights into tensor memory: a warpgroup takes every third step, always into the same stage
        const int quad = warp & 3, stage = warp >> 2, g = lane >> 2;
        const uint32_t to = tmem + MXT_A_COL + stage * 64 + ((uint32_t)(32 * quad) << 16);
        constexpr int AHEAD = S::AHEAD, SLOT = 4 * MX_UNIT_BYTES;  // two tiles' two units
        uint8_t* ring = sm + BATCHES * BATCH * STEP_BYTES + warp * (AHEAD * SLOT);
        bool more = walk.find();
        int64_t left = more ? (walk.items - walk.item + walk.step - 1) / walk.step * steps - stage : 0;  // of the CTA, from this warp's on
        int u = 0;
        const uint8_t* from[2];
        bool there[2];
        auto locate = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tile = tile_of(quad, i);
                there[i] = tile < tiles;
                from[i] = weight(i) + walk.e * a.L.expert_bytes() + (there[i] ? tile : 0) * a.L.tile_bytes();
            }
        };
        auto advance = [&](int n) {  // steps
            u += 2 * n;
            while (more && u >= 2 * steps) {
                u -= 2 * steps;
                more = walk.next();
                if (more) locate();
            }
        };
        int slot = 0;
        // A step's codes and scales into the warp's ring.  (A tile behind the last leaves what
        // was there: rows of the product that go nowhere; so does a unit behind the last.)
        auto fetch = [&]() {
            if (more) {
                const int n = min(2, units - u) * (MX_UNIT_BYTES / 16);
                uint8_t* at = ring + slot * SLOT + lane * 16;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t* p = from[i] + u * MX_UNIT_BYTES + lane * 16;
                    if (there[i] && QG_OK(qg_in(from[i] - weight(i) + (int64_t)u * MX_UNIT_BYTES, n * 16, a.L.bytes()), status, 331)) {
                        cp_async16(at + i * 2 * MX_UNIT_BYTES, p);
                        if (lane + 32 < n) cp_async16(at + i * 2 * MX_UNIT_BYTES + 512, p + 512);
                        if (lane + 64 < n) cp_async16(at + i * 2 * MX_UNIT_BYTES + 1024, p + 1024);
                    }
                }
                if (++slot == AHEAD) slot = 0;
                advance(MXT_A_STAGES);
            }
            cp_async_commit();
        };
        if (more) locate();
        advance(stage);
#pragma unroll
        for (int j = 0; j < AHEAD - 1; ++j) fetch();
        int mine = 0, at_step = stage;  // of the CTA's, over all items
        uint32_t phase = 1;
        // (one body, not unrolled: the roles' loops share the instruction caches)
#pragma unroll 1
        for (; left > 0; left -= MXT_A_STAGES, at_step += MXT_A_STAGES, phase ^= 1) {
            cp_async_wait<AHEAD - 2>();
            __syncwarp();
            const uint8_t* at = ring + mine * SLOT;
            if (++mine == AHEAD) mine = 0;
            fetch();  // (into the slot read one step ago)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[2][16];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t* unit = at + (2 * i + h) * MX_UNIT_BYTES;
                    const uint4 code = *reinterpret_cast<const uint4*>(unit + lane * 16);
                    const uint32_t scale = *reinterpret_cast<const uint32_t*>(unit + MX_UNIT_CODES + g * 4);
                    const uint32_t wd[4] = {code.x, code.y, code.z, code.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // rows g and g + 8 of the first block, then of the second
                        // 2^(b - 127 + 13) as a half, twice
                        const uint32_t e = (__byte_perm(scale, 0, 0x4040 + 0x0101 * k) - (127 - MXT_SHIFT - 15) * 0x10001u) << 10;
                        const int o = 8 * (k >> 1) + 2 * (k & 1);
                        e2m1_scaled(wd[k], e, r[i][o], r[i][o + 1], r[i][o + 4], r[i][o + 5]);
                    }
                }
                if (h == 0) {
                    if (!wait(empty_a + stage, phase)) goto stop;
                    tc_fence_after();
                }
                tc_st_16x256b_x4(to + 32 * h, r[0]);
                tc_st_16x256b_x4(to + 32 * h + (16u << 16), r[1]);
            }
            tc_wait_st();
            tc_fence_before();
            // one of the four announces the rows of x too, which came long ago
            if (quad == 0 && at_step % BATCH == 0) {
                const int b = at_step / BATCH;
                if (!wait(full_b + b % BATCHES, b / BATCHES & 1)) break;
            }
            __syncwarp();
            if (lane == 0) arrive_first(full_a + stage);
        }
    stop:
        cp_async_wait<0>();
    } else if (warp >= MXT_LOAD_WARP) {
        // ---- rows of x into shared memory: this CTA's half of a row tile, a 16-byte piece of every 16th row a thread
        constexpr int STEP = MXT_LOAD * 4, EACH = (ROWS / 2 + STEP - 1) / STEP, LAG = BATCHES - 2;
        const int id = threadIdx.x - MXT_LOAD_WARP * 32, c = id & 7, r0 = id >> 3;
        static_assert(STEP % 8 == 4, "every other row: the swizzle's other half");
        const uint32_t at[2] = {smem_u32(sm) + r0 * 128 + ((c ^ (r0 & 7)) << 4), smem_u32(sm) + r0 * 128 + ((c ^ (r0 & 7) ^ 4) << 4)};
        const int64_t plane = x.plane * 2;
        MxtStage<BATCHES> st, told;
        int in = 0, issued = 0;  // steps of the batch, batches not yet announced
        bool ok = true, dropped = x.drop && blockIdx.x == 0;
        auto tell = [&]() {  // the oldest of them has landed
            fence_proxy_async();
            __syncwarp();
            if (lane == 0 && !dropped) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(full_b + told.i)) : "memory");
            dropped = false;
            told.next();
            --issued;
        };
        for (bool more = walk.find(); more && ok; more = walk.next()) {
            const int half = walk.n / 2;
            const uint8_t* from[EACH];
#pragma unroll
            for (int j = 0; j < EACH; ++j) {  // (rows behind the last repeat it and go nowhere)
                const int place = walk.s0 + min((int)rank * half + r0 + j * STEP, walk.cnt - 1);
                from[j] = reinterpret_cast<const uint8_t*>(x.x + (int64_t)(max(0, mxt_slot(a, place)) / a.x_div) * x.ld + c * 8);
            }
            const int rows = (half - r0 + STEP - 1) / STEP;  // of this thread
            for (int u = 0; u < units; u += 2) {
                if (in == 0) ok = wait(empty_b + st.i, st.phase ^ 1);
                if (!ok) break;
                const uint32_t step = (st.i * BATCH + in) * STEP_BYTES;
                const uint32_t to[2] = {at[0] + step, at[1] + step};
                // zeros behind a row, nothing read (16 bytes a piece: it is there or it is not)
                const int b0 = u * MX_UNIT_K + c * 8 < x.values ? 16 : 0, b1 = (u + 1) * MX_UNIT_K + c * 8 < x.values ? 16 : 0;
#pragma unroll
                for (int j = 0; j < EACH; ++j) {
                    if (j < rows)
#pragma unroll
                        for (int i = 0; i < TERMS; ++i) {
                            const uint32_t d = to[j & 1] + j * STEP * 128 + i * TERM_BYTES;
                            asm volatile("cp.async.cg.shared.global [%0], [%2], 16, %3;\n\t"
                                         "cp.async.cg.shared.global [%1], [%2 + 128], 16, %4;" ::"r"(d),
                                         "r"(d + UNIT_BYTES), "l"(from[j] + i * plane), "r"(b0), "r"(b1)
                                         : "memory");
                        }
                    from[j] += 4 * MX_UNIT_K;
                }
                if (++in == BATCH) {
                    in = 0;
                    cp_async_commit();
                    st.next();
                    if (++issued > LAG) {
                        cp_async_wait<LAG>();
                        tell();
                    }
                }
            }
        }
        cp_async_commit();
        if (in) ++issued;  // (a last batch that is not full)
        cp_async_wait<0>();
        while (issued > 0) tell();
        asm volatile("bar.sync 2, %0;" ::"n"((MXT_LOAD + MXT_EPI) * 32) : "memory");  // every result of this CTA is written
        uint32_t zero = 0;
        asm volatile("" : "+r"(zero));
        mxt_marked_rows<T, MODE>(mx_hidden(a), x, mxt_before<TERMS>(sm_raw + zero), status);
    } else if (warp == MXT_MMA_WARP) {
        // ---- products: a wait, eight products and a commit or two a step
        if (rank == 0) {
            const bool on = elected();
            const uint32_t full = smem_u32(full_a), empty = smem_u32(empty_a), spent = smem_u32(empty_b), done = smem_u32(acc_full);
            const uint64_t b0 = tc_desc(smem_u32(sm));
            MxtStage<BATCHES> sb;
            MxtStage<MXT_A_STAGES> sa;
            MxtStage<2> acc;
            int in = 0;
            bool ok = true;
            for (bool more = walk.find(); more && ok; more = walk.next()) {
                const uint32_t idesc = tc_idesc(__shfl_sync(~0u, walk.n, 0));
                uint32_t d = tmem + acc.i * ROWS, add = 0;
                if constexpr (TERMS == 1) ok = wait(acc_empty + acc.i, acc.phase ^ 1);
                for (int u = 0; u < units && ok; u += 2) {
                    if constexpr (TERMS == 2)
                        if (u % (2 * MXT_CHUNK) == 0) {
                            d = tmem + acc.i * ROWS;
                            add = 0;
                            ok = wait(acc_empty + acc.i, acc.phase ^ 1);
                            if (!ok) break;
                        }
                    ok = wait_at(full + 8 * sa.i, sa.phase);  // of both CTAs, and their rows of x
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t b = b0 + (uint64_t)((sb.i * BATCH + in) * (STEP_BYTES / 16));
                    const uint32_t at = tmem + MXT_A_COL + sa.i * 64;
#pragma unroll
                    for (int i = TERMS - 1; i >= 0; --i)  // (the small terms first, while the sum cuts little of them)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (h == 0 || u + 1 < units) {
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    tc_mma_f16(d, at + h * 32 + k * 8, b + (uint64_t)(h * (UNIT_BYTES / 16) + i * (TERM_BYTES / 16) + k * 2),
                                               idesc, add, on);
                                    add = 1;
                                }
                            }
                    tc_commit_both(empty + 8 * sa.i, on);
                    if (++in == BATCH) {
                        in = 0;
                        tc_commit_both(spent + 8 * sb.i, on);
                        sb.next();
                    }
                    sa.next();
                    if constexpr (TERMS == 2)
                        if ((u + 2) % (2 * MXT_CHUNK) == 0 || u + 2 >= units) {
                            tc_commit_both(done + 8 * acc.i, on);
                            acc.next();
                        }
                }
                if constexpr (TERMS == 1) {
                    if (ok) tc_commit_both(done + 8 * acc.i, on);
                    acc.next();
                }
            }
        }
    } else {
        // ---- results: 16 columns at a time, rows of slots (anywhere) through shared memory, so that a lane
        // stores 16 bytes of a column
        constexpr int WIDE = MODE == MX_GATE_UP ? 64 : 128;  // neighbouring outputs of a column
        constexpr int EACH = 16 / sizeof(O), LANES = WIDE / EACH, COLUMNS = 32 / LANES;  // a column's outputs by so many lanes
        constexpr int PER = (ROWS + 31) / 32;
        constexpr bool SCALED = !std::is_same<T, __half>::value;
        const int quad = warp & 3, i = lane >> 4;
        const uint32_t from = tmem + ((uint32_t)(32 * quad) << 16);
        O* y = static_cast<O*>(a.y);
        O* stage = reinterpret_cast<O*>(epi_stage);
        // this lane's place among a column's
        const int in_column = MODE == MX_GATE_UP ? 16 * quad + (lane & 15) : 32 * quad + lane;
        // An item's slots, their powers of two and this lane's row's, read ahead.
        int next_slot[PER], next_e;
        float next_scale[PER];
        auto look = [&](const MxtWalk<ROWS>& w) {
#pragma unroll
            for (int j = 0; j < PER; ++j) next_slot[j] = lane + 32 * j < w.cnt ? mxt_slot(a, w.s0 + lane + 32 * j) : -1;
            const int tile = w.g * GROUP_TILES + (int)rank * (GROUP_TILES / 2) + (MODE == MX_GATE_UP ? quad : 2 * quad + i);
            next_e = tile < tiles ? weight(i)[w.e * a.L.expert_bytes() + tile * a.L.tile_bytes() + (int64_t)units * MX_UNIT_BYTES + (lane & 15)]
                                  : 127;
        };
        auto look_scales = [&]() {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                next_scale[j] = SCALED && next_slot[j] >= 0 ? x.scale[next_slot[j] / a.x_div] : 1.0f;
        };
        const bool wide = ((reinterpret_cast<uintptr_t>(y) | (uintptr_t)(a.ldy * (int64_t)sizeof(O))) & 15u) == 0;
        MxtStage<2> acc;
        MxtStage<MXT_SETS> set;
        int half = 0;  // of the staging buffer
        bool stopped = false;
        bool more = walk.find();
        if (more) {
            look(walk);
            look_scales();
        }
        while (more) {
            int* slots = epi_slots + set.i * ROWS;  // (the four warps write the same)
            float* scales = epi_scale + set.i * ROWS;
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (lane + 32 * j < ROWS) {
                    slots[lane + 32 * j] = next_slot[j];
                    if (SCALED) scales[lane + 32 * j] = next_scale[j];
                }
            __syncwarp();
            // the weight's power of two, and whether its product with a row's is sure to be an
            // fp32 number (nearly always), exact then
            const int e = next_e, p = e - 127 - MXT_SHIFT;
            if (e == 255) *marks = 1;
            const float f0 = e == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(max(p, -126) + 127) << 23);
            bool mild = e == 255 || (p >= (SCALED ? -63 : -126) && p <= (SCALED ? 63 : 127));
            if constexpr (SCALED)
#pragma unroll
                for (int j = 0; j < PER; ++j) mild &= next_scale[j] >= 0x1p-63f && next_scale[j] <= 0x1p64f;
            mild = __all_sync(~0u, mild);
            const int n0 = (walk.g * GROUP_TILES + (int)rank * (GROUP_TILES / 2)) * MX_TILE_N;
            const int outputs = max(0, min(WIDE, a.L.N - n0)), columns = (walk.cnt + 15) & ~15;
            if (MODE == MX_DOWN && walk.g == 0 && rank == 0 && quad == 0)
                for (int r = lane; r < walk.cnt; r += 32)
                    if (slots[r] >= 0 && QG_OK(qg_in(slots[r], 1, a.slots), status, 334)) a.place_of[slots[r]] = walk.s0 + r;
            MxtWalk<ROWS> after = walk;
            more = after.next();
            if (more) look(after);
            const uint32_t sums_at = from + 2 * ROWS;
            const bool summed = TERMS == 2 && units > 2 * MXT_CHUNK;
            if constexpr (TERMS == 2)
#pragma unroll 1
                for (int u = 2 * MXT_CHUNK; u < units && !stopped; u += 2 * MXT_CHUNK) {  // all accumulators of the item but the last
                    stopped = !wait(acc_full + acc.i, acc.phase);
                    if (stopped) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < columns; c0 += 16) {
                        uint32_t v[16], s[16];
                        tc_ld_32x32b_x16(from + acc.i * ROWS + c0, v);
                        if (u > 2 * MXT_CHUNK) {
                            tc_ld_32x32b_x16(sums_at + c0, s);
                            tc_wait_ld();
                            add_sums(v, s);
                        } else {
                            tc_wait_ld();
                        }
                        tc_st_32x32b_x16(sums_at + c0, v);
                    }
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_first(acc_empty + acc.i);
                    acc.next();
                }
            const uint32_t d = from + acc.i * ROWS;
            auto results = [&](auto exact) {
                uint32_t v[16], s[16];
                tc_ld_32x32b_x16(d, v);
                if (summed) tc_ld_32x32b_x16(sums_at, s);
#pragma unroll 1
                for (int c0 = 0; c0 < columns; c0 += 16) {
                    tc_wait_ld();
                    if (summed) add_sums(v, s);
                    float z[16];
                    if (exact) {
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const float4 f = SCALED ? *reinterpret_cast<const float4*>(scales + c0 + c) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                            z[c] = __uint_as_float(v[c]) * (f.x * f0);
                            z[c + 1] = __uint_as_float(v[c + 1]) * (f.y * f0);
                            z[c + 2] = __uint_as_float(v[c + 2]) * (f.z * f0);
                            z[c + 3] = __uint_as_float(v[c + 3]) * (f.w * f0);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            z[c] = e == 255 ? f0 : mul_pow2(__uint_as_float(v[c]), p + (SCALED ? mxt_exponent(scales[c0 + c]) : 0));
                    }
                    if (c0 + 16 < columns) {
                        tc_ld_32x32b_x16(d + c0 + 16, v);  // on its way meanwhile
                        if (summed) tc_ld_32x32b_x16(sums_at + c0 + 16, s);
                    } else {  // the accumulator is free again
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_first(acc_empty + acc.i);
                    }
                    if (c0 == 0 && more) look_scales();
                    if constexpr (MODE == MX_DOWN) {
                        // rows of the partial results lie next to one another: straight from the registers
                        O* at = y + (int64_t)(walk.s0 + c0) * a.ldy + n0 + in_column;
                        if (in_column < outputs)
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                if (c0 + c < walk.cnt && QG_OK(qg_in(at - y, 1, (int64_t)a.slots * a.ldy), status, 333)) *at = z[c];
                                at += a.ldy;
                            }
                        continue;
                    }
                    O* to = stage + half * (16 * 128) + in_column;
                    if constexpr (MODE == MX_GATE_UP) {
                        // a lane of the gate's rows and the one of the same row of up
                        // have two columns: one each
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            const float other = __shfl_xor_sync(~0u, i ? z[c] : z[c + 1], 16);
                            to[(c + i) * WIDE] = from_f32<O>(mx_silu<T>(i ? other : z[c]) * (i ? z[c + 1] : other));
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; ++c) to[c * WIDE] = from_f32<O>(z[c]);
                    }
                    asm volatile("bar.sync 1, %0;" ::"n"(MXT_EPI * 32) : "memory");  // (the next write to this half comes after the next one)
                    const O* have = stage + half * (16 * 128);
#pragma unroll
                    for (int j = 0; j < 16; j += 4 * COLUMNS) {
                        const int c = j + quad * COLUMNS + lane / LANES, r = lane % LANES * EACH;
                        const int64_t s = slots[c0 + c];
                        O* at = y + s * a.ldy + n0 + r;
                        if (s < 0 || r >= outputs || !QG_OK(qg_in(s * a.ldy + n0 + r, min(EACH, outputs - r), (int64_t)a.slots * a.ldy), status, 332))
                            continue;
                        if (wide && r + EACH <= outputs)
                            *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(have + c * WIDE + r);
                        else
                            for (int k = 0; k < EACH && r + k < outputs; ++k) at[k] = have[c * WIDE + r + k];
                    }
                    half ^= 1;
                }
            };
            if (!stopped) stopped = !wait(acc_full + acc.i, acc.phase);
            if (!stopped) {
                tc_fence_after();
                if (MODE != MX_GEMM) results(mild);  // (as two loops, down takes 468 us for 404)
                else if (mild) results(std::true_type{});
                else results(std::false_type{});
            } else if constexpr (MODE != MX_DOWN) {  // it still comes to the barriers that the four warps have together
                for (int c0 = 0; c0 < columns; c0 += 16) asm volatile("bar.sync 1, %0;" ::"n"(MXT_EPI * 32) : "memory");
            }
            acc.next();
            set.next();
            walk = after;
        }
        asm volatile("bar.arrive 2, %0;" ::"n"((MXT_LOAD + MXT_EPI) * 32) : "memory");
    }
    if (warp == MXT_MMA_WARP && rank == 0) {  // what was issued ends before tensor memory is given back
        tc_commit_both(smem_u32(all_done), elected());
    }
    if (warp == MXT_MMA_WARP) {
        const long long t0 = clock64();
        while (!mbar_try_wait(all_done, 0))
            if (clock64() - t0 > MXT_WAIT_CLOCKS) {
                if (lane == 0) atomicAdd_system(status, 1u);
                break;
            }
        __syncwarp();
    }
    __syncwarp();
    tc_fence_before();
    cluster_barrier();
    if (warp == MXT_MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

}  // namespace qgemv
