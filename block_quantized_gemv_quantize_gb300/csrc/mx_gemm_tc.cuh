// Products of MXFP4 experts with many rows each (tcgen05 kernel).
//
// y[s][n] = sum_k w[n][k] x[s][k] with the weights as operand A (128 rows of
// a tcgen05.mma, from tensor memory) and up to MXT_ROWS rows of x as operand B
// (shared memory).  A code times its scale is a bf16 number exactly; rows of x
// are one bf16 term (bf16), two (fp16) or three (fp32), which hold them
// exactly, so that only the tensor core's fp32 sums round.  The codes come
// from the pack's words with integer operations, one multiplication in pairs
// for the scale, and go to tensor memory as fragments (16x256b): that operand
// then costs no shared-memory bandwidth, which is what bounds such a kernel
// with both operands there (64 KB a step of 256 x 192 x 64 for A alone).
//
// Scales in A are relative to the row's largest and times 2^-20, so that the
// sums stay in range wherever x is a bf16 number; the epilogue multiplies by
// the row's power of two.
//
// A CTA an SM: 8 warps convert weights (each the 32 rows of its quadrant of
// tensor memory), 3 gather rows of x into 128-byte-swizzled shared memory by asynchronous
// copies, one thread issues the products, 4 warps write the results.  256 rows
// of weights (128 of gate and of up) by one row tile is an item; items go
// round-robin over CTAs, row tiles of an expert are of even size, N is the row
// tile's count rounded up to 16.
#pragma once

#include "mx_gemm.cuh"

namespace qgemv {

constexpr int MXT_THREADS = 512;
constexpr int MXT_CONVERT = 8, MXT_EPI = 4, MXT_MMA_WARP = 12, MXT_LOAD_WARP = 13, MXT_LOAD = 3;
constexpr int MXT_A_STAGES = 2;
constexpr long long MXT_WAIT_CLOCKS = 2000000000;  // about a second

template <typename T>
struct MxtShape;
template <>
struct MxtShape<__nv_bfloat16> {
    static constexpr int TERMS = 1, ROWS = 192, STAGES = 7;
};
template <>
struct MxtShape<__half> {
    static constexpr int TERMS = 2, ROWS = 192, STAGES = 4;
};
template <>
struct MxtShape<float> {
    static constexpr int TERMS = 3, ROWS = 128, STAGES = 4;
};

struct MxtRows {
    const __nv_bfloat16* x;  // row r of term i at x + i * plane + r * ld
    int64_t ld, plane;
    int values;  // of a row that are there
    bool wide;
};

template <typename T>
constexpr size_t mxt_smem(int experts)
{
    using S = MxtShape<T>;
    return 1024 + (size_t)S::STAGES * S::TERMS * S::ROWS * 128 + 2 * S::ROWS * sizeof(void*) +
           MXT_EPI * S::ROWS * sizeof(int64_t) + (2 * S::STAGES + 2 * MXT_A_STAGES + 3) * sizeof(uint64_t) +
           (size_t)(2 * (experts + 1) + 32 + 4) * sizeof(int);
}

// ---- tcgen05 --------------------------------------------------------------------

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tc_mma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
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
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// K-major operand in shared memory, rows of 128 bytes, 8 rows a 1024-byte
// swizzle atom: start address, 1024 bytes from eight rows to the next.
__device__ __forceinline__ uint64_t tc_desc(uint32_t smem)
{
    return (uint64_t)((smem & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

// D fp32, A and B bf16, both K-major, 128 x n.
__device__ __forceinline__ uint32_t tc_idesc(int n) { return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(n >> 3) << 17 | 8u << 24; }

// A word's eight codes, times a scale (in both halves), as four pairs of bf16.
__device__ __forceinline__ void e2m1_bf16(uint32_t w, uint32_t scale, uint32_t& p0, uint32_t& p1, uint32_t& p2, uint32_t& p3)
{
    // exponent and mantissa to bits 8 .. 6: the code times 2^-126 (0.5 is subnormal there as here)
    const uint32_t m = 0x01C001C0u, s = 0x80008000u;
    const uint32_t t0 = ((w << 6) & m) | ((w << 12) & s), t1 = ((w << 2) & m) | ((w << 8) & s);
    const uint32_t t2 = ((w >> 2) & m) | ((w << 4) & s), t3 = ((w >> 6) & m) | (w & s);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p0) : "r"(t0), "r"(scale));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p1) : "r"(t1), "r"(scale));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p2) : "r"(t2), "r"(scale));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p3) : "r"(t3), "r"(scale));
}

constexpr int MXT_SHIFT = 20;  // the scales in A are 2^-20 of what they are

// ---- rows of x as bf16 terms ------------------------------------------------------

template <typename T>
__device__ __forceinline__ void mxt_terms(float v, uint16_t (&t)[MxtShape<T>::TERMS])
{
    // cut off, not rounded: the largest numbers stay finite, and what is left is exact
    float left = v;
#pragma unroll
    for (int i = 0; i < MxtShape<T>::TERMS; ++i) {
        const uint32_t u = __float_as_uint(left);
        t[i] = (uint16_t)(left != left ? 0x7FC0u : u >> 16);
        left = isfinite(v) ? left - __uint_as_float(u & 0xFFFF0000u) : 0.0f;
    }
}

// x [rows][K] -> planes [term][rows][padded], zeros behind a row.  One read, TERMS
// writes of half its bytes (or all); bound by memory.
template <typename T>
__global__ void __launch_bounds__(256) mxt_planes_kernel(const T* __restrict__ x, int64_t ld, uint16_t* planes, int64_t rows,
                                                         int K, int padded, bool wide, unsigned int* status)
{
    constexpr int TERMS = MxtShape<T>::TERMS;
    pdl_launch_dependents();
    pdl_wait();
    const int pieces = padded / 8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * pieces; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / pieces;
        const int k = (int)(i - row * pieces) * 8;
        float v[8];
        mx_load8(x + row * ld + k, wide, max(0, K - k), v);
        uint16_t t[8][TERMS];
#pragma unroll
        for (int j = 0; j < 8; ++j) mxt_terms<T>(v[j], t[j]);
        if (!QG_OK(qg_in(row * padded + k, 8, rows * padded), status, 330)) continue;
#pragma unroll
        for (int j = 0; j < TERMS; ++j) {
            alignas(16) uint16_t o[8];
#pragma unroll
            for (int m = 0; m < 8; ++m) o[m] = t[m][j];
            *reinterpret_cast<uint4*>(planes + (j * rows + row) * padded + k) = *reinterpret_cast<uint4*>(o);
        }
    }
}

// ---- the kernel -------------------------------------------------------------------

// An item: a row tile and a group of weight tiles.  Every role walks the same ones.
struct MxtWalk {
    const int *before, *start;
    int rows_most, groups;
    int64_t item, items;
    int step;
    int e, g, s0, cnt, n;  // expert, group, first place, rows, rows rounded up to 16
    __device__ bool find()
    {
        if (item >= items) return false;
        const int rt = (int)(item / groups);
        g = (int)(item - (int64_t)rt * groups);
        while (rt >= before[e + 1]) ++e;
        const int first = start[e], all = start[e + 1] - first;
        const int tiles = before[e + 1] - before[e];
        const int each = min(rows_most, ((all + tiles - 1) / tiles + 15) & ~15);
        s0 = first + (rt - before[e]) * each;
        cnt = min(each, first + all - s0);
        n = (cnt + 15) & ~15;
        return true;
    }
    __device__ bool next()
    {
        item += step;
        return find();
    }
};

__device__ __forceinline__ int mxt_slot(const MxArgs& a, int place)
{
    const int s = a.order ? a.order[place] : place;
    return s < 0 || s >= a.slots ? -1 : s;
}

template <typename T, int MODE>
__global__ void __launch_bounds__(MXT_THREADS, 1) mxt_kernel(MxArgs a, MxtRows x, unsigned int* status)
{
    using S = MxtShape<T>;
    using O = typename std::conditional<MODE == MX_DOWN, float, T>::type;
    constexpr int ROWS = S::ROWS, TERMS = S::TERMS, STAGES = S::STAGES, LAG = STAGES - 2;
    constexpr int STAGE_BYTES = TERMS * ROWS * 128;
    constexpr uint32_t A_COL = 2 * ROWS;  // tensor memory: two accumulators of ROWS columns, then the stages of A
    static_assert(A_COL + MXT_A_STAGES * 64 <= 512, "tensor memory");
    extern __shared__ uint8_t sm_raw[];
    uint8_t* sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
    const __nv_bfloat16** ptrs = reinterpret_cast<const __nv_bfloat16**>(sm + STAGES * STAGE_BYTES);
    uint64_t* full_b = reinterpret_cast<uint64_t*>(ptrs + 2 * ROWS);
    uint64_t *empty_b = full_b + STAGES, *full_a = empty_b + STAGES, *empty_a = full_a + MXT_A_STAGES;
    uint64_t *acc_full = empty_a + MXT_A_STAGES, *acc_empty = acc_full + 1, *all_done = acc_empty + 1;
    int64_t* epi_offs = reinterpret_cast<int64_t*>(all_done + 1);
    int* before = reinterpret_cast<int*>(epi_offs + MXT_EPI * ROWS);
    int* start = before + a.L.experts + 1;
    int* sums = start + a.L.experts + 1;
    volatile int* gave_up = sums + 32;
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(sums + 33);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full_b + i, MXT_LOAD);
            mbar_init(empty_b + i, 1);
        }
        for (int i = 0; i < MXT_A_STAGES; ++i) {
            mbar_init(full_a + i, MXT_CONVERT);
            mbar_init(empty_a + i, 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, MXT_EPI);
        mbar_init(all_done, 1);
        fence_barrier_init();
        *gave_up = 0;
    }
    if (warp == MXT_MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_at)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    pdl_wait();
    const int n_rt = mx_row_tiles<MXT_THREADS>(a, ROWS, before, start, sums);  // (ends with a barrier)
    tc_fence_after();
    const uint32_t tmem = *tmem_at;
    mx_zero_rest(a, static_cast<O*>(a.y), status);

    constexpr int GROUP_TILES = MODE == MX_GATE_UP ? 8 : 16;
    const int units = a.L.units(), tiles = a.L.tiles();
    MxtWalk walk;
    walk.before = before;
    walk.start = start;
    walk.rows_most = ROWS;
    walk.groups = (tiles + GROUP_TILES - 1) / GROUP_TILES;
    walk.items = (int64_t)n_rt * walk.groups;
    walk.item = blockIdx.x;
    walk.step = gridDim.x;
    walk.e = 0;

    // A bounded wait; where one runs out, all roles stop.
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        const long long t0 = clock64();  // (the wall clock's register takes longer to read than most waits)
        while (!mbar_try_wait(bar, parity)) {
            if (*gave_up) return false;
            if (clock64() - t0 > MXT_WAIT_CLOCKS) {
                *gave_up = 1;
                if (lane == 0) atomicAdd_system(status, 1u);
                return false;
            }
        }
        return true;
    };

    if (warp < MXT_CONVERT) {
        // ---- weights into tensor memory
        const int quad = warp & 3, half = warp >> 2, g = lane >> 2;
        const uint8_t* w = MODE == MX_GATE_UP && half ? a.w2 : a.w;
        const int tile0 = (MODE == MX_GATE_UP ? 0 : half * 8) + quad * 2;
        const uint32_t to = tmem + A_COL + half * 32 + ((uint32_t)(32 * quad) << 16);
        constexpr int AHEAD = 3;
        uint4 code[AHEAD][2];
        uint32_t scale[AHEAD][2];
        bool more = walk.find();
        int64_t left = more ? (walk.items - walk.item + walk.step - 1) / walk.step * units : 0;  // steps
        int u = 0;
        const uint8_t* from[2] = {nullptr, nullptr};
        auto locate = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tile = walk.g * GROUP_TILES + tile0 + i;
                from[i] = tile < tiles ? w + walk.e * a.L.expert_bytes() + tile * a.L.tile_bytes() : nullptr;
            }
        };
        auto fetch = [&](uint4 (&c)[2], uint32_t (&s)[2]) {
            if (!more) return;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                c[i] = make_uint4(0, 0, 0, 0);
                s[i] = 0x7F7F7F7Fu;
                const uint8_t* p = from[i] + (int64_t)u * MX_UNIT_BYTES;
                if (from[i] && QG_OK(qg_in(p - w, MX_UNIT_BYTES, a.L.bytes()), status, 331)) {
                    c[i] = __ldg(reinterpret_cast<const uint4*>(p) + lane);
                    s[i] = __ldg(reinterpret_cast<const uint32_t*>(p + MX_UNIT_CODES) + g);
                }
            }
            if (++u == units) {
                u = 0;
                more = walk.next();
                if (more) locate();
            }
        };
        if (more) locate();
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) fetch(code[i], scale[i]);
        int stage = 0;
        uint32_t phase = 1;
        bool ok = true;
        while (left > 0 && ok) {
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                if (left <= 0 || !ok) break;
                uint32_t r[2][16];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t wd[4] = {code[j][i].x, code[j][i].y, code[j][i].z, code[j][i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // rows g and g + 8 of the first block, then of the second
                        // 2^(b - 127) 2^126 2^-20 as bf16
                        const uint32_t e = ((scale[j][i] >> (8 * k) & 255u) + 126 - MXT_SHIFT) << 7;
                        const int o = 8 * (k >> 1) + 2 * (k & 1);
                        e2m1_bf16(wd[k], e | e << 16, r[i][o], r[i][o + 1], r[i][o + 4], r[i][o + 5]);
                    }
                }
                fetch(code[j], scale[j]);
                ok = wait(empty_a + stage, phase);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                tc_st_16x256b_x4(to + stage * 64, r[0]);
                tc_st_16x256b_x4(to + stage * 64 + (16u << 16), r[1]);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(full_a + stage)) : "memory");
                if (++stage == MXT_A_STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
                --left;
            }
        }
    } else if (warp >= MXT_LOAD_WARP) {
        // ---- rows of x into shared memory
        const int id = threadIdx.x - MXT_LOAD_WARP * 32, c = id & 7, r0 = id >> 3;
        constexpr int STEP = MXT_LOAD * 32 / 8;
        int stage = 0, flip = 0, issued = 0, told = 0;
        uint32_t phase = 1;
        bool ok = true;
        auto tell = [&]() {  // the oldest stage not yet announced has landed
            fence_proxy_async();
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(full_b + told)) : "memory");
            if (++told == STAGES) told = 0;
            --issued;
        };
        for (bool more = walk.find(); more && ok; more = walk.next()) {
            const __nv_bfloat16** rows = ptrs + flip * ROWS;
            flip ^= 1;
            for (int r = id; r < walk.n; r += MXT_LOAD * 32) {  // (rows behind the last repeat it and go nowhere)
                const int s = mxt_slot(a, walk.s0 + min(r, walk.cnt - 1));
                rows[r] = x.x + (int64_t)(max(0, s) / a.x_div) * x.ld;
            }
            asm volatile("bar.sync 1, %0;" ::"n"(MXT_LOAD * 32) : "memory");
            for (int u = 0; u < units && ok; ++u) {
                ok = __all_sync(~0u, wait(empty_b + stage, phase));
                if (!ok) break;
                uint8_t* to = sm + stage * STAGE_BYTES;
                const int k = u * MX_UNIT_K + c * 8;
                const bool there = k < x.values;
#pragma unroll 4
                for (int r = r0; r < walk.n; r += STEP) {
                    const __nv_bfloat16* p = rows[r] + k;
                    uint8_t* at = to + r * 128 + ((c ^ (r & 7)) << 4);
#pragma unroll
                    for (int i = 0; i < TERMS; ++i) {
                        if (x.wide) {
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(at + i * ROWS * 128)),
                                         "l"(there ? p + i * x.plane : x.x), "r"(there ? 16 : 0)
                                         : "memory");
                        } else {
                            uint32_t v[4];
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const uint16_t* q = reinterpret_cast<const uint16_t*>(p + i * x.plane) + 2 * m;
                                v[m] = there ? (uint32_t)q[0] | (uint32_t)q[1] << 16 : 0u;
                            }
                            *reinterpret_cast<uint4*>(at + i * ROWS * 128) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    }
                }
                cp_async_commit();
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
                if (++issued > LAG) {
                    cp_async_wait<LAG>();
                    tell();
                }
            }
        }
        cp_async_wait<0>();
        while (issued > 0) tell();
    } else if (warp == MXT_MMA_WARP) {
        // ---- products
        int sa = 0, sb = 0;
        uint32_t pa = 0, pb = 0, pe = 1;
        bool ok = true;
        for (bool more = walk.find(); more && ok; more = walk.next()) {
            const uint32_t idesc = tc_idesc(walk.n);
            ok = __all_sync(~0u, wait(acc_empty, pe));
            pe ^= 1;
            for (int u = 0; u < units && ok; ++u) {
                ok = wait(full_b + sb, pb) && wait(full_a + sa, pa);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t b = tc_desc(smem_u32(sm + sb * STAGE_BYTES));
                    const uint32_t at = tmem + A_COL + sa * 64;
#pragma unroll
                    for (int i = 0; i < TERMS; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                tc_mma_f16(tmem + h * ROWS, at + h * 32 + k * 8,
                                           b + (uint64_t)(i * (ROWS * 128 / 16) + k * 2), idesc, u > 0 || i > 0 || k > 0);
                    tc_commit(empty_b + sb);
                    tc_commit(empty_a + sa);
                }
                __syncwarp();
                if (++sb == STAGES) {
                    sb = 0;
                    pb ^= 1;
                }
                if (++sa == MXT_A_STAGES) {
                    sa = 0;
                    pa ^= 1;
                }
            }
            if (ok && lane == 0) tc_commit(acc_full);
            __syncwarp();
        }
        // what was issued ends before tensor memory is given back
        if (lane == 0) tc_commit(all_done);
        __syncwarp();
        if (!mbar_wait_bounded(all_done, 0) && lane == 0) atomicAdd_system(status, 1u);
    } else {
        // ---- results
        const int quad = warp & 3;
        int64_t* offs = epi_offs + quad * ROWS;  // where the rows' outputs are, -1 for none
        const uint32_t from = tmem + ((uint32_t)(32 * quad) << 16);
        O* y = static_cast<O*>(a.y);
        uint32_t phase = 0;
        bool ok = true;
        for (bool more = walk.find(); more && ok; more = walk.next()) {
            __syncwarp();
            for (int r = lane; r < walk.n; r += 32) {
                const int s = r < walk.cnt ? mxt_slot(a, walk.s0 + r) : -1;
                offs[r] = s < 0 ? -1 : s * a.ldy;
            }
            int n[2];
            float f[2][2];  // the row's power of two, in two factors
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                n[h] = walk.g * GROUP_TILES * MX_TILE_N + quad * 32 + lane + (MODE == MX_GATE_UP ? 0 : h * 128);
                const uint8_t* w = MODE == MX_GATE_UP && h ? a.w2 : a.w;
                const int e = n[h] < a.L.N ? w[walk.e * a.L.expert_bytes() + (n[h] / MX_TILE_N) * a.L.tile_bytes() +
                                               (int64_t)units * MX_UNIT_BYTES + n[h] % MX_TILE_N]
                                           : 127;
                const int p = e - 127 + MXT_SHIFT;
                f[h][0] = e == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(min(p, 127) + 127) << 23);
                f[h][1] = __uint_as_float((uint32_t)(max(p - 127, 0) + 127) << 23);
            }
            __syncwarp();
            ok = __all_sync(~0u, wait(acc_full, phase));
            phase ^= 1;
            if (!ok) break;
            tc_fence_after();
            // 16 columns a step, the next ones on their way from tensor memory meanwhile
            auto store = [&](const uint32_t (&v)[16], const uint32_t (&v2)[16], int c0, int h) {
                const bool mine = n[h] < a.L.N;
                O* to = y + n[h];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    float o = __uint_as_float(v[c]) * f[h][0] * f[h][1];
                    if constexpr (MODE == MX_GATE_UP) o = mx_silu(o) * (__uint_as_float(v2[c]) * f[1][0] * f[1][1]);
                    const int64_t at = offs[c0 + c];
                    if (mine && at >= 0 && QG_OK(qg_in(at + n[h], 1, (int64_t)a.slots * a.ldy), status, 332)) to[at] = from_f32<O>(o);
                }
            };
            const int steps = (MODE == MX_GATE_UP ? 1 : 2) * (walk.n / 16);
            auto load = [&](int i, uint32_t (&v)[16], uint32_t (&v2)[16]) {
                if constexpr (MODE == MX_GATE_UP) {
                    tc_ld_32x32b_x16(from + 16 * i, v);
                    tc_ld_32x32b_x16(from + ROWS + 16 * i, v2);
                } else {
                    const int h = i >= walk.n / 16;
                    tc_ld_32x32b_x16(from + h * ROWS + 16 * (i - h * (walk.n / 16)), v);
                }
            };
            auto put = [&](int i, const uint32_t (&v)[16], const uint32_t (&v2)[16]) {
                const int h = MODE == MX_GATE_UP ? 0 : i >= walk.n / 16;
                const int c0 = 16 * (i - h * (walk.n / 16));
                if (h) store(v, v2, c0, 1);
                else store(v, v2, c0, 0);
            };
            uint32_t va[16], va2[16], vb[16], vb2[16];
            load(0, va, va2);
            for (int i = 0; i < steps; i += 2) {
                tc_wait_ld();
                if (i + 1 < steps) load(i + 1, vb, vb2);
                put(i, va, va2);
                if (i + 1 < steps) {
                    tc_wait_ld();
                    if (i + 2 < steps) load(i + 2, va, va2);
                    put(i + 1, vb, vb2);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(acc_empty)) : "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MXT_MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

}  // namespace qgemv
