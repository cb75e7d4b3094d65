// attn_paged: attention of a few new tokens over the block-quantized paged
// cache, on the tensor cores straight from the blocks.
//
// Mathematics.  A row is one (new token, q head); the rows that share a kv
// head go together.  With codes c and block scales d (kvcache.cuh),
//     s[row][p] = scale sum_b d_k[p][b] sum_{i in b} q[row][i] c_k[p][i]
//     out[row][i] = sum_p w[row][p] d_v[p][b(i)] c_v[p][i] / sum_p w[row][p]
// with w = 2^(s log2 e - m), m the running maximum of the row.  The codes are
// small integers, so they are fp16 exactly and are the tensor cores' B operand
// without ever being scaled: K's scales multiply the fp32 block sums, V's the
// weights before they are rounded to fp16.  q and w d_v are fp16 pairs hi + lo
// (22 bits) in the two halves of the A operand, eight rows to an instruction
// of 16 (TWO; fp32 and fp16 callers), or 16 rows of one fp16 each (bf16
// callers, whose output keeps 8 bits).  q is brought to 2^13 .. 2^14 by an exact
// power of two per row, w d_v to below 2^14 by one that follows the largest
// d_v seen so far, so that neither leaves fp16's range.
//
// Split.  An item is a (sequence, kv head, group of row tiles).  All items'
// tiles of 16 tokens stand in one line, cut into equal pieces, one a CTA: the
// load is even however the lengths differ, and the lengths are read on the
// device, so that a captured graph serves any.  In a CTA, WS warps take an
// item's tiles in turn, pairs at a time, each through a ring of its own in
// shared memory that bulk copies fill (a tile of a kv head is contiguous: one
// copy); WR warps share each ring, one for every tile of rows.  The WS partial
// results meet in shared memory; an item cut between CTAs leaves one partial
// result a CTA in the workspace, and the CTA that finds itself last (a counter)
// joins them in CTA order, so the result does not depend on the order in which
// CTAs finish.
#pragma once

#include "kvcache.cuh"

namespace qgemv {

constexpr int ATTN_GRID = 160;  // most CTAs (one an SM): the workspace holds two partial results of each

template <int FMT, int NB, bool TWO>
struct AttnShape {
    static constexpr int ROWS = TWO ? 8 : 16;            // rows of a row tile
    static constexpr int NR = TWO ? 1 : 2;               // rows whose statistics a lane keeps
    static constexpr int NO = NB * 4 * (TWO ? 2 : 4);    // output values of a lane in a partial result
    static constexpr int PART = (NO + 2 * NR) * 32;      // floats of one row tile's partial result
    static constexpr int TILE = kv_tile_bytes(FMT, NB), HALF = kv_half_bytes(FMT, NB);
    static constexpr bool Q_SMEM = NB > 4;               // q's fragments do not fit the registers next to the sums
    static constexpr int MAX_WARPS = 8;
};

struct AttnPlan {
    int type;
    int ws, wr;          // splits, row tiles at a time
    int row_tiles, row_groups;
    int stages;          // tiles a ring holds
    int min_chunk;       // least tiles of a CTA
    uint32_t off_merge, off_q, off_bar, bytes;  // shared memory
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// Codes to fp16 without a conversion: 0x6400 | n is the fp16 number 1024 + n.
// Two bytes of w, as 1024 + byte (code + 128), less 1152.
template <int SEL>
__device__ __forceinline__ uint32_t codes_q8(uint32_t w)
{
    return h2_bits(__hsub2(bits_h2(__byte_perm(w, 0x64646464u, SEL)), bits_h2(0x64806480u)));
}
// The low nibbles of bytes 0 and 2: 1024 + code less 1032 (code - 8).
__device__ __forceinline__ uint32_t codes_q4_lo(uint32_t w)
{
    return h2_bits(__hsub2(bits_h2((w & 0x000F000Fu) | 0x64006400u), bits_h2(0x64086408u)));
}
// Their high nibbles: (1024 + 16 code) / 16 - 72, exact in one fma.
__device__ __forceinline__ uint32_t codes_q4_hi(uint32_t w)
{
    return h2_bits(__hfma2(bits_h2((w & 0x00F000F0u) | 0x64006400u), bits_h2(0x2C002C00u), bits_h2(0xD480D480u)));
}

// The four tokens of a tile that column pair t of the products holds: i = 0..3
// are the tokens 4 i + (t ^ 3 (i & 1)), an order in which neither K's loads (a
// token a lane quad) nor V's (four tokens a lane) meet in a bank.
__device__ __forceinline__ int tile_token(int t, int i) { return 4 * i + (t ^ (3 * (i & 1))); }

// K's B fragments of block b, columns 8 j .. 8 j + 7 of the tile: the values
// 8 t .. 8 t + 7 of the lane's token (q8_0, f16); or (q4_0) 4 t + {0, 2, 1, 3},
// then 16 + 4 t + {0, 2, 1, 3}.  q's fragments follow the same order.
template <int FMT>
__device__ __forceinline__ void k_fragment(const uint8_t* k, int b, int tok, int t, uint32_t (&f)[4])
{
    const uint8_t* p = k + (b * KV_TILE + tok) * kv_code_bytes(FMT) + t * (kv_code_bytes(FMT) / 4);
    if constexpr (FMT == QGEMV_KV_F16) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        f[0] = w.x, f[1] = w.y, f[2] = w.z, f[3] = w.w;
    } else if constexpr (FMT == QGEMV_KV_Q8_0) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        f[0] = codes_q8<0x4140>(w.x), f[1] = codes_q8<0x4342>(w.x);
        f[2] = codes_q8<0x4140>(w.y), f[3] = codes_q8<0x4342>(w.y);
    } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p), v = w >> 8;
        f[0] = codes_q4_lo(w), f[1] = codes_q4_lo(v), f[2] = codes_q4_hi(w), f[3] = codes_q4_hi(v);
    }
}

// V's B fragments of block b for its four column tiles: token pairs (0, 1) in
// lo, (2, 3) in hi; column n of tile nn is the block's value 4 n + nn, or (q4_0)
// 2 n + {0, 16, 1, 17}[nn].
template <int FMT>
__device__ __forceinline__ void v_fragments(const uint8_t* v, int b, int g, int t, uint32_t (&lo)[4], uint32_t (&hi)[4])
{
    const uint8_t* p = v + b * KV_TILE * kv_code_bytes(FMT) + g * (kv_code_bytes(FMT) / 8);
    auto at = [&](int i) { return p + tile_token(t, i) * kv_code_bytes(FMT); };
    if constexpr (FMT == QGEMV_KV_F16) {
        uint2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint2*>(at(i));
        lo[0] = __byte_perm(w[0].x, w[1].x, 0x5410), lo[1] = __byte_perm(w[0].x, w[1].x, 0x7632);
        lo[2] = __byte_perm(w[0].y, w[1].y, 0x5410), lo[3] = __byte_perm(w[0].y, w[1].y, 0x7632);
        hi[0] = __byte_perm(w[2].x, w[3].x, 0x5410), hi[1] = __byte_perm(w[2].x, w[3].x, 0x7632);
        hi[2] = __byte_perm(w[2].y, w[3].y, 0x5410), hi[3] = __byte_perm(w[2].y, w[3].y, 0x7632);
    } else if constexpr (FMT == QGEMV_KV_Q8_0) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(at(i));
        uint32_t x = __byte_perm(w[0], w[1], 0x5140), y = __byte_perm(w[0], w[1], 0x7362);
        lo[0] = codes_q8<0x4140>(x), lo[1] = codes_q8<0x4342>(x), lo[2] = codes_q8<0x4140>(y), lo[3] = codes_q8<0x4342>(y);
        x = __byte_perm(w[2], w[3], 0x5140), y = __byte_perm(w[2], w[3], 0x7362);
        hi[0] = codes_q8<0x4140>(x), hi[1] = codes_q8<0x4342>(x), hi[2] = codes_q8<0x4140>(y), hi[3] = codes_q8<0x4342>(y);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint16_t*>(at(i));
        uint32_t x = __byte_perm(w[0], w[1], 0x5410), y = x >> 8;
        lo[0] = codes_q4_lo(x), lo[1] = codes_q4_hi(x), lo[2] = codes_q4_lo(y), lo[3] = codes_q4_hi(y);
        x = __byte_perm(w[2], w[3], 0x5410), y = x >> 8;
        hi[0] = codes_q4_lo(x), hi[1] = codes_q4_hi(x), hi[2] = codes_q4_lo(y), hi[3] = codes_q4_hi(y);
    }
}

// The tiles of a sequence that its rows see.
struct AttnTiles {
    int first, count;
    __host__ __device__ AttnTiles() : first(0), count(0) {}
    __host__ __device__ explicit AttnTiles(const AttnSpan& sp)
    {
        first = sp.first() / KV_TILE;
        count = sp.last() > sp.first() ? (sp.last() + KV_TILE - 1) / KV_TILE - first : 0;
    }
};

// A CTA's walk over its piece of the line of tiles: segments, each a run of
// one item's tiles.
struct AttnWalk {
    int64_t left;        // tiles of the piece from this segment's first on
    int b, item;         // sequence, (kv head, row group) within it
    int first, count;    // the item's tiles
    int ta, tb;          // the segment's, counted from `first`
    __device__ __forceinline__ bool done() const { return left <= 0; }
    __device__ __forceinline__ void clip() { tb = left < (int64_t)(count - ta) ? ta + (int)left : count; }
    __device__ __forceinline__ void next(const AttnArgs& a, int items)
    {
        left -= tb - ta;
        if (left <= 0) return;
        ta = 0;
        if (++item == items) {
            item = 0;
            do {
                const AttnTiles n{AttnSpan(a, a.lens[++b])};  // left > 0: a later sequence has tiles
                first = n.first;
                count = n.count;
            } while (count == 0);
        }
        clip();
    }
};

// By one warp: the total of all sequences' tiles times `items`, and the walk
// that starts at tile `start` of the line (when start < total).
__device__ __forceinline__ int64_t attn_total(const AttnArgs& a, int items, int lane)
{
    int64_t n = 0;
    for (int b = lane; b < a.batch; b += 32) n += AttnTiles(AttnSpan(a, a.lens[b])).count;
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n * items;
}

__device__ __forceinline__ AttnWalk attn_find(const AttnArgs& a, int items, int64_t start, int64_t left, int lane)
{
    AttnWalk w{};
    w.left = left;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        const AttnTiles t = b < a.batch ? AttnTiles(AttnSpan(a, a.lens[b])) : AttnTiles();
        int64_t sum = (int64_t)t.count * items;
        const int64_t own = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + sum > start && own > 0);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int64_t off = start - (before + __shfl_sync(0xffffffffu, sum - own, src));
            w.b = b0 + src;
            w.first = __shfl_sync(0xffffffffu, t.first, src);
            w.count = __shfl_sync(0xffffffffu, t.count, src);
            w.item = (int)(off / w.count);
            w.ta = (int)(off - (int64_t)w.item * w.count);
            w.clip();
            return w;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    w.left = 0;
    return w;
}

template <int N>
__device__ __forceinline__ void load_row_part(const void* p, int64_t at, int type, bool wide, float (&v)[N])
{
    if (type == QGEMV_F32) load_values(static_cast<const float*>(p) + at, wide, v);
    else if (type == QGEMV_F16) load_values(static_cast<const __half*>(p) + at, wide, v);
    else load_values(static_cast<const __nv_bfloat16*>(p) + at, wide, v);
}

template <int N>
__device__ __forceinline__ void store_row_part(void* p, int64_t at, int type, bool wide, const float (&v)[N])
{
    if (type == QGEMV_F32) store_values(static_cast<float*>(p) + at, wide, v);
    else if (type == QGEMV_F16) store_values(static_cast<__half*>(p) + at, wide, v);
    else store_values(static_cast<__nv_bfloat16*>(p) + at, wide, v);
}

__device__ __forceinline__ bool rows_wide(const void* p, int64_t row, int64_t head, int type)
{
    const KvRows r{const_cast<void*>(p), row, head};
    return type == QGEMV_F32 ? r.wide<float>() : r.wide<__half>();
}

// What a warp keeps of its row tile: running maximum (of s log2 e), sum of
// weights and unnormalised outputs.  While a segment runs, l is this lane's
// share and o is scaled by 2^(28 - e) (f16: 2^14), in the fragments' 16 rows.
template <int FMT, int NB, bool TWO>
struct AttnState {
    using Sh = AttnShape<FMT, NB, TWO>;
    float m[Sh::NR], l[Sh::NR];
    float o[NB][4][4];
    int e;

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int r = 0; r < Sh::NR; ++r) m[r] = -INFINITY, l[r] = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[b][n][c] = 0.0f;
        e = 0;
    }
    // a finite base for exponents: a row that has seen nothing has m = -inf
    static __device__ __forceinline__ float base(float m) { return m == -INFINITY ? 0.0f : m; }

    // End of a segment: sums over the quad, the two halves of a split row
    // added (an infinite output stands in the high half alone), the scale out.
    __device__ __forceinline__ void finish(bool poison)
    {
#pragma unroll
        for (int r = 0; r < Sh::NR; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (poison) l[r] = __int_as_float(0x7fffffff);
        }
        const float back = FMT == QGEMV_KV_F16 ? 0x1p-14f : __int_as_float((127 + e - 28) << 23);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (TWO && c >= 2) continue;
                    float v = o[b][n][c];
                    if (TWO) v = isinf(v) ? v : v + o[b][n][c + 2];
                    o[b][n][c] = v * back;
                }
    }
    // this and another partial result of the same rows
    template <typename Load>
    __device__ __forceinline__ void join(Load load)
    {
        float wa[2], wb[2];
#pragma unroll
        for (int r = 0; r < Sh::NR; ++r) {
            const float m2 = load(Sh::NO + r), l2 = load(Sh::NO + Sh::NR + r);
            const float mn = fmaxf(m[r], m2), bs = base(mn);
            wa[r] = ex2(m[r] - bs);
            wb[r] = ex2(m2 - bs);
            l[r] = l[r] * wa[r] + l2 * wb[r];
            m[r] = mn;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int c = 0; c < (TWO ? 2 : 4); ++c) {
                    const int r = TWO ? 0 : c >> 1;
                    o[b][n][c] = o[b][n][c] * wa[r] + load((b * 4 + n) * (TWO ? 2 : 4) + c) * wb[r];
                }
    }
    template <typename Store>
    __device__ __forceinline__ void put(Store store) const
    {
#pragma unroll
        for (int r = 0; r < Sh::NR; ++r) store(Sh::NO + r, m[r]), store(Sh::NO + Sh::NR + r, l[r]);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int c = 0; c < (TWO ? 2 : 4); ++c) store((b * 4 + n) * (TWO ? 2 : 4) + c, o[b][n][c]);
    }
};

template <int FMT, int NB, bool TWO>
__global__ void __launch_bounds__(AttnShape<FMT, NB, TWO>::MAX_WARPS * 32, 1)
    attn_split_kernel(const AttnArgs a, const AttnPlan p, unsigned int* status)
{
    using Sh = AttnShape<FMT, NB, TWO>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ AttnWalk s_walk;
    __shared__ int64_t s_chunk;
    __shared__ int s_last, s_dead;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int split = warp / p.wr, wrow = warp - split * p.wr;
    const int items = a.L.heads * p.row_groups;
    const int S = p.stages;
    uint8_t* ring = smem + (size_t)split * S * Sh::TILE;
    float* merge = reinterpret_cast<float*>(smem + p.off_merge);
    uint4* q_smem = reinterpret_cast<uint4*>(smem + p.off_q) + wrow * (NB * 2 * 32) + lane;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.off_bar) + split * S;
    uint64_t* empty = reinterpret_cast<uint64_t*>(smem + p.off_bar) + (p.ws + split) * S;
    int* bad_page = reinterpret_cast<int*>(smem + p.off_bar + 16 * p.ws * S) + split * S;

    pdl_launch_dependents();
    if (wrow == 0 && lane == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], p.wr);
        }
        fence_barrier_init();
    }
    if (threadIdx.x == 0) s_dead = 0;
    pdl_wait();

    if (warp == 0) {
        const int64_t total = attn_total(a, items, lane);
        int64_t chunk = (total + gridDim.x - 1) / gridDim.x;
        if (chunk < p.min_chunk) chunk = p.min_chunk;
        const int64_t start = chunk * blockIdx.x;
        const int64_t left = total - start < chunk ? total - start : chunk;
        AttnWalk w{};
        if (left > 0) w = attn_find(a, items, start, left, lane);
        if (lane == 0) {
            s_walk = w;
            s_chunk = chunk;
        }
    }
    // sequences of which no row sees anything: zeros (NaN where the length is bad)
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
        const AttnSpan sp(a, a.lens[b]);
        if (AttnTiles(sp).count) continue;
        const float none[4] = {sp.bad ? __int_as_float(0x7fffffff) : 0.0f, sp.bad ? __int_as_float(0x7fffffff) : 0.0f,
                               sp.bad ? __int_as_float(0x7fffffff) : 0.0f, sp.bad ? __int_as_float(0x7fffffff) : 0.0f};
        for (int i = threadIdx.x; i < a.rows * a.heads * NB * 8; i += blockDim.x) {
            const int rh = i / (NB * 8), d = (i - rh * (NB * 8)) * 4;
            const int64_t row = (int64_t)b * a.rows + rh / a.heads;
            const int head = rh % a.heads;
            store_row_part(a.out, row * a.o_row + head * a.o_head + d, p.type, false, none);
            if (a.lse && d == 0) a.lse[row * a.heads + head] = sp.bad ? none[0] : -INFINITY;
        }
    }
    __syncthreads();
    AttnWalk seg = s_walk;
    if (seg.done()) return;

    // ---- the ring: the lane that issues walks the same segments on its own
    const bool issuer = wrow == 0 && lane == 0;
    AttnWalk ahead = seg;
    int ah_tile = 2 * split, ah_slot = 0, ah_round = 0, issued = 0;  // next tile, counted from ahead.ta
    const uint64_t policy = l2_evict_first_policy();
    bool dead = false;
    const int tpp = a.L.tiles();
    auto issue = [&](int upto) {  // tiles of this split until `upto` are in flight or done
        while (issued < upto) {
            while (!ahead.done() && ahead.ta + ah_tile >= ahead.tb) {
                ahead.next(a, items);
                ah_tile = 2 * split;
            }
            if (ahead.done()) return;
            if (ah_round > 0 && !mbar_wait_bounded(&empty[ah_slot], (ah_round - 1) & 1)) {
                dead = true;
                return;
            }
            const int tile = ahead.first + ahead.ta + ah_tile, pg = tile / tpp;
            const int page = a.table[ahead.b * a.ld_table + pg];
            const int64_t off = a.L.tile_offset(page, ahead.item / p.row_groups, tile - pg * tpp);
            const bool ok = off >= 0 && QG_OK(qg_in(off, Sh::TILE, a.L.bytes()), status, 731);
            bad_page[ah_slot] = !ok;
            mbar_arrive_expect_tx(&full[ah_slot], ok ? Sh::TILE : 0u);
            if (ok) bulk_g2s(ring + (size_t)ah_slot * Sh::TILE, a.cache + off, Sh::TILE, &full[ah_slot], policy);
            ++issued;
            ah_tile += (ah_tile & 1) ? 2 * p.ws - 1 : 1;
            if (++ah_slot == S) ah_slot = 0, ++ah_round;
        }
    };
    if (issuer) issue(S);
    int taken = 0, slot = 0, phase = 0;  // tiles of this split

    AttnState<FMT, NB, TWO> st;
    const bool q_wide = rows_wide(a.q, a.q_row, a.q_head, p.type);
    const bool o_wide = rows_wide(a.out, a.o_row, a.o_head, p.type);
    int n_seg = 0;

    for (; !seg.done(); seg.next(a, items), ++n_seg) {
        const AttnSpan sp(a, a.lens[seg.b]);
        const int kvh = seg.item / p.row_groups;
        const int row_tile = (seg.item - kvh * p.row_groups) * p.wr + wrow;
        // ---- q: this lane's rows, scaled to 2^13 .. 2^14, as A fragments
        uint32_t qf[Sh::Q_SMEM ? 1 : NB * 2][4];
        float rs[Sh::NR];
        int end[Sh::NR], begin[Sh::NR];
        if (Sh::Q_SMEM) __syncthreads();  // the previous segment's readers are done
#pragma unroll
        for (int r = 0; r < Sh::NR; ++r) {
            const int rr = row_tile * Sh::ROWS + g + 8 * r;
            const bool in = rr < a.rows * a.group;
            const int i = in ? rr / a.group : 0;
            end[r] = in ? sp.end(i) : 0;
            begin[r] = in ? sp.begin(i) : 0;
            const int64_t at = ((int64_t)seg.b * a.rows + i) * a.q_row + (int64_t)(kvh * a.group + rr - i * a.group) * a.q_head;
            float qv[NB][8];
            uint32_t top = 0;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    const int d = b * 32 + (FMT == QGEMV_KV_Q4_0 ? 16 * h + 4 * t : 8 * t + 4 * h);
                    if (in) load_row_part(a.q, at + d, p.type, q_wide, x);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // q4_0: values 4 t + {0, 1, 2, 3} go to places {0, 2, 1, 3}
                        const int place = FMT == QGEMV_KV_Q4_0 ? 4 * h + ((k & 1) << 1) + (k >> 1) : 4 * h + k;
                        qv[b][place] = x[k];
                        top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
                    }
                }
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            int ex = (int)(top >> 23) - 127;  // |q| < 2^(ex + 1)
            ex = max(-100, min(127, ex));
            const float up = __int_as_float((127 + 13 - ex) << 23);
            rs[r] = a.scale * 1.4426950408889634f * __int_as_float((127 - 13 + max(ex, -113)) << 23);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x = qv[b][2 * k] * up, y = qv[b][2 * k + 1] * up;
                    const __half2 h = __floats2half2_rn(x, y);
                    hi[k] = h2_bits(h);
                    if (TWO) {
                        const float2 f = __half22float2(h);
                        lo[k] = h2_bits(__floats2half2_rn(x - f.x, y - f.y));
                    }
                }
                // k step s: a0, a2 of row g (+ 8: a1, a3)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if constexpr (Sh::Q_SMEM) {
                        uint32_t* w = reinterpret_cast<uint32_t*>(q_smem + (b * 2 + s) * 32);
                        if (split == 0) {
                            w[r] = hi[2 * s], w[2 + r] = hi[2 * s + 1];
                            if (TWO) w[1] = lo[2 * s], w[3] = lo[2 * s + 1];
                        }
                    } else {
                        qf[b * 2 + s][r] = hi[2 * s], qf[b * 2 + s][2 + r] = hi[2 * s + 1];
                        if (TWO) qf[b * 2 + s][1] = lo[2 * s], qf[b * 2 + s][3] = lo[2 * s + 1];
                    }
                }
            }
        }
        if (Sh::Q_SMEM) __syncthreads();
        // tiles all of whose tokens every row sees need no mask
        const int clear_from = sp.begin(a.rows - 1), clear_to = sp.end(0);
        bool poison = false;
        st.clear();

        for (int tl = seg.ta + 2 * split; tl < seg.tb; tl += 2 * p.ws) {
            const int n = min(2, seg.tb - tl);
            if (issuer && !dead) issue(taken + S);
            const uint8_t* tile[2];
            uint64_t* done[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                tile[u] = ring + (size_t)slot * Sh::TILE;
                done[u] = &empty[slot];
                if (u < n) {
                    dead = __any_sync(0xffffffffu, dead) || !__all_sync(0xffffffffu, mbar_wait_bounded(&full[slot], phase));
                    if (!dead && bad_page[slot]) poison = true;
                    if (++slot == S) slot = 0, phase ^= 1;
                }
            }
            taken += n;
            if (dead) break;
            if (poison) {  // a stage without its tile: the rows are NaN whatever comes
                __syncwarp();
                if (lane == 0)
                    for (int u = 0; u < n; ++u) mbar_arrive(done[u]);
                continue;
            }

            // ---- scores
            float y[2][4 * Sh::NR];
            uint32_t hidden = 0;  // bit (tile, value): masked
            bool edge[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int k = 0; k < 4 * Sh::NR; ++k) y[u][k] = u < n ? 0.0f : -INFINITY;
                const int pos = (seg.first + tl + u) * KV_TILE;
                edge[u] = pos < clear_from || pos + KV_TILE > clear_to;
                if (u >= n) continue;
                const uint8_t* k8 = tile[u];
                float c16[2][4] = {};
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float c[2][4] = {};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t f[4];
                        k_fragment<FMT>(k8, b, tile_token(g >> 1, 2 * j + (g & 1)), t, f);
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            uint32_t qa[4];
                            if constexpr (Sh::Q_SMEM) {
                                const uint4 w = q_smem[(b * 2 + s) * 32];
                                qa[0] = w.x, qa[1] = w.y, qa[2] = w.z, qa[3] = w.w;
                            } else {
#pragma unroll
                                for (int z = 0; z < 4; ++z) qa[z] = qf[b * 2 + s][z];
                            }
                            mma_f16(FMT == QGEMV_KV_F16 ? c16[j] : c[j], qa, f[2 * s], f[2 * s + 1]);
                        }
                    }
                    if constexpr (FMT != QGEMV_KV_F16) {
                        const uint2 w = *reinterpret_cast<const uint2*>(k8 + NB * KV_TILE * kv_code_bytes(FMT) + b * 32 + 8 * t);
                        const float2 d01 = __half22float2(bits_h2(w.x)), d23 = __half22float2(bits_h2(w.y));
                        const float d[4] = {d01.x, d01.y, d23.x, d23.y};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (TWO) {
                                y[u][i] = fmaf(d[i], c[i >> 1][i & 1] + c[i >> 1][2 + (i & 1)], y[u][i]);
                            } else {
                                y[u][i] = fmaf(d[i], c[i >> 1][i & 1], y[u][i]);
                                y[u][4 * (Sh::NR - 1) + i] = fmaf(d[i], c[i >> 1][2 + (i & 1)], y[u][4 * (Sh::NR - 1) + i]);
                            }
                        }
                    }
                }
                if constexpr (FMT == QGEMV_KV_F16) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (TWO) {
                            y[u][i] = c16[i >> 1][i & 1] + c16[i >> 1][2 + (i & 1)];
                        } else {
                            y[u][i] = c16[i >> 1][i & 1];
                            y[u][4 * (Sh::NR - 1) + i] = c16[i >> 1][2 + (i & 1)];
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 4 * Sh::NR; ++k) y[u][k] *= rs[k >> 2];
                if (edge[u]) {
#pragma unroll
                    for (int k = 0; k < 4 * Sh::NR; ++k) {
                        const int x = pos + tile_token(t, k & 3);
                        if (x >= end[k >> 2] || x < begin[k >> 2]) {
                            y[u][k] = -INFINITY;
                            hidden |= 1u << (u * 8 + k);
                        }
                    }
                }
            }

            // ---- V's scales and the largest of them, among tokens that any row sees
            uint2 dv[FMT == QGEMV_KV_F16 ? 1 : 2][NB];
            int e = st.e;
            if constexpr (FMT != QGEMV_KV_F16) {
                __half2 top = bits_h2(0u);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (u >= n) continue;
                    uint32_t live[2] = {0xffffffffu, 0xffffffffu};
                    if (edge[u]) {
                        const int pos = (seg.first + tl + u) * KV_TILE;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int x = pos + tile_token(t, i);
                            if (x < sp.first() || x >= sp.last()) live[i >> 1] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
                        }
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint2 w = *reinterpret_cast<const uint2*>(tile[u] + Sh::HALF + NB * KV_TILE * kv_code_bytes(FMT) +
                                                                  b * 32 + 8 * t);
                        w.x &= live[0], w.y &= live[1];
                        dv[u][b] = w;
                        top = __hmax2(top, __hmax2(__habs2(bits_h2(w.x)), __habs2(bits_h2(w.y))));
                    }
                }
                uint32_t bits = max((uint32_t)__half_as_ushort(__low2half(top)), (uint32_t)__half_as_ushort(__high2half(top)));
                bits = __reduce_max_sync(0xffffffffu, bits);
                if (bits < 0x7c00u) e = max(e, (int)(bits >> 10));  // d_v < 2^(e - 14)
            }

            // ---- the running maximum; the sums are rescaled only where it or e grows
            float mx[Sh::NR];
            bool grow = e > st.e;
#pragma unroll
            for (int r = 0; r < Sh::NR; ++r) {
                float v = -INFINITY;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) v = fmaxf(v, y[u][4 * r + i]);
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                mx[r] = v;
                grow |= v > st.m[r];
            }
            if (__any_sync(0xffffffffu, grow)) {
                const float down = __int_as_float((127 + st.e - e) << 23);
                float f[Sh::NR];
#pragma unroll
                for (int r = 0; r < Sh::NR; ++r) {
                    const float mn = fmaxf(st.m[r], mx[r]);
                    f[r] = ex2(st.m[r] - st.base(mn));
                    st.l[r] *= f[r];
                    f[r] *= down;
                    st.m[r] = mn;
                }
                st.e = e;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int nn = 0; nn < 4; ++nn)
#pragma unroll
                        for (int c = 0; c < 4; ++c) st.o[b][nn][c] *= f[TWO ? 0 : c >> 1];
            }
#pragma unroll
            for (int r = 0; r < Sh::NR; ++r) {
                const float bs = st.base(st.m[r]);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[u][4 * r + i] = ex2(y[u][4 * r + i] - bs);
                        st.l[r] += y[u][4 * r + i];
                    }
            }

            // ---- outputs
            const float up = FMT == QGEMV_KV_F16 ? 0x1p14f : __int_as_float((127 + 28 - st.e) << 23);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (u >= n) continue;
                const uint8_t* v8 = tile[u] + Sh::HALF;
                uint32_t pa[4];
                auto weights = [&](const float (&d)[4]) {
                    float w[4 * Sh::NR];
#pragma unroll
                    for (int k = 0; k < 4 * Sh::NR; ++k) w[k] = y[u][k] * d[k & 3];
                    if (edge[u]) {
#pragma unroll
                        for (int k = 0; k < 4 * Sh::NR; ++k)
                            if (hidden >> (u * 8 + k) & 1) w[k] = 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const __half2 h = __floats2half2_rn(w[2 * j], w[2 * j + 1]);
                        pa[2 * j] = h2_bits(h);
                        if (TWO) {
                            const float2 f = __half22float2(h);
                            pa[2 * j + 1] = h2_bits(__floats2half2_rn(w[2 * j] - f.x, w[2 * j + 1] - f.y));
                        } else {
                            pa[2 * j + 1] = h2_bits(__floats2half2_rn(w[4 * (Sh::NR - 1) + 2 * j], w[4 * (Sh::NR - 1) + 2 * j + 1]));
                        }
                    }
                };
                bool odd_values = false;  // f16 at the edge: infinities or NaN among the values that some row sees
                uint32_t live[2] = {0xffffffffu, 0xffffffffu};
                if constexpr (FMT == QGEMV_KV_F16) {
                    const float one[4] = {up, up, up, up};
                    weights(one);
                    if (edge[u]) {
                        const int pos = (seg.first + tl + u) * KV_TILE;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int x = pos + tile_token(t, i);
                            if (x < sp.first() || x >= sp.last()) live[i >> 1] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
                        }
                    }
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if constexpr (FMT != QGEMV_KV_F16) {
                        const float2 d01 = __half22float2(bits_h2(dv[u][b].x)), d23 = __half22float2(bits_h2(dv[u][b].y));
                        const float d[4] = {d01.x * up, d01.y * up, d23.x * up, d23.y * up};
                        weights(d);
                    }
                    uint32_t lo[4], hi[4];
                    v_fragments<FMT>(v8, b, g, t, lo, hi);
                    if constexpr (FMT == QGEMV_KV_F16) {
                        if (edge[u]) {
#pragma unroll
                            for (int nn = 0; nn < 4; ++nn) {
                                lo[nn] &= live[0], hi[nn] &= live[1];
                                auto finite = [&](uint32_t w) {
                                    if ((w & 0x7c00u) == 0x7c00u) w &= 0xffff0000u, odd_values = true;
                                    if ((w & 0x7c000000u) == 0x7c000000u) w &= 0x0000ffffu, odd_values = true;
                                    return w;
                                };
                                lo[nn] = finite(lo[nn]), hi[nn] = finite(hi[nn]);
                            }
                        }
                    }
#pragma unroll
                    for (int nn = 0; nn < 4; ++nn) mma_f16(st.o[b][nn], pa, lo[nn], hi[nn]);
                }
                if constexpr (FMT == QGEMV_KV_F16) {
                    // such values went in as zeros; add them to the rows that see them
                    if (edge[u] && __any_sync(0xffffffffu, odd_values)) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            for (int tt = 0; tt < 4; ++tt) {
                                const int tok = tile_token(tt, i);
                                float w[Sh::NR];
                                bool see[Sh::NR];
#pragma unroll
                                for (int r = 0; r < Sh::NR; ++r) {
                                    w[r] = __shfl_sync(0xffffffffu, y[u][4 * r + i], (lane & 28) | tt) * up;
                                    see[r] = !(__shfl_sync(0xffffffffu, hidden, (lane & 28) | tt) >> (u * 8 + 4 * r + i) & 1);
                                }
#pragma unroll
                                for (int b = 0; b < NB; ++b)
#pragma unroll
                                    for (int nn = 0; nn < 4; ++nn)
#pragma unroll
                                        for (int c = 0; c < 2; ++c) {
                                            const float x = __half2float(reinterpret_cast<const __half*>(v8)[(b * KV_TILE + tok) * 32 + 4 * (2 * t + c) + nn]);
                                            if (isfinite(x)) continue;
#pragma unroll
                                            for (int r = 0; r < Sh::NR; ++r)
                                                if (see[r]) st.o[b][nn][2 * r + c] += w[r] * x;
                                        }
                            }
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                for (int u = 0; u < n; ++u) mbar_arrive(done[u]);
        }
        st.finish(poison || dead);
        if (dead && lane == 0) s_dead = 1;

        // ---- the splits' partial results, in shared memory
        auto meet = [&]() {
            for (int k = p.ws; k > 1;) {
                const int h = (k + 1) / 2;
                float* buf = merge + (size_t)((split >= h ? split - h : split) * p.wr + wrow) * Sh::PART + lane;
                __syncthreads();
                if (split >= h && split < k) st.put([&](int i, float v) { buf[i * 32] = v; });
                __syncthreads();
                if (split < k - h) st.join([&](int i) { return buf[i * 32]; });
                k = h;
            }
        };
        auto write_out = [&]() {
#pragma unroll
            for (int r = 0; r < Sh::NR; ++r) {
                const int rr = row_tile * Sh::ROWS + g + 8 * r;
                if (rr >= a.rows * a.group) continue;
                const int i = rr / a.group;
                const int64_t row = (int64_t)seg.b * a.rows + i;
                const int head = kvh * a.group + rr - i * a.group;
                const float inv = st.l[r] == 0.0f ? 0.0f : __fdiv_rn(1.0f, st.l[r]);
                const bool none = st.l[r] == 0.0f;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            // q4_0: values 16 h + 4 t + k; else 8 t + 4 h + k
                            const float x = FMT == QGEMV_KV_Q4_0 ? st.o[b][2 * (k & 1) + h][2 * r + (k >> 1)] : st.o[b][k][2 * r + h];
                            v[k] = none ? 0.0f : x * inv;
                        }
                        const int d = b * 32 + (FMT == QGEMV_KV_Q4_0 ? 16 * h + 4 * t : 8 * t + 4 * h);
                        store_row_part(a.out, row * a.o_row + head * a.o_head + d, p.type, o_wide, v);
                    }
                if (a.lse && t == 0)
                    a.lse[row * a.heads + head] = none ? -INFINITY : 0.6931471805599453f * st.m[r] + logf(st.l[r]);
            }
        };
        meet();
        if (seg.ta == 0 && seg.tb == seg.count) {
            if (split == 0) write_out();
            continue;
        }
        // ---- an item cut between CTAs
        const int64_t chunk = s_chunk, here = chunk * blockIdx.x;
        // the item's first tile in the line, and the CTAs that share it
        const int64_t line = n_seg == 0 ? here - seg.ta : chunk * (blockIdx.x + 1) - seg.tb;
        const int c0 = (int)(line / chunk), c1 = (int)((line + seg.count - 1) / chunk);
        auto part = [&](int c) {
            const int second = c == c0 && line != chunk * c;
            return a.partials + ((size_t)(2 * c + second) * p.wr + wrow) * Sh::PART + lane;
        };
        if (split == 0) {
            float* w = part(blockIdx.x);
            st.put([&](int i, float v) { __stcg(w + i * 32, v); });
            __threadfence();
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            const unsigned int before = atomicAdd(&a.counters[c0], 1u);
            s_last = before == (unsigned)(c1 - c0);
            if (s_last) a.counters[c0] = 0;
            __threadfence();
        }
        __syncthreads();
        if (!s_last) continue;
        st.clear();
        for (int c = c0 + split; c <= c1; c += p.ws) {
            const float* w = part(c);
            st.join([&](int i) { return __ldcg(w + i * 32); });
        }
        meet();
        if (split == 0) write_out();
    }

    if (issuer && dead) {  // copies of its own that it did not wait for
        for (int q = taken < 2 ? 0 : taken - 2; q < issued; ++q) mbar_wait_bounded(&full[q % S], (q / S) & 1);
    }
    __syncthreads();
    if (threadIdx.x == 0 && s_dead) atomicAdd_system(status, 1u);
}

template <int FMT, int NB, bool TWO>
AttnPlan attn_plan(const DeviceInfo& di, int type, int rows)
{
    using Sh = AttnShape<FMT, NB, TWO>;
    AttnPlan p{};
    p.type = type;
    p.row_tiles = (rows + Sh::ROWS - 1) / Sh::ROWS;
    p.row_groups = (p.row_tiles + Sh::MAX_WARPS - 1) / Sh::MAX_WARPS;
    p.wr = (p.row_tiles + p.row_groups - 1) / p.row_groups;
    p.ws = Sh::MAX_WARPS / p.wr;
    for (;; --p.ws) {
        const uint32_t merge = (uint32_t)(p.ws / 2) * p.wr * Sh::PART * 4;
        const uint32_t q = Sh::Q_SMEM ? (uint32_t)p.wr * NB * 2 * 32 * 16 : 0;
        const uint32_t per_stage = (uint32_t)p.ws * (Sh::TILE + 2 * 8 + 4);
        const uint32_t fixed = merge + q + 256;
        const uint32_t budget = (uint32_t)di.smem_optin - 1024;
        const int stages = budget > fixed ? (int)((budget - fixed) / per_stage) : 0;
        if (stages < 4 && p.ws > 1) continue;
        p.stages = stages > 8 ? 8 : stages;
        p.off_merge = (uint32_t)p.ws * p.stages * Sh::TILE;
        p.off_q = p.off_merge + merge;
        p.off_bar = p.off_q + q;
        p.bytes = p.off_bar + (uint32_t)p.ws * p.stages * 20;
        break;
    }
    p.min_chunk = 2 * p.ws;
    return p;
}

template <int FMT, int NB, bool TWO>
int launch_attn_split(int type, const AttnArgs& a, cudaStream_t s)
{
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return QGEMV_CUDA_ERROR;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return QGEMV_CUDA_ERROR;
    const AttnPlan p = attn_plan<FMT, NB, TWO>(di, type, a.rows * a.group);
    if (p.stages < 2) return QGEMV_UNSUPPORTED_SHAPE;
    auto kern = attn_split_kernel<FMT, NB, TWO>;
    static std::once_flag once[64];
    static bool ok[64];
    std::call_once(once[dev], [&]() {
        ok[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, di.smem_optin - 1024) ==
                      cudaSuccess &&
                  wait_timeout_counter() != nullptr;
        if (!ok[dev]) cudaGetLastError();
    });
    if (!ok[dev]) return QGEMV_CUDA_ERROR;
    const int grid = di.sms < ATTN_GRID ? di.sms : ATTN_GRID;
    if (launch_pdl(kern, dim3(grid), dim3(p.ws * p.wr * 32), p.bytes, s, a, p, wait_timeout_counter()) != cudaSuccess)
        return QGEMV_CUDA_ERROR;
    return cudaGetLastError() == cudaSuccess ? QGEMV_OK : QGEMV_CUDA_ERROR;
}

template <int FMT, bool TWO>
int launch_attn_dim(int type, const AttnArgs& a, cudaStream_t s)
{
    switch (a.L.nb) {
    case 2: return launch_attn_split<FMT, 2, TWO>(type, a, s);
    case 3: return launch_attn_split<FMT, 3, TWO>(type, a, s);
    case 4: return launch_attn_split<FMT, 4, TWO>(type, a, s);
    default: return launch_attn_split<FMT, 8, TWO>(type, a, s);
    }
}

template <int FMT>
int launch_attn_type(int type, const AttnArgs& a, cudaStream_t s)
{
    return type == QGEMV_BF16 ? launch_attn_dim<FMT, false>(type, a, s) : launch_attn_dim<FMT, true>(type, a, s);
}

int launch_attn_f16(int type, const AttnArgs& a, cudaStream_t s);
int launch_attn_q8_0(int type, const AttnArgs& a, cudaStream_t s);
int launch_attn_q4_0(int type, const AttnArgs& a, cudaStream_t s);

}  // namespace qgemv
