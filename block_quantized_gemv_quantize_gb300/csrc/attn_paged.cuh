// attn_paged: attention of a few new tokens over the block-quantized paged
// cache, on the tensor cores straight from the blocks.
//
// Mathematics.  A row is one (new token, q head); the rows that share a kv
// head go together.  With codes c and block scales d (kvcache.cuh),
//     s[row][p] = scale sum_b d_k[p][b] sum_{i in b} q[row][i] c_k[p][i]
//     out[row][i] = sum_p w[row][p] d_v[p][b(i)] c_v[p][i] / sum_p w[row][p]
// with w = 2^(s log2 e - m), m a maximum of the row that lags its true one by
// at most 4 (so sums are rescaled a few times, not at every new maximum).  The
// codes are small integers, so they are fp16 exactly and are the tensor cores'
// B operand without ever being scaled: K's scales multiply the fp32 block
// sums, V's the weights before they are rounded to fp16.  q and w d_v are fp16
// pairs hi + lo of 22 bits, whatever the rows' type (bf16 rows with one term of 11
// bits had one output in a hundred at a neighbouring value and were no faster: 46
// ragged sequences 80.5 us, 79.6 with a pair).  q is brought to 2^13 .. 2^14 by an
// exact power of two per row, w d_v to below 2^15 by one that follows the largest
// d_v seen so far, so that neither leaves fp16's range.  That one power for all rows
// and blocks loses nothing while the scales are within 2^12 of one another.  A warp
// that has met scales further apart, or some of zero, goes through its tiles again
// (ATTN_AGAIN), with powers for each row and block: then neither what other rows see,
// nor what other blocks hold, nor tokens without weight take bits from a product.  That
// makes a split two to four times as long (all of them, two of 131071 tokens in q4_0:
// 335 us, not 95); such powers in every step cost every call (17 rows at D = 256 98 us,
// not 76).  An fp16 cache's infinities and NaN, too, are left for such a second pass.
//
// Rows in an instruction of 16 (MODE):
//   ATTN_PAIR  8 rows: their hi in the lower half, their lo in the upper
//   ATTN_TWO   16 rows, hi and lo in two instructions; the blocks are unpacked
//              once for 16 rows, which from 9 rows on beats two ATTN_PAIR tiles
//
// Split.  An item is a (sequence, kv head, group of row tiles).  All items'
// tiles of 16 tokens stand in one line, each item with ATTN_ITEM_COST units in
// front for what it costs besides its tiles, and the line is cut into equal
// pieces, one a split: the load is even however the lengths differ, and the
// lengths are read on the device, so that a captured graph serves any.  A CTA
// has WS splits; each streams its piece through a ring of its own in shared
// memory that bulk copies fill, two tiles a stage (tiles of a kv head follow one
// another in a page: one copy for both, or two where a page ends between them),
// and WR warps share the ring, one for every tile of rows.  One more warp issues
// the copies, a lane a ring.  A split writes the outputs of an item that it has
// whole; of one that it shares it leaves a partial result (at most two) in the
// workspace, and the split that has the item's first tile leaves its record.  A
// second kernel joins the partial results of every recorded item, each output by
// as many warps as there are to spare, in the order of the splits: the result
// does not depend on the order in which CTAs finish.
//
// What bounds it.  46 ragged sequences of up to 8192 tokens (q8_0, bf16 rows):
// 80 us, 5.6 TB/s, nearly what the copies and the join take without the arithmetic.
// One kv head a query head in f16: 40 us, 5.2 TB/s, likewise.  Two sequences of
// 131071 tokens in q4_0 (fp16 rows): 95 us where the copies alone take 58: 415
// instructions a tile of 16 tokens and 8 rows, of which 32 are the products, at 0.56
// an SM quarter and cycle.  Width 6 over 17391 tokens (30 rows a kv head): 30 us, of
// them 20 in the splits at two instructions in five cycles an SM quarter (two warps
// each, 232 registers a thread).  17 rows with a window at D = 256: 76 us, six warps a
// CTA that each unpack every tile, at one instruction in three cycles.  A call of 197
// tokens takes 10 us: two launches, three dependent reads before the first tile arrives
// (lengths, page number, tile) and the join.
//
// Registers: 255 a thread do not hold all of D = 256.  Over 8 rows q8_0 and q4_0 spill
// 44 bytes at most; an f16 cache 190 bytes up to 8 rows, where memory bounds it all the
// same (8 sequences of 8192 tokens, 8 kv heads: 86 us, 6.3 TB/s), and 230 above.
#pragma once

#include <type_traits>

#include "kvcache.cuh"

namespace qgemv {

constexpr int ATTN_GRID = 160;       // most CTAs (one an SM): the workspace holds their partial results
constexpr int ATTN_JOIN_WARPS = 16;  // of a CTA of the joining kernel
// What an item costs besides its tiles (q, a cut into partial results), in tiles;
// even.  46 ragged sequences, and 17 rows with a window at D = 256, as they stood
// then: 94 and 84 us with 4, 87 and 79 with 8, 90 and 80 with 16.
constexpr int ATTN_ITEM_COST = 8;
// Least units of a split: a single sequence of 197 tokens takes 10.8 us with 2,
// 12.2 with 4, 15.1 with 8.
constexpr int ATTN_MIN_PIECE = 2;

enum AttnMode { ATTN_PAIR = 1, ATTN_TWO = 2 };

// The mode for a call: by the rows of a kv head.
inline int attn_mode(int rows) { return rows > 8 ? ATTN_TWO : ATTN_PAIR; }

// Shares of a split whose warps share their schedulers with another's, and of one
// whose warps do not.  The latter is faster where arithmetic bounds the kernel, by the
// rows a kv head and, for few of them, the format and D; where memory does it is not.
// 8 and 10, 8 kv heads, 8 sequences of 16384 * 128 / D tokens (from 30 rows on half):
//     rows       1              16             30
//     q8_0 D=64  61.6, 67.2 us  83.2, 80.8     97.4, 90.4
//     q8_0 D=128 54.4, 52.8     74.9, 73.0     86.4, 80.4
//     q4_0 D=64  64.1, 67.6     84.4, 82.6     99.5, 92.3
//     f16 D=64   85.9, 91.5     88.4, 93.4     77.6, 74.5
//     f16 D=128  87.8, 89.9     89.1, 87.6     65.3, 61.4
// (D = 96 and 256 like 128; from 48 rows on no split is alone, or all are.)
constexpr int ATTN_SHARE = 8;
inline int attn_share_alone(int fmt, int nb, int rows)
{
    return rows > (fmt == QGEMV_KV_F16 ? 16 : (nb > 2 ? 0 : 8)) ? 10 : ATTN_SHARE;
}

// Warps that compute (one more copies): eight warps leave a thread 255 registers.
// Eleven (168 registers, q in shared memory) measured 1 to 4 % faster where the
// cache is long and 15 to 20 % slower on short sequences.
constexpr int ATTN_WARPS = 7;

template <int FMT, int NB, int MODE>
struct AttnShape {
    static constexpr int ROWS = MODE == ATTN_PAIR ? 8 : 16;  // rows of a row tile
    static constexpr int NR = ROWS / 8;                      // rows whose statistics a lane keeps
    static constexpr int NC = 2 * NR;                        // output values of a lane and column tile
    static constexpr int NO = NB * 4 * NC;                   // output values of a lane
    static constexpr int PART = (NO + 2 * NR) * 32;          // floats of one row tile's partial result
    static constexpr int TILE = kv_tile_bytes(FMT, NB), HALF = kv_half_bytes(FMT, NB);
    static constexpr bool Q_SMEM = NB > 4 || MODE == ATTN_TWO;  // else q's fragments stay in registers
    static constexpr int Q_TERMS = MODE == ATTN_TWO ? 2 : 1;
    static constexpr int WARPS = ATTN_WARPS;
    static constexpr int STEP = 2;                           // tiles of a step without an edge
    static constexpr int RUNS = NB * NR;                     // runs of eight output values of a lane: (block b, row g + 8 r)
    // where value k of a run's half h stands among a lane's outputs
    __host__ __device__ static constexpr int place(int b, int h, int r, int k)
    {
        return FMT == QGEMV_KV_Q4_0 ? (b * 4 + 2 * (k & 1) + h) * NC + 2 * r + (k >> 1) : (b * 4 + k) * NC + 2 * r + h;
    }
    // and the first of them in the row, for lane column t
    __device__ static int column(int b, int h, int t) { return b * 32 + (FMT == QGEMV_KV_Q4_0 ? 16 * h + 4 * t : 8 * t + 4 * h); }
};

struct AttnPlan {
    int splits;          // of the whole grid
    uint32_t magic;      // attn_magic
    int ws, wr;          // splits, row tiles at a time
    int row_groups;
    int stages;          // pairs of tiles a ring holds
    int cum[ATTN_WARPS + 1];  // shares of a CTA's part of the line: split s has cum[s] .. cum[s + 1] of cum[ws]
    uint32_t off_q, off_bar, bytes;  // shared memory
    int drop_copy;       // test only: no copy for the stage with the first tile of the line
};

// How the line is cut: a CTA has `chunk` units of it, split s of the CTA those from
// start(s) on.  All even.
struct AttnCut {
    int64_t chunk, piece;
    bool even;  // all splits alike: too few units to weigh
    __device__ __forceinline__ AttnCut(const AttnPlan& p, int64_t total)
    {
        piece = (total + p.splits - 1) / p.splits;
        piece += piece & 1;
        if (piece < ATTN_MIN_PIECE) piece = ATTN_MIN_PIECE;
        even = piece < 8;  // (else the least share is of 4 units)
        const int ctas = p.splits / p.ws;
        chunk = even ? piece * p.ws : (total + ctas - 1) / ctas;
        chunk += chunk & 1;
    }
    __device__ __forceinline__ int64_t start(const AttnPlan& p, int s) const
    {
        if (even) return piece * s;
        return s == p.ws ? chunk : (chunk * p.cum[s] / p.cum[p.ws] + 1) & ~(int64_t)1;
    }
    // the split that has a unit of the line
    __device__ __forceinline__ int split_of(const AttnPlan& p, int64_t unit) const
    {
        const int64_t cta = unit / chunk;
        unit -= cta * chunk;
        int s = 0;
        while (s + 1 < p.ws && start(p, s + 1) <= unit) ++s;
        return (int)cta * p.ws + s;
    }
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

// Whether a phase is over, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// Codes to fp16 without a conversion, by the well-known technique of an integer in
// the mantissa of a power of two: 0x6400 | n is the fp16 number 1024 + n.
// The 0x64 bytes (`magic`) are an argument of the kernel, which the compiler does
// not see through: an instruction has room for one constant, so with two of them
// it would spend a second instruction on every word.
constexpr uint32_t attn_magic(int fmt) { return fmt == QGEMV_KV_Q8_0 ? 0x64646464u : 0x64006400u; }
// Two bytes of w, as 1024 + byte (code + 128), less 1152.
template <int SEL>
__device__ __forceinline__ uint32_t codes_q8(uint32_t w, uint32_t magic)
{
    return h2_bits(__hsub2(bits_h2(__byte_perm(w, magic, SEL)), bits_h2(0x64806480u)));
}
// The low nibbles of bytes 0 and 2: 1024 + code less 1032 (code - 8).
__device__ __forceinline__ uint32_t codes_q4_lo(uint32_t w, uint32_t magic)
{
    return h2_bits(__hsub2(bits_h2((w & 0x000F000Fu) | magic), bits_h2(0x64086408u)));
}
// Their high nibbles: (1024 + 16 code) / 16 - 72, exact in one fma.
__device__ __forceinline__ uint32_t codes_q4_hi(uint32_t w, uint32_t magic)
{
    return h2_bits(__hfma2(bits_h2((w & 0x00F000F0u) | magic), bits_h2(0x2C002C00u), bits_h2(0xD480D480u)));
}

// The four tokens of a tile that column pair t of the products holds: i = 0..3
// are the tokens 4 i + (t ^ 3 (i & 1)), an order in which neither K's loads (a
// token a lane quad) nor V's (four tokens a lane) meet in a bank.
__device__ __forceinline__ int tile_token(int t, int i) { return 4 * i + (t ^ (3 * (i & 1))); }

// K's B fragments of block b, columns 8 j .. 8 j + 7 of the tile: the values
// 8 t .. 8 t + 7 of the lane's token (q8_0, f16); or (q4_0) 4 t + {0, 2, 1, 3},
// then 16 + 4 t + {0, 2, 1, 3}.  q's fragments follow the same order.
template <int FMT>
__device__ __forceinline__ void k_fragment(const uint8_t* k, int b, int tok, int t, uint32_t magic, uint32_t (&f)[4])
{
    const uint8_t* p = k + (b * KV_TILE + tok) * kv_code_bytes(FMT) + t * (kv_code_bytes(FMT) / 4);
    if constexpr (FMT == QGEMV_KV_F16) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        f[0] = w.x, f[1] = w.y, f[2] = w.z, f[3] = w.w;
    } else if constexpr (FMT == QGEMV_KV_Q8_0) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        f[0] = codes_q8<0x4140>(w.x, magic), f[1] = codes_q8<0x4342>(w.x, magic);
        f[2] = codes_q8<0x4140>(w.y, magic), f[3] = codes_q8<0x4342>(w.y, magic);
    } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p), v = w >> 8;
        f[0] = codes_q4_lo(w, magic), f[1] = codes_q4_lo(v, magic), f[2] = codes_q4_hi(w, magic), f[3] = codes_q4_hi(v, magic);
    }
}

// V's B fragments of block b for its four column tiles: token pairs (0, 1) in
// lo, (2, 3) in hi; column n of tile nn is the block's value 4 n + nn, or (q4_0)
// 2 n + {0, 16, 1, 17}[nn].
template <int FMT>
__device__ __forceinline__ void v_fragments(const uint8_t* v, int b, int g, int t, uint32_t magic, uint32_t (&lo)[4],
                                            uint32_t (&hi)[4])
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
        lo[0] = codes_q8<0x4140>(x, magic), lo[1] = codes_q8<0x4342>(x, magic);
        lo[2] = codes_q8<0x4140>(y, magic), lo[3] = codes_q8<0x4342>(y, magic);
        x = __byte_perm(w[2], w[3], 0x5140), y = __byte_perm(w[2], w[3], 0x7362);
        hi[0] = codes_q8<0x4140>(x, magic), hi[1] = codes_q8<0x4342>(x, magic);
        hi[2] = codes_q8<0x4140>(y, magic), hi[3] = codes_q8<0x4342>(y, magic);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint16_t*>(at(i));
        uint32_t x = __byte_perm(w[0], w[1], 0x5410), y = x >> 8;
        lo[0] = codes_q4_lo(x, magic), lo[1] = codes_q4_hi(x, magic);
        lo[2] = codes_q4_lo(y, magic), lo[3] = codes_q4_hi(y, magic);
        x = __byte_perm(w[2], w[3], 0x5410), y = x >> 8;
        hi[0] = codes_q4_lo(x, magic), hi[1] = codes_q4_hi(x, magic);
        hi[2] = codes_q4_lo(y, magic), hi[3] = codes_q4_hi(y, magic);
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

// Units of an item on the line: even, as the pieces are, so that a split starts
// at an even tile of an item and takes its tiles in pairs.
__host__ __device__ constexpr int attn_item_units(int count) { return ATTN_ITEM_COST + count + (count & 1); }

// A split's walk over its piece of the line: segments, each a run of one item's
// tiles.
struct AttnWalk {
    int64_t left;      // units of the piece from this segment's first on
    int64_t line;      // the item's first unit
    int b, item;       // sequence, (kv head, row group) within it
    int first, count;  // the item's tiles
    int ta, tb;        // the segment's, counted from `first`
    int used;          // units of it
    __device__ __forceinline__ bool done() const { return left <= 0; }
    __device__ __forceinline__ void clip(int off)
    {
        const int units = attn_item_units(count) - off;
        used = left < (int64_t)units ? (int)left : units;
        ta = max(0, off - ATTN_ITEM_COST);
        tb = min(count, max(0, off + used - ATTN_ITEM_COST));
    }
    // to the next segment with tiles in it
    __device__ __forceinline__ void next(const AttnArgs& a, int items)
    {
        do {
            left -= used;
            if (left <= 0) return;
            line += attn_item_units(count);
            if (++item == items) {
                item = 0;
                do {
                    const AttnTiles n{AttnSpan(a, a.lens[++b])};  // left > 0: a later sequence has tiles
                    first = n.first;
                    count = n.count;
                } while (count == 0);
            }
            clip(0);
        } while (tb <= ta);
    }
};

__device__ __forceinline__ int64_t attn_units(const AttnTiles& t, int items)
{
    return t.count ? (int64_t)attn_item_units(t.count) * items : 0;
}

// By one warp: the length of the line, and the walk that starts at its unit
// `start`.
__device__ __forceinline__ int64_t attn_total(const AttnArgs& a, int items, int lane)
{
    int64_t n = 0;
    for (int b = lane; b < a.batch; b += 32) n += attn_units(AttnTiles(AttnSpan(a, a.lens[b])), items);
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n;
}

__device__ __forceinline__ AttnWalk attn_find(const AttnArgs& a, int items, int64_t start, int64_t left, int lane)
{
    AttnWalk w{};
    if (left <= 0) return w;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        const AttnTiles t = b < a.batch ? AttnTiles(AttnSpan(a, a.lens[b])) : AttnTiles();
        const int64_t own = attn_units(t, items);
        int64_t sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, own > 0 && before + sum > start);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int64_t at = before + __shfl_sync(0xffffffffu, sum - own, src);  // the sequence's first unit
            w.left = left;
            w.b = b0 + src;
            w.first = __shfl_sync(0xffffffffu, t.first, src);
            w.count = __shfl_sync(0xffffffffu, t.count, src);
            w.item = (int)((start - at) / attn_item_units(w.count));
            w.line = at + (int64_t)w.item * attn_item_units(w.count);
            w.clip((int)(start - w.line));
            if (w.tb <= w.ta) w.next(a, items);
            return w;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    return w;
}

// The fp16 pair hi + lo of two fp32 values.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    float dx, dy;
    add_f32x2(dx, dy, x, y, -f.x, -f.y);
    hi = h2_bits(h);
    lo = h2_bits(__floats2half2_rn(dx, dy));
}

// The least scale that the power of the largest still serves, as fp16 bits, for scales
// below 2^(e - 14): 2^(e - 27), whose products with a weight of 1 (every row has one)
// stand at 2^-2 or above, so that a rounding to hi + lo (2^-25 at most there) is off by
// 2^-23 of the row's and block's largest product.  (A scale of zero is too small: the
// row's weight may be all on such a token.)
__device__ __forceinline__ uint32_t attn_least_scale(int e)
{
    return e > 13 ? (uint32_t)(e - 12) << 10 : 1u << max(e - 3, 0);
}

// Powers of two for each row and block, a byte each: the upper byte of the float 2^s,
// s odd.  They start at the largest, which brings a weight of 1 and the smallest fp16
// number to 2^13, and fall where a product passes 2^15, to one that leaves the largest
// at 2^10 .. 2^12 (weights reach 2^4, so the smallest, 2^-7, suffices for any scale).
// Where the row's reference maximum grows, and all its weights shrink by f, they rise
// by 1 / f or a little more.  So the largest product of a row and block stands at 2^10
// or above, and no rounding is off by more than 2^-35 of it.
constexpr int ATTN_POWER_MOST = 82, ATTN_POWER_LEAST = 60;  // 2^37, 2^-7
__device__ __forceinline__ float attn_power(uint32_t word, int b)
{
    return __uint_as_float(__byte_perm(word, 0, 0x444 | (b & 3) << 12));
}
__device__ __forceinline__ float attn_inverse(float power) { return __int_as_float(0x7f000000 - __float_as_int(power)); }

template <int NB, int NR>
struct AttnPowers {
    static constexpr int WORDS = (NB + 3) / 4;
    uint32_t w[NR][WORDS];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (uint32_t& x : w[r]) x = ATTN_POWER_MOST * 0x01010101u;
    }
    __device__ __forceinline__ float of(int r, int b) const { return attn_power(w[r][b / 4], b); }
    // the power times 4^rise (of either sign), within the ends; returns by what it changed
    __device__ __forceinline__ float change(int r, int b, int rise)
    {
        uint32_t& x = w[r][b / 4];
        const int at = 8 * (b & 3), old = x >> at & 0xff, now = max(ATTN_POWER_LEAST, min(old + rise, ATTN_POWER_MOST));
        x += (uint32_t)(now - old) << at;
        return __int_as_float((127 + 2 * (now - old)) << 23);
    }
};

// What a warp keeps of its row tile while a segment runs: the rows' reference
// maximum (of s log2 e), this lane's share of the sum of weights, and the
// outputs times 2^(25 - e) (fp16 caches: 2^11) in the products' layout.
template <int FMT, int NB, int MODE>
struct AttnState {
    using Sh = AttnShape<FMT, NB, MODE>;
    float m[Sh::NR], l[Sh::NR], rs[Sh::NR];
    float o[NB][4][4];
    int e;  // V's scales are below 2^(e - 14); -1: all are zero so far
    __half2 least;  // of the scales that some row sees, as far as this lane looks at them
    uint32_t magic;

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
        e = -1;
        least = bits_h2(0x7c007c00u);
    }
    // the outputs of row r and block b times f
    __device__ __forceinline__ void scale(int r, int b, float f)
    {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (MODE == ATTN_PAIR || c >> 1 == r) o[b][n][c] *= f;
    }
    // Whether the segment has to be gone through again: its scales are too far apart for
    // one power; or its values, in an fp16 cache, hold an infinity or a NaN, which two
    // terms of a weight (lo is often negative or zero) and weights of zero make NaN of.
    __device__ __forceinline__ bool again() const
    {
        if constexpr (FMT == QGEMV_KV_F16) {
            float sum = 0.0f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) sum += o[b][n][c];
            return __any_sync(0xffffffffu, !isfinite(sum));
        }
        const uint32_t two = h2_bits(least), low = __reduce_min_sync(0xffffffffu, min(two & 0xffffu, two >> 16));
        return e >= 0 && low < attn_least_scale(e);
    }
    // End of a segment: l over the quad; the two halves of a split row added
    // (an infinite output stands in the high half alone); the scale out.
    __device__ __forceinline__ void finish(bool poison)
    {
#pragma unroll
        for (int r = 0; r < Sh::NR; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (poison) l[r] = __int_as_float(0x7fffffff);
        }
        const float back = FMT == QGEMV_KV_F16 ? 0x1p-11f : __int_as_float((127 + e - 25) << 23);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int c = 0; c < Sh::NC; ++c) {
                    float v = o[b][n][c];
                    if (MODE == ATTN_PAIR) v = isinf(v) ? v : v + o[b][n][c + 2];
                    o[b][n][c] = v * back;
                }
    }
};

// a finite base for exponents: a row that has seen nothing has m = -inf
__device__ __forceinline__ float attn_base(float m) { return m == -INFINITY ? 0.0f : m; }

// How a step takes its tiles: two whose tokens all rows see; one, of which some tokens
// may be hidden from some rows; and such a one with powers for each row and block, or
// with the infinities and NaN of an fp16 cache's values apart from the products.
enum AttnKind { ATTN_FULL, ATTN_EDGE, ATTN_AGAIN };

// What one step needs to know of its tiles.
struct AttnStep {
    const uint8_t* tile;  // the first one's, the other behind it
    int pos;          // position of its first token
    int first, last;  // positions that any row sees
};

// One step of a split, into a warp's row tile.
template <int FMT, int NB, int MODE, AttnKind KIND>
__device__ __forceinline__ void attn_step(AttnState<FMT, NB, MODE>& st, const AttnStep& x,
                                          AttnPowers<NB, AttnShape<FMT, NB, MODE>::NR>& powers,
                                          const uint32_t (&qf)[AttnShape<FMT, NB, MODE>::Q_SMEM ? 1 : NB * 2][4],
                                          const uint4* q_smem, const int (&begin)[AttnShape<FMT, NB, MODE>::NR],
                                          const int (&end)[AttnShape<FMT, NB, MODE>::NR], int lane)
{
    using Sh = AttnShape<FMT, NB, MODE>;
    constexpr bool EDGE = KIND != ATTN_FULL, POWERS = KIND == ATTN_AGAIN && FMT != QGEMV_KV_F16;
    constexpr bool APART = KIND == ATTN_AGAIN && FMT == QGEMV_KV_F16;
    constexpr int NT = EDGE ? 1 : Sh::STEP, NR = Sh::NR, NV = 4 * NR, SCALES = NB * KV_TILE * kv_code_bytes(FMT);
    const int g = lane >> 2, t = lane & 3;

    // ---- scores: y[u][4 r + i], row g + 8 r, token i of the lane's column pairs
    float y[NT][NV];
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int k = 0; k < NV; ++k) y[u][k] = 0.0f;
    float c16[NT][2][4] = {};
    // the tiles u0 .. u1 - 1 of block b: both at once where that halves the loads
    // of q's fragments, else one after the other, which needs fewer registers
    auto block = [&](int b, int u0, int u1) {
        float c[2][2][4] = {};
        uint32_t f[2][2][4];
#pragma unroll
        for (int u = u0; u < u1; ++u) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                k_fragment<FMT>(x.tile + u * Sh::TILE, b, tile_token(g >> 1, 2 * j + (g & 1)), t, st.magic, f[u][j]);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int term = 0; term < Sh::Q_TERMS; ++term) {
                uint32_t qa[4];
                if constexpr (Sh::Q_SMEM) {
                    const uint4 w = q_smem[((b * 2 + s) * Sh::Q_TERMS + term) * 32];
                    qa[0] = w.x, qa[1] = w.y, qa[2] = w.z, qa[3] = w.w;
                } else {
#pragma unroll
                    for (int z = 0; z < 4; ++z) qa[z] = qf[b * 2 + s][z];
                }
#pragma unroll
                for (int u = u0; u < u1; ++u) {
        #pragma unroll
                    for (int j = 0; j < 2; ++j)
                        mma_f16(FMT == QGEMV_KV_F16 ? c16[u][j] : c[u][j], qa, f[u][j][2 * s], f[u][j][2 * s + 1]);
                }
            }
        if constexpr (FMT != QGEMV_KV_F16) {
#pragma unroll
            for (int u = u0; u < u1; ++u) {
                    const uint2 w = *reinterpret_cast<const uint2*>(x.tile + u * Sh::TILE + SCALES + b * 32 + 8 * t);
                const float2 d[2] = {__half22float2(bits_h2(w.x)), __half22float2(bits_h2(w.y))};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (MODE == ATTN_PAIR) add_f32x2(c[u][j][0], c[u][j][1], c[u][j][0], c[u][j][1], c[u][j][2], c[u][j][3]);
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        fma_f32x2(y[u][4 * r + 2 * j], y[u][4 * r + 2 * j + 1], c[u][j][2 * r], c[u][j][2 * r + 1], d[j].x, d[j].y);
                }
            }
        }
    };
    if constexpr (Sh::Q_SMEM) {
#pragma unroll
        for (int b = 0; b < NB; ++b) block(b, 0, NT);
    } else {
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int b = 0; b < NB; ++b) block(b, u, u + 1);
    }
    // An infinite key of an fp16 cache: the low term makes NaN of the high term's
    // infinity, which alone is the score.
    auto together = [](float hi, float lo) { return isfinite(hi) ? hi + lo : hi; };
    if constexpr (FMT == QGEMV_KV_F16 && MODE == ATTN_TWO) {
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int p = x.pos + u * KV_TILE + tile_token(t, 2 * j + (c & 1));
                    if (!EDGE || (p >= x.first && p < x.last)) sum += c16[u][j][c];  // (the others may be anything)
                }
        if (__any_sync(0xffffffffu, !isfinite(sum))) {
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                float hi[2][4] = {};
#pragma unroll 1
                for (int bs = 0; bs < NB * 2; ++bs) {
                    const uint4 w = q_smem[bs * Sh::Q_TERMS * 32];
                    const uint32_t qa[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t f[4];
                        k_fragment<FMT>(x.tile + u * Sh::TILE, bs >> 1, tile_token(g >> 1, 2 * j + (g & 1)), t, st.magic, f);
                        mma_f16(hi[j], qa, bs & 1 ? f[2] : f[0], bs & 1 ? f[3] : f[1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (!isfinite(c16[u][j][c])) c16[u][j][c] = hi[j][c];
            }
        }
    }
    uint32_t hidden = 0;  // bit 8 u + k: y[u][k] is masked
#pragma unroll
    for (int u = 0; u < NT; ++u) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float &v0 = y[u][4 * r + 2 * j], &v1 = y[u][4 * r + 2 * j + 1];
                if constexpr (FMT == QGEMV_KV_F16) {
                    v0 = c16[u][j][2 * r], v1 = c16[u][j][2 * r + 1];
                    if (MODE == ATTN_PAIR) v0 = together(v0, c16[u][j][2]), v1 = together(v1, c16[u][j][3]);
                }
                mul_f32x2(v0, v1, v0, v1, st.rs[r], st.rs[r]);
            }
        if constexpr (EDGE) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int p = x.pos + u * KV_TILE + tile_token(t, k & 3);
                if (p >= end[k >> 2] || p < begin[k >> 2]) {
                    y[u][k] = -INFINITY;
                    hidden |= 1u << (u * 8 + k);
                }
            }
        }
    }
    // tokens that no row sees: their scales and values are anything
    uint32_t live[NT][2];
#pragma unroll
    for (int u = 0; u < NT; ++u) live[u][0] = live[u][1] = ~0u;
    if constexpr (EDGE) {
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = x.pos + u * KV_TILE + tile_token(t, i);
                if (p < x.first || p >= x.last) live[u][i >> 1] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
            }
    }

    // ---- the largest of V's scales, and the least: lane g's of block g
    int e = st.e;
    if constexpr (FMT != QGEMV_KV_F16 && !POWERS) {
        __half2 top = bits_h2(0u);  // hmax2 and hmin2 take the number of a number and a NaN
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            uint2 w = *reinterpret_cast<const uint2*>(x.tile + u * Sh::TILE + Sh::HALF + SCALES + g % NB * 32 + 8 * t);
            if (FMT == QGEMV_KV_Q4_0) w.x &= 0x7fff7fffu, w.y &= 0x7fff7fffu;  // q8_0's are never negative
            uint2 v = w;
            if (EDGE) {
                w.x &= live[u][0], w.y &= live[u][1];
                v.x |= ~live[u][0], v.y |= ~live[u][1];
            }
            top = __hmax2(top, __hmax2(bits_h2(w.x), bits_h2(w.y)));
            st.least = __hmin2(st.least, __hmin2(bits_h2(v.x), bits_h2(v.y)));
        }
        top = __hmax2(top, __lowhigh2highlow(top));
        const uint32_t bits = __reduce_max_sync(0xffffffffu, h2_bits(top) & 0xffffu);
        if (bits > 0 && bits < 0x7c00u) e = max(e, (int)(bits >> 10));
    }

    // ---- the sums are rescaled only where a maximum is passed by 4 (a factor
    // 2^4 in the weights, so w d_v stays below 2^15) or d_v takes another power of two
    float mx[NR];
    bool grow = e > st.e;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        float v = y[0][4 * r];
#pragma unroll
        for (int k = 1; k < 4 * NT; ++k) v = fmaxf(v, y[k >> 2][4 * r + (k & 3)]);
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
        mx[r] = v;
        grow |= v > st.m[r] + 4.0f;
    }
    if (__any_sync(0xffffffffu, grow)) {
        const float down = __int_as_float((127 + st.e - e) << 23);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float mn = fmaxf(st.m[r], mx[r]), f = ex2(st.m[r] - attn_base(mn));
            st.l[r] *= f;
            st.m[r] = mn;
            const int rise = (128 - (int)(__float_as_uint(f) >> 23)) >> 1;  // 4^rise >= 1 / f
#pragma unroll
            for (int b = 0; b < NB; ++b) st.scale(r, b, POWERS ? f * powers.change(r, b, rise) : f * down);
        }
        st.e = e;
    }
    // weights, and from here on times the outputs' scale
    const float up = FMT == QGEMV_KV_F16 ? 0x1p11f : (POWERS ? 1.0f : __int_as_float((127 + 25 - st.e) << 23));
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const float bs = -attn_base(st.m[r]);
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float &v0 = y[u][4 * r + 2 * j], &v1 = y[u][4 * r + 2 * j + 1];
                add_f32x2(v0, v1, v0, v1, bs, bs);
                v0 = ex2(v0);
                v1 = ex2(v1);
                add_f32x2(s0, s1, s0, s1, v0, v1);
                mul_f32x2(v0, v1, v0, v1, up, up);
            }
        st.l[r] += s0 + s1;
    }

    // ---- outputs
#pragma unroll
    for (int u = 0; u < NT; ++u) {
        const uint8_t* v8 = x.tile + u * Sh::TILE + Sh::HALF;
        uint32_t hi[4], lo[4];  // A fragments; ATTN_PAIR: hi alone, with the low terms in its upper rows
        auto weights = [&](const float2 (&d)[2], int b) {
            float w[NV];
#pragma unroll
            for (int k = 0; k < NV; k += 2) mul_f32x2(w[k], w[k + 1], y[u][k], y[u][k + 1], d[(k >> 1) & 1].x, d[(k >> 1) & 1].y);
            if constexpr (EDGE) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (hidden >> (u * 8 + k) & 1) w[k] = 0.0f;
            }
            if constexpr (POWERS) {
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    float most = 0.0f;  // (a number of a number and a NaN)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        w[4 * r + k] *= powers.of(r, b);
                        most = fmaxf(most, fabsf(w[4 * r + k]));
                    }
                    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                    const int fall = most >= 0x1p15f ? ((int)(__float_as_uint(most) >> 23) - 127 - 10) >> 1 : 0;
                    if (__any_sync(0xffffffffu, fall > 0)) {
                        const float by = powers.change(r, b, -fall);
                        st.scale(r, b, by);
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[4 * r + k] *= by;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if constexpr (MODE == ATTN_PAIR) {
                    split_pair(w[2 * j], w[2 * j + 1], hi[2 * j], hi[2 * j + 1]);
                } else {
#pragma unroll
                    for (int r = 0; r < 2; ++r) split_pair(w[4 * r + 2 * j], w[4 * r + 2 * j + 1], hi[2 * j + r], lo[2 * j + r]);
                }
            }
        };
        bool odd_values = false;  // infinities or NaN that some row sees
        if constexpr (FMT == QGEMV_KV_F16) {
            const float2 one[2] = {{1.0f, 1.0f}, {1.0f, 1.0f}};
            weights(one, 0);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if constexpr (FMT != QGEMV_KV_F16) {
                uint2 w = *reinterpret_cast<const uint2*>(v8 + SCALES + b * 32 + 8 * t);
                const float2 d[2] = {__half22float2(bits_h2(w.x)), __half22float2(bits_h2(w.y))};
                weights(d, b);
            }
            uint32_t v0[4], v1[4];
            v_fragments<FMT>(v8, b, g, t, st.magic, v0, v1);
            if constexpr (FMT == QGEMV_KV_F16 && EDGE) {
#pragma unroll
                for (int nn = 0; nn < 4; ++nn) {
                    auto finite = [&](uint32_t w) {
                        if (!APART) return w;
                        if ((w & 0x7c00u) == 0x7c00u) w &= 0xffff0000u, odd_values = true;
                        if ((w & 0x7c000000u) == 0x7c000000u) w &= 0x0000ffffu, odd_values = true;
                        return w;
                    };
                    v0[nn] = finite(v0[nn] & live[u][0]), v1[nn] = finite(v1[nn] & live[u][1]);
                }
            }
#pragma unroll
            for (int nn = 0; nn < 4; ++nn) {
                mma_f16(st.o[b][nn], hi, v0[nn], v1[nn]);
                if constexpr (MODE == ATTN_TWO) mma_f16(st.o[b][nn], lo, v0[nn], v1[nn]);
            }
        }
        if constexpr (APART) {
            // such values went in as zeros; add them to the rows that see them
            if (__any_sync(0xffffffffu, odd_values)) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll 1
                    for (int tt = 0; tt < 4; ++tt) {
                        const int tok = tile_token(tt, i);
                        float w[NR];
                        bool see[NR];
#pragma unroll
                        for (int r = 0; r < NR; ++r) {
                            w[r] = __shfl_sync(0xffffffffu, y[u][4 * r + i], (lane & 28) | tt);
                            see[r] = !(__shfl_sync(0xffffffffu, hidden, (lane & 28) | tt) >> (u * 8 + 4 * r + i) & 1);
                        }
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int nn = 0; nn < 4; ++nn)
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    const float v = __half2float(
                                        reinterpret_cast<const __half*>(v8)[(b * KV_TILE + tok) * 32 + 4 * (2 * t + c) + nn]);
                                    if (isfinite(v)) continue;
#pragma unroll
                                    for (int r = 0; r < NR; ++r)
                                        if (see[r]) st.o[b][nn][2 * r + c] += w[r] * v;
                                }
                    }
            }
        }
    }
}

// What the split that has a shared item's first tile leaves of it, in one word:
// the partial results from this split's on (0: none), the item ((kv head, row
// group) within the sequence, below 2^24: at most 2^16 heads of 17 rows) and the
// sequence.
struct AttnRecord {
    uint64_t bits;
    static __device__ __forceinline__ AttnRecord of(int parts, int b, int item)
    {
        return {(uint64_t)parts | (uint64_t)item << 16 | (uint64_t)b << 40};
    }
    __device__ __forceinline__ int parts() const { return (int)(bits & 0xffffu); }
    __device__ __forceinline__ int item() const { return (int)(bits >> 16 & 0xffffffu); }
    __device__ __forceinline__ int b() const { return (int)(bits >> 40); }
};

__device__ __forceinline__ float* attn_part(const AttnArgs& a, const AttnPlan& p, int split, int which, int tile, int floats)
{
    return a.partials + (((size_t)split * 2 + which) * p.wr + tile) * floats;
}

// A row's four values of one run, normalised; and with the first run its
// log-sum-exp.
template <int FMT, int NB, int MODE, typename T>
__device__ __forceinline__ void attn_emit(const AttnArgs& a, const AttnPlan& p, bool wide, int b_seq, int item, int tile,
                                          int b, int h, int r, int lane, const float (&v)[4], float m, float l)
{
    using Sh = AttnShape<FMT, NB, MODE>;
    const int g = lane >> 2, t = lane & 3, kvh = item / p.row_groups;
    const int rr = ((item - kvh * p.row_groups) * p.wr + tile) * Sh::ROWS + g + 8 * r;
    if (rr >= a.rows * a.group) return;
    const int i = rr / a.group;
    const int64_t row = (int64_t)b_seq * a.rows + i;
    const int head = kvh * a.group + rr - i * a.group;
    const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
    float o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = l == 0.0f ? 0.0f : v[k] * inv;
    store_values(static_cast<T*>(a.out) + row * a.o_row + head * a.o_head + Sh::column(b, h, t), wide, o);
    if (a.lse && t == 0 && b == 0 && h == 0)
        a.lse[row * a.heads + head] = l == 0.0f ? -INFINITY : 0.6931471805599453f * m + logf(l);
}

template <int FMT, int NB, int MODE, typename T>
__global__ void __launch_bounds__((AttnShape<FMT, NB, MODE>::WARPS + 1) * 32, 1)
    attn_split_kernel(const AttnArgs a, const __grid_constant__ AttnPlan p, unsigned int* status)
{
    using Sh = AttnShape<FMT, NB, MODE>;
    constexpr int NR = Sh::NR;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ AttnWalk s_walk[Sh::WARPS];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int warps = p.ws * p.wr;  // those that compute
    const int split = warp / p.wr, wrow = warp - split * p.wr;
    static_assert(ATTN_GRID * Sh::WARPS <= ATTN_MAX_SPLITS, "a record for every split");
    const int items = a.L.heads * p.row_groups;
    const int S = p.stages;
    constexpr int STAGE = 2 * Sh::TILE;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.off_bar);
    uint64_t* empty = full + p.ws * S;
    int* bad_page = reinterpret_cast<int*>(empty + p.ws * S);

    pdl_launch_dependents();
    if (warp == warps) {
        for (int i = lane; i < p.ws * S; i += 32) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], p.wr);
        }
        fence_barrier_init();
    }
    pdl_wait();

    // the line, and this split's piece of it
    const int64_t total = attn_total(a, items, lane);
    const AttnCut cut(p, total);
    const int split_id = blockIdx.x * p.ws + split;
    AttnWalk seg{};
    if (warp < warps) {
        const int64_t first = cut.start(p, split), start = cut.chunk * blockIdx.x + first;
        const int64_t piece = cut.start(p, split + 1) - first;
        seg = attn_find(a, items, start, total - start < piece ? total - start : piece, lane);
        if (wrow == 0 && lane == 0) s_walk[split] = seg;
    }
    // sequences of which no row sees anything: zeros (NaN where the length is bad)
    const bool o_wide = KvRows{a.out, a.o_row, a.o_head}.wide<T>();
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
        const AttnSpan sp(a, a.lens[b]);
        if (AttnTiles(sp).count) continue;
        const float v = sp.bad ? __int_as_float(0x7fffffff) : 0.0f;
        const float none[4] = {v, v, v, v};
        for (int i = threadIdx.x; i < a.rows * a.heads * NB * 8; i += blockDim.x) {
            const int rh = i / (NB * 8), d = (i - rh * (NB * 8)) * 4;
            const int64_t row = (int64_t)b * a.rows + rh / a.heads;
            const int head = rh % a.heads;
            store_values(static_cast<T*>(a.out) + row * a.o_row + head * a.o_head + d, o_wide, none);
            if (a.lse && d == 0) a.lse[row * a.heads + head] = sp.bad ? v : -INFINITY;
        }
    }
    __syncthreads();

    if (warp == warps) {
        // ---- the copies: lane s walks split s's tiles.  All lanes stay
        // together: in each round those whose next stage is free issue a copy
        // (lanes that wait on their own stage, each in a loop of its own, ran
        // one after the other and bounded the kernel at 150 ns a tile).
        const uint64_t policy = l2_evict_first_policy();
        const int tpp = a.L.tiles();
        const bool mine = lane < p.ws;
        uint8_t* ring = smem + (size_t)(mine ? lane : 0) * S * STAGE;
        uint64_t *fl = full + (mine ? lane : 0) * S, *em = empty + (mine ? lane : 0) * S;
        int* bad = bad_page + (mine ? lane : 0) * S;
        AttnWalk w{};
        if (mine) w = s_walk[lane];
        int at = w.ta, slot = 0, round = 0, issued = 0;
        bool more = !w.done();
        // the tile's page and the next one's number, which is on the way early
        const int32_t* row = a.table;
        int page = -1, page_next = -1, n = 0, tile_in = 0, head = 0;
        auto after = [&]() {  // the number of page n + 1, if the segment has tiles there
            if ((n + 1) * tpp < w.first + w.tb) page_next = row[n + 1];
        };
        auto settle = [&]() {  // a segment's first tile
            const int tile = w.first + at;
            n = tile / tpp;
            tile_in = tile - n * tpp;
            head = w.item / p.row_groups;
            row = a.table + w.b * a.ld_table;
            page = row[n];
            after();
        };
        if (more) settle();
        const int dropped = p.drop_copy && more && w.line == 0 && w.ta == 0 ? 0 : -1;
        int idle = 0;
        while (__any_sync(0xffffffffu, more)) {
            const bool go = more && (round == 0 || mbar_test_wait(&em[slot], (round - 1) & 1));
            if (!__any_sync(0xffffffffu, go)) {
                if (++idle > (1 << 24)) break;  // a second or more
                __nanosleep(32);
                continue;
            }
            idle = 0;
            if (!go) continue;
            const int two = w.tb - at >= 2, apart = two && tile_in + 1 == tpp;
            const int64_t off = a.L.tile_offset(page, head, tile_in);
            const int64_t off2 = apart ? a.L.tile_offset(page_next, head, 0) : off;
            const bool ok = off >= 0 && off2 >= 0 &&
                            QG_OK(qg_in(off, apart ? Sh::TILE : (1 + two) * Sh::TILE, a.L.bytes()) &&
                                      qg_in(off2, Sh::TILE, a.L.bytes()), status, 731);
            bad[slot] = !ok;
            if (issued != dropped) mbar_arrive_expect_tx(&fl[slot], ok ? (1 + two) * Sh::TILE : 0u);
            if (ok && issued != dropped) {
                uint8_t* to = ring + (size_t)slot * STAGE;
                bulk_g2s(to, a.cache + off, two && !apart ? 2 * Sh::TILE : Sh::TILE, &fl[slot], policy);
                if (apart) bulk_g2s(to + Sh::TILE, a.cache + off2, Sh::TILE, &fl[slot], policy);
            }
            ++issued;
            if (++slot == S) slot = 0, ++round;
            at += 1 + two;
            if (at >= w.tb) {
                w.next(a, items);
                at = w.ta;
                more = !w.done();
                if (more) settle();
            } else if ((tile_in += 2) >= tpp) {
                if (tpp == 1) {
                    n += 2;
                    page = row[n];
                    tile_in = 0;
                } else {
                    ++n;
                    page = page_next;
                    tile_in -= tpp;
                }
                after();
            }
        }
        // No copy outlives the CTA, whose warps may have given up waiting for theirs.
        for (int q = issued > S ? issued - S : 0; q < issued; ++q)
            if (q != dropped) mbar_wait_bounded(&fl[q % S], (q / S) & 1);
        if (more) atomicAdd_system(status, 1u);  // gave up
        return;
    }

    // ---- the warps that compute
    const uint8_t* ring = smem + (size_t)split * S * STAGE;
    uint4* q_smem = reinterpret_cast<uint4*>(smem + p.off_q) + warp * (NB * 2 * Sh::Q_TERMS * 32) + lane;
    const bool q_wide = KvRows{const_cast<void*>(a.q), a.q_row, a.q_head}.wide<T>();
    int slot = 0, phase = 0;
    bool dead = false;
    AttnState<FMT, NB, MODE> st;
    st.magic = p.magic;
    AttnRecord record{0};

    for (; !seg.done(); seg.next(a, items)) {
        const int kvh = seg.item / p.row_groups;
        const int row0 = ((seg.item - kvh * p.row_groups) * p.wr + wrow) * Sh::ROWS;
        const AttnSpan sp(a, a.lens[seg.b]);
        // ---- q: this lane's rows, scaled to 2^13 .. 2^14, as A fragments.  All
        // loads first (a row that does not exist loads the last one that does):
        // behind a branch each they came one after the other, 3.3 us for 16 rows.
        uint32_t qf[Sh::Q_SMEM ? 1 : NB * 2][4];
        int end[NR], begin[NR];
        bool in[NR];
        alignas(16) T raw[NR][NB * 2][4];
        {
            const T* row[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const int all = a.rows * a.group, rr = min(row0 + g + 8 * r, all - 1), i = rr / a.group;
                in[r] = row0 + g + 8 * r < all;
                end[r] = in[r] ? sp.end(i) : 0;
                begin[r] = in[r] ? sp.begin(i) : 0;
                row[r] = static_cast<const T*>(a.q) + ((int64_t)seg.b * a.rows + i) * a.q_row +
                         (int64_t)(kvh * a.group + rr - i * a.group) * a.q_head;
            }
            if (q_wide) {
                using Vec = std::conditional_t<sizeof(T) == 4, uint4, uint2>;
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int k = 0; k < NB * 2; ++k)
                        *reinterpret_cast<Vec*>(raw[r][k]) =
                            *reinterpret_cast<const Vec*>(row[r] + Sh::column(k >> 1, k & 1, t));
            } else {
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int k = 0; k < NB * 2; ++k)
#pragma unroll
                        for (int z = 0; z < 4; ++z) raw[r][k][z] = row[r][Sh::column(k >> 1, k & 1, t) + z];
            }
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float qv[NB][8];
            uint32_t top = 0;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // q4_0: values 4 t + {0, 1, 2, 3} go to places {0, 2, 1, 3}
                        const int place = FMT == QGEMV_KV_Q4_0 ? 4 * h + ((k & 1) << 1) + (k >> 1) : 4 * h + k;
                        const float x = in[r] ? to_f32(raw[r][2 * b + h][k]) : 0.0f;
                        qv[b][place] = x;
                        top = max(top, __float_as_uint(x) & 0x7fffffffu);
                    }
                }
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            int ex = (int)(top >> 23) - 127;  // |q| < 2^(ex + 1)
            ex = max(-100, min(127, ex));
            const float up = __int_as_float((127 + 13 - ex) << 23);
            st.rs[r] = a.scale * 1.4426950408889634f * __int_as_float((127 - 13 + ex) << 23);
            if (top >= 0x7f800000u) st.rs[r] = __int_as_float(0x7fffffff);  // no softmax of this row
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) split_pair(qv[b][2 * k] * up, qv[b][2 * k + 1] * up, hi[k], lo[k]);
                // k step s: a0, a2 of row g (+ 8: a1, a3)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if constexpr (Sh::Q_SMEM) {
                        uint32_t* w = reinterpret_cast<uint32_t*>(q_smem + (b * 2 + s) * Sh::Q_TERMS * 32);
                        w[r] = hi[2 * s], w[2 + r] = hi[2 * s + 1];
                        if (MODE == ATTN_PAIR) w[1] = lo[2 * s], w[3] = lo[2 * s + 1];
                        if (MODE == ATTN_TWO) w[128 + r] = lo[2 * s], w[130 + r] = lo[2 * s + 1];
                    } else {
                        qf[b * 2 + s][r] = hi[2 * s], qf[b * 2 + s][2 + r] = hi[2 * s + 1];
                        if (MODE == ATTN_PAIR) qf[b * 2 + s][1] = lo[2 * s], qf[b * 2 + s][3] = lo[2 * s + 1];
                    }
                }
            }
        }
        // (a lane reads back what it wrote itself: no barrier)
        // tiles all of whose tokens every row sees need no mask
        const int clear_from = sp.begin(a.rows - 1), clear_to = sp.end(0);
        bool poison = false;
        st.clear();

        AttnPowers<NB, NR> powers;
        for (int tl = seg.ta; tl < seg.tb; tl += 2) {
            const int used = split * S + slot;
            if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait_bounded(&full[used], phase));
            if (dead) break;
            // (a stage without its tiles: the rows are NaN whatever comes)
            if (bad_page[used]) poison = true;
            AttnStep x;
            x.tile = ring + (size_t)slot * STAGE;
            x.pos = (seg.first + tl) * KV_TILE;
            x.first = sp.first();
            x.last = sp.last();
            if (++slot == S) slot = 0, phase ^= 1;
            if (!poison) {
                if (tl + 2 <= seg.tb && x.pos >= clear_from && x.pos + 2 * KV_TILE <= clear_to) {
                    attn_step<FMT, NB, MODE, ATTN_FULL>(st, x, powers, qf, q_smem, begin, end, lane);
                } else {
#pragma unroll 1
                    for (int u = 0; u < 2 && tl + u < seg.tb; ++u) {
                        attn_step<FMT, NB, MODE, ATTN_EDGE>(st, x, powers, qf, q_smem, begin, end, lane);
                        x.tile += Sh::TILE;
                        x.pos += KV_TILE;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[used]);
        }
        if (!poison && !dead && st.again()) {
            // once more, from the cache itself: the ring has gone on.  (Its tiles all had
            // their addresses checked by the copying warp; a page whose number has
            // changed meanwhile is no page.)
            st.clear();
            st.e = 0;
            powers.clear();
            const int tpp = a.L.tiles();
#pragma unroll 1
            for (int tl = seg.ta; tl < seg.tb; ++tl) {
                const int tile = seg.first + tl, n = tile / tpp;
                const int64_t off = a.L.tile_offset(a.table[seg.b * a.ld_table + n], kvh, tile - n * tpp);
                if (off < 0 || !QG_OK(qg_in(off, Sh::TILE, a.L.bytes()), status, 732)) {
                    poison = true;
                    break;
                }
                const AttnStep x{a.cache + off, tile * KV_TILE, sp.first(), sp.last()};
                attn_step<FMT, NB, MODE, ATTN_AGAIN>(st, x, powers, qf, q_smem, begin, end, lane);
            }
            if constexpr (FMT != QGEMV_KV_F16) {  // as if with one power, 2^25
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int b = 0; b < NB; ++b) st.scale(r, b, 0x1p25f * attn_inverse(powers.of(r, b)));
            }
        }
        st.finish(poison || dead);

        if (seg.ta == 0 && seg.tb == seg.count) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        float v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int at = Sh::place(b, h, r, k);
                            v[k] = st.o[at / (4 * Sh::NC)][at / Sh::NC % 4][at % Sh::NC];
                        }
                        attn_emit<FMT, NB, MODE, T>(a, p, o_wide, seg.b, seg.item, wrow, b, h, r, lane, v, st.m[r], st.l[r]);
                    }
        } else {
            // an item that goes on after this piece is the last of it; one that began before, the first
            float* to = attn_part(a, p, split_id, seg.ta == 0, wrow, Sh::PART) + lane;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int c = 0; c < Sh::NC; ++c) __stcg(to + ((b * 4 + n) * Sh::NC + c) * 32, st.o[b][n][c]);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                __stcg(to + (Sh::NO + r) * 32, st.m[r]);
                __stcg(to + (Sh::NO + NR + r) * 32, st.l[r]);
            }
            if (seg.ta == 0) {
                const int last = cut.split_of(p, seg.line + ATTN_ITEM_COST + seg.count - 1);
                record = AttnRecord::of(last - split_id + 1, seg.b, seg.item);
            }
        }
    }
    if (wrow == 0 && lane == 0) a.records[split_id] = record;
    if (dead && lane == 0) atomicAdd_system(status, 1u);
}

// The items that splits share: out of their partial results, in the order of
// the splits.  A job is a run of eight values of a row of an item, or half of it: a warp's
// lanes hold its rows and columns as the splits' lanes did.  `per` warps of a
// CTA take a job's partial results in turn.
template <int FMT, int NB, int MODE, typename T>
__global__ void __launch_bounds__(ATTN_JOIN_WARPS * 32) attn_join_kernel(const AttnArgs a, const AttnPlan p)
{
    using Sh = AttnShape<FMT, NB, MODE>;
    constexpr int NR = Sh::NR;
    __shared__ int s_split[ATTN_MAX_SPLITS], s_items;
    __shared__ AttnRecord s_rec[ATTN_MAX_SPLITS];
    __shared__ uint32_t s_has[ATTN_MAX_SPLITS / 32];
    __shared__ float s_sum[ATTN_JOIN_WARPS][10][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();
    // the splits with a record, in order (the same for every CTA)
    constexpr int WORDS = ATTN_MAX_SPLITS / 32;
    AttnRecord got[WORDS / ATTN_JOIN_WARPS];
#pragma unroll
    for (int j = 0; j < WORDS / ATTN_JOIN_WARPS; ++j) {  // (all on the way at once)
        const int i = (j * ATTN_JOIN_WARPS + warp) * 32 + lane;
        got[j] = i < p.splits ? a.records[i] : AttnRecord{0};
    }
#pragma unroll
    for (int j = 0; j < WORDS / ATTN_JOIN_WARPS; ++j) {
        const int w = j * ATTN_JOIN_WARPS + warp;
        s_rec[w * 32 + lane] = got[j];
        const uint32_t has = __ballot_sync(0xffffffffu, got[j].parts() > 0);
        if (lane == 0) s_has[w] = has;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < WORDS / ATTN_JOIN_WARPS; ++j) {
        const int w = j * ATTN_JOIN_WARPS + warp;
        int before = 0;
#pragma unroll
        for (int k = 0; k < WORDS; k += 32) before += k + lane < w ? __popc(s_has[k + lane]) : 0;
        before = __reduce_add_sync(0xffffffffu, before);
        const uint32_t has = s_has[w];
        if (has >> lane & 1) s_split[before + __popc(has & ((1u << lane) - 1))] = w * 32 + lane;
        if (w == WORDS - 1 && lane == 0) s_items = before + __popc(has);
    }
    __syncthreads();
    // one job a run where that fills the GPU, else one a half of it
    const int halves = s_items * p.wr * Sh::RUNS * 2 > (int)gridDim.x * ATTN_JOIN_WARPS ? 1 : 2;
    const int in_item = p.wr * Sh::RUNS * halves, jobs = s_items * in_item;
    int per = ATTN_JOIN_WARPS;
    while (per > 1 && jobs * per > (int)gridDim.x * ATTN_JOIN_WARPS) per >>= 1;
    const int at_once = ATTN_JOIN_WARPS / per, part0 = warp % per;
    const bool o_wide = KvRows{a.out, a.o_row, a.o_head}.wide<T>();
    for (int base = blockIdx.x * at_once; base < jobs; base += gridDim.x * at_once) {
        const int job = base + warp / per;
        const int run = job % in_item / halves, tile = run / Sh::RUNS, r = run % NR, b = run % Sh::RUNS / NR;
        const int h = halves == 2 ? job & 1 : 0;  // of the run, its first half or all
        float m = -INFINITY, l = 0.0f, v[8] = {};
        AttnRecord rec{0};
        if (job < jobs) {
            const int s0 = s_split[job / in_item];
            rec = s_rec[s0];
            // (two loops, so that the loads of four partial results go together)
            auto gather = [&](auto whole) {
#pragma unroll 4
                for (int i = part0; i < rec.parts(); i += per) {
                    const float* from = attn_part(a, p, s0 + i, i == 0, tile, Sh::PART) + lane;
                    const float m2 = __ldcg(from + (Sh::NO + r) * 32), l2 = __ldcg(from + (Sh::NO + NR + r) * 32);
                    float x[whole ? 8 : 4];
#pragma unroll
                    for (int k = 0; k < (whole ? 8 : 4); ++k)
                        x[k] = __ldcg(from + Sh::place(b, whole ? k >> 2 : h, r, k & 3) * 32);
                    const float mn = fmaxf(m, m2), bs = attn_base(mn), f1 = ex2(m - bs), f2 = ex2(m2 - bs);
                    m = mn;
                    l = l * f1 + l2 * f2;
#pragma unroll
                    for (int k = 0; k < (whole ? 8 : 4); ++k) v[k] = v[k] * f1 + x[k] * f2;
                }
            };
            if (halves == 1) gather(std::true_type{});
            else gather(std::false_type{});
        }
        if (per > 1) {
            float(*mine)[32] = s_sum[warp];
            mine[0][lane] = m, mine[1][lane] = l;
#pragma unroll
            for (int k = 0; k < 8; ++k) mine[2 + k][lane] = v[k];
            __syncthreads();
            if (part0 == 0) {
                float top = m;
#pragma unroll 5
                for (int i = 1; i < per; ++i) top = fmaxf(top, s_sum[warp + i][0][lane]);
                const float bs = attn_base(top), f0 = ex2(m - bs);
                l *= f0;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= f0;
#pragma unroll 5
                for (int i = 1; i < per; ++i) {
                    const float f = ex2(s_sum[warp + i][0][lane] - bs);
                    l += s_sum[warp + i][1][lane] * f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] += s_sum[warp + i][2 + k][lane] * f;
                }
                m = top;
            }
            __syncthreads();
        }
        if (part0 == 0 && job < jobs) {
            const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
            attn_emit<FMT, NB, MODE, T>(a, p, o_wide, rec.b(), rec.item(), tile, b, h, r, lane, lo, m, l);
            if (halves == 1) attn_emit<FMT, NB, MODE, T>(a, p, o_wide, rec.b(), rec.item(), tile, b, 1, r, lane, hi, m, l);
        }
    }
}

template <int FMT, int NB, int MODE>
AttnPlan attn_plan(const DeviceInfo& di, int rows)
{
    using Sh = AttnShape<FMT, NB, MODE>;
    AttnPlan p{};
    p.magic = attn_magic(FMT);
    const int tiles = (rows + Sh::ROWS - 1) / Sh::ROWS;
    p.row_groups = (tiles + Sh::WARPS - 1) / Sh::WARPS;
    p.wr = (tiles + p.row_groups - 1) / p.row_groups;
    for (p.ws = Sh::WARPS / p.wr; p.ws > 0; --p.ws) {
        const uint32_t q = Sh::Q_SMEM ? (uint32_t)p.ws * p.wr * NB * 2 * Sh::Q_TERMS * 512 : 0;
        const uint32_t per_stage = (uint32_t)p.ws * (2 * Sh::TILE + 2 * 8 + 4);
        const uint32_t budget = (uint32_t)di.smem_optin - 2048;  // beside the static shared memory
        const int stages = budget > q ? (int)((budget - q) / per_stage) : 0;
        if (stages < 2 && p.ws > 1) continue;
        p.stages = stages > 3 ? 3 : stages;
        p.off_q = (uint32_t)p.ws * p.stages * 2 * Sh::TILE;
        p.off_bar = p.off_q + q;
        p.bytes = p.off_bar + (uint32_t)p.ws * p.stages * 20;
        break;
    }
    p.splits = (di.sms < ATTN_GRID ? di.sms : ATTN_GRID) * p.ws;
    // A warp that has its scheduler (warp number mod 4) to itself is faster; the
    // split whose warps all are gets more.
    int on[4] = {0, 0, 0, 0};
    for (int w = 0; w < p.ws * p.wr; ++w) ++on[w % 4];
    for (int s = 0; s < p.ws; ++s) {
        bool alone = true;
        for (int w = s * p.wr; w < (s + 1) * p.wr; ++w) alone = alone && on[w % 4] == 1;
        p.cum[s + 1] = p.cum[s] + (alone ? attn_share_alone(FMT, NB, rows) : ATTN_SHARE);
    }
    return p;
}

template <int FMT, int NB, int MODE, typename T>
int launch_attn(const AttnArgs& a, cudaStream_t s)
{
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return QGEMV_CUDA_ERROR;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return QGEMV_CUDA_ERROR;
    AttnPlan p = attn_plan<FMT, NB, MODE>(di, a.rows * a.group);
    if (p.stages < 2) return QGEMV_UNSUPPORTED_SHAPE;
    auto kern = attn_split_kernel<FMT, NB, MODE, T>;
    static std::once_flag once[64];
    static bool ok[64];
    std::call_once(once[dev], [&]() {
        ok[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, di.smem_optin - 2048) ==
                      cudaSuccess &&
                  wait_timeout_counter() != nullptr;
        if (!ok[dev]) cudaGetLastError();
    });
    if (!ok[dev]) return QGEMV_CUDA_ERROR;
    p.drop_copy = take_drop_request();
    if (launch_pdl(kern, dim3(p.splits / p.ws), dim3((p.ws * p.wr + 1) * 32), p.bytes, s, a, p, wait_timeout_counter()) !=
        cudaSuccess)
        return QGEMV_CUDA_ERROR;
    if (launch_pdl(attn_join_kernel<FMT, NB, MODE, T>, dim3(2 * di.sms), dim3(ATTN_JOIN_WARPS * 32), 0, s, a, p) != cudaSuccess)
        return QGEMV_CUDA_ERROR;
    return cudaGetLastError() == cudaSuccess ? QGEMV_OK : QGEMV_CUDA_ERROR;
}

template <int FMT, int MODE, typename T>
int launch_attn_dim(const AttnArgs& a, cudaStream_t s)
{
    switch (a.L.nb) {
    case 2: return launch_attn<FMT, 2, MODE, T>(a, s);
    case 3: return launch_attn<FMT, 3, MODE, T>(a, s);
    case 4: return launch_attn<FMT, 4, MODE, T>(a, s);
    default: return launch_attn<FMT, 8, MODE, T>(a, s);
    }
}

// One translation unit for each format and type.
template <int FMT, typename T>
int launch_attn_rows(const AttnArgs& a, cudaStream_t s)
{
    if (attn_mode(a.rows * a.group) == ATTN_PAIR) return launch_attn_dim<FMT, ATTN_PAIR, T>(a, s);
    return launch_attn_dim<FMT, ATTN_TWO, T>(a, s);
}

}  // namespace qgemv
