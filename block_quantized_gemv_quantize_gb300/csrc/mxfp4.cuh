// Microscaled 4-bit floating point (MXFP4) and the sparse layer's calls on it:
// formats, layouts and launch arguments (include/qgemv.h has the definitions).
#pragma once

#include <type_traits>

#include "kvcache.cuh"  // element types of rows

namespace qgemv {

constexpr int MX_BYTES = 17;        // a block: the scale byte, 16 bytes of codes
constexpr int MX_UNIT_K = 64;       // values of a row in one unit of the pack
constexpr int MX_TILE_N = 16;       // rows of a tile
constexpr int MX_UNIT_CODES = MX_TILE_N * MX_UNIT_K / 2;
constexpr int MX_UNIT_BYTES = MX_UNIT_CODES + MX_TILE_N * MX_UNIT_K / 32;  // codes, scale bytes
constexpr int MX_NEAR = 27;  // how far (in powers of two) a block's scale may be below its row's largest
constexpr int MX_MAX_K = 1 << 15, MX_MAX_N = 1 << 24, MX_MAX_EXPERTS = 1024, MX_MAX_TOP_K = 32;

// The pack: [expert][tile of 16 rows], a tile being
//   units  [K / 64][544 B], the last one filled up with zeros.  512 bytes of
//          codes, 16 for each lane 4 g + t of a warp: four words, of row g in
//          the unit's first block, row g + 8 there, row g in its second block,
//          row g + 8 there.  A word has the block's values 4 t .. 4 t + 3 and
//          16 + 4 t .. 16 + 4 t + 3, a nibble each in that order.  Then 32
//          scale bytes [g][4] in the order of a lane's words: 127 - l for a block
//          whose scale is 2^-l of the row's largest (l = 0 for a block of zeros), the
//          block's own byte in a row marked by 255
//   tops   [16] bytes: the row's largest scale byte among blocks that are not all
//          zeros; 255 for a row that holds a NaN block, or one that is farther than
//          2^-27 (MX_NEAR) below the largest: no half holds its values beside those
// A lane's 16 bytes are its operands of four m16n8k16 products, if the K index
// runs through a block in the order in which the words have it; and its pairs
// are the fragments of a 16 x 256-bit store to tensor memory with K in its own
// order.
struct MxLayout {
    int experts, N, K;
    __host__ __device__ int tiles() const { return (N + MX_TILE_N - 1) / MX_TILE_N; }
    __host__ __device__ int units() const { return (K + MX_UNIT_K - 1) / MX_UNIT_K; }
    __host__ __device__ int64_t tile_bytes() const { return (int64_t)units() * MX_UNIT_BYTES + MX_TILE_N; }
    __host__ __device__ int64_t expert_bytes() const { return tiles() * tile_bytes(); }
    __host__ __device__ int64_t bytes() const { return experts * expert_bytes(); }
};

// The value of scale byte e (255: NaN).  2^-127 is subnormal.
__device__ __forceinline__ float mx_scale(int e)
{
    return __uint_as_float(e == 0 ? 0x00400000u : (e == 255 ? 0x7FC00000u : (uint32_t)e << 23));
}

// v * 2^p in one rounding (p: -378 .. 380): factors that are fp32 numbers, the least of
// them first.  Where the product is 2^-150 or more, all before the last are exact;
// one that leaves the range does so as the exact one would.
__device__ __forceinline__ float mul_pow2(float v, int p)
{
    const int a = max(-126, min(127, p)), r = p - a, b = max(-126, min(127, r)), c = r - b;
    if (c) v *= __uint_as_float((uint32_t)(c + 127) << 23);
    return v * __uint_as_float((uint32_t)(b + 127) << 23) * __uint_as_float((uint32_t)(a + 127) << 23);
}

// ---- rows of values -------------------------------------------------------------

// Sixteen bytes that are read once.  (Not by the read-only path: under programmatic
// launch an earlier kernel may have been writing them when this one started.)
__device__ __forceinline__ uint4 load_once(const void* p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// Eight values as they lie in memory.
template <typename T>
struct Raw {
    uint32_t w[2 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, bool wide)
{
    Raw<T> r;
    if (wide) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            const uint4 v = load_once(reinterpret_cast<const uint4*>(p) + i);
            r.w[4 * i] = v.x;
            r.w[4 * i + 1] = v.y;
            r.w[4 * i + 2] = v.z;
            r.w[4 * i + 3] = v.w;
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(p[i]);
    } else {
        const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = (uint32_t)u[2 * i] | (uint32_t)u[2 * i + 1] << 16;
    }
    return r;
}

// Four values, of which the first sits in w[0].
template <typename T>
__device__ __forceinline__ void values4(const uint32_t* w, float (&v)[4])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(w + i));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

int launch_quantize_mxfp4(int type, const void* x, int64_t ldx, void* blocks, int64_t N, int K, cudaStream_t s);
int launch_dequantize_mxfp4(int type, const void* blocks, void* y, int64_t ldy, int64_t N, int K, cudaStream_t s);
int launch_qpack_mxfp4(const void* canon, void* pack, const MxLayout& L, cudaStream_t s);

// ---- router -------------------------------------------------------------------

struct RouteArgs {
    const void* logits;  // null: the ids are given
    int64_t ld;
    int32_t* ids;
    float* weights;
    int32_t* offsets;
    int32_t* order;
    int32_t* counts;  // workspace [MAX_RANGES + 1][experts + 1]
    unsigned int* status;  // of the bounds-checking build
    int tokens, experts, top_k;
    bool sigmoid, renormalize;
    float scale;
};

size_t route_workspace_bytes(int tokens, int experts);
int launch_route(int type, const RouteArgs& a, cudaStream_t s);

// ---- the experts' products ------------------------------------------------------

enum MxMode { MX_GEMM = 0, MX_GATE_UP = 1, MX_DOWN = 2 };

struct MxArgs {
    const uint8_t* w;   // the pack (gate's)
    const uint8_t* w2;  // up's
    MxLayout L;
    const void* x;
    int64_t ldx, ldy;
    const int32_t* offsets;
    const int32_t* order;  // null: slot i is row i
    int slots, top_k;      // x's row of slot s is s / x_div
    int x_div;
    void* y;               // gemm, gate_up: [slots]; down: fp32 partial results [place][N]
    int32_t* place_of;     // down, [slots]: a slot's place (its row of the partial results), -1 for none; of a slot that order does not name: anything
    void* planes;          // workspace for rows of x as halves (mx_planes_bytes)
};

// Whether a call takes the tcgen05 kernel: its experts have many rows each, about (or
// rows of x that are too long for the other's shared memory).
bool mx_many_rows(int64_t slots, int experts, int K);
// Workspace of that kernel: rows of x as halves, and their powers of two.
size_t mx_planes_bytes(int type, int64_t rows, int K);

int launch_mx_gemm(int mode, int type, const MxArgs& a, cudaStream_t s);
int launch_mx_combine(int type, const float* parts, const int32_t* place_of, const int32_t* order, const float* weights,
                      void* out, int64_t ldo, int tokens, int top_k, int N, cudaStream_t s);

}  // namespace qgemv
