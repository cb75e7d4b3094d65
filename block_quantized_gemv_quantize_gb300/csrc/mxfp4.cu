// MXFP4: quantizer, its inverse, and the repacker of weights.
#include "mxfp4.cuh"

namespace qgemv {
namespace {

constexpr int THREADS = 256;
constexpr int QUANTIZE_CTAS = 5;            // an SM
constexpr int RUN = 32;                     // blocks that a warp takes at a time
constexpr int RUN_BYTES = RUN * MX_BYTES;   // 544, a multiple of 16: runs of the output stay aligned

// A warp's run of blocks: 4 lanes a block, 8 blocks a step, 4 steps.  Lane
// `sub` of a block has its values 8 sub .. 8 sub + 7.
struct RunAt {
    int64_t row;
    int col;  // block of the row
    int nb;
    __device__ void next()
    {
        col += 8;
        while (col >= nb) {
            col -= nb;
            ++row;
        }
    }
};

__device__ __forceinline__ RunAt run_at(uint32_t block, int nb)
{
    const uint32_t row = block / (uint32_t)nb;
    return {row, (int)(block - row * (uint32_t)nb), nb};
}

// Four bytes of two codes each, lo[i] in the low nibble: nearest, of two equally near the
// even one, at most 6 in magnitude (what the format asks for).
__device__ __forceinline__ uint32_t e2m1_bytes(const float (&lo)[4], const float (&hi)[4])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %5, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %6, %2;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %7, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %4;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(lo[0]), "f"(lo[1]), "f"(lo[2]), "f"(lo[3]), "f"(hi[0]), "f"(hi[1]), "f"(hi[2]), "f"(hi[3]));
    return r;
}

// The largest magnitude's fp32 bits.  (Magnitudes order like their bits; NaN and infinity come last.)
template <typename T>
__device__ __forceinline__ uint32_t top_bits(const Raw<T>& r)
{
    if constexpr (sizeof(T) == 4) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, r.w[i] & 0x7FFFFFFFu);
        return top;
    } else {
        uint32_t m = r.w[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __vmaxu2(m, r.w[i] & 0x7FFF7FFFu);
        const uint32_t top = max(m & 0xFFFFu, m >> 16);
        if constexpr (std::is_same<T, __nv_bfloat16>::value) return top << 16;
        else return __float_as_uint(__half2float(__ushort_as_half((unsigned short)top)));
    }
}

// One pass over the data: reads 32 s bytes (s: bytes of an element), writes 17 a block.  The
// scale is an exponent, so both the quotient and the code are exact but for the
// code's own rounding.  Bound by instructions next to HBM (2.9 issued a clock): 163840 x
// 1408 bf16 values in and back 220 us, 5.3 TB/s; with the codes put together from
// nibbles of two lanes, and a second wave of CTAs, 272.
template <typename T>
__global__ void __launch_bounds__(THREADS, QUANTIZE_CTAS) quantize_kernel(const T* x, int64_t ldx, uint8_t* out,
                                                           uint32_t blocks, int nb, bool wide, int64_t rows,
                                                           unsigned int* status)
{
    __shared__ __align__(16) uint8_t buf[THREADS / 32][RUN_BYTES];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 3;
    uint8_t* mine = buf[warp];
    const uint32_t runs = (blocks + RUN - 1) / RUN;
    for (uint32_t run = blockIdx.x * (THREADS / 32) + warp; run < runs; run += gridDim.x * (THREADS / 32)) {
        const uint32_t first = run * RUN;
        RunAt at = run_at(first + (lane >> 2), nb);
        Raw<T> v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (first + 8 * i + (lane >> 2) < blocks &&
                QG_OK(at.row < rows && qg_in((int64_t)at.col * 32 + sub * 8, 8, (int64_t)nb * 32), status, 300))
                v[i] = load_raw(x + at.row * ldx + (int64_t)at.col * 32 + sub * 8, wide);
            else
                v[i] = Raw<T>{};
            at.next();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t top = top_bits<T>(v[i]);
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            const bool fine = top < 0x7F800000u;
            const int e = fine ? max(0, (int)(top >> 23) - 2) : 255;
            const float f = __uint_as_float((uint32_t)(254 - min(e, 253)) << 23);  // 2^(127 - e)
            // lane sub < 2 has values 8 sub .., lane sub + 2 those 16 further on, which share
            // bytes 8 sub ..: each takes four of them, the first two words of both or the last
            constexpr int H = sizeof(T);  // words of four values
            uint32_t lo[H], hi[H];
#pragma unroll
            for (int k = 0; k < H; ++k) {
                const uint32_t other = __shfl_xor_sync(~0u, sub < 2 ? v[i].w[H + k] : v[i].w[k], 2);
                lo[k] = sub < 2 ? v[i].w[k] : other;
                hi[k] = sub < 2 ? other : v[i].w[H + k];
            }
            float a[4], c[4];
            values4<T>(lo, a);
            values4<T>(hi, c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                a[k] *= f;
                c[k] *= f;
            }
            const uint32_t bytes = fine ? e2m1_bytes(a, c) : 0u;
            uint8_t* b = mine + (8 * i + (lane >> 2)) * MX_BYTES;
            if (sub == 0) b[0] = (uint8_t)e;
            b += 1 + 8 * (sub & 1) + 4 * (sub >> 1);
#pragma unroll
            for (int k = 0; k < 4; ++k) b[k] = (uint8_t)(bytes >> (8 * k));
        }
        __syncwarp();
        uint8_t* to = out + (int64_t)first * MX_BYTES;
        if (first + RUN <= blocks) {
            for (int i = lane; i < RUN_BYTES / 16; i += 32) reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<uint4*>(mine)[i];
        } else {
            for (int i = lane; i < (int)(blocks - first) * MX_BYTES; i += 32) to[i] = mine[i];
        }
        __syncwarp();
    }
}

// The eight codes of nibble half `high` of eight bytes as fp32 values.
__device__ __forceinline__ void e2m1_values(uint2 bytes, bool high, float (&v)[8])
{
    const uint32_t w[2] = {(high ? bytes.x >> 4 : bytes.x) & 0x0F0F0F0Fu, (high ? bytes.y >> 4 : bytes.y) & 0x0F0F0F0Fu};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t p = w[i] | w[i] >> 4;  // bytes 0 and 2: two codes each
        uint32_t a, b;
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b2;\n\t}"
            : "=r"(a), "=r"(b)
            : "r"(p));
        const float2 f = __half22float2(*reinterpret_cast<__half2*>(&a)), g = __half22float2(*reinterpret_cast<__half2*>(&b));
        v[4 * i] = f.x;
        v[4 * i + 1] = f.y;
        v[4 * i + 2] = g.x;
        v[4 * i + 3] = g.y;
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 8) dequantize_kernel(const uint8_t* in, T* y, int64_t ldy,
                                                             uint32_t blocks, int nb, bool wide, int64_t rows,
                                                             unsigned int* status)
{
    __shared__ __align__(16) uint8_t buf[THREADS / 32][RUN_BYTES + 16];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 3;
    uint8_t* mine = buf[warp];
    const uint32_t runs = (blocks + RUN - 1) / RUN;
    for (uint32_t run = blockIdx.x * (THREADS / 32) + warp; run < runs; run += gridDim.x * (THREADS / 32)) {
        const uint32_t first = run * RUN;
        const uint8_t* from = in + (int64_t)first * MX_BYTES;
        if (first + RUN <= blocks) {
            for (int i = lane; i < RUN_BYTES / 16; i += 32)
                reinterpret_cast<uint4*>(mine)[i] = load_once(reinterpret_cast<const uint4*>(from) + i);
        } else {
            for (int i = lane; i < (int)(blocks - first) * MX_BYTES; i += 32) mine[i] = from[i];
        }
        __syncwarp();
        RunAt at = run_at(first + (lane >> 2), nb);
#pragma unroll
        for (int i = 0; i < 4; ++i, at.next()) {
            const int b = 8 * i + (lane >> 2);
            if (first + b < blocks) {
                const int o = b * MX_BYTES + 1 + 8 * (sub & 1);
                const uint32_t* w = reinterpret_cast<const uint32_t*>(mine) + (o >> 2);
                const int shift = 8 * (o & 3);
                const uint2 bytes = make_uint2(__funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift));
                const float scale = mx_scale(mine[b * MX_BYTES]);
                float v[8];
                e2m1_values(bytes, sub >= 2, v);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= scale;
                if (QG_OK(at.row < rows && qg_in((int64_t)at.col * 32 + sub * 8, 8, (int64_t)nb * 32), status, 301))
                    store_values<8>(y + at.row * ldy + (int64_t)at.col * 32 + sub * 8, wide, v);
            }
        }
        __syncwarp();
    }
}

// One CTA a tile: the rows' largest scales (of blocks that are not all zeros), then the units, a warp a unit.
__global__ void __launch_bounds__(128) pack_kernel(const uint8_t* canon, uint8_t* pack, MxLayout L,
                                                   int64_t tiles, unsigned int* status)
{
    __shared__ int tops[MX_TILE_N];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nb = L.K / 32;
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int expert = (int)(tile / L.tiles()), n0 = (int)(tile % L.tiles()) * MX_TILE_N;
        const uint8_t* rows = canon + ((int64_t)expert * L.N + n0) * nb * MX_BYTES;
        uint8_t* to = pack + tile * L.tile_bytes();
        {
            const int r = threadIdx.x / 8;
            int top = 0, least = 255;
            for (int b = threadIdx.x & 7; b < nb && n0 + r < L.N; b += 8) {
                const uint8_t* block = rows + ((int64_t)r * nb + b) * MX_BYTES;
                const int e = block[0];
                if (e <= top && e >= least) continue;
                uint32_t any = e == 255;  // (NaN, whatever the codes)
#pragma unroll
                for (int k = 1; k <= 16; ++k) any |= block[k] & 0x77u;
                if (any) top = max(top, e), least = min(least, e);  // (a block of zeros has no scale to keep)
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                top = max(top, __shfl_xor_sync(~0u, top, o));
                least = min(least, __shfl_xor_sync(~0u, least, o));
            }
            if ((threadIdx.x & 7) == 0) tops[r] = top - least > MX_NEAR ? 255 : top;
        }
        __syncthreads();
        const int g = lane >> 2, t = lane & 3;
        for (int u = warp; u < L.units(); u += 4) {
            uint32_t word[4], live = 0;  // bit j: block j is not all zeros
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = g + 8 * (j & 1), b = 2 * u + (j >> 1);
                word[j] = 0;
                const uint8_t* block = rows + ((int64_t)r * nb + b) * MX_BYTES;
                if (n0 + r < L.N && b < nb) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)  // value 4 t + k % 4 of the block's half k / 4
                        word[j] |= (uint32_t)((block[1 + 4 * t + (k & 3)] >> (k < 4 ? 0 : 4)) & 15u) << (4 * k);
                }
                if (word[j] & 0x77777777u) live |= 1u << j;
            }
            live |= __shfl_xor_sync(~0u, live, 1);
            live |= __shfl_xor_sync(~0u, live, 2);
            // this lane's scale: block t's
            const int r = g + 8 * (t & 1), b = 2 * u + (t >> 1);
            const int own = n0 + r < L.N && b < nb ? rows[((int64_t)r * nb + b) * MX_BYTES] : 0;
            const int scale = tops[r] == 255 ? own : 127 - (live >> t & 1u ? tops[r] - own : 0);
            uint8_t* unit = to + (int64_t)u * MX_UNIT_BYTES;
            if (QG_OK(qg_in(unit - pack, MX_UNIT_BYTES, L.bytes()), status, 302)) {
                reinterpret_cast<uint4*>(unit)[lane] = make_uint4(word[0], word[1], word[2], word[3]);
                unit[MX_UNIT_CODES + lane] = (uint8_t)scale;
            }
        }
        if (threadIdx.x < MX_TILE_N) to[(int64_t)L.units() * MX_UNIT_BYTES + threadIdx.x] = (uint8_t)tops[threadIdx.x];
        __syncthreads();
    }
}

template <typename T>
bool rows_wide(const void* p, int64_t ld)
{
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * (int64_t)sizeof(T))) & 15u) == 0;
}

// (as many CTAs an SM as are there at once: a second wave would end half empty)
unsigned run_grid(const DeviceInfo& di, int64_t blocks, int ctas)
{
    const int64_t per_cta = THREADS / 32 * RUN, grid = (blocks + per_cta - 1) / per_cta;
    return (unsigned)(grid < (int64_t)di.sms * ctas ? grid : (int64_t)di.sms * ctas);
}

template <typename T>
int quantize_t(const void* x, int64_t ldx, void* blocks, int64_t N, int K, cudaStream_t s)
{
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return QGEMV_CUDA_ERROR;
    const int nb = K / 32;
    return launch_pdl(quantize_kernel<T>, dim3(run_grid(di, N * nb, QUANTIZE_CTAS)), dim3(THREADS), 0, s, static_cast<const T*>(x), ldx,
                      static_cast<uint8_t*>(blocks), (uint32_t)(N * nb), nb, rows_wide<T>(x, ldx), N,
                      wait_timeout_counter()) == cudaSuccess
               ? QGEMV_OK
               : QGEMV_CUDA_ERROR;
}

template <typename T>
int dequantize_t(const void* blocks, void* y, int64_t ldy, int64_t N, int K, cudaStream_t s)
{
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return QGEMV_CUDA_ERROR;
    const int nb = K / 32;
    return launch_pdl(dequantize_kernel<T>, dim3(run_grid(di, N * nb, 8)), dim3(THREADS), 0, s,
                      static_cast<const uint8_t*>(blocks), static_cast<T*>(y), ldy, (uint32_t)(N * nb), nb,
                      rows_wide<T>(y, ldy), N, wait_timeout_counter()) == cudaSuccess
               ? QGEMV_OK
               : QGEMV_CUDA_ERROR;
}

}  // namespace

int launch_quantize_mxfp4(int type, const void* x, int64_t ldx, void* blocks, int64_t N, int K, cudaStream_t s)
{
    if (type == QGEMV_F32) return quantize_t<float>(x, ldx, blocks, N, K, s);
    if (type == QGEMV_F16) return quantize_t<__half>(x, ldx, blocks, N, K, s);
    return quantize_t<__nv_bfloat16>(x, ldx, blocks, N, K, s);
}

int launch_dequantize_mxfp4(int type, const void* blocks, void* y, int64_t ldy, int64_t N, int K, cudaStream_t s)
{
    if (type == QGEMV_F32) return dequantize_t<float>(blocks, y, ldy, N, K, s);
    if (type == QGEMV_F16) return dequantize_t<__half>(blocks, y, ldy, N, K, s);
    return dequantize_t<__nv_bfloat16>(blocks, y, ldy, N, K, s);
}

int launch_qpack_mxfp4(const void* canon, void* pack, const MxLayout& L, cudaStream_t s)
{
    const int64_t tiles = (int64_t)L.experts * L.tiles();
    return launch_pdl(pack_kernel, dim3((unsigned)(tiles < 65535 ? tiles : 65535)), dim3(128), 0, s,
                      static_cast<const uint8_t*>(canon), static_cast<uint8_t*>(pack), L, tiles,
                      wait_timeout_counter()) == cudaSuccess
               ? QGEMV_OK
               : QGEMV_CUDA_ERROR;
}

}  // namespace qgemv
