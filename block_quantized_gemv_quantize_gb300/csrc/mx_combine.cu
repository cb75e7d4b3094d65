// The last step of the down product: out[t] = sum_j weight[t][j] part[place of
// slot t k + j], in the order of j, in fp32.  A slot's place is written where the order names
// the slot; of one that it does not name the workspace holds anything, so a place counts
// only if the order has the slot there.  Reads the partial results once; bound by
// them (HBM, or L2 where they are few): 4096 tokens x 6 x 5120, 503 MB, 80 us.
#include "mxfp4.cuh"

namespace qgemv {
namespace {

constexpr int THREADS = 256;

// Four outputs of one token a thread, TERMS of the sum in flight.  (Eight where a thread has one
// quad: 96 tokens x 8 x 2048, product and sum, 43.3 us by eight and 44.6 by two; two beyond: 4096
// tokens x 6 x 5120 384 us and 452 by eight, whose registers leave fewer threads.)
template <typename T, int TERMS>
__global__ void __launch_bounds__(THREADS) combine_kernel(const float* parts, const int32_t* place_of,
                                                          const int32_t* order, const float* weights, T* out, int64_t ldo, int tokens,
                                                          int top_k, int N, int quads, bool wide, unsigned int* status)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t all = (int64_t)tokens * quads;
    const int slots = tokens * top_k;
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < all; i += (int64_t)gridDim.x * THREADS) {
        const int t = (int)(i / quads), n = (int)(i - (int64_t)t * quads) * 4;
        const float* w = weights + (int64_t)t * top_k;
        const int32_t* places = place_of + (int64_t)t * top_k;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (!QG_OK(qg_in(t * ldo + n, 1, tokens * ldo), status, 320)) continue;
#pragma unroll TERMS
        for (int j = 0; j < top_k; ++j) {
            const int s = t * top_k + j, place = places[j];
            const int at = place < 0 || place >= slots ? 0 : place;  // (loads that wait for no other: place 0 is there)
            const int named = order ? order[at] : at;
            const float f = w[j];
            const float* p = parts + (int64_t)at * N + n;
            float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (N % 4 == 0) {
                const float4 r = *reinterpret_cast<const float4*>(p);
                q[0] = r.x, q[1] = r.y, q[2] = r.z, q[3] = r.w;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (n + k < N) q[k] = p[k];
            }
            if (at == place && named == s)  // (not a slot without an expert)
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = fmaf(f, q[k], v[k]);
        }
        T* o = out + t * ldo + n;
        if (wide) {
            alignas(16) T r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = from_f32<T>(v[k]);
            if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(o) = *reinterpret_cast<uint4*>(r);
            else *reinterpret_cast<uint2*>(o) = *reinterpret_cast<uint2*>(r);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (n + k < N) o[k] = from_f32<T>(v[k]);
        }
    }
}

template <typename T>
int combine_t(const float* parts, const int32_t* place_of, const int32_t* order, const float* weights, void* out, int64_t ldo, int tokens, int top_k,
              int N, cudaStream_t s)
{
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return QGEMV_CUDA_ERROR;
    const int quads = (N + 3) / 4;
    const int64_t ctas = ((int64_t)tokens * quads + THREADS - 1) / THREADS;
    const bool wide = N % 4 == 0 && ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(ldo * (int64_t)sizeof(T))) &
                                     (4 * sizeof(T) - 1)) == 0;
    return launch_pdl(ctas <= di.sms * 8 ? combine_kernel<T, 8> : combine_kernel<T, 2>,
                      dim3((unsigned)(ctas < di.sms * 8 ? ctas : di.sms * 8)), dim3(THREADS), 0, s,
                      parts, place_of, order, weights, static_cast<T*>(out), ldo, tokens, top_k, N, quads, wide,
                      wait_timeout_counter()) == cudaSuccess
               ? QGEMV_OK
               : QGEMV_CUDA_ERROR;
}

}  // namespace

int launch_mx_combine(int type, const float* parts, const int32_t* place_of, const int32_t* order, const float* weights,
                      void* out, int64_t ldo, int tokens, int top_k, int N, cudaStream_t s)
{
    if (type == QGEMV_F32) return combine_t<float>(parts, place_of, order, weights, out, ldo, tokens, top_k, N, s);
    if (type == QGEMV_F16) return combine_t<__half>(parts, place_of, order, weights, out, ldo, tokens, top_k, N, s);
    return combine_t<__nv_bfloat16>(parts, place_of, order, weights, out, ldo, tokens, top_k, N, s);
}

// From 8 rows an expert on (of those that can have any: how the slots fall the host does not know).
// By the mma.sync kernel and by this one, bf16 rows if not said otherwise: 64 experts of 1408 x 5120, gate
// and up, 8 rows each 112 and 132 us, 12 rows 183 and 126 (a second row tile reads the weights again); one of
// 17408 x 5120, 4 rows 17.5 and 21.8, 8 rows 22.7 and 22.0 (fp32 33.4 and 27.0), 9 rows 32 and 22; one of 4096 x
// 4096, 8 rows 13.0 and 15.0 (fp32 15.0 and 17.6), 9 rows 16 and 15.  512 slots all of one expert of 64 take 95 us,
// less than the even ones, where this one would take 24.
bool mx_many_rows(int64_t slots, int experts, int K)
{
    return slots > 8 * (slots < experts ? slots : (int64_t)experts) || K > 16384;
}

size_t mx_planes_bytes(int type, int64_t rows, int K)
{
    const size_t halves = (size_t)((K + MX_UNIT_K - 1) / MX_UNIT_K) * MX_UNIT_K * (type == QGEMV_F32 ? 2 : 1);
    return (size_t)rows * (halves * 2 + sizeof(float));
}

int launch_mx_gemm_f32(int mode, const MxArgs& a, cudaStream_t s);
int launch_mx_gemm_f16(int mode, const MxArgs& a, cudaStream_t s);
int launch_mx_gemm_bf16(int mode, const MxArgs& a, cudaStream_t s);

int launch_mx_gemm(int mode, int type, const MxArgs& a, cudaStream_t s)
{
    if (type == QGEMV_F32) return launch_mx_gemm_f32(mode, a, s);
    if (type == QGEMV_F16) return launch_mx_gemm_f16(mode, a, s);
    return launch_mx_gemm_bf16(mode, a, s);
}

}  // namespace qgemv
