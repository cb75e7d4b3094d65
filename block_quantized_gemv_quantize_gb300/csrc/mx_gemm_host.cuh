// Launch plans of the experts' products.
#pragma once

#include "mx_gemm_tc.cuh"

#include <algorithm>
#include <mutex>

namespace qgemv {

// Rows a tile, warps a tile's K, CTAs.
template <typename T, int MODE>
bool mxs_plan(const DeviceInfo& di, const MxArgs& a, MxsPlan& p)
{
    constexpr int TERMS = MX_TERMS<T>;
    const int units = a.L.units();
    p.x_bytes = units * MX_UNIT_K * 2 + 64;  // (neighbouring rows half of the banks apart)
    const size_t fixed = (size_t)MXS_WARPS * MXS_STAGES * 2 * MX_UNIT_BYTES + MXS_WARPS * 2 * MXS_ROWS * MXS_RED * sizeof(float) +
                         (size_t)(2 * (a.L.experts + 1) + 32 + 3 * MXS_ROWS) * sizeof(int);
    const size_t row = (size_t)TERMS * p.x_bytes;
    const int want = std::max(1, std::min(MXS_ROWS, a.slots));
    const int fit = (size_t)di.smem_optin > fixed ? (int)(((size_t)di.smem_optin - fixed) / row) : 0;
    if (fit < 1) return false;
    p.rows = std::min(want, fit);
    p.smem = fixed + row * p.rows;
    // Warps that share a pair of tiles: 8 to 20 units each keep the ring and the
    // sum over the warps in proportion, more warps where a CTA has too few pairs.  (64 experts, a row
    // each: gate and up of 1408 x 5120 with 2, 4, 8 warps 95, 89, 95 us, down of
    // 5120 x 1408 57, 60, 76; a token of 6 experts, gate and up 26, 20, 19.5.)
    const int pairs = MODE == MX_GATE_UP ? a.L.tiles() : (a.L.tiles() + 1) / 2;
    const int64_t all = pairs * std::min<int64_t>(a.L.experts, a.slots);
    p.parts = units >= 32 ? 4 : units >= 12 ? 2 : 1;
    while (p.parts < MXS_WARPS && all * p.parts < (int64_t)di.sms * MXS_WARPS && units >= p.parts * 6) p.parts *= 2;
    const int64_t most = (int64_t)pairs * std::min<int64_t>(a.slots, (int64_t)a.slots / p.rows + a.L.experts);
    p.grid = (int)std::min<int64_t>(most, di.sms);
    return true;
}

template <typename T, int MODE>
int launch_mxs(const MxArgs& a, cudaStream_t s)
{
    const DeviceInfo di = device_info();
    int dev = 0;
    if (di.sms <= 0 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return QGEMV_CUDA_ERROR;
    MxsPlan p;
    if (!mxs_plan<T, MODE>(di, a, p)) return QGEMV_UNSUPPORTED_SHAPE;
    auto kern = mxs_kernel<T, MODE>;
    static std::once_flag once[64];
    static bool ok[64];
    std::call_once(once[dev], [&]() {
        ok[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, di.smem_optin) == cudaSuccess;
        if (!ok[dev]) cudaGetLastError();
    });
    if (!ok[dev]) return QGEMV_CUDA_ERROR;
    return launch_pdl(kern, dim3((unsigned)p.grid), dim3(MXS_THREADS), p.smem, s, a, p, wait_timeout_counter()) == cudaSuccess
               ? QGEMV_OK
               : QGEMV_CUDA_ERROR;
}

template <typename T, int MODE>
int launch_mxt(const MxArgs& a, cudaStream_t s)
{
    const DeviceInfo di = device_info();
    int dev = 0;
    if (di.sms <= 0 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return QGEMV_CUDA_ERROR;
    auto kern = mxt_kernel<T, MODE>;
    static std::once_flag once[64];
    static bool ok[64];
    static unsigned int* timeouts[64];
    std::call_once(once[dev], [&]() {
        timeouts[dev] = wait_timeout_counter();
        ok[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, di.smem_optin) == cudaSuccess &&
                  timeouts[dev] != nullptr;
        if (!ok[dev]) cudaGetLastError();
    });
    if (!ok[dev]) return QGEMV_CUDA_ERROR;
    // x itself where its rows are halves and aligned, halves in the workspace otherwise
    constexpr int TERMS = MX_TERMS<T>;
    constexpr bool HALVES = std::is_same<T, __half>::value;
    const int padded = a.L.units() * MX_UNIT_K;
    const int64_t rows = a.slots / a.x_div;
    const bool wide = ((reinterpret_cast<uintptr_t>(a.x) | (uintptr_t)(a.ldx * (int64_t)sizeof(T))) & 15u) == 0;
    MxtRows x{static_cast<const __half*>(a.x), a.ldx, 0, a.L.K, nullptr, 0};
    if (!HALVES || !wide) {
        __half* planes = static_cast<__half*>(a.planes);
        float* scale = reinterpret_cast<float*>(planes + TERMS * rows * padded);
        x = {planes, padded, rows * padded, padded, HALVES ? nullptr : scale, 0};
        // (a warp a row where that fills the GPU and a row its registers)
        const bool narrow = padded <= (int)(4096 / sizeof(T)) && rows >= 4 * (int64_t)di.sms;
        const unsigned ctas = (unsigned)std::min<int64_t>(narrow ? (rows + 3) / 4 : rows, (int64_t)di.sms * 8);
        if (launch_pdl(narrow ? mxt_rows_kernel<T, 1> : mxt_rows_kernel<T, 4>, dim3(ctas), dim3(MXT_ROW_THREADS), 0, s,
                       static_cast<const T*>(a.x), a.ldx, planes, scale, rows, a.L.K, padded, wide, timeouts[dev]) != cudaSuccess)
            return QGEMV_CUDA_ERROR;
    }
    x.drop = take_drop_request();
    constexpr int GROUP = MODE == MX_GATE_UP ? 8 : 16;
    const int64_t groups = (a.L.tiles() + GROUP - 1) / GROUP;
    const int64_t most = groups * std::min<int64_t>(a.slots, (int64_t)a.slots / MXT_ROWS<TERMS> + a.L.experts);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u * (unsigned)std::min<int64_t>(most, di.sms / 2));
    cfg.blockDim = dim3(MXT_THREADS);
    cfg.dynamicSmemBytes = mxt_smem<TERMS>(a.L.experts);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a, x, timeouts[dev]) == cudaSuccess ? QGEMV_OK : QGEMV_CUDA_ERROR;
}

template <typename T, int MODE>
int launch_mx_mode(const MxArgs& a, cudaStream_t s)
{
    return mx_many_rows(a.slots, a.L.experts, a.L.K) ? launch_mxt<T, MODE>(a, s) : launch_mxs<T, MODE>(a, s);
}

template <typename T>
int launch_mx_gemm_t(int mode, const MxArgs& a, cudaStream_t s)
{
    if (mode == MX_GEMM) return launch_mx_mode<T, MX_GEMM>(a, s);
    if (mode == MX_GATE_UP) return launch_mx_mode<T, MX_GATE_UP>(a, s);
    return launch_mx_mode<T, MX_DOWN>(a, s);
}

}  // namespace qgemv
