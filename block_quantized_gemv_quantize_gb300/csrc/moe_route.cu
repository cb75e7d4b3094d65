// The router of a sparse layer: each token's experts and weights, and the
// slots sorted by expert.
//
// Choice: the top_k largest logits, by rounds of a warp's maximum (a token a
// warp, its logits in registers): exact, and of equal logits the lowest
// expert.  Weights from the same registers.  Sort: a stable counting sort
// over contiguous ranges of slots, one a CTA.  Every count is an integer, so
// that neither the order of atomics nor the grid changes the result.
// Up to SMALL_TOKENS tokens one CTA does all of it in one launch (latency);
// beyond, a first kernel routes and counts, a second adds up each bin's counts
// over the ranges, a third places the slots.  Bound by the instructions of a
// token's top_k rounds (2.5 of 4 issued a clock), and the three launches (17391 tokens, 8 of 128 experts: 18.5 us,
// one token 3.6; a second kernel in which each CTA added up all ranges' counts took 25 us more).
#include "mxfp4.cuh"

#include <mutex>

namespace qgemv {
namespace {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int SMALL_TOKENS = 4 * WARPS;
constexpr int MAX_RANGES = 1024;  // CTAs of a large call

// A range a CTA: a token a warp, or as many more as keep to MAX_RANGES.
__host__ __device__ inline int range_tokens(int tokens)
{
    return WARPS * max(1, (tokens + WARPS * MAX_RANGES - 1) / (WARPS * MAX_RANGES));
}

// Larger value, larger key; of -0 and +0 one key; NaN and minus infinity 0.
__device__ __forceinline__ uint32_t logit_key(float v)
{
    if (!(v > -INFINITY)) return 0u;
    const uint32_t u = v == 0.0f ? 0u : __float_as_uint(v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The same for the 16-bit types, whose key leaves room for the expert (the lower, the
// larger), so that one maximum finds both.
template <typename T>
__device__ __forceinline__ uint32_t logit_key16(T v, int e)
{
    const float f = to_f32(v);
    if (!(f > -INFINITY)) return 0u;
    const uint32_t u = f == 0.0f ? 0u : (uint32_t)*reinterpret_cast<const uint16_t*>(&v);
    return (((u & 0x8000u) ? ~u & 0xFFFFu : (u | 0x8000u)) << 16) | (uint32_t)(0xFFFF - e);
}
template <typename T>
__device__ __forceinline__ float key16_logit(uint32_t k)
{
    const uint32_t o = k >> 16;
    const uint16_t u = (uint16_t)((o & 0x8000u) ? (o & 0x7FFFu) : ~o);
    return to_f32(*reinterpret_cast<const T*>(&u));
}

__device__ __forceinline__ float key_logit(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// One token by one warp: lane j gets place j's expert (-1: none) and weight.
template <typename T, int PER>
__device__ __forceinline__ void route_token(const T* row, const RouteArgs& a, int lane, int& id, float& weight)
{
    constexpr bool SHORT = sizeof(T) == 2;
    auto value = [](uint32_t k) { if constexpr (SHORT) return key16_logit<T>(k); else return key_logit(k); };
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        if constexpr (SHORT) key[i] = e < a.experts ? logit_key16(row[e], e) : 0u;
        else key[i] = e < a.experts ? logit_key(row[e]) : 0u;
    }
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine = max(mine, key[i]);
    const uint32_t top = __reduce_max_sync(~0u, mine);
    const float best = top ? value(top) : 0.0f;
    float total = 1.0f;
    if (!a.sigmoid && !a.renormalize) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i]) s += expf(value(key[i]) - best);
        total = warp_sum(s);
    }
    id = -1;
    uint32_t chosen = 0;
    for (int j = 0; j < a.top_k; ++j) {
        const uint32_t k = __reduce_max_sync(~0u, mine);
        if (k == 0) break;
        if (lane == j) chosen = k;
        if constexpr (SHORT) {  // (no two keys are the same)
            mine = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (key[i] == k) key[i] = 0;
                mine = max(mine, key[i]);
            }
        } else {
            int at = MX_MAX_EXPERTS;
            if (mine == k) {
#pragma unroll
                for (int i = PER - 1; i >= 0; --i)
                    if (key[i] == k) at = lane + 32 * i;
            }
            at = __reduce_min_sync(~0u, at);
            if (lane == j) id = at;
            if ((at & 31) == lane) {
                mine = 0;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    if (at == lane + 32 * i) key[i] = 0;
                    mine = max(mine, key[i]);
                }
            }
        }
    }
    if (SHORT && chosen) id = 0xFFFF - (int)(chosen & 0xFFFFu);
    const float logit = chosen ? value(chosen) : -INFINITY;
    if (a.sigmoid) {
        // sigmoid(l) over the sum of them: from their logarithms, so that logits far below zero keep their ratios
        const float ls = logit > 0.0f ? -log1pf(expf(-logit)) : logit - log1pf(expf(logit));
        if (a.renormalize) {
            float most = id < 0 ? -INFINITY : ls;
#pragma unroll
            for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
            weight = id < 0 ? 0.0f : expf(ls - most);
            total = warp_sum(weight);
        } else {
            weight = 1.0f / (1.0f + expf(-logit));
        }
    } else {
        weight = id < 0 ? 0.0f : expf(logit - best);
        if (a.renormalize) total = warp_sum(weight);
    }
    weight = id < 0 ? 0.0f : weight / total * a.scale;
}

// The tokens [t0, t1) of a CTA: ids and weights out, or ids given.
template <typename T, int PER>
__device__ __forceinline__ void route_range(const RouteArgs& a, int t0, int t1)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int t = t0 + warp; t < t1; t += WARPS) {
        int id;
        float weight;
        route_token<T, PER>(static_cast<const T*>(a.logits) + t * a.ld, a, lane, id, weight);
        if (lane < a.top_k && QG_OK(qg_in((int64_t)t * a.top_k + lane, 1, (int64_t)a.tokens * a.top_k), a.status, 340)) {
            a.ids[(int64_t)t * a.top_k + lane] = id;
            a.weights[(int64_t)t * a.top_k + lane] = weight;
        }
    }
}

// An index of the workspace's counts.
__device__ __forceinline__ bool counts_in(int64_t i, int bins) { return qg_in(i, 1, (int64_t)(MAX_RANGES + 1) * bins); }

// The bin of an id: its expert, or `experts` for a slot without one.
__device__ __forceinline__ int bin_of(int id, int experts) { return id >= 0 && id < experts ? id : experts; }

// Exclusive sums of v[0 .. n) in place, by the whole CTA; returns the total.
__device__ int scan_bins(int* v, int n, int* sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int base = 0;
    for (int lo = 0; lo < n; lo += THREADS) {
        const int i = lo + threadIdx.x;
        const int mine = i < n ? v[i] : 0;
        int s = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(~0u, s, o);
            if (lane >= o) s += up;
        }
        if (lane == 31) sums[warp] = s;
        __syncthreads();
        int before = base, all = 0;
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) before += sums[w];
            all += sums[w];
        }
        if (i < n) v[i] = before + s - mine;
        base += all;
        __syncthreads();
    }
    return base;
}

// Places the slots [s0, s1) of a CTA, in order within each bin.  first[bin] is the
// place of the range's first slot of the bin; per_warp [WARPS][bins] scratch.
// Each warp has a contiguous part of the range: it counts its bins, the warps'
// counts add up before it, then it places 32 slots at a time.
__device__ void place_range(const RouteArgs& a, const int32_t* ids, int s0, int s1, const int* first, int* per_warp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = a.experts + 1;
    const int part = ((s1 - s0 + WARPS - 1) / WARPS + 31) & ~31;
    const int lo = min(s1, s0 + warp * part), hi = min(s1, lo + part);
    for (int i = threadIdx.x; i < WARPS * bins; i += THREADS) per_warp[i] = 0;
    __syncthreads();
    int* mine = per_warp + warp * bins;
    for (int s = lo + lane; s < hi; s += 32) atomicAdd(&mine[bin_of(ids[s], a.experts)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += THREADS) {
        int at = first[b];
        for (int w = 0; w < WARPS; ++w) {
            const int n = per_warp[w * bins + b];
            per_warp[w * bins + b] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int base = lo; base < hi; base += 32) {
        const int s = base + lane;
        const int b = s < hi ? bin_of(ids[s], a.experts) : -1;
        const uint32_t same = __match_any_sync(~0u, b);
        const int rank = __popc(same & ((1u << lane) - 1u));
        int at = 0;
        if (b >= 0) at = mine[b];
        __syncwarp();
        if (b >= 0) {
            if (QG_OK(qg_in(at + rank, 1, (int64_t)a.tokens * a.top_k), a.status, 341)) a.order[at + rank] = s;
            if (rank == 0) mine[b] = at + __popc(same);
        }
        __syncwarp();
    }
}

__host__ __device__ constexpr int smem_ints(int experts) { return (WARPS + 1) * (experts + 1) + WARPS; }

template <typename T, int PER, bool ROUTE>
__global__ void __launch_bounds__(THREADS) small_kernel(RouteArgs a)
{
    extern __shared__ int sm[];
    const int bins = a.experts + 1, slots = a.tokens * a.top_k;
    int *first = sm, *per_warp = sm + bins, *sums = per_warp + WARPS * bins;
    pdl_launch_dependents();
    pdl_wait();
    if constexpr (ROUTE) route_range<T, PER>(a, 0, a.tokens);
    for (int i = threadIdx.x; i < bins; i += THREADS) first[i] = 0;
    __syncthreads();  // (this CTA's ids are visible to it)
    for (int s = threadIdx.x; s < slots; s += THREADS) atomicAdd(&first[bin_of(a.ids[s], a.experts)], 1);
    __syncthreads();
    scan_bins(first, bins, sums);
    for (int i = threadIdx.x; i < bins; i += THREADS) a.offsets[i] = first[i];
    place_range(a, a.ids, 0, slots, first, per_warp);
}

template <typename T, int PER, bool ROUTE>
__global__ void __launch_bounds__(THREADS) count_kernel(RouteArgs a, int per)
{
    extern __shared__ int sm[];
    const int bins = a.experts + 1;
    const int t0 = min(a.tokens, (int)blockIdx.x * per), t1 = min(a.tokens, t0 + per);
    pdl_launch_dependents();
    pdl_wait();
    for (int i = threadIdx.x; i < bins; i += THREADS) sm[i] = 0;
    if constexpr (ROUTE) route_range<T, PER>(a, t0, t1);
    __syncthreads();
    for (int s = t0 * a.top_k + threadIdx.x; s < t1 * a.top_k; s += THREADS)
        atomicAdd(&sm[bin_of(a.ids[s], a.experts)], 1);
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += THREADS)
        if (QG_OK(counts_in((int64_t)blockIdx.x * bins + i, bins), a.status, 342)) a.counts[(int64_t)blockIdx.x * bins + i] = sm[i];
}

// Each bin's counts become the sums over the ranges before, its total goes behind them all.  Eight
// bins a CTA (a sector of a range's counts), 32 ranges a thread.  (A bin a warp, its lanes a row
// apart each, makes the whole call 20.8 us instead of 18.5.)
constexpr int SUM_BINS = 8, SUM_THREADS = 32 * SUM_BINS;

__global__ void __launch_bounds__(SUM_THREADS) sum_kernel(RouteArgs a, int ranges)
{
    constexpr int PER = MAX_RANGES / 32;
    static_assert(PER * 32 == MAX_RANGES, "a range a thread and step");
    __shared__ int part[32][SUM_BINS + 1];
    const int sub = threadIdx.x % SUM_BINS, group = threadIdx.x / SUM_BINS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int bins = a.experts + 1, b = blockIdx.x * SUM_BINS + sub;
    const int mine = b < bins ? max(0, min(PER, ranges - group * PER)) : 0;
    pdl_launch_dependents();
    pdl_wait();
    int32_t* counts = a.counts + (int64_t)group * PER * bins + b;
    int n[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) n[i] = i < mine ? counts[i * bins] : 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += n[i];
    part[group][sub] = sum;
    __syncthreads();
    {
        const int own = part[lane][warp];
        int at = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(~0u, at, o);
            if (lane >= o) at += up;
        }
        part[lane][warp] = at - own;
        const int whose = blockIdx.x * SUM_BINS + warp;
        if (lane == 31 && whose < bins && QG_OK(counts_in((int64_t)MAX_RANGES * bins + whose, bins), a.status, 343))
            a.counts[(int64_t)MAX_RANGES * bins + whose] = at;
    }
    __syncthreads();
    int at = part[group][sub];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (i < mine && QG_OK(counts_in(counts - a.counts + i * bins, bins), a.status, 344)) counts[i * bins] = at;
        at += n[i];
    }
}

__global__ void __launch_bounds__(THREADS) place_kernel(RouteArgs a, int per)
{
    extern __shared__ int sm[];
    const int bins = a.experts + 1;
    int *first = sm, *per_warp = sm + bins, *sums = per_warp + WARPS * bins;
    const int t0 = min(a.tokens, (int)blockIdx.x * per), t1 = min(a.tokens, t0 + per);
    pdl_launch_dependents();
    pdl_wait();
    constexpr int PER = (MX_MAX_EXPERTS + THREADS) / THREADS;
    int before[PER];  // this range's first place in the bin
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = threadIdx.x + i * THREADS;
        before[i] = b < bins ? a.counts[(int64_t)blockIdx.x * bins + b] : 0;
        if (b < bins) first[b] = a.counts[(int64_t)MAX_RANGES * bins + b];
    }
    __syncthreads();
    scan_bins(first, bins, sums);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < bins; i += THREADS) a.offsets[i] = first[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if ((int)threadIdx.x + i * THREADS < bins) first[threadIdx.x + i * THREADS] += before[i];
    __syncthreads();
    place_range(a, a.ids, t0 * a.top_k, t1 * a.top_k, first, per_warp);
}

template <typename T, int PER, bool ROUTE>
int route_tp(const RouteArgs& a, cudaStream_t s)
{
    const DeviceInfo di = device_info();
    int dev = 0;
    if (di.sms <= 0 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return QGEMV_CUDA_ERROR;
    const size_t smem = (size_t)smem_ints(a.experts) * sizeof(int);
    if (a.tokens <= SMALL_TOKENS) {
        static std::once_flag once[64];
        static bool ok[64];
        auto kern = small_kernel<T, PER, ROUTE>;
        std::call_once(once[dev], [&]() {
            ok[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, di.smem_optin) == cudaSuccess;
            if (!ok[dev]) cudaGetLastError();
        });
        if (!ok[dev]) return QGEMV_CUDA_ERROR;
        return launch_pdl(kern, dim3(1), dim3(THREADS), smem, s, a) == cudaSuccess ? QGEMV_OK : QGEMV_CUDA_ERROR;
    }
    const int per = range_tokens(a.tokens);
    const unsigned grid = (unsigned)((a.tokens + per - 1) / per);
    static std::once_flag once[64];
    static bool ok[64];
    std::call_once(once[dev], [&]() {
        ok[dev] =
            cudaFuncSetAttribute(place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, di.smem_optin) == cudaSuccess;
        if (!ok[dev]) cudaGetLastError();
    });
    if (!ok[dev]) return QGEMV_CUDA_ERROR;
    if (launch_pdl(count_kernel<T, PER, ROUTE>, dim3(grid), dim3(THREADS), (size_t)(a.experts + 1) * sizeof(int), s, a,
                   per) != cudaSuccess)
        return QGEMV_CUDA_ERROR;
    if (launch_pdl(sum_kernel, dim3((unsigned)(a.experts + SUM_BINS) / SUM_BINS), dim3(SUM_THREADS), 0, s, a, (int)grid) != cudaSuccess)
        return QGEMV_CUDA_ERROR;
    return launch_pdl(place_kernel, dim3(grid), dim3(THREADS), smem, s, a, per) == cudaSuccess ? QGEMV_OK
                                                                                               : QGEMV_CUDA_ERROR;
}

template <typename T>
int route_t(const RouteArgs& a, cudaStream_t s)
{
    if (a.experts <= 64) return route_tp<T, 2, true>(a, s);
    if (a.experts <= 128) return route_tp<T, 4, true>(a, s);
    if (a.experts <= 256) return route_tp<T, 8, true>(a, s);
    return route_tp<T, 32, true>(a, s);
}

}  // namespace

size_t route_workspace_bytes(int tokens, int experts)
{
    return tokens <= SMALL_TOKENS ? 0 : (size_t)(MAX_RANGES + 1) * (experts + 1) * sizeof(int32_t);
}

int launch_route(int type, const RouteArgs& args, cudaStream_t s)
{
    RouteArgs a = args;
    a.status = wait_timeout_counter();
    if (!a.logits) return route_tp<float, 1, false>(a, s);
    if (type == QGEMV_F32) return route_t<float>(a, s);
    if (type == QGEMV_F16) return route_t<__half>(a, s);
    return route_t<__nv_bfloat16>(a, s);
}

}  // namespace qgemv
