// rq_route.cu -- expert routing around the grouped products: the top-k choice
// of each token with its softmax weights, the stable grouping of the chosen
// (token, expert) pairs by expert, and the weighted sum of a token's expert
// outputs.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rq_device.cuh"
#include "rq_internal.h"

namespace rq {
namespace {

constexpr int kRouteThreads = 256;

__device__ __forceinline__ float load_logit(const void* p, size_t i, int bf16) {
    const float v = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
    // NaN is never chosen; +inf counts as the largest finite value, so that weights stay finite
    return v != v ? -INFINITY : fminf(v, 3.402823466e38f);
}

// One warp per token: k rounds of "largest logit after the last choice in
// (value descending, index ascending) order", then the softmax weights.
__global__ void topk_kernel(RouteArgs a) {
    const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (warp >= a.T) return;
    const size_t row = (size_t)warp * a.E;
    float last = INFINITY, top = 0.0f, sum_k = 0.0f, mine = 0.0f;
    int last_i = -1, my_id = -1;
    for (int j = 0; j < a.k; ++j) {
        float b = -INFINITY;
        int bi = 0x7fffffff;
        for (int e = lane; e < a.E; e += 32) {
            const float v = load_logit(a.logits, row + e, a.bf16);
            if (v < last || (v == last && e > last_i))
                if (v > b) { b = v; bi = e; }
        }
        for (int o = 16; o; o >>= 1) {
            const float ob = __shfl_xor_sync(~0u, b, o);
            const int oi = __shfl_xor_sync(~0u, bi, o);
            if (ob > b || (ob == b && oi < bi)) { b = ob; bi = oi; }
        }
        if (b == -INFINITY) break;
        if (j == 0) top = b;
        if (lane == j) { mine = b; my_id = bi; }
        sum_k += expf(b - top);
        last = b;
        last_i = bi;
    }
    float den = sum_k;
    if (!a.renorm) {
        den = 0.0f;
        for (int e = lane; e < a.E; e += 32) den += expf(load_logit(a.logits, row + e, a.bf16) - top);
        for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(~0u, den, o);
    }
    if (lane < a.k) {
        a.ids[(size_t)warp * a.k + lane] = my_id;
        a.weights[(size_t)warp * a.k + lane] = my_id >= 0 ? expf(mine - top) / den : 0.0f;
    }
}

// One CTA per expert: its rank among the experts' counts, then its pairs in order.
__global__ void group_kernel(RouteArgs a) {
    __shared__ int warp_sum[kRouteThreads / 32];
    __shared__ int base_s, run_s;
    const int e = blockIdx.x, P = a.T * a.k, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    if (tid == 0) base_s = 0;
    __syncthreads();
    int below = 0;                                       // pairs of experts below e (e == E: all chosen pairs)
    for (int i = tid; i < P; i += kRouteThreads) below += a.ids[i] >= 0 && a.ids[i] < e;
    atomicAdd(&base_s, below);
    __syncthreads();
    const int base = base_s;
    if (tid == 0) { a.offsets[e] = base; run_s = base; }
    __syncthreads();
    for (int i0 = 0; i0 < P; i0 += kRouteThreads) {
        const int i = i0 + tid;
        const bool hit = i < P && (e == a.E ? a.ids[i] < 0 : a.ids[i] == e);
        const unsigned m = __ballot_sync(~0u, hit);
        if (lane == 0) warp_sum[w] = __popc(m);
        __syncthreads();
        int before = run_s, total = 0;
        for (int v = 0; v < kRouteThreads / 32; ++v) {
            if (v < w) before += warp_sum[v];
            total += warp_sum[v];
        }
        if (hit) {
            const int at = before + __popc(m & ((1u << lane) - 1u));
            a.in_rows[at] = e == a.E ? -1 : i / a.k;
            a.slots[at] = e == a.E ? -1 : i;
        }
        __syncthreads();
        if (tid == 0) run_s += total;
        __syncthreads();
    }
}

__global__ void combine_kernel(CombineArgs a) {
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (size_t)a.T * a.N) return;
    const int t = (int)(i / a.N), n = (int)(i % a.N);
    float s = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const size_t p = (size_t)t * a.k + j;
        if (a.ids[p] < 0) continue;
        const float v = a.ybf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.y)[p * a.N + n])
                                : static_cast<const float*>(a.y)[p * a.N + n];
        s = fmaf(a.weights[p], v, s);
    }
    store_y(a.out, i, s, a.obf16);
}

}  // namespace

size_t route_workspace(int, int, int) { return 16; }

cudaError_t launch_route(const RouteArgs& a, cudaStream_t st) {
    topk_kernel<<<(a.T + 7) / 8, 256, 0, st>>>(a);
    group_kernel<<<a.E + 1, kRouteThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t st) {
    const size_t n = (size_t)a.T * a.N;
    combine_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace rq
