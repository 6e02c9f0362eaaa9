// rq_route.cu -- expert routing around the grouped products: the top-k choice
// of each token with its softmax weights, the stable grouping of the chosen
// (token, expert) pairs by expert, and the weighted sum of a token's expert
// outputs.
//
// Routing is a counting sort. Blocks of tokens (at most kMaxBlocks) choose
// their experts and count them (choose_kernel); then each block of the same
// tokens sums the counts before it and places its pairs (place_kernel), in
// order, so that the result does not depend on scheduling. Up to kOneBlock
// tokens one block does both in one launch: a decode step pays for latency,
// not for work. The combine reads k rows and writes one per token: bound by
// memory, 16 bytes per load.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rq_device.cuh"
#include "rq_internal.h"

namespace rq {
namespace {

constexpr int kRouteThreads = 1024;
constexpr int kMaxBlocks = 256;
constexpr int kOneBlock = 64;

// fp32 as an unsigned key with the same order; 0 for a logit that is never
// chosen (-inf, NaN). +inf counts as the largest finite value, so that the
// weights stay finite; -0 as 0.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (!(v > -INFINITY)) return 0u;
    v = fminf(v, 3.402823466e38f) + 0.0f;
    const uint32_t u = __float_as_uint(v);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

__device__ __forceinline__ float load_logit(const void* p, size_t i, int bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// One warp chooses for one token, its logits in registers (V per lane, expert
// lane + 32 i): k times the largest key and the lowest expert that has it.
// Lane j keeps choice j.
template <int V>
__device__ __forceinline__ void choose(const RouteArgs& a, int t, int lane, int& my_id, float& my_w) {
    const size_t row = (size_t)t * a.E;
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < a.E ? order_key(load_logit(a.logits, row + e, a.bf16)) : 0u;
    }
    my_id = -1;
    my_w = 0.0f;
    float top = 0.0f, den = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = max(m, key[i]);
        m = __reduce_max_sync(~0u, m);
        if (m == 0u) break;
        if (j == 0) {
            top = key_value(m);
            if (!a.renorm) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (key[i]) den += expf(key_value(key[i]) - top);
            }
        }
        int e = 0x7fffffff;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            if (key[i] == m) e = lane + 32 * i;
        e = __reduce_min_sync(~0u, e);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i == e) key[i] = 0u;
        const float w = expf(key_value(m) - top);
        if (lane == j) { my_id = e; my_w = w; }
        if (a.renorm) den += w;                          // the same in every lane
    }
    if (!a.renorm)
        for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(~0u, den, o);
    if (my_id >= 0) my_w = my_w / den;
}

// Places a block's pairs [i0, i1) by expert: one warp, 32 pairs at a time in
// order, at[e] the next free row of expert e.
__device__ __forceinline__ void place(const RouteArgs& a, int* at, int i0, int i1, int lane) {
    for (int i = i0; i < i1; i += 32) {
        const int e = i + lane < i1 ? a.ids[i + lane] : -1;
        const unsigned same = __match_any_sync(~0u, e);
        const int before = __popc(same & ((1u << lane) - 1u));
        int row = 0;
        if (e >= 0) row = at[e] + before;
        __syncwarp();
        if (e >= 0 && before == 0) at[e] += __popc(same);
        __syncwarp();
        if (e >= 0) {
            a.in_rows[row] = (i + lane) / a.k;
            a.slots[row] = i + lane;
        }
    }
}

// Exclusive sums of v[0..E - 1] in place, by one warp; returns the total.
__device__ __forceinline__ int scan_warp(int* v, int E, int lane) {
    int run = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int x = e0 + lane < E ? v[e0 + lane] : 0;
        int s = x;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, s, o);
            if (lane >= o) s += y;
        }
        if (e0 + lane < E) v[e0 + lane] = run + s - x;
        run += __shfl_sync(~0u, s, 31);
    }
    __syncwarp();
    return run;
}

// Tokens [blockIdx.x per, + per): choices, and the block's count of each
// expert; with one block also the places.
template <int V>
__global__ void __launch_bounds__(kRouteThreads) choose_kernel(RouteArgs a, int per) {
    __shared__ int count[1024];
    const int tid = threadIdx.x, lane = tid & 31;
    for (int e = tid; e < a.E; e += blockDim.x) count[e] = 0;
    grid_dep_wait();
    grid_dep_launch();
    __syncthreads();
    const int t0 = blockIdx.x * per, t1 = min(a.T, t0 + per);
    for (int t = t0 + (tid >> 5); t < t1; t += blockDim.x >> 5) {
        int id;
        float w;
        choose<V>(a, t, lane, id, w);
        if (lane < a.k) {
            a.ids[(size_t)t * a.k + lane] = id;
            a.weights[(size_t)t * a.k + lane] = w;
            if (id >= 0) atomicAdd(&count[id], 1);
        }
    }
    __syncthreads();
    if (gridDim.x > 1) {
        for (int e = tid; e < a.E; e += blockDim.x) static_cast<int*>(a.ws)[(size_t)blockIdx.x * a.E + e] = count[e];
        return;
    }
    const int P = a.T * a.k;
    __shared__ int total;
    if (tid < 32) {
        const int n = scan_warp(count, a.E, lane);
        if (lane == 0) total = n;
        for (int e = lane; e <= a.E; e += 32) a.offsets[e] = e < a.E ? count[e] : n;
        __syncwarp();
        place(a, count, 0, P, lane);
    }
    __syncthreads();
    for (int i = total + tid; i < P; i += blockDim.x) a.in_rows[i] = a.slots[i] = -1;
}

constexpr int kPlaceThreads = 256;

__global__ void __launch_bounds__(kPlaceThreads) place_kernel(RouteArgs a, int per) {
    extern __shared__ int sm[];                          // at[E], then before[E] summed over threads
    int* at = sm;
    int* before = sm + a.E;
    const int tid = threadIdx.x, lane = tid & 31, nb = gridDim.x;
    for (int e = tid; e < 2 * a.E; e += kPlaceThreads) sm[e] = 0;
    grid_dep_wait();
    grid_dep_launch();
    __syncthreads();
    const int* c = static_cast<const int*>(a.ws);
    // several threads per expert while there are fewer experts than threads
    const int ways = a.E >= kPlaceThreads ? 1 : kPlaceThreads / a.E;
    for (int x = tid; x < ways * a.E; x += kPlaceThreads) {
        const int e = x % a.E;
        int all = 0, low = 0;
#pragma unroll 8
        for (int b = x / a.E; b < nb; b += ways) {
            const int v = c[(size_t)b * a.E + e];
            all += v;
            if (b < (int)blockIdx.x) low += v;
        }
        atomicAdd(&at[e], all);
        atomicAdd(&before[e], low);
    }
    __syncthreads();
    __shared__ int total;
    const int P = a.T * a.k;
    if (tid < 32) {
        const int n = scan_warp(at, a.E, lane);
        if (lane == 0) total = n;
        if (blockIdx.x == 0)
            for (int e = lane; e <= a.E; e += 32) a.offsets[e] = e < a.E ? at[e] : n;
        __syncwarp();
        for (int e = lane; e < a.E; e += 32) at[e] += before[e];
        __syncwarp();
        const int t0 = blockIdx.x * per;
        place(a, at, t0 * a.k, min(a.T, t0 + per) * a.k, lane);
    }
    __syncthreads();
    for (int i = total + (int)blockIdx.x * kPlaceThreads + tid; i < P; i += nb * kPlaceThreads) a.in_rows[i] = a.slots[i] = -1;
}

// ---------------------------------------------------------------- combine
template <bool YB>
__device__ __forceinline__ void load8(const void* y, size_t i, float (&v)[8]) {
    if constexpr (YB) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(y) + i));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) { v[2 * q] = bf16lo_f32(w[q]); v[2 * q + 1] = bf16hi_f32(w[q]); }
    } else {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(y) + i);
        const float4 a = __ldcs(f), b = __ldcs(f + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

// Eight columns of a token per thread (N a multiple of 8), two choices'
// loads at a time.
template <bool YB, bool OB>
__global__ void __launch_bounds__(256) combine8_kernel(CombineArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const int per = a.N / 8;                             // vectors of a row
    const long long n = (long long)a.T * per;
    for (long long x = (long long)blockIdx.x * 256 + threadIdx.x; x < n; x += (long long)gridDim.x * 256) {
        const int t = (int)(x / per), c = (int)(x - (long long)t * per) * 8;
        float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        for (int j = 0; j < a.k; j += 2) {
            const size_t p = (size_t)t * a.k + j;
            const bool on0 = __ldg(a.ids + p) >= 0, on1 = j + 1 < a.k && __ldg(a.ids + p + 1) >= 0;
            float v0[8], v1[8];
            if (on0) load8<YB>(a.y, p * a.N + c, v0);
            if (on1) load8<YB>(a.y, (p + 1) * a.N + c, v1);
            const float w0 = on0 ? __ldg(a.weights + p) : 0.0f, w1 = on1 ? __ldg(a.weights + p + 1) : 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (on0) s[q] = fmaf(w0, v0[q], s[q]);
                if (on1) s[q] = fmaf(w1, v1[q], s[q]);
            }
        }
        const size_t o = (size_t)t * a.N + c;
        if constexpr (OB) {
            uint32_t u[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(s[2 * q], s[2 * q + 1]);
                u[q] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + o) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
            float4* f = reinterpret_cast<float4*>(static_cast<float*>(a.out) + o);
            f[0] = make_float4(s[0], s[1], s[2], s[3]);
            f[1] = make_float4(s[4], s[5], s[6], s[7]);
        }
    }
}

// Any N: one column per thread.
__global__ void __launch_bounds__(256) combine1_kernel(CombineArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const long long n = (long long)a.T * a.N;
    for (long long x = (long long)blockIdx.x * 256 + threadIdx.x; x < n; x += (long long)gridDim.x * 256) {
        const int t = (int)(x / a.N), c = (int)(x - (long long)t * a.N);
        float s = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const size_t p = (size_t)t * a.k + j;
            if (a.ids[p] < 0) continue;
            const float v = a.ybf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.y)[p * a.N + c])
                                    : static_cast<const float*>(a.y)[p * a.N + c];
            s = fmaf(a.weights[p], v, s);
        }
        store_y(a.out, (size_t)x, s, a.obf16);
    }
}

template <class K, class... A>
cudaError_t launch(K kernel, int grid, int block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Tokens per block: one block for few tokens, else a multiple of the block's
// 32 warps with at most kMaxBlocks blocks.
int tokens_per_block(int T) {
    if (T <= kOneBlock) return T;
    const int per = (T + kMaxBlocks - 1) / kMaxBlocks;
    return (per + 31) / 32 * 32;
}

}  // namespace

size_t route_workspace(int T, int E, int) {
    const int per = tokens_per_block(T);
    return round16((size_t)((T + per - 1) / per) * E * 4);
}

cudaError_t launch_route(const RouteArgs& a, cudaStream_t st) {
    const int per = tokens_per_block(a.T), blocks = (a.T + per - 1) / per;
    const int warps = per < 32 ? per : 32;
    const int threads = warps * 32;
    const int v = (a.E + 31) / 32;
    const cudaError_t e = v <= 1  ? launch(choose_kernel<1>, blocks, threads, 0, st, a, per)
                        : v <= 2  ? launch(choose_kernel<2>, blocks, threads, 0, st, a, per)
                        : v <= 4  ? launch(choose_kernel<4>, blocks, threads, 0, st, a, per)
                        : v <= 8  ? launch(choose_kernel<8>, blocks, threads, 0, st, a, per)
                        : v <= 16 ? launch(choose_kernel<16>, blocks, threads, 0, st, a, per)
                                  : launch(choose_kernel<32>, blocks, threads, 0, st, a, per);
    if (e != cudaSuccess || blocks == 1) return e;
    return launch(place_kernel, blocks, kPlaceThreads, (size_t)2 * a.E * 4, st, a, per);
}

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t st) {
    const bool wide = a.N % 8 == 0;
    const long long n = (long long)a.T * (wide ? a.N / 8 : a.N);
    const long long want = (n + 255) / 256, most = (long long)sm_count() * 64;
    const int grid = (int)(want < most ? want : most);
    if (!wide) return launch(combine1_kernel, grid, 256, 0, st, a);
    if (a.ybf16) return a.obf16 ? launch(combine8_kernel<true, true>, grid, 256, 0, st, a)
                                : launch(combine8_kernel<true, false>, grid, 256, 0, st, a);
    return a.obf16 ? launch(combine8_kernel<false, true>, grid, 256, 0, st, a)
                   : launch(combine8_kernel<false, false>, grid, 256, 0, st, a);
}

}  // namespace rq
