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
// Measured: 8191 tokens, E 64, k 4, bf16: 11.0 us: two launches, and in the
// second one warp of a block places its pairs while the others wait (an expert's
// counts summed by several threads with shared atomics instead of one warp:
// 16.4; 256 blocks instead of 128: 2 us more). 1 token: 3.4 us.
// Combine of 8192 tokens, k 2, N 4096, bf16: 35 us, 5.7 TB/s (87 % of a copy);
// where N is no multiple of 8, one element per load: N 4095 240 us, 0.84 TB/s.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rq_device.cuh"
#include "rq_internal.h"

namespace rq {
namespace {

constexpr int kRouteThreads = 1024;
constexpr int kMaxBlocks = 128;                        // a lane of a warp sums four of them
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

// Places a block's pairs i0 .. i0 + n - 1 by expert: one warp, 32 pairs at a
// time in order, ids in shared memory, at[e] the next free row of expert e.
__device__ __forceinline__ void place(const RouteArgs& a, int* at, const int* ids, int i0, int n, int lane) {
    for (int i = 0; i < n; i += 32) {
        const int e = i + lane < n ? ids[i + lane] : -1;
        const unsigned same = __match_any_sync(~0u, e);
        const int before = __popc(same & ((1u << lane) - 1u));
        int row = 0;
        if (e >= 0) row = at[e] + before;
        __syncwarp();
        if (e >= 0 && before == 0) at[e] += __popc(same);
        __syncwarp();
        if (e >= 0) {
            a.in_rows[row] = (i0 + i + lane) / a.k;
            a.slots[row] = i0 + i + lane;
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
    __shared__ int chosen[kOneBlock * 16];               // with one block: the ids
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
            if (gridDim.x == 1) chosen[t * a.k + lane] = id;
            if (id >= 0) atomicAdd(&count[id], 1);
        }
    }
    __syncthreads();
    if (gridDim.x > 1) {
        // an expert's counts lie together; a token counts once for an expert, so that 16 bits hold a block's
        for (int e = tid; e < a.E; e += blockDim.x)
            static_cast<uint16_t*>(a.ws)[(size_t)e * kMaxBlocks + blockIdx.x] = (uint16_t)count[e];
        return;
    }
    const int P = a.T * a.k;
    __shared__ int total;
    if (tid < 32) {
        const int n = scan_warp(count, a.E, lane);
        if (lane == 0) total = n;
        for (int e = lane; e <= a.E; e += 32) a.offsets[e] = e < a.E ? count[e] : n;
        __syncwarp();
        place(a, count, chosen, 0, P, lane);
    }
    __syncthreads();
    for (int i = total + tid; i < P; i += blockDim.x) a.in_rows[i] = a.slots[i] = -1;
}

constexpr int kPlaceThreads = 1024;

__global__ void __launch_bounds__(kPlaceThreads) place_kernel(RouteArgs a, int per) {
    extern __shared__ int sm[];                          // per expert: all blocks' sum, the sum before this block; the block's ids
    int* at = sm;
    int* before = sm + a.E;
    int* ids = sm + 2 * a.E;
    const int tid = threadIdx.x, lane = tid & 31, nb = gridDim.x;
    grid_dep_wait();
    grid_dep_launch();
    const int i0 = blockIdx.x * per * a.k, n = min(a.T * a.k - i0, per * a.k);
    for (int i = tid; i < n; i += kPlaceThreads) ids[i] = a.ids[i0 + i];
    // a warp per expert, four blocks' counts per lane
#pragma unroll 4
    for (int e = tid >> 5; e < a.E; e += kPlaceThreads / 32) {
        const uint2 c = static_cast<const uint2*>(a.ws)[(size_t)e * (kMaxBlocks / 4) + lane];
        const int v[4] = {(int)(c.x & 0xffff), (int)(c.x >> 16), (int)(c.y & 0xffff), (int)(c.y >> 16)};
        int all = 0, low = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (4 * lane + i < nb) all += v[i];
            if (4 * lane + i < (int)blockIdx.x) low += v[i];
        }
        all = __reduce_add_sync(~0u, all);
        low = __reduce_add_sync(~0u, low);
        if (lane == 0) {
            at[e] = all;
            before[e] = low;
        }
    }
    __syncthreads();
    __shared__ int total;
    const int P = a.T * a.k;
    if (tid < 32) {
        const int all = scan_warp(at, a.E, lane);
        if (lane == 0) total = all;
        if (blockIdx.x == 0)
            for (int e = lane; e <= a.E; e += 32) a.offsets[e] = e < a.E ? at[e] : all;
        __syncwarp();
        for (int e = lane; e < a.E; e += 32) at[e] += before[e];
        __syncwarp();
        place(a, at, ids, i0, n, lane);
    }
    __syncthreads();
    for (int i = total + (int)blockIdx.x * kPlaceThreads + tid; i < P; i += nb * kPlaceThreads) a.in_rows[i] = a.slots[i] = -1;
}

// ---------------------------------------------------------------- combine
// Eight consecutive values of y as they lie in memory.
template <bool YB>
struct Raw8 {
    uint4 a[YB ? 1 : 2];
    __device__ __forceinline__ void load(const void* y, size_t i) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(y) + i * (YB ? 2 : 4));
        a[0] = __ldcs(p);
        if (!YB) a[YB ? 0 : 1] = __ldcs(p + 1);
    }
    __device__ __forceinline__ float at(int q) const {
        const uint4 v = a[YB ? 0 : q >> 2];
        const int i = YB ? q >> 1 : q & 3;
        const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
        return !YB ? __uint_as_float(w) : q & 1 ? bf16hi_f32(w) : bf16lo_f32(w);
    }
};

// A block takes 512 vectors of eight columns of one token (N a multiple of 8):
// two per thread, with two choices' loads of both in flight.
constexpr int kCombineVecs = 512;

template <bool YB, bool OB>
__global__ void __launch_bounds__(256) combine8_kernel(CombineArgs a, int chunks) {
    grid_dep_wait();
    grid_dep_launch();
    const int per = a.N / 8, t = blockIdx.x / chunks, v0 = (blockIdx.x - t * chunks) * kCombineVecs + threadIdx.x;
    const size_t row = (size_t)t * a.k;
    float s[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 8; ++q) s[h][q] = 0.0f;
    for (int j = 0; j < a.k; j += 2) {
        // The rows are loaded beside their ids, not after them (what a row without an expert holds is dropped), and
        // all loads are unconditional (a choice or column past the end reads the last one).
        Raw8<YB> v[2][2];
        bool on[2];
        float w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) v[i][h].load(a.y, (row + min(j + i, a.k - 1)) * a.N + 8 * min(v0 + 256 * h, per - 1));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            on[i] = __ldg(a.ids + row + min(j + i, a.k - 1)) >= 0 && j + i < a.k;
            w[i] = __ldg(a.weights + row + min(j + i, a.k - 1));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (on[i])
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < 8; ++q) s[h][q] = fmaf(w[i], v[i][h].at(q), s[h][q]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (v0 + 256 * h >= per) break;
        const size_t o = (size_t)t * a.N + 8 * (v0 + 256 * h);
        if constexpr (OB) {
            uint32_t u[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(s[h][2 * q], s[h][2 * q + 1]);
                u[q] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + o) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
            float4* f = reinterpret_cast<float4*>(static_cast<float*>(a.out) + o);
            f[0] = make_float4(s[h][0], s[h][1], s[h][2], s[h][3]);
            f[1] = make_float4(s[h][4], s[h][5], s[h][6], s[h][7]);
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
    return T <= kOneBlock ? 16 : round16((size_t)E * kMaxBlocks * 2);
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
    // at most 43 KB: E <= 1024, T k <= 2^20
    return launch(place_kernel, blocks, kPlaceThreads, (size_t)(2 * a.E + per * a.k) * 4, st, a, per);
}

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t st) {
    const int chunks = (a.N / 8 + kCombineVecs - 1) / kCombineVecs;
    if (a.N % 8 || (long long)a.T * chunks > 0x7fffffff) {
        const long long want = ((long long)a.T * a.N + 255) / 256, most = (long long)sm_count() * 64;
        return launch(combine1_kernel, (int)(want < most ? want : most), 256, 0, st, a);
    }
    const int grid = a.T * chunks;
    if (a.ybf16) return a.obf16 ? launch(combine8_kernel<true, true>, grid, 256, 0, st, a, chunks)
                                : launch(combine8_kernel<true, false>, grid, 256, 0, st, a, chunks);
    return a.obf16 ? launch(combine8_kernel<false, true>, grid, 256, 0, st, a, chunks)
                   : launch(combine8_kernel<false, false>, grid, 256, 0, st, a, chunks);
}

}  // namespace rq
