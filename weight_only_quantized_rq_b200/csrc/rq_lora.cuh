// rq_lora.cuh -- the first half of the adapters' term, for the kernels that make
// it above eight rows: t = s_a A_a x, and the rows' order by adapter.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "rq_internal.h"
#include "rq_rows.cuh"

namespace rq {

constexpr int kBlockRows = 1024;       // rows per round of launches

// K over 16 warps where few rows leave SMs idle (32 rows: 25.5 us against 27.0 with 8, 1024: 131 against 103)
inline int shrink_threads(int R) { return R <= 128 ? 512 : 256; }

// Block (m, j) makes ranks j .. j + 7 of t for row m and the next seven rows of
// the same adapter, if m is the first of such eight: A is read once for them.
// A (8 ranks of the 16-row operand) times x^T on mma.sync, K shared out over
// the warps; a lane loads 16 bytes (8 K) of a rank and of a row, and what is k
// to the instruction is permuted alike in both. The blocks of j = 0 also give
// their row its place in adapter order (rows without an adapter last).
template <int THREADS>
__device__ __forceinline__ void shrink_block(const Adapters& p, const __nv_bfloat16* x, int R, int* order, int block) {
    constexpr int kWarps = THREADS / 32, kDeep = 1024 / THREADS;
    __shared__ float part[kWarps][64];
    __shared__ unsigned same[kBlockRows / 32];           // rows of the block's adapter
    __shared__ int lower[kWarps], rows[8];
    __shared__ bool first;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = p.r / 8, m = block / per, j = 8 * (block % per);
    if (tid < 8) rows[tid] = -1;
    auto key = [&](int q) { const int a = p.row[q]; return a >= 0 && a < p.n ? a : 0x7fffffff; };
    const int a = key(m);
    const bool idle = a == 0x7fffffff;
    if (idle && j > 0) return;
    const int own = !idle && p.ranks ? p.ranks[a] : p.r;
    const float alpha = idle ? 0.0f : p.alpha[a];
    int less = 0;
    for (int q0 = 0; q0 < R; q0 += THREADS) {
        const int q = q0 + tid, b = q < R ? key(q) : 0;
        const unsigned eq = __ballot_sync(~0u, q < R && b == a);
        less += __popc(__ballot_sync(~0u, q < R && b < a));
        if (lane == 0) same[(q0 >> 5) + warp] = eq;
    }
    if (lane == 0) lower[warp] = less;
    __syncthreads();
    if (warp == 0) {
        const unsigned w = 32 * lane < R ? same[lane] : 0u;
        const unsigned past = lane < (m >> 5) ? w : lane == (m >> 5) ? w & ((1u << (m & 31)) - 1u) : 0u;
        unsigned from = w & ~past;
        const int before = __reduce_add_sync(~0u, __popc(past));
        int at = __popc(from);
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, at, o);
            if (lane >= o) at += v;
        }
        at -= __popc(from);
        for (; from && at < 8; from &= from - 1) rows[at++] = 32 * lane + __ffs(from) - 1;
        const int l = __reduce_add_sync(~0u, lane < kWarps ? lower[lane] : 0);
        if (lane == 0) {
            first = before % 8 == 0;
            if (j == 0) order[l + before] = m;
        }
    }
    __syncthreads();
    if (idle || !first || j >= own) return;
    const int g = lane >> 2, q = lane & 3, row = rows[g];
    const uint4* xr = reinterpret_cast<const uint4*>(x + (size_t)max(row, 0) * p.K);
    const uint4* ar = reinterpret_cast<const uint4*>(p.A + ((size_t)a * p.r + j + g) * p.K);
    const int nc = p.K / 8;
    float d[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    for (int c0 = 4 * warp; c0 < nc; c0 += 4 * kDeep * kWarps) {
        uint4 u[kDeep], v[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {                // unconditional
            const int c = min(c0 + 4 * kWarps * i + q, nc - 1);
            v[i] = __ldg(ar + c);
            u[i] = __ldg(xr + c);
        }
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const bool in = c0 + 4 * kWarps * i + q < nc;
            const uint32_t lo[4] = {in ? v[i].x : 0u, 0u, in ? v[i].y : 0u, 0u}, hi[4] = {in ? v[i].z : 0u, 0u, in ? v[i].w : 0u, 0u};
            mma16816(d[0], lo, in ? u[i].x : 0u, in ? u[i].y : 0u, d[0][0], d[0][1], d[0][2], d[0][3]);
            mma16816(d[1], hi, in ? u[i].z : 0u, in ? u[i].w : 0u, d[1][0], d[1][1], d[1][2], d[1][3]);
        }
    }
    part[warp][8 * g + 2 * q] = d[0][0] + d[1][0];
    part[warp][8 * g + 2 * q + 1] = d[0][1] + d[1][1];
    __syncthreads();
    if (tid < 64) {
        const int o = rows[tid & 7];
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) t += part[i][tid];
        if (o >= 0) p.t[(size_t)o * p.r + j + (tid >> 3)] = t * alpha;
    }
}

}  // namespace rq
