// rq_rows.cuh -- what the kernels of the row-dependent products share: the
// mma.sync wrapper and the low-rank adapters' two halves.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rq_device.cuh"
#include "rq_internal.h"

namespace rq {

// D = A B + C, A 16 x 16 (row), B 16 x 8 (col), bf16 with fp32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1,
                                         float c2, float c3) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// fp32 pair -> bf16x2 (nearest even), lo in the low half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// fp32 pair -> bf16x2, cut off towards zero.
__device__ __forceinline__ uint32_t cut2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// t[m][j .. j + 7] = alpha A . x[m] by a block of WARPS warps that share out K,
// so that each lane has one load of x and eight of A in flight per round. Ranks
// past the slot's are not read.
template <int WARPS>
__device__ __forceinline__ void shrink8(const Adapters& p, const __nv_bfloat16* xs, int m, int j, float (&part)[WARPS][8]) {
    const int a = p.row[m], lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (a < 0 || a >= p.n) return;                       // the same for the whole block
    if (p.ranks && j >= p.ranks[a]) return;
    const uint4* x = reinterpret_cast<const uint4*>(xs + (size_t)m * p.K);
    const uint4* w = reinterpret_cast<const uint4*>(p.A + ((size_t)a * p.r + j) * p.K);
    const int nc = p.K / 8;
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = 32 * warp + lane; c < nc; c += 32 * WARPS) {
        const uint4 u = x[c];
        uint4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = __ldg(w + (size_t)q * nc + c);
        const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint32_t vv[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[q] = fmaf(bf16lo_f32(uu[i]), bf16lo_f32(vv[i]), s[q]);
                s[q] = fmaf(bf16hi_f32(uu[i]), bf16hi_f32(vv[i]), s[q]);
            }
        }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
#pragma unroll
        for (int o = 16; o; o >>= 1) s[q] += __shfl_xor_sync(~0u, s[q], o);
    if (lane == 0)
#pragma unroll
        for (int q = 0; q < 8; ++q) part[warp][q] = s[q];
    __syncthreads();
    if (threadIdx.x < 8) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) t += part[i][threadIdx.x];
        p.t[(size_t)m * p.r + j + threadIdx.x] = t * p.alpha[a];
    }
}

// Adds the adapters' term over ranks 32 c .. 32 c + 31 to one 8-row tile's
// sums: for each adapter among the tile's rows D = B_a t^T with t zero for the
// other rows, and D added to the adapter's own rows only (an infinite or NaN
// B_a stays with them). t is split into three bf16 parts (24 bits), so that nothing
// of it is lost to the tensor core's operand type; the first is cut off, so that
// a finite t keeps a finite one. The lower parts have sums of their own, which
// count where the first part's is finite: where t or B is infinite, they, zero or
// of the other sign, would make NaN of the formula's infinity. Lane 4 g + q holds ranks
// 8 q .. 8 q + 7 of the chunk: of weight rows n + 8 i (i = 0..3) and of
// activation row g, which is row m of the call (negative: none).
__device__ __forceinline__ void add_adapters(const Adapters& p, int m, int c, int n, int lane, float (&acc0)[4], float (&acc1)[4]) {
    const int j0 = 32 * c + 8 * (lane & 3);
    int a = -1, rank = 0;
    if (m >= 0) {
        a = p.row[m];
        if (a >= 0 && a < p.n) rank = p.ranks ? min(p.ranks[a], p.r) : p.r;
        if (rank <= 32 * c) a = -1;
    }
    uint32_t t[3][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float2 v = make_float2(0.0f, 0.0f);
        if (a >= 0 && j0 + 2 * q < rank) {
            v = *reinterpret_cast<const float2*>(p.t + (size_t)m * p.r + j0 + 2 * q);
            if (j0 + 2 * q + 1 >= rank) v.y = 0.0f;
        }
        t[0][q] = cut2(v.x, v.y);
        v.x -= bf16lo_f32(t[0][q]);
        v.y -= bf16hi_f32(t[0][q]);
        t[1][q] = pack2(v.x, v.y);
        v.x -= bf16lo_f32(t[1][q]);
        v.y -= bf16hi_f32(t[1][q]);
        t[2][q] = pack2(v.x, v.y);
    }
    unsigned todo = __ballot_sync(~0u, a >= 0);
    while (todo) {
        const int src = __ffs(todo) - 1, aa = __shfl_sync(~0u, a, src), rk = __shfl_sync(~0u, rank, src);
        const bool same = a == aa;
        const unsigned with = __ballot_sync(~0u, same);
        todo &= ~with;
        uint4 b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            b[q] = make_uint4(0u, 0u, 0u, 0u);
            if (j0 < rk) b[q] = __ldg(reinterpret_cast<const uint4*>(p.B + ((size_t)aa * p.N + min(n + 8 * q, p.N - 1)) * p.r + j0));
            const int keep = rk - j0;                    // past the rank the slot may hold anything
            if (keep < 8) {
                const auto cut = [&](uint32_t w, int k) { return k + 1 < keep ? w : k < keep ? w & 0xffffu : 0u; };
                b[q] = make_uint4(cut(b[q].x, 0), cut(b[q].y, 2), cut(b[q].z, 4), cut(b[q].w, 6));
            }
        }
        float d[2][2][4];                                // [first part, lower parts][weight rows n + 16 i]
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            const uint32_t t0 = same ? t[s][0] : 0u, t1 = same ? t[s][1] : 0u, t2 = same ? t[s][2] : 0u, t3 = same ? t[s][3] : 0u;
            const uint32_t a0[4] = {b[0].x, b[1].x, b[0].y, b[1].y}, a1[4] = {b[2].x, b[3].x, b[2].y, b[3].y};
            const uint32_t a2[4] = {b[0].z, b[1].z, b[0].w, b[1].w}, a3[4] = {b[2].z, b[3].z, b[2].w, b[3].w};
            auto& e = d[s > 0];
            if (s < 2) {
                mma16816(e[0], a0, t0, t1, 0.0f, 0.0f, 0.0f, 0.0f);
                mma16816(e[1], a1, t0, t1, 0.0f, 0.0f, 0.0f, 0.0f);
            } else {
                mma16816(e[0], a0, t0, t1, e[0][0], e[0][1], e[0][2], e[0][3]);
                mma16816(e[1], a1, t0, t1, e[1][0], e[1][1], e[1][2], e[1][3]);
            }
            mma16816(e[0], a2, t2, t3, e[0][0], e[0][1], e[0][2], e[0][3]);
            mma16816(e[1], a3, t2, t3, e[1][0], e[1][1], e[1][2], e[1][3]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {                    // columns: activation rows 2 (lane & 3) + (i & 1)
            const bool own = with >> (4 * (2 * (lane & 3) + (i & 1))) & 1u;
            const auto sum = [&](int h) { return d[0][h][i] + (fabsf(d[0][h][i]) < INFINITY ? d[1][h][i] : 0.0f); };
            acc0[i] += own ? sum(0) : 0.0f;
            acc1[i] += own ? sum(1) : 0.0f;
        }
    }
}

}  // namespace rq
