// rq_lora.cu -- a low-rank adapter per row beside a shared packed product:
// y[m] = x[m] W^T + s_a B_a (A_a x[m]), a = row_adapter[m].
//
// Up to eight rows the product's own kernels do it (rq_rows.cu): two launches.
// Above, the adapters' term is made beside the product and added in its
// epilogue, in fp32 before the one rounding:
//   shrink_kernel  t = s_a A_a x (a block per eight rows of an adapter and eight
//                  ranks), and the rows' order by adapter
//   expand_kernel  z = B_a t for eight rows x 128 weight rows per block, rows in
//                  adapter order so that a block reads the B of few adapters
// The product starts while expand runs and waits for it only at its end.
// Measured (the whole call): 32 rows of 16 adapters, r 32, w8g16 4096 x 4096,
// 27 MB: 25.5 us; 128 rows of 24, r 64, w4sb32 2560 -> 10240, 40 MB: 45 us (34
// without expand); 1024 rows of 64, r 64, w4g64 4096 x 4096: 106 us. What bounds
// it is the chain of launches ahead of the product's sums, not the bytes.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rq_device.cuh"
#include "rq_internal.h"
#include "rq_rows.cuh"

namespace rq {
namespace {

constexpr int kFewRows = 8;
constexpr int kBlockRows = 1024;       // rows per round of launches
constexpr int kExpandThreads = 128;

// Block (m, j) makes ranks j .. j + 7 of t for row m and the next seven rows of
// the same adapter, if m is the first of such eight: A is read once for them.
// A (8 ranks of the 16-row operand) times x^T on mma.sync, K shared out over
// the warps; a lane loads 16 bytes (8 K) of a rank and of a row, and what is k
// to the instruction is permuted alike in both. The blocks of j = 0 also give
// their row its place in adapter order (rows without an adapter last).
template <int THREADS>
__global__ void __launch_bounds__(THREADS) shrink_kernel(const __grid_constant__ Adapters p, const __nv_bfloat16* x, int R, int* order) {
    constexpr int kWarps = THREADS / 32, kDeep = 1024 / THREADS;
    __shared__ float part[kWarps][64];
    __shared__ unsigned same[kBlockRows / 32];           // rows of the block's adapter
    __shared__ int lower[kWarps], rows[8];
    __shared__ bool first;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = p.r / 8, m = blockIdx.x / per, j = 8 * (blockIdx.x % per);
    if (tid < 8) rows[tid] = -1;
    grid_dep_wait();
    grid_dep_launch();                                   // all work before this call is done
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

__global__ void __launch_bounds__(kExpandThreads) expand_kernel(const __grid_constant__ Adapters p, const int* order, int R, float* z, int ldz) {
    __shared__ float4 scratch[kExpandThreads / 32][64];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_wait();
    grid_dep_launch();
    const int n0 = blockIdx.x * 128 + 32 * warp, i = 8 * blockIdx.y + (lane >> 2);
    if (n0 >= ldz) return;
    const int m = i < R ? order[i] : -1;
    float acc[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    for (int c = 0; 32 * c < p.r; ++c) add_adapters(p, m, c, n0 + (lane >> 2), lane, acc[0], acc[1]);
    // [activation row][weight row], 16-byte chunks swizzled by the row
    float* f = reinterpret_cast<float*>(scratch[warp]);
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = 2 * (lane & 3) + (q & 1), c = 16 * mt + (lane >> 2) + 8 * (q >> 1);
            f[r * 32 + (((c >> 2) ^ r) << 2) + (c & 3)] = acc[mt][q];
        }
    __syncwarp();
    const int r = lane >> 2, n = n0 + 8 * (lane & 3);
    if (m < 0 || n >= ldz) return;
    float4* o = reinterpret_cast<float4*>(z + (size_t)m * ldz + n);
    o[0] = scratch[warp][r * 8 + ((2 * (lane & 3)) ^ r)];
    o[1] = scratch[warp][r * 8 + ((2 * (lane & 3) + 1) ^ r)];
}

template <class K, class... A>
cudaError_t launch(K kernel, dim3 grid, int block, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int ld_of(int N) { return (N + 7) & ~7; }

struct LoraLayout { size_t t, order, z, product, total; };

LoraLayout lora_layout(int fmt, int R, int K, int N, int rank) {
    const int b = R < kBlockRows ? R : kBlockRows;
    LoraLayout l;
    l.t = 0;
    l.order = round16((size_t)b * rank * 4);
    l.z = l.order + round16((size_t)b * 4);
    l.product = l.z + (R > kFewRows ? (size_t)b * ld_of(N) * 4 : 0);
    const size_t narrow = rows_workspace(fmt, b, K, 1), wide = wide_rows(b, 1) ? wide_workspace(b, K, 1) : 0;
    l.total = l.product + (narrow > wide ? narrow : wide);
    return l;
}

}  // namespace

cudaError_t launch_expand(const Adapters& ad, const int* order, int R, float* z, int ldz, cudaStream_t st) {
    return launch(expand_kernel, dim3((unsigned)((ldz + 127) / 128), (unsigned)((R + 7) / 8)), kExpandThreads, st, ad, order, R, z, ldz);
}

size_t lora_workspace(int fmt, int R, int K, int N, int rank) { return lora_layout(fmt, R, K, N, rank).total; }

cudaError_t launch_lora(const RowsArgs& a0, cudaStream_t st) {
    const LoraLayout l = lora_layout(a0.fmt, a0.R, a0.K, a0.N, a0.ad.r);
    uint8_t* ws = static_cast<uint8_t*>(a0.ws);
    for (int m0 = 0; m0 < a0.R; m0 += kBlockRows) {
        RowsArgs a = a0;
        a.R = a.T = a.Ty = a0.R - m0 < kBlockRows ? a0.R - m0 : kBlockRows;
        a.x = static_cast<const __nv_bfloat16*>(a0.x) + (size_t)m0 * a0.K;
        a.y = static_cast<uint8_t*>(a0.y) + (size_t)m0 * a0.N * (a0.ybf16 ? 2 : 4);
        a.ws = ws + l.product;
        a.ad.row = a0.ad.row + m0;
        a.ad.t = reinterpret_cast<float*>(ws + l.t);
        if (a0.R > kFewRows) {
            int* order = reinterpret_cast<int*>(ws + l.order);
            // K over 16 warps where few rows leave SMs idle (32 rows: 25.5 us against 27.0 with 8, 1024: 131 against 103)
            const bool few = a.R <= 128;
            const cudaError_t e = launch(few ? shrink_kernel<512> : shrink_kernel<256>, dim3((unsigned)(a.R * (a.ad.r / 8))), few ? 512 : 256,
                                         st, a.ad, static_cast<const __nv_bfloat16*>(a.x), a.R, order);
            if (e != cudaSuccess) return e;
            a.order = order;
            a.z = reinterpret_cast<float*>(ws + l.z);
            a.ldz = ld_of(a0.N);
        }
        const cudaError_t e = a.ybf16 && wide_rows(a.R, 1) ? launch_wide(a, st) : launch_rows(a, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace rq
