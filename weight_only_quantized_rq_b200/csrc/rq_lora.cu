// rq_lora.cu -- a low-rank adapter per row beside a shared packed product:
// y[m] = x[m] W^T + s_a B_a (A_a x[m]), a = row_adapter[m].
//
// Up to eight rows the product's own kernels do it (rq_rows.cu): two launches.
// Above, the adapters' term is made beside the product and added in its
// epilogue, in fp32 before the one rounding:
//   shrink         t = s_a A_a x (a block per eight rows of an adapter and eight
//                  ranks), and the rows' order by adapter: a launch of its own, or
//                  in one with the rows' layout (rq_wide.cu)
//   expand_kernel  z = B_a t for eight rows x 128 weight rows per block, rows in
//                  adapter order so that a block reads the B of few adapters
// The product starts while expand runs and waits for it only at its end.
// Shrink and layout in one launch instead of two: 128 rows 45.5 -> 44.1 us, 1024
// rows of 8 adapters 72 -> 67, but 32 rows 26.0 -> 26.8.
// Measured (the whole call): 32 rows of 16 adapters, r 32, w8g16 4096 x 4096,
// 27 MB: 27 us; 128 rows of 24, r 64, w4sb32 2560 -> 10240, 40 MB: 45 us (33
// without expand); 1024 rows of 64, r 64, w4g64 4096 x 4096: 104 us. What bounds
// it is the chain of launches ahead of the product's sums, not the bytes.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rq_device.cuh"
#include "rq_internal.h"
#include "rq_lora.cuh"
#include "rq_rows.cuh"

namespace rq {
namespace {

constexpr int kFewRows = 8;
constexpr int kExpandThreads = 128;

template <int THREADS>
__global__ void __launch_bounds__(THREADS) shrink_kernel(const __grid_constant__ Adapters p, const __nv_bfloat16* x, int R, int* order) {
    grid_dep_wait();
    grid_dep_launch();                                   // all work before this call is done
    shrink_block<THREADS>(p, x, R, order, blockIdx.x);
}

__global__ void __launch_bounds__(kExpandThreads, 7) expand_kernel(const __grid_constant__ Adapters p, const int* order, int R, float* z, int ldz) {
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
    const bool wide = a0.ybf16 && wide_rows(a0.R, 1);    // of the call, not of a round: a short last round is multiplied as the others
    for (int m0 = 0; m0 < a0.R; m0 += kBlockRows) {
        RowsArgs a = a0;
        a.R = a.T = a.Ty = a0.R - m0 < kBlockRows ? a0.R - m0 : kBlockRows;
        a.x = static_cast<const __nv_bfloat16*>(a0.x) + (size_t)m0 * a0.K;
        a.y = static_cast<uint8_t*>(a0.y) + (size_t)m0 * a0.N * (a0.ybf16 ? 2 : 4);
        a.ws = ws + l.product;
        a.ad.row = a0.ad.row + m0;
        a.ad.t = reinterpret_cast<float*>(ws + l.t);
        if (a0.R > kFewRows) {
            a.order = reinterpret_cast<int*>(ws + l.order);
            if (!wide) {
                const bool few = shrink_threads(a.R) == 512;
                const cudaError_t e = launch(few ? shrink_kernel<512> : shrink_kernel<256>, dim3((unsigned)(a.R * (a.ad.r / 8))), few ? 512 : 256,
                                             st, a.ad, static_cast<const __nv_bfloat16*>(a.x), a.R, a.order);
                if (e != cudaSuccess) return e;
            }
            a.z = reinterpret_cast<float*>(ws + l.z);
            a.ldz = ld_of(a0.N);
        }
        const cudaError_t e = wide ? launch_wide(a, st) : launch_rows(a, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace rq
