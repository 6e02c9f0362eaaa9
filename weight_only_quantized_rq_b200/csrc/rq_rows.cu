// rq_rows.cu -- packed products whose weights depend on the activation row:
// products grouped by expert, and low-rank adapters beside a shared packed
// projection.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rq_device.cuh"
#include "rq_internal.h"

namespace rq {
namespace {

// Eight consecutive weights k8 .. k8 + 7 of one packed row, as fp32 (exact for
// the symmetric formats, one rounding of S q - M for the superblocks).
template <int FMT>
__device__ __forceinline__ void w_hat8(const uint8_t* codes, const uint8_t* scales, size_t row, int K, int k8, float (&w)[8]) {
    if constexpr (is_sb(FMT)) {
        constexpr int BITS = sb_bits(FMT);
        const uint8_t* r = codes + (row * (K / 256) + k8 / 256) * sb_record(FMT);
        const uint4 hd = *reinterpret_cast<const uint4*>(r);
        const int kk = k8 % 256, j = kk / 32;
        const float S = __half2float(__ushort_as_half((uint16_t)(hd.x & 0xffffu))) * (float)sb_field(hd.y, hd.z, hd.w, 0, j);
        const float M = __half2float(__ushort_as_half((uint16_t)(hd.x >> 16))) * (float)sb_field(hd.y, hd.z, hd.w, 1, j);
        const uint32_t c = *reinterpret_cast<const uint32_t*>(r + 16 + kk / 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t q = (c >> (4 * i)) & 15u;
            if (BITS == 5) q |= ((r[144 + kk / 8] >> i) & 1u) << 4;
            if (BITS == 6) q |= ((r[144 + kk / 4 + i / 4] >> (2 * (i % 4))) & 3u) << 4;
            w[i] = fmaf(S, (float)q, -M);
        }
    } else {
        constexpr int G = sym_group(FMT);
        const float s = __half2float(reinterpret_cast<const __half*>(scales)[row * (K / G) + k8 / G]);
        if constexpr (FMT == kFmtW4G64) {
            const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + (row * K + k8) / 2);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = s * (float)((int)((c >> (4 * i)) & 15u) - 8);
        } else if constexpr (FMT == kFmtW6G16) {
            const uint8_t* r = codes + (row * (K / 64) + k8 / 64) * 48;
            const int kk = k8 % 64;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int q = ((r[(kk + i) / 2] >> (4 * (i & 1))) & 15) | (((r[32 + (kk + i) / 4] >> (2 * (i % 4))) & 3) << 4);
                w[i] = s * (float)(q - 32);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = s * (float)((int)codes[row * K + k8 + i] - 128);
        }
    }
}

// t[m][j] = scale_a * (x[m] . A_a[j]): one warp per (m, j).
__global__ void shrink_kernel(RowsArgs a) {
    const int j = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), m = blockIdx.y, lane = threadIdx.x & 31;
    const int ad = a.adapter[m];
    if (j >= a.r || ad < 0 || ad >= a.n_adapters || (a.ranks && j >= a.ranks[ad])) return;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + (size_t)m * a.K;
    const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(a.A) + ((size_t)ad * a.r + j) * a.K;
    float s = 0.0f;
    for (int k = lane; k < a.K; k += 32) s = fmaf(__bfloat162float(x[k]), __bfloat162float(A[k]), s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (lane == 0) static_cast<float*>(a.ws)[(size_t)m * a.r + j] = s * a.alpha[ad];
}

// One warp per packed row (one output feature of one expert), eight
// activation rows of the group at a time.
template <int FMT>
__global__ void rows_kernel(RowsArgs a) {
    const size_t row = (size_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (size_t)a.E * a.N) return;
    const int e = (int)(row / a.N), n = (int)(row % a.N);
    int o0 = 0, o1 = a.R;
    if (a.offsets) {                                     // the running maximum keeps any offsets in order and in range
        for (int i = 0; i <= e; ++i) o0 = max(o0, min(a.offsets[i], a.R));
        o1 = max(o0, min(a.offsets[e + 1], a.R));
    }
    const uint8_t* codes = static_cast<const uint8_t*>(a.codes);
    const uint8_t* scales = static_cast<const uint8_t*>(a.scales);
    for (int i0 = o0; i0 < o1; i0 += 8) {
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const __nv_bfloat16* xr[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i0 + i < o1 ? (a.in_rows ? a.in_rows[i0 + i] : i0 + i) : -1;
            xr[i] = r >= 0 && r < a.T ? static_cast<const __nv_bfloat16*>(a.x) + (size_t)r * a.K : nullptr;
        }
        for (int k8 = 8 * lane; k8 < a.K; k8 += 256) {
            float w[8];
            w_hat8<FMT>(codes, scales, row, a.K, k8, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!xr[i]) continue;
                const uint4 v = *reinterpret_cast<const uint4*>(xr[i] + k8);
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i] = fmaf(w[2 * j], bf16lo_f32(u[j]), acc[i]);
                    acc[i] = fmaf(w[2 * j + 1], bf16hi_f32(u[j]), acc[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            for (int o = 16; o; o >>= 1) acc[i] += __shfl_xor_sync(~0u, acc[i], o);
            if (lane != 0 || i0 + i >= o1) continue;
            const int m = i0 + i;
            float v = acc[i];
            if (a.adapter) {
                const int ad = a.adapter[m];
                if (ad >= 0 && ad < a.n_adapters) {
                    const int rank = a.ranks ? min(a.ranks[ad], a.r) : a.r;
                    const __nv_bfloat16* B = static_cast<const __nv_bfloat16*>(a.B) + ((size_t)ad * a.N + n) * a.r;
                    float s = 0.0f;
                    for (int j = 0; j < rank; ++j) s = fmaf(static_cast<float*>(a.ws)[(size_t)m * a.r + j], __bfloat162float(B[j]), s);
                    v += s;
                }
            }
            if (a.act == 1) { v = v > 0.0f || v != v ? v : 0.0f; v *= v; }
            const int out = a.out_rows ? a.out_rows[m] : m;
            if (out >= 0 && out < a.Ty) store_y(a.y, (size_t)out * a.N + n, v, a.ybf16);
        }
    }
}

}  // namespace

size_t rows_workspace(int, int R, int, int, int, int rank) { return round16((size_t)R * rank * 4) + 16; }

cudaError_t launch_rows(const RowsArgs& a, cudaStream_t st) {
    if (a.adapter) shrink_kernel<<<dim3((a.r + 7) / 8, a.R), 256, 0, st>>>(a);
    const unsigned grid = (unsigned)(((size_t)a.E * a.N + 7) / 8);
    switch (a.fmt) {
        case kFmtW4G64: rows_kernel<kFmtW4G64><<<grid, 256, 0, st>>>(a); break;
        case kFmtW8G16: rows_kernel<kFmtW8G16><<<grid, 256, 0, st>>>(a); break;
        case kFmtW8G64: rows_kernel<kFmtW8G64><<<grid, 256, 0, st>>>(a); break;
        case kFmtW6G16: rows_kernel<kFmtW6G16><<<grid, 256, 0, st>>>(a); break;
        case kFmtW4SB32: rows_kernel<kFmtW4SB32><<<grid, 256, 0, st>>>(a); break;
        case kFmtW5SB32: rows_kernel<kFmtW5SB32><<<grid, 256, 0, st>>>(a); break;
        default: rows_kernel<kFmtW6SB32><<<grid, 256, 0, st>>>(a); break;
    }
    return cudaGetLastError();
}

}  // namespace rq
