// rq_wide.cu -- the grouped products for groups of many rows (prompts), on the
// 5th-generation tensor cores: y[i] = act(x[in(i)] W_e^T) with bf16 results.
//
// lay_rows_kernel gathers the rows into group order as fp16 under a power of
// two per row (the largest value in [2^14, 2^15); bf16 values are exact there
// down to 2^-31 of the row's largest), in the order in which the codes unpack.
// wide_kernel multiplies:
//   * A unit is 256 weight rows x K x up to MC activation rows of one expert:
//     two tiles of 128 weight rows that share the activations. tcgen05.mma takes
//     the weights from tensor memory (A) and the activations from shared memory
//     (B); the fp32 sums stay in tensor memory until the unit's end. Two tiles
//     of weights and 128 rows beat one tile and 256 rows (the same sums): the
//     weights are the narrow operand, so a CTA fetches 24 instead of 36 KB per
//     64 K, and it was the fetching that bound it.
//   * Sixteen warps unpack: a thread owns one weight row of a tile (its
//     tensor-memory lane) and half of its K. A weight is q s rounded once to
//     fp16 (half a step, 2^-11 of it, an eighth of the result's own rounding to
//     bf16; q s is a multiple of 2^-24, so that small ones are exact); fp16
//     instead of bf16 for both operands buys that. The superblocks' weights are
//     within 2^-10 (|w| + |w(c)|), w(c) the group's weight of the middle code
//     (unpack_atom). Scales under which a code could pass fp16's 65504 are seen
//     while unpacking; such a row's sums are made again in fp32 (exact_sums).
//   * Units are cut where an even share of the work (rows x K) ends, so every
//     CTA (one per SM) has the same; a cut unit's parts are summed through the
//     workspace in K order by whichever CTA arrives last.
// Measured: 4096 rows of 8 experts, w4g64, K 2048, N 8192: 173 us back to back, 794
// TFLOP/s (195 with other work between the calls, 705); w4sb32 183, w6sb32 215.
// A unit takes 11.7 us of products, 1.4 to drain, 3.1 to move its sums out;
// without the last 150 us. An MMA of 128 x 128 x 16 takes 97 cycles where the
// pipe's rate gives 64; 90 of them are its own (nothing unpacked or stored to
// tensor memory beside it: 90), the rest is what unpacking adds. Not kept: the
// next unit's first stages unpacked before the sums move out (185 us), sums
// stored 16 bytes at a time through more shuffles (176).
// Roles: 16 unpacking warps (they also move the sums out), a warp per weight
// tile that issues its MMAs (one warp alone issued for 380 of the 256 cycles
// that the products of an atom take), one thread that copies codes and one
// that copies rows.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rq_device.cuh"
#include "rq_internal.h"
#include "rq_lora.cuh"
#include "rq_rows.cuh"
#include "rq_tc.cuh"

namespace rq {
namespace {

constexpr int kWorkers = 16;
constexpr int kTiles = 2;               // weight tiles of a unit; warps 8 t .. 8 t + 7 unpack tile t, four of them
                                        // the first 64 of each 128 K, four the others
constexpr int kUnitRows = kTiles * kTcRows;
constexpr int kWideThreads = 32 * (kWorkers + 4);
constexpr int kMaxX = 4;                // activation slots at most (128 K each)
constexpr int kMaxCodes = 4;            // code slots at most
constexpr int kDescs = 8;
constexpr size_t kWideSmem = 227 * 1024;
constexpr int kWideMaxCtas = 256;
constexpr int kOverBytes = 2 * kUnitRows * 2;
constexpr int kA = 4;                   // A slots: 128 K of one tile, 64 columns
constexpr int kBarBytes = (2 * kMaxCodes + 2 * kMaxX + 2 * kA + kDescs + 4 * 2 + 3) * 8;

template <int FMT>
struct Wide {
    static constexpr int KS = is_w8(FMT) || FMT == kFmtW6G16 ? 128 : 256;         // K per code slot
    static constexpr int RB = FMT == kFmtW4G64 || is_w8(FMT) ? 128 : FMT == kFmtW6G16 ? 96 : sb_record(FMT);
    static constexpr int CB = (kUnitRows * RB + 1023) & ~1023;
    static constexpr int PAIRS = KS / 128;                                        // 128-K steps of a stage
    // order of a row's values: within 8 (1: 0 4 1 5 2 6 3 7) or within 4 (2: 0 2 1 3)
    static constexpr int ORDER = is_w8(FMT) ? 2 : 1;
};

struct WidePlan {
    const int* offsets;                 // NULL: one group of all rows
    int E, R, N, K, T, MC;
};

struct WideParams {
    CUtensorMap cmap;                   // codes: uint8 [E N][row bytes], box [256][RB]
    CUtensorMap xmap;                   // rows: fp16 [R][K] viewed as [K / 64][R][64], box [1][32][64]
    WidePlan pl;
    const uint8_t* codes;
    const uint8_t* scales;
    unsigned long long total_rows;
    uint32_t crb, srb;                  // code and scale bytes per weight row
    const uint4* xg;                    // the laid-out rows
    const float* rscale;                // [R] inverse of a row's power of two
    float* part;                        // partial tiles, two per CTA
    unsigned* count;                    // stages summed of a cut unit, by its first CTA and warp
    const int* out_rows;
    void* y;
    int Ty, act;
    const float* z;                     // [R][ldz] the adapters' term, or NULL
    int ldz;
    int xslots, cslots, over_at;
    unsigned long long wait_ns;
    int test_flags;
};

// ------------------------------------------------------------------- rows
constexpr int kLayThreads = 256;

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight bf16 values under the power of two f, as fp16 in the order that the codes unpack in.
template <int ORDER>
__device__ __forceinline__ uint4 lay8(uint4 v, float f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = half2_bits(bf16lo_f32(w[i]) * f, bf16hi_f32(w[i]) * f);
    if (ORDER == 1) return make_uint4(prmt(h[0], h[2], 0x5410u), prmt(h[0], h[2], 0x7632u), prmt(h[1], h[3], 0x5410u), prmt(h[1], h[3], 0x7632u));
    return make_uint4(prmt(h[0], h[1], 0x5410u), prmt(h[0], h[1], 0x7632u), prmt(h[2], h[3], 0x5410u), prmt(h[2], h[3], 0x7632u));
}
__device__ __forceinline__ uint32_t top8(uint4 v) {
    const uint32_t m = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
}

struct LayParams {
    const __nv_bfloat16* x;
    const int* in_rows;
    int rows_x, K;
    uint4* out;
    float* rscale;
    unsigned* count;
    int n_count;
};

// One block per row: the largest exponent, then the row under its power of
// two. Rows of up to 32 THREADS values stay in registers between the two.
template <int ORDER, int THREADS>
__device__ __forceinline__ void lay_row(const LayParams& l, int row) {
    __shared__ uint32_t tops[THREADS / 32];
    const int tid = threadIdx.x, K = l.K;
    if (row == 0)
        for (int i = tid; i < l.n_count; i += THREADS) l.count[i] = 0u;
    int src = l.in_rows ? l.in_rows[row] : row;
    if (src < 0 || src >= l.rows_x) src = -1;
    const uint4* p = reinterpret_cast<const uint4*>(l.x + (size_t)(src < 0 ? 0 : src) * K);
    const int nc = src < 0 ? 0 : K / 8;
    constexpr int KEEP = 4;
    uint4 v[KEEP];
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
        const int c = tid + i * THREADS;
        v[i] = c < nc ? p[c] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < KEEP; ++i) top = __vmaxu2(top, top8(v[i]));
    for (int c = tid + KEEP * THREADS; c < nc; c += THREADS) top = __vmaxu2(top, top8(p[c]));
    top = max(top & 0xffffu, top >> 16);
    top = __reduce_max_sync(~0u, top);
    if ((tid & 31) == 0) tops[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) top = max(top, tops[i]);
    // biased exponent of the largest value; 255 (not finite) as 254, so that no finite value beside it becomes infinite
    const int ex = min(254, (int)(top >> 7));
    const int sh = top ? max(-126, min(126, 141 - ex)) : 0;
    const float f = __uint_as_float((uint32_t)(127 + sh) << 23);
    if (tid == 0) l.rscale[row] = __uint_as_float((uint32_t)(127 - sh) << 23);
    uint4* o = l.out + (size_t)row * (K / 8);
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
        const int c = tid + i * THREADS;
        if (c < K / 8) o[c] = lay8<ORDER>(v[i], f);
    }
    for (int c = tid + KEEP * THREADS; c < K / 8; c += THREADS) o[c] = lay8<ORDER>(c < nc ? p[c] : make_uint4(0u, 0u, 0u, 0u), f);
}

template <int ORDER>
__global__ void __launch_bounds__(kLayThreads) lay_rows_kernel(const __grid_constant__ LayParams l) {
    grid_dep_wait();
    grid_dep_launch();
    lay_row<ORDER, kLayThreads>(l, blockIdx.x);
}

// With adapters: their first product's blocks, then the rows'.
template <int ORDER, int THREADS>
__global__ void __launch_bounds__(THREADS) lay_shrink_kernel(const __grid_constant__ LayParams l, const __grid_constant__ Adapters ad, int R, int* order) {
    grid_dep_wait();
    grid_dep_launch();
    const int n = R * (ad.r / 8), b = blockIdx.x;
    if (b < n) shrink_block<THREADS>(ad, l.x, R, order, b);
    else lay_row<ORDER, THREADS>(l, b - n);
}

// ------------------------------------------------------------------ groups
// Per expert: first row, and the cost of all K stages before it. An expert's
// rows are cut into equal chunks (a multiple of 16 rows, at most MC).
struct WGroups {
    long long* cost;   // [E + 1]
    int* row;          // [E + 1]
    int* ctas;         // CTAs that share the work
};
__host__ __device__ inline size_t wgroups_bytes(int E) { return round16((size_t)(E + 1) * 12 + 4); }

__device__ __forceinline__ int chunk_rows(int m, int MC) {
    const int c = (m + MC - 1) / MC;
    return c ? ((m + c - 1) / c + 15) & ~15 : 16;
}
// Cost of a stage: the rows that the tensor cores multiply, at least what
// unpacking takes.
__device__ __forceinline__ int stage_cost(int rows) { return max(rows, 96); }

__device__ __forceinline__ void scan_wide(const WidePlan& pl, WGroups g, int lane) {
    const int tiles_n = (pl.N + kUnitRows - 1) / kUnitRows;
    int top = 0;
    long long base = 0, units = 0;
    for (int e0 = 0; e0 <= pl.E; e0 += 32) {
        const int e = e0 + lane;
        int v = 0;
        if (pl.offsets) v = e <= pl.E ? min(max(pl.offsets[e], 0), pl.R) : 0;
        else v = e >= 1 ? pl.R : 0;                       // one group of all rows
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(~0u, v, o);
            if (lane >= o) v = max(v, w);
        }
        v = max(v, top);
        const int prev = __shfl_up_sync(~0u, v, 1);
        const int m = lane == 0 ? (e0 ? v - top : 0) : v - prev;       // rows of group e - 1
        const int rc = chunk_rows(m, pl.MC);
        long long un = (long long)((m + rc - 1) / rc) * tiles_n, c = un * pl.T * stage_cost(rc);
        for (int o = 1; o < 32; o <<= 1) {
            const long long b = __shfl_up_sync(~0u, c, o), n = __shfl_up_sync(~0u, un, o);
            if (lane >= o) {
                c += b;
                un += n;
            }
        }
        if (e <= pl.E) {
            g.row[e] = v;
            g.cost[e] = base + c;
        }
        top = __shfl_sync(~0u, v, 31);
        base += __shfl_sync(~0u, c, 31);
        units += __shfl_sync(~0u, un, 31);
    }
    // A unit's K loop takes about 0.65 us per 128 K, and summing the parts of a cut unit 0.5 us per part and 2.5 more
    // per 128 rows. Units that do not fill the SMs are either cut into p equal parts each (p = the root of the two's
    // ratio, as far as there are SMs), or shared out evenly over all SMs, most of which then have parts of two units to
    // sum (4 us more). 80 units of 10 stages: whole 50.0, in even shares 57.7 us.
    if (lane == 0) {
        const float loop = 0.65f * (float)((pl.K + 127) / 128), part = 0.5f + 2.5f / 128.0f * (float)min(pl.MC, (top + pl.E - 1) / pl.E);
        const int G = (int)gridDim.x;
        int ctas = G;
        if (units < G) {
            const int p = max(1, min(G / (int)max(units, 1ll), (int)(sqrtf(loop / part) + 0.5f)));
            const float even = (float)G / (float)max(units, 1ll);        // parts of a unit in even shares
            if (loop / (float)p + (p > 1 ? part * (float)p : 0.0f) < loop / even + part * (even + 1.0f) + 4.0f) ctas = max(1, (int)units * p);
        }
        *g.ctas = ctas;
    }
    __syncwarp();
}

// A stretch of a unit in one CTA.
struct __align__(16) WDesc {
    int done;          // no more work
    int row0, rows;    // rows of the call
    int n0, wrow;      // first weight row within the expert, and in the plane
    int k0, k1;        // stages
    int first, last;   // CTAs that share the unit
    int cost;          // of a stage
    long long pos;     // cost position of the unit's first stage
};

__device__ __forceinline__ long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Walks a CTA's stretches: cost positions [ceil(b W / G), ceil((b + 1) W / G)).
struct Walk {
    const WidePlan& pl;
    const WGroups& g;
    long long W, Gc, P1, w, st, stages;                  // w: cost of a stage of expert e, st: its next stage
    int e, m, rc, chunks;
    bool live;

    __device__ __forceinline__ Walk(const WidePlan& plan, const WGroups& groups) : pl(plan), g(groups) {
        W = g.cost[pl.E];
        Gc = *g.ctas;
        const long long P0 = ceil_div(blockIdx.x * W, Gc);
        P1 = ceil_div((blockIdx.x + 1) * W, Gc);
        live = blockIdx.x < Gc && P0 < P1;
        if (!live) return;
        int lo = 0, hi = pl.E - 1;                       // last expert whose first position is at most P0
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (g.cost[mid] <= P0) lo = mid;
            else hi = mid - 1;
        }
        enter(lo);
        st = ceil_div(P0 - g.cost[e], w);
    }
    __device__ __forceinline__ void enter(int expert) {
        e = expert;
        m = g.row[e + 1] - g.row[e];
        rc = chunk_rows(m, pl.MC);
        chunks = (m + rc - 1) / rc;
        w = stage_cost(rc);
        stages = (g.cost[e + 1] - g.cost[e]) / w;
    }
    __device__ __forceinline__ bool next(WDesc& d) {
        if (!live) return false;
        while (st >= stages && e + 1 < pl.E) {           // to the next expert with rows
            enter(e + 1);
            st = 0;
        }
        const long long pos = g.cost[e] + st * w;
        if (st >= stages || pos >= P1) return live = false;
        const int T = pl.T;
        const long long unit = st / T;
        const int nt = (int)(unit / chunks), c = (int)(unit - (long long)nt * chunks);
        d.done = 0;
        d.row0 = g.row[e] + c * rc;
        d.rows = min(rc, m - c * rc);
        d.n0 = nt * kUnitRows;
        d.wrow = e * pl.N + d.n0;
        d.k0 = (int)(st - unit * T);
        d.k1 = (int)min((long long)T, d.k0 + ceil_div(P1 - pos, w));
        d.cost = (int)w;
        d.pos = g.cost[e] + unit * T * w;
        d.first = d.k0 > 0 ? (int)(d.pos * Gc / W) : (int)blockIdx.x;
        d.last = d.k1 < T ? (int)((d.pos + (T - 1) * w) * Gc / W) : (int)blockIdx.x;
        st = unit * T + d.k1;
        return true;
    }
};

// An activation row at the end of a unit: where it goes (NULL: nowhere), its
// power of two as fp32, and what the stored bf16 pairs are multiplied by.
struct __align__(16) RowInfo {
    __nv_bfloat16* y;
    float scale;
    uint32_t scale2;
};

// ------------------------------------------------------------------ unpack
__device__ __forceinline__ uint32_t h2(uint16_t v) { return (uint32_t)v * 0x10001u; }
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) { uint32_t d; asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b)); return d; }
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) { uint32_t d; asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b)); return d; }
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// (v & m) | c
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t m, uint32_t c) { return lop_mask_or(v, m, c); }
__device__ __forceinline__ uint4 lds4(uint32_t a) { return lds128_a(a); }

// Largest magnitude (as bits) of four fp16 scales.
__device__ __forceinline__ uint32_t top_scale(const uint32_t (&sc)[2]) {
    const uint32_t m = __vmaxu2(sc[0] & 0x7fff7fffu, sc[1] & 0x7fff7fffu);
    return max(m & 0xffffu, m >> 16);
}

// 64 weights of the thread's row in an atom -> 32 fp16 pairs. cs: the row's
// bytes of the slot; at: atom of the slot; sc: its scale words (two fp16
// each); sw: swizzle of 16-byte chunks (row % 8, or 0). True if a code under
// these scales could pass 65504 (0x7BFF; a power of two of codes less, as many
// exponents less).
template <int FMT>
__device__ __forceinline__ bool unpack_atom(uint32_t cs, int at, int sw, const uint32_t (&sc)[2], uint32_t (&o)[32]) {
    if constexpr (FMT == kFmtW4G64) {
        // (1024 + u) - 1032 and (1024 + 16 u) / 16 - 72 give q exactly; q s is rounded once
        const uint4 c0 = lds4(cs + (((2 * at) ^ sw) << 4)), c1 = lds4(cs + (((2 * at + 1) ^ sw) << 4));
        const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const uint32_t s = h2((uint16_t)(sc[0] & 0xffffu));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t v = w[i] >> 8;
            o[4 * i + 0] = hmul2(hadd2(and_or(w[i], 0x000F000Fu, 0x64006400u), 0xE408E408u), s);
            o[4 * i + 1] = hmul2(hfma2(and_or(w[i], 0x00F000F0u, 0x64006400u), 0x2C002C00u, 0xD480D480u), s);
            o[4 * i + 2] = hmul2(hadd2(and_or(v, 0x000F000Fu, 0x64006400u), 0xE408E408u), s);
            o[4 * i + 3] = hmul2(hfma2(and_or(v, 0x00F000F0u, 0x64006400u), 0x2C002C00u, 0xD480D480u), s);
        }
        return (sc[0] & 0x7fffu) > 0x7BFFu - 3 * 0x400;
    } else if constexpr (is_w8(FMT)) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 v = lds4(cs + (((4 * at + c) ^ sw) << 4));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            const uint32_t s = FMT == kFmtW8G64 ? h2((uint16_t)(sc[0] & 0xffffu)) : h2((uint16_t)(c & 1 ? sc[c >> 1] >> 16 : sc[c >> 1] & 0xffffu));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[8 * c + 2 * i] = hmul2(hadd2(and_or(w[i], 0x00FF00FFu, 0x64006400u), 0xE480E480u), s);        // - 1152
                o[8 * c + 2 * i + 1] = hmul2(hadd2(and_or(w[i] >> 8, 0x00FF00FFu, 0x64006400u), 0xE480E480u), s);
            }
        }
        return top_scale(sc) > 0x7BFFu - 7 * 0x400;
    } else if constexpr (FMT == kFmtW6G16) {
        const uint4 c0 = lds4(cs + 48 * at), c1 = lds4(cs + 48 * at + 16), pl = lds4(cs + 48 * at + 32);
        const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w}, p[4] = {pl.x, pl.y, pl.z, pl.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t ph = (p[i >> 1] >> (16 * (i & 1))) & 0xffffu, h = ph | (ph << 8);
            const uint32_t s = h2((uint16_t)((i >> 1) & 1 ? sc[i >> 2] >> 16 : sc[i >> 2] & 0xffffu));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t hs = q < 2 ? h << (4 - 2 * q) : h >> (2 * q - 4);
                const uint32_t u = and_or(hs, 0x00300030u, and_or(w[i] >> (4 * q), 0x000F000Fu, 0x64006400u));
                o[4 * i + q] = hmul2(hadd2(u, 0xE420E420u), s);                                                // - 1056
            }
        }
        return top_scale(sc) > 0x7BFFu - 5 * 0x400;
    } else {
        // v = u - c exactly (c = 2^(B - 1)), then S v + (c S - M) in one step, S = d sc and c S - M rounded to fp16 (half a
        // step, 2^-11, each): within 2^-11 (S |v| + |c S - M| + |w|) <= 2^-10 (|w| + |c S - M|). Subtracting M from S u
        // instead would leave 2^-11 of both parts where they cancel. In fp32 with one rounding: 4096 rows of 8 experts,
        // K 2048, N 8192, w4sb32 178 -> 200 us, w6sb32 217 -> 260.
        constexpr float C = (float)(1 << (sb_bits(FMT) - 1));
        bool over = false;
        const uint4 hd = lds4(cs);
        const float d = __half2float(__ushort_as_half((uint16_t)(hd.x & 0xffffu)));
        const float dm = __half2float(__ushort_as_half((uint16_t)(hd.x >> 16)));
#pragma unroll
        for (int gl = 0; gl < 2; ++gl) {
            const int j = 2 * at + gl;
            const float s = d * (float)sb_field(hd.y, hd.z, hd.w, 0, j);
            const __half sh = __float2half_rn(s);
            // below fp16's normal range the middle goes by the rounded S, so that a code of 0 with M 0 stays 0
            const float mid = fmaf(C, fabsf(s) < 6.103515625e-5f ? __half2float(sh) : s, -dm * (float)sb_field(hd.y, hd.z, hd.w, 1, j));
            const uint32_t S = h2(__half_as_ushort(sh)), M = h2(__half_as_ushort(__float2half_rn(mid)));
            over |= !(fmaf(C, fabsf(s), fabsf(mid)) <= 65504.0f);
            const uint4 cw = lds4(cs + 16 + 16 * j);
            const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};
            uint32_t pl[2] = {0u, 0u};
            if constexpr (FMT == kFmtW5SB32) pl[0] = lds32_a(cs + 144 + 4 * j);
            if constexpr (FMT == kFmtW6SB32) {
                pl[0] = lds32_a(cs + 144 + 8 * j);
                pl[1] = lds32_a(cs + 148 + 8 * j);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t u[4];
                if constexpr (FMT == kFmtW4SB32) {
                    const uint32_t v = w[i] >> 8;
                    u[0] = hadd2(and_or(w[i], 0x000F000Fu, 0x64006400u), 0xE408E408u);                          // - 1032
                    u[1] = hfma2(and_or(w[i], 0x00F000F0u, 0x64006400u), 0x2C002C00u, 0xD480D480u);             // / 16 - 72
                    u[2] = hadd2(and_or(v, 0x000F000Fu, 0x64006400u), 0xE408E408u);
                    u[3] = hfma2(and_or(v, 0x00F000F0u, 0x64006400u), 0x2C002C00u, 0xD480D480u);
                } else {
                    // the higher bits of weights k and k + 4 to bits 4 and 20 on
                    constexpr int B = FMT == kFmtW5SB32 ? 1 : 2;
                    constexpr uint32_t HM = B == 1 ? 0x00100010u : 0x00300030u;
                    uint32_t h = B == 1 ? (pl[0] >> (8 * i)) & 0xffu : (pl[i >> 1] >> (16 * (i & 1))) & 0xffffu;
                    h |= h << (B == 1 ? 12 : 8);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t hs = 4 - B * q >= 0 ? h << (4 - B * q < 0 ? 0 : 4 - B * q) : h >> (B * q - 4 < 0 ? 0 : B * q - 4);
                        u[q] = hadd2(and_or(hs, HM, and_or(w[i] >> (4 * q), 0x000F000Fu, 0x64006400u)), B == 1 ? 0xE410E410u : 0xE420E420u);
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) o[16 * gl + 4 * i + q] = hfma2(u[q], S, M);
            }
        }
        return over;
    }
}

// Eight weights of a plane's row from K 8 c on, in fp32.
template <int FMT>
__device__ __forceinline__ void weights8(const WideParams& p, unsigned long long row, int c, float (&w)[8]) {
    const uint8_t* code = p.codes + row * p.crb;
    uint32_t lo = 0u, hi = 0u;                           // nibbles (bytes for the 8-bit codes), and the bits above them
    int bits = 0, off = 0;
    float s = 0.0f, m = 0.0f;
    if constexpr (is_sb(FMT)) {
        const uint8_t* rec = code + (c >> 5) * sb_record(FMT);
        const int i = c & 31, j = i >> 2;
        const uint4 hd = __ldg(reinterpret_cast<const uint4*>(rec));
        lo = __ldg(reinterpret_cast<const uint32_t*>(rec + 16) + i);
        if (FMT == kFmtW5SB32) hi = __ldg(rec + 144 + i);
        if (FMT == kFmtW6SB32) hi = __ldg(reinterpret_cast<const uint16_t*>(rec + 144) + i);
        bits = sb_bits(FMT) - 4;
        s = __half2float(__ushort_as_half((uint16_t)(hd.x & 0xffffu))) * (float)sb_field(hd.y, hd.z, hd.w, 0, j);
        m = __half2float(__ushort_as_half((uint16_t)(hd.x >> 16))) * (float)sb_field(hd.y, hd.z, hd.w, 1, j);
    } else {
        s = __half2float(__ushort_as_half(__ldg(reinterpret_cast<const uint16_t*>(p.scales + row * p.srb) + 8 * c / sym_group(FMT))));
        if (FMT == kFmtW4G64) {
            lo = __ldg(reinterpret_cast<const uint32_t*>(code) + c);
            off = 8;
        } else if (FMT == kFmtW6G16) {
            const uint8_t* b = code + (c >> 3) * 48;
            lo = __ldg(reinterpret_cast<const uint32_t*>(b) + (c & 7));
            hi = __ldg(reinterpret_cast<const uint16_t*>(b + 32) + (c & 7));
            bits = 2;
            off = 32;
        } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(code) + c);
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = s * (float)((int)((k < 4 ? v.x : v.y) >> (8 * (k & 3)) & 255u) - 128);
            return;
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int u = (int)(lo >> (4 * k) & 15u) + (int)((hi >> (bits * k) & ((1u << bits) - 1u)) << 4);
        w[k] = fmaf(s, (float)(u - off), -m);
    }
}

// The sums of one weight row over K 8 c0 .. 8 c1 - 1 with the laid-out rows m0 .. m0 + 15 in fp32: for weights out of
// fp16's range, which trained matrices do not have. Slow (512 rows, 2 experts, w4g64 2048 x 512: 1.8 ms), but a unit of
// 128 rows and the longest K ends in 56 ms, far below the limit of the waits beside it. Looking for such scales costs
// the other calls 1 % (4096 rows of 8 experts, w4g64 2048 x 8192: 171 -> 173 us).
template <int FMT>
__device__ __noinline__ void exact_sums(const WideParams& p, unsigned long long row, int c0, int c1, int m0, float* sums) {
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = 0.0f;
    for (int c = c0; c < c1; ++c) {
        float w[8];
        weights8<FMT>(p, row, c, w);
#pragma unroll 4
        for (int j = 0; j < 16; ++j) {
            const uint4 u = __ldg(p.xg + (size_t)min(m0 + j, p.pl.R - 1) * (p.pl.K / 8) + c);
            const uint32_t h[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {                // the pairs that lay8 makes
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
                const int k = Wide<FMT>::ORDER == 1 ? i : (i & 1) + 4 * (i >> 1);
                v[j] = fmaf(w[k], f.x, v[j]);
                v[j] = fmaf(w[k + (Wide<FMT>::ORDER == 1 ? 4 : 2)], f.y, v[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) sums[j] = v[j];
}

// Scale words of the row's atom (64 weights from K 64 a on).
template <int FMT>
__device__ __forceinline__ void atom_scales(const uint8_t* row, int a, int K, uint32_t (&sc)[2]) {
    sc[0] = sc[1] = 0u;
    if constexpr (!is_sb(FMT)) {
        if (64 * a >= K) return;
        if constexpr (sym_group(FMT) == 16) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + 8 * a));
            sc[0] = v.x;
            sc[1] = v.y;
        } else {
            sc[0] = __ldg(reinterpret_cast<const uint16_t*>(row) + a);
        }
    }
}

// max(v, 0), NaN stays NaN
__device__ __forceinline__ float relu_nan(float v) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(v), "f"(0.0f));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// ----------------------------------------------------------------- product
template <int FMT, int MC>
__global__ void __launch_bounds__(kWideThreads, 1) wide_kernel(const __grid_constant__ WideParams p) {
    using G = Wide<FMT>;
    constexpr int ND = MC == 64 ? 2 : 1;                                 // buffers of sums
    constexpr uint32_t A0 = ND * kTiles * MC;                            // the A slots lie behind them
    static_assert(A0 + 64 * kA <= 512, "tensor memory");
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int NX = p.xslots, NC = p.cslots;
    uint8_t* at = smem + NC * G::CB + (size_t)NX * MC * 256;
    WDesc* desc = reinterpret_cast<WDesc*>(at);
    at += kDescs * sizeof(WDesc);
    RowInfo* rowinfo = reinterpret_cast<RowInfo*>(at) + (warp & (kWorkers - 1)) * (MC / 2);
    at += kWorkers * (MC / 2) * sizeof(RowInfo);
    uint64_t* cfull = reinterpret_cast<uint64_t*>(at);
    uint64_t* cempty = cfull + kMaxCodes;
    uint64_t* xfull = cempty + kMaxCodes;
    uint64_t* xempty = xfull + kMaxX;
    uint64_t* afull = xempty + kMaxX;
    uint64_t* aempty = afull + kA;
    uint64_t* ufull = aempty + kA;
    uint64_t* dfull = ufull + kDescs;
    uint64_t* dempty = dfull + ND * kTiles;
    uint64_t* mdone = dempty + ND * kTiles;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(mdone + kTiles);
    at += kBarBytes;
    WGroups g;
    g.cost = reinterpret_cast<long long*>(at);
    g.row = reinterpret_cast<int*>(g.cost + p.pl.E + 1);
    g.ctas = g.row + p.pl.E + 1;
    // Per weight row, for even and odd units (a row's two unpacking warps are less than two units apart): 1 + the last
    // unit with weights past fp16.
    volatile uint16_t* over = reinterpret_cast<uint16_t*>(smem + p.over_at);

    for (int i = tid; i < 2 * kUnitRows; i += kWideThreads) over[i] = 0;
    if (tid == 0) {
        for (int s = 0; s < NC; ++s) {
            mbar_init(&cfull[s], 1);
            mbar_init(&cempty[s], kWorkers);
        }
        for (int s = 0; s < NX; ++s) {
            mbar_init(&xfull[s], 1);
            mbar_init(&xempty[s], kTiles);
        }
        for (int s = 0; s < kA; ++s) {
            mbar_init(&afull[s], kWorkers / kTiles);
            mbar_init(&aempty[s], 1);
        }
        for (int s = 0; s < kDescs; ++s) mbar_init(&ufull[s], 1);
        for (int s = 0; s < ND * kTiles; ++s) {
            mbar_init(&dfull[s], 1);
            mbar_init(&dempty[s], kWorkers / kTiles);
        }
        for (int s = 0; s < kTiles; ++s) mbar_init(&mdone[s], 1);
        fence_mbar_init();
    }
    if (warp == kWorkers) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tslot)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (warp == kWorkers + 1) {
        scan_wide(p.pl, g, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    grid_dep_launch();

    const int T = p.pl.T;
    const uint32_t cbase = smem_u32(smem), xbase = cbase + NC * G::CB;
    auto wait = [&](uint64_t* bar, int phase, unsigned flag) {
        return __all_sync(~0u, mbar_try_wait(bar, (uint32_t)phase & 1u)) ||
               __all_sync(~0u, mbar_wait_bounded(bar, (uint32_t)phase & 1u, flag, 0u, p.wait_ns));
    };

    if (warp == kWorkers + 1) {
        // ------------------------------------------------ work and its rows
        if (lane == 0) {
            if (!p.z) grid_dep_wait();                   // the rows (with z, the kernel before this one waited for them)
            asm volatile("fence.proxy.async.global;" ::: "memory");
            Walk walk(p.pl, g);
            WDesc d;
            int u = 0, xs = 0, xwrap = 0, issued = 0;
            bool ok = !(p.test_flags & kTestNoCopies);
            for (; ok && walk.next(d); ++u) {
                desc[u % kDescs] = d;
                mbar_arrive(&ufull[u % kDescs]);
                const int boxes = (((d.rows + 15) & ~15) + 31) / 32;
                for (int a = d.k0 * G::PAIRS; ok && a < d.k1 * G::PAIRS; ++a) {
                    if (xwrap && !mbar_wait_bounded(&xempty[xs], (uint32_t)(xwrap - 1) & 1u, kStatusSlotWait, 32u, p.wait_ns)) { ok = false; break; }
                    mbar_arrive_expect_tx(&xfull[xs], (uint32_t)boxes * 8192u);
                    for (int h = 0; h < 2; ++h)
                        for (int b = 0; b < boxes; ++b)
                            tma_3d(xbase + xs * (MC * 256) + h * (MC * 128) + b * 4096, &p.xmap, 0, d.row0 + 32 * b, 2 * a + h, &xfull[xs]);
                    ++issued;
                    if (++xs == NX) { xs = 0; ++xwrap; }
                }
            }
            if (!(p.test_flags & kTestNoCopies)) {
                desc[u % kDescs].done = 1;
                mbar_arrive(&ufull[u % kDescs]);
            }
            // copies in flight (a warp gave up) land before the CTA leaves
            for (int q = 0; q < NX && q < issued; ++q)
                mbar_wait_bounded(&xfull[q], (uint32_t)(issued / NX + (q < issued % NX ? 1 : 0) - 1) & 1u, kStatusTmaWait, 64u, p.wait_ns);
        }
        __syncwarp();
    } else if (warp == kWorkers + 2) {
        // ------------------------------------------------------------ codes
        if (lane == 0 && !(p.test_flags & kTestNoCopies)) {
            Walk walk(p.pl, g);
            WDesc d;
            int cs = 0, cwrap = 0, issued = 0;
            bool ok = true;
            while (ok && walk.next(d)) {
                if constexpr (!is_sb(FMT)) {             // the tile's scales into L2
                    const unsigned long long b0 = (unsigned long long)d.wrow * p.srb & ~15ull;
                    const unsigned long long b1 = (min((unsigned long long)d.wrow + kUnitRows, p.total_rows) * p.srb + 15) & ~15ull;
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(p.scales + b0), "r"((uint32_t)(b1 - b0)) : "memory");
                }
                for (int k = d.k0; k < d.k1; ++k) {
                    if (cwrap && !mbar_wait_bounded(&cempty[cs], (uint32_t)(cwrap - 1) & 1u, kStatusSlotWait, 32u, p.wait_ns)) { ok = false; break; }
                    mbar_arrive_expect_tx(&cfull[cs], (uint32_t)(kUnitRows * G::RB));
                    tma_2d(cbase + cs * G::CB, &p.cmap, k * G::RB, d.wrow, &cfull[cs]);
                    ++issued;
                    if (++cs == NC) { cs = 0; ++cwrap; }
                }
            }
            for (int q = 0; q < NC && q < issued; ++q)
                mbar_wait_bounded(&cfull[q], (uint32_t)(issued / NC + (q < issued % NC ? 1 : 0) - 1) & 1u, kStatusTmaWait, 64u, p.wait_ns);
        }
        __syncwarp();
    } else if (warp >= kWorkers) {
        // ------------------------------------------------------- MMA issue
        const int t = warp == kWorkers ? 0 : 1;
        int xs = 0, xwrap = 0, as = t, awrap = 0;        // the tile's A slots: t, t + 2
        bool ok = true;
        for (int u = 0; ok; ++u) {
            if (!wait(&ufull[u % kDescs], u / kDescs, kStatusTmaWait)) break;
            const WDesc d = desc[u % kDescs];
            if (d.done) break;
            const int db = u % ND;
            if (u >= ND && !wait(&dempty[db * kTiles + t], u / ND - 1, kStatusMmaWait)) break;
            tc_fence_after();
            const int np = (d.rows + 15) & ~15;
            const uint32_t idesc = (1u << 4) | ((uint32_t)(np >> 3) << 17) | ((uint32_t)(kTcRows >> 4) << 24);   // fp16, fp32 sums
            const uint32_t dc = tmem + (db * kTiles + t) * MC;
            const int n = (d.k1 - d.k0) * G::PAIRS;
            for (int i = 0; i < n; ++i) {
                if (!wait(&xfull[xs], xwrap, kStatusTmaWait) || !wait(&afull[as], awrap, kStatusTmaWait)) { ok = false; break; }
                tc_fence_after();
                const uint64_t xd = sw128_desc(xbase + xs * (MC * 256));
                const uint32_t ac = tmem + A0 + 64u * as;
                mma_atom(dc, ac, xd, idesc, i ? 1u : 0u);
                mma_atom(dc, ac + 32u, xd + (uint64_t)(MC * 128 >> 4), idesc, 1u);
                mma_commit(&aempty[as]);
                mma_commit(&xempty[xs]);
                as += kTiles;
                if (as >= kA) { as = t; ++awrap; }
                if (++xs == NX) { xs = 0; ++xwrap; }
            }
            if (ok) mma_commit(&dfull[db * kTiles + t]);
        }
        mma_commit(&mdone[t]);
        wait(&mdone[t], 0, kStatusMmaWait);              // no MMA in flight at teardown
    } else {
        // ------------------------------------------- unpack, then the sums
        const int q = warp & 3, tile = warp >> 3, h = (warp >> 2) & 1, r = 32 * q + lane, rr = kTcRows * tile + r;
        const uint32_t tl = (uint32_t)(32 * q) << 16;
        int cs = 0, cwrap = 0, as = tile, awrap = 0;     // this tile's A slots: tile, tile + 2
        bool waited = false;
        const long long W = g.cost[p.pl.E], Gc = *g.ctas;
        for (int u = 0;; ++u) {
            if (!wait(&ufull[u % kDescs], u / kDescs, kStatusTmaWait)) break;
            const WDesc d = desc[u % kDescs];
            if (d.done) break;
            const uint8_t* srow = p.scales + min((unsigned long long)d.wrow + rr, p.total_rows - 1) * p.srb;
            uint32_t sc[2], nx[2];
            const int a1 = d.k1 * 2 * G::PAIRS;
            atom_scales<FMT>(srow, d.k0 * 2 * G::PAIRS + h, p.pl.K, nx);
            bool ok = true;
            for (int k = d.k0; ok && k < d.k1; ++k) {
                if (!wait(&cfull[cs], cwrap, kStatusTmaWait)) { ok = false; break; }
#pragma unroll
                for (int i = 0; i < G::PAIRS; ++i) {
                    const int a = (k * G::PAIRS + i) * 2 + h;            // 64-K atom of the row
                    sc[0] = nx[0];
                    sc[1] = nx[1];
                    if (a + 2 < a1) atom_scales<FMT>(srow, a + 2, p.pl.K, nx);
                    uint32_t o[32];
                    if (unpack_atom<FMT>(cbase + cs * G::CB + rr * G::RB, 2 * i + h, G::RB == 128 ? r & 7 : 0, sc, o)) over[(u & 1) * kUnitRows + rr] = (uint16_t)(u + 1);
                    if (i == G::PAIRS - 1) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&cempty[cs]);
                    }
                    if (awrap && !wait(&aempty[as], awrap - 1, kStatusMmaWait)) { ok = false; break; }
                    tc_fence_after();
                    tmem_st32(tmem + tl + A0 + 64u * as + 32u * h, o);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&afull[as]);
                    as += kTiles;
                    if (as >= kA) { as = tile; ++awrap; }
                }
                if (++cs == NC) { cs = 0; ++cwrap; }
            }
            if (!ok) break;
            if (!waited) {
                grid_dep_wait();                         // counters and powers of two come from lay_rows_kernel
                waited = true;
            }
            bool safe = true;                            // a row's power of two squared stays in range
            // this warp's activation rows, 16 of every 32: row of y (negative: none) and scale
            const int blocks = (d.rows + 15) / 16;
            for (int b = h, x = 0; b < blocks; b += 4, x += 32) {
                const int i = 16 * (b + (lane >> 4) * 2) + (lane & 15), m = d.row0 + i;
                RowInfo info = {nullptr, 0.0f, 0u};
                if (i < d.rows) {
                    const int o = p.out_rows ? __ldg(p.out_rows + m) : m;
                    if (o >= 0 && o < p.Ty) info.y = static_cast<__nv_bfloat16*>(p.y) + (size_t)o * p.pl.N + d.n0;
                    info.scale = __ldcg(p.rscale + m);
                    const float f = p.act ? info.scale * info.scale : info.scale;
                    info.scale2 = (__float_as_uint(f) >> 16) * 0x10001u;
                    if (p.act && !(info.scale > 1e-18f && info.scale < 1e18f)) safe = false;
                }
                if (x + lane < MC / 2) rowinfo[x + lane] = info;
            }
            safe = __all_sync(~0u, safe);
            __syncwarp();
            const int db = u % ND;
            if (!wait(&dfull[db * kTiles + tile], u / ND, kStatusMmaWait)) break;
            tc_fence_after();
            // sums: this warp's 32 weight rows, 16 activation rows at a time
            const uint32_t dcol = tmem + tl + (db * kTiles + tile) * MC;
            // made again where a weight passed fp16's range (a row past the expert's end is not stored)
            const bool again = over[(u & 1) * kUnitRows + rr] == (uint16_t)(u + 1) && d.n0 + rr < p.pl.N, any_again = __any_sync(~0u, again);
            auto load16 = [&](int b, float (&v)[16]) {
                tmem_ld16(dcol + 16u * b, v);
                if (any_again) {
                    float t[16];
                    if (again) exact_sums<FMT>(p, (unsigned long long)d.wrow + rr, d.k0 * (G::KS / 8), min(d.k1 * (G::KS / 8), p.pl.K / 8), d.row0 + 16 * b, t);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = again ? t[j] : v[j];
                    __syncwarp();
                }
            };
            const bool cut = d.first != d.last || d.k0 > 0 || d.k1 < T;
            constexpr size_t kPart = (size_t)MC * kUnitRows;
            bool store = true;
            // which of CTAs c0 .. c0 + 31 have stages of the unit
            auto parts_from = [&](int c0) {
                const int c = c0 + lane;
                const long long q0 = ceil_div((long long)c * W, Gc) - d.pos, q1 = ceil_div(((long long)c + 1) * W, Gc) - d.pos;
                const long long k0 = q0 <= 0 ? 0 : ceil_div(q0, d.cost), k1 = q1 <= 0 ? 0 : ceil_div(q1, d.cost);
                return __ballot_sync(~0u, c <= d.last && k0 < k1 && k0 < T);
            };
            unsigned parts0 = 0u;
            if (cut) {
                float* mine = p.part + (2 * (size_t)blockIdx.x + (d.k0 == 0)) * kPart + rr;
                for (int b = h; b < blocks; b += 2) {
                    float v[16];
                    load16(b, v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) __stcg(mine + (size_t)(16 * b + j) * kUnitRows, v[j]);
                }
                __threadfence();
                __syncwarp();
                unsigned old = 0;
                if (lane == 0) old = atomicAdd(&p.count[d.first * kWorkers + warp], (unsigned)(d.k1 - d.k0));
                old = __shfl_sync(~0u, old, 0);
                store = old + (unsigned)(d.k1 - d.k0) == (unsigned)T;    // the last part: all stages are summed
                if (store) {
                    __threadfence();
                    parts0 = parts_from(d.first);
                }
            }
            for (int b = h; store && b < blocks; b += 2) {
                float v[16];
                if (!cut) {
                    load16(b, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = 0.0f;
                    for (int c0 = d.first; c0 <= d.last; c0 += 32) {
                        unsigned todo = c0 == d.first ? parts0 : parts_from(c0);
                        while (todo) {                   // two parts' loads at a time, added in order
                            const int ca = __ffs(todo) - 1;
                            todo &= todo - 1;
                            const int cb = todo ? __ffs(todo) - 1 : -1;
                            todo &= todo - 1;
                            const float* fa = p.part + (2 * (size_t)(c0 + ca) + (c0 + ca == d.first)) * kPart + (size_t)(16 * b) * kUnitRows + rr;
                            const float* fb = p.part + 2 * (size_t)(c0 + max(cb, 0)) * kPart + (size_t)(16 * b) * kUnitRows + rr;
                            float xa[16], xb[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) xa[j] = __ldcg(fa + j * kUnitRows);
#pragma unroll
                            for (int j = 0; j < 16; ++j) xb[j] = cb >= 0 ? __ldcg(fb + j * kUnitRows) : 0.0f;
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = (v[j] + xa[j]) + xb[j];
                        }
                    }
                }
                const int left = p.pl.N - d.n0 - rr;                     // columns from this lane's on
                const RowInfo* info = rowinfo + (b >> 1) * 16;
                if ((p.pl.N & 1) == 0 && !p.z && safe) {
                    // The row's power of two commutes with the rounding, so it is applied to the packed bf16 results.
                    // Lanes in pairs: the even one stores columns n, n + 1 of row j, the odd one those of row j + 1.
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        float v0 = v[j], v1 = v[j + 1];
                        if (p.act) {
                            v0 = relu_nan(v0);
                            v1 = relu_nan(v1);
                            v0 *= v0;
                            v1 *= v1;
                        }
                        const uint32_t own = pack2(v0, v1), other = __shfl_xor_sync(~0u, own, 1);
                        const RowInfo f = info[j + (lane & 1)];
                        const uint32_t h = mul_bf16x2(lane & 1 ? prmt(other, own, 0x7632u) : prmt(own, other, 0x5410u), f.scale2);
                        if (f.y && left > 0) *reinterpret_cast<uint32_t*>(f.y + (rr & ~1)) = h;
                    }
                } else {
                    if (p.z) {                           // all loads before the first store
                        const float* z = p.z + (size_t)(d.row0 + 16 * b) * p.ldz + d.n0 + rr;
                        float zv[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) zv[j] = 16 * b + j < d.rows && left > 0 ? __ldcg(z + (size_t)j * p.ldz) : 0.0f;
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = fmaf(v[j], info[j].scale, zv[j]);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const RowInfo f = info[j];
                        float r1 = p.z ? v[j] : v[j] * f.scale;
                        if (p.act) {
                            r1 = relu_nan(r1);
                            r1 *= r1;
                        }
                        if (f.y && left > 0) f.y[rr] = __float2bfloat16_rn(r1);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&dempty[db * kTiles + tile]);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kWorkers) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// ------------------------------------------------------------------ host
struct WLayout { size_t xg, rscale, part, count, total; };

WLayout wide_layout(int R, int K, int MC) {
    WLayout l;
    l.xg = 0;
    l.rscale = (size_t)R * K * 2;
    l.part = l.rscale + round16((size_t)R * 4);
    l.count = l.part + (size_t)2 * kWideMaxCtas * MC * kUnitRows * 4;
    l.total = l.count + kWideMaxCtas * kWorkers * 4;
    return l;
}

// Activation rows of a unit at most: 128 where that still makes a unit for
// every second SM.
int wide_mc(int R, int E, int N) {
    const int per = (R + E - 1) / E;
    if (per <= 64) return 64;
    return (long long)((N + kUnitRows - 1) / kUnitRows) * E * ((per + 127) / 128) >= sm_count() / 2 ? 128 : 64;
}

template <int FMT, int MC>
cudaError_t launch_wide_mc(const RowsArgs& a, WideParams& p, cudaStream_t st) {
    using G = Wide<FMT>;
    const size_t fixed = kDescs * sizeof(WDesc) + kWorkers * (MC / 2) * sizeof(RowInfo) + kBarBytes + wgroups_bytes(a.E) + kOverBytes;
    p.xslots = kMaxX;
    auto codes = [&]() { return (int)((kWideSmem - fixed - (size_t)p.xslots * MC * 256) / G::CB); };
    if (fixed + (size_t)p.xslots * MC * 256 + 2 * (size_t)G::CB > kWideSmem) p.xslots = 2;   // wide codes, many experts
    p.cslots = codes();
    if (p.cslots > kMaxCodes) p.cslots = kMaxCodes;
    if (p.cslots < 2) return cudaErrorInvalidValue;
    auto kern = wide_kernel<FMT, MC>;
    static unsigned long long attr_done = 0ull;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(__atomic_load_n(&attr_done, __ATOMIC_ACQUIRE) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWideSmem);
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(&attr_done, bit, __ATOMIC_RELEASE);
    }
    const int sms = sm_count();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms < kWideMaxCtas ? sms : kWideMaxCtas));
    cfg.blockDim = dim3(kWideThreads);
    cfg.dynamicSmemBytes = fixed + (size_t)p.xslots * MC * 256 + (size_t)p.cslots * G::CB;
    p.over_at = (int)(cfg.dynamicSmemBytes - kOverBytes);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int FMT>
cudaError_t launch_wide_fmt(const RowsArgs& a, cudaStream_t st) {
    using G = Wide<FMT>;
    const EncodeTiled enc = encoder();
    if (!enc) return cudaErrorNotSupported;
    const int MC = wide_mc(a.R, a.E, a.N);
    const WLayout l = wide_layout(a.R, a.K, MC);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    unsigned* count = reinterpret_cast<unsigned*>(ws + l.count);
    float* rscale = reinterpret_cast<float*>(ws + l.rscale);

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.R);
    cfg.blockDim = dim3(kLayThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const LayParams lay = {static_cast<const __nv_bfloat16*>(a.x), a.in_rows, a.T, a.K, reinterpret_cast<uint4*>(ws + l.xg), rscale, count,
                           kWideMaxCtas * kWorkers};
    cudaError_t e;
    if (!a.z) {
        e = cudaLaunchKernelEx(&cfg, lay_rows_kernel<G::ORDER>, lay);
    } else {
        const int threads = shrink_threads(a.R);
        cfg.gridDim = dim3((unsigned)(a.R * (a.ad.r / 8) + a.R));
        cfg.blockDim = dim3((unsigned)threads);
        e = threads == 512 ? cudaLaunchKernelEx(&cfg, lay_shrink_kernel<G::ORDER, 512>, lay, a.ad, a.R, a.order)
                           : cudaLaunchKernelEx(&cfg, lay_shrink_kernel<G::ORDER, 256>, lay, a.ad, a.R, a.order);
    }
    if (e != cudaSuccess) return e;
    if (a.z) {
        e = launch_expand(a.ad, a.order, a.R, const_cast<float*>(a.z), a.ldz, st);
        if (e != cudaSuccess) return e;
    }

    WideParams p = {};
    const uint64_t crb = code_row_bytes(FMT, a.K), rows = (uint64_t)a.E * a.N;
    const cuuint64_t cd[2] = {crb, rows}, cst[1] = {crb};
    const cuuint32_t cb[2] = {(cuuint32_t)G::RB, (cuuint32_t)kUnitRows}, ones[3] = {1, 1, 1};
    const cuuint64_t xd[3] = {64, (cuuint64_t)a.R, (cuuint64_t)(a.K / 64)}, xst[2] = {(cuuint64_t)a.K * 2, 128};
    const cuuint32_t xb[3] = {64, 32, 1};
    if (enc(&p.cmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(a.codes), cd, cst, cb, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            G::RB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
        enc(&p.xmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, ws + l.xg, xd, xst, xb, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    p.pl = {a.offsets, a.E, a.R, a.N, a.K, (a.K + G::KS - 1) / G::KS, MC};
    p.codes = static_cast<const uint8_t*>(a.codes);
    p.scales = static_cast<const uint8_t*>(a.scales);
    p.total_rows = rows;
    p.crb = (uint32_t)crb;
    p.srb = (uint32_t)scale_row_bytes(FMT, a.K);
    p.xg = reinterpret_cast<const uint4*>(ws + l.xg);
    p.rscale = rscale;
    p.part = reinterpret_cast<float*>(ws + l.part);
    p.count = count;
    p.out_rows = a.out_rows;
    p.y = a.y;
    p.Ty = a.Ty;
    p.act = a.act;
    p.z = a.z;
    p.ldz = a.ldz;
    p.wait_ns = wait_limit_ns();
    p.test_flags = test_flags();
    return MC == 128 ? launch_wide_mc<FMT, 128>(a, p, st) : launch_wide_mc<FMT, 64>(a, p, st);
}

}  // namespace

size_t wide_workspace(int R, int K, int E) { return wide_layout(R, K, (R + E - 1) / E > 64 ? 128 : 64).total; }

cudaError_t launch_wide(const RowsArgs& a, cudaStream_t st) {
    switch (a.fmt) {
        case kFmtW4G64: return launch_wide_fmt<kFmtW4G64>(a, st);
        case kFmtW8G16: return launch_wide_fmt<kFmtW8G16>(a, st);
        case kFmtW8G64: return launch_wide_fmt<kFmtW8G64>(a, st);
        case kFmtW6G16: return launch_wide_fmt<kFmtW6G16>(a, st);
        case kFmtW4SB32: return launch_wide_fmt<kFmtW4SB32>(a, st);
        case kFmtW5SB32: return launch_wide_fmt<kFmtW5SB32>(a, st);
        default: return launch_wide_fmt<kFmtW6SB32>(a, st);
    }
}

cudaError_t status_wide(cudaStream_t st, unsigned* word) {
    unsigned v = 0, z = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_status, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    *word = v;
    return e;
}

}  // namespace rq
