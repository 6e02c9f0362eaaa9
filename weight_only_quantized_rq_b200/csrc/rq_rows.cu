// rq_rows.cu -- packed products whose weights depend on the activation row:
// products grouped by expert with ragged sizes, and a low-rank adapter per row
// beside a shared packed projection. fp32 results, and bf16 ones of groups with
// few rows (rq_wide.cu makes those of many rows).
//
//   grouped  y[i] = act(x[in(i)] W_e^T),            i in [offsets[e], offsets[e + 1])
//   adapter  y[m] = x[m] W^T + s_a B_a (A_a x[m]),  a = row_adapter[m]
//
// Two launches per call:
//
// prep_kernel  lays the rows out for the tensor cores: per group, tiles of
//   eight rows (the last one padded with zeros), each tile as the B fragments
//   of mma.m16n8k16 in the order that the weights' codes unpack in, so that the
//   product kernel reads 16 bytes per lane with no bank conflict and no
//   permutation. For the superblocks it adds -sum x per group of 32 (w = S u - M
//   needs it beside the products). It clears the counters of the cut units, and up to eight
//   rows with adapters it computes t = s_a A_a x[m] in fp32. The product kernel
//   starts beside it: its weight copies run while prep works.
//
// rows_kernel  multiplies. Bound by the weight stream while a group has few
//   rows: what has to be read is the packed plane of each expert in use.
//   * Codes are exact small integers in bf16 (q, |q| <= 128; u <= 63 for the
//     superblocks), x is bf16: every product is exact in the tensor core's
//     fp32 sums, and the group's scale multiplies the fp32 group sum. So no
//     weight is rounded, and fp32 results are good to fp32 (2e-7 on the
//     sums here), unlike weights rounded to bf16 before the product (2e-3).
//     The offset that a code unpacks under is subtracted from the code, not from
//     the sum: a code of zero adds nothing however large its x (16 + u summed
//     against a start of -24 sum x saved that subtraction, but its error
//     followed 24 sum |x|: 20 times as large with outliers of 200 on zero codes).
//     Codes carry a factor of 2^-14, so that no sum of a group leaves fp32's
//     range before its scale is applied; a unit's sums get it back at the end
//     (exact, but for results below 2^-112, which keep 2^-135 absolute).
//   * mma.sync, not tcgen05: with a handful of rows the products are not what
//     counts. The A operand of mma.sync comes straight from the registers that
//     unpacked it, and its result is in registers when the group's scale is
//     applied; through tensor memory each 64-weight group would need its own
//     accumulator and a read back (measured for this library's other kernel:
//     1.9 against 2.4 TB/s).
//   * A unit of work is 128 weight rows x K x up to 8 NB activation rows. Four
//     warps take 32 weight rows each, from the codes to y with no barrier among
//     them (16 rows per warp would double the shared-memory reads of x); a
//     fifth copies: codes by TMA through a ring of their own, activations and
//     scales through two slots. Small CTAs, three or four per SM: one CTA's
//     start and end run beside the others' stream (eight warps with barriers, two
//     CTAs per SM: 66 against 51 us at the time for 141 MB of w4g64 codes and 4
//     rows per expert).
//   * All units' K stages form one line that the CTAs share out evenly, so
//     neither ragged groups nor few tiles leave SMs idle. A unit cut by a CTA
//     border is summed through the workspace: each part is written, the last to
//     arrive adds all parts in K order (the same bits whoever is last; nobody
//     waits).
// Measured (both kernels, device time): 16 experts of w4g64, K 2048, N 8192, 4
// rows each, 141 MB: 42 us, 3.4 TB/s; the stream alone takes 33 of it, the rest
// is the front (7 us from the call to the first products) and the CTAs' uneven
// ends. Two rows, 2 experts, 18 MB: 13 us.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rq_device.cuh"
#include "rq_internal.h"
#include "rq_rows.cuh"
#include "rq_tc.cuh"

namespace rq {
namespace {

constexpr int kRowsPerTile = 128;      // weight rows of a unit
constexpr int kMathWarps = 4;          // 32 weight rows each
constexpr int kRowsThreads = 32 * (kMathWarps + 1);
constexpr int kMaxRing = 6;            // code slots at most
constexpr int kXRing = 2;              // slots of activations and scales
constexpr int kDescs = 8;              // unit descriptors in flight: more than kMaxRing + 1
constexpr size_t kSmemPerSm = 228 * 1024;

// Geometry of a format's K stage.
template <int FMT>
struct Geo {
    static constexpr int KS = is_w8(FMT) || FMT == kFmtW6G16 ? 128 : 256;         // K per stage
    static constexpr int RB = FMT == kFmtW4G64 ? 128 : is_w8(FMT) ? 128 : FMT == kFmtW6G16 ? 96 : sb_record(FMT);
    // Activations of one 8-row tile's stage: the fragments, then for the superblocks minus the rows' sums
    // over each group, 32 bytes per group (of rows 0..7).
    static constexpr int XB = KS * 16 + (is_sb(FMT) ? KS : 0);
    static constexpr int SB = is_sb(FMT) ? 0 : KS / sym_group(FMT) * 2;           // scale bytes of a weight row's stage
    static constexpr bool SWZ = RB == 128;
    static constexpr int CB = (kRowsPerTile * RB + 1023) & ~1023;                 // a code slot
    static constexpr int SCRATCH = is_sb(FMT) ? 2048 : 1024;                      // shared bytes of a math warp
};

// Codes are multiplied as q 2^-kDown (u 2^-kDown): with 64 codes of up to 128 in a group's sum, a quarter of fp32's
// largest value is not passed.
constexpr int kDown = 14;

// CTAs per SM: four while their accumulators and two stages each fit.
__host__ __device__ constexpr int ctas_per_sm(int fmt, int nb) {
    return nb == 4 || fmt == kFmtW5SB32 || fmt == kFmtW6SB32 ? 3 : 4;
}

struct Plan {                          // what both kernels know of a call
    const int* offsets;
    int E, R, N, K, T;                 // T: stages per unit
    int NB;                            // 8-row tiles per unit at most
};

struct RowsParams {
    CUtensorMap cmap;                  // codes: uint8 [E N][row bytes], box [128][RB]
    Plan pl;
    const uint8_t* scales;
    unsigned long long total_rows;     // E N
    uint32_t srb;                      // scale bytes per weight row
    const uint8_t* xf;                 // prepared activations
    float* part;                       // partial tiles, two per CTA
    unsigned* count;                   // arrivals per split unit, by its first CTA
    const int* out_rows;
    void* y;
    int Ty, ybf16, act;
    Adapters ad;                       // row NULL: none; used where a unit holds one 8-row tile
    const float* z;                    // [R][ldz] the adapters' term, or NULL
    int ldz;
    int ring, xslot;                   // code slots; bytes of an activation slot
    unsigned long long wait_ns;
    int test_flags;
};

struct PrepParams {
    Plan pl;
    const __nv_bfloat16* x;
    const int* in_rows;
    int rows_x;
    uint8_t* xf;
    unsigned* count;
    int n_count;
    int tiles_max, kblocks;
    Adapters ad;
    int late;                          // the kernel before this one is waited for at the end
};

// ------------------------------------------------------------------ groups
// First row and first 8-row tile of each group, and its first unit, computed
// by one warp from the offsets (their running maximum, clamped to [0, R]).
struct Groups {
    int* row;          // [E + 1]
    int* tile;         // [E + 1]
    long long* unit;   // [E + 1]
};
__host__ __device__ inline size_t groups_bytes(int E) { return round16((size_t)(E + 1) * 16); }

__device__ __forceinline__ Groups groups_at(void* p, int E) {
    Groups g;
    g.unit = static_cast<long long*>(p);
    g.row = reinterpret_cast<int*>(g.unit + E + 1);
    g.tile = g.row + E + 1;
    return g;
}

__device__ __forceinline__ void scan_groups(const Plan& pl, Groups g, int lane) {
    const int tiles_n = (pl.N + kRowsPerTile - 1) / kRowsPerTile, chunk = 8 * pl.NB;
    int top = 0, tile0 = 0;
    long long unit0 = 0;
    for (int e0 = 0; e0 <= pl.E; e0 += 32) {
        const int e = e0 + lane;
        // end of group e - 1 = start of group e
        int v = 0;
        if (pl.offsets) v = e <= pl.E ? min(max(pl.offsets[e], 0), pl.R) : 0;
        else v = e >= 1 ? pl.R : 0;
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(~0u, v, o);
            if (lane >= o) v = max(v, w);
        }
        v = max(v, top);
        const int prev = __shfl_up_sync(~0u, v, 1);
        const int m = lane == 0 ? (e0 ? v - top : 0) : v - prev;       // rows of group e - 1
        int tl = (m + 7) / 8;
        long long un = (long long)((m + chunk - 1) / chunk) * tiles_n;
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(~0u, tl, o);
            const long long b = __shfl_up_sync(~0u, un, o);
            if (lane >= o) { tl += a; un += b; }
        }
        if (e <= pl.E) {
            g.row[e] = v;
            g.tile[e] = tile0 + tl;
            g.unit[e] = unit0 + un;
        }
        top = __shfl_sync(~0u, v, 31);
        tile0 += __shfl_sync(~0u, tl, 31);
        unit0 += __shfl_sync(~0u, un, 31);
    }
    __syncwarp();
}

// Last e with a[e] <= v (a ascending, a[0] <= v): the group that holds v, as
// groups without members repeat their successor's start.
template <class T>
__device__ __forceinline__ int find_group(const T* a, int E, T v) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= v) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// ------------------------------------------------------------------- prep
constexpr int kPrepThreads = 128;
constexpr int kPrepUnroll = 4;         // 16-byte chunks per thread
constexpr int kPrepChunks = 4 * (kPrepThreads / 32) * kPrepUnroll;   // of each of a block's eight rows

// -2^-kDown times the sum of eight values.
__device__ __forceinline__ float bf16_sum8(uint4 v) {
    constexpr float F = -1.0f / (1 << kDown);
    float a = bf16lo_f32(v.x) * F, b = bf16hi_f32(v.x) * F;
    a = fmaf(bf16lo_f32(v.y), F, a);
    b = fmaf(bf16hi_f32(v.y), F, b);
    a = fmaf(bf16lo_f32(v.z), F, a);
    b = fmaf(bf16hi_f32(v.z), F, b);
    a = fmaf(bf16lo_f32(v.w), F, a);
    return fmaf(bf16hi_f32(v.w), F, b) + a;
}

// With 32 registers its blocks fit beside the CTAs of a product that is still
// running; with SHRINK (adapters of few rows) it takes 64.
template <int FMT, bool SHRINK>
__global__ void __launch_bounds__(kPrepThreads, SHRINK ? 8 : 16) prep_kernel(const PrepParams p) {
    using G = Geo<FMT>;
    extern __shared__ __align__(16) uint8_t sm[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!p.late) grid_dep_wait();
    grid_dep_launch();                                   // the next kernel may start: all work before this call is done
    const int nx = p.tiles_max * p.kblocks;
    if ((int)blockIdx.x < nx) {
        if (blockIdx.x == 0)
            for (int i = tid; i < p.n_count; i += kPrepThreads) p.count[i] = 0u;
        Groups g = groups_at(sm, p.pl.E);
        if (warp == 0) scan_groups(p.pl, g, lane);
        __syncthreads();
        const int tile = blockIdx.x / p.kblocks, kb = blockIdx.x % p.kblocks;
        if (tile >= g.tile[p.pl.E]) {
            if (p.late) grid_dep_wait();
            return;
        }
        const int e = find_group(g.tile, p.pl.E, tile);
        const int row = g.row[e] + 8 * (tile - g.tile[e]) + (lane >> 2);     // lane = 4 (row in tile) + chunk in four
        int src = -1;
        if (row < g.row[e + 1]) {
            src = p.in_rows ? p.in_rows[row] : row;
            if (src < 0 || src >= p.rows_x) src = -1;
        }
        const int c_end = p.pl.T * G::KS / 8;                                // 8-value chunks of a row, padded to whole stages
        uint8_t* out = p.xf + (size_t)tile * p.pl.T * G::XB;
        uint4 vv[kPrepUnroll];
#pragma unroll
        for (int q = 0; q < kPrepUnroll; ++q) {
            const int c = kb * kPrepChunks + 4 * (kPrepUnroll * warp + q) + (lane & 3);
            vv[q] = make_uint4(0u, 0u, 0u, 0u);
            if (src >= 0 && 8 * c < p.pl.K) vv[q] = *reinterpret_cast<const uint4*>(p.x + (size_t)src * p.pl.K + 8 * c);
        }
#pragma unroll
        for (int q = 0; q < kPrepUnroll; ++q) {
            const int c = kb * kPrepChunks + 4 * (kPrepUnroll * warp + q) + (lane & 3);
            if (c >= c_end) break;                       // the same for the whole warp
            const uint4 v = vv[q];
            const int st = 8 * c / G::KS, cs = c - st * (G::KS / 8);         // stage, chunk in the stage
            uint8_t* o = out + (size_t)st * G::XB;
            if constexpr (G::KS == 256) {
                // nibble words unpack as the pairs (0, 4), (1, 5), (2, 6), (3, 7)
                uint4 w;
                w.x = prmt(v.x, v.z, 0x5410u);
                w.y = prmt(v.x, v.z, 0x7632u);
                w.z = prmt(v.y, v.w, 0x5410u);
                w.w = prmt(v.y, v.w, 0x7632u);
                *reinterpret_cast<uint4*>(o + ((cs >> 2) * 32 + lane) * 16) = w;
                if constexpr (is_sb(FMT)) {              // the row's sum over 32 weights, behind the fragments
                    float s = bf16_sum8(v);
                    s += __shfl_xor_sync(~0u, s, 1);
                    s += __shfl_xor_sync(~0u, s, 2);
                    if ((lane & 3) == 0) reinterpret_cast<float*>(o + G::KS * 16)[(cs >> 2) * 8 + (lane >> 2)] = s;
                }
            } else {
                // four-weight words unpack as the pairs (0, 2), (1, 3); lane t of a quad takes weights
                // 4t .. 4t + 3 of each 16-weight step, two steps per 16 bytes
                const int g8 = lane >> 2;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t a = h ? v.z : v.x, b = h ? v.w : v.y;
                    const int t = 2 * (cs & 1) + h, half = (cs >> 1) & 1;
                    const uint2 w = make_uint2(prmt(a, b, 0x5410u), prmt(a, b, 0x7632u));
                    *reinterpret_cast<uint2*>(o + ((cs >> 2) * 32 + g8 * 4 + t) * 16 + half * 8) = w;
                }
            }
        }
    } else if constexpr (SHRINK) {
        __shared__ float part[kPrepThreads / 32][8];
        const int per = p.ad.r / 8, b = blockIdx.x - nx;
        shrink8<kPrepThreads / 32>(p.ad, p.x, b / per, 8 * (b % per), part);
    }
    if (p.late) grid_dep_wait();                         // done means that the kernel before is done too
}

// ------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ void prefetch_l2_bulk(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_x(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}
// Asynchronous copy of B (4 or 8) bytes, or zeros where !in; cp_async_arrive
// makes the mbarrier receive one arrival when this thread's copies so far are
// in shared memory.
template <int B>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" :: "r"(dst), "l"(src), "n"(B), "r"(in ? B : 0) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(bar)) : "memory");
}

// (v & m) | c
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t m, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(v), "r"(m), "r"(c));
    return d;
}
// (v & m) ^ c
__device__ __forceinline__ uint32_t and_xor(uint32_t v, uint32_t m, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(v), "r"(m), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// ------------------------------------------------------------------ unpack
// A bf16 has seven fraction bits. Codes of B < 7 bits go to the top B of them
// under the exponent of 2^B (less kDown): 2^B + u, from which 2^B (superblocks) or
// 1.5 2^B (symmetric) is subtracted, all exact: a shift, a logic operation and a
// subtraction per two weights (two more for the bits above a nibble).
constexpr uint32_t code_base(int B) { return (uint32_t)(127 + B - kDown) << 7; }
__device__ __forceinline__ uint32_t shift_to(uint32_t w, int from, int to) { return from >= to ? w >> (from - to) : w << (to - from); }

// Eight nibbles of w as the pairs (0, 4), (1, 5), (2, 6), (3, 7); h holds the
// codes' B - 4 higher bits at bits 16 (k / 4) + (B - 4) (k % 4).
template <int B, bool SYM>
__device__ __forceinline__ void unpack_nibbles(uint32_t w, uint32_t h, uint32_t (&o)[4]) {
    if constexpr (B == 4) {
        // every other nibble stays at the bottom of the fraction, under the exponent of 2^7: one shift less
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t P = i & 1 ? 3u : 0u, E = code_base(i & 1 ? 4 : 7) * 0x10001u;
            o[i] = sub_bf16x2(and_or(shift_to(w, 4 * i, P), 0x000F000Fu << P, E), E | (SYM ? 0x00080008u << P : 0u));
        }
        return;
    }
    constexpr uint32_t P = 7 - B, M = 0x000F000Fu << P, E = code_base(B) * 0x10001u, OFF = E | (SYM ? 0x00400040u : 0u);
    constexpr uint32_t HM = (B == 5 ? 0x00010001u : 0x00030003u) << (P + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[i] = and_or(shift_to(w, 4 * i, P), M, E);
        if (B > 4) o[i] = and_or(shift_to(h, (B - 4) * i, P + 4), HM, o[i]);
        o[i] = sub_bf16x2(o[i], OFF);
    }
}
// Four bytes u = q + 128 of w as the pairs (0, 2), (1, 3): the low seven bits
// under 128, minus 128 where the byte's top bit is set and 256 where it is not
// (the next exponent, whose lowest bit is 1 as kDown is even).
__device__ __forceinline__ void unpack_bytes(uint32_t w, uint32_t (&o)[2]) {
    static_assert(kDown % 2 == 0, "the exponent of 128 is even");
    constexpr uint32_t E = code_base(7) * 0x10001u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t v = i ? w >> 8 : w;
        o[i] = sub_bf16x2(and_or(v, 0x007F007Fu, E), and_xor(v, 0x00800080u, E + 0x00800080u));
    }
}

// --------------------------------------------------------------- one stage
__device__ __forceinline__ float half_at(uint32_t w, int h) {
    return __half2float(__ushort_as_half((uint16_t)(h ? w >> 16 : w & 0xffffu)));
}

// A superblock stage's scales, each lane those of weight row wr + lane: S_j and
// M_j of the eight groups to shared memory.
template <int FMT>
__device__ __forceinline__ void decode_superblock(uint32_t cs, uint32_t smin, int wr, int lane) {
    using G = Geo<FMT>;
    const uint4 hd = lds128_a(cs + (uint32_t)(wr + lane) * G::RB);
    const float d = half_at(hd.x, 0), dm = half_at(hd.x, 1);
    __syncwarp();                                        // the previous stage's values have been read
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        // fields 2q and 2q + 1 of the scales (from bit 12 q of the string) and of the mins (from bit 48 + 12 q)
        const uint32_t f0 = q < 2 ? hd.y >> (12 * q) : __funnelshift_r(q == 2 ? hd.y : hd.z, q == 2 ? hd.z : 0u, (12 * q) & 31);
        const uint32_t f1 = q < 2 ? __funnelshift_r(hd.z, hd.w, 16 + 12 * q) : hd.w >> (12 * q - 16);
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};"
                     :: "r"(smin + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)), "f"(__fmul_rn(d, (float)(f0 & 63u))), "f"(__fmul_rn(dm, (float)(f1 & 63u))),
                        "f"(__fmul_rn(d, (float)((f0 >> 6) & 63u))), "f"(__fmul_rn(dm, (float)((f1 >> 6) & 63u))) : "memory");
    }
    __syncwarp();
}

__device__ __forceinline__ float lds_half(uint32_t a) { return __half2float(__ushort_as_half((uint16_t)lds16_a(a))); }

// One warp's share of a stage: weight rows wr .. wr + 31, all live 8-row
// tiles. acc[m16][tile]: D fragment (weight rows 16 m16 + lane / 4, + 8;
// activation rows 2 (lane % 4), + 1). cs, xs, ss: code, activation and scale
// blocks; smin: the warp's decoded superblock scales.
template <int FMT, int NB>
__device__ __forceinline__ void stage_math(uint32_t cs, uint32_t xs, uint32_t ss, uint32_t smin, int wr, int lane, int tiles,
                                           float (&acc)[2][NB][4]) {
    using G = Geo<FMT>;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t xl = xs + lane * 16;
    const uint32_t rb = cs + (uint32_t)(wr + g) * G::RB;                 // first of the thread's weight rows, 8 apart
    const uint32_t rs = ss + (uint32_t)(wr + g) * G::SB;
    if constexpr (FMT == kFmtW4G64 || FMT == kFmtW8G64) {
        // a group of 64: four steps into one sum
        constexpr int NG = G::KS / 64;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
            uint32_t a[2][4][4];                         // [m16][step][register]
            float s[4];
#pragma unroll
            for (int mr = 0; mr < 4; ++mr) {
                s[mr] = lds_half(rs + 8 * mr * G::SB + 2 * gr);
                if constexpr (FMT == kFmtW4G64) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t o[4];
                        unpack_nibbles<4, true>(lds32_a(rb + 8 * mr * G::RB + (((2 * gr + j) ^ g) << 4) + 4 * t), 0u, o);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            a[mr >> 1][2 * j + h][mr & 1] = o[2 * h];
                            a[mr >> 1][2 * j + h][2 + (mr & 1)] = o[2 * h + 1];
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t o[2];
                        unpack_bytes(lds32_a(rb + 8 * mr * G::RB + (((4 * gr + j) ^ g) << 4) + 4 * t), o);
                        a[mr >> 1][j][mr & 1] = o[0];
                        a[mr >> 1][j][2 + (mr & 1)] = o[1];
                    }
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if (NB > 1 && nb >= tiles) break;
                const uint4 x0 = lds128_a(xl + nb * G::XB + (2 * gr) * 512), x1 = lds128_a(xl + nb * G::XB + (2 * gr + 1) * 512);
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    float d[4];
                    mma16816(d, a[mt][0], x0.x, x0.y, 0.0f, 0.0f, 0.0f, 0.0f);
                    mma16816(d, a[mt][1], x0.z, x0.w, d[0], d[1], d[2], d[3]);
                    mma16816(d, a[mt][2], x1.x, x1.y, d[0], d[1], d[2], d[3]);
                    mma16816(d, a[mt][3], x1.z, x1.w, d[0], d[1], d[2], d[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[mt][nb][i] = fmaf(s[2 * mt + (i >> 1)], d[i], acc[mt][nb][i]);
                }
            }
        }
    } else if constexpr (FMT == kFmtW8G16 || FMT == kFmtW6G16) {
        // pairs of 16-weight steps, each a group of its own
#pragma unroll
        for (int sp = 0; sp < G::KS / 32; ++sp) {
            uint32_t a[2][2][4];
            float s[2][4];
#pragma unroll
            for (int mr = 0; mr < 4; ++mr) {
                const uint32_t w = lds32_a(rs + 8 * mr * G::SB + 4 * sp);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int st = 2 * sp + h;
                    s[h][mr] = half_at(w, h);
                    uint32_t o[2];
                    if constexpr (FMT == kFmtW6G16) {
                        const uint32_t b = rb + 8 * mr * G::RB + 48 * (st >> 2);
                        const uint32_t n = lds16_a(b + 8 * (st & 3) + 2 * t);
                        uint32_t pl;
                        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(pl) : "r"(b + 32 + 4 * (st & 3) + t));
                        const uint32_t v = n | (n << 8), hh = pl | (pl << 12);     // pairs (0, 2), (1, 3), as for the bytes
                        constexpr uint32_t E = code_base(6) * 0x10001u;
                        o[0] = sub_bf16x2(and_or(hh << 5, 0x00600060u, and_or(v << 1, 0x001E001Eu, E)), E | 0x00400040u);
                        o[1] = sub_bf16x2(and_or(hh << 3, 0x00600060u, and_or(v >> 3, 0x001E001Eu, E)), E | 0x00400040u);
                    } else {
                        unpack_bytes(lds32_a(rb + 8 * mr * G::RB + ((st ^ g) << 4) + 4 * t), o);
                    }
                    a[mr >> 1][h][mr & 1] = o[0];
                    a[mr >> 1][h][2 + (mr & 1)] = o[1];
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if (NB > 1 && nb >= tiles) break;
                const uint4 x = lds128_a(xl + nb * G::XB + sp * 512);
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    float d0[4], d1[4];
                    mma16816(d0, a[mt][0], x.x, x.y, 0.0f, 0.0f, 0.0f, 0.0f);
                    mma16816(d1, a[mt][1], x.z, x.w, 0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[mt][nb][i] = fmaf(s[0][2 * mt + (i >> 1)], d0[i], acc[mt][nb][i]);
                        acc[mt][nb][i] = fmaf(s[1][2 * mt + (i >> 1)], d1[i], acc[mt][nb][i]);
                    }
                }
            }
        }
    } else {
        // superblock groups of 32
        decode_superblock<FMT>(cs, smin, wr, lane);
#pragma unroll 2
        for (int gr = 0; gr < 8; ++gr) {
            uint32_t a[2][2][4];
            float2 sm2[4];
#pragma unroll
            for (int mr = 0; mr < 4; ++mr) {
                uint32_t o[4], h = 0u;
                const uint32_t r = rb + 8 * mr * G::RB;
                if constexpr (FMT == kFmtW5SB32) {
                    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(h) : "r"(r + 144 + 4 * gr + t));
                    h |= h << 12;
                } else if constexpr (FMT == kFmtW6SB32) {
                    h = lds16_a(r + 144 + 8 * gr + 2 * t);
                    h |= h << 8;
                }
                unpack_nibbles<sb_bits(FMT), false>(lds32_a(r + 16 + 16 * gr + 4 * t), h, o);
                sm2[mr] = lds64f_a(smin + (8 * mr + g) * 64 + (((gr >> 1) ^ ((g >> 1) & 3)) << 4) + 8 * (gr & 1));
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    a[mr >> 1][s][mr & 1] = o[2 * s];
                    a[mr >> 1][s][2 + (mr & 1)] = o[2 * s + 1];
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if (NB > 1 && nb >= tiles) break;
                const uint4 x = lds128_a(xl + nb * G::XB + gr * 512);
                const float2 c = lds64f_a(xs + nb * G::XB + G::KS * 16 + gr * 32 + t * 8);       // rows 2t, 2t + 1
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    float d[4];
                    mma16816(d, a[mt][0], x.x, x.y, 0.0f, 0.0f, 0.0f, 0.0f);
                    mma16816(d, a[mt][1], x.z, x.w, d[0], d[1], d[2], d[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 m = sm2[2 * mt + (i >> 1)];
                        acc[mt][nb][i] = fmaf(m.x, d[i], acc[mt][nb][i]);
                        acc[mt][nb][i] = fmaf(m.y, i & 1 ? c.y : c.x, acc[mt][nb][i]);
                    }
                }
            }
        }
    }
}

// ----------------------------------------------------------------- product
// One stretch of a unit in one CTA, written by the copy warp ahead of the
// stretch's first stage.
struct __align__(16) Desc {
    int rows;          // rows of the call
    int k0, k1;        // stages
    int n0;            // first weight row within the expert
    int row0;          // first row
    int first, last;   // CTAs that share the unit
    int pad;
};

__device__ __forceinline__ Desc read_desc(const Desc* p) {
    const uint4 a = lds128_a(smem_u32(p)), b = lds128_a(smem_u32(p) + 16);
    return {(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

struct Work { int e, n0, row0, rows, tile0; };   // a unit: expert, first weight row, first row and rows, first 8-row tile

__device__ __forceinline__ Work get_work(const Plan& pl, const Groups& g, long long unit) {
    const int e = find_group(g.unit, pl.E, unit), m = g.row[e + 1] - g.row[e];
    const int chunk = 8 * pl.NB, chunks = (m + chunk - 1) / chunk;
    const long long i = unit - g.unit[e];
    const int nt = i < 0x7fffffff ? (int)i / chunks : (int)(i / chunks), c = (int)(i - (long long)nt * chunks);
    Work w;
    w.e = e;
    w.n0 = nt * kRowsPerTile;
    w.row0 = g.row[e] + c * chunk;
    w.rows = min(chunk, m - c * chunk);
    w.tile0 = g.tile[e] + c * pl.NB;
    return w;
}

// v[0..7] to columns n .. n + 7 of y's row `out`.
__device__ __forceinline__ void store8(const RowsParams& p, int out, int n, const float (&v)[8]) {
    const int N = p.pl.N;
    const size_t o = (size_t)out * N + n;
    if ((N & 7) == 0 || ((N & 3) == 0 && !p.ybf16 && n + 8 <= N)) {
        if (p.ybf16) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.y) + o) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
            float* y = static_cast<float*>(p.y) + o;
            *reinterpret_cast<float4*>(y) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(y + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (n + q < N) store_y(p.y, o + q, v[q], p.ybf16);
    }
}

template <int FMT, int NB>
__global__ void __launch_bounds__(kRowsThreads, ctas_per_sm(FMT, NB)) rows_kernel(const __grid_constant__ RowsParams p) {
    using G = Geo<FMT>;
    extern __shared__ __align__(1024) uint8_t smem[];                    // the swizzled code tiles need this alignment
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ring = p.ring;
    uint8_t* at = smem + (size_t)ring * G::CB;
    const uint32_t xbase = smem_u32(at);
    at += kXRing * p.xslot;
    float* scratch = reinterpret_cast<float*>(at + warp * G::SCRATCH);   // of a math warp
    at += kMathWarps * G::SCRATCH;
    uint64_t* cfull = reinterpret_cast<uint64_t*>(at);
    uint64_t* cempty = cfull + kMaxRing;
    uint64_t* xfull = cempty + kMaxRing;
    uint64_t* xempty = xfull + kXRing;
    at += 2 * (kMaxRing + kXRing) * 8;
    Desc* desc = reinterpret_cast<Desc*>(at);
    at += kDescs * sizeof(Desc);
    const Groups g = groups_at(at, p.pl.E);

    if (tid == 0) {
        for (int s = 0; s < ring; ++s) {
            mbar_init(&cfull[s], 1);
            mbar_init(&cempty[s], kMathWarps);
        }
        for (int s = 0; s < kXRing; ++s) {
            mbar_init(&xfull[s], is_sb(FMT) ? 1 : 33);                   // the copy thread, and the scale copies of 32 lanes
            mbar_init(&xempty[s], kMathWarps);
        }
        fence_mbar_init();
    }
    if (warp == kMathWarps) scan_groups(p.pl, g, lane);
    __syncthreads();
    grid_dep_launch();

    const int T = p.pl.T;
    const long long S = g.unit[p.pl.E] * T;
    const long long Gc = min((long long)gridDim.x, S);                   // CTAs with work
    if ((long long)blockIdx.x >= Gc) {
        grid_dep_wait();                                                 // no kernel after this one runs beside prep_kernel
        return;
    }
    const long long s0 = blockIdx.x * S / Gc, s1 = ((long long)blockIdx.x + 1) * S / Gc;
    const int n = (int)(s1 - s0);                                        // stages of this CTA
    const uint32_t base = smem_u32(smem);
    constexpr uint32_t kSOff = NB * G::XB;                               // scales behind the activations of a slot

    if (warp == kMathWarps) {
        // ------------------------------------------------------------ copies
        // Two streams: code tiles, and activations with scales. The codes of
        // the first `ring` stages are asked for before the prepared
        // activations are waited for.
        const bool copies = !(p.test_flags & kTestNoCopies);
        if (!copies) return;
        struct Cursor {                                                  // walks the CTA's stages
            long long unit;
            int i, k, u;
            Work w;
        };
        auto begin = [&](Cursor& c) {
            c.unit = s0 / T;
            c.k = (int)(s0 - c.unit * T);
            c.i = c.u = 0;
            c.w = get_work(p.pl, g, c.unit);
        };
        auto next = [&](Cursor& c) {
            if (++c.i < n && ++c.k == T) {
                c.k = 0;
                ++c.u;
                c.w = get_work(p.pl, g, ++c.unit);
            }
        };
        auto codes = [&](const Cursor& c, int slot) {
            if (lane == 0) {
                mbar_arrive_expect_tx(&cfull[slot], (uint32_t)(kRowsPerTile * G::RB));
                tma_2d(base + slot * G::CB, &p.cmap, c.k * G::RB, c.w.e * p.pl.N + c.w.n0, &cfull[slot]);
            }
        };
        Cursor cc, cx;
        begin(cc);
        cx = cc;
        int cslot = 0, cwrap = 0, xslot = 0, xwrap = 0;
        bool ok = true;
        while (cc.i < min(n, ring)) {
            codes(cc, cslot);
            if (++cslot == ring) { cslot = 0; ++cwrap; }
            next(cc);
        }
        if (!p.z) grid_dep_wait();                       // with z, the kernel before this one waited for prep_kernel
        asm volatile("fence.proxy.async.global;" ::: "memory");
        // In the order in which slots come free: a stage's activations when
        // the stage kXRing before has been used, then the codes that follow
        // the ones taken out for the next stage.
        while (cx.i < n) {
            if (xwrap && !__all_sync(~0u, mbar_wait_bounded(&xempty[xslot], (uint32_t)(xwrap - 1) & 1u, kStatusSlotWait, 32u, p.wait_ns))) {
                ok = false;
                break;
            }
            const Work& w = cx.w;
            const uint32_t xs = xbase + xslot * p.xslot;
            const int tiles = (w.rows + 7) / 8, k = cx.k;
            if (lane == 0) {
                if (k == 0 || cx.i == 0) {
                    const long long us = cx.unit * T;
                    Desc d = {w.rows, k, min(T, k + n - cx.i), w.n0, w.row0, (int)blockIdx.x, (int)blockIdx.x, 0};
                    if (d.k0 > 0) d.first = (int)(((us + 1) * Gc - 1) / S);
                    if (d.k1 < T) d.last = (int)(((us + T) * Gc - 1) / S);
                    desc[cx.u % kDescs] = d;
                }
                mbar_arrive_expect_tx(&xfull[xslot], (uint32_t)(tiles * G::XB));
            }
            __syncwarp();
            if (NB == 1 && p.ad.row && k == 0) {                         // the adapters' B rows into L2, by the unit's first CTA
                const int a = lane < w.rows ? p.ad.row[w.row0 + lane] : -1;
                if (a >= 0 && a < p.ad.n && (lane == 0 || p.ad.row[w.row0 + lane - 1] != a))
                    prefetch_l2_bulk(p.ad.B + ((size_t)a * p.pl.N + w.n0) * p.ad.r, (uint32_t)(min(kRowsPerTile, p.pl.N - w.n0) * p.ad.r * 2));
            }
            if (lane < tiles)
                bulk_x(xs + lane * G::XB, p.xf + ((size_t)(w.tile0 + lane) * T + k) * G::XB, G::XB, &xfull[xslot]);
            if constexpr (!is_sb(FMT)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 32 * i + lane;
                    const unsigned long long row = min((unsigned long long)w.e * p.pl.N + w.n0 + r, p.total_rows - 1);
                    const uint8_t* src = p.scales + row * p.srb;
                    const uint32_t dst = xs + kSOff + r * G::SB;
                    const uint32_t b0 = k * G::SB;
                    if (G::SB >= 8 && (p.srb & 7u) == 0u) {
#pragma unroll
                        for (int b = 0; b < G::SB; b += 8) cp_async<8>(dst + b, b0 + b < p.srb ? src + b0 + b : src, b0 + b < p.srb);
                    } else if ((p.srb & 3u) == 0u) {
#pragma unroll
                        for (int b = 0; b < G::SB; b += 4) cp_async<4>(dst + b, b0 + b < p.srb ? src + b0 + b : src, b0 + b < p.srb);
                    } else {                                             // an odd number of scales per row
#pragma unroll
                        for (int b = 0; b < G::SB; b += 2) {
                            const uint16_t v = b0 + b < p.srb ? *reinterpret_cast<const uint16_t*>(src + b0 + b) : (uint16_t)0;
                            asm volatile("st.shared.u16 [%0], %1;" :: "r"(dst + b), "h"(v) : "memory");
                        }
                    }
                }
                if ((p.srb & 3u) == 0u) cp_async_arrive(&xfull[xslot]);
                else mbar_arrive(&xfull[xslot]);
            }
            next(cx);
            if (++xslot == kXRing) { xslot = 0; ++xwrap; }
            if (cc.i < n && cx.i >= kXRing) {
                if (!__all_sync(~0u, mbar_wait_bounded(&cempty[cslot], (uint32_t)(cwrap - 1) & 1u, kStatusSlotWait, 32u, p.wait_ns))) {
                    ok = false;
                    break;
                }
                codes(cc, cslot);
                if (++cslot == ring) { cslot = 0; ++cwrap; }
                next(cc);
            }
        }
        (void)ok;
        // copies in flight (a math warp gave up) land before the CTA leaves
        if (lane == 0) {
            for (int q = 0; q < ring && q < cc.i; ++q)
                mbar_wait_bounded(&cfull[q], (uint32_t)(cc.i / ring + (q < cc.i % ring ? 1 : 0) - 1) & 1u, kStatusTmaWait, 64u, p.wait_ns);
            for (int q = 0; q < kXRing && q < cx.i; ++q)
                mbar_wait_bounded(&xfull[q], (uint32_t)(cx.i / kXRing + (q < cx.i % kXRing ? 1 : 0) - 1) & 1u, kStatusTmaWait, 64u, p.wait_ns);
        }
        return;
    }

    // ---------------------------------------------------------------- math
    // A warp keeps to its own 32 weight rows from the codes to y: no barrier
    // among the warps. One whose wait runs out leaves.
    const int wr = 32 * warp;
    const uint32_t sm = smem_u32(scratch);
    int cslot = 0, cwrap = 0, xslot = 0, xwrap = 0, left = n;
    auto wait = [&](uint64_t* bar, int wrap) {
        return __all_sync(~0u, mbar_try_wait(bar, (uint32_t)wrap & 1u)) ||
               __all_sync(~0u, mbar_wait_bounded(bar, (uint32_t)wrap & 1u, kStatusTmaWait, 0u, p.wait_ns));
    };
    bool waited = false;
    for (int u = 0; left > 0; ++u) {
        if (!wait(&xfull[xslot], xwrap)) return;
        // The descriptor is read again after the stages, so that they keep no registers for it (its place is not
        // written before the copy warp is kDescs units ahead, more than the slots allow).
        const uint4 d0 = lds128_a(smem_u32(&desc[u % kDescs]));
        const int tiles = ((int)d0.x + 7) / 8, count = (int)d0.z - (int)d0.y;
        float acc[2][NB][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mt][nb][i] = 0.0f;
#pragma unroll 1
        for (int k = 0; k < count; ++k) {
            if (!wait(&cfull[cslot], cwrap)) return;
            const uint32_t cs = base + cslot * G::CB, xs = xbase + xslot * p.xslot;
            if (k && !wait(&xfull[xslot], xwrap)) return;
            stage_math<FMT, NB>(cs, xs, xs + kSOff, sm, wr, lane, tiles, acc);
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&cempty[cslot]);
                mbar_arrive(&xempty[xslot]);
            }
            if (++cslot == ring) { cslot = 0; ++cwrap; }
            if (++xslot == kXRing) { xslot = 0; ++xwrap; }
        }
        left -= count;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mt][nb][i] *= (float)(1 << kDown);

        const Desc d = read_desc(&desc[u % kDescs]);
        int out[NB];                                      // this lane's rows of y
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int i = 8 * nb + (lane >> 2), m = d.row0 + i;
            out[nb] = i >= d.rows ? -1 : p.out_rows ? p.out_rows[m] : m;
        }
        const int parts = d.last - d.first + 1;
        if (!waited) {
            grid_dep_wait();                              // counters and the adapters' terms come from the kernels before
            waited = true;
        }
        if constexpr (NB == 1) {
            if (p.ad.row) {
                // the parts of a unit share its ranks, 32 at a time
                const int i = lane >> 2, m = i < d.rows ? d.row0 + i : -1;
                for (int c = (int)blockIdx.x - d.first; 32 * c < p.ad.r; c += parts)
                    add_adapters(p.ad, m, c, d.n0 + wr + (lane >> 2), lane, acc[0][0], acc[1][0]);
            }
        }
        if (parts > 1) {
            // a part of a unit: CTA c's part lies in slot 2c (it began in an earlier CTA) or 2c + 1
            constexpr int kPart = kMathWarps * 2 * NB * 32;              // float4 per slot
            float4* part = reinterpret_cast<float4*>(p.part) + warp * (2 * NB * 32) + lane;
            float4* mypart = part + (size_t)(2 * blockIdx.x + (d.k0 == 0)) * kPart;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    if (nb < tiles)
                        __stcg(mypart + (mt * NB + nb) * 32, make_float4(acc[mt][nb][0], acc[mt][nb][1], acc[mt][nb][2], acc[mt][nb][3]));
                    acc[mt][nb][0] = acc[mt][nb][1] = acc[mt][nb][2] = acc[mt][nb][3] = 0.0f;
                }
            __threadfence();
            __syncwarp();
            unsigned old = 0;
            if (lane == 0) old = atomicAdd(&p.count[d.first * kMathWarps + warp], 1u);
            old = __shfl_sync(~0u, old, 0);
            if (old != (unsigned)(parts - 1)) continue;           // not the last to arrive
            __threadfence();
            constexpr int kAhead = NB == 1 ? 4 : NB == 2 ? 2 : 1;        // parts read together
            for (int c0 = d.first; c0 <= d.last; c0 += kAhead) {
                float4 v[kAhead][2][NB];
#pragma unroll
                for (int q = 0; q < kAhead; ++q)
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            const int c = c0 + q;
                            v[q][mt][nb] = c <= d.last && nb < tiles
                                ? __ldcg(part + (size_t)(2 * c + (c == d.first)) * kPart + (mt * NB + nb) * 32)
                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        }
#pragma unroll
                for (int q = 0; q < kAhead; ++q)
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            acc[mt][nb][0] += v[q][mt][nb].x;
                            acc[mt][nb][1] += v[q][mt][nb].y;
                            acc[mt][nb][2] += v[q][mt][nb].z;
                            acc[mt][nb][3] += v[q][mt][nb].w;
                        }
            }
        }
        // through shared memory to eight consecutive weight rows per lane
        const int nn = d.n0 + wr + 8 * (lane & 3);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            if (nb >= tiles) break;
            __syncwarp();
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // [activation row r][weight row], 16-byte chunks swizzled by r: no bank conflict either way
                    const int r = 2 * (lane & 3) + (i & 1), c = 16 * mt + (lane >> 2) + 8 * (i >> 1);
                    scratch[r * 32 + (((c >> 2) ^ r) << 2) + (c & 3)] = acc[mt][nb][i];
                }
            __syncwarp();
            if (out[nb] < 0 || out[nb] >= p.Ty || nn >= p.pl.N) continue;
            const float4* f = reinterpret_cast<const float4*>(scratch) + (lane >> 2) * 8;
            const float4 f0 = f[(2 * (lane & 3)) ^ (lane >> 2)], f1 = f[(2 * (lane & 3) + 1) ^ (lane >> 2)];
            float v[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
            if (p.z) {
                const float4* z = reinterpret_cast<const float4*>(p.z + (size_t)(d.row0 + 8 * nb + (lane >> 2)) * p.ldz + nn);
                const float4 z0 = __ldcg(z), z1 = __ldcg(z + 1);
                v[0] += z0.x; v[1] += z0.y; v[2] += z0.z; v[3] += z0.w;
                v[4] += z1.x; v[5] += z1.y; v[6] += z1.z; v[7] += z1.w;
            }
            if (p.act) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    v[q] = v[q] > 0.0f || v[q] != v[q] ? v[q] : 0.0f;
                    v[q] *= v[q];
                }
            }
            store8(p, out[nb], nn, v);
        }
        __syncwarp();                                     // scratch is read before it is written again
    }
}

// ------------------------------------------------------------------ host
constexpr int kMaxCtas = 768;          // CTAs of a launch at most

// 8-row tiles per unit: as many as an even split of the rows fills, since a
// group with more rows than a unit holds streams its weights once per unit. One
// tile up to four rows on average (w4g64, 64 rows of 16 experts: 42 us against
// 44 with two; a group of up to 16 rows then streams twice, from the L2), since
// a second tile costs a CTA per SM its registers and every stage its MMAs. Two
// up to 16 rows, for w4sb32 up to 64: four tiles of a superblock stage leave
// room for two CTAs per SM instead of three (8 experts, K 2560, N 2501, fp32:
// w4sb32 16 rows 28 against 34 us, 64 rows 59 and 64, 128 rows 102 both; w5sb32
// 16 rows 43 and 49, 32 rows 65 and 63; w4g64 16 rows 39.8 and 39.3).
template <int FMT>
int pick_nb(int R, int E) {
    const int per = (R + E - 1) / E;
    return R <= 8 || per <= 4 ? 1 : per <= (FMT == kFmtW4SB32 ? 64 : is_sb(FMT) ? 16 : 12) ? 2 : 4;
}

struct Layout { size_t xf, part, count, total; int tiles, T; };

template <int FMT>
Layout layout(int R, int K, int E) {
    Layout l;
    l.T = (K + Geo<FMT>::KS - 1) / Geo<FMT>::KS;
    l.tiles = R / 8 + (E < R ? E : R);                   // sum of ceil(m_e / 8) at most
    l.xf = 0;
    l.part = round16((size_t)l.tiles * l.T * Geo<FMT>::XB);
    l.count = l.part + (size_t)2 * kMaxCtas * pick_nb<FMT>(R, E) * 4096;
    l.total = l.count + kMaxCtas * kMathWarps * 4;
    return l;
}

template <int FMT, int NB>
cudaError_t launch_product(const RowsParams& p0, cudaStream_t st) {
    using G = Geo<FMT>;
    RowsParams p = p0;
    p.xslot = (NB * G::XB + kRowsPerTile * G::SB + 127) & ~127;
    const size_t fixed = kXRing * (size_t)p.xslot + kMathWarps * G::SCRATCH + 2 * (kMaxRing + kXRing) * 8 + kDescs * sizeof(Desc) +
                         groups_bytes(p.pl.E);
    constexpr size_t smem_max = kSmemPerSm / 2 - 1024;
    int per_sm = ctas_per_sm(FMT, NB);
    while (per_sm > 2 && kSmemPerSm / per_sm - 1024 < fixed + 2 * (size_t)G::CB) --per_sm;   // two code slots at least
    p.ring = (int)((kSmemPerSm / per_sm - 1024 - fixed) / G::CB);
    if (p.ring > kMaxRing) p.ring = kMaxRing;
    if (p.ring < 2) return cudaErrorInvalidValue;
    auto kern = rows_kernel<FMT, NB>;
    static unsigned long long attr_done = 0ull;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(__atomic_load_n(&attr_done, __ATOMIC_ACQUIRE) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_max);
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(&attr_done, bit, __ATOMIC_RELEASE);
    }
    int ctas = per_sm * sm_count();
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = fixed + (size_t)p.ring * G::CB;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int FMT>
cudaError_t launch_fmt(const RowsArgs& a, cudaStream_t st) {
    using G = Geo<FMT>;
    const EncodeTiled enc = encoder();
    if (!enc) return cudaErrorNotSupported;
    const Layout l = layout<FMT>(a.R, a.K, a.E);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    Plan pl = {a.offsets, a.E, a.R, a.N, a.K, l.T, pick_nb<FMT>(a.R, a.E)};

    PrepParams q = {};
    q.pl = pl;
    q.x = static_cast<const __nv_bfloat16*>(a.x);
    q.in_rows = a.in_rows;
    q.rows_x = a.T;
    q.xf = ws + l.xf;
    q.count = reinterpret_cast<unsigned*>(ws + l.count);
    q.n_count = kMaxCtas * kMathWarps;
    q.tiles_max = l.tiles;
    q.kblocks = (l.T * G::KS / 8 + kPrepChunks - 1) / kPrepChunks;
    if (!a.z) q.ad = a.ad;                                // with z the adapters' term is made elsewhere
    q.late = a.z != nullptr;
    const long long blocks = (long long)q.tiles_max * q.kblocks + (q.ad.row ? (long long)a.R * (q.ad.r / 8) : 0);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kPrepThreads);
    cfg.dynamicSmemBytes = groups_bytes(a.E);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = q.ad.row ? cudaLaunchKernelEx(&cfg, prep_kernel<FMT, true>, q) : cudaLaunchKernelEx(&cfg, prep_kernel<FMT, false>, q);
    if (e != cudaSuccess) return e;
    if (a.z) {
        e = launch_expand(a.ad, a.order, a.R, const_cast<float*>(a.z), a.ldz, st);
        if (e != cudaSuccess) return e;
    }

    RowsParams p = {};
    const uint64_t crb = code_row_bytes(FMT, a.K), rows = (uint64_t)a.E * a.N;
    const cuuint64_t dims[2] = {crb, rows}, strides[1] = {crb};
    const cuuint32_t box[2] = {(cuuint32_t)G::RB, (cuuint32_t)kRowsPerTile}, es[2] = {1, 1};
    if (enc(&p.cmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(a.codes), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, G::SWZ ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    p.pl = pl;
    p.scales = static_cast<const uint8_t*>(a.scales);
    p.total_rows = rows;
    p.srb = (uint32_t)scale_row_bytes(FMT, a.K);
    p.xf = ws + l.xf;
    p.part = reinterpret_cast<float*>(ws + l.part);
    p.count = reinterpret_cast<unsigned*>(ws + l.count);
    p.out_rows = a.out_rows;
    p.y = a.y;
    p.Ty = a.Ty;
    p.ybf16 = a.ybf16;
    p.act = a.act;
    p.ad = q.ad;
    p.z = a.z;
    p.ldz = a.ldz;
    p.wait_ns = wait_limit_ns();
    p.test_flags = test_flags();
    if (pl.NB == 1) return launch_product<FMT, 1>(p, st);
    if (pl.NB == 2) return launch_product<FMT, 2>(p, st);
    return launch_product<FMT, 4>(p, st);
}

}  // namespace

size_t rows_workspace(int fmt, int R, int K, int E) {
    switch (fmt) {
        case kFmtW4G64: return layout<kFmtW4G64>(R, K, E).total;
        case kFmtW8G16: return layout<kFmtW8G16>(R, K, E).total;
        case kFmtW8G64: return layout<kFmtW8G64>(R, K, E).total;
        case kFmtW6G16: return layout<kFmtW6G16>(R, K, E).total;
        case kFmtW4SB32: return layout<kFmtW4SB32>(R, K, E).total;
        case kFmtW5SB32: return layout<kFmtW5SB32>(R, K, E).total;
        default: return layout<kFmtW6SB32>(R, K, E).total;
    }
}

cudaError_t launch_rows(const RowsArgs& a, cudaStream_t st) {
    switch (a.fmt) {
        case kFmtW4G64: return launch_fmt<kFmtW4G64>(a, st);
        case kFmtW8G16: return launch_fmt<kFmtW8G16>(a, st);
        case kFmtW8G64: return launch_fmt<kFmtW8G64>(a, st);
        case kFmtW6G16: return launch_fmt<kFmtW6G16>(a, st);
        case kFmtW4SB32: return launch_fmt<kFmtW4SB32>(a, st);
        case kFmtW5SB32: return launch_fmt<kFmtW5SB32>(a, st);
        default: return launch_fmt<kFmtW6SB32>(a, st);
    }
}

cudaError_t status_rows(cudaStream_t st, unsigned* word) {
    unsigned v = 0, z = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_status, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    *word = v;
    return e;
}

}  // namespace rq
