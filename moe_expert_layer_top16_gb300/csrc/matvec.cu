// Products of a few rows with four-bit weights.
//
//   y[n][m] = sum_k w[m][k] x[n][k]     w: an E2M1 code times the E8M0 scale of
//             its 32, or (code - 8) times the scale of its 32, 64 or 128 in
//             fp16, bf16 or fp32;  x: fp32, bf16 or fp16, not quantised
//
// for one matrix and a few rows; for the expert of each slot; with a second
// matrix, SiLU(gate) up; or summed over a token's slots with its gates.
//
// The weights' way from HBM bounds it: every other cost has to hide behind some
// 45 bytes a nanosecond and SM, 22 a cycle, 44 weights.  Turning each weight into
// an fp32 and an FMA (three to four instructions a weight) would not, so that the
// products go through the tensor cores as well, m16n8k16 in fp16:
//
// - A lane holds 16 (or 8) consecutive bytes of codes of two rows, g and g + 8,
//   as they lie in memory: with the order of k inside an MMA free, those are the
//   A fragments of eight (four) MMAs, after one conversion for two weights.
//   E2M1 codes and integers from -8 to 7 are exact in fp16.
// - The four lanes of a row hold codes of four (two) different groups of 32, whose
//   scales differ.  B is block diagonal: its column (vector, group) holds the
//   vector's values in the rows of that group's lanes and zeros elsewhere, so that
//   each column of the accumulator belongs to one group and is scaled after its
//   32 products.  Of the MMA's eight columns four (two) serve a vector.
// - x goes to fp16 without losing its range: each 32 values are multiplied with the
//   power of two that brings the largest into [2^14, 2^15).  A bf16 or fp16 value is
//   then exact down to 2^-28 of the largest in its 32, and off by at most 2^-39 of
//   it below: eight bits of exponent less than an fp32 sum of the 32 would keep.
//   An fp32 value is three such parts, 12 bits apart, in three vectors.
// - Products and their sums over 32 (MMA) and over all groups are fp32.
//
// A team of warps takes 16 rows of the matrix, its warps take the units of K (what
// the MMAs of one load cover) in turn and add their sums in shared memory in a fixed
// order.
#include <algorithm>
#include <cuda_fp16.h>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace moe {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kRows = 16;                // rows of a team's tile
constexpr int kMvMaxThreads = 512;
constexpr int kMaxSegs = 32;             // slots of a token

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight codes as four pairs of fp16: E2M1 in order, (0, 1) (2, 3) (4, 5) (6, 7).
__device__ __forceinline__ void e2m1_pairs(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 p, q, r, s;\n\t"
        "mov.b32 {p, q, r, s}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, p;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, q;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, r;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, s;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// Integers c - 8, in the order (0, 4) (1, 5) (2, 6) (3, 7): a code in the low
// bits of an fp16 1024 is 1024 + c, four bits higher 1024 + 16 c.
__device__ __forceinline__ void int4_pairs(uint32_t w, uint32_t (&h)[4]) {
    const __half2 low = __float2half2_rn(-1032.0f), sixteenth = __float2half2_rn(0.0625f), high = __float2half2_rn(-72.0f);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint32_t a = ((w >> (8 * u)) & 0x000F000Fu) | 0x64006400u, b = ((w >> (8 * u)) & 0x00F000F0u) | 0x64006400u;
        __half2 p, q;
        memcpy(&p, &a, 4);
        memcpy(&q, &b, 4);
        p = __hadd2(p, low);
        q = __hfma2(q, sixteenth, high);
        memcpy(&h[2 * u], &p, 4);
        memcpy(&h[2 * u + 1], &q, 4);
    }
}

// Kinds of scale: E8M0 (with E2M1 codes), two bytes or four (with integers).
enum ScaleKind : int { SCALE_E8M0 = 0, SCALE_16 = 1, SCALE_32 = 2 };

// How a row's scales are loaded: a pair of groups of 32 as one word (rows start on
// whole words), one scale for both (groups of 64 and 128), or one by one.
enum ScaleLoad : int { LOAD_PAIR = 0, LOAD_ONE = 1, LOAD_TWO = 2 };

// What a lane loads for a unit of K of one matrix: its codes of rows g and g + 8
// and the scales of its two accumulator columns in both rows, as they lie in memory
// (a pair of 8 or 16 bits in s[0], s[2]).
template <int LV>
struct Codes {
    uint32_t lo[LV / 4], hi[LV / 4];
    uint32_t s[4];                       // row g: column 0, 1; row g + 8: column 0, 1
};

// The scales of groups kb and kb + 1 (of 32; the second may lie behind the last) of
// the row at `row`.
template <int SK>
__device__ __forceinline__ void load_scales(const uint8_t* row, int kb, int KB, int shift, int how, uint32_t& s0, uint32_t& s1) {
    using T = typename std::conditional<SK == SCALE_E8M0, uint8_t, typename std::conditional<SK == SCALE_16, uint16_t, uint32_t>::type>::type;
    const T* r = reinterpret_cast<const T*>(row);
    if (how == LOAD_PAIR) {
        if constexpr (SK == SCALE_E8M0)
            s0 = __ldg(reinterpret_cast<const uint16_t*>(r + kb));
        else if constexpr (SK == SCALE_16)
            s0 = __ldg(reinterpret_cast<const uint32_t*>(r + kb));
        else {
            const uint2 both = __ldg(reinterpret_cast<const uint2*>(r + kb));
            s0 = both.x;
            s1 = both.y;
        }
    } else if (how == LOAD_ONE) {
        s0 = __ldg(r + (kb >> shift));
    } else {
        s0 = __ldg(r + kb);
        s1 = kb + 1 < KB ? __ldg(r + kb + 1) : 0;
    }
}
template <int SK>
__device__ __forceinline__ float2 scale_values(uint32_t s0, uint32_t s1, int how, bool bf16) {
    if constexpr (SK == SCALE_E8M0) {
        const uint16_t two = static_cast<uint16_t>(how == LOAD_PAIR ? s0 : s0 | (s1 << 8));
        uint32_t v;                      // 2^-127 for code 0, NaN for 255
        asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(v) : "h"(two));
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    } else if constexpr (SK == SCALE_32) {
        return make_float2(__uint_as_float(s0), __uint_as_float(how == LOAD_ONE ? s0 : s1));
    } else {
        const uint32_t v = how == LOAD_PAIR ? s0 : s0 | ((how == LOAD_ONE ? s0 : s1) << 16);
        if (bf16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
        __half2 h;
        memcpy(&h, &v, 4);
        return __half22float2(h);
    }
}

// Weights go by once: past L1.
template <int LV>
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&w)[LV / 4]) {
    if constexpr (LV == 16) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "l"(p));
    } else {
        asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    }
}

__device__ __forceinline__ void ld_shared(uint32_t (&b)[4], uint32_t addr) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]) : "r"(addr));
}

// Shared memory: x as fp16 [unit][word of 8][vector][lane of the row], 16 bytes each;
// as many zero bytes as a unit has; factors [unit][vector][group] in fp32; the warps'
// sums [2][team][matrix][warp][row][vector].
template <int LV, int NT, bool DUAL>
struct Layout {
    static constexpr int UK = 8 * LV;            // k of a unit: four lanes' codes
    static constexpr int GP = UK / 32;           // groups of 32 in it
    static constexpr int VT = 8 / GP;            // vectors of an MMA's columns
    static constexpr int VS = NT * VT;           // vectors there is room for
    static constexpr int NM = DUAL ? 2 : 1;
    static constexpr int PF = 64 / LV / NM;      // units whose loads are in flight
    static constexpr int kUnitX = UK * VS * 2, kUnitF = VS * GP * 4;
    static constexpr int sums(int warps) { return 2 * NM * warps * kRows * VS * 4; }
};

template <int SK, int LV, int NT, bool DUAL>
__global__ void __launch_bounds__(kMvMaxThreads) matvec_kernel(const MatvecArgs a) {
    using L = Layout<LV, NT, DUAL>;
    constexpr int UK = L::UK, GP = L::GP, VT = L::VT, VS = L::VS, NM = L::NM, PF = L::PF;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int s_expert[kMaxSegs];
    __shared__ int64_t s_row[kMaxSegs];
    __shared__ float s_gate[kMaxSegs];
    __shared__ int s_segs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int KW = a.kw, team = warp / KW, kwarp = warp % KW, teams = (blockDim.x >> 5) / KW;
    const int64_t set = static_cast<int64_t>(blockIdx.x) % a.sets;
    const int part = static_cast<int>(blockIdx.x / a.sets);
    const int K = a.K, KB = K / 32, M = a.M, how = a.scale_load;
    const int cps = (K + UK - 1) / UK;   // units of a segment
    // the vectors: rows of x (one matrix), a slot's row, or a token's slots one behind the other
    const int nv = a.idx ? 1 : static_cast<int>(min(static_cast<int64_t>(a.nv), a.N - set * a.nv));
    if (warp == 0) {
        int n = 1;
        if (!a.idx) {
            if (lane == 0) {
                s_expert[0] = 0;
                s_row[0] = set * a.nv;
                s_gate[0] = 1.0f;
            }
        } else {
            const int per = a.weights ? a.k : 1;
            const int64_t slot = set * per + lane;
            const int e = lane < per ? a.idx[slot] : -1;
            const bool kept = e >= 0 && e < a.G;
            const uint32_t all = __ballot_sync(kAll, kept);
            n = __popc(all);
            if (kept) {
                const int at = __popc(all & ((1u << lane) - 1));
                s_expert[at] = e;
                s_row[at] = a.x_per_slot ? slot : slot / a.k;
                s_gate[at] = a.weights ? a.weights[slot] : 1.0f;
            }
        }
        if (lane == 0) s_segs = n;
    }
    const int cap = a.cap;               // units that fit
    uint8_t* xv = sm;
    uint8_t* zero = xv + static_cast<size_t>(cap) * L::kUnitX;
    float* xf = reinterpret_cast<float*>(zero + L::kUnitX);
    float* red = xf + static_cast<size_t>(cap) * (VS * GP);
    for (int i = threadIdx.x * 16; i < L::kUnitX; i += blockDim.x * 16) *reinterpret_cast<uint4*>(zero + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const int segs = s_segs, units = segs * cps;

    // x of the units [u0, u1) to shared memory: a thread takes eight values, four threads a group
    auto stage = [&](int u0, int u1) {
        constexpr int per_unit = UK / 8;
        const int vvt = nv * a.parts, total = (u1 - u0) * per_unit * nv;
        for (int i0 = 0; i0 < total; i0 += blockDim.x) {
            const int i = i0 + threadIdx.x;
            const bool in = i < total;
            const int c = i % per_unit, rest = in ? i / per_unit : 0, u = nv == 1 ? rest : rest / nv, n = rest - u * nv;
            const int seg = segs == 1 ? 0 : (u0 + u) / cps, k = ((u0 + u) - seg * cps) * UK + c * 8;
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 0.0f;
            if (in && k < K) {
                const int64_t off = (s_row[seg] + n) * a.ld_x + k;
                if (a.x_wide) {
                    raw_to_f32(load_raw<8>(a.x, off, a.dt_x), a.dt_x, f);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float e[1];
                        raw_to_f32(load_raw<1>(a.x, off + j, a.dt_x), a.dt_x, e);
                        f[j] = e[0];
                    }
                }
            }
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float m = fabsf(f[j]);
                if (m < INFINITY) top = fmaxf(top, m);          // infinities and NaN stay what they are
            }
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
            // 2^-ex brings it into [2^14, 2^15); the factors, with those of the parts, stay normal numbers
            int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14;
            ex = max(ex, a.parts == 1 ? -126 : -100);
            if (top == 0.0f) ex = 0;
            const float to = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);     // 2^-126 at least: ex <= 113
            const float back = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= to;
            const int word = LV == 16 ? c % 4 : c % 2, t = LV == 16 ? c / 4 : c / 2;
            uint4* xo = reinterpret_cast<uint4*>(xv) + ((u * (LV / 4) + word) * VS) * 4 + t;
            float* fo = xf + u * (VS * GP) + c / 4;
            for (int p = 0; p < a.parts; ++p) {
                __half h[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) h[j] = __float2half_rn(f[j]);
                if (a.parts > 1)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float r = (f[j] - __half2float(h[j])) * 4096.0f;
                        f[j] = r == r ? r : 0.0f;                // nothing is left of an infinity
                    }
                __half o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)                      // integers come in the order (0, 4) (1, 5) (2, 6) (3, 7)
                    o[j] = SK == SCALE_E8M0 ? h[j] : h[(j & 1) * 4 + j / 2];
                uint4 v;
                memcpy(&v, o, 16);
                const int vv = n * a.parts + p;
                if (in) {
                    xo[vv * 4] = v;
                    if ((c & 3) == 0) fo[vv * GP] = s_gate[seg] * back * __uint_as_float(static_cast<uint32_t>(127 - 12 * p) << 23);
                }
            }
            if (in && n == 0)                                    // vectors that are not there
                for (int vv = vvt; vv < VS; ++vv) {
                    xo[vv * 4] = make_uint4(0, 0, 0, 0);
                    if ((c & 3) == 0) fo[vv * GP] = 0.0f;
                }
        }
    };

    // this lane's places
    const int64_t row_bytes = K / 2, srow_bytes = static_cast<int64_t>(KB >> a.shift) * (SK == SCALE_E8M0 ? 1 : SK == SCALE_16 ? 2 : 4);
    const int kb_lane = LV == 16 ? 2 * (t4 & 1) : 0;                      // first group of its two columns
    const bool bf16 = a.dt_scale == ELEM_BF16;
    // B fragments: the lane's column is that of vector vb in group gb; values in the rows of that group's lanes,
    // zeros elsewhere
    const int vb = g / GP, gb = g % GP;
    const bool diagonal = gb == (LV == 16 ? t4 : t4 / 2);
    const uint32_t x_base = smem_u32(diagonal ? xv + (vb * 4 + t4) * 16 : zero);
    const uint32_t x_step = diagonal ? L::kUnitX : 0;
    const int vc = LV == 16 ? t4 / 2 : t4;                               // vector of its accumulator columns
    const float* f_lane = xf + vc * GP + kb_lane;

    const int tiles = (M + kRows - 1) / kRows;
    const int tile_step = a.blocks * teams;
    struct Place {                       // the rows of a tile
        int64_t lo, hi;
    };
    auto place = [&](int tile) {
        return Place{min(static_cast<int64_t>(tile) * kRows + g, static_cast<int64_t>(M) - 1),
                     min(static_cast<int64_t>(tile) * kRows + g + 8, static_cast<int64_t>(M) - 1)};
    };
    Codes<LV> q[PF][NM];
    // unit u of the rows at p
    auto fetch = [&](Codes<LV> (&w)[NM], const Place& p, int u) {
        int64_t e = s_expert[0];
        int c = u;
        if (segs > 1) {
            const int seg = u / cps;
            c = u - seg * cps;
            e = s_expert[seg];
        }
        const int64_t lo = e * M + p.lo, hi = e * M + p.hi;
        const int k = c * UK + t4 * (2 * LV), kb = c * GP + kb_lane;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const uint8_t* codes = (m ? a.up_codes : a.codes) + k / 2;
            const uint8_t* scales = m ? a.up_scales : a.scales;
            if (k < K) {
                load_codes<LV>(codes + lo * row_bytes, w[m].lo);
                load_codes<LV>(codes + hi * row_bytes, w[m].hi);
            } else {
#pragma unroll
                for (int i = 0; i < LV / 4; ++i) w[m].lo[i] = w[m].hi[i] = 0;
            }
            w[m].s[0] = w[m].s[1] = w[m].s[2] = w[m].s[3] = 0;
            if (kb < KB) {
                load_scales<SK>(scales + lo * srow_bytes, kb, KB, a.shift, how, w[m].s[0], w[m].s[1]);
                load_scales<SK>(scales + hi * srow_bytes, kb, KB, a.shift, how, w[m].s[2], w[m].s[3]);
            }
        }
    };

    float acc[NM][NT][2];
    // adds the products of a unit whose x is number ul in shared memory
    auto work = [&](const Codes<LV> (&w)[NM], int ul) {
        const uint32_t x_at = x_base + ul * x_step;
        float c[NM][NT][4];
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) c[m][n][0] = c[m][n][1] = c[m][n][2] = c[m][n][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < LV / 4; ++i) {
            uint32_t b[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) ld_shared(b[n], x_at + (i * VS + n * VT) * 64);
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                uint32_t lo[4], hi[4];
                if constexpr (SK == SCALE_E8M0) {
                    e2m1_pairs(w[m].lo[i], lo);
                    e2m1_pairs(w[m].hi[i], hi);
                } else {
                    int4_pairs(w[m].lo[i], lo);
                    int4_pairs(w[m].hi[i], hi);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_16816(c[m][n], lo[0], hi[0], lo[1], hi[1], b[n][0], b[n][1]);
                    mma_16816(c[m][n], lo[2], hi[2], lo[3], hi[3], b[n][2], b[n][3]);
                }
            }
        }
        // behind the last group codes, values and scales are zero
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const float2 s = scale_values<SK>(w[m].s[0], w[m].s[1], how, bf16), r = scale_values<SK>(w[m].s[2], w[m].s[3], how, bf16);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 f = *reinterpret_cast<const float2*>(f_lane + (ul * VS + n * VT) * GP);
                acc[m][n][0] = fmaf(c[m][n][1] * s.y, f.y, fmaf(c[m][n][0] * s.x, f.x, acc[m][n][0]));
                acc[m][n][1] = fmaf(c[m][n][3] * r.y, f.y, fmaf(c[m][n][2] * r.x, f.x, acc[m][n][1]));
            }
        }
    };

    // A warp's units of a tile are a run of them, PF of them in flight; the loads of the next tile's first ones are
    // issued while the last of this one's are worked on.
    const bool whole = units <= cap;     // all of x fits: staged once
    bool ahead = false;                  // q holds the first units already
    int flip = 0;
    for (int tile0 = part * teams; tile0 < tiles; tile0 += tile_step) {
        const int tile = tile0 + team;
        const bool live = tile < tiles;
        const Place here = place(tile), next = place(tile + tile_step);
        const bool more = whole && tile + tile_step < tiles;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = 0.0f;
        for (int u0 = 0; u0 < units; u0 += cap) {
            const int u1 = min(u0 + cap, units), per = (u1 - u0 + KW - 1) / KW;
            const int first = min(u0 + kwarp * per, u1), last = min(first + per, u1);
            if (live && !ahead)
#pragma unroll
                for (int i = 0; i < PF; ++i)
                    if (first + i < last) fetch(q[i], here, first + i);
            if (!whole || tile0 == part * teams) {
                __syncthreads();
                stage(u0, u1);
                __syncthreads();
            }
            if (!live) continue;
            for (int ub = first; ub < last; ub += PF) {
                const bool end = ub + PF >= last;
#pragma unroll
                for (int i = 0; i < PF; ++i) {
                    if (ub + i < last) work(q[i], ub + i - u0);
                    if (!end) {
                        if (ub + PF + i < last) fetch(q[i], here, ub + PF + i);
                    } else if (more && first + i < last) {
                        fetch(q[i], next, first + i);
                    }
                }
            }
            ahead = more;
        }
        // the warps' sums, then the rows' outputs
        float* mine = red + (flip * teams + team) * (NM * KW * kRows * VS);
        flip ^= 1;
        if (live) {
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float lo = acc[m][n][0], hi = acc[m][n][1];
                    if (LV == 16) {
                        lo += __shfl_xor_sync(kAll, lo, 1);
                        hi += __shfl_xor_sync(kAll, hi, 1);
                    }
                    if (LV == 8 || (t4 & 1) == 0) {
                        mine[((m * KW + kwarp) * VS + n * VT + vc) * kRows + g] = lo;
                        mine[((m * KW + kwarp) * VS + n * VT + vc) * kRows + g + 8] = hi;
                    }
                }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(KW * 32) : "memory");
            for (int o = threadIdx.x - team * KW * 32; o < kRows * nv; o += KW * 32) {
                const int r = o % kRows, n = o / kRows;
                const int64_t m = static_cast<int64_t>(tile) * kRows + r;
                if (m >= M) continue;
                float y[NM];
#pragma unroll
                for (int x = 0; x < NM; ++x) {
                    y[x] = 0.0f;
                    for (int w = 0; w < KW; ++w)
                        for (int p = 0; p < a.parts; ++p) y[x] += mine[((x * KW + w) * VS + n * a.parts + p) * kRows + r];
                }
                float v[1] = {y[0]};
                if constexpr (DUAL) v[0] = y[0] / (1.0f + expf(-y[0])) * y[1];
                store_vec(a.out, (set * a.nv + n) * a.ld_out + m, a.dt_out, v);
            }
        }
    }
}

// Warps of a block, of a team and blocks of a set.  Two blocks of 8 warps an SM where x fits, else one of 16.  A block
// takes a set's tiles in rounds, a round as long as a warp's run of units and some three more for its start and end:
// the split of K among a team's warps that makes that shortest.
template <int SK, int LV, int NT, bool DUAL>
cudaError_t matvec_as(MatvecArgs a, cudaStream_t s) {
    using L = Layout<LV, NT, DUAL>;
    const int tiles = (a.M + kRows - 1) / kRows;
    const int64_t units = static_cast<int64_t>(a.weights ? a.k : 1) * ((a.K + L::UK - 1) / L::UK);
    const size_t unit_bytes = L::kUnitX + L::kUnitF;
    const bool two = units * unit_bytes + L::kUnitX + L::sums(8) <= 108 * 1024;
    const int warps = two ? 8 : 16, resident = two ? 304 : 152;
    a.cap = static_cast<int>(std::min<int64_t>(units, (220 * 1024 - L::kUnitX - L::sums(16)) / unit_bytes));
    const size_t smem = a.cap * unit_bytes + L::kUnitX + L::sums(warps);
    if (smem > 40 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(matvec_kernel<SK, LV, NT, DUAL>, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
        if (err != cudaSuccess) return err;
    }
    // a set of its own for each slot: some four rounds of blocks, as many of them may have nothing to do
    const int64_t most = a.idx ? std::max<int64_t>(1, (4 * resident + a.sets - 1) / a.sets) : std::max<int64_t>(1, resident / a.sets);
    int64_t best = INT64_MAX;
    for (int kw = 1; kw <= warps; kw *= 2) {
        const int teams = warps / kw;
        const int64_t blocks = std::min<int64_t>((tiles + teams - 1) / teams, most);
        const int64_t rounds = (tiles + blocks * teams - 1) / (blocks * teams), waves = (a.sets * blocks + resident - 1) / resident;
        const int64_t cost = waves * rounds * ((units + kw - 1) / kw + 3);
        if (cost < best) {
            best = cost;
            a.kw = kw;
            a.blocks = static_cast<int>(blocks);
        }
    }
    matvec_kernel<SK, LV, NT, DUAL><<<static_cast<unsigned>(a.sets * a.blocks), warps * 32, smem, s>>>(a);
    return cudaGetLastError();
}

template <int SK, bool DUAL>
cudaError_t matvec_of(const MatvecArgs& a, cudaStream_t s) {
    const int vv = a.nv * a.parts;
    if (vv <= 2) return matvec_as<SK, 16, 1, DUAL>(a, s);
    if (vv <= 4) return matvec_as<SK, 8, 1, DUAL>(a, s);
    if (vv <= 8) return matvec_as<SK, 8, 2, DUAL>(a, s);
    return matvec_as<SK, 8, 3, DUAL>(a, s);
}

}  // namespace

cudaError_t launch_matvec(MatvecArgs a, cudaStream_t s) {
    a.parts = a.dt_x == ELEM_F32 ? 3 : 1;
    if (a.idx) {
        a.nv = 1;
        a.sets = a.weights ? a.N : a.N * a.k;
    } else {
        const int most = a.parts == 3 ? 4 : 8;
        a.nv = static_cast<int>(std::min<int64_t>(a.N, most));
        a.sets = (a.N + a.nv - 1) / a.nv;
    }
    if (a.sets == 0) return cudaSuccess;
    a.x_wide = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.ld_x * elem_bytes(a.dt_x)) % 16 == 0;
    const int size = a.format == 0 ? 1 : elem_bytes(a.dt_scale);
    const bool pairs = (a.K / 32) % 2 == 0 && reinterpret_cast<uintptr_t>(a.scales) % (2 * size) == 0 &&
                       reinterpret_cast<uintptr_t>(a.up_scales) % (2 * size) == 0;
    a.scale_load = a.shift > 0 ? LOAD_ONE : pairs ? LOAD_PAIR : LOAD_TWO;
    if (a.format == 0) return a.up_codes ? matvec_of<SCALE_E8M0, true>(a, s) : matvec_of<SCALE_E8M0, false>(a, s);
    if (a.dt_scale == ELEM_F32) return a.up_codes ? matvec_of<SCALE_32, true>(a, s) : matvec_of<SCALE_32, false>(a, s);
    return a.up_codes ? matvec_of<SCALE_16, true>(a, s) : matvec_of<SCALE_16, false>(a, s);
}

}  // namespace moe
