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

__device__ __forceinline__ float e8m0_value(uint32_t c) {
    return __uint_as_float(c == 0 ? 0x00400000u : (c == 255u ? 0x7FC00000u : c << 23));
}

// What a lane loads for a unit of K of one matrix: its codes of rows g and g + 8
// and the scales of its two accumulator columns in both rows, as they lie in memory.
template <int LV>
struct Codes {
    uint32_t lo[LV / 4], hi[LV / 4];
    uint32_t s[4];                       // row g: column 0, 1; row g + 8: column 0, 1
};

struct RowPart {                         // of one matrix, for one lane
    const uint8_t *lo, *hi;              // codes of the rows, at the lane's place in unit 0
    const uint8_t *slo, *shi;            // scales of the rows
};

// The scales of groups kb and kb + 1 (units of 32 along K; the second may lie behind
// the last) of one row.  Two groups of 32 that lie in one word are loaded together
// where rows start on whole words.
template <int SK>
__device__ __forceinline__ void load_scales(const uint8_t* row, int kb, int KB, int shift, bool pairs, uint32_t& s0, uint32_t& s1) {
    s0 = s1 = 0;
    if (kb >= KB) return;
    if constexpr (SK == SCALE_E8M0) {
        if (pairs) {
            const uint32_t both = *reinterpret_cast<const uint16_t*>(row + kb);
            s0 = both & 0xFFu;
            s1 = both >> 8;
        } else {
            s0 = row[kb];
            if (kb + 1 < KB) s1 = row[kb + 1];
        }
    } else if constexpr (SK == SCALE_16) {
        const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
        if (shift > 0) {
            s0 = s1 = r[kb >> shift];
        } else if (pairs) {
            const uint32_t both = *reinterpret_cast<const uint32_t*>(r + kb);
            s0 = both & 0xFFFFu;
            s1 = both >> 16;
        } else {
            s0 = r[kb];
            if (kb + 1 < KB) s1 = r[kb + 1];
        }
    } else {
        const uint32_t* r = reinterpret_cast<const uint32_t*>(row);
        if (shift > 0) {
            s0 = s1 = r[kb >> shift];
        } else if (pairs) {
            const uint2 both = *reinterpret_cast<const uint2*>(r + kb);
            s0 = both.x;
            s1 = both.y;
        } else {
            s0 = r[kb];
            if (kb + 1 < KB) s1 = r[kb + 1];
        }
    }
}
template <int SK>
__device__ __forceinline__ float scale_value(uint32_t s, bool bf16) {
    if constexpr (SK == SCALE_E8M0) return e8m0_value(s);
    if constexpr (SK == SCALE_32) return __uint_as_float(s);
    return bf16 ? __uint_as_float(s << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(s)));
}

template <int LV>
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&w)[LV / 4]) {
    if constexpr (LV == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[1] = v.y;
    }
}

// 16 bytes of shared memory where `on`; the registers keep what they hold (zeros) elsewhere.
__device__ __forceinline__ void ld_shared_if(uint32_t (&b)[4], uint32_t addr, bool on) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3])
                 : "r"(addr), "r"(static_cast<int>(on))
                 : "memory");
}

template <int SK, int LV, int NT, bool DUAL>
__global__ void __launch_bounds__(kMvMaxThreads) matvec_kernel(const MatvecArgs a) {
    constexpr int UK = 8 * LV;           // k of a unit: four lanes' codes
    constexpr int GP = UK / 32;          // groups of 32 in it
    constexpr int VT = 8 / GP;           // vectors of an MMA's columns
    constexpr int NM = DUAL ? 2 : 1;
    constexpr int PF = 2;                // units whose loads are in flight
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int s_expert[kMaxSegs];
    __shared__ int64_t s_row[kMaxSegs];
    __shared__ float s_gate[kMaxSegs];
    __shared__ int s_segs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int KW = a.kw, team = warp / KW, kwarp = warp % KW, teams = (blockDim.x >> 5) / KW;
    const int64_t set = static_cast<int64_t>(blockIdx.x) % a.sets;
    const int part = static_cast<int>(blockIdx.x / a.sets);
    const int K = a.K, KB = K / 32, M = a.M;
    const int cps = (K + UK - 1) / UK;   // units of a segment
    // the vectors: rows of x (one matrix), a slot's row, or a token's slots one behind the other
    const int nv = a.idx ? 1 : static_cast<int>(min(static_cast<int64_t>(a.nv), a.N - set * a.nv));
    const int vvt = nv * a.parts;
    if (threadIdx.x == 0) {
        int n = 0;
        if (!a.idx) {
            s_expert[0] = 0;
            s_row[0] = set * a.nv;
            s_gate[0] = 1.0f;
            n = 1;
        } else {
            const int64_t first = a.weights ? set * a.k : set;
            for (int j = 0; j < (a.weights ? a.k : 1); ++j) {
                const int e = a.idx[first + j];
                if (e < 0 || e >= a.G) continue;
                s_expert[n] = e;
                s_row[n] = a.x_per_slot ? first + j : (first + j) / a.k;
                s_gate[n] = a.weights ? a.weights[first + j] : 1.0f;
                ++n;
            }
        }
        s_segs = n;
    }
    __syncthreads();
    const int segs = s_segs, units = segs * cps;
    // shared memory: fp16 values [unit][word of 8][vector][lane of the row], 16 bytes each; scales
    // [unit][vector][group]; the warps' sums [2][team][matrix][kwarp][row][vector]
    const int cap = a.cap;               // units that fit
    uint4* xv = reinterpret_cast<uint4*>(sm);
    const int vmax = a.nv * a.parts;
    float* xs = reinterpret_cast<float*>(sm + static_cast<size_t>(cap) * vmax * UK * 2);
    float* red = xs + static_cast<size_t>(cap) * vmax * GP;
    const int red_team = NM * KW * kRows * vmax;

    // x of the units [u0, u1) to shared memory: a thread takes eight values, four threads a group
    auto stage = [&](int u0, int u1) {
        const int per_unit = UK / 8;
        const int total = (u1 - u0) * per_unit * nv;
        for (int i0 = 0; i0 < total; i0 += blockDim.x) {
            const int i = i0 + threadIdx.x;
            const bool in = i < total;
            const int c = in ? i % per_unit : 0, rest = in ? i / per_unit : 0, n = rest % nv, u = rest / nv;
            const int seg = (u0 + u) / cps, k = ((u0 + u) - seg * cps) * UK + c * 8;
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
            const float down = ex >= 0 ? __uint_as_float(static_cast<uint32_t>(127 - ex) << 23) : 1.0f;
            const float up = ex < 0 ? __uint_as_float(static_cast<uint32_t>(127 - ex) << 23) : 1.0f;
            const float back = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] * down * up;
            const int word = LV == 16 ? c % 4 : c % 2, t = LV == 16 ? c / 4 : c / 2;
            for (int p = 0; p < a.parts; ++p) {
                __half h[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    h[j] = __float2half_rn(f[j]);
                    const float r = (f[j] - __half2float(h[j])) * 4096.0f;
                    f[j] = r == r ? r : 0.0f;                    // nothing is left of an infinity
                }
                __half o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)                      // integers come in the order (0, 4) (1, 5) (2, 6) (3, 7)
                    o[j] = SK == SCALE_E8M0 ? h[j] : h[(j & 1) * 4 + j / 2];
                uint4 v;
                memcpy(&v, o, 16);
                if (in) {
                    const int vv = n * a.parts + p;
                    xv[((u * (LV / 4) + word) * vvt + vv) * 4 + t] = v;
                    if ((c & 3) == 0)
                        xs[(u * vvt + vv) * GP + c / 4] = s_gate[seg] * back * __uint_as_float(static_cast<uint32_t>(127 - 12 * p) << 23);
                }
            }
        }
    };

    // this lane's places
    const int64_t row_bytes = K / 2, srow_bytes = static_cast<int64_t>(KB >> a.shift) * (SK == SCALE_E8M0 ? 1 : SK == SCALE_16 ? 2 : 4);
    const int kb_lane = LV == 16 ? 2 * (t4 & 1) : 0;                      // first group of its two columns
    auto load = [&](Codes<LV>& q, const RowPart& r, int64_t e, int c) {
        const int k = c * UK + t4 * (2 * LV);
        const int64_t at = e * M * row_bytes + static_cast<int64_t>(c) * (UK / 2);
        if (k < K) {
            load_codes<LV>(r.lo + at, q.lo);
            load_codes<LV>(r.hi + at, q.hi);
        } else {
#pragma unroll
            for (int w = 0; w < LV / 4; ++w) q.lo[w] = q.hi[w] = 0;
        }
        const int64_t sat = e * M * srow_bytes;
        load_scales<SK>(r.slo + sat, c * GP + kb_lane, KB, a.shift, a.scale_pairs, q.s[0], q.s[1]);
        load_scales<SK>(r.shi + sat, c * GP + kb_lane, KB, a.shift, a.scale_pairs, q.s[2], q.s[3]);
    };

    const bool bf16 = a.dt_scale == ELEM_BF16;
    // B fragments: the lane's column is that of vector vb in group gb; nonzero in the rows of that group's lanes
    const int vb = g / GP, gb = g % GP;
    const bool diagonal = gb == (LV == 16 ? t4 : t4 / 2);
    const uint32_t xv_base = smem_u32(xv);
    const int vc = LV == 16 ? t4 / 2 : t4;                               // vector of its accumulator columns

    const int tiles = (M + kRows - 1) / kRows;
    int flip = 0;
    bool staged = false;
    for (int tile0 = part * teams; tile0 < tiles; tile0 += a.blocks * teams) {
        const int tile = tile0 + team;
        const bool live = tile < tiles;
        const int r0 = min(tile * kRows + g, M - 1), r1 = min(tile * kRows + g + 8, M - 1);
        RowPart rp[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const uint8_t* codes = m ? a.up_codes : a.codes;
            const uint8_t* scales = m ? a.up_scales : a.scales;
            rp[m] = {codes + r0 * row_bytes + t4 * LV, codes + r1 * row_bytes + t4 * LV, scales + r0 * srow_bytes,
                     scales + r1 * srow_bytes};
        }
        float acc[NM][NT][2];
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = 0.0f;
        for (int u0 = 0; u0 < units; u0 += cap) {
            const int u1 = min(u0 + cap, units);
            Codes<LV> q[PF][NM];
            auto fetch = [&](int i, int u) {
                int64_t e = s_expert[0];
                int c = u;
                if (segs > 1) {
                    const int seg = u / cps;
                    c = u - seg * cps;
                    e = s_expert[seg];
                }
#pragma unroll
                for (int m = 0; m < NM; ++m) load(q[i][m], rp[m], e, c);
            };
            if (live)
#pragma unroll
                for (int i = 0; i < PF; ++i)
                    if (u0 + kwarp + i * KW < u1) fetch(i, u0 + kwarp + i * KW);
            if (!staged || units > cap) {
                if (staged) __syncthreads();
                stage(u0, u1);
                __syncthreads();
                staged = true;
            }
            if (!live) continue;
            uint32_t b[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n][0] = b[n][1] = b[n][2] = b[n][3] = 0;
            for (int ub = u0 + kwarp; ub < u1; ub += PF * KW) {
#pragma unroll
                for (int i = 0; i < PF; ++i) {
                    const int u = ub + i * KW;
                    if (u >= u1) break;
                    float c[NM][NT][4];
#pragma unroll
                    for (int m = 0; m < NM; ++m)
#pragma unroll
                        for (int n = 0; n < NT; ++n) c[m][n][0] = c[m][n][1] = c[m][n][2] = c[m][n][3] = 0.0f;
                    const int ul = u - u0;
#pragma unroll
                    for (int w = 0; w < LV / 4; ++w) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            ld_shared_if(b[n], xv_base + (((ul * (LV / 4) + w) * vvt + n * VT + vb) * 4 + t4) * 16,
                                         diagonal && n * VT + vb < vvt);
#pragma unroll
                        for (int m = 0; m < NM; ++m) {
                            uint32_t lo[4], hi[4];
                            if constexpr (SK == SCALE_E8M0) {
                                e2m1_pairs(q[i][m].lo[w], lo);
                                e2m1_pairs(q[i][m].hi[w], hi);
                            } else {
                                int4_pairs(q[i][m].lo[w], lo);
                                int4_pairs(q[i][m].hi[w], hi);
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                mma_16816(c[m][n], lo[0], hi[0], lo[1], hi[1], b[n][0], b[n][1]);
                                mma_16816(c[m][n], lo[2], hi[2], lo[3], hi[3], b[n][2], b[n][3]);
                            }
                        }
                    }
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        const float s0 = scale_value<SK>(q[i][m].s[0], bf16), s1 = scale_value<SK>(q[i][m].s[1], bf16);
                        const float s2 = scale_value<SK>(q[i][m].s[2], bf16), s3 = scale_value<SK>(q[i][m].s[3], bf16);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const int vv = n * VT + vc;
                            if (vv < vvt) {
                                const float2 f = *reinterpret_cast<const float2*>(xs + (ul * vvt + vv) * GP + kb_lane);
                                // behind the last group codes, values and scales are zero
                                acc[m][n][0] = fmaf(c[m][n][1] * s1, f.y, fmaf(c[m][n][0] * s0, f.x, acc[m][n][0]));
                                acc[m][n][1] = fmaf(c[m][n][3] * s3, f.y, fmaf(c[m][n][2] * s2, f.x, acc[m][n][1]));
                            }
                        }
                    }
                    if (u + PF * KW < u1) fetch(i, u + PF * KW);
                }
            }
        }
        // the warps' sums, then the rows' outputs
        float* mine = red + (flip * teams + team) * red_team;
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
                    const int vv = n * VT + vc;
                    if (vv < vvt && (LV == 8 || (t4 & 1) == 0)) {
                        mine[((m * KW + kwarp) * kRows + g) * vmax + vv] = lo;
                        mine[((m * KW + kwarp) * kRows + g + 8) * vmax + vv] = hi;
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
                        for (int p = 0; p < a.parts; ++p) y[x] += mine[((x * KW + w) * kRows + r) * vmax + n * a.parts + p];
                }
                float v[1] = {y[0]};
                if constexpr (DUAL) v[0] = y[0] / (1.0f + expf(-y[0])) * y[1];
                store_vec(a.out, (set * a.nv + n) * a.ld_out + m, a.dt_out, v);
            }
        }
    }
}

template <int SK, int LV, int NT, bool DUAL>
cudaError_t matvec_as(MatvecArgs a, cudaStream_t s) {
    constexpr int UK = 8 * LV, GP = UK / 32, NM = DUAL ? 2 : 1;
    const int vmax = a.nv * a.parts, tiles = (a.M + kRows - 1) / kRows;
    const int64_t units = static_cast<int64_t>(a.weights ? a.k : 1) * ((a.K + UK - 1) / UK);
    const size_t unit_bytes = static_cast<size_t>(vmax) * (UK * 2 + GP * 4);
    a.kw = 8;
    int teams = 1;
    auto sums = [&](int tm) { return sizeof(float) * 2 * static_cast<size_t>(tm) * NM * a.kw * kRows * vmax; };
    if (units * unit_bytes > 40 * 1024) teams = 2;
    a.cap = static_cast<int>(std::min<int64_t>(units, (200 * 1024 - sums(teams)) / unit_bytes));
    const size_t smem = a.cap * unit_bytes + sums(teams);
    if (smem > 40 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(matvec_kernel<SK, LV, NT, DUAL>, cudaFuncAttributeMaxDynamicSharedMemorySize, 201 * 1024);
        if (err != cudaSuccess) return err;
    }
    // blocks for a set of vectors: about as many as run at once
    const int64_t at_once = 152 * std::max<int64_t>(1, std::min<int64_t>(4 / teams, 220 * 1024 / (smem + 1024)));
    a.blocks = static_cast<int>(std::min<int64_t>((tiles + teams - 1) / teams, std::max<int64_t>(1, (at_once + a.sets - 1) / a.sets)));
    matvec_kernel<SK, LV, NT, DUAL><<<static_cast<unsigned>(a.sets * a.blocks), teams * a.kw * 32, smem, s>>>(a);
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
    a.scale_pairs = a.shift == 0 && (a.K / 32) % 2 == 0 && reinterpret_cast<uintptr_t>(a.scales) % (2 * size) == 0 &&
                    reinterpret_cast<uintptr_t>(a.up_scales) % (2 * size) == 0;
    if (a.format == 0) return a.up_codes ? matvec_of<SCALE_E8M0, true>(a, s) : matvec_of<SCALE_E8M0, false>(a, s);
    if (a.dt_scale == ELEM_F32) return a.up_codes ? matvec_of<SCALE_32, true>(a, s) : matvec_of<SCALE_32, false>(a, s);
    return a.up_codes ? matvec_of<SCALE_16, true>(a, s) : matvec_of<SCALE_16, false>(a, s);
}

}  // namespace moe
