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
constexpr int kStage = 4;                // loads of x that a thread has in flight
constexpr int kMvSmem = 224 * 1024;      // dynamic shared memory of a block at most

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with nothing to add to.
__device__ __forceinline__ void mma_16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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
__device__ __forceinline__ uint32_t merged(uint32_t w, uint32_t mask, uint32_t bits) {
    uint32_t r;                          // (w & mask) | bits
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
    return r;
}
__device__ __forceinline__ void int4_pairs(uint32_t w, uint32_t (&h)[4], uint32_t mask, uint32_t bits) {
    const __half2 low = __float2half2_rn(-1032.0f), sixteenth = __float2half2_rn(0.0625f), high = __float2half2_rn(-72.0f);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint32_t v = u ? w >> 8 : w, a = merged(v, mask, bits), b = merged(v, mask << 4, bits);
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

template <int N>
__device__ __forceinline__ void ld_words(uint32_t (&b)[N], const uint8_t* p) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        b[0] = v.x;
        b[1] = v.y;
        b[2] = v.z;
        b[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        b[0] = v.x;
        b[1] = v.y;
    } else {
        b[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// Asynchronous copies to shared memory; zeros instead where `on` is not set.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(on ? N : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Two scales as they lie in a word.
template <int SK>
__device__ __forceinline__ float2 two_scales(uint32_t v, bool bf16) {
    if constexpr (SK == SCALE_E8M0) {
        uint32_t r;                      // 2^-127 for code 0, NaN for 255
        asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
        return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xFFFF0000u));
    } else {
        if (bf16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
        __half2 h;
        memcpy(&h, &v, 4);
        return __half22float2(h);
    }
}
// The scales of N (2 or 4) groups of 32 from group gi of a unit on; the row's scales of the unit lie at `row`.
template <int SK, int N>
__device__ __forceinline__ void read_scales(const uint8_t* row, int gi, int shift, bool bf16, float (&s)[N]) {
    if constexpr (SK == SCALE_E8M0) {
        if constexpr (N == 2) {
            const float2 v = two_scales<SK>(*reinterpret_cast<const uint16_t*>(row + gi), false);
            s[0] = v.x;
            s[1] = v.y;
        } else {
            uint32_t w[1];
            ld_words(w, row + gi);
            const float2 v = two_scales<SK>(w[0] & 0xFFFFu, false), u = two_scales<SK>(w[0] >> 16, false);
            s[0] = v.x;
            s[1] = v.y;
            s[2] = u.x;
            s[3] = u.y;
        }
    } else if constexpr (SK == SCALE_16) {
        if (shift == 0) {
            uint32_t w[N / 2];
            ld_words(w, row + 2 * gi);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float2 v = two_scales<SK>(w[i], bf16);
                s[2 * i] = v.x;
                s[2 * i + 1] = v.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) s[2 * i] = s[2 * i + 1] = two_scales<SK>(*reinterpret_cast<const uint16_t*>(row + 2 * ((gi + 2 * i) >> shift)), bf16).x;
        }
    } else {
        uint32_t w[N];
        if (shift == 0) {
            ld_words(w, row + 4 * gi);
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                uint32_t v[1];
                ld_words(v, row + 4 * ((gi + 2 * i) >> shift));
                s[2 * i] = s[2 * i + 1] = __uint_as_float(v[0]);
            }
        }
    }
}

// The warps of a team: at most eight teams have more than one.
__device__ __forceinline__ void team_sync(int team, int warps) {
    if (warps == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(warps * 32) : "memory");
}

// A unit is 256 k of a team's 16 rows: 128 bytes of a row.  Its codes go by cp.async to a ring of D slots that each
// warp has for itself, [half of 64 bytes][row][16 bytes], the four pieces of a row's half in an order that keeps the
// reads free of bank conflicts.
constexpr int kUK = 256;
constexpr int kUnitGroups = kUK / 32;
constexpr int kCodeBytes = kRows * kUK / 2;
__device__ __forceinline__ int piece(int row, int i) { return i ^ (((row >> 2) & 1) | (row & 2)); }

// GP groups of 32 share an MMA's columns (1, 2 or 4), 8 / GP vectors a tile of columns, NT tiles.  Shared memory: x as
// fp16 [unit][half][part of GP groups][word of 8][vector][lane of the row], 16 bytes each; as many zero bytes as a
// unit has (read by the lanes off the diagonal); factors of the groups in fp32; the warps' sums
// [team][matrix][warp][vector][row]; the rings.
template <int SK, int GP, int NT, bool DUAL, int D>
struct Layout {
    static constexpr int VT = 8 / GP;            // vectors of a tile
    static constexpr int VS = NT * VT;           // vectors there is room for
    static constexpr int NM = DUAL ? 2 : 1;
    static constexpr int kUnitX = kUK * VS * 2, kUnitF = VS * kUnitGroups * 4;
    static constexpr int kZero = GP == 1 ? 0 : kUnitX;
    static constexpr int kScaleRow = kUnitGroups * (SK == SCALE_E8M0 ? 1 : SK == SCALE_16 ? 2 : 4);
    static constexpr int kSlot = NM * (kCodeBytes + kRows * kScaleRow);
    static constexpr int kWarp = NM * kRows * VS * 4 + D * kSlot;     // of a warp: sums and ring
};

template <int SK, int GP, int NT, bool DUAL, int D>
__global__ void __launch_bounds__(kMvMaxThreads) matvec_kernel(const MatvecArgs a) {
    using L = Layout<SK, GP, NT, DUAL, D>;
    constexpr int VT = L::VT, VS = L::VS, NM = L::NM, PARTS = 4 / GP;
    constexpr int AC = GP == 1 ? 4 : 2;  // sums of a lane and tile: two rows, and two vectors where a column is one
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int s_expert[kMaxSegs];
    __shared__ int64_t s_row[kMaxSegs];
    __shared__ float s_gate[kMaxSegs];
    __shared__ int s_segs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int KW = a.kw, team = warp / KW, kwarp = warp % KW, warps = blockDim.x >> 5, teams = warps / KW;
    const int64_t set = static_cast<int64_t>(blockIdx.x) % a.sets;
    const int part = static_cast<int>(blockIdx.x / a.sets);
    const int K = a.K, M = a.M;
    const int cps = (K + kUK - 1) / kUK;   // units of a segment
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
    const int cap = a.cap;               // units of x that fit
    uint8_t* xv = sm;
    uint8_t* zero = xv + static_cast<size_t>(cap) * L::kUnitX;
    float* xf = reinterpret_cast<float*>(zero + L::kZero);
    float* red = xf + static_cast<size_t>(cap) * (VS * kUnitGroups);
    uint8_t* ring = reinterpret_cast<uint8_t*>(red) + warps * (NM * kRows * VS * 4) + warp * (D * L::kSlot);
    for (int i = threadIdx.x * 16; i < L::kZero; i += blockDim.x * 16) *reinterpret_cast<uint4*>(zero + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const int segs = s_segs, units = segs * cps;

    // x of the units [u0, u1) to shared memory: a thread takes eight values, four threads a group
    auto stage = [&](int u0, int u1) {
        constexpr int per_unit = kUK / 8;
        const int vvt = nv * a.parts, total = (u1 - u0) * per_unit * nv;
        for (int i0 = 0; i0 < total; i0 += kStage * blockDim.x) {
            RawVec<8> raw[kStage];
#pragma unroll
            for (int j = 0; j < kStage; ++j) {
                const int i = i0 + j * blockDim.x + threadIdx.x;
                const int c = i % per_unit, rest = i / per_unit, u = nv == 1 ? rest : rest / nv, n = rest - u * nv;
                const int seg = segs == 1 ? 0 : (u0 + u) / cps, k = ((u0 + u) - seg * cps) * kUK + c * 8;
                raw[j].a = raw[j].b = make_uint4(0, 0, 0, 0);
                if (a.x_wide && i < total && k < K) raw[j] = load_raw<8>(a.x, (s_row[seg] + n) * a.ld_x + k, a.dt_x);
            }
#pragma unroll
          for (int j = 0; j < kStage; ++j) {
            if (i0 + j * blockDim.x >= total) break;
            const int i = i0 + j * blockDim.x + threadIdx.x;
            const bool in = i < total;
            const int c = i % per_unit, rest = in ? i / per_unit : 0, u = nv == 1 ? rest : rest / nv, n = rest - u * nv;
            const int seg = segs == 1 ? 0 : (u0 + u) / cps, k = ((u0 + u) - seg * cps) * kUK + c * 8;
            float f[8];
            raw_to_f32(raw[j], a.dt_x, f);
            if (!a.x_wide && in && k < K) {
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    float e[1];
                    raw_to_f32(load_raw<1>(a.x, (s_row[seg] + n) * a.ld_x + k + x, a.dt_x), a.dt_x, e);
                    f[x] = e[0];
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
            const float to = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
            const float back = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= to;
            // lane t of a row holds the codes of 8 GP values of each part of 32 GP
            const int of_part = c % (4 * GP), t = of_part / GP, word = of_part % GP, gi = c / 4;
            uint4* xo = reinterpret_cast<uint4*>(xv) + ((u * (kUK / 32) + c / (4 * GP) * GP + word) * VS) * 4 + t;
            float* fo = xf + u * (VS * kUnitGroups) + (GP == 1 ? gi * VS : gi);
            constexpr int fs = GP == 1 ? 1 : kUnitGroups;
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
                    if ((c & 3) == 0) fo[vv * fs] = s_gate[seg] * back * __uint_as_float(static_cast<uint32_t>(127 - 12 * p) << 23);
                }
            }
            if (in && n == 0)                                    // vectors that are not there
                for (int vv = vvt; vv < VS; ++vv) {
                    xo[vv * 4] = make_uint4(0, 0, 0, 0);
                    if ((c & 3) == 0) fo[vv * fs] = 0.0f;
                }
          }
        }
    };

    // this lane's places
    constexpr int kScaleSize = SK == SCALE_E8M0 ? 1 : SK == SCALE_16 ? 2 : 4;
    const int64_t row_bytes = K / 2, srow_bytes = static_cast<int64_t>(K / 32 >> a.shift) * kScaleSize;
    const bool bf16 = a.dt_scale == ELEM_BF16;
    // B fragments: the lane's column is that of vector vb in group gb of a part; values in the rows of that group's
    // lanes, zeros elsewhere
    const int vb = g / GP;
    const bool diagonal = g % GP == t4 * GP / 4;
    const uint8_t* x_base = diagonal ? xv + (vb * 4 + t4) * 16 : zero;
    const uint32_t x_step = diagonal ? L::kUnitX : 0;
    // its two accumulator columns: groups g2 and g2 + 1 of vector vc, or vectors vc and vc + 1
    const int vc = GP == 4 ? t4 / 2 : GP == 2 ? t4 : 2 * t4, g2 = GP == 4 ? 2 * (t4 & 1) : 0;
    const float* f_lane = xf + (GP == 1 ? vc : vc * kUnitGroups + g2);

    const int tiles = (M + kRows - 1) / kRows;
    const int tile_step = a.blocks * teams;
    // The next unit to copy: pointers of this lane's pieces of codes (row g, row g + 8) and of scales, which move along a
    // segment.  Scales go by pieces of 16, 8 or 4 bytes where all rows start on whole pieces, else one by one.
    const int unit_scales = (kUnitGroups >> a.shift) * kScaleSize;                    // bytes of a row
    const int size = a.scale_piece > 0 ? a.scale_piece : kScaleSize, lg = 31 - __clz(unit_scales / size);
    const int srow = lane >> lg, soff = (lane & ((1 << lg) - 1)) * size, sstep = 32 >> lg;
    const uint32_t put = g * 64 + piece(g, t4) * 16;
    struct {
        int tile, u, c;                  // tile, unit, unit in its segment
        const uint8_t *lo[NM], *hi[NM], *s[NM];
        int64_t back;                    // from the scales' pointer to the first row's
        int rows;                        // from the tile's first to the matrix' last
    } cur;
    auto aim = [&](int tile, int u) {
        cur.tile = tile;
        cur.u = u;
        const int seg = segs > 1 ? u / cps : 0;
        cur.c = u - seg * cps;
        const int r = tile * kRows;
        cur.rows = M - r;
        const int64_t row = static_cast<int64_t>(s_expert[seg]) * M + r;
        const int64_t lo = (row + (g < cur.rows ? g : 0)) * row_bytes + cur.c * (kUK / 2) + t4 * 16, up = g + 8 < cur.rows ? 8 * row_bytes : 0;
        const int64_t of_row = min(srow, kRows) * srow_bytes + soff, sc = row * srow_bytes + static_cast<int64_t>(cur.c) * unit_scales + of_row;
        cur.back = -of_row;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            cur.lo[m] = (m ? a.up_codes : a.codes) + lo;
            cur.hi[m] = cur.lo[m] + up;
            cur.s[m] = (m ? a.up_scales : a.scales) + sc;
        }
    };
    auto copy_scales = [&](uint32_t dst, const uint8_t* src, bool on) {
        if (a.scale_piece == 8)
            copy_small<8>(dst, src, on);
        else if (a.scale_piece == 16)
            copy16(dst, src, on);
        else if (a.scale_piece == 4)
            copy_small<4>(dst, src, on);
        else if (kScaleSize == 1)
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(dst), "r"(static_cast<uint32_t>(on ? *src : 0)) : "memory");
        else
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst), "h"(on ? *reinterpret_cast<const uint16_t*>(src) : static_cast<uint16_t>(0)) : "memory");
    };
    auto fetch = [&](uint8_t* slot) {
        const int left = K - cur.c * kUK;
        const uint32_t to = smem_u32(slot) + put, sto = smem_u32(slot) + NM * kCodeBytes + srow * L::kScaleRow + soff;
        if (left >= kUK && cur.rows >= kRows) {
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                copy16(to + m * kCodeBytes, cur.lo[m], true);
                copy16(to + m * kCodeBytes + 512, cur.hi[m], true);
                copy16(to + m * kCodeBytes + 1024, cur.lo[m] + 64, true);
                copy16(to + m * kCodeBytes + 1536, cur.hi[m] + 64, true);
                if (srow < kRows) copy_scales(sto + m * (kRows * L::kScaleRow), cur.s[m], true);
                for (int row = sstep; srow + row < kRows; row += sstep)
                    copy_scales(sto + m * (kRows * L::kScaleRow) + row * L::kScaleRow, cur.s[m] + row * srow_bytes, true);
            }
        } else {
            // behind the row's end the first address of its unit, which is not read
            const bool on0 = t4 * 32 < left, on1 = t4 * 32 + 128 < left;
            const int sleft = static_cast<int>(srow_bytes) - cur.c * unit_scales;        // K / 8 at most
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const uint8_t *lo = cur.lo[m] - (on0 ? 0 : t4 * 16), *hi = cur.hi[m] - (on0 ? 0 : t4 * 16);
                copy16(to + m * kCodeBytes, lo, on0 && g < cur.rows);
                copy16(to + m * kCodeBytes + 512, hi, on0 && g + 8 < cur.rows);
                copy16(to + m * kCodeBytes + 1024, lo + (on1 ? 64 : 0), on1 && g < cur.rows);
                copy16(to + m * kCodeBytes + 1536, hi + (on1 ? 64 : 0), on1 && g + 8 < cur.rows);
                for (int row = 0; srow + row < kRows; row += sstep) {
                    const bool on = soff < sleft && srow + row < cur.rows;
                    copy_scales(sto + m * (kRows * L::kScaleRow) + row * L::kScaleRow, cur.s[m] + (on ? row * srow_bytes : cur.back), on);
                }
            }
        }
        ++cur.u;
        if (++cur.c == cps && cur.u < units) {
            aim(cur.tile, cur.u);
        } else {
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                cur.lo[m] += kUK / 2;
                cur.hi[m] += kUK / 2;
                cur.s[m] += unit_scales;
            }
        }
    };

    // in registers: an instruction takes one constant
    uint32_t mask4 = 0x000F000Fu, bits4 = 0x64006400u;
    asm volatile("" : "+r"(mask4), "+r"(bits4));
    float acc[NM][NT][AC];
    // adds the products of the unit in a slot, whose x is number ul in shared memory
    auto work = [&](const uint8_t* slot, int ul) {
        const uint8_t* x_at = x_base + ul * x_step;
        const float* f_at = f_lane + ul * (VS * kUnitGroups);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float s4[NM][2][4];
            if constexpr (GP == 1) {
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    const uint8_t* row = slot + NM * kCodeBytes + (m * kRows + g) * L::kScaleRow;
                    read_scales<SK, 4>(row, half * 4, a.shift, bf16, s4[m][0]);
                    read_scales<SK, 4>(row + 8 * L::kScaleRow, half * 4, a.shift, bf16, s4[m][1]);
                }
            }
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                uint32_t lo[NM][GP], hi[NM][GP];
                // the lane's 4 GP bytes of the part's 16 GP in a row
                const uint8_t* at = slot + half * 1024 + g * 64 +
                                    (GP == 4 ? piece(g, t4) * 16 : GP == 2 ? piece(g, 2 * part + t4 / 2) * 16 + (t4 & 1) * 8 : piece(g, part) * 16 + t4 * 4);
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    ld_words(lo[m], at + m * kCodeBytes);
                    ld_words(hi[m], at + m * kCodeBytes + 512);
                }
                float c[NM][NT][4];
#pragma unroll
                for (int w = 0; w < GP; ++w) {
                    uint32_t b[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n) ld_words(b[n], x_at + (((half * PARTS + part) * GP + w) * VS + n * VT) * 64);
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        uint32_t p[4], q[4];
                        if constexpr (SK == SCALE_E8M0) {
                            e2m1_pairs(lo[m][w], p);
                            e2m1_pairs(hi[m][w], q);
                        } else {
                            int4_pairs(lo[m][w], p, mask4, bits4);
                            int4_pairs(hi[m][w], q, mask4, bits4);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (w == 0)
                                mma_16816_first(c[m][n], p[0], q[0], p[1], q[1], b[n][0], b[n][1]);
                            else
                                mma_16816(c[m][n], p[0], q[0], p[1], q[1], b[n][0], b[n][1]);
                            mma_16816(c[m][n], p[2], q[2], p[3], q[3], b[n][2], b[n][3]);
                        }
                    }
                }
                // behind the last group codes, values and scales are zero
                const int gi = half * 4 + part * GP;
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    if constexpr (GP == 1) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const float2 f = *reinterpret_cast<const float2*>(f_at + gi * VS + n * VT);
                            acc[m][n][0] = fmaf(c[m][n][0] * s4[m][0][part], f.x, acc[m][n][0]);
                            acc[m][n][1] = fmaf(c[m][n][1] * s4[m][0][part], f.y, acc[m][n][1]);
                            acc[m][n][2] = fmaf(c[m][n][2] * s4[m][1][part], f.x, acc[m][n][2]);
                            acc[m][n][3] = fmaf(c[m][n][3] * s4[m][1][part], f.y, acc[m][n][3]);
                        }
                    } else {
                        const uint8_t* row = slot + NM * kCodeBytes + (m * kRows + g) * L::kScaleRow;
                        float s[2], r[2];
                        read_scales<SK, 2>(row, gi + g2, a.shift, bf16, s);
                        read_scales<SK, 2>(row + 8 * L::kScaleRow, gi + g2, a.shift, bf16, r);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const float2 f = *reinterpret_cast<const float2*>(f_at + n * VT * kUnitGroups + gi);
                            acc[m][n][0] = fmaf(c[m][n][1] * s[1], f.y, fmaf(c[m][n][0] * s[0], f.x, acc[m][n][0]));
                            acc[m][n][1] = fmaf(c[m][n][3] * r[1], f.y, fmaf(c[m][n][2] * r[0], f.x, acc[m][n][1]));
                        }
                    }
                }
            }
        }
    };

    // A warp's units of a tile are a run of them; the copies of D units are in flight, those of the next tile's first
    // ones while the last of this one's are worked on.  Each unit is a group of copies (or an empty one).
    const bool whole = units <= cap;     // all of x fits: staged once
    bool ahead = false;                  // the ring holds the first units already
    int at = 0;                          // slot of the next unit
    float* mine = red + team * (NM * KW * kRows * VS);
    for (int tile0 = part * teams; tile0 < tiles; tile0 += tile_step) {
        const int tile = tile0 + team;
        const bool live = tile < tiles;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < AC; ++i) acc[m][n][i] = 0.0f;
        for (int u0 = 0; u0 < units; u0 += cap) {
            const int u1 = min(u0 + cap, units), per = (u1 - u0 + KW - 1) / KW;
            const int first = min(u0 + kwarp * per, u1), last = min(first + per, u1), run = last - first;
            // the next unit of this run, or (if x stays) the first of the next tile's
            auto issue = [&](uint8_t* slot) {
                if (cur.u >= last && whole && run > 0 && cur.tile + tile_step < tiles) aim(cur.tile + tile_step, first);
                if (cur.u < last) fetch(slot);
                copy_commit();
            };
            if (live && !ahead) {
                at = 0;
                aim(tile, first);
                for (int i = 0; i < D; ++i) issue(ring + i * L::kSlot);
            }
            if (!whole || tile0 == part * teams) {
                __syncthreads();
                stage(u0, u1);
                __syncthreads();
            }
            if (!live) continue;
            for (int i = 0; i < run; ++i) {
                copy_wait<D - 1>();
                __syncwarp();
                uint8_t* slot = ring + at * L::kSlot;
                work(slot, first + i - u0);
                __syncwarp();
                issue(slot);
                at = at + 1 == D ? 0 : at + 1;
            }
            ahead = whole;
        }
        // the warps' sums, then the rows' outputs
        if (live) {
            team_sync(team, KW);         // the last tile's are read
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float* to = mine + ((m * KW + kwarp) * VS + n * VT + vc) * kRows + g;
                    if constexpr (GP == 1) {
                        to[0] = acc[m][n][0];
                        to[kRows] = acc[m][n][1];
                        to[8] = acc[m][n][2];
                        to[kRows + 8] = acc[m][n][3];
                    } else {
                        float lo = acc[m][n][0], hi = acc[m][n][1];
                        if (GP == 4) {
                            lo += __shfl_xor_sync(kAll, lo, 1);
                            hi += __shfl_xor_sync(kAll, hi, 1);
                        }
                        if (GP == 2 || (t4 & 1) == 0) {
                            to[0] = lo;
                            to[8] = hi;
                        }
                    }
                }
            team_sync(team, KW);
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
template <int SK, int GP, int NT, bool DUAL, int D>
cudaError_t matvec_as(MatvecArgs a, cudaStream_t s) {
    using L = Layout<SK, GP, NT, DUAL, D>;
    const int tiles = (a.M + kRows - 1) / kRows;
    const int64_t units = static_cast<int64_t>(a.weights ? a.k : 1) * ((a.K + kUK - 1) / kUK);
    const size_t unit_bytes = L::kUnitX + L::kUnitF;
    const bool two = units * unit_bytes + L::kZero + 8 * L::kWarp <= 110 * 1024;
    const int warps = two ? 8 : 16, resident = two ? 304 : 152;
    a.cap = static_cast<int>(std::min<int64_t>(units, (kMvSmem - L::kZero - warps * L::kWarp) / unit_bytes));
    const size_t smem = a.cap * unit_bytes + L::kZero + warps * L::kWarp;
    if (smem > 40 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(matvec_kernel<SK, GP, NT, DUAL, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMvSmem);
        if (err != cudaSuccess) return err;
    }
    // a set of its own for each slot: some four rounds of blocks, as many of them may have nothing to do
    const int64_t most = a.idx ? std::max<int64_t>(1, (4 * resident + a.sets - 1) / a.sets) : std::max<int64_t>(1, resident / a.sets);
    int64_t best = INT64_MAX;
    for (int kw = 1; kw <= warps; kw *= 2) {
        const int teams = warps / kw;
        const int64_t blocks = std::min<int64_t>((tiles + teams - 1) / teams, most);
        const int64_t rounds = (tiles + blocks * teams - 1) / (blocks * teams), waves = (a.sets * blocks + resident - 1) / resident;
        const int64_t cost = waves * rounds * (2 * ((units + kw - 1) / kw) + 1);
        if (cost < best) {
            best = cost;
            a.kw = kw;
            a.blocks = static_cast<int>(blocks);
        }
    }
    matvec_kernel<SK, GP, NT, DUAL, D><<<static_cast<unsigned>(a.sets * a.blocks), warps * 32, smem, s>>>(a);
    return cudaGetLastError();
}

// Vectors (three for an fp32 row) against the columns of one MMA: four groups of a row's lanes and two vectors, two and
// four, one and eight, or two MMAs of eight.
template <int SK, bool DUAL>
cudaError_t matvec_of(const MatvecArgs& a, cudaStream_t s) {
    const int vv = a.nv * a.parts;
    if (vv <= 2) return matvec_as<SK, 4, 1, DUAL, DUAL ? 2 : 3>(a, s);
    if (vv <= 4) return matvec_as<SK, 2, 1, DUAL, DUAL ? 2 : 3>(a, s);
    if (vv <= 8) return matvec_as<SK, 1, 1, DUAL, 2>(a, s);
    return matvec_as<SK, 1, 2, DUAL, 2>(a, s);
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
    // pieces of a row's scales of a unit, as large as addresses and rows allow
    const uint64_t lie = reinterpret_cast<uintptr_t>(a.scales) | reinterpret_cast<uintptr_t>(a.up_scales) |
                         static_cast<uint64_t>((a.K / 32) >> a.shift) * size | static_cast<uint64_t>((kUnitGroups >> a.shift) * size);
    a.scale_piece = lie % 16 == 0 ? 16 : lie % 8 == 0 ? 8 : lie % 4 == 0 ? 4 : 0;
    if (a.format == 0) return a.up_codes ? matvec_of<SCALE_E8M0, true>(a, s) : matvec_of<SCALE_E8M0, false>(a, s);
    if (a.dt_scale == ELEM_F32) return a.up_codes ? matvec_of<SCALE_32, true>(a, s) : matvec_of<SCALE_32, false>(a, s);
    return a.up_codes ? matvec_of<SCALE_16, true>(a, s) : matvec_of<SCALE_16, false>(a, s);
}

}  // namespace moe
