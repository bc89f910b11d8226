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
// Measured, K = 7,168: MXFP4 and one bf16 vector, 8,192 rows 13.9 us (31 MB: 2.2 TB/s),
// 65,536 rows 60 us (4.2 TB/s).  A block's start takes some 6 us of that (first
// instructions, x from memory to its fp16 form), a unit of 16 x 256 weights 350
// instructions, at which 16 warps an SM keep up with two thirds of HBM.  Integers in
// groups of 128 and eight fp16 vectors, 65,536 rows 86 us: 576 instructions a unit,
// which the schedulers issue in 65% of the cycles (the tensor pipe is at 12%, shared
// memory at a fifth).
//
// Two matrices of 4,096 rows (gate and up with SiLU), MXFP4, bf16: one vector 16 us,
// four 21, eight 25; fp32: one 18, two 25, four 39.  (16 warps' rings and sums are then
// 132 to 160 KB, so that K = 7,168 of five bf16 or two fp32 vectors is staged in parts,
// for each round of tiles anew; with one matrix, of three fp32 vectors.)  At 128
// registers a thread the forms with two matrices, and those of nine to sixteen vectors,
// store up to 200 bytes to local memory.
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
constexpr int D = 2;                     // units in a warp's ring
constexpr int kUK = 256;                 // k of a unit
constexpr int kUnitGroups = kUK / 32;
constexpr int kMvMaxThreads = 512;
constexpr int kMaxSegs = 32;             // slots of a token
constexpr int kMvSmem = 222 * 1024;      // dynamic shared memory of a block at most, but for the first 1,024-byte boundary

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
// bits of an fp16 1024 is 1024 + c, four bits higher 1024 + 16 c.  (A known method:
// Kim, Henry, Fahim and Awadalla, "Who Says Elephants Can't Run: Bringing Large Scale
// MoE Models into Cloud Scale Production", 2022, on conversion without I2F.)
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

// Kinds of scale: E8M0 (with E2M1 codes), fp16, bf16 or fp32 (with integers).
enum ScaleKind : int { SCALE_E8M0 = 0, SCALE_F16 = 1, SCALE_BF16 = 2, SCALE_F32 = 3 };

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
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Two scales as they lie in a word.
template <int SK>
__device__ __forceinline__ float2 two_scales(uint32_t v) {
    if constexpr (SK == SCALE_E8M0) {
        uint32_t r;                      // 2^-127 for code 0, NaN for 255
        asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
        v = r;
    }
    if constexpr (SK == SCALE_F16) {
        __half2 h;
        memcpy(&h, &v, 4);
        return __half22float2(h);
    }
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
// A row's scales of a unit, W words as they lie in memory: `bytes` of them, in pieces of 16, 8 or 4 bytes.
__device__ __forceinline__ void ld_global(uint32_t& a, const uint8_t* p) { asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(a) : "l"(p)); }
__device__ __forceinline__ void ld_global(uint32_t& a, uint32_t& b, const uint8_t* p) {
    asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "l"(p));
}
__device__ __forceinline__ void ld_global(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d, const uint8_t* p) {
    asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "l"(p));
}
template <int W>
__device__ __forceinline__ void load_row_scales(uint32_t (&w)[W], const uint8_t* p, int bytes, int piece) {
    if (W >= 4 && piece == 16) {
#pragma unroll
        for (int i = 0; i + 3 < W; i += 4)
            if (4 * i < bytes) ld_global(w[i], w[i + 1], w[i + 2], w[i + 3], p + 4 * i);
    } else if (piece == 8) {
#pragma unroll
        for (int i = 0; i + 1 < W; i += 2)
            if (4 * i < bytes) ld_global(w[i], w[i + 1], p + 4 * i);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (4 * i < bytes) ld_global(w[i], p + 4 * i);
    }
}
// The same one by one, `left` bytes of them; behind them zeros.
template <int SK, int W>
__device__ __forceinline__ void load_row_scales_one(uint32_t (&w)[W], const uint8_t* p, int n, int left) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
    constexpr int size = SK == SCALE_E8M0 ? 1 : SK == SCALE_F32 ? 4 : 2;
#pragma unroll
    for (int i = 0; i < kUnitGroups; ++i) {
        if (i >= n || i * size >= left) break;
        if constexpr (SK == SCALE_E8M0) w[i / 4] |= static_cast<uint32_t>(__ldg(p + i)) << (8 * (i % 4));
        if constexpr (SK == SCALE_F16 || SK == SCALE_BF16) w[i / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(p) + i)) << (16 * (i % 2));
        if constexpr (SK == SCALE_F32) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
    }
}
// Scales as loaded, each for 2^shift groups of 32, as one for each of the unit's groups.
template <int SK, int W>
__device__ __forceinline__ void spread_scales(uint32_t (&to)[W], const uint32_t (&w)[W], int shift) {
#pragma unroll
    for (int i = 0; i < W; ++i) to[i] = w[i];
    if constexpr (SK == SCALE_F32) {
        if (shift > 0)
#pragma unroll
            for (int i = 0; i < W; ++i) to[i] = shift == 1 ? w[i / 2] : w[i / 4];
    } else if constexpr (SK != SCALE_E8M0) {
        if (shift > 0)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int n = shift == 1 ? i : i / 2;
                to[i] = __byte_perm(shift == 1 ? w[i / 2] : w[0], 0, n & 1 ? 0x3232 : 0x1010);
            }
    }
}
// The scales of groups 2 q and 2 q + 1, or with `odd` (q even then) of the two behind them.
template <int SK, int W>
__device__ __forceinline__ void pair_of_scales(const uint32_t (&w)[W], int q, int odd, float (&s)[2]) {
    if constexpr (SK == SCALE_F32) {
        s[0] = __uint_as_float(odd ? w[(2 * q + 2) % W] : w[2 * q]);
        s[1] = __uint_as_float(odd ? w[(2 * q + 3) % W] : w[2 * q + 1]);
    } else {
        const float2 v = two_scales<SK>(SK == SCALE_E8M0 ? w[q / 2] >> (16 * (q % 2) + 16 * odd) : odd ? w[(q + 1) % W] : w[q]);
        s[0] = v.x;
        s[1] = v.y;
    }
}

// The warps of a team: at most eight teams have more than one.
__device__ __forceinline__ void team_sync(int team, int warps) {
    if (warps == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(warps * 32) : "memory");
}

// A unit is 256 k of a team's 16 rows: 128 bytes of a row.  Each warp has a ring of D units for itself: the codes come
// by TMA, a box of 16 rows of 128 bytes in the 128-byte swizzle (piece i of 16 bytes of row r lies at piece i ^ (r % 8)).
// Two units in the ring do as well as more in long runs and better at the start, where x comes behind them: 8,192 rows of
// 7,168 and one token 14.6 us, with four 15.8.  (Tiles of 32 rows, with x read once for two MMAs, are no faster: shared
// memory is at a fifth of its rate, and 256 tiles leave 24 of 152 SMs idle.)
// The scales go to registers, a unit ahead: four lanes read the same 8 bytes of an MXFP4 row.  (By cp.async or by TMA to
// shared memory and from there they cost more instructions than all else but the conversion of the codes: 155,648 rows
// of 7,168 120 us, without scales 100.)  The MMA's row g is row `row_of(g)` of the tile and g + 8 eight behind it: with the three
// bits of g in reverse order, the lanes that shared memory serves at once, a quarter, half or whole warp of them, find
// their pieces in different banks.
constexpr int kCodeBytes = kRows * kUK / 2;
__device__ __forceinline__ int row_of(int g) { return (g >> 2) | (g & 2) | ((g & 1) << 2); }

// GP groups of 32 share an MMA's columns (1, 2 or 4), 8 / GP vectors a tile of columns, NT tiles.  Shared memory: the
// rings' codes, [warp][slot][matrix]; x as fp16 [unit][half][part of GP groups][word of 8][vector][lane of the row], 16
// bytes each; as many zero bytes as a unit has (read by the lanes off the diagonal); factors of the groups in fp32; the
// warps' sums [team][matrix][warp][vector][row].
template <int SK, int GP, int NT, bool DUAL>
struct Layout {
    static constexpr int VT = 8 / GP;            // vectors of a tile
    static constexpr int VS = NT * VT;           // vectors there is room for
    static constexpr int NM = DUAL ? 2 : 1;
    static constexpr int kUnitX = kUK * VS * 2, kUnitF = VS * kUnitGroups * 4;
    static constexpr int kZero = GP == 1 ? 0 : kUnitX;
    static constexpr int W = SK == SCALE_E8M0 ? 2 : SK == SCALE_F32 ? 8 : 4;     // words of a row's scales in a unit
    static constexpr int kWarp = NM * kRows * VS * 4 + D * NM * kCodeBytes;             // of a warp: sums and ring
};

// Waits, with a limit, for a copy that nobody will use.
__device__ __noinline__ void matvec_drain(uint64_t* bar, uint32_t parity, int* status) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            if (status) atomicCAS(status, 0, DEV_TIMEOUT_TEARDOWN);
            return;
        }
}

template <int SK, int GP, int NT, bool DUAL>
__global__ void __launch_bounds__(kMvMaxThreads) matvec_kernel(const __grid_constant__ MatvecArgs a) {
    using L = Layout<SK, GP, NT, DUAL>;
    constexpr int VT = L::VT, VS = L::VS, NM = L::NM, PARTS = 4 / GP;
    constexpr int AC = GP == 1 ? 4 : 2;  // sums of a lane and tile: two rows, and two vectors where a column is one
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const sm = smem_raw + (-smem_u32(smem_raw) & 1023u);        // (by an offset: it stays known as shared memory)
    __shared__ int s_expert[kMaxSegs], s_row[kMaxSegs], s_segs, s_abort;
    __shared__ __align__(8) uint64_t s_full[kMvMaxThreads / 32][D];
    __shared__ float s_gate[kMaxSegs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int KW = 1 << a.kw_log, team = warp >> a.kw_log, kwarp = warp & (KW - 1), warps = blockDim.x >> 5, teams = warps >> a.kw_log;
    const uint32_t sets = static_cast<uint32_t>(a.sets), part = sets == 1 ? blockIdx.x : blockIdx.x / sets, set = blockIdx.x - part * sets;
    const int K = a.K, M = a.M, cps = a.cps;
    uint64_t* const full = s_full[warp];
    volatile int* const abort_flag = &s_abort;
    if (threadIdx.x == 0) s_abort = 0;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < D; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    // the vectors: rows of x (one matrix), a slot's row, or a token's slots one behind the other, whose numbers below 2^31
    // go to shared memory
    const int nv = a.idx ? 1 : static_cast<int>(min(static_cast<int64_t>(a.nv), a.N - static_cast<int64_t>(set) * a.nv));
    int segs = 1, expert = 0;
    int64_t xrow = static_cast<int64_t>(set) * a.nv;
    if (a.weights) {
        if (warp == 0) {
            const int slot = static_cast<int>(set) * a.k + lane;
            const int e = lane < a.k ? a.idx[slot] : -1;
            const bool kept = e >= 0 && e < a.G;
            const uint32_t all = __ballot_sync(kAll, kept);
            if (kept) {
                const int at = __popc(all & ((1u << lane) - 1));
                s_expert[at] = e;
                s_row[at] = a.x_per_slot ? slot : static_cast<int>(set);
                s_gate[at] = a.weights[slot];
            }
            if (lane == 0) s_segs = __popc(all);
        }
        __syncthreads();
        segs = s_segs;
    } else if (a.idx) {
        expert = a.idx[set];
        segs = expert >= 0 && expert < a.G ? 1 : 0;
        xrow = a.x_per_slot ? set : set / static_cast<uint32_t>(a.k);
    }
    const int units = segs * cps;
    const int cap = a.cap;               // units of x that fit
    uint8_t* const codes = sm + warp * (D * NM * kCodeBytes);
    uint8_t* xv = sm + warps * (D * NM * kCodeBytes);
    uint8_t* zero = xv + static_cast<size_t>(cap) * L::kUnitX;
    float* xf = reinterpret_cast<float*>(zero + L::kZero);
    float* red = xf + static_cast<size_t>(cap) * (VS * kUnitGroups);
    for (int i = threadIdx.x * 16; i < L::kZero; i += blockDim.x * 16) *reinterpret_cast<uint4*>(zero + i) = make_uint4(0, 0, 0, 0);

    // x of the units [u0, u1) to shared memory.  A warp takes a unit of a vector, a lane eight values, four lanes a
    // group.  The values come by cp.async to where their fp16 parts go, and are made these parts in place by the lane
    // that copied them.
    constexpr int fs = GP == 1 ? 1 : kUnitGroups;                // from a vector's factor to the next one's
    const int x_word = lane / (4 * GP) * GP + lane % (4 * GP) % GP;      // lane t of a row holds the codes of 8 GP values of each part of 32 GP
    uint8_t* const x_lane = xv + (x_word * (VS * 4) + lane % (4 * GP) / GP) * 16;
    const int64_t x0 = xrow * a.ld_x + lane * 8;
    auto copy_x = [&](int u0, int u1) {
        const int items = (u1 - u0) * nv;
#pragma unroll 1
        for (int j = warp; j < items; j += warps) {
            int u = j, n = 0, k = (u0 + j) * kUK;
            int64_t off = x0;
            if (nv > 1) {                // one segment
                u = j / nv;
                n = j - u * nv;
                off += n * a.ld_x;
                k = (u0 + u) * kUK;
            } else if (a.weights) {
                const int seg = (u0 + j) / cps;
                off = s_row[seg] * a.ld_x + lane * 8;
                k = (u0 + j - seg * cps) * kUK;
            }
            const bool on = k + lane * 8 < K;
            const uint8_t* src = static_cast<const uint8_t*>(a.x) + (off + (on ? k : -lane * 8)) * (a.parts > 1 ? 4 : 2);
            const uint32_t dst = smem_u32(x_lane + u * L::kUnitX + n * a.parts * 64);
            copy16(dst, src, on);
            if (a.parts > 1) copy16(dst + 64, src + 16, on);
        }
    };
    auto stage = [&](int u0, int u1) {
        const int vvt = nv * a.parts, items = (u1 - u0) * nv;
        float* const f_to = xf + (GP == 1 ? lane / 4 * VS : lane / 4);
#pragma unroll 1
        for (int j = warp; j < items; j += warps) {
            const int u = nv == 1 ? j : j / nv, n = j - u * nv, seg = a.weights ? (u0 + u) / cps : 0;
            uint8_t* xo = x_lane + u * L::kUnitX + n * a.parts * 64;
            const float gate = a.weights ? s_gate[seg] : 1.0f;
            float f[8];
            if (a.x_wide) {
                RawVec<8> raw;
                raw.a = *reinterpret_cast<const uint4*>(xo);
                if (a.parts > 1) raw.b = *reinterpret_cast<const uint4*>(xo + 64);
                raw_to_f32(raw, a.dt_x, f);
            } else {
                const int64_t off = a.weights ? s_row[seg] * a.ld_x + lane * 8 : x0 + n * a.ld_x;
                const int k = (u0 + u - seg * cps) * kUK;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    float e[1] = {0.0f};
                    if (k + lane * 8 < K) raw_to_f32(load_raw<1>(a.x, off + k + x, a.dt_x), a.dt_x, e);
                    f[x] = e[0];
                }
            }
            float top = 0.0f;                                    // (fmaxf goes past NaN)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
            if (top == INFINITY) {                               // infinities stay what they are
                top = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fabsf(f[i]) < INFINITY ? fmaxf(top, fabsf(f[i])) : top;
            }
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
            // 2^-ex brings it into [2^14, 2^15); the factors, with those of the parts, stay normal numbers
            int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14;
            ex = top == 0.0f ? 0 : max(ex, a.parts == 1 ? -126 : -100);
            const float to = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
            const float back = gate * __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= to;
            float* fo = f_to + u * (VS * kUnitGroups) + n * a.parts * fs;
            for (int p = 0; p < a.parts; ++p) {
                __half2 h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)                      // integers come in the order (0, 4) (1, 5) (2, 6) (3, 7)
                    h[i] = SK == SCALE_E8M0 ? __floats2half2_rn(f[2 * i], f[2 * i + 1]) : __floats2half2_rn(f[i], f[i + 4]);
                if (a.parts > 1)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 v = __half22float2(h[i]);
                        float& lo = f[SK == SCALE_E8M0 ? 2 * i : i];
                        float& hi = f[SK == SCALE_E8M0 ? 2 * i + 1 : i + 4];
                        const float r = (lo - v.x) * 4096.0f, s = (hi - v.y) * 4096.0f;
                        lo = r == r ? r : 0.0f;                  // nothing is left of an infinity
                        hi = s == s ? s : 0.0f;
                    }
                uint4 v;
                memcpy(&v, h, 16);
                *reinterpret_cast<uint4*>(xo + p * 64) = v;
                if ((lane & 3) == 0) fo[p * fs] = back * __uint_as_float(static_cast<uint32_t>(127 - 12 * p) << 23);
            }
            if (n == 0)                                          // vectors that are not there
                for (int p = vvt; p < VS; ++p) {
                    *reinterpret_cast<uint4*>(xo + p * 64) = make_uint4(0, 0, 0, 0);
                    if ((lane & 3) == 0) fo[p * fs] = 0.0f;
                }
        }
    };

    // this lane's places
    // B fragments: the lane's column is that of vector vb in group gb of a part; values in the rows of that group's
    // lanes, zeros elsewhere
    const int vb = g / GP;
    const bool diagonal = g % GP == t4 * GP / 4;
    const uint8_t* x_base = diagonal ? xv + (vb * 4 + t4) * 16 : zero;
    const uint32_t x_step = diagonal ? L::kUnitX : 0;
    // its two accumulator columns: groups g2 and g2 + 1 of vector vc, or vectors vc and vc + 1
    const int vc = GP == 4 ? t4 / 2 : GP == 2 ? t4 : 2 * t4, g2 = GP == 4 ? 2 * (t4 & 1) : 0;
    const float* f_lane = xf + (GP == 1 ? vc : vc * kUnitGroups + g2);

    const int tiles = a.tiles, tile_step = a.blocks * teams;
    // The next unit to copy: its tile, its number, those left of the run, its number in its segment, its row of all
    // matrices.  Rows behind the last of all matrices and codes behind a row's end come as zeros; rows of the next matrix
    // are not stored.
    int c_tile = 0, c_u = 0, c_left = 0, c_c = 0, c_row = 0;
    auto copy_next = [&](int at) {
        if (c_c == cps) {
            const int seg = segs > 1 ? c_u / cps : 0;
            c_c = c_u - seg * cps;
            c_row = (a.weights ? s_expert[seg] : expert) * M + c_tile * kRows;           // G M < 2^31
        }
        if (elect_one()) {
            mbar_arrive_expect_tx(&full[at], NM * kCodeBytes);
#pragma unroll
            for (int m = 0; m < NM; ++m)
                tma_load_2d(codes + (at * NM + m) * kCodeBytes, m ? &a.up_map : &a.map, &full[at], c_c * (kUK / 2), c_row);
        }
        ++c_u;
        ++c_c;
        --c_left;
    };
    // The next unit's scales: where its row lies, the bytes from there to the row's end, and to row g + 8.
    const int row0 = row_of(g), unit_scales = a.unit_scales;
    uint32_t next[NM][2][L::W], now[NM][2][L::W];
    const uint8_t* s_at = nullptr;
    int s_left = 0, s_below = 0;
    auto aim_scales = [&](int tile, int u) {
        const int seg = segs > 1 ? u / cps : 0, lo = min(tile * kRows + row0, M - 1), hi = min(tile * kRows + row0 + 8, M - 1);
        const int64_t row = static_cast<int64_t>(a.weights ? s_expert[seg] : expert) * M + lo;
        const int off = (u - seg * cps) * unit_scales;
        s_at = a.scales + row * a.srow + off;
        s_left = a.srow - off;
        s_below = (hi - lo) * a.srow;
    };
    auto load_scales = [&] {
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const uint8_t* p = m ? s_at + (a.up_scales - a.scales) : s_at;
            if (a.scale_piece > 0 && s_left >= unit_scales) {
                load_row_scales(next[m][0], p, unit_scales, a.scale_piece);
                load_row_scales(next[m][1], p + s_below, unit_scales, a.scale_piece);
            } else {
                load_row_scales_one<SK>(next[m][0], p, kUnitGroups >> a.shift, s_left);
                load_row_scales_one<SK>(next[m][1], p + s_below, kUnitGroups >> a.shift, s_left);
            }
        }
        s_at += unit_scales;
        s_left -= unit_scales;
    };

    // in registers: an instruction takes one constant
    uint32_t mask4 = 0x000F000Fu, bits4 = 0x64006400u;
    asm volatile("" : "+r"(mask4), "+r"(bits4));
    float acc[NM][NT][AC];
    // adds the products of the unit in a slot, whose x is number ul in shared memory
    const uint8_t* const c_lane = codes + row0 * 128;
    const int odd = GP == 4 ? t4 & 1 : 0;
    auto work = [&](int at_slot, int ul) {
        const uint8_t* slot = c_lane + at_slot * (NM * kCodeBytes);
        const uint8_t* x_at = x_base + ul * x_step;
        const float* f_at = f_lane + ul * (VS * kUnitGroups);
        // The MMAs of a part follow one another in one accumulator, some 22 cycles each: two parts at a time.
#pragma unroll
        for (int pair = 0; pair < PARTS; ++pair) {
            // parts 2 pair and 2 pair + 1 of the unit's 2 PARTS
            uint32_t lo[2][NM][GP], hi[2][NM][GP];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int q = 2 * pair + h, half = q / PARTS, part = q % PARTS;
                // the lane's 4 GP bytes of the part's 16 GP in a row
                const int piece = half * 4 + (GP == 4 ? t4 : GP == 2 ? 2 * part + t4 / 2 : part);
                const uint8_t* at = slot + (piece ^ row0) * 16 + (GP == 4 ? 0 : GP == 2 ? (t4 & 1) * 8 : t4 * 4);
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    ld_words(lo[h][m], at + m * kCodeBytes);
                    ld_words(hi[h][m], at + m * kCodeBytes + 1024);
                }
            }
            float c[2][NM][NT][4];
#pragma unroll
            for (int w = 0; w < GP; ++w) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t b[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n) ld_words(b[n], x_at + (((2 * pair + h) * GP + w) * VS + n * VT) * 64);
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        uint32_t p[4], q[4];
                        if constexpr (SK == SCALE_E8M0) {
                            e2m1_pairs(lo[h][m][w], p);
                            e2m1_pairs(hi[h][m][w], q);
                        } else {
                            int4_pairs(lo[h][m][w], p, mask4, bits4);
                            int4_pairs(hi[h][m][w], q, mask4, bits4);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (w == 0)
                                mma_16816_first(c[h][m][n], p[0], q[0], p[1], q[1], b[n][0], b[n][1]);
                            else
                                mma_16816(c[h][m][n], p[0], q[0], p[1], q[1], b[n][0], b[n][1]);
                            mma_16816(c[h][m][n], p[2], q[2], p[3], q[3], b[n][2], b[n][3]);
                        }
                    }
                }
            }
            // behind the last group codes, values and scales are zero
            const int gi = 2 * pair * GP;
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                if constexpr (GP == 1) {
                    float s[2], r[2];
                    pair_of_scales<SK>(now[m][0], pair, 0, s);
                    pair_of_scales<SK>(now[m][1], pair, 0, r);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const float2 f = *reinterpret_cast<const float2*>(f_at + (gi + h) * VS + n * VT);
                            acc[m][n][0] = fmaf(c[h][m][n][0] * s[h], f.x, acc[m][n][0]);
                            acc[m][n][1] = fmaf(c[h][m][n][1] * s[h], f.y, acc[m][n][1]);
                            acc[m][n][2] = fmaf(c[h][m][n][2] * r[h], f.x, acc[m][n][2]);
                            acc[m][n][3] = fmaf(c[h][m][n][3] * r[h], f.y, acc[m][n][3]);
                        }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float s[2], r[2];
                        pair_of_scales<SK>(now[m][0], (2 * pair + h) * GP / 2, odd, s);
                        pair_of_scales<SK>(now[m][1], (2 * pair + h) * GP / 2, odd, r);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const float2 f = *reinterpret_cast<const float2*>(f_at + n * VT * kUnitGroups + gi + h * GP);
                            acc[m][n][0] = fmaf(c[h][m][n][1] * s[1], f.y, fmaf(c[h][m][n][0] * s[0], f.x, acc[m][n][0]));
                            acc[m][n][1] = fmaf(c[h][m][n][3] * r[1], f.y, fmaf(c[h][m][n][2] * r[0], f.x, acc[m][n][1]));
                        }
                    }
                }
            }
        }
    };

    // A warp's units of a tile are a run of them; the copies of D units are in flight, those of the next tile's first
    // ones while the last of this one's are worked on.
    const bool whole = units <= cap;     // all of x fits: staged once
    bool ahead = false;                  // the ring holds the first units already
    int at = 0, flying = 0;              // slot of the next unit, slots with a copy that was not waited for
    uint32_t phase = 0;                  // of the next slot's barrier
    bool ok = true;                      // no wait has run out
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
            const int u1 = min(u0 + cap, units), per = (u1 - u0 + KW - 1) >> a.kw_log;
            const int first = min(u0 + kwarp * per, u1), run = min(first + per, u1) - first;
            const bool need = !whole || tile0 == static_cast<int>(part) * teams;      // x of these units
            if (need && a.x_wide) {
                if (tile0 != static_cast<int>(part) * teams || u0 > 0) __syncthreads();   // the last ones are read
                copy_x(u0, u1);
            }
            const bool fill = live && !ahead && ok && run > 0;
            if (fill) {
                c_tile = tile;
                c_u = first;
                c_c = cps;
                c_left = run;
                aim_scales(tile, first);
                load_scales();
            }
            // D copies ahead, the wait for x, the units in turn
            for (int i = fill ? -D : 0; i < run || (need && i <= 0); ++i) {
                if (i == 0 && need) {
                    copy_wait();
                    if (!a.x_wide) __syncthreads();
                    stage(u0, u1);
                    __syncthreads();
                }
                if (i >= 0) {
                    if (i >= run || !live || !ok) break;
#pragma unroll
                    for (int m = 0; m < NM; ++m)
                        for (int r = 0; r < 2; ++r) spread_scales<SK>(now[m][r], next[m][r], a.shift);
                    if (i + 1 < run) {
                        if (segs > 1 && s_left <= 0) aim_scales(tile, first + i + 1);
                        load_scales();
                    } else if (whole && tile + tile_step < tiles) {
                        aim_scales(tile + tile_step, first);
                        load_scales();
                    }
                    ok = __all_sync(kAll, mbar_wait(&full[at], phase, abort_flag, a.status, DEV_TIMEOUT_PRODUCER));
                    if (!ok) break;
                    --flying;
                    work(at, first + i - u0);
                    __syncwarp();
                }
                // the next unit of this run, or (if x stays) the first of the next tile's
                if (c_left == 0 && whole && c_tile + tile_step < tiles) {
                    c_tile += tile_step;
                    c_u = first;
                    c_c = cps;
                    c_left = run;
                }
                if (c_left > 0) {
                    copy_next(at);
                    ++flying;
                }
                if (++at == D) {
                    at = 0;
                    if (i >= 0) phase ^= 1;
                }
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
                    float* to = mine + ((m * KW + kwarp) * VS + n * VT + vc) * kRows + row0;
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
                store_vec(a.out, (static_cast<int64_t>(set) * a.nv + n) * a.ld_out + m, a.dt_out, v);
            }
        }
    }
    // a wait ran out: this warp's copies land before its shared memory goes to another block
    for (; !ok && flying > 0; --flying) {
        matvec_drain(&full[at], phase, a.status);
        if (++at == D) {
            at = 0;
            phase ^= 1;
        }
    }
}

int ilog2(int n) { return n > 1 ? 1 + ilog2(n / 2) : 0; }

// Warps of a block and of a team, and blocks of a set.  16 warps an SM, in one block or, where both fit, in two.  A
// block's time, in halves of a unit (0.35 us): its start, some 6 us of first instructions and first loads; its share of
// x; rounds of tiles, each as long as a warp's run and an end.  Taken is what makes the waves of blocks shortest.  (With
// no start counted and half the waves, four tokens of 16 slots, down, took 25 us for 12; twelve of 16 slots kept by
// nobody, or all kept, within 2%.)
template <int SK, int GP, int NT, bool DUAL>
cudaError_t matvec_as(MatvecArgs a, cudaStream_t s) {
    using L = Layout<SK, GP, NT, DUAL>;
    const int tiles = a.tiles;
    const int64_t units = static_cast<int64_t>(a.weights ? a.k : 1) * a.cps;
    const size_t unit_bytes = L::kUnitX + L::kUnitF;
    const bool two = units * unit_bytes + L::kZero + 8 * L::kWarp <= 110 * 1024;
    int64_t best = INT64_MAX;
    int warps = 16;
    for (int w = two ? 8 : 16; w <= 16; w *= 2) {
        // a set of its own for each slot: up to eight waves of blocks, as many of them may have nothing to do
        const int64_t resident = 152 * 16 / w, most = std::max<int64_t>(1, a.idx ? (8 * resident + a.sets - 1) / a.sets : resident / a.sets);
        for (int kw = 1; kw <= w; kw *= 2) {
            const int teams = w / kw;
            const int64_t blocks = std::min<int64_t>((tiles + teams - 1) / teams, most);
            const int64_t rounds = (tiles + blocks * teams - 1) / (blocks * teams), waves = (a.sets * blocks + resident - 1) / resident;
            const int64_t cost = waves * (18 + units * a.nv / w + rounds * (2 * ((units + kw - 1) / kw) + 1));
            if (cost < best) {
                best = cost;
                warps = w;
                a.kw_log = ilog2(kw);
                a.blocks = static_cast<int>(blocks);
            }
        }
    }
    a.cap = static_cast<int>(std::min<int64_t>(units, (kMvSmem - L::kZero - warps * L::kWarp) / unit_bytes));
    const size_t smem = 1024 + a.cap * unit_bytes + L::kZero + warps * L::kWarp;
    // (also gives a host thread its context, which the tensor maps' encoder, a driver call, wants)
    const cudaError_t err = cudaFuncSetAttribute(matvec_kernel<SK, GP, NT, DUAL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMvSmem + 1024);
    if (err != cudaSuccess) return err;
    if (!a.make_maps(a)) return cudaErrorInvalidValue;
    matvec_kernel<SK, GP, NT, DUAL><<<static_cast<unsigned>(a.sets * a.blocks), warps * 32, smem, s>>>(a);
    return cudaGetLastError();
}

// Vectors (three for an fp32 row) against the columns of one MMA: four groups of a row's lanes and two vectors, two and
// four, one and eight, or two MMAs of eight.
template <int SK, bool DUAL>
cudaError_t matvec_of(const MatvecArgs& a, cudaStream_t s) {
    const int vv = a.nv * a.parts;
    if (vv <= 2) return matvec_as<SK, 4, 1, DUAL>(a, s);
    if (vv <= 4) return matvec_as<SK, 2, 1, DUAL>(a, s);
    if (vv <= 8) return matvec_as<SK, 1, 1, DUAL>(a, s);
    return matvec_as<SK, 1, 2, DUAL>(a, s);
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
    a.srow = (a.K / 32 >> a.shift) * size;
    a.unit_scales = (kUnitGroups >> a.shift) * size;
    const uint64_t lie = reinterpret_cast<uintptr_t>(a.scales) | reinterpret_cast<uintptr_t>(a.up_scales) |
                         static_cast<uint64_t>(a.srow) | static_cast<uint64_t>(a.unit_scales);
    a.scale_piece = lie % 16 == 0 ? 16 : lie % 8 == 0 ? 8 : lie % 4 == 0 ? 4 : 0;
    a.cps = (a.K + kUK - 1) / kUK;
    a.tiles = static_cast<int>((static_cast<int64_t>(a.M) + kRows - 1) / kRows);
    if (a.format == 0) return a.up_codes ? matvec_of<SCALE_E8M0, true>(a, s) : matvec_of<SCALE_E8M0, false>(a, s);
    if (a.dt_scale == ELEM_F32) return a.up_codes ? matvec_of<SCALE_F32, true>(a, s) : matvec_of<SCALE_F32, false>(a, s);
    if (a.dt_scale == ELEM_BF16) return a.up_codes ? matvec_of<SCALE_BF16, true>(a, s) : matvec_of<SCALE_BF16, false>(a, s);
    return a.up_codes ? matvec_of<SCALE_F16, true>(a, s) : matvec_of<SCALE_F16, false>(a, s);
}

}  // namespace moe
