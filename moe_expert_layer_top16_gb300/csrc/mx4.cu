// Four-bit activations and four-bit products.
//
//   quantise   MXFP4 codes and scales of fp32, bf16 or fp16 rows, by the rule
//              of the weight encoder: per 32 elements the scale 2^e with
//              e = floor(log2 amax) - 2, each magnitude to the nearest E2M1
//              level, a tie to the smaller one
//   decode     the values that codes and scales stand for
//              (both bound by HBM: 8,192 x 7,168 bf16, 149 MB, 23.8 us to four
//              bits and 23.2 back; 22.0 at the rate of a plain copy)
//   product    out[n][m] = sum_k dq(B[n][k]) dq(A[g(n)][m][k]), A and B both
//              MXFP4, on tcgen05 kind::mxf4 (K = 64 an instruction, twice the
//              rate of the MXFP8 kind), fp32 accumulation
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace moe {

namespace {

// ------------------------------------------------------------------ codec
// Two E2M1 codes (nearest even, saturating) as a byte, `lo` in the low nibble.
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
        "cvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// 2^-14 below one: a 16-bit input on a midpoint of the E2M1 levels, times
// this, lies below it, and the next larger 16-bit value (at least 2^-11 above)
// still lies above, so that rounding to nearest sends ties to the smaller
// level.
constexpr float kTieDown = 1.0f - 0x1p-14f;

// The same for any fp32 value: the low 12 bits become one sticky bit and the
// magnitude goes down by a quarter of the remaining unit, which moves a
// midpoint (few significant bits) below itself and no other value across one.
__device__ __forceinline__ float tie_down(float v) {
    const uint32_t b = __float_as_uint(v), m = b & 0x7FFFFFFFu;
    uint32_t s = (m & 0x7FFFF000u) | ((m & 0xFFFu) ? 0x800u : 0u);
    s = s >= 0x01000000u ? s - 0x400u : 0u;          // below 2^-125: zero in any case
    return __uint_as_float(s | (b & 0x80000000u));
}

// Scale code of a block whose largest magnitude has the bits `top`: 255 (not
// a number) if that is an infinity or a NaN, 0 for a block of zeros.
__device__ __forceinline__ uint32_t mx4_scale_code(uint32_t top) {
    if (top >= 0x7F800000u) return 255u;
    const int biased = static_cast<int>(top >> 23);
    return biased > 2 ? static_cast<uint32_t>(biased - 2) : 0u;      // e = -127 at least
}

// Factor 2^-e for scale code c <= 252.
__device__ __forceinline__ float mx4_inverse(uint32_t c) { return __uint_as_float((254u - c) << 23); }

// Where vector i of a matrix with per_row vectors a row starts: row and vector
// in the row.  Contiguous rows are one long row.
template <bool FLAT>
__device__ __forceinline__ void row_of(int64_t i, int64_t per_row, bool small, int64_t& r, int64_t& c) {
    if (FLAT) {
        r = 0;
        c = i;
    } else if (small) {
        const uint32_t q = static_cast<uint32_t>(i) / static_cast<uint32_t>(per_row);
        r = q;
        c = static_cast<uint32_t>(i) - q * static_cast<uint32_t>(per_row);
    } else {
        r = i / per_row;
        c = i - r * per_row;
    }
}

// Four lanes hold a block of 32, a lane 8 elements; kQuantBatch vectors of a
// thread are loaded before the first is used.  Bound by HBM: 2.53 bytes move
// for a 16-bit element.
constexpr int kQuantBatch = 4;

template <int DT, bool FLAT>
__global__ void __launch_bounds__(256) mxfp4_quantize_kernel(const void* __restrict__ x, int64_t ld, int64_t n,
                                                             int64_t per_row, uint8_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales) {
    pdl_trigger();                             // the product may come up meanwhile
    const bool small = n <= 0xffffffffll;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (256 * kQuantBatch) + threadIdx.x;
    RawVec<8> raw[kQuantBatch];
#pragma unroll
    for (int u = 0; u < kQuantBatch; ++u) {
        const int64_t i = i0 + 256 * u;
        raw[u].a = raw[u].b = make_uint4(0, 0, 0, 0);
        if (i < n) {
            int64_t r, c;
            row_of<FLAT>(i, per_row, small, r, c);
            raw[u] = load_stream<8, DT>(x, r * ld + c * 8);
        }
    }
#pragma unroll
    for (int u = 0; u < kQuantBatch; ++u) {
        const int64_t i = i0 + 256 * u;
        float v[8];
        raw_to_f32(raw[u], DT, v);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        // n is a multiple of 4: a block's four lanes are all inside or all outside
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t sc = mx4_scale_code(top);
        const bool none = top == 0 || sc == 255u;
        const float f = none ? 0.0f : mx4_inverse(sc) * (DT == ELEM_F32 ? 1.0f : kTieDown);
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo = v[2 * j] * f, hi = v[2 * j + 1] * f;
            if (DT == ELEM_F32) {
                lo = tie_down(lo);
                hi = tie_down(hi);
            }
            word |= e2m1_pair(lo, hi) << (8 * j);
        }
        if (i < n) {
            // codes and scales are contiguous: vector i's follow from i alone
            reinterpret_cast<uint32_t*>(codes)[i] = none ? 0u : word;
            if ((threadIdx.x & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(sc);
        }
    }
}

// Rows off 16 bytes: a warp holds a block, a lane an element.
__global__ void __launch_bounds__(256) mxfp4_quantize_plain_kernel(const void* __restrict__ x, int64_t ld, int dt,
                                                                   int64_t n, int64_t K, uint8_t* __restrict__ codes,
                                                                   uint8_t* __restrict__ scales) {
    const bool small = n <= 0xffffffffll;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if ((i & ~31ll) >= n) return;              // whole warps: n is a multiple of 32
    int64_t r, c;
    row_of<false>(i, K, small, r, c);
    float v[1];
    raw_to_f32(load_raw<1>(x, r * ld + c, dt), dt, v);
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(v[0]) & 0x7FFFFFFFu);
    const uint32_t sc = mx4_scale_code(top);
    const bool none = top == 0 || sc == 255u;
    const float f = tie_down(v[0] * (none ? 0.0f : mx4_inverse(sc)));
    const float g = __shfl_down_sync(0xffffffffu, f, 1);
    if (!(threadIdx.x & 1)) codes[i >> 1] = none ? 0 : static_cast<uint8_t>(e2m1_pair(f, g));
    if ((threadIdx.x & 31) == 0) scales[i >> 5] = static_cast<uint8_t>(sc);
}

// 2^e of a scale code: subnormal for code 0, NaN for 255.
__device__ __forceinline__ float mx4_scale(uint32_t c) {
    return __uint_as_float(c == 0 ? 0x00400000u : (c == 255u ? 0x7FC00000u : c << 23));
}

// Two codes of a byte as fp32 (the low nibble first).
__device__ __forceinline__ float2 e2m1_values(uint32_t byte) {
    uint32_t h;
    asm("{\n\t.reg .b8 t;\n\t.reg .b16 w;\n\t"
        "cvt.u16.u32 w, %1;\n\t"
        "mov.b16 {t, _}, w;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
        : "=r"(h)
        : "r"(byte));
    __half2 v;
    memcpy(&v, &h, 4);
    return __half22float2(v);
}

// One thread per 8 codes, kQuantBatch of them in flight.
template <int DT, bool FLAT, int V>
__global__ void __launch_bounds__(256) mxfp4_decode_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int64_t n,
                                                           int64_t per_row, void* __restrict__ x, int64_t ld) {
    const bool small = n <= 0xffffffffll;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (256 * kQuantBatch) + threadIdx.x;
    uint32_t w[kQuantBatch], sc[kQuantBatch];
#pragma unroll
    for (int u = 0; u < kQuantBatch; ++u) {
        const int64_t i = i0 + 256 * u;
        if (i < n) {
            w[u] = __ldcs(reinterpret_cast<const uint32_t*>(codes) + i);
            sc[u] = scales[i >> 2];
        }
    }
#pragma unroll
    for (int u = 0; u < kQuantBatch; ++u) {
        const int64_t i = i0 + 256 * u;
        if (i >= n) break;
        const float f = mx4_scale(sc[u]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 p = e2m1_values((w[u] >> (8 * j)) & 0xFFu);
            v[2 * j] = p.x * f;
            v[2 * j + 1] = p.y * f;
        }
        int64_t r, c;
        row_of<FLAT>(i, per_row, small, r, c);
        if (V == 8) {
            store_stream<8, DT>(x, r * ld + c * 8, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float o[1] = {v[j]};
                store_vec(x, r * ld + c * 8 + j, DT, o);
            }
        }
    }
}

// ------------------------------------------------------------------ product
// A persistent CTA on each SM takes work items (group g, 128 rows of A, up to
// nt rows of B of that group): A is the MMA's M operand, so that a short group
// pads B's rows to 16 only.  A stage is 256 elements of K: 128 bytes a row of
// A and of B, in the 128-byte swizzle.  Roles:
//   warp 0      TMA producer of both operands
//   warp 1      MMA issuer: four MMAs of K = 64 a stage, and a commit
//   warps 4-7   scales: the row-major scales of the item's rows come to shared
//               memory four stages at a time (32 bytes of a row), and the four
//               warps write each its quarter of TMEM, which holds up to four
//               stages' scales: row r of 128 in lane r % 32, column r / 32.
//               The caller's scales need no launch that rearranges them, and
//               the MMA thread issues no copies: with six shared-memory-to-
//               TMEM copies a stage its issue rate set the pace.
//   warp 3      TMA producer of the scales, where their rows are multiples of
//               16 bytes (K a multiple of 512); else warps 4-7 load them
//               themselves, a batch ahead in registers.  Their gathers of 16
//               bytes a row then cost the scale warps 215 to 290 cycles a stage.
//   warps 8-11  epilogue
// A warp writes and reads the TMEM lanes of its number modulo 4.
//
// Wide items run on CTA pairs (clusters of two, cta_group::2): M = 256, each
// CTA holds its 128 rows of A, half of the item's rows of B and, in its TMEM,
// the scales of its rows of A and of all of B's.  The even CTA issues the MMAs
// of both; copies and scale writes of both count on its barriers, its commits
// arrive on both CTAs'.
//
// 8,192 x 8,192 x 7,168 takes 153 us, 6.3 PFLOP/s, with the tensor pipe active
// 66% of the launch (the MMAs' 102 us); K = 14,336 295, so that 28 stages more an
// item cost 141.  What bounds a stage is not settled.  Paired (256 x 192 x 256)
// it moves 28 KB in by TMA, out again to the MMAs, and 11 KB of scales: some 540
// cycles at 128 bytes a cycle, more than the MMAs need.  But items of 208 rows,
// two rounds of items fewer, gained less than 2%, as did the scales' columns
// written by two groups of warps or two stages at a time, or lost.  1,376 items
// on 76 pairs are 18.1 rounds: the last holds eight items, 4% of the time.
// Items of few stages are bound by the epilogue: an output of 8,192 x 8,192 takes
// 118 us at K = 512 and 137 at 3,584, in bf16 and in fp32.  Gathered scales: K =
// 7,040 235 us, 3,456 147; 64 groups of 146 rows (M = 1,024) 38 us at K = 3,456,
// 36 at 3,584.
// Decode (73 rows for 64 groups of 1,024 x 3,584) is bound by the weights' way
// from HBM: 20 us for 85 MB; at K = 3,456 28.
//
// Unpaired, 41 KB of operands a stage came into an SM at
// 64 bytes a cycle, which bounded the product; a pair's CTA takes 28 KB.  Groups
// of few rows are bound by A's way from HBM, which pairs do not shorten.  Pairs
// against single CTAs, M = 8192, K = 7168: 4,096 rows 82.3 and 90.5 us, 1,024
// rows 31.3 and 33.4, 512 rows 24.4 and 24.9; 64 groups of 146 rows (M = 1024,
// K = 3584) 37.9 and 35.9, 16 of 125 rows 13.5 and 12.4.
constexpr int kMx4PairRows = 512;                 // rows of B a group, on average, from which on pairs are used
constexpr int kMx4BlockM = 128;
constexpr int kMx4BlockK = 256;
constexpr int kMx4NtMax = 192;                    // two accumulators and four sets of scale columns in 512;
                                                  // five stages (208: four)
constexpr int kMx4ABytes = kMx4BlockM * 128;
constexpr int kMx4Threads = 12 * 32;
constexpr int kMx4MaxStages = 16;
constexpr int kMx4MinStages = 4;
constexpr int kMx4MaxSets = 4;
constexpr int kMx4SetCols = 24;                   // 2 x 4 columns of A's scales, 2 x 8 of B's
constexpr int kMx4Batch = 4;                      // stages whose scales are loaded together: 32 bytes of a row
constexpr int kMx4ScaleRows = kMx4BlockM + (kMx4NtMax + 31) / 32 * 32;
constexpr int kMx4ScaleBuf = kMx4ScaleRows * 32;  // a batch: 128 rows of A, then B's
constexpr int kMx4ScaleBytes = 2 * kMx4ScaleBuf;
constexpr int kMx4RowLoads = (2 * (kMx4BlockM + kMx4NtMax) + 127) / 128;      // 16-byte pieces of a batch a thread
constexpr int kMx4TmemCols = 512;
constexpr int kMx4MaxGroups = 1024;
constexpr int kMx4BarBytes = (3 * kMx4MaxStages + 9) * 8 + 24;

struct Mx4Item {
    int a_row, m0, b_row, n;
};

struct Mx4Geometry {
    int M, m_rows, m_first, m_tiles, nt, G;      // m_rows: rows of A of an item, m_first: this CTA's first of them
    const int* tile_off;     // [G + 1] first token tile of each group
    const int* first;        // [G + 1] first row; first[G]: unused
    const int* count;        // [G]
};

__device__ __forceinline__ Mx4Item mx4_item(const Mx4Geometry& g, int64_t it) {
    const int tile = static_cast<int>(it / g.m_tiles);
    const int mt = static_cast<int>(it - static_cast<int64_t>(tile) * g.m_tiles);
    int lo = 0, hi = g.G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.tile_off[mid] <= tile) lo = mid;
        else hi = mid - 1;
    }
    const int j = tile - g.tile_off[lo];
    Mx4Item w;
    w.m0 = mt * g.m_rows + g.m_first;
    w.a_row = lo * g.M + w.m0;
    w.b_row = g.first[lo] + j * g.nt;
    w.n = min(g.nt, g.count[lo] - j * g.nt);
    return w;
}

// Sixteen scale codes (two stages) of a row, of which `left` codes (a multiple
// of 4) belong to the row, as words; codes behind the row read as 0.  Plain
// loads: the kernel before this one, which it overlaps, may have written them.
__device__ __forceinline__ uint4 load_scales(const uint8_t* at, int left) {
    uint4 r = make_uint4(0, 0, 0, 0);
    const uint32_t* p = reinterpret_cast<const uint32_t*>(at);
    r.x = p[0];
    if (left > 4) r.y = p[1];
    if (left > 8) r.z = p[2];
    if (left > 12) r.w = p[3];
    return r;
}

// Place of 16-byte half `h` of row r in the shared rows of 32 bytes: halves
// swap every four rows, so that eight rows' halves lie in different banks.
__device__ __forceinline__ int scale_place(int r, int h) { return r * 32 + ((h ^ ((r >> 2) & 1)) << 4); }

__device__ __forceinline__ bool mx4_drain(uint64_t* bar, uint32_t parity, int* status) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            if (status) atomicCAS(status, 0, DEV_TIMEOUT_TEARDOWN);
            return false;
        }
    }
    return true;
}

template <int DT>
__device__ __forceinline__ void store_out(void* out, int64_t off, float v) {
    if (DT == ELEM_F32) static_cast<float*>(out)[off] = v;
    else if (DT == ELEM_BF16) static_cast<__nv_bfloat16*>(out)[off] = __float2bfloat16_rn(v);
    else static_cast<__half*>(out)[off] = __float2half_rn(v);
}

template <int DT, bool SFT, bool PAIR>
__global__ void __launch_bounds__(kMx4Threads, 1) mx4_gemm_kernel(const __grid_constant__ Mx4Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    pdl_trigger();
    const int S = pin(p.stages), stage_bytes = pin(p.stage_bytes);
    const int M = pin(p.M), K = pin(p.K), nt = pin(p.nt), G = pin(p.G), b_box = pin(p.b_box);
    const int off_b = kMx4ABytes;
    const int sets = min(kMx4MaxSets, (kMx4TmemCols - 2 * nt) / kMx4SetCols);
    uint8_t* tail = base + S * stage_bytes;
    uint8_t* scales = tail;                                  // [2][128 of A, then nt of B][32]
    uint64_t* full = reinterpret_cast<uint64_t*>(tail + kMx4ScaleBytes);      // operands of a stage have landed
    uint64_t* sfull = full + kMx4MaxStages;                  // its scales are in TMEM
    uint64_t* empty = sfull + kMx4MaxStages;
    uint64_t* tfull = empty + kMx4MaxStages;                 // [2]
    uint64_t* tempty = tfull + 2;                            // [2]
    uint64_t* cfull = tempty + 2;                            // [2] a batch of scales has landed
    uint64_t* cempty = cfull + 2;                            // [2]
    uint64_t* tdown = cempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tdown + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* tile_off = reinterpret_cast<int*>(tail + kMx4ScaleBytes + kMx4BarBytes);
    int* first = tile_off + G + 1;
    int* count = first + G + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* status = pin(p.status);
    const int cta = PAIR ? static_cast<int>(cluster_ctarank()) : 0;      // the even CTA (0) issues the MMAs
    const int unit = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
    const int units = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&sfull[s], PAIR && cta == 0 ? 8 : 4);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], PAIR && cta == 0 ? 8 : 4);
            mbar_init(&cfull[b], 1);
            mbar_init(&cempty[b], 4);
        }
        mbar_init(tdown, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&p.tmA);
        prefetch_tmap(&p.tmB);
        if (SFT) {
            prefetch_tmap(&p.tmSA);
            prefetch_tmap(&p.tmSB);
        }
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(tmem_slot, kMx4TmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, kMx4TmemCols);
            tmem_relinquish();
        }
    }
    // the launch overlaps the end of the kernel before (the quantiser of B, as a
    // rule), whose results are read from here on: 512 rows quantised and
    // multiplied by 16 groups 8.8 us, 9.3 without
    pdl_wait();
    if (warp == 2) {
        // token tiles of each group, from the offsets (kept inside [0, N])
        const int per = (G + 31) / 32;
        int sum = 0;
        for (int u = 0; u < per; ++u) {
            const int g = lane * per + u;
            if (g >= G) break;
            int lo = 0, hi = p.N;
            if (p.offsets) {
                lo = min(max(p.offsets[g], 0), p.N);
                hi = min(max(p.offsets[g + 1], lo), p.N);
            }
            first[g] = lo;
            count[g] = hi - lo;
            tile_off[g] = sum;
            sum += (hi - lo + nt - 1) / nt;
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        for (int u = 0; u < per; ++u) {
            const int g = lane * per + u;
            if (g < G) tile_off[g] += incl - sum;
        }
        if (lane == 31) tile_off[G] = incl;
    }
    tc_fence_before();
    __syncthreads();
    // a pair's barriers are initialised before either CTA signals the other's
    if constexpr (PAIR) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    constexpr int kRows = PAIR ? 2 * kMx4BlockM : kMx4BlockM;
    const int m_tiles = (M + kRows - 1) / kRows;
    const Mx4Geometry geo{M, kRows, cta * kMx4BlockM, m_tiles, nt, G, tile_off, first, count};
    const int64_t items = static_cast<int64_t>(tile_off[G]) * m_tiles;
    const int KT = (K + kMx4BlockK - 1) / kMx4BlockK;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        uint32_t stage = 0, phase = 0, issued = 0, issued_parity = 0;
        bool ok = true;
        for (int64_t it = unit; ok && it < items; it += units) {
            const Mx4Item w = mx4_item(geo, it);
            const int nm = (w.n + 15) & ~15;
            const int nbox = (nm + b_box - 1) / b_box;
            // (a pair: one box of half of the item's rows in each CTA, both
            // counted on the even one's barrier)
            const uint32_t tx = PAIR ? 2u * static_cast<uint32_t>(kMx4ABytes + b_box * 128)
                                     : static_cast<uint32_t>(kMx4ABytes + nbox * b_box * 128);
            for (int kt = 0; kt < KT; ++kt) {
                ok = mbar_wait(&empty[stage], phase ^ 1, abort_flag, status, DEV_TIMEOUT_PRODUCER);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                if constexpr (PAIR) {
                    if (elect_one()) {
                        uint8_t* sb = base + stage * stage_bytes;
                        const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
                        if (cta == 0) mbar_arrive_expect_tx(&full[stage], tx);
                        tma_load_2d_pair(sb, &p.tmA, fb, kt * 128, w.a_row);
                        tma_load_2d_pair(sb + off_b, &p.tmB, fb, kt * 128, w.b_row + cta * (nm >> 1));
                    }
                } else if (elect_one()) {
                    uint8_t* sb = base + stage * stage_bytes;
                    mbar_arrive_expect_tx(&full[stage], tx);
                    tma_load_2d(sb, &p.tmA, &full[stage], kt * 128, w.a_row);
                    for (int c = 0; c < nbox; ++c)
                        tma_load_2d(sb + off_b + c * b_box * 128, &p.tmB, &full[stage], kt * 128, w.b_row + c * b_box);
                }
                __syncwarp();
                issued |= 1u << stage;
                issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == static_cast<uint32_t>(S)) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if constexpr (PAIR) {
            // the even CTA's MMAs read this CTA's stages and its commits arrive
            // here: every stage is released before this CTA leaves
            for (int i = 0; ok && i < S; ++i) {
                ok = mbar_wait(&empty[stage], phase ^ 1, abort_flag, status, DEV_TIMEOUT_PRODUCER);
                ok = __all_sync(0xffffffffu, ok);
                if (++stage == static_cast<uint32_t>(S)) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (*abort_flag && lane == 0 && cta == 0) {
            // every copy in flight lands before the CTA leaves (a pair's all
            // count on the even CTA's barriers)
            for (int s = 0; s < S; ++s)
                if (issued & (1u << s)) mx4_drain(&full[s], (issued_parity >> s) & 1u, status);
        }
        __syncwarp();
    } else if (warp == 1 && cta == 0) {
        // ------------------------------------------------------------ MMA issuer
        uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0, set = 0;
        bool any = false;
        // descriptors of stage 0; a stage further on adds its offset (the
        // start-address field counts 16-byte units)
        const uint64_t ad0 = sdesc_sw128(smem_u32(base)), bd0 = sdesc_sw128(smem_u32(base + off_b));
        const uint32_t sf0 = tmem + 2u * static_cast<uint32_t>(nt);
        for (int64_t it = unit; it < items; it += units) {
            const Mx4Item w = mx4_item(geo, it);
            const int nm = (w.n + 15) & ~15;
            bool ok = mbar_wait(&tempty[acc], acc_phase ^ 1, abort_flag, status, DEV_TIMEOUT_MMA);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const uint32_t d = tmem + acc * static_cast<uint32_t>(nt);
            const uint32_t idesc0 = idesc_mxf4(kRows, nm);
            for (int kt = 0; kt < KT; ++kt) {
                // a stage that is already there is seen so by every lane at
                // once: the warp-wide vote only on the waiting path
                if (!mbar_try_wait(&full[stage], phase) || !mbar_try_wait(&sfull[stage], phase)) {
                    ok = mbar_wait(&full[stage], phase, abort_flag, status, DEV_TIMEOUT_MMA) &&
                         mbar_wait(&sfull[stage], phase, abort_flag, status, DEV_TIMEOUT_MMA);
                    if (!__all_sync(0xffffffffu, ok)) goto mma_done;
                }
                tc_fence_after();                      // the scales were written by other threads
                const uint64_t off = static_cast<uint64_t>(stage) * (static_cast<uint32_t>(stage_bytes) >> 4);
                const uint64_t ad = ad0 + off, bd = bd0 + off;
                const uint32_t sfa = sf0 + set * kMx4SetCols, sfb = sfa + 8u;
                const bool both = K - kt * kMx4BlockK > 128;
                if (elect_one()) {
                    // scale ids 0 and 2: the low and high half of each scale word
                    constexpr uint32_t high = 2u << 4 | 2u << 29;
                    auto mma = [&](int j, uint32_t id, uint32_t fa, uint32_t fb, uint32_t add) {
                        if constexpr (PAIR) mma_mxf4_pair(d, ad + 2 * j, bd + 2 * j, id, fa, fb, add);
                        else mma_mxf4(d, ad + 2 * j, bd + 2 * j, id, fa, fb, add);
                    };
                    mma(0, idesc0, sfa, sfb, kt != 0 ? 1u : 0u);
                    mma(1, idesc0 | high, sfa, sfb, 1u);
                    if (both) {
                        mma(2, idesc0, sfa + 4u, sfb + 8u, 1u);
                        mma(3, idesc0 | high, sfa + 4u, sfb + 8u, 1u);
                    }
                    if constexpr (PAIR) tc_commit_pair(&empty[stage], 3);
                    else tc_commit(&empty[stage]);
                }
                any = true;
                __syncwarp();
                if (++set == static_cast<uint32_t>(sets)) set = 0;
                if (++stage == static_cast<uint32_t>(S)) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (elect_one()) {
                if constexpr (PAIR) tc_commit_pair(&tfull[acc], 3);
                else tc_commit(&tfull[acc]);
            }
            __syncwarp();
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1;
        }
    mma_done:
        // every tcgen05 operation finishes before TMEM is freed
        if (any) {
            if (elect_one()) {
                if constexpr (PAIR) tc_commit_pair(tdown, 1);
                else tc_commit(tdown);
                mx4_drain(tdown, 0, status);
            }
            __syncwarp();
        }
    } else if (SFT && warp == 3) {
        // ------------------------------------------------------------ producer of the scales
        const int batches = (KT + kMx4Batch - 1) / kMx4Batch;
        uint32_t buf = 0, phase = 0, issued = 0, issued_parity = 0;
        bool ok = true;
        for (int64_t it = unit; ok && it < items; it += units) {
            const Mx4Item w = mx4_item(geo, it);
            for (int b = 0; b < batches; ++b) {
                ok = mbar_wait(&cempty[buf], phase ^ 1, abort_flag, status, DEV_TIMEOUT_PRODUCER);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    uint8_t* d = scales + buf * kMx4ScaleBuf;
                    mbar_arrive_expect_tx(&cfull[buf], static_cast<uint32_t>((kMx4BlockM + nt) * 32));
                    tma_load_2d(d, &p.tmSA, &cfull[buf], b * 32, w.a_row);
                    tma_load_2d(d + kMx4BlockM * 32, &p.tmSB, &cfull[buf], b * 32, w.b_row);
                }
                __syncwarp();
                issued |= 1u << buf;
                issued_parity = (issued_parity & ~(1u << buf)) | (phase << buf);
                buf ^= 1;
                if (buf == 0) phase ^= 1;
            }
        }
        if (*abort_flag && lane == 0) {
            for (int b = 0; b < 2; ++b)
                if (issued & (1u << b)) mx4_drain(&cfull[b], (issued_parity >> b) & 1u, status);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------------ scales
        const int q = warp & 3, tid = threadIdx.x & 127;
        const uint32_t t_lane = static_cast<uint32_t>(32 * q) << 16;
        const int pitch = K / 32;
        const int batches = (KT + kMx4Batch - 1) / kMx4Batch;
        // without TMA: piece i of this thread is half (tid & 1) of row 64 i +
        // tid / 2, rows of A first; a batch is read while the one before it is
        // in use
        constexpr int kPieces = SFT ? 1 : kMx4RowLoads;
        uint4 piece[kPieces];
        const uint8_t* at[kPieces];                    // this thread's rows of the item, null: none
        auto aim = [&](const Mx4Item& w) {
            if constexpr (!SFT) {
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int r = 64 * i + (tid >> 1), b = r - kMx4BlockM;
                    at[i] = nullptr;
                    if (i < 2 && w.m0 + r < M) at[i] = p.sfa + static_cast<int64_t>(w.a_row + r) * pitch + (tid & 1) * 16;
                    if (i >= 2 && b < w.n) at[i] = p.sfb + static_cast<int64_t>(w.b_row + b) * pitch + (tid & 1) * 16;
                }
            }
        };
        auto read = [&](int batch) {
            if constexpr (!SFT) {
                const int c = batch * (8 * kMx4Batch), left = pitch - c - (tid & 1) * 16;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    piece[i] = make_uint4(0, 0, 0, 0);
                    if (at[i] && left > 0) piece[i] = load_scales(at[i] + c, left);
                }
            }
        };
        int64_t it = unit;
        int batch = 0, n = 0, n_next = 0;
        if (it < items) {
            const Mx4Item w = mx4_item(geo, it);
            n_next = w.n;
            aim(w);
            read(0);
        }
        uint32_t stage = 0, set = 0, turn = 0;
        uint32_t old_stage = 0, old_phase = 0;         // of the turn that last used the set
        uint32_t buf = 0, buf_phase = 0;
        bool ok = true;
        while (it < items) {
            n = n_next;
            if (SFT) {
                if (!mbar_try_wait(&cfull[buf], buf_phase)) {
                    ok = mbar_wait(&cfull[buf], buf_phase, abort_flag, status, DEV_TIMEOUT_PRODUCER);
                    ok = __all_sync(0xffffffffu, ok);
                }
                if (!ok) break;
            } else {
                // the four warps have read the batch before, and leave together
                // if a wait of one of them ran out
                uint32_t all;
                __syncwarp();
                asm volatile(
                    "{\n\t.reg .pred p, r;\n\t"
                    "setp.ne.u32 p, %1, 0;\n\t"
                    "bar.red.and.pred r, 1, 128, p;\n\t"
                    "selp.u32 %0, 1, 0, r;\n\t}"
                    : "=r"(all)
                    : "r"(ok ? 1u : 0u)
                    : "memory");
                if (!all) break;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int r = 64 * i + (tid >> 1);
                    if (i < 2 || r - kMx4BlockM < n) *reinterpret_cast<uint4*>(scales + scale_place(r, tid & 1)) = piece[i];
                }
                named_bar_sync(2, 128);
            }
            const int stages_here = min(kMx4Batch, KT - batch * kMx4Batch);
            if (++batch == batches) {
                batch = 0;
                it += units;
                if (it < items) {
                    const Mx4Item w = mx4_item(geo, it);
                    n_next = w.n;
                    aim(w);
                }
            }
            if (it < items) read(batch);
            const uint8_t* rows = scales + buf * kMx4ScaleBuf;
            // two stages from each 16-byte half
#pragma unroll
            for (int h = 0; h < kMx4Batch / 2; ++h) {
                uint4 a[4], b[8];
                if (2 * h < stages_here) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const uint4*>(rows + scale_place(32 * i + lane, h));
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // rows behind the item's last: their columns are never stored
                        b[i] = make_uint4(0, 0, 0, 0);
                        if (32 * i < kMx4NtMax && 32 * i < n)
                            b[i] = *reinterpret_cast<const uint4*>(rows + scale_place(kMx4BlockM + 32 * i + lane, h));
                    }
                }
                if (SFT && h == kMx4Batch / 2 - 1) {   // the buffer has been read
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&cempty[buf]);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (2 * h + k >= stages_here || !ok) break;
                    // the MMAs that read this set's last scales are done
                    if (turn >= static_cast<uint32_t>(sets)) {
                        if (!mbar_try_wait(&empty[old_stage], old_phase)) {
                            ok = mbar_wait(&empty[old_stage], old_phase, abort_flag, status, DEV_TIMEOUT_PRODUCER);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                        }
                        if (++old_stage == static_cast<uint32_t>(S)) {
                            old_stage = 0;
                            old_phase ^= 1;
                        }
                    }
                    tc_fence_after();
                    const uint32_t cols = tmem + t_lane + 2u * static_cast<uint32_t>(nt) + set * kMx4SetCols;
                    uint32_t lo[8], hi[8], av[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        lo[i] = k ? b[i].z : b[i].x;
                        hi[i] = k ? b[i].w : b[i].y;
                        av[i] = i < 4 ? (k ? a[i & 3].z : a[i & 3].x) : (k ? a[i & 3].w : a[i & 3].y);
                    }
                    tmem_st8(cols, av);
                    tmem_st8(cols + 8, lo);
                    tmem_st8(cols + 16, hi);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        // (the columns are written: tcgen05.wait::st; nothing in memory
                        // to order, and a release at cluster scope costs a microsecond)
                        if (PAIR && cta == 1) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&sfull[stage]), 0));
                        else mbar_arrive(&sfull[stage]);
                    }
                    ++turn;
                    if (++set == static_cast<uint32_t>(sets)) set = 0;
                    if (++stage == static_cast<uint32_t>(S)) stage = 0;
                }
            }
            if (SFT) {
                buf ^= 1;
                if (buf == 0) buf_phase ^= 1;
            }
        }
    } else if (warp >= 8) {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3;         // TMEM lanes this warp may read
        const uint32_t t_lane = static_cast<uint32_t>(32 * quarter) << 16;
        uint32_t acc = 0, acc_phase = 0;
        for (int64_t it = unit; it < items; it += units) {
            const Mx4Item w = mx4_item(geo, it);
            const bool ok = mbar_wait(&tfull[acc], acc_phase, abort_flag, status, DEV_TIMEOUT_EPILOGUE);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const uint32_t a0 = tmem + t_lane + acc * static_cast<uint32_t>(nt);
            const int col = w.m0 + 32 * quarter + lane;
            const bool in = col < M;
            const int nm = (w.n + 15) & ~15;
            uint32_t cur[16], nxt[16];
            tmem_ld16_async(a0, cur);
            tmem_wait16(cur);
            for (int n0 = 0; n0 < nm; n0 += 16) {
                const bool more = n0 + 16 < nm;
                if (more) tmem_ld16_async(a0 + static_cast<uint32_t>(n0 + 16), nxt);
                const int nv = min(16, w.n - n0);
                int64_t o = static_cast<int64_t>(w.b_row + n0) * p.ld_out + col;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (i >= nv) break;
                    if (in) store_out<DT>(p.out, o, __uint_as_float(cur[i]));
                    o += p.ld_out;
                }
                if (more) {
                    tmem_wait16(nxt);
#pragma unroll
                    for (int i = 0; i < 16; ++i) cur[i] = nxt[i];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                // (this warp's TMEM loads are complete: nothing else to order)
                if (PAIR && cta == 1) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&tempty[acc]), 0));
                else mbar_arrive(&tempty[acc]);
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    // neither CTA of a pair frees TMEM or leaves while the other may still
    // signal its barriers
    if constexpr (PAIR) cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, kMx4TmemCols);
        else tmem_dealloc(tmem, kMx4TmemCols);
    }
}

template <bool SFT, bool PAIR>
auto mx4_kernel_as(int dt_out) {
    return dt_out == ELEM_F32 ? mx4_gemm_kernel<ELEM_F32, SFT, PAIR>
                              : (dt_out == ELEM_BF16 ? mx4_gemm_kernel<ELEM_BF16, SFT, PAIR> : mx4_gemm_kernel<ELEM_F16, SFT, PAIR>);
}
auto mx4_kernel(int dt_out, bool sf_tma, bool pair) {
    if (pair) return sf_tma ? mx4_kernel_as<true, true>(dt_out) : mx4_kernel_as<false, true>(dt_out);
    return sf_tma ? mx4_kernel_as<true, false>(dt_out) : mx4_kernel_as<false, false>(dt_out);
}

int mx4_stage_bytes(int nt, bool pair) { return (kMx4ABytes + (pair ? nt / 2 : nt) * 128 + 1023) & ~1023; }

int mx4_table_bytes(int G) { return (3 * (G + 1) * 4 + 15) & ~15; }

}  // namespace

cudaError_t mx4_pair_clusters(int M, int N, int G, int* clusters) {
    *clusters = 0;
    if (N < static_cast<int64_t>(kMx4PairRows) * G || M <= kMx4BlockM) return cudaSuccess;
    // (its instances differ in neither threads nor shared memory, which decide)
    static PerDevice counts;
    return once_a_device(
        counts, [](int* c) { return resident_pairs(mx4_gemm_kernel<ELEM_F32, true, true>, kMx4Threads, kSmemLimit, c); }, clusters);
}

cudaError_t mx4_setup(const Mx4Params& p) {
    return cudaFuncSetAttribute(mx4_kernel(p.dt_out, p.sf_tma, p.pair_clusters > 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmemLimit);
}

void mx4_tiles(int N, int G, bool pair, int* nt, int* b_box) {
    if (G == 1) {
        // equal tiles, a box each
        const int tiles = (N + kMx4NtMax - 1) / kMx4NtMax;
        *nt = ((N + tiles - 1) / tiles + 15) & ~15;
        *b_box = *nt;
    } else {
        // room for about twice the mean; boxes that follow a short group's rows
        int64_t n = (2 * static_cast<int64_t>(N) + G - 1) / G;
        n = n > kMx4NtMax ? kMx4NtMax : (n < 16 ? 16 : n);
        *b_box = n > 64 ? 32 : 16;
        *nt = static_cast<int>((n + *b_box - 1) / *b_box * *b_box);
    }
    if (pair) *b_box = *nt / 2;
}

cudaError_t launch_mx4_gemm(const Mx4Params& in, cudaStream_t s) {
    Mx4Params p = in;
    if (p.M < 1 || p.N < 1 || p.K < 128 || p.K % 128 || p.G < 1 || p.G > kMx4MaxGroups) return cudaErrorInvalidValue;
    const bool pair = p.pair_clusters > 0;
    if (p.nt < 16 || p.nt > kMx4NtMax || p.nt % 16 || (pair ? 2 * p.b_box != p.nt : (p.b_box < 16 || p.nt % p.b_box)))
        return cudaErrorInvalidValue;
    p.stage_bytes = mx4_stage_bytes(p.nt, pair);
    const int fixed = 1024 + kMx4ScaleBytes + kMx4BarBytes + mx4_table_bytes(p.G);
    p.stages = (kSmemLimit - fixed) / p.stage_bytes;
    if (p.stages > kMx4MaxStages) p.stages = kMx4MaxStages;
    if (p.stages < kMx4MinStages) return cudaErrorInvalidValue;
    const size_t smem = fixed + static_cast<size_t>(p.stages) * p.stage_bytes;
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    const int64_t m_tiles = (p.M + (pair ? 2 : 1) * kMx4BlockM - 1) / ((pair ? 2 : 1) * kMx4BlockM);
    const int64_t most = m_tiles * ((p.N + p.nt - 1) / p.nt + p.G - 1);
    const int64_t units = std::min<int64_t>(most, pair ? p.pair_clusters : sms);
    void (*kern)(Mx4Params) = mx4_kernel(p.dt_out, p.sf_tma, pair);
    if (pair)
        return launch_ex_cluster(kern, dim3(static_cast<unsigned>(2 * units)), dim3(kMx4Threads), smem, s, true, 2, p);
    return launch_ex(kern, dim3(static_cast<unsigned>(units)), dim3(kMx4Threads), smem, s, true, p);
}

namespace {

template <int DT>
void quantize_as(const void* x, int64_t ld, int64_t rows, int64_t K, uint8_t* codes, uint8_t* scales, unsigned grid,
                 cudaStream_t s) {
    const int64_t n = rows * (K / 8);
    if (ld == K || rows == 1) mxfp4_quantize_kernel<DT, true><<<grid, 256, 0, s>>>(x, ld, n, K / 8, codes, scales);
    else mxfp4_quantize_kernel<DT, false><<<grid, 256, 0, s>>>(x, ld, n, K / 8, codes, scales);
}

template <int DT>
void decode_as(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* x, int64_t ld, bool v8,
               unsigned grid, cudaStream_t s) {
    const int64_t n = rows * (K / 8);
    if (!v8) mxfp4_decode_kernel<DT, false, 1><<<grid, 256, 0, s>>>(codes, scales, n, K / 8, x, ld);
    else if (ld == K || rows == 1) mxfp4_decode_kernel<DT, true, 8><<<grid, 256, 0, s>>>(codes, scales, n, K / 8, x, ld);
    else mxfp4_decode_kernel<DT, false, 8><<<grid, 256, 0, s>>>(codes, scales, n, K / 8, x, ld);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const void* x, int64_t ld, int dt, int64_t rows, int64_t K, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t s) {
    if (rows < 0 || K <= 0 || K % 32) return cudaErrorInvalidValue;
    if (rows == 0) return cudaSuccess;
    const bool v8 = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (rows == 1 || (ld * elem_bytes(dt)) % 16 == 0);
    const int64_t per_block = v8 ? 256 * kQuantBatch : 256;
    const int64_t blocks = (rows * (K / (v8 ? 8 : 1)) + per_block - 1) / per_block;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(blocks);
    if (!v8) mxfp4_quantize_plain_kernel<<<grid, 256, 0, s>>>(x, ld, dt, rows * K, K, codes, scales);
    else if (dt == ELEM_F32) quantize_as<ELEM_F32>(x, ld, rows, K, codes, scales, grid, s);
    else if (dt == ELEM_BF16) quantize_as<ELEM_BF16>(x, ld, rows, K, codes, scales, grid, s);
    else quantize_as<ELEM_F16>(x, ld, rows, K, codes, scales, grid, s);
    return cudaGetLastError();
}

cudaError_t launch_mxfp4_decode(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* x,
                                int64_t ld, int dt, cudaStream_t s) {
    if (rows < 0 || K <= 0 || K % 32) return cudaErrorInvalidValue;
    if (rows == 0) return cudaSuccess;
    const bool v8 = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (rows == 1 || (ld * elem_bytes(dt)) % 16 == 0);
    const int64_t blocks = (rows * (K / 8) + 256 * kQuantBatch - 1) / (256 * kQuantBatch);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(blocks);
    if (dt == ELEM_F32) decode_as<ELEM_F32>(codes, scales, rows, K, x, ld, v8, grid, s);
    else if (dt == ELEM_BF16) decode_as<ELEM_BF16>(codes, scales, rows, K, x, ld, v8, grid, s);
    else decode_as<ELEM_F16>(codes, scales, rows, K, x, ld, v8, grid, s);
    return cudaGetLastError();
}

}  // namespace moe
