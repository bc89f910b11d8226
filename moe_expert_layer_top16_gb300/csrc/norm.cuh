// What the forward pass and the gradients of the norms round a block share:
// rows by windows, their sums, and how a launch covers them.
#pragma once
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace moe {

constexpr int kNormMaxWarps = 32;
constexpr int kNormMaxStages = 8;

// ------------------------------------------------------------------ rows by windows
// A row is cut at the windows of its matrix (8 elements: 16 bytes of a 16-bit
// type; 4 for an fp32 x), not at its own start: for rows of any
// length the windows inside a row are whole 16-byte words, and only its first
// and last window may be partial.  All matrices of a launch have 16-byte
// aligned bases and row strides that are equal modulo a window, so a row lies
// alike in all of them; a block takes every (8 m)-th row, so that its rows all
// start at the same place in their first window and thread i owns the same
// columns in each.
//
// A row is owned by a group of tpr threads; a block holds blockDim / tpr
// groups, which share its weights.  A row too wide for one block is split over
// the blocks of a cluster (each one group), a part of the columns each.
constexpr int kNormMaxSplit = 4;
struct Rows {
    int tpr, lane_in_group, group, groups;
    int unit, units;            // this block among the blocks (its cluster among the clusters)
    int part, parts;            // this block in its cluster
    int first, step;            // rows first, first + step, ...
    int shift;                  // elements of the first window that belong to the row before
};

template <bool SPLIT>
__device__ __forceinline__ Rows rows_of(int tpr, int64_t ld, int window) {
    Rows r;
    r.tpr = tpr;
    r.part = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
    r.parts = SPLIT ? static_cast<int>(cluster_ctas()) : 1;
    r.unit = SPLIT ? static_cast<int>(blockIdx.x) / r.parts : static_cast<int>(blockIdx.x);
    r.units = SPLIT ? static_cast<int>(gridDim.x) / r.parts : static_cast<int>(gridDim.x);
    r.groups = blockDim.x / tpr;
    r.group = threadIdx.x / tpr;
    r.lane_in_group = threadIdx.x - r.group * tpr;
    r.first = r.unit + r.units * r.group;
    r.step = r.units * r.groups;
    r.shift = static_cast<int>((r.unit * ld) & (window - 1));
    return r;
}

// Element types that an instance of the kernels is made for (RUN: as the
// arguments say): of x, dx, h and dh, and of y.  u has x's type, except in the
// forward F32 instance, whose u has any.  The backward instances other than
// RUN have both norms and every matrix of them.  F32_Y16 (forward only): y of
// either 16-bit type, by windows of four like x.
enum NormKind : int { NORM_RUN, NORM_BF16, NORM_BF16_Y32, NORM_F16, NORM_F16_Y32, NORM_F32, NORM_F32_Y16 };
template <int KIND>
struct Kind {
    static constexpr bool wide = KIND == NORM_F32 || KIND == NORM_F32_Y16, full = KIND != NORM_RUN;
    static constexpr bool half = KIND == NORM_F16 || KIND == NORM_F16_Y32, small = full && !wide;
    static constexpr int window = wide ? 4 : 8;
    static constexpr int x = !full ? -1 : (wide ? ELEM_F32 : (half ? ELEM_F16 : ELEM_BF16));
    static constexpr int y = KIND == NORM_BF16 || KIND == NORM_F16 ? x : (full && KIND != NORM_F32_Y16 ? ELEM_F32 : -1);
};

// The kind of a launch whose x is of a 16-bit type (RUN: another pair).
inline int small_kind(int x, int y) {
    if (x == ELEM_BF16) return y == ELEM_BF16 ? NORM_BF16 : (y == ELEM_F32 ? NORM_BF16_Y32 : NORM_RUN);
    if (x == ELEM_F16) return y == ELEM_F16 ? NORM_F16 : (y == ELEM_F32 ? NORM_F16_Y32 : NORM_RUN);
    return NORM_RUN;
}

// f with the instance's EDGE and KIND as types (RUN: with EDGE).
template <typename F>
cudaError_t with_kind(int kind, bool edge, F f) {
    auto one = [&](auto k) {
        return edge ? f(std::true_type{}, k) : f(std::false_type{}, k);
    };
    switch (kind) {
        case NORM_BF16: return one(std::integral_constant<int, NORM_BF16>{});
        case NORM_BF16_Y32: return one(std::integral_constant<int, NORM_BF16_Y32>{});
        case NORM_F16: return one(std::integral_constant<int, NORM_F16>{});
        case NORM_F16_Y32: return one(std::integral_constant<int, NORM_F16_Y32>{});
        case NORM_F32: return one(std::integral_constant<int, NORM_F32>{});
        default: return f(std::true_type{}, std::integral_constant<int, NORM_RUN>{});
    }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most n of this thread's copy groups are in flight (one: the
// widest rows, tested first).
__device__ __forceinline__ void cp_async_wait(int n) {
    if (n == 1) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        return;
    }
    switch (n) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
        case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    }
}

// Two fp32 values in a register pair: the packed multiply and add take two
// elements an instruction.
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair(float lo, float hi) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ float2 split(Pair p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float sum2(Pair p) {
    const float2 f = split(p);
    return f.x + f.y;
}
// A 16-bit pair as fp32.
__device__ __forceinline__ Pair widen(uint32_t w, int dt) {
    if (dt == ELEM_BF16) return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    __half2 h;
    memcpy(&h, &w, 4);
    const float2 f = __half22float2(h);
    return pair(f.x, f.y);
}
__device__ __forceinline__ uint32_t narrow(Pair p, int dt) {
    const float2 f = split(p);
    return pack2(f.x, f.y, dt);
}

// Whether a window lies in its row as a whole: EDGE instances have first and
// last windows that do not.
template <bool EDGE, int W>
__device__ __forceinline__ bool whole(int c, int D) {
    return !EDGE || (c >= 0 && c + W <= D);
}

// One window of a row into this thread's own slots (a 16-byte slot; two,
// `pitch` bytes apart, for eight fp32): what a thread copies it alone reads, so
// that the ring needs no barriers.  src: the window's first element; c: its
// column, negative in a first window that starts in the row before; left: the
// matrix's elements from the window's first on.  A partial window is copied
// whole while it lies inside the matrix (the values outside the row are masked
// later); a window that reaches behind the matrix's last element goes element
// by element.
template <bool EDGE, int W>
__device__ __forceinline__ void fetch(uint8_t* slot, int pitch, const uint8_t* src, int c, int D, int dt, int64_t left) {
    if constexpr (EDGE) {
        if (left < W) {
#pragma unroll 1
            for (int j = 0; j < W; ++j) {
                if (c + j < 0 || c + j >= D) continue;
                if (dt == ELEM_F32)
                    reinterpret_cast<uint32_t*>(slot + (j >> 2) * pitch)[j & 3] = reinterpret_cast<const uint32_t*>(src)[j];
                else
                    reinterpret_cast<uint16_t*>(slot)[j] = reinterpret_cast<const uint16_t*>(src)[j];
            }
            return;
        }
    }
    const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(slot));
    if (W == 4 && dt != ELEM_F32) cp_async8(dst, src);
    else cp_async16(dst, src);
    if (W == 8 && dt == ELEM_F32) cp_async16(dst + pitch, src + 16);
}

// A window's words as they were copied (b: of eight fp32 only).
struct Words {
    uint4 a, b;
};
template <int W>
__device__ __forceinline__ Words words(const uint8_t* slot, int pitch, int dt) {
    Words w;
    if (W == 4 && dt != ELEM_F32) {
        const uint2 a = *reinterpret_cast<const uint2*>(slot);
        w.a = make_uint4(a.x, a.y, 0, 0);
        return w;
    }
    w.a = *reinterpret_cast<const uint4*>(slot);
    if (W == 8 && dt == ELEM_F32) w.b = *reinterpret_cast<const uint4*>(slot + pitch);
    return w;
}

// The window's values, zero outside the row.
template <bool EDGE, int W>
__device__ __forceinline__ void unpack(const Words& w, int dt, int c, int D, Pair (&v)[W / 2]) {
    const uint4& a = w.a;
    if (dt == ELEM_F32) {
        v[0] = pair(__uint_as_float(a.x), __uint_as_float(a.y));
        v[1] = pair(__uint_as_float(a.z), __uint_as_float(a.w));
        if constexpr (W == 8) {
            const uint4& b = w.b;
            v[2] = pair(__uint_as_float(b.x), __uint_as_float(b.y));
            v[3] = pair(__uint_as_float(b.z), __uint_as_float(b.w));
        }
    } else {
        v[0] = widen(a.x, dt);
        v[1] = widen(a.y, dt);
        if constexpr (W == 8) {
            v[2] = widen(a.z, dt);
            v[3] = widen(a.w, dt);
        }
    }
    if (!whole<EDGE, W>(c, D)) {
#pragma unroll
        for (int j = 0; j < W / 2; ++j) {
            const float2 f = split(v[j]);
            const int e = c + 2 * j;
            v[j] = pair(e >= 0 && e < D ? f.x : 0.0f, e + 1 >= 0 && e + 1 < D ? f.y : 0.0f);
        }
    }
}

template <bool EDGE, int W>
__device__ __forceinline__ void unpack(const uint8_t* slot, int pitch, int dt, int c, int D, Pair (&v)[W / 2]) {
    unpack<EDGE, W>(words<W>(slot, pitch, dt), dt, c, D, v);
}

// Store a window, and (BACK) leave in v the values as stored.
template <bool EDGE, int W, bool BACK>
__device__ __forceinline__ void put(uint8_t* dst, int c, int D, int dt, Pair (&v)[W / 2]) {
    const bool all = EDGE ? whole<EDGE, W>(c, D) : c < D;
    if (dt == ELEM_F32) {
        if (all) {
#pragma unroll
            for (int j = 0; j < W / 4; ++j) {
                const float2 p = split(v[2 * j]), q = split(v[2 * j + 1]);
                reinterpret_cast<float4*>(dst)[j] = make_float4(p.x, p.y, q.x, q.y);
            }
        }
        if constexpr (EDGE) {
            if (all) return;
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
                const float2 f = split(v[j]);
                const int e = c + 2 * j;
                if (e >= 0 && e < D) reinterpret_cast<float*>(dst)[2 * j] = f.x;
                if (e + 1 >= 0 && e + 1 < D) reinterpret_cast<float*>(dst)[2 * j + 1] = f.y;
            }
        }
        return;
    }
    uint32_t w[W / 2];
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
        w[j] = narrow(v[j], dt);
        if (BACK) v[j] = widen(w[j], dt);
    }
    if (all) {
        if constexpr (W == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    }
    if constexpr (EDGE) {
        if (all) return;
#pragma unroll
        for (int j = 0; j < W / 2; ++j) {
            const int e = c + 2 * j;
            if (e >= 0 && e < D) reinterpret_cast<uint16_t*>(dst)[2 * j] = static_cast<uint16_t>(w[j] & 0xFFFFu);
            if (e + 1 >= 0 && e + 1 < D) reinterpret_cast<uint16_t*>(dst)[2 * j + 1] = static_cast<uint16_t>(w[j] >> 16);
        }
    }
}

// A thread behind the row's last window computes like the others, on zeros,
// and stores nothing (a test and two branches less in every step of a row):
// EDGE instances mask what it reads, the others clear its slots once.
template <int NV, bool EDGE>
__device__ __forceinline__ void clear_behind(uint8_t* mine, int pitch, int stages, int slots, int c0, int step, int D) {
    if constexpr (!EDGE) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (c0 + i * step >= D)
                for (int k = 0; k < stages; ++k)
                    for (int j = 0; j < slots; ++j)
                        *reinterpret_cast<uint4*>(mine + ((k * NV + i) * slots + j) * pitch) = make_uint4(0, 0, 0, 0);
    }
}

// A column block's weights in shared memory, as fp32: W / 4 16-byte slots
// `pitch` bytes apart.
template <int W>
__device__ __forceinline__ void keep(uint8_t* slot, int pitch, const float (&v)[W]) {
#pragma unroll
    for (int j = 0; j < W / 4; ++j)
        *reinterpret_cast<float4*>(slot + j * pitch) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
template <int W>
__device__ __forceinline__ void kept(const uint8_t* slot, int pitch, Pair (&v)[W / 2]) {
#pragma unroll
    for (int j = 0; j < W / 4; ++j) {
        const float4 a = *reinterpret_cast<const float4*>(slot + j * pitch);
        v[2 * j] = pair(a.x, a.y);
        v[2 * j + 1] = pair(a.z, a.w);
    }
}

// Columns c .. c + W - 1 of a weight vector (1 outside the row, or without one).
// The loads are in flight together: one at a time they cost a launch of
// few rows more than its rows.
template <int W>
__device__ __forceinline__ void load_columns(float (&v)[W], const void* w, int c, int D, int dt) {
    const uint8_t* at = static_cast<const uint8_t*>(w) + static_cast<int64_t>(c) * elem_bytes(dt);
    const bool words = c >= 0 && c + W <= D && reinterpret_cast<uintptr_t>(at) % (W * elem_bytes(dt) < 16 ? 8 : 16) == 0;
    if (!w) {
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = 1.0f;
    } else if (words && dt == ELEM_F32) {
        float4 q[W / 4];
#pragma unroll
        for (int j = 0; j < W / 4; ++j) q[j] = __ldg(reinterpret_cast<const float4*>(at) + j);
#pragma unroll
        for (int j = 0; j < W / 4; ++j) v[4 * j] = q[j].x, v[4 * j + 1] = q[j].y, v[4 * j + 2] = q[j].z, v[4 * j + 3] = q[j].w;
    } else if (words) {
        uint2 q[W / 4];
#pragma unroll
        for (int j = 0; j < W / 4; ++j) q[j] = __ldg(reinterpret_cast<const uint2*>(at) + j);
#pragma unroll
        for (int j = 0; j < W / 4; ++j) {
            const float2 lo = split(widen(q[j].x, dt)), hi = split(widen(q[j].y, dt));
            v[4 * j] = lo.x, v[4 * j + 1] = lo.y, v[4 * j + 2] = hi.x, v[4 * j + 3] = hi.y;
        }
    } else if (dt == ELEM_F32) {
        const float* p = static_cast<const float*>(w);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = (c + j >= 0 && c + j < D) ? __ldg(p + c + j) : 1.0f;
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(w);
        uint16_t u[W];
#pragma unroll
        for (int j = 0; j < W; ++j)
            u[j] = (c + j >= 0 && c + j < D) ? __ldg(p + c + j)
                                             : static_cast<uint16_t>(dt == ELEM_BF16 ? 0x3F80 : 0x3C00);
#pragma unroll
        for (int j = 0; j < W; ++j)
            v[j] = dt == ELEM_BF16 ? __uint_as_float(static_cast<uint32_t>(u[j]) << 16) : __half2float(__ushort_as_half(u[j]));
    }
}

// The block's weights: NV windows of w_post times a channel gate, then of
// w_pre, 2 W / 4 slots each.
template <int NV, int W, typename Args>
__device__ __forceinline__ void keep_weights(uint8_t* slots, int pitch, const Args& a, int c0, int step) {
    const void* gate = a.gate_kind == NORM_GATE_CHANNEL ? a.gate : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float w[W], f[W], n[W];
        load_columns<W>(w, a.w_post, c0 + i * step, a.D, a.dt_w);
        load_columns<W>(f, gate, c0 + i * step, a.D, a.dt_w);
        load_columns<W>(n, a.w_pre, c0 + i * step, a.D, a.dt_w);
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] *= f[j];
        keep<W>(slots + i * (W / 2) * pitch, pitch, w);
        keep<W>(slots + (i * (W / 2) + W / 4) * pitch, pitch, n);
    }
}

// Sums of N values over a group's threads in a fixed order (butterflies in the
// warps, then over the warps' sums).  `buf` alternates between calls, so that
// one barrier a call is enough; a group of one warp needs none.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], const Rows& g, float (*red)[N][kNormMaxWarps], int& buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (g.tpr == 32) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = g.tpr >> 5, warp0 = g.group * warps;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[buf][i][warp] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + g.group), "r"(g.tpr) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane < warps ? red[buf][i][warp0 + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    buf ^= 1;
}

// Split rows: a warp's value goes to every block of the cluster by a store that
// counts on the receiver's mbarrier.  (A cluster barrier's release also waits
// for the thread's stores to memory, a microsecond a row.)  A buffer and its
// mbarrier are used in every other turn: a block sends for turn n + 2 once it
// has every warp's values of turn n + 1, which they send after they have read
// those of turn n.  Nothing a user can do makes a wait run out; if one does,
// the sums become NaN.
struct Exchange {
    uint64_t bar[2];
    int lost;
};
__device__ __forceinline__ void exchange_start(Exchange* x) {
    if (threadIdx.x == 0) {
        mbar_init(&x->bar[0], 1);
        mbar_init(&x->bar[1], 1);
        x->lost = 0;
        fence_mbar_init();
    }
    __syncthreads();
    cluster_sync_all();
}
__device__ __forceinline__ void send_all(const float* here, Exchange* x, int turn, const Rows& g, float v) {
    const uint32_t at = smem_u32(here), bar = smem_u32(&x->bar[turn & 1]);
    for (int r = 0; r < g.parts; ++r) st_async_f32(mapa_shared(at, r), v, mapa_shared(bar, r));
}
// Values of this turn that a block gets: one of each of `count` a warp.
__device__ __forceinline__ bool receive_all(Exchange* x, int turn, const Rows& g, int count) {
    if (threadIdx.x == 0)
        mbar_arrive_expect_tx(&x->bar[turn & 1], static_cast<uint32_t>(g.parts * (g.tpr >> 5) * count * 4));
    return mbar_wait(&x->bar[turn & 1], (turn >> 1) & 1, &x->lost, nullptr, 0);
}
__device__ __forceinline__ float cluster_sum(float v, const Rows& g, float (*red)[kNormMaxSplit * kNormMaxWarps], Exchange* x,
                                             int& turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int lane = threadIdx.x & 31, warps = g.tpr >> 5;
    if (lane == 0) send_all(&red[turn & 1][g.part * warps + (threadIdx.x >> 5)], x, turn, g, v);
    __syncwarp();
    v = receive_all(x, turn, g, 1) ? 0.0f : __uint_as_float(0x7FC00000u);
    for (int w = lane; w < g.parts * warps; w += 32) v += red[turn & 1][w];
    __syncwarp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    ++turn;
    return v;
}

__device__ __forceinline__ float token_gate(const void* gate, int64_t t, int dt) {
    float g[1];
    raw_to_f32(load_raw<1>(gate, t, dt), dt, g);
    return g[0];
}

// Slots a thread has for one window of type dt (none: no such matrix).
__host__ __device__ __forceinline__ int window_slots(bool there, int dt, int window) {
    return there ? (dt == ELEM_F32 ? window / 4 : 1) : 0;
}

// This thread's first window of the next row of a matrix that goes by.
__device__ __forceinline__ uint8_t* run(const void* base, int64_t ld, int dt, const Rows& g, int c0) {
    return static_cast<uint8_t*>(const_cast<void*>(base)) + (g.first * ld + c0) * elem_bytes(dt);
}
// Bytes from a group's row to its next one, in each matrix (kernel arguments,
// so that they take no registers).
struct Steps {
    int64_t x, y, h, u, dh, du, dx, dy;
};

// ------------------------------------------------------------------ rows element by element
// For matrices whose rows do not lie alike in their windows (bases off 16
// bytes, strides that differ modulo 8).
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*red)[N][kNormMaxWarps], int& buf) {
    Rows g;
    g.tpr = blockDim.x;
    g.group = 0;
    group_sums<N>(v, g, red, buf);
}

// ------------------------------------------------------------------ launches
inline cudaError_t sm_count(int* sms) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    return err;
}

// Collects whether a launch's matrices lie alike in their windows.
struct Alike {
    int window;
    bool ok = true;
    int64_t ld = -1;
    bool odd = false;           // rows start at different places in their windows
    explicit Alike(int w) : window(w) {}
    void add(const void* p, int64_t l) {
        if (!p) return;
        if (reinterpret_cast<uintptr_t>(p) % 16) ok = false;
        if (ld >= 0 && ((ld ^ l) & (window - 1))) ok = false;
        ld = l;
        odd = odd || (l & (window - 1));
    }
};

// How a launch covers T rows of D elements: a group of tpr threads owns a row,
// nv windows a thread; the ring takes the shared memory that is left, up to
// eight rows a group.
struct Shape {
    int nv, tpr, threads, stages, grid, split;
    bool edge;                  // some windows lie only partly in their row
    size_t smem;
};
constexpr int kNormStatic = 2304;                // the sums' static part at most
constexpr int kNormSmem = kSmemLimit - kNormStatic;

// Dynamic shared memory of each of `blocks` blocks on one SM (1 KB a block is
// the system's).
constexpr int room_of(int blocks) {
    return blocks == 1 ? kNormSmem : (kSmemLimit + 1024) / blocks - 1024 - kNormStatic;
}

// What a kernel allows: rows of more than two_from windows have two a thread;
// group_threads: threads of a block's groups together at most, row_threads of
// one, part_threads of a block of a split row; regs: of a thread; deep: rows of a group in the ring, where there is
// room, rows_used: in use at once; split: blocks that share a row at most; slots_for: slots of a window
// that have to fit, if there are as many or not (0: as there are).
struct Rule {
    int two_from, group_threads, row_threads, part_threads, regs, deep, rows_used, split, slots_for;
};

// slots: of a window in the ring; most: blocks (clusters).
inline bool shape_of(int64_t T, int D, const Alike& al, int slots, const Rule& rule, int sms, int64_t most, int split, Shape* s) {
    const int W = al.window;
    const int row = (D + (al.odd ? W - 1 : 0) + W - 1) / W, windows = (row + split - 1) / split;
    if (windows > 2 * (split > 1 ? rule.part_threads : rule.row_threads)) return false;
    // the order of a row's sums does not depend on which matrices there are
    if (rule.slots_for && (rule.slots_for * 16 + W / 2 * 16) * 2 * ((windows + 63) / 64 * 32) > kNormSmem) return false;
    s->split = split;
    s->edge = al.odd || D % W;
    s->nv = split > 1 || windows > rule.two_from ? 2 : 1;
    s->tpr = ((windows + s->nv - 1) / s->nv + 31) / 32 * 32;
    const int stage = s->nv * slots * 16, fixed = s->nv * (W / 2) * s->tpr * 16;      // bytes a thread; a block
    int groups = split > 1 ? 1 : std::max(1, std::min(rule.group_threads / s->tpr, 8));
    while (groups > 1 && (static_cast<int64_t>(groups) * sms > T || rule.deep * groups * s->tpr * stage + fixed > kNormSmem)) --groups;
    s->threads = s->tpr * groups;
    int per_sm = std::max(1, std::min(65536 / (rule.regs * s->threads), 2048 / s->threads));
    // at least `deep` rows in the ring of a group
    while (per_sm > 1 && rule.deep * stage * s->threads + fixed > room_of(per_sm)) --per_sm;
    // clusters of four: the SMs of a GPC are not all multiples of four (with 38
    // clusters for 152 SMs two waited for the others: twice the time)
    const int units = sms * per_sm / split - (split > 2 ? 2 : 0);
    int64_t grid = std::min<int64_t>((T + groups - 1) / groups, std::max(1, units));
    if (grid > most) grid = most;
    // a row's place in its windows has to be the same in all rows of a block
    if (al.odd && (groups > 1 || grid < T)) {
        if (grid < 8) return false;
        grid = grid / 8 * 8;
    }
    s->grid = static_cast<int>(grid);
    const int per_block = std::min<int>(per_sm, static_cast<int>((grid * split + sms - 1) / sms));
    const int64_t rows = (T + grid * groups - 1) / (grid * groups);                        // of a group at most
    int st = (room_of(per_block) - fixed) / (stage * s->threads);
    st = std::max(1, std::min<int>(st, kNormMaxStages));
    s->stages = static_cast<int>(std::min<int64_t>(st, rows));
    if (s->stages < std::min<int64_t>(rule.rows_used, rows)) return false;
    s->smem = static_cast<size_t>(s->stages) * stage * s->threads + fixed;
    return s->smem <= static_cast<size_t>(kNormSmem);
}

// The fewest blocks a row that its windows and the ring's rows fit in.
inline bool shape_of(int64_t T, int D, const Alike& al, int slots, const Rule& rule, int sms, int64_t most, Shape* s) {
    if (!al.ok) return false;
    for (int split = 1; split <= rule.split; split *= 2)
        if (shape_of(T, D, al, slots, rule, sms, most, split, s)) return true;
    return false;
}

inline Steps steps_of(const NormArgs& a, int64_t rows) {
    Steps s = {};
    s.x = rows * a.ld_x * elem_bytes(a.dt_x);
    s.y = rows * a.ld_y * elem_bytes(a.dt_y);
    s.h = rows * a.ld_h * elem_bytes(a.dt_x);
    s.u = rows * a.ld_u * elem_bytes(a.dt_u);
    return s;
}
inline Steps steps_of(const NormBackArgs& a, int64_t rows) {
    Steps s = {};
    s.h = rows * a.ld_h * elem_bytes(a.dt_x);
    s.du = rows * a.ld_du * elem_bytes(a.dt_u);
    s.dh = rows * a.ld_dh * elem_bytes(a.dt_x);
    s.y = rows * a.ld_y * elem_bytes(a.dt_y);
    s.dx = rows * a.ld_dx * elem_bytes(a.dt_x);
    s.dy = rows * a.ld_dy * elem_bytes(a.dt_y);
    return s;
}

template <typename Args>
cudaError_t run_rows(void (*kern)(Args, int, int, Steps), const Args& a, const Shape& sh, size_t smem, cudaStream_t s) {
    if (smem > 40 * 1024) {         // with the static part, up to 48 KB need no attribute
        const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem);
        if (err != cudaSuccess) return err;
    }
    const int64_t rows = static_cast<int64_t>(sh.grid) * (sh.threads / sh.tpr);
    if (sh.split > 1)
        return launch_ex_cluster(kern, dim3(sh.grid * sh.split), dim3(sh.threads), smem, s, false, sh.split, a, sh.tpr,
                                 sh.stages, steps_of(a, rows));
    kern<<<sh.grid, sh.threads, smem, s>>>(a, sh.tpr, sh.stages, steps_of(a, rows));
    return cudaGetLastError();
}

}  // namespace moe
