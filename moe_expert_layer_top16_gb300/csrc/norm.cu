// The norms behind and before a block, with the block's gate and the residual
// scale, in one pass over the rows; and its gradients.
//
//   rms(v)  = sqrt(mean(v^2) + eps)
//   h       = r x + g w_post y / rms(y)       r: residual scale, g: gate of the
//                                              channel, of the token, or none
//   u       = w_pre h / rms(h)                 of h as it is stored
//
// With no y only the second line is computed (h = x), with no u only the
// first.  Backward, from dh (gradient of h as the residual stream), du:
//   a = du w_pre,  total = dh + (a - h^ mean(a h^)) / rms(h),  h^ = h / rms(h)
//   dx = r total,  p = total g w_post,  dy = (p - y^ mean(p y^)) / rms(y)
//   dw_pre = sum_t du h^,  dw_post = sum_t total g y^,
//   dg = sum total w_post y^  over t (channel) or over the row (token)
//
// Bound by HBM: every row of every matrix goes by once.  A row's windows wait
// in shared memory (a ring that cp.async fills some rows ahead), so that the
// sums over the row (of y^2, then of h^2) need no second read.  All sums are
// fp32.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace moe {

namespace {

constexpr int kNormMaxWarps = 32;
constexpr int kNormMaxStages = 8;

// ------------------------------------------------------------------ rows by windows
// A row is cut at the windows of its matrix (8 elements: 16 bytes of a 16-bit
// type; 4 where every matrix is fp32), not at its own start: for rows of any
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
// RUN have both norms and every matrix of them.
enum NormKind : int { NORM_RUN = 0, NORM_BF16 = 1, NORM_BF16_Y32 = 2, NORM_F32 = 3 };
template <int KIND>
struct Kind {
    static constexpr int window = KIND == NORM_F32 ? 4 : 8;
    static constexpr bool full = KIND != NORM_RUN;
    static constexpr int x = KIND == NORM_RUN ? -1 : (KIND == NORM_F32 ? ELEM_F32 : ELEM_BF16);
    static constexpr int y = KIND == NORM_RUN ? -1 : (KIND == NORM_BF16 ? ELEM_BF16 : ELEM_F32);
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
    cp_async16(dst, src);
    if (W == 8 && dt == ELEM_F32) cp_async16(dst + pitch, src + 16);
}

// A window's words as they were copied (b: of eight fp32 only).
struct Words {
    uint4 a, b;
};
template <int W>
__device__ __forceinline__ Words words(const uint8_t* slot, int pitch, int dt) {
    Words w;
    w.a = *reinterpret_cast<const uint4*>(slot);
    if (W == 8 && dt == ELEM_F32) w.b = *reinterpret_cast<const uint4*>(slot + pitch);
    return w;
}

// The window's values, zero outside the row.
template <bool EDGE, int W>
__device__ __forceinline__ void unpack(const Words& w, int dt, int c, int D, Pair (&v)[W / 2]) {
    const uint4& a = w.a;
    if (W == 4 || dt == ELEM_F32) {
        v[0] = pair(__uint_as_float(a.x), __uint_as_float(a.y));
        v[1] = pair(__uint_as_float(a.z), __uint_as_float(a.w));
        if constexpr (W == 8) {
            const uint4& b = w.b;
            v[2] = pair(__uint_as_float(b.x), __uint_as_float(b.y));
            v[3] = pair(__uint_as_float(b.z), __uint_as_float(b.w));
        }
    } else if constexpr (W == 8) {
        v[0] = widen(a.x, dt);
        v[1] = widen(a.y, dt);
        v[2] = widen(a.z, dt);
        v[3] = widen(a.w, dt);
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
    if (!w) {
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = 1.0f;
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

// Four sums at once: the lanes halve what they carry with each exchange (two
// values after the first, one after the second), so that six exchanges do what
// twenty would; lane 8 k then holds value k of the warp.
// `between` is done before the barrier: what the threads that arrive first do
// while they would wait.  Split rows: each warp's sums go to every block of the
// cluster, whose barrier takes the place of the group's (a block writes a
// buffer again one barrier after the others have read it).
template <bool SPLIT, int WARPS, typename F>
__device__ __forceinline__ void group_sums4(float (&v)[4], const Rows& g, float (*red)[4][WARPS], int& buf, F between) {
    const int lane = threadIdx.x & 31;
    const bool up = lane & 16, odd = lane & 8;
    // lanes 0-15 keep values 0 and 1, lanes 16-31 values 2 and 3
    const float a = __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16) + (up ? v[2] : v[0]);
    const float b = __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16) + (up ? v[3] : v[1]);
    float s = __shfl_xor_sync(0xffffffffu, odd ? a : b, 8) + (odd ? b : a);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (SPLIT || g.tpr > 32) {
        const int warp = threadIdx.x >> 5, warps = (g.tpr >> 5) * g.parts, warp0 = g.group * warps;
        if constexpr (SPLIT) {
            if ((lane & 7) == 0) {
                const uint32_t at = smem_u32(&red[buf][lane >> 3][g.part * (g.tpr >> 5) + warp]);
                for (int r = 0; r < g.parts; ++r)
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(at, r)), "f"(s) : "memory");
            }
            between();
            __syncwarp();
            cluster_sync_all();
        } else {
            if ((lane & 7) == 0) red[buf][lane >> 3][warp] = s;
            between();
            asm volatile("bar.sync %0, %1;" ::"r"(1 + g.group), "r"(g.tpr) : "memory");
        }
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; w += 8)
            if (w + (lane & 7) < warps) s += red[buf][lane >> 3][warp0 + w + (lane & 7)];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        buf ^= 1;
    } else {
        between();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, s, 8 * i);
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

// Forward.  A group keeps `stages` rows in flight by cp.async.
template <int NV, bool EDGE, int KIND>
__global__ void __launch_bounds__(1024) block_norm_kernel(const NormArgs a, int tpr, int stages, const Steps st) {
    using K = Kind<KIND>;
    constexpr int W = K::window;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][1][kNormMaxWarps];
    int buf = 0;
    const int dx = K::x >= 0 ? K::x : a.dt_x, dy = K::y >= 0 ? K::y : a.dt_y;
    const int du = KIND == NORM_BF16 || KIND == NORM_BF16_Y32 ? K::x : a.dt_u;
    const bool post = a.y != nullptr, pre = a.u != nullptr;
    const Rows g = rows_of<false>(tpr, a.ld_x, W);
    const int D = a.D, T = static_cast<int>(a.T);
    const int pitch = blockDim.x * 16, wpitch = tpr * 16;
    const int yw = window_slots(post, dy, W), slots = yw + window_slots(true, dx, W);
    uint8_t* weights = ring + g.lane_in_group * 16;
    uint8_t* mine = ring + NV * (W / 2) * wpitch + threadIdx.x * 16;        // [stages][NV][slots]
    const int c0 = g.lane_in_group * W - g.shift, step = tpr * W;
    const int stage_pitch = NV * slots * pitch;
    uint8_t *rx = run(a.x, a.ld_x, dx, g, c0), *ry = run(a.y, a.ld_y, dy, g, c0);
    uint8_t *rh = run(a.h, a.ld_h, dx, g, c0), *ru = run(a.u, a.ld_u, du, g, c0);
    int ahead = 0;                        // stage that the next row goes to
    auto issue = [&](int t) {
        if (t < T) {
            uint8_t* s = mine + ahead * stage_pitch;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * step;
                if (c >= D) break;
                uint8_t* p = s + i * slots * pitch;
                // only the last rows have windows that reach behind the matrix
                const int64_t rows_left = (EDGE && t + W >= T) ? T - 1 - t : W;
                if (post) fetch<EDGE, W>(p, pitch, ry + i * step * elem_bytes(dy), c, D, dy, rows_left * a.ld_y + D - c);
                fetch<EDGE, W>(p + yw * pitch, pitch, rx + i * step * elem_bytes(dx), c, D, dx, rows_left * a.ld_x + D - c);
            }
            ry += st.y;
            rx += st.x;
        }
        cp_async_commit();
        if (++ahead == stages) ahead = 0;
    };
    clear_behind<NV, EDGE>(mine, pitch, stages, slots, c0, step, D);
    for (int k = 0; k + 1 < stages; ++k) issue(g.first + k * g.step);
    if (g.group == 0) keep_weights<NV, W>(weights, wpitch, a, c0, step);
    __syncthreads();
    int stage = 0;
    const float inv_d = 1.0f / static_cast<float>(D);
    const Pair res = pair(a.res_scale, a.res_scale);
    for (int t = g.first; t < T; t += g.step) {
        issue(t + (stages - 1) * g.step);
        cp_async_wait(stages - 1);
        const uint8_t* s = mine + stage * stage_pitch;
        if (++stage == stages) stage = 0;
        Pair v[NV][W / 2];
        float q = 0.0f;
        if (post) {
            Pair acc = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * step;
                unpack<EDGE, W>(s + i * slots * pitch, pitch, dy, c, D, v[i]);
#pragma unroll
                for (int j = 0; j < W / 2; ++j) acc = fma2(v[i][j], v[i][j], acc);
            }
            float ss[1] = {sum2(acc)};
            group_sums<1>(ss, g, red, buf);
            q = rsqrtf(ss[0] * inv_d + a.eps);
            if (a.gate_kind == NORM_GATE_TOKEN) q *= token_gate(a.gate, t, a.dt_w);
        }
        const Pair qq = pair(q, q);
        Pair acc = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            const uint8_t* p = s + (i * slots + yw) * pitch;
            if (post) {
                Pair x[W / 2], w[W / 2];
                unpack<EDGE, W>(p, pitch, dx, c, D, x);
                kept<W>(weights + i * (W / 2) * wpitch, wpitch, w);
#pragma unroll
                for (int j = 0; j < W / 2; ++j) v[i][j] = fma2(res, x[j], mul2(mul2(qq, w[j]), v[i][j]));
                put<EDGE, W, true>(rh + i * step * elem_bytes(dx), c, D, dx, v[i]);
            } else {
                unpack<EDGE, W>(p, pitch, dx, c, D, v[i]);
            }
#pragma unroll
            for (int j = 0; j < W / 2; ++j) acc = fma2(v[i][j], v[i][j], acc);
        }
        rh += st.h;
        if (pre) {
            float ss[1] = {sum2(acc)};
            group_sums<1>(ss, g, red, buf);
            const float r = rsqrtf(ss[0] * inv_d + a.eps);
            const Pair rr = pair(r, r);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * step;
                Pair w[W / 2];
                kept<W>(weights + (i * (W / 2) + W / 4) * wpitch, wpitch, w);
#pragma unroll
                for (int j = 0; j < W / 2; ++j) v[i][j] = mul2(mul2(v[i][j], rr), w[j]);
                put<EDGE, W, false>(ru + i * step * elem_bytes(du), c, D, du, v[i]);
            }
            ru += st.u;
        }
    }
}

// Gradients, with the same ring.  The column sums of a thread's rows stay in
// registers (sum du h^ and sum total y^, times the token's gate), are added
// over the block's groups through shared memory and go to part[block][2][D].
// The weights wait in shared memory, which leaves registers for 28 warps.  The
// sums over row t + 1 that its norms need are taken together with the one over
// row t that its dy needs: one barrier a row, and the work of both before it.
template <int NV, int MAXT, bool EDGE, int KIND, bool SPLIT>
__global__ void __launch_bounds__(MAXT) block_norm_backward_kernel(const NormBackArgs a, int tpr, int stages,
                                                                   const Steps st) {
    using K = Kind<KIND>;
    constexpr int W = K::window;
    extern __shared__ __align__(16) uint8_t ring[];
    constexpr int kWarps = MAXT / 32 * (SPLIT ? kNormMaxSplit : 1);
    __shared__ float red[2][4][(kWarps + 7) / 8 * 8];
    int buf = 0;
    const int tx = K::x >= 0 ? K::x : a.dt_x, ty = K::y >= 0 ? K::y : a.dt_y, tu = K::x >= 0 ? K::x : a.dt_u;
    const bool post = K::full || a.y != nullptr, pre = K::full || a.du != nullptr, has_dh = K::full || a.dh != nullptr;
    const bool want_dx = K::full || a.dx != nullptr, want_dy = K::full || a.dy != nullptr;
    const Rows g = rows_of<SPLIT>(tpr, pre ? a.ld_h : a.ld_dh, W);
    if constexpr (SPLIT) cluster_sync_all();           // the others' shared memory is there
    const int D = a.D, T = static_cast<int>(a.T);
    const int pitch = blockDim.x * 16, wpitch = tpr * 16;
    const int off_u = window_slots(pre, tx, W), off_d = off_u + window_slots(pre, tu, W),
              off_y = off_d + window_slots(has_dh, tx, W), slots = off_y + window_slots(post, ty, W);     // a window's
    uint8_t* weights = ring + g.lane_in_group * 16;
    uint8_t* mine = ring + NV * (W / 2) * wpitch + threadIdx.x * 16;        // [stages][NV][slots]
    const int step = tpr * W, c0 = g.lane_in_group * W - g.shift + g.part * NV * step;
    const int stage_pitch = NV * slots * pitch;
    uint8_t *rh = run(a.h, a.ld_h, tx, g, c0), *ru = run(a.du, a.ld_du, tu, g, c0);
    uint8_t *rd = run(a.dh, a.ld_dh, tx, g, c0), *ry = run(a.y, a.ld_y, ty, g, c0);
    uint8_t *ox = run(a.dx, a.ld_dx, tx, g, c0), *oy = run(a.dy, a.ld_dy, ty, g, c0);
    int ahead = 0;                        // stage that the next row goes to
    auto issue = [&](int t) {
        if (t < T) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * step;
                if (c >= D) break;
                uint8_t* s = mine + ahead * stage_pitch + i * slots * pitch;
                // only the last rows have windows that reach behind the matrix
                const int64_t rows_left = (EDGE && t + W >= T) ? T - 1 - t : W;
                if (pre) {
                    fetch<EDGE, W>(s, pitch, rh + i * step * elem_bytes(tx), c, D, tx, rows_left * a.ld_h + D - c);
                    fetch<EDGE, W>(s + off_u * pitch, pitch, ru + i * step * elem_bytes(tu), c, D, tu, rows_left * a.ld_du + D - c);
                }
                if (has_dh)
                    fetch<EDGE, W>(s + off_d * pitch, pitch, rd + i * step * elem_bytes(tx), c, D, tx, rows_left * a.ld_dh + D - c);
                if (post)
                    fetch<EDGE, W>(s + off_y * pitch, pitch, ry + i * step * elem_bytes(ty), c, D, ty, rows_left * a.ld_y + D - c);
            }
            rh += st.h;
            ru += st.du;
            rd += st.dh;
            ry += st.y;
        }
        cp_async_commit();
        if (++ahead == stages) ahead = 0;
    };
    for (int k = 0; k < stages; ++k) issue(g.first + k * g.step);
    if (g.group == 0) keep_weights<NV, W>(weights, wpitch, a, c0, step);
    Pair s_pre[NV][W / 2], s_post[NV][W / 2];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W / 2; ++j) s_pre[i][j] = s_post[i][j] = 0;
    __syncthreads();
    int stage = 0;
    const float inv_d = 1.0f / static_cast<float>(D);
    // h^2, a h and y^2 of this thread's part of the row in stage `s`
    auto squares = [&](const uint8_t* s, float (&v)[4]) {
        Pair hh = 0, uh = 0, yy = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c >= D) break;
            const uint8_t* p = s + i * slots * pitch;
            if (pre) {
                Pair h[W / 2], u[W / 2], w[W / 2];
                unpack<EDGE, W>(p, pitch, tx, c, D, h);
                unpack<EDGE, W>(p + off_u * pitch, pitch, tu, c, D, u);
                kept<W>(weights + (i * (W / 2) + W / 4) * wpitch, wpitch, w);
#pragma unroll
                for (int j = 0; j < W / 2; ++j) {
                    hh = fma2(h[j], h[j], hh);
                    uh = fma2(mul2(u[j], w[j]), h[j], uh);
                }
            }
            if (post) {
                Pair y[W / 2];
                unpack<EDGE, W>(p + off_y * pitch, pitch, ty, c, D, y);
#pragma unroll
                for (int j = 0; j < W / 2; ++j) yy = fma2(y[j], y[j], yy);
            }
        }
        v[0] = sum2(hh);
        v[1] = sum2(uh);
        v[2] = sum2(yy);
    };
    float r = 0.0f, m = 0.0f, q = 0.0f;                // 1 / rms(h), mean(a h^) / rms(h), 1 / rms(y)
    auto norms = [&](const float (&v)[4]) {
        r = rsqrtf(v[0] * inv_d + a.eps);
        m = r * r * v[1] * inv_d;
        q = rsqrtf(v[2] * inv_d + a.eps);
    };
    if (g.first < T) {
        cp_async_wait(stages - 1);
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        squares(mine, v);
        group_sums4<SPLIT>(v, g, red, buf, [] {});
        norms(v);
    }
    for (int t = g.first; t < T; t += g.step) {
        const uint8_t* s = mine + stage * stage_pitch;
        if (++stage == stages) stage = 0;
        const float gt = (post && a.gate_kind == NORM_GATE_TOKEN) ? token_gate(a.gate, t, a.dt_w) : 1.0f;
        const Pair rr = pair(r, r), rm = pair(-r * m, -r * m), qg = pair(q * gt, q * gt);
        Pair total[NV][W / 2];
        Words kept_y[NV];
        Pair py = 0;                                   // sum total w_post (channel gate) y
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c >= D) break;
            const uint8_t* p = s + i * slots * pitch;
#pragma unroll
            for (int j = 0; j < W / 2; ++j) total[i][j] = 0;
            if (has_dh) unpack<EDGE, W>(p + off_d * pitch, pitch, tx, c, D, total[i]);
            if (pre) {
                Pair h[W / 2], u[W / 2], w[W / 2];
                unpack<EDGE, W>(p, pitch, tx, c, D, h);
                unpack<EDGE, W>(p + off_u * pitch, pitch, tu, c, D, u);
                kept<W>(weights + (i * (W / 2) + W / 4) * wpitch, wpitch, w);
#pragma unroll
                for (int j = 0; j < W / 2; ++j) {
                    const Pair ur = mul2(u[j], rr);
                    s_pre[i][j] = fma2(ur, h[j], s_pre[i][j]);
                    total[i][j] = fma2(h[j], rm, fma2(ur, w[j], total[i][j]));
                }
            }
            if (want_dx) {
                const float rs = post ? a.res_scale : 1.0f;
                const Pair res = pair(rs, rs);
                Pair o[W / 2];
#pragma unroll
                for (int j = 0; j < W / 2; ++j) o[j] = mul2(res, total[i][j]);
                put<EDGE, W, false>(ox + i * step * elem_bytes(tx), c, D, tx, o);
            }
            if (post) {
                Pair y[W / 2], w[W / 2];
                kept_y[i] = words<W>(p + off_y * pitch, pitch, ty);
                unpack<EDGE, W>(kept_y[i], ty, c, D, y);
                kept<W>(weights + i * (W / 2) * wpitch, wpitch, w);
#pragma unroll
                for (int j = 0; j < W / 2; ++j) {
                    s_post[i][j] = fma2(total[i][j], mul2(y[j], qg), s_post[i][j]);
                    total[i][j] = mul2(total[i][j], w[j]);
                    py = fma2(total[i][j], y[j], py);
                }
            }
        }
        ox += st.dx;
        float v[4] = {0.0f, 0.0f, 0.0f, sum2(py)};
        const bool more = t + g.step < T;
        if (more) {
            // the next row has landed: later ones may be in flight
            cp_async_wait(stages - 2);
            squares(mine + stage * stage_pitch, v);
        }
        // this thread is through with row t's slots
        group_sums4<SPLIT>(v, g, red, buf, [&] { issue(t + stages * g.step); });
        if (post) {
            if (a.d_gate_token && g.lane_in_group == 0 && g.part == 0) a.d_gate_token[t] = v[3] * q;
            if (want_dy) {
                const float n = -q * q * v[3] * inv_d;     // -mean(p y^) / (g rms(y))
                const Pair nn = pair(n, n);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = c0 + i * step;
                    if (c >= D) break;
                    Pair y[W / 2];
                    unpack<EDGE, W>(kept_y[i], ty, c, D, y);
#pragma unroll
                    for (int j = 0; j < W / 2; ++j) y[j] = mul2(qg, fma2(y[j], nn, total[i][j]));
                    put<EDGE, W, false>(oy + i * step * elem_bytes(ty), c, D, ty, y);
                }
            }
        }
        oy += st.dy;
        norms(v);
    }
    if (!a.part) return;
    float* out = a.part + static_cast<int64_t>(g.unit) * 2 * D;
    // the groups in turn add their columns to the block's, in the ring's
    // memory (one group: straight to the part)
    float* acc = g.groups == 1 ? out : reinterpret_cast<float*>(ring);
    cp_async_wait(0);
    __syncthreads();
    for (int k = 0; k < g.groups; ++k) {
        if (g.group == k) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < W / 2; ++j) {
                    const int c = c0 + i * step + 2 * j;
                    const float2 f = split(s_pre[i][j]), e = split(s_post[i][j]);
                    if (c >= 0 && c < D) {
                        acc[c] = (k ? acc[c] : 0.0f) + f.x;
                        acc[D + c] = (k ? acc[D + c] : 0.0f) + e.x;
                    }
                    if (c + 1 >= 0 && c + 1 < D) {
                        acc[c + 1] = (k ? acc[c + 1] : 0.0f) + f.y;
                        acc[D + c + 1] = (k ? acc[D + c + 1] : 0.0f) + e.y;
                    }
                }
        }
        __syncthreads();
    }
    if (g.groups > 1)
        for (int c = threadIdx.x; c < 2 * D; c += blockDim.x) out[c] = acc[c];
}

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

__global__ void __launch_bounds__(1024) block_norm_plain_kernel(const NormArgs a) {
    __shared__ float red[2][1][kNormMaxWarps];
    int buf = 0;
    const bool post = a.y != nullptr, pre = a.u != nullptr;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    auto at = [](const void* p, int64_t i, int dt) {
        float f[1];
        raw_to_f32(load_raw<1>(p, i, dt), dt, f);
        return f[0];
    };
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        float q = 0.0f;
        if (post) {
            float ss[1] = {0.0f};
            for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
                const float y = at(a.y, t * a.ld_y + c, a.dt_y);
                ss[0] = fmaf(y, y, ss[0]);
            }
            block_sums<1>(ss, red, buf);
            q = rsqrtf(ss[0] * inv_d + a.eps);
            if (a.gate_kind == NORM_GATE_TOKEN) q *= token_gate(a.gate, t, a.dt_w);
        }
        // h as it is stored: computed once, then read back by the same thread
        float ss[1] = {0.0f};
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
            float h[1] = {at(a.x, t * a.ld_x + c, a.dt_x)};
            if (post) {
                float w = a.w_post ? at(a.w_post, c, a.dt_w) : 1.0f;
                if (a.gate_kind == NORM_GATE_CHANNEL) w *= at(a.gate, c, a.dt_w);
                h[0] = fmaf(a.res_scale, h[0], q * w * at(a.y, t * a.ld_y + c, a.dt_y));
                store_vec(a.h, t * a.ld_h + c, a.dt_x, h);
                h[0] = round_to(h[0], a.dt_x);
            }
            ss[0] = fmaf(h[0], h[0], ss[0]);
        }
        if (!pre) continue;
        block_sums<1>(ss, red, buf);
        const float r = rsqrtf(ss[0] * inv_d + a.eps);
        const void* hp = post ? a.h : a.x;
        const int64_t ld = post ? a.ld_h : a.ld_x;
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
            const float o[1] = {at(hp, t * ld + c, a.dt_x) * r * (a.w_pre ? at(a.w_pre, c, a.dt_w) : 1.0f)};
            store_vec(a.u, t * a.ld_u + c, a.dt_u, o);
        }
    }
}

constexpr int kPlainColumns = 16;       // columns a thread: widths up to 16 * 1024

__global__ void __launch_bounds__(1024) block_norm_backward_plain_kernel(const NormBackArgs a) {
    __shared__ float red[2][3][kNormMaxWarps];
    __shared__ float red1[2][1][kNormMaxWarps];
    int buf = 0, buf1 = 0;
    const bool post = a.y != nullptr, pre = a.du != nullptr;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    auto at = [](const void* p, int64_t i, int dt) {
        float f[1];
        raw_to_f32(load_raw<1>(p, i, dt), dt, f);
        return f[0];
    };
    float s_pre[kPlainColumns], s_post[kPlainColumns];
#pragma unroll
    for (int i = 0; i < kPlainColumns; ++i) s_pre[i] = s_post[i] = 0.0f;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        float sums[3] = {0.0f, 0.0f, 0.0f};
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
            if (pre) {
                const float h = at(a.h, t * a.ld_h + c, a.dt_x);
                const float u = at(a.du, t * a.ld_du + c, a.dt_u) * (a.w_pre ? at(a.w_pre, c, a.dt_w) : 1.0f);
                sums[0] = fmaf(h, h, sums[0]);
                sums[1] = fmaf(u, h, sums[1]);
            }
            if (post) {
                const float y = at(a.y, t * a.ld_y + c, a.dt_y);
                sums[2] = fmaf(y, y, sums[2]);
            }
        }
        block_sums<3>(sums, red, buf);
        const float r = rsqrtf(sums[0] * inv_d + a.eps);
        const float m = r * r * sums[1] * inv_d;
        const float q = rsqrtf(sums[2] * inv_d + a.eps);
        const float gt = (post && a.gate_kind == NORM_GATE_TOKEN) ? token_gate(a.gate, t, a.dt_w) : 1.0f;
        float total[kPlainColumns], yv[kPlainColumns];
        float d[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kPlainColumns; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= a.D) break;
            total[i] = a.dh ? at(a.dh, t * a.ld_dh + c, a.dt_x) : 0.0f;
            if (pre) {
                const float h = at(a.h, t * a.ld_h + c, a.dt_x);
                const float u = at(a.du, t * a.ld_du + c, a.dt_u);
                s_pre[i] = fmaf(u, h * r, s_pre[i]);
                total[i] += r * (u * (a.w_pre ? at(a.w_pre, c, a.dt_w) : 1.0f) - h * m);
            }
            if (post) {
                yv[i] = at(a.y, t * a.ld_y + c, a.dt_y);
                s_post[i] = fmaf(total[i] * gt, yv[i] * q, s_post[i]);
            }
            if (a.dx) {
                const float o[1] = {post ? a.res_scale * total[i] : total[i]};
                store_vec(a.dx, t * a.ld_dx + c, a.dt_x, o);
            }
            if (post) {
                float w = a.w_post ? at(a.w_post, c, a.dt_w) : 1.0f;
                if (a.gate_kind == NORM_GATE_CHANNEL) w *= at(a.gate, c, a.dt_w);
                total[i] *= w;
                d[0] = fmaf(total[i], yv[i], d[0]);
            }
        }
        if (!post) continue;
        block_sums<1>(d, red1, buf1);
        if (a.d_gate_token && threadIdx.x == 0) a.d_gate_token[t] = d[0] * q;
        if (a.dy) {
            const float n = q * q * d[0] * inv_d, f = q * gt;
#pragma unroll
            for (int i = 0; i < kPlainColumns; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c >= a.D) break;
                const float o[1] = {f * (total[i] - yv[i] * n)};
                store_vec(a.dy, t * a.ld_dy + c, a.dt_y, o);
            }
        }
    }
    if (a.part) {
        float* out = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.D;
#pragma unroll
        for (int i = 0; i < kPlainColumns; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= a.D) break;
            out[c] = s_pre[i];
            out[a.D + c] = s_post[i];
        }
    }
}

// Column sums of the CTAs' parts, in a fixed order, and the weights' and the
// channel gate's gradients from them.
constexpr int kColGroups = 16;
__global__ void __launch_bounds__(32 * kColGroups) norm_columns_kernel(const NormBackArgs a, int parts) {
    __shared__ float red[kColGroups][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const int which = blockIdx.y;                 // 0: sum du h^, 1: sum total g y^
    float s = 0.0f;
    if (c < a.D)
        for (int p = g; p < parts; p += kColGroups) s += a.part[(static_cast<int64_t>(p) * 2 + which) * a.D + c];
    red[g][lane] = s;
    __syncthreads();
    if (g != 0 || c >= a.D) return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kColGroups; ++i) s += red[i][lane];
    if (which == 0) {
        if (a.dw_pre) a.dw_pre[c] = s;
        return;
    }
    float gate[1] = {1.0f}, w[1] = {1.0f};
    if (a.gate_kind == NORM_GATE_CHANNEL) raw_to_f32(load_raw<1>(a.gate, c, a.dt_w), a.dt_w, gate);
    if (a.w_post) raw_to_f32(load_raw<1>(a.w_post, c, a.dt_w), a.dt_w, w);
    if (a.dw_post) a.dw_post[c] = s * gate[0];
    if (a.d_gate_channel) a.d_gate_channel[c] = s * w[0];
}

__global__ void norm_zero_kernel(const NormBackArgs a) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= a.D) return;
    if (a.dw_pre) a.dw_pre[c] = 0.0f;
    if (a.dw_post) a.dw_post[c] = 0.0f;
    if (a.d_gate_channel) a.d_gate_channel[c] = 0.0f;
}

cudaError_t sm_count(int* sms) {
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
constexpr int kNormSmem = kSmemLimit - 2048;     // without the sums' static part

// What a kernel allows: rows of more than two_from windows have two a thread;
// group_threads: threads of a block's groups together at most, row_threads of
// one; regs: of a thread; deep: rows of a group in the ring, where there is
// room; split: blocks that share a row at most.
struct Rule {
    int two_from, group_threads, row_threads, regs, deep, split;
};

// slots: of a window in the ring; most: blocks (clusters).
bool shape_of(int64_t T, int D, const Alike& al, int slots, const Rule& rule, int sms, int64_t most, int split, Shape* s) {
    const int W = al.window;
    const int row = (D + (al.odd ? W - 1 : 0) + W - 1) / W, windows = (row + split - 1) / split;
    if (windows > 2 * rule.row_threads) return false;
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
    while (per_sm > 1 && per_sm * (rule.deep * stage * s->threads + fixed + 1024) > kNormSmem) --per_sm;
    int64_t grid = std::min<int64_t>((T + groups - 1) / groups, std::max(1, sms * per_sm / split));
    if (grid > most) grid = most;
    // a row's place in its windows has to be the same in all rows of a block
    if (al.odd && (groups > 1 || grid < T)) {
        if (grid < 8) return false;
        grid = grid / 8 * 8;
    }
    s->grid = static_cast<int>(grid);
    const int per_block = std::min<int>(per_sm, static_cast<int>((grid * split + sms - 1) / sms));
    const int64_t rows = (T + grid * groups - 1) / (grid * groups);                        // of a group at most
    int st = (kNormSmem / per_block - 1024 - fixed) / (stage * s->threads);
    st = std::max(1, std::min<int>(st, kNormMaxStages));
    s->stages = static_cast<int>(std::min<int64_t>(st, rows));
    if (rule.deep > 2 && s->stages < 2 && rows > 1) return false;         // two rows are in use at once
    s->smem = static_cast<size_t>(s->stages) * stage * s->threads + fixed;
    return s->smem <= static_cast<size_t>(kNormSmem);
}

// The fewest blocks a row that its windows and the ring's rows fit in.
bool shape_of(int64_t T, int D, const Alike& al, int slots, const Rule& rule, int sms, int64_t most, Shape* s) {
    if (!al.ok) return false;
    for (int split = 1; split <= rule.split; split *= 2)
        if (shape_of(T, D, al, slots, rule, sms, most, split, s)) return true;
    return false;
}

Steps steps_of(const NormArgs& a, int64_t rows) {
    Steps s = {};
    s.x = rows * a.ld_x * elem_bytes(a.dt_x);
    s.y = rows * a.ld_y * elem_bytes(a.dt_y);
    s.h = rows * a.ld_h * elem_bytes(a.dt_x);
    s.u = rows * a.ld_u * elem_bytes(a.dt_u);
    return s;
}
Steps steps_of(const NormBackArgs& a, int64_t rows) {
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

template <bool EDGE, int KIND>
cudaError_t forward_as(const NormArgs& a, const Shape& sh, cudaStream_t s) {
    if (sh.nv == 2) return run_rows(block_norm_kernel<2, EDGE, KIND>, a, sh, sh.smem, s);
    return run_rows(block_norm_kernel<1, EDGE, KIND>, a, sh, sh.smem, s);
}
// Two windows a thread in one block of up to 512 threads a SM, 128 registers
// each: the sums' exchange, the copies' and the loop's instructions are paid
// for 16 elements at a time.  4,096 x 7,168 bf16 70 us, one window a thread in
// 896 threads of 72 registers 84; 4,096 x 3,584 fp32 53 and 86.  Narrow rows
// have one window a thread; where that takes 72 registers, 896 threads.
template <bool EDGE, int KIND>
constexpr bool lean = !EDGE && (KIND == NORM_BF16 || KIND == NORM_F32);
template <bool EDGE, int KIND>
cudaError_t backward_as(const NormBackArgs& a, const Shape& sh, size_t smem, cudaStream_t s) {
    constexpr int kNarrow = lean<EDGE, KIND> ? 896 : 512;
    if (sh.split > 1) return run_rows(block_norm_backward_kernel<2, 512, EDGE, KIND, true>, a, sh, smem, s);
    if (sh.nv == 2) return run_rows(block_norm_backward_kernel<2, 512, EDGE, KIND, false>, a, sh, smem, s);
    return run_rows(block_norm_backward_kernel<1, kNarrow, EDGE, KIND, false>, a, sh, smem, s);
}

// Windows of four for rows of fp32, as long as two a thread cover the row.  The
// forward rule does not ask for u's type: a fused call and its two parts then
// add in the same order, and give the same bits.
bool fours(int D, int x, int y) { return D <= 8000 && x == ELEM_F32 && y == ELEM_F32; }

int plain_threads(int D) { return std::min(1024, std::max(32, (D + kPlainColumns / 4 - 1) / (kPlainColumns / 4) + 31) / 32 * 32); }

}  // namespace

int norm_parts(int64_t T, int D) {
    // narrow rows: more blocks, each with a short part
    const int64_t most = std::max<int64_t>(kNormParts, (1 << 19) / D);
    return static_cast<int>(std::max<int64_t>(1, std::min(T, most)));
}

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t s) {
    if (a.D < 1 || a.D > kNormMaxWidth || a.T < 0) return cudaErrorInvalidValue;
    if (a.T == 0) return cudaSuccess;
    int sms = 0;
    cudaError_t err = sm_count(&sms);
    if (err != cudaSuccess) return err;
    const int ty = a.y ? a.dt_y : a.dt_x, tu = a.u ? a.dt_u : a.dt_x;
    int kind = NORM_RUN;
    if (a.dt_x == ELEM_BF16 && tu == ELEM_BF16)
        kind = ty == ELEM_BF16 ? NORM_BF16 : (ty == ELEM_F32 ? NORM_BF16_Y32 : NORM_RUN);
    else if (fours(a.D, a.dt_x, ty))
        kind = NORM_F32;
    const int W = kind == NORM_F32 ? 4 : 8;
    Alike al(W);
    al.add(a.x, a.ld_x);
    al.add(a.y, a.ld_y);
    al.add(a.h, a.ld_h);
    al.add(a.u, a.ld_u);
    Shape sh;
    const int slots = window_slots(true, a.dt_x, W) + window_slots(a.y, a.dt_y, W);
    // 896 threads in two groups of 448 for 7,168 elements: the one group's
    // sums overlap the other's loads and stores
    if (shape_of(a.T, a.D, al, slots, Rule{256, 1024, 1024, 64, 2, 1}, sms, 1 << 30, &sh)) {
        if (kind == NORM_BF16) return sh.edge ? forward_as<true, NORM_BF16>(a, sh, s) : forward_as<false, NORM_BF16>(a, sh, s);
        if (kind == NORM_F32) return sh.edge ? forward_as<true, NORM_F32>(a, sh, s) : forward_as<false, NORM_F32>(a, sh, s);
        if (kind == NORM_BF16_Y32 && !sh.edge) return forward_as<false, NORM_BF16_Y32>(a, sh, s);
        return forward_as<true, NORM_RUN>(a, sh, s);
    }
    const int threads = plain_threads(a.D);
    block_norm_plain_kernel<<<static_cast<unsigned>(std::min<int64_t>(a.T, static_cast<int64_t>(sms) * (2048 / threads))),
                              threads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_block_norm_backward(const NormBackArgs& a, cudaStream_t s) {
    if (a.D < 1 || a.D > kNormMaxWidth || a.T < 0) return cudaErrorInvalidValue;
    if (a.T == 0) {
        if (!a.dw_pre && !a.dw_post && !a.d_gate_channel) return cudaSuccess;
        norm_zero_kernel<<<(a.D + 255) / 256, 256, 0, s>>>(a);
        return cudaGetLastError();
    }
    int sms = 0;
    cudaError_t err = sm_count(&sms);
    if (err != cudaSuccess) return err;
    int kind = NORM_RUN;
    if (a.y && a.du && a.dh && a.dx && a.dy && a.dt_u == a.dt_x) {
        if (a.dt_x == ELEM_BF16) kind = a.dt_y == ELEM_BF16 ? NORM_BF16 : (a.dt_y == ELEM_F32 ? NORM_BF16_Y32 : NORM_RUN);
        else if (fours(a.D, a.dt_x, a.dt_y)) kind = NORM_F32;
    }
    const int W = kind == NORM_F32 ? 4 : 8;
    Alike al(W);
    al.add(a.h, a.ld_h);
    al.add(a.du, a.ld_du);
    al.add(a.dh, a.ld_dh);
    al.add(a.y, a.ld_y);
    al.add(a.dx, a.ld_dx);
    al.add(a.dy, a.ld_dy);
    const int slots = window_slots(a.du, a.dt_x, W) + window_slots(a.du, a.dt_u, W) + window_slots(a.dh, a.dt_x, W) +
                      window_slots(a.y, a.dt_y, W);
    const int most = norm_parts(a.T, a.D);
    Shape sh;
    int parts;
    // the widest row with one window a thread: 1,024 elements of bf16 (28 us for
    // 8,192 rows, two windows 30; 2,048 elements 46 and 38), of fp32 too (32 and
    // 32), 2,048 with y in fp32 (53 and 56)
    const int two_from = kind == NORM_BF16 ? 128 : 256;
    const bool lean_row = !al.odd && a.D % W == 0 && (kind == NORM_BF16 || kind == NORM_F32) && a.D <= two_from * W;
    const Rule rule = {two_from, lean_row ? 896 : 512, 512, lean_row ? 72 : 128, 3, kNormMaxSplit};
    if (shape_of(a.T, a.D, al, slots, rule, sms, most, &sh)) {
        // the end of the kernel adds the groups' columns in the ring's memory
        size_t smem = sh.smem;
        if (a.part && sh.threads > sh.tpr) smem = std::max(smem, sizeof(float) * 2 * static_cast<size_t>(a.D));
        parts = sh.grid;
        if (kind == NORM_BF16)
            err = sh.edge ? backward_as<true, NORM_BF16>(a, sh, smem, s) : backward_as<false, NORM_BF16>(a, sh, smem, s);
        else if (kind == NORM_F32)
            err = sh.edge ? backward_as<true, NORM_F32>(a, sh, smem, s) : backward_as<false, NORM_F32>(a, sh, smem, s);
        else if (kind == NORM_BF16_Y32 && !sh.edge)
            err = backward_as<false, NORM_BF16_Y32>(a, sh, smem, s);
        else
            err = backward_as<true, NORM_RUN>(a, sh, smem, s);
    } else {
        parts = static_cast<int>(std::min<int64_t>(std::min<int64_t>(a.T, most), 2 * sms));
        const int threads = std::min(1024, (a.D + 31) / 32 * 32);
        block_norm_backward_plain_kernel<<<parts, threads, 0, s>>>(a);
        err = cudaGetLastError();
    }
    if (err != cudaSuccess || !a.part) return err;
    norm_columns_kernel<<<dim3((a.D + 31) / 32, 2), 32 * kColGroups, 0, s>>>(a, parts);
    return cudaGetLastError();
}

}  // namespace moe
