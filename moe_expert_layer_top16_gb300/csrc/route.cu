// Tokens sorted by expert and back, as operators of their own.
//
//   sort       slots i = t k + j (token t, slot j) ordered by expert, earlier
//              slots first: offsets[e] = number of kept slots of experts < e,
//              slot_pos[i] = offsets[e_i] + number of earlier slots of e_i,
//              sorted_slot[slot_pos[i]] = i.  A slot whose expert is outside
//              [0, E) is dropped: slot_pos -1, and nothing is read or written
//              for it below.
//   permute    rows[slot_pos[t, j]] = x[t]
//   unpermute  y[t] = sum_j w[t, j] rows[slot_pos[t, j]], slots in order, in
//              fp32 (w = 1 where none is given: the gradient of permute)
//   backward   d_rows[slot_pos[t, j]] = w[t, j] dy[t],
//              d_w[t, j] = <dy[t], rows[slot_pos[t, j]]>
//
// Every place is written by exactly one thread and every sum runs in a fixed
// order: results do not depend on scheduling.
#include <algorithm>

#include "internal.h"
#include "vec.cuh"

namespace moe {

namespace {

// ------------------------------------------------------------------ sort
// A counting sort.  Warp w of a CTA owns a contiguous strip of slots and counts
// its experts in a row of its own (cnt[w][E], shared memory; integer atomics,
// whose order does not matter).  A scan over the CTA's warps, then over the
// CTAs, then over experts turns the counts into each strip's first place of
// every expert.  A second pass over the strip hands the places out, 32 slots a
// step: match.any finds a slot's equals, the lanes below it are its rank, and
// the lowest lane of each set moves the strip's next place on.  The loads of
// kSortBatch steps are in flight together: a strip's steps are short, and one
// at a time each would pay a round trip to memory.
//
// Up to kSortOne slots one CTA does it all in one launch.  Beyond, a first
// launch counts each CTA's experts into the workspace, and every CTA of the
// second sums the counts of the CTAs before it: a cluster of eight CTAs with
// distributed shared memory took 33 us for 131,072 slots, bound by the
// shared-memory pipes of eight SMs, 64 CTAs in two launches take 14.5.  (One
// launch up to 4,096 slots, 11.7 us at most on the device, where two would take
// 7.3: the second launch and its workspace cost the host four.)
constexpr int kSortMaxE = 1024;
constexpr int kSortMaxWarps = 32;
constexpr int kSortBatch = 4;
constexpr int64_t kSortOne = 4096;         // slots of a single-CTA sort
constexpr int kSortSlots = 2048;
constexpr int kSortMaxCtas = 152;
constexpr int kSortCounts = 1 << 16;

// CTAs of a sort of n slots.  Each reads all CTAs' counts, so that many of them
// pay for short strips only with few experts: half of kSortSlots a CTA up to 32
// (16,384 slots 8.0 us, 9.2 with half as many CTAs; 65,536 on 32 CTAs 11.1, on
// 64 13.0), then kSortSlots until every SM has one or there are kSortCounts
// counts (262,144 slots of 896 experts on 128 CTAs 33.6 us, on 73 17.5).
int sort_ctas(int64_t n, int E) {
    if (n <= kSortOne) return 1;
    const int64_t half = (2 * n + kSortSlots - 1) / kSortSlots, whole = (n + kSortSlots - 1) / kSortSlots;
    const int64_t c = std::max(whole, std::min<int64_t>(half, 32));
    const int most = std::min(kSortMaxCtas, std::max(32, kSortCounts / E));
    return static_cast<int>(c < most ? c : most);
}

// Slots of CTA c of C: [first, last), whole 32-slot steps.
__device__ __forceinline__ void sort_range(int64_t n, int C, int c, int64_t& first, int64_t& last) {
    const int64_t steps = (n + 31) / 32;
    const int64_t per = (steps + C - 1) / C;
    first = min(c * per, steps);
    last = min(first + per, steps);
}

__global__ void __launch_bounds__(512) sort_count_kernel(const int32_t* __restrict__ idx, int64_t n, int E,
                                                         int32_t* __restrict__ counts) {
    extern __shared__ __align__(16) int32_t sm[];
    pdl_trigger();
    for (int e = threadIdx.x; e < E; e += blockDim.x) sm[e] = 0;
    __syncthreads();
    int64_t s0, s1;
    sort_range(n, gridDim.x, blockIdx.x, s0, s1);
    const int64_t i1 = min(s1 * 32, n);
    for (int64_t i = s0 * 32 + threadIdx.x; i < i1; i += 4 * blockDim.x) {
        int32_t e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) e[u] = i + u * blockDim.x < i1 ? idx[i + u * blockDim.x] : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (e[u] >= 0 && e[u] < E) atomicAdd(&sm[e[u]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) counts[static_cast<int64_t>(blockIdx.x) * E + e] = sm[e];
}

// counts is written by the launch that this one overlaps: plain loads, as the
// non-coherent path is for memory that nobody writes while the kernel lives.
__global__ void __launch_bounds__(kSortMaxWarps * 32)
    sort_kernel(const int32_t* __restrict__ idx, int64_t n, int E, const int32_t* counts,
                int32_t* __restrict__ offsets, int32_t* __restrict__ sorted_slot, int32_t* __restrict__ slot_pos) {
    extern __shared__ __align__(16) int32_t sm[];
    __shared__ int32_t warp_sum[32];
    const int W = blockDim.x >> 5, C = gridDim.x, rank = blockIdx.x;
    const int Ep = (E + 3) & ~3;       // rows of whole 16-byte words
    int32_t* cnt = sm;                 // [W][Ep]
    int32_t* start = sm + W * Ep;      // [Ep] this CTA's first place of each expert
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t first, last;
    sort_range(n, C, rank, first, last);
    // strips of whole 32-slot steps
    const int64_t per = (last - first + W - 1) / W;
    const int64_t s0 = min(first + warp * per, last), s1 = min(s0 + per, last);
    int32_t ex[kSortBatch];
    auto load = [&](int64_t s) {
#pragma unroll
        for (int u = 0; u < kSortBatch; ++u) {
            const int64_t i = (s + u) * 32 + lane;
            ex[u] = (s + u < s1 && i < n) ? idx[i] : -1;
        }
    };
    load(s0);
    for (int i = threadIdx.x; i < W * Ep / 4; i += blockDim.x) reinterpret_cast<int4*>(cnt)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    int32_t* mine = cnt + warp * Ep;
    for (int64_t s = s0; s < s1; s += kSortBatch) {
        if (s != s0) load(s);
#pragma unroll
        for (int u = 0; u < kSortBatch; ++u)
            if (ex[u] >= 0 && ex[u] < E) atomicAdd(&mine[ex[u]], 1);
    }
    __syncthreads();
    // each thread's run of consecutive experts: the strips before each strip,
    // the CTAs before this one, and all of them
    if (C > 1) pdl_wait();             // the counts of the launch before
    const int per_thread = (E + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    const int e0 = threadIdx.x * per_thread;
    int32_t sum = 0;
    for (int u = 0; u < per_thread; ++u) {
        const int e = e0 + u;
        if (e >= E) break;
        int32_t run = 0;
        for (int w0 = 0; w0 < W; w0 += 8) {
            int32_t c[8];
#pragma unroll
            for (int v = 0; v < 8; ++v) c[v] = w0 + v < W ? cnt[(w0 + v) * Ep + e] : 0;
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                if (w0 + v < W) cnt[(w0 + v) * Ep + e] = run;
                run += c[v];
            }
        }
        int32_t before = 0, all = run;
        if (C > 1) {
            all = 0;
            for (int c0 = 0; c0 < C; c0 += 16) {
                int32_t v[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) v[c] = c0 + c < C ? counts[static_cast<int64_t>(c0 + c) * E + e] : 0;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    before += c0 + c < rank ? v[c] : 0;
                    all += v[c];
                }
            }
        }
        start[e] = sum + before;       // within this thread's run so far
        sum += all;
    }
    int32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    // every warp scans the warps' sums for itself
    const int32_t ws = lane < W ? warp_sum[lane] : 0;
    int32_t winc = ws;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, winc, o);
        if (lane >= o) winc += v;
    }
    const int32_t total = __shfl_sync(0xffffffffu, winc, 31);
    const int32_t base = __shfl_sync(0xffffffffu, winc - ws, warp) + incl - sum;
    for (int u = 0; u < per_thread; ++u) {
        const int e = e0 + u;
        if (e >= E) break;
        start[e] += base;
        // no CTA before rank 0: its first places are the experts' offsets
        if (rank == 0) offsets[e] = start[e];
    }
    if (rank == 0 && threadIdx.x == 0) offsets[E] = total;
    __syncthreads();
    // the strips' places in order
    if (per > kSortBatch) load(s0);
    for (int64_t s = s0; s < s1; s += kSortBatch) {
        if (s != s0) load(s);
        uint32_t peers[kSortBatch];
#pragma unroll
        for (int u = 0; u < kSortBatch; ++u) {
            if (ex[u] < 0 || ex[u] >= E) ex[u] = E;
            peers[u] = __match_any_sync(0xffffffffu, ex[u]);
        }
#pragma unroll
        for (int u = 0; u < kSortBatch; ++u) {
            const int64_t i = (s + u) * 32 + lane;
            if (s + u >= s1) break;
            const uint32_t below = peers[u] & ((1u << lane) - 1);
            int32_t p = -1;
            if (ex[u] < E) p = start[ex[u]] + mine[ex[u]] + __popc(below);
            __syncwarp();
            if (ex[u] < E && below == 0) mine[ex[u]] += __popc(peers[u]);
            __syncwarp();
            if (i < n) {
                slot_pos[i] = p;
                if (p >= 0) sorted_slot[p] = static_cast<int32_t>(i);
            }
        }
    }
    for (int64_t p = total + static_cast<int64_t>(rank) * blockDim.x + threadIdx.x; p < n;
         p += static_cast<int64_t>(C) * blockDim.x)
        sorted_slot[p] = -1;
}

// ------------------------------------------------------------------ permute
// One warp per (token, chunk of the row, group of slots): the chunk's loads
// are issued once, then stored to each slot's place.  V: the widest word that
// both matrices' addresses, strides and the row's length are multiples of.
// Bound by HBM writes: 8,192 tokens of 3,584 bf16 to 16 places each 150 us (1.0
// GB, 6.6 TB/s; 147 at the rate of a plain copy).
constexpr int kPermWords = 4;     // words a lane holds

template <typename V>
__global__ void permute_kernel(const uint8_t* __restrict__ x, int64_t x_stride, int64_t row_words, int64_t T, int k,
                               const int32_t* __restrict__ slot_pos, int64_t n_rows, uint8_t* __restrict__ rows,
                               int64_t rows_stride, int64_t chunks, int groups, int spw) {
    const int64_t gw = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (gw >= T * chunks * groups) return;
    const int64_t t = gw / (chunks * groups);
    const int64_t rest = gw - t * chunks * groups;
    const int64_t ch = rest / groups;
    const int j0 = static_cast<int>(rest - ch * groups) * spw;
    const int j1 = min(j0 + spw, k);
    const int64_t w0 = ch * (32 * kPermWords) + lane;
    const V* src = reinterpret_cast<const V*>(x + t * x_stride);
    V v[kPermWords];
#pragma unroll
    for (int u = 0; u < kPermWords; ++u)
        if (w0 + 32 * u < row_words) v[u] = src[w0 + 32 * u];
    const int p_lane = (lane < k) ? slot_pos[t * k + lane] : -1;
    for (int j = j0; j < j1; ++j) {
        const int64_t p = __shfl_sync(0xffffffffu, p_lane, j);
        if (p < 0 || p >= n_rows) continue;
        V* dst = reinterpret_cast<V*>(rows + p * rows_stride);
#pragma unroll
        for (int u = 0; u < kPermWords; ++u)
            if (w0 + 32 * u < row_words) dst[w0 + 32 * u] = v[u];
    }
}

// ------------------------------------------------------------------ unpermute
// One warp per (token, 32 V columns), or, element by element, per 4 times 32
// columns, so that a warp that reads 64 bytes at a time has enough of them in
// flight: the slots' loads are issued a batch at a time, their FMAs run in
// slot order.  4,096 x 16 rows of 3,584 bf16: 68 us, 7.2 TB/s (mostly reads).
constexpr int kUnpermBatch = 8;

template <int V, int U, int DT>
__global__ void __launch_bounds__(128) unpermute_kernel(const void* __restrict__ rows, int64_t ld_rows, int64_t n_rows,
                                                        const int32_t* __restrict__ slot_pos,
                                                        const float* __restrict__ w, int64_t T, int k, int D,
                                                        void* __restrict__ y, int64_t ld_y, int dty, uint32_t chunks) {
    const int lane = threadIdx.x & 31;
    const uint32_t warp = threadIdx.x >> 5;
    const uint32_t per_block = blockDim.x >> 5;
    // grid: (chunks of columns in blocks of warps, tokens)
    const uint32_t ch = blockIdx.x * per_block + warp;
    if (ch >= chunks) return;
    const int64_t t = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
    if (t >= T) return;
    const int col = static_cast<int>(ch) * (32 * V * U) + lane * V;
    int32_t p_lane = (lane < k) ? slot_pos[t * k + lane] : -1;
    if (p_lane >= n_rows) p_lane = -1;
    const float w_lane = (lane < k) ? (w ? w[t * k + lane] : 1.0f) : 0.0f;
    float acc[U][V];
#pragma unroll
    for (int g = 0; g < U; ++g)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[g][i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += kUnpermBatch) {
        RawVec<V> r[kUnpermBatch][U];
#pragma unroll
        for (int u = 0; u < kUnpermBatch; ++u) {
            const int64_t p = __shfl_sync(0xffffffffu, p_lane, (j0 + u) & 31);
            if (j0 + u < k && p >= 0)
#pragma unroll
                for (int g = 0; g < U; ++g)
                    if (col + 32 * V * g < D) r[u][g] = load_stream<V, DT>(rows, p * ld_rows + col + 32 * V * g);
        }
#pragma unroll
        for (int u = 0; u < kUnpermBatch; ++u) {
            const int32_t p = __shfl_sync(0xffffffffu, p_lane, (j0 + u) & 31);
            const float wj = __shfl_sync(0xffffffffu, w_lane, (j0 + u) & 31);
            if (j0 + u < k && p >= 0)
#pragma unroll
                for (int g = 0; g < U; ++g)
                    if (col + 32 * V * g < D) {
                        float f[V];
                        raw_to_f32(r[u][g], DT, f);
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[g][i] = fmaf(wj, f[i], acc[g][i]);
                    }
        }
    }
#pragma unroll
    for (int g = 0; g < U; ++g)
        if (col + 32 * V * g < D) store_vec(y, t * ld_y + col + 32 * V * g, dty, acc[g]);
}

// ------------------------------------------------------------------ unpermute, backward
// One warp per SL slots of a token: the token's gradient and the slots' rows
// go by once, the dot products are summed over the lanes in a fixed order.
// Measured at 4,096 x 16 rows of 3,584 bf16: one slot a warp and four vectors
// in flight 167 us, two slots 164, two and three vectors 154 (6.2 TB/s), four
// slots and four vectors 186.
constexpr int kBackSlots = 2;
constexpr int kBackBatch = 3;

template <int V, int SL, int DT>
__global__ void __launch_bounds__(256) unpermute_backward_kernel(
    const void* __restrict__ dy, int64_t ld_dy, int dty, const void* __restrict__ rows, int64_t ld_rows,
    int64_t n_rows, const int32_t* __restrict__ slot_pos, const float* __restrict__ w, int64_t warps, int k, int D,
    void* __restrict__ d_rows, int64_t ld_d, float* __restrict__ d_w) {
    const int64_t gw = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (gw >= warps) return;
    const uint32_t per = static_cast<uint32_t>((k + SL - 1) / SL);               // warps of a token
    const int64_t t = static_cast<uint32_t>(gw) / per;                           // warps < 2^31
    const int j0 = static_cast<int>(static_cast<uint32_t>(gw) % per) * SL;
    int64_t p[SL];
    float wj[SL], dot[SL];
    bool any = false;
#pragma unroll
    for (int a = 0; a < SL; ++a) {
        const int64_t s = t * k + j0 + a;
        p[a] = j0 + a < k ? slot_pos[s] : -1;
        if (p[a] >= n_rows) p[a] = -1;
        wj[a] = w && p[a] >= 0 ? w[s] : 1.0f;
        dot[a] = 0.0f;
        any = any || p[a] >= 0;
    }
    for (int c0 = lane * V; any && c0 < D; c0 += 32 * V * kBackBatch) {
        RawVec<V> g[kBackBatch], r[SL][kBackBatch];
#pragma unroll
        for (int u = 0; u < kBackBatch; ++u) {
            const int c = c0 + 32 * V * u;
            if (c < D) {
                g[u] = load_raw<V>(dy, t * ld_dy + c, dty);
                if (d_w)
#pragma unroll
                    for (int a = 0; a < SL; ++a)
                        if (p[a] >= 0) r[a][u] = load_stream<V, DT>(rows, p[a] * ld_rows + c);
            }
        }
#pragma unroll
        for (int u = 0; u < kBackBatch; ++u) {
            const int c = c0 + 32 * V * u;
            if (c < D) {
                float f[V];
                raw_to_f32(g[u], dty, f);
#pragma unroll
                for (int a = 0; a < SL; ++a) {
                    if (p[a] < 0) continue;
                    if (d_w) {
                        float q[V];
                        raw_to_f32(r[a][u], DT, q);
#pragma unroll
                        for (int i = 0; i < V; ++i) dot[a] = fmaf(f[i], q[i], dot[a]);
                    }
                    if (d_rows) {
                        float o[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) o[i] = f[i] * wj[a];
                        store_stream<V, DT>(d_rows, p[a] * ld_d + c, o);
                    }
                }
            }
        }
    }
    if (!d_w) return;
#pragma unroll
    for (int a = 0; a < SL; ++a) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[a] += __shfl_xor_sync(0xffffffffu, dot[a], o);
        if (lane == 0 && j0 + a < k) d_w[t * k + j0 + a] = dot[a];
    }
}

unsigned blocks_of(int64_t warps, int threads) {
    return static_cast<unsigned>((warps * 32 + threads - 1) / threads);
}

// Grids are one-dimensional: at most 2^31 - 1 blocks.
bool grid_ok(int64_t warps, int threads) { return (warps * 32 + threads - 1) / threads <= 0x7fffffffll; }

template <typename V>
cudaError_t permute_as(const uint8_t* x, int64_t x_stride, int64_t row_bytes, int64_t T, int k, const int32_t* slot_pos,
                       int64_t n_rows, uint8_t* rows, int64_t rows_stride, cudaStream_t s) {
    const int64_t words = row_bytes / static_cast<int64_t>(sizeof(V));
    const int64_t chunks = (words + 32 * kPermWords - 1) / (32 * kPermWords);
    // all slots of a token in one warp read its row once; a small batch is
    // split over the slots too, until it has warps for every SM
    int spw = k;
    while (spw > 1 && T * chunks * ((k + spw - 1) / spw) < 152 * 16) spw = (spw + 1) / 2;
    const int groups = (k + spw - 1) / spw;
    const int64_t warps = T * chunks * groups;
    if (!grid_ok(warps, 256)) return cudaErrorInvalidValue;
    permute_kernel<V><<<blocks_of(warps, 256), 256, 0, s>>>(x, x_stride, words, T, k, slot_pos, n_rows, rows,
                                                             rows_stride, chunks, groups, spw);
    return cudaGetLastError();
}

}  // namespace

size_t sort_workspace_bytes(int64_t n, int E) {
    const int C = sort_ctas(n, E);
    return C > 1 ? sizeof(int32_t) * static_cast<size_t>(C) * E : 0;
}

cudaError_t launch_sort(const int32_t* idx, int64_t n, int E, int32_t* offsets, int32_t* sorted_slot,
                        int32_t* slot_pos, int32_t* work, cudaStream_t s) {
    if (n < 0 || E < 1 || E > kSortMaxE) return cudaErrorInvalidValue;
    const int C = sort_ctas(n, E);
    if (C > 1 && !work) return cudaErrorInvalidValue;
    const int64_t steps = ((n + 31) / 32 + C - 1) / C;
    int W = 4;
    // (more warps than a short strip each needs make the scan over them longer)
    while (W < (C > 1 && steps <= kSortSlots / 32 ? 16 : kSortMaxWarps) && W < steps) W *= 2;
    const size_t row = sizeof(int32_t) * static_cast<size_t>((E + 3) & ~3), smem = row * (W + 1);
    static_assert(sizeof(int32_t) * (kSortMaxWarps + 1) * kSortMaxE <= kSmemLimit - 1024, "sort tables");
    if (smem > 40 * 1024) {         // with the static part, up to 48 KB need no attribute
        const cudaError_t err = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(sizeof(int32_t) * (kSortMaxWarps + 1) * kSortMaxE));
        if (err != cudaSuccess) return err;
    }
    if (C > 1) {
        sort_count_kernel<<<C, 512, row, s>>>(idx, n, E, work);
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess) return err;
    }
    return launch_ex(sort_kernel, dim3(C), dim3(W * 32), smem, s, C > 1, idx, n, E,
                     static_cast<const int32_t*>(work), offsets, sorted_slot, slot_pos);
}

cudaError_t launch_permute(const uint8_t* x, int64_t x_stride, int64_t row_bytes, int64_t T, int k,
                           const int32_t* slot_pos, int64_t n_rows, uint8_t* rows, int64_t rows_stride,
                           cudaStream_t s) {
    const uint64_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(rows) |
                         static_cast<uint64_t>(x_stride) | static_cast<uint64_t>(rows_stride) |
                         static_cast<uint64_t>(row_bytes);
    if (!(all & 15)) return permute_as<uint4>(x, x_stride, row_bytes, T, k, slot_pos, n_rows, rows, rows_stride, s);
    if (!(all & 7)) return permute_as<uint2>(x, x_stride, row_bytes, T, k, slot_pos, n_rows, rows, rows_stride, s);
    if (!(all & 3)) return permute_as<uint32_t>(x, x_stride, row_bytes, T, k, slot_pos, n_rows, rows, rows_stride, s);
    if (!(all & 1)) return permute_as<uint16_t>(x, x_stride, row_bytes, T, k, slot_pos, n_rows, rows, rows_stride, s);
    return permute_as<uint8_t>(x, x_stride, row_bytes, T, k, slot_pos, n_rows, rows, rows_stride, s);
}

// Whether rows of this matrix can be read 8 elements at a time.
bool rows_by_8(const void* p, int64_t ld, int dt, int D) {
    return D % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * elem_bytes(dt)) % 16 == 0;
}

namespace {

template <int V, int DT>
cudaError_t unpermute_as(const void* rows, int64_t ld_rows, int64_t n_rows, const int32_t* slot_pos, const float* w,
                         int64_t T, int k, int D, void* y, int64_t ld_y, int dty, cudaStream_t s) {
    constexpr int U = V == 1 ? 4 : 1;
    const uint32_t chunks = static_cast<uint32_t>((D + 32 * V * U - 1) / (32 * V * U));
    const uint32_t warps = chunks < 4 ? chunks : 4;
    const uint32_t gy = T < 65535 ? static_cast<uint32_t>(T) : 65535u;
    const dim3 grid((chunks + warps - 1) / warps, gy, static_cast<unsigned>((T + gy - 1) / gy));
    unpermute_kernel<V, U, DT><<<grid, warps * 32, 0, s>>>(rows, ld_rows, n_rows, slot_pos, w, T, k, D, y, ld_y, dty, chunks);
    return cudaGetLastError();
}

// Two slots a warp read the token's gradient half as often; a small batch takes
// one, for more warps.
template <int V, int DT>
cudaError_t unpermute_backward_as(const void* dy, int64_t ld_dy, int dty, const void* rows, int64_t ld_rows,
                                  int64_t n_rows, const int32_t* slot_pos, const float* w, int64_t T, int k, int D,
                                  void* d_rows, int64_t ld_d, float* d_w, cudaStream_t s) {
    constexpr int SL = kBackSlots;
    const bool few = k == 1 || T * k < 152 * 64;
    const int64_t warps = T * (few ? k : (k + SL - 1) / SL);
    if (few)
        unpermute_backward_kernel<V, 1, DT><<<blocks_of(warps, 256), 256, 0, s>>>(
            dy, ld_dy, dty, rows, ld_rows, n_rows, slot_pos, w, warps, k, D, d_rows, ld_d, d_w);
    else
        unpermute_backward_kernel<V, SL, DT><<<blocks_of(warps, 256), 256, 0, s>>>(
            dy, ld_dy, dty, rows, ld_rows, n_rows, slot_pos, w, warps, k, D, d_rows, ld_d, d_w);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_unpermute(const void* rows, int64_t ld_rows, int dt, int64_t n_rows, const int32_t* slot_pos,
                             const float* w, int64_t T, int k, int D, void* y, int64_t ld_y, int dty, cudaStream_t s) {
    const bool v8 = rows_by_8(rows, ld_rows, dt, D) && rows_by_8(y, ld_y, dty, D);
    auto run = [&](auto f) { return f(rows, ld_rows, n_rows, slot_pos, w, T, k, D, y, ld_y, dty, s); };
    if (v8) {
        if (dt == ELEM_F32) return run(unpermute_as<8, ELEM_F32>);
        if (dt == ELEM_BF16) return run(unpermute_as<8, ELEM_BF16>);
        return run(unpermute_as<8, ELEM_F16>);
    }
    if (dt == ELEM_F32) return run(unpermute_as<1, ELEM_F32>);
    if (dt == ELEM_BF16) return run(unpermute_as<1, ELEM_BF16>);
    return run(unpermute_as<1, ELEM_F16>);
}

cudaError_t launch_unpermute_backward(const void* dy, int64_t ld_dy, int dty, const void* rows, int64_t ld_rows, int dt,
                                      int64_t n_rows, const int32_t* slot_pos, const float* w, int64_t T, int k, int D,
                                      void* d_rows, int64_t ld_d, float* d_w, cudaStream_t s) {
    const bool v8 = rows_by_8(dy, ld_dy, dty, D) && (!d_w || rows_by_8(rows, ld_rows, dt, D)) &&
                    (!d_rows || rows_by_8(d_rows, ld_d, dt, D));
    if (!grid_ok(T * k, 256)) return cudaErrorInvalidValue;
    auto run = [&](auto f) {
        return f(dy, ld_dy, dty, rows, ld_rows, n_rows, slot_pos, w, T, k, D, d_rows, ld_d, d_w, s);
    };
    if (v8) {
        if (dt == ELEM_F32) return run(unpermute_backward_as<8, ELEM_F32>);
        if (dt == ELEM_BF16) return run(unpermute_backward_as<8, ELEM_BF16>);
        return run(unpermute_backward_as<8, ELEM_F16>);
    }
    if (dt == ELEM_F32) return run(unpermute_backward_as<1, ELEM_F32>);
    if (dt == ELEM_BF16) return run(unpermute_backward_as<1, ELEM_BF16>);
    return run(unpermute_backward_as<1, ELEM_F16>);
}

}  // namespace moe
