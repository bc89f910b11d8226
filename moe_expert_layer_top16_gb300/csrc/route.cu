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
#include <cooperative_groups.h>

#include "internal.h"
#include "vec.cuh"

namespace moe {

namespace cg = cooperative_groups;

namespace {

// ------------------------------------------------------------------ sort
// A counting sort in one launch of one cluster.  Warp w of the cluster owns a
// contiguous strip of slots and counts its experts in a row of its own
// (cnt[w][E], shared memory): the 32 slots of a step find their equals with
// match.any, and the lowest lane of each set adds the set's size.  A scan over
// the CTA's warps, then over the cluster's CTAs (distributed shared memory),
// then over experts turns the counts into each strip's first place of every
// expert, and a second pass over the strip hands the places out.
constexpr int kSortMaxE = 1024;
constexpr int kSortMaxWarps = 32;

__global__ void sort_kernel(const int32_t* __restrict__ idx, int64_t n, int E, int32_t* __restrict__ offsets,
                            int32_t* __restrict__ sorted_slot, int32_t* __restrict__ slot_pos, int C) {
    extern __shared__ int32_t sm[];
    __shared__ int32_t warp_sum[32];
    const int W = blockDim.x >> 5;
    int32_t* cnt = sm;                 // [W][E]
    int32_t* tot = sm + W * E;         // [E] this CTA's counts
    int32_t* start = tot + E;          // [E] this CTA's first place of each expert
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x);
    for (int i = threadIdx.x; i < W * E; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    // strips of whole 32-slot steps
    const int64_t steps = (n + 31) / 32;
    const int64_t per = (steps + static_cast<int64_t>(C) * W - 1) / (static_cast<int64_t>(C) * W);
    const int64_t s0 = (static_cast<int64_t>(rank) * W + warp) * per;
    const int64_t s1 = s0 + per < steps ? s0 + per : steps;
    int32_t* mine = cnt + warp * E;
    for (int64_t s = s0; s < s1; ++s) {
        const int64_t i = s * 32 + lane;
        int e = (i < n) ? idx[i] : -1;
        if (e < 0 || e >= E) e = E;
        const uint32_t peers = __match_any_sync(0xffffffffu, e);
        if (e < E && (peers & ((1u << lane) - 1)) == 0) mine[e] += __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int32_t run = 0;
        for (int w = 0; w < W; ++w) {
            const int32_t c = cnt[w * E + e];
            cnt[w * E + e] = run;
            run += c;
        }
        tot[e] = run;
    }
    // each thread's run of consecutive experts: earlier CTAs' counts and the
    // cluster's total
    if (C > 1) cg::this_cluster().sync();
    else __syncthreads();
    const int per_thread = (E + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    const int e0 = threadIdx.x * per_thread;
    int32_t sum = 0;
    for (int u = 0; u < per_thread; ++u) {
        const int e = e0 + u;
        if (e >= E) break;
        int32_t before = 0, all = 0;
        if (C > 1) {
            for (int c = 0; c < C; ++c) {
                const int32_t v = cg::this_cluster().map_shared_rank(tot, c)[e];
                before += (c < rank) ? v : 0;
                all += v;
            }
        } else {
            all = tot[e];
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
    int32_t base = incl - sum, total = 0;
    for (int w = 0; w < W; ++w) {
        if (w < warp) base += warp_sum[w];
        total += warp_sum[w];
    }
    {
        for (int u = 0; u < per_thread; ++u) {
            const int e = e0 + u;
            if (e >= E) break;
            start[e] += base;
        }
    }
    if (rank == 0 && threadIdx.x == 0) offsets[E] = total;
    __syncthreads();
    // rank 0 has no earlier CTA: its first places are the experts' offsets
    if (rank == 0)
        for (int e = threadIdx.x; e < E; e += blockDim.x) offsets[e] = start[e];
    // the strips' places in order
    for (int64_t s = s0; s < s1; ++s) {
        const int64_t i = s * 32 + lane;
        int e = (i < n) ? idx[i] : -1;
        if (e < 0 || e >= E) e = E;
        const uint32_t peers = __match_any_sync(0xffffffffu, e);
        const uint32_t below = peers & ((1u << lane) - 1);
        int32_t p = -1;
        if (e < E) p = start[e] + mine[e] + __popc(below);
        __syncwarp();
        if (e < E && below == 0) mine[e] += __popc(peers);
        if (i < n) {
            slot_pos[i] = p;
            if (p >= 0) sorted_slot[p] = static_cast<int32_t>(i);
        }
        __syncwarp();
    }
    for (int64_t p = total + static_cast<int64_t>(rank) * blockDim.x + threadIdx.x; p < n;
         p += static_cast<int64_t>(C) * blockDim.x)
        sorted_slot[p] = -1;
    // no CTA leaves while another may still read its counts
    if (C > 1) cg::this_cluster().sync();
}

// ------------------------------------------------------------------ permute
// One warp per (token, chunk of the row, group of slots): the chunk's loads
// are issued once, then stored to each slot's place.  V: the widest word that
// both matrices' addresses, strides and the row's length are multiples of.
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
// One warp per (token, 32 V columns): the slots' loads are issued a batch at
// a time, their FMAs run in slot order.
constexpr int kUnpermBatch = 8;

template <int V>
__global__ void __launch_bounds__(128) unpermute_kernel(const void* __restrict__ rows, int64_t ld_rows, int dt,
                                                        int64_t n_rows, const int32_t* __restrict__ slot_pos,
                                                        const float* __restrict__ w, int64_t T, int k, int D,
                                                        void* __restrict__ y, int64_t ld_y, int dty, int64_t chunks) {
    const int64_t gw = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (gw >= T * chunks) return;
    const int64_t t = gw / chunks;
    const int64_t col = (gw - t * chunks) * (32 * V) + lane * V;
    int32_t p_lane = (lane < k) ? slot_pos[t * k + lane] : -1;
    if (p_lane >= n_rows) p_lane = -1;
    const float w_lane = (lane < k) ? (w ? w[t * k + lane] : 1.0f) : 0.0f;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += kUnpermBatch) {
        RawVec<V> r[kUnpermBatch];
#pragma unroll
        for (int u = 0; u < kUnpermBatch; ++u) {
            const int64_t p = __shfl_sync(0xffffffffu, p_lane, (j0 + u) & 31);
            if (j0 + u < k && p >= 0 && col < D) r[u] = load_raw<V>(rows, p * ld_rows + col, dt);
        }
#pragma unroll
        for (int u = 0; u < kUnpermBatch; ++u) {
            const int32_t p = __shfl_sync(0xffffffffu, p_lane, (j0 + u) & 31);
            const float wj = __shfl_sync(0xffffffffu, w_lane, (j0 + u) & 31);
            if (j0 + u < k && p >= 0 && col < D) {
                float f[V];
                raw_to_f32(r[u], dt, f);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(wj, f[i], acc[i]);
            }
        }
    }
    if (col < D) store_vec(y, t * ld_y + col, dty, acc);
}

// ------------------------------------------------------------------ unpermute, backward
// One warp per slot: the token's gradient and the slot's row go by once, the
// dot product is summed over the lanes in a fixed order.
constexpr int kBackBatch = 4;

template <int V>
__global__ void __launch_bounds__(256) unpermute_backward_kernel(
    const void* __restrict__ dy, int64_t ld_dy, int dty, const void* __restrict__ rows, int64_t ld_rows, int dt,
    int64_t n_rows, const int32_t* __restrict__ slot_pos, const float* __restrict__ w, int64_t T, int k, int D,
    void* __restrict__ d_rows, int64_t ld_d, float* __restrict__ d_w) {
    const int64_t s = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (s >= T * k) return;
    const int64_t t = s / k;
    const int64_t p = slot_pos[s];
    if (p < 0 || p >= n_rows) {
        if (d_w && lane == 0) d_w[s] = 0.0f;
        return;
    }
    const float wj = w ? w[s] : 1.0f;
    float dot = 0.0f;
    for (int64_t c0 = lane * V; c0 < D; c0 += 32 * V * kBackBatch) {
        RawVec<V> g[kBackBatch], r[kBackBatch];
#pragma unroll
        for (int u = 0; u < kBackBatch; ++u) {
            const int64_t c = c0 + 32 * V * u;
            if (c < D) {
                g[u] = load_raw<V>(dy, t * ld_dy + c, dty);
                if (d_w) r[u] = load_raw<V>(rows, p * ld_rows + c, dt);
            }
        }
#pragma unroll
        for (int u = 0; u < kBackBatch; ++u) {
            const int64_t c = c0 + 32 * V * u;
            if (c < D) {
                float f[V];
                raw_to_f32(g[u], dty, f);
                if (d_w) {
                    float q[V];
                    raw_to_f32(r[u], dt, q);
#pragma unroll
                    for (int i = 0; i < V; ++i) dot = fmaf(f[i], q[i], dot);
                }
                if (d_rows) {
#pragma unroll
                    for (int i = 0; i < V; ++i) f[i] *= wj;
                    store_vec(d_rows, p * ld_d + c, dt, f);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (d_w && lane == 0) d_w[s] = dot;
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

cudaError_t launch_sort(const int32_t* idx, int64_t n, int E, int32_t* offsets, int32_t* sorted_slot,
                        int32_t* slot_pos, cudaStream_t s) {
    if (n < 0 || E < 1 || E > kSortMaxE) return cudaErrorInvalidValue;
    // one CTA up to 8,192 slots, then up to 8 (the portable cluster size)
    int C = 1;
    while (C < 8 && n > static_cast<int64_t>(C) * 8192) C *= 2;
    const int64_t steps = (n + 31) / 32;
    int W = 4;
    while (W < kSortMaxWarps && static_cast<int64_t>(W) * C < steps) W *= 2;
    const size_t smem = sizeof(int32_t) * (static_cast<size_t>(W) + 2) * E;
    static_assert(sizeof(int32_t) * (kSortMaxWarps + 2) * kSortMaxE <= kSmemLimit, "sort tables");
    if (smem > 48 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(sizeof(int32_t) * (kSortMaxWarps + 2) * kSortMaxE));
        if (err != cudaSuccess) return err;
    }
    return launch_ex_cluster(sort_kernel, dim3(C), dim3(W * 32), smem, s, false, C, idx, n, E, offsets, sorted_slot,
                             slot_pos, C);
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

cudaError_t launch_unpermute(const void* rows, int64_t ld_rows, int dt, int64_t n_rows, const int32_t* slot_pos,
                             const float* w, int64_t T, int k, int D, void* y, int64_t ld_y, int dty, cudaStream_t s) {
    const bool v8 = rows_by_8(rows, ld_rows, dt, D) && rows_by_8(y, ld_y, dty, D);
    const int64_t chunks = (D + (v8 ? 255 : 31)) / (v8 ? 256 : 32);
    const int64_t warps = T * chunks;
    if (!grid_ok(warps, 128)) return cudaErrorInvalidValue;
    if (v8)
        unpermute_kernel<8><<<blocks_of(warps, 128), 128, 0, s>>>(rows, ld_rows, dt, n_rows, slot_pos, w, T, k, D, y,
                                                                  ld_y, dty, chunks);
    else
        unpermute_kernel<1><<<blocks_of(warps, 128), 128, 0, s>>>(rows, ld_rows, dt, n_rows, slot_pos, w, T, k, D, y,
                                                                  ld_y, dty, chunks);
    return cudaGetLastError();
}

cudaError_t launch_unpermute_backward(const void* dy, int64_t ld_dy, int dty, const void* rows, int64_t ld_rows, int dt,
                                      int64_t n_rows, const int32_t* slot_pos, const float* w, int64_t T, int k, int D,
                                      void* d_rows, int64_t ld_d, float* d_w, cudaStream_t s) {
    const bool v8 = rows_by_8(dy, ld_dy, dty, D) && (!d_w || rows_by_8(rows, ld_rows, dt, D)) &&
                    (!d_rows || rows_by_8(d_rows, ld_d, dt, D));
    const int64_t warps = T * k;
    if (!grid_ok(warps, 256)) return cudaErrorInvalidValue;
    if (v8)
        unpermute_backward_kernel<8><<<blocks_of(warps, 256), 256, 0, s>>>(
            dy, ld_dy, dty, rows, ld_rows, dt, n_rows, slot_pos, w, T, k, D, d_rows, ld_d, d_w);
    else
        unpermute_backward_kernel<1><<<blocks_of(warps, 256), 256, 0, s>>>(
            dy, ld_dy, dty, rows, ld_rows, dt, n_rows, slot_pos, w, T, k, D, d_rows, ld_d, d_w);
    return cudaGetLastError();
}

}  // namespace moe
