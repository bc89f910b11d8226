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
// Bound by HBM: every row of every matrix goes by once.  A CTA holds whole
// rows in registers, so the two block-wide sums (of y^2, then of h^2) need no
// second read.  All sums are fp32.
#include <atomic>

#include "internal.h"
#include "vec.cuh"

namespace moe {

namespace {

constexpr int kNormMaxWarps = 32;

// Block-wide sums of N values in a fixed order: lanes by butterfly, then the
// warps' sums in warp order (every thread adds them itself).  `buf` alternates
// between calls, so that one barrier a call is enough.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*red)[N][kNormMaxWarps], int& buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[buf][i][threadIdx.x >> 5] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = 0.0f;
        for (int w = 0; w < warps; ++w) s += red[buf][i][w];
        v[i] = s;
    }
    buf ^= 1;
}

template <int V, int NV>
__global__ void __launch_bounds__(V == 8 ? 512 : 1024) block_norm_kernel(const NormArgs a) {
    __shared__ float red[2][1][kNormMaxWarps];
    int buf = 0;
    const int step = blockDim.x * V;
    const int c0 = threadIdx.x * V;
    const bool post = a.y != nullptr, pre = a.u != nullptr;
    float wp[NV][V], wn[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) wp[i][j] = wn[i][j] = 1.0f;
        const int c = c0 + i * step;
        if (c >= a.D) continue;
        if (post && a.w_post) raw_to_f32(load_raw<V>(a.w_post, c, a.dt_w), a.dt_w, wp[i]);
        if (post && a.gate_kind == NORM_GATE_CHANNEL) {
            float g[V];
            raw_to_f32(load_raw<V>(a.gate, c, a.dt_w), a.dt_w, g);
#pragma unroll
            for (int j = 0; j < V; ++j) wp[i][j] *= g[j];
        }
        if (pre && a.w_pre) raw_to_f32(load_raw<V>(a.w_pre, c, a.dt_w), a.dt_w, wn[i]);
    }
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        RawVec<V> rx[NV], ry[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c < a.D) {
                if (post) ry[i] = load_raw<V>(a.y, t * a.ld_y + c, a.dt_y);
                rx[i] = load_raw<V>(a.x, t * a.ld_x + c, a.dt_x);
            }
        }
        float h[NV][V];
        if (post) {
            float y[NV][V];
            float s[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (c0 + i * step >= a.D) continue;
                raw_to_f32(ry[i], a.dt_y, y[i]);
#pragma unroll
                for (int j = 0; j < V; ++j) s[0] = fmaf(y[i][j], y[i][j], s[0]);
            }
            block_sums<1>(s, red, buf);
            float q = 1.0f / sqrtf(s[0] / static_cast<float>(a.D) + a.eps);
            if (a.gate_kind == NORM_GATE_TOKEN) {
                float g[1];
                raw_to_f32(load_raw<1>(a.gate, t, a.dt_w), a.dt_w, g);
                q *= g[0];
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * step;
                if (c >= a.D) continue;
                float x[V];
                raw_to_f32(rx[i], a.dt_x, x);
#pragma unroll
                for (int j = 0; j < V; ++j) h[i][j] = fmaf(a.res_scale, x[j], q * wp[i][j] * y[i][j]);
                store_vec(a.h, t * a.ld_h + c, a.dt_x, h[i]);
#pragma unroll
                for (int j = 0; j < V; ++j) h[i][j] = round_to(h[i][j], a.dt_x);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (c0 + i * step < a.D) raw_to_f32(rx[i], a.dt_x, h[i]);
        }
        if (pre) {
            float s[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (c0 + i * step >= a.D) continue;
#pragma unroll
                for (int j = 0; j < V; ++j) s[0] = fmaf(h[i][j], h[i][j], s[0]);
            }
            block_sums<1>(s, red, buf);
            const float r = 1.0f / sqrtf(s[0] / static_cast<float>(a.D) + a.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * step;
                if (c >= a.D) continue;
#pragma unroll
                for (int j = 0; j < V; ++j) h[i][j] = h[i][j] * r * wn[i][j];
                store_vec(a.u, t * a.ld_u + c, a.dt_u, h[i]);
            }
        }
    }
}

// Gradients.  The column sums of a CTA's rows stay in registers and go to
// part[blockIdx.x][2][D] at the end: sum du h^ and sum total y^ (times the
// token's gate).
template <int V, int NV>
__global__ void __launch_bounds__(V == 8 ? 512 : 1024) block_norm_backward_kernel(const NormBackArgs a) {
    __shared__ float red[2][3][kNormMaxWarps];
    __shared__ float red1[2][1][kNormMaxWarps];
    int buf = 0, buf1 = 0;
    const int step = blockDim.x * V;
    const int c0 = threadIdx.x * V;
    const bool post = a.y != nullptr, pre = a.du != nullptr;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    float s_pre[NV][V], s_post[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) s_pre[i][j] = s_post[i][j] = 0.0f;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        RawVec<V> rh[NV], rdu[NV], rdh[NV], ry[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c < a.D) {
                if (pre) {
                    rh[i] = load_raw<V>(a.h, t * a.ld_h + c, a.dt_x);
                    rdu[i] = load_raw<V>(a.du, t * a.ld_du + c, a.dt_u);
                }
                if (post) ry[i] = load_raw<V>(a.y, t * a.ld_y + c, a.dt_y);
                if (a.dh) rdh[i] = load_raw<V>(a.dh, t * a.ld_dh + c, a.dt_x);
            }
        }
        float total[NV][V];
        float s[3] = {0.0f, 0.0f, 0.0f};     // h^2, a h, y^2
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c >= a.D) continue;
            if (pre) {
                float h[V], g[V];
                raw_to_f32(rh[i], a.dt_x, h);
                raw_to_f32(rdu[i], a.dt_u, g);
                if (a.w_pre) {
                    float w[V];
                    raw_to_f32(load_raw<V>(a.w_pre, c, a.dt_w), a.dt_w, w);
#pragma unroll
                    for (int j = 0; j < V; ++j) g[j] *= w[j];
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    s[0] = fmaf(h[j], h[j], s[0]);
                    s[1] = fmaf(g[j], h[j], s[1]);
                    total[i][j] = g[j];
                }
            }
            if (post) {
                float y[V];
                raw_to_f32(ry[i], a.dt_y, y);
#pragma unroll
                for (int j = 0; j < V; ++j) s[2] = fmaf(y[j], y[j], s[2]);
            }
        }
        block_sums<3>(s, red, buf);
        const float r = 1.0f / sqrtf(s[0] * inv_d + a.eps);
        const float m = r * r * s[1] * inv_d;          // mean(a h^) / rms(h)
        const float q = 1.0f / sqrtf(s[2] * inv_d + a.eps);
        float gt = 1.0f;
        if (post && a.gate_kind == NORM_GATE_TOKEN) {
            float g[1];
            raw_to_f32(load_raw<1>(a.gate, t, a.dt_w), a.dt_w, g);
            gt = g[0];
        }
        float d[1] = {0.0f};                           // sum total w_post (channel gate) y
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c >= a.D) continue;
            float dh[V];
#pragma unroll
            for (int j = 0; j < V; ++j) dh[j] = 0.0f;
            if (a.dh) raw_to_f32(rdh[i], a.dt_x, dh);
            if (pre) {
                float h[V], g[V];
                raw_to_f32(rh[i], a.dt_x, h);
                raw_to_f32(rdu[i], a.dt_u, g);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    s_pre[i][j] = fmaf(g[j], h[j] * r, s_pre[i][j]);
                    total[i][j] = dh[j] + r * (total[i][j] - h[j] * m);
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) total[i][j] = dh[j];
            }
            if (a.dx) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = post ? a.res_scale * total[i][j] : total[i][j];
                store_vec(a.dx, t * a.ld_dx + c, a.dt_x, o);
            }
            if (post) {
                float y[V], w[V];
                raw_to_f32(ry[i], a.dt_y, y);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    s_post[i][j] = fmaf(total[i][j] * gt, y[j] * q, s_post[i][j]);
                    w[j] = 1.0f;
                }
                if (a.w_post) raw_to_f32(load_raw<V>(a.w_post, c, a.dt_w), a.dt_w, w);
                if (a.gate_kind == NORM_GATE_CHANNEL) {
                    float g[V];
                    raw_to_f32(load_raw<V>(a.gate, c, a.dt_w), a.dt_w, g);
#pragma unroll
                    for (int j = 0; j < V; ++j) w[j] *= g[j];
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    total[i][j] *= w[j];
                    d[0] = fmaf(total[i][j], y[j], d[0]);
                }
            }
        }
        if (post) {
            block_sums<1>(d, red1, buf1);
            if (a.d_gate_token && threadIdx.x == 0) a.d_gate_token[t] = d[0] * q;
            if (a.dy) {
                const float n = q * q * d[0] * inv_d;      // mean(p y^) / (g rms(y))
                const float f = q * gt;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = c0 + i * step;
                    if (c >= a.D) continue;
                    float y[V], o[V];
                    raw_to_f32(ry[i], a.dt_y, y);
#pragma unroll
                    for (int j = 0; j < V; ++j) o[j] = f * (total[i][j] - y[j] * n);
                    store_vec(a.dy, t * a.ld_dy + c, a.dt_y, o);
                }
            }
        }
    }
    if (a.part) {
        float* out = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.D;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = c0 + i * step + j;
                if (c < a.D) {
                    out[c] = s_pre[i][j];
                    out[a.D + c] = s_post[i][j];
                }
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

bool vec8(const void* p, int64_t ld, int dt) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * elem_bytes(dt)) % 16 == 0);
}

// Threads of a CTA and register vectors a thread for rows of D elements.
void norm_shape(int D, bool v8, int& threads, int& nv) {
    const int n = v8 ? D / 8 : D;
    if (v8) nv = n <= 512 ? 1 : (n <= 1024 ? 2 : 4);
    else nv = n <= 4096 ? 4 : 16;
    threads = ((n + nv - 1) / nv + 31) / 32 * 32;
}

// Blocks of `threads` threads of this kernel instance that fit on an SM.
template <auto Kern>
int resident(int threads) {
    static std::atomic<int> cache[kNormMaxWarps + 1];
    int n = cache[threads / 32].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, Kern, threads, 0) != cudaSuccess || n < 1) n = 1;
        cache[threads / 32].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int V, int NV>
cudaError_t forward_as(const NormArgs& a, int threads, int sms, cudaStream_t s) {
    const int64_t most = static_cast<int64_t>(sms) * resident<block_norm_kernel<V, NV>>(threads);
    block_norm_kernel<V, NV><<<static_cast<unsigned>(a.T < most ? a.T : most), threads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int V, int NV>
cudaError_t backward_as(const NormBackArgs& a, int threads, int sms, cudaStream_t s) {
    int64_t grid = static_cast<int64_t>(sms) * resident<block_norm_backward_kernel<V, NV>>(threads);
    if (grid > kNormParts) grid = kNormParts;
    if (grid > a.T) grid = a.T;
    block_norm_backward_kernel<V, NV><<<static_cast<unsigned>(grid), threads, 0, s>>>(a);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || !a.part) return err;
    norm_columns_kernel<<<dim3((a.D + 31) / 32, 2), 32 * kColGroups, 0, s>>>(a, static_cast<int>(grid));
    return cudaGetLastError();
}

cudaError_t sm_count(int* sms) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    return err;
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t s) {
    if (a.D < 1 || a.D > kNormMaxWidth || a.T < 0) return cudaErrorInvalidValue;
    if (a.T == 0) return cudaSuccess;
    int sms = 0;
    cudaError_t err = sm_count(&sms);
    if (err != cudaSuccess) return err;
    const bool v8 = a.D % 8 == 0 && vec8(a.x, a.ld_x, a.dt_x) && vec8(a.y, a.ld_y, a.dt_y) && vec8(a.h, a.ld_h, a.dt_x) &&
                    vec8(a.u, a.ld_u, a.dt_u) && vec8(a.w_post, 0, a.dt_w) && vec8(a.w_pre, 0, a.dt_w) &&
                    (a.gate_kind != NORM_GATE_CHANNEL || vec8(a.gate, 0, a.dt_w));
    int threads, nv;
    norm_shape(a.D, v8, threads, nv);
    if (v8) {
        if (nv == 1) return forward_as<8, 1>(a, threads, sms, s);
        if (nv == 2) return forward_as<8, 2>(a, threads, sms, s);
        return forward_as<8, 4>(a, threads, sms, s);
    }
    if (nv == 4) return forward_as<1, 4>(a, threads, sms, s);
    return forward_as<1, 16>(a, threads, sms, s);
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
    const bool v8 = a.D % 8 == 0 && vec8(a.h, a.ld_h, a.dt_x) && vec8(a.y, a.ld_y, a.dt_y) && vec8(a.dh, a.ld_dh, a.dt_x) &&
                    vec8(a.du, a.ld_du, a.dt_u) && vec8(a.dx, a.ld_dx, a.dt_x) && vec8(a.dy, a.ld_dy, a.dt_y) &&
                    vec8(a.w_post, 0, a.dt_w) && vec8(a.w_pre, 0, a.dt_w) &&
                    (a.gate_kind != NORM_GATE_CHANNEL || vec8(a.gate, 0, a.dt_w));
    int threads, nv;
    norm_shape(a.D, v8, threads, nv);
    if (v8) {
        if (nv == 1) return backward_as<8, 1>(a, threads, sms, s);
        if (nv == 2) return backward_as<8, 2>(a, threads, sms, s);
        return backward_as<8, 4>(a, threads, sms, s);
    }
    if (nv == 4) return backward_as<1, 4>(a, threads, sms, s);
    return backward_as<1, 16>(a, threads, sms, s);
}

}  // namespace moe
