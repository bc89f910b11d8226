// Gradients of the norms round a block (the formulas stand in norm.cu).
#include "norm.cuh"

namespace moe {

namespace {

// Four sums at once: the lanes halve what they carry with each exchange (two
// values after the first, one after the second), so that six exchanges do what
// twenty would; lane 8 k then holds value k of the warp.
// `between` is done before the barrier: what the threads that arrive first do
// while they would wait.
template <bool SPLIT, int WARPS, typename F>
__device__ __forceinline__ void group_sums4(float (&v)[4], const Rows& g, float (*red)[4][WARPS], Exchange* exchange, int& buf,
                                            F between) {
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
            if ((lane & 7) == 0) send_all(&red[buf & 1][lane >> 3][g.part * (g.tpr >> 5) + warp], exchange, buf, g, s);
            between();
            __syncwarp();
            s = receive_all(exchange, buf, g, 4) ? 0.0f : __uint_as_float(0x7FC00000u);
        } else {
            if ((lane & 7) == 0) red[buf][lane >> 3][warp] = s;
            between();
            asm volatile("bar.sync %0, %1;" ::"r"(1 + g.group), "r"(g.tpr) : "memory");
            s = 0.0f;
        }
#pragma unroll
        for (int w = 0; w < WARPS; w += 8)
            if (w + (lane & 7) < warps) s += red[SPLIT ? buf & 1 : buf][lane >> 3][warp0 + w + (lane & 7)];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        buf = SPLIT ? buf + 1 : buf ^ 1;
    } else {
        between();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, s, 8 * i);
}

// Gradients, with the same ring.  The column sums of a thread's rows stay in
// registers (sum du h^ and sum total y^, times the token's gate), are added
// over the block's groups through shared memory and go to the block's part.
// The weights wait in shared memory, which leaves registers for the sums.  The
// sums over row t + 1 that its norms need are taken together with the one over
// row t that its dy needs: one barrier a row, and the work of both before it.
// What bounds it: HBM for whole rows (4,096 x 7,168 bf16 62 us, 352 MB, 5.7
// TB/s; 52 us at the rate of a plain copy; fp32, split over two blocks, 113 and
// 104); for rows of odd lengths the few warps that mask partial windows (4,096
// x 7,167 bf16 99).  Calls without dh, du or y, or with du of another type than
// h, take the instance whose types are looked up at run time and whose registers
// spill: 4,096 x 7,168 bf16 without y 118 us (35), without du 121 (35), without dh
// 152 (43); fp32 with du in bf16 430 (95).  Element by element, bases off 16
// bytes: bf16 688, fp32 539.
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
    __shared__ Exchange exchange;
    if constexpr (SPLIT) exchange_start(&exchange);
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
        group_sums4<SPLIT>(v, g, red, &exchange, buf, [] {});
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
        group_sums4<SPLIT>(v, g, red, &exchange, buf, [&] { issue(t + stages * g.step); });
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
    pdl_trigger();                     // the columns' kernel may come up while the parts are written
    const int pitch_c = a.pitch, shift_c = g.shift & a.mask;
    float* out = a.part + static_cast<int64_t>(g.unit) * 2 * pitch_c;
    // the groups in turn add their columns to the block's, in the ring's
    // memory (one group: straight to the part)
    float* acc = g.groups == 1 ? out : reinterpret_cast<float*>(ring);
    cp_async_wait(0);
    __syncthreads();
    for (int k = 0; k < g.groups; ++k) {
        if (g.group == k) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                // the window's place in the part (outside the row its sums are zero)
                const int c = c0 + i * step + shift_c;
                if (c - shift_c >= D) break;
                auto add = [&](const Pair (&sum)[W / 2], float* to) {
                    if (c >= 0 && c + W <= pitch_c && reinterpret_cast<uintptr_t>(to + c) % 16 == 0) {
#pragma unroll
                        for (int j = 0; j < W / 4; ++j) {
                            const float2 f = split(sum[2 * j]), e = split(sum[2 * j + 1]);
                            float4* at = reinterpret_cast<float4*>(to + c) + j;
                            const float4 o = k ? *at : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            *at = make_float4(o.x + f.x, o.y + f.y, o.z + e.x, o.w + e.y);
                        }
                        return;
                    }
#pragma unroll
                    for (int j = 0; j < W / 2; ++j) {
                        const float2 f = split(sum[j]);
                        const int e = c + 2 * j;
                        if (e >= 0 && e < pitch_c) to[e] = (k ? to[e] : 0.0f) + f.x;
                        if (e + 1 >= 0 && e + 1 < pitch_c) to[e + 1] = (k ? to[e + 1] : 0.0f) + f.y;
                    }
                };
                add(s_pre[i], acc);
                add(s_post[i], acc + pitch_c);
            }
        }
        __syncthreads();
    }
    if (g.groups > 1)
        for (int c = threadIdx.x; c < 2 * pitch_c; c += blockDim.x) out[c] = acc[c];
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
        pdl_trigger();
        float* out = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.pitch;
#pragma unroll
        for (int i = 0; i < kPlainColumns; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= a.D) break;
            out[c] = s_pre[i];
            out[a.pitch + c] = s_post[i];
        }
    }
}

// Column sums of the CTAs' parts, in a fixed order, and the weights' and the
// channel gate's gradients from them.
constexpr int kColGroups = 16, kColBatch = 10;     // loads in flight: 152 parts in one go
__global__ void __launch_bounds__(32 * kColGroups) norm_columns_kernel(const NormBackArgs a, int parts, int ld) {
    __shared__ float red[kColGroups][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const int which = blockIdx.y;                 // 0: sum du h^, 1: sum total g y^
    pdl_wait();
    float s = 0.0f;
    if (c < a.D) {
        const float* from = a.part + static_cast<int64_t>(which) * a.pitch + c;
        const int64_t part = 2 * static_cast<int64_t>(a.pitch);
        for (int p = g; p < parts; p += kColBatch * kColGroups) {
            float v[kColBatch];
#pragma unroll
            for (int u = 0; u < kColBatch; ++u) {
                const int q = p + u * kColGroups;
                v[u] = q < parts ? from[q * part + (q * ld & a.mask)] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < kColBatch; ++u) s += v[u];
        }
    }
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

// Two windows a thread in one block of up to 512 threads a SM, 128 registers
// each: the sums' exchange, the copies' and the loop's instructions are paid
// for 16 elements at a time.  With all else alike, 4,096 x 7,168 bf16 70 us, one
// window a thread in 896 threads of 72 registers 87; 4,096 x 3,584 fp32 (h, du
// and dh one tensor) 53 and 86.  Narrow rows have one window a thread.
// Wider rows than 1,024 windows are split, where one block of 704 threads would
// do too (4,096 x 5,120 fp32 83.5 us, one block 88.6).
template <bool EDGE, int KIND>
cudaError_t backward_as(const NormBackArgs& a, const Shape& sh, size_t smem, cudaStream_t s) {
    if (sh.split > 1) return run_rows(block_norm_backward_kernel<2, 512, EDGE, KIND, true>, a, sh, smem, s);
    if (sh.nv == 2) return run_rows(block_norm_backward_kernel<2, 512, EDGE, KIND, false>, a, sh, smem, s);
    return run_rows(block_norm_backward_kernel<1, 512, EDGE, KIND, false>, a, sh, smem, s);
}

}  // namespace

int norm_parts(int64_t T, int D) {
    // narrow rows: more blocks, each with a short part
    const int64_t most = std::max<int64_t>(kNormParts, (1 << 19) / D);
    return static_cast<int>(std::max<int64_t>(1, std::min(T, most)));
}

cudaError_t launch_block_norm_backward(const NormBackArgs& in, cudaStream_t s) {
    NormBackArgs a = in;
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
        // windows of four: as many as two a thread of four blocks cover
        if (a.dt_x == ELEM_F32 && a.dt_y == ELEM_F32 && (a.D <= 16376 || a.D % 4 == 0)) kind = NORM_F32;
        else kind = small_kind(a.dt_x, a.dt_y);
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
    a.pitch = norm_pitch(a.D);
    a.mask = a.D % 8 ? W - 1 : 0;
    Shape sh;
    int parts;
    // one window a thread up to 64 (one tensor for h, du and dh: 8,192 rows of 1,024 bf16 25.7 us, two 23.7);
    // with y in fp32 up to 256 (29.5 and 31.7), and two groups a block rather
    // than a third row in the ring (3,584 columns 79 and 96)
    const bool mixed = a.dt_x != ELEM_F32 && a.y && a.dt_y == ELEM_F32;
    const Rule rule = {mixed ? 256 : 64, 512, 512, 512, 128, mixed ? 2 : 3, 2, kNormMaxSplit, 0};
    if (shape_of(a.T, a.D, al, slots, rule, sms, most, &sh)) {
        // the end of the kernel adds the groups' columns in the ring's memory
        size_t smem = sh.smem;
        if (a.part && sh.threads > sh.tpr) smem = std::max(smem, sizeof(float) * 2 * static_cast<size_t>(a.pitch));
        parts = sh.grid;
        err = with_kind(kind, sh.edge, [&](auto edge, auto k) {
            return backward_as<decltype(edge)::value, decltype(k)::value>(a, sh, smem, s);
        });
    } else {
        parts = static_cast<int>(std::min<int64_t>(std::min<int64_t>(a.T, most), 2 * sms));
        const int threads = std::min(1024, (a.D + 31) / 32 * 32);
        a.mask = 0;
        block_norm_backward_plain_kernel<<<parts, threads, 0, s>>>(a);
        err = cudaGetLastError();
    }
    if (err != cudaSuccess || !a.part) return err;
    return launch_ex(norm_columns_kernel, dim3((a.D + 31) / 32, 2), dim3(32 * kColGroups), 0, s, true, a, parts,
                     static_cast<int>((a.du ? a.ld_h : a.ld_dh) & 7));
}

}  // namespace moe
