// The norms behind and before a block, with the block's gate and the residual
// scale, in one pass over the rows (its gradients: norm_back.cu).
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
// fp32.  Measured: 8,192 x 7,168 bf16 81 us (470 MB, 5.8 TB/s; 69 us at the
// rate of a plain copy), fp32 163 (139), bf16 with y in fp32 118 (87); 2,048 x
// 16,384 fp32, split over two blocks, 90 (79); 64 rows of bf16 with y in fp32 5
// us, which is the launch, two trips to memory and two sums in turn.  Element by
// element (bases off 16 bytes) 8,192 x 7,168 bf16 361, fp32 382.
#include "norm.cuh"

namespace moe {

namespace {

// Forward.  A group keeps `stages` rows in flight by cp.async.
template <int NV, bool EDGE, int KIND, bool SPLIT>
__global__ void __launch_bounds__(1024) block_norm_kernel(const NormArgs a, int tpr, int stages, const Steps st) {
    using K = Kind<KIND>;
    constexpr int W = K::window;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][SPLIT ? kNormMaxSplit * kNormMaxWarps : kNormMaxWarps];
    int buf = 0;
    const int dx = K::x >= 0 ? K::x : a.dt_x, dy = K::y >= 0 ? K::y : a.dt_y;
    const int du = K::small ? K::x : a.dt_u;
    const bool post = a.y != nullptr, pre = a.u != nullptr;
    const Rows g = rows_of<SPLIT>(tpr, a.ld_x, W);
    __shared__ Exchange exchange;
    if constexpr (SPLIT) exchange_start(&exchange);
    auto row_sum = [&](float v) {
        if constexpr (SPLIT) return cluster_sum(v, g, red, &exchange, buf);
        else {
            float ss[1] = {v};
            group_sums<1>(ss, g, reinterpret_cast<float (*)[1][kNormMaxWarps]>(red), buf);
            return ss[0];
        }
    };
    const int D = a.D, T = static_cast<int>(a.T);
    const int pitch = blockDim.x * 16, wpitch = tpr * 16;
    const int yw = window_slots(post, dy, W), slots = yw + window_slots(true, dx, W);
    uint8_t* weights = ring + g.lane_in_group * 16;
    uint8_t* mine = ring + NV * (W / 2) * wpitch + threadIdx.x * 16;        // [stages][NV][slots]
    const int step = tpr * W, c0 = g.lane_in_group * W - g.shift + g.part * NV * step;
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
            q = rsqrtf(row_sum(sum2(acc)) * inv_d + a.eps);
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
            const float r = rsqrtf(row_sum(sum2(acc)) * inv_d + a.eps);
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

template <bool EDGE, int KIND>
cudaError_t forward_as(const NormArgs& a, const Shape& sh, cudaStream_t s) {
    if (sh.split > 1) return run_rows(block_norm_kernel<2, EDGE, KIND, true>, a, sh, sh.smem, s);
    if (sh.nv == 2) return run_rows(block_norm_kernel<2, EDGE, KIND, false>, a, sh, sh.smem, s);
    return run_rows(block_norm_kernel<1, EDGE, KIND, false>, a, sh, sh.smem, s);
}

// About four columns a thread.
int plain_threads(int D) { return std::min(1024, ((D + 3) / 4 + 31) / 32 * 32); }

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t s) {
    if (a.D < 1 || a.D > kNormMaxWidth || a.T < 0) return cudaErrorInvalidValue;
    if (a.T == 0) return cudaSuccess;
    int sms = 0;
    cudaError_t err = sm_count(&sms);
    if (err != cudaSuccess) return err;
    // the window goes by x's type alone: where the matrices lie alike, at equal
    // strides, a fused call and its two parts sum a row in the same order and
    // give the same bits
    const int ty = a.y ? a.dt_y : a.dt_x, tu = a.u ? a.dt_u : a.dt_x;
    int kind = NORM_RUN;
    if (a.dt_x == ELEM_F32) kind = ty == ELEM_F32 ? NORM_F32 : NORM_F32_Y16;
    else if (tu == a.dt_x) kind = small_kind(a.dt_x, ty);
    const int W = a.dt_x == ELEM_F32 ? 4 : 8;
    Alike al(W);
    al.add(a.x, a.ld_x);
    al.add(a.y, a.ld_y);
    al.add(a.h, a.ld_h);
    al.add(a.u, a.ld_u);
    Shape sh;
    const int slots = window_slots(true, a.dt_x, W) + window_slots(a.y, a.dt_y, W);
    // Two windows a thread from 65 on (8,192 x 2,048 bf16 22 us, one 26; 1,024
    // fp32 21 and 24).  Two groups a block overlap the one's sums with the
    // other's loads and stores; many whole rows of 448 windows or more are
    // better off with one group and a ring of four rows (8,192 x 7,168 bf16 81.5
    // and 84.6 us, 4,096 fp32 80.5 and 94.5; of 1,024 rows 15.3 and 12.9).  Near
    // the rule's borders the two are within 5%, or 10% for the widest: four rows
    // and three, 8,192 x 3,456 bf16 38.5 and 40.3, 3,584 40.7 and 40.8; 4,560 x
    // 7,168 bf16 48.4 and 46.8, 4,864 51.1 and 49.4; 4,560 x 4,096 fp32 48.0 and
    // 52.1, 4,864 50.6 and 56.6.  Odd rows are better off with two groups than
    // with a third row (7,167 48 and 63).
    const bool mixed = a.dt_x != ELEM_F32 && ty == ELEM_F32, whole_row = !al.odd && a.D % W == 0;
    const int deep = mixed || !whole_row ? 2 : (a.D >= 448 * W && a.T >= 32 * static_cast<int64_t>(sms) ? 4 : 3);
    if (shape_of(a.T, a.D, al, slots, Rule{64, 1024, 1024, 1024, 64, deep, 1, kNormMaxSplit, W == 4 ? 2 : 3}, sms, 1 << 30, &sh)) {
        if (kind == NORM_F32_Y16) return forward_as<true, NORM_F32_Y16>(a, sh, s);
        return with_kind(kind, sh.edge, [&](auto edge, auto k) {
            return forward_as<decltype(edge)::value, decltype(k)::value>(a, sh, s);
        });
    }
    const int threads = plain_threads(a.D);
    block_norm_plain_kernel<<<static_cast<unsigned>(std::min<int64_t>(a.T, static_cast<int64_t>(sms) * (2048 / threads))),
                              threads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
