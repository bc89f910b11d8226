// The router as operators of their own.
//
//   select     the k experts of each token with the largest keys, and their
//              gates.  Key: the logit l, or with a bias sigmoid(l) + b; equal
//              keys by the lower expert.  Gates: the winners' scores over
//              their sum, or as they are
//   balance    for each sequence of tokens the counts c_e of its slots, the
//              mean share P_e of each expert in its tokens' scores, and
//              L = E / (k n) sum_e c_e P_e   (1 when both are even)
//   backward   the gradient of gates and losses with respect to the logits,
//              both in one pass over them
//
// A token's logits are one warp's: a lane holds them in registers, eight
// neighbours at a time where rows allow it (one at a time the loads are eight
// times as many).  Every sum runs in a fixed order.
//
// Large batches should be bound by the logits' way from HBM, 4.4 us for 8,192 rows
// of 896 in fp32, k = 16; they take 22 us (selection), 21 (loss) and 24 (gradient): a row
// is 650 (loss) to some 1,200 instructions of one warp, most of them in chains
// (sorts and sums over the lanes, 25 to 35 cycles a step), which 17 to 28 warps
// an SM hide in part.  Small calls are the host's: 11 to 15 us a call for 3 to 5 us
// on the device.
#include <algorithm>
#include <cfloat>

#include "internal.h"
#include "ptx.cuh"
#include "norm.cuh"
#include "vec.cuh"

namespace moe {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// A logit as the operators read it: what is not a number closes an expert like
// minus infinity, plus infinity counts as the largest number.
// (fmaxf and fminf go past NaN.)
__device__ __forceinline__ float open_logit(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX); }

template <bool OPEN, int V, int NI>
__device__ __forceinline__ void open_row(const RawVec<V> (&raw)[NI], int E, int dt, int lane, float (&v)[NI * V]) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = (32 * i + lane) * V;
        float f[V];
        if (e < E) raw_to_f32(raw[i], dt, f);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i * V + j] = e < E ? (OPEN ? open_logit(f[j]) : f[j]) : -INFINITY;
    }
}

// A lane's part of a row: value i V + j is that of expert (32 i + lane) V + j;
// minus infinity behind the last expert.  DT: the type, or -1 where dt has it
// (rows that are read by single elements).  OPEN: as open_logit has them.
template <int DT, bool OPEN, int V, int NI>
__device__ __forceinline__ void load_row(const void* base, int64_t off, int E, int dt, int lane, float (&v)[NI * V]) {
    if (DT >= 0) dt = DT;
    RawVec<V> raw[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = (32 * i + lane) * V;
        if (e < E) raw[i] = load_raw<V>(base, off + e, dt);
    }
    open_row<OPEN, V, NI>(raw, E, dt, lane, v);
}

// ------------------------------------------------------------------ reductions over a warp
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// e^x and 1 / x by the instructions for them.  2^(x log2 e) is off by two units in
// the last place and by |x| of them for the product's rounding: as much as the
// rounding of an argument l - top, which e^-|x| turns into less than a unit of the
// largest score.  (expf takes 8 instructions for this one's 2, and the row's
// exponentials were more than half of these kernels.)
__device__ __forceinline__ float fast_exp(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504f));
    return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / d of four values from 1 to 2^30 by one reciprocal: the special functions
// take four of a warp's lanes a clock, and with two for each logit they were what
// a row took longest for.  Off by 6 x 2^-24 at most.
__device__ __forceinline__ void rcp4(const float (&d)[4], float (&q)[4]) {
    const float a = d[0] * d[1], b = d[2] * d[3], r = fast_rcp(a * b);
    const float ra = r * b, rb = r * a;
    q[0] = ra * d[1];
    q[1] = ra * d[0];
    q[2] = rb * d[3];
    q[3] = rb * d[2];
}

// ------------------------------------------------------------------ scores
// Scores of values v[N] as multiples of a common factor that keeps them from
// underflow, and their sum over the warp.  Softmax: e^(v - max).  Sigmoid:
// sigmoid(v) = e^min(v, 0) / (1 + e^-|v|), its numerator over the largest one,
// which is 1 unless every value is negative.  Closed values give 0.
template <bool SIG, int N>
__device__ __forceinline__ float scores(float (&v)[N]) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, v[i]);
    top = warp_max(top);
    float sum = 0.0f;
    if (top == -INFINITY) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
    } else if (!SIG) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = fast_exp(v[i] - top);
            sum += v[i];
        }
    } else if (top >= 0.0f) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            float u[4], d[4], q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u[j] = fast_exp(-fabsf(v[i + j]));
                d[j] = 1.0f + u[j];
            }
            rcp4(d, q);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i + j] = (v[i + j] >= 0.0f ? 1.0f : u[j]) * q[j];
                sum += v[i + j];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = fast_exp(v[i] - top) * fast_rcp(1.0f + fast_exp(v[i]));
            sum += v[i];
        }
    }
    return warp_sum(sum);
}
// The same for one value a lane, which the gates are made of.
__device__ __forceinline__ float slot_scores(float& v, bool sigmoid) {
    const float top = warp_max(sigmoid ? fminf(v, 0.0f) : v);
    v = top == -INFINITY ? 0.0f : expf((sigmoid ? fminf(v, 0.0f) : v) - top) / (sigmoid ? 1.0f + expf(-fabsf(v)) : 1.0f);
    return warp_sum(v);
}

__device__ __forceinline__ float sigmoid_of(float v) {
    const float u = expf(-fabsf(v));
    return (v >= 0.0f ? 1.0f : u) / (1.0f + u);
}
// 1 - sigmoid(v) without the cancellation.
__device__ __forceinline__ float sigmoid_rest(float v) {
    const float u = expf(-fabsf(v));
    return (v >= 0.0f ? u : 1.0f) / (1.0f + u);
}

// ------------------------------------------------------------------ select
// The k-th largest of the lanes' largest keys (for k > 16: of the lanes' halves')
// is at most the k-th largest key: what reaches it are the candidates, whose
// numbers go to shared memory.  Up to 32 of them are sorted over the lanes, up to
// kCand ranked by counting the better ones; rows with more take k rounds of a
// maximum over the row.
//
// How many there are depends on how many of those sets hold an expert: 1.1 to 1.4 k
// where all do and k is at most half of them (896 or 256 experts, k = 16: 21; element
// by element from 61 up).  Rows that go by eight values fill E / 8 lanes, and with
// fewer sets than k every expert is a candidate; for k > 16 element by element one
// half of each lane is empty up to E = 512 (and for E <= 256 up to 128).  Ordinary
// rows then take the slow ways too.  8,192 rows in fp32, with a bias and without:
//   k = 16   256 experts 15, 12 us   128: 149, 46   96: 775, 191   64: 50, 26
//   k = 32   896: 55, 30   512: 47, 27   256: 42, 24   384: 455, 134   128: 1,954, 431
//            384, not aligned: 5,643, 971
//   k = 8    64 to 256: 12 to 21, 10 to 15
// One row that takes rounds is enough for most of it: 501 experts and k = 32, 560 and 150
// us for a single token, and up to 1,115 and 283 us where a few rows of 896 or 1,024 do.
//
// Keys with a bias are defined in 64 bits, whose exponentials would take some
// ten times as long as the logits' way from memory.  They are estimated in 32:
// |estimate - key| <= 5e-7 + 2^-24 |estimate|.  (With u = e^-l and s = 1 / (1 + u),
// u is off by (2^-22 + 1.3 |l| 2^-24) u, of which s (1 - s) <= 1/4 and |l| s (1 - s)
// <= 0.23 leave 1.3 x 2^-24; the sum 1 + u and rcp4 add 7 x 2^-24, the u kept below
// 2^30 1e-9, together less than 5e-7; the last term is the sum with b.)  Candidates
// are what reaches the bound less twice that, and only where two neighbours in the
// order are nearer than that and not equal in logit and bias are the candidates
// ranked by keys of 64 bits: a row in some hundreds, at which a launch's last rows
// wait longest.  The neighbours looked at are those up to the end of the run of
// equals that holds the last slot: of two candidates in the wrong order, the better
// one behind, those from the first to the last are all near, and the first two of
// them that differ stand at the end of a run that begins before or at the last slot.
// 8,192 rows of 896, k = 16: 22 us with a bias, 16 without.
constexpr int kCand = 64;
constexpr int kSelectWarps = 4;
constexpr float kNear = 1e-6f, kNearRel = 0x1p-22f;

struct Candidate {
    float key, l, b;
    int e;
};

__device__ __forceinline__ float key32(float l, float b) {
    const float s = fast_rcp(1.0f + fminf(fast_exp(-l), 0x1p30f)) + b;
    return l > -INFINITY ? s : -INFINITY;
}
__device__ __forceinline__ void keys32(float* l, const float* b) {
    float d[4], q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = 1.0f + fminf(fast_exp(-l[j]), 0x1p30f);
    rcp4(d, q);
#pragma unroll
    for (int j = 0; j < 4; ++j) l[j] = l[j] > -INFINITY ? q[j] + b[j] : -INFINITY;
}
__device__ __forceinline__ double key64(float l, float b) {
    return 1.0 / (1.0 + exp(-static_cast<double>(l))) + static_cast<double>(b);
}
// A bias of minus infinity or not a number closes an expert as well.
__device__ __forceinline__ float open_bias(float b) { return open_logit(b); }

// Descending over the lanes.
__device__ __forceinline__ float bitonic_step(float x, int lane, int stride, bool down) {
    const float y = __shfl_xor_sync(kAll, x, stride);
    return (((lane & stride) == 0) == down) ? fmaxf(x, y) : fminf(x, y);
}
__device__ __forceinline__ float sort_lanes(float x, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int stride = size / 2; stride > 0; stride /= 2) x = bitonic_step(x, lane, stride, (lane & size) == 0);
    return x;
}
// Keys with their experts, by (key descending, expert ascending).
__device__ __forceinline__ void sort_keys(float& key, int& e, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int stride = size / 2; stride > 0; stride /= 2) {
            const float k2 = __shfl_xor_sync(kAll, key, stride);
            const int e2 = __shfl_xor_sync(kAll, e, stride);
            const bool other = k2 > key || (k2 == key && e2 < e);            // the partner's is the better one
            const bool take = other == (((lane & stride) == 0) == ((lane & size) == 0));
            key = take ? k2 : key;
            e = take ? e2 : e;
        }
}

// Rows with too many candidates: k rounds, each the largest key of 64 bits
// below the pick before, in the order (key descending, expert ascending).
__device__ __noinline__ void select_rounds(const SelectArgs& a, int64_t t, int lane, int* win, float* win_l) {
    double last = INFINITY;
    int last_e = -1;
    for (int j = 0; j < a.k; ++j) {
        double best = -INFINITY;
        int best_e = 0x7fffffff;
        float best_l = 0.0f;
        for (int e = lane; e < a.E; e += 32) {
            float f[1];
            raw_to_f32(load_raw<1>(a.logits, t * a.ld + e, a.dt), a.dt, f);
            const float l = open_logit(f[0]), b = a.bias ? open_bias(a.bias[e]) : 0.0f;
            if (l == -INFINITY || b == -INFINITY) continue;
            const double key = a.bias ? key64(l, b) : static_cast<double>(l);
            if ((key < last || (key == last && e > last_e)) && key > best) {
                best = key;
                best_e = e;
                best_l = l;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double k2 = __shfl_xor_sync(kAll, best, o);
            const int e2 = __shfl_xor_sync(kAll, best_e, o);
            const float l2 = __shfl_xor_sync(kAll, best_l, o);
            if (k2 > best || (k2 == best && e2 < best_e)) {
                best = k2;
                best_e = e2;
                best_l = l2;
            }
        }
        if (lane == 0 && best_e < a.E) {
            win[j] = best_e;
            win_l[j] = best_l;
        }
        last = best;
        last_e = best_e;
        if (best_e >= a.E) break;
    }
}

template <int DT, int V, int NI>
__global__ void __launch_bounds__(kSelectWarps * 32, 7) select_kernel(const SelectArgs a) {
    __shared__ __align__(16) Candidate s_cand[kSelectWarps][kCand];
    __shared__ double s_key[kSelectWarps][kCand];
    __shared__ int s_win[kSelectWarps][32];
    __shared__ float s_win_l[kSelectWarps][32];
    constexpr int N = NI * V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kSelectWarps + warp;
    if (t >= a.T) return;
    const int E = a.E, k = a.k;
    if (a.mask && !a.mask[t]) {
        if (lane < k) {
            a.idx[t * k + lane] = -1;
            a.gates[t * k + lane] = 0.0f;
        }
        return;
    }
    Candidate* cand = s_cand[warp];
    auto logit = [&](int e) {
        float f[1];
        raw_to_f32(load_raw<1>(a.logits, t * a.ld + e, DT >= 0 ? DT : a.dt), ELEM_F32, f);
        return open_logit(f[0]);
    };
    // keys; without a bias these are the logits
    float v[N];
    load_row<DT, false, V, NI>(a.logits, t * a.ld, E, a.dt, lane, v);
    if (a.bias) {
        constexpr int W = V == 8 ? 8 : 4;                // keys at a time
#pragma unroll
        for (int i = 0; i < N; i += W) {
            float b[W];
#pragma unroll
            for (int j = 0; j < W; j += V) {
                const int e0 = (32 * ((i + j) / V) + lane) * V;
                float f[V];
#pragma unroll
                for (int c = 0; c < V; ++c) f[c] = 0.0f;
                if (e0 < E) raw_to_f32(load_raw<V>(a.bias, e0, ELEM_F32), ELEM_F32, f);
#pragma unroll
                for (int c = 0; c < V; ++c) b[j + c] = f[c];
            }
#pragma unroll
            for (int j = 0; j < W; j += 4) keys32(v + i + j, b + j);
        }
    }
    // (a key that is not a number is passed over by maxima and reaches no bound)
    // the bound: the k-th largest of 32 or 64 disjoint sets' largest keys
    float h0 = -INFINITY, h1 = -INFINITY;
#pragma unroll
    for (int c = 0; c < N; ++c) {
        if (c < N / 2)
            h0 = fmaxf(h0, v[c]);
        else
            h1 = fmaxf(h1, v[c]);
    }
    float least;
    if (k <= 16) {
        least = sort_lanes(fmaxf(h0, h1), lane);
    } else {
        h0 = sort_lanes(h0, lane);
        h1 = __shfl_sync(kAll, sort_lanes(h1, lane), 31 - lane);
        least = fmaxf(h0, h1);           // the 32 largest of both, as a bitonic sequence
#pragma unroll
        for (int stride = 16; stride > 0; stride /= 2) least = bitonic_step(least, lane, stride, true);
    }
    least = __shfl_sync(kAll, least, k - 1);
    least = fminf(least, FLT_MAX);
    if (a.bias) least -= kNear + kNearRel * fabsf(least);
    least = fmaxf(least, -FLT_MAX);      // (fewer than k sets have an open expert: all that are open)
    uint32_t mask = 0;
#pragma unroll
    for (int c = 0; c < N; ++c) mask |= v[c] >= least ? 1u << c : 0u;
    const int mine = __popc(mask);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += n;
    }
    const int n = __shfl_sync(kAll, incl, 31);
    int e = -1;                          // of slot `lane`; -1 behind the last slot and where no expert was left
    float l[1] = {-INFINITY};
    if (n <= kCand) {
        int pos = incl - mine;
        while (mask) {
            const int c = __ffs(mask) - 1;
            mask &= mask - 1;
            cand[pos++].e = (32 * (c / V) + lane) * V + c % V;
        }
        __syncwarp();
    }
    if (n <= 32) {
        float key = -INFINITY, bias = 0.0f;
        int at = 0x7fffffff;             // the expert and the lane that has its logit and bias
        if (lane < n) {
            e = cand[lane].e;
            l[0] = key = logit(e);
            if (a.bias) {
                bias = open_bias(a.bias[e]);
                key = key32(key, bias);
            }
            at = e * 32 + lane;
        }
        sort_keys(key, at, lane);
        e = at >> 5;
        l[0] = __shfl_sync(kAll, l[0], at & 31);
        if (a.bias) {
            bias = __shfl_sync(kAll, bias, at & 31);
            const float key2 = __shfl_down_sync(kAll, key, 1), l2 = __shfl_down_sync(kAll, l[0], 1), b2 = __shfl_down_sync(kAll, bias, 1);
            const bool differ = lane + 1 >= n || l2 != l[0] || b2 != bias;
            const uint32_t ends = __ballot_sync(kAll, differ);           // of runs of equals; lane 31 is always one
            const uint32_t near = __ballot_sync(kAll, lane + 1 < n && differ && key - key2 <= kNear + kNearRel * fabsf(key));
            // as far as the run that has the last slot: what is behind its end may be better than its equals
            const int last = k - 1 + __ffs(ends >> (k - 1)) - 1;
            if (near & (0xffffffffu >> (31 - last))) {
                const double exact = lane < n ? key64(l[0], bias) : -INFINITY;
                int rank = 0;
                for (int p = 0; p < n; ++p) {
                    const double q = __shfl_sync(kAll, exact, p);
                    const int f = __shfl_sync(kAll, e, p);
                    rank += (q > exact || (q == exact && f < e)) ? 1 : 0;
                }
                if (lane < n) {
                    s_win[warp][rank] = e;
                    s_win_l[warp][rank] = l[0];
                }
                __syncwarp();
                if (lane < n) {
                    e = s_win[warp][lane];
                    l[0] = s_win_l[warp][lane];
                }
            }
        }
        if (lane >= min(n, k)) {
            e = -1;
            l[0] = -INFINITY;
        }
    } else {
        s_win[warp][lane] = -1;
        s_win_l[warp][lane] = -INFINITY;
        __syncwarp();
        if (n > kCand) {
            select_rounds(a, t, lane, s_win[warp], s_win_l[warp]);
        } else {
            // two candidates a lane
            Candidate own[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int p = lane + 32 * u;
                if (p < n) {
                    own[u].e = cand[p].e;
                    own[u].l = logit(own[u].e);
                    own[u].b = a.bias ? open_bias(a.bias[own[u].e]) : 0.0f;
                    own[u].key = a.bias ? key32(own[u].l, own[u].b) : own[u].l;
                    cand[p] = own[u];
                }
            }
            __syncwarp();
            int rank[2] = {0, 0};
            bool near = false;
            for (int p = 0; p < n; ++p) {
                const Candidate q = cand[p];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (lane + 32 * u >= n) continue;
                    rank[u] += (q.key > own[u].key || (q.key == own[u].key && q.e < own[u].e)) ? 1 : 0;
                    if (a.bias)
                        near |= fabsf(q.key - own[u].key) <= kNear + kNearRel * fabsf(own[u].key) &&
                                !(q.l == own[u].l && q.b == own[u].b);
                }
            }
            if (a.bias && __any_sync(kAll, near)) {
                double exact[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    rank[u] = 0;
                    if (lane + 32 * u < n) s_key[warp][lane + 32 * u] = exact[u] = key64(own[u].l, own[u].b);
                }
                __syncwarp();
                for (int p = 0; p < n; ++p) {
                    const double q = s_key[warp][p];
                    const int f = cand[p].e;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        if (lane + 32 * u < n) rank[u] += (q > exact[u] || (q == exact[u] && f < own[u].e)) ? 1 : 0;
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (lane + 32 * u < n && rank[u] < k) {
                    s_win[warp][rank[u]] = own[u].e;
                    s_win_l[warp][rank[u]] = own[u].l;
                }
        }
        __syncwarp();
        e = s_win[warp][lane];
        l[0] = s_win_l[warp][lane];
    }
    float w;
    if (a.normalize) {
        w = l[0];
        const float sum = slot_scores(w, a.sigmoid != 0);
        w = sum > 0.0f ? w / sum : 0.0f;
    } else if (a.sigmoid) {
        w = e >= 0 ? sigmoid_of(l[0]) : 0.0f;
    } else {
        float top = -INFINITY, sum = 0.0f;           // (no bias goes with softmax: v are the logits)
#pragma unroll
        for (int c = 0; c < N; ++c) top = fmaxf(top, open_logit(v[c]));
        top = warp_max(top);
        if (top > -INFINITY)
#pragma unroll
            for (int c = 0; c < N; ++c) sum += fast_exp(open_logit(v[c]) - top);
        sum = warp_sum(sum);
        w = e >= 0 ? fast_exp(l[0] - top) / sum : 0.0f;
    }
    if (lane < k) {
        a.idx[t * k + lane] = e;
        a.gates[t * k + lane] = a.scale * w;
    }
}

// ------------------------------------------------------------------ sequences
// Borders of the sequences, kept inside the rows.
__device__ __forceinline__ int64_t border(const int32_t* seq, int s, int S, int64_t T) {
    if (!seq) return s == 0 ? 0 : T;
    return min(max(static_cast<int64_t>(seq[s]), static_cast<int64_t>(0)), T);
}

// The sequence that row t is in, -1: in none.  32 borders at a time.
__device__ __forceinline__ int sequence_of(const int32_t* seq, int S, int64_t T, int64_t t, int lane) {
    if (!seq) return 0;
    // number of sequences that end at or before t
    int lo = 0, hi = S;
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int at = min(lo + (lane + 1) * step, hi) - 1;            // last sequence of the lane's part
        const uint32_t over = __ballot_sync(kAll, border(seq, at + 1, S, T) > t);
        if (over == 0) {
            lo = hi;
        } else {
            const int part = __ffs(over) - 1;
            const int first = lo + part * step, last = min(first + step, hi) - 1;
            lo = first;
            hi = last;                   // the last one ends behind t: the answer is at most its number
        }
    }
    return lo < S && border(seq, lo, S, T) <= t ? lo : -1;
}

// ------------------------------------------------------------------ balance
// Block b takes the tokens [b per, (b + 1) per).  Its warps add up their
// tokens' shares in registers; at the end of each sequence inside the block the
// warps' sums are added in shared memory, and the block's part of the sequence
// goes to row b + s of the workspace: both numbers only grow along the tokens,
// so that no two parts share a row.  A cluster of eight CTAs for each sequence
// then adds its parts, each CTA an eighth of the experts, however short the sequence
// is: 16,384 rows of 896 in bf16 take 19 us in one sequence, 21 in 9, 40 in 64, 279 in
// 1,000.
//
// A warp's rows come through a ring in shared memory, of which a lane copies and
// reads its own words: with a warp's loads and its arithmetic in turn, the loss
// of 16,384 rows of 896 in bf16 took 34 us for 21.
constexpr int kBalCtas = 8;
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__host__ __device__ constexpr int bal_warps(int n) { return n <= 8 ? 24 : n <= 16 ? 16 : 12; }       // of n values a lane: what the registers hold
__host__ __device__ constexpr int bal_depth(int n) { return n <= 8 ? 4 : n <= 16 ? 3 : 2; }
template <int DT, int V, int NI>
__host__ __device__ constexpr int bal_slot() { return V == 8 ? 512 * NI * (DT == ELEM_F32 ? 2 : 1) : 0; }

// A warp's rows t0, t0 + step, ... before `end`: their shares to acc, their slots to hist; the rows that have one.
template <bool SIG, int DT, int V, int NI>
__device__ __forceinline__ int balance_rows(const BalanceArgs& a, int64_t t0, int64_t end, int step, int lane, int32_t* hist,
                                            const uint8_t* rings, float (&acc)[NI * V]) {
    constexpr int N = NI * V, D = bal_depth(NI * V), kSlot = bal_slot<DT, V, NI>();
    const uint32_t ring = smem_u32(rings);
    const int E = a.E, k = a.k;
#pragma unroll
    for (int c = 0; c < N; ++c) acc[c] = 0.0f;
    int used = 0, slot = 0;
    auto fetch = [&](int64_t t, int to) {
        if constexpr (V == 8) {
            if (t < end) {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int e0 = (32 * i + lane) * V;
                    if (e0 >= E) continue;
                    const uint8_t* src = static_cast<const uint8_t*>(a.logits) + (t * a.ld + e0) * (DT == ELEM_F32 ? 4 : 2);
                    const uint32_t dst = ring + static_cast<uint32_t>(to * kSlot + i * (kSlot / NI) + lane * 16);
                    cp_async16(dst, src);
                    if (DT == ELEM_F32) cp_async16(dst + 512, src + 16);
                }
            }
            cp_async_commit();
        }
    };
    int e_next = t0 < end && lane < k ? a.idx[t0 * k + lane] : -1;
#pragma unroll
    for (int d = 0; d < D - 1; ++d) fetch(t0 + d * step, d);
#pragma unroll 1
    for (int64_t t = t0; t < end; t += step) {
        const int e = e_next;
        if (t + step < end && lane < k) e_next = a.idx[(t + step) * k + lane];
        fetch(t + (D - 1) * step, slot == 0 ? D - 1 : slot - 1);
        if constexpr (V == 8) cp_async_wait(D - 1);      // (of rows without a slot too: their words of the ring are copied to again)
        const int from = slot;
        slot = slot + 1 == D ? 0 : slot + 1;
        const bool kept = e >= 0 && e < E;
        if (!__any_sync(kAll, kept)) continue;
        if (kept) atomicAdd(&hist[e], 1);
        ++used;
        float v[N];
        if constexpr (V == 8) {
            RawVec<V> raw[NI];
            const uint8_t* p = rings + from * kSlot + lane * 16;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                raw[i].a = ld16(p + i * (kSlot / NI));
                if (DT == ELEM_F32) raw[i].b = ld16(p + i * (kSlot / NI) + 512);
            }
            open_row<true, V, NI>(raw, E, DT, lane, v);
        } else {
            load_row<DT, true, V, NI>(a.logits, t * a.ld, E, a.dt, lane, v);
        }
        const float sum = scores<SIG>(v);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int c = 0; c < N; ++c) acc[c] = fmaf(v[c], inv, acc[c]);
    }
    return used;
}

template <bool SIG, int DT, int V, int NI>
__global__ void __launch_bounds__(bal_warps(NI * V) * 32, 1) balance_parts_kernel(const BalanceArgs a) {
    constexpr int kBalWarps = bal_warps(NI * V), D = bal_depth(NI * V), kSlot = bal_slot<DT, V, NI>();
    extern __shared__ __align__(16) float s_sum[];       // [kBalWarps][pitch], int32 [pitch] counts, rings [kBalWarps][D][kSlot]
    __shared__ int s_tokens;
    constexpr int N = NI * V;
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E, P = a.pitch;
    int32_t* hist = reinterpret_cast<int32_t*>(s_sum + kBalWarps * P);
    const uint8_t* rings = reinterpret_cast<const uint8_t*>(hist + P) + warp * (D * kSlot);
    const int64_t t0 = blockIdx.x * a.per, t1 = min(t0 + a.per, a.T);
    // the first sequence that ends behind t0 (every warp finds the same)
    int s = 0;
    if (a.seq) {
        int lo = 0, hi = a.S;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (border(a.seq, mid + 1, a.S, a.T) > t0)
                hi = mid;
            else
                lo = mid + 1;
        }
        s = lo;
    }
    for (; s < a.S; ++s) {
        const int64_t first = border(a.seq, s, a.S, a.T);
        if (first >= t1) break;
        const int64_t f = max(first, t0), l = min(border(a.seq, s + 1, a.S, a.T), t1);
        if (l <= f) continue;
        for (int e = threadIdx.x; e < P; e += blockDim.x) hist[e] = 0;
        if (threadIdx.x == 0) s_tokens = 0;
        __syncthreads();
        float acc[N];
        const int used = balance_rows<SIG, DT, V, NI>(a, f + warp, l, kBalWarps, lane, hist, rings, acc);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e0 = (32 * i + lane) * V;
            if (e0 < E)
#pragma unroll
                for (int j = 0; j < V; ++j) s_sum[warp * P + e0 + j] = acc[i * V + j];
        }
        if (lane == 0) atomicAdd(&s_tokens, used);
        __syncthreads();
        float* part = a.part + (blockIdx.x + static_cast<int64_t>(s)) * (2 * P + 4);
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kBalWarps; ++w) sum += s_sum[w * P + e];
            part[e] = sum;
            reinterpret_cast<int32_t*>(part)[P + e] = hist[e];
        }
        if (threadIdx.x == 0) reinterpret_cast<int32_t*>(part)[2 * P] = s_tokens;
        __syncthreads();
    }
}

// Few rows in one launch: a cluster for each sequence, whose CTAs take every eighth row and exchange their sums
// through each other's shared memory.  (A second launch costs a small call's host more than the rows cost the device:
// loss and gradient of 64 rows of 32 experts 35 us a call among others with two launches for the loss, 31 with one; 1,001
// rows of 131 in 13 sequences 7.8 us on the device with two, 4.9 with one.)
constexpr int kSmallRounds = 6;          // rows of a warp at most
constexpr int kSmallSequences = 38;      // two waves of clusters
template <bool SIG, int DT, int V, int NI>
__global__ void __launch_bounds__(bal_warps(NI * V) * 32, 1) balance_small_kernel(const BalanceArgs a) {
    constexpr int kBalWarps = bal_warps(NI * V), D = bal_depth(NI * V), kSlot = bal_slot<DT, V, NI>();
    extern __shared__ __align__(16) float s_sum[];       // as in balance_parts_kernel
    __shared__ int s_tokens;
    __shared__ float s_part[kBalWarps], s_loss[kBalCtas];
    constexpr int N = NI * V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E, P = a.pitch;
    const int rank = blockIdx.x % kBalCtas, s = blockIdx.x / kBalCtas;
    int32_t* hist = reinterpret_cast<int32_t*>(s_sum + kBalWarps * P);
    const uint8_t* rings = reinterpret_cast<const uint8_t*>(hist + P) + warp * (D * kSlot);
    const int64_t first = border(a.seq, s, a.S, a.T), last = border(a.seq, s + 1, a.S, a.T);
    for (int e = threadIdx.x; e < P; e += blockDim.x) hist[e] = 0;
    if (threadIdx.x == 0) s_tokens = 0;
    __syncthreads();
    float acc[N];
    const int used = balance_rows<SIG, DT, V, NI>(a, first + rank + kBalCtas * warp, last, kBalCtas * kBalWarps, lane, hist, rings, acc);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e0 = (32 * i + lane) * V;
        if (e0 < E)
#pragma unroll
            for (int j = 0; j < V; ++j) s_sum[warp * P + e0 + j] = acc[i * V + j];
    }
    if (lane == 0) atomicAdd(&s_tokens, used);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kBalWarps; ++w) sum += s_sum[w * P + e];
        s_sum[e] = sum;
    }
    cluster_sync_all();
    const int per = (E + kBalCtas - 1) / kBalCtas, end = min((rank + 1) * per, E);
    float mine = 0.0f;
    for (int e = rank * per + threadIdx.x; e < end; e += blockDim.x) {
        float x = 0.0f;
        int n = 0;
#pragma unroll
        for (int r = 0; r < kBalCtas; ++r) {
            x += __uint_as_float(ld_cluster(mapa_shared(smem_u32(&s_sum[e]), r)));
            n += static_cast<int>(ld_cluster(mapa_shared(smem_u32(&hist[e]), r)));
        }
        a.counts[static_cast<int64_t>(s) * E + e] = n;
        mine = fmaf(static_cast<float>(n), x, mine);
    }
    mine = warp_sum(mine);
    if (lane == 0) s_part[warp] = mine;
    __syncthreads();
    int n = 0;
    if (threadIdx.x == 0) {
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < kBalWarps; ++w) x += s_part[w];
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&s_loss[rank]), 0)), "f"(x) : "memory");
        if (rank == 0)
            for (int r = 0; r < kBalCtas; ++r) n += static_cast<int>(ld_cluster(mapa_shared(smem_u32(&s_tokens), r)));
    }
    cluster_sync_all();
    if (rank == 0 && threadIdx.x == 0) {
        float x = 0.0f;
        for (int r = 0; r < kBalCtas; ++r) x += s_loss[r];
        const float m = static_cast<float>(max(n, 1));
        a.loss[s] = (static_cast<float>(E) / static_cast<float>(a.k)) * (x / m) / m;
        a.tokens[s] = n;
    }
}

// Experts that a CTA of the sums takes, a multiple of four.
__device__ __forceinline__ int sum_cols(int E) { return ((E + kBalCtas - 1) / kBalCtas + 3) & ~3; }

// The parts are written by the launch that this one overlaps: plain loads.  A warp
// takes four experts a lane of every 32nd part and has its loads of five parts,
// which are those of 152 blocks, in flight at once: the kernel is one latency long.
constexpr int kSumRows = 32, kSumAhead = 5;
__global__ void __launch_bounds__(32 * kSumRows) balance_sum_kernel(const BalanceArgs a) {
    __shared__ __align__(16) float s_sum[kSumRows][128];
    __shared__ __align__(16) int s_cnt[kSumRows][128];
    __shared__ int s_tok[kSumRows];
    __shared__ float s_loss[kBalCtas];
    const int rank = blockIdx.x % kBalCtas, s = blockIdx.x / kBalCtas;
    const int col = (threadIdx.x & 31) * 4, row = threadIdx.x >> 5;
    const int per = sum_cols(a.E);
    const int e0 = rank * per + col;
    const int64_t stride = 2 * a.pitch + 4;
    const int64_t first = border(a.seq, s, a.S, a.T), last = border(a.seq, s + 1, a.S, a.T);
    const int64_t b0 = last > first ? first / a.per : 0, b1 = last > first ? (last - 1) / a.per + 1 : 0;
    cluster_sync_all();                // every CTA runs before its shared memory is written to
    pdl_wait();
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    int4 cnt = make_int4(0, 0, 0, 0);
    int tok = 0;
    if (col < per && e0 < a.pitch) {   // (experts between E and the pitch, a multiple of four, count for nothing)
        for (int64_t b = b0 + row; b < b1; b += kSumRows * kSumAhead) {
            float4 x[kSumAhead];
            int4 c[kSumAhead];
#pragma unroll
            for (int u = 0; u < kSumAhead; ++u) {
                const float* part = a.part + (b + u * kSumRows + s) * stride + e0;
                const bool in = b + u * kSumRows < b1;
                x[u] = in ? *reinterpret_cast<const float4*>(part) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                c[u] = in ? *reinterpret_cast<const int4*>(part + a.pitch) : make_int4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < kSumAhead; ++u) {
                sum = make_float4(sum.x + x[u].x, sum.y + x[u].y, sum.z + x[u].z, sum.w + x[u].w);
                cnt = make_int4(cnt.x + c[u].x, cnt.y + c[u].y, cnt.z + c[u].z, cnt.w + c[u].w);
            }
        }
    }
    for (int64_t b = b0 + threadIdx.x; b < b1; b += blockDim.x)
        tok += reinterpret_cast<const int32_t*>(a.part + (b + s) * stride)[2 * a.pitch];
    tok = __reduce_add_sync(kAll, tok);
    if ((threadIdx.x & 31) == 0) s_tok[threadIdx.x >> 5] = tok;
    *reinterpret_cast<float4*>(&s_sum[row][col]) = sum;
    *reinterpret_cast<int4*>(&s_cnt[row][col]) = cnt;
    __syncthreads();
    if (threadIdx.x < 128) {
        const int c = threadIdx.x, e = rank * per + c;
        float x = 0.0f;
        int n = 0;
#pragma unroll
        for (int r = 0; r < kSumRows; ++r) {
            x += s_sum[r][c];
            n += s_cnt[r][c];
        }
        const bool mine = c < per && e < a.E;
        if (mine) a.counts[static_cast<int64_t>(s) * a.E + e] = n;
        s_sum[0][c] = mine ? static_cast<float>(n) * x : 0.0f;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const float x = warp_sum((s_sum[0][threadIdx.x] + s_sum[0][threadIdx.x + 32]) +
                                 (s_sum[0][threadIdx.x + 64] + s_sum[0][threadIdx.x + 96]));
        if (threadIdx.x == 0) {
            const uint32_t at = mapa_shared(smem_u32(&s_loss[rank]), 0);
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
        }
    }
    cluster_sync_all();
    if (rank == 0 && threadIdx.x == 0) {
        int n = 0;
        for (int w = 0; w < kSumRows; ++w) n += s_tok[w];
        float x = 0.0f;
        for (int r = 0; r < kBalCtas; ++r) x += s_loss[r];
        const float m = static_cast<float>(max(n, 1));
        a.loss[s] = (static_cast<float>(a.E) / static_cast<float>(a.k)) * (x / m) / m;
        a.tokens[s] = n;
    }
}

// ------------------------------------------------------------------ backward
// With shares p, a_e = dL E c_e / (k n^2) and r_e = 1 - sigmoid(l_e) (1 for
// softmax), the loss gives p_e r_e (a_e - sum p a).  With g = scale d_gates and
// the gates w over the winners, the gates give w_j r_j (g_j - sum g w); not
// normalised, g_j s_j r_j, or for the softmax over all p_e ([e won] g_e - sum g p).
// A lane holds slot j = lane; the slots' values meet their experts' lanes in a row
// of shared memory.  One exponential a logit: with u = e^-|l|, sigmoid(l) is {1, u} /
// (1 + u) and sigmoid(l) (1 - sigmoid(l)) = u / (1 + u)^2, which is kept for the second pass.
// (Rows of more than 512 experts by eight values: 96 registers, of which a thread stores 56 to
// 124 bytes to local memory.)
constexpr int kBackWarps = 4;

// Eight (or one) counts as floats.
template <int V>
__device__ __forceinline__ void load_counts(const int32_t* p, bool wide, float (&c)[V]) {
    if constexpr (V == 8) {
        if (wide) {
            const int4 a = *reinterpret_cast<const int4*>(p), b = *(reinterpret_cast<const int4*>(p) + 1);
            c[0] = static_cast<float>(a.x);
            c[1] = static_cast<float>(a.y);
            c[2] = static_cast<float>(a.z);
            c[3] = static_cast<float>(a.w);
            c[4] = static_cast<float>(b.x);
            c[5] = static_cast<float>(b.y);
            c[6] = static_cast<float>(b.z);
            c[7] = static_cast<float>(b.w);
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) c[j] = static_cast<float>(p[j]);
}

template <bool SIG, int DT, int V, int NI>
__global__ void __launch_bounds__(kBackWarps * 32, 5) router_backward_kernel(const RouterBackArgs a) {
    extern __shared__ __align__(16) float s_rows[];      // [kBackWarps][pitch]
    constexpr int N = NI * V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kBackWarps + warp;
    if (t >= a.T) return;
    const int E = a.E, k = a.k;
    float* srow = s_rows + warp * a.pitch;
    const bool all = !SIG && !a.normalize && a.d_gates;          // gates by the softmax over all
    // (all that has no need of another load's value is asked for first)
    RawVec<V> raw[NI];
    if (a.d_loss || all) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e0 = (32 * i + lane) * V;
            if (e0 < E) raw[i] = load_raw<V>(a.logits, t * a.ld + e0, DT >= 0 ? DT : a.dt);
        }
    }
    int e = lane < k ? a.idx[t * k + lane] : -1;
    int s = a.d_loss ? sequence_of(a.seq, a.S, a.T, t, lane) : -1;
    if (e < 0 || e >= E) e = -1;
    const bool any = __any_sync(kAll, e >= 0);
    if (!any) s = -1;
    float x[N], ac[N];                                   // x: p r as multiples of 1 / inv; ac: a_e
    float inv = 0.0f, top = -INFINITY, inner = 0.0f;
    const bool shared = any && (s >= 0 || all);
    if (shared) {
        if (s >= 0) {
            const bool wide = E % 4 == 0 && (reinterpret_cast<uintptr_t>(a.counts) & 15) == 0;
            const float n = static_cast<float>(max(a.tokens[s], 1));
            const float f = a.d_loss[s] * (static_cast<float>(E) / static_cast<float>(k)) / n / n;
            const int32_t* cnt = a.counts + static_cast<int64_t>(s) * E;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e0 = (32 * i + lane) * V;
                float ct[V];
#pragma unroll
                for (int j = 0; j < V; ++j) ct[j] = 0.0f;
                if (e0 < E) load_counts<V>(cnt + e0, wide, ct);
#pragma unroll
                for (int j = 0; j < V; ++j) ac[i * V + j] = f * ct[j];
            }
        } else {
#pragma unroll
            for (int c = 0; c < N; ++c) ac[c] = 0.0f;
        }
        open_row<true, V, NI>(raw, E, DT >= 0 ? DT : a.dt, lane, x);
#pragma unroll
        for (int c = 0; c < N; ++c) top = fmaxf(top, x[c]);
        top = warp_max(top);
        float sum = 0.0f;
        if (top == -INFINITY) {
#pragma unroll
            for (int c = 0; c < N; ++c) x[c] = 0.0f;
        } else if (!SIG) {
#pragma unroll
            for (int c = 0; c < N; ++c) {
                x[c] = fast_exp(x[c] - top);
                sum += x[c];
                inner = fmaf(x[c], ac[c], inner);
            }
        } else if (top >= 0.0f) {
#pragma unroll
            for (int c = 0; c < N; c += 4) {
                float u[4], d[4], q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u[j] = fast_exp(-fabsf(x[c + j]));
                    d[j] = 1.0f + u[j];
                }
                rcp4(d, q);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float z = u[j] * q[j], y = x[c + j] >= 0.0f ? q[j] : z;
                    x[c + j] = z * q[j];
                    sum += y;
                    inner = fmaf(y, ac[c + j], inner);
                }
            }
        } else {
#pragma unroll
            for (int c = 0; c < N; ++c) {
                const float q = fast_rcp(1.0f + fast_exp(x[c]));
                const float y = fast_exp(x[c] - top) * q;
                x[c] = y * q;                            // with 1 - s = q
                sum += y;
                inner = fmaf(y, ac[c], inner);
            }
        }
        sum = warp_sum(sum);
        inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        inner = warp_sum(inner) * inv;
    }
    float shift = 0.0f;                                  // what is taken from every share
    const bool gates = a.d_gates && any;
    if (gates) {
        float l = -INFINITY, g = 0.0f;
        if (e >= 0) {
            float q[1];
            raw_to_f32(load_raw<1>(a.logits, t * a.ld + e, a.dt), a.dt, q);
            l = open_logit(q[0]);
            if (l > -INFINITY) g = a.scale * a.d_gates[t * k + lane];     // (0 times what stands there could be NaN)
        }
        float val;
        if (a.normalize) {
            float w = l;
            const float sum = slot_scores(w, SIG);
            w = sum > 0.0f ? w / sum : 0.0f;
            val = w * (g - warp_sum(w * g));
            if (SIG) val *= sigmoid_rest(l);
        } else if (SIG) {
            val = g * sigmoid_of(l) * sigmoid_rest(l);
        } else {
            val = l > -INFINITY ? g * fast_exp(l - top) * inv : 0.0f;
            shift = warp_sum(val);
        }
        if (l == -INFINITY) val = 0.0f;
        for (int c = lane * 4; c < a.pitch; c += 128) *reinterpret_cast<float4*>(srow + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        __syncwarp();
        const uint32_t same = __match_any_sync(kAll, e);
        if (__any_sync(kAll, e >= 0 && (same & (same - 1)))) {
            for (int j = 0; j < k; ++j) {                // an expert named twice: slots in turn
                if (lane == j && e >= 0) srow[e] += val;
                __syncwarp();
            }
        } else if (e >= 0) {
            srow[e] = val;
        }
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e0 = (32 * i + lane) * V;
        float o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = 0.0f;
        if (gates && e0 < E) {
            if constexpr (V == 8) {
                const float4 p = *reinterpret_cast<const float4*>(srow + e0), q = *reinterpret_cast<const float4*>(srow + e0 + 4);
                o[0] = p.x;
                o[1] = p.y;
                o[2] = p.z;
                o[3] = p.w;
                o[4] = q.x;
                o[5] = q.y;
                o[6] = q.z;
                o[7] = q.w;
            } else {
                o[0] = srow[e0];
            }
        }
        if (shared) {
            // p r (a - inner), and for gates by the softmax over all -p shift
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = i * V + j;
                o[j] = fmaf(x[c] * inv, ac[c] - (inner + shift), o[j]);
            }
        }
        if (e0 < E) store_vec(a.d_logits, t * a.ld_d + e0, DT >= 0 ? DT : a.dt, o);
    }
}

// Whether rows go by eight values at a time.
bool rows_wide(const void* p, int64_t ld, int dt, int E) {
    return E % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * elem_bytes(dt)) % 16 == 0;
}

// RUN(SIG, DT, V, NI) with the type and the fewest registers that hold E values a warp.
#define MOE_ROW_FORMS_OF(RUN, SIG, wide, dt, E)            \
    do {                                                   \
        if (!(wide)) {                                     \
            if ((E) <= 256) return RUN(SIG, -1, 1, 8);     \
            return RUN(SIG, -1, 1, 32);                    \
        }                                                  \
        if ((dt) == ELEM_F32) MOE_ROW_WIDE(RUN, SIG, ELEM_F32, E);   \
        if ((dt) == ELEM_BF16) MOE_ROW_WIDE(RUN, SIG, ELEM_BF16, E); \
        MOE_ROW_WIDE(RUN, SIG, ELEM_F16, E);               \
    } while (0)
#define MOE_ROW_WIDE(RUN, SIG, DT, E)                      \
    do {                                                   \
        if ((E) <= 256) return RUN(SIG, DT, 8, 1);         \
        if ((E) <= 512) return RUN(SIG, DT, 8, 2);         \
        return RUN(SIG, DT, 8, 4);                         \
    } while (0)
#define MOE_ROW_FORMS(RUN, sigmoid, wide, dt, E)           \
    if (sigmoid) MOE_ROW_FORMS_OF(RUN, true, wide, dt, E); \
    MOE_ROW_FORMS_OF(RUN, false, wide, dt, E)

int64_t balance_per(int64_t T) {
    const int64_t per = (T + 151) / 152;
    return std::max<int64_t>(per, 1);
}

template <bool SIG, int DT, int V, int NI>
cudaError_t balance_as(const BalanceArgs& a, cudaStream_t s) {
    if (a.T > 0) {
        const unsigned blocks = static_cast<unsigned>((a.T + a.per - 1) / a.per);
        constexpr int kBalWarps = bal_warps(NI * V), kRings = kBalWarps * bal_depth(NI * V) * bal_slot<DT, V, NI>();
        const size_t smem = sizeof(float) * static_cast<size_t>(kBalWarps + 1) * a.pitch + kRings;
        if (a.T <= kSmallRounds * kBalCtas * kBalWarps && a.S <= kSmallSequences) {
            if (smem > 48 * 1024 - 256) {
                const cudaError_t err = cudaFuncSetAttribute(balance_small_kernel<SIG, DT, V, NI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                             static_cast<int>(sizeof(float) * (kBalWarps + 1) * 32 * V * NI) + kRings);
                if (err != cudaSuccess) return err;
            }
            return launch_ex_cluster(balance_small_kernel<SIG, DT, V, NI>, dim3(static_cast<unsigned>(a.S) * kBalCtas), dim3(kBalWarps * 32), smem, s,
                                     false, kBalCtas, a);
        }
        if (smem > 48 * 1024 - 256) {
            const cudaError_t err = cudaFuncSetAttribute(balance_parts_kernel<SIG, DT, V, NI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                         static_cast<int>(sizeof(float) * (kBalWarps + 1) * 32 * V * NI) + kRings);
            if (err != cudaSuccess) return err;
        }
        balance_parts_kernel<SIG, DT, V, NI><<<blocks, kBalWarps * 32, smem, s>>>(a);
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess) return err;
    }
    return launch_ex_cluster(balance_sum_kernel, dim3(static_cast<unsigned>(a.S) * kBalCtas), dim3(32 * kSumRows), 0, s, a.T > 0, kBalCtas, a);
}

}  // namespace

size_t balance_workspace_bytes(int64_t T, int E, int S) {
    if (T == 0) return 0;
    const int64_t per = balance_per(T), blocks = (T + per - 1) / per;
    return sizeof(float) * static_cast<size_t>(blocks + S) * static_cast<size_t>(2 * ((E + 3) & ~3) + 4);
}

cudaError_t launch_select(const SelectArgs& a, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    const unsigned blocks = static_cast<unsigned>((a.T + kSelectWarps - 1) / kSelectWarps);
#define MOE_RUN(SIG, DT, V, NI) (select_kernel<DT, V, NI><<<blocks, kSelectWarps * 32, 0, s>>>(a), cudaGetLastError())
    MOE_ROW_FORMS_OF(MOE_RUN, , rows_wide(a.logits, a.ld, a.dt, a.E) && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0, a.dt, a.E);
#undef MOE_RUN
}

cudaError_t launch_balance(BalanceArgs a, cudaStream_t s) {
    a.per = balance_per(a.T);
    a.pitch = (a.E + 3) & ~3;
#define MOE_RUN(SIG, DT, V, NI) balance_as<SIG, DT, V, NI>(a, s)
    MOE_ROW_FORMS(MOE_RUN, a.sigmoid, rows_wide(a.logits, a.ld, a.dt, a.E), a.dt, a.E);
#undef MOE_RUN
}

cudaError_t launch_router_backward(RouterBackArgs a, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    a.pitch = (a.E + 3) & ~3;
    const unsigned blocks = static_cast<unsigned>((a.T + kBackWarps - 1) / kBackWarps);
    const size_t smem = a.d_gates ? sizeof(float) * kBackWarps * static_cast<size_t>(a.pitch) : 0;
#define MOE_RUN(SIG, DT, V, NI) (router_backward_kernel<SIG, DT, V, NI><<<blocks, kBackWarps * 32, smem, s>>>(a), cudaGetLastError())
    MOE_ROW_FORMS(MOE_RUN, a.sigmoid, rows_wide(a.logits, a.ld, a.dt, a.E) && rows_wide(a.d_logits, a.ld_d, a.dt, a.E), a.dt, a.E);
#undef MOE_RUN
}

}  // namespace moe
