// route_scores.cu -- routing rules on given logits (sigmoid or softmax scores, a balance bias that
// takes part in the choice only, expert groups, top-k, renormalised weights) and their gradient.
//
// One warp per token; lane l holds the experts l + 32 i in registers (i < NV, E <= 32 NV <= 1024).
//
// The choice is the one that 64-bit arithmetic makes.  Without a bias the scores are monotone in the
// logits, so the logits themselves are ranked and nothing is rounded.  With a bias (and for the sums of
// a group's two best) the ranking values are computed in fp32 with a bound on their error; where the
// value kept last and the value left out first are closer than twice that bound, the values that could
// stand on either side are computed again in 64 bits and ordered there.  fp64 runs at about two
// operations per clock and SM on this GPU, so ranking everything in fp64 is out of the question: the
// bound leaves a handful of values in a prompt of thousands of tokens.  Ties go to the lower id.
#include "ops.cuh"
#include "route_common.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRouteWarps = 8;    // tokens per CTA
constexpr uint32_t kOutKey = 1u;  // ranks an expert out of service: below every logit's key, above "not a candidate" (0)
constexpr float kMaxF32 = 3.402823466e38f;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// A logit of -inf (or NaN) takes its expert out of service; +inf scores like the largest finite number.
__device__ __forceinline__ bool in_service(float l) { return l > -INFINITY; }
__device__ __forceinline__ float clamp_logit(float l) { return fminf(l, kMaxF32); }

__device__ __forceinline__ float sigmoid_f32(float l) { return 1.f / (1.f + expf(-l)); }
__device__ __forceinline__ double sigmoid_f64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(kFull, v, m);
    return v;
}
__device__ __forceinline__ float warp_max_f32(float v) { return key_logit(__reduce_max_sync(kFull, logit_key(v))); }

// The softmax of a row needs its largest logit and the sum of exp(l - max); unused for sigmoid scores.
struct RowNorm {
    float max, inv_sum;
};

template <int NV>
__device__ __forceinline__ RowNorm softmax_norm(const float (&l)[NV]) {
    float m = -kMaxF32;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in_service(l[i])) m = fmaxf(m, clamp_logit(l[i]));
    m = warp_max_f32(m);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in_service(l[i])) sum += expf(clamp_logit(l[i]) - m);
    sum = warp_butterfly_sum(sum);
    return {m, sum > 0.f ? 1.f / sum : 0.f};
}

__device__ __forceinline__ float score_f32(float l, bool softmax, const RowNorm& n) {
    if (!in_service(l)) return 0.f;
    return softmax ? expf(clamp_logit(l) - n.max) * n.inv_sum : sigmoid_f32(l);
}

// A picked score as a ratio to exp(ref), for renormalised weights: ref is the largest picked logit
// (sigmoid: at most 0, where exp(l) and the score part), so that a row of tiny scores keeps its ratios.
__device__ __forceinline__ float score_ratio(float l, bool softmax, float ref) {
    if (!in_service(l)) return 0.f;
    if (softmax) return expf(clamp_logit(l) - ref);
    return l > 0.f ? sigmoid_f32(l) : expf(l - ref) / (1.f + expf(l));
}

// Group of an expert: e / S as a product, exact for e < 1024 (its error e / 2^20 stays below 1 / S).
struct GroupOf {
    uint32_t mul;
    __device__ explicit GroupOf(int S) : mul(((1u << 20) + S - 1) / S) {}
    __device__ __forceinline__ int operator()(int e) const { return (int)(((uint32_t)e * mul) >> 20); }
};

// The two largest of a stream of values.
template <typename F>
struct Top2 {
    F a, b;
    __device__ __forceinline__ void add(F v) {
        if (v > a) {
            b = a;
            a = v;
        } else if (v > b) {
            b = v;
        }
    }
    __device__ __forceinline__ void merge(int xor_lane) {
        const F oa = __shfl_xor_sync(kFull, a, xor_lane), ob = __shfl_xor_sync(kFull, b, xor_lane);
        add(oa);
        add(ob);
    }
    // sum of the (up to) two best, or the best alone
    __device__ __forceinline__ F score(bool top2) const { return (top2 && b > -INFINITY) ? a + b : a; }
};

// 2^shift lanes share an expert group: as many as G groups leave to each.
__device__ __forceinline__ int group_lane_shift(int G) { return G <= 1 ? 5 : G <= 2 ? 4 : G <= 4 ? 3 : G <= 8 ? 2 : G <= 16 ? 1 : 0; }

// Score of group lane >> sh from values val[e] (-inf: out of service); every lane of the group gets it.
template <typename F>
__device__ __forceinline__ F group_score(const F* val, int G, int S, int sh, bool top2) {
    const int lane = threadIdx.x & 31, g = lane >> sh, lp = 1 << sh;
    Top2<F> t{(F)-INFINITY, (F)-INFINITY};
    if (g < G)
        for (int j = lane & (lp - 1); j < S; j += lp) t.add(val[g * S + j]);
    for (int m = 1; m < lp; m <<= 1) t.merge(m);
    return t.score(top2);
}

// Bit g of the result: group g is among the `keep` best of the candidate groups (ties to the lower group).
template <typename F>
__device__ __forceinline__ uint32_t best_groups(F score, uint32_t cand, int G, int sh, int keep) {
    const int lane = threadIdx.x & 31, g = lane >> sh;
    int before = 0;
    for (int j = 0; j < G; ++j) {
        const F o = __shfl_sync(kFull, score, j << sh);
        if ((cand >> j) & 1) before += (o > score || (o == score && j < g)) ? 1 : 0;
    }
    const bool in = g < G && ((cand >> g) & 1) && before < keep;
    const uint32_t lanes = __ballot_sync(kFull, in);
    uint32_t mask = 0;
    for (int j = 0; j < G; ++j) mask |= ((lanes >> (j << sh)) & 1u) << j;
    return mask;
}

template <int NV, typename T>
__global__ void __launch_bounds__(32 * kRouteWarps) route_scores_kernel(const RouteScoresArgs a) {
    extern __shared__ double scratch[];  // per warp E values, where the rule has groups or a bias
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    const int E = a.E, k = a.k, G = a.rule.groups;
    const bool softmax = a.rule.score == MOE_SCORE_SOFTMAX, biased = a.bias != nullptr;
    const bool top2 = a.rule.group_score == MOE_GROUP_TOP2;
    double* v64 = scratch + (size_t)warp * E;

    float l[NV];
    const T* row = static_cast<const T*>(a.logits) + (int64_t)t * a.ld;
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = lane + 32 * i < E ? to_f32(row[lane + 32 * i]) : -INFINITY;
    RowNorm norm = {0.f, 0.f};
    if (softmax) norm = softmax_norm<NV>(l);

    // Ranking values and the bound on the error of a difference of two of them.  fp32 sigmoid: expf and
    // a division are within 2^-22 of it; softmax: the sum's (NV + 16) roundings dominate, relative to the
    // row's largest score; the sum with the bias rounds once more.
    float v[NV];
    float vmax = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        v[i] = l[i];
        if (biased) {
            v[i] = in_service(l[i]) ? score_f32(l[i], softmax, norm) + __ldg(a.bias + e) : -INFINITY;
            if (in_service(l[i])) vmax = fmaxf(vmax, fabsf(v[i]));
        }
        if (e < E && a.scores) a.scores[(int64_t)t * E + e] = score_f32(l[i], softmax, norm);
    }
    const float err_s = softmax ? (float)(NV + 16) * 1.1920929e-7f * norm.inv_sum : 9.5367432e-7f;
    float err = 0.f;
    if (biased) err = err_s + 4.7683716e-7f * warp_max_f32(vmax);

    double norm64 = 0.0;  // 1 / sum exp(l - max) in 64 bits, computed when a choice needs it
    auto exact_value = [&](float lv, int e) -> double {
        double s = softmax ? exp((double)clamp_logit(lv) - (double)norm.max) * norm64 : sigmoid_f64(lv);
        if (biased) s += (double)__ldg(a.bias + e);
        return s;
    };
    auto need_exact = [&]() {
        if (!softmax || norm64 != 0.0) return;
        double sum = 0.0;
#pragma unroll 1
        for (int i = 0; i < NV; ++i) {
            const float lv = lane + 32 * i < E ? to_f32(row[lane + 32 * i]) : -INFINITY;
            if (in_service(lv)) sum += exp((double)clamp_logit(lv) - (double)norm.max);
        }
        norm64 = 1.0 / warp_sum_f64(sum);
    };

    // ---------------------------------------------------------------- groups
    uint32_t kept = 0xffffffffu;
    const int S = E / G;
    const GroupOf group_of(S);
    if (G > 1 && a.rule.top_groups < G) {
        const int sh = group_lane_shift(G), keep = a.rule.top_groups;
        const bool raw = !biased && !top2;  // the groups' best logits: exact
        float* vs = reinterpret_cast<float*>(v64);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 32 * i < E)
                vs[lane + 32 * i] = (biased || raw) ? v[i] : in_service(l[i]) ? score_f32(l[i], softmax, norm) : -INFINITY;
        __syncwarp();
        const float gs = group_score<float>(vs, G, S, sh, top2);
        const uint32_t all = G == 32 ? kFull : (1u << G) - 1;
        kept = best_groups<float>(gs, all, G, sh, keep);
        if (!raw) {
            const int g = lane >> sh;
            const bool mine = g < G && gs > -INFINITY;
            const bool in = g < G && ((kept >> g) & 1);
            const float lo = warp_max_f32(mine && !in ? gs : -INFINITY);   // best left out
            const float hi = -warp_max_f32(mine && in ? -gs : -INFINITY);  // worst kept
            const float gerr = 2.f * (biased ? err : err_s) + 4.7683716e-7f * fmaxf(fabsf(lo), fabsf(hi));
            if (lo > -INFINITY && hi < INFINITY && hi - lo <= gerr) {
                need_exact();
                const uint32_t lanes = __ballot_sync(kFull, mine && gs >= hi - gerr && gs <= lo + gerr);
                const uint32_t sure = __ballot_sync(kFull, mine && gs > lo + gerr);
                uint32_t open = 0, in_mask = 0;
                for (int j = 0; j < G; ++j) {
                    open |= ((lanes >> (j << sh)) & 1u) << j;
                    in_mask |= ((sure >> (j << sh)) & 1u) << j;
                }
                __syncwarp();
#pragma unroll 1
                for (int i = 0; i < NV; ++i) {
                    const int e = lane + 32 * i;
                    if (e >= E || !((open >> group_of(e)) & 1)) continue;
                    const float lv = to_f32(row[e]);
                    v64[e] = in_service(lv) ? exact_value(lv, e) : -(double)INFINITY;
                }
                __syncwarp();
                const bool is_open = g < G && ((open >> g) & 1);
                const double gx = group_score<double>(v64, is_open ? G : 0, S, sh, top2);
                kept = in_mask | best_groups<double>(gx, open, G, sh, keep - __popc(in_mask));
            }
        }
    }

    // ---------------------------------------------------------------- top-k: the k-th key and who ties with it
    uint32_t key[NV];
    uint32_t chosen = 0;  // bit i: expert lane + 32 i is picked
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        const bool cand = e < E && (G == 1 || ((kept >> group_of(e)) & 1));
        // (a NaN value comes from a NaN bias: ranked like an expert out of service)
        key[i] = !cand ? 0u : in_service(l[i]) && v[i] == v[i] ? logit_key(v[i]) : kOutKey;
    }
    uint32_t last = 0, next = 0;  // key of the pick that completes the k, largest key left out
    int above = 0;                // picks with a larger key than `last`
    {
        uint32_t gone = 0;
        int n = 0;
        while (true) {
            uint32_t lb = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (!((gone >> i) & 1)) lb = max(lb, key[i]);
            const uint32_t wb = __reduce_max_sync(kFull, lb);
            if (n >= k) {
                next = n > k ? last : wb;
                break;
            }
            if (wb != last) above = n;
            last = wb;
            n += __popc(__ballot_sync(kFull, lb == wb));
            if (lb == wb) {
                bool done = false;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (!done && !((gone >> i) & 1) && key[i] == wb) {
                        gone |= 1u << i;
                        done = true;
                    }
            }
        }
    }
    const bool close = biased && last > kOutKey && next > kOutKey && key_logit(last) - key_logit(next) <= err;
    if (!close) {
        int ties = k - above;  // how many of the experts at `last` are picked, lowest ids first
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (key[i] > last) chosen |= 1u << i;
            const uint32_t tie = __ballot_sync(kFull, key[i] == last);
            if (key[i] == last && __popc(tie & ((1u << lane) - 1)) < ties) chosen |= 1u << i;
            ties -= __popc(tie);
        }
    } else {
        need_exact();
        const float top = key_logit(next) + err, bottom = key_logit(last) - err;
        uint32_t open = 0;
        int sure = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (key[i] <= kOutKey) continue;
            const float x = key_logit(key[i]);
            if (x > top) {
                chosen |= 1u << i;
                ++sure;
            } else if (x >= bottom) {
                open |= 1u << i;
            }
        }
        sure = __reduce_add_sync(kFull, sure);
        __syncwarp();
        // the open experts' values, in id order (NaN elsewhere: compares false)
#pragma unroll 1
        for (int i = 0; i < NV; ++i) {
            const int e = lane + 32 * i;
            if (e < E) v64[e] = ((open >> i) & 1) ? exact_value(to_f32(row[e]), e) : nan("");
        }
        __syncwarp();
        uint32_t rest = open;
        while (rest) {
            const int i = __ffs(rest) - 1;
            rest &= rest - 1;
            const int e = lane + 32 * i;
            const double mine = v64[e];
            int before = sure;
            for (int j = 0; j < E; ++j) before += (v64[j] > mine || (v64[j] == mine && j < e)) ? 1 : 0;
            if (before < k) chosen |= 1u << i;
        }
        __syncwarp();
    }

    // ---------------------------------------------------------------- weights of the picks, in id order
    const bool renorm = a.rule.renormalize != 0;
    float ref = 0.f;
    if (renorm) {
        float m = -kMaxF32;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (((chosen >> i) & 1) && in_service(l[i])) m = fmaxf(m, clamp_logit(l[i]));
        ref = warp_max_f32(m);
        if (!softmax) ref = fminf(ref, 0.f);
    }
    float u[NV];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        u[i] = 0.f;
        if (!((chosen >> i) & 1)) continue;
        u[i] = renorm ? score_ratio(l[i], softmax, ref) : score_f32(l[i], softmax, norm);
        sum += u[i];
    }
    float scale = a.rule.scale;
    if (renorm) {
        sum = warp_butterfly_sum(sum);
        scale = sum > 0.f ? scale / sum : 0.f;
    }
    int base = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool in = (chosen >> i) & 1;
        const uint32_t who = __ballot_sync(kFull, in);
        if (in) {
            const int at = base + __popc(who & ((1u << lane) - 1));
            a.ids[(int64_t)t * k + at] = lane + 32 * i;
            a.w[(int64_t)t * k + at] = u[i] * scale;
            if (a.counts) atomicAdd(a.counts + lane + 32 * i, 1);
        }
        base += __popc(who);
    }
}

// Gradient of the logits from the gradient of the weights (and, optionally, of all the scores).
// u_j: the picked scores, c the rule's factor.  Renormalised: du_j = c (dw_j - sum_i dw_i u_i / S) / S with
// S = sum u (taken in ratios to the largest score, as above), else du_j = c dw_j.  Sigmoid: dl = ds s (1 - s), with
// 1 - s = sigmoid(-l).  Softmax: dl = s (ds - sum ds s); with renormalised weights and no other gradient of
// the scores that sum is zero by itself and only the picked experts get a gradient.
template <int NV, typename T>
__global__ void __launch_bounds__(32 * kRouteWarps) route_scores_backward_kernel(const RouteBackwardArgs a) {
    extern __shared__ float rows[];  // per warp: the gradient of the scores [E], times the scores
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    const int E = a.E, k = a.k;
    const bool softmax = a.rule.score == MOE_SCORE_SOFTMAX, renorm = a.rule.renormalize != 0;
    float* ds = rows + (size_t)warp * E;
    const T* row = static_cast<const T*>(a.logits) + (int64_t)t * a.ld;
    T* out = static_cast<T*>(a.dlogits) + (int64_t)t * a.ldd;

    float l[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < E ? to_f32(row[e]) : -INFINITY;
        if (e < E) ds[e] = 0.f;
    }
    RowNorm norm = {0.f, 0.f};
    if (softmax) norm = softmax_norm<NV>(l);
    __syncwarp();

    // lane j < k: pick j; g = u_j du_j, the product that the logits' gradient needs
    const int id = lane < k ? a.ids[(int64_t)t * k + lane] : -1;
    const bool valid = id >= 0 && id < E;
    const float lp = valid ? to_f32(row[id]) : -INFINITY;
    const float dw = valid && in_service(lp) ? a.dw[(int64_t)t * k + lane] * a.rule.scale : 0.f;
    float g = 0.f;
    if (renorm) {
        float ref = warp_max_f32(in_service(lp) ? clamp_logit(lp) : -kMaxF32);
        if (!softmax) ref = fminf(ref, 0.f);
        const float u = score_ratio(lp, softmax, ref);
        const float S = warp_butterfly_sum(u);
        const float r = S > 0.f ? u / S : 0.f;
        g = r * (dw - warp_butterfly_sum(dw * r));
    } else {
        g = dw * score_f32(lp, softmax, norm);
    }
    if (valid) ds[id] = g;
    __syncwarp();
    float total = 0.f;  // softmax: sum of ds s over all experts
    float gs[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        gs[i] = 0.f;
        if (e >= E) continue;
        gs[i] = ds[e];
        float extra = 0.f;
        if (a.dscores && in_service(l[i])) extra = a.dscores[(int64_t)t * E + e] * score_f32(l[i], softmax, norm);
        if (!renorm) total += gs[i];
        total += extra;
        gs[i] += extra;
    }
    if (softmax && (!renorm || a.dscores)) total = warp_butterfly_sum(total);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        if (e >= E) continue;
        float dl = 0.f;
        if (in_service(l[i])) dl = softmax ? gs[i] - score_f32(l[i], true, norm) * total : gs[i] * sigmoid_f32(-l[i]);
        out[e] = from_f32<T>(dl);
    }
}

template <typename T>
const void* scores_kernel(int E) {
    const int nv = (E + 31) / 32;
    return nv <= 1    ? (const void*)route_scores_kernel<1, T>
           : nv <= 2  ? (const void*)route_scores_kernel<2, T>
           : nv <= 4  ? (const void*)route_scores_kernel<4, T>
           : nv <= 8  ? (const void*)route_scores_kernel<8, T>
           : nv <= 16 ? (const void*)route_scores_kernel<16, T>
                      : (const void*)route_scores_kernel<32, T>;
}

template <typename T>
const void* backward_kernel(int E) {
    const int nv = (E + 31) / 32;
    return nv <= 1    ? (const void*)route_scores_backward_kernel<1, T>
           : nv <= 2  ? (const void*)route_scores_backward_kernel<2, T>
           : nv <= 4  ? (const void*)route_scores_backward_kernel<4, T>
           : nv <= 8  ? (const void*)route_scores_backward_kernel<8, T>
           : nv <= 16 ? (const void*)route_scores_backward_kernel<16, T>
                      : (const void*)route_scores_backward_kernel<32, T>;
}

}  // namespace

cudaError_t launch_route_scores(const RouteScoresArgs& a, moe_dtype dtype, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const void* f = dtype == MOE_F32    ? scores_kernel<float>(a.E)
                    : dtype == MOE_BF16 ? scores_kernel<__nv_bfloat16>(a.E)
                                        : scores_kernel<__half>(a.E);
    const size_t smem = a.bias || a.rule.groups > 1 ? sizeof(double) * kRouteWarps * (size_t)a.E : 0;
    void* args[] = {const_cast<RouteScoresArgs*>(&a)};
    return launch_kernel(f, dim3((a.T + kRouteWarps - 1) / kRouteWarps), dim3(32 * kRouteWarps), smem, st, false, args);
}

cudaError_t launch_route_scores_backward(const RouteBackwardArgs& a, moe_dtype dtype, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const void* f = dtype == MOE_F32    ? backward_kernel<float>(a.E)
                    : dtype == MOE_BF16 ? backward_kernel<__nv_bfloat16>(a.E)
                                        : backward_kernel<__half>(a.E);
    void* args[] = {const_cast<RouteBackwardArgs*>(&a)};
    return launch_kernel(f, dim3((a.T + kRouteWarps - 1) / kRouteWarps), dim3(32 * kRouteWarps),
                         sizeof(float) * kRouteWarps * (size_t)a.E, st, false, args);
}

}  // namespace moe
