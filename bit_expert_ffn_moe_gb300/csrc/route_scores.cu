// route_scores.cu -- routing rules on given logits (sigmoid or softmax scores, a balance bias that
// takes part in the choice only, expert groups, top-k, renormalised weights) and their gradient.
//
// One warp per token; lane l holds the experts NV l .. NV l + NV - 1 in registers (E <= 32 NV <= 1024).
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
// Largest value of the warp (NaN ignored unless every lane has one).
__device__ __forceinline__ float warp_max_f32(float v) {
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

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
// Sigmoid: exp(min(l, 0) - ref) / (1 + exp(-|l|)), for ref = 0 wherever l > 0.
__device__ __forceinline__ float score_ratio(float l, bool softmax, float ref) {
    if (!in_service(l)) return 0.f;
    if (softmax) return expf(clamp_logit(l) - ref);
    return __fdividef(expf(fminf(l, 0.f) - ref), 1.f + expf(-fabsf(l)));
}

// Group of an expert: e / S as a product with mul = ceil(2^20 / S), exact for e < 1024 (its error e / 2^20 stays
// below 1 / S).
struct GroupOf {
    uint32_t mul;
    __device__ __forceinline__ int operator()(int e) const { return (int)(((uint32_t)e * mul) >> 20); }
};

__device__ __forceinline__ float larger(float x, float y) { return fmaxf(x, y); }
__device__ __forceinline__ float smaller(float x, float y) { return fminf(x, y); }
__device__ __forceinline__ double larger(double x, double y) { return x > y ? x : y; }
__device__ __forceinline__ double smaller(double x, double y) { return x > y ? y : x; }

__device__ __forceinline__ float lowest(float) { return -kMaxF32; }
__device__ __forceinline__ double lowest(double) { return -1.7976931348623157e308; }

// The two largest of a stream of values.
template <typename F>
struct Top2 {
    F a, b;
    __device__ __forceinline__ void add(F v) {
        b = larger(b, smaller(a, v));
        a = larger(a, v);
    }
    __device__ __forceinline__ void merge(int xor_lane) {
        const F oa = __shfl_xor_sync(kFull, a, xor_lane), ob = __shfl_xor_sync(kFull, b, xor_lane);
        b = larger(larger(b, ob), smaller(a, oa));
        a = larger(a, oa);
    }
    // sum of the (up to) two best (finite where they are low: -inf is a group without any), or the best alone; the smaller of the
    // values it is made of
    __device__ __forceinline__ bool two(bool top2) const { return top2 && b > -INFINITY; }
    __device__ __forceinline__ F score(bool top2) const { return two(top2) ? larger(a + b, lowest(a)) : a; }
    __device__ __forceinline__ F least(bool top2) const { return two(top2) ? b : a; }
};

// 2^shift lanes share an expert group: as many as G groups leave to each.
__device__ __forceinline__ int group_lane_shift(int G) { return G <= 1 ? 5 : G <= 2 ? 4 : G <= 4 ? 3 : G <= 8 ? 2 : G <= 16 ? 1 : 0; }

// The best two of group lane >> sh from values val[e] (-inf: out of service), in every lane of the group.
__device__ __forceinline__ Top2<float> group_best(const float* val, int G, int S, int sh) {
    const int lane = threadIdx.x & 31, g = lane >> sh, lp = 1 << sh;
    Top2<float> t{-INFINITY, -INFINITY};
    if (g < G)
        for (int j = lane & (lp - 1); j < S; j += lp) t.add(val[g * S + j]);
    for (int m = 1; m < lp; m <<= 1) t.merge(m);
    return t;
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

// What a warp needs of a row: NV values per lane, lane l the experts NV l .. NV l + NV - 1.
template <int NV, typename T>
__device__ __forceinline__ void load_chunk(const T* row, int E, bool wide, float (&l)[NV]) {
    const int e0 = NV * (int)(threadIdx.x & 31);
    constexpr int bytes = NV * (int)sizeof(T);
    if (bytes >= 4 && wide && e0 + NV <= E) {
        constexpr int words = bytes >= 4 ? bytes / 4 : 1;
        uint32_t u[words];
        const T* p = row + e0;
        if constexpr (words % 4 == 0) {
#pragma unroll
            for (int i = 0; i < words / 4; ++i) {
                const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
                u[4 * i] = q.x, u[4 * i + 1] = q.y, u[4 * i + 2] = q.z, u[4 * i + 3] = q.w;
            }
        } else if constexpr (words == 2) {
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
            u[0] = q.x, u[1] = q.y;
        } else {
            u[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
        }
        const T* v = reinterpret_cast<const T*>(u);
#pragma unroll
        for (int i = 0; i < NV; ++i) l[i] = to_f32(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) l[i] = e0 + i < E ? to_f32(row[e0 + i]) : -INFINITY;
    }
}

// Error bounds of differences of two fp32 ranking values.  Sigmoid s = 1 / (1 + e), e = exp2 of the rounded exponent
// by the hardware's approximation (relative error 2^-22 + |l| 2^-24), 1 / by the hardware's (1 ulp): an error of
// s (1 - s) (2^-22 + |l| 2^-24) + s (2^-24 + 2^-23) < 2.3 * 2^-23, as s (1 - s) <= 1/4 and s (1 - s) |l| < 0.23.
// Softmax: the sum's NV + 5 roundings and the two exp, relative to the row's largest score.  The sum with
// the bias rounds once more, 2^-24 of the value.
constexpr float kSigmoidErr = 5.6e-7f;  // 2 * 2.3 * 2^-23
__device__ __forceinline__ float softmax_err(int nv, float largest) { return (float)(nv + 16) * 1.1920929e-7f * largest; }
constexpr float kSumErr = 1.8e-7f;  // 1.5 * 2^-23 of the largest value

// Bounds of a group's score in 64 bits: half of the above for each value in it (values that cancel keep their errors) and for
// their sum.  No bound below a score of +inf, which may be a sum that overflowed; none above one of -inf.
struct Range {
    float low, high;
};
__device__ __forceinline__ Range group_range(const Top2<float>& best, bool top2, float err_s) {
    const float gs = best.score(top2), two = best.two(top2) ? 1.f : 0.f;
    const float sizes = fabsf(best.a) + fabsf(gs) + (two != 0.f ? fabsf(best.b) : 0.f);
    const float err = 0.5f * ((1.f + two) * err_s + kSumErr * sizes);
    return {fmaxf(gs - err, -INFINITY), fmaxf(gs + err, -INFINITY)};  // (fmaxf: of NaN)
}

__device__ __forceinline__ float sigmoid_fast(float l) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.44269504f * l));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
    return s;
}

// ------------------------------------------------------------------ the careful choice
// A 64-bit key in the order of doubles (no NaN), and back: comparisons of keys are integer instructions.
__device__ __forceinline__ unsigned long long key64(double v) {
    const long long u = __double_as_longlong(v == 0.0 ? 0.0 : v);
    return u < 0 ? ~(unsigned long long)u : (unsigned long long)u | 0x8000000000000000ull;
}
__device__ __forceinline__ double key_double(unsigned long long k) {
    return __longlong_as_double((long long)(k >> 63 ? k & 0x7fffffffffffffffull : ~k));
}
__device__ __forceinline__ unsigned long long warp_max_key(unsigned long long k) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) k = max(k, __shfl_xor_sync(kFull, k, m));
    return k;
}

// What the launcher works out once: experts per group, ceil(2^20 / that), whether rows and bias may be read in wide
// pieces, and how many lanes (2^lane_shift) hold exactly one group (-1: groups and lanes do not match).
struct RoutePlan {
    int S;
    uint32_t group_mul;
    int lane_shift;
    bool wide, wide_bias;
};

struct Scratch {  // of a warp, in shared memory
    unsigned long long* v64;  // [E]
    uint32_t* key;            // [E]
    uint16_t* list;           // [E]
    int* picks;               // [32]
};
constexpr int kScratchPerExpert = 14;
__device__ __forceinline__ Scratch warp_scratch(void* smem, int E, int warps, int warp) {
    Scratch s;
    char* p = static_cast<char*>(smem);
    s.v64 = reinterpret_cast<unsigned long long*>(p) + (size_t)warp * E;
    p += (size_t)8 * warps * E;
    s.picks = reinterpret_cast<int*>(p) + 32 * warp;
    p += (size_t)128 * warps;
    s.key = reinterpret_cast<uint32_t*>(p) + (size_t)warp * E;
    p += (size_t)4 * warps * E;
    s.list = reinterpret_cast<uint16_t*>(p) + (size_t)warp * E;
    return s;
}

// The whole choice for one token by one warp from shared memory: experts out of service inside the
// choice, and values closer than their error, of which those that could stand on either side of the border
// (a few) are computed in 64 bits, one per lane.  Writes the k ids in ascending order to picks[].
//   An infinite bias ranks its expert before or behind all finite values: such a value is exact, so the error's bound is
// that of the finite ones, and no border between values of which one is infinite is in doubt (each comparison below is
// false for a difference of inf or NaN).  Groups' sums are 64-bit, where those of finite values stay finite.
template <typename T>
__device__ __noinline__ void choose_careful(const RouteScoresArgs& a, const RoutePlan& plan, const T* row, const Scratch sc) {
    const int lane = threadIdx.x & 31;
    const uint32_t below = (1u << lane) - 1;
    const int E = a.E, k = a.k, G = a.rule.groups, S = plan.S, nv = (E + 31) / 32;
    const bool softmax = a.rule.score == MOE_SCORE_SOFTMAX, biased = a.bias != nullptr;
    const bool top2 = a.rule.group_score == MOE_GROUP_TOP2;
    float mx = -kMaxF32, inv_sum = 0.f;
    if (softmax && (biased || top2)) {
        for (int e = lane; e < E; e += 32)
            if (in_service(to_f32(row[e]))) mx = fmaxf(mx, clamp_logit(to_f32(row[e])));
        mx = warp_max_f32(mx);
        float sum = 0.f;
        for (int e = lane; e < E; e += 32)
            if (in_service(to_f32(row[e]))) sum += expf(clamp_logit(to_f32(row[e])) - mx);
        sum = warp_butterfly_sum(sum);
        inv_sum = sum > 0.f ? 1.f / sum : 0.f;
    }
    const RowNorm norm = {mx, inv_sum};
    const float err_s = softmax ? softmax_err(nv, inv_sum) : kSigmoidErr;
    double inv64 = 0.0;
    // 64-bit values of the n listed experts
    auto exact_list = [&](int n) {
        if (softmax && inv64 == 0.0) {
            double sum = 0.0;
            for (int e = lane; e < E; e += 32)
                if (in_service(to_f32(row[e]))) sum += exp((double)clamp_logit(to_f32(row[e])) - (double)mx);
            inv64 = 1.0 / warp_sum_f64(sum);
        }
        for (int i = lane; i < n; i += 32) {
            const int e = sc.list[i];
            const float lv = to_f32(row[e]);
            double s = softmax ? exp((double)clamp_logit(lv) - (double)mx) * inv64 : sigmoid_f64(lv);
            if (biased) s += (double)__ldg(a.bias + e);
            sc.v64[i] = __double_as_longlong(s);
        }
        __syncwarp();
    };
    auto score32 = [&](float lv) { return softmax ? score_f32(lv, true, norm) : sigmoid_fast(clamp_logit(lv)); };

    // keys of the ranking values; ranked values are the logits or scores + bias
    float vmax = 0.f;
    for (int e = lane; e < E; e += 32) {
        const float lv = to_f32(row[e]);
        float v = lv;
        if (biased && in_service(lv)) {
            v = score32(lv) + __ldg(a.bias + e);
            if (fabsf(v) < INFINITY) vmax = fmaxf(vmax, fabsf(v));
        }
        // (a NaN value comes from a NaN bias: ranked like an expert out of service)
        sc.key[e] = in_service(lv) && v == v ? logit_key(v) : kOutKey;
    }
    const float err = biased ? err_s + kSumErr * warp_max_f32(vmax) : 0.f;
    __syncwarp();

    uint32_t kept = kFull;
    const GroupOf group_of{plan.group_mul};
    if (G > 1 && a.rule.top_groups < G) {
        const int sh = group_lane_shift(G), keep = a.rule.top_groups, g = lane >> sh;
        const bool raw = !biased && !top2;  // the groups' best logits: exact
        float* val = reinterpret_cast<float*>(sc.v64);
        for (int e = lane; e < E; e += 32) {
            const uint32_t q = sc.key[e];
            val[e] = q == kOutKey ? -INFINITY : (biased || raw) ? key_logit(q) : score32(to_f32(row[e]));
        }
        __syncwarp();
        constexpr double kInf = INFINITY;
        const Top2<float> best = group_best(val, G, S, sh);
        const double gs = best.two(top2) ? (double)best.a + (double)best.b : (double)best.a;
        const unsigned long long gkey = key64(gs);
        kept = best_groups<unsigned long long>(gkey, G == 32 ? kFull : (1u << G) - 1, G, sh, keep);
        if (!raw) {
            const bool mine = g < G && gs > -kInf;
            const bool in = g < G && ((kept >> g) & 1);
            const unsigned long long none = key64(-kInf);
            const double lo = key_double(warp_max_key(mine && !in ? gkey : none));     // best left out
            const double hi = key_double(~warp_max_key(mine && in ? ~gkey : ~key64(kInf)));  // worst kept
            const double verr = biased ? err : err_s, gerr = 2.0 * verr;
            if (lo > -kInf && hi < kInf && hi - lo <= gerr) {
                const bool is_open = mine && gs >= hi - gerr && gs <= lo + gerr;
                const uint32_t lanes = __ballot_sync(kFull, is_open);
                const uint32_t sure = __ballot_sync(kFull, mine && gs > lo + gerr);
                uint32_t open = 0, in_mask = 0;
                for (int j = 0; j < G; ++j) {
                    open |= ((lanes >> (j << sh)) & 1u) << j;
                    in_mask |= ((sure >> (j << sh)) & 1u) << j;
                }
                // of the open groups, the values that may be among a group's best one or two
                if ((lane & ((1 << sh) - 1)) == 0) sc.picks[g] = __float_as_int(__fsub_rd(best.least(top2), biased ? err : err_s));
                __syncwarp();
                int n = 0;
                for (int i = 0; i < nv; ++i) {
                    const int e = lane + 32 * i;
                    bool take = e < E && ((open >> group_of(e < E ? e : 0)) & 1);
                    if (take) take = val[e] > -INFINITY && val[e] >= __int_as_float(sc.picks[group_of(e)]);
                    const uint32_t who = __ballot_sync(kFull, take);
                    if (take) sc.list[n + __popc(who & below)] = (uint16_t)e;
                    n += __popc(who);
                }
                __syncwarp();
                exact_list(n);
                double x = -(double)INFINITY, y = -(double)INFINITY;
                if (is_open && (lane & ((1 << sh) - 1)) == 0)
                    for (int i = 0; i < n; ++i) {
                        if (group_of(sc.list[i]) != g) continue;
                        const double v = __longlong_as_double(sc.v64[i]);
                        if (v > x) y = x, x = v;
                        else if (v > y) y = v;
                    }
                const double gx = top2 && y > -(double)INFINITY ? x + y : x;
                kept = in_mask | best_groups<unsigned long long>(key64(gx), open, G, sh, keep - __popc(in_mask));
            }
        }
        __syncwarp();
        for (int e = lane; e < E; e += 32)
            if (!((kept >> group_of(e)) & 1)) sc.key[e] = 0u;
        __syncwarp();
    }

    // the k-th key and who ties with it
    uint32_t gone = 0, chosen = 0;  // bit i: expert lane + 32 i
    uint32_t last = 0, next = 0;    // key of the pick that completes the k, largest key left out
    int above = 0, n = 0;           // picks with a larger key than `last`, picks so far
    uint32_t lb = 0;
    int li = -1;
    while (true) {
        if (li < 0) {
            lb = 0;
            for (int i = 0; i < nv; ++i) {
                const uint32_t q = lane + 32 * i < E && !((gone >> i) & 1) ? sc.key[lane + 32 * i] : 0u;
                if (q > lb) lb = q, li = i;
            }
        }
        const uint32_t wb = __reduce_max_sync(kFull, lb);
        if (n >= k) {
            next = n > k ? last : wb;
            break;
        }
        if (wb != last) above = n;
        last = wb;
        n += __popc(__ballot_sync(kFull, lb == wb));
        if (lb == wb) gone |= 1u << (li & 31), li = -1;
    }
    if (!(biased && last > kOutKey && next > kOutKey && key_logit(last) - key_logit(next) <= err)) {
        int ties = k - above;  // how many of the experts at `last` are picked, lowest ids first
        for (int i = 0; i < nv; ++i) {
            const uint32_t q = lane + 32 * i < E ? sc.key[lane + 32 * i] : 0u;
            if (q > last) chosen |= 1u << i;
            const uint32_t tie = __ballot_sync(kFull, q == last);
            if (q == last && __popc(tie & below) < ties) chosen |= 1u << i;
            ties -= __popc(tie);
        }
    } else {
        const float top = key_logit(next) + err, bottom = key_logit(last) - err;
        uint32_t open = 0;
        int sure = 0, m = 0;
        for (int i = 0; i < nv; ++i) {
            const int e = lane + 32 * i;
            const uint32_t q = e < E ? sc.key[e] : 0u;
            const bool up = q > kOutKey && key_logit(q) > top, take = q > kOutKey && !up && key_logit(q) >= bottom;
            if (up) chosen |= 1u << i;
            if (take) open |= 1u << i;
            sure += __popc(__ballot_sync(kFull, up));
            const uint32_t who = __ballot_sync(kFull, take);
            if (take) sc.list[m + __popc(who & below)] = (uint16_t)e;
            m += __popc(who);
        }
        __syncwarp();
        exact_list(m);
        // list entries are in id order: an equal value before an entry has the lower id
        int at = 0;
        for (int i = 0; i < nv; ++i) {
            const uint32_t who = __ballot_sync(kFull, (open >> i) & 1);
            if ((open >> i) & 1) {
                const int me = at + __popc(who & below);
                const unsigned long long mine = key64(__longlong_as_double(sc.v64[me]));
                int before = sure;
                for (int j = 0; j < m; ++j) {
                    const unsigned long long o = key64(__longlong_as_double(sc.v64[j]));
                    before += (o > mine || (o == mine && j < me)) ? 1 : 0;
                }
                if (before < k) chosen |= 1u << i;
            }
            at += __popc(who);
        }
    }
    int base = 0;
    for (int i = 0; i < nv; ++i) {
        const uint32_t who = __ballot_sync(kFull, (chosen >> i) & 1);
        const int at = base + __popc(who & below);
        if (((chosen >> i) & 1) && at < k) sc.picks[at] = lane + 32 * i;
        base += __popc(who);
    }
}

// A lower bound of the k-th largest of the lanes' values (the k-th largest itself where they differ): k rounds that drop the
// largest, at most 12 of them, else the lanes sorted (bitonic, 15 exchanges).
__device__ __forceinline__ float kth_of_lanes(float v, int k) {
    if (k <= 12) {
        float m = 0.f;
        for (int r = 0; r < k; ++r) {
            m = warp_max_f32(v);
            if (v == m) v = -INFINITY;
        }
        return m;
    }
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 2; n <= 32; n *= 2)
#pragma unroll
        for (int j = n / 2; j >= 1; j /= 2) {
            const float o = __shfl_xor_sync(kFull, v, j);
            v = ((lane & n) == 0) == ((lane & j) == 0) ? fmaxf(v, o) : fminf(v, o);
        }
    return __shfl_sync(kFull, v, k - 1);
}

// ------------------------------------------------------------------ the few at a border
// For sigmoid scores, whose 64-bit value depends on one logit: the common case of two values (or two groups) on
// either side of a border needs no pass over the row.  Kept small: this code runs for one token in some
// thousands, so its time is mostly that of fetching it.
__device__ __noinline__ double exact_sigmoid(float l, const float* bias) {
    const double s = sigmoid_f64(clamp_logit(l));
    return bias ? s + (double)__ldg(bias) : s;
}

// Lanes of `set` with a larger value than this lane's, or an equal one in a lower lane.
__device__ __forceinline__ int lanes_before(uint32_t set, double v) {
    const unsigned long long mine = key64(v);
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (uint32_t rest = set; rest; rest &= rest - 1) {
        const int j = __ffs(rest) - 1;
        const unsigned long long o = __shfl_sync(kFull, mine, j);
        before += (o > mine || (o == mine && j < lane)) ? 1 : 0;
    }
    return before;
}

// ------------------------------------------------------------------ the rules
// The k-th largest of the lanes' maxima is a lower bound of the k-th largest value, and few values beyond k pass it
// (about k^2 / 64 at random): those go to lanes of their own, in id order, and the smallest are dropped one
// by one until k are left.  With fp32 ranking values the bound is lowered by their error, so that every value
// which might belong to the picks is among these; what is too close to the border is settled in 64 bits.
// Issue-bound, hence the care for instructions: 16384 tokens of 256 fp32 logits (2.5 us of reading) take 14.0 us with 8 groups and
// a bias (about 700 warp instructions a token, 68% of the issue slots), 9.8 us without.
template <int NV, typename T>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_scores_kernel(const __grid_constant__ RouteScoresArgs a, const __grid_constant__ RoutePlan plan) {
    constexpr int kBits = NV == 1 ? 1 : NV == 2 ? 2 : NV == 4 ? 3 : NV == 8 ? 4 : NV == 16 ? 5 : 6;  // of a count up to NV
    extern __shared__ double scratch[];
    __shared__ float2 slots[kRouteWarps][32];  // id (bits) and ranking value of the values that pass
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * warps + warp;
    if (t >= a.T) return;
    const uint32_t below = (1u << lane) - 1;
    const int E = a.E, k = a.k, G = a.rule.groups;
    const bool softmax = a.rule.score == MOE_SCORE_SOFTMAX, biased = a.bias != nullptr, renorm = a.rule.renormalize != 0;
    const bool grouped = G > 1 && a.rule.top_groups < G, top2 = a.rule.group_score == MOE_GROUP_TOP2;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    const int e0 = NV * lane;

    float l[NV];
    load_chunk<NV>(row, E, plan.wide, l);
    const bool want_scores = biased || (grouped && top2);
    RowNorm norm = {0.f, 0.f};
    if (softmax && (want_scores || !renorm || a.scores)) norm = softmax_norm<NV>(l);
    if (a.scores) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (e0 + i < E) a.scores[t * E + e0 + i] = score_f32(l[i], softmax, norm);
    }

    // ranking values: the logits, or scores (+ bias).  An expert out of service has -inf (NaN logits: NaN, which no
    // comparison below lets pass; sigmoid_fast(-inf) is 0 and needs the test).  A NaN bias ranks like -inf (the fmaxf), an infinite
    // one makes its value infinite: where that reaches a border, the choice is the careful one.
    float v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = l[i];
    if (want_scores) {
        float b[NV];
        if (biased) load_chunk<NV>(a.bias, E, plan.wide_bias, b);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float s = softmax ? score_f32(l[i], true, norm) : sigmoid_fast(l[i]);
            v[i] = in_service(l[i]) ? (biased ? fmaxf(s + b[i], -INFINITY) : s) : -INFINITY;
        }
    }
    const float err_s = softmax ? softmax_err(NV, norm.inv_sum) : kSigmoidErr;
    bool careful = false;

    if (grouped) {
        const int S = plan.S, sh = plan.lane_shift, lanes = 1 << (sh & 31);
        const bool raw = !want_scores;
        float hi = 0.f, lo = -INFINITY;  // lower bound of the worst group kept, upper bound of the best left out
        bool in = false, decided = false;
        uint32_t kept = 0;
        if (sh >= 0) {  // 2^sh whole lanes share a group
            Top2<float> best{-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < NV; ++i) best.add(v[i]);
            for (int m = 1; m < lanes; m <<= 1) best.merge(m);
            const float gs = best.score(top2);
            float left = e0 < E ? gs : NAN;
            for (int r = 0; r < a.rule.top_groups; ++r) {  // the best group left, ties to the lower group
                const float most = warp_max_f32(left);
                const int first = __ffs(__ballot_sync(kFull, left == most)) - 1;
                if (lane >> sh == first >> sh) in = true, left = NAN;
            }
            Range range = {0.f, 0.f};
            if (!raw) {
                range = group_range(best, top2, err_s);
                lo = warp_max_f32(in ? -INFINITY : range.high);
                hi = -warp_max_f32(in ? -range.low : -INFINITY);
            }
            if (!softmax && lo > -INFINITY && !(hi > lo)) {
                // Kept groups that lie above all left out are in, those left out below all kept are out; the scores of the others (all in
                // service) in 64 bits, from the values that may be among a group's best
                const bool live = gs > -INFINITY, open = live && (in ? range.low <= lo : range.high >= hi);
                const float small = best.least(top2), least = small - (err_s + kSumErr * fabsf(small));
                uint32_t take = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (open && v[i] > -INFINITY && !(v[i] < least)) take |= 1u << i;  // (a bound of inf - inf takes all)
                Top2<double> x{-(double)INFINITY, -(double)INFINITY};
                for (; take; take &= take - 1) {
                    const int e = e0 + __ffs(take) - 1;
                    x.add(exact_sigmoid(to_f32(row[e]), biased ? a.bias + e : nullptr));
                }
                __syncwarp();
                for (int m = 1; m < lanes; m <<= 1) x.merge(m);
                const bool head = (lane & (lanes - 1)) == 0;
                const bool above = in && range.low > lo;
                const uint32_t set = __ballot_sync(kFull, open && head), sure = __ballot_sync(kFull, above && head);
                int before = lanes_before(set, x.score(top2));
                before = __shfl_sync(kFull, before, lane & ~(lanes - 1));
                in = above || (open && before + __popc(sure) < a.rule.top_groups);
                decided = true;
            }
        } else {  // through shared memory
            float* val = reinterpret_cast<float*>(warp_scratch(scratch, E, warps, warp).v64);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (e0 + i < E) val[e0 + i] = v[i];
            __syncwarp();
            const int gsh = group_lane_shift(G), g = lane >> gsh;
            const Top2<float> best = group_best(val, G, S, gsh);
            kept = best_groups<float>(best.score(top2), G == 32 ? kFull : (1u << G) - 1, G, gsh, a.rule.top_groups);
            if (!raw) {
                const bool mine = g < G && ((kept >> g) & 1);
                const Range range = group_range(best, top2, err_s);
                lo = warp_max_f32(g < G && !mine ? range.high : -INFINITY);
                hi = -warp_max_f32(mine ? -range.low : -INFINITY);
            }
            __syncwarp();
        }
        careful = !decided && lo > -INFINITY && !(hi > lo);
        if (!biased) {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = l[i];
        }
        if (sh >= 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = in ? v[i] : -INFINITY;
        } else {
            const GroupOf group_of{plan.group_mul};
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (e0 + i >= E || !((kept >> group_of(e0 + i < E ? e0 + i : 0)) & 1)) v[i] = -INFINITY;
        }
    }

    // candidates: every value that might be among the k largest, one per lane in id order
    float head = v[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) head = fmaxf(head, v[i]);
    head = fmaxf(head, -INFINITY);  // (a NaN sorts nowhere)
    const float bound = kth_of_lanes(head, k);
    float floor_v = biased ? bound - (err_s + kSumErr * fabsf(bound)) : bound;
    int at = 0, m = 0;
    uint32_t take = 0;
    auto count = [&](float least) {
        take = 0;
        least = fmaxf(least, -kMaxF32);  // (-inf: out of service, or not open)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (v[i] >= least) take |= 1u << i;
        const int c = __popc(take);
        at = m = 0;
#pragma unroll
        for (int b = 0; b < kBits; ++b) {
            const uint32_t lanes = __ballot_sync(kFull, (c >> b) & 1);
            at += __popc(lanes & below) << b;
            m += __popc(lanes) << b;
        }
    };
    count(floor_v);
    if (m > 32) {
        // fewer lanes than k hold the open groups' experts: search a bound that 32 lanes take
        uint32_t few = logit_key(INFINITY), many = logit_key(floor_v);  // (the key of -inf is above 0)
        for (int r = 0; r < 32 && few - many > 1 && (m > 32 || m < k); ++r) {
            const uint32_t mid = many + (few - many) / 2;
            floor_v = key_logit(mid);
            count(floor_v);
            if (m > 32) many = mid;
            else few = mid;
        }
        if (biased && m >= k && m <= 32) count(floor_v - (err_s + kSumErr * fabsf(floor_v)));
    }
    careful = careful || m < k || m > 32;

    bool pick = false;
    int id = 0;
    if (!careful) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((take >> i) & 1) slots[warp][at++] = make_float2(__int_as_float(e0 + i), v[i]);
        __syncwarp();
        const float2 mine = slots[warp][lane < m ? lane : 0];
        id = __float_as_int(mine.x);
        const float x = lane < m ? mine.y : INFINITY;
        uint32_t alive = m == 32 ? kFull : (1u << m) - 1;
        float next = -INFINITY;  // largest value dropped
        for (int r = m; r > k; --r) {  // the smallest left, ties to the higher id
            next = -warp_max_f32((alive >> lane) & 1 ? -x : -INFINITY);
            const uint32_t who = __ballot_sync(kFull, x == next) & alive;
            alive &= ~(0x80000000u >> __clz(who));
        }
        const float last = -warp_max_f32((alive >> lane) & 1 ? -x : -INFINITY);
        if (biased) {
            const float err = err_s + kSumErr * fabsf(last);
            if (!(last - next > err)) {  // settled in 64 bits
                if (softmax || !(err < INFINITY)) {
                    careful = true;
                } else {
                    const bool in_play = lane < m && x >= last - err;
                    const bool open = in_play && x <= next + err;
                    const uint32_t set = __ballot_sync(kFull, open), sure = __ballot_sync(kFull, in_play && !open);
                    double v64 = 0.0;
                    if (open) v64 = exact_sigmoid(to_f32(row[id]), a.bias + id);
                    __syncwarp();
                    const bool wins = lanes_before(set, v64) + __popc(sure) < k;
                    alive = sure | __ballot_sync(kFull, open && wins);
                }
            }
        }
        pick = (alive >> lane) & 1;
    }
    if (careful) {
        const Scratch sc = warp_scratch(scratch, E, warps, warp);
        choose_careful<T>(a, plan, row, sc);
        __syncwarp();
        pick = lane < k;
        id = pick ? sc.picks[lane] : 0;
    }

    // weights of the picks, in lane order, which is id order
    const float lp = pick ? to_f32(row[id]) : -INFINITY;
    float u, scale = a.rule.scale;
    if (renorm) {
        float ref = warp_max_f32(in_service(lp) ? clamp_logit(lp) : -kMaxF32);
        if (!softmax) ref = fminf(ref, 0.f);
        u = score_ratio(lp, softmax, ref);
        const float sum = warp_butterfly_sum(u);
        scale = sum > 0.f ? __fdividef(scale, sum) : 0.f;
    } else {
        u = score_f32(lp, softmax, norm);
    }
    const int rank = __popc(__ballot_sync(kFull, pick) & below);
    if (pick && rank < k) {
        a.ids[t * k + rank] = id;
        a.w[t * k + rank] = u * scale;
        if (a.counts) atomicAdd(a.counts + id, 1);
    }
}

// ------------------------------------------------------------------ gradient
// Gradient of the logits from the gradient of the weights (and, optionally, of all the scores).
// u_j: the picked scores, c the rule's factor.  Renormalised: du_j = c (dw_j - sum_i dw_i u_i / S) / S with
// S = sum u (taken in ratios to the largest score, as above), else du_j = c dw_j.  Sigmoid: dl = ds s (1 - s), with
// 1 - s = sigmoid(-l).  Softmax: dl = s (ds - sum ds s); with renormalised weights and no other gradient of
// the scores that sum is zero by itself, so that, as for sigmoid scores, only the picked experts get a
// gradient: the row is then written as zeros and the picks' values on top, and only the picked logits are read.
// The sparse form: 2^seg_log lanes (k or a few more) share a token, so that a warp's chain of dependent loads (ids, logits)
// serves several tokens; sums over a segment.  8192 tokens of 256 fp32 logits: 2.9 us (4.2 with a
// warp per token; 1.3 us is what writing them takes), 65536 of 64 bf16: 5.8 (12.5).
constexpr int kSparseWarps = 4;
template <typename T>
__global__ void __launch_bounds__(32 * kSparseWarps)
    route_scores_backward_sparse_kernel(const __grid_constant__ RouteBackwardArgs a, const bool wide, const int seg_log) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seg = 1 << seg_log, per = 32 >> seg_log;
    const int64_t t0 = ((int64_t)blockIdx.x * kSparseWarps + warp) * per, t = t0 + (lane >> seg_log);
    if (t0 >= a.T) return;
    const int E = a.E, k = a.k, j = lane & (seg - 1);
    const bool softmax = a.rule.score == MOE_SCORE_SOFTMAX, renorm = a.rule.renormalize != 0, on = t < a.T && j < k;
    T* out = static_cast<T*>(a.dlogits) + t * a.ldd;
    const int id = on ? a.ids[t * k + j] : -1;
    const float dw_in = on ? a.dw[t * k + j] : 0.f;
    const bool valid = id >= 0 && id < E;
    const float lp = valid ? to_f32(static_cast<const T*>(a.logits)[t * a.ld + id]) : -INFINITY;
    // zeros, over which the picks' values go
    const int rows = (int)min((int64_t)per, a.T - t0);
    T* to = static_cast<T*>(a.dlogits) + t0 * a.ldd;
    for (int r = 0; r < rows; ++r, to += a.ldd) {
        if (wide) {
            for (int p = lane; p < E * (int)sizeof(T) / 16; p += 32) reinterpret_cast<uint4*>(to)[p] = make_uint4(0, 0, 0, 0);
        } else {
            for (int e = lane; e < E; e += 32) to[e] = from_f32<T>(0.f);
        }
    }
    __syncwarp();
    const float dw = valid && in_service(lp) ? dw_in * a.rule.scale : 0.f;
    auto sum = [&](float v) {
        for (int m = seg >> 1; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        return v;
    };
    float g;  // u_j du_j, the product that the logits' gradient needs
    if (renorm) {
        float ref = in_service(lp) ? clamp_logit(lp) : -kMaxF32;
        for (int m = seg >> 1; m > 0; m >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, m));
        if (!softmax) ref = fminf(ref, 0.f);
        const float u = score_ratio(lp, softmax, ref);
        const float S = sum(u);
        const float r = S > 0.f ? u / S : 0.f;
        g = r * (dw - sum(dw * r));
    } else {
        g = dw * sigmoid_f32(lp);
    }
    if (valid) out[id] = from_f32<T>(in_service(lp) ? (softmax ? g : g * sigmoid_f32(-lp)) : 0.f);
}

// The dense form: one warp per token, as the rules' kernel.
template <int NV, typename T>
__global__ void __launch_bounds__(32 * kRouteWarps) route_scores_backward_kernel(const __grid_constant__ RouteBackwardArgs a, const bool wide) {
    extern __shared__ float rows[];  // per warp: the gradient of the scores times the scores [E]
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * warps + warp;
    if (t >= a.T) return;
    const int E = a.E, k = a.k, e0 = NV * lane;
    const bool softmax = a.rule.score == MOE_SCORE_SOFTMAX, renorm = a.rule.renormalize != 0;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    T* out = static_cast<T*>(a.dlogits) + t * a.ldd;

    // lane j < k: pick j
    const int id = lane < k ? a.ids[t * k + lane] : -1;
    const bool valid = id >= 0 && id < E;
    const float lp = valid ? to_f32(row[id]) : -INFINITY;
    const float dw = valid && in_service(lp) ? a.dw[t * k + lane] * a.rule.scale : 0.f;
    float l[NV];
    RowNorm norm = {0.f, 0.f};
    float* ds = rows + (size_t)warp * E;
    load_chunk<NV>(row, E, wide, l);
    if (softmax) norm = softmax_norm<NV>(l);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (e0 + i < E) ds[e0 + i] = 0.f;
    __syncwarp();
    float g;  // u_j du_j, the product that the logits' gradient needs
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
        gs[i] = 0.f;
        if (e0 + i >= E) continue;
        gs[i] = ds[e0 + i];
        float extra = 0.f;
        if (a.dscores && in_service(l[i])) extra = a.dscores[t * E + e0 + i] * score_f32(l[i], softmax, norm);
        if (!renorm) total += gs[i];
        total += extra;
        gs[i] += extra;
    }
    if (softmax) total = warp_butterfly_sum(total);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (e0 + i >= E) continue;
        float dl = 0.f;
        if (in_service(l[i])) dl = softmax ? gs[i] - score_f32(l[i], true, norm) * total : gs[i] * sigmoid_f32(-l[i]);
        out[e0 + i] = from_f32<T>(dl);
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

// Rows start on 16-byte boundaries: lanes read their experts in wide pieces.
static bool rows_wide(const void* p, int64_t ld, moe_dtype dtype) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (dtype == MOE_F32 ? 4 : 2) % 16 == 0;
}

cudaError_t launch_route_scores(const RouteScoresArgs& a, moe_dtype dtype, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const void* f = dtype == MOE_F32    ? scores_kernel<float>(a.E)
                    : dtype == MOE_BF16 ? scores_kernel<__nv_bfloat16>(a.E)
                                        : scores_kernel<__half>(a.E);
    int nv = 1;  // experts per lane, as the kernel's
    while (32 * nv < a.E) nv *= 2;
    RoutePlan plan;
    plan.S = a.E / a.rule.groups;
    plan.group_mul = ((1u << 20) + plan.S - 1) / plan.S;
    plan.lane_shift = -1;
    for (int sh = 0; sh <= 5; ++sh)
        if (plan.S == nv << sh) plan.lane_shift = sh;
    plan.wide = rows_wide(a.logits, a.ld, dtype);
    plan.wide_bias = reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    const int warps = a.E > 512 ? kRouteWarps / 2 : kRouteWarps;  // (less than 60 KB of scratch)
    const size_t smem = (size_t)warps * (kScratchPerExpert * (size_t)a.E + 128);
    void* args[] = {const_cast<RouteScoresArgs*>(&a), &plan};
    return launch_kernel(f, dim3((a.T + warps - 1) / warps), dim3(32 * warps), smem, st, true, args);
}

cudaError_t launch_route_scores_backward(const RouteBackwardArgs& a, moe_dtype dtype, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const bool dense = a.dscores || (a.rule.score == MOE_SCORE_SOFTMAX && !a.rule.renormalize);
    bool wide = rows_wide(a.dlogits, a.ldd, dtype);
    if (!dense) {
        wide = wide && a.E * (dtype == MOE_F32 ? 4 : 2) % 16 == 0;
        int seg_log = 2;
        while (1 << seg_log < a.k) ++seg_log;
        const int tokens = kSparseWarps * (32 >> seg_log);
        const void* f = dtype == MOE_F32    ? (const void*)route_scores_backward_sparse_kernel<float>
                        : dtype == MOE_BF16 ? (const void*)route_scores_backward_sparse_kernel<__nv_bfloat16>
                                            : (const void*)route_scores_backward_sparse_kernel<__half>;
        void* args[] = {const_cast<RouteBackwardArgs*>(&a), &wide, &seg_log};
        return launch_kernel(f, dim3((a.T + tokens - 1) / tokens), dim3(32 * kSparseWarps), 0, st, true, args);
    }
    const void* f = dtype == MOE_F32    ? backward_kernel<float>(a.E)
                    : dtype == MOE_BF16 ? backward_kernel<__nv_bfloat16>(a.E)
                                        : backward_kernel<__half>(a.E);
    wide = wide && rows_wide(a.logits, a.ld, dtype);
    void* args[] = {const_cast<RouteBackwardArgs*>(&a), &wide};
    return launch_kernel(f, dim3((a.T + kRouteWarps - 1) / kRouteWarps), dim3(32 * kRouteWarps),
                         sizeof(float) * kRouteWarps * (size_t)a.E, st, true, args);
}

}  // namespace moe
