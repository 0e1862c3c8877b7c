// route.cu -- routing of tokens to experts: scores, the choice of top-k experts
// within groups, the combine's weights, the order of the routed rows that the
// dispatch and the grouped products read, and the logits' gradient.
//
//   s = softmax(l) or sigmoid(l);  choice by s + bias (the bias steers the
//   choice only), within the topk_groups groups whose group_top best scores sum
//   highest;  w_j = scale * s_j, or scale * s_j / sum over the chosen s.
//
// The choice is a whole number next to others, so it is taken as the exact
// scores order it.  Without bias and groups that is the order of the logits
// themselves, which both score functions keep.  Otherwise FP32 scores are
// compared, each with a bound on its error; a token whose choice hangs on a
// difference within those bounds is chosen again from scores in FP64.  That is one
// token in a thousand where logits are FP32 or biased; bf16 logits without a bias are
// often equal where they are compared (256 experts, 4 of 8 groups, top-8: in a third
// of the tokens, 32 us for 4099 of them against 28), and equal scores, which go to
// the lower index, are found equal in FP64 only.
//
// What bounds it: at 16384 tokens of 64 experts the logits are 4.2 MB (0.6 us), and
// the call takes 17.7 us on the device, the choice 13 of them and the row order, a
// second launch that starts early, 4.  A warp works on one token at a time, 337
// instructions each: every round of maximum, ballot and shuffles takes a whole warp's
// instructions for one token.  More lanes a token would not shorten the rounds; fewer,
// several tokens to a warp, have not been tried.  4099 tokens of 256 experts in 8
// groups, sigmoid and bias: 27.5 us.
#include "common.cuh"

#include <algorithm>

namespace nvfp4 {
namespace {

constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 32;   // lane j of a warp holds slot j
constexpr int kMaxRouteGroups = 32;
constexpr int kRouteThreads = 1024;
constexpr int kPlanThreads = 512;
// Up to here one CTA does the whole call in one launch, which the host feels.  On
// the device, one CTA against two launches: 8 tokens 5.4 us against 5.8 (64 experts)
// and 9.9 against 10.5 (256, biased, in groups); 32 tokens 6.2 against 5.9 and 15.5
// against 10.6; 128 tokens 12.0 against 6.1 and 49 against 16.
constexpr int kSingleTokens = 16;
constexpr size_t kRouteWorkspaceHead = 256;
constexpr unsigned kFull = 0xffffffffu;

struct RouteArgs {
    const void* logits;
    int64_t ld;
    const float* bias;
    int64_t tokens;
    int experts, top_k, groups, topk_groups, group_top;
    int group_lanes;        // lanes of a group where that is a power of two whole lanes, else 0
    int softmax, renorm;
    float scale;
    int32_t* expert;
    float* weight;
    int32_t* group_offsets;
    int32_t* row_index;
    int32_t* slot_row;
    uint32_t* status;
    int32_t* hist;          // [CTAs, hist_ld]
    int hist_ld;            // experts up to a power of two, at least 4
    int64_t tokens_per_cta;
};

// Floats and doubles as unsigned numbers of the same order; -0 as +0, NaN as 1
// (below every number), 0 left for "not eligible".
__device__ __forceinline__ uint32_t ordered(float v)
{
    if (v != v) return 1u;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double v)
{
    if (v != v) return 1ull;
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ double value_of(uint64_t k)
{
    return __longlong_as_double(static_cast<long long>(k ^ ((k >> 63) ? 1ull << 63 : ~0ull)));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kFull, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v)
{
    const uint32_t hi = __reduce_max_sync(kFull, static_cast<uint32_t>(v >> 32));
    const uint32_t lo =
        __reduce_max_sync(kFull, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}
// Largest float of the warp, none of them NaN.
__device__ __forceinline__ float warp_max(float v) { return value_of(__reduce_max_sync(kFull, ordered(v))); }
template <typename T>
__device__ __forceinline__ T warp_sum(T v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// exp and 1 / x for the FP32 scores, whose errors choose() bounds, and in FP64.
__device__ __forceinline__ float score_exp(float v) { return __expf(v); }
__device__ __forceinline__ double score_exp(double v) { return exp(v); }
__device__ __forceinline__ float score_reciprocal(float v) { return __fdividef(1.0f, v); }
__device__ __forceinline__ double score_reciprocal(double v) { return 1.0 / v; }

template <typename S> struct KeyOf;
template <> struct KeyOf<float> { using type = uint32_t; };
template <> struct KeyOf<double> { using type = uint64_t; };

// The lowest finite bf16 value: a logit at or below it (FP32's lowest and -inf
// among them) takes its expert out of the choice.
constexpr float kMaskedLogit = -3.38953138925153547590e+38f;

template <int EPL, bool BF16>
__device__ __forceinline__ void load_logits(const void* logits, int64_t ld, int64_t token, int lane, int experts,
                                            float (&l)[EPL])
{
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane * EPL + i;
        l[i] = -INFINITY;
        if (e < experts) {
            if constexpr (BF16)
                l[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(logits)[token * ld + e]);
            else
                l[i] = static_cast<const float*>(logits)[token * ld + e];
        }
    }
}

// The k best experts of one token, lane j returning slot j's expert (-1: none
// left) and its logit.  Lane i holds the EPL experts from i * EPL on.
//
// With float scores, `close` says that the choice hangs on less than the scores'
// error bounds.  Those differ from expert to expert (a score that a bias cancels
// has a far larger one than a small score under a small bias), so that each of the
// chosen is compared with all that rank behind it, not with the next alone: its
// score less its bound has to exceed their largest score plus bound.  For groups,
// whose rank is a sum of their best scores, every member's bound is taken to be
// the group's largest: the n-th best exact score is then within that bound of the
// n-th best FP32 score, whichever members they belong to.  (Groups that are ranked
// one after the other take the token's largest bound, which saves a reduction each.)
template <typename S, int EPL>
__device__ __forceinline__ void choose(const RouteArgs& a, const float (&l)[EPL], int lane, int& id, float& logit,
                                       bool& close)
{
    using K = typename KeyOf<S>::type;
    constexpr bool F32 = sizeof(S) == 4;
    K key[EPL];
    float err[EPL], largest = 0.0f;
    close = false;
    const bool by_logit = !a.bias && a.groups == 1;
    if (by_logit) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            key[i] = l[i] <= kMaskedLogit ? 0 : ordered(static_cast<S>(l[i]));
            err[i] = 0.0f;
        }
    } else {
        S s[EPL];
        S top = 0, total = 1;
        if (a.softmax) {
            K m = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (!(l[i] <= kMaskedLogit)) m = max(m, ordered(static_cast<S>(l[i])));
            m = warp_max(m);
            top = m > 1 ? value_of(m) : static_cast<S>(0);
            total = 0;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (l[i] <= kMaskedLogit)
                s[i] = 0;
            else if (a.softmax)
                s[i] = score_exp(static_cast<S>(l[i]) - top);
            else
                s[i] = score_reciprocal(static_cast<S>(1) + score_exp(-static_cast<S>(l[i])));
            if (a.softmax) total += s[i];
        }
        if (a.softmax) total = score_reciprocal(warp_sum(total));
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane * EPL + i;
            if (a.softmax) s[i] *= total;
            const S v = s[i] + (a.bias && e < a.experts ? static_cast<S>(a.bias[e]) : static_cast<S>(0));
            key[i] = l[i] <= kMaskedLogit ? 0 : ordered(v);
            // FP32.  __expf is off by (2 + 1.173 |x|) ulp, 2^-22 + |x| 2^-22.7 of its
            // value.  Sigmoid: that times 1 - s, and the sum's and quotient's roundings.
            // Softmax: that and the argument's rounding for the term; in the total the
            // terms' errors are weighted by the scores, whose mean |x| is at most ln 512,
            // and 21 additions follow one another: 2^-18.4; then a quotient and a product.
            // Both: the bias's addition, and numbers below the smallest normal one, which
            // may come out as zero.
            err[i] = 0.0f;
            if (F32 && key[i]) {
                const float sf = static_cast<float>(s[i]);
                const float rel = a.softmax ? 0x1p-18f + fabsf(static_cast<float>(l[i] - top)) * 0x1p-22f
                                            : 0x1p-21f + (1.0f - sf) * (1.0f + fabsf(l[i])) * 0x1p-22f;
                err[i] = sf * rel + fabsf(static_cast<float>(v)) * 0x1p-23f + 0x1p-125f;
            }
        }
    }
    if (F32 && !by_logit) {
        // infinities and NaN have no bound: such a token is left to FP64, and all is finite below
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) most = max(most, __float_as_uint(err[i]));
        most = warp_max(most);
        close = most >= 0x7F800000u;
        if (close) return;
        largest = __uint_as_float(most);
    }
    if (a.groups > 1) {
        const int size = a.experts / a.groups;
        K mine = 0;         // lane g (or the first of its lanes): group g's key
        float mine_err = 0.0f;
        if (a.group_lanes) {
            // a group is group_lanes whole lanes: each lane's two best, then merged
            // pairwise within the group's lanes
            K best = 0, second = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                if (key[i] > best)
                    second = best, best = key[i];
                else if (key[i] > second)
                    second = key[i];
                if (F32) mine_err = fmaxf(mine_err, err[i]);
            }
#pragma unroll 1
            for (int d = 1; d < a.group_lanes; d <<= 1) {
                const K ob = __shfl_xor_sync(kFull, best, d), os = __shfl_xor_sync(kFull, second, d);
                if (F32) mine_err = fmaxf(mine_err, __shfl_xor_sync(kFull, mine_err, d));
                second = max(max(second, os), min(best, ob));
                best = max(best, ob);
            }
            if (best && lane % a.group_lanes == 0 && lane < a.groups * a.group_lanes) {
                S sum = best == 1 ? static_cast<S>(NAN) : value_of(best);
                if (a.group_top == 2 && second) {
                    sum += second == 1 ? static_cast<S>(NAN) : value_of(second);
                    mine_err *= 2.0f;
                }
                mine = ordered(sum);
                mine_err += fabsf(static_cast<float>(sum)) * 0x1p-23f;
            }
        } else for (int g = 0; g < a.groups; ++g) {
            S sum = 0;
            bool any = false;
            int taken = -1;
            float sum_err = 0.0f;
            for (int n = 0; n < a.group_top; ++n) {
                K m = 0;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = lane * EPL + i;
                    if (e >= g * size && e < (g + 1) * size && e != taken) m = max(m, key[i]);
                }
                const K best = warp_max(m);
                if (best == 0) break;
                const int src = __ffs(__ballot_sync(kFull, m == best)) - 1;
                int at = -1;
#pragma unroll
                for (int i = EPL - 1; i >= 0; --i) {
                    const int e = lane * EPL + i;
                    if (e >= g * size && e < (g + 1) * size && e != taken && key[i] == best) at = e;
                }
                taken = __shfl_sync(kFull, at, src);
                sum_err += largest;
                sum += best == 1 ? static_cast<S>(NAN) : value_of(best);
                any = true;
            }
            if (lane == g) {
                mine = any ? ordered(sum) : 0;
                mine_err = sum_err + fabsf(static_cast<float>(sum)) * 0x1p-23f;
            }
        }
        unsigned kept = 0;
        const K rank = mine;
        for (int n = 0; n < a.topk_groups; ++n) {
            const K best = warp_max(mine);
            if (best == 0) break;
            const int src = __ffs(__ballot_sync(kFull, mine == best)) - 1;
            kept |= 1u << src;
            if (lane == src) mine = 0;
        }
        if (F32) {  // the kept groups' smallest value against the largest one left out
            const float v = rank ? static_cast<float>(value_of(rank)) : 0.0f;
            const bool in = (kept >> lane) & 1u;
            const float least = -warp_max(in ? -__fsub_rd(v, mine_err) : -INFINITY);
            const float most = warp_max(rank && !in ? __fadd_ru(v, mine_err) : -INFINITY);
            close = !(least > most) && kept;
            if (close) return;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int g = a.group_lanes ? lane & -a.group_lanes : (lane * EPL + i) / size;
            if (g >= 32 || !((kept >> g) & 1)) key[i] = 0;
        }
    }
    id = -1;
    logit = 0.0f;
    float score = 0.0f, bound = 0.0f;  // of slot j, lane j
    for (int j = 0; j < a.top_k; ++j) {
        K m = key[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) m = max(m, key[i]);
        const K best = warp_max(m);
        if (best == 0) break;
        const int src = __ffs(__ballot_sync(kFull, m == best)) - 1;
        int at = 0;
        float l_at = 0.0f, e_at = 0.0f;
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i)
            if (key[i] == best) at = i, l_at = l[i], e_at = err[i];
        if (lane == src) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i == at) key[i] = 0;
        }
        const int e = src * EPL + __shfl_sync(kFull, at, src);
        const float lv = __shfl_sync(kFull, l_at, src);
        if (F32 && !by_logit) {
            const float eb = __shfl_sync(kFull, e_at, src);
            if (lane == j) score = static_cast<float>(value_of(best)), bound = eb;
        }
        if (lane == j) id = e, logit = lv;
    }
    if (F32 && !by_logit) {
        // the largest score plus bound of all behind slot j: of the experts left, and of
        // the later slots
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i]) most = fmaxf(most, __fadd_ru(static_cast<float>(value_of(key[i])), err[i]));
        most = warp_max(most);
        float upper = id >= 0 ? __fadd_ru(score, bound) : -INFINITY;  // of this slot, and then of it and the later ones
        float later = __shfl_down_sync(kFull, upper, 1);
        if (lane == 31) later = -INFINITY;
#pragma unroll 1
        for (int d = 1; d < a.top_k; d <<= 1) {
            const float v = __shfl_down_sync(kFull, later, d);
            if (lane + d < 32) later = fmaxf(later, v);
        }
        most = fmaxf(most, later);
        close = __any_sync(kFull, id >= 0 && !(__fsub_rd(score, bound) > most));
    }
}

// sigmoid(l) times exp(-m), m = min(the largest chosen logit, 0): the factor
// cancels in sigmoid(l) / sum and keeps both finite for very negative logits.
__device__ __forceinline__ float scaled_sigmoid(float l, float m)
{
    return l <= 0.0f ? expf(l - m) / (1.0f + expf(l)) : 1.0f / (1.0f + expf(-l));
}

__device__ __forceinline__ float max_chosen(int id, float logit)
{
    const uint32_t m = __reduce_max_sync(kFull, id >= 0 ? ordered(logit) : 0u);
    return m > 1 ? value_of(m) : 0.0f;
}

// Largest logit and sum of exp(l - largest) over a token's eligible experts.
template <int EPL>
__device__ __forceinline__ void softmax_stats(const float (&l)[EPL], float& top, float& total)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (!(l[i] <= kMaskedLogit)) m = max(m, ordered(l[i]));
    m = warp_max(m);
    top = m > 1 ? value_of(m) : 0.0f;
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) total += l[i] <= kMaskedLogit ? 0.0f : expf(l[i] - top);
    total = warp_sum(total);
}

// Rows of the slots [s0, s1), by expert and then by slot: base[e] is the first
// row of expert e for these slots.  Each warp takes a run of the slots; counts
// [warps, experts] in `cnt`.
__device__ void place_rows(const RouteArgs& a, int64_t s0, int64_t s1, const int* base, int* cnt)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int E = a.experts;
    for (int i = threadIdx.x; i < warps * E; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    const int64_t run = ((s1 - s0 + warps - 1) / warps + 31) / 32 * 32;
    const int64_t w0 = min(s0 + warp * run, s1), w1 = min(w0 + run, s1);
    int* mine = cnt + warp * E;
    for (int64_t c = w0; c < w1; c += 32) {
        const int id = c + lane < w1 ? a.expert[c + lane] : -1;
        const unsigned same = __match_any_sync(kFull, id);
        if (id >= 0 && lane == __ffs(same) - 1) mine[id] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int at = base[e];
        for (int w = 0; w < warps; ++w) {
            const int n = cnt[w * E + e];
            cnt[w * E + e] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int64_t c = w0; c < w1; c += 32) {
        const int64_t s = c + lane;
        const int id = s < w1 ? a.expert[s] : -1;
        const unsigned same = __match_any_sync(kFull, id);
        const int row = id >= 0 ? mine[id] + __popc(same & ((1u << lane) - 1)) : -1;
        __syncwarp();
        if (id >= 0 && lane == __ffs(same) - 1) mine[id] += __popc(same);
        __syncwarp();
        if (s < w1) {
            a.slot_row[s] = row;
            if (row >= 0) a.row_index[row] = static_cast<int32_t>(s / a.top_k);
        }
    }
}

// Exclusive prefix sums of count[0..n) into off[0..n], by the whole block;
// returns the total.
__device__ int block_prefix(const int* count, int* off, int n, int* warp_total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // n <= 512 <= blockDim.x
    const int v = static_cast<int>(threadIdx.x) < n ? count[threadIdx.x] : 0;
    int incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int t = __shfl_up_sync(kFull, incl, d);
        if (lane >= d) incl += t;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
        if (w < warp) before += warp_total[w];
        total += warp_total[w];
    }
    if (static_cast<int>(threadIdx.x) < n) off[threadIdx.x] = before + incl - v;
    if (threadIdx.x == 0) off[n] = total;
    __syncthreads();
    return total;
}

// One warp per token.  SINGLE: one CTA, which also places the rows; otherwise
// each CTA counts its tokens' experts into its row of a.hist.
template <int EPL, bool BF16, bool SINGLE>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteArgs a)
{
    extern __shared__ int s_dyn[];
    int* s_count = s_dyn;  // [experts]
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) s_count[e] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.status) *a.status = 0u;
    __syncthreads();
    const int64_t t0 = blockIdx.x * a.tokens_per_cta, t1 = min(t0 + a.tokens_per_cta, a.tokens);
    float next[EPL];  // the following token's logits, on their way
    if (t0 + warp < t1) load_logits<EPL, BF16>(a.logits, a.ld, t0 + warp, lane, a.experts, next);
    for (int64_t t = t0 + warp; t < t1; t += warps) {
        float l[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) l[i] = next[i];
        if (t + warps < t1) load_logits<EPL, BF16>(a.logits, a.ld, t + warps, lane, a.experts, next);
        int id;
        float logit;
        bool close;
        choose<float, EPL>(a, l, lane, id, logit, close);
        if (close) {
            bool unused;
            choose<double, EPL>(a, l, lane, id, logit, unused);
        }
        float v = 0.0f;
        if (a.renorm) {
            const float m = max_chosen(id, logit);
            if (id >= 0) v = a.softmax ? expf(logit - m) : scaled_sigmoid(logit, fminf(m, 0.0f));
            const float total = warp_sum(v);
            if (id >= 0) v = v / total * a.scale;
        } else if (a.softmax) {
            float top, total;
            softmax_stats<EPL>(l, top, total);
            if (id >= 0) v = expf(logit - top) / total * a.scale;
        } else if (id >= 0) {
            v = a.scale / (1.0f + expf(-logit));
        }
        if (lane < a.top_k) {
            a.expert[t * a.top_k + lane] = id;
            a.weight[t * a.top_k + lane] = v;
            if (id >= 0) atomicAdd(&s_count[id], 1);
        }
    }
    __syncthreads();
    if constexpr (SINGLE) {
        int* s_off = s_count + a.experts;      // [experts + 1]
        int* s_warp = s_off + a.experts + 1;   // [32]
        int* s_cnt = s_warp + 32;              // [warps, experts]
        const int total = block_prefix(s_count, s_off, a.experts, s_warp);
        for (int e = threadIdx.x; e <= a.experts; e += blockDim.x) a.group_offsets[e] = s_off[e];
        for (int64_t r = total + threadIdx.x; r < a.tokens * a.top_k; r += blockDim.x) a.row_index[r] = -1;
        place_rows(a, 0, a.tokens * a.top_k, s_off, s_cnt);
    } else {
        for (int e = threadIdx.x; e < a.hist_ld; e += blockDim.x)
            a.hist[blockIdx.x * a.hist_ld + e] = e < a.experts ? s_count[e] : 0;
    }
}

// Second launch of a large call: CTA b finds where its tokens' rows start (all
// experts before, and the earlier CTAs' rows of the same expert) and places them.
__global__ void __launch_bounds__(kPlanThreads) route_plan_kernel(const RouteArgs a)
{
    extern __shared__ int s_dyn[];
    const int E = a.experts;
    int* s_count = s_dyn;             // [E] all CTAs
    int* s_before = s_count + E;      // [E] earlier CTAs
    int* s_off = s_before + E;        // [E + 1]
    int* s_warp = s_off + E + 1;      // [32]
    int* s_cnt = s_warp + 32;         // [warps, E]
    const int b = blockIdx.x;
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_count[e] = s_before[e] = 0;
    __syncthreads();
    wait_for_previous_kernel();
    let_next_kernel_start();
    {
        // four experts a thread, the CTAs' rows over the threads that share them
        const int vecs = a.hist_ld / 4, v = threadIdx.x % vecs;
        int4 all = make_int4(0, 0, 0, 0), before = all;
#pragma unroll 4
        for (int c = threadIdx.x / vecs; c < static_cast<int>(gridDim.x); c += kPlanThreads / vecs) {
            const int4 n = reinterpret_cast<const int4*>(a.hist)[c * vecs + v];
            all.x += n.x, all.y += n.y, all.z += n.z, all.w += n.w;
            if (c < b) before.x += n.x, before.y += n.y, before.z += n.z, before.w += n.w;
        }
        const int n_all[4] = {all.x, all.y, all.z, all.w}, n_before[4] = {before.x, before.y, before.z, before.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * v + i < E) {
                if (n_all[i]) atomicAdd(&s_count[4 * v + i], n_all[i]);
                if (n_before[i]) atomicAdd(&s_before[4 * v + i], n_before[i]);
            }
    }
    __syncthreads();
    const int total = block_prefix(s_count, s_off, E, s_warp);
    if (b == 0) {
        for (int e = threadIdx.x; e <= E; e += blockDim.x) a.group_offsets[e] = s_off[e];
        for (int64_t r = total + threadIdx.x; r < a.tokens * a.top_k; r += blockDim.x) a.row_index[r] = -1;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_before[e] += s_off[e];
    __syncthreads();
    const int64_t t0 = b * a.tokens_per_cta, t1 = min(t0 + a.tokens_per_cta, a.tokens);
    place_rows(a, t0 * a.top_k, t1 * a.top_k, s_before, s_cnt);
}

struct RouteBackArgs {
    const float* dweight;
    const void* logits;
    int64_t ld;
    const int32_t* expert;
    int64_t tokens;
    int experts, top_k, softmax, renorm;
    float scale;
    void* dlogits;
    int64_t ldd;
};

// One warp per token; lane j holds slot j.
//   softmax:  dl_e = p_e (dp_e - sum_i dp_i p_i), dp the chosen weights' gradients
//   renormalised over the chosen, q = s_j / sum: dl_j = scale q_j (g_j - sum g q) f_j,
//   f_j = 1 (softmax) or 1 - sigmoid(l_j); zero for the others
template <int EPL, bool BF16>
__global__ void __launch_bounds__(256) route_backward_kernel(const RouteBackArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    wait_for_previous_kernel();
    let_next_kernel_start();
    for (int64_t t = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5); t < a.tokens; t += warps) {
        int id = -1;
        float g = 0.0f, l = 0.0f;
        if (lane < a.top_k) {
            id = a.expert[t * a.top_k + lane];
            if (id >= a.experts) id = -1;
            if (id >= 0) {
                g = a.dweight[t * a.top_k + lane] * a.scale;
                if constexpr (BF16)
                    l = __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[t * a.ld + id]);
                else
                    l = static_cast<const float*>(a.logits)[t * a.ld + id];
            }
        }
        float d = 0.0f;
        float out[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) out[i] = 0.0f;
        if (a.renorm) {
            const float m = max_chosen(id, l);
            float v = 0.0f;
            if (id >= 0) v = a.softmax ? expf(l - m) : scaled_sigmoid(l, fminf(m, 0.0f));
            const float total = warp_sum(v);
            const float q = id >= 0 ? v / total : 0.0f;
            const float dot = warp_sum(q * g);
            d = q * (g - dot);
            if (!a.softmax) d *= 1.0f / (1.0f + expf(l));
        } else if (a.softmax) {
            float all[EPL], top, total;
            load_logits<EPL, BF16>(a.logits, a.ld, t, lane, a.experts, all);
            softmax_stats<EPL>(all, top, total);
            const float p = id >= 0 ? expf(l - top) / total : 0.0f;
            const float dot = warp_sum(p * g);
            d = p * g;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                out[i] = all[i] <= kMaskedLogit ? 0.0f : -(expf(all[i] - top) / total) * dot;
        } else if (id >= 0) {
            d = g / (1.0f + expf(-l)) * (1.0f / (1.0f + expf(l)));
        }
        for (int j = 0; j < a.top_k; ++j) {
            const int e = __shfl_sync(kFull, id, j);
            const float v = __shfl_sync(kFull, d, j);
            if (e >= 0 && e / EPL == lane) {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (e % EPL == i) out[i] += v;
            }
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane * EPL + i;
            if (e >= a.experts) continue;
            if constexpr (BF16)
                static_cast<__nv_bfloat16*>(a.dlogits)[t * a.ldd + e] = __float2bfloat16_rn(out[i]);
            else
                static_cast<float*>(a.dlogits)[t * a.ldd + e] = out[i];
        }
    }
}

size_t route_smem(int experts, bool single, bool plan)
{
    const int warps = (single ? kRouteThreads : kPlanThreads) / 32;
    if (single) return sizeof(int) * (2 * experts + 1 + 32 + warps * experts);
    if (plan) return sizeof(int) * (3 * experts + 1 + 32 + warps * experts);
    return sizeof(int) * experts;
}

int hist_stride(int experts)
{
    int n = 4;
    while (n < experts) n *= 2;
    return n;
}

int route_ctas(int64_t tokens, int sms)
{
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((tokens + 7) / 8, std::min(sms, 160))));
}

nvfp4_status route_common(const void* logits, int logits_dtype, int64_t ld, int64_t tokens, int experts, int top_k,
                          int score)
{
    if (logits_dtype != NVFP4_OUT_F32 && logits_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
    if (score != NVFP4_SOFTMAX && score != NVFP4_SIGMOID) return NVFP4_ERR_INVALID_ARG;
    if (tokens < 0 || experts < 1 || experts > kMaxExperts || top_k < 1 || top_k > kMaxTopK || top_k > experts ||
        ld < experts || tokens > 0x7fffffffll / top_k)
        return NVFP4_ERR_SHAPE;
    if (tokens > 0 && !logits) return NVFP4_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) & (logits_dtype == NVFP4_OUT_F32 ? 3u : 1u)) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" size_t nvfp4_route_workspace_size(int64_t tokens, int experts)
{
    if (tokens <= kSingleTokens || experts <= 0) return kRouteWorkspaceHead;
    return kRouteWorkspaceHead + sizeof(int32_t) * static_cast<size_t>(route_ctas(tokens, 160)) * hist_stride(experts);
}

extern "C" nvfp4_status nvfp4_route(const void* logits, int logits_dtype, int64_t ld, const float* bias,
                                    int64_t tokens, int experts, const nvfp4_route_params* p, int32_t* expert,
                                    float* weight, int32_t* group_offsets, int32_t* row_index, int32_t* slot_row,
                                    void* workspace, size_t ws_bytes, void* stream)
{
    if (!p || !group_offsets || (tokens > 0 && (!expert || !weight || !row_index || !slot_row)))
        return NVFP4_ERR_INVALID_ARG;
    if (const nvfp4_status s = route_common(logits, logits_dtype, ld, tokens, experts, p->top_k, p->score)) return s;
    if (p->groups < 1 || p->groups > kMaxRouteGroups || experts % p->groups || p->topk_groups < 1 ||
        p->topk_groups > p->groups || p->top_k > experts / p->groups * p->topk_groups)
        return NVFP4_ERR_SHAPE;
    if ((p->group_top != 1 && p->group_top != 2) || (p->renormalize != 0 && p->renormalize != 1))
        return NVFP4_ERR_INVALID_ARG;
    for (const void* q : {static_cast<const void*>(bias), static_cast<const void*>(expert),
                          static_cast<const void*>(weight), static_cast<const void*>(group_offsets),
                          static_cast<const void*>(row_index), static_cast<const void*>(slot_row)})
        if (reinterpret_cast<uintptr_t>(q) & 3u) return NVFP4_ERR_ALIGN;
    const bool single = tokens <= kSingleTokens;
    if ((!single && !workspace) || (workspace && (off16(workspace) || ws_bytes < nvfp4_route_workspace_size(tokens, experts))))
        return NVFP4_ERR_WORKSPACE;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    const int sms = sm100_sms(dev);
    if (!sms) return NVFP4_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    RouteArgs a{};
    a.logits = logits, a.ld = ld, a.bias = bias, a.tokens = tokens;
    a.experts = experts, a.top_k = p->top_k;
    a.groups = p->groups == p->topk_groups ? 1 : p->groups;  // every group kept: no limit
    a.topk_groups = p->topk_groups, a.group_top = p->group_top;
    a.softmax = p->score == NVFP4_SOFTMAX, a.renorm = p->renormalize, a.scale = p->scale;
    a.expert = expert, a.weight = weight;
    a.group_offsets = group_offsets, a.row_index = row_index, a.slot_row = slot_row;
    a.status = workspace ? static_cast<uint32_t*>(workspace) + 2 : nullptr;
    const int ctas = single ? 1 : route_ctas(tokens, sms);
    a.tokens_per_cta = (tokens + ctas - 1) / ctas;
    a.hist_ld = hist_stride(experts);
    const int per_lane = experts <= 32 ? 1 : experts <= 64 ? 2 : experts <= 128 ? 4 : experts <= 256 ? 8 : 16;
    const int size = experts / a.groups, lanes = size / per_lane;
    a.group_lanes = size % per_lane == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    a.hist = single ? nullptr : reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + kRouteWorkspaceHead);
    const size_t smem = route_smem(experts, single, false);
    bool ok = true;
    const auto go = [&](auto kernel) {
        if (smem > 48 * 1024)
            ok = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) == cudaSuccess;
        if (ok) ok = launch_early(true, kernel, ctas, kRouteThreads, smem, st, a) == cudaSuccess;
    };
    const bool h = logits_dtype == NVFP4_OUT_BF16;
#define NVFP4_ROUTE(EPL)                                                                          \
    single ? (h ? go(route_kernel<EPL, true, true>) : go(route_kernel<EPL, false, true>))         \
           : (h ? go(route_kernel<EPL, true, false>) : go(route_kernel<EPL, false, false>))
    if (experts <= 32) NVFP4_ROUTE(1);
    else if (experts <= 64) NVFP4_ROUTE(2);
    else if (experts <= 128) NVFP4_ROUTE(4);
    else if (experts <= 256) NVFP4_ROUTE(8);
    else NVFP4_ROUTE(16);
#undef NVFP4_ROUTE
    if (!ok || cudaGetLastError() != cudaSuccess) return NVFP4_ERR_CUDA;
    if (!single) {
        if (launch_early(true, route_plan_kernel, ctas, kPlanThreads, route_smem(experts, false, true), st, a) !=
            cudaSuccess)
            return NVFP4_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

extern "C" nvfp4_status nvfp4_route_backward(const float* dweight, const void* logits, int logits_dtype, int64_t ld,
                                             const int32_t* expert, int64_t tokens, int experts,
                                             const nvfp4_route_params* p, void* dlogits, int64_t ldd, void* stream)
{
    if (!p || (tokens > 0 && (!dweight || !expert || !dlogits))) return NVFP4_ERR_INVALID_ARG;
    if (const nvfp4_status s = route_common(logits, logits_dtype, ld, tokens, experts, p->top_k, p->score)) return s;
    if (ldd < experts) return NVFP4_ERR_SHAPE;
    if (p->renormalize != 0 && p->renormalize != 1) return NVFP4_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(dweight) & 3u) || (reinterpret_cast<uintptr_t>(expert) & 3u) ||
        (reinterpret_cast<uintptr_t>(dlogits) & (logits_dtype == NVFP4_OUT_F32 ? 3u : 1u)))
        return NVFP4_ERR_ALIGN;
    if (tokens == 0) return NVFP4_OK;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    const int sms = sm100_sms(dev);
    if (!sms) return NVFP4_ERR_UNSUPPORTED;
    RouteBackArgs a{dweight, logits, ld, expert, tokens, experts, p->top_k, p->score == NVFP4_SOFTMAX,
                    p->renormalize, p->scale, dlogits, ldd};
    const int grid = static_cast<int>(std::min<int64_t>((tokens + 7) / 8, static_cast<int64_t>(sms) * 8));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    const auto go = [&](auto kernel) { err = launch_early(true, kernel, grid, 256, 0, st, a); };
    const bool h = logits_dtype == NVFP4_OUT_BF16;
    if (experts <= 32) h ? go(route_backward_kernel<1, true>) : go(route_backward_kernel<1, false>);
    else if (experts <= 64) h ? go(route_backward_kernel<2, true>) : go(route_backward_kernel<2, false>);
    else if (experts <= 128) h ? go(route_backward_kernel<4, true>) : go(route_backward_kernel<4, false>);
    else if (experts <= 256) h ? go(route_backward_kernel<8, true>) : go(route_backward_kernel<8, false>);
    else h ? go(route_backward_kernel<16, true>) : go(route_backward_kernel<16, false>);
    return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
