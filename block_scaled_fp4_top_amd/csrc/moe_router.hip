// The router's choice of experts for each token, and its gradient.
//
//   score s = softmax or sigmoid of the logits, choice c = s + bias; of the best groups of
//   experts the K largest choices, in descending order, ties to the lower expert;
//   weight = scale * s, divided by the sum of the chosen s if renormalised.
//
// An expert whose logit or bias is -inf is never chosen. A NaN makes its token's weights
// NaN and counts as the lowest choice, so that ids stay distinct experts.
//
// Choices are compared exactly: without a bias (and without sums of two choices) the logits
// decide, as both scores rise with them; otherwise c is computed in fp64, so that no
// choice depends on the rounding of an fp32 score.
//
// A token belongs to LPT lanes of a wave (16 up to 256 experts, else 64), each of which
// holds EPL consecutive experts in registers. K rounds of a maximum over the lanes' best
// pick the experts; the lane that holds a round's winner looks for its next best.
#include <algorithm>

#include "moe_args.h"
#include "moe_rows_dev.h"
#include "moe_wave_dev.h"

#define INLINE __attribute__((always_inline))

namespace moe {

constexpr float kInf = __builtin_huge_valf();
constexpr float kLowest = -3.402823466e38f;

struct RouteArgs {
    const void* logits;
    int64_t ld;
    const float* bias;  // or null
    int T, E, K;
    int softmax;        // else sigmoid
    int groups, top_groups, group_top;
    int renormalize;
    float scale;
    int32_t* ids;
    float* weights;
};

// What the lanes of a wave wrote to the LDS is read by its other lanes: LDS accesses of a
// wave are in order, the compiler has to leave them so.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int CTRL>
__device__ __forceinline__ double dpp_move(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp_move<CTRL>((uint32_t)b), hi = dpp_move<CTRL>((uint32_t)(b >> 32));
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) { return u2f(dpp_move<CTRL>(f2u(v))); }
__device__ __forceinline__ float lane_value(float v, int l) { return lane_f32(v, l); }
__device__ __forceinline__ double lane_value(double v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, l), hi = __builtin_amdgcn_readlane((int)(b >> 32), l);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Over a token's lanes; the same bits in each.
template <int LPT, typename V, typename OP>
__device__ __forceinline__ V token_all(V v, OP op) {
    v = op(v, dpp_move<kRor8>(v));
    v = op(v, dpp_move<kRor4>(v));
    v = op(v, dpp_move<kRor2>(v));
    v = op(v, dpp_move<kRor1>(v));
    if constexpr (LPT == 64) v = op(op(lane_value(v, 0), lane_value(v, 16)), op(lane_value(v, 32), lane_value(v, 48)));
    return v;
}
template <int LPT, typename V>
__device__ __forceinline__ V token_max(V v) {
    return token_all<LPT>(v, [](V a, V b) INLINE { return a > b ? a : b; });
}
template <int LPT, typename V>
__device__ __forceinline__ V token_sum(V v) {
    return token_all<LPT>(v, [](V a, V b) INLINE { return a + b; });
}
// This token's bits of a ballot.
template <int LPT>
__device__ __forceinline__ uint64_t token_ballot(bool b) {
    const uint64_t all = __ballot(b);
    if constexpr (LPT == 64) return all;
    return (all >> ((threadIdx.x & 63) / LPT * LPT)) & ((1ull << LPT) - 1);
}

// exp(x - top) with equal infinities 0 apart
template <typename V>
__device__ __forceinline__ V exp_below(V x, V top) {
    const V d = x == top ? (V)0 : x - top;
    if constexpr (sizeof(V) == 8) return exp(d);
    else return expf(d);
}

// Logits of EPL consecutive experts from `first` on, -inf behind the last.
template <int EPL, typename X>
__device__ __forceinline__ void load_logits(const X* row, int first, int E, float* x) {
    constexpr int V = 16 / sizeof(X);
    if constexpr (EPL % V == 0 || EPL * sizeof(X) == 8) {
        if (first + EPL <= E) {
            load_floats<EPL>(row + first, x);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = first + i < E ? to_f32(row[first + i]) : -kInf;
}

template <typename V>
struct Top2 {
    V a, b;  // the largest and the second, -inf where there is none
};
template <typename V>
__device__ __forceinline__ void insert(Top2<V>& t, V v) {
    const bool first = v > t.a;
    t.b = first ? t.a : v > t.b ? v : t.b;
    t.a = first ? v : t.a;
}

// Takes the experts of all but the top_groups best groups out of c. LDS: `room` holds E + G
// values for choices (G padding), G scores and G flags.
template <typename V, int LPT, int EPL>
__device__ __forceinline__ void keep_groups(const RouteArgs& p, int sub, V* c, char* room) {
    const int G = p.groups, S = p.E / G, pad = S | 1;
    V* choice = (V*)room;
    V* score = choice + G * pad;
    int* stays = (int*)(score + G);
    const int first = sub * EPL;
    int g = first / S, at = first - g * S;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (first + i < p.E) choice[g * pad + at] = c[i];
        if (++at == S) at = 0, ++g;
    }
    wave_fence();
    for (int h = sub; h < G; h += LPT) {
        Top2<V> t{(V)-kInf, (V)-kInf};
        for (int j = 0; j < S; ++j) insert(t, choice[h * pad + j]);
        score[h] = p.group_top == 2 && t.b > (V)-kInf ? t.a + t.b : t.a;
    }
    wave_fence();
    for (int h = sub; h < G; h += LPT) {
        const V mine = score[h];
        int better = 0;
        for (int o = 0; o < G; ++o) better += score[o] > mine || (score[o] == mine && o < h);
        stays[h] = better < p.top_groups;
    }
    wave_fence();
    g = first / S, at = first - g * S;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (first + i < p.E && !stays[g]) c[i] = (V)-kInf;
        if (++at == S) at = 0, ++g;
    }
}
static size_t group_room(const RouteArgs& p, size_t v) {
    return p.groups > 1 ? (size_t)p.groups * ((p.E / p.groups) | 1) * v + p.groups * (v + 4) + 8 : 0;
}

// V: what choices are compared in, float for the logits themselves.
template <typename X, typename V, int LPT, int EPL>
__global__ __launch_bounds__(64) void route_kernel(RouteArgs p, int room) {
    constexpr int TOKENS = 64 / LPT;
    constexpr bool kByLogits = sizeof(V) == 4;
    __shared__ int s_ids[TOKENS][kMaxK];
    extern __shared__ __align__(8) char s_room[];
    const int sub = threadIdx.x % LPT, tok = threadIdx.x / LPT, first = sub * EPL;
    const int t = blockIdx.x * TOKENS + tok;
    const bool live = t < p.T;
    const X* row = (const X*)p.logits + (int64_t)(live ? t : p.T - 1) * p.ld;  // (lanes without a token do another's work)
    float x[EPL];
    load_logits<EPL>(row, first, p.E, x);
    V c[EPL];
    bool nan = false;
    float top = -kInf, sum = 0.0f;  // of the softmax
    if (p.softmax && (!kByLogits || !p.renormalize)) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) top = x[i] > top ? x[i] : top;
        top = token_max<LPT>(top);
        if constexpr (kByLogits) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) sum += x[i] > -kInf ? exp_below(x[i], top) : 0.0f;
            sum = token_sum<LPT>(sum);
        }
    }
    if constexpr (kByLogits) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            nan |= x[i] != x[i];
            c[i] = x[i] != x[i] ? kLowest : x[i];
        }
    } else {
        V total = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const V v = x[i];
            if (p.softmax) {
                c[i] = x[i] > -kInf ? exp_below(v, (V)top) : 0.0;
                total += c[i];
            } else {
                const V e = exp(-fabs(v));
                c[i] = (v >= 0.0 ? 1.0 : e) / (1.0 + e);
            }
        }
        if (p.softmax) total = token_sum<LPT>(total);
        sum = (float)total;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (p.softmax) c[i] = c[i] / total;
            const bool in = first + i < p.E;
            const float b = p.bias && in ? p.bias[first + i] : 0.0f;
            const bool bad = x[i] != x[i] || b != b;
            nan |= bad;
            const bool masked = x[i] == -kInf || b == -kInf || !in;
            c[i] = masked ? (V)-kInf : bad ? (V)kLowest : c[i] + (V)b;
        }
    }
    nan = token_ballot<LPT>(nan) != 0;
    if (p.groups > 1) keep_groups<V, LPT, EPL>(p, sub, c, s_room + tok * room);
    // K rounds
    V best;
    int at;
    auto look = [&]() INLINE {
        best = (V)-kInf;
        at = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const bool more = c[i] > best;
            best = more ? c[i] : best;
            at = more ? i : at;
        }
    };
    look();
    for (int k = 0; k < p.K; ++k) {
        const V most = token_max<LPT>(best);
        const uint64_t who = token_ballot<LPT>(best == most && best > (V)-kInf);
        const int winner = who ? __ffsll((unsigned long long)who) - 1 : -1;
        if (winner < 0 && sub == 0) s_ids[tok][k] = -1;
        if (sub == winner) {
            s_ids[tok][k] = first + at;
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] = i == at ? (V)-kInf : c[i];
            look();
        }
    }
    wave_fence();
    // weights: LPT of them at a time (K <= 64)
    constexpr int SLOTS = kMaxK / LPT;
    int id[SLOTS];
    float l[SLOTS], w[SLOTS];
    float high = -kInf;
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) {
        const int k = sub + u * LPT;
        id[u] = k < p.K ? s_ids[tok][k] : -1;
        l[u] = id[u] >= 0 ? to_f32(row[id[u]]) : -kInf;
        const float v = p.softmax ? l[u] : fminf(l[u], 0.0f);  // exp of it, up to 1 + exp(-|l|)
        high = v > high ? v : high;
    }
    if (p.renormalize) {
        high = token_max<LPT>(high);
        float all = 0.0f;
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            w[u] = 0.0f;
            if (id[u] >= 0) {
                w[u] = exp_below(p.softmax ? l[u] : fminf(l[u], 0.0f), high);
                if (!p.softmax) w[u] = __fdiv_rn(w[u], 1.0f + expf(-fabsf(l[u])));
            }
            all += w[u];
        }
        all = token_sum<LPT>(all);
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) w[u] = id[u] >= 0 ? __fdiv_rn(w[u], all) : 0.0f;
    } else {
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            w[u] = 0.0f;
            if (id[u] < 0) continue;
            const float e = p.softmax ? exp_below(l[u], top) : expf(-fabsf(l[u]));
            w[u] = p.softmax ? __fdiv_rn(e, sum) : __fdiv_rn(l[u] >= 0.0f ? 1.0f : e, 1.0f + e);
        }
    }
    if (!live) return;
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) {
        const int k = sub + u * LPT;
        if (k >= p.K) continue;
        p.ids[(int64_t)t * p.K + k] = id[u];
        p.weights[(int64_t)t * p.K + k] = nan ? __builtin_nanf("") : w[u] * p.scale;
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
// q = scale * dweights of the chosen, s their scores.
//   softmax renormalised: p = softmax over the chosen, dx_k = p_k (q_k - sum p q)
//   sigmoid renormalised: p = s / sum s,               dx_k = p_k (1 - s_k) (q_k - sum p q)
//   sigmoid:              dx_k = q_k s_k (1 - s_k)
//   softmax:              dx_j = s_j (q_j - sum_k s_k q_k) for every expert j
// 0 elsewhere. A choice outside [0, E) or of a -inf logit adds nothing; an expert chosen
// twice gets the sum. The choice itself has no gradient, so the bias has none either.
struct RouteGradArgs {
    const void* logits;
    int64_t ld;
    const int32_t* ids;
    const float* dweights;
    int T, E, K;
    int softmax, renormalize;
    float scale;
    void* dlogits;
    int64_t ld_out;
};

template <typename X, int LPT, int EPL>
__global__ __launch_bounds__(64) void route_grad_kernel(RouteGradArgs p) {
    constexpr int TOKENS = 64 / LPT, SLOTS = kMaxK / LPT;
    __shared__ int s_ids[TOKENS][kMaxK];
    __shared__ float s_q[TOKENS][kMaxK];
    __shared__ float s_row[TOKENS][LPT * EPL];
    const int sub = threadIdx.x % LPT, tok = threadIdx.x / LPT, first = sub * EPL;
    const int t = blockIdx.x * TOKENS + tok;
    const bool live = t < p.T, dense = p.softmax && !p.renormalize;
    const int64_t t0 = live ? t : p.T - 1;
    const X* row = (const X*)p.logits + t0 * p.ld;
    float x[EPL], top = -kInf, sum = 0.0f;
    if (dense) {
        load_logits<EPL>(row, first, p.E, x);
#pragma unroll
        for (int i = 0; i < EPL; ++i) top = x[i] > top ? x[i] : top;
        top = token_max<LPT>(top);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            x[i] = x[i] == -kInf ? 0.0f : exp_below(x[i], top);
            sum += x[i];
        }
        sum = token_sum<LPT>(sum);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) s_row[tok][first + i] = 0.0f;
    int id[SLOTS];
    float l[SLOTS], q[SLOTS], high = -kInf;
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) {
        const int k = sub + u * LPT;
        id[u] = k < p.K ? p.ids[t0 * p.K + k] : -1;
        if ((uint32_t)id[u] >= (uint32_t)p.E) id[u] = -1;
        l[u] = id[u] >= 0 ? to_f32(row[id[u]]) : -kInf;
        if (l[u] == -kInf) id[u] = -1;
        q[u] = id[u] >= 0 ? p.dweights[t0 * p.K + k] * p.scale : 0.0f;
        const float v = p.softmax ? l[u] : fminf(l[u], 0.0f);
        high = v > high ? v : high;
    }
    float d[SLOTS];
    if (p.renormalize) {
        high = token_max<LPT>(high);
        float w[SLOTS], rest[SLOTS], all = 0.0f, dot = 0.0f;
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            w[u] = 0.0f, rest[u] = 1.0f;
            if (id[u] >= 0) {
                w[u] = exp_below(p.softmax ? l[u] : fminf(l[u], 0.0f), high);
                if (!p.softmax) {
                    const float e = expf(-fabsf(l[u]));
                    w[u] = __fdiv_rn(w[u], 1.0f + e);
                    rest[u] = __fdiv_rn(l[u] >= 0.0f ? e : 1.0f, 1.0f + e);
                }
            }
            all += w[u];
        }
        all = token_sum<LPT>(all);
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            w[u] = id[u] >= 0 ? __fdiv_rn(w[u], all) : 0.0f;
            dot = __fmaf_rn(w[u], q[u], dot);
        }
        dot = token_sum<LPT>(dot);
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) d[u] = w[u] * rest[u] * (q[u] - dot);
    } else {
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            d[u] = q[u];
            if (!p.softmax && id[u] >= 0) {
                const float e = expf(-fabsf(l[u])), r = __fdiv_rn(1.0f, 1.0f + e);
                d[u] = q[u] * r * (e * r);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) {
        const int k = sub + u * LPT;
        if (k < p.K) s_ids[tok][k] = id[u], s_q[tok][k] = d[u];
    }
    wave_fence();
    // the first of equal ids takes the sum, k ascending
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) {
        const int k = sub + u * LPT;
        if (k >= p.K || id[u] < 0) continue;
        float v = 0.0f;
        bool mine = true;
        for (int j = 0; j < p.K; ++j)
            if (s_ids[tok][j] == id[u]) {
                mine &= j >= k;
                v += s_q[tok][j];
            }
        if (mine) s_row[tok][id[u]] = v;
    }
    wave_fence();
    float o[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) o[i] = s_row[tok][first + i];
    if (dense) {
        float dot = 0.0f;
        const float inv = sum > 0.0f || sum != sum ? __fdiv_rn(1.0f, sum) : 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            x[i] *= inv;
            dot = __fmaf_rn(x[i], o[i], dot);
        }
        dot = token_sum<LPT>(dot);
#pragma unroll
        for (int i = 0; i < EPL; ++i) o[i] = x[i] * (o[i] - dot);
    }
    if (!live) return;
    X* out = (X*)p.dlogits + t0 * p.ld_out;
    constexpr int V = 16 / sizeof(X);
    if constexpr (EPL % V == 0) {
        if (first + EPL <= p.E) {
#pragma unroll
            for (int g = 0; g < EPL / V; ++g) {
                Vec<X> v;
#pragma unroll
                for (int i = 0; i < V; ++i) v.e[i] = from_f32<X>(o[g * V + i]);
                store_vec<false>(out + first + g * V, v);
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (first + i < p.E) out[first + i] = from_f32<X>(o[i]);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Calls f(LPT, EPL) as integral constants for E experts.
template <typename F>
static void with_lanes(int E, F f) {
    using std::integral_constant;
    typedef integral_constant<int, 16> L16;
    typedef integral_constant<int, 64> L64;
    if (E <= 16) f(L16(), integral_constant<int, 1>());
    else if (E <= 32) f(L16(), integral_constant<int, 2>());
    else if (E <= 64) f(L16(), integral_constant<int, 4>());
    else if (E <= 128) f(L16(), integral_constant<int, 8>());
    else if (E <= 256) f(L16(), integral_constant<int, 16>());
    else if (E <= 512) f(L64(), integral_constant<int, 8>());
    else f(L64(), integral_constant<int, 16>());
}

template <typename X>
static hipError_t launch_route(const RouteArgs& p, hipStream_t s) {
    const bool by_logits = !p.bias && (p.groups == 1 || p.group_top == 1);
    with_lanes(p.E, [&](auto lpt, auto epl) {
        constexpr int LPT = decltype(lpt)::value, EPL = decltype(epl)::value, TOKENS = 64 / LPT;
        const dim3 grid((p.T + TOKENS - 1) / TOKENS);
        if (by_logits) {
            const int room = (int)((group_room(p, 4) + 7) / 8 * 8);
            hipLaunchKernelGGL((route_kernel<X, float, LPT, EPL>), grid, dim3(64), room * TOKENS, s, p, room);
        } else {
            const int room = (int)((group_room(p, 8) + 7) / 8 * 8);
            hipLaunchKernelGGL((route_kernel<X, double, LPT, EPL>), grid, dim3(64), room * TOKENS, s, p, room);
        }
    });
    return hipGetLastError();
}

template <typename X>
static hipError_t launch_route_grad(const RouteGradArgs& p, hipStream_t s) {
    with_lanes(p.E, [&](auto lpt, auto epl) {
        constexpr int LPT = decltype(lpt)::value, EPL = decltype(epl)::value, TOKENS = 64 / LPT;
        hipLaunchKernelGGL((route_grad_kernel<X, LPT, EPL>), dim3((p.T + TOKENS - 1) / TOKENS), dim3(64), 0, s, p);
    });
    return hipGetLastError();
}

static int check_route_sizes(int dtype, int T, int E, int K, int score, float scale) {
    if (!dtype_ok(dtype)) return reject(MOE_ERR_INVALID, "dtype=%d is not a moe_dtype", dtype);
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return reject(MOE_ERR_INVALID, "score=%d is not a moe_score", score);
    if (E < 1 || E > kMaxE) return reject(MOE_ERR_INVALID, "E=%d outside [1, %d]", E, kMaxE);
    if (K < 1 || K > kMaxK || K > E) return reject(MOE_ERR_INVALID, "K=%d outside [1, min(E, %d)]", K, kMaxK);
    if (T < 0) return reject(MOE_ERR_INVALID, "T=%d is negative", T);
    if ((long long)T * K > (long long)kMaxRows)
        return reject(MOE_ERR_UNSUPPORTED, "T*K=%lld routes above %lld", (long long)T * K, (long long)kMaxRows);
    if (!(scale > -3.4e38f && scale < 3.4e38f)) return reject(MOE_ERR_INVALID, "scale must be finite");
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_route(const void* logits, int64_t logits_stride, int32_t dtype, const float* bias, int32_t T, int32_t E,
                         int32_t K, int32_t score, int32_t groups, int32_t top_groups, int32_t group_top, int32_t renormalize,
                         float scale, int32_t* ids, float* weights, hipStream_t stream) {
    const int rc = check_route_sizes(dtype, T, E, K, score, scale);
    if (rc) return rc;
    if (groups < 1 || groups > E || E % groups) return reject(MOE_ERR_INVALID, "groups=%d must divide E=%d", groups, E);
    if (top_groups < 1 || top_groups > groups) return reject(MOE_ERR_INVALID, "top_groups=%d outside [1, %d]", top_groups, groups);
    if (group_top != 1 && group_top != 2) return reject(MOE_ERR_INVALID, "group_top must be 1 or 2");
    if (renormalize != 0 && renormalize != 1) return reject(MOE_ERR_INVALID, "renormalize must be 0 or 1");
    if (T == 0) return MOE_OK;
    if (!logits || !ids || !weights) return reject(MOE_ERR_INVALID, "NULL pointer argument");
    if (logits_stride < 0 || logits_stride > ((int64_t)1 << 32)) return reject(MOE_ERR_INVALID, "a row stride is out of range");
    const int es = dtype_bytes(dtype);
    if (!is_aligned(logits, es) || !is_aligned(bias, 4) || !is_aligned(ids, 4) || !is_aligned(weights, 4))
        return reject(MOE_ERR_INVALID, "misaligned pointer");
    const int64_t r4 = (int64_t)T * K * 4;
    const Bytes in[] = {matrix(logits, T, logits_stride, E, es), flat(bias, (int64_t)E * 4)}, out[] = {flat(ids, r4), flat(weights, r4)};
    for (const Bytes& o : out)
        for (const Bytes& i : in)
            if (overlap(i, o)) return reject(MOE_ERR_INVALID, "an output overlaps an input");
    if (overlap(out[0], out[1])) return reject(MOE_ERR_INVALID, "the outputs overlap");
    // (one group, or all of them: the groups decide nothing)
    if (top_groups == groups) groups = top_groups = 1;
    const RouteArgs p{logits, logits_stride, bias, T, E, K, score == MOE_SCORE_SOFTMAX, groups, top_groups, group_top, renormalize,
                      scale, ids, weights};
    hipError_t e;
    if (dtype == MOE_DT_BF16) e = launch_route<Bf16>(p, stream);
    else if (dtype == MOE_DT_FP16) e = launch_route<Fp16>(p, stream);
    else e = launch_route<float>(p, stream);
    return launched(e, "routing");
}

extern "C" int moe_route_grad(const float* dweights, const void* logits, int64_t logits_stride, int32_t dtype, const int32_t* ids,
                              int32_t T, int32_t E, int32_t K, int32_t score, int32_t renormalize, float scale, void* dlogits,
                              int64_t dlogits_stride, hipStream_t stream) {
    const int rc = check_route_sizes(dtype, T, E, K, score, scale);
    if (rc) return rc;
    if (renormalize != 0 && renormalize != 1) return reject(MOE_ERR_INVALID, "renormalize must be 0 or 1");
    if (T == 0) return MOE_OK;
    if (!dweights || !logits || !ids || !dlogits) return reject(MOE_ERR_INVALID, "NULL pointer argument");
    const int64_t far = (int64_t)1 << 32;
    if (logits_stride < 0 || logits_stride > far || dlogits_stride > far || (T > 1 && dlogits_stride < E))
        return reject(MOE_ERR_INVALID, "a row stride is out of range");
    const int es = dtype_bytes(dtype);
    if (!is_aligned(logits, es) || !is_aligned(dlogits, es) || !is_aligned(ids, 4) || !is_aligned(dweights, 4))
        return reject(MOE_ERR_INVALID, "misaligned pointer");
    const int64_t r4 = (int64_t)T * K * 4;
    const Bytes o = matrix(dlogits, T, dlogits_stride, E, es);
    for (const Bytes& i : {matrix(logits, T, logits_stride, E, es), flat(ids, r4), flat(dweights, r4)})
        if (overlap(i, o)) return reject(MOE_ERR_INVALID, "an output overlaps an input");
    const RouteGradArgs p{logits, logits_stride, ids, dweights, T, E, K, score == MOE_SCORE_SOFTMAX, renormalize, scale, dlogits,
                          dlogits_stride};
    hipError_t e;
    if (dtype == MOE_DT_BF16) e = launch_route_grad<Bf16>(p, stream);
    else if (dtype == MOE_DT_FP16) e = launch_route_grad<Fp16>(p, stream);
    else e = launch_route_grad<float>(p, stream);
    return launched(e, "routing gradient");
}
