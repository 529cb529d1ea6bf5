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
// A token belongs to LPT lanes of a wave, each of which holds EPL consecutive experts in
// registers. fp32 scores choose first: every expert gets a key of 32 bits, the choice as a
// fixed-point number on top of its inverted index, and K rounds of a maximum over keys
// below the last one pick the experts (keys differ, so no round needs to know its winner).
// That is the exact order unless two neighbours of it lie closer than the scores' error
// bound; then the wave goes on to the first gap and ranks these candidates by their exact
// values.
//
// Bound by the vector units: 16383 tokens, 256 experts, K = 8, fp32 (16.8 MB, 3.4 us of
// memory) 13 us by sigmoid and bias, 13.5 - 18 with 8 groups too (1235 vector instructions
// for four tokens, counted), 8 us by bf16 logits alone. With fp64 scores and 64-bit rounds
// throughout 28 us. A launch ends with its slowest wave, so what a few tokens need is kept
// short: a fallback of a whole wave of tokens to fp64 cost 8 us at the end (and what is left
// of it is the range above).
//
// Two kinds of tokens always need the exact choice, one after the other in their wave: those
// with equal groups at the border (padded rows of zeros with equal biases and sums of two:
// half of 16383 tokens such rows, 87 us), and those of whose experts one lies further above
// the rest than the keys reach (a bias of 3 for one expert, 90 us; with groups 100).
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

__device__ __forceinline__ float lane_value(float v, int l) { return lane_f32(v, l); }
__device__ __forceinline__ double lane_value(double v, int l) { return lane_f64(v, l); }

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
// A key's maximum over a token's lanes.
template <int LPT>
__device__ __forceinline__ uint32_t token_key_max(uint32_t v) {
    if constexpr (LPT == 64) return lanes_max(v);
    return row_max(v);
}
template <int EPL>
__device__ __forceinline__ int first_expert(int sub) { return sub * EPL; }
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

// Takes the experts of all but the top_groups best groups out of a token's c, the whole wave
// at it. LDS: `room` holds the choices (rows of a group padded to an odd length), G scores
// and G flags.
template <typename V, int EPL>
__device__ __forceinline__ void keep_groups(const RouteArgs& p, V* c, char* room) {
    const int lane = threadIdx.x & 63, G = p.groups, S = p.E / G, pad = S | 1, first = lane * EPL;
    V* choice = (V*)room;
    V* score = choice + G * pad;
    int* stays = (int*)(score + G);
    int g = first / S, at = first - g * S;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (first + i < p.E) choice[g * pad + at] = c[i];
        if (++at == S) at = 0, ++g;
    }
    wave_fence();
    int parts = 1;  // lanes of a group
    while (parts * 2 * G <= 64) parts *= 2;
    for (int h0 = 0; h0 < G; h0 += 64 / parts) {
        const int h = h0 + lane / parts;
        Top2<V> t{(V)-kInf, (V)-kInf};
        if (h < G)
            for (int j = lane % parts; j < S; j += parts) insert(t, choice[h * pad + j]);
        for (int off = 1; off < parts; off *= 2) {
            const V a = __shfl_xor(t.a, off), b = __shfl_xor(t.b, off);
            insert(t, a);
            insert(t, b);
        }
        if (h < G && lane % parts == 0) score[h] = p.group_top == 2 && t.b > (V)-kInf ? t.a + t.b : t.a;
    }
    wave_fence();
    for (int h = lane; h < G; h += 64) {
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
// Bytes of LDS for a token: its candidates (64 values and ids), or its groups.
static int token_room(const RouteArgs& p, size_t v) {
    const size_t groups = p.groups > 1 ? (size_t)p.groups * ((p.E / p.groups) | 1) * v + p.groups * (v + 4) : 0;
    return (int)((std::max(groups, (size_t)kMaxK * 12) + 7) / 8 * 8);
}

// The exact choice of one token, the whole wave at it (a few tokens of a launch need it, and
// the launch waits for them), by V: float for the logits themselves, else double. Leaves
// the ids in s_ids.
template <typename X, typename V, int EPL>
__device__ __forceinline__ void choose_exact(const RouteArgs& p, const X* row, float top, int* s_ids, char* room) {
    constexpr bool kByLogits = sizeof(V) == 4;
    const int lane = threadIdx.x & 63, first = lane * EPL;
    float x[EPL];
    load_logits<EPL>(row, first, p.E, x);
    V c[EPL], total = 0;
    if constexpr (kByLogits) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = x[i] != x[i] ? kLowest : x[i];
    } else {
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
        if (p.softmax) total = token_sum<64>(total);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (p.softmax) c[i] = c[i] / total;
            const bool in = first + i < p.E;
            const float b = p.bias && in ? p.bias[first + i] : 0.0f;
            const bool masked = x[i] == -kInf || b == -kInf || !in;
            c[i] = masked ? (V)-kInf : x[i] != x[i] || b != b ? (V)kLowest : c[i] + (V)b;
        }
    }
    if (p.groups > 1) keep_groups<V, EPL>(p, c, room);
    // K rounds; the lane that holds a round's winner looks for its next best
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
        const V most = token_max<64>(best);
        const uint64_t who = __ballot(best == most && best > (V)-kInf);
        const int winner = who ? __ffsll((unsigned long long)who) - 1 : -1;
        if (winner < 0 && lane == 0) s_ids[k] = -1;
        if (lane == winner) {
            s_ids[k] = first + at;
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] = i == at ? (V)-kInf : c[i];
            look();
        }
    }
    wave_fence();
}

// Whether groups can be scored in registers: a power of two of lanes each, in one row of 16.
__device__ __forceinline__ bool groups_of_lanes(int epl, int S) {
    const int n = S / epl;
    return S % epl == 0 && n <= 16 && (n & (n - 1)) == 0;
}

// The same by fp32 choices c (-inf: none). False if a group that stays lies within the error
// bound of one that goes: `slack` for the scores of both, and four roundings of each
// group's two choices (slack 0: c is exact, ties go to the lower group).
// A sum of two of the lowest values counts as the lowest, not as -inf: such a group has something
// to choose (and its error bound sends it to the exact choice).
__device__ __forceinline__ float group_score(const Top2<float>& t, int group_top) {
    return group_top == 2 && t.b > -kInf ? fmaxf(t.a + t.b, kLowest) : t.a;
}
__device__ __forceinline__ float lowest_of(float score, const Top2<float>& t, float slack) {
    return score - (slack + 0x1p-22f * (fabsf(t.a) + (t.b > -kInf ? fabsf(t.b) : 0.0f)));
}
__device__ __forceinline__ float highest_of(float score, const Top2<float>& t, float slack) {
    return score == -kInf ? score : score + (slack + 0x1p-22f * (fabsf(t.a) + (t.b > -kInf ? fabsf(t.b) : 0.0f)));
}
template <int LPT, int EPL>
__device__ __forceinline__ bool keep_groups_fast(const RouteArgs& p, int sub, float* c, char* room, float slack) {
    const int G = p.groups, S = p.E / G;
    bool mine_stays = true;
    float score;
    if (groups_of_lanes(EPL, S)) {
        const int n = S / EPL;  // lanes of a group
        Top2<float> t{-kInf, -kInf};
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            t.b = __builtin_amdgcn_fmed3f(t.a, t.b, c[i]);
            t.a = fmaxf(t.a, c[i]);
        }
        auto join = [&](float a, float b) INLINE {
            t.b = fmaxf(fminf(t.a, a), fmaxf(t.b, b));
            t.a = fmaxf(t.a, a);
        };
        if (n > 1) join(dpp_move<0xB1>(t.a), dpp_move<0xB1>(t.b));    // lane ^ 1
        if (n > 2) join(dpp_move<0x4E>(t.a), dpp_move<0x4E>(t.b));    // lane ^ 2
        if (n > 4) join(dpp_move<0x141>(t.a), dpp_move<0x141>(t.b));  // mirrored in 8 lanes
        if (n > 8) join(dpp_move<0x140>(t.a), dpp_move<0x140>(t.b));  // in 16
        score = group_score(t, p.group_top);
        if (first_expert<EPL>(sub) >= p.E) score = -kInf;
        int better = 0;
        // (lanes of the same group have the same score and are no better)
        auto against = [&](float o, int other) INLINE { better += o > score || (o == score && other / n < sub / n); };
        if constexpr (LPT == 64) {
            for (int g = 0; g < G; ++g) against(lane_f32(score, g * n), g * n);
        } else {
#define AGAINST(R) against(dpp_move<0x120 + R>(score), (int)dpp_move<0x120 + R>((uint32_t)sub))
        if (n < 2) { AGAINST(1); AGAINST(3); AGAINST(5); AGAINST(7); AGAINST(9); AGAINST(11); AGAINST(13); AGAINST(15); }
        if (n < 4) { AGAINST(2); AGAINST(6); AGAINST(10); AGAINST(14); }
        if (n < 8) { AGAINST(4); AGAINST(12); }
        if (n < 16) AGAINST(8);
#undef AGAINST
        }
        mine_stays = better < p.top_groups;
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = mine_stays ? c[i] : -kInf;
        if (slack == 0.0f) return true;
        const float in = token_all<LPT>(mine_stays ? lowest_of(score, t, slack) : kInf, [](float a, float b) INLINE { return a < b ? a : b; });
        const float out = token_max<LPT>(mine_stays ? -kInf : highest_of(score, t, slack));
        return out == -kInf || in > out;
    }
    // through the LDS, as in keep_groups
    const int pad = S | 1, first = sub * EPL;
    float* choice = (float*)room;
    float* scores = choice + G * pad;
    int* stays = (int*)(scores + G);
    int g = first / S, at = first - g * S;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (first + i < p.E) choice[g * pad + at] = c[i];
        if (++at == S) at = 0, ++g;
    }
    wave_fence();
    for (int h = sub; h < G; h += LPT) {
        Top2<float> t{-kInf, -kInf};
        for (int j = 0; j < S; ++j) {
            const float v = choice[h * pad + j];
            t.b = __builtin_amdgcn_fmed3f(t.a, t.b, v);
            t.a = fmaxf(t.a, v);
        }
        scores[h] = group_score(t, p.group_top);
        // (the group's own choices are no longer needed: its error bound instead)
        choice[h * pad] = lowest_of(scores[h], t, slack);
        if (S > 1) choice[h * pad + 1] = highest_of(scores[h], t, slack);
    }
    wave_fence();
    float in = kInf, out = -kInf;
    for (int h = sub; h < G; h += LPT) {
        const float mine = scores[h];
        int better = 0;
        for (int o = 0; o < G; ++o) better += scores[o] > mine || (scores[o] == mine && o < h);
        stays[h] = better < p.top_groups;
        const float lowest = choice[h * pad], highest = S > 1 ? choice[h * pad + 1] : mine + (mine - lowest);
        if (stays[h]) in = lowest < in ? lowest : in;
        else if (mine > -kInf) out = highest > out ? highest : out;
    }
    wave_fence();
    g = first / S, at = first - g * S;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (first + i < p.E && !stays[g]) c[i] = -kInf;
        if (++at == S) at = 0, ++g;
    }
    if (slack == 0.0f) return true;
    in = token_all<LPT>(in, [](float a, float b) INLINE { return a < b ? a : b; });
    out = token_max<LPT>(out);
    return out == -kInf || in > out;
}

// Keys: 10 bits of inverted index, above them the choice in 22 bits: the 16 bits of a 16-bit
// logit (exact), or (c - top) / reach + 1 as a fixed-point number (0 for everything more
// than `reach` below the token's top).
constexpr int kIndexBits = 10;
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1;
constexpr float kKeyUnits = 4194302.0f;  // 2^22 - 2: keys from 1 to 2^22 - 1
constexpr float kReachLogits = 32.0f, kReachScores = 2.0f;

// BY_LOGITS: the logits decide (no bias, no sums of two), else s + bias.
template <typename X, bool BY_LOGITS, int LPT, int EPL>
__global__ __launch_bounds__(64) void route_kernel(RouteArgs p, int room) {
    constexpr int TOKENS = 64 / LPT, SLOTS = kMaxK / LPT;
    constexpr bool kExactKeys = BY_LOGITS && sizeof(X) == 2;
    __shared__ int s_ids[TOKENS][kMaxK];
    extern __shared__ __align__(8) char s_room[];
    const int sub = threadIdx.x % LPT, tok = threadIdx.x / LPT, first = sub * EPL;
    const int t = blockIdx.x * TOKENS + tok;
    const bool live = t < p.T;
    const X* row = (const X*)p.logits + (int64_t)(live ? t : p.T - 1) * p.ld;  // (lanes without a token do another's work)
    float x[EPL], bias[EPL];
    load_logits<EPL>(row, first, p.E, x);
    auto load_bias = [&]() INLINE {
#pragma unroll
        for (int i = 0; i < EPL; ++i) bias[i] = 0.0f;
        if (p.bias) {
            if (first + EPL <= p.E) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) bias[i] = p.bias[first + i];
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (first + i < p.E) bias[i] = p.bias[first + i];
            }
        }
    };
    if (!BY_LOGITS) load_bias();
    bool nan = false;
    float top = -kInf, sum = 0.0f;  // of the softmax
    float c[EPL], slack = 0.0f;     // choices, and twice what they may be off
    if (p.softmax && (!BY_LOGITS || !p.renormalize)) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) top = fmaxf(top, x[i]);  // (fmaxf passes over a NaN)
        top = token_max<LPT>(top);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            c[i] = x[i] > -kInf ? exp_below(x[i], top) : 0.0f;
            sum += c[i];
        }
        sum = token_sum<LPT>(sum);
    }
    if constexpr (BY_LOGITS) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            nan |= x[i] != x[i];
            c[i] = x[i] != x[i] ? kLowest : x[i];
        }
    } else {
        // sigmoid: exp and reciprocal 1 ulp each, x log2(e) rounded (s (1 - s) |x| <= 0.23): below
        // 2^-22. softmax: an exponent's rounding (0.37 2^-24), exp, 30 additions and the
        // division: below 2^-19 of the largest score, 1 / sum
        const float inv = p.softmax ? __fdiv_rn(1.0f, sum) : 0.0f;
        slack = p.softmax ? 0x1p-18f * inv : 0x1p-21f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float s = p.softmax ? c[i] * inv : __builtin_amdgcn_rcpf(1.0f + __expf(-x[i]));
            const bool bad = x[i] != x[i] || bias[i] != bias[i], masked = x[i] == -kInf || bias[i] == -kInf;
            nan |= bad;
            c[i] = masked ? -kInf : bad ? kLowest : s + bias[i];
        }
    }
    nan = token_ballot<LPT>(nan) != 0;
    bool sure = true;
    if (p.groups > 1) sure = keep_groups_fast<LPT, EPL>(p, sub, c, s_room + tok * room, slack);
    // keys
    uint32_t key[EPL];
    float high = 0.0f;
    constexpr float kReach = BY_LOGITS ? kReachLogits : kReachScores;
    if constexpr (!kExactKeys) {
        high = c[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) high = fmaxf(high, c[i]);
        high = token_max<LPT>(high);
        sure &= high < 1e30f;  // (infinities, and rows of lowest values: by the exact choice)
    }
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        uint32_t q;
        if constexpr (kExactKeys) {
            const uint32_t b = f2u(c[i] + 0.0f);  // (-0 and 0 are one logit)
            uint32_t o;
            if constexpr (std::is_same<X, Bf16>::value) o = ((b & 0x80000000u) ? ~b : b | 0x80000000u) >> 16;
            else {
                // fp16: its own bits (a NaN counts as the lowest finite value)
                const uint32_t h = __builtin_bit_cast(uint16_t, (_Float16)fmaxf(c[i] + 0.0f, -65504.0f));
                o = (h & 0x8000u) ? ~h & 0xFFFFu : h | 0x8000u;
            }
            q = o + 1;
        } else {
            q = (uint32_t)fmaxf(__fmaf_rn(c[i] - high, kKeyUnits / kReach, kKeyUnits), 0.0f) + 1;
        }
        key[i] = c[i] > -kInf ? (q << kIndexBits) | (kIndexMask - (first + i)) : 0;
        best = max(best, key[i]);
    }
    // candidate k of the token in lane k % LPT, slot k / LPT
    uint32_t mine[SLOTS], last = 0xFFFFFFFFu, end_gap = 0;
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) mine[u] = 0;
    auto next_key = [&]() INLINE {
        const uint32_t before = last;
        last = token_key_max<LPT>(best);
        end_gap = (before >> kIndexBits) - (last >> kIndexBits);
        best = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) best = max(best, key[i] < last ? key[i] : 0);
    };
    int found = 0;
    // candidates up to number `end`; while(more()) for those behind it
    auto pick = [&](int end, auto more) INLINE {
#pragma unroll
        for (int u = 0; u < SLOTS; ++u)
            while (found < min(end, (u + 1) * LPT) && found >= u * LPT && more()) {
                next_key();
                if (sub == found - u * LPT) mine[u] = last;
                ++found;
            }
    };
    pick(p.K, [] { return true; });
    // weights: LPT of them at a time (K <= 64)
    int id[SLOTS];
    float l[SLOTS], w[SLOTS];
    auto look_up = [&]() INLINE {
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) l[u] = id[u] >= 0 ? to_f32(row[id[u]]) : -kInf;
    };
    auto ids_of = [&](int end) INLINE {
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) id[u] = sub + u * LPT < end && mine[u] ? (int)(kIndexMask - (mine[u] & kIndexMask)) : -1;
        look_up();
    };
    ids_of(p.K);
    if constexpr (!kExactKeys) {
        // Neighbours closer than the bound: two units for the keys' own roundings and two for their
        // truncation, the scores' error and the addition's. The first key that was not taken
        // (`best`'s maximum) is the last one's neighbour.
        const float bound = 4.0f + (slack + (BY_LOGITS ? 0.0f : 0x1p-22f * (fabsf(high) + kReach))) * (kKeyUnits / kReach);
        const uint32_t limit = (uint32_t)fminf(bound, 4.0e9f);
        auto near = [&](uint32_t above, uint32_t below) INLINE {
            return above && below && (above >> kIndexBits) - (below >> kIndexBits) <= limit;
        };
        // The same logit and bias make the same key but for the index, which decides then: these two
        // stand as they are, but say nothing of what follows them. Among the keys taken the next
        // pair does; across the last place, the first key behind it of another choice.
        auto too_close = [&](uint32_t above, uint32_t below) INLINE {
            if (!near(above, below)) return false;
            const int i = kIndexMask - (above & kIndexMask), j = kIndexMask - (below & kIndexMask);
            return to_f32(row[i]) != to_f32(row[j]) || (!BY_LOGITS && p.bias && p.bias[i] != p.bias[j]);
        };
        const uint32_t rest = token_key_max<LPT>(best);
        bool close = too_close(last, rest);
        const bool run = !close && near(last, rest);
        if (__ballot(run)) {
            asm volatile("" ::: "memory");  // (loads again, instead of registers for the biases until here)
            load_logits<EPL>(row, first, p.E, x);
            if (!BY_LOGITS) load_bias();
            const int at = run ? kIndexMask - (last & kIndexMask) : 0;
            const float l = to_f32(row[at]), b = !BY_LOGITS && p.bias ? p.bias[at] : 0.0f;
            uint32_t other = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (key[i] < last && (x[i] != l || (!BY_LOGITS && bias[i] != b))) other = max(other, key[i]);
            close |= run && near(last, token_key_max<LPT>(other));
        }
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            if (u * LPT >= p.K) continue;
            // the key before this lane's: of the lane below, or of the last lane's slot before
            uint32_t prior = (uint32_t)__shfl((int)mine[u], (threadIdx.x & 63) - 1);
            const uint32_t wrap = u ? (uint32_t)__shfl((int)mine[u ? u - 1 : 0], (threadIdx.x & 63) | (LPT - 1)) : 0;
            prior = sub ? prior : wrap;
            if (sub + u * LPT < p.K) close |= too_close(prior, mine[u]);
        }
        if (__ballot(close || !sure)) {
            // Candidates up to one that lies behind a gap, ranked by exact values. Where 64 of them
            // hold no gap, or groups are close: all experts by exact values.
            end_gap = 0;
            pick(kMaxK, [&]() INLINE { return __ballot(last && end_gap <= limit) != 0; });
            const uint32_t open = token_key_max<LPT>(best);
            const bool all = !sure || (found == kMaxK && end_gap <= limit && open && (last >> kIndexBits) - (open >> kIndexBits) <= limit);
            {
                ids_of(found);
                double total = 1.0;
                if (!BY_LOGITS && p.softmax) {
                    total = 0.0;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) total += x[i] > -kInf ? exp_below((double)x[i], (double)top) : 0.0;
                    total = token_sum<LPT>(total);
                }
                double* s_exact = (double*)(s_room + tok * room);
                int* s_who = (int*)(s_exact + kMaxK);
                double exact[SLOTS];
#pragma unroll
                for (int u = 0; u < SLOTS; ++u) {
                    exact[u] = -kInf;
                    if (id[u] < 0) continue;
                    const double v = l[u];
                    if (BY_LOGITS) {
                        exact[u] = v;
                    } else {
                        const double e = p.softmax ? exp_below(v, (double)top) : exp(-fabs(v));
                        exact[u] = p.softmax ? e / total : (v >= 0.0 ? 1.0 : e) / (1.0 + e);
                        exact[u] += p.bias ? (double)p.bias[id[u]] : 0.0;
                    }
                    exact[u] = exact[u] != exact[u] ? (double)kLowest : exact[u];
                }
#pragma unroll
                for (int u = 0; u < SLOTS; ++u) {
                    if (sub + u * LPT < p.K) s_ids[tok][sub + u * LPT] = -1;
                    s_exact[sub + u * LPT] = exact[u];
                    s_who[sub + u * LPT] = id[u];
                }
                wave_fence();
#pragma unroll
                for (int u = 0; u < SLOTS; ++u) {
                    if (id[u] < 0) continue;
                    int rank = 0;
                    for (int j = 0; j < found; ++j) {
                        const int other = s_who[j];
                        const double v = s_exact[j];
                        rank += other >= 0 && (v > exact[u] || (v == exact[u] && other < id[u]));
                    }
                    if (rank < p.K) s_ids[tok][rank] = id[u];
                }
                wave_fence();
            }
            for (uint64_t left = __ballot(all && sub == 0); left; left &= left - 1) {
                const int l = __ffsll((unsigned long long)left) - 1;
                choose_exact<X, typename std::conditional<BY_LOGITS, float, double>::type, LPT * EPL / 64 ? LPT * EPL / 64 : 1>(
                    p, (const X*)p.logits + (int64_t)min((int)blockIdx.x * TOKENS + l / LPT, p.T - 1) * p.ld, lane_f32(top, l),
                    s_ids[l / LPT], s_room + l / LPT * room);
            }
#pragma unroll
            for (int u = 0; u < SLOTS; ++u) id[u] = sub + u * LPT < p.K ? s_ids[tok][sub + u * LPT] : -1;
            look_up();
        }
    }
    if (p.renormalize) {
        float most = -kInf, all = 0.0f;
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) most = fmaxf(most, p.softmax ? l[u] : fminf(l[u], 0.0f));  // exp of it, up to 1 + exp(-|l|)
        most = token_max<LPT>(most);
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            w[u] = 0.0f;
            if (id[u] >= 0) {
                w[u] = exp_below(p.softmax ? l[u] : fminf(l[u], 0.0f), most);
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
// Calls f(LPT, EPL) as integral constants for E experts: 16 lanes a token up to 256 experts,
// else (and for few tokens) all 64.
template <typename F>
static void with_lanes(int E, bool few, F f) {
    using std::integral_constant;
    typedef integral_constant<int, 16> L16;
    typedef integral_constant<int, 64> L64;
    if (E <= 16) f(L16(), integral_constant<int, 1>());
    else if (E <= 32) f(L16(), integral_constant<int, 2>());
    else if (E <= 64) f(L16(), integral_constant<int, 4>());
    else if (E <= 128 && !few) f(L16(), integral_constant<int, 8>());
    else if (E <= 256 && !few) f(L16(), integral_constant<int, 16>());
    else if (E <= 128) f(L64(), integral_constant<int, 2>());
    else if (E <= 256) f(L64(), integral_constant<int, 4>());
    else if (E <= 512) f(L64(), integral_constant<int, 8>());
    else f(L64(), integral_constant<int, 16>());
}
// (256 experts, sigmoid and bias, 64 lanes a token against 16, us: 64 tokens 3.7 / 5.2, 1024
// tokens 5.4 / 7.3, 16383 tokens 15.5 / 12.3)
constexpr int kFewTokens = 1024;

template <typename X>
static hipError_t launch_route(const RouteArgs& p, hipStream_t s) {
    const bool by_logits = !p.bias && (p.groups == 1 || p.group_top == 1);
    with_lanes(p.E, p.T <= kFewTokens, [&](auto lpt, auto epl) {
        constexpr int LPT = decltype(lpt)::value, EPL = decltype(epl)::value, TOKENS = 64 / LPT;
        const dim3 grid((p.T + TOKENS - 1) / TOKENS);
        const int room = token_room(p, by_logits ? 4 : 8);
        if (by_logits) hipLaunchKernelGGL((route_kernel<X, true, LPT, EPL>), grid, dim3(64), room * TOKENS, s, p, room);
        else hipLaunchKernelGGL((route_kernel<X, false, LPT, EPL>), grid, dim3(64), room * TOKENS, s, p, room);
    });
    return hipGetLastError();
}

template <typename X>
static hipError_t launch_route_grad(const RouteGradArgs& p, hipStream_t s) {
    with_lanes(p.E, false, [&](auto lpt, auto epl) {
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
