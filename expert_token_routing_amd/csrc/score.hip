// Routing by scores: the router whose choice and weights come from softmax or
// sigmoid scores, with a bias that acts on the choice alone, expert groups
// chosen first and renormalised weights; its gradient; and the step of the
// bias that evens the experts' load.
//
// Mathematics, for a token with logits l and bias b:
//   s = softmax(l) or 1 / (1 + exp(-l)),  c = s + b (an order like l without b)
//   a group's score: its best c, or the sum of its best two
//   the top groups, then the top k experts by c in them, ties to the lower index
//   w_j = scale s_j / (sum over the chosen s, or 1)
// and from the gradient dw of w, the choice held fixed, with r_j = s_j / sum s:
//   sigmoid:  dl_j = scale r_j (1 - s_j) (dw_j - sum_i dw_i r_i), or
//             dl_j = scale s_j (1 - s_j) dw_j where weights are not renormalised
//   softmax:  dl_j = scale r_j (dw_j - sum_i dw_i r_i) on the chosen, or
//             dl_e = scale p_e ([chosen] dw_e - sum_i dw_i p_i) on every expert
#include <algorithm>

#include "launch.h"

namespace occ {
namespace {

constexpr int kScoreThreads = 256;
constexpr unsigned kScoreGrid = 1 << 20;  // workgroups; more tokens loop

// A double's place in the order of the doubles, above 0; NaN reads as -inf.
__device__ __forceinline__ uint64_t order_key(double v) {
    v = v == v ? v + 0. : -INFINITY;
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return b >> 63 ? ~b : b | 1ull << 63;
}

template <int L, typename V, typename F>
__device__ __forceinline__ V team_reduce(V v, F f) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = f(v, __shfl_xor(v, o));
    return v;
}

// A float's place in the order of the floats, above 0, and back; NaN reads as -inf.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v == v ? v + 0.f : -INFINITY);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_key(uint32_t k) {
    return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
}

// LDS written by some lanes of a wave and read by others of it.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int L>
__device__ __forceinline__ uint32_t team_max(uint32_t v) {
    const auto larger = [](uint32_t x, uint32_t y) { return max(x, y); };
    v = group_reduce<16>(v, larger);
    if constexpr (L == 64) {
        v = max(v, static_cast<uint32_t>(dpp_i<kDppRowBcast15, 0xa>(0, static_cast<int>(v))));
        v = max(v, static_cast<uint32_t>(dpp_i<kDppRowBcast31, 0xc>(0, static_cast<int>(v))));
        v = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
    }
    return v;
}
template <int L>
__device__ __forceinline__ float team_sum(float v) {
    if constexpr (L == 64) return wave_sum(v);
    else return group_sum<L>(v);
}
// Whether it holds in a lane of the team: bit i for its lane i.
template <int L>
__device__ __forceinline__ uint64_t team_ballot(bool v) {
    const uint64_t all = __ballot(v);
    if constexpr (L == 64) return all;
    else return all >> (lane_id() / L * L) & ((1ull << L) - 1);
}

// How a team of L lanes walks the groups: GL lanes a group, `per` groups at once.
template <int L>
struct GroupWalk {
    int shift, per;  // GL = 1 << shift
    __device__ explicit GroupWalk(int Nd) {
        int s = L == 64 ? 6 : 4;
        while (s > 0 && (L >> s) < Nd) s--;
        shift = s;
        per = L >> s;
    }
};

// A token's LDS: the choice by place (a group's places together, groups
// n + 1 apart: other banks), the groups' scores, and what was chosen.
template <int L, int NI>
struct TokenLds {
    double choice[L * NI + kMaxNd];
    double group[kMaxNd];
};

// The best two of two pairs.
template <typename V>
__device__ __forceinline__ void best_two(V &a, V &b, V c, V d) {
    const V lo = a < c ? a : c, hi = a < c ? c : a;
    const V next = b < d ? d : b;
    a = hi;
    b = lo < next ? next : lo;
}

// The groups' scores from the choice in LDS, one after another `per` groups;
// f(g, score) for each (in all its lanes; past the last group, g >= Nd).
template <int L, typename V, typename F>
__device__ __forceinline__ void group_scores(const V *choice, int Nd, int n, int group_best, F f) {
    const GroupWalk<L> walk(Nd);
    const int l = threadIdx.x % L, i = l & ((1 << walk.shift) - 1);
    for (int g0 = 0; g0 < Nd; g0 += walk.per) {
        const int g = g0 + (l >> walk.shift);
        V top = -INFINITY, next = -INFINITY;
        if (g < Nd)
            for (int j = i; j < n; j += 1 << walk.shift)
                best_two(top, next, choice[g * (n + 1) + j], static_cast<V>(-INFINITY));
        for (int o = 1; o < 1 << walk.shift; o <<= 1) {
            const V ot = __shfl_xor(top, o), on = __shfl_xor(next, o);
            best_two(top, next, ot, on);
        }
        f(g, group_best > 1 && next > -INFINITY ? top + next : top);
    }
}

// What a lane knows of its experts: at places l + L j of the placement where
// groups matter (which puts a group's experts together), of 0..Ne-1 otherwise.
template <int NI>
struct Experts {
    int e[NI];
    float v[NI], b[NI];  // logit (-inf for one that is left out), bias
};

// A softmax's terms over the largest logit m; a logit of -inf has none.
__device__ __forceinline__ double exp_over(float v, float m) {
    return v == -INFINITY ? 0. : v == m ? 1. : exp(static_cast<double>(v) - static_cast<double>(m));
}
__device__ __forceinline__ double sigmoid64(float v) {
    const double e = exp(-fabs(static_cast<double>(v)));
    return (v < 0.f ? e : 1.) / (1. + e);
}

// The choice in 64 bits throughout, for the tokens whose choice 32 bits cannot
// tell: s_ids and s_v, the k chosen experts and their logits in order.
template <int L, int NI, bool GROUPS>
__device__ __forceinline__ void choose64(const ScoreArgs &a, const Experts<NI> &x,
                                                   TokenLds<L, NI> &lds, int *s_ids, float *s_v) {
    const int l = threadIdx.x % L, Ne = a.Ne, n = a.tab.n, Nd = a.tab.Nd;
    double c[NI];
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < NI; j++) c[j] = sigmoid64(x.v[j]);
    } else {
        float m = x.v[0];
#pragma unroll
        for (int j = 1; j < NI; j++) m = fmaxf(m, x.v[j]);
        m = team_reduce<L>(m, [](float p, float q) { return fmaxf(p, q); });
        double sum = 0.;
#pragma unroll
        for (int j = 0; j < NI; j++) {
            c[j] = exp_over(x.v[j], m);
            sum += c[j];
        }
        sum = team_reduce<L>(sum, [](double p, double q) { return p + q; });
#pragma unroll
        for (int j = 0; j < NI; j++) c[j] = sum > 0. ? c[j] / sum : 0.;
    }
#pragma unroll
    for (int j = 0; j < NI; j++) c[j] = x.v[j] == -INFINITY ? -INFINITY : c[j] + x.b[j];
    uint64_t allowed = ~0ull;
    if constexpr (GROUPS) {
#pragma unroll
        for (int j = 0; j < NI; j++) {
            const int p = l + L * j;
            if (p < Ne) lds.choice[p + p / n] = c[j];
        }
        wave_sync();
        group_scores<L>(lds.choice, Nd, n, a.group_best, [&](int g, double v) {
            if (g < Nd) lds.group[g] = v;
        });
        wave_sync();
        allowed = 0;
        for (int g = l; g < Nd; g += L) {
            const double v = lds.group[g];
            int ahead = 0;
            for (int o = 0; o < Nd; o++) {
                const double y = lds.group[o];
                ahead += y > v || (y == v && o < g);
            }
            if (ahead < a.top_groups) allowed |= 1ull << g;
        }
        allowed = team_reduce<L>(allowed, [](uint64_t p, uint64_t q) { return p | q; });
    }
    uint64_t key[NI];
#pragma unroll
    for (int j = 0; j < NI; j++) {
        const int p = l + L * j;
        bool ok = p < Ne;
        if constexpr (GROUPS) ok = ok && allowed >> (p / n) & 1;
        key[j] = ok ? order_key(a.bias ? c[j] : static_cast<double>(x.v[j])) : 0;
    }
    for (int i = 0; i < a.k; i++) {
        uint64_t best = 0;
        int who = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < NI; j++)
            if (key[j] > best || (key[j] == best && x.e[j] < who)) {
                best = key[j];
                who = x.e[j];
            }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            const uint64_t ob = __shfl_xor(best, o);
            const int ow = __shfl_xor(who, o);
            if (ob > best || (ob == best && ow < who)) {
                best = ob;
                who = ow;
            }
        }
#pragma unroll
        for (int j = 0; j < NI; j++)
            if (key[j] && x.e[j] == who) {
                key[j] = 0;
                s_ids[i] = who;
                s_v[i] = x.v[j];
            }
    }
    wave_sync();
}

// A team of L lanes a token, NI experts a lane.  A choice is a border, and near
// ties would fall differently in 32 bits than in 64 for a token in some
// thousands.  Scores in 32 bits are off by less than half of margin(c), so a
// choice whose neighbours (the chosen, the first not chosen, the groups at
// their border) lie further apart is the one that 64 bits make; logits alone
// order without an error, and experts of equal logit and bias tie in both.  The
// tokens that are left take choose64.  The chosen experts' scores and the
// weights are formed in 64 bits, a lane an expert.
constexpr float kMargin = 0x1p-18f;
template <int L, int NI, bool GROUPS>
__global__ __launch_bounds__(kScoreThreads) void k_route_scored(ScoreArgs a) {
    constexpr int TOK = kScoreThreads / L, KPL = L == 64 ? 1 : kMaxK / L;
    __shared__ TokenLds<L, NI> s_lds[GROUPS ? TOK : 1];
    __shared__ float s_v[TOK][kMaxK + 1], s_b[TOK][kMaxK + 1], s_c[TOK][kMaxK + 1];
    __shared__ int s_ids[TOK][kMaxK + 1];
    const int l = threadIdx.x % L, q = threadIdx.x / L;
    const int Ne = a.Ne, k = a.k, n = a.tab.n, Nd = a.tab.Nd;
    const bool biased = a.bias != nullptr;
    for (size_t t0 = static_cast<size_t>(blockIdx.x) * TOK; t0 < static_cast<size_t>(a.T);
         t0 += static_cast<size_t>(gridDim.x) * TOK) {
        const size_t t = t0 + q;
        const bool live = t < static_cast<size_t>(a.T);
        const float *row = a.logits + (live ? t : a.T - 1) * Ne;
        Experts<NI> x;
#pragma unroll
        for (int j = 0; j < NI; j++) {
            const int p = min(l + L * j, Ne - 1);
            x.e[j] = GROUPS && !a.in_order ? a.tab.expert[p] : p;
            x.v[j] = row[x.e[j]];
            x.b[j] = biased ? a.bias[x.e[j]] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < NI; j++)
            if (!(l + L * j < Ne) || x.v[j] != x.v[j]) x.v[j] = -INFINITY;
        float top = 0.f;  // the largest logit, for a softmax
        if (!a.sigmoid) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < NI; j++) m = max(m, order_key(x.v[j]));
            top = from_key(team_max<L>(m));
        }
        float c[NI];
        bool sure = true;
        if (GROUPS || biased) {
            if (a.sigmoid) {
#pragma unroll
                for (int j = 0; j < NI; j++) {
                    const float e = __expf(-fabsf(x.v[j]));
                    c[j] = (x.v[j] < 0.f ? e : 1.f) * __builtin_amdgcn_rcpf(1.f + e);
                }
            } else {
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < NI; j++) {
                    c[j] = x.v[j] == -INFINITY ? 0.f : x.v[j] == top ? 1.f : __expf(x.v[j] - top);
                    sum += c[j];
                }
                sum = team_sum<L>(sum);
                const float inv = sum > 0.f ? __builtin_amdgcn_rcpf(sum) : 0.f;
#pragma unroll
                for (int j = 0; j < NI; j++) c[j] *= inv;
            }
#pragma unroll
            for (int j = 0; j < NI; j++) c[j] = x.v[j] == -INFINITY ? -INFINITY : c[j] + x.b[j];
        }
        uint32_t key[NI];
#pragma unroll
        for (int j = 0; j < NI; j++) key[j] = l + L * j < Ne ? order_key(biased ? c[j] : x.v[j]) : 0u;
        if constexpr (GROUPS) {
            float *choice = reinterpret_cast<float *>(s_lds[q].choice), *group = reinterpret_cast<float *>(s_lds[q].group);
            int g_of[NI];
#pragma unroll
            for (int j = 0; j < NI; j++) {
                const int p = l + L * j;
                g_of[j] = p * a.over_n >> 16;
                if (p < Ne) choice[p + g_of[j]] = c[j];
            }
            wave_sync();
            group_scores<L>(choice, Nd, n, a.group_best, [&](int g, float v) {
                if (g < Nd) group[g] = v;
            });
            wave_sync();
            uint64_t allowed = 0;
            for (int g0 = 0; g0 < Nd; g0 += L) {
                const float v = g0 + l < Nd ? group[g0 + l] : -INFINITY;
                const float off = 2.f * kMargin * (1.f + fabsf(v));
                int ahead = 0, near = 0;  // surely; perhaps
                for (int o = 0; o < Nd; o++) {
                    const float y = group[o];
                    ahead += y - v > off;
                    near += !(v - y > off) && o != g0 + l;
                }
                const bool in = near < a.top_groups, out = ahead >= a.top_groups;
                sure = sure && (g0 + l >= Nd || in || out);
                allowed |= team_ballot<L>(in && g0 + l < Nd) << g0;
            }
            sure = team_ballot<L>(!sure) == 0;
#pragma unroll
            for (int j = 0; j < NI; j++)
                if (!(allowed >> g_of[j] & 1)) key[j] = 0;
        }
        // one more than k where the choice's border has to be looked at
        const int rounds = biased ? k + 1 : k;
        for (int i = 0; i < rounds; i++) {
            uint32_t best = key[0];
#pragma unroll
            for (int j = 1; j < NI; j++) best = max(best, key[j]);
            best = team_max<L>(best);
            uint32_t low = 0;  // the lowest expert that has it, as 256 - e
#pragma unroll
            for (int j = NI - 1; j >= 0; j--) low = key[j] == best ? max(low, 256u - x.e[j]) : low;
            const uint64_t with = team_ballot<L>(low != 0);
            // (wave-uniform: a lane alone has it in every team, as nearly always)
            if (__ballot((with & (with - 1)) != 0)) low = low == team_max<L>(low) ? low : 0;
#pragma unroll
            for (int j = 0; j < NI; j++)
                if (low && key[j] == best && 256u - x.e[j] == low) {
                    key[j] = 0;
                    s_ids[q][i] = x.e[j];
                    s_v[q][i] = x.v[j];
                    if (biased) {
                        s_b[q][i] = x.b[j];
                        s_c[q][i] = best ? c[j] : -INFINITY;
                    }
                }
        }
        wave_sync();
        if (biased) {
#pragma unroll
            for (int i = 0; i < KPL; i++) {
                const int o = l + L * i + 1;  // against the one in front
                if (o <= k) {
                    const float c0 = s_c[q][o - 1], c1 = s_c[q][o];
                    const bool same = s_v[q][o - 1] == s_v[q][o] && s_b[q][o - 1] == s_b[q][o];
                    if (c0 - c1 <= kMargin * (1.f + fabsf(c0)) && !same) sure = false;
                }
            }
        }
        if (__ballot(!sure)) {
            wave_sync();
            choose64<L, NI, GROUPS>(a, x, s_lds[GROUPS ? q : 0], s_ids[q], s_v[q]);
        }
        // Renormalised, scores are taken over the largest that was chosen, so
        // that none of them vanishes in the sum: softmax terms over its logit;
        // sigmoids as they are but where all of them are below e^-600.
        double s[KPL], sum = 0.;
        float m = top;
        if (a.renormalise) {
            m = -INFINITY;
#pragma unroll
            for (int i = 0; i < KPL; i++)
                if (l + L * i < k) m = fmaxf(m, s_v[q][l + L * i]);
            m = from_key(team_max<L>(order_key(m)));
        }
        const bool deep = a.sigmoid && a.renormalise && m < -600.f;
#pragma unroll
        for (int i = 0; i < KPL; i++) {
            const float v = l + L * i < k ? s_v[q][l + L * i] : -INFINITY;
            s[i] = a.sigmoid && !deep ? sigmoid64(v) : exp_over(v, m);
            sum += s[i];
        }
        if (!a.renormalise) {
            sum = 0.;
            if (!a.sigmoid) {
#pragma unroll
                for (int j = 0; j < NI; j++) sum += exp_over(x.v[j], top);
            }
        }
        if (a.renormalise || !a.sigmoid) sum = team_reduce<L>(sum, [](double y, double z) { return y + z; });
        else sum = 1.;
        const double over = sum > 0. ? sum : INFINITY;
#pragma unroll
        for (int i = 0; i < KPL; i++)
            if (live && l + L * i < k) {
                a.ids[t * k + l + L * i] = s_ids[q][l + L * i];
                a.w[t * k + l + L * i] = static_cast<float>(a.scale * (s[i] / over));
            }
        wave_sync();
    }
}

// The gradient: a team of L lanes a token, lane j < k (and j + L) with the
// token's j-th expert, then lane l with experts l + L i of the row.
template <int L, int NI, bool FULL>
__global__ __launch_bounds__(kScoreThreads) void k_route_scored_back(
    const float *logits, const int32_t *__restrict__ ids, const float *__restrict__ dw,
    const float *dlogits_in, int T, int Ne, int k, int sigmoid, int renormalise, float scale,
    float *dlogits) {
    constexpr int KPL = kMaxK / L > 0 ? kMaxK / L : 1;  // slots a lane
    const int l = threadIdx.x % L;
    for (size_t t = static_cast<size_t>(blockIdx.x) * (kScoreThreads / L) + threadIdx.x / L; t < static_cast<size_t>(T);
         t += static_cast<size_t>(gridDim.x) * (kScoreThreads / L)) {  // a team's lanes leave together
    const auto add = [](float x, float y) { return x + y; };
    const auto most = [](float x, float y) { return fmaxf(x, y); };
    int id[KPL];
    float g[KPL], x[KPL];
#pragma unroll
    for (int i = 0; i < KPL; i++) {
        const int j = l + L * i;
        id[i] = j < k ? ids[t * k + j] : -1;
        if (id[i] < 0 || id[i] >= Ne) id[i] = -1;
        g[i] = id[i] < 0 ? 0.f : dw[t * k + j];
        x[i] = id[i] < 0 ? -INFINITY : logits[t * Ne + id[i]];
        if (x[i] != x[i]) x[i] = -INFINITY;
    }
    float p[NI], in[NI];
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const size_t at = t * Ne + min(l + L * i, Ne - 1);
        in[i] = dlogits_in ? dlogits_in[at] : 0.f;
        if constexpr (FULL) p[i] = l + L * i < Ne ? logits[at] : -INFINITY;
    }
    float sub = 0.f;  // FULL: what every expert's gradient has less
    if constexpr (FULL) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            p[i] = p[i] == p[i] ? p[i] : -INFINITY;
            m = fmaxf(m, p[i]);
        }
        m = team_reduce<L>(m, most);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            p[i] = p[i] == -INFINITY ? 0.f : p[i] == m ? 1.f : __expf(p[i] - m);
            sum += p[i];
        }
        sum = team_reduce<L>(sum, add);
        const float inv = sum > 0.f ? scale / sum : 0.f, unit = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int i = 0; i < KPL; i++)
            sub += x[i] == -INFINITY ? 0.f : g[i] * unit * (x[i] == m ? 1.f : __expf(x[i] - m));
        sub = team_reduce<L>(sub, add);
#pragma unroll
        for (int i = 0; i < NI; i++) p[i] *= inv;
    } else {
        // r = s / sum s from the scores over the largest one's power of e,
        // which no sum of small scores makes 0
        float m = -INFINITY, s[KPL], rest[KPL];
#pragma unroll
        for (int i = 0; i < KPL; i++) m = fmaxf(m, sigmoid ? fminf(x[i], 0.f) : x[i]);
        m = team_reduce<L>(m, most);
        if (sigmoid && !renormalise) m = 0.f;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < KPL; i++) {
            const float e = sigmoid ? __expf(-fabsf(x[i])) : 0.f;  // of the smaller side
            const float over = 1.f / (1.f + e);
            const float low = sigmoid ? fminf(x[i], 0.f) : x[i];
            s[i] = x[i] == -INFINITY ? 0.f : (low == m ? 1.f : __expf(low - m)) * over;
            rest[i] = sigmoid ? (x[i] < 0.f ? 1.f : e) * over : 1.f;
            sum += s[i];
        }
        sum = team_reduce<L>(sum, add);
        const float inv = !renormalise ? 1.f : sum > 0.f ? 1.f / sum : 0.f;
        float mean = 0.f;
#pragma unroll
        for (int i = 0; i < KPL; i++) {
            s[i] *= inv;
            mean += s[i] == 0.f ? 0.f : g[i] * s[i];
        }
        mean = renormalise ? team_reduce<L>(mean, add) : 0.f;
#pragma unroll
        for (int i = 0; i < KPL; i++) g[i] = s[i] == 0.f ? 0.f : scale * s[i] * rest[i] * (g[i] - mean);
    }
    float out[NI];
#pragma unroll
    for (int i = 0; i < NI; i++) out[i] = FULL ? -sub : 0.f;
    for (int j = 0; j < k; j++) {
        int e = -1;
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < KPL; i++) {
            const int ei = __shfl(id[i], j % L, L);
            const float vi = __shfl(g[i], j % L, L);
            if (j / L == i) {
                e = ei;
                v = vi;
            }
        }
#pragma unroll
        for (int i = 0; i < NI; i++) out[i] += l + L * i == e ? v : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NI; i++)
        if (l + L * i < Ne) dlogits[t * Ne + l + L * i] = in[i] + (FULL ? (p[i] == 0.f ? 0.f : p[i] * out[i]) : out[i]);
    }
}

// The bias's step: a workgroup counts its share of the entries in LDS (whole
// numbers, so that their order changes nothing); where there are several they
// leave their counts in the workspace and one adds them.
constexpr int kBiasThreads = 1024, kBiasBlocks = 64, kBiasShare = 8192;  // entries a workgroup
int bias_blocks(size_t entries) {
    return static_cast<int>(std::max<size_t>(1, std::min<size_t>(kBiasBlocks, ceil_div(entries, kBiasShare))));
}

__device__ __forceinline__ void bias_finish(int c, int Ne, const float *bias_in, float rate,
                                            int32_t *counts, float *bias) {
    __shared__ int s_total;
    const int e = threadIdx.x;
    if (e == 0) s_total = 0;
    __syncthreads();
    if (e < Ne) atomicAdd(&s_total, c);
    __syncthreads();
    if (e <= Ne) counts[e] = c;
    if (e < Ne) {
        const int64_t over = static_cast<int64_t>(s_total) - static_cast<int64_t>(Ne) * c;
        bias[e] = bias_in[e] + (over > 0 ? rate : over < 0 ? -rate : 0.f);
    }
}

__global__ __launch_bounds__(kBiasThreads) void k_bias_count(
    const int32_t *__restrict__ ids, const uint8_t *__restrict__ valid, int T, int k, int Ne,
    const float *bias_in, float rate, int32_t *__restrict__ counts, float *bias,
    int32_t *__restrict__ part) {
    __shared__ int s_cnt[kMaxNe + 1];
    for (int e = threadIdx.x; e <= Ne; e += kBiasThreads) s_cnt[e] = 0;
    __syncthreads();
    const size_t step = static_cast<size_t>(gridDim.x) * kBiasThreads;
    const size_t first = static_cast<size_t>(blockIdx.x) * kBiasThreads + threadIdx.x;
    const uint32_t entries = static_cast<uint32_t>(T) * static_cast<uint32_t>(k);
    for (size_t i = first; i < entries; i += step) {
        const uint32_t t = static_cast<uint32_t>(i) / static_cast<uint32_t>(k);
        if (valid && !valid[t]) continue;
        const int e = ids[i];
        if (e >= 0 && e < Ne) atomicAdd(&s_cnt[e], 1);
        if (i == static_cast<size_t>(t) * k) atomicAdd(&s_cnt[Ne], 1);
    }
    __syncthreads();
    const int e = threadIdx.x;
    if (gridDim.x == 1) bias_finish(e <= Ne ? s_cnt[e] : 0, Ne, bias_in, rate, counts, bias);
    else if (e <= Ne) part[static_cast<size_t>(blockIdx.x) * (Ne + 1) + e] = s_cnt[e];
}

// The workgroups' counts: kBiasShares threads an expert, each with all of its
// loads in flight (one thread's 32 loads in turn took 9 us).
constexpr int kBiasShares = 4, kBiasEach = kBiasBlocks / kBiasShares;
__global__ __launch_bounds__(kBiasThreads) void k_bias_step(const int32_t *__restrict__ part, int blocks,
                                                            int Ne, const float *bias_in, float rate,
                                                            int32_t *__restrict__ counts, float *bias) {
    __shared__ int s_cnt[kMaxNe + 1];
    for (int e = threadIdx.x; e <= Ne; e += kBiasThreads) s_cnt[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < kBiasShares * (Ne + 1); i += kBiasThreads) {
        const int e = i % (Ne + 1), b0 = i / (Ne + 1);
        int v[kBiasEach], c = 0;
#pragma unroll
        for (int j = 0; j < kBiasEach; j++)
            v[j] = part[static_cast<size_t>(min(b0 + kBiasShares * j, blocks - 1)) * (Ne + 1) + e];
#pragma unroll
        for (int j = 0; j < kBiasEach; j++) c += b0 + kBiasShares * j < blocks ? v[j] : 0;
        atomicAdd(&s_cnt[e], c);
    }
    __syncthreads();
    const int e = threadIdx.x;
    bias_finish(e <= Ne ? s_cnt[e] : 0, Ne, bias_in, rate, counts, bias);
}

}  // namespace

hipError_t launch_route_scored(const ScoreArgs &a, hipStream_t s) {
    const bool groups = a.top_groups < a.tab.Nd;
    ScoreArgs b = a;
    b.over_n = static_cast<int>(ceil_div(1 << 16, a.tab.n));  // p / n = p over_n >> 16 for p < 256
    b.in_order = 1;
    for (int p = 0; groups && p < a.Ne; p++) b.in_order = b.in_order && a.tab.expert[p] == p;
#define OCC_SCORED(L, NI)                                                              \
    do {                                                                               \
        const unsigned grid = std::min(ceil_div(a.T, kScoreThreads / L), kScoreGrid);   \
        if (groups) k_route_scored<L, NI, true><<<grid, kScoreThreads, 0, s>>>(b);     \
        else k_route_scored<L, NI, false><<<grid, kScoreThreads, 0, s>>>(b);           \
    } while (0)
    if (a.Ne <= 16) OCC_SCORED(16, 1);
    else if (a.Ne <= 32) OCC_SCORED(16, 2);
    else if (a.Ne <= 64) OCC_SCORED(16, 4);
    else if (a.Ne <= 128) OCC_SCORED(64, 2);
    else OCC_SCORED(64, 4);
#undef OCC_SCORED
    return hipGetLastError();
}

hipError_t launch_route_scored_back(const float *logits, const int32_t *ids, const float *dw,
                                    const float *dlogits_in, int T, int Ne, int k, int sigmoid,
                                    int renormalise, float scale, float *dlogits, hipStream_t s) {
    const bool full = !sigmoid && !renormalise;
#define OCC_SCORED(L, NI)                                                                            \
    do {                                                                                             \
        const unsigned grid = std::min(ceil_div(T, kScoreThreads / L), kScoreGrid);                   \
        if (full) k_route_scored_back<L, NI, true><<<grid, kScoreThreads, 0, s>>>(                   \
                logits, ids, dw, dlogits_in, T, Ne, k, sigmoid, renormalise, scale, dlogits);        \
        else k_route_scored_back<L, NI, false><<<grid, kScoreThreads, 0, s>>>(                       \
                logits, ids, dw, dlogits_in, T, Ne, k, sigmoid, renormalise, scale, dlogits);        \
    } while (0)
    if (Ne <= 16) OCC_SCORED(16, 1);
    else if (Ne <= 32) OCC_SCORED(16, 2);
    else if (Ne <= 64) OCC_SCORED(16, 4);
    else if (Ne <= 128) OCC_SCORED(64, 2);
    else OCC_SCORED(64, 4);
#undef OCC_SCORED
    return hipGetLastError();
}

size_t bias_part_bytes(int T, int Ne, int k) {
    const int blocks = bias_blocks(static_cast<size_t>(T) * k);
    return blocks > 1 ? static_cast<size_t>(blocks) * (Ne + 1) * 4 : 0;
}

hipError_t launch_bias_step(const int32_t *ids, const uint8_t *valid, int T, int k, int Ne,
                            const float *bias_in, float rate, int32_t *counts, float *bias,
                            int32_t *part, hipStream_t s) {
    const int blocks = bias_blocks(static_cast<size_t>(T) * k);
    k_bias_count<<<blocks, kBiasThreads, 0, s>>>(ids, valid, T, k, Ne, bias_in, rate, counts, bias, part);
    if (blocks > 1) k_bias_step<<<1, kBiasThreads, 0, s>>>(part, blocks, Ne, bias_in, rate, counts, bias);
    return hipGetLastError();
}

}  // namespace occ
