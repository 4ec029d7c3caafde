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

// A team of L lanes a token; lane l has the experts at places l + L j (of the
// placement where groups matter, which puts a group's experts together).
// Scores are made and compared in 64 bits: a choice is a border, and near ties
// would fall differently in 32 bits for a token in some thousands.
template <int L, int NI, bool GROUPS>
__global__ __launch_bounds__(kScoreThreads) void k_route_scored(ScoreArgs a) {
    constexpr int TOK = kScoreThreads / L;
    __shared__ double s_choice[TOK][GROUPS ? L * NI + kMaxNd : 1];
    __shared__ double s_group[TOK][GROUPS ? kMaxNd : 1];
    __shared__ double s_chosen[TOK][kMaxK];
    __shared__ int s_ids[TOK][kMaxK];
    const int l = threadIdx.x % L, q = threadIdx.x / L;
    const int Ne = a.Ne, k = a.k, n = a.tab.n, Nd = a.tab.Nd;
    for (size_t t0 = static_cast<size_t>(blockIdx.x) * TOK; t0 < static_cast<size_t>(a.T);
         t0 += static_cast<size_t>(gridDim.x) * TOK) {
    const size_t t = t0 + q;
    const bool live = t < static_cast<size_t>(a.T);

    double s[NI], c[NI];
    int e[NI];
    float v[NI], b[NI];
#pragma unroll
    for (int j = 0; j < NI; j++) {
        const int p = min(l + L * j, Ne - 1);
        e[j] = GROUPS ? a.tab.expert[p] : p;
        v[j] = a.logits[(live ? t : a.T - 1) * Ne + e[j]];
        b[j] = a.bias ? a.bias[e[j]] : 0.f;
        if (!(l + L * j < Ne) || v[j] != v[j]) v[j] = -INFINITY;
    }
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < NI; j++) {
            const double e = exp(-fabs(static_cast<double>(v[j])));
            s[j] = (v[j] < 0.f ? e : 1.) / (1. + e);
        }
    } else {
        float m = v[0];
#pragma unroll
        for (int j = 1; j < NI; j++) m = fmaxf(m, v[j]);
        m = group_max<L>(m);
        double sum = 0.;
#pragma unroll
        for (int j = 0; j < NI; j++) {
            s[j] = v[j] == -INFINITY ? 0. : v[j] == m ? 1. : exp(static_cast<double>(v[j]) - m);
            sum += s[j];
        }
        sum = team_reduce<L>(sum, [](double x, double y) { return x + y; });
#pragma unroll
        for (int j = 0; j < NI; j++) s[j] = sum > 0. ? s[j] / sum : 0.;
    }
#pragma unroll
    for (int j = 0; j < NI; j++) c[j] = v[j] == -INFINITY ? -INFINITY : s[j] + b[j];

    uint64_t allowed = ~0ull;
    if constexpr (GROUPS) {
        // the groups' scores: a lane a group, its experts one after another
#pragma unroll
        for (int j = 0; j < NI; j++) {
            const int p = l + L * j;
            if (p < Ne) s_choice[q][p + p / n] = c[j];  // groups n + 1 apart: other banks
        }
        __syncthreads();
        for (int g = l; g < Nd; g += L) {
            double top = -INFINITY, next = -INFINITY;
            for (int i = 0; i < n; i++) {
                const double x = s_choice[q][g * (n + 1) + i];
                if (x > top) {
                    next = top;
                    top = x;
                } else if (x > next) {
                    next = x;
                }
            }
            s_group[q][g] = a.group_best > 1 && next > -INFINITY ? top + next : top;
        }
        __syncthreads();
        allowed = 0;
        for (int g = l; g < Nd; g += L) {
            const double x = s_group[q][g];
            int ahead = 0;
            for (int o = 0; o < Nd; o++) {
                const double y = s_group[q][o];
                ahead += y > x || (y == x && o < g);
            }
            if (ahead < a.top_groups) allowed |= 1ull << g;
        }
        allowed = team_reduce<L>(allowed, [](uint64_t x, uint64_t y) { return x | y; });
    }

    uint64_t key[NI];
#pragma unroll
    for (int j = 0; j < NI; j++) {
        const int p = l + L * j;
        bool ok = p < Ne;
        if constexpr (GROUPS) ok = ok && allowed >> (p / n) & 1;
        key[j] = ok ? order_key(a.bias ? c[j] : static_cast<double>(v[j])) : 0;
    }
    for (int i = 0; i < k; i++) {
        uint64_t best = 0;
        int who = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < NI; j++)
            if (key[j] > best || (key[j] == best && e[j] < who)) {
                best = key[j];
                who = e[j];
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
            if (key[j] && e[j] == who) {
                key[j] = 0;
                s_ids[q][i] = who;
                s_chosen[q][i] = s[j];
            }
    }
    __syncthreads();
    double sum = 0.;
    for (int i = 0; i < k; i++) sum += s_chosen[q][i];
    const double over = !a.renormalise ? 1. : sum > 0. ? sum : INFINITY;
    for (int i = l; live && i < k; i += L) {
        a.ids[t * k + i] = s_ids[q][i];
        a.w[t * k + i] = static_cast<float>(a.scale * (s_chosen[q][i] / over));
    }
    __syncthreads();
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
        const bool none = sigmoid && m < -745.f;  // as in the forward, where no score is left in 64 bits
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
        const float inv = !renormalise ? 1.f : sum > 0.f && !none ? 1.f / sum : 0.f;
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

__global__ __launch_bounds__(kBiasThreads) void k_bias_step(const int32_t *__restrict__ part, int blocks,
                                                            int Ne, const float *bias_in, float rate,
                                                            int32_t *__restrict__ counts, float *bias) {
    int c = 0;
    if (static_cast<int>(threadIdx.x) <= Ne)
        for (int b = 0; b < blocks; b++) c += part[static_cast<size_t>(b) * (Ne + 1) + threadIdx.x];
    bias_finish(c, Ne, bias_in, rate, counts, bias);
}

}  // namespace

hipError_t launch_route_scored(const ScoreArgs &a, hipStream_t s) {
    const bool groups = a.top_groups < a.tab.Nd;
#define OCC_SCORED(L, NI)                                                              \
    do {                                                                               \
        const unsigned grid = std::min(ceil_div(a.T, kScoreThreads / L), kScoreGrid);   \
        if (groups) k_route_scored<L, NI, true><<<grid, kScoreThreads, 0, s>>>(a);     \
        else k_route_scored<L, NI, false><<<grid, kScoreThreads, 0, s>>>(a);           \
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
