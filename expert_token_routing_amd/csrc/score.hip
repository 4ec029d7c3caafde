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
// Tokens from which a wave of 64 lanes a token takes four one after another, so
// that their weights in 64 bits fill its lanes once: at 4096 / 8192 / 16384 /
// 65536 tokens of 128 experts (top 8, no bias) 6.8 / 7.5 / 9.7 / 30.7 us
// against 5.2 / 8.4 / 14.7 / 52.6 one at a time, of 256 in groups (top 8, bias)
// 19.5 / 21.7 / 26.1 / 74 against 16.2 / 22.6 / 36.6 / 116; a single token 6.1
// against 3.3.
constexpr int kScoreSerial = 8192;
// Tokens up to which 33 to 64 experts with groups or a bias take a wave a token,
// one expert a lane: its steps are fewer where one token's chain is what a
// launch waits for.  64 experts, top 8, in groups with a bias: 1 / 64 / 512 /
// 2048 tokens 4.5 / 5.0 / 5.1 / 6.8 us against 6.1 / 6.5 / 6.7 / 8.1 with 16
// lanes, 4096 8.0 against 8.2, 8192 13.8 against 11.5.  Without either, or with
// fewer experts, within a tenth on both sides.
constexpr int kScoreWide = 2048;
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

// LDS of a wave in choose64: the choice by place (a group's places together,
// groups n + 1 apart: other banks) and the groups' scores; of a team in
// keep_groups the same in 32 bits, with how far off a score may be.
struct ChoiceLds {
    double choice[kMaxNe + kMaxNd];
    double group[kMaxNd];
};
struct alignas(8) GroupScore {
    float v, err;
};
template <int L, int NI>
struct GroupLds {
    uint32_t key[L * NI + kMaxNd];
    GroupScore group[kMaxNd];
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

// e^x for x <= 0, within 2^-50: x = n ln 2 + r, |r| <= ln 2 / 2, and the series
// of e^r up to r^12 (the rest is below 2^-52); a third of the instructions of a
// general exp.
__device__ __forceinline__ double exp64(double x) {
    x = fmax(x, -800.);  // 0 from -746 on
    const double n = rint(x * 0x1.71547652b82fep+0);
    double r = fma(n, -0x1.62e42fefa3800p-1, x);
    r = fma(n, -0x1.ef35793c76730p-45, r);
    double p = 1. / 479001600.;
    p = fma(p, r, 1. / 39916800.);
    p = fma(p, r, 1. / 3628800.);
    p = fma(p, r, 1. / 362880.);
    p = fma(p, r, 1. / 40320.);
    p = fma(p, r, 1. / 5040.);
    p = fma(p, r, 1. / 720.);
    p = fma(p, r, 1. / 120.);
    p = fma(p, r, 1. / 24.);
    p = fma(p, r, 1. / 6.);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.);
    p = fma(p, r, 1.);
    return ldexp(p, static_cast<int>(n));
}
// 1 / x of a normal number, within 2^-51: the hardware's estimate and two
// steps of Newton's method.
__device__ __forceinline__ double over64(double x) {
    double y = __builtin_amdgcn_rcp(x);
    y = fma(y, fma(-x, y, 1.), y);
    return fma(y, fma(-x, y, 1.), y);
}
// A softmax's terms over the largest logit m; a logit of -inf has none.
__device__ __forceinline__ double exp_over(float v, float m) {
    return v == -INFINITY ? 0. : v == m ? 1. : exp64(static_cast<double>(v) - static_cast<double>(m));
}
__device__ __forceinline__ double sigmoid64(float v) {
    const double e = exp64(-fabs(static_cast<double>(v)));
    return (v < 0.f ? e : 1.) * over64(1. + e);
}

struct Chosen {
    int e;
    uint32_t key;
};

// The `need` best of a wave's experts in order: by key, then by `fine` (of
// experts of one key; the same in all for none), then by the lower index (the
// larger rev = 256 - e).  A key that between `need` and kMoreHeads more lanes'
// largest ones reach, bit by bit by ballots; then every expert that reaches it,
// one a lane through LDS, counts those ahead of it; all experts with a key where
// they lie in fewer lanes than `need`.  False where that is more than a wave of
// experts or fewer than `need`.  `tie` (by key alone): whether the last two have
// one key.
constexpr int kMoreHeads = 3;
struct alignas(8) Candidate {
    uint32_t rev, key;
};
template <int NI, bool FINE>
__device__ __forceinline__ bool few_best(const uint32_t (&key)[NI], const uint32_t (&rev)[NI], const uint64_t *fine,
                                         int need, Candidate *best, uint64_t *best_fine, Chosen *chosen,
                                         bool *tie = nullptr) {
    uint32_t head = key[0];
#pragma unroll
    for (int j = 1; j < NI; j++) head = max(head, key[j]);
    uint32_t reach = 0;
    for (uint32_t bit = 1u << 31; bit; bit >>= 1) {
        const int n = __popcll(__ballot(head >= (reach | bit)));
        if (n >= need) {
            reach |= bit;
            if (n <= need + kMoreHeads) break;
        }
    }
    reach = max(reach, 1u);
    int n = 0;
#pragma unroll
    for (int j = 0; j < NI; j++) {
        const uint64_t in = __ballot(key[j] >= reach);
        const int at = n + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(in >> 32),
                                                     __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(in), 0));
        if (key[j] >= reach && at < kWave) {
            best[at] = Candidate{rev[j], key[j]};
            if constexpr (FINE) best_fine[at] = fine[j];
        }
        n += __popcll(in);
    }
    if (n > kWave || n < need) return false;
    wave_sync();
    const int lane = lane_id();
    Candidate mine = best[lane];
    if (lane >= n) mine = Candidate{0, 0};
    int rank = 0;
    if constexpr (FINE) {
        const uint64_t at = best_fine[lane];
        for (int i = 0; i < n; i++) {
            const uint64_t o = best_fine[i];
            const uint32_t r = best[i].rev;
            rank += o > at || (o == at && r > mine.rev);
        }
    } else {
        // four at once, zeros behind the last (from other lanes' registers instead:
        // 35.7 us against 32.7 for 65536 tokens of 128 experts)
        if (lane >= n) best[lane] = mine;
        wave_sync();
        const auto whole = [](Candidate c) { return static_cast<uint64_t>(c.key) << 32 | c.rev; };
        const uint64_t at = whole(mine);
        for (int i = 0; i < n; i += 4) {
            const Candidate c0 = best[i], c1 = best[i + 1], c2 = best[i + 2], c3 = best[i + 3];
            rank += (whole(c0) > at) + (whole(c1) > at) + (whole(c2) > at) + (whole(c3) > at);
        }
    }
    if (lane < n && rank < need) chosen[rank] = Chosen{256 - static_cast<int>(mine.rev), mine.key};
    if (tie) {
        const auto at = [&](int r) { return __builtin_ctzll(__ballot(lane < n && rank == r)); };
        *tie = need > 1 && __builtin_amdgcn_readlane(static_cast<int>(mine.key), at(need - 1)) ==
                               __builtin_amdgcn_readlane(static_cast<int>(mine.key), at(need - 2));
    }
    return true;
}

// Where the first expert that is not chosen (`last`) is an exact tie of the last
// chosen one, of one logit and bias, that pair is in order but says nothing of
// what stands behind it: whether an expert that is no such tie lies within the
// margin of theirs, so that 64 bits may put it in front.  `key` and `rev` hold
// the experts that are left, or all of them.
template <int L, int NI>
__device__ __forceinline__ bool hidden_behind(const uint32_t (&key)[NI], const uint32_t (&rev)[NI], Chosen last,
                                              const float *row, const float *bias, float margin) {
    const float c = from_key(last.key), off = margin * (1.f + fabsf(c)), v = row[last.e], b = bias[last.e];
    bool any = false;
#pragma unroll
    for (int j = 0; j < NI; j++)
        if (key[j] != 0 && key[j] <= last.key && c - from_key(key[j]) <= off) {
            const int e = 256 - static_cast<int>(rev[j]);
            any = any || row[e] != v || bias[e] != b;
        }
    return team_ballot<L>(any) != 0;
}

// The choice in 64 bits throughout, for the tokens whose choice 32 bits cannot
// tell: the k chosen experts in order, by all lanes of a wave.  A call of its
// own, which loads its row anew.  Few tokens take it, but a launch ends with the
// last of them.
struct Choice {
    const float *row, *bias;
    const uint8_t *place;  // LDS: expert at each place
    int Ne, k, n, Nd, sigmoid, top_groups, group_best;
};
template <int NI, bool GROUPS>
__device__ __attribute__((noinline)) void choose64(Choice a, ChoiceLds *lds, Candidate *best, Chosen *chosen) {
    constexpr int L = kWave;
    const int l = lane_id(), Ne = a.Ne, n = a.n, Nd = a.Nd;
    const float *row = a.row;
    struct {
        int e[NI];
        float v[NI], b[NI];
    } x;
#pragma unroll
    for (int j = 0; j < NI; j++) {
        const int p = min(l + L * j, Ne - 1);
        x.e[j] = GROUPS ? a.place[p] : p;
        x.v[j] = row[x.e[j]];
        x.b[j] = a.bias ? a.bias[x.e[j]] : 0.f;
        if (!(l + L * j < Ne) || x.v[j] != x.v[j]) x.v[j] = -INFINITY;
    }
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
        for (int j = 0; j < NI; j++) c[j] = sum > 0. ? c[j] * over64(sum) : 0.;
    }
#pragma unroll
    for (int j = 0; j < NI; j++) {
        c[j] += x.b[j];
        if (x.v[j] == -INFINITY || c[j] != c[j]) c[j] = -INFINITY;
    }
    uint64_t allowed = ~0ull;
    if constexpr (GROUPS) {
#pragma unroll
        for (int j = 0; j < NI; j++) {
            const int p = l + L * j;
            if (p < Ne) lds->choice[p + p / n] = c[j];
        }
        wave_sync();
        group_scores<L>(lds->choice, Nd, n, a.group_best, [&](int g, double v) {
            if (g < Nd) lds->group[g] = v;
        });
        wave_sync();
        allowed = 0;
        for (int g = l; g < Nd; g += L) {
            const double v = lds->group[g];
            int ahead = 0;
            for (int o = 0; o < Nd; o++) {
                const double y = lds->group[o];
                ahead += y > v || (y == v && o < g);
            }
            if (ahead < a.top_groups) allowed |= 1ull << g;
        }
        allowed = team_reduce<L>(allowed, [](uint64_t p, uint64_t q) { return p | q; });
    }
    uint64_t fine[NI];
    uint32_t key[NI], rev[NI];
#pragma unroll
    for (int j = 0; j < NI; j++) {
        const int p = l + L * j;
        bool ok = p < Ne;
        if constexpr (GROUPS) ok = ok && allowed >> (p / n) & 1;
        const double o = a.bias ? c[j] : static_cast<double>(x.v[j]);
        fine[j] = ok ? order_key(o) : 0;
        key[j] = ok ? order_key(static_cast<float>(o)) : 0;  // (rounding keeps the order but for ties)
        rev[j] = ok ? 256u - x.e[j] : 0;
    }
    if (few_best<NI, true>(key, rev, fine, a.k, best, reinterpret_cast<uint64_t *>(lds->choice), chosen)) {
        wave_sync();
        return;
    }
    for (int i = 0; i < a.k; i++) {  // one after another
        uint64_t most = 0;
        uint32_t low = 0;
#pragma unroll
        for (int j = 0; j < NI; j++)
            if (fine[j] > most || (fine[j] == most && rev[j] > low)) {
                most = fine[j];
                low = rev[j];
            }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            const uint64_t om = __shfl_xor(most, o);
            const uint32_t ow = __shfl_xor(low, o);
            if (om > most || (om == most && ow > low)) {
                most = om;
                low = ow;
            }
        }
#pragma unroll
        for (int j = 0; j < NI; j++)
            if (fine[j] && rev[j] == low) {
                fine[j] = 0;
                chosen[i] = Chosen{256 - static_cast<int>(low), 0};
            }
    }
    wave_sync();
}

// The groups' scores from the order keys of c in LDS (as group_scores), and of
// the kept groups: bit g << shift of the result; `sure` is whether the scores
// at the border lie further apart than both may be off.  A sum's error goes by
// its terms, which may cancel: margin / 2 (1 + |c|) of each, 2^-24 of the sum
// besides, below margin (1 + |c1| + |c2|) together.  A group without an expert
// is -inf exactly.
template <int L>
__device__ __forceinline__ uint64_t keep_groups(const uint32_t *key, GroupScore *s_group, const ScoreArgs &a,
                                                float margin, int &shift, bool &sure) {
    const GroupWalk<L> walk(a.tab.Nd);
    const int l = threadIdx.x % L, Nd = a.tab.Nd, n = a.tab.n, GL = 1 << walk.shift;
    const int i = l & (GL - 1);
    const auto score = [&](int g) -> GroupScore {
        uint32_t top = 0, next = 0;
        const uint32_t *at = key + min(g, Nd - 1) * (n + 1);
        for (int j0 = 0; j0 < n; j0 += 4 * GL) {
            uint32_t k[4];
#pragma unroll
            for (int j = 0; j < 4; j++) k[j] = at[min(j0 + GL * j + i, n - 1)];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t one = g < Nd && j0 + GL * j + i < n ? k[j] : 0;
                next = max(next, min(top, one));
                top = max(top, one);
            }
        }
        const auto join = [&](uint32_t ot, uint32_t on) {
            next = max(max(next, on), min(top, ot));
            top = max(top, ot);
        };
        if (GL >= 2) join(dpp_partner<kDppXor1>(top), dpp_partner<kDppXor1>(next));
        if (GL >= 4) join(dpp_partner<kDppXor2>(top), dpp_partner<kDppXor2>(next));
        if (GL >= 8) join(dpp_partner<kDppHalfMirror>(top), dpp_partner<kDppHalfMirror>(next));
        if (GL >= 16) join(dpp_partner<kDppMirror>(top), dpp_partner<kDppMirror>(next));
        if (GL >= 32) join(__shfl_xor(top, 16), __shfl_xor(next, 16));
        if (GL >= 64) join(__shfl_xor(top, 32), __shfl_xor(next, 32));
        // none left: -inf; one: no second
        const float ft = top ? from_key(top) : -INFINITY, fn = next ? from_key(next) : -INFINITY;
        const bool both = a.group_best > 1 && fn > -INFINITY;
        const float size = fabsf(ft) + (both ? fabsf(fn) : 0.f);
        return GroupScore{both ? ft + fn : ft, ft > -INFINITY ? margin * (1.f + size) : 0.f};
    };
    uint64_t kept = 0;
    shift = 0;
    if (GL >= Nd) {  // (all groups at once) a group's lane i compares it with group i
        const int g = l >> walk.shift;
        const GroupScore own = score(g);
        const float v = own.v, y = __shfl(v, i << walk.shift, L);
        const float off = own.err + __shfl(own.err, i << walk.shift, L);
        const bool other = i < Nd && g < Nd && i != g;
        const uint64_t fields = GL >= 64 ? ~0ull : (1ull << GL) - 1;
        const int ahead = __popcll(team_ballot<L>(other && y - v > off) >> (g << walk.shift) & fields);
        const int near = __popcll(team_ballot<L>(other && !(v - y > off)) >> (g << walk.shift) & fields);
        const bool in = near < a.top_groups, out = ahead >= a.top_groups;
        sure = team_ballot<L>(g < Nd && !in && !out) == 0;
        kept = team_ballot<L>(g < Nd && in && i == 0);
        shift = walk.shift;
        return kept;
    }
    for (int g0 = 0; g0 < Nd; g0 += walk.per) {
        const int g = g0 + (l >> walk.shift);
        const GroupScore own = score(g);
        if (g < Nd && i == 0) s_group[g] = own;
    }
    wave_sync();
    for (int g0 = 0; g0 < Nd; g0 += L) {
        const int g = g0 + l;
        const GroupScore own = s_group[min(g, Nd - 1)];
        int ahead = 0, near = 0;
        for (int o = 0; o < Nd; o++) {
            const GroupScore y = s_group[o];
            const float off = own.err + y.err;
            ahead += y.v - own.v > off;
            near += !(own.v - y.v > off) && o != g;
        }
        const bool in = near < a.top_groups, out = ahead >= a.top_groups;
        sure = sure && team_ballot<L>(g < Nd && !in && !out) == 0;
        kept |= team_ballot<L>(g < Nd && in) << g0;
    }
    return kept;
}

// A team of L lanes a token, NI experts a lane.  A choice is a border, and near
// ties would fall differently in 32 bits than in 64 for a token in some
// thousands.  Scores in 32 bits are off by less than half of a margin, so a
// choice whose neighbours (the chosen, the first not chosen, the groups at
// their border) lie further apart is the one that 64 bits make; logits alone
// order without an error, and experts of equal logit and bias tie in both; where
// they tie across the border of the chosen, the experts behind them count (by
// hidden_behind).  The tokens that are left take choose64.
//
// Bound by instructions, but for few tokens, where the launch and its chain of
// dependent steps count.  With 16 lanes a token a lane sorts its experts once,
// and a round is the team's largest head and the winner's next one; all lanes
// of a wave take few_best.  A wave makes the choice of four tokens (16 lanes
// each, or all lanes one token after another) and then forms their weights in
// 64 bits, 16 lanes a token.  Up to 64 experts 16 lanes a token (but see
// kScoreWide): at 512 / 8192 / 65536 tokens of 60 experts, top 4, 3.6 / 3.9 /
// 11.0 us against 3.7 / 7.0 / 29.5 with 64, 65536 of 64 in groups with a bias,
// top 8, 33 against 78.  The 65536 tokens of 60 experts read and write 18 MB (1.7
// TB/s) in 93 vector and 38 scalar instructions a token, of 64 in groups with a
// bias 21 MB (0.6 TB/s) in 246 and 86, 32768 of 256 in groups 36 MB in 43 us (0.8
// TB/s) in 433 and 308.  choose64 is what they are far from: 65536 tokens of 64
// experts in groups take 111 us where most of them need it (sigmoids of logits of
// a deviation of 8, rounded to bf16, a bias of zeros).
template <int L, int NI, bool GROUPS, bool BIASED>
__global__ __launch_bounds__(kScoreThreads, 4) void k_route_scored(ScoreArgs a) {
    constexpr int TEAMS = kWave / L, WAVES = kScoreThreads / kWave, TOK = 4, W = 16, KPL = kMaxK / W;
    constexpr bool DOUBT = GROUPS || BIASED || L == 64;  // (logits alone order for sure)
    __shared__ Candidate s_best[DOUBT ? WAVES : 1][kWave];
    __shared__ union {
        GroupLds<L, NI> team[GROUPS ? TEAMS : 1];
        ChoiceLds all;
    } s_lds[DOUBT ? WAVES : 1];
    __shared__ Chosen s_chosen[WAVES][TOK][kMaxK + 1];
    __shared__ double s_sum[WAVES][TOK];
    __shared__ float s_top[WAVES][TOK], s_margin[WAVES][TOK];  // INFINITY: not sure already
    __shared__ uint8_t s_place[GROUPS ? kMaxNe : 1];
    if constexpr (GROUPS) {
        for (int p = threadIdx.x; p < a.Ne; p += kScoreThreads) s_place[p] = a.in_order ? p : a.tab.expert[p];
        __syncthreads();
    }
    const int lane = lane_id(), wv = threadIdx.x / kWave, l = lane % L, team = lane / L;
    const int Ne = a.Ne, k = a.k;
    const bool full = !a.sigmoid && !a.renormalise;
    int e_of[NI], g_of[NI];  // the lane's experts: at places l + L j of the placement where groups
    float bias[NI];          // matter (which puts a group's together), of 0..Ne-1 otherwise
#pragma unroll
    for (int j = 0; j < NI; j++) {
        const int p = min(l + L * j, Ne - 1);
        e_of[j] = GROUPS ? s_place[p] : p;
        bias[j] = BIASED ? a.bias[e_of[j]] : 0.f;
        g_of[j] = GROUPS ? p * a.over_n >> 16 : 0;
    }
    const size_t T = a.T, step = static_cast<size_t>(gridDim.x) * WAVES * a.per_wave;
    for (size_t t0 = (static_cast<size_t>(blockIdx.x) * WAVES + wv) * a.per_wave; t0 < T; t0 += step) {
        float ahead[NI];  // the token's row; where a wave takes several, loaded while the
                          // one before is in work (4 to 6% from 32768 tokens on)
        const auto load = [&](int q) {
            const float *row = a.logits + min(t0 + q, T - 1) * Ne;  // (behind the last one: again, and not written)
#pragma unroll
            for (int j = 0; j < NI; j++) ahead[j] = row[e_of[j]];
        };
        if constexpr (L == kWave) load(0);
        for (int it = 0; it < a.per_wave; it += TEAMS) {
            const int q = it + team;
            if constexpr (L < kWave) load(q);
            Chosen *chosen = s_chosen[wv][q];
            float v[NI];
#pragma unroll
            for (int j = 0; j < NI; j++) v[j] = ahead[j];
            if (L == kWave && it + 1 < a.per_wave) load(it + 1);
#pragma unroll
            for (int j = 0; j < NI; j++)
                if (!(l + L * j < Ne) || v[j] != v[j]) v[j] = -INFINITY;
            float top = 0.f;  // the largest logit, for a softmax
            if (!a.sigmoid && (GROUPS || BIASED || full)) {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < NI; j++) m = max(m, order_key(v[j]));
                top = from_key(team_max<L>(m));
            }
            // How far apart two choices in 32 bits must be, over 1 + |c|, to be
            // sure: twice the error of one.  A sigmoid's is below 2^-22 (2^-23
            // for the reciprocal, 2^-24 for the sum in it, 0.42 2^-23 for the
            // exponential, whose own is 2^-23 + 1.5 |v| 2^-24) and 2^-24 |c| for
            // the bias; a softmax's below 2^-19 of the largest p (the terms'
            // exponentials, their sum and its reciprocal) besides.
            float margin = 0x1p-21f;
            float c[NI];
            bool sure = true;
            if constexpr (GROUPS || BIASED) {
                if (a.sigmoid) {
#pragma unroll
                    for (int j = 0; j < NI; j++) {
                        c[j] = __builtin_amdgcn_rcpf(1.f + __expf(-v[j]));
                    }
                } else {
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < NI; j++) {
                        c[j] = v[j] == -INFINITY ? 0.f : v[j] == top ? 1.f : __expf(v[j] - top);
                        sum += c[j];
                    }
                    sum = team_sum<L>(sum);
                    const float inv = sum > 0.f ? __builtin_amdgcn_rcpf(sum) : 0.f;
#pragma unroll
                    for (int j = 0; j < NI; j++) c[j] *= inv;
                    margin += 0x1p-18f * inv;
                }
#pragma unroll
                for (int j = 0; j < NI; j++) c[j] = v[j] == -INFINITY ? -INFINITY : c[j] + bias[j];
            }
            uint32_t key[NI], rev[NI];  // rev: 256 - e, larger for the lower index
#pragma unroll
            for (int j = 0; j < NI; j++) {
                const bool in = l + L * j < Ne;
                key[j] = in ? order_key(BIASED ? c[j] : v[j]) : 0u;
                rev[j] = in ? 256u - e_of[j] : 0u;
            }
            if constexpr (GROUPS) {
                GroupLds<L, NI> &lds = s_lds[wv].team[team];
#pragma unroll
                for (int j = 0; j < NI; j++) {
                    const int p = l + L * j;
                    if (p < Ne) lds.key[p + g_of[j]] = BIASED ? key[j] : order_key(c[j]);
                }
                wave_sync();
                int shift;
                const uint64_t kept = keep_groups<L>(lds.key, lds.group, a, margin, shift, sure);
#pragma unroll
                for (int j = 0; j < NI; j++)
                    if (!(kept >> (g_of[j] << shift) & 1)) key[j] = 0;
            }
            const bool border = BIASED && a.rounds > k;
            const auto hidden = [&] {
                return hidden_behind<L, NI>(key, rev, chosen[k], a.logits + min(t0 + q, T - 1) * Ne, a.bias, margin);
            };
            if constexpr (L == 64) {
                bool tie = false;
                sure = few_best<NI, false>(key, rev, nullptr, a.rounds, s_best[wv], nullptr, chosen, BIASED ? &tie : nullptr) && sure;
                if (border && tie) {
                    wave_sync();
                    sure = !hidden() && sure;
                }
            } else {
                // the lane's experts, the best first
                const auto order = [&](int i, int j) {
                    const bool swap = key[j] > key[i] || (key[j] == key[i] && rev[j] > rev[i]);
                    const uint32_t k0 = key[i], r0 = rev[i];
                    key[i] = swap ? key[j] : k0;
                    rev[i] = swap ? rev[j] : r0;
                    key[j] = swap ? k0 : key[j];
                    rev[j] = swap ? r0 : rev[j];
                };
                if constexpr (NI == 2) order(0, 1);
                if constexpr (NI == 4) {
                    order(0, 1);
                    order(2, 3);
                    order(0, 2);
                    order(1, 3);
                    order(1, 2);
                }
                for (int i = 0; i < a.rounds; i++) {
                    const uint32_t best = team_max<L>(key[0]);
                    bool has = key[0] == best;
                    const uint64_t with = team_ballot<L>(has);
                    if (__ballot((with & (with - 1)) != 0)) {  // ties, in any team of the wave
                        const uint32_t low = team_max<L>(has ? rev[0] : 0u);
                        has = has && rev[0] == low;
                    }
                    if (has) chosen[i] = Chosen{256 - static_cast<int>(rev[0]), best};
#pragma unroll
                    for (int j = 0; j + 1 < NI; j++) {
                        key[j] = has ? key[j + 1] : key[j];
                        rev[j] = has ? rev[j + 1] : rev[j];
                    }
                    key[NI - 1] = has ? 0u : key[NI - 1];
                }
                if (border) {
                    wave_sync();
                    const bool tie = chosen[k].key == chosen[k - 1].key && chosen[k].key != 0;
                    if (__ballot(tie)) {
                        const bool h = hidden();
                        sure = sure && !(tie && h);
                    }
                }
            }
            if (DOUBT && l == 0) s_margin[wv][q] = sure ? margin : INFINITY;
            if (full) {
                double sum = 0.;
#pragma unroll
                for (int j = 0; j < NI; j++) sum += exp_over(v[j], top);
                sum = team_reduce<L>(sum, [](double y, double z) { return y + z; });
                if (l == 0) {
                    s_sum[wv][q] = sum;
                    s_top[wv][q] = top;
                }
            }
        }
        wave_sync();
        const int r = lane % W, q = lane / W;
        const size_t t = t0 + q;
        const bool live = q < a.per_wave && t < T;
        // The choices that are not sure, found 16 lanes a token.
        if constexpr (DOUBT) {
            const float margin = live ? s_margin[wv][q] : 0.f;
            bool sure = margin < INFINITY;
            if (BIASED && sure && live) {
#pragma unroll
                for (int i = 0; i < KPL; i++) {
                    const int o = r + W * i + 1;  // against the one in front
                    if (o < a.rounds) {
                        const Chosen y = s_chosen[wv][q][o - 1], z = s_chosen[wv][q][o];
                        const float cy = from_key(y.key), cz = from_key(z.key);
                        if (cy - cz <= margin * (1.f + fabsf(cy)))
                            sure = sure && a.logits[t * Ne + y.e] == a.logits[t * Ne + z.e] && a.bias[y.e] == a.bias[z.e];
                    }
                }
            }
            if (const uint64_t unsure = __ballot(!sure)) {
                wave_sync();
                for (int i = 0; i < a.per_wave; i++)
                    if (unsure >> (W * i) & 0xffff)
                        choose64<(L * NI + kWave - 1) / kWave, GROUPS>(
                            Choice{a.logits + (t0 + i) * Ne, a.bias, s_place, Ne, k, a.tab.n, a.tab.Nd, a.sigmoid, a.top_groups,
                                   a.group_best},
                            &s_lds[wv].all, s_best[wv], s_chosen[wv][i]);
            }
        }
        // The weights.  Renormalised, scores are taken over the largest that
        // was chosen, so that none of them vanishes in the sum: softmax terms
        // over its logit; sigmoids as they are but where all of them are below
        // e^-600.
        float v[KPL], m = -INFINITY;
        int e[KPL];
#pragma unroll
        for (int i = 0; i < KPL; i++) {
            const int j = r + W * i;
            e[i] = live && j < k ? s_chosen[wv][q][j].e : 0;
            v[i] = live && j < k ? a.logits[t * Ne + e[i]] : -INFINITY;
            if (v[i] != v[i]) v[i] = -INFINITY;
        }
        if (a.renormalise) {
#pragma unroll
            for (int i = 0; i < KPL; i++) m = fmaxf(m, v[i]);
            m = group_max<W>(m);
        } else if (full && live) {
            m = s_top[wv][q];
        }
        const bool deep = a.sigmoid && a.renormalise && m < -600.f;
        double s[KPL], sum = 0.;
#pragma unroll
        for (int i = 0; i < KPL; i++) {
            s[i] = 0.;
            if (i * W < k) {  // (wave-uniform)
                s[i] = a.sigmoid && !deep ? sigmoid64(v[i]) : exp_over(v[i], m);
                sum += s[i];
            }
        }
        if (a.renormalise) sum = team_reduce<W>(sum, [](double y, double z) { return y + z; });
        else sum = full && live ? s_sum[wv][q] : 1.;
        const double over = sum > 0. ? a.scale * over64(sum) : 0.;
#pragma unroll
        for (int i = 0; i < KPL; i++)
            if (live && r + W * i < k) {
                a.ids[t * k + r + W * i] = e[i];
                a.w[t * k + r + W * i] = static_cast<float>(over * s[i]);
            }
        wave_sync();
    }
}

// The gradient: a team of L lanes a token, lane j < k (and j + L) with the
// token's j-th expert, then lane l with experts l + L i of the row.  In fp32: it
// has no border, and an error stays a rounding.  Bound by memory where tokens
// are many, since every row is written, zeros too: 65536 tokens of 60 experts,
// softmax, added to an earlier gradient, 11.9 us (49 MB, 4.1 TB/s).  Up to 64
// experts 16 lanes a token: renormalised, 3.4 / 3.8 / 10.5 us at 512 / 8192 /
// 65536 tokens against 3.1 / 4.8 / 23.2 with 64.
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
// leave their counts in the workspace and one adds them.  Bound by latency: 512
// tokens of top 8 4.9 us in one launch, 65536 of top 4 (1 MB) 5.4 + 3.6 in two.
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
    const int kept = groups ? a.top_groups * a.tab.n : a.Ne;
    ScoreArgs b = a;
    // one more than k where the choice has a border and that has to be looked at
    b.rounds = a.bias ? std::min(a.k + 1, kept) : a.k;
    b.over_n = static_cast<int>(ceil_div(1 << 16, a.tab.n));  // p / n = p over_n >> 16 for p < 256
    b.in_order = 1;
    for (int p = 0; groups && p < a.Ne; p++) b.in_order = b.in_order && a.tab.expert[p] == p;
#define OCC_SCORED(L, NI)                                                              \
    do {                                                                               \
        b.per_wave = L == 16 || a.T >= kScoreSerial ? 4 : 1;                            \
        const unsigned grid = std::min(ceil_div(a.T, kScoreThreads / kWave * b.per_wave), kScoreGrid); \
        if (groups && a.bias) k_route_scored<L, NI, true, true><<<grid, kScoreThreads, 0, s>>>(b);  \
        else if (groups) k_route_scored<L, NI, true, false><<<grid, kScoreThreads, 0, s>>>(b);      \
        else if (a.bias) k_route_scored<L, NI, false, true><<<grid, kScoreThreads, 0, s>>>(b);      \
        else k_route_scored<L, NI, false, false><<<grid, kScoreThreads, 0, s>>>(b);                 \
    } while (0)
    if (a.Ne <= 16) OCC_SCORED(16, 1);
    else if (a.Ne <= 32) OCC_SCORED(16, 2);
    else if (a.Ne <= 64 && a.T <= kScoreWide && (groups || a.bias)) {
        b.per_wave = 1;
        const unsigned grid = std::min(ceil_div(a.T, kScoreThreads / kWave), kScoreGrid);
        if (groups && a.bias) k_route_scored<64, 1, true, true><<<grid, kScoreThreads, 0, s>>>(b);
        else if (groups) k_route_scored<64, 1, true, false><<<grid, kScoreThreads, 0, s>>>(b);
        else k_route_scored<64, 1, false, true><<<grid, kScoreThreads, 0, s>>>(b);
    } else if (a.Ne <= 64) OCC_SCORED(16, 4);
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
