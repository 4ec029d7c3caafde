// The router's losses (load balance over experts and over expert groups, and
// the z-loss), the per-expert counts, and their gradient in the logits.
//
// Mathematics, over the n valid tokens with p = softmax of a token's logits:
//   f_e = Ne counts[e] / (k n), P_e = mean p_e, F_g = mean of f over group g,
//   loss = cb sum f P + cg sum_g F_g P(g) + cz mean lse^2
//   dlogits = dlogits_in + u / n * p (c - <c, p> + 2 cz lse),
//   c_e = cb (f_e - 1) + cg (F_g(e) - 1).
// Since p sums to 1, c may be shifted by a constant: taken from 1, the value
// of f and F at an even load, p (c - <c, p>) does not cancel.
//
// Bound by latency at a training step's smaller batches and by reading the
// logits (4 T Ne bytes each way) at the largest.  A token's softmax takes a
// team of 16, 32 or 64 lanes, the fewest that hold its logits as at most four
// per lane (consecutive ones, one vector, or expert l + L i with lane l), so
// that a wave works on up to four tokens and reduces over a team in 4 to 6 lane exchanges.  The forward adds
// p in registers over a workgroup's tokens and counts in LDS with integer
// atomics (whose order changes nothing); each workgroup leaves its sums in
// the workspace and one workgroup adds them, in a fixed order and in fp64.
// Logits are loaded before the work that does not need them (the counts, the
// backward's coefficients) and a step ahead of their softmax.  exp and log are
// the hardware's base-2 ones behind a product with log2 e or ln 2: an error
// of u |l - max| in p beside expf's, the size that the rounding of l - max has.
// Measured at T = 65536, Ne = 60 (mask, k = 4): 6.4 + 5.8 us forward, 10.1 us
// backward for 48 MB (10.8 with a load for each logit); at T = 512, Ne = 64:
// 7.8 and 4.0 us.
#include <algorithm>

#include "launch.h"

namespace occ {
namespace {

constexpr int kBalThreads = 1024;
constexpr int kBalWaves = kBalThreads / kWave;
constexpr int kBackThreads = 512;

// Loads come a step ahead of their use and are unconditional, so that none
// waits for another: what lies behind the last expert or token is the last
// one's again, and left out when it is used.  A wave's tokens share a scalar
// base; `row` is the token's distance from it.
template <int L, int NI, bool VEC>
__device__ __forceinline__ int expert(int l, int i) {
    return VEC ? NI * l + i : l + L * i;
}
template <int L, int NI, bool VEC>
__device__ __forceinline__ void team_load(const float *base, unsigned row, int l, int Ne,
                                          float (&x)[NI]) {
    const char *at = reinterpret_cast<const char *>(base);
    if constexpr (VEC) {
        const f32x4 v = *reinterpret_cast<const f32x4 *>(at + 4 * (row * Ne + min(4 * l, Ne - 4)));
#pragma unroll
        for (int i = 0; i < 4; i++) x[i] = v[i];
    } else {
#pragma unroll
        for (int i = 0; i < NI; i++)
            x[i] = *reinterpret_cast<const float *>(at + 4 * (row * Ne + min(l + L * i, Ne - 1)));
    }
}

// A token's logits: -inf behind Ne, and everywhere when the token does not
// count.
template <int L, int NI, bool VEC>
__device__ __forceinline__ void team_mask(bool in, int l, int Ne, float (&x)[NI]) {
#pragma unroll
    for (int i = 0; i < NI; i++) x[i] = in && expert<L, NI, VEC>(l, i) < Ne ? x[i] : -INFINITY;
}

// Their softmax in place (0 behind Ne); returns their log-sum-exp.  A row of
// -inf alone has p = 0 and a log-sum-exp of 0; NaN and +inf give NaN.
template <int L, int NI>
__device__ __forceinline__ float team_softmax(float (&p)[NI]) {
    float m = p[0];
#pragma unroll
    for (int i = 1; i < NI; i++) m = fmaxf(m, p[i]);
    m = group_max<L>(m);
    const float shift = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        p[i] = __expf(p[i] - shift);
        s += p[i];
    }
    s = group_sum<L>(s);
    // s is 0 or in [1, 256]: the hardware's reciprocal and logarithm (2^-23
    // relative each) need no care for subnormal values
    const bool none = s == 0.f;
    const float inv = none ? 0.f : __builtin_amdgcn_rcpf(s);
#pragma unroll
    for (int i = 0; i < NI; i++) p[i] *= inv;
    return none ? 0.f : fmaf(__builtin_amdgcn_logf(s), 0x1.62e43p-1f, shift);
}

// One workgroup's part: prob sums (Ne floats), z sum, then counts (Ne) and
// valid tokens as int32.
__host__ __device__ inline int part_words(int Ne) { return 2 * Ne + 2; }

struct BalanceOut {
    float cb, cg, cz;
    int32_t *counts;
    float *probs, *loss;
};

// Thread (e, share) = (x mod (Ne + 1), x / (Ne + 1)) brings a share of column
// e's sums: of p over the tokens and of the counts for an expert, of the
// squared log-sum-exps and of the valid tokens in column Ne.  The workgroup
// adds the shares in order and makes the outputs.
__device__ __forceinline__ void finish(double p, int c, int shares, int Ne, int k,
                                       const PlaceTab &tab, const BalanceOut &o) {
    __shared__ double s_sum[kBalThreads];
    __shared__ int s_cnt[kBalThreads];
    __shared__ float s_f[kMaxNe];
    __shared__ double s_p[kMaxNe + 1];
    const int cols = Ne + 1, e = threadIdx.x;
    s_sum[e] = p;
    s_cnt[e] = c;
    __syncthreads();
    if (e < cols) {
        for (int q = 1; q < shares; q++) {
            p += s_sum[q * cols + e];
            c += s_cnt[q * cols + e];
        }
        s_cnt[e] = c;
        o.counts[e] = c;
    }
    __syncthreads();
    const int n = s_cnt[Ne];
    if (e < cols) {
        s_p[e] = n ? p / n : 0.;
        if (e < Ne) {
            o.probs[e] = static_cast<float>(s_p[e]);
            s_f[e] = n ? static_cast<float>(c) * Ne / (static_cast<float>(k) * n) : 0.f;
        }
    }
    __syncthreads();
    if (e >= kWave) return;
    double lb = 0., lg = 0.;  // lane l: experts l + 64 j, group l
    for (int i = e; i < Ne; i += kWave) lb += s_f[i] * s_p[i];
    if (o.cg != 0.f && e < tab.Nd) {
        double f = 0., q = 0.;
        for (int j = 0; j < tab.n; j++) {
            const int i = tab.expert[e * tab.n + j];
            f += s_f[i];
            q += s_p[i];
        }
        lg = f / tab.n * q;
    }
    for (int d = kWave / 2; d > 0; d >>= 1) {
        lb += __shfl_xor(lb, d);
        lg += __shfl_xor(lg, d);
    }
    if (e) return;
    lb = o.cb != 0.f ? o.cb * lb : 0.;
    lg *= o.cg;
    const double lz = o.cz != 0.f ? o.cz * s_p[Ne] : 0.;
    o.loss[0] = static_cast<float>(lb + lg + lz);
    o.loss[1] = static_cast<float>(lb);
    o.loss[2] = static_cast<float>(lg);
    o.loss[3] = static_cast<float>(lz);
}

// Workgroup b's tokens are [b per_block, ...).  A single workgroup finishes;
// of several each leaves its sums in part.
template <int L, int NI, bool VEC>
__global__ __launch_bounds__(kBalThreads) void k_balance(const float *__restrict__ logits,
                                                         const int32_t *__restrict__ ids,
                                                         const uint8_t *__restrict__ valid,
                                                         unsigned T, int Ne, int k,
                                                         unsigned per_block,
                                                         float *__restrict__ part, PlaceTab tab,
                                                         BalanceOut o) {
    constexpr unsigned kTeams = kBalThreads / L;
    __shared__ int s_hits[kMaxNe + 1];
    __shared__ float s_w[kBalWaves][kMaxNe], s_z[kBalWaves];
    for (int e = threadIdx.x; e <= Ne; e += kBalThreads) s_hits[e] = 0;
    __syncthreads();
    const unsigned t0 = blockIdx.x * per_block, t1 = min(T, t0 + per_block);
    const int l = threadIdx.x % L, team = threadIdx.x / L;
    const int w = threadIdx.x / kWave, lane = lane_id();

    float pn[NI];
    uint8_t ok;
    const float *base = logits + static_cast<size_t>(t0) * Ne;
    const uint8_t *mask = valid ? valid : reinterpret_cast<const uint8_t *>(logits);
    auto load = [&](unsigned t) {
        t = min(t, t1 - 1);
        ok = mask[t];
        team_load<L, NI, VEC>(base, t - t0, l, Ne, pn);
    };
    load(t0 + team);

    // counts, an id at a time
    const unsigned slots = t1 > t0 ? (t1 - t0) * k : 0;
    const int32_t *own_ids = ids + static_cast<size_t>(t0) * k;
    for (unsigned i = threadIdx.x; i < slots; i += 4 * kBalThreads) {
        unsigned e[4];
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const unsigned iq = i + q * kBalThreads;
            const bool counts = iq < slots && (!valid || valid[t0 + iq / k]);
            e[q] = counts ? static_cast<unsigned>(own_ids[iq]) : 0xffffffffu;
        }
#pragma unroll
        for (int q = 0; q < 4; q++)
            if (e[q] < static_cast<unsigned>(Ne)) atomicAdd(&s_hits[e[q]], 1);
    }
    int n_valid = 0;
    for (unsigned t = t0 + threadIdx.x; t < t1; t += kBalThreads) n_valid += !valid || valid[t];
    n_valid = wave_sum_i(n_valid);
    if (lane == 0 && n_valid) atomicAdd(&s_hits[Ne], n_valid);

    float acc[NI], z = 0.f;
#pragma unroll
    for (int i = 0; i < NI; i++) acc[i] = 0.f;
    for (unsigned t = t0 + team; t < t1; t += kTeams) {
        float p[NI];
#pragma unroll
        for (int i = 0; i < NI; i++) p[i] = pn[i];
        team_mask<L, NI, VEC>(!valid || ok, l, Ne, p);
        load(t + kTeams);
        // a token that does not count is a row of -inf: p = 0, lse = 0
        const float lse = team_softmax<L, NI>(p);
#pragma unroll
        for (int i = 0; i < NI; i++) acc[i] += p[i];
        z = fmaf(lse, lse, z);
    }
    // the teams of a wave, then the waves in order
#pragma unroll
    for (int i = 0; i < NI; i++) {
        if constexpr (L <= 16) acc[i] += __shfl_xor(acc[i], 16);
        if constexpr (L <= 32) acc[i] += __shfl_xor(acc[i], 32);
        const int e = expert<L, NI, VEC>(l, i);
        if (lane < L && e < Ne) s_w[w][e] = acc[i];
    }
    if constexpr (L <= 16) z += __shfl_xor(z, 16);
    if constexpr (L <= 32) z += __shfl_xor(z, 32);
    if (lane == 0) s_z[w] = z;
    __syncthreads();
    const int e = threadIdx.x;
    float sum = 0.f;
    if (e <= Ne)
        for (int q = 0; q < kBalWaves; q++) sum += e < Ne ? s_w[q][e] : s_z[q];
    const int hits = e <= Ne ? s_hits[e] : 0;
    if (gridDim.x == 1) {
        finish(sum, hits, 1, Ne, k, tab, o);
    } else if (e <= Ne) {
        float *out = part + static_cast<size_t>(blockIdx.x) * part_words(Ne);
        out[e] = sum;
        out[Ne + 1 + e] = __int_as_float(hits);
    }
}

// The workgroups' parts added up.
__global__ __launch_bounds__(kBalThreads) void k_balance_final(const float *__restrict__ part,
                                                               int blocks, int Ne, int k,
                                                               PlaceTab tab, BalanceOut o) {
    const int cols = Ne + 1, shares = kBalThreads / cols;
    const int e = threadIdx.x % cols, sh = threadIdx.x / cols;
    double p = 0.;
    int c = 0;
    if (sh < shares)
#pragma unroll 8
        for (int b = sh; b < blocks; b += shares) {
            const float *row = part + static_cast<size_t>(b) * part_words(Ne);
            p += row[e];
            c += __float_as_int(row[cols + e]);
        }
    finish(p, c, shares, Ne, k, tab, o);
}

template <int L, int NI, bool VEC>
__global__ __launch_bounds__(kBackThreads) void k_balance_back(
    const float *logits, const uint8_t *__restrict__ valid, const int32_t *__restrict__ counts,
    PlaceTab tab, unsigned T, int Ne, int k, float cb, float cg, float cz, float dloss,
    const float *dlogits_in, float *dlogits) {
    constexpr unsigned kTeams = kBackThreads / L;
    __shared__ float s_f[kMaxNe], s_c[kMaxNe];
    const int l = threadIdx.x % L;
    const unsigned stride = gridDim.x * kTeams;
    float pn[NI], gn[NI];
    uint8_t ok;
    const uint8_t *mask = valid ? valid : reinterpret_cast<const uint8_t *>(logits);
    const float *into = dlogits_in ? dlogits_in : logits;
    const unsigned team = threadIdx.x / L;
    auto load = [&](unsigned t) {  // t: the workgroup's first token
        t = min(t, T - 1);
        const unsigned row = min(team, T - 1 - t);
        const size_t base = static_cast<size_t>(t) * Ne;
        ok = mask[t + row];
        team_load<L, NI, VEC>(logits + base, row, l, Ne, pn);
        team_load<L, NI, VEC>(into + base, row, l, Ne, gn);
    };
    load(blockIdx.x * kTeams);  // in flight while the workgroup makes its coefficients
    const int n = counts[Ne];
    for (int e = threadIdx.x; e < Ne; e += kBackThreads)
        s_f[e] = n ? static_cast<float>(counts[e]) * Ne / (static_cast<float>(k) * n) : 0.f;
    __syncthreads();
    for (int e = threadIdx.x; e < Ne; e += kBackThreads) {
        float c = cb * (s_f[e] - 1.f);
        if (cg != 0.f) {
            const int g = tab.grp[e];
            float f = 0.f;
            for (int j = 0; j < tab.n; j++) f += s_f[tab.expert[g * tab.n + j]];
            c += cg * (f / tab.n - 1.f);
        }
        s_c[e] = c;
    }
    __syncthreads();
    float c[NI];
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int e = expert<L, NI, VEC>(l, i);
        c[i] = e < Ne ? s_c[e] : 0.f;
    }
    const float up = n ? dloss / n : 0.f;
    for (unsigned t = blockIdx.x * kTeams; t < T; t += stride) {
        float p[NI], g[NI], dot = 0.f;
        const bool in = !valid || ok;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            p[i] = pn[i];
            g[i] = dlogits_in ? gn[i] : 0.f;
        }
        team_mask<L, NI, VEC>(in, l, Ne, p);
        load(t + stride);
        const float lse = team_softmax<L, NI>(p);
#pragma unroll
        for (int i = 0; i < NI; i++) dot = fmaf(c[i], p[i], dot);
        const float add = 2.f * cz * lse - group_sum<L>(dot);
        // a token that does not count keeps what came in
#pragma unroll
        for (int i = 0; i < NI; i++) g[i] = in ? fmaf(up * p[i], c[i] + add, g[i]) : g[i];
        if (t + team >= T) continue;
        float *to = dlogits + static_cast<size_t>(t + team) * Ne;
        if constexpr (VEC) {
            if (4 * l < Ne) *reinterpret_cast<f32x4 *>(to + 4 * l) = f32x4{g[0], g[1], g[2], g[3]};
        } else {
#pragma unroll
            for (int i = 0; i < NI; i++)
                if (l + L * i < Ne) to[l + L * i] = g[i];
        }
    }
}

// f(L, NI, VEC): the smallest team that holds Ne logits, four consecutive
// ones to a lane where they can be moved as one vector.
template <typename F>
void by_experts(int Ne, bool aligned, F f) {
    using std::integral_constant;
    typedef integral_constant<int, 4> I4;
    const bool vec = aligned && Ne % 4 == 0;
    const auto four = [&](auto L) {
        if (vec)
            f(L, I4{}, std::true_type{});
        else
            f(L, I4{}, std::false_type{});
    };
    if (Ne <= 16)
        f(integral_constant<int, 16>{}, integral_constant<int, 1>{}, std::false_type{});
    else if (Ne <= 32)
        f(integral_constant<int, 16>{}, integral_constant<int, 2>{}, std::false_type{});
    else if (Ne <= 64)
        four(integral_constant<int, 16>{});
    else if (Ne <= 128)
        four(integral_constant<int, 32>{});
    else
        four(integral_constant<int, 64>{});
}
bool vector_aligned(const float *a, const float *b = nullptr, const float *c = nullptr) {
    return (reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
            reinterpret_cast<uintptr_t>(c)) % 16 == 0;
}

// Forward workgroups at most: one per CU (at T = 65536, Ne = 60 6.4 us and 5.8
// for the sum of the parts; half as many 8.3 and 4.7).
constexpr int kBalBlocks = 256;
// Up to this many tokens for each of its teams a batch takes one workgroup,
// which finishes too: at T = 512, Ne = 64 a call of 9.2 us, where several
// workgroups and their sum take 13.1 since the host launches twice (captured:
// 7.6 against 6.7); with twice the tokens 11.8 against 12.9 (11.1 and 7.0).
constexpr int kOneBlockSteps = 8;
// Backward workgroups at most: four per CU (10.1 us at T = 65536; two 10.2,
// eight 12.2).
constexpr unsigned kBackBlocks = 1024;

}  // namespace

static int balance_blocks(int T, int Ne) {
    const int team = Ne <= 64 ? 16 : Ne <= 128 ? 32 : 64;  // as in by_experts
    if (T <= kOneBlockSteps * (kBalThreads / team)) return 1;
    return static_cast<int>(std::min(ceil_div(T, 64), static_cast<unsigned>(kBalBlocks)));
}

size_t balance_part_bytes(int T, int Ne) {
    return static_cast<size_t>(balance_blocks(T, Ne)) * part_words(Ne) * 4;
}

hipError_t launch_balance(const float *logits, const int32_t *ids, const uint8_t *valid, int T,
                          int k, const PlaceTab &tab, float cb, float cg, float cz,
                          int32_t *counts, float *probs, float *loss, float *part, hipStream_t s) {
    const int Ne = tab.Ne;
    const unsigned per = ceil_div(T, balance_blocks(T, Ne)), grid = ceil_div(T, per);
    const BalanceOut o{cb, cg, cz, counts, probs, loss};
    by_experts(Ne, vector_aligned(logits), [&](auto L, auto NI, auto VEC) {
        k_balance<decltype(L)::value, decltype(NI)::value, decltype(VEC)::value>
            <<<grid, kBalThreads, 0, s>>>(logits, ids, valid, T, Ne, k, per, part, tab, o);
    });
    if (grid > 1)
        k_balance_final<<<1, kBalThreads, 0, s>>>(part, static_cast<int>(grid), Ne, k, tab, o);
    return hipGetLastError();
}

hipError_t launch_balance_back(const float *logits, const uint8_t *valid, const int32_t *counts,
                               const PlaceTab &tab, int T, int k, float cb, float cg, float cz,
                               float dloss, const float *dlogits_in, float *dlogits,
                               hipStream_t s) {
    const int Ne = tab.Ne;
    by_experts(Ne, vector_aligned(logits, dlogits_in, dlogits), [&](auto L, auto NI, auto VEC) {
        constexpr int kTeams = kBackThreads / decltype(L)::value;
        const unsigned grid = std::min(ceil_div(T, kTeams), kBackBlocks);
        k_balance_back<decltype(L)::value, decltype(NI)::value, decltype(VEC)::value>
            <<<grid, kBackThreads, 0, s>>>(logits, valid, counts, tab, T, Ne, k, cb, cg, cz, dloss,
                                           dlogits_in, dlogits);
    });
    return hipGetLastError();
}

}  // namespace occ
