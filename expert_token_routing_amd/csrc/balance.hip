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
// per lane (expert l + L i with lane l), so that a wave works on up to four
// tokens and reduces over a team in 4 to 6 lane exchanges.  The forward adds
// p in registers over a workgroup's tokens and counts in LDS with integer
// atomics (whose order changes nothing); each workgroup leaves its sums in
// the workspace and one workgroup adds them, in a fixed order and in fp64.
#include "launch.h"

namespace occ {
namespace {

constexpr int kBalThreads = 512;
constexpr int kBalWaves = kBalThreads / kWave;
constexpr int kFinalThreads = 1024;

constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

// Reductions over teams of L lanes; every lane of the team gets the result.
template <int L, typename F>
__device__ __forceinline__ float team_reduce(float v, F f) {
    v = f(v, dpp_f<kDppXor1, 0xf>(v, v));
    v = f(v, dpp_f<kDppXor2, 0xf>(v, v));
    v = f(v, dpp_f<kDppHalfMirror, 0xf>(v, v));
    v = f(v, dpp_f<kDppMirror, 0xf>(v, v));
    if constexpr (L >= 32) v = f(v, __shfl_xor(v, 16));
    if constexpr (L >= 64) v = f(v, __shfl_xor(v, 32));
    return v;
}
template <int L>
__device__ __forceinline__ float team_sum(float v) {
    return team_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float team_max(float v) {
    return team_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}

// The softmax of a token's logits (p[i] of expert l + L i, 0 behind Ne) and
// their log-sum-exp.  A row of -inf alone has p = 0 and a log-sum-exp of 0;
// NaN and +inf give NaN.
template <int L, int NI>
__device__ __forceinline__ float team_softmax(const float *__restrict__ row, int l, int Ne,
                                              float (&p)[NI]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int e = l + L * i;
        p[i] = e < Ne ? row[e] : -INFINITY;
        m = fmaxf(m, p[i]);
    }
    m = team_max<L>(m);
    float s = 0.f;
    const float shift = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        p[i] = expf(p[i] - shift);
        s += p[i];
    }
    s = team_sum<L>(s);
    if (s == 0.f) return 0.f;
    const float inv = 1.f / s;
#pragma unroll
    for (int i = 0; i < NI; i++) p[i] *= inv;
    return shift + logf(s);
}

// One workgroup's part: prob sums (Ne floats), z sum, then counts (Ne) and
// valid tokens as int32.
__host__ __device__ inline int part_words(int Ne) { return 2 * Ne + 2; }

template <int L, int NI>
__global__ __launch_bounds__(kBalThreads) void k_balance(const float *__restrict__ logits,
                                                         const int32_t *__restrict__ ids,
                                                         const uint8_t *__restrict__ valid, int T,
                                                         int Ne, int k, int per_block,
                                                         float *__restrict__ part) {
    constexpr int kTeams = kBalThreads / L;
    __shared__ int s_cnt[kMaxNe + 1];
    __shared__ float s_p[kBalWaves][kMaxNe], s_z[kBalWaves];
    for (int e = threadIdx.x; e <= Ne; e += kBalThreads) s_cnt[e] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * per_block, t1 = min(T, t0 + per_block);
    const int l = threadIdx.x % L, team = threadIdx.x / L;
    const int w = threadIdx.x / kWave, lane = lane_id();

    // counts: one thread per token
    int n_valid = 0;
    for (int t = t0 + static_cast<int>(threadIdx.x); t < t1; t += kBalThreads) {
        if (valid && !valid[t]) continue;
        n_valid++;
        const int32_t *row = ids + static_cast<size_t>(t) * k;
        for (int j = 0; j < k; j++) {
            const unsigned e = static_cast<unsigned>(row[j]);
            if (e < static_cast<unsigned>(Ne)) atomicAdd(&s_cnt[e], 1);
        }
    }
    if (n_valid) atomicAdd(&s_cnt[Ne], n_valid);

    float acc[NI], z = 0.f;
#pragma unroll
    for (int i = 0; i < NI; i++) acc[i] = 0.f;
    for (int t = t0 + team; t < t1; t += kTeams) {
        if (valid && !valid[t]) continue;  // the whole team
        float p[NI];
        const float lse = team_softmax<L, NI>(logits + static_cast<size_t>(t) * Ne, l, Ne, p);
#pragma unroll
        for (int i = 0; i < NI; i++) acc[i] += p[i];
        z = fmaf(lse, lse, z);
    }
    // the teams of a wave, then the waves in order
#pragma unroll
    for (int i = 0; i < NI; i++) {
        if constexpr (L <= 16) acc[i] += __shfl_xor(acc[i], 16);
        if constexpr (L <= 32) acc[i] += __shfl_xor(acc[i], 32);
        const int e = l + L * i;
        if (lane < L && e < Ne) s_p[w][e] = acc[i];
    }
    if constexpr (L <= 16) z += __shfl_xor(z, 16);
    if constexpr (L <= 32) z += __shfl_xor(z, 32);
    if (lane == 0) s_z[w] = z;
    __syncthreads();
    float *out = part + static_cast<size_t>(blockIdx.x) * part_words(Ne);
    for (int e = threadIdx.x; e <= Ne; e += kBalThreads) {
        float s = 0.f;
        for (int q = 0; q < kBalWaves; q++) s += e < Ne ? s_p[q][e] : s_z[q];
        out[e] = s;
        out[Ne + 1 + e] = __int_as_float(s_cnt[e]);
    }
}

// The workgroups' parts added up: thread (e, share) takes every shares-th
// part, then the shares are added in order; thread e finishes expert e.
__global__ __launch_bounds__(kFinalThreads) void k_balance_final(
    const float *__restrict__ part, int blocks, int Ne, int k, PlaceTab tab, float cb, float cg,
    float cz, int32_t *__restrict__ counts, float *__restrict__ probs, float *__restrict__ loss) {
    __shared__ double s_sum[kFinalThreads];
    __shared__ int s_cnt[kFinalThreads];
    __shared__ float s_f[kMaxNe];
    __shared__ double s_p[kMaxNe + 1];
    const int cols = Ne + 1, shares = kFinalThreads / cols;
    const int e = threadIdx.x % cols, sh = threadIdx.x / cols;
    double p = 0.;
    int c = 0;
    if (sh < shares)
        for (int b = sh; b < blocks; b += shares) {
            const float *row = part + static_cast<size_t>(b) * part_words(Ne);
            p += row[e];
            c += __float_as_int(row[cols + e]);
        }
    s_sum[threadIdx.x] = p;
    s_cnt[threadIdx.x] = c;
    __syncthreads();
    if (threadIdx.x < cols) {
        for (int q = 1; q < shares; q++) {
            p += s_sum[q * cols + e];
            c += s_cnt[q * cols + e];
        }
        s_cnt[e] = c;
        counts[e] = c;
    }
    __syncthreads();
    const int n = s_cnt[Ne];
    if (threadIdx.x < cols) {
        s_p[e] = n ? p / n : 0.;
        if (e < Ne) {
            probs[e] = static_cast<float>(s_p[e]);
            s_f[e] = n ? static_cast<float>(c) * Ne / (static_cast<float>(k) * n) : 0.f;
        }
    }
    __syncthreads();
    if (threadIdx.x >= kWave) return;
    double lb = 0., lg = 0.;  // lane l: experts l + 64 j, group l
    for (int i = threadIdx.x; i < Ne; i += kWave) lb += s_f[i] * s_p[i];
    if (cg != 0.f && static_cast<int>(threadIdx.x) < tab.Nd) {
        double f = 0., q = 0.;
        for (int j = 0; j < tab.n; j++) {
            const int i = tab.expert[threadIdx.x * tab.n + j];
            f += s_f[i];
            q += s_p[i];
        }
        lg = f / tab.n * q;
    }
    for (int o = kWave / 2; o > 0; o >>= 1) {
        lb += __shfl_xor(lb, o);
        lg += __shfl_xor(lg, o);
    }
    if (threadIdx.x) return;
    lb = cb != 0.f ? cb * lb : 0.;
    lg *= cg;
    const double lz = cz != 0.f ? cz * s_p[Ne] : 0.;
    loss[0] = static_cast<float>(lb + lg + lz);
    loss[1] = static_cast<float>(lb);
    loss[2] = static_cast<float>(lg);
    loss[3] = static_cast<float>(lz);
}

template <int L, int NI>
__global__ __launch_bounds__(kBalThreads) void k_balance_back(
    const float *__restrict__ logits, const uint8_t *__restrict__ valid,
    const int32_t *__restrict__ counts, PlaceTab tab, int T, int Ne, int k, float cb, float cg,
    float cz, float dloss, const float *dlogits_in, float *dlogits) {
    constexpr int kTeams = kBalThreads / L;
    __shared__ float s_f[kMaxNe], s_c[kMaxNe];
    const int n = counts[Ne];
    for (int e = threadIdx.x; e < Ne; e += kBalThreads)
        s_f[e] = n ? static_cast<float>(counts[e]) * Ne / (static_cast<float>(k) * n) : 0.f;
    __syncthreads();
    for (int e = threadIdx.x; e < Ne; e += kBalThreads) {
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
    const int l = threadIdx.x % L;
    float c[NI];
#pragma unroll
    for (int i = 0; i < NI; i++) c[i] = l + L * i < Ne ? s_c[l + L * i] : 0.f;
    const float up = n ? dloss / n : 0.f;
    for (int t = blockIdx.x * kTeams + threadIdx.x / L; t < T; t += gridDim.x * kTeams) {
        const size_t base = static_cast<size_t>(t) * Ne;
        float g[NI];
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int e = l + L * i;
            g[i] = dlogits_in && e < Ne ? dlogits_in[base + e] : 0.f;
        }
        if (!valid || valid[t]) {  // the whole team
            float p[NI], dot = 0.f;
            const float lse = team_softmax<L, NI>(logits + base, l, Ne, p);
#pragma unroll
            for (int i = 0; i < NI; i++) dot = fmaf(c[i], p[i], dot);
            dot = team_sum<L>(dot);
            const float add = 2.f * cz * lse - dot;
#pragma unroll
            for (int i = 0; i < NI; i++) g[i] = fmaf(up * p[i], c[i] + add, g[i]);
        }
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int e = l + L * i;
            if (e < Ne) dlogits[base + e] = g[i];
        }
    }
}

// f(L, NI): the smallest team that holds Ne logits.
template <typename F>
void by_experts(int Ne, F f) {
    using std::integral_constant;
    if (Ne <= 16)
        f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    else if (Ne <= 32)
        f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    else if (Ne <= 64)
        f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    else if (Ne <= 128)
        f(integral_constant<int, 32>{}, integral_constant<int, 4>{});
    else
        f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
}

constexpr int kBalBlocks = 512;  // forward workgroups at most: two per CU

}  // namespace

int balance_blocks(int T) {
    // at least 32 tokens each (two per team of 16 lanes)
    const int need = static_cast<int>(ceil_div(T, 32));
    return need < kBalBlocks ? need : kBalBlocks;
}

size_t balance_part_bytes(int T, int Ne) {
    return static_cast<size_t>(balance_blocks(T)) * part_words(Ne) * 4;
}

hipError_t launch_balance(const float *logits, const int32_t *ids, const uint8_t *valid, int T,
                          int k, const PlaceTab &tab, float cb, float cg, float cz,
                          int32_t *counts, float *probs, float *loss, float *part, hipStream_t s) {
    const int Ne = tab.Ne;
    const int per = static_cast<int>(ceil_div(T, balance_blocks(T)));
    const unsigned grid = ceil_div(T, per);
    by_experts(Ne, [&](auto L, auto NI) {
        k_balance<decltype(L)::value, decltype(NI)::value>
            <<<grid, kBalThreads, 0, s>>>(logits, ids, valid, T, Ne, k, per, part);
    });
    k_balance_final<<<1, kFinalThreads, 0, s>>>(part, static_cast<int>(grid), Ne, k, tab, cb, cg, cz,
                                                counts, probs, loss);
    return hipGetLastError();
}

hipError_t launch_balance_back(const float *logits, const uint8_t *valid, const int32_t *counts,
                               const PlaceTab &tab, int T, int k, float cb, float cg, float cz,
                               float dloss, const float *dlogits_in, float *dlogits,
                               hipStream_t s) {
    const int Ne = tab.Ne;
    by_experts(Ne, [&](auto L, auto NI) {
        constexpr int kTeams = kBalThreads / decltype(L)::value;
        const unsigned need = ceil_div(T, kTeams);
        const unsigned grid = need < 1024 ? need : 1024;
        k_balance_back<decltype(L)::value, decltype(NI)::value><<<grid, kBalThreads, 0, s>>>(
            logits, valid, counts, tab, T, Ne, k, cb, cg, cz, dloss, dlogits_in, dlogits);
    });
    return hipGetLastError();
}

}  // namespace occ
