// The layer with 8-bit experts for few tokens (single tokens of a decode
// step), in two launches.  Each slot (token, expert) multiplies its expert's
// weights by one row, so that the weights' bytes are all that counts: waves
// read whole weight rows, 16 bytes a lane, and sum them with
// v_dot4_i32_i8; nothing is gathered, sorted or padded.
//   up    a workgroup takes kFewF features of a slot: it asks for its weights,
//         quantises the token's row while they come, and leaves h in fp32;
//   down  a workgroup takes kFewC columns of a token over all of its slots: it
//         asks for its weights, quantises the slots' h while they come, and
//         adds the terms.
// One token of top 8 (d = 2048, F = 1024): 8.2 + 8.6 us for 33.6 + 16.8 MB (4.1
// and 1.9 TB/s), where the shortest kernel with one load takes 3 us.
// Codes, integer sums, terms and the order of their sum are those of the
// general path: a token's y does not depend on the batch that it came in.
#include "int8_rows.h"

namespace occ {
namespace {

constexpr int kFewThreads = 256, kFewWaves = kFewThreads / kWave;
constexpr int kFewF = 16;  // features a workgroup, 4 a wave
constexpr int kFewC = 8;   // columns a workgroup, 2 a wave
constexpr int kFewSlots = 8;  // slots whose weights a wave asks for at once

__device__ __forceinline__ int dot16(u32x4 a, u32x4 b, int c) {
#pragma unroll
    for (int i = 0; i < 4; i++)
        c = __builtin_amdgcn_sdot4(static_cast<int>(a[i]), static_cast<int>(b[i]), c, false);
    return c;
}

// Lane j < k: the expert of the token's slot j and its weight, after the rule
// for ids that are out of range or repeated (the lowest unused expert, weight
// 0); the lanes behind hold expert 0.  Every lane of the wave calls it.
__device__ __forceinline__ void token_slots(const int32_t *ids, const float *w, int t, int k, int Ne,
                                            int &e, float &wt) {
    const int lane = lane_id();
    const size_t at = static_cast<size_t>(t) * k + min(lane, k - 1);
    e = lane < k ? ids[at] : 0;
    wt = w[at];
    bool odd = lane < k && (e < 0 || e >= Ne);
    for (int i = 0; i < k; i++) {
        const int ei = __builtin_amdgcn_readlane(e, i);
        odd = odd || (lane > i && lane < k && e == ei);
    }
    if (__ballot(odd) == 0) return;
    // one slot after another; lane l keeps whether experts l + 64 q are used
    bool used[kMaxNe / kWave];
#pragma unroll
    for (int q = 0; q < kMaxNe / kWave; q++) used[q] = false;
    for (int i = 0; i < k; i++) {
        int to = __builtin_amdgcn_readlane(e, i);
        int taken = 0, free = Ne - 1;
#pragma unroll
        for (int q = kMaxNe / kWave - 1; q >= 0; q--) {
            const uint64_t open = __ballot(!used[q] && lane + kWave * q < Ne);
            if (open) free = kWave * q + __builtin_ctzll(open);
            taken |= __ballot(used[q] && lane + kWave * q == to) != 0;
        }
        const bool good = to >= 0 && to < Ne && !taken;
        to = good ? to : free;
#pragma unroll
        for (int q = 0; q < kMaxNe / kWave; q++) used[q] = used[q] || lane + kWave * q == to;
        if (lane == i) {
            e = to;
            wt = good ? wt : 0.f;
        }
    }
}

// h of one slot's features: blocks of the routed slots first (slot by slot),
// then of the shared experts'.
template <int NC>  // 16-byte chunks of a weight row a lane has at once
__global__ __launch_bounds__(kFewThreads) void k_few_up(FewArgs a) {
    __shared__ u32x4 s_x[kFewMaxD / 16];
    __shared__ uint32_t s_top[kFewWaves];
    const int lane = lane_id(), wv = threadIdx.x / kWave, d = a.d;
    const int per = (a.F + kFewF - 1) / kFewF, routed = a.T * a.k * per;
    int b = blockIdx.x, t, f0, F, e;
    float wt = 1.f;
    float *h;
    Int8Weights W = a.routed;
    // the row first: what is asked for last is waited for last
    const bool shared = b >= routed;
    int slot;
    if (shared) {
        b -= routed;
        F = a.F_shared;
        const int per_sh = (F + kFewF - 1) / kFewF;
        slot = b / per_sh;
        f0 = (b - slot * per_sh) * kFewF;
        t = slot / a.n_shared;
        e = slot - t * a.n_shared;
        W = a.shared;
        h = a.h_sh + static_cast<size_t>(slot) * F;
    } else {
        F = a.F;
        slot = b / per;
        f0 = (b - slot * per) * kFewF;
        t = slot / a.k;
        h = a.h + static_cast<size_t>(slot) * F;
    }
    const int chunks8 = d / 8, chunks = d / 16;  // of the bf16 row, of the codes
    const u32x4 *x = reinterpret_cast<const u32x4 *>(a.x) + static_cast<size_t>(t) * chunks8;
    constexpr int XPT = kFewMaxD / 8 / kFewThreads;
    u32x4 raw[XPT];
#pragma unroll
    for (int i = 0; i < XPT; i++)
        if (i == 0 || i * kFewThreads < chunks8) raw[i] = x[min(static_cast<int>(threadIdx.x) + i * kFewThreads, chunks8 - 1)];
    if (!shared) {
        int ej;
        float wj;
        token_slots(a.ids, a.w, t, a.k, a.Ne, ej, wj);
        const int j = slot - t * a.k;
        e = __builtin_amdgcn_readlane(ej, j);
        wt = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wj), j));
    }
    const int fw = f0 + 4 * wv;
    const u32x4 *row[8];  // gate rows of 4 features, then up rows
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int f = min(fw + (i & 3), F - 1);
        row[i] = reinterpret_cast<const u32x4 *>((i < 4 ? W.gate : W.up) + (static_cast<size_t>(e) * F + f) * d);
    }
    u32x4 v[8][NC];
#pragma unroll
    for (int c = 0; c < NC; c++)
#pragma unroll
        for (int i = 0; i < 8; i++) v[i][c] = __builtin_nontemporal_load(row[i] + min(lane + kWave * c, chunks - 1));
    float sg = 0.f, su = 0.f;  // lane i < 4: of feature i
    {
        const size_t at = static_cast<size_t>(e) * F + min(fw + (lane & 3), F - 1);
        sg = W.gate_scale[at];
        su = W.up_scale[at];
    }
    // the row's codes
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < XPT; i++)
        if (i == 0 || i * kFewThreads < chunks8) {
            Chunk<true> cx;
            cx.from(raw[i]);
            m = max(m, cx.top());
        }
    m = wave_top(m);
    if (lane == 0) s_top[wv] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFewWaves; i++) m = max(m, s_top[i]);
    const RowScale r(m);
#pragma unroll
    for (int i = 0; i < XPT; i++) {
        const int c = threadIdx.x + i * kFewThreads;
        if (c < chunks8) {
            Chunk<true> cx;
            cx.from(raw[i]);
            reinterpret_cast<u32x2 *>(s_x)[c] = u32x2{r.code4(cx.v[0], cx.v[1], cx.v[2], cx.v[3]),
                                                      r.code4(cx.v[4], cx.v[5], cx.v[6], cx.v[7])};
        }
    }
    __syncthreads();
    int acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int c0 = 0; c0 < chunks; c0 += NC * kWave) {
#pragma unroll
        for (int c = 0; c < NC; c++) {
            const int at = c0 + lane + kWave * c;
            const u32x4 xq = at < chunks ? s_x[at] : u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; i++) acc[i] = dot16(v[i][c], xq, acc[i]);
        }
        if (c0 + NC * kWave < chunks) {
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int i = 0; i < 8; i++)
                    v[i][c] = __builtin_nontemporal_load(row[i] + min(c0 + (NC + c) * kWave + lane, chunks - 1));
        }
    }
    int g = 0, u = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int gi = wave_sum_i(acc[i]), ui = wave_sum_i(acc[i + 4]);
        g = lane == i ? gi : g;
        u = lane == i ? ui : u;
    }
    if (lane < 4 && fw + lane < F)
        h[fw + lane] = swiglu(static_cast<float>(g) * (r.scale * sg), static_cast<float>(u) * (r.scale * su)) * wt;
}

// A row of h as codes in LDS (rows of F, a multiple of 64), by one wave;
// returns its scale.
__device__ __forceinline__ float quantise_h(const float *h, int F, uint32_t *codes) {
    const int lane = lane_id(), chunks = F / 4;
    const u32x4 *src = reinterpret_cast<const u32x4 *>(h);
    constexpr int NH = 4;
    u32x4 raw[NH];
    uint32_t m = 0;
    for (int c0 = 0; c0 < chunks; c0 += NH * kWave) {
#pragma unroll
        for (int i = 0; i < NH; i++) raw[i] = src[min(c0 + lane + kWave * i, chunks - 1)];
#pragma unroll
        for (int i = 0; i < NH; i++) {
            Chunk<false> x;
            x.from(raw[i]);
            m = max(m, x.top());
        }
    }
    const RowScale r(wave_top(m));
    for (int c0 = 0; c0 < chunks; c0 += NH * kWave) {
        if (chunks > NH * kWave) {
#pragma unroll
            for (int i = 0; i < NH; i++) raw[i] = src[min(c0 + lane + kWave * i, chunks - 1)];
        }
#pragma unroll
        for (int i = 0; i < NH; i++) {
            Chunk<false> x;
            x.from(raw[i]);
            if (c0 + lane + kWave * i < chunks) codes[c0 + lane + kWave * i] = r.code4(x.v[0], x.v[1], x.v[2], x.v[3]);
        }
    }
    return r.scale;
}

// kFewC columns of a token.  Slots in batches: their weights are asked for,
// the first batch's before the codes are made.
template <int NC>
__global__ __launch_bounds__(kFewThreads) void k_few_down(FewArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint32_t s_codes[];
    __shared__ float s_scale[kMaxK + kFewMaxShared];
    const int lane = lane_id(), wv = threadIdx.x / kWave;
    const int per = (a.d + kFewC - 1) / kFewC;
    const int t = blockIdx.x / per, c0 = (blockIdx.x - t * per) * kFewC + 2 * wv;
    const int k = a.k, F = a.F, Fs = a.F_shared, chunks = F / 16;
    int e;
    float wt;
    token_slots(a.ids, a.w, t, k, a.Ne, e, wt);
    const int col[2] = {min(c0, a.d - 1), min(c0 + 1, a.d - 1)};
    const float sd0 = a.routed.down_scale[static_cast<size_t>(e) * a.d + col[0]];  // lane j: of slot j
    const float sd1 = a.routed.down_scale[static_cast<size_t>(e) * a.d + col[1]];
    u32x4 v[kFewSlots][2][NC];
    const auto ask = [&](int j0) {
#pragma unroll
        for (int j = 0; j < kFewSlots; j++) {
            const int ej = __builtin_amdgcn_readlane(e, min(j0 + j, k - 1));
            if (j0 + j < k) {
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const u32x4 *row = reinterpret_cast<const u32x4 *>(a.routed.down + (static_cast<size_t>(ej) * a.d + col[i]) * F);
#pragma unroll
                    for (int c = 0; c < NC; c++) v[j][i][c] = __builtin_nontemporal_load(row + min(lane + kWave * c, chunks - 1));
                }
            }
        }
    };
    ask(0);
    for (int j = wv; j < k; j += kFewWaves) {
        const float s = quantise_h(a.h + (static_cast<size_t>(t) * k + j) * F, F, s_codes + j * (F / 4));
        if (lane == 0) s_scale[j] = s;
    }
    uint32_t *codes_sh = s_codes + k * (F / 4);
    for (int j = wv; j < a.n_shared; j += kFewWaves) {
        const float s = quantise_h(a.h_sh + (static_cast<size_t>(t) * a.n_shared + j) * Fs, Fs, codes_sh + j * (Fs / 4));
        if (lane == 0) s_scale[kMaxK + j] = s;
    }
    __syncthreads();
    float y[2] = {0.f, 0.f};
    // a term, rounded as the general path's
    const auto term = [](int sum, float hs, float sd) {
        return bf16_bits_to_f32(f32_to_bf16_bits(static_cast<float>(sum) * (hs * sd)));
    };
    for (int j0 = 0; j0 < k; j0 += kFewSlots) {
        if (j0) ask(j0);
#pragma unroll
        for (int j = 0; j < kFewSlots; j++) {
            if (j0 + j < k) {
                const u32x4 *hq = reinterpret_cast<const u32x4 *>(s_codes + (j0 + j) * (F / 4));
                int acc[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    const int at = lane + kWave * c;
                    const u32x4 q = at < chunks ? hq[at] : u32x4{0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < 2; i++) acc[i] = dot16(v[j][i][c], q, acc[i]);
                }
                if (chunks > NC * kWave) {  // the rest of a long row
                    const int ej = __builtin_amdgcn_readlane(e, j0 + j);
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const u32x4 *row = reinterpret_cast<const u32x4 *>(a.routed.down + (static_cast<size_t>(ej) * a.d + col[i]) * F);
#pragma unroll 4
                        for (int at = NC * kWave + lane; at < chunks; at += kWave) acc[i] = dot16(row[at], hq[at], acc[i]);
                    }
                }
                const float hs = s_scale[j0 + j];
                const float d0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sd0), j0 + j));
                const float d1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sd1), j0 + j));
                y[0] += term(wave_sum_i(acc[0]), hs, d0);
                y[1] += term(wave_sum_i(acc[1]), hs, d1);
            }
        }
    }
    for (int j = 0; j < a.n_shared; j++) {
        const u32x4 *hq = reinterpret_cast<const u32x4 *>(codes_sh + j * (Fs / 4));
        const u32x4 *r0 = reinterpret_cast<const u32x4 *>(a.shared.down + (static_cast<size_t>(j) * a.d + col[0]) * Fs);
        const u32x4 *r1 = reinterpret_cast<const u32x4 *>(a.shared.down + (static_cast<size_t>(j) * a.d + col[1]) * Fs);
        int acc0 = 0, acc1 = 0;
#pragma unroll 4
        for (int at = lane; at < Fs / 16; at += kWave) {
            const u32x4 q = hq[at];
            acc0 = dot16(r0[at], q, acc0);
            acc1 = dot16(r1[at], q, acc1);
        }
        y[0] += term(wave_sum_i(acc0), s_scale[kMaxK + j], a.shared.down_scale[static_cast<size_t>(j) * a.d + col[0]]);
        y[1] += term(wave_sum_i(acc1), s_scale[kMaxK + j], a.shared.down_scale[static_cast<size_t>(j) * a.d + col[1]]);
    }
    if (lane < 2 && c0 + lane < a.d)
        a.y[static_cast<size_t>(t) * a.d + c0 + lane] = f32_to_bf16_bits(lane ? y[1] : y[0]);
}

}  // namespace

// The codes of a token's hidden states, which the down kernel keeps in LDS.
static size_t few_lds(const FewArgs &a) {
    return static_cast<size_t>(a.k) * a.F + static_cast<size_t>(a.n_shared) * a.F_shared;
}

bool few_fits(int d, int k, int F, int n_shared, int F_shared) {
    FewArgs a{};
    a.k = k;
    a.F = F;
    a.n_shared = n_shared;
    a.F_shared = F_shared;
    return d <= kFewMaxD && n_shared <= kFewMaxShared && few_lds(a) <= 48 * 1024;
}

hipError_t launch_few(const FewArgs &a, hipStream_t s) {
    const size_t up = static_cast<size_t>(a.T) * (static_cast<size_t>(a.k) * ceil_div(a.F, kFewF) +
                                                  static_cast<size_t>(a.n_shared) * ceil_div(a.F_shared, kFewF));
    const unsigned grid = static_cast<unsigned>(up);
    if (a.d <= 1024) k_few_up<1><<<grid, kFewThreads, 0, s>>>(a);
    else k_few_up<2><<<grid, kFewThreads, 0, s>>>(a);
    const unsigned down = static_cast<unsigned>(a.T) * ceil_div(a.d, kFewC);
    const size_t lds = few_lds(a);
    if (a.F <= 1024) k_few_down<1><<<down, kFewThreads, lds, s>>>(a);
    else k_few_down<2><<<down, kFewThreads, lds, s>>>(a);
    return hipGetLastError();
}

}  // namespace occ
