// The row movers of the layer with 8-bit experts: the quantiser of rows
// (tokens, hidden states, weights) and the sum of a token's terms.  Both are
// bound by memory.
#include <algorithm>

#include "launch.h"

namespace occ {
namespace {

constexpr int kQuantThreads = 256;
constexpr size_t kMaxGrid = 1 << 22;  // workgroups; larger problems loop
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

// A 16-byte chunk of a row as floats: 8 bf16 or 4 fp32.
template <bool BF16>
struct Chunk {
    static constexpr int N = BF16 ? 8 : 4;
    float v[N];
    __device__ __forceinline__ void from(u32x4 raw) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (BF16) {
                v[2 * i] = __uint_as_float(raw[i] << 16);
                v[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u);
            } else {
                v[i] = __uint_as_float(raw[i]);
            }
        }
    }
    // The largest magnitude's bits: as whole numbers in the order of the
    // magnitudes, infinity and NaN above all others.
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < N; i++) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        return m;
    }
};

__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d, float inv) {
    const auto code = [inv](float x) {
        return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(x * inv), -127.f), 127.f))) & 0xffu;
    };
    return code(a) | code(b) << 8 | code(c) << 16 | code(d) << 24;
}

// The row's factor of its values and what a code stands for, from its largest
// magnitude's bits.  Not finite: codes of zero and a scale of NaN.
__device__ __forceinline__ void row_scale(uint32_t bits, float &inv, float &scale) {
    const float a = __uint_as_float(bits);
    const bool bad = bits >= 0x7f800000u, held = !bad && a >= kInt8Tiny;
    inv = held ? 127.f / a : 0.f;
    scale = bad ? __uint_as_float(0x7fc00000u) : held ? a / 127.f : 0.f;
}

template <bool BF16>
__device__ __forceinline__ void store_codes(const Chunk<BF16> &x, bool bad, float inv, int8_t *q) {
    uint32_t c[Chunk<BF16>::N / 4];
#pragma unroll
    for (int i = 0; i < Chunk<BF16>::N / 4; i++)
        c[i] = bad ? 0u : code4(x.v[4 * i], x.v[4 * i + 1], x.v[4 * i + 2], x.v[4 * i + 3], inv);
    if constexpr (BF16) *reinterpret_cast<u32x2 *>(q) = u32x2{c[0], c[1]};
    else *reinterpret_cast<uint32_t *>(q) = c[0];
}

// One wave a row of at most 64 NV chunks, held in registers between the
// maximum and the codes; longer rows (NV = 0) take a workgroup and are read
// twice, the second time from the caches.
template <bool BF16, int NV>
__global__ __launch_bounds__(kQuantThreads) void k_quantize_rows(
    const u32x4 *__restrict__ x, size_t rows, int chunks, int8_t *__restrict__ q, size_t ldq,
    float *__restrict__ scale, const int32_t *__restrict__ tok_epd, int k,
    int32_t *__restrict__ epd_tok) {
    constexpr int kTeam = NV ? kWave : kQuantThreads, kTeams = kQuantThreads / kTeam, per = Chunk<BF16>::N;
    const int i = threadIdx.x % kTeam;
    for (size_t row = static_cast<size_t>(blockIdx.x) * kTeams + threadIdx.x / kTeam; row < rows;
         row += static_cast<size_t>(gridDim.x) * kTeams) {
        const u32x4 *src = x + row * chunks;
        if (tok_epd)
            for (int j = i; j < k; j += kTeam) epd_tok[tok_epd[row * k + j]] = static_cast<int32_t>(row);
        Chunk<BF16> v[NV ? NV : 1];
        uint32_t m = 0;
        if constexpr (NV != 0) {
#pragma unroll
            for (int j = 0; j < NV; j++) v[j].from(src[min(i + kWave * j, chunks - 1)]);
#pragma unroll
            for (int j = 0; j < NV; j++) m = max(m, v[j].top());
        } else {
            for (int c = i; c < chunks; c += kTeam) {
                v[0].from(src[c]);
                m = max(m, v[0].top());
            }
        }
        // (the bits of a magnitude have no sign: signed order is theirs)
        m = static_cast<uint32_t>(group_reduce<kWave>(static_cast<int>(m), [](int a, int b) { return max(a, b); }));
        if constexpr (NV == 0) {
            __shared__ uint32_t part[kQuantThreads / kWave];
            __syncthreads();  // the last row's maxima have been read
            if (lane_id() == 0) part[threadIdx.x / kWave] = m;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kQuantThreads / kWave; j++) m = max(m, part[j]);
        }
        float inv, sc;
        row_scale(m, inv, sc);
        const bool bad = m >= 0x7f800000u;
        if (i == 0) scale[row] = sc;
        int8_t *dst = q + row * ldq;
        if constexpr (NV != 0) {
#pragma unroll
            for (int j = 0; j < NV; j++) {
                const int c = i + kWave * j;
                if (c < chunks) store_codes(v[j], bad, inv, dst + static_cast<size_t>(c) * per);
            }
        } else {
            for (int c = i; c < chunks; c += kTeam) {
                v[0].from(src[c]);
                store_codes(v[0], bad, inv, dst + static_cast<size_t>(c) * per);
            }
        }
        for (int c = chunks + i; c < static_cast<int>(ldq / per); c += kTeam)
            store_codes(v[0], true, 0.f, dst + static_cast<size_t>(c) * per);
    }
}

// A thread a 16-byte chunk of y; a token's terms are loaded together, kTerms
// at a time.
constexpr int kCombThreads = 256, kTerms = 8;
__global__ __launch_bounds__(kCombThreads) void k_combine_rows(
    const u32x4 *__restrict__ y_epd, const int32_t *__restrict__ tok_epd,
    const u32x4 *__restrict__ y_sh, int n_shared, int T, int k, int chunks, int team_shift,
    u32x4 *__restrict__ y) {
    const int team = 1 << team_shift, i = threadIdx.x & (team - 1);
    const int teams = kCombThreads >> team_shift;
    for (size_t t = static_cast<size_t>(blockIdx.x) * teams + (threadIdx.x >> team_shift); t < static_cast<size_t>(T);
         t += static_cast<size_t>(gridDim.x) * teams) {
        for (int c = i; c < chunks; c += team) {
            float acc[8] = {};
            for (int j0 = 0; j0 < k; j0 += kTerms) {
                u32x4 v[kTerms];
#pragma unroll
                for (int j = 0; j < kTerms; j++) {
                    const size_t row = tok_epd[t * k + min(j0 + j, k - 1)];
                    if (j0 + j < k) v[j] = __builtin_nontemporal_load(y_epd + row * chunks + c);
                }
#pragma unroll
                for (int j = 0; j < kTerms; j++) {
                    if (j0 + j >= k) break;
                    Chunk<true> x;
                    x.from(v[j]);
#pragma unroll
                    for (int e = 0; e < 8; e++) acc[e] += x.v[e];
                }
            }
            for (int s = 0; s < n_shared; s++) {
                Chunk<true> x;
                x.from(__builtin_nontemporal_load(y_sh + (static_cast<size_t>(s) * T + t) * chunks + c));
#pragma unroll
                for (int e = 0; e < 8; e++) acc[e] += x.v[e];
            }
            u32x4 o;
#pragma unroll
            for (int e = 0; e < 4; e++)
                o[e] = static_cast<uint32_t>(f32_to_bf16_bits(acc[2 * e])) |
                       static_cast<uint32_t>(f32_to_bf16_bits(acc[2 * e + 1])) << 16;
            y[t * chunks + c] = o;
        }
    }
}

}  // namespace

hipError_t launch_quantize_rows(const void *x, int bf16, size_t rows, int cols, int8_t *q,
                                size_t ldq, float *scale, const int32_t *tok_epd, int k,
                                int32_t *epd_tok, hipStream_t s) {
    const int chunks = cols / (bf16 ? 8 : 4);
    const u32x4 *xs = static_cast<const u32x4 *>(x);
    const int nv = (chunks + kWave - 1) / kWave;
    const size_t rows_per = nv <= 8 ? kQuantThreads / kWave : 1;
    const unsigned grid = static_cast<unsigned>(std::min<size_t>(ceil_div(rows, rows_per), kMaxGrid));
#define OCC_QUANT(NV)                                                                          \
    do {                                                                                       \
        if (bf16) k_quantize_rows<true, NV><<<grid, kQuantThreads, 0, s>>>(xs, rows, chunks, q, ldq, scale, tok_epd, k, epd_tok);  \
        else k_quantize_rows<false, NV><<<grid, kQuantThreads, 0, s>>>(xs, rows, chunks, q, ldq, scale, tok_epd, k, epd_tok);      \
    } while (0)
    if (nv <= 1) OCC_QUANT(1);
    else if (nv <= 2) OCC_QUANT(2);
    else if (nv <= 4) OCC_QUANT(4);
    else if (nv <= 8) OCC_QUANT(8);
    else OCC_QUANT(0);
#undef OCC_QUANT
    return hipGetLastError();
}

hipError_t launch_combine_rows(const uint16_t *y_epd, const int32_t *tok_epd, const uint16_t *y_sh,
                               int n_shared, int T, int k, int d, uint16_t *y, hipStream_t s) {
    const int chunks = d / 8;
    int shift = 3;  // threads a token: its chunks, at most a workgroup
    while ((1 << shift) < std::min(chunks, kCombThreads)) shift++;
    const unsigned grid = static_cast<unsigned>(std::min<size_t>(ceil_div(T, kCombThreads >> shift), kMaxGrid));
    k_combine_rows<<<grid, kCombThreads, 0, s>>>(
        reinterpret_cast<const u32x4 *>(y_epd), tok_epd, reinterpret_cast<const u32x4 *>(y_sh),
        n_shared, T, k, chunks, shift, reinterpret_cast<u32x4 *>(y));
    return hipGetLastError();
}

}  // namespace occ
