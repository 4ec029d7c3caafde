// The row movers of the layer with 8-bit experts: the quantiser of rows
// (tokens, hidden states, weights) and the sum of a token's terms.  Both are
// bound by memory: 65536 rows of 2048 bf16 72.7 us (5.5 TB/s), the fp32 hidden
// states of 65536 slots of 1024 behind the up-projection 54.7 (6.1 TB/s, some
// from the caches); the terms of 8192 tokens of 2048, eight each, 48.4 us (302
// MB, 6.2 TB/s).
#include <algorithm>

#include "int8_rows.h"

namespace occ {
namespace {

constexpr int kQuantThreads = 256;
constexpr size_t kMaxGrid = 1 << 22;  // workgroups; larger problems loop
// One wave a row of at most 64 NV chunks; longer rows (NV = 0) take a workgroup
// and are read twice, the second time from the caches (8192 rows of 16384 bf16
// 107.6 us, 3.7 TB/s).
template <bool BF16, int NV>
__global__ __launch_bounds__(kQuantThreads) void k_quantize_rows(const u32x4 *__restrict__ x, size_t rows,
                                                                 int chunks, int8_t *__restrict__ q,
                                                                 size_t ldq, float *__restrict__ scale) {
    if constexpr (NV != 0) {
        constexpr int kTeams = kQuantThreads / kWave;
        for (size_t row = static_cast<size_t>(blockIdx.x) * kTeams + threadIdx.x / kWave; row < rows;
             row += static_cast<size_t>(gridDim.x) * kTeams)
            quantise_row<BF16, NV>(x + row * chunks, chunks, q + row * ldq, ldq, scale + row);
    } else {
        constexpr int per = Chunk<BF16>::N;
        __shared__ uint32_t part[kQuantThreads / kWave];
        const int i = threadIdx.x;
        for (size_t row = blockIdx.x; row < rows; row += gridDim.x) {
            const u32x4 *src = x + row * chunks;
            Chunk<BF16> v;
            uint32_t m = 0;
            for (int c = i; c < chunks; c += kQuantThreads) {
                v.from(src[c]);
                m = max(m, v.top());
            }
            m = wave_top(m);
            __syncthreads();  // the last row's maxima have been read
            if (lane_id() == 0) part[threadIdx.x / kWave] = m;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kQuantThreads / kWave; j++) m = max(m, part[j]);
            const RowScale r(m);
            if (i == 0) scale[row] = r.scale;
            int8_t *dst = q + row * ldq;
            for (int c = i; c < chunks; c += kQuantThreads) {
                v.from(src[c]);
                store_codes(v, r, dst + static_cast<size_t>(c) * per);
            }
            for (size_t c = static_cast<size_t>(chunks) * per + 4 * i; c < ldq; c += 4 * kQuantThreads)
                *reinterpret_cast<uint32_t *>(dst + c) = 0u;
        }
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
                                size_t ldq, float *scale, hipStream_t s) {
    const int chunks = cols / (bf16 ? 8 : 4);
    const u32x4 *xs = static_cast<const u32x4 *>(x);
    const int nv = (chunks + kWave - 1) / kWave;
    const size_t rows_per = nv <= 8 ? kQuantThreads / kWave : 1;
    const unsigned grid = static_cast<unsigned>(std::min<size_t>(ceil_div(rows, rows_per), kMaxGrid));
#define OCC_QUANT(NV)                                                                                       \
    do {                                                                                                    \
        if (bf16) k_quantize_rows<true, NV><<<grid, kQuantThreads, 0, s>>>(xs, rows, chunks, q, ldq, scale); \
        else k_quantize_rows<false, NV><<<grid, kQuantThreads, 0, s>>>(xs, rows, chunks, q, ldq, scale);     \
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
