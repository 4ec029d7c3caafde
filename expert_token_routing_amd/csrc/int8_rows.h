// Rows as 8-bit codes with a scale: the quantiser's arithmetic, shared by the
// row movers (int8.hip) and the few-token kernels (int8_few.hip), whose codes
// must be the same.
#pragma once

#include "launch.h"

namespace occ {

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

// A row's factor of its values and what a code stands for, from its largest
// magnitude's bits.  Not finite: codes of zero and a scale of NaN.
struct RowScale {
    float inv, scale;
    bool bad;
    __device__ __forceinline__ explicit RowScale(uint32_t bits) {
        const float a = __uint_as_float(bits);
        bad = bits >= 0x7f800000u;
        const bool held = !bad && a >= kInt8Tiny;
        inv = held ? 127.f / a : 0.f;
        scale = bad ? __uint_as_float(0x7fc00000u) : held ? a / 127.f : 0.f;
    }
    __device__ __forceinline__ uint32_t code(float x) const {
        return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(x * inv), -127.f), 127.f))) & 0xffu;
    }
    __device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) const {
        return bad ? 0u : code(a) | code(b) << 8 | code(c) << 16 | code(d) << 24;
    }
};

// The largest of a wave's values, in every lane.
__device__ __forceinline__ uint32_t wave_top(uint32_t m) {
    // (the bits of a magnitude have no sign: signed order is theirs)
    return static_cast<uint32_t>(group_reduce<kWave>(static_cast<int>(m), [](int a, int b) { return max(a, b); }));
}

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

// The codes of a chunk at dst (aligned to their number).
template <bool BF16>
__device__ __forceinline__ void store_codes(const Chunk<BF16> &x, const RowScale &r, int8_t *dst) {
    if constexpr (BF16)
        *reinterpret_cast<u32x2 *>(dst) = u32x2{r.code4(x.v[0], x.v[1], x.v[2], x.v[3]),
                                                r.code4(x.v[4], x.v[5], x.v[6], x.v[7])};
    else
        *reinterpret_cast<uint32_t *>(dst) = r.code4(x.v[0], x.v[1], x.v[2], x.v[3]);
}

// A row of at most 64 NV chunks by one wave, held in registers between the
// maximum and the codes where it is at most 8 chunks a lane and read twice
// otherwise; zeros behind it up to ldq bytes.
template <bool BF16, int NV>
__device__ __forceinline__ void quantise_row(const u32x4 *src, int chunks, int8_t *dst, size_t ldq,
                                             float *scale) {
    constexpr int per = Chunk<BF16>::N, B = NV < 8 ? NV : 8;
    const int lane = lane_id();
    u32x4 raw[B];
    uint32_t m = 0;
    Chunk<BF16> x;
#pragma unroll
    for (int j0 = 0; j0 < NV; j0 += B) {
#pragma unroll
        for (int j = 0; j < B; j++) raw[j] = src[min(lane + kWave * (j0 + j), chunks - 1)];
#pragma unroll
        for (int j = 0; j < B; j++) {
            x.from(raw[j]);
            m = max(m, x.top());
        }
    }
    const RowScale r(wave_top(m));
    if (lane == 0) *scale = r.scale;
#pragma unroll
    for (int j0 = 0; j0 < NV; j0 += B) {
        if constexpr (NV > B) {
#pragma unroll
            for (int j = 0; j < B; j++) raw[j] = src[min(lane + kWave * (j0 + j), chunks - 1)];
        }
#pragma unroll
        for (int j = 0; j < B; j++) {
            const int c = lane + kWave * (j0 + j);
            x.from(raw[j]);
            if (c < chunks) store_codes(x, r, dst + static_cast<size_t>(c) * per);
        }
    }
    for (size_t c = static_cast<size_t>(chunks) * per + 4 * lane; c < ldq; c += 4 * kWave)
        *reinterpret_cast<uint32_t *>(dst + c) = 0u;
}

}  // namespace occ
