// Backward pass of the gate projection logits = x W_r^T:
//   dx = dx_in + dlogits W_r  (contracts the Ne experts),
//   dW_r = dlogits^T x        (contracts the T tokens).
//
// Ne <= 256 against d in the thousands: both products move far more bytes
// than they need matrix cycles, so each kernel is built around one pass over
// its T x d tensors (dx_in and dx; x) and keeps the small operand on chip.
//
// bf16: v_mfma_f32_16x16x32_bf16.  dlogits are fp32 and enter as a sum of
// bf16 terms, each the rounding of what the ones before it leave: two terms
// (16 bits, far below the bf16 rounding of dx) in dx, three (all 24 bits of
// an fp32 value) in dW_r, whose outputs are fp32.
//   k_gate_dx   a wave owns 64 columns and keeps W_r's fragments for them in
//               registers (Ne x 64) while it walks over 16-token tiles.  The
//               product is issued transposed and column m of fragment ni is
//               mapped to 16 (m / 4) + 4 ni + m mod 4, so that a lane ends
//               with 16 consecutive columns of one token: two 16-byte loads
//               of dx_in and stores of dx.
//   k_gate_dw   a wave owns 128 columns and up to 64 experts and walks over
//               tokens 32 at a time.  MFMA wants 8 consecutive tokens of one
//               column per lane, x holds columns consecutively: each lane
//               loads 16 bytes (8 columns) of its 8 tokens and transposes the
//               8 x 8 block in registers (32 byte permutes), which yields the
//               fragments of 8 column sets (column 8 i + q in fragment q).  No
//               LDS, every x value is loaded once.  The tokens are split over
//               the 4 waves of a workgroup, added through LDS, and over
//               workgroups, whose partial sums a second kernel adds in order.
// fp32: v_mfma_f32_16x16x4_f32 on the operands as they lie (one value per
// lane and step), exact products.
#include <algorithm>

#include "launch.h"

namespace occ {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kDxCols = 64;    // columns of a wave in k_gate_dx
constexpr int kDwCols = 128;   // columns of a workgroup in k_gate_dw (bf16)
constexpr int kDwColsF = 64;   // (fp32)
constexpr int kDwExperts = 64; // experts of a workgroup in k_gate_dw

// v as bf16 terms, most significant first, four values' bits side by side.
template <int TERMS>
__device__ __forceinline__ void split_terms(const float (&v)[8], bf16x8_t (&out)[TERMS]) {
    float rest[8];
#pragma unroll
    for (int j = 0; j < 8; j++) rest[j] = v[j];
#pragma unroll
    for (int q = 0; q < TERMS; q++)
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const __bf16 b = static_cast<__bf16>(rest[j]);
            out[q][j] = b;
            if (q + 1 < TERMS) rest[j] -= static_cast<float>(b);
        }
}

// Eight consecutive values row[k .. k+7] of a row of n, zeros behind n.
template <bool VEC>
__device__ __forceinline__ void load8(const float *__restrict__ row, int k, int n, float (&v)[8]) {
    if constexpr (VEC) {  // n % 4 == 0, 16-byte aligned rows
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const bool in = k + 4 * h < n;
            const f32x4 x = in ? *reinterpret_cast<const f32x4 *>(row + k + 4 * h)
                               : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; j++) v[4 * h + j] = x[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = k + j < n ? row[k + j] : 0.f;
    }
}

// KS: 32-deep steps over the experts.  Waves are independent (no barrier).
template <int KS, bool VEC>
__global__ __launch_bounds__(kThreads) void k_gate_dx(const float *__restrict__ dl,
                                                      const uint16_t *__restrict__ wr,
                                                      const uint16_t *dx_in, uint16_t *dx, int T,
                                                      int d, int Ne) {
    const int l = lane_id(), i16 = l & 15, G = l >> 4;
    const int c0 = (blockIdx.x * kWaves + threadIdx.x / kWave) * kDxCols;
    if (c0 >= d) return;  // d is a multiple of kDxCols
    bf16x8_t w[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int ni = 0; ni < 4; ni++) {
            const int c = c0 + 16 * (i16 >> 2) + 4 * ni + (i16 & 3);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int e = 32 * ks + 8 * G + j;
                const uint16_t b = e < Ne ? wr[static_cast<size_t>(e) * d + c] : uint16_t{0};
                w[ks][ni][j] = __builtin_bit_cast(__bf16, b);
            }
        }
    const int tiles = (T + 15) / 16;
    for (int tile = blockIdx.y; tile < tiles; tile += gridDim.y) {
        const int t = tile * 16 + i16;
        const float *row = dl + static_cast<size_t>(min(t, T - 1)) * Ne;
        f32x4 acc[4];
#pragma unroll
        for (int ni = 0; ni < 4; ni++) acc[ni] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
            float v[8];
            load8<VEC>(row, 32 * ks + 8 * G, Ne, v);
            bf16x8_t a[2];
            split_terms<2>(v, a);
#pragma unroll
            for (int q = 0; q < 2; q++)
#pragma unroll
                for (int ni = 0; ni < 4; ni++)
                    acc[ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[ks][ni], a[q], acc[ni], 0, 0, 0);
        }
        // lane: token t, columns c0 + 16 G + 4 ni + v
        if (t >= T) continue;
        const size_t at = static_cast<size_t>(t) * d + c0 + 16 * G;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            u32x4 in = {0, 0, 0, 0}, out;
            if (dx_in) in = *reinterpret_cast<const u32x4 *>(dx_in + at + 8 * h);
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const f32x4 &s = acc[2 * h + (q >> 1)];
                const float lo = s[2 * (q & 1)] + __uint_as_float(in[q] << 16);
                const float hi = s[2 * (q & 1) + 1] + __uint_as_float(in[q] & 0xffff0000u);
                out[q] = static_cast<uint32_t>(f32_to_bf16_bits(lo)) |
                         static_cast<uint32_t>(f32_to_bf16_bits(hi)) << 16;
            }
            *reinterpret_cast<u32x4 *>(dx + at + 8 * h) = out;
        }
    }
}

// MB: 16-expert blocks of the workgroup.  part: [token share][Ne][d].
template <int MB>
__global__ __launch_bounds__(kThreads) void k_gate_dw(const float *__restrict__ dl,
                                                      const uint16_t *__restrict__ x, int T, int d,
                                                      int Ne, int per_share,
                                                      float *__restrict__ part) {
    __shared__ f32x4 s_acc[kWaves / 2][MB * 8][kWave];
    const int l = lane_id(), i16 = l & 15, G = l >> 4, wv = threadIdx.x / kWave;
    const int c0 = blockIdx.x * kDwCols, e0 = blockIdx.y * kDwExperts;
    const bool col_in = c0 + 8 * i16 < d;  // d is a multiple of 64
    const int t0 = blockIdx.z * per_share, t1 = min(T, t0 + per_share);
    f32x4 acc[MB][8];
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int q = 0; q < 8; q++) acc[m][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int t = t0 + 32 * wv; t < t1; t += 32 * kWaves) {
        const int tl = t + 8 * G;  // this lane's 8 tokens
        u32x4 row[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            // tokens behind the share meet zero dlogits below; their x is zero
            // too, since 0 times a NaN read past the end would not be 0
            row[j] = u32x4{0, 0, 0, 0};
            if (tl + j < t1 && col_in)
                row[j] = *reinterpret_cast<const u32x4 *>(x + static_cast<size_t>(tl + j) * d + c0 +
                                                          8 * i16);
        }
        bf16x8_t b[8];
#pragma unroll
        for (int q = 0; q < 8; q++) {
            u32x4 f;
#pragma unroll
            for (int j = 0; j < 4; j++)
                f[j] = __builtin_amdgcn_perm(row[2 * j + 1][q >> 1], row[2 * j][q >> 1],
                                             q & 1 ? 0x07060302u : 0x05040100u);
            b[q] = __builtin_bit_cast(bf16x8_t, f);
        }
#pragma unroll
        for (int m = 0; m < MB; m++) {
            const int e = e0 + 16 * m + i16;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                v[j] = tl + j < t1 && e < Ne ? dl[static_cast<size_t>(tl + j) * Ne + e] : 0.f;
            bf16x8_t a[3];
            split_terms<3>(v, a);
#pragma unroll
            for (int q = 0; q < 8; q++)
#pragma unroll
                for (int s = 2; s >= 0; s--)
                    acc[m][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[s], b[q], acc[m][q], 0, 0, 0);
        }
    }
    // waves 2 and 3 into 0 and 1, then 1 into 0
#pragma unroll
    for (int half = kWaves / 2; half > 0; half >>= 1) {
        if (wv >= half && wv < 2 * half)
#pragma unroll
            for (int m = 0; m < MB; m++)
#pragma unroll
                for (int q = 0; q < 8; q++) s_acc[wv - half][m * 8 + q][l] = acc[m][q];
        __syncthreads();
        if (wv < half)
#pragma unroll
            for (int m = 0; m < MB; m++)
#pragma unroll
                for (int q = 0; q < 8; q++) acc[m][q] += s_acc[wv][m * 8 + q][l];
        __syncthreads();
    }
    if (wv || !col_in) return;
    // lane: experts e0 + 16 m + 4 G + v, columns c0 + 8 i16 + q
    float *out = part + static_cast<size_t>(blockIdx.z) * Ne * d;
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int v = 0; v < 4; v++) {
            const int e = e0 + 16 * m + 4 * G + v;
            if (e >= Ne) continue;
            float *o = out + static_cast<size_t>(e) * d + c0 + 8 * i16;
            *reinterpret_cast<f32x4 *>(o) = f32x4{acc[m][0][v], acc[m][1][v], acc[m][2][v], acc[m][3][v]};
            *reinterpret_cast<f32x4 *>(o + 4) =
                f32x4{acc[m][4][v], acc[m][5][v], acc[m][6][v], acc[m][7][v]};
        }
}

// fp32: a wave makes 64 tokens x 64 columns of dx, contracting 4 experts per
// step; the product is transposed and its columns mapped as in k_gate_dx.
__global__ __launch_bounds__(kThreads) void k_gate_dx_f32(const float *__restrict__ dl,
                                                          const float *__restrict__ wr,
                                                          const float *dx_in, float *dx, int T,
                                                          int d, int Ne) {
    const int l = lane_id(), i16 = l & 15, G = l >> 4;
    const int c0 = (blockIdx.x * kWaves + threadIdx.x / kWave) * kDxCols;
    if (c0 >= d) return;
    for (int t0 = blockIdx.y * 64; t0 < T; t0 += gridDim.y * 64) {
        f32x4 acc[4][4];  // [token block][ni]
#pragma unroll
        for (int m = 0; m < 4; m++)
#pragma unroll
            for (int ni = 0; ni < 4; ni++) acc[m][ni] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int e0 = 0; e0 < Ne; e0 += 4) {
            const int e = e0 + G;
            float a[4], w[4];
#pragma unroll
            for (int m = 0; m < 4; m++)
                a[m] = e < Ne ? dl[static_cast<size_t>(min(t0 + 16 * m + i16, T - 1)) * Ne + e] : 0.f;
#pragma unroll
            for (int ni = 0; ni < 4; ni++) {
                const int c = c0 + 16 * (i16 >> 2) + 4 * ni + (i16 & 3);
                w[ni] = e < Ne && c < d ? wr[static_cast<size_t>(e) * d + c] : 0.f;
            }
#pragma unroll
            for (int m = 0; m < 4; m++)
#pragma unroll
                for (int ni = 0; ni < 4; ni++)
                    acc[m][ni] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[ni], a[m], acc[m][ni], 0, 0, 0);
        }
        if (c0 + 16 * G >= d) continue;  // d is a multiple of 16
#pragma unroll
        for (int m = 0; m < 4; m++) {
            const int t = t0 + 16 * m + i16;
            if (t >= T) continue;
            const size_t at = static_cast<size_t>(t) * d + c0 + 16 * G;
#pragma unroll
            for (int ni = 0; ni < 4; ni++) {
                f32x4 v = acc[m][ni];
                if (dx_in) v += *reinterpret_cast<const f32x4 *>(dx_in + at + 4 * ni);
                *reinterpret_cast<f32x4 *>(dx + at + 4 * ni) = v;
            }
        }
    }
}

// fp32: a wave makes 64 experts x 64 columns of dW_r from a quarter of the
// workgroup's tokens, 8 at a time.
__global__ __launch_bounds__(kThreads) void k_gate_dw_f32(const float *__restrict__ dl,
                                                          const float *__restrict__ x, int T, int d,
                                                          int Ne, int per_share,
                                                          float *__restrict__ part) {
    __shared__ f32x4 s_acc[kWaves / 2][16][kWave];
    const int l = lane_id(), i16 = l & 15, G = l >> 4, wv = threadIdx.x / kWave;
    const int c0 = blockIdx.x * kDwColsF, e0 = blockIdx.y * kDwExperts;
    const int t0 = blockIdx.z * per_share, t1 = min(T, t0 + per_share);
    f32x4 acc[4][4];  // [expert block][column block]
#pragma unroll
    for (int m = 0; m < 4; m++)
#pragma unroll
        for (int q = 0; q < 4; q++) acc[m][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    // two steps of 4 tokens at a time, their loads first
    for (int tt = t0 + 8 * wv; tt < t1; tt += 8 * kWaves) {
        float a[2][4], b[2][4];
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const int t = tt + 4 * u + G;
#pragma unroll
            for (int m = 0; m < 4; m++) {
                const int e = e0 + 16 * m + i16;
                a[u][m] = t < t1 && e < Ne ? dl[static_cast<size_t>(t) * Ne + e] : 0.f;
            }
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int c = c0 + 16 * q + i16;
                b[u][q] = t < t1 && c < d ? x[static_cast<size_t>(t) * d + c] : 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int m = 0; m < 4; m++)
#pragma unroll
                for (int q = 0; q < 4; q++)
                    acc[m][q] =
                        __builtin_amdgcn_mfma_f32_16x16x4f32(a[u][m], b[u][q], acc[m][q], 0, 0, 0);
    }
#pragma unroll
    for (int half = kWaves / 2; half > 0; half >>= 1) {
        if (wv >= half && wv < 2 * half)
#pragma unroll
            for (int m = 0; m < 4; m++)
#pragma unroll
                for (int q = 0; q < 4; q++) s_acc[wv - half][m * 4 + q][l] = acc[m][q];
        __syncthreads();
        if (wv < half)
#pragma unroll
            for (int m = 0; m < 4; m++)
#pragma unroll
                for (int q = 0; q < 4; q++) acc[m][q] += s_acc[wv][m * 4 + q][l];
        __syncthreads();
    }
    if (wv) return;
    float *out = part + static_cast<size_t>(blockIdx.z) * Ne * d;
#pragma unroll
    for (int m = 0; m < 4; m++)
#pragma unroll
        for (int v = 0; v < 4; v++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int e = e0 + 16 * m + 4 * G + v, c = c0 + 16 * q + i16;
                if (e < Ne && c < d) out[static_cast<size_t>(e) * d + c] = acc[m][q][v];
            }
}

// dw = the token shares' sums in order.
__global__ __launch_bounds__(kThreads) void k_gate_dw_fold(const f32x4 *__restrict__ part,
                                                           int shares, size_t n4,
                                                           f32x4 *__restrict__ dw) {
    const size_t i = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= n4) return;
    f32x4 s = part[i];
    for (int q = 1; q < shares; q++) s += part[q * n4 + i];
    dw[i] = s;
}

}  // namespace

// Token shares of dW_r: enough workgroups for two per CU, each share at
// least 256 tokens (its sums cost Ne x d fp32 written and read).  From the
// shape alone, so that sums do not depend on the device's state.
int gate_dw_shares(int T, int d, int Ne, int bf16) {
    const int cols = static_cast<int>(ceil_div(d, bf16 ? kDwCols : kDwColsF));
    const int groups = cols * static_cast<int>(ceil_div(Ne, kDwExperts));
    const int want = static_cast<int>(ceil_div(512, groups));
    const int most = static_cast<int>(ceil_div(T, 256));
    return want < most ? want : most;
}

hipError_t launch_gate_dx(const float *dl, const void *w_router, const void *dx_in, int T, int d,
                          int Ne, int bf16, void *dx, hipStream_t s) {
    const unsigned cols = ceil_div(d, kWaves * kDxCols);
    if (!bf16) {
        k_gate_dx_f32<<<dim3(cols, std::min(ceil_div(T, 64), 4096u)), kThreads, 0, s>>>(
            dl, static_cast<const float *>(w_router), static_cast<const float *>(dx_in),
            static_cast<float *>(dx), T, d, Ne);
        return hipGetLastError();
    }
    // waves walk over enough token tiles to pay for their W_r fragments
    const unsigned tiles = ceil_div(T, 16);
    const unsigned rows = std::min(ceil_div(2048, cols), tiles);
    const bool vec = Ne % 4 == 0 && reinterpret_cast<uintptr_t>(dl) % 16 == 0;
#define OCC_GATE_DX(KS)                                                                        \
    do {                                                                                       \
        const auto *w = static_cast<const uint16_t *>(w_router);                               \
        const auto *in = static_cast<const uint16_t *>(dx_in);                                 \
        auto *out = static_cast<uint16_t *>(dx);                                               \
        if (vec)                                                                               \
            k_gate_dx<KS, true><<<dim3(cols, rows), kThreads, 0, s>>>(dl, w, in, out, T, d, Ne);  \
        else                                                                                   \
            k_gate_dx<KS, false><<<dim3(cols, rows), kThreads, 0, s>>>(dl, w, in, out, T, d, Ne); \
    } while (0)
    if (Ne <= 32)
        OCC_GATE_DX(1);
    else if (Ne <= 64)
        OCC_GATE_DX(2);
    else if (Ne <= 128)
        OCC_GATE_DX(4);
    else
        OCC_GATE_DX(8);
#undef OCC_GATE_DX
    return hipGetLastError();
}

hipError_t launch_gate_dw(const float *dl, const void *x, int T, int d, int Ne, int bf16,
                          float *part, float *dw, hipStream_t s) {
    const int shares = gate_dw_shares(T, d, Ne, bf16);
    // whole 32-token steps of the 4 waves; a share may then be empty, and sums to zero
    const int per = static_cast<int>(ceil_div(ceil_div(T, shares), 128) * 128);
    const unsigned eg = ceil_div(Ne, kDwExperts);
    if (bf16) {
        const dim3 grid(ceil_div(d, kDwCols), eg, shares);
        const auto *xb = static_cast<const uint16_t *>(x);
        if (Ne <= 16)
            k_gate_dw<1><<<grid, kThreads, 0, s>>>(dl, xb, T, d, Ne, per, part);
        else if (Ne <= 32)
            k_gate_dw<2><<<grid, kThreads, 0, s>>>(dl, xb, T, d, Ne, per, part);
        else
            k_gate_dw<4><<<grid, kThreads, 0, s>>>(dl, xb, T, d, Ne, per, part);
    } else {
        k_gate_dw_f32<<<dim3(ceil_div(d, kDwColsF), eg, shares), kThreads, 0, s>>>(
            dl, static_cast<const float *>(x), T, d, Ne, per, part);
    }
    const size_t n4 = static_cast<size_t>(Ne) * d / 4;
    k_gate_dw_fold<<<ceil_div(n4, kThreads), kThreads, 0, s>>>(
        reinterpret_cast<const f32x4 *>(part), shares, n4, reinterpret_cast<f32x4 *>(dw));
    return hipGetLastError();
}

}  // namespace occ
