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
//   k_gate_dx   a wave owns 128 columns, keeps W_r's fragments for them in
//               registers (Ne x 128, transposed there once) and walks over
//               16-token tiles.  Column 8 i + ni is column i of fragment ni,
//               so that a lane ends with 8 consecutive columns of four tokens
//               and 16 lanes move 256 bytes of a row at once (in 64-byte
//               pieces: 118 us at T = 65536, d = 2048, Ne = 60 against 95).
//   k_gate_dw   a workgroup owns 256 columns, 64 experts and a share of the
//               tokens, 64 per step.  MFMA wants 8 consecutive tokens of one
//               column per lane, x holds columns consecutively: each lane
//               loads 4 columns of its 8 tokens and transposes them in
//               registers (16 byte permutes), no LDS, every x value loaded
//               once.  The step's dlogits are split once for all waves, a
//               quarter of a half step by each, and passed through LDS as
//               fragments, while the step before is multiplied.  The two
//               halves are added at the end, and the shares by a second
//               kernel in order.
// Measured at d = 2048, Ne = 60, T = 65536: dW_r 75 us + 6 for the shares, dx
// 95 us (5.8 TB/s of 553 MB), 174 us as one call (4.7 TB/s of its 822 MB; one
// bf16 term in place of three leaves the call as it is: the memory bounds
// it); Ne = 64, T = 8192: 17 + 4.5 and 17 us.
// fp32: v_mfma_f32_16x16x4_f32 on the operands as they lie (one value per
// lane and step), exact products.
#include <algorithm>

#include "launch.h"

namespace occ {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kDxCols = 64;     // columns of a wave in k_gate_dx_f32
constexpr int kDwThreads = 512; // k_gate_dw
constexpr int kDwCols = 256;    // columns of a workgroup in k_gate_dw
constexpr int kDwColsF = 64;    // in k_gate_dw_f32
constexpr int kDwExperts = 64;  // experts of a workgroup in either

// Workgroup b runs on XCD b mod 8, each with an L2 of its own.  A token range
// meets every column group, so its groups get numbers that share an XCD: the
// range's dlogits are fetched into one L2 instead of eight.
__device__ __forceinline__ void share_of(int groups, int &group, unsigned &share) {
    const unsigned r = blockIdx.x >> 3;
    group = static_cast<int>(r % groups);
    share = r / groups * 8 + (blockIdx.x & 7);
}
unsigned share_grid(int groups, unsigned shares) { return groups * ceil_div(shares, 8) * 8; }

// Two values as bf16, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __attribute__((ext_vector_type(2))) float f32x2;
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ float low_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// v as bf16 terms, most significant first.
template <int TERMS>
__device__ __forceinline__ void split_terms(const float (&v)[8], bf16x8_t (&out)[TERMS]) {
    float rest[8];
#pragma unroll
    for (int j = 0; j < 8; j++) rest[j] = v[j];
#pragma unroll
    for (int q = 0; q < TERMS; q++) {
        u32x4 pk;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            pk[j] = pack_bf16(rest[2 * j], rest[2 * j + 1]);
            rest[2 * j] -= low_bf16(pk[j]);
            rest[2 * j + 1] -= high_bf16(pk[j]);
        }
        out[q] = __builtin_bit_cast(bf16x8_t, pk);
    }
}

// The loops load ahead of their use, from a base that the whole wave shares
// (scalar arithmetic) and 32-bit lane offsets that stay the same from step to
// step.  These loads are unconditional -- behind a load under a condition the
// wait for an older one has to wait for both -- so a step that would reach
// past the last token starts early enough not to, and the tokens that it then
// repeats are left out afterwards; with fewer tokens than a step has, the
// last one is repeated.
template <typename V>
__device__ __forceinline__ V load_at(const void *base, unsigned offset) {
    return *reinterpret_cast<const V *>(static_cast<const char *>(base) + offset);
}

// Eight rows of NI consecutive bf16 values (row j in r[j]) transposed: value q
// of all rows in out[q].
template <int NI, typename V>
__device__ __forceinline__ void transpose8(const V (&r)[8], bf16x8_t (&out)[NI]) {
#pragma unroll
    for (int q = 0; q < NI; q++) {
        u32x4 f;
#pragma unroll
        for (int j = 0; j < 4; j++)
            f[j] = __builtin_amdgcn_perm(r[2 * j + 1][q >> 1], r[2 * j][q >> 1],
                                         q & 1 ? 0x07060302u : 0x05040100u);
        out[q] = __builtin_bit_cast(bf16x8_t, f);
    }
}

// KS: 32-deep steps over the experts; NI: 16-column fragments of a wave, 8 or
// 4.  Waves are independent (no barrier).
template <int KS, int NI, bool VEC>
__global__ __launch_bounds__(kThreads) void k_gate_dx(const float *__restrict__ dl,
                                                      const uint16_t *__restrict__ wr,
                                                      const uint16_t *dx_in, uint16_t *dx,
                                                      unsigned T, int d, int Ne, int groups,
                                                      unsigned shares) {
    typedef __attribute__((ext_vector_type(NI / 2))) unsigned int Cols;  // NI columns
    const int l = lane_id(), i16 = l & 15, G = l >> 4;
    int group;
    unsigned tile;
    share_of(groups, group, tile);
    const int c0 = (group * kWaves + threadIdx.x / kWave) * (16 * NI);
    if (c0 >= d || tile >= shares) return;
    bf16x8_t w[KS][NI];
    // column i of fragment ni is NI i + ni
    const int cw = c0 + NI * i16;
#pragma unroll
    for (int ks = 0; ks < KS; ks++) {
        Cols r[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int e = 32 * ks + 8 * G + j;
            r[j] = e < Ne && cw < d
                       ? *reinterpret_cast<const Cols *>(wr + static_cast<size_t>(e) * d + cw)
                       : Cols{};
        }
        transpose8<NI>(r, w[ks]);
    }
    // the next tile's dlogits and dx_in, loaded while this one is multiplied;
    // lane offsets: this lane's token of a tile and its experts or columns
    const unsigned tiles = (T + 15) / 16, rows = min(T, 16u), last = T - rows;
    const unsigned r = min(static_cast<unsigned>(i16), rows - 1);  // dlogits' token
    constexpr int kPieces = VEC ? 2 : 8;  // of 4 values or 1
    unsigned at_e[KS][kPieces], at_c[4];
#pragma unroll
    for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int j = 0; j < kPieces; j++)
            at_e[ks][j] = 4 * (r * Ne + min(32 * ks + 8 * G + 8 / kPieces * j, Ne - 8 / kPieces));
#pragma unroll
    for (int v = 0; v < 4; v++)
        at_c[v] = 2 * (min(static_cast<unsigned>(4 * G + v), rows - 1) * d + min(cw, d - NI));
    float vn[KS][8];
    Cols in[4];
    const uint16_t *from = dx_in ? dx_in : dx;  // not used without dx_in
    auto load = [&](unsigned t) {
        const float *row = dl + static_cast<size_t>(t) * Ne;
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
            for (int j = 0; j < kPieces; j++) {
                if constexpr (VEC) {
                    const f32x4 x = load_at<f32x4>(row, at_e[ks][j]);
#pragma unroll
                    for (int q = 0; q < 4; q++) vn[ks][4 * j + q] = x[q];
                } else {
                    vn[ks][j] = load_at<float>(row, at_e[ks][j]);
                }
            }
#pragma unroll
        for (int v = 0; v < 4; v++) in[v] = load_at<Cols>(from + static_cast<size_t>(t) * d, at_c[v]);
    };
    load(min(tile * 16, last));
    for (; tile < tiles; tile += shares) {
        const unsigned t = min(tile * 16, last);
        f32x4 acc[NI];
#pragma unroll
        for (int v = 0; v < 4; v++)
#pragma unroll
            for (int q = 0; q < NI / 2; q++) {
                acc[2 * q][v] = dx_in ? low_bf16(in[v][q]) : 0.f;
                acc[2 * q + 1][v] = dx_in ? high_bf16(in[v][q]) : 0.f;
            }
        bf16x8_t a[KS][2];
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
            if (32 * ks + 32 > Ne)  // experts behind the last
#pragma unroll
                for (int j = 0; j < 8; j++)
                    vn[ks][j] = 32 * ks + 8 * G + j < Ne ? vn[ks][j] : 0.f;
            split_terms<2>(vn[ks], a[ks]);
        }
        load(min((tile + shares) * 16, last));
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
            for (int q = 0; q < 2; q++)
#pragma unroll
                for (int ni = 0; ni < NI; ni++)
                    acc[ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[ks][q], w[ks][ni], acc[ni], 0, 0, 0);
        // lane: tokens t + 4 G + v, columns cw + ni; tokens of an earlier tile
        // and repeated ones are not stored
        char *to = reinterpret_cast<char *>(dx + static_cast<size_t>(t) * d);
#pragma unroll
        for (int v = 0; v < 4; v++) {
            Cols out;
#pragma unroll
            for (int q = 0; q < NI / 2; q++) out[q] = pack_bf16(acc[2 * q][v], acc[2 * q + 1][v]);
            const unsigned own = t + 4 * G + v;
            if (own >= tile * 16 && own < T && cw < d) *reinterpret_cast<Cols *>(to + at_c[v]) = out;
        }
    }
}

// MB: 16-expert blocks of the workgroup.  part: [token share][Ne][d].  Waves
// 0..3 and 4..7 take the two 32-token halves of a step, wave w the 64 columns
// from 64 (w mod 4).
template <int MB>
__global__ __launch_bounds__(kDwThreads) void k_gate_dw(const float *__restrict__ dl,
                                                        const uint16_t *__restrict__ x, unsigned T,
                                                        int d, int Ne, int groups, unsigned shares,
                                                        unsigned per_share,
                                                        float *__restrict__ part) {
    typedef bf16x8_t Terms[2][2][MB][3][kWave];  // [buffer][half][expert block][term][lane]
    typedef f32x4 Sums[4][MB * 4][kWave];
    __shared__ __attribute__((aligned(16))) char lds[sizeof(Terms) > sizeof(Sums) ? sizeof(Terms) : sizeof(Sums)];
    Terms &s_a = *reinterpret_cast<Terms *>(lds);
    Sums &s_sum = *reinterpret_cast<Sums *>(lds);
    const int l = lane_id(), i16 = l & 15, G = l >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), half = wv >> 2, cg = wv & 3;
    int group;
    unsigned share;
    share_of(groups, group, share);
    if (share >= shares) return;
    const int c0 = group * kDwCols + 64 * cg, e0 = blockIdx.y * kDwExperts;
    const bool col_in = c0 < d;  // d is a multiple of 64
    const unsigned t0 = share * per_share, t1 = min(T, t0 + per_share);
    f32x4 acc[MB][4];
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int q = 0; q < 4; q++) acc[m][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    // Step n's 8 tokens of this lane: 4 columns of x, and the dlogits of one
    // expert (behind Ne the last one's again, whose sums are not stored)
    typedef __attribute__((ext_vector_type(2))) unsigned int u32x2;
    const unsigned rows = min(T, 64u), last = T - rows;
    unsigned at_x[8], at_e[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const unsigned r = min(static_cast<unsigned>(32 * half + 8 * G + j), rows - 1);
        at_x[j] = 2 * (r * d + min(c0, d - 64) + 4 * i16);
        at_e[j] = 4 * (r * Ne + min(e0 + 16 * cg + i16, Ne - 1));
    }
    u32x2 row[2][8];
    float v[2][8];
    auto load_x = [&](unsigned t, u32x2(&r)[8]) {
        const uint16_t *from = x + static_cast<size_t>(min(t, last)) * d;
#pragma unroll
        for (int j = 0; j < 8; j++) r[j] = load_at<u32x2>(from, at_x[j]);
    };
    auto load_dl = [&](unsigned t, float(&o)[8]) {
        const float *from = dl + static_cast<size_t>(min(t, last)) * Ne;
#pragma unroll
        for (int j = 0; j < 8; j++) o[j] = load_at<float>(from, at_e[j]);
    };
    auto split = [&](unsigned t, float(&o)[8], int buf) {
        if (cg >= MB) return;
        if (t + 64 > t1) {  // tokens before the step, behind the share, or repeated count nothing
            const unsigned first = min(t, last);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const unsigned r = 32 * half + 8 * G + j, own = first + r;
                o[j] = own >= t && own < t1 && r < rows ? o[j] : 0.f;
            }
        }
        bf16x8_t terms[3];
        split_terms<3>(o, terms);
#pragma unroll
        for (int s = 0; s < 3; s++) s_a[buf][half][cg][s][l] = terms[s];
    };
    load_dl(t0, v[0]);
    load_x(t0, row[0]);
    load_dl(t0 + 64, v[1]);
    load_x(t0 + 64, row[1]);
    split(t0, v[0], 0);
    load_dl(t0 + 128, v[0]);
    __syncthreads();
    // Step n multiplies from buffer n mod 2 while the next step's dlogits are
    // split into the other one, whose readers have passed the barrier.
    for (unsigned t = t0; t < t1; t += 128) {
#pragma unroll
        for (int u = 0; u < 2; u++) {  // the second step may lie behind the share: zeros
            bf16x8_t b[4];
            transpose8<4>(row[u], b);
            load_x(t + 64 * u + 128, row[u]);
            split(t + 64 * u + 64, v[u ^ 1], u ^ 1);
            load_dl(t + 64 * u + 192, v[u ^ 1]);
            // (without columns of its own a wave multiplies the last ones' and stores nothing)
#pragma unroll
            for (int m = 0; m < MB; m++)
#pragma unroll
                for (int s = 2; s >= 0; s--) {
                    const bf16x8_t a = s_a[u][half][m][s][l];
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        acc[m][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[q], acc[m][q], 0, 0, 0);
                }
            __syncthreads();
        }
    }
    // the second half's sums into the first's
    if (half)
#pragma unroll
        for (int m = 0; m < MB; m++)
#pragma unroll
            for (int q = 0; q < 4; q++) s_sum[cg][m * 4 + q][l] = acc[m][q];
    __syncthreads();
    if (half || !col_in) return;
    // lane: experts e0 + 16 m + 4 G + v, columns c0 + 4 i16 + q
    float *out = part + static_cast<size_t>(share) * Ne * d;
#pragma unroll
    for (int m = 0; m < MB; m++) {
#pragma unroll
        for (int q = 0; q < 4; q++) acc[m][q] += s_sum[cg][m * 4 + q][l];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int er = e0 + 16 * m + 4 * G + i;
            if (er < Ne)
                *reinterpret_cast<f32x4 *>(out + static_cast<size_t>(er) * d + c0 + 4 * i16) =
                    f32x4{acc[m][0][i], acc[m][1][i], acc[m][2][i], acc[m][3][i]};
        }
    }
}

// fp32: a wave makes 64 tokens x 64 columns of dx, contracting 4 experts per
// step; the product is transposed and its columns mapped as in k_gate_dx.
__global__ __launch_bounds__(kThreads) void k_gate_dx_f32(const float *__restrict__ dl,
                                                          const float *__restrict__ wr,
                                                          const float *dx_in, float *dx,
                                                          unsigned T, int d, int Ne) {
    const int l = lane_id(), i16 = l & 15, G = l >> 4;
    const int c0 = (blockIdx.x * kWaves + threadIdx.x / kWave) * kDxCols;
    if (c0 >= d) return;
    for (unsigned t0 = blockIdx.y * 64; t0 < T; t0 += gridDim.y * 64) {
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
            const unsigned t = t0 + 16 * m + i16;
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
                                                          const float *__restrict__ x, unsigned T,
                                                          int d, int Ne, unsigned per_share,
                                                          float *__restrict__ part) {
    __shared__ f32x4 s_acc[kWaves / 2][16][kWave];
    const int l = lane_id(), i16 = l & 15, G = l >> 4, wv = threadIdx.x / kWave;
    const int c0 = blockIdx.x * kDwColsF, e0 = blockIdx.y * kDwExperts;
    const unsigned t0 = blockIdx.z * per_share, t1 = min(T, t0 + per_share);
    f32x4 acc[4][4];  // [expert block][column block]
#pragma unroll
    for (int m = 0; m < 4; m++)
#pragma unroll
        for (int q = 0; q < 4; q++) acc[m][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    // two steps of 4 tokens at a time, their loads first
    for (unsigned tt = t0 + 8 * wv; tt < t1; tt += 8 * kWaves) {
        float a[2][4], b[2][4];
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const unsigned t = tt + 4 * u + G;
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

// dw = the sum of the token shares' partial sums: thread (i, q) adds shares q,
// q + 4, ..., then the four are added in order.
constexpr int kFoldOut = kThreads / 4;
__global__ __launch_bounds__(kThreads) void k_gate_dw_fold(const f32x4 *__restrict__ part,
                                                           int shares, size_t n4,
                                                           f32x4 *__restrict__ dw) {
    __shared__ f32x4 s_sum[4][kFoldOut];
    const int o = threadIdx.x % kFoldOut, q = threadIdx.x / kFoldOut;
    const size_t i = static_cast<size_t>(blockIdx.x) * kFoldOut + o;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (i < n4)
#pragma unroll 8
        for (int t = q; t < shares; t += 4) s += part[t * n4 + i];
    s_sum[q][o] = s;
    __syncthreads();
    if (q || i >= n4) return;
#pragma unroll
    for (int r = 1; r < 4; r++) s += s_sum[r][o];
    dw[i] = s;
}

}  // namespace

// Token shares of dW_r, from the shape alone, so that sums do not depend on
// the device's state: enough for one workgroup per CU, of one step each at
// least (64 tokens, 32 in fp32).  A share costs Ne x d fp32 written and read.
int gate_dw_shares(int T, int d, int Ne, int bf16) {
    const unsigned cols = ceil_div(d, bf16 ? kDwCols : kDwColsF);
    const unsigned want = ceil_div(256, cols * ceil_div(Ne, kDwExperts));
    return static_cast<int>(std::min(want, ceil_div(T, bf16 ? 64 : 32)));
}

hipError_t launch_gate_dx(const float *dl, const void *w_router, const void *dx_in, int T, int d,
                          int Ne, int bf16, void *dx, hipStream_t s) {
    if (!bf16) {
        k_gate_dx_f32<<<dim3(ceil_div(d, kWaves * kDxCols), std::min(ceil_div(T, 64), 4096u)), kThreads,
                        0, s>>>(dl, static_cast<const float *>(w_router),
                                static_cast<const float *>(dx_in), static_cast<float *>(dx), T, d, Ne);
        return hipGetLastError();
    }
    const bool vec = Ne % 4 == 0 && reinterpret_cast<uintptr_t>(dl) % 16 == 0;
    auto run = [&](auto ks, auto ni) {
        constexpr int KS = decltype(ks)::value, NI = decltype(ni)::value;
        // waves walk over enough token tiles to pay for their W_r fragments
        const unsigned cols = ceil_div(d, kWaves * 16 * NI);
        const unsigned shares = std::min(ceil_div(512, cols), ceil_div(T, 16));
        const unsigned grid = share_grid(cols, shares);
        const auto *w = static_cast<const uint16_t *>(w_router);
        const auto *in = static_cast<const uint16_t *>(dx_in);
        auto *out = static_cast<uint16_t *>(dx);
        if (vec)
            k_gate_dx<KS, NI, true><<<grid, kThreads, 0, s>>>(dl, w, in, out, T, d, Ne, cols, shares);
        else
            k_gate_dx<KS, NI, false><<<grid, kThreads, 0, s>>>(dl, w, in, out, T, d, Ne, cols, shares);
    };
    using std::integral_constant;
    if (Ne <= 32)
        run(integral_constant<int, 1>{}, integral_constant<int, 8>{});
    else if (Ne <= 64)
        run(integral_constant<int, 2>{}, integral_constant<int, 8>{});
    else if (Ne <= 128)
        run(integral_constant<int, 4>{}, integral_constant<int, 8>{});
    else
        run(integral_constant<int, 8>{}, integral_constant<int, 4>{});
    return hipGetLastError();
}

hipError_t launch_gate_dw(const float *dl, const void *x, int T, int d, int Ne, int bf16,
                          float *part, float *dw, hipStream_t s) {
    const int shares = gate_dw_shares(T, d, Ne, bf16);
    // whole steps; the last shares may then be empty, and sum to zero
    const unsigned step = bf16 ? 64 : 32, per = ceil_div(ceil_div(T, shares), step) * step;
    const unsigned eg = ceil_div(Ne, kDwExperts);
    float *out = shares > 1 ? part : dw;
    if (bf16) {
        const int groups = ceil_div(d, kDwCols);
        const dim3 grid(share_grid(groups, shares), eg);
        const auto *xb = static_cast<const uint16_t *>(x);
        if (Ne <= 16)
            k_gate_dw<1><<<grid, kDwThreads, 0, s>>>(dl, xb, T, d, Ne, groups, shares, per, out);
        else if (Ne <= 32)
            k_gate_dw<2><<<grid, kDwThreads, 0, s>>>(dl, xb, T, d, Ne, groups, shares, per, out);
        else
            k_gate_dw<4><<<grid, kDwThreads, 0, s>>>(dl, xb, T, d, Ne, groups, shares, per, out);
    } else {
        k_gate_dw_f32<<<dim3(ceil_div(d, kDwColsF), eg, shares), kThreads, 0, s>>>(
            dl, static_cast<const float *>(x), T, d, Ne, per, out);
    }
    if (shares > 1) {
        const size_t n4 = static_cast<size_t>(Ne) * d / 4;
        k_gate_dw_fold<<<ceil_div(n4, kFoldOut), kThreads, 0, s>>>(
            reinterpret_cast<const f32x4 *>(part), shares, n4, reinterpret_cast<f32x4 *>(dw));
    }
    return hipGetLastError();
}

}  // namespace occ
