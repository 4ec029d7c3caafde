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
//   gate_dx     a wave owns 128 columns, keeps W_r's fragments for them in
//               registers (up to 64 experts x 128, transposed there once) and
//               walks over 16-token tiles.  Column 8 i + ni is column i of
//               fragment ni, so that a lane ends with 8 consecutive columns of
//               four tokens and 16 lanes move 256 bytes of a row at once (in
//               64-byte pieces: 118 us at T = 65536, d = 2048, Ne = 60
//               against 95).
//   gate_dx_tile  more than 64 experts, through LDS.
//   gate_dw     a workgroup owns 256 columns, 64 experts and a share of the
//               tokens, 64 per step.  MFMA wants 8 consecutive tokens of one
//               column per lane, x holds columns consecutively: each lane
//               loads 4 columns of its 8 tokens and transposes them in
//               registers (16 byte permutes), no LDS, every x value loaded
//               once.  The step's dlogits are split once for all waves, a
//               quarter of a half step by each, and passed through LDS as
//               fragments, while the step before is multiplied.  The two
//               halves are added at the end, and the shares by a second
//               kernel in order.
// fp32: v_mfma_f32_16x16x4_f32, exact products, in gate_dx_tile and gate_dw_f32.
//
// One launch makes both products, each by workgroups of its own, so that one's
// start, its waits and its last workgroups lie under the other's work
// (k_gate_bwd, k_gate_bwd_f32).  Against a launch for each: T = 256, d = 2048,
// 64 experts 10.4 us against 14.6 (bf16), 11.7 against 17.2 (fp32); T = 8192
// 30 against 39, 60 against 65; T = 32768 90 against 96, 202 against 201; 250
// experts in bf16 T = 1024 19 against 28, T = 32768 218 against 209.
// Measured at d = 2048 bf16: Ne = 60, T = 65536 166 us + 5.4 for the shares
// (4.8 TB/s of 822 MB, with one bf16 term in place of three as long: the
// memory bounds it); Ne = 64, T = 8192 24.3 + 4.1 us (3.6 TB/s of 104 MB).
// Above 64 experts the groups of dW_r each load and transpose x again: T = 8192,
// Ne = 65 36 + 4.7 us, 130 56 + 4.8, 250 62 + 4.9 (83 to 105 MB read from HBM
// against 85 at 64: the repeated work bounds them, not HBM).
#include <algorithm>
#include <type_traits>

#include "launch.h"

namespace occ {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2;
typedef f32x4 f32x4_unaligned __attribute__((aligned(4)));  // the hardware takes dword alignment

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kDxCols = 128;    // columns of a wave in gate_dx
constexpr int kBfThreads = 512; // k_gate_bwd
constexpr int kDwCols = 256;    // columns of a workgroup in gate_dw
constexpr int kDwColsF = 64;    // in gate_dw_f32
constexpr int kDwExperts = 64;  // experts of a workgroup in either

// Workgroup b runs on XCD b mod 8, each with an L2 of its own.  A token range
// meets every column group, so its groups get numbers that share an XCD: the
// range's dlogits are fetched into one L2 instead of eight.  Fewer ranges
// than XCDs spread their groups over all of them instead.
__device__ __forceinline__ bool share_of(unsigned block, int groups, unsigned shares, int &group,
                                         unsigned &share) {
    const unsigned r = shares < 8 ? block : block >> 3;
    group = static_cast<int>(r % groups);
    share = shares < 8 ? r / groups : r / groups * 8 + (block & 7);
    return share < shares;
}
unsigned share_grid(int groups, unsigned shares) {
    return groups * (shares < 8 ? shares : ceil_div(shares, 8) * 8);
}

// What the workgroups of one product need.  blocks: how many of a launch are
// its own, whole multiples of the XCDs (0: not computed).
struct DxArgs {
    const void *w_router, *dx_in;
    void *dx;
    int groups;
    unsigned shares;  // or tiles
    unsigned blocks;
};
struct DwArgs {
    const void *x;
    float *out;  // [share][Ne][d]
    int groups, col_groups;
    unsigned shares, per_share, blocks;
};
unsigned whole_xcds(unsigned blocks) { return ceil_div(blocks, 8) * 8; }

// This workgroup's number among those of its product; dx_first: dx's come first.
__device__ __forceinline__ unsigned own_block(const DwArgs &dw, const DxArgs &dx, bool dx_first,
                                              bool &is_dw) {
    const unsigned first = dx_first ? dx.blocks : dw.blocks;
    is_dw = (blockIdx.x < first) != dx_first;
    return blockIdx.x < first ? blockIdx.x : blockIdx.x - first;
}

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

// KS: 32-deep steps over the experts.  Waves are independent (no barrier).
template <int KS, bool VEC>
__device__ __forceinline__ void gate_dx(unsigned block, const float *__restrict__ dl, unsigned T,
                                        int d, int Ne, const DxArgs &A) {
    const auto *__restrict__ wr = static_cast<const uint16_t *>(A.w_router);
    const auto *dx_in = static_cast<const uint16_t *>(A.dx_in);
    auto *dx = static_cast<uint16_t *>(A.dx);
    const int groups = A.groups;
    const unsigned shares = A.shares;
    constexpr int NI = kDxCols / 16;  // 16-column fragments
    typedef u32x4 Cols;               // NI columns
    const int l = lane_id(), i16 = l & 15, G = l >> 4;
    int group;
    unsigned tile;
    if (!share_of(block, groups, shares, group, tile)) return;
    const int c0 = (group * (blockDim.x / kWave) + threadIdx.x / kWave) * (16 * NI);
    if (c0 >= d) return;
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
struct DwLds {
    typedef bf16x8_t Terms[2][2][MB][3][kWave];  // [buffer][half][expert block][term][lane]
    typedef f32x4 Sums[4][MB * 4][kWave];
    static constexpr size_t kBytes = std::max(sizeof(Terms), sizeof(Sums));
};
template <int MB>
__device__ __forceinline__ void gate_dw(unsigned block, const float *__restrict__ dl, unsigned T,
                                        int d, int Ne, const DwArgs &A, char *lds) {
    typedef typename DwLds<MB>::Terms Terms;
    typedef typename DwLds<MB>::Sums Sums;
    const auto *__restrict__ x = static_cast<const uint16_t *>(A.x);
    float *__restrict__ part = A.out;
    const int col_groups = A.col_groups;
    Terms &s_a = *reinterpret_cast<Terms *>(lds);
    Sums &s_sum = *reinterpret_cast<Sums *>(lds);
    const int l = lane_id(), i16 = l & 15, G = l >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), half = wv >> 2, cg = wv & 3;
    int group;
    unsigned share;
    if (!share_of(block, A.groups, A.shares, group, share)) return;
    const int c0 = group % col_groups * kDwCols + 64 * cg, e0 = group / col_groups * kDwExperts;
    const bool col_in = c0 < d;  // d is a multiple of 64
    const unsigned t0 = share * A.per_share, t1 = min(T, t0 + A.per_share);
    f32x4 acc[MB][4];
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int q = 0; q < 4; q++) acc[m][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    // Step n's 8 tokens of this lane: 4 columns of x, and the dlogits of one
    // expert (behind Ne the last one's again, whose sums are not stored)
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

// dx for every fp32 shape and for bf16 with more than 64 experts: tiles of
// 32 MB tokens x 64 WN columns by 2 WN waves (32 x 64 to 128 x 256), the
// experts contracted in steps of kDepth through LDS (two buffers; the next
// step's operands are in flight in registers).  Wave (wm, wn) of 2 x WN makes
// 16 MB tokens x 64 columns; column 4 i + ni of those is column i of fragment
// ni, so that a lane ends with 4 consecutive columns.
// bf16: 32 experts a step; dlogits are split into their two terms on the way
// into LDS and W_r's columns transposed in registers, both stored as the
// 16-byte operands (8 consecutive experts) that a lane feeds to the MFMA.
// fp32: 16 experts a step; a lane's operand of MFMA s is expert 4 (lane / 16)
// + s, so that one 16-byte read of a token's dlogits feeds four MFMAs.
template <typename E, int MB, int WN>
struct DxTile;
template <int MB, int WN>
struct DxTile<uint16_t, MB, WN> {
    static constexpr int kDepth = 32;
    // 16-byte operands: dlogits [term][expert / 8][token], W_r [expert / 8][column]
    bf16x8_t a[2][4][32 * MB], b[4][64 * WN];
    struct Next {
        float dl[8];
        u32x2 w[8];
    };
};
template <int MB, int WN>
struct DxTile<float, MB, WN> {
    static constexpr int kDepth = 16;
    f32x4 a[4][32 * MB];       // [expert / 4][token]
    float b[16][64 * WN + 4];  // padded: a lane's four reads of 16 columns miss each other's banks
    struct Next {
        f32x4 dl, w[2];
    };
};

// One tile by the 2 WN waves of thread tid; all threads of a workgroup, with
// tiles or without, meet the same barriers.  Without SMALL there are a tile's
// tokens and a step's experts at least: a tile (a step) that would reach past
// the last token (expert) starts early enough not to, and leaves out what
// others do.  SMALL takes the rest, with clamped addresses.
template <typename E, int MB, int WN, bool SMALL>
__device__ __forceinline__ void gate_dx_tile(unsigned block, int tid, const float *__restrict__ dl,
                                             unsigned T, int d, int Ne, const DxArgs &A,
                                             DxTile<E, MB, WN> (&lds)[2]) {
    const auto *__restrict__ wr = static_cast<const E *>(A.w_router);
    const auto *dx_in = static_cast<const E *>(A.dx_in);
    auto *dx = static_cast<E *>(A.dx);
    typedef DxTile<E, MB, WN> Tile;
    constexpr int kTokens = 32 * MB, kDepth = Tile::kDepth, kOwn = kDepth / 4;
    constexpr bool kBf16 = sizeof(E) == 2;
    int group;
    unsigned tile;
    const bool mine = share_of(block, A.groups, A.shares, group, tile);
    if (!mine) tile = 0;  // computed once more and not stored
    const int l = lane_id(), i16 = l & 15, G = l >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid / kWave), wm = wv / WN, wn = wv % WN;
    const int c0 = group * 64 * WN;
    const unsigned first = tile * kTokens, t0 = SMALL ? first : min(first, T - kTokens);

    // This thread's share of a step: dlogits of one token, kOwn consecutive
    // experts, and W_r: 16 WN lanes hold 4 columns each of a row; bf16 8 rows
    // of one operand (the first waves alone), fp32 two rows.
    constexpr int kRowLanes = 16 * WN, kRowsAtOnce = kWave / kRowLanes;
    const int a_tok = tid / 4, a_k = tid % 4 * kOwn;
    const unsigned a_at = 4 * (a_tok * Ne + a_k);
    const int w_sub = l / kRowLanes, w_col = l % kRowLanes * 4;
    const int w_rows = kBf16 ? 8 : 1;  // consecutive rows of a lane
    const unsigned w_at = sizeof(E) * (w_sub * w_rows * d + min(c0 + w_col, d - 4));
    const float *dl0 = dl + static_cast<size_t>(t0) * Ne;
    typename Tile::Next next;
    // first expert of a step's operands
    auto start = [&](int e0) { return __builtin_amdgcn_readfirstlane(SMALL ? e0 : min(e0, Ne - kDepth)); };
    auto weights = [&](int row) {  // row: the first of the kRowsAtOnce rows, or operands of rows
        if constexpr (SMALL) {
            const int own = min(row + w_sub * w_rows, Ne - 1);
            return wr + static_cast<size_t>(own) * d + min(c0 + w_col, d - 4);
        } else {
            return reinterpret_cast<const E *>(
                reinterpret_cast<const char *>(wr + static_cast<size_t>(row) * d) + w_at);
        }
    };
    auto load = [&](int e0) {
        const int e = start(e0);
        if constexpr (SMALL) {
            const float *row = dl + static_cast<size_t>(min(t0 + a_tok, T - 1)) * Ne;
#pragma unroll
            for (int j = 0; j < kOwn; j++) next.dl[j] = row[min(e + a_k + j, Ne - 1)];
        } else {
#pragma unroll
            for (int j = 0; j < kOwn; j += 4) {
                const f32x4 v = load_at<f32x4_unaligned>(dl0 + e + j, a_at);
#pragma unroll
                for (int q = 0; q < 4; q++) next.dl[j + q] = v[q];
            }
        }
        if constexpr (kBf16) {
            if (wv * kRowsAtOnce < 4) {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    next.w[j] = *reinterpret_cast<const u32x2 *>(
                        weights(e + 8 * kRowsAtOnce * wv + j));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; j++)
                next.w[j] = *reinterpret_cast<const f32x4 *>(weights(e + (2 * wv + j) * kRowsAtOnce));
        }
    };
    auto store = [&](int e0, Tile &to) {
        // experts of another step, and behind the last, have zero dlogits
        const int e = start(e0);
        float v[kOwn];
#pragma unroll
        for (int j = 0; j < kOwn; j++) {
            const int ej = e + a_k + j;
            v[j] = ej >= e0 && ej < Ne ? next.dl[j] : 0.f;
        }
        if constexpr (kBf16) {
            bf16x8_t terms[2];
            split_terms<2>(v, terms);
            to.a[0][tid % 4][a_tok] = terms[0];
            to.a[1][tid % 4][a_tok] = terms[1];
            if (wv * kRowsAtOnce < 4) {
                bf16x8_t b[4];
                transpose8<4>(next.w, b);
#pragma unroll
                for (int q = 0; q < 4; q++) to.b[wv * kRowsAtOnce + w_sub][w_col + q] = b[q];
            }
        } else {
            to.a[tid % 4][a_tok] = f32x4{v[0], v[1], v[2], v[3]};
#pragma unroll
            for (int j = 0; j < 2; j++)
                *reinterpret_cast<f32x4 *>(&to.b[(2 * wv + j) * kRowsAtOnce + w_sub][w_col]) = next.w[j];
        }
    };

    // This lane's outputs: tokens t0 + own + 16 m + v, columns c .. c + 3.
    typedef typename std::conditional<kBf16, u32x2, f32x4>::type Cols;
    const int c = c0 + 64 * wn + 4 * i16, own = 16 * MB * wm + 4 * G;
    const unsigned o_at = sizeof(E) * (own * d + min(c, d - 4));
    load(0);
    // sums start from dx_in
    f32x4 acc[MB][4];  // [16 tokens][ni]
    if (dx_in) {
        const E *from = dx_in + static_cast<size_t>(t0) * d;
#pragma unroll
        for (int m = 0; m < MB; m++)
#pragma unroll
            for (int v = 0; v < 4; v++) {
                Cols in = {};
                if (!SMALL || t0 + own + 16 * m + v < T)
                    in = load_at<Cols>(from + (16 * m + v) * d, o_at);
                if constexpr (kBf16) {
                    acc[m][0][v] = low_bf16(in[0]);
                    acc[m][1][v] = high_bf16(in[0]);
                    acc[m][2][v] = low_bf16(in[1]);
                    acc[m][3][v] = high_bf16(in[1]);
                } else {
#pragma unroll
                    for (int ni = 0; ni < 4; ni++) acc[m][ni][v] = in[ni];
                }
            }
    } else {
#pragma unroll
        for (int m = 0; m < MB; m++)
#pragma unroll
            for (int ni = 0; ni < 4; ni++) acc[m][ni] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    int buf = 0;
    for (int e0 = 0; e0 < Ne; e0 += kDepth, buf ^= 1) {
        Tile &at = lds[buf];
        store(e0, at);
        if (e0 + kDepth < Ne) load(e0 + kDepth);
        // the other buffer's readers have passed the barrier before this one
        __syncthreads();
        if constexpr (kBf16) {
            bf16x8_t b[4];
#pragma unroll
            for (int ni = 0; ni < 4; ni++) b[ni] = at.b[G][64 * wn + 4 * i16 + ni];
#pragma unroll
            for (int m = 0; m < MB; m++)
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    const bf16x8_t a = at.a[q][G][16 * MB * wm + 16 * m + i16];
#pragma unroll
                    for (int ni = 0; ni < 4; ni++)
                        acc[m][ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[ni], acc[m][ni], 0, 0, 0);
                }
        } else {
            f32x4 a[MB];
#pragma unroll
            for (int m = 0; m < MB; m++) a[m] = at.a[G][16 * MB * wm + 16 * m + i16];
#pragma unroll
            for (int q = 0; q < 4; q++) {  // expert 4 G + q
                const f32x4 b = *reinterpret_cast<const f32x4 *>(&at.b[4 * G + q][64 * wn + 4 * i16]);
#pragma unroll
                for (int m = 0; m < MB; m++)
#pragma unroll
                    for (int ni = 0; ni < 4; ni++)
                        acc[m][ni] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[m][q], b[ni], acc[m][ni], 0, 0, 0);
            }
        }
    }
    if (c >= d || !mine) return;
    E *to = dx + static_cast<size_t>(t0) * d;
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int v = 0; v < 4; v++) {
            Cols o;
            if constexpr (kBf16)
                o = Cols{pack_bf16(acc[m][0][v], acc[m][1][v]), pack_bf16(acc[m][2][v], acc[m][3][v])};
            else
                o = Cols{acc[m][0][v], acc[m][1][v], acc[m][2][v], acc[m][3][v]};
            const unsigned t = t0 + own + 16 * m + v;
            if (t >= first && t < T)
                *reinterpret_cast<Cols *>(reinterpret_cast<char *>(to + (16 * m + v) * d) + o_at) = o;
        }
}

template <typename E, int MB, int WN, bool SMALL>
__global__ __launch_bounds__(2 * WN *kWave, 4) void k_gate_dx_tile(const float *__restrict__ dl,
                                                                   unsigned T, int d, int Ne,
                                                                   const DxArgs dx) {
    __shared__ DxTile<E, MB, WN> lds[2];
    gate_dx_tile<E, MB, WN, SMALL>(blockIdx.x, threadIdx.x, dl, T, d, Ne, dx, lds);
}

// bf16, both products: those of dx in the form that DX names.  A pair of
// small tiles lies dx.blocks apart, on one XCD.
enum DxKind { kRegsVec, kRegs, kTile, kSmallTile, kPair, kSmallPair };
template <int MB, int DX>
__global__ __launch_bounds__(kBfThreads) void k_gate_bwd(const float *__restrict__ dl, unsigned T,
                                                         int d, int Ne, const DwArgs dw,
                                                         const DxArgs dx, bool dx_first) {
    typedef DxTile<uint16_t, 4, 4> Tile;
    typedef DxTile<uint16_t, 2, 2> Half;
    constexpr size_t kTileBytes = DX >= kPair ? 4 * sizeof(Half) : DX >= kTile ? 2 * sizeof(Tile) : 0;
    __shared__ __attribute__((aligned(16))) char lds[std::max(DwLds<MB>::kBytes, kTileBytes)];
    bool is_dw;
    const unsigned block = own_block(dw, dx, dx_first, is_dw);
    if (is_dw) {
        gate_dw<MB>(block, dl, T, d, Ne, dw, lds);
    } else if constexpr (DX >= kPair) {
        const int half = threadIdx.x / (kBfThreads / 2);
        gate_dx_tile<uint16_t, 2, 2, DX == kSmallPair>(
            block + half * dx.blocks, threadIdx.x % (kBfThreads / 2), dl, T, d, Ne, dx,
            reinterpret_cast<Half(*)[2]>(lds)[half]);
    } else if constexpr (DX >= kTile) {
        gate_dx_tile<uint16_t, 4, 4, false>(block, threadIdx.x, dl, T, d, Ne, dx,
                                            *reinterpret_cast<Tile(*)[2]>(lds));
    } else {
        gate_dx<(MB + 1) / 2, DX == kRegsVec>(block, dl, T, d, Ne, dx);
    }
}

// fp32: a wave makes 16 MB experts x 64 columns of dW_r from a quarter of the
// workgroup's tokens, 16 per step.  Expert MB i + m is row i of block m and
// column 4 i + q column i of block q, so that a lane's operands of 4 MB MFMAs
// are one piece of a token's dlogits and one of its x, of 16 bytes (MB = 4).
// Fewer experts take fewer blocks (8 experts, d = 2048: T = 256 6.9 us a call
// against 11.4 with four, T = 32768 163 against 181).
// What lies behind a token's last expert is read with it (its sums are not
// stored), except near the end of the array.
template <int MB>
using DwSums = f32x4[kWaves / 2][4 * MB][kWave];
template <int MB>
__device__ __forceinline__ void gate_dw_f32(unsigned block, const float *__restrict__ dl, unsigned T,
                                            int d, int Ne, const DwArgs &A, DwSums<MB> &s_acc) {
    const auto *__restrict__ x = static_cast<const float *>(A.x);
    float *__restrict__ part = A.out;
    const int col_groups = A.col_groups;
    int group;
    unsigned share;
    if (!share_of(block, A.groups, A.shares, group, share)) return;
    const int l = lane_id(), i16 = l & 15, G = l >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int c0 = group % col_groups * kDwColsF, e0 = group / col_groups * kDwExperts;
    const unsigned t0 = share * A.per_share, t1 = min(T, t0 + A.per_share);
    const int col = min(c0 + 4 * i16, d - 4), exp = min(e0 + MB * i16, Ne - 1);
    typedef float Experts __attribute__((ext_vector_type(MB), aligned(4)));
    f32x4 acc[MB][4];  // [m][q]
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int q = 0; q < 4; q++) acc[m][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    Experts an[4];
    f32x4 bn[4];  // the next step's tokens t + 4 u + G
    auto load = [&](unsigned t) {
        // MB - 1 values behind a row lie in the next rows, as many at most
        const bool inside = t + 16 + MB - 1 <= T;
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const size_t tu = min(t + 4 * u + G, T - 1);
            const float *row = dl + tu * Ne;
            if (inside) {
                an[u] = *reinterpret_cast<const Experts *>(row + exp);
            } else {
#pragma unroll
                for (int m = 0; m < MB; m++) an[u][m] = row[min(exp + m, Ne - 1)];
            }
            bn[u] = *reinterpret_cast<const f32x4 *>(x + tu * d + col);
        }
    };
    load(t0 + 16 * wv);
    for (unsigned t = t0 + 16 * wv; t < t1; t += 16 * kWaves) {
        Experts a[4];
        f32x4 b[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
            // tokens behind the share count nothing
            a[u] = t + 4 * u + G < t1 ? an[u] : Experts{};
            b[u] = bn[u];
        }
        load(t + 16 * kWaves);
#pragma unroll
        for (int u = 0; u < 4; u++)
#pragma unroll
            for (int m = 0; m < MB; m++)
#pragma unroll
                for (int q = 0; q < 4; q++)
                    acc[m][q] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[u][m], b[u][q], acc[m][q], 0, 0, 0);
    }
#pragma unroll
    for (int half = kWaves / 2; half > 0; half >>= 1) {
        if (wv >= half && wv < 2 * half)
#pragma unroll
            for (int m = 0; m < MB; m++)
#pragma unroll
                for (int q = 0; q < 4; q++) s_acc[wv - half][m * 4 + q][l] = acc[m][q];
        __syncthreads();
        if (wv < half)
#pragma unroll
            for (int m = 0; m < MB; m++)
#pragma unroll
                for (int q = 0; q < 4; q++) acc[m][q] += s_acc[wv][m * 4 + q][l];
        __syncthreads();
    }
    if (wv || c0 + 4 * i16 >= d) return;
    // lane: experts e0 + MB (4 G + v) + m, columns c0 + 4 i16 + q
    float *out = part + static_cast<size_t>(share) * Ne * d;
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int v = 0; v < 4; v++) {
            const int e = e0 + MB * (4 * G + v) + m;
            if (e < Ne)
                *reinterpret_cast<f32x4 *>(out + static_cast<size_t>(e) * d + col) =
                    f32x4{acc[m][0][v], acc[m][1][v], acc[m][2][v], acc[m][3][v]};
        }
}

// fp32, both products.
template <int MB, int DX>
__global__ __launch_bounds__(kThreads) void k_gate_bwd_f32(const float *__restrict__ dl, unsigned T,
                                                           int d, int Ne, const DwArgs dw,
                                                           const DxArgs dx) {
    typedef DxTile<float, 2, 2> Tile;
    typedef DxTile<float, 1, 1> Half;
    __shared__ __attribute__((aligned(16))) char
        lds[std::max(sizeof(DwSums<MB>), DX >= kPair ? 4 * sizeof(Half) : 2 * sizeof(Tile))];
    bool is_dw;
    const unsigned block = own_block(dw, dx, false, is_dw);
    if (is_dw) {
        gate_dw_f32<MB>(block, dl, T, d, Ne, dw, *reinterpret_cast<DwSums<MB> *>(lds));
    } else if constexpr (DX >= kPair) {
        const int half = threadIdx.x / (kThreads / 2);
        gate_dx_tile<float, 1, 1, DX == kSmallPair>(
            block + half * dx.blocks, threadIdx.x % (kThreads / 2), dl, T, d, Ne, dx,
            reinterpret_cast<Half(*)[2]>(lds)[half]);
    } else {
        gate_dx_tile<float, 2, 2, DX == kSmallTile>(block, threadIdx.x, dl, T, d, Ne, dx,
                                                    *reinterpret_cast<Tile(*)[2]>(lds));
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

// Token shares of dW_r: enough of them for a workgroup (two in fp32, of half
// the waves) on every CU if that leaves 512 tokens to a share, for half as
// many otherwise, beside dx's workgroups and with half the partial sums (each
// Ne x d fp32, written and read); of 128 tokens at least, and of all up to
// 256, which saves the launch that adds them.  From the shape alone, so that
// a sum does not depend on the device or on what else a call computes.
// Measured as one call at d = 2048, the larger count and half of it: bf16 T =
// 4096, 8 to 64 experts 18 to 26 us against 16 to 21, T = 32768 78 to 90
// against 81 to 97; fp32 T = 4096, 250 experts 88 against 86 (dW_r alone, T =
// 32768: 85 against 101); T = 256, d = 128, one share against two 12.1 against
// 14.8, T = 512 13.7 against 11.0.
static unsigned gate_dw_full(int d, int Ne, int bf16) {
    const unsigned groups = ceil_div(d, bf16 ? kDwCols : kDwColsF) * ceil_div(Ne, kDwExperts);
    return ceil_div(bf16 ? 256 : 512, groups);
}
static bool gate_dw_long(int T, int d, int Ne, int bf16) {
    return T / 512 >= static_cast<int>(gate_dw_full(d, Ne, bf16));
}
int gate_dw_shares(int T, int d, int Ne, int bf16) {
    if (T <= 256) return 1;
    const unsigned full = gate_dw_full(d, Ne, bf16);
    return static_cast<int>(
        std::min(gate_dw_long(T, d, Ne, bf16) ? full : ceil_div(full, 2), ceil_div(T, 128)));
}

hipError_t launch_gate_bwd(const float *dl, const void *x, const void *w_router, const void *dx_in,
                           int T, int d, int Ne, int bf16, void *dx, float *part, float *dw,
                           hipStream_t s) {
    const size_t bytes = static_cast<size_t>(T) * d * (bf16 ? 2 : 4);
    const auto xa = reinterpret_cast<uintptr_t>(x), da = reinterpret_cast<uintptr_t>(dx);
    if (dx && dw && xa < da + bytes && da < xa + bytes) {
        // dx lies in x: it is written when dW_r has read it
        const hipError_t e = launch_gate_bwd(dl, x, nullptr, nullptr, T, d, Ne, bf16, nullptr, part, dw, s);
        if (e != hipSuccess) return e;
        return launch_gate_bwd(dl, nullptr, w_router, dx_in, T, d, Ne, bf16, dx, nullptr, nullptr, s);
    }
    DwArgs W = {};
    if (dw) {
        W.x = x;
        W.shares = gate_dw_shares(T, d, Ne, bf16);
        W.out = W.shares > 1 ? part : dw;
        // whole steps; the last shares may then be empty, and sum to zero
        W.per_share = ceil_div(ceil_div(T, W.shares), 64) * 64;
        W.col_groups = ceil_div(d, bf16 ? kDwCols : kDwColsF);
        W.groups = W.col_groups * static_cast<int>(ceil_div(Ne, kDwExperts));
        W.blocks = whole_xcds(share_grid(W.groups, W.shares));
    }
    DxArgs X = {w_router, dx_in, dx, 0, 0, 0};
    using std::integral_constant;
    typedef integral_constant<int, 1> I1;
    typedef integral_constant<int, 2> I2;
    typedef integral_constant<int, 4> I4;
    // dx in tiles of 32 MB x 64 WN; true: fewer tokens or experts than one takes
    const auto tiles_of = [&](auto e, auto mb, auto wn) {
        constexpr int MB = decltype(mb)::value, WN = decltype(wn)::value;
        X.groups = ceil_div(d, 64 * WN);
        X.shares = ceil_div(T, 32 * MB);
        X.blocks = whole_xcds(share_grid(X.groups, X.shares));
        return T < 32 * MB || Ne < DxTile<decltype(e), MB, WN>::kDepth;
    };
    const auto small_tiles_alone = [&](auto e) {
        typedef decltype(e) E;
        if (tiles_of(e, I2{}, I2{}))
            k_gate_dx_tile<E, 2, 2, true><<<X.blocks, 4 * kWave, 0, s>>>(dl, T, d, Ne, X);
        else
            k_gate_dx_tile<E, 2, 2, false><<<X.blocks, 4 * kWave, 0, s>>>(dl, T, d, Ne, X);
    };
    // Long shares of dW_r are the finer work and follow dx's workgroups, which
    // each walk over many tiles (T = 32768, d = 2048, 30 experts: 83 us against
    // 90); few of them come first.
    const bool dx_first = Ne <= 64 && gate_dw_long(T, d, Ne, bf16);
    const auto both = [&](auto mb, auto kind, int threads) {
        k_gate_bwd<decltype(mb)::value, decltype(kind)::value>
            <<<W.blocks + X.blocks, threads, 0, s>>>(dl, T, d, Ne, W, X, dx_first);
    };
    if (!bf16) {
        const auto both_f32 = [&](auto mb, auto kind) {
            k_gate_bwd_f32<decltype(mb)::value, decltype(kind)::value>
                <<<W.blocks + X.blocks, kThreads, 0, s>>>(dl, T, d, Ne, W, X);
        };
        const auto run = [&](auto mb) {
            if (dx && tiles_of(float{}, I2{}, I2{}))
                both_f32(mb, integral_constant<int, kSmallTile>{});
            else
                both_f32(mb, integral_constant<int, kTile>{});
        };
        // Fewer 64 x 128 tiles than CUs: 32 x 64 (dx alone, d = 2048, 250 experts:
        // T = 64 10.0 us against 14.9, T = 512 14.9 against 16.1, T = 2048 28.9
        // against 27.4), beside dW_r a pair of them with several groups of
        // experts (T = 64 12.2 against 15.2; 64 experts 7.5 against 7.2).
        const bool few = static_cast<int64_t>(ceil_div(T, 64)) * ceil_div(d, 128) < 256;
        if (!dw) {
            // dx alone has more waves on a CU in its own kernel (T = 4096, d =
            // 2048: 8 experts 16 us against 21, 250 47 against 49)
            if (few) {
                if (tiles_of(float{}, I1{}, I1{}))
                    k_gate_dx_tile<float, 1, 1, true><<<X.blocks, 2 * kWave, 0, s>>>(dl, T, d, Ne, X);
                else
                    k_gate_dx_tile<float, 1, 1, false><<<X.blocks, 2 * kWave, 0, s>>>(dl, T, d, Ne, X);
            } else {
                small_tiles_alone(float{});
            }
        } else if (Ne <= 16) {
            run(I1{});
        } else if (Ne <= 32) {
            run(I2{});
        } else if (dx && few && Ne > kDwExperts) {
            const bool small = tiles_of(float{}, I1{}, I1{});
            X.blocks = whole_xcds(ceil_div(X.blocks, 2));
            if (small)
                both_f32(I4{}, integral_constant<int, kSmallPair>{});
            else
                both_f32(I4{}, integral_constant<int, kPair>{});
        } else {
            run(I4{});
        }
    } else if (dx && Ne > 64) {
        // W_r no longer fits a wave's registers.  Large tiles where there is one
        // for every CU (130 experts, d = 2048, dx alone: T = 4096 15.8 us against
        // 16.0, T = 8192 25.7 against 30.5) and small ones below (T = 512 6.8
        // against 11.0); beside dW_r, whose registers leave a CU one workgroup,
        // for every fourth, and two small ones to a workgroup (250 experts: T =
        // 64 12.2 against 18.4, T = 512 16.2 against 17.8, T = 2048 27.8 against
        // 22.9).  (d is at most 8192: a large tile is full.)
        const bool large =
            static_cast<int64_t>(ceil_div(T, 128)) * ceil_div(d, 256) >= (dw ? 64 : 256);
        if (!dw) {
            if (large) {
                tiles_of(uint16_t{}, I4{}, I4{});
                k_gate_dx_tile<uint16_t, 4, 4, false><<<X.blocks, 8 * kWave, 0, s>>>(dl, T, d, Ne, X);
            } else {
                small_tiles_alone(uint16_t{});
            }
        } else if (large) {
            tiles_of(uint16_t{}, I4{}, I4{});
            both(I4{}, integral_constant<int, kTile>{}, kBfThreads);
        } else {
            const bool small = tiles_of(uint16_t{}, I2{}, I2{});
            X.blocks = whole_xcds(ceil_div(X.blocks, 2));
            if (small)
                both(I4{}, integral_constant<int, kSmallPair>{}, kBfThreads);
            else
                both(I4{}, integral_constant<int, kPair>{}, kBfThreads);
        }
    } else {
        // dx alone in smaller workgroups, for the same waves on more CUs
        // (T = 256, d = 2048, 64 experts: 4.5 us against 5.9)
        const int threads = dw ? kBfThreads : kThreads;
        if (dx) {
            // waves walk over enough token tiles to pay for their W_r fragments
            X.groups = ceil_div(d, threads / kWave * kDxCols);
            X.shares = std::min(ceil_div(2048 / (threads / kWave), X.groups), ceil_div(T, 16));
            X.blocks = whole_xcds(share_grid(X.groups, X.shares));
        }
        const bool vec = Ne % 4 == 0 && reinterpret_cast<uintptr_t>(dl) % 16 == 0;
        const auto run = [&](auto mb) {
            if (vec)
                both(mb, integral_constant<int, kRegsVec>{}, threads);
            else
                both(mb, integral_constant<int, kRegs>{}, threads);
        };
        if (Ne <= 16)
            run(I1{});
        else if (Ne <= 32)
            run(I2{});
        else
            run(I4{});
    }
    if (W.shares > 1) {
        const size_t n4 = static_cast<size_t>(Ne) * d / 4;
        k_gate_dw_fold<<<ceil_div(n4, kFoldOut), kThreads, 0, s>>>(
            reinterpret_cast<const f32x4 *>(part), W.shares, n4, reinterpret_cast<f32x4 *>(dw));
    }
    return hipGetLastError();
}

}  // namespace occ
