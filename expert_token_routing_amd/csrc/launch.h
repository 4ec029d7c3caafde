// Host-side launchers of the library's kernels (internal; the C ABI is in
// include/occ.h).  Each queues its kernels on `stream` and returns the launch
// status.  Shapes have been validated by the caller.
#pragma once

#include "common.h"

namespace occ {

// Compute units of the current device (read once per device; 256 on MI355X).
int compute_units();

// --- routing (route.hip) ---
// prune_rule 0 none, 1 TRAVERSE, 2 GROUPSUM, 3 similarity (sim_rank: Ne x Ne
// ranked table, used only by rule 3).
hipError_t launch_route(const float *logits, int T, int Ne, int k, int prune_rule, int G,
                        const PlaceTab &tab, const int32_t *sim_rank, int32_t *ids, float *w,
                        hipStream_t s);
// Copies caller routing into ids/w, replacing out-of-range or repeated ids of
// a token by the lowest unused experts with weight 0.
hipError_t launch_sanitize_ids(const int32_t *ids_in, const float *w_in, int T, int k, int Ne,
                               int32_t *ids, float *w, hipStream_t s);

// --- gate projection (gate.hip) ---
// logits (T x Ne fp32) = x (T x d) . w_router (Ne x d)^T, bf16 or fp32 inputs.
hipError_t launch_gate(const void *x, const void *w_router, int T, int d, int Ne, int bf16,
                       float *logits, hipStream_t s);

// --- expert similarity table (similarity.hip) ---
// gram += H^T H (fp64, tokens ascending); H is T x Ne fp32.
hipError_t launch_sim_gram(const float *H, int T, int Ne, double *gram, hipStream_t s);
// Squared cosine similarities (t2 may be NULL) and each row's ranking.
hipError_t launch_sim_rank(const double *gram, int Ne, double *t2, int32_t *rank, hipStream_t s);

// --- BRIM (brim.hip) ---
constexpr int kBrimChunk = 128;  // tokens per BRIM workgroup
// Batches of at most kBrimSmallT tokens and kBrimSmallEntries routing
// entries build the BRIM in one workgroup (more entries are faster over
// the three kernels' several workgroups).
constexpr int kBrimSmallT = 512, kBrimSmallEntries = 1024;
struct BrimBufs {
    int32_t *brim0, *sfd_off, *epd_off, *tile_off, *epd_src, *tok_epd, *brim1;
    float *epd_w;
    int32_t *down_rows, *first_cnt, *tile_off_first, *tile_off_rest;
    int32_t *chunk_cnt, *chunk_base;
};
// tile_rows: the grouped GEMMs' row-tile capacity.  fill_cols > 0: the
// up-projection's column tiles; the experts then take extra row tiles (at
// most kBrimMaxFill) until the up-projection's tiles fill their last round
// of the CUs.
constexpr int kBrimMaxFill = 64;
hipError_t launch_brim(const int32_t *ids, const float *w, int T, int k, const PlaceTab &tab,
                       int tile_rows, int fill_cols, int dense_brim1, const BrimBufs &b,
                       hipStream_t s);

// --- row movers (rows.hip) ---
// x_sfd[brim0[g, t]] = x[t] for every group the token uses; with zero_out,
// also zero_out[brim0[g, t]][0 .. zero_cols) = 0 (fp32, zero_cols % 4 == 0).
hipError_t launch_dispatch(const void *x, int T, int Nd, size_t row_bytes, const int32_t *brim0,
                           void *x_sfd, hipStream_t s, float *zero_out = nullptr,
                           int zero_cols = 0);
// Deterministic stage one: each SFD row holds its first contributor's result
// (the token's lowest-position expert in the group) and y_epd[tok_epd[t, j]]
// holds the others'; sfd_out[brim0[g, t]] becomes the sum over the token's
// experts in group g in ascending placement position (fp32), written back
// only for groups with several experts.  With y, also stage two, as
// launch_combine would compute it (same order).
hipError_t launch_merge_slots(const float *y_epd, const int32_t *ids, const int32_t *tok_epd,
                              const int32_t *brim0, const PlaceTab &tab, int T, int k, int d,
                              float *sfd_out, const float *y_sh, void *y, int y_bf16,
                              hipStream_t s);
// y[t] = dtype( sum over g of sfd_out[brim0[g, t]] (+ y_sh[t]) ), fp32 sums in
// ascending group order.
hipError_t launch_combine(const float *sfd_out, const int32_t *brim0, const float *y_sh, int T,
                          int Nd, int d, int out_bf16, void *y, hipStream_t s);
hipError_t launch_fill_i32(int32_t *p, size_t n, int32_t v, hipStream_t s);

// --- grouped GEMMs, bf16 MFMA (gemm_bf16.hip) ---
// Up-projection with SwiGLU and routing-weight modulation:
//   out[r, f] = bf16( row_w[r] * silu(a_r . Wg[e][f]) * (a_r . Wu[e][f]) )
// a_r = A[a_rows[r]] (or A[r] when a_rows is NULL).  Routed mode walks the
// segments [seg_off[p], seg_off[p+1]) of each placement position p with the
// tile schedule tile_off; shared mode (seg_off NULL) is one segment of M rows.
// gu_out (optional, training): the pre-activations are also stored, row r
// holding bf16 g = a_r . Wg[e] in columns [0, N) and u in [N, 2N).
struct UpArgs {
    const void *A;
    const int32_t *a_rows;
    const void *Wg, *Wu;
    const int32_t *seg_off, *tile_off;
    const float *row_w;
    void *out;
    void *gu_out;
    int M, K, N, Ne;
    PlaceTab tab;
    int m_tiles;  // dense mode: row tiles (set by the bf16 launchers)
};
hipError_t launch_gemm_up_bf16(const UpArgs &a, size_t max_m_tiles, hipStream_t s);

// Down-projection.  Routed: the EPD rows of expert position p are
// rows[seg_off[p] ..  seg_off[p+1]), first_cnt[p] of them first contributors
// to their SFD row; phase 1 multiplies those and stores
// out[dst_rows[r], :] = A[r] . W[e]^T, which writes every SFD row once;
// phase 2 multiplies the others and adds with fp32 atomics (several experts
// of one group share an SFD row).  tile_off is the phase's row-tile schedule.
// Phase 3 (the deterministic merge's first half) multiplies every row, with
// the all-rows schedule: first contributors store into their SFD rows, the
// others into epd_out at their own EPD rows.
// Shared (seg_off NULL): out[r, :] = A[r] . W^T with W = n_sh blocks of
// (N x k_split) laid end to end along K.
struct DownArgs {
    const void *A;
    const void *W;
    const int32_t *seg_off, *tile_off;
    const int32_t *rows, *first_cnt;
    const int32_t *dst_rows;
    float *out;
    float *epd_out;  // phase 3
    int M, K, N, Ne, k_split, phase;
    PlaceTab tab;
    int m_tiles;  // dense mode: row tiles (set by the bf16 launchers)
};
hipError_t launch_gemm_down_bf16(const DownArgs &a, size_t max_m_tiles, hipStream_t s);
// The same with 128-row tiles (gemm_bf16_m128.hip), taken by bf16 batches
// whose experts average fewer than kSmallTileRows rows.
constexpr int kGemmBmBf16Small = 128;
constexpr int kSmallTileRows = 96;
hipError_t launch_gemm_up_bf16_m128(const UpArgs &a, size_t max_m_tiles, hipStream_t s);
hipError_t launch_gemm_down_bf16_m128(const DownArgs &a, size_t max_m_tiles, hipStream_t s);
// The same, four-wave and software-pipelined with 256 x 256 tiles
// (gemm_bf16_dense.hip), for dense products only (seg_off NULL; a routed
// launch returns hipErrorInvalidValue).  Taken by dense products of at least
// kDensePipeRounds rounds of tiles on the CUs.
constexpr int kDensePipeRounds = 4;
hipError_t launch_gemm_up_bf16_dense(const UpArgs &a, size_t max_m_tiles, hipStream_t s);
hipError_t launch_gemm_down_bf16_dense(const DownArgs &a, size_t max_m_tiles, hipStream_t s);

// --- the same two GEMMs in fp32 on the vector ALUs (gemm_f32.hip) ---
hipError_t launch_gemm_up_f32(const UpArgs &a, size_t max_m_tiles, hipStream_t s);
hipError_t launch_gemm_down_f32(const DownArgs &a, size_t max_m_tiles, hipStream_t s);

// --- the layer with experts in 8-bit integers ---
// Rows of K codes lie round_line(K) bytes apart, zeros behind K.
inline size_t round_line(size_t k) { return (k + 127) / 128 * 128; }
// (int8.hip) Rows of x (bf16 or fp32) as codes and a scale each: scale = a / 127,
// code = rint(v * (127 / a)), a the row's largest magnitude; a row with a below
// kInt8Tiny is held as zeros, one that is not finite gets a scale of NaN.  Rows
// of q lie ldq bytes apart, with zeros in cols .. ldq (multiples of 16).
constexpr float kInt8Tiny = 0x1p-100f;
hipError_t launch_quantize_rows(const void *x, int bf16, size_t rows, int cols, int8_t *q,
                                size_t ldq, float *scale, hipStream_t s);
// (slots.hip) The slots sorted by expert: EPD row of each slot (tok_epd, T x k), token and
// weight of each EPD row (epd_tok, epd_w), segments of the placement's positions (epd_off) and
// their row tiles (tile_off) as launch_brim's; ids and w are the caller's, made safe as by
// launch_sanitize_ids.  Beside that the rows of x as codes (xq, ldx bytes apart) with scales xs.
constexpr int kSlotsSmall = 1024, kSlotsSmallEntries = 8192;  // tokens and entries of one workgroup
constexpr int kSlotsMaxShares = 256;
struct SlotArgs {
    const int32_t *ids;
    const float *w;
    const u32x4 *x;
    int8_t *xq;
    float *xs;
    int32_t *tok_epd, *epd_tok, *epd_off, *tile_off;
    float *epd_w;
    int32_t *counts;  // kSlotsMaxShares x Ne
    size_t ldx;
    int T, d, k, tile_rows, fill_cols;
    PlaceTab tab;
    int share, shares, cus;  // set by the launcher
};
// Tokens a workgroup sorts; 0: one workgroup sorts all.
inline int slot_shares(int T, int k) {
    if (T <= kSlotsSmall && static_cast<size_t>(T) * k <= kSlotsSmallEntries) return 0;
    const int per = static_cast<int>(ceil_div(T, kSlotsMaxShares));
    return per > 256 ? per : 256;
}
hipError_t launch_slots(const SlotArgs &a, hipStream_t s);
// y[t] = bf16( sum over j of y_epd[tok_epd[t k + j]] + sum over s of y_sh[s T + t] ), bf16
// rows of d, fp32 sums in that order.
hipError_t launch_combine_rows(const uint16_t *y_epd, const int32_t *tok_epd, const uint16_t *y_sh,
                               int n_shared, int T, int k, int d, uint16_t *y, hipStream_t s);
// (gemm_int8.hip) h[r, f] = w_r silu(g) u in fp32, g = (xs_r sg[e][f]) (xq_r . Wg[e][f]), row
// r's codes and xs at a_rows[r] (or r); segments and tiles as in UpArgs.  lda in bytes.
struct Up8Args {
    const int8_t *A;
    const int32_t *a_rows;
    const float *a_scale;
    const int8_t *Wg, *Wu;
    const float *sg, *su;
    const int32_t *seg_off, *tile_off;
    const float *row_w;
    float *out;
    int M, K, N, Ne, lda;
    PlaceTab tab;
    int m_tiles;
};
// out[r, c] = bf16( (hs_r sd[e][c]) (hq_r . Wd[e][c]) ).
struct Down8Args {
    const int8_t *A;
    const float *a_scale;
    const int8_t *W;
    const float *sd;
    const int32_t *seg_off, *tile_off;
    uint16_t *out;
    int M, K, N, Ne, lda;
    PlaceTab tab;
    int m_tiles;
};
hipError_t launch_gemm_up8(const Up8Args &a, size_t max_m_tiles, hipStream_t s);
hipError_t launch_gemm_down8(const Down8Args &a, size_t max_m_tiles, hipStream_t s);
// The same with 80 x 128 tiles (gemm_int8_m80.hip), for batches whose experts average fewer
// than kSmallTileRows8 rows.
constexpr int kGemmBmInt8Small = 80, kSmallTileRows8 = 128;
hipError_t launch_gemm_up8_m80(const Up8Args &a, size_t max_m_tiles, hipStream_t s);
hipError_t launch_gemm_down8_m80(const Down8Args &a, size_t max_m_tiles, hipStream_t s);

// (int8_few.hip) The whole layer for few tokens: x, y T x d bf16, ids and w as
// the caller gave them; h (T k x F) and h_sh (T n_shared x F_shared) are
// scratch.  Shapes that few_fits refuses take the general path.
constexpr int kFewMaxD = 8192, kFewMaxShared = 16;
struct Int8Weights {
    const int8_t *gate, *up, *down;
    const float *gate_scale, *up_scale, *down_scale;
};
struct FewArgs {
    const uint16_t *x;
    const int32_t *ids;
    const float *w;
    Int8Weights routed, shared;
    float *h, *h_sh;
    uint16_t *y;
    int T, d, Ne, k, F, n_shared, F_shared;
};
bool few_fits(int d, int k, int F, int n_shared, int F_shared);
hipError_t launch_few(const FewArgs &a, hipStream_t s);

// --- routing by scores (score.hip) ---
struct ScoreArgs {
    const float *logits, *bias;  // bias may be NULL
    int T, Ne, k, sigmoid, top_groups, group_best, renormalise;
    float scale;
    PlaceTab tab;
    int32_t *ids;
    float *w;
    int over_n, in_order, per_wave, rounds;  // set by the launcher
};
hipError_t launch_route_scored(const ScoreArgs &a, hipStream_t s);
hipError_t launch_route_scored_back(const float *logits, const int32_t *ids, const float *dw,
                                    const float *dlogits_in, int T, int Ne, int k, int sigmoid,
                                    int renormalise, float scale, float *dlogits, hipStream_t s);
size_t bias_part_bytes(int T, int Ne, int k);
hipError_t launch_bias_step(const int32_t *ids, const uint8_t *valid, int T, int k, int Ne,
                            const float *bias_in, float rate, int32_t *counts, float *bias,
                            int32_t *part, hipStream_t s);

// --- backward grouped GEMMs, bf16 MFMA (gemm_bwd.hip) ---
// Input-gradient GEMM over row tiles of up to kBwdRowTile rows (tile_off over the segments
// seg_off of placement positions; first_cnt and phase select rows as in
// DownArgs):  C[pos, :] = A_row . B_e, K contracted, with A_row the K values
// at column a_col of row a_rows[pos] (or pos) of A (rows lda apart), and row
// k of B_e = B1[e] row k for k < ksplit, else B2[e] row k - ksplit (both N
// wide, so B is read K-major; e = tab.expert[p]).  N >= 256.  With b_kcontig
// (SWIGLU only, no B2, ksplit = K) B1 holds the weights transposed instead:
// expert e's block of N rows of K contiguous values, B_e[k][n] = B1[(e N + n) K + k].
// Epilogue SWIGLU: C is dh; with g = gu[pos*gu_ld + gu_col + f], u at
// + gu_uoff, and w = row_w[pos] (1 if NULL), writes bf16 dg, du to
// out[pos*out_ld + out_col + f] and + out_uoff, and (dw_part non-NULL)
// dw_part[pos * dw_stride + q] = this tile half's sum of dh * silu(g) u.
// Epilogue MERGE: C goes to merge_out[dst_rows[a_rows[pos]]] (identity
// without dst_rows / a_rows), N wide fp32: stored (merge_store) or added;
// with split (phase 0), the rows of a segment after its first_cnt first
// contributors are stored to epd_out[a_rows[pos]] instead.
enum { BWD_EPI_SWIGLU = 0, BWD_EPI_MERGE = 1 };
// Row capacity of the input-gradient tiles: the row schedules tile_off are
// built with it (ceil(rows / kBwdRowTile) tiles per segment, the all-rows
// schedule filled to whole rounds of the CUs; rows shared out evenly in
// 16-row blocks).
constexpr int kBwdRowTile = 320;
struct BwdDgradArgs {
    const void *A;
    const int32_t *a_rows;
    const void *B1, *B2;
    const int32_t *seg_off, *tile_off, *first_cnt, *dst_rows;
    const void *gu;
    const float *row_w;
    void *out;
    float *dw_part;
    float *merge_out;
    float *epd_out;
    int N, K, ksplit, Ne, phase, epilogue, dw_stride, merge_store, split, b_kcontig;
    int lda, a_col, gu_ld, gu_col, gu_uoff, out_ld, out_col, out_uoff;
    PlaceTab tab;
};
hipError_t launch_bwd_dgrad(const BwdDgradArgs &a, size_t max_m_tiles, hipStream_t s);

// Weight-gradient GEMM, one group of K rows per expert (routed: the expert
// segments seg_off, placement position order, e = tab.expert[p]; dense:
// seg_off NULL, n_groups blocks of `rows` rows, e = block):
//   C_e[m, n] = sum over the group's rows pos of A[a_rows[pos]][a_col + m] *
//               B[b_rows[pos]][b_col + n],   a_col = a_col0 + group * a_col_grp
// both operands K-major (rows lda / ldb elements apart); at most one of
// a_rows, b_rows is given (hipErrorInvalidValue otherwise).  Rows m < msplit go
// to C1[e] (msplit x N), the rest to C2[e].  M, N >= 256; tail rows of a
// group read zero_row (at least 256 zero elements).
// Dense launches (seg_off NULL) may split K (the rows) into k_parts chunks
// of k_chunk rows: each chunk's fp32 tiles go to `part` (k_parts x n_groups
// x M x N) and a second kernel adds them in chunk order into C1 / C2, so
// the result stays deterministic.
struct BwdWgradArgs {
    const void *A, *B;
    const int32_t *a_rows, *b_rows, *seg_off;
    const void *zero_row;
    float *C1, *C2;
    int M, N, msplit, lda, ldb, a_col0, a_col_grp, b_col0, b_col_grp, n_groups, rows;
    PlaceTab tab;
    int k_parts, k_chunk;
    float *part;
};
hipError_t launch_bwd_wgrad(const BwdWgradArgs &a, hipStream_t s);
// K chunks for a dense weight-gradient product of n_groups x M x N outputs
// over `rows` rows (1: no split), chosen from the shape alone; rows per
// chunk for that count.
int wgrad_k_parts(int n_groups, int M, int N, int rows);
int wgrad_k_chunk(int rows, int parts);

// Row-tile schedules for `tile_rows`-row tiles from the expert segments
// epd_off and first-contributor counts first_cnt (all rows, first, rest).
hipError_t launch_tile_sched(const int32_t *epd_off, const int32_t *first_cnt, int Ne,
                             int tile_rows, int fill_cols, int32_t *tile_off,
                             int32_t *tile_off_first, int32_t *tile_off_rest, hipStream_t s);
// A one-segment schedule for a dense GEMM over T rows: seg_off = {0, T},
// tile_off = {0, m_tiles} (the rows shared out evenly over m_tiles tiles).
hipError_t launch_dense_sched(int T, int m_tiles, int32_t *seg_off, int32_t *tile_off,
                              hipStream_t s);
// nz bf16 matrices of R x C, the z-th at src + z * src_z (elements), each
// written transposed: dst[z * dst_z + c * ldd + r] = src[z * src_z + r * C + c].
// R and C multiples of 64, ldd >= R, 16-byte aligned rows.
hipError_t launch_transpose_bf16(const void *src, int R, int C, size_t src_z, void *dst, int ldd,
                                 size_t dst_z, int nz, hipStream_t s);
// Routing-weight and logit gradients: dw[t, j] = sum of dw_part over the
// EPD row tok_epd[t*k + j]'s nparts partials (in order); dlogits through the
// full softmax of the logits (logits may be NULL: dw only).
hipError_t launch_route_backward(const float *logits, const int32_t *ids, const int32_t *tok_epd,
                                 const float *dw_part, int nparts, int dw_stride, int T, int Ne,
                                 int k, float *dw, float *dlogits, hipStream_t s);

// --- norms, gate and residual between two blocks (norm.hip) ---
// r = x + scale gate w_post n(y), h = w_pre n(r); gate_kind as occ_block_gate;
// y, w_post, gate, w_pre with h may be NULL.
hipError_t launch_block_norm(const void *x, const void *y, const void *w_post, const void *gate,
                             const void *w_pre, int T, int d, int bf16, int gate_kind, float eps,
                             float scale, void *r, void *h, hipStream_t s);
// Its backward; part holds norm_back_blocks x 2 x d floats.
int norm_back_blocks(int T, int chunks);  // chunks: 16-byte pieces of a row
hipError_t launch_block_norm_back(const void *dr, const void *dh, const void *r, const void *y,
                                  const void *w_post, const void *gate, const void *w_pre, int T,
                                  int d, int bf16, int gate_kind, float eps, float scale, void *dx,
                                  void *dy, float *dw_post, float *dgate, float *dw_pre,
                                  float *part, hipStream_t s);

// --- router losses (balance.hip) ---
size_t balance_part_bytes(int T, int Ne);
hipError_t launch_balance(const float *logits, const int32_t *ids, const uint8_t *valid, int T,
                          int k, const PlaceTab &tab, float cb, float cg, float cz,
                          int32_t *counts, float *probs, float *loss, float *part, hipStream_t s);
hipError_t launch_balance_back(const float *logits, const uint8_t *valid, const int32_t *counts,
                               const PlaceTab &tab, int T, int k, float cb, float cg, float cz,
                               float dloss, const float *dlogits_in, float *dlogits,
                               hipStream_t s);

// --- gate projection, backward (gate_bwd.hip) ---
// dx = dx_in + dl w_router (dx_in may be NULL);  dw = dl^T x through
// gate_dw_shares x Ne x d partial sums in part.  NULL dx or dw: not computed.
// dx may lie in x.
int gate_dw_shares(int T, int d, int Ne, int bf16);
hipError_t launch_gate_bwd(const float *dl, const void *x, const void *w_router, const void *dx_in,
                           int T, int d, int Ne, int bf16, void *dx, float *part, float *dw,
                           hipStream_t s);

// --- optimizer step (adamw.hip) ---
constexpr int64_t kAdamwMaxElements = 1ll << 33;  // of one tensor
struct AdamwTensor {
    int64_t n;
    const float *p;
    const void *g, *m, *v;
    const float *m_scale, *v_scale;
    float *p_out;
    void *m_out, *v_out;
    float *m_scale_out, *v_scale_out;
    void *p_bf16;
    int64_t aligned;  // every array may be moved four elements at a time
};
struct AdamwStep {
    float lr, beta1, one_b1, beta2, one_b2, eps, weight_decay, grad_scale;
    float c1, c2_rsqrt;     // 1 - beta1^step, 1 / sqrt(1 - beta2^step)
    float log_b1, log_b2;   // for a step read from `dynamic`
    const float *dynamic;   // NULL or {lr, step, grad_scale} on the device
};
hipError_t launch_adamw(const AdamwTensor *tensors, int count, const AdamwStep &st, int q8,
                        int grad_bf16, hipStream_t s);

// --- co-activation statistics (coact.hip) ---
hipError_t launch_coact(const int32_t *ids, int T, int k, const PlaceTab &tab, int32_t *C,
                        float *P, int64_t *n_sfd, double *ct, double *intra, hipStream_t s);

}  // namespace occ
