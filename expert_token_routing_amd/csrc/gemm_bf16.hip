// Grouped expert GEMMs on the bf16 matrix cores of gfx950 (MFMA
// v_mfma_f32_16x16x32_bf16, fp32 accumulation).
//
// These are the paper's sparse matrix multiplications (appendix A.2):
//   up    SMM scattering SFD -> EPD (Algorithm 6) fused with the SwiGLU
//         activation and the weight modulation (Algorithm 7): for each
//         expert, its EPD rows gather their SFD rows (the condensed BRIM_1,
//         section 3.1 footnote 2) and produce
//           epd[r, f] = bf16( w_r * silu(a_r . Wg[f]) * (a_r . Wu[f]) );
//         the weight scales the hidden state after the activation, which is
//         exact because the down-projection is linear;
//   down  SMM merging EPD -> SFD (Algorithm 8): each EPD row's product with
//         W_down is added in fp32 to its SFD row (several experts of one group
//         share that row -- the intra-group pre-aggregation of section 3.1).
//
// Tiling (the grouped build; the dense build's four-wave pipelined loop is
// described where it is defined): a 512-thread workgroup (8 waves, one
// workgroup per CU, two waves per SIMD) computes a tile of up to 320 rows x
// 256 MFMA output columns.  The
// rows come in 16-row blocks dealt to the four wave rows in turn, and each
// wave holds 128 columns of its blocks.  In the up GEMM the 256 columns
// are 128 gate and 128 up rows of the same output features, so the SwiGLU
// epilogue has both operands in registers.  K is consumed in 64-deep slices
// (each row's slice is one 128-byte line) through two 72 KB LDS buffers
// filled by direct global->LDS loads: slice kt+1 is issued right after the
// barrier that opens slice kt and lands during its MFMA work.  Measured on
// the OLMoE-shaped layer, this beats 32-deep slices in a 3- to 5-deep ring
// by 9% in the up-projection (a deeper ring of 64-byte slices did not help:
// the load path, not its depth, is the limit).  The 16-byte chunks of an LDS
// row are XOR-swizzled by row so that fragment reads of 16 consecutive rows
// hit distinct banks.  The up GEMM's bf16 output tile is staged through LDS
// and written as whole 16-byte row chunks.
//
// Scheduling: the BRIM scan gives each expert ceil(rows / BM) row tiles
// (tile_off), so every tile reads one expert's weights, and the expert's
// row blocks are shared out evenly among them.  With 320-row capacity an
// expert of 1025-1067 rows is four tiles of 256-272 rows instead of four
// full 256-row tiles and a fifth of at most 43 rows that costs as much as a
// full one (the tile's time is set by its weight loads).  Measured on the
// OLMoE-shaped layer (287 -> 255 row tiles): -3% in both projections; the
// balance is imperfect because a 17-block tile gives one SIMD pair 9 blocks.
// A wave skips the MFMAs and the direct loads of blocks that hold no rows.
// Workgroup b runs on
// XCD b % 8; tiles are renumbered so that each XCD takes a contiguous range
// of an expert-major tile order (inside an expert, bands of 8 row tiles
// walked column by column, except in the atomic merge phase; a dense product
// the same way): the workgroups sharing an expert's weights and a row tile's
// activations share one L2.
// 256-row tiles halve the weight bytes fetched per flop against 128-row
// tiles (measured: 1.6 vs 2.5 GB beyond L2 per up-projection launch on the
// OLMoE-shaped layer).  The 128-row build (the decode regime) shares all of
// this with four two-block wave rows.
#include "gemm_tile.h"

namespace occ {
namespace {

// Second bound: waves per SIMD = workgroups per CU x NT / 256.
__global__ __launch_bounds__(NT, OCC_GEMM_WG_PER_CU * NT / 256) void OCC_NAMED(k_gemm_up)(UpArgs a) {
    __shared__ __attribute__((aligned(16))) uint16_t smem[RING];
    __shared__ float s_w[BM];
    Tile t;
    if (!tile_of(a.seg_off, a.tile_off, a.M, a.m_tiles, a.Ne, a.tab, (a.N + 127) / 128, 128, t))
        return;

    const int tid = threadIdx.x, r0 = tid / CHUNKS;
    const int K = a.K, N = a.N;
    const uint16_t *A = static_cast<const uint16_t *>(a.A);
    const uint16_t *Wg = static_cast<const uint16_t *>(a.Wg) + static_cast<size_t>(t.e) * N * K;
    const uint16_t *Wu = static_cast<const uint16_t *>(a.Wu) + static_cast<size_t>(t.e) * N * K;
    PtrSrc src;
#pragma unroll
    for (int i = 0; i < A_LD; i++) {
        const int r = min(r0 + i * ROWS_PER_PASS, t.rows - 1);
        const int row = t.seg + t.m0 + r;
        const int arow = a.a_rows ? a.a_rows[row] : row;
        src.a[i] = A + static_cast<size_t>(arow) * K + fetch_chunk(r0 + i * ROWS_PER_PASS) * 8;
    }
#pragma unroll
    for (int i = 0; i < B_LD; i++) {
        const int rb = r0 + i * ROWS_PER_PASS;
        const int f = min(t.n0 + (rb & 127), N - 1);
        src.b[i] = (rb < 128 ? Wg : Wu) + static_cast<size_t>(f) * K + fetch_chunk(rb) * 8;
    }

    const int l = lane_id(), wv = tid / kWave, wm = wv >> 1, wn = wv & 1;  // wm < WAVES_M
    int brow[NI];
#pragma unroll
    for (int ni = 0; ni < NI; ni++)
        brow[ni] = (ni < NI / 2 ? 0 : 128) + wn * 64 + (ni % (NI / 2)) * 16 + (l & 15);
    acc_t acc[MI][NI];
#pragma unroll
    for (int mi = 0; mi < MI; mi++)
#pragma unroll
        for (int ni = 0; ni < NI; ni++) acc[mi][ni] = acc_t{0.f, 0.f, 0.f, 0.f};

    int nv, na;
    wave_share(t.rows, wm, nv, na);
    // The rows' routing weights, loaded once by one thread per row (loaded by
    // every lane in the epilogue, they were waited for one by one).
    auto pre = [&] {
        if (tid < t.rows) s_w[tid] = a.row_w ? a.row_w[t.seg + t.m0 + tid] : 1.f;
    };
    run_k_loop<true>(nv, src, K, K, 0, smem, wm, brow, acc, na, pre);

    // SwiGLU + modulation in registers (the sigmoid's division by the
    // hardware reciprocal: the result is rounded to bf16, and the IEEE
    // division sequence made the epilogue -- during which the matrix cores
    // idle -- several times longer); bf16 tiles staged in LDS (the K
    // buffers are free after the loop's last barrier) and written as whole
    // 16-byte row chunks: the hidden state, then in training the gate and up
    // pre-activations the backward pass reads (two more passes through the
    // same staging rows; written lane by lane they were 2-byte stores).
    // All three are non-temporal: the hidden states are read back only by
    // the next launch and the pre-activations by the backward pass, and kept
    // out of the L2 they leave the weight and activation slices that the
    // running tiles share (measured on the OLMoE-shaped layer: -1.5% here,
    // -4% in the decode step; the same hint on the down-projection's fp32
    // stores cost 6-10%).
    constexpr int CH = 128 / 8;  // 16-byte chunks per staged row
    auto stage = [&](int which) {  // 0: h, 1: g, 2: u
        // lane l holds row (l & 15) of each block and features 4 (l >> 4) .. + 3
        // of each 16-feature group (the MFMAs ran with their operands
        // exchanged): one 8-byte LDS write per group
#pragma unroll
        for (int mi = 0; mi < MI; mi++) {
            const int r = block_row(wm, mi) + (l & 15);
            const float wr = s_w[min(r, t.rows - 1)];
#pragma unroll
            for (int ni = 0; ni < NI / 2; ni++) {
                u16x4 o;
#pragma unroll
                for (int v = 0; v < 4; v++) {
                    const float g = acc[mi][ni][v], u = acc[mi][ni + NI / 2][v];
                    const float x = which == 0 ? g * __builtin_amdgcn_rcpf(1.f + __expf(-g)) * u * wr
                                               : (which == 1 ? g : u);
                    o[v] = f32_to_bf16_bits(x);
                }
                *reinterpret_cast<u16x4 *>(smem + r * OUT_PITCH + wn * 64 + ni * 16 + 4 * (l >> 4)) = o;
            }
        }
        __syncthreads();
    };
    auto flush = [&](uint16_t *base, size_t ld) {  // staged rows -> base[row * ld + n0 ..]
#pragma unroll 4
        for (int i = tid; i < BM * CH; i += NT) {
            const int r = i / CH, c = (i % CH) * 8;
            if (r >= t.rows || t.n0 + c >= N) continue;
            const u32x4 v = *reinterpret_cast<const u32x4 *>(smem + r * OUT_PITCH + c);
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(
                                               base + (static_cast<size_t>(t.seg) + t.m0 + r) * ld + t.n0 + c));
        }
    };
    stage(0);
    flush(static_cast<uint16_t *>(a.out), N);
    if (a.gu_out) {
        // training: keep the pre-activations for the backward pass, row r
        // holding g in columns [0, N) and u in [N, 2N)
        uint16_t *gu = static_cast<uint16_t *>(a.gu_out);
        __syncthreads();
        stage(1);
        flush(gu, 2 * static_cast<size_t>(N));
        __syncthreads();
        stage(2);
        flush(gu + N, 2 * static_cast<size_t>(N));
    }
}

__global__ __launch_bounds__(NT, OCC_GEMM_WG_PER_CU * NT / 256) void OCC_NAMED(k_gemm_down)(DownArgs a) {
    __shared__ __attribute__((aligned(16))) uint16_t smem[RING];
    __shared__ int s_dst[BM];
    Tile t;
    if (!tile_of(a.seg_off, a.tile_off, a.M, a.m_tiles, a.Ne, a.tab, (a.N + BN - 1) / BN, BN, t,
                 a.first_cnt, a.phase, kBandDown))
        return;

    const int tid = threadIdx.x, r0 = tid / CHUNKS;
    const int K = a.K, N = a.N, ksp = a.k_split;
    const uint16_t *A = static_cast<const uint16_t *>(a.A);
    // W is (blocks of N x ksp) along K; routed experts have one block (ksp = K).
    const uint16_t *W = static_cast<const uint16_t *>(a.W) + static_cast<size_t>(t.e) * N * K;
    PtrSrc src;
#pragma unroll
    for (int i = 0; i < A_LD; i++) {
        const int r = min(r0 + i * ROWS_PER_PASS, t.rows - 1);
        const int row = t.seg + t.m0 + r;
        const int arow = a.rows ? a.rows[row] : row;
        src.a[i] = A + static_cast<size_t>(arow) * K + fetch_chunk(r0 + i * ROWS_PER_PASS) * 8;
    }
#pragma unroll
    for (int i = 0; i < B_LD; i++) {
        const int n = min(t.n0 + r0 + i * ROWS_PER_PASS, N - 1);
        src.b[i] = W + static_cast<size_t>(n) * ksp + fetch_chunk(r0 + i * ROWS_PER_PASS) * 8;
    }
    const size_t blk = static_cast<size_t>(N) * ksp;

    const int l = lane_id(), wv = tid / kWave, wm = wv >> 1, wn = wv & 1;  // wm < WAVES_M
    int brow[NI];
#pragma unroll
    for (int ni = 0; ni < NI; ni++) brow[ni] = wn * WN + ni * 16 + (l & 15);
    acc_t acc[MI][NI];
#pragma unroll
    for (int mi = 0; mi < MI; mi++)
#pragma unroll
        for (int ni = 0; ni < NI; ni++) acc[mi][ni] = acc_t{0.f, 0.f, 0.f, 0.f};

    int nv, na;
    wave_share(t.rows, wm, nv, na);
    // The SFD row of each of the tile's rows, looked up once by one thread
    // per row (two dependent loads): looked up by every lane in the
    // epilogue, the lookups ran in series, one L2 round trip pair per row
    // (measured on the OLMoE-shaped layer: -10% in the first merge phase,
    // -5% in the atomic phase).  Phase 3 sends the rows after the first
    // contributors to their own EPD rows instead, marked by a negative entry
    // ~erow.
    auto pre = [&] {
        if (a.dst_rows && tid < t.rows) {
            const size_t row = static_cast<size_t>(t.seg) + t.m0 + tid;
            const int erow = a.rows ? a.rows[row] : static_cast<int>(row);
            s_dst[tid] = a.phase == 3 && tid >= t.first ? ~erow : a.dst_rows[erow];
        }
    };
    run_k_loop<false>(nv, src, K, ksp, blk, smem, wm, brow, acc, na, pre);

    float *out = a.out;
#pragma unroll
    for (int mi = 0; mi < MI; mi++)
#pragma unroll
        for (int v = 0; v < 4; v++) {
            const int r = block_row(wm, mi) + 4 * (l >> 4) + v;
            if (r >= t.rows) continue;
            const size_t row = static_cast<size_t>(t.seg) + t.m0 + r;
            if (a.dst_rows) {
                const int d = s_dst[r];
                float *dst = d < 0 ? a.epd_out + static_cast<size_t>(~d) * N
                                   : out + static_cast<size_t>(d) * N;
                if (a.phase == 1 || a.phase == 3) {
#pragma unroll
                    for (int ni = 0; ni < NI; ni++) {
                        const int c = t.n0 + wn * WN + ni * 16 + (l & 15);
                        if (c < N) dst[c] = acc[mi][ni][v];
                    }
                } else {
#pragma unroll
                    for (int ni = 0; ni < NI; ni++) {
                        const int c = t.n0 + wn * WN + ni * 16 + (l & 15);
                        if (c < N) unsafeAtomicAdd(dst + c, acc[mi][ni][v]);
                    }
                }
            } else {
#pragma unroll
                for (int ni = 0; ni < NI; ni++) {
                    const int c = t.n0 + wn * WN + ni * 16 + (l & 15);
                    if (c < N) out[row * N + c] = acc[mi][ni][v];
                }
            }
        }
}

}  // namespace

hipError_t OCC_NAMED(launch_gemm_up_bf16)(const UpArgs &a, size_t max_m_tiles, hipStream_t s) {
    UpArgs b = a;
#ifdef OCC_GEMM_DENSE_ONLY
    // routed row-tile schedules are cut for the grouped builds' tile height
    if (a.seg_off) return hipErrorInvalidValue;
#endif
    const int n_tiles = static_cast<int>(ceil_div(a.N, 128));
    if (!a.seg_off) {
        b.m_tiles = dense_row_tiles(a.M, n_tiles);
        max_m_tiles = static_cast<size_t>(b.m_tiles);
    }
    const unsigned grid = grid_for(max_m_tiles, n_tiles);
    if (grid == 0) return hipSuccess;
    OCC_NAMED(k_gemm_up)<<<grid, NT, 0, s>>>(b);
    return hipGetLastError();
}

hipError_t OCC_NAMED(launch_gemm_down_bf16)(const DownArgs &a, size_t max_m_tiles, hipStream_t s) {
    DownArgs b = a;
#ifdef OCC_GEMM_DENSE_ONLY
    // routed row-tile schedules are cut for the grouped builds' tile height
    if (a.seg_off) return hipErrorInvalidValue;
#endif
    const int n_tiles = static_cast<int>(ceil_div(a.N, BN));
    if (!a.seg_off) {
        b.m_tiles = dense_row_tiles(a.M, n_tiles);
        max_m_tiles = static_cast<size_t>(b.m_tiles);
    }
    const unsigned grid = grid_for(max_m_tiles, n_tiles);
    if (grid == 0) return hipSuccess;
    OCC_NAMED(k_gemm_down)<<<grid, NT, 0, s>>>(b);
    return hipGetLastError();
}

}  // namespace occ
