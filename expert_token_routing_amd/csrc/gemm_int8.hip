// Grouped expert GEMMs on the int8 matrix cores of gfx950 (MFMA
// v_mfma_i32_16x16x64_i8), for experts whose weights are 8-bit integers with
// an fp32 scale for each output channel and whose rows are 8-bit integers
// with an fp32 scale for each row:
//   up    h[r, f] = w_r * silu(g) * u,  g = (xs_r sg[f]) * (xq_r . Wg[f]),
//         u likewise; fp32, for the row quantiser that follows;
//   down  out[r, c] = (hs_r sd[c]) * (hq_r . Wd[c]), rounded to bf16.
// The integer sums are exact (|code| <= 127: K <= 2^17 products stay below
// 2^31), so a result does not depend on the order or the tile it was summed in.
//
// The tile and its K loop are the bf16 kernels' (gemm_tile.h), since a tile
// moves bytes: a 128-byte line holds 128 int8 instead of 64 bf16, a 16-byte
// fragment 16, and the int8 instruction multiplies 64 bytes of K in the
// cycles that the bf16 one does.  Half the bytes and half the instructions a
// product.  Measured (d = 2048, 64 experts of F = 1024, top 8, 320-row tiles):
// 8192 tokens up 298 us, down 190 (1.84 and 1.45 POP/s, against 2.04 of a plain
// 8192 x 8192 x 8192 int8 product), bound by the matrix cores and, in the
// down-projection, the epilogue's stores; 512 tokens on 80-row tiles 64 and 39
// us for 282 and 141 MB of weights and rows (4.4 and 3.6 TB/s), bound by memory.  K need only be a multiple of 64: rows of codes are padded with
// zeros to whole lines (lda), and in the last line the loads of weights that
// would pass the row's end read what lies before it again, which meets zeros.
#ifndef OCC_GEMM_INT8
#define OCC_GEMM_INT8 1
#endif
#include "gemm_tile.h"

namespace occ {
namespace {

constexpr int FT = BN / 2;  // features of an up-projection tile: as many gate and up columns

// The direct loads' addresses; where the last K slice is not a whole line it
// starts at `last`, and the threads behind the row's end step back into it.
struct LineEndSrc {
    const uint16_t *a[A_LD], *b[B_LD];
    size_t last;
    int back;
    __device__ const uint16_t *a_at(int i, int k0) const { return a[i] + k0; }
    __device__ const uint16_t *b_at(int i, size_t bo) const { return b[i] + bo - (bo == last ? back : 0); }
};
__device__ __forceinline__ void line_end(LineEndSrc &src, int K, int chunk) {
    const int rest = K % BK, chunks = rest / 8;
    src.last = rest ? static_cast<size_t>(K - rest) : ~static_cast<size_t>(0);
    src.back = rest && chunk >= chunks ? (chunk - chunk % chunks) * 8 : 0;
}

__device__ __forceinline__ void clear(acc_t (&acc)[MI][NI]) {
#pragma unroll
    for (int mi = 0; mi < MI; mi++)
#pragma unroll
        for (int ni = 0; ni < NI; ni++) acc[mi][ni] = acc_t{0, 0, 0, 0};
}

__global__ __launch_bounds__(NT, OCC_GEMM_WG_PER_CU * NT / 256) void OCC_NAMED(k_gemm_up8)(Up8Args a) {
    __shared__ __attribute__((aligned(16))) uint16_t smem[RING];
    __shared__ float s_x[BM], s_w[BM];
    __shared__ f32x4 s_g[FT / 4], s_u[FT / 4];
    Tile t;
    if (!tile_of(a.seg_off, a.tile_off, a.M, a.m_tiles, a.Ne, a.tab, (a.N + FT - 1) / FT, FT, t))
        return;

    const int tid = threadIdx.x, r0 = tid / CHUNKS;
    const int K = a.K / 2, lda = a.lda / 2, N = a.N;  // in 2-byte units
    const uint16_t *A = reinterpret_cast<const uint16_t *>(a.A);
    const size_t w0 = static_cast<size_t>(t.e) * N;
    const uint16_t *Wg = reinterpret_cast<const uint16_t *>(a.Wg) + w0 * K;
    const uint16_t *Wu = reinterpret_cast<const uint16_t *>(a.Wu) + w0 * K;
    LineEndSrc src;
#pragma unroll
    for (int i = 0; i < A_LD; i++) {
        const int r = min(r0 + i * ROWS_PER_PASS, t.rows - 1);
        const int row = t.seg + t.m0 + r;
        const int arow = a.a_rows ? a.a_rows[row] : row;
        src.a[i] = A + static_cast<size_t>(arow) * lda + fetch_chunk(r0 + i * ROWS_PER_PASS) * 8;
    }
#pragma unroll
    for (int i = 0; i < B_LD; i++) {
        const int rb = r0 + i * ROWS_PER_PASS;
        const int f = min(t.n0 + rb % FT, N - 1);
        src.b[i] = (rb < FT ? Wg : Wu) + static_cast<size_t>(f) * K + fetch_chunk(rb) * 8;
    }
    // rows a whole number of passes apart share their swizzle key, and so a
    // thread's chunk
    static_assert(ROWS_PER_PASS % 16 == 0, "one fetch chunk a thread");
    line_end(src, K, fetch_chunk(r0));

    const int l = lane_id(), wv = tid / kWave, wm = wv >> 1, wn = wv & 1;
    int brow[NI];
#pragma unroll
    for (int ni = 0; ni < NI; ni++)
        brow[ni] = (ni < NI / 2 ? 0 : FT) + wn * (FT / 2) + (ni % (NI / 2)) * 16 + (l & 15);
    acc_t acc[MI][NI];
    clear(acc);

    int nv, na;
    wave_share(t.rows, wm, nv, na);
    auto pre = [&] {
        if (tid < t.rows) {
            const int row = t.seg + t.m0 + tid;
            s_x[tid] = a.a_scale[a.a_rows ? a.a_rows[row] : row];
            s_w[tid] = a.row_w ? a.row_w[row] : 1.f;
        }
        if (tid < FT) {
            const int f = min(t.n0 + tid, N - 1);
            reinterpret_cast<float *>(s_g)[tid] = a.sg[w0 + f];
            reinterpret_cast<float *>(s_u)[tid] = a.su[w0 + f];
        }
    };
    run_k_loop<true>(nv, src, K, K, 0, smem, wm, brow, acc, na, pre);

    // Scales and SwiGLU in registers: with the operands exchanged a lane
    // holds row (l & 15) and features 4 (l >> 4) .. + 3 of each group of 16,
    // one 16-byte store (through LDS, as 256-byte pieces of rows, the layer took
    // 620 us at 8192 tokens against 608: unlike bf16 rows, four lanes fill a
    // 64-byte sector).  Stored through the caches, where the quantiser finds
    // part of them: past them the kernel took 317 us against 298.  h stays fp32 until its row's largest magnitude is
    // known: rounded to bf16 first, an eighth of the codes would come out one
    // step off (0.8% of h's size), as much as the quantisation itself.
#pragma unroll
    for (int mi = 0; mi < MI; mi++) {
        const int r = block_row(wm, mi) + (l & 15);
        if (r >= t.rows) continue;
        const float xs = s_x[r], wr = s_w[r];
        float *dst = a.out + (static_cast<size_t>(t.seg) + t.m0 + r) * N;
#pragma unroll
        for (int ni = 0; ni < NI / 2; ni++) {
            const int c = wn * (FT / 2) + ni * 16 + 4 * (l >> 4);
            if (t.n0 + c >= N) continue;
            const f32x4 cg = s_g[c / 4], cu = s_u[c / 4];
            f32x4 o;
#pragma unroll
            for (int v = 0; v < 4; v++) {
                const float g = static_cast<float>(acc[mi][ni][v]) * (xs * cg[v]);
                const float u = static_cast<float>(acc[mi][ni + NI / 2][v]) * (xs * cu[v]);
                o[v] = swiglu(g, u) * wr;
            }
            *reinterpret_cast<f32x4 *>(dst + t.n0 + c) = o;
        }
    }
}

__global__ __launch_bounds__(NT, OCC_GEMM_WG_PER_CU * NT / 256) void OCC_NAMED(k_gemm_down8)(Down8Args a) {
    __shared__ __attribute__((aligned(16))) uint16_t smem[RING];
    __shared__ float s_h[BM];
    __shared__ f32x4 s_d[BN / 4];
    Tile t;
    if (!tile_of(a.seg_off, a.tile_off, a.M, a.m_tiles, a.Ne, a.tab, (a.N + BN - 1) / BN, BN, t,
                 nullptr, 0, kBandDown))
        return;

    const int tid = threadIdx.x, r0 = tid / CHUNKS;
    const int K = a.K / 2, lda = a.lda / 2, N = a.N;
    const uint16_t *A = reinterpret_cast<const uint16_t *>(a.A);
    const size_t w0 = static_cast<size_t>(t.e) * N;
    const uint16_t *W = reinterpret_cast<const uint16_t *>(a.W) + w0 * K;
    LineEndSrc src;
#pragma unroll
    for (int i = 0; i < A_LD; i++) {
        const int r = min(r0 + i * ROWS_PER_PASS, t.rows - 1);
        src.a[i] = A + (static_cast<size_t>(t.seg) + t.m0 + r) * lda + fetch_chunk(r0 + i * ROWS_PER_PASS) * 8;
    }
#pragma unroll
    for (int i = 0; i < B_LD; i++) {
        const int n = min(t.n0 + r0 + i * ROWS_PER_PASS, N - 1);
        src.b[i] = W + static_cast<size_t>(n) * K + fetch_chunk(r0 + i * ROWS_PER_PASS) * 8;
    }
    line_end(src, K, fetch_chunk(r0));

    const int l = lane_id(), wv = tid / kWave, wm = wv >> 1, wn = wv & 1;
    int brow[NI];
#pragma unroll
    for (int ni = 0; ni < NI; ni++) brow[ni] = wn * WN + ni * 16 + (l & 15);
    acc_t acc[MI][NI];
    clear(acc);

    int nv, na;
    wave_share(t.rows, wm, nv, na);
    auto pre = [&] {
        if (tid < t.rows) s_h[tid] = a.a_scale[static_cast<size_t>(t.seg) + t.m0 + tid];
        if (tid < BN) reinterpret_cast<float *>(s_d)[tid] = a.sd[w0 + min(t.n0 + tid, N - 1)];
    };
    run_k_loop<true, false>(nv, src, K, K, 0, smem, wm, brow, acc, na, pre);

    // bf16 rows staged in LDS, 64 columns of each wave column at a time (the K buffers are
    // free after the loop), and written as 16-byte chunks.  The terms of a
    // token's sum are rounded to bf16 here (2^-9, a fifth of the codes' own
    // error) since in fp32 they would be most of what the layer moves: the
    // sum over them is fp32.
    constexpr int CH = 128 / 8;
    uint16_t *out = a.out;
#pragma unroll
    for (int part = 0; part < WN / 64; part++) {
#pragma unroll
        for (int mi = 0; mi < MI; mi++) {
            const int r = block_row(wm, mi) + (l & 15);
            const float hs = s_h[min(r, t.rows - 1)];
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int ni = part * 4 + q;
                const f32x4 cd = s_d[(wn * WN + ni * 16) / 4 + (l >> 4)];
                u16x4 o;
#pragma unroll
                for (int v = 0; v < 4; v++)
                    o[v] = f32_to_bf16_bits(static_cast<float>(acc[mi][ni][v]) * (hs * cd[v]));
                *reinterpret_cast<u16x4 *>(smem + r * OUT_PITCH + wn * 64 + q * 16 + 4 * (l >> 4)) = o;
            }
        }
        __syncthreads();
#pragma unroll 4
        for (int i = tid; i < BM * CH; i += NT) {
            const int r = i / CH, c = (i % CH) * 8;
            const int col = t.n0 + (c >> 6) * WN + part * 64 + (c & 63);
            if (r >= t.rows || col >= N) continue;
            const u32x4 v = *reinterpret_cast<const u32x4 *>(smem + r * OUT_PITCH + c);
            *reinterpret_cast<u32x4 *>(out + (static_cast<size_t>(t.seg) + t.m0 + r) * N + col) = v;
        }
        if (part + 1 < WN / 64) __syncthreads();
    }
}

}  // namespace

hipError_t OCC_NAMED(launch_gemm_up8)(const Up8Args &a, size_t max_m_tiles, hipStream_t s) {
    Up8Args b = a;
    const int n_tiles = static_cast<int>(ceil_div(a.N, FT));
    if (!a.seg_off) {
        b.m_tiles = dense_row_tiles(a.M, n_tiles);
        max_m_tiles = static_cast<size_t>(b.m_tiles);
    }
    const unsigned grid = grid_for(max_m_tiles, n_tiles);
    if (grid == 0) return hipSuccess;
    OCC_NAMED(k_gemm_up8)<<<grid, NT, 0, s>>>(b);
    return hipGetLastError();
}

hipError_t OCC_NAMED(launch_gemm_down8)(const Down8Args &a, size_t max_m_tiles, hipStream_t s) {
    Down8Args b = a;
    const int n_tiles = static_cast<int>(ceil_div(a.N, BN));
    if (!a.seg_off) {
        b.m_tiles = dense_row_tiles(a.M, n_tiles);
        max_m_tiles = static_cast<size_t>(b.m_tiles);
    }
    const unsigned grid = grid_for(max_m_tiles, n_tiles);
    if (grid == 0) return hipSuccess;
    OCC_NAMED(k_gemm_down8)<<<grid, NT, 0, s>>>(b);
    return hipGetLastError();
}

}  // namespace occ
