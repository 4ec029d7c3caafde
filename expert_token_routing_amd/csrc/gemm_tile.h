// The row-tile GEMM on gfx950's matrix cores that the bf16 kernels
// (gemm_bf16.hip) and the int8 kernels (gemm_int8.hip) are built around: the
// tile's place in a launch, its direct global->LDS loads and its K loop.  The
// includer adds the operands' addresses and the epilogues.  Tiling and
// scheduling are described in gemm_bf16.hip, where they were measured.
#pragma once

#include <algorithm>

#include "launch.h"

namespace occ {
namespace {

// The matrix instruction of the build: 16 x 16 outputs, 64 bytes of K a step,
// 16 bytes of each operand a lane.  The tile moves bytes and does not care
// which: K and row pitches count 2-byte units (one bf16 value or two int8).
#ifndef OCC_GEMM_INT8
#define OCC_GEMM_INT8 0
#endif
#if OCC_GEMM_INT8
typedef __attribute__((ext_vector_type(4))) int frag_t;
typedef __attribute__((ext_vector_type(4))) int acc_t;
__device__ __forceinline__ acc_t mma(frag_t a, frag_t b, acc_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}
#else
typedef __attribute__((ext_vector_type(8))) __bf16 frag_t;
typedef f32x4 acc_t;
__device__ __forceinline__ acc_t mma(frag_t a, frag_t b, acc_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
#endif
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

#ifndef OCC_GEMM_BK
#define OCC_GEMM_BK 64
#endif
#ifndef OCC_GEMM_WG_PER_CU
#define OCC_GEMM_WG_PER_CU 1
#endif
#ifndef OCC_XCD_MAP
#define OCC_XCD_MAP 1
#endif
// One source, several builds: kGemmBmBf16-row tiles unless the includer
// defines another height (and, for the dense build, four waves and the
// pipelined K loop, OCC_GEMM_PIPE), each with suffixed kernel and launcher
// names.
#ifndef OCC_GEMM_TILE_M
#define OCC_GEMM_TILE_M kGemmBmBf16
#endif
#ifndef OCC_GEMM_SUFFIX
#define OCC_GEMM_SUFFIX
#endif
#define OCC_CAT2(a, b) a##b
#define OCC_CAT(a, b) OCC_CAT2(a, b)
#define OCC_NAMED(name) OCC_CAT(name, OCC_GEMM_SUFFIX)
constexpr int BM = OCC_GEMM_TILE_M;  // rows (tokens) per tile
#ifndef OCC_GEMM_TILE_N
#define OCC_GEMM_TILE_N 256
#endif
constexpr int BN = OCC_GEMM_TILE_N;  // MFMA columns per tile
constexpr int BK = OCC_GEMM_BK;   // K slice
#ifndef OCC_GEMM_NT
#define OCC_GEMM_NT 512
#endif
constexpr int NT = OCC_GEMM_NT;          // threads: (NT/128) x 2 waves
constexpr int WAVES_M = NT / kWave / 2;
constexpr int WN = BN / 2;               // columns of a wave
constexpr int MI = (BM / 16 + WAVES_M - 1) / WAVES_M, NI = WN / 16;  // its 16 x 16 blocks
constexpr int CHUNKS = BK / 8;           // 16-byte chunks per LDS row
constexpr int ROWS_PER_PASS = NT / CHUNKS;  // rows one pass of the workgroup moves
constexpr int A_LD = (BM + ROWS_PER_PASS - 1) / ROWS_PER_PASS;
constexpr int B_LD = BN / ROWS_PER_PASS;
constexpr int STAGE = (BM + BN) * BK;    // 2-byte units per LDS buffer
#ifndef OCC_GEMM_NSTAGE
#define OCC_GEMM_NSTAGE 2
#endif
constexpr int NSTAGE = OCC_GEMM_NSTAGE;  // LDS ring filled by direct global->LDS loads
static_assert(NSTAGE >= 2 && NSTAGE <= 5, "ring depth");
static_assert(BK == 32 || BK == 64, "a wave load moves 1 KB: 16 rows of 64 bytes or 8 of 128");
constexpr int OUT_PITCH = 128 + 8;       // up epilogue staging row (elements)
constexpr int RING = NSTAGE * STAGE;     // its elements
static_assert(RING * 2 * OCC_GEMM_WG_PER_CU <= 160 * 1024, "LDS");
static_assert(MI * WAVES_M * 16 * OUT_PITCH <= RING, "epilogue staging fits in the K buffers");

// Chunk c of row r sits at chunk slot c ^ ((r >> 1) mod chunks-per-row).  A
// 16-byte fragment read covers 16 consecutive rows at one logical chunk;
// measured on gfx950 (one workgroup timing ds_read_b128 patterns), this key
// reads such a fragment without bank conflicts for both 64- and 128-byte
// rows, while r mod 4 or (r >> 2) mod 4 on 64-byte rows cost 35-45% more
// LDS time.
__device__ __forceinline__ int swz_key(int row) { return row >> 1; }
__device__ __forceinline__ int swz(int row, int chunk) { return row * BK + ((chunk ^ (swz_key(row) & (BK / 8 - 1))) << 3); }

// The K chunk of tile row `row` that this thread fetches.  Thread t moves
// rows (t / CHUNKS) + i * ROWS_PER_PASS, i.e. wave w owns 16-row groups; the
// direct loads write LDS slot t % CHUNKS of the row, so the thread fetches
// the logical chunk that the swizzle puts in that slot.
__device__ __forceinline__ int fetch_chunk(int row) {
    const int c = threadIdx.x % CHUNKS;
    return c ^ (swz_key(row) & (CHUNKS - 1));
}

// Workgroup -> (row tile, column tile).  Returns false when there is no tile.
__device__ __forceinline__ bool map_tile(int m_tiles, int n_tiles, int &tm, int &tn) {
    const int total = m_tiles * n_tiles;
    const int per = (total + 7) >> 3;
    const int b = blockIdx.x, idx = b >> 3;
    if (idx >= per) return false;
#if OCC_XCD_MAP
    const int logical = (b & 7) * per + idx;
#else
    const int logical = b;
#endif
    if (logical >= total) return false;
    tm = logical / n_tiles;
    tn = logical - tm * n_tiles;
    return true;
}

// Order of the tiles of one expert (or of a dense product): an r x c grid of
// row x column tiles is walked in bands of OCC_GEMM_BAND row tiles, and
// inside a band column by column, so the 32 workgroups an XCD runs at a time
// hold 8 row tiles x 4 column tiles of one band (448 KB of distinct operand
// bytes per 64-deep K slice at 320 x 256 tiles) rather than one row tile x 32
// column tiles (the row-major order of a dense product: 1.06 MB) or, for an
// expert of 14 row tiles walked column by column, 14 x 2-3 (650 KB).
// Measured (bands of 1, 2, 4, 8 and unbounded): 8 is best for the
// up-projection, though by little -- the Qwen-shaped layer's step -1.5%, the
// OLMoE- and DeepSeek-shaped ones -0.5% against unbounded bands -- so L2
// reuse is not what bounds these GEMMs.  The routed down-projection (8
// column tiles of d = 2048) takes bands of 16, which for these batches'
// experts of at most 14 row tiles is column by column over the whole expert:
// against 8, 2% faster on the Qwen-shaped and pruned OLMoE batches, even on
// the others (bands of 2 and 4 slower); dense launches keep 8 (the
// Qwen-shaped shared down-projection measured 8% slower with 16).  Local
// index `local` -> (row tile lm, column tn).
#ifndef OCC_GEMM_BAND
#define OCC_GEMM_BAND 8
#endif
constexpr int kBandDown = 16;
__device__ __forceinline__ void band_order(int local, int r, int c, int &lm, int &tn, int B = OCC_GEMM_BAND) {
    const int band = local / (B * c);
    const int rb0 = band * B;
    const int rb = min(B, r - rb0);
    const int idx = local - band * B * c;
    tn = idx / rb;
    lm = rb0 + idx - tn * rb;
}

struct Tile {
    int e;     // expert
    int seg;   // first row of the expert's segment
    int m0;    // first row of the tile inside the segment
    int rows;  // valid rows in the tile (at most BM)
    int n0;    // first column (output feature) of the tile
    int first; // phase 3: the tile's first `first` rows are first contributors
};

// A segment of len rows in n = ceil(len / BM) row tiles: its ceil(len / 16)
// MFMA row blocks are dealt out as evenly as possible (the first B mod n
// tiles take one more), so an expert of 1030 rows is four tiles of 272, 256,
// 256 and 246 rows rather than four full tiles and one of 6 rows.  Tile j's
// first row and row count.
__device__ __forceinline__ void split_rows(int len, int n, int j, int &m0, int &rows) {
    const int B = (len + 15) >> 4, base = B / n, rem = B - base * n;
    m0 = 16 * (j * base + min(j, rem));
    rows = min(16 * (base + (j < rem ? 1 : 0)), len - m0);
}

// Routed tiles walk expert segments [seg_off[p], seg_off[p+1]) -- all rows
// (phases 0 and 3), the first first_cnt[p] rows (phase 1) or the rest (phase 2) --
// with the phase's row-tile schedule tile_off; shared tiles (seg_off NULL)
// walk M rows.
__device__ __forceinline__ bool tile_of(const int32_t *seg_off, const int32_t *tile_off, int M,
                                        int m_tiles_dense, int Ne, const PlaceTab &tab,
                                        int n_tiles, int n_step, Tile &t,
                                        const int32_t *first_cnt = nullptr, int phase = 0,
                                        int band = OCC_GEMM_BAND) {  // routed launches
    int tm, tn;
    if (seg_off) {
        const int m_tiles = tile_off[Ne];
        if (!map_tile(m_tiles, n_tiles, tm, tn)) return false;
        const int p = tile_owner(tile_off, Ne, tm);
        if (phase != 2) {
            // Bands of row tiles, column tiles outermost inside a band: the
            // workgroups that run together on an XCD then share fewer weight
            // column tiles (the larger share of the L2 misses).  Column tiles
            // outermost was measured on the OLMoE-shaped layer at -4% in the
            // up-projection and in the first merge phase against row order;
            // the atomic phase is faster in row order.
            int lm;
            band_order((tm - tile_off[p]) * n_tiles + tn, tile_off[p + 1] - tile_off[p], n_tiles,
                       lm, tn, band);
            tm = tile_off[p] + lm;
        }
        const int seg0 = seg_off[p], len = seg_off[p + 1] - seg0;
        const int nf = phase == 1 || phase == 2 ? first_cnt[p] : 0;
        t.e = tab.expert[p];
        t.seg = phase == 2 ? seg0 + nf : seg0;
        split_rows(phase == 1 ? nf : len - nf, tile_off[p + 1] - tile_off[p], tm - tile_off[p],
                   t.m0, t.rows);
        t.first = phase == 3 ? first_cnt[p] - t.m0 : 0;
    } else {
        const int m_tiles = m_tiles_dense;
        if (!map_tile(m_tiles, n_tiles, tm, tn)) return false;
        band_order(tm * n_tiles + tn, m_tiles, n_tiles, tm, tn);
        t.e = 0;
        t.seg = 0;
        split_rows(M, m_tiles, tm, t.m0, t.rows);
        t.first = 0;
    }
    t.n0 = tn * n_step;
    return true;
}

// The tile's 16-row blocks are dealt to the wave rows in turn: wave row wm
// owns blocks wm, wm + WAVES_M, ...; its mi-th block starts at this row.
// The two wave rows that share a SIMD (wm and wm + 2) then hold
// ceil(blocks / 2) blocks between them whatever the tile's height.
__device__ __forceinline__ int block_row(int wm, int mi) { return (wm + WAVES_M * mi) * 16; }

// NV: the wave's blocks that hold rows (the others are not multiplied).
// SWAP issues the MFMA with the operands' roles exchanged, which yields the
// transposed 16 x 16 block: lane l then holds row (l & 15) and the four
// consecutive columns 4 (l >> 4) .. + 3 (the plain layout gives a lane four
// rows of one column).
template <int NV, bool SWAP>
__device__ __forceinline__ void mma_slice(const uint16_t *sA, const uint16_t *sB, int wm,
                                          const int (&brow)[NI], acc_t (&acc)[MI][NI]) {
    if constexpr (NV > 0) {
        const int l = lane_id();
#pragma unroll
        for (int ks = 0; ks < BK / 32; ks++) {
            const int chunk = ks * 4 + (l >> 4);
            frag_t a[NV], b[NI];
#pragma unroll
            for (int mi = 0; mi < NV; mi++)
                a[mi] = *reinterpret_cast<const frag_t *>(sA + swz(block_row(wm, mi) + (l & 15), chunk));
#pragma unroll
            for (int ni = 0; ni < NI; ni++)
                b[ni] = *reinterpret_cast<const frag_t *>(sB + swz(brow[ni], chunk));
            // The matrix-core burst runs at raised wave priority: of the two
            // waves sharing a SIMD, the one whose MFMAs are ready issues
            // first and the other's fragment reads fall in between
            // (up-projection -2% on the OLMoE-shaped batch).
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int mi = 0; mi < NV; mi++)
#pragma unroll
                for (int ni = 0; ni < NI; ni++)
                    acc[mi][ni] = SWAP ? mma(b[ni], a[mi], acc[mi][ni]) : mma(a[mi], b[ni], acc[mi][ni]);
            __builtin_amdgcn_s_setprio(0);
        }
    }
}

// Direct global->LDS load of 16 bytes per lane (global_load_lds_dwordx4):
// lane l writes LDS bytes [m0 + 16 l, m0 + 16 l + 16).  m0 must be
// wave-uniform.  Issued as inline assembly because the compiler's builtin
// does not model the LDS write; completion is tracked with vmcnt below.  The
// LDS address is an input operand bound to M0 ("{m0}"), so the compiler
// itself writes M0 before the instruction and knows the register is live
// (M0 is reserved and may not be named as a clobber); the s_nop is the wait
// state between that write and the load.
__device__ __forceinline__ void dma16(const void *g, uint32_t m0) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(g), "{m0}"(m0)
                 : "memory");
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// Wait until at most n (wave-uniform, 0 <= n <= N) loads are in flight; the
// count is an immediate of the instruction, hence the chain.
template <int N>
__device__ __forceinline__ void wait_vmcnt_le(int n) {
    if constexpr (N == 0) {
        wait_vmcnt<0>();
    } else {
        if (n >= N) wait_vmcnt<N>();
        else wait_vmcnt_le<N - 1>(n);
    }
}

#ifndef OCC_GEMM_PIPE
#define OCC_GEMM_PIPE 0
#endif

// Where a thread's direct loads read: its A rows (the tile's rows, gathered)
// and its B rows (weight rows), at the thread's fetch chunk.  a_at(i, k0) is
// load slot i's A address at K offset k0, b_at(i, bo) slot i's B address at
// B offset bo.
struct PtrSrc {  // one 64-bit address per slot
    const uint16_t *a[A_LD], *b[B_LD];
    __device__ const uint16_t *a_at(int i, int k0) const { return a[i] + k0; }
    __device__ const uint16_t *b_at(int i, size_t bo) const { return b[i] + bo; }
};
// K loop shared by both GEMMs; src gives the direct loads' addresses.  A ring of NSTAGE LDS buffers is filled
// by direct loads: slice kt+NSTAGE-1 is issued right after the barrier that
// opens slice kt, so each load has NSTAGE-1 slices of MFMA work to land,
// and the barrier also certifies that every wave has finished reading the
// buffer it overwrites (slice kt-1's).  B is laid out as blocks of ksp-wide
// K ranges, blk elements apart (the shared experts' down weights); one block
// (ksp = K) is the plain case.
// The wave issues only its first na A loads per slice (the 8-row groups
// that hold rows; the LDS rows it skips keep stale values, which reach only
// output rows that are never stored) and multiplies its first NV blocks.
// pre() runs once the first slices are issued: per-row tables the epilogue
// needs are loaded there, their latency hidden under those slices' (the
// loop's first barrier publishes what it writes to LDS).
#if !OCC_GEMM_PIPE
template <int NV, bool SWAP, bool UP, class Src, class Pre>
__device__ __forceinline__ void k_loop(const Src &src, int K, int ksp, size_t blk, uint16_t *smem,
                                       int wm, const int (&brow)[NI], acc_t (&acc)[MI][NI], int na,
                                       Pre &pre) {
    constexpr int LOADS = A_LD + B_LD;
    const int per_slice = na + B_LD;  // loads the wave issues per slice
    const int nk = (K + BK - 1) / BK;
    const int w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<size_t>(smem));
    auto issue = [&](int kt) {
        const int k0 = kt * BK;
        const size_t bo = ksp == K ? static_cast<size_t>(k0)
                                   : static_cast<size_t>(k0 / ksp) * blk + static_cast<size_t>(k0 % ksp);
        const uint32_t st = lds0 + static_cast<uint32_t>((kt % NSTAGE) * STAGE * 2);
#pragma unroll
        for (int i = 0; i < A_LD; i++)
            if (i < na)
                dma16(src.a_at(i, k0), __builtin_amdgcn_readfirstlane(st + (i * (NT / kWave) + w) * kWave * 16));
#pragma unroll
        for (int i = 0; i < B_LD; i++)
            dma16(src.b_at(i, bo), __builtin_amdgcn_readfirstlane(st + BM * BK * 2 + (i * (NT / kWave) + w) * kWave * 16));
    };
    constexpr int D = NSTAGE - 1;  // slices in flight ahead of the one consumed
    for (int kt = 0; kt < D && kt < nk; kt++) issue(kt);
    pre();
    for (int kt = 0; kt < nk; kt++) {
        // Slices kt+1 .. min(kt+D, nk)-1 may stay in flight.
        const int ahead = min(kt + D, nk) - 1 - kt;
        wait_vmcnt_le<(D - 1) * LOADS>(ahead * per_slice);
        __syncthreads();
        if (kt + D < nk) issue(kt + D);
        uint16_t *buf = smem + (kt % NSTAGE) * STAGE;
        mma_slice<NV, SWAP>(buf, buf + BM * BK, wm, brow, acc);
    }
    __syncthreads();
}
#endif

#if OCC_GEMM_PIPE
// The pipelined K loop of the four-wave build (gemm_bf16_dense.hip: one
// wave per SIMD, 128 x 128 per wave, 256 accumulators per lane).  With no
// second wave on the SIMD to fill the gaps, the loop is software-pipelined
// inside the wave: the fragments of a 32-deep step are double-buffered in
// registers, so the next step's LDS reads, and the next slice's direct
// loads, are issued between the current step's MFMAs.  One barrier per
// 64-deep slice, after the slice's first step, once the next slice has
// landed; it also certifies that every wave has read the slice whose buffer
// the following loads overwrite.  Per 256 x 256 x 32 step a wave reads 16
// fragments for 64 MFMAs (0.25 per MFMA against 0.33 in the eight-wave
// build), and every wave issues all of its load slots (rows past the
// tile's repeat its last row), since a load skipped under a branch would
// split the MFMA stream into blocks.
static_assert(NT == 256 && NSTAGE == 2 && BK == 64, "pipelined loop: 4 waves, two 64-deep slots");

// Fragment registers of one 32-deep step: the wave's NV A blocks and NI B
// blocks; the loop keeps two sets, one multiplied while the other is read.
template <int NV>
struct Frags {
    frag_t a[NV > 0 ? NV : 1];
    frag_t b[NI];
};

// Fragment reads with constant offsets: every block's 16 rows start at a
// multiple of 16, so the swizzle key of a lane's row is (l & 15) >> 1 for
// all of them and a lane's offset inside any block is the same.  `ab` / `bb`
// point at that lane offset in the wave's first A / B block of one buffer
// and one 32-deep half; block i then sits a constant number of rows further
// (A: WAVES_M * 16 i; B: the up-projection pairs gate and up blocks 128
// rows apart, the down-projection's are consecutive), so the compiler folds
// it into the read's immediate offset.  Read r of a step: B blocks first,
// since the MFMAs take every B block with A block 0 first.
template <bool UP>
__device__ constexpr int b_block_off(int ni) {
    return UP ? (ni < NI / 2 ? 0 : 128) + (ni % (NI / 2)) * 16 : ni * 16;
}
template <int NV, bool UP>
__device__ __forceinline__ void frag_read(Frags<NV> &f, int r, const uint16_t *ab, const uint16_t *bb) {
    if (r < NI)
        f.b[r] = *reinterpret_cast<const frag_t *>(bb + b_block_off<UP>(r) * BK);
    else
        f.a[r - NI] = *reinterpret_cast<const frag_t *>(ab + WAVES_M * 16 * (r - NI) * BK);
}

// One 32-deep step: the NV x NI MFMAs on `cur`, with the reads of the next
// step's fragments (into `nxt`, when READ) spread over its first three
// quarters and the `nd` direct loads dma(d) over all of it, at most one of
// each after an MFMA (those that find no MFMA follow the last).  A
// scheduling barrier after each MFMA keeps that order.  (The loads issued
// in the step's first quarter or half instead were measured 2-5% slower in
// both products.)
template <int NV, bool SWAP, bool UP, bool READ, class Dma>
__device__ __forceinline__ void pipe_step(const Frags<NV> &cur, Frags<NV> &nxt, const uint16_t *ab,
                                          const uint16_t *bb, acc_t (&acc)[MI][NI], int nd,
                                          Dma &dma) {
    constexpr int NM = NV * NI, NR = NV + NI, ND = A_LD + B_LD;
    constexpr int RSPAN = NM * 3 / 4 > NR ? NM * 3 / 4 : NR;  // read r after MFMA r * RSPAN / NR
    constexpr int DSPAN = NM > ND ? NM : ND;                  // load d after MFMA d * DSPAN / ND
#pragma unroll
    for (int m = 0; m < NM; m++) {
        const int mi = m / NI, ni = m % NI;
        acc[mi][ni] = SWAP ? mma(cur.b[ni], cur.a[mi], acc[mi][ni]) : mma(cur.a[mi], cur.b[ni], acc[mi][ni]);
        const int r = (m * NR + RSPAN - 1) / RSPAN;
        if (READ && r < NR && r * RSPAN / NR == m) frag_read<NV, UP>(nxt, r, ab, bb);
        const int d = (m * ND + DSPAN - 1) / DSPAN;
        if (d < ND && d * DSPAN / ND == m && d < nd) dma(d);
        __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (READ) {
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (r * RSPAN / NR >= NM) frag_read<NV, UP>(nxt, r, ab, bb);
    }
#pragma unroll
    for (int d = 0; d < ND; d++)
        if (d * DSPAN / ND >= NM && d < nd) dma(d);
}

template <int NV, bool SWAP, bool UP, class Src, class Pre>
__device__ __forceinline__ void k_loop(const Src &src, int K, int ksp, size_t blk, uint16_t *smem,
                                       int wm, const int (&brow)[NI], acc_t (&acc)[MI][NI], int,
                                       Pre &pre) {
    constexpr int LOADS = A_LD + B_LD;
    const int nk = (K + BK - 1) / BK;
    const int w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int c0 = lane_id() >> 4;
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<size_t>(smem));
    // Direct load d of slice kt: A rows (d < A_LD) or B rows.  The B offset
    // of the slice (blocks of ksp along K) is computed once per slice.
    auto b_off = [&](int kt) {
        const int k0 = kt * BK;
        return ksp == K ? static_cast<size_t>(k0)
                        : static_cast<size_t>(k0 / ksp) * blk + static_cast<size_t>(k0 % ksp);
    };
    auto load = [&](int kt, size_t bo, int d) {
        const uint32_t st = lds0 + static_cast<uint32_t>((kt & 1) * STAGE * 2);
        if (d < A_LD) {
            dma16(src.a_at(d, kt * BK), __builtin_amdgcn_readfirstlane(st + (d * (NT / kWave) + w) * kWave * 16));
        } else {
            const int i = d - A_LD;
            dma16(src.b_at(i, bo), __builtin_amdgcn_readfirstlane(st + BM * BK * 2 + (i * (NT / kWave) + w) * kWave * 16));
        }
    };
    for (int d = 0; d < LOADS; d++) load(0, b_off(0), d);
    pre();
    if (nk > 1)
        for (int d = 0; d < LOADS; d++) load(1, b_off(1), d);
    wait_vmcnt_le<LOADS>(nk > 1 ? LOADS : 0);
    __syncthreads();
    // Lane offsets of the two 32-deep halves of a slice (see frag_read).
    const int key = (lane_id() & 15) >> 1;
    const int h0 = (c0 ^ key) << 3, h1 = ((4 + c0) ^ key) << 3;
    const int ao = (wm * 16 + (lane_id() & 15)) * BK, bo0 = (BM + brow[0]) * BK;
    auto ab = [&](int slot, int h) { return smem + slot * STAGE + ao + h; };
    auto bb = [&](int slot, int h) { return smem + slot * STAGE + bo0 + h; };
    Frags<NV> f0, f1;
#pragma unroll
    for (int r = 0; r < NV + NI; r++) frag_read<NV, UP>(f0, r, ab(0, h0), bb(0, h0));
    auto none = [](int) {};
    int kt = 0;
    for (; kt + 2 < nk; kt++) {  // slice kt; slice kt+2's loads go out during its second step
        const int slot = kt & 1;
        pipe_step<NV, SWAP, UP, true>(f0, f1, ab(slot, h1), bb(slot, h1), acc, 0, none);
        wait_vmcnt<0>();
        __syncthreads();
        const size_t bo = b_off(kt + 2);
        auto dma = [&](int d) { load(kt + 2, bo, d); };
        pipe_step<NV, SWAP, UP, true>(f1, f0, ab(slot ^ 1, h0), bb(slot ^ 1, h0), acc, LOADS, dma);
    }
    if (kt + 1 < nk) {  // the last but one slice: nothing left to load
        const int slot = kt & 1;
        pipe_step<NV, SWAP, UP, true>(f0, f1, ab(slot, h1), bb(slot, h1), acc, 0, none);
        wait_vmcnt<0>();
        __syncthreads();
        pipe_step<NV, SWAP, UP, true>(f1, f0, ab(slot ^ 1, h0), bb(slot ^ 1, h0), acc, 0, none);
        kt++;
    }
    {  // the last slice
        const int slot = kt & 1;
        pipe_step<NV, SWAP, UP, true>(f0, f1, ab(slot, h1), bb(slot, h1), acc, 0, none);
        pipe_step<NV, SWAP, UP, false>(f1, f0, ab(slot, h0), bb(slot, h0), acc, 0, none);
    }
    __syncthreads();
}
#endif

// Runs the K loop with the wave's block count as a constant.
// UP: the B columns are pairs of gate and up blocks.
template <bool SWAP, bool UP = SWAP, int NV = MI, class Src, class Pre>
__device__ __forceinline__ void run_k_loop(int nv, const Src &src, int K, int ksp, size_t blk,
                                           uint16_t *smem, int wm, const int (&brow)[NI],
                                           acc_t (&acc)[MI][NI], int na, Pre &pre) {
    if constexpr (NV == 0) {
        k_loop<0, SWAP, UP>(src, K, ksp, blk, smem, wm, brow, acc, na, pre);
    } else if constexpr (OCC_GEMM_PIPE) {
        // a wave with rows multiplies all of its blocks (those past the
        // tile's rows hold repeated rows whose results are not stored)
        if (nv > 0) k_loop<MI, SWAP, UP>(src, K, ksp, blk, smem, wm, brow, acc, na, pre);
        else k_loop<0, SWAP, UP>(src, K, ksp, blk, smem, wm, brow, acc, na, pre);
    } else {
        if (nv >= NV) k_loop<NV, SWAP, UP>(src, K, ksp, blk, smem, wm, brow, acc, na, pre);
        else run_k_loop<SWAP, UP, NV - 1>(nv, src, K, ksp, blk, smem, wm, brow, acc, na, pre);
    }
}

// The wave's share of a tile of `rows` rows: its blocks that hold rows, and
// its A loads (wave w's load i moves rows i * ROWS_PER_PASS + w * 8 .. + 7)
// that do.
__device__ __forceinline__ void wave_share(int rows, int wm, int &nv, int &na) {
    const int blocks = (rows + 15) >> 4;
    nv = __builtin_amdgcn_readfirstlane(min(MI, max(0, (blocks - wm + WAVES_M - 1) / WAVES_M)));
    const int first = static_cast<int>(threadIdx.x) / kWave * (kWave / CHUNKS);
    na = __builtin_amdgcn_readfirstlane(
        min(A_LD, max(0, (rows - first + ROWS_PER_PASS - 1) / ROWS_PER_PASS)));
}

unsigned grid_for(size_t m_tiles, size_t n_tiles) {
    const size_t total = m_tiles * n_tiles;
    return static_cast<unsigned>(8 * ((total + 7) / 8));
}

// Row tiles of a dense product of M rows against n_tiles column tiles: the
// fewest that hold every row (ceil(M / BM)), raised as far as the launch
// still takes the same number of rounds of the GPU's workgroup slots, so the
// last round is filled with shorter tiles instead of running partly empty
// (the Qwen-shaped layer's shared down-projection: 205 x 8 tiles are 6.4
// rounds of 256 CUs, run as 7; 224 x 8 tiles of 293 rows fill the 7 rounds).
// At most one 16-row block per tile.
int dense_row_tiles(int M, int n_tiles) {
    const int m0 = static_cast<int>(ceil_div(M, BM));
    const long slots = static_cast<long>(compute_units()) * OCC_GEMM_WG_PER_CU;
    if (m0 == 0 || n_tiles == 0 || slots <= 0) return m0;
    const long rounds = (static_cast<long>(m0) * n_tiles + slots - 1) / slots;
    const long m = std::min<long>(rounds * slots / n_tiles, (M + 15) / 16);
    return static_cast<int>(std::max<long>(m0, m));
}

}  // namespace
}  // namespace occ
