// C ABI of the Occult MoE-layer library: argument checks, workspace layout,
// and the stage sequence of the layer (declarations and contracts in occ.h).
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>
#include <vector>

#include "launch.h"

#pragma GCC visibility push(default)
#include "occ.h"
#pragma GCC visibility pop

using namespace occ;

namespace occ {
int compute_units() {
    constexpr int kDevices = 64;
    static int cached[kDevices] = {};  // 0: not read yet
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kDevices) return 256;
    int v = __atomic_load_n(&cached[dev], __ATOMIC_RELAXED);
    if (v == 0) {
        if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            v <= 0)
            v = 256;
        __atomic_store_n(&cached[dev], v, __ATOMIC_RELAXED);
    }
    return v;
}
}  // namespace occ

// The allocation-free forward's workspace: a file-scope device array that
// each GPU holds (at its own address) from the library's load until the
// process ends.  In host code `scratch` is only a stand-in for the symbol;
// its device address on the current GPU is looked up once per device with
// hipGetSymbolAddress (noalloc_scratch below) and that address is what
// kernels receive.  Every call on one GPU uses the same array, so calls that
// overlap on a GPU race.
static __device__ __align__(256) unsigned char scratch[OCC_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

size_t elem_bytes(const occ_layer_desc &D) { return D.dtype == OCC_BF16 ? 2 : 4; }
// The grouped GEMM kernels for a shape.  bf16 batches whose experts average
// fewer than kSmallTileRows rows (T*k < 96*Ne, e.g. decode steps) take the
// 128-row tiles, whose smaller LDS slices leave room for a third ring slot:
// such launches stream the weights from HBM.  The choice is made from the
// shape alone (nothing is read back): an average of 96 keeps the largest
// expert within one 128-row tile at the spread of expert loads seen in
// routed batches (the largest about 1.25x the average), and above it an
// expert's second 128-row tile costs a round of the CUs that one 320-row
// tile avoids (OLMoE shape: 128-row tiles 7% faster at 700 tokens, 5%
// slower at 1000).
struct GemmOps {
    hipError_t (*up)(const UpArgs &, size_t, hipStream_t);
    hipError_t (*down)(const DownArgs &, size_t, hipStream_t);
    int bm;
};
GemmOps gemm_ops(const occ_layer_desc &D) {
    if (D.dtype != OCC_BF16) return {launch_gemm_up_f32, launch_gemm_down_f32, kGemmBmF32};
    if (static_cast<int64_t>(D.T) * D.k < static_cast<int64_t>(kSmallTileRows) * D.Ne)
        return {launch_gemm_up_bf16_m128, launch_gemm_down_bf16_m128, kGemmBmBf16Small};
    return {launch_gemm_up_bf16, launch_gemm_down_bf16, kGemmBmBf16};
}
int tile_rows(const occ_layer_desc &D) { return gemm_ops(D).bm; }
// The routed row-tile schedule fills the up-projection's last round of the
// CUs on the 320-row build (column tiles of 128 features); the other builds
// take ceil(rows / capacity) tiles per expert.
int fill_cols(const occ_layer_desc &D) {
    return gemm_ops(D).up == launch_gemm_up_bf16 ? static_cast<int>(ceil_div(D.F, 128)) : 0;
}

// Dense products (the shared experts) that fill at least kDensePipeRounds
// rounds of the CUs with 256 x 256 tiles take the pipelined four-wave build;
// cols is the product's MFMA output width (the up-projection's gate and up
// columns together).
bool dense_pipelined(const GemmOps &ops, int64_t M, int64_t cols) {
    if (ops.up != launch_gemm_up_bf16) return false;  // fp32, or the decode regime
    const int64_t tiles = ((M + 255) / 256) * ((cols + 255) / 256);
    return tiles >= static_cast<int64_t>(kDensePipeRounds) * compute_units();
}

// Byte offsets of every buffer inside the workspace.  Sized for the worst
// case N_sfd = T * min(k, Nd), so no data-dependent size is read back.
struct Layout {
    size_t logits, ids, w, brim0, sfd_off, epd_off, tile_off, tile_off_first, tile_off_rest, first_cnt,
        chunk_cnt, chunk_base, epd_src, epd_w, tok_epd, down_rows, brim1, brim_end, x_sfd, epd,
        sfd_out, h_sh, y_sh, y_epd;
    // training only (flags & OCC_FLAG_TRAIN): saved pre-activations and the
    // backward pass's buffers
    size_t gu, gu_sh, dy_sfd, dgu, dx_sfd, dw_part, zero_row, bt_all, bt_first, bt_rest, dgu_sh,
        dx_sh, wt_sh, wt_down, dense_seg, dense_tile, wg_part;
    int dw_stride;
    size_t total;
};

constexpr int kBwdTile = 256;  // rows and columns of a backward GEMM tile

Layout layout(const occ_layer_desc &D) {
    const size_t T = D.T, k = D.k, Nd = D.Nd, Ne = D.Ne, d = D.d, F = D.F, es = elem_bytes(D);
    const size_t n = Ne / Nd, nsfd_max = T * std::min(k, Nd), nepd = T * k;
    const size_t nchunks = (T + kBrimChunk - 1) / kBrimChunk, nb = Nd + 2 * Ne;
    Layout L{};
    size_t o = 0;
    auto take = [&o](size_t bytes) {
        const size_t r = o;
        o = align_up(o + std::max<size_t>(bytes, 1));
        return r;
    };
    L.logits = take(T * Ne * 4);
    L.ids = take(nepd * 4);
    L.w = take(nepd * 4);
    L.brim0 = take(Nd * T * 4);
    L.sfd_off = take((Nd + 1) * 4);
    L.epd_off = take((Ne + 1) * 4);
    L.tile_off = take((Ne + 1) * 4);
    L.tile_off_first = take((Ne + 1) * 4);
    L.tile_off_rest = take((Ne + 1) * 4);
    L.first_cnt = take(Ne * 4);
    L.chunk_cnt = take(nchunks * nb * 4);
    L.chunk_base = take(nchunks * nb * 4);
    L.epd_src = take(nepd * 4);
    L.epd_w = take(nepd * 4);
    L.tok_epd = take(nepd * 4);
    L.down_rows = take(nepd * 4);
    L.brim1 = take(n * nsfd_max * 4);
    L.brim_end = o;
    L.x_sfd = take(nsfd_max * d * es);
    L.epd = take(nepd * F * es);
    L.sfd_out = take(nsfd_max * d * 4);
    // deterministic merge: every EPD row's fp32 result (the backward reuses
    // it for dx)
    if (D.flags & OCC_FLAG_DETERMINISTIC) L.y_epd = take(nepd * d * 4);
    const size_t Nsh = static_cast<size_t>(D.n_shared) * D.F_shared;
    if (D.n_shared > 0) {
        L.h_sh = take(T * Nsh * es);
        L.y_sh = take(T * d * 4);
    }
    if (D.flags & OCC_FLAG_TRAIN) {
        L.dw_stride = 2 * static_cast<int>((F + kBwdTile - 1) / kBwdTile);
        L.gu = take(nepd * 2 * F * es);
        L.dy_sfd = take(nsfd_max * d * es);
        L.dgu = take(nepd * 2 * F * es);
        L.dx_sfd = take(nsfd_max * d * 4);
        L.dw_part = take(nepd * L.dw_stride * 4);
        L.zero_row = take(std::max<size_t>({d, 2 * F, 2 * Nsh, kBwdTile}) * es);
        L.bt_all = take((Ne + 1) * 4);
        L.bt_first = take((Ne + 1) * 4);
        L.bt_rest = take((Ne + 1) * 4);
        L.dense_seg = take(2 * 4);
        L.dense_tile = take(2 * 4);
        if (D.n_shared > 0) {
            L.gu_sh = take(T * 2 * Nsh * es);
            L.dgu_sh = take(T * 2 * Nsh * es);
            L.dx_sh = take(T * d * 4);
            // the shared gate and up weights transposed, d x 2 F_shared per
            // expert (the input gradient's contraction index contiguous)
            L.wt_sh = take(Nsh * d * 2 * es);
            // and the shared down-projection weights, F_shared x d per
            // expert, for dh_sh = dy W_d read K-contiguous
            L.wt_down = take(Nsh * d * es);
            // the shared weight gradients' split-K partials (dense, K = T)
            const size_t Fs = D.F_shared, nsh = D.n_shared;
            const size_t p3 = wgrad_k_parts(D.n_shared, D.d, D.F_shared, D.T);
            const size_t p4 = wgrad_k_parts(D.n_shared, 2 * D.F_shared, D.d, D.T);
            const size_t need = std::max(p3 > 1 ? p3 * nsh * d * Fs : 0,
                                         p4 > 1 ? p4 * nsh * 2 * Fs * d : 0);
            L.wg_part = need ? take(need * 4) : 0;
        }
    }
    L.total = o;
    return L;
}

occ_status check_desc(const occ_layer_desc *D) {
    if (!D) return OCC_ERR_INVALID_ARG;
    if (D->T < 1 || D->d < 1 || D->Ne < 1 || D->k < 1 || D->Nd < 1 || D->F < 1)
        return OCC_ERR_INVALID_ARG;
    if (D->k > D->Ne || D->Ne % D->Nd != 0) return OCC_ERR_INVALID_ARG;
    if (D->n_shared < 0 || (D->n_shared > 0 && D->F_shared < 1)) return OCC_ERR_INVALID_ARG;
    if (D->dtype != OCC_F32 && D->dtype != OCC_BF16) return OCC_ERR_INVALID_ARG;
    if (D->prune_rule < OCC_PRUNE_OFF || D->prune_rule > OCC_PRUNE_SIMILARITY)
        return OCC_ERR_INVALID_ARG;
    if (D->prune_rule != OCC_PRUNE_OFF &&
        (D->prune_groups < 1 ||
         static_cast<int64_t>(D->prune_groups) * (D->Ne / D->Nd) < D->k))
        return OCC_ERR_INVALID_ARG;
    if (D->flags & ~(OCC_FLAG_TRAIN | OCC_FLAG_DETERMINISTIC)) return OCC_ERR_INVALID_ARG;
    // training keeps bf16 pre-activations for the bf16 backward GEMMs, whose
    // 256-wide tiles need d, F (and F_shared) of at least 256
    if ((D->flags & OCC_FLAG_TRAIN) &&
        (D->dtype != OCC_BF16 || D->d < kBwdTile || D->F < kBwdTile ||
         (D->n_shared > 0 && D->F_shared < kBwdTile)))
        return OCC_ERR_UNSUPPORTED;
    if (D->Ne > kMaxNe || D->Nd > kMaxNd || D->k > kMaxK) return OCC_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(D->T) * D->k >= (1ll << 31) ||
        static_cast<int64_t>(D->T) * D->Nd >= (1ll << 31))
        return OCC_ERR_UNSUPPORTED;
    const int mult = D->dtype == OCC_BF16 ? 64 : 16;
    if (D->d % mult || D->F % mult || (D->n_shared > 0 && D->F_shared % mult))
        return OCC_ERR_UNSUPPORTED;
    if (D->d > (D->dtype == OCC_BF16 ? 8192 : 4096)) return OCC_ERR_UNSUPPORTED;
    return OCC_OK;
}

occ_status make_tab(const occ_layer_desc &D, const int32_t *L, PlaceTab *tab) {
    if (!L) return OCC_ERR_INVALID_ARG;
    const int n = D.Ne / D.Nd;
    bool seen[kMaxNe] = {};
    *tab = PlaceTab{};
    for (int g = 0; g < D.Nd; g++)
        for (int j = 0; j < n; j++) {
            const int e = L[g * n + j];
            if (e < 0 || e >= D.Ne || seen[e]) return OCC_ERR_INVALID_ARG;
            seen[e] = true;
            tab->grp[e] = static_cast<uint8_t>(g);
            tab->slot[e] = static_cast<uint8_t>(j);
            tab->expert[g * n + j] = static_cast<uint8_t>(e);
        }
    tab->Ne = D.Ne;
    tab->Nd = D.Nd;
    tab->n = n;
    return OCC_OK;
}

occ_status check_ws(const occ_layer_desc &D, const void *ws, size_t ws_bytes, size_t need) {
    (void)D;
    if (!ws || reinterpret_cast<uintptr_t>(ws) % kAlign != 0 || ws_bytes < need)
        return OCC_ERR_WORKSPACE;
    return OCC_OK;
}

template <typename T>
T *at(void *ws, size_t off) {
    return reinterpret_cast<T *>(static_cast<char *>(ws) + off);
}

occ_brim brim_view(void *ws, const Layout &L) {
    occ_brim b;
    b.brim0 = at<int32_t>(ws, L.brim0);
    b.sfd_off = at<int32_t>(ws, L.sfd_off);
    b.epd_off = at<int32_t>(ws, L.epd_off);
    b.epd_src = at<int32_t>(ws, L.epd_src);
    b.epd_w = at<float>(ws, L.epd_w);
    b.tok_epd = at<int32_t>(ws, L.tok_epd);
    b.brim1 = at<int32_t>(ws, L.brim1);
    b.down_rows = at<int32_t>(ws, L.down_rows);
    b.first_cnt = at<int32_t>(ws, L.first_cnt);
    b.tile_off = at<int32_t>(ws, L.tile_off);
    return b;
}

BrimBufs brim_bufs(void *ws, const Layout &L) {
    BrimBufs b;
    b.brim0 = at<int32_t>(ws, L.brim0);
    b.sfd_off = at<int32_t>(ws, L.sfd_off);
    b.epd_off = at<int32_t>(ws, L.epd_off);
    b.tile_off = at<int32_t>(ws, L.tile_off);
    b.epd_src = at<int32_t>(ws, L.epd_src);
    b.tok_epd = at<int32_t>(ws, L.tok_epd);
    b.brim1 = at<int32_t>(ws, L.brim1);
    b.epd_w = at<float>(ws, L.epd_w);
    b.down_rows = at<int32_t>(ws, L.down_rows);
    b.first_cnt = at<int32_t>(ws, L.first_cnt);
    b.tile_off_first = at<int32_t>(ws, L.tile_off_first);
    b.tile_off_rest = at<int32_t>(ws, L.tile_off_rest);
    b.chunk_cnt = at<int32_t>(ws, L.chunk_cnt);
    b.chunk_base = at<int32_t>(ws, L.chunk_base);
    return b;
}

occ_status hip_status(hipError_t e) { return e == hipSuccess ? OCC_OK : OCC_ERR_HIP; }

// Row tiles of a dense backward input-gradient product over T rows against
// n_tiles column tiles: ceil(T / kBwdRowTile), raised as far as the launch
// keeps the same number of rounds of the CUs (one workgroup each), so the
// last round is filled with shorter tiles; at most one 16-row block per tile.
int dense_row_tiles_bwd(int T, int n_tiles) {
    const long m0 = (T + kBwdRowTile - 1) / kBwdRowTile, cus = compute_units();
    if (m0 == 0 || n_tiles <= 0) return static_cast<int>(m0);
    const long rounds = (m0 * n_tiles + cus - 1) / cus;
    const long m = std::min<long>(rounds * cus / n_tiles, (T + 15) / 16);
    return static_cast<int>(std::max(m0, m));
}

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices] = {};

occ_status noalloc_scratch(void **out) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return OCC_ERR_HIP;
    if (dev < 0 || dev >= kMaxDevices) return OCC_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void *p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return OCC_ERR_HIP;
        if (reinterpret_cast<uintptr_t>(p) % kAlign != 0) return OCC_ERR_HIP;
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return OCC_OK;
}

#define OCC_TRY(expr)                              \
    do {                                           \
        const occ_status st_ = (expr);             \
        if (st_ != OCC_OK) return st_;             \
    } while (0)

#define OCC_HIP(expr) OCC_TRY(hip_status(expr))

bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Whether each of these arrays (NULL among them) starts on a 16-byte border.
template <typename... P>
bool rows_aligned(P... p) {
    return (aligned_to(p, 16) && ...);
}

// Whether this output (or NULL) is none of these arrays.
template <typename... P>
bool apart(const void *out, P... p) {
    return !out || ((out != static_cast<const void *>(p)) && ...);
}

int row_chunks(const occ_layer_desc &D) { return static_cast<int>(D.d * elem_bytes(D) / 16); }

// Scratch of the operators around the layer: the largest of their needs.
size_t block_ws_bytes(const occ_layer_desc &D) {
    const size_t d = D.d, bf16 = D.dtype == OCC_BF16;
    return align_up(std::max<size_t>(
        {norm_back_blocks(D.T, row_chunks(D)) * 2 * d * 4, balance_part_bytes(D.T, D.Ne),
         static_cast<size_t>(gate_dw_shares(D.T, D.d, D.Ne, bf16)) * D.Ne * d * 4,
         bias_part_bytes(D.T, D.Ne, D.k)}));
}

occ_status check_norm(const occ_layer_desc *desc, const occ_norm_desc *opt) {
    OCC_TRY(check_desc(desc));
    if (!opt || !std::isfinite(opt->eps) || opt->eps < FLT_MIN || !std::isfinite(opt->scale) ||
        opt->gate < OCC_GATE_NONE || opt->gate > OCC_GATE_TOKEN)
        return OCC_ERR_INVALID_ARG;
    return OCC_OK;
}

// The gate's pointer matches its kind: rows of 16-byte chunks or floats.
bool gate_fits(const occ_norm_desc &opt, const void *gate) {
    if (opt.gate == OCC_GATE_NONE) return !gate;
    return gate && aligned_to(gate, opt.gate == OCC_GATE_CHANNEL ? 16 : 4);
}

// The placement table for the router's losses, which use it for the group
// term alone: experts in order when there is none.
occ_status balance_tab(const occ_layer_desc &D, const occ_balance_desc *opt, const int32_t *L,
                       PlaceTab *tab) {
    if (!opt || !std::isfinite(opt->balance) || !std::isfinite(opt->group) ||
        !std::isfinite(opt->z))
        return OCC_ERR_INVALID_ARG;
    if (L) return make_tab(D, L, tab);
    if (opt->group != 0.f) return OCC_ERR_INVALID_ARG;
    int32_t order[kMaxNe];
    for (int e = 0; e < D.Ne; e++) order[e] = e;
    return make_tab(D, order, tab);
}

// The options of routing by scores, for this layer.
occ_status check_score(const occ_layer_desc *desc, const occ_score_desc *opt) {
    OCC_TRY(check_desc(desc));
    if (!opt || desc->prune_rule != OCC_PRUNE_OFF || !std::isfinite(opt->scale) ||
        opt->score < OCC_SCORE_SOFTMAX || opt->score > OCC_SCORE_SIGMOID ||
        (opt->renormalise != 0 && opt->renormalise != 1))
        return OCC_ERR_INVALID_ARG;
    const int n = desc->Ne / desc->Nd;
    if (opt->top_groups < 1 || opt->top_groups > desc->Nd ||
        static_cast<int64_t>(opt->top_groups) * n < desc->k)
        return OCC_ERR_INVALID_ARG;
    if (opt->group_best < 1 || opt->group_best > 2 ||
        (opt->top_groups < desc->Nd && opt->group_best > n))
        return OCC_ERR_INVALID_ARG;
    return OCC_OK;
}

// The 8-bit layer's buffers: the sorted slots, then codes, scales and terms.
struct Int8Layout {
    size_t tok_epd, epd_tok, epd_w, epd_off, tile_off, counts, xq, xs, h, hq, hs, y_epd, y_sh, total;
};

// The row tiles of its products: the capacity, and the columns by which the
// schedule fills the last round (0: not).
bool small_tiles8(const occ_layer_desc &D) {
    return static_cast<int64_t>(D.T) * D.k < static_cast<int64_t>(kSmallTileRows8) * D.Ne;
}
// The shared experts see every token, whatever a routed expert's share of them:
// their products take the low tiles up to this many.  Layer with few routed
// rows, 80-row / 320-row tiles (us): two of F_shared = 1408 (d = 2048) 128 / 140
// at 1024 tokens, 144 / 150 at 1536, 168 / 158 at 2048, 234 / 197 at 4096; one of
// 5632 94 / 101 at 768, 144 / 144 at 1024, 174 / 162 at 1536, 312 / 269 at 4096; one
// of 1024 55 / 62, 95 / 101, 104 / 108, 139 / 131.
constexpr int kSmallTileShared8 = 1536;
int tile_rows8(const occ_layer_desc &D) { return small_tiles8(D) ? kGemmBmInt8Small : kGemmBmBf16; }
int fill_cols8(const occ_layer_desc &D) { return small_tiles8(D) ? 0 : static_cast<int>(ceil_div(D.F, 128)); }

// The most row tiles that a routing can make: E experts with rows have at most
// (slots - E) / capacity + E, and filling the last round of the CUs adds no
// more than that round holds.
size_t most_row_tiles8(const occ_layer_desc &D) {
    const int64_t slots = static_cast<int64_t>(D.T) * D.k, E = std::min<int64_t>(D.Ne, slots);
    const int64_t most = (slots - E) / tile_rows8(D) + E, cols = fill_cols8(D);
    if (cols == 0) return static_cast<size_t>(most);
    const int64_t cus = compute_units(), rounds = (most * cols + cus - 1) / cus;
    return static_cast<size_t>(std::min(std::max(most, rounds * cus / cols), most + kBrimMaxFill));
}

// Whether the layer runs without sorting its slots (int8_few.hip): each slot
// then reads its expert's weights for itself, so what decides is the bytes that
// all slots read, and the three launches that the general path spends on each
// shared expert.  Weights of T tokens where the few-token form stops being the
// faster one (MiB), and us there, few / general: 64 experts of F = 1024, top 8,
// 192 to 240 (4 tokens 42 / 45, 5 51 / 47); 60 of 1408, top 4, 165 to 198; 128 of
// 768, top 8, 216 to 252; with one shared expert 330 (60 of 1408, top 4, one of
// 5632: 5 tokens 75 / 76, 6 83 / 80; 64 of 1024, top 8, one of 1024: 324, 6 tokens
// 65 / 66); with two 462 (64 of 1408, top 6, two of 1408: 6 tokens 86 / 92, 7 100 /
// 103, 8 112 / 106); with four above 768 (64 of 1024, top 4, four of 1024: 16 tokens
// 119 / 125).  Few tokens of small experts win throughout: 128 of 768, d = 1024,
// top 2, with a shared one: 16 tokens 27 / 42.
constexpr int64_t kFewBytes = 200 << 20, kFewSharedBytes = 130 << 20;
constexpr int kFewTokenSlots = 64;
bool few_tokens(const occ_layer_desc &D) {
    const int64_t shared = D.n_shared > 0 ? static_cast<int64_t>(D.n_shared) * D.F_shared : 0;
    const int64_t token = 3ll * D.d * (static_cast<int64_t>(D.k) * D.F + shared);
    return static_cast<int64_t>(D.T) * D.k <= kFewTokenSlots &&
           few_fits(D.d, D.k, D.F, D.n_shared, D.F_shared) &&
           D.T * token <= kFewBytes + D.n_shared * kFewSharedBytes;
}

Int8Layout int8_layout(const occ_layer_desc &D) {
    const size_t T = D.T, d = D.d, F = D.F, nepd = T * D.k, Fs = D.n_shared > 0 ? D.F_shared : 0;
    Int8Layout L{};
    size_t o = 0;
    auto take = [&o](size_t bytes) {
        const size_t r = o;
        o = align_up(o + std::max<size_t>(bytes, 1));
        return r;
    };
    L.tok_epd = take(nepd * 4);
    L.epd_tok = take(nepd * 4);
    L.epd_w = take(nepd * 4);
    L.epd_off = take((D.Ne + 1) * 4);
    L.tile_off = take((D.Ne + 1) * 4);
    L.counts = take(static_cast<size_t>(kSlotsMaxShares) * D.Ne * 4);
    L.xq = take(T * round_line(d));
    L.xs = take(T * 4);
    // the shared experts' hidden states go through the routed ones' buffers first
    // (few tokens keep both)
    L.h = take(few_tokens(D) ? (nepd * F + T * D.n_shared * Fs) * 4 : std::max(nepd * F, T * Fs) * 4);
    L.hq = take(std::max(nepd * round_line(F), T * round_line(Fs)));
    L.hs = take(nepd * 4);
    L.y_epd = take(nepd * d * 2);
    L.y_sh = take(D.n_shared * T * d * 2);
    L.total = o;
    return L;
}

occ_status check_int8(const occ_layer_desc *desc) {
    OCC_TRY(check_desc(desc));
    // K products of codes up to 127 stay below 2^31 up to K = 133144
    constexpr int kMaxWidth = 131072;
    if (desc->dtype != OCC_BF16 || (desc->flags & OCC_FLAG_TRAIN) || desc->F > kMaxWidth ||
        (desc->n_shared > 0 && desc->F_shared > kMaxWidth))
        return OCC_ERR_UNSUPPORTED;
    return OCC_OK;
}

bool experts_given(const occ_int8_experts *e) {
    return e && e->gate && e->up && e->down && e->gate_scale && e->up_scale && e->down_scale &&
           rows_aligned(e->gate, e->up, e->down) && aligned_to(e->gate_scale, 4) &&
           aligned_to(e->up_scale, 4) && aligned_to(e->down_scale, 4);
}

bool apart_from(const void *out, const occ_int8_experts *e) {
    return !e || apart(out, e->gate, e->up, e->down, e->gate_scale, e->up_scale, e->down_scale);
}

}  // namespace

extern "C" {

const char *occ_status_string(occ_status s) {
    switch (s) {
        case OCC_OK: return "OCC_OK";
        case OCC_ERR_INVALID_ARG: return "OCC_ERR_INVALID_ARG";
        case OCC_ERR_UNSUPPORTED: return "OCC_ERR_UNSUPPORTED";
        case OCC_ERR_WORKSPACE: return "OCC_ERR_WORKSPACE";
        case OCC_ERR_HIP: return "OCC_ERR_HIP";
    }
    return "OCC_ERR_UNKNOWN";
}

occ_status occ_workspace_size(const occ_layer_desc *desc, size_t *bytes_host) {
    OCC_TRY(check_desc(desc));
    if (!bytes_host) return OCC_ERR_INVALID_ARG;
    *bytes_host = layout(*desc).total;
    return OCC_OK;
}

occ_status occ_route(const occ_layer_desc *desc, const float *logits,
                     const int32_t *placement_host, int32_t *ids, float *w, void *stream) {
    OCC_TRY(check_desc(desc));
    if (!logits || !ids || !w || desc->prune_rule == OCC_PRUNE_SIMILARITY)
        return OCC_ERR_INVALID_ARG;
    PlaceTab tab;
    OCC_TRY(make_tab(*desc, placement_host, &tab));
    OCC_HIP(launch_route(logits, desc->T, desc->Ne, desc->k, desc->prune_rule,
                         desc->prune_groups, tab, nullptr, ids, w,
                         static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_similarity_accumulate(int32_t T, int32_t Ne, const float *logits, double *gram,
                                     void *stream) {
    if (T < 0 || Ne < 1 || Ne > kMaxNe || !gram || (T > 0 && !logits)) return OCC_ERR_INVALID_ARG;
    OCC_HIP(launch_sim_gram(logits, T, Ne, gram, static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_similarity_rank(int32_t Ne, const double *gram, double *t2, int32_t *rank,
                               void *stream) {
    if (Ne < 1 || Ne > kMaxNe || !gram || !rank) return OCC_ERR_INVALID_ARG;
    OCC_HIP(launch_sim_rank(gram, Ne, t2, rank, static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_route_similarity(const occ_layer_desc *desc, const float *logits,
                                const int32_t *placement_host, const int32_t *sim_rank,
                                int32_t *ids, float *w, void *stream) {
    OCC_TRY(check_desc(desc));
    if (!logits || !ids || !w || !sim_rank || desc->prune_rule != OCC_PRUNE_SIMILARITY)
        return OCC_ERR_INVALID_ARG;
    PlaceTab tab;
    OCC_TRY(make_tab(*desc, placement_host, &tab));
    OCC_HIP(launch_route(logits, desc->T, desc->Ne, desc->k, desc->prune_rule,
                         desc->prune_groups, tab, sim_rank, ids, w,
                         static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_build_brim(const occ_layer_desc *desc, const int32_t *ids, const float *w,
                          const int32_t *placement_host, int dense_brim1, void *workspace,
                          size_t ws_bytes, occ_brim *out_host, void *stream) {
    OCC_TRY(check_desc(desc));
    if (!ids || !w || !out_host) return OCC_ERR_INVALID_ARG;
    PlaceTab tab;
    OCC_TRY(make_tab(*desc, placement_host, &tab));
    const Layout L = layout(*desc);
    OCC_TRY(check_ws(*desc, workspace, ws_bytes, L.brim_end));
    hipStream_t s = static_cast<hipStream_t>(stream);
    int32_t *ids_ws = at<int32_t>(workspace, L.ids);
    float *w_ws = at<float>(workspace, L.w);
    OCC_HIP(launch_sanitize_ids(ids, w, desc->T, desc->k, desc->Ne, ids_ws, w_ws, s));
    OCC_HIP(launch_brim(ids_ws, w_ws, desc->T, desc->k, tab, tile_rows(*desc), fill_cols(*desc),
                        dense_brim1 != 0, brim_bufs(workspace, L), s));
    *out_host = brim_view(workspace, L);
    return OCC_OK;
}

occ_status occ_forward_views(const occ_layer_desc *desc, void *workspace,
                             occ_forward_view *out_host) {
    OCC_TRY(check_desc(desc));
    if (!workspace || !out_host) return OCC_ERR_INVALID_ARG;
    const Layout L = layout(*desc);
    occ_forward_view v;
    v.logits = at<float>(workspace, L.logits);
    v.ids = at<int32_t>(workspace, L.ids);
    v.w = at<float>(workspace, L.w);
    v.brim = brim_view(workspace, L);
    v.x_sfd = at<void>(workspace, L.x_sfd);
    v.epd = at<void>(workspace, L.epd);
    v.sfd_out = at<float>(workspace, L.sfd_out);
    v.h_shared = desc->n_shared > 0 ? at<void>(workspace, L.h_sh) : nullptr;
    v.y_shared = desc->n_shared > 0 ? at<float>(workspace, L.y_sh) : nullptr;
    *out_host = v;
    return OCC_OK;
}

// The layer's stage sequence.  Stage 0 routes `logits` (the desc's rule),
// or first computes them as x w_router^T when w_router is given, or, with
// neither, copies the caller's routing ids_in / w_in.
static occ_status forward(const occ_layer_desc *desc, const void *x, const float *logits,
                          const void *w_router, const int32_t *ids_in, const float *w_in,
                          const int32_t *placement_host, const void *w_gate, const void *w_up,
                          const void *w_down, const void *ws_gate, const void *ws_up,
                          const void *ws_down, void *y, void *workspace, size_t ws_bytes,
                          void *const *stage_events, void *stream) {
    OCC_TRY(check_desc(desc));
    const occ_layer_desc &D = *desc;
    if (!x || !w_gate || !w_up || !w_down || !y) return OCC_ERR_INVALID_ARG;
    const bool routes = logits || w_router;
    if (routes ? D.prune_rule == OCC_PRUNE_SIMILARITY : (!ids_in || !w_in))
        return OCC_ERR_INVALID_ARG;
    if (D.n_shared > 0 && (!ws_gate || !ws_up || !ws_down)) return OCC_ERR_INVALID_ARG;
    if (stage_events)
        for (int i = 0; i <= OCC_STAGE_COUNT; i++)
            if (!stage_events[i]) return OCC_ERR_INVALID_ARG;
    PlaceTab tab;
    OCC_TRY(make_tab(D, placement_host, &tab));
    const Layout L = layout(D);
    OCC_TRY(check_ws(D, workspace, ws_bytes, L.total));

    hipStream_t s = static_cast<hipStream_t>(stream);
    auto mark = [&](int i) -> occ_status {
        if (!stage_events) return OCC_OK;
        return hip_status(hipEventRecord(static_cast<hipEvent_t>(stage_events[i]), s));
    };
    const bool bf16 = D.dtype == OCC_BF16;
    const size_t es = elem_bytes(D);
    const BrimBufs bb = brim_bufs(workspace, L);
    int32_t *ids = at<int32_t>(workspace, L.ids);
    float *w = at<float>(workspace, L.w);
    void *x_sfd = at<void>(workspace, L.x_sfd);
    void *epd = at<void>(workspace, L.epd);
    float *sfd_out = at<float>(workspace, L.sfd_out);
    float *y_sh = D.n_shared > 0 ? at<float>(workspace, L.y_sh) : nullptr;
    const size_t T = D.T;
    const GemmOps ops = gemm_ops(D);
    const size_t bm = ops.bm;
    const size_t routed_tiles = (T * D.k + bm - 1) / bm + D.Ne + kBrimMaxFill;
    const size_t shared_tiles = (T + bm - 1) / bm;

    OCC_TRY(mark(0));
    // Eq. 2: router, behind the gate projection g(x) when its weights are
    // given (or the caller's routing, checked)
    if (w_router) {
        float *lg = at<float>(workspace, L.logits);
        OCC_HIP(launch_gate(x, w_router, D.T, D.d, D.Ne, bf16, lg, s));
        logits = lg;
    }
    if (logits)
        OCC_HIP(launch_route(logits, D.T, D.Ne, D.k, D.prune_rule, D.prune_groups, tab, nullptr,
                             ids, w, s));
    else
        OCC_HIP(launch_sanitize_ids(ids_in, w_in, D.T, D.k, D.Ne, ids, w, s));
    OCC_TRY(mark(1));
    // Algorithms 3 and 5: BRIM_0, BRIM_1 (condensed), GEMM tile schedule
    OCC_HIP(launch_brim(ids, w, D.T, D.k, tab, static_cast<int>(bm), fill_cols(D), 0, bb, s));
    OCC_TRY(mark(2));
    // Small batches (experts averaging fewer than 128 rows) merge in one
    // down-projection launch of atomic adds, whose SFD accumulator rows the
    // dispatch zeroes as it writes the same rows of x_sfd.
    const bool det = D.flags & OCC_FLAG_DETERMINISTIC;
    const bool one_launch = !det && static_cast<int64_t>(D.T) * D.k < 128ll * D.Ne;
    // Algorithm 4: ORI -> SFD
    OCC_HIP(launch_dispatch(x, D.T, D.Nd, static_cast<size_t>(D.d) * es, bb.brim0, x_sfd, s,
                            one_launch ? sfd_out : nullptr, D.d));
    OCC_TRY(mark(3));
    // shared experts: dense SwiGLU over all T tokens, fp32 result
    if (D.n_shared > 0) {
        UpArgs su{};
        su.A = x;
        su.Wg = ws_gate;
        su.Wu = ws_up;
        su.out = at<void>(workspace, L.h_sh);
        su.gu_out = (D.flags & OCC_FLAG_TRAIN) ? at<void>(workspace, L.gu_sh) : nullptr;
        su.M = D.T;
        su.K = D.d;
        su.N = D.n_shared * D.F_shared;
        su.Ne = 1;
        su.tab = tab;
        DownArgs sd{};
        sd.A = su.out;
        sd.W = ws_down;
        sd.out = y_sh;
        sd.M = D.T;
        sd.K = su.N;
        sd.N = D.d;
        sd.Ne = 1;
        sd.k_split = D.F_shared;
        sd.tab = tab;
        if (dense_pipelined(ops, D.T, 2ll * su.N))
            OCC_HIP(launch_gemm_up_bf16_dense(su, shared_tiles, s));
        else
            OCC_HIP(ops.up(su, shared_tiles, s));
        OCC_TRY(mark(4));
        if (dense_pipelined(ops, D.T, sd.N))
            OCC_HIP(launch_gemm_down_bf16_dense(sd, shared_tiles, s));
        else
            OCC_HIP(ops.down(sd, shared_tiles, s));
    } else {
        OCC_TRY(mark(4));
    }
    OCC_TRY(mark(5));
    // Algorithms 6-7: SFD -> EPD, SwiGLU, weight modulation
    UpArgs up{};
    up.A = x_sfd;
    up.a_rows = bb.epd_src;
    up.Wg = w_gate;
    up.Wu = w_up;
    up.seg_off = bb.epd_off;
    up.tile_off = bb.tile_off;
    up.row_w = bb.epd_w;
    up.out = epd;
    up.gu_out = (D.flags & OCC_FLAG_TRAIN) ? at<void>(workspace, L.gu) : nullptr;
    up.M = D.T * D.k;
    up.K = D.d;
    up.N = D.F;
    up.Ne = D.Ne;
    up.tab = tab;
    OCC_HIP(ops.up(up, routed_tiles, s));
    OCC_TRY(mark(6));
    // Algorithm 8: EPD -> SFD, summed inside each group in fp32.  The first
    // contributor to every SFD row stores (so no zero-fill is needed), then
    // the other rows of the group add with atomics.  Small batches are bound
    // by reading the weights, which the two launches would read twice: there
    // the SFD rows were zeroed by the dispatch and one launch adds every row.
    DownArgs dn{};
    dn.A = epd;
    dn.W = w_down;
    dn.seg_off = bb.epd_off;
    dn.rows = bb.down_rows;
    dn.first_cnt = bb.first_cnt;
    dn.dst_rows = bb.epd_src;
    dn.out = sfd_out;
    dn.M = D.T * D.k;
    dn.K = D.F;
    dn.N = D.d;
    dn.Ne = D.Ne;
    dn.k_split = D.F;
    dn.tab = tab;
    if (det) {
        // first contributors store into their SFD rows, the others at their
        // own EPD rows; the merge then adds those to the SFD rows in slot order
        float *y_epd = at<float>(workspace, L.y_epd);
        dn.epd_out = y_epd;
        dn.phase = 3;
        dn.tile_off = bb.tile_off;
        OCC_HIP(ops.down(dn, routed_tiles, s));
        OCC_TRY(mark(7));
        // stage one (SFD rows) and, in the same pass over each token, stage
        // two (Algorithm 9) with the combine's order of additions
        OCC_HIP(launch_merge_slots(y_epd, ids, bb.tok_epd, bb.brim0, tab, D.T, D.k, D.d, sfd_out,
                                   y_sh, y, bf16, s));
    } else if (one_launch) {
        dn.phase = 0;
        dn.tile_off = bb.tile_off;
        OCC_HIP(ops.down(dn, routed_tiles, s));
        OCC_TRY(mark(7));
    } else {
        dn.phase = 1;
        dn.tile_off = bb.tile_off_first;
        OCC_HIP(ops.down(dn, routed_tiles, s));
        OCC_TRY(mark(7));
        dn.phase = 2;
        dn.tile_off = bb.tile_off_rest;
        OCC_HIP(ops.down(dn, routed_tiles, s));
    }
    OCC_TRY(mark(8));
    // Algorithm 9: SFD -> ORI across groups (+ shared experts), cast once
    if (!det) OCC_HIP(launch_combine(sfd_out, bb.brim0, y_sh, D.T, D.Nd, D.d, bf16, y, s));
    OCC_TRY(mark(9));
    return OCC_OK;
}

occ_status occ_moe_forward(const occ_layer_desc *desc, const void *x, const float *logits,
                           const int32_t *placement_host, const void *w_gate, const void *w_up,
                           const void *w_down, const void *ws_gate, const void *ws_up,
                           const void *ws_down, void *y, void *workspace, size_t ws_bytes,
                           void *const *stage_events, void *stream) {
    if (!logits) return OCC_ERR_INVALID_ARG;
    return forward(desc, x, logits, nullptr, nullptr, nullptr, placement_host, w_gate, w_up,
                   w_down, ws_gate, ws_up, ws_down, y, workspace, ws_bytes, stage_events, stream);
}

occ_status occ_moe_forward_noalloc(const occ_layer_desc *desc, const void *x, const float *logits,
                                   const int32_t *placement_host, const void *w_gate,
                                   const void *w_up, const void *w_down, const void *ws_gate,
                                   const void *ws_up, const void *ws_down, void *y,
                                   void *const *stage_events, void *stream) {
    OCC_TRY(check_desc(desc));
    if (!logits) return OCC_ERR_INVALID_ARG;
    // the backward pass reads the training forward's state from a caller
    // workspace, which this variant does not have
    if (desc->flags & OCC_FLAG_TRAIN) return OCC_ERR_UNSUPPORTED;
    if (layout(*desc).total > OCC_NOALLOC_SCRATCH_BYTES) return OCC_ERR_WORKSPACE;
    void *ws = nullptr;
    OCC_TRY(noalloc_scratch(&ws));
    return forward(desc, x, logits, nullptr, nullptr, nullptr, placement_host, w_gate, w_up,
                   w_down, ws_gate, ws_up, ws_down, y, ws, OCC_NOALLOC_SCRATCH_BYTES,
                   stage_events, stream);
}

occ_status occ_moe_forward_gated(const occ_layer_desc *desc, const void *x, const void *w_router,
                                 const int32_t *placement_host, const void *w_gate,
                                 const void *w_up, const void *w_down, const void *ws_gate,
                                 const void *ws_up, const void *ws_down, void *y,
                                 void *workspace, size_t ws_bytes, void *const *stage_events,
                                 void *stream) {
    if (!w_router) return OCC_ERR_INVALID_ARG;
    return forward(desc, x, nullptr, w_router, nullptr, nullptr, placement_host, w_gate, w_up,
                   w_down, ws_gate, ws_up, ws_down, y, workspace, ws_bytes, stage_events, stream);
}

occ_status occ_gate(const occ_layer_desc *desc, const void *x, const void *w_router,
                    float *logits, void *stream) {
    OCC_TRY(check_desc(desc));
    if (!x || !w_router || !logits) return OCC_ERR_INVALID_ARG;
    OCC_HIP(launch_gate(x, w_router, desc->T, desc->d, desc->Ne, desc->dtype == OCC_BF16, logits,
                        static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_block_workspace_size(const occ_layer_desc *desc, size_t *bytes_host) {
    OCC_TRY(check_desc(desc));
    if (!bytes_host) return OCC_ERR_INVALID_ARG;
    *bytes_host = block_ws_bytes(*desc);
    return OCC_OK;
}

occ_status occ_block_norm(const occ_layer_desc *desc, const occ_norm_desc *opt, const void *x,
                          const void *y, const void *w_post, const void *gate, const void *w_pre,
                          void *r, void *h, void *stream) {
    OCC_TRY(check_norm(desc, opt));
    if (!x || !gate_fits(*opt, gate) || !w_pre != !h) return OCC_ERR_INVALID_ARG;
    if (y ? !r : r || w_post || gate || !h) return OCC_ERR_INVALID_ARG;
    if (!rows_aligned(x, y, w_post, w_pre, r, h) || !apart(r, h, w_post, gate, w_pre) ||
        !apart(h, w_post, gate, w_pre))
        return OCC_ERR_INVALID_ARG;
    OCC_HIP(launch_block_norm(x, y, w_post, gate, w_pre, desc->T, desc->d,
                              desc->dtype == OCC_BF16, opt->gate, opt->eps, opt->scale, r, h,
                              static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_block_norm_backward(const occ_layer_desc *desc, const occ_norm_desc *opt,
                                   const void *dr, const void *dh, const void *r, const void *y,
                                   const void *w_post, const void *gate, const void *w_pre,
                                   void *dx, void *dy, float *dw_post, float *dgate,
                                   float *dw_pre, void *workspace, size_t ws_bytes,
                                   void *stream) {
    OCC_TRY(check_norm(desc, opt));
    if (!dx || !gate_fits(*opt, gate) || (!dr && !dh)) return OCC_ERR_INVALID_ARG;
    if (!w_pre != !dh || !w_pre != !dw_pre || !w_post != !dw_post || !gate != !dgate)
        return OCC_ERR_INVALID_ARG;
    if ((w_pre && !r) || ((w_post || gate) && (!y || !dy)) || (y && !dy))
        return OCC_ERR_INVALID_ARG;
    if (!rows_aligned(dr, dh, r, y, w_post, w_pre, dx, dy) || !aligned_to(dw_post, 4) ||
        !aligned_to(dgate, 4) || !aligned_to(dw_pre, 4))
        return OCC_ERR_INVALID_ARG;
    if (!apart(dx, dy, w_post, gate, w_pre, dw_post, dgate, dw_pre) ||
        !apart(dy, w_post, gate, w_pre, dw_post, dgate, dw_pre) ||
        !apart(dw_post, dr, dh, r, y, w_post, gate, w_pre, dgate, dw_pre) ||
        !apart(dw_pre, dr, dh, r, y, w_post, gate, w_pre, dgate) ||
        !apart(dgate, dr, dh, r, y, w_post, w_pre, opt->gate == OCC_GATE_TOKEN ? nullptr : gate) ||
        !apart(workspace, dr, dh, r, y, w_post, gate, w_pre, dx, dy, dw_post, dgate, dw_pre))
        return OCC_ERR_INVALID_ARG;
    OCC_TRY(check_ws(*desc, workspace, ws_bytes, block_ws_bytes(*desc)));
    OCC_HIP(launch_block_norm_back(dr, dh, r, y, w_post, gate, w_pre, desc->T, desc->d,
                                   desc->dtype == OCC_BF16, opt->gate, opt->eps, opt->scale, dx,
                                   dy, dw_post, dgate, dw_pre, static_cast<float *>(workspace),
                                   static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_balance_loss(const occ_layer_desc *desc, const occ_balance_desc *opt,
                            const float *logits, const int32_t *ids, const uint8_t *valid,
                            const int32_t *placement_host, int32_t *counts, float *probs,
                            float *loss, void *workspace, size_t ws_bytes, void *stream) {
    OCC_TRY(check_desc(desc));
    if (!logits || !ids || !counts || !probs || !loss) return OCC_ERR_INVALID_ARG;
    if (!aligned_to(logits, 4) || !aligned_to(ids, 4) || !aligned_to(counts, 4) ||
        !aligned_to(probs, 4) || !aligned_to(loss, 4) || !apart(counts, logits, ids, valid, probs, loss) ||
        !apart(probs, logits, ids, valid, loss) || !apart(loss, logits, ids, valid) ||
        !apart(workspace, logits, ids, valid, counts, probs, loss))
        return OCC_ERR_INVALID_ARG;
    PlaceTab tab;
    OCC_TRY(balance_tab(*desc, opt, placement_host, &tab));
    OCC_TRY(check_ws(*desc, workspace, ws_bytes, block_ws_bytes(*desc)));
    OCC_HIP(launch_balance(logits, ids, valid, desc->T, desc->k, tab, opt->balance, opt->group,
                           opt->z, counts, probs, loss, static_cast<float *>(workspace),
                           static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_balance_backward(const occ_layer_desc *desc, const occ_balance_desc *opt,
                                const float *logits, const uint8_t *valid,
                                const int32_t *placement_host, const int32_t *counts, float dloss,
                                const float *dlogits_in, float *dlogits, void *stream) {
    OCC_TRY(check_desc(desc));
    if (!logits || !counts || !dlogits || !std::isfinite(dloss)) return OCC_ERR_INVALID_ARG;
    if (!aligned_to(logits, 4) || !aligned_to(counts, 4) || !aligned_to(dlogits_in, 4) ||
        !aligned_to(dlogits, 4) || !apart(dlogits, valid, counts))
        return OCC_ERR_INVALID_ARG;
    PlaceTab tab;
    OCC_TRY(balance_tab(*desc, opt, placement_host, &tab));
    OCC_HIP(launch_balance_back(logits, valid, counts, tab, desc->T, desc->k, opt->balance,
                                opt->group, opt->z, dloss, dlogits_in, dlogits,
                                static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_gate_backward(const occ_layer_desc *desc, const float *dlogits, const void *x,
                             const void *w_router, const void *dx_in, void *dx, float *dw_router,
                             void *workspace, size_t ws_bytes, void *stream) {
    OCC_TRY(check_desc(desc));
    if (!dlogits || (!dx && !dw_router)) return OCC_ERR_INVALID_ARG;
    if (dx ? !w_router : !!dx_in) return OCC_ERR_INVALID_ARG;
    if (dw_router && !x) return OCC_ERR_INVALID_ARG;
    if (!aligned_to(dlogits, 4) || !rows_aligned(x, w_router, dx_in, dx, dw_router) ||
        !apart(dx, dlogits, w_router) || !apart(dw_router, dlogits, x, w_router, dx_in, dx) ||
        (dw_router && !apart(workspace, dlogits, x, w_router, dx_in, dx, dw_router)))
        return OCC_ERR_INVALID_ARG;
    if (dw_router) OCC_TRY(check_ws(*desc, workspace, ws_bytes, block_ws_bytes(*desc)));
    const int bf16 = desc->dtype == OCC_BF16;
    hipStream_t s = static_cast<hipStream_t>(stream);
    OCC_HIP(launch_gate_bwd(dlogits, x, w_router, dx_in, desc->T, desc->d, desc->Ne, bf16, dx,
                            static_cast<float *>(workspace), dw_router, s));
    return OCC_OK;
}

occ_status occ_adamw_step(const occ_adamw_desc *opt, const occ_adamw_tensor *tensors_host,
                          int32_t count, const float *dynamic, void *stream) {
    if (!opt || count < 0 || (count > 0 && !tensors_host)) return OCC_ERR_INVALID_ARG;
    // as the fp32 values that the kernel computes with
    const auto finite = [](double v) { return std::isfinite(static_cast<float>(v)); };
    const auto ranged = [&](double v) { return finite(v) && v >= 0.; };
    if ((opt->state != OCC_ADAMW_32BIT && opt->state != OCC_ADAMW_8BIT) ||
        (opt->grad_dtype != OCC_F32 && opt->grad_dtype != OCC_BF16) || !ranged(opt->lr) ||
        !ranged(opt->beta1) || opt->beta1 >= 1. || !ranged(opt->beta2) || opt->beta2 >= 1. ||
        !(static_cast<float>(opt->eps) >= FLT_MIN) || !finite(opt->eps) ||
        !ranged(opt->weight_decay) || !finite(opt->grad_scale) || opt->step < 1 ||
        !aligned_to(dynamic, 4))
        return OCC_ERR_INVALID_ARG;
    const bool q8 = opt->state == OCC_ADAMW_8BIT, gb = opt->grad_dtype == OCC_BF16;
    const size_t ms = q8 ? 1 : 4;
    std::vector<AdamwTensor> list;
    std::vector<const void *> written;  // each once
    constexpr int kOutputs = 6;
    try {
        list.reserve(count);
        written.reserve(static_cast<size_t>(count) * kOutputs);
    } catch (...) {
        return OCC_ERR_UNSUPPORTED;
    }
    for (int i = 0; i < count; i++) {
        const occ_adamw_tensor &t = tensors_host[i];
        if (t.n < 0) return OCC_ERR_INVALID_ARG;
        if (t.n == 0) continue;
        if (t.n > kAdamwMaxElements) return OCC_ERR_UNSUPPORTED;
        if (!t.p || !t.g || !t.m || !t.v || !t.p_out || !t.m_out || !t.v_out)
            return OCC_ERR_INVALID_ARG;
        if (!t.m_scale == q8 || !t.v_scale == q8 || !t.m_scale_out == q8 || !t.v_scale_out == q8)
            return OCC_ERR_INVALID_ARG;
        const auto fits = [&](size_t k) {  // arrays aligned to k elements
            return aligned_to(t.p, 4 * k) && aligned_to(t.g, (gb ? 2 : 4) * k) &&
                   aligned_to(t.m, ms * k) && aligned_to(t.v, ms * k) &&
                   aligned_to(t.p_out, 4 * k) && aligned_to(t.m_out, ms * k) &&
                   aligned_to(t.v_out, ms * k) && aligned_to(t.p_bf16, 2 * k);
        };
        if (!fits(1) || !aligned_to(t.m_scale, 4) || !aligned_to(t.v_scale, 4) ||
            !aligned_to(t.m_scale_out, 4) || !aligned_to(t.v_scale_out, 4))
            return OCC_ERR_INVALID_ARG;
        list.push_back({t.n, t.p, t.g, t.m, t.v, t.m_scale, t.v_scale, t.p_out, t.m_out, t.v_out,
                        t.m_scale_out, t.v_scale_out, t.p_bf16, fits(4)});
        for (const void *out : {static_cast<const void *>(t.p_out), static_cast<const void *>(t.m_out),
                                static_cast<const void *>(t.v_out),
                                static_cast<const void *>(t.m_scale_out),
                                static_cast<const void *>(t.v_scale_out),
                                static_cast<const void *>(t.p_bf16)})
            if (out) written.push_back(out);
    }
    std::sort(written.begin(), written.end());
    if (std::adjacent_find(written.begin(), written.end()) != written.end())
        return OCC_ERR_INVALID_ARG;
    // an array that is read is written by its own new value or not at all
    const auto kept = [&](const void *in, const void *own) {
        return !in || in == own || !std::binary_search(written.begin(), written.end(), in);
    };
    for (const AdamwTensor &t : list)
        if (!kept(t.p, t.p_out) || !kept(t.g, nullptr) || !kept(t.m, t.m_out) ||
            !kept(t.v, t.v_out) || !kept(t.m_scale, t.m_scale_out) ||
            !kept(t.v_scale, t.v_scale_out))
            return OCC_ERR_INVALID_ARG;
    if (!kept(dynamic, nullptr)) return OCC_ERR_INVALID_ARG;
    AdamwStep st;
    const double step = static_cast<double>(opt->step);
    st.lr = static_cast<float>(opt->lr);
    st.beta1 = static_cast<float>(opt->beta1);
    st.one_b1 = static_cast<float>(1. - opt->beta1);
    st.beta2 = static_cast<float>(opt->beta2);
    st.one_b2 = static_cast<float>(1. - opt->beta2);
    st.eps = static_cast<float>(opt->eps);
    st.weight_decay = static_cast<float>(opt->weight_decay);
    st.grad_scale = static_cast<float>(opt->grad_scale);
    st.log_b1 = static_cast<float>(std::log(opt->beta1));
    st.log_b2 = static_cast<float>(std::log(opt->beta2));
    st.c1 = static_cast<float>(-std::expm1(step * std::log(opt->beta1)));
    st.c2_rsqrt = static_cast<float>(1. / std::sqrt(-std::expm1(step * std::log(opt->beta2))));
    st.dynamic = dynamic;
    OCC_HIP(launch_adamw(list.data(), static_cast<int>(list.size()), st, q8, gb,
                         static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_moe_forward_routed(const occ_layer_desc *desc, const void *x, const int32_t *ids,
                                  const float *w, const int32_t *placement_host,
                                  const void *w_gate, const void *w_up, const void *w_down,
                                  const void *ws_gate, const void *ws_up, const void *ws_down,
                                  void *y, void *workspace, size_t ws_bytes,
                                  void *const *stage_events, void *stream) {
    if (!ids || !w) return OCC_ERR_INVALID_ARG;
    return forward(desc, x, nullptr, nullptr, ids, w, placement_host, w_gate, w_up, w_down, ws_gate,
                   ws_up, ws_down, y, workspace, ws_bytes, stage_events, stream);
}

occ_status occ_moe_backward(const occ_layer_desc *desc, const void *dy, const void *x,
                            const float *logits, const int32_t *placement_host,
                            const void *w_gate, const void *w_up, const void *w_down,
                            const void *ws_gate, const void *ws_up, const void *ws_down,
                            void *dx, float *dw_gate, float *dw_up, float *dw_down,
                            float *dws_gate, float *dws_up, float *dws_down, float *dw,
                            float *dlogits, void *workspace, size_t ws_bytes,
                            void *const *stage_events, void *stream) {
    OCC_TRY(check_desc(desc));
    const occ_layer_desc &D = *desc;
    if (!(D.flags & OCC_FLAG_TRAIN)) return OCC_ERR_INVALID_ARG;
    if (!dy || !x || !w_gate || !w_up || !w_down || !dx || !dw_gate || !dw_up || !dw_down)
        return OCC_ERR_INVALID_ARG;
    if (D.n_shared > 0 && (!ws_gate || !ws_up || !ws_down || !dws_gate || !dws_up || !dws_down))
        return OCC_ERR_INVALID_ARG;
    if (dlogits && !logits) return OCC_ERR_INVALID_ARG;
    if (stage_events)
        for (int i = 0; i <= OCC_BSTAGE_COUNT; i++)
            if (!stage_events[i]) return OCC_ERR_INVALID_ARG;
    PlaceTab tab;
    OCC_TRY(make_tab(D, placement_host, &tab));
    const Layout L = layout(D);
    OCC_TRY(check_ws(D, workspace, ws_bytes, L.total));

    hipStream_t s = static_cast<hipStream_t>(stream);
    auto mark = [&](int i) -> occ_status {
        if (!stage_events) return OCC_OK;
        return hip_status(hipEventRecord(static_cast<hipEvent_t>(stage_events[i]), s));
    };
    const size_t es = elem_bytes(D), T = D.T, d = D.d, F = D.F;
    const size_t Nsh = static_cast<size_t>(D.n_shared) * D.F_shared;
    const BrimBufs bb = brim_bufs(workspace, L);
    const void *x_sfd = at<void>(workspace, L.x_sfd);
    const void *h = at<void>(workspace, L.epd);
    void *dy_sfd = at<void>(workspace, L.dy_sfd);
    void *dgu = at<void>(workspace, L.dgu);
    float *dx_sfd = at<float>(workspace, L.dx_sfd);
    float *dw_part = at<float>(workspace, L.dw_part);
    void *zero_row = at<void>(workspace, L.zero_row);
    int32_t *bt_all = at<int32_t>(workspace, L.bt_all);
    int32_t *bt_first = at<int32_t>(workspace, L.bt_first);
    int32_t *bt_rest = at<int32_t>(workspace, L.bt_rest);
    float *dx_sh = D.n_shared > 0 ? at<float>(workspace, L.dx_sh) : nullptr;
    const size_t routed_tiles = (T * D.k + kBwdRowTile - 1) / kBwdRowTile + D.Ne + kBrimMaxFill;
    const bool det = D.flags & OCC_FLAG_DETERMINISTIC;
    const bool one_launch = !det && static_cast<int64_t>(D.T) * D.k < 128ll * D.Ne;

    OCC_TRY(mark(0));
    // row schedules of the input-gradient tiles, a zero row for the tails of
    // K-major operands
    const size_t zero_elems = std::max<size_t>({d, 2 * F, 2 * Nsh, kBwdTile});
    OCC_HIP(launch_fill_i32(static_cast<int32_t *>(zero_row), zero_elems * es / 4, 0, s));
    // the all-rows schedule filled for the SwiGLU backward's ceil(F / 256)
    // column tiles (the input gradient's product runs on the same schedule),
    // where the forward's is filled too (not in the decode regime, whose
    // products stream their weights and gain nothing from more tiles)
    const int bwd_fill = fill_cols(D) > 0 ? static_cast<int>(ceil_div(F, kBwdTile)) : 0;
    OCC_HIP(launch_tile_sched(bb.epd_off, bb.first_cnt, D.Ne, kBwdRowTile, bwd_fill, bt_all,
                              bt_first, bt_rest, s));
    // dy ORI -> SFD: the combine's transpose copies dy into each replica (and
    // zeroes the dx accumulator rows when the merge is one launch of adds)
    OCC_HIP(launch_dispatch(dy, D.T, D.Nd, d * es, bb.brim0, dy_sfd, s,
                            one_launch ? dx_sfd : nullptr, D.d));
    OCC_TRY(mark(1));
    // dh = dy W_d for every EPD row (its SFD row's gradient, BRIM_1), then
    // the SwiGLU and modulation backward
    BwdDgradArgs g1{};
    g1.A = dy_sfd;
    g1.a_rows = bb.epd_src;
    g1.lda = D.d;
    g1.B1 = w_down;
    g1.seg_off = bb.epd_off;
    g1.tile_off = bt_all;
    g1.first_cnt = bb.first_cnt;
    g1.gu = at<void>(workspace, L.gu);
    g1.gu_ld = 2 * D.F;
    g1.gu_uoff = D.F;
    g1.row_w = bb.epd_w;
    g1.out = dgu;
    g1.out_ld = 2 * D.F;
    g1.out_uoff = D.F;
    g1.dw_part = dw_part;
    g1.dw_stride = L.dw_stride;
    g1.N = D.F;
    g1.K = D.d;
    g1.ksplit = D.d;
    g1.Ne = D.Ne;
    g1.epilogue = BWD_EPI_SWIGLU;
    g1.tab = tab;
    OCC_HIP(launch_bwd_dgrad(g1, routed_tiles, s));
    OCC_TRY(mark(2));
    // dx_epd = dg W_g + du W_u, merged into SFD rows inside each group (fp32)
    BwdDgradArgs g2{};
    g2.A = dgu;
    g2.a_rows = bb.down_rows;
    g2.lda = 2 * D.F;
    g2.B1 = w_gate;
    g2.B2 = w_up;
    g2.seg_off = bb.epd_off;
    g2.first_cnt = bb.first_cnt;
    g2.dst_rows = bb.epd_src;
    g2.merge_out = dx_sfd;
    g2.N = D.d;
    g2.K = 2 * D.F;
    g2.ksplit = D.F;
    g2.Ne = D.Ne;
    g2.epilogue = BWD_EPI_MERGE;
    g2.tab = tab;
    if (det) {
        // first contributors store into their SFD rows of dx, the others at
        // their own EPD rows; summed per SFD row in slot order after the
        // shared experts, with the combine
        g2.epd_out = at<float>(workspace, L.y_epd);
        g2.split = 1;
        g2.phase = 0;
        g2.tile_off = bt_all;
        g2.merge_store = 1;
        OCC_HIP(launch_bwd_dgrad(g2, routed_tiles, s));
    } else if (one_launch) {
        g2.phase = 0;
        g2.tile_off = bt_all;
        g2.merge_store = 0;
        OCC_HIP(launch_bwd_dgrad(g2, routed_tiles, s));
    } else {
        g2.phase = 1;
        g2.tile_off = bt_first;
        g2.merge_store = 1;
        OCC_HIP(launch_bwd_dgrad(g2, routed_tiles, s));
        g2.phase = 2;
        g2.tile_off = bt_rest;
        g2.merge_store = 0;
        OCC_HIP(launch_bwd_dgrad(g2, routed_tiles, s));
    }
    OCC_TRY(mark(3));
    // shared experts: dense over the T tokens, one expert at a time for the
    // input gradients, all at once for the weight gradients
    if (D.n_shared > 0) {
        int32_t *dseg = at<int32_t>(workspace, L.dense_seg);
        int32_t *dtile = at<int32_t>(workspace, L.dense_tile);
        // the row-tile schedule of dh -> dg, du against F_shared columns,
        // balanced over the CUs' rounds (dx_sh below schedules its own)
        const int m_gu = dense_row_tiles_bwd(D.T, ceil_div(D.F_shared, kBwdTile));
        OCC_HIP(launch_dense_sched(D.T, m_gu, dseg, dtile, s));
        PlaceTab one{};
        one.Ne = 1;
        one.Nd = 1;
        one.n = 1;
        void *dgu_sh = at<void>(workspace, L.dgu_sh);
        // the shared W_d transposed (F_shared x d per expert), so that
        // dh_sh = dy W_d reads both operands K-contiguous.  (The routed
        // experts keep transpose reads: there the copy of all their W_d
        // costs what the faster product saves.)
        void *wt_down = at<void>(workspace, L.wt_down);
        OCC_HIP(launch_transpose_bf16(ws_down, D.d, D.F_shared, d * D.F_shared, wt_down, D.d,
                                      static_cast<size_t>(D.F_shared) * d, D.n_shared, s));
        for (int sx = 0; sx < D.n_shared; sx++) {
            const size_t Fs = D.F_shared;
            BwdDgradArgs s1{};
            s1.A = dy;
            s1.lda = D.d;
            s1.B1 = static_cast<const char *>(wt_down) + sx * Fs * d * es;
            s1.b_kcontig = 1;
            s1.seg_off = dseg;
            s1.tile_off = dtile;
            s1.gu = at<void>(workspace, L.gu_sh);
            s1.gu_ld = static_cast<int>(2 * Nsh);
            s1.gu_col = static_cast<int>(sx * Fs);
            s1.gu_uoff = static_cast<int>(Nsh);
            s1.out = dgu_sh;
            s1.out_ld = static_cast<int>(2 * Nsh);
            s1.out_col = static_cast<int>(sx * 2 * Fs);
            s1.out_uoff = static_cast<int>(Fs);
            s1.N = D.F_shared;
            s1.K = D.d;
            s1.ksplit = D.d;
            s1.Ne = 1;
            s1.epilogue = BWD_EPI_SWIGLU;
            s1.tab = one;
            OCC_HIP(launch_bwd_dgrad(s1, m_gu, s));
        }
        // dx_sh = sum over the shared experts of dg W_g + du W_u: one dense
        // product with K = 2 n_shared F_shared against the weights
        // transposed (expert sx's block holds W_g^T then W_u^T), on the
        // forward's down-projection build, whose operands both have the
        // contraction index contiguous (no LDS transpose reads)
        void *wt_sh = at<void>(workspace, L.wt_sh);
        const size_t Fs = D.F_shared, blk = d * 2 * Fs;
        OCC_HIP(launch_transpose_bf16(ws_gate, D.F_shared, D.d, Fs * d, wt_sh,
                                      static_cast<int>(2 * Fs), blk, D.n_shared, s));
        OCC_HIP(launch_transpose_bf16(ws_up, D.F_shared, D.d, Fs * d,
                                      static_cast<char *>(wt_sh) + Fs * es,
                                      static_cast<int>(2 * Fs), blk, D.n_shared, s));
        DownArgs s2{};
        s2.A = dgu_sh;
        s2.W = wt_sh;
        s2.out = dx_sh;
        s2.M = D.T;
        s2.K = static_cast<int>(2 * Nsh);
        s2.N = D.d;
        s2.Ne = 1;
        s2.k_split = static_cast<int>(2 * Fs);
        s2.tab = one;
        const GemmOps ops = gemm_ops(D);
        if (dense_pipelined(ops, D.T, D.d))
            OCC_HIP(launch_gemm_down_bf16_dense(s2, 0, s));
        else
            OCC_HIP(ops.down(s2, 0, s));
        BwdWgradArgs w3{};
        w3.A = dy;
        w3.lda = D.d;
        w3.B = at<void>(workspace, L.h_sh);
        w3.ldb = static_cast<int>(Nsh);
        w3.b_col_grp = D.F_shared;
        w3.zero_row = zero_row;
        w3.C1 = dws_down;
        w3.M = D.d;
        w3.N = D.F_shared;
        w3.msplit = D.d;
        w3.n_groups = D.n_shared;
        w3.rows = D.T;
        w3.tab = one;
        // K = all T tokens against a small output: split into chunks summed
        // in order (enough tiles for the CUs, still deterministic)
        w3.k_parts = wgrad_k_parts(D.n_shared, D.d, D.F_shared, D.T);
        w3.k_chunk = wgrad_k_chunk(D.T, w3.k_parts);
        w3.part = w3.k_parts > 1 ? at<float>(workspace, L.wg_part) : nullptr;
        OCC_HIP(launch_bwd_wgrad(w3, s));
        BwdWgradArgs w4{};
        w4.A = dgu_sh;
        w4.lda = static_cast<int>(2 * Nsh);
        w4.a_col_grp = 2 * D.F_shared;
        w4.B = x;
        w4.ldb = D.d;
        w4.zero_row = zero_row;
        w4.C1 = dws_gate;
        w4.C2 = dws_up;
        w4.M = 2 * D.F_shared;
        w4.N = D.d;
        w4.msplit = D.F_shared;
        w4.n_groups = D.n_shared;
        w4.rows = D.T;
        w4.tab = one;
        w4.k_parts = wgrad_k_parts(D.n_shared, 2 * D.F_shared, D.d, D.T);
        w4.k_chunk = wgrad_k_chunk(D.T, w4.k_parts);
        w4.part = w4.k_parts > 1 ? at<float>(workspace, L.wg_part) : nullptr;
        OCC_HIP(launch_bwd_wgrad(w4, s));
    }
    OCC_TRY(mark(4));
    // dx: SFD -> ORI, summed across groups (the dispatch's transpose), plus
    // the shared experts' part, cast once
    if (det)
        OCC_HIP(launch_merge_slots(at<float>(workspace, L.y_epd), at<int32_t>(workspace, L.ids),
                                   bb.tok_epd, bb.brim0, tab, D.T, D.k, D.d, dx_sfd, dx_sh, dx,
                                   D.dtype == OCC_BF16, s));
    else
        OCC_HIP(launch_combine(dx_sfd, bb.brim0, dx_sh, D.T, D.Nd, D.d, D.dtype == OCC_BF16, dx,
                               s));
    OCC_TRY(mark(5));
    // dW_d[e] = sum over e's rows of dy_sfd[row's SFD row] (x) h[row]
    BwdWgradArgs w1{};
    w1.A = dy_sfd;
    w1.a_rows = bb.epd_src;
    w1.lda = D.d;
    w1.B = h;
    w1.ldb = D.F;
    w1.seg_off = bb.epd_off;
    w1.zero_row = zero_row;
    w1.C1 = dw_down;
    w1.M = D.d;
    w1.N = D.F;
    w1.msplit = D.d;
    w1.n_groups = D.Ne;
    w1.tab = tab;
    OCC_HIP(launch_bwd_wgrad(w1, s));
    OCC_TRY(mark(6));
    // [dW_g; dW_u][e] = sum over e's rows of [dg; du] (x) x_sfd[row's SFD row]
    BwdWgradArgs w2{};
    w2.A = dgu;
    w2.lda = 2 * D.F;
    w2.B = x_sfd;
    w2.b_rows = bb.epd_src;
    w2.ldb = D.d;
    w2.seg_off = bb.epd_off;
    w2.zero_row = zero_row;
    w2.C1 = dw_gate;
    w2.C2 = dw_up;
    w2.M = 2 * D.F;
    w2.N = D.d;
    w2.msplit = D.F;
    w2.n_groups = D.Ne;
    w2.tab = tab;
    OCC_HIP(launch_bwd_wgrad(w2, s));
    OCC_TRY(mark(7));
    // routing-weight and logit gradients
    if (dw || dlogits)
        OCC_HIP(launch_route_backward(logits, at<int32_t>(workspace, L.ids), bb.tok_epd, dw_part,
                                      L.dw_stride, L.dw_stride, D.T, D.Ne, D.k, dw, dlogits, s));
    OCC_TRY(mark(8));
    return OCC_OK;
}

occ_status occ_route_scored(const occ_layer_desc *desc, const occ_score_desc *opt,
                            const float *logits, const float *bias, const int32_t *placement_host,
                            int32_t *ids, float *w, void *stream) {
    OCC_TRY(check_score(desc, opt));
    if (!logits || !ids || !w || !aligned_to(logits, 4) || !aligned_to(bias, 4) ||
        !aligned_to(ids, 4) || !aligned_to(w, 4) || !apart(ids, logits, bias, w) ||
        !apart(w, logits, bias))
        return OCC_ERR_INVALID_ARG;
    ScoreArgs a{};
    if (placement_host) {
        OCC_TRY(make_tab(*desc, placement_host, &a.tab));
    } else {
        if (opt->top_groups < desc->Nd) return OCC_ERR_INVALID_ARG;
        a.tab.Nd = desc->Nd;
        a.tab.n = desc->Ne / desc->Nd;
    }
    a.logits = logits;
    a.bias = bias;
    a.T = desc->T;
    a.Ne = desc->Ne;
    a.k = desc->k;
    a.sigmoid = opt->score == OCC_SCORE_SIGMOID;
    a.top_groups = opt->top_groups;
    a.group_best = opt->group_best;
    a.renormalise = opt->renormalise;
    a.scale = opt->scale;
    a.ids = ids;
    a.w = w;
    OCC_HIP(launch_route_scored(a, static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_route_scored_backward(const occ_layer_desc *desc, const occ_score_desc *opt,
                                     const float *logits, const int32_t *ids, const float *dw,
                                     const float *dlogits_in, float *dlogits, void *stream) {
    OCC_TRY(check_score(desc, opt));
    if (!logits || !ids || !dw || !dlogits || !aligned_to(logits, 4) || !aligned_to(ids, 4) ||
        !aligned_to(dw, 4) || !aligned_to(dlogits_in, 4) || !aligned_to(dlogits, 4) ||
        !apart(dlogits, ids, dw))
        return OCC_ERR_INVALID_ARG;
    OCC_HIP(launch_route_scored_back(logits, ids, dw, dlogits_in, desc->T, desc->Ne, desc->k,
                                     opt->score == OCC_SCORE_SIGMOID, opt->renormalise, opt->scale,
                                     dlogits, static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_route_bias_step(const occ_layer_desc *desc, float rate, const int32_t *ids,
                               const uint8_t *valid, const float *bias_in, int32_t *counts,
                               float *bias, void *workspace, size_t ws_bytes, void *stream) {
    OCC_TRY(check_desc(desc));
    if (!ids || !bias_in || !counts || !bias || !std::isfinite(rate) || !aligned_to(ids, 4) ||
        !aligned_to(bias_in, 4) || !aligned_to(counts, 4) || !aligned_to(bias, 4) ||
        !apart(counts, ids, valid, bias_in, bias) || !apart(bias, ids, valid) ||
        !apart(workspace, ids, valid, bias_in, counts, bias))
        return OCC_ERR_INVALID_ARG;
    OCC_TRY(check_ws(*desc, workspace, ws_bytes, block_ws_bytes(*desc)));
    OCC_HIP(launch_bias_step(ids, valid, desc->T, desc->k, desc->Ne, bias_in, rate, counts, bias,
                             static_cast<int32_t *>(workspace), static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_quantize_int8(int64_t rows, int32_t cols, int32_t dtype, const void *x, int8_t *q,
                             float *scale, void *stream) {
    if (rows < 1 || cols < 1 || (dtype != OCC_F32 && dtype != OCC_BF16) || !x || !q || !scale ||
        !rows_aligned(x, q) || !aligned_to(scale, 4) || !apart(q, x, scale) || !apart(scale, x))
        return OCC_ERR_INVALID_ARG;
    if (cols % 16 || rows >= (1ll << 31)) return OCC_ERR_UNSUPPORTED;
    OCC_HIP(launch_quantize_rows(x, dtype == OCC_BF16, static_cast<size_t>(rows), cols, q,
                                 static_cast<size_t>(cols), scale, static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

occ_status occ_int8_workspace_size(const occ_layer_desc *desc, size_t *bytes_host) {
    OCC_TRY(check_int8(desc));
    if (!bytes_host) return OCC_ERR_INVALID_ARG;
    *bytes_host = int8_layout(*desc).total;
    return OCC_OK;
}

occ_status occ_moe_forward_int8(const occ_layer_desc *desc, const void *x, const int32_t *ids_in,
                                const float *w_in, const int32_t *placement_host,
                                const occ_int8_experts *experts_host,
                                const occ_int8_experts *shared_host, void *y, void *workspace,
                                size_t ws_bytes, void *stream) {
    OCC_TRY(check_int8(desc));
    const occ_layer_desc &D = *desc;
    if (!x || !ids_in || !w_in || !y || !experts_given(experts_host) || !rows_aligned(x, y) ||
        !aligned_to(ids_in, 4) || !aligned_to(w_in, 4) ||
        (D.n_shared > 0 ? !experts_given(shared_host) : shared_host != nullptr) ||
        !apart(y, x, ids_in, w_in) || !apart_from(y, experts_host) ||
        !apart_from(y, shared_host) || !apart(workspace, x, ids_in, w_in, y) ||
        !apart_from(workspace, experts_host) || !apart_from(workspace, shared_host))
        return OCC_ERR_INVALID_ARG;
    PlaceTab tab;
    OCC_TRY(make_tab(D, placement_host, &tab));
    const Int8Layout L = int8_layout(D);
    OCC_TRY(check_ws(D, workspace, ws_bytes, L.total));

    hipStream_t s = static_cast<hipStream_t>(stream);
    int8_t *xq = at<int8_t>(workspace, L.xq), *hq = at<int8_t>(workspace, L.hq);
    float *xs = at<float>(workspace, L.xs), *hs = at<float>(workspace, L.hs);
    float *h = at<float>(workspace, L.h);
    uint16_t *y_epd = at<uint16_t>(workspace, L.y_epd), *y_sh = at<uint16_t>(workspace, L.y_sh);
    const size_t T = D.T, d = D.d, nepd = T * D.k;
    if (few_tokens(D)) {
        const auto weights = [](const occ_int8_experts *e) {
            return e ? Int8Weights{e->gate, e->up, e->down, e->gate_scale, e->up_scale, e->down_scale}
                     : Int8Weights{};
        };
        FewArgs f{};
        f.x = static_cast<const uint16_t *>(x);
        f.ids = ids_in;
        f.w = w_in;
        f.routed = weights(experts_host);
        f.shared = weights(shared_host);
        f.h = h;
        f.h_sh = h + nepd * D.F;
        f.y = static_cast<uint16_t *>(y);
        f.T = D.T;
        f.d = D.d;
        f.Ne = D.Ne;
        f.k = D.k;
        f.F = D.F;
        f.n_shared = D.n_shared;
        f.F_shared = D.n_shared > 0 ? D.F_shared : 0;
        OCC_HIP(launch_few(f, s));
        return OCC_OK;
    }
    const bool small = small_tiles8(D), small_sh = D.T < kSmallTileShared8;
    const auto gemm_up = small ? launch_gemm_up8_m80 : launch_gemm_up8;
    const auto gemm_down = small ? launch_gemm_down8_m80 : launch_gemm_down8;
    const auto gemm_up_sh = small_sh ? launch_gemm_up8_m80 : launch_gemm_up8;
    const auto gemm_down_sh = small_sh ? launch_gemm_down8_m80 : launch_gemm_down8;
    const size_t routed_tiles = most_row_tiles8(D);

    // a token's row of codes is kept once and gathered by each of its experts
    SlotArgs sl{};
    sl.ids = ids_in;
    sl.w = w_in;
    sl.x = static_cast<const u32x4 *>(x);
    sl.xq = xq;
    sl.xs = xs;
    sl.tok_epd = at<int32_t>(workspace, L.tok_epd);
    sl.epd_tok = at<int32_t>(workspace, L.epd_tok);
    sl.epd_off = at<int32_t>(workspace, L.epd_off);
    sl.tile_off = at<int32_t>(workspace, L.tile_off);
    sl.epd_w = at<float>(workspace, L.epd_w);
    sl.counts = at<int32_t>(workspace, L.counts);
    sl.ldx = round_line(d);
    sl.T = D.T;
    sl.d = D.d;
    sl.k = D.k;
    sl.tile_rows = tile_rows8(D);
    sl.fill_cols = fill_cols8(D);
    sl.tab = tab;
    OCC_HIP(launch_slots(sl, s));
    for (int sx = 0; sx < D.n_shared; sx++) {
        const size_t Fs = D.F_shared, wo = sx * Fs * d;
        Up8Args up{};
        up.A = xq;
        up.a_scale = xs;
        up.Wg = shared_host->gate + wo;
        up.Wu = shared_host->up + wo;
        up.sg = shared_host->gate_scale + sx * Fs;
        up.su = shared_host->up_scale + sx * Fs;
        up.out = h;
        up.M = D.T;
        up.K = D.d;
        up.N = D.F_shared;
        up.Ne = 1;
        up.lda = static_cast<int>(round_line(d));
        up.tab = tab;
        OCC_HIP(gemm_up_sh(up, 0, s));
        OCC_HIP(launch_quantize_rows(h, 0, T, D.F_shared, hq, round_line(Fs), hs, s));
        Down8Args dn{};
        dn.A = hq;
        dn.a_scale = hs;
        dn.W = shared_host->down + wo;
        dn.sd = shared_host->down_scale + sx * d;
        dn.out = y_sh + sx * T * d;
        dn.M = D.T;
        dn.K = D.F_shared;
        dn.N = D.d;
        dn.Ne = 1;
        dn.lda = static_cast<int>(round_line(Fs));
        dn.tab = tab;
        OCC_HIP(gemm_down_sh(dn, 0, s));
    }
    Up8Args up{};
    up.A = xq;
    up.a_rows = sl.epd_tok;
    up.a_scale = xs;
    up.Wg = experts_host->gate;
    up.Wu = experts_host->up;
    up.sg = experts_host->gate_scale;
    up.su = experts_host->up_scale;
    up.seg_off = sl.epd_off;
    up.tile_off = sl.tile_off;
    up.row_w = sl.epd_w;
    up.out = h;
    up.M = D.T * D.k;
    up.K = D.d;
    up.N = D.F;
    up.Ne = D.Ne;
    up.lda = static_cast<int>(round_line(d));
    up.tab = tab;
    OCC_HIP(gemm_up(up, routed_tiles, s));
    OCC_HIP(launch_quantize_rows(h, 0, nepd, D.F, hq, round_line(D.F), hs, s));
    Down8Args dn{};
    dn.A = hq;
    dn.a_scale = hs;
    dn.W = experts_host->down;
    dn.sd = experts_host->down_scale;
    dn.seg_off = sl.epd_off;
    dn.tile_off = sl.tile_off;
    dn.out = y_epd;
    dn.M = D.T * D.k;
    dn.K = D.F;
    dn.N = D.d;
    dn.Ne = D.Ne;
    dn.lda = static_cast<int>(round_line(D.F));
    dn.tab = tab;
    OCC_HIP(gemm_down(dn, routed_tiles, s));
    OCC_HIP(launch_combine_rows(y_epd, sl.tok_epd, y_sh, D.n_shared, D.T, D.k, D.d,
                                static_cast<uint16_t *>(y), s));
    return OCC_OK;
}

occ_status occ_coactivation_stats(const occ_layer_desc *desc, const int32_t *ids,
                                  const int32_t *placement_host, int32_t *C, float *P,
                                  int64_t *n_sfd, double *ct, double *intra, void *stream) {
    OCC_TRY(check_desc(desc));
    if (!ids || !C || !P || !n_sfd || !ct || !intra) return OCC_ERR_INVALID_ARG;
    PlaceTab tab;
    OCC_TRY(make_tab(*desc, placement_host, &tab));
    OCC_HIP(launch_coact(ids, desc->T, desc->k, tab, C, P, n_sfd, ct, intra,
                         static_cast<hipStream_t>(stream)));
    return OCC_OK;
}

// Algorithm 1 (paper section 3.2).  The 1/|L| and 1/max C scalings of the
// paper's scores do not change any argmax / argmin, so the integer counts are
// used directly; each unused expert's summed collaboration with all placed
// experts and with the current group is kept up to date as experts are
// placed.
occ_status occ_place_experts(const int32_t *C_host, int32_t Ne, int32_t Nd,
                             int32_t *placement_host) {
    if (!C_host || !placement_host || Ne < 1 || Nd < 1 || Ne % Nd != 0 || Ne > 65536)
        return OCC_ERR_INVALID_ARG;
    const int n = Ne / Nd;
    std::vector<char> used(Ne, 0);
    std::vector<int64_t> with_placed(Ne, 0), with_group(Ne, 0);
    for (int g = 0; g < Nd; g++) {
        std::fill(with_group.begin(), with_group.end(), 0);
        int32_t *Lg = placement_host + static_cast<size_t>(g) * n;
        int len = 0;
        auto push = [&](int e) {
            Lg[len++] = e;
            used[e] = 1;
            const int32_t *row = C_host + static_cast<size_t>(e) * Ne;
            for (int q = 0; q < Ne; q++) {
                with_placed[q] += row[q];
                with_group[q] += row[q];
            }
        };
        if (g == 0 && n >= 2) {
            int bi = 0, bj = 1;
            for (int i = 0; i < Ne; i++)
                for (int j = i + 1; j < Ne; j++)
                    if (C_host[static_cast<size_t>(i) * Ne + j] >
                        C_host[static_cast<size_t>(bi) * Ne + bj]) {
                        bi = i;
                        bj = j;
                    }
            push(bi);
            push(bj);
        } else if (g > 0) {
            int best = -1;
            for (int e = 0; e < Ne; e++)
                if (!used[e] && (best < 0 || with_placed[e] < with_placed[best])) best = e;
            push(best);
        }
        while (len < n) {
            int best = -1;
            for (int e = 0; e < Ne; e++)
                if (!used[e] && (best < 0 || with_group[e] > with_group[best])) best = e;
            push(best);
        }
    }
    return OCC_OK;
}

occ_status occ_events_create(int32_t n, void **events_host) {
    if (n < 0 || (n > 0 && !events_host)) return OCC_ERR_INVALID_ARG;
    for (int i = 0; i < n; i++) {
        hipEvent_t e;
        OCC_HIP(hipEventCreate(&e));
        events_host[i] = e;
    }
    return OCC_OK;
}

occ_status occ_events_destroy(int32_t n, void **events_host) {
    if (n < 0 || (n > 0 && !events_host)) return OCC_ERR_INVALID_ARG;
    for (int i = 0; i < n; i++)
        if (events_host[i]) OCC_HIP(hipEventDestroy(static_cast<hipEvent_t>(events_host[i])));
    return OCC_OK;
}

occ_status occ_event_elapsed_ms(void *start, void *stop, float *ms_host) {
    if (!start || !stop || !ms_host) return OCC_ERR_INVALID_ARG;
    OCC_HIP(hipEventSynchronize(static_cast<hipEvent_t>(stop)));
    OCC_HIP(hipEventElapsedTime(ms_host, static_cast<hipEvent_t>(start),
                                static_cast<hipEvent_t>(stop)));
    return OCC_OK;
}

}  // extern "C"
