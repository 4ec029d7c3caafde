// The slots of the layer with 8-bit experts sorted by expert, and the tokens
// quantised beside that.  A slot (token t, its j-th expert) gets an EPD row in
// its expert's segment, segments in placement order as in Algorithm 5.  The
// order of the rows inside a segment is left open (LDS counters hand them
// out): an EPD row's results do not depend on where it stands, and a token's
// terms are summed in the order of its ids.
//
// Bound by latency: the entries are few (12 bytes a slot), so what counts is
// the launches and the dependent steps in them.  Batches of up to kSlotsSmall
// tokens and kSlotsSmallEntries entries are sorted by one workgroup, counted,
// scanned and placed in LDS; larger ones in two launches, the workgroups
// counting their tokens into a table and then each adding up the table for
// itself.  The quantiser's rows ride in the first launch's other workgroups,
// where the GPU would wait.  Measured with the tokens' codes (d = 2048, top 8,
// 64 experts): 512 tokens 11.0 us in one launch, 8192 12.8 + 10.7 in two.
#include <algorithm>

#include "int8_rows.h"

namespace occ {
namespace {

constexpr int kPlaceThreads = 256;

// A token's experts, safe: one that is out of range or repeats an earlier one
// becomes the lowest not yet used, with weight 0 (as launch_sanitize_ids).
// f(j, expert, weight) for each slot; kAhead entries are loaded at once.  ONCE:
// there are no more (k <= kAhead), so that j is a constant where f is inlined.
constexpr int kAhead = 8;
template <bool ONCE = false, typename F>
__device__ __forceinline__ void for_slots(const int32_t *__restrict__ ids, const float *__restrict__ w,
                                          size_t t, int k, int Ne, F f) {
    const size_t o = t * k;
    uint64_t u0 = 0, u1 = 0, u2 = 0, u3 = 0;
    for (int j0 = 0; j0 < (ONCE ? 1 : k); j0 += kAhead) {
        int e_in[kAhead];
        float w_in[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            const size_t at = o + min(j0 + j, k - 1);
            e_in[j] = ids[at];
            w_in[j] = w ? w[at] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            const int e = e_in[j], word = e >> 6;
            const uint64_t in = word == 0 ? u0 : word == 1 ? u1 : word == 2 ? u2 : u3;
            const bool good = e >= 0 && e < Ne && !(in >> (e & 63) & 1);
            // k <= Ne leaves one below Ne
            const int free = ~u0 ? __builtin_ctzll(~u0)
                                 : ~u1 ? 64 + __builtin_ctzll(~u1)
                                       : ~u2 ? 128 + __builtin_ctzll(~u2) : 192 + __builtin_ctzll(~u3 | 1ull << 63);
            const int to = good ? e : free;
            const uint64_t bit = 1ull << (to & 63);
            u0 |= to < 64 ? bit : 0;
            u1 |= to >> 6 == 1 ? bit : 0;
            u2 |= to >> 6 == 2 ? bit : 0;
            u3 |= to >> 6 == 3 ? bit : 0;
            if (j0 + j < k) f(ONCE ? j : j0 + j, to, good ? w_in[j] : 0.f);
        }
    }
}

// Segment starts and, with `schedule`, the row-tile schedule (as the BRIM
// scan's) from the experts' rows by placement position; by one wave.  start
// gets Ne entries (LDS), epd_off and tile_off Ne + 1.
__device__ void segments(const int *rows, int *tiles, const SlotArgs &a, int *start, bool schedule) {
    const int lane = lane_id(), Ne = a.tab.Ne;
    if (schedule) {
        for (int p = lane; p < Ne; p += kWave) tiles[p] = (rows[p] + a.tile_rows - 1) / a.tile_rows;
        wave_sync();
        if (a.fill_cols > 0) fill_rounds(rows, tiles, Ne, a.fill_cols, a.cus, kBrimMaxFill);
        wave_sync();
    }
    int run = 0, run_t = 0;
    for (int p0 = 0; p0 < Ne; p0 += kWave) {
        const int p = p0 + lane;
        const int v = p < Ne ? rows[p] : 0, vt = schedule && p < Ne ? tiles[p] : 0;
        const int inc = wave_incl_scan(v), inc_t = wave_incl_scan(vt);
        if (p < Ne) {
            start[p] = run + inc - v;
            if (schedule) {
                a.epd_off[p] = run + inc - v;
                a.tile_off[p] = run_t + inc_t - vt;
            }
        }
        run += __shfl(inc, kWave - 1);
        run_t += __shfl(inc_t, kWave - 1);
    }
    if (schedule && lane == 0) {
        a.epd_off[Ne] = run;
        a.tile_off[Ne] = run_t;
    }
}

// Where an expert stands in the placement, in LDS.
__device__ __forceinline__ void load_places(const PlaceTab &tab, int *s_pos) {
    for (int p = threadIdx.x; p < tab.Ne; p += blockDim.x) s_pos[tab.expert[p]] = p;
}

__device__ __forceinline__ void place_token(const SlotArgs &a, size_t t, const int *s_pos, int *next) {
    for_slots(a.ids, a.w, t, a.k, a.tab.Ne, [&](int j, int e, float w) {
        const int row = atomicAdd(next + s_pos[e], 1);
        a.tok_epd[t * a.k + j] = row;
        a.epd_tok[row] = static_cast<int32_t>(t);
        a.epd_w[row] = w;
    });
}

template <int NV>
__device__ __forceinline__ void quantise_tokens(const SlotArgs &a, int block, int blocks) {
    const size_t waves = blockDim.x / kWave, step = static_cast<size_t>(blocks) * waves;
    for (size_t t = static_cast<size_t>(block) * waves + threadIdx.x / kWave; t < static_cast<size_t>(a.T); t += step)
        quantise_row<true, NV>(a.x + t * (a.d / 8), a.d / 8, a.xq + t * a.ldx, a.ldx, a.xs + t);
}

template <int NV>
__global__ __launch_bounds__(kSlotsSmall) void k_slots_small(SlotArgs a) {
    if (blockIdx.x > 0) {
        quantise_tokens<NV>(a, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    __shared__ int s_rows[kMaxNe], s_tiles[kMaxNe], s_next[kMaxNe], s_pos[kMaxNe];
    for (int p = threadIdx.x; p < kMaxNe; p += kSlotsSmall) s_rows[p] = 0;
    load_places(a.tab, s_pos);
    __syncthreads();
    const int t = threadIdx.x;
    // Up to kAhead slots a token stay in registers, each with its position in
    // the placement and its count so far, its row's place in the segment.
    const bool held = a.k <= kAhead;
    int pos[kAhead], rank[kAhead];
    float w[kAhead];
    if (t < a.T) {
        if (held)
            for_slots<true>(a.ids, a.w, t, a.k, a.tab.Ne, [&](int j, int e, float wj) {
                pos[j] = s_pos[e];
                rank[j] = atomicAdd(s_rows + pos[j], 1);
                w[j] = wj;
            });
        else
            for_slots(a.ids, nullptr, t, a.k, a.tab.Ne, [&](int, int e, float) { atomicAdd(s_rows + s_pos[e], 1); });
    }
    __syncthreads();
    if (threadIdx.x < kWave) segments(s_rows, s_tiles, a, s_next, true);
    __syncthreads();
    if (t >= a.T) return;
    if (!held) {
        place_token(a, t, s_pos, s_next);
        return;
    }
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
        if (j >= a.k) continue;
        const int row = s_next[pos[j]] + rank[j];
        a.tok_epd[static_cast<size_t>(t) * a.k + j] = row;
        a.epd_tok[row] = t;
        a.epd_w[row] = w[j];
    }
}

template <int NV>
__global__ __launch_bounds__(kPlaceThreads) void k_slots_count(SlotArgs a) {
    const int b = blockIdx.x;
    if (b >= a.shares) {
        quantise_tokens<NV>(a, b - a.shares, gridDim.x - a.shares);
        return;
    }
    __shared__ int s_rows[kMaxNe], s_pos[kMaxNe];
    for (int p = threadIdx.x; p < kMaxNe; p += kPlaceThreads) s_rows[p] = 0;
    load_places(a.tab, s_pos);
    __syncthreads();
    const int end = min(a.T, (b + 1) * a.share);
    for (int t = b * a.share + threadIdx.x; t < end; t += kPlaceThreads)
        for_slots(a.ids, nullptr, t, a.k, a.tab.Ne, [&](int, int e, float) { atomicAdd(s_rows + s_pos[e], 1); });
    __syncthreads();
    for (int p = threadIdx.x; p < a.tab.Ne; p += kPlaceThreads) a.counts[static_cast<size_t>(b) * a.tab.Ne + p] = s_rows[p];
}

// Workgroup b < shares places its tokens; the last one makes the schedule.
__global__ __launch_bounds__(kPlaceThreads) void k_slots_place(SlotArgs a) {
    __shared__ int s_rows[kMaxNe], s_below[kMaxNe], s_tiles[kMaxNe], s_next[kMaxNe], s_pos[kMaxNe];
    const int b = blockIdx.x, Ne = a.tab.Ne;
    for (int p = threadIdx.x; p < kMaxNe; p += kPlaceThreads) s_rows[p] = s_below[p] = 0;
    load_places(a.tab, s_pos);
    __syncthreads();
    // position p's column of the table, shared out over the threads
    int per = 1;
    while (per * 2 * Ne <= kPlaceThreads) per *= 2;
    for (int i = threadIdx.x; i < per * Ne; i += kPlaceThreads) {
        const int p = i % Ne, first = i / Ne;
        int all = 0, below = 0;
#pragma unroll 8
        for (int q = first; q < a.shares; q += per) {
            const int v = a.counts[static_cast<size_t>(q) * Ne + p];
            all += v;
            below += q < b ? v : 0;
        }
        atomicAdd(s_rows + p, all);
        atomicAdd(s_below + p, below);
    }
    __syncthreads();
    if (threadIdx.x < kWave) segments(s_rows, s_tiles, a, s_next, b == a.shares);
    if (b == a.shares) return;
    __syncthreads();
    for (int p = threadIdx.x; p < Ne; p += kPlaceThreads) s_next[p] += s_below[p];
    __syncthreads();
    const int end = min(a.T, (b + 1) * a.share);
    for (int t = b * a.share + threadIdx.x; t < end; t += kPlaceThreads) place_token(a, t, s_pos, s_next);
}

}  // namespace

hipError_t launch_slots(const SlotArgs &args, hipStream_t s) {
    SlotArgs a = args;
    const int nv = static_cast<int>(ceil_div(a.d / 8, kWave));
    const bool small = slot_shares(a.T, a.k) == 0;
    const size_t waves = (small ? kSlotsSmall : kPlaceThreads) / kWave;
    const unsigned quant = static_cast<unsigned>(std::min<size_t>(ceil_div(a.T, waves), 1 << 20));
    a.cus = compute_units();
    if (!small) {
        a.share = slot_shares(a.T, a.k);
        a.shares = static_cast<int>(ceil_div(a.T, a.share));
    }
#define OCC_SLOTS(NV)                                                                       \
    do {                                                                                    \
        if (small) k_slots_small<NV><<<1 + quant, kSlotsSmall, 0, s>>>(a);                  \
        else k_slots_count<NV><<<a.shares + quant, kPlaceThreads, 0, s>>>(a);               \
    } while (0)
    if (nv <= 1) OCC_SLOTS(1);
    else if (nv <= 2) OCC_SLOTS(2);
    else if (nv <= 4) OCC_SLOTS(4);
    else if (nv <= 8) OCC_SLOTS(8);
    else OCC_SLOTS(16);
#undef OCC_SLOTS
    if (!small) k_slots_place<<<a.shares + 1, kPlaceThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace occ
