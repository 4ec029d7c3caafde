// The boundary between two transformer blocks: the norm behind a block, its
// gate and residual scale, the residual addition and the norm in front of the
// next block in one pass over the rows, and the backward pass of that.
//
// Mathematics (n(v) = v rstd(v), rstd = 1 / sqrt(mean v^2 + eps) by rows):
//   r = x + s g w_post n(y),   h = w_pre n(r).
// The gradient of <q, n(v)> in v is rstd (q - n(v) mean(q n(v))), so a row's
// backward needs three sums before dr' = dr + (gradient through h) is known
// (r.r, (dh w_pre).r, y.y) and one after it ((dr' g w_post).n(y)), which is also
// a token gate's gradient.  (With v rstd^3 mean(q v) behind rstd q a cube leaves
// fp32 where rows and eps are small, and the gradient does not.)  The gradients
// of w_post and of a channel gate come from one column sum, S = sum over rows of
// s g_token dr' n(y): gate S and w_post S.
//
// Memory bound: the forward reads x and y and writes r and h once, the
// backward reads dr, dh, r and y and writes dx and dy once.  A row stays in
// registers as 16-byte chunks from its loads to its stores, and a team of
// threads shares it (chunk c with thread c mod NT, so that a wave's loads are
// contiguous).  Teams are as wide as leaves each thread one or two chunks:
// short dependent chains and few registers, so that many rows are in flight;
// a team of several waves adds its sums through LDS, and a row of up to 32
// chunks takes 16 or 32 lanes of a wave (T = 65536, d = 128 forward 12 us, 24
// with a wave to a row; backward 26 against 50).  At d = 2048 in bf16
// (256 chunks), T = 65536 forward, compared when loads and stores stood under
// conditions: 188 us with 128 threads a row (186 now), 211 with 256, 200 with
// 64 (one wave, no barrier).
// The forward gives each row to a team of its own.  In the backward each
// thread also keeps fp32 sums of its columns' weight gradients, so its teams
// walk over rows with a fixed stride, the next row's loads issued before this
// one's sums; a workgroup's sums go to the workspace once and a second kernel
// adds the workgroups' in order, so results do not depend on timing.
// Workgroups of 1024 threads, one per CU, leave the fewest such sums: 299 us
// at T = 65536, d = 2048 (297 now) against 313 with two of 256 threads.
// A workgroup's row takes 1.6 us (1.2 of them the vector units'), 2.6 with
// loads and stores under conditions, IEEE roots and divisions and values
// rounded one by one.
// Measured at d = 2048 bf16, all parts present: forward T = 65536 186 us
// (5.8 TB/s of the bytes it cannot do without), one token 2.2; backward
// T = 65536 297 + 4.6 us (5.3 TB/s), T = 8192 39.6 + 4.7 us (4.5 TB/s).
// Stores past the caches measure 3% faster alone and slower by 2 to 5% with
// the kernel that reads their rows, so they are ordinary.
#include <algorithm>

#include "launch.h"

namespace occ {
namespace {

// NT threads share a row: forward in workgroups of at least 256 threads,
// backward in workgroups of 1024.
template <int NT>
constexpr int kBlock = NT > 256 ? NT : 256;
constexpr int kBackBlock = 1024;

// A chunk is 16 bytes of a row: E values.
template <typename E>
struct Chunk;
template <>
struct Chunk<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const u32x4 &c, float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(c[i] << 16);
            v[2 * i + 1] = __uint_as_float(c[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ u32x4 pack(const float (&v)[N]) {
        typedef __attribute__((ext_vector_type(2))) float f32x2;
        typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
        u32x4 c;
#pragma unroll
        for (int i = 0; i < 4; i++)
            c[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * i], v[2 * i + 1]}, bf16x2));
        return c;
    }
};
template <>
struct Chunk<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const u32x4 &c, float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = __uint_as_float(c[i]);
    }
    static __device__ __forceinline__ u32x4 pack(const float (&v)[N]) {
        u32x4 c;
#pragma unroll
        for (int i = 0; i < 4; i++) c[i] = __float_as_uint(v[i]);
        return c;
    }
};

// Arrays are reached through buffer descriptors, whose bounds take the place
// of conditions: loads behind the last row or chunk, or of an array that a
// call does not have (no bytes), give zero, stores there do nothing.  With
// every access unconditional a wait can count the ones behind it, so that the
// next row's loads and the last one's stores stay in flight.
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr unsigned kNowhere = 0x40000000;  // behind every buffer's end
__device__ __forceinline__ Buffer buffer_of(const void *p, unsigned bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, p ? bytes : 0, 0x00020000);
}
__device__ __forceinline__ u32x4 load_chunk(Buffer b, unsigned at) {
    return __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, 0);
}
__device__ __forceinline__ void store_chunk(Buffer b, unsigned at, u32x4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(v, b, at, 0, 0);
}
__device__ __forceinline__ float load_float(Buffer b, unsigned at) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, at, 0, 0));
}
// Rows [t0, t0 + rows) of arrays of T rows of `bytes` each.
struct Rows {
    size_t from;
    unsigned bytes;
    __device__ __forceinline__ Rows(unsigned t0, unsigned rows, unsigned T, unsigned row_bytes)
        : from(static_cast<size_t>(t0) * row_bytes), bytes(t0 < T ? min(rows, T - t0) * row_bytes : 0) {}
    __device__ __forceinline__ Buffer of(const void *p) const {
        return __builtin_amdgcn_make_buffer_rsrc(static_cast<char *>(const_cast<void *>(p)) + from, 0,
                                                 p ? bytes : 0, 0x00020000);
    }
};

// 1 / sqrt(mean + eps) by the hardware, 2^-23 relative (eps is a normal number).
__device__ __forceinline__ float rstd_of(float squares, float inv_d, float eps) {
    return __builtin_amdgcn_rsqf(fmaf(squares, inv_d, eps));
}

// Sums over a wave, a step of all M at a time: each fills the wait that the
// lane network asks for behind another.
template <int M>
__device__ __forceinline__ void wave_sums(float (&v)[M]) {
#define OCC_STEP(CTRL, MASK)   \
    _Pragma("unroll") for (int i = 0; i < M; i++) v[i] += dpp_f<CTRL, MASK>(0.f, v[i]);
    OCC_STEP(kDppRowShr1, 0xf)
    OCC_STEP(kDppRowShr2, 0xf)
    OCC_STEP(kDppRowShr4, 0xf)
    OCC_STEP(kDppRowShr8, 0xf)
    OCC_STEP(kDppRowBcast15, 0xa)
    OCC_STEP(kDppRowBcast31, 0xc)
#undef OCC_STEP
#pragma unroll
    for (int i = 0; i < M; i++)
        v[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v[i]), kWave - 1));
}

// Sums over the NT threads that share a row.  Rows of several waves go
// through LDS, with two sets of slots used in turn (the next sum's writes
// cannot meet this one's reads, since the barrier in between orders them).
constexpr int kMaxWaves = kBackBlock / kWave;
typedef float Slots[2][3][kMaxWaves];
template <int NT, int M>
__device__ __forceinline__ void row_sums(float (&v)[M], Slots &slots, int &turn) {
    constexpr int kRowWaves = NT / kWave;
    if constexpr (NT < kWave) {
#pragma unroll
        for (int i = 0; i < M; i++) v[i] = group_sum<NT>(v[i]);
    } else {
        wave_sums(v);
    }
    if constexpr (kRowWaves > 1) {
        const int w = threadIdx.x / kWave, w0 = threadIdx.x / NT * kRowWaves;
        if (lane_id() == 0) {
#pragma unroll
            for (int i = 0; i < M; i++) slots[turn][i][w] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < M; i++)
            v[i] = group_sum<kRowWaves>(slots[turn][i][w0 + lane_id() % kRowWaves]);
        turn ^= 1;
    }
}

struct NormArgs {
    const u32x4 *x, *y, *w_post, *w_pre;
    const void *gate;
    u32x4 *r, *h;
    unsigned T;     // rows
    int chunks;     // 16-byte chunks of a row
    int gate_kind;  // occ_block_gate
    float inv_d, eps, scale;
};

template <typename E, int NT, int VPT>
__global__ __launch_bounds__(kBlock<NT>) void k_norm(NormArgs a) {
    constexpr int N = Chunk<E>::N;
    __shared__ Slots slots;
    int turn = 0;
    constexpr int kRows = kBlock<NT> / NT;
    const unsigned c = threadIdx.x % NT, sub = threadIdx.x / NT, bytes = a.chunks * 16;
    const bool gate_ch = a.gate_kind == 1, gate_tok = a.gate_kind == 2;
    unsigned at[VPT];  // in a row
#pragma unroll
    for (int j = 0; j < VPT; j++)
        at[j] = c + NT * j < static_cast<unsigned>(a.chunks) ? 16 * (c + NT * j) : kNowhere;
    u32x4 xr[VPT], yr[VPT], wpost[VPT], wpre[VPT], wgate[VPT];
    float gt;
    auto load = [&](unsigned t0) {
        const Rows rows(t0, kRows, a.T, bytes);
        const Buffer x = rows.of(a.x), y = rows.of(a.y);
#pragma unroll
        for (int j = 0; j < VPT; j++) {
            xr[j] = load_chunk(x, sub * bytes + at[j]);
            yr[j] = load_chunk(y, sub * bytes + at[j]);
        }
        gt = load_float(Rows(t0, kRows, a.T, 4).of(gate_tok ? a.gate : nullptr), sub * 4);
    };
    unsigned t0 = blockIdx.x * kRows;
    load(t0);
#pragma unroll
    for (int j = 0; j < VPT; j++) {
        wpost[j] = load_chunk(buffer_of(a.w_post, bytes), at[j]);
        wpre[j] = load_chunk(buffer_of(a.w_pre, bytes), at[j]);
        wgate[j] = load_chunk(buffer_of(gate_ch ? a.gate : nullptr, bytes), at[j]);
    }
    // the trip count is the workgroup's: its rows' sums may need barriers
    while (true) {
        float s = a.scale;
        if (gate_tok) s *= gt;
        if (a.w_post) {
            float ssq[1] = {0.f};
#pragma unroll
            for (int j = 0; j < VPT; j++) {
                float v[N];
                Chunk<E>::unpack(yr[j], v);
#pragma unroll
                for (int i = 0; i < N; i++) ssq[0] = fmaf(v[i], v[i], ssq[0]);
            }
            row_sums<NT>(ssq, slots, turn);
            s *= rstd_of(ssq[0], a.inv_d, a.eps);
        }
        const Rows rows(t0, kRows, a.T, bytes);
        const Buffer to_r = rows.of(a.r), to_h = rows.of(a.h);
        float r[VPT][N];
        float ssq[1] = {0.f};
#pragma unroll
        for (int j = 0; j < VPT; j++) {
            Chunk<E>::unpack(xr[j], r[j]);
            if (a.y) {
                float z[N], w[N];
                Chunk<E>::unpack(yr[j], z);
                if (a.w_post) {
                    Chunk<E>::unpack(wpost[j], w);
#pragma unroll
                    for (int i = 0; i < N; i++) z[i] *= w[i];
                }
                if (gate_ch) {
                    Chunk<E>::unpack(wgate[j], w);
#pragma unroll
                    for (int i = 0; i < N; i++) z[i] *= w[i];
                }
#pragma unroll
                for (int i = 0; i < N; i++) r[j][i] = fmaf(s, z[i], r[j][i]);
                store_chunk(to_r, sub * bytes + at[j], Chunk<E>::pack(r[j]));
            }
#pragma unroll
            for (int i = 0; i < N; i++) ssq[0] = fmaf(r[j][i], r[j][i], ssq[0]);
        }
        if (a.h) {
            row_sums<NT>(ssq, slots, turn);
            const float rstd = rstd_of(ssq[0], a.inv_d, a.eps);
#pragma unroll
            for (int j = 0; j < VPT; j++) {
                float w[N];
                Chunk<E>::unpack(wpre[j], w);
#pragma unroll
                for (int i = 0; i < N; i++) w[i] *= r[j][i] * rstd;
                store_chunk(to_h, sub * bytes + at[j], Chunk<E>::pack(w));
            }
        }
        t0 += gridDim.x * kRows;
        if (t0 >= a.T) break;
        load(t0);
    }
}

// What the column sums end as.  With S of dz n(y), dz without the channel
// gate: dw_post = gate S, dgate = w_post S.
template <typename E>
struct ColumnOut {
    const E *w_post, *gate_ch;
    float *dw_post, *dgate_ch, *dw_pre;

    __device__ __forceinline__ bool wants(int k) const { return k ? dw_pre != nullptr : dw_post || dgate_ch; }
    __device__ __forceinline__ void store(int k, int c, float v) const {
        const auto value = [](E e) {
            if constexpr (sizeof(E) == 2)
                return bf16_bits_to_f32(e);
            else
                return e;
        };
        if (k) {
            dw_pre[c] = v;
            return;
        }
        if (dw_post) dw_post[c] = gate_ch ? value(gate_ch[c]) * v : v;
        if (dgate_ch) dgate_ch[c] = w_post ? value(w_post[c]) * v : v;
    }
};

struct NormBackArgs {
    const u32x4 *dr, *dh, *r, *y, *w_post, *w_pre;
    const void *gate;
    u32x4 *dx, *dy;
    float *dgate_tok;  // T values (gate_kind 2)
    float *part;       // [workgroup][2][d]: column sums of dz n(y) and of dh n(r)
    unsigned T;
    int chunks, gate_kind;
    float inv_d, eps, scale;
};

// One chunk of a row per thread.
template <typename E, int NT>
__global__ __launch_bounds__(kBackBlock) void k_norm_back(NormBackArgs a, ColumnOut<E> o) {
    constexpr int N = Chunk<E>::N, kRows = kBackBlock / NT;
    __shared__ Slots slots;
    int turn = 0;
    const unsigned c = threadIdx.x % NT, sub = threadIdx.x / NT, bytes = a.chunks * 16;
    const bool gate_ch = a.gate_kind == 1, gate_tok = a.gate_kind == 2;
    const unsigned at = c < static_cast<unsigned>(a.chunks) ? 16 * c : kNowhere;  // in a row
    u32x4 drn, dhn, rn, yn;  // the next row's chunk
    float gtn;
    auto load = [&](unsigned t0) {
        const Rows rows(t0, kRows, a.T, bytes);
        const auto chunk = [&](const u32x4 *p) { return load_chunk(rows.of(p), sub * bytes + at); };
        drn = chunk(a.dr);
        dhn = chunk(a.dh);
        rn = chunk(a.dh ? a.r : nullptr);
        yn = chunk(a.y);
        gtn = load_float(Rows(t0, kRows, a.T, 4).of(gate_tok ? a.gate : nullptr), sub * 4);
    };
    const unsigned stride = gridDim.x * kRows;
    load(blockIdx.x * kRows);
    const u32x4 wpre = load_chunk(buffer_of(a.w_pre, bytes), at);
    const u32x4 wpost = load_chunk(buffer_of(a.w_post, bytes), at);
    const u32x4 wgate = load_chunk(buffer_of(gate_ch ? a.gate : nullptr, bytes), at);
    float gw[N];  // channel gate times w_post
    float acc_y[N], acc_r[N];
    {
        float g[N];
        Chunk<E>::unpack(wpost, gw);
        Chunk<E>::unpack(wgate, g);
#pragma unroll
        for (int i = 0; i < N; i++) {
            gw[i] = (a.w_post ? gw[i] : 1.f) * (gate_ch ? g[i] : 1.f);
            acc_y[i] = acc_r[i] = 0.f;
        }
    }
    // the trip count is the workgroup's: its rows' sums may need barriers
    for (unsigned t0 = blockIdx.x * kRows; t0 < a.T; t0 += stride) {
        float q[N], dh[N], r[N], y[N], w[N];
        Chunk<E>::unpack(drn, q);
        Chunk<E>::unpack(dhn, dh);
        Chunk<E>::unpack(rn, r);
        Chunk<E>::unpack(yn, y);
        Chunk<E>::unpack(wpre, w);
        const float gt = gate_tok ? gtn : 1.f;
        load(t0 + stride);
        float sums[3] = {0.f, 0.f, 0.f};  // r.r, (dh w_pre).r, y.y
#pragma unroll
        for (int i = 0; i < N; i++) {
            w[i] *= dh[i];
            sums[0] = fmaf(r[i], r[i], sums[0]);
            sums[1] = fmaf(w[i], r[i], sums[1]);
            sums[2] = fmaf(y[i], y[i], sums[2]);
        }
        row_sums<NT>(sums, slots, turn);
        const float rstd_r = rstd_of(sums[0], a.inv_d, a.eps);
        const float mean_r = sums[1] * a.inv_d * rstd_r;  // of (dh w_pre) n(r)
        const float rstd_y = a.w_post ? rstd_of(sums[2], a.inv_d, a.eps) : 1.f;
        const float sg = a.scale * gt;
        // (without dh or y their terms are zero)
#pragma unroll
        for (int i = 0; i < N; i++) {
            r[i] *= rstd_r;  // n(r)
            acc_r[i] = fmaf(dh[i], r[i], acc_r[i]);
            q[i] = fmaf(rstd_r, fmaf(-mean_r, r[i], w[i]), q[i]);
        }
        // q is dr', and then dr' gate_ch w_post
        const Rows rows(t0, kRows, a.T, bytes);
        store_chunk(rows.of(a.dx), sub * bytes + at, Chunk<E>::pack(q));
        float dot[1] = {0.f};  // (dr' gate_ch w_post).n(y)
#pragma unroll
        for (int i = 0; i < N; i++) {
            y[i] *= rstd_y;  // n(y)
            acc_y[i] = fmaf(q[i] * sg, y[i], acc_y[i]);
            q[i] *= gw[i];
            dot[0] = fmaf(q[i], y[i], dot[0]);
        }
        float mean_y = 0.f;
        if (a.w_post || gate_tok) {
            row_sums<NT>(dot, slots, turn);
            if (a.w_post) mean_y = dot[0] * a.inv_d;
            if (gate_tok)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(a.scale * dot[0]),
                                                      Rows(t0, kRows, a.T, 4).of(a.dgate_tok),
                                                      c == 0 ? sub * 4 : kNowhere, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < N; i++) q[i] = sg * rstd_y * fmaf(-mean_y, y[i], q[i]);
        store_chunk(rows.of(a.dy), sub * bytes + at, Chunk<E>::pack(q));
    }

    // this workgroup's column sums, its rows' added in order; a single
    // workgroup's are the outputs
    const int d = a.chunks * N;
    float *out = a.part + static_cast<size_t>(blockIdx.x) * 2 * d;
    __shared__ float col[kRows][NT * N];
#pragma unroll
    for (int k = 0; k < 2; k++) {
        if (!o.wants(k)) continue;
        __syncthreads();  // the sums before these have been read
#pragma unroll
        for (int i = 0; i < N; i++) col[sub][c * N + i] = k ? acc_r[i] : acc_y[i];
        __syncthreads();
        for (int j = threadIdx.x; j < d; j += kBackBlock) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < kRows; q++) s += col[q][j];
            if (gridDim.x == 1)
                o.store(k, j, s);
            else
                out[k * d + j] = s;
        }
    }
}

// Column c's sums over the workgroups: each of 16 interleaved shares in
// order, then the shares in order.
constexpr int kFoldCols = 64, kFoldShares = 16;
template <typename E>
__global__ __launch_bounds__(kFoldCols *kFoldShares) void k_norm_fold(const float *__restrict__ part,
                                                                      int blocks, int d,
                                                                      ColumnOut<E> o) {
    __shared__ float s_sum[kFoldShares][kFoldCols];
    if (!o.wants(blockIdx.y)) return;
    const int c = blockIdx.x * kFoldCols + threadIdx.x % kFoldCols, sh = threadIdx.x / kFoldCols;
    float v = 0.f;
    if (c < d)
#pragma unroll 8
        for (int b = sh; b < blocks; b += kFoldShares)
            v += part[(static_cast<size_t>(b) * 2 + blockIdx.y) * d + c];
    s_sum[sh][threadIdx.x % kFoldCols] = v;
    __syncthreads();
    if (sh || c >= d) return;
    for (int q = 1; q < kFoldShares; q++) v += s_sum[q][threadIdx.x];
    o.store(blockIdx.y, c, v);
}

// Forward: threads that share a row of `chunks` chunks and chunks of each.
template <typename F>
void by_width(int chunks, F f) {
    using std::integral_constant;
    if (chunks <= 16)
        f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    else if (chunks <= 32)
        f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
    else if (chunks <= 64)
        f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (chunks <= 128)
        f(integral_constant<int, 128>{}, integral_constant<int, 1>{});
    else if (chunks <= 256)
        f(integral_constant<int, 128>{}, integral_constant<int, 2>{});
    else if (chunks <= 512)
        f(integral_constant<int, 512>{}, integral_constant<int, 1>{});
    else
        f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
}

// Backward: threads that share a row, one per chunk.
template <typename F>
void by_width_back(int chunks, F f) {
    using std::integral_constant;
    if (chunks <= 16)
        f(integral_constant<int, 16>{});
    else if (chunks <= 32)
        f(integral_constant<int, 32>{});
    else if (chunks <= 64)
        f(integral_constant<int, 64>{});
    else if (chunks <= 128)
        f(integral_constant<int, 128>{});
    else if (chunks <= 256)
        f(integral_constant<int, 256>{});
    else if (chunks <= 512)
        f(integral_constant<int, 512>{});
    else
        f(integral_constant<int, 1024>{});
}

}  // namespace

// Backward workgroups at most: one per CU, since each leaves 2 d fp32 sums
// behind (T = 8192, d = 2048: 48 us a call; two per CU 54).
constexpr int kNormBackBlocks = 256;

// Up to this many rows for each of its teams a batch takes one workgroup,
// whose sums need no second kernel: T = 16, d = 2048 12.0 us a call, where the
// host launching twice takes 15.5 (captured: 11.1 against 8.5).
constexpr unsigned kOneBlockRows = 4;

int norm_back_blocks(int T, int chunks) {
    unsigned need = 0;
    by_width_back(chunks, [&](auto nt) { need = ceil_div(T, kBackBlock / decltype(nt)::value); });
    if (need <= kOneBlockRows) return 1;
    return static_cast<int>(std::min(need, static_cast<unsigned>(kNormBackBlocks)));
}

hipError_t launch_block_norm(const void *x, const void *y, const void *w_post, const void *gate,
                             const void *w_pre, int T, int d, int bf16, int gate_kind, float eps,
                             float scale, void *r, void *h, hipStream_t s) {
    NormArgs a;
    a.x = static_cast<const u32x4 *>(x);
    a.y = static_cast<const u32x4 *>(y);
    a.w_post = static_cast<const u32x4 *>(w_post);
    a.w_pre = static_cast<const u32x4 *>(w_pre);
    a.gate = gate;
    a.r = static_cast<u32x4 *>(r);
    a.h = static_cast<u32x4 *>(h);
    a.T = T;
    a.chunks = d / (bf16 ? 8 : 4);
    a.gate_kind = gate_kind;
    a.inv_d = 1.f / static_cast<float>(d);
    a.eps = eps;
    a.scale = scale;
    by_width(a.chunks, [&](auto nt, auto vpt) {
        constexpr int NT = decltype(nt)::value, VPT = decltype(vpt)::value;
        // one row per team, up to the most threads that a launch holds
        const unsigned grid = std::min(ceil_div(T, kBlock<NT> / NT), 1u << 22);
        if (bf16)
            k_norm<uint16_t, NT, VPT><<<grid, kBlock<NT>, 0, s>>>(a);
        else
            k_norm<float, NT, VPT><<<grid, kBlock<NT>, 0, s>>>(a);
    });
    return hipGetLastError();
}

hipError_t launch_block_norm_back(const void *dr, const void *dh, const void *r, const void *y,
                                  const void *w_post, const void *gate, const void *w_pre, int T,
                                  int d, int bf16, int gate_kind, float eps, float scale, void *dx,
                                  void *dy, float *dw_post, float *dgate, float *dw_pre,
                                  float *part, hipStream_t s) {
    NormBackArgs a;
    a.dr = static_cast<const u32x4 *>(dr);
    a.dh = static_cast<const u32x4 *>(dh);
    a.r = static_cast<const u32x4 *>(r);
    // y matters to its norm's and its gate's gradients only
    a.y = w_post || gate ? static_cast<const u32x4 *>(y) : nullptr;
    a.w_post = static_cast<const u32x4 *>(w_post);
    a.w_pre = static_cast<const u32x4 *>(w_pre);
    a.gate = gate;
    a.dx = static_cast<u32x4 *>(dx);
    a.dy = static_cast<u32x4 *>(dy);
    a.dgate_tok = gate_kind == 2 ? dgate : nullptr;
    a.part = part;
    a.T = T;
    a.chunks = d / (bf16 ? 8 : 4);
    a.gate_kind = gate_kind;
    a.inv_d = 1.f / static_cast<float>(d);
    a.eps = eps;
    a.scale = scale;
    const int grid = norm_back_blocks(T, a.chunks);
    const auto run = [&](auto e) {
        typedef decltype(e) E;
        const bool ch = gate_kind == 1;
        const ColumnOut<E> o = {static_cast<const E *>(w_post),
                                ch ? static_cast<const E *>(gate) : nullptr, dw_post,
                                ch ? dgate : nullptr, dw_pre};
        by_width_back(a.chunks, [&](auto nt) {
            k_norm_back<E, decltype(nt)::value><<<grid, kBackBlock, 0, s>>>(a, o);
        });
        if (grid > 1 && (dw_post || o.dgate_ch || dw_pre))
            k_norm_fold<E><<<dim3(ceil_div(d, kFoldCols), 2), kFoldCols * kFoldShares, 0, s>>>(
                part, grid, d, o);
    };
    if (bf16)
        run(uint16_t{});
    else
        run(float{});
    return hipGetLastError();
}

}  // namespace occ
