// One AdamW step over many tensors, moments in fp32 or in 8 bits.
//
// Mathematics, g' = grad_scale g:
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2,
//   p = (1 - lr wd) p - (lr / c1) m / (sqrt(v) / sqrt(c2) + eps),  c = 1 - b^step.
// In 8 bits m and sqrt(v) are e4m3 codes (the hardware's conversions) with an
// fp32 unit per 256 elements, the largest magnitude / 448: the moments are
// formed and used in fp32 and rounded once, to 4 significant bits (2^-4
// relative), which the block's unit keeps within e4m3's range down to 2^-17
// of the largest.
//
// Memory bound: per element 16 bytes in and 12 out in fp32 (14 with the bf16
// copy), 10 + 6 in 8 bits.  One launch takes up to kMaxTensors tensors, whose
// table travels by value in the kernel's arguments (no device copy of it to
// keep), and cuts them into pieces of kPiece elements; a workgroup finds its
// tensor from its number and moves one piece with 16-byte accesses, four
// elements per lane.  A wave's 64 lanes then hold the 256 elements of one
// 8-bit block, whose largest magnitude is a wave maximum.  The workgroups cross
// the tensors in order: pieces of 4 elements per lane measure 2110 us for 403 M
// elements in fp32 (5.7 TB/s; 2050 to 2190 with the addresses), of 8 2297, of 16
// 2250, of 32 2319.  All of a lane's loads are in flight at once (one behind
// the other, 8 bits 127 us for 35 M elements against 112, 5.6 TB/s), but for
// the largest fp32 states.  Workgroups of 1024 threads: small tensors 40%
// slower, the largest 3% either way.  IEEE square roots and divisions cost 8
// bits 10%.
#include <type_traits>

#include "launch.h"

namespace occ {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = kThreads * 4;  // elements of a workgroup
constexpr int kMaxTensors = 30;
constexpr uint64_t kMaxBlocks = 0xffffffffull / kThreads;  // a launch holds fewer than 2^32 threads
static_assert(kAdamwMaxElements / kPiece < kMaxBlocks, "one tensor fits a launch");
constexpr int kQBlock = kWave * 4;  // OCC_ADAMW_BLOCK

constexpr float kE4m3Max = 448.f, kE4m3Min = 0x1p-9f, kSmallest = 0x1p-100f;

struct Table {
    AdamwTensor t[kMaxTensors];
    uint32_t first[kMaxTensors];  // first workgroup of each tensor
    int count;
};
static_assert(sizeof(Table) + sizeof(AdamwStep) <= 4096, "kernel arguments");

// Four consecutive values from element i of n, as one vector (WHOLE) or each by
// itself, zero behind the end.  No load is under a condition, so that all of a
// lane's are in flight at once.
template <bool WHOLE, typename V, typename E>
__device__ __forceinline__ void load4(const void *p, int64_t i, int64_t n, E (&v)[4]) {
    const E *q = static_cast<const E *>(p);
    if constexpr (WHOLE) {
        const V x = *reinterpret_cast<const V *>(q + i);
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] = reinterpret_cast<const E *>(&x)[j];
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] = q[min(i + j, n - 1)];
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] = i + j < n ? v[j] : static_cast<E>(0);
    }
}
template <bool WHOLE, typename V, typename E>
__device__ __forceinline__ void store4(void *p, int64_t i, int64_t n, const E (&v)[4]) {
    E *q = static_cast<E *>(p) + i;
    if constexpr (WHOLE) {
        V x;
#pragma unroll
        for (int j = 0; j < 4; j++) reinterpret_cast<E *>(&x)[j] = v[j];
        *reinterpret_cast<V *>(q) = x;
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (i + j < n) q[j] = v[j];
    }
}

__device__ __forceinline__ void from_e4m3(uint32_t codes, float unit, float (&v)[4]) {
    v[0] = unit * __builtin_amdgcn_cvt_f32_fp8(codes, 0);
    v[1] = unit * __builtin_amdgcn_cvt_f32_fp8(codes, 1);
    v[2] = unit * __builtin_amdgcn_cvt_f32_fp8(codes, 2);
    v[3] = unit * __builtin_amdgcn_cvt_f32_fp8(codes, 3);
}
__device__ __forceinline__ uint32_t to_e4m3(const float (&v)[4]) {
    int c = 0;
    c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], c, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], c, true);
    return static_cast<uint32_t>(c);
}

// The wave's 256 values as codes, and their unit.  keep[j]: a value that is
// not zero keeps a code that is not.  One value that is not finite makes the
// unit so and with it all 256: an infinity is the largest magnitude, a NaN,
// which a maximum passes over, is looked for by itself.
template <bool KEEP>
__device__ __forceinline__ uint32_t quantise(const float (&v)[4], const float (&keep)[4],
                                             float &unit) {
    float top = wave_max(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])),
                               fmaxf(fabsf(v[2]), fabsf(v[3]))));
    if (__any(__builtin_isunordered(v[0], v[1]) || __builtin_isunordered(v[2], v[3]))) top = NAN;
    unit = 0.f;
    float c[4] = {0.f, 0.f, 0.f, 0.f};
    if (!(top < kSmallest)) {
        unit = top / kE4m3Max;
        const float per = kE4m3Max / top;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            c[j] = v[j] * per;
            // NaN passes both
            c[j] = c[j] > kE4m3Max ? kE4m3Max : c[j] < -kE4m3Max ? -kE4m3Max : c[j];
            if (KEEP && keep[j] > 0.f && c[j] < kE4m3Min) c[j] = kE4m3Min;
        }
    }
    return to_e4m3(c);
}

// STAGED: one load of a lane behind the other.  Waves fill the memory's queues
// either way; above kStagedElements the four streams disturb each other less
// (fp32, 403 M elements 2125 us against 2215, 268 M 1414 against 1476; 134 M 700
// and 699, 34 M 194 against 190, six small tensors 4.3 against 3.6).
constexpr uint64_t kStagedElements = 1ull << 27;
template <bool STAGED>
__device__ __forceinline__ void stage_end() {
    if constexpr (STAGED) {
        __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <bool Q8, bool GBF16, bool STAGED, bool WHOLE>
__device__ __forceinline__ void update(const AdamwTensor &T, int64_t i, const AdamwStep &st) {
    const int64_t n = T.n;
    float p[4], g[4], m[4], v[4];
    load4<WHOLE, f32x4, float>(T.p, i, n, p);
    stage_end<STAGED>();
    if constexpr (GBF16) {
        typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
        uint16_t gb[4];
        load4<WHOLE, u16x4, uint16_t>(T.g, i, n, gb);
#pragma unroll
        for (int j = 0; j < 4; j++) g[j] = bf16_bits_to_f32(gb[j]);
    } else {
        load4<WHOLE, f32x4, float>(T.g, i, n, g);
    }
    stage_end<STAGED>();
    const int64_t qb = i / kQBlock;
    if constexpr (Q8) {
        typedef uint8_t u8x4 __attribute__((ext_vector_type(4)));
        uint8_t mc[4], vc[4];
        load4<WHOLE, u8x4, uint8_t>(T.m, i, n, mc);
        load4<WHOLE, u8x4, uint8_t>(T.v, i, n, vc);
        // a lane behind the end holds zeros; its block exists (the wave's first lane's does)
        from_e4m3(mc[0] | mc[1] << 8 | mc[2] << 16 | static_cast<uint32_t>(mc[3]) << 24,
                  T.m_scale[qb], m);
        from_e4m3(vc[0] | vc[1] << 8 | vc[2] << 16 | static_cast<uint32_t>(vc[3]) << 24,
                  T.v_scale[qb], v);
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] *= v[j];
    } else {
        load4<WHOLE, f32x4, float>(T.m, i, n, m);
        stage_end<STAGED>();
        load4<WHOLE, f32x4, float>(T.v, i, n, v);
    }
    float lr = st.lr, c1 = st.c1, c2_rsqrt = st.c2_rsqrt, gs = st.grad_scale;
    if (st.dynamic) {
        lr = st.dynamic[0];
        const float step = st.dynamic[1];
        gs = st.dynamic[2];
        c1 = -expm1f(step * st.log_b1);
        c2_rsqrt = 1.f / sqrtf(-expm1f(step * st.log_b2));
    }
    const float decay = fmaf(-lr, st.weight_decay, 1.f), rate = lr / c1;
    float root[4];
    uint16_t copy[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float gj = g[j] * gs;
        m[j] = fmaf(st.beta1, m[j], st.one_b1 * gj);
        v[j] = fmaf(st.beta2, v[j], st.one_b2 * gj * gj);
        // hardware square root and reciprocal: 2^-23 relative of the step each;
        // they take no subnormal value (eps keeps the divisor a normal one)
        const bool low = v[j] < 0x1p-96f;
        root[j] = __builtin_amdgcn_sqrtf(low ? 0x1p64f * v[j] : v[j]) * (low ? 0x1p-32f : 1.f);
        p[j] = fmaf(decay, p[j], -rate * (m[j] * __builtin_amdgcn_rcpf(fmaf(root[j], c2_rsqrt, st.eps))));
        copy[j] = f32_to_bf16_bits(p[j]);
    }
    store4<WHOLE, f32x4, float>(T.p_out, i, n, p);
    if (T.p_bf16) {
        typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
        store4<WHOLE, u16x4, uint16_t>(T.p_bf16, i, n, copy);
    }
    if constexpr (Q8) {
        typedef uint8_t u8x4 __attribute__((ext_vector_type(4)));
        float um, uv;
        const uint32_t qm = quantise<false>(m, m, um), qv = quantise<true>(root, v, uv);
        const uint8_t mc[4] = {static_cast<uint8_t>(qm), static_cast<uint8_t>(qm >> 8),
                               static_cast<uint8_t>(qm >> 16), static_cast<uint8_t>(qm >> 24)};
        const uint8_t vc[4] = {static_cast<uint8_t>(qv), static_cast<uint8_t>(qv >> 8),
                               static_cast<uint8_t>(qv >> 16), static_cast<uint8_t>(qv >> 24)};
        store4<WHOLE, u8x4, uint8_t>(T.m_out, i, n, mc);
        store4<WHOLE, u8x4, uint8_t>(T.v_out, i, n, vc);
        if (lane_id() == 0) {
            T.m_scale_out[qb] = um;
            T.v_scale_out[qb] = uv;
        }
    } else {
        store4<WHOLE, f32x4, float>(T.m_out, i, n, m);
        store4<WHOLE, f32x4, float>(T.v_out, i, n, v);
    }
}

// A whole piece of a tensor moves in vectors, a tensor's last one and pieces of
// arrays off the vectors' borders value by value.
template <bool Q8, bool GBF16, bool STAGED>
__global__ __launch_bounds__(kThreads) void k_adamw(Table tab, AdamwStep st) {
    int a = 0;
    for (int hi = tab.count; hi - a > 1;) {  // the last tensor with first <= blockIdx.x
        const int mid = (a + hi) >> 1;
        if (tab.first[mid] <= blockIdx.x)
            a = mid;
        else
            hi = mid;
    }
    const AdamwTensor &T = tab.t[a];
    const int64_t i0 = static_cast<int64_t>(blockIdx.x - tab.first[a]) * kPiece;
    // a wave whose elements all lie behind the tensor's end has nothing to do
    if (i0 + (threadIdx.x & ~(kWave - 1)) * 4 >= T.n) return;
    if (T.aligned && i0 + kPiece <= T.n)
        update<Q8, GBF16, STAGED, true>(T, i0 + threadIdx.x * 4, st);
    else
        update<Q8, GBF16, STAGED, false>(T, i0 + threadIdx.x * 4, st);
}

}  // namespace

hipError_t launch_adamw(const AdamwTensor *tensors, int count, const AdamwStep &st, int q8,
                        int grad_bf16, hipStream_t s) {
    int i = 0;
    while (i < count) {
        Table tab;
        tab.count = 0;
        uint64_t blocks = 0;
        for (; i < count && tab.count < kMaxTensors; i++) {
            if (tensors[i].n == 0) continue;
            const uint64_t need = static_cast<uint64_t>((tensors[i].n + kPiece - 1) / kPiece);
            if (blocks && blocks + need > kMaxBlocks) break;
            tab.t[tab.count] = tensors[i];
            tab.first[tab.count] = static_cast<uint32_t>(blocks);
            tab.count++;
            blocks += need;
        }
        if (tab.count == 0) continue;
        const unsigned grid = static_cast<unsigned>(blocks);
        const bool staged = blocks * kPiece > kStagedElements;
        const auto run = [&](auto q, auto g, auto staging) {
            k_adamw<decltype(q)::value, decltype(g)::value, decltype(staging)::value>
                <<<grid, kThreads, 0, s>>>(tab, st);
        };
        const auto by_grad = [&](auto q, auto staging) {
            if (grad_bf16)
                run(q, std::true_type{}, staging);
            else
                run(q, std::false_type{}, staging);
        };
        if (q8)
            by_grad(std::true_type{}, std::false_type{});
        else if (staged)
            by_grad(std::false_type{}, std::true_type{});
        else
            by_grad(std::false_type{}, std::false_type{});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace occ
