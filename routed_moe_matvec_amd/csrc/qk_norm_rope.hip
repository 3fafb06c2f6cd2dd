// RMS norm of queries and keys, head by head, and their rotation by position.
//
//   u_c = x_c / sqrt(mean_c x_c^2 + eps) * w_c;  a pair (a, b) of channels turns by t = position * freq_i:
//   y_a = u_a cos t - u_b sin t,  y_b = u_b cos t + u_a sin t;  channels from R on stay u.
//
// One pass: a lane holds 16 channels of a head (Dh / 16 lanes a head), whole pairs
// among them, so the rotation needs no exchange and the norm's sum four steps between
// neighbours at most.  The angle is taken in 64 bits, exact but for one rounding of
// position * freq, and brought to within an eighth of a turn; sine and cosine are
// sums of their power series there, in fp32.  A wave computes those of its token
// once, a lane each, and shares them through LDS.
//
// Bound by memory: 31 k tokens of 40 heads of 128 in bf16 112 to 124 us, 5.1 to 5.7 TB/s (copies
// of such sizes reach 5.1 to 5.5), 4094 tokens of 20 heads of 256 from fp32 to bf16 21 us,
// 6.0 TB/s, part of it in the last-level cache.  A wave with two to five groups of heads, its
// sines shared by them, took 3% less to 8% more for these two, and 3.8 to 5.5 us for 32 tokens in
// place of 3.4.  Small calls are one round trip to memory, so everything is asked for at once.
#include <type_traits>

#include "common.h"
#include "kv4_device.h"

namespace qg {

struct RopeArgs {
    const void *x[2];       // queries, keys
    void *y[2];
    const float *w[2];
    const float *freq;
    const int32_t *cu, *lens;
    int32_t *status;
    int ldx[2], ldy[2];
    int n, B, H, heads, R;  // heads: of queries and keys
    int waves;              // of a token
    float eps;
};

constexpr int kRopeWaves = 4;
constexpr int kRopeMaxLen = 0x3fffffff;

// cos and sin of x, of any size below 2^40.
__device__ __forceinline__ f32x2 cos_sin(double x) {
    const double n = __builtin_rint(x * 0.63661977236758134308);  // quarter turns
    // pi / 2 as the sum of two doubles
    const double r = __builtin_fma(-n, 6.12323399573676588613e-17, __builtin_fma(-n, 1.57079632679489661923, x));
    const int quarter = (int)(n - 4.0 * __builtin_floor(n * 0.25));
    const float f = (float)r, z = f * f;  // |f| <= pi / 4: the first term left out is below 2^-28 of the sum
    float s = __builtin_fmaf(z, 1.f / 362880, -1.f / 5040);
    s = __builtin_fmaf(z, s, 1.f / 120);
    s = __builtin_fmaf(z, s, -1.f / 6);
    s = __builtin_fmaf(z * f, s, f);
    float c = __builtin_fmaf(z, -1.f / 3628800, 1.f / 40320);
    c = __builtin_fmaf(z, c, -1.f / 720);
    c = __builtin_fmaf(z, c, 1.f / 24);
    c = __builtin_fmaf(z, c, -0.5f);
    c = __builtin_fmaf(z, c, 1.f);
    const float cc = quarter & 1 ? s : c, ss = quarter & 1 ? c : s;
    return f32x2{quarter == 1 || quarter == 2 ? -cc : cc, quarter & 2 ? -ss : ss};
}

// Sum over the 4, 8 or 16 lanes of a head, the same in each.
template <int LANES>
__device__ __forceinline__ float head_sum(float x) {
    auto from = [](float v, auto ctrl) {
        return __builtin_bit_cast(
            float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    x += from(x, std::integral_constant<int, 0xb1>{});                        // lane ^ 1
    x += from(x, std::integral_constant<int, 0x4e>{});                        // lane ^ 2
    if (LANES > 4) x += from(x, std::integral_constant<int, 0x141>{});  // the other four of eight
    if (LANES > 8) x += from(x, std::integral_constant<int, 0x140>{});  // the other eight of sixteen
    return x;
}

__device__ __forceinline__ bool rope_lengths_ok(const RopeArgs &a, int c0, int c1, int len) {
    return c0 >= 0 && c1 >= c0 && c1 <= a.n && len >= c1 - c0 && len <= kRopeMaxLen;
}

// Element j of 16 bytes.
template <class T>
__device__ __forceinline__ float element(u32x4 w, int j) {
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(float, (uint32_t)w[j]);
    } else {
        typedef T pair __attribute__((ext_vector_type(2)));
        return (float)__builtin_bit_cast(pair, (uint32_t)w[j / 2])[j % 2];
    }
}

template <int TIN, int TOUT, int DH, bool NEIGHBOURS>
__global__ __launch_bounds__(kRopeWaves *kWave) void qk_norm_rope_kernel(RopeArgs a) {
    typedef typename ElemOf<TIN>::type T;
    typedef typename ElemOf<TOUT>::type U;
    constexpr int LANES = DH / 16, HEADS = kWave / LANES;  // lanes of a head, heads of a wave
    constexpr int E = 16 / (int)sizeof(T), NP = 16 / E;    // elements of 16 bytes, places of a lane
    constexpr int NF = (DH / 2 + kWave - 1) / kWave;       // frequencies of a lane
    __shared__ __attribute__((aligned(16))) f32x2 turns[kRopeWaves][DH / 2];
    const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wave = blockIdx.x * kRopeWaves + wv;
    if (blockIdx.x == 0)  // every length once: one out of order may otherwise go unseen
        for (int b = threadIdx.x; b < a.B; b += kRopeWaves * kWave)
            if (!rope_lengths_ok(a, a.cu[b], a.cu[b + 1], a.lens[b])) kv4_report(a.status, QG_DEV_BAD_LENGTH);
    const int tok = wave / a.waves;
    if (tok >= a.n) return;

    // The lane's 16 channels: 16 bytes each of NP places, neighbouring lanes' side by side.
    // Of the R / 16 lanes that turn, elements j and 8 + j are a pair of QG_ROPE_HALVES, 2 j and 2 j + 1 of
    // QG_ROPE_NEIGHBOURS.
    const int i = lane % LANES, turning = a.R / 16, asked = wave % a.waves * HEADS + lane / LANES;
    const bool turned = i < turning, mine = asked < a.heads;
    const int h = mine ? asked : 0;  // lanes behind the last head read the first, and write nothing
    const bool key = h >= a.H;
    int at[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int halves = k < NP / 2 ? E * (i + turning * k) : a.R / 2 + E * (i + turning * (k - NP / 2));
        at[k] = !turned ? a.R + E * (i - turning + (LANES - turning) * k) : NEIGHBOURS ? E * (i + turning * k) : halves;
    }
    // all that is read, at once
    u32x4 raw[NP];
    f32x4 w[4];
    float freq[NF];
    const T *xp = key ? (const T *)a.x[1] + (size_t)tok * a.ldx[1] + (h - a.H) * DH
                      : (const T *)a.x[0] + (size_t)tok * a.ldx[0] + h * DH;
    const float *wp = a.w[key];
#pragma unroll
    for (int k = 0; k < NP; ++k) raw[k] = *(const u32x4 *)(xp + at[k]);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = f32x4{1.f, 1.f, 1.f, 1.f};
    if (wp)
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = *(const f32x4 *)(wp + at[4 * j / E] + 4 * j % E);
#pragma unroll
    for (int f = 0; f < NF; ++f) freq[f] = f * kWave + lane < a.R / 2 ? a.freq[f * kWave + lane] : 0.f;
    int c0, c1, len;
    if (a.B <= kWave) {  // a sequence a lane: no second round trip
        const int s = min(lane, a.B - 1), first = a.cu[s], end = a.cu[s + 1], held = a.lens[s];
        const unsigned long long le = __ballot(lane < a.B && (lane == 0 || first <= tok));
        const int b = 63 - __builtin_clzll(le);
        c0 = __builtin_amdgcn_readlane(first, b);
        c1 = __builtin_amdgcn_readlane(end, b);
        len = __builtin_amdgcn_readlane(held, b);
    } else {
        const int b = wave_find_last(a.B, tok, [&](int s) { return a.cu[s]; });
        c0 = load_uniform(a.cu + b);
        c1 = load_uniform(a.cu + b + 1);
        len = load_uniform(a.lens + b);
    }
    if (!rope_lengths_ok(a, c0, c1, len) || tok < c0 || tok >= c1) return;

    const double pos = (double)(len - c1 + tok);
#pragma unroll
    for (int f = 0; f < NF; ++f)
        if (f * kWave + lane < DH / 2) turns[wv][f * kWave + lane] = cos_sin(pos * (double)freq[f]);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    f32x2 turn[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {  // two frequencies side by side
        const int own = NEIGHBOURS ? at[2 * j / E] / 2 + j % (E / 2) : at[j / E] + j % E, f = turned ? own : 0;
        const f32x4 t = *(const f32x4 *)&turns[wv][f];
        turn[j] = f32x2{t[0], t[1]};
        turn[j + 1] = f32x2{t[2], t[3]};
    }
    if (!mine) return;
    float x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = element<T>(raw[j / E], j % E);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) sum = __builtin_fmaf(x[j], x[j], sum);
    sum = head_sum<LANES>(sum);
    auto inverse = [](float sum, float eps) { return 1.f / __builtin_sqrtf(sum * (1.f / DH) + eps); };
    float r;
    // Squares beyond fp32: those of elements 2^72 times smaller, of which 256 of the largest stay inside it.  Half of the
    // factor goes to the elements and half to r, which would be subnormal with all of it.
    if (TIN != QG_TYPE_F16 && !(sum <= 0x1p126f)) {
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float y = x[j] * 0x1p-72f;
            sum = __builtin_fmaf(y, y, sum);
            x[j] *= 0x1p-36f;
        }
        r = inverse(head_sum<LANES>(sum), a.eps * 0x1p-144f) * 0x1p-36f;
    } else {
        r = inverse(sum, a.eps);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] *= r;
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] *= w[j / 4][j % 4];
    U *y = key ? (U *)a.y[1] + (size_t)tok * a.ldy[1] + (h - a.H) * DH : (U *)a.y[0] + (size_t)tok * a.ldy[0] + h * DH;
    typedef U out_t __attribute__((ext_vector_type(E)));
    out_t out[NP];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int ja = NEIGHBOURS ? 2 * j : j, jb = NEIGHBOURS ? 2 * j + 1 : 8 + j;
        // what does not turn is not multiplied with its neighbour's 0 either: that may be Inf or NaN
        const float ya = __builtin_fmaf(x[ja], turn[j][0], -(x[jb] * turn[j][1]));
        const float yb = __builtin_fmaf(x[jb], turn[j][0], x[ja] * turn[j][1]);
        out[ja / E][ja % E] = (U)(turned ? ya : x[ja]);
        out[jb / E][jb % E] = (U)(turned ? yb : x[jb]);
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) *(out_t *)(y + at[k]) = out[k];
}

template <int TIN, int TOUT, int DH, bool NEIGHBOURS>
static int launch_rope(RopeArgs a, hipStream_t stream) {
    constexpr int HEADS = 1024 / DH;
    a.waves = (a.heads + HEADS - 1) / HEADS;
    const long long grid = ((long long)a.n * a.waves + kRopeWaves - 1) / kRopeWaves;
    hipLaunchKernelGGL((qk_norm_rope_kernel<TIN, TOUT, DH, NEIGHBOURS>), dim3((unsigned)grid), dim3(kRopeWaves * kWave), 0,
                       stream, a);
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

template <int TIN, int TOUT>
static int launch_rope_types(const RopeArgs &a, int Dh, bool neighbours, hipStream_t s) {
    switch (Dh) {
        case 64: return neighbours ? launch_rope<TIN, TOUT, 64, true>(a, s) : launch_rope<TIN, TOUT, 64, false>(a, s);
        case 128: return neighbours ? launch_rope<TIN, TOUT, 128, true>(a, s) : launch_rope<TIN, TOUT, 128, false>(a, s);
        default: return neighbours ? launch_rope<TIN, TOUT, 256, true>(a, s) : launch_rope<TIN, TOUT, 256, false>(a, s);
    }
}

}  // namespace qg

extern "C" int qk_norm_rope(int type, const void *q, int ldq, const void *k, int ldk, int n, const int32_t *cu,
                            const int32_t *lens, int B, int H, int Hkv, int Dh, const float *wq, const float *wk,
                            float eps, int R, int style, const float *freq, int out_type, void *q_out, int ldq_out,
                            void *k_out, int ldk_out, int32_t *d_status, void *stream) {
    using namespace qg;
    if (type != QG_TYPE_F32 && type != QG_TYPE_F16 && type != QG_TYPE_BF16) return QG_ERR_FORMAT;
    if (out_type != type && (type != QG_TYPE_F32 || (out_type != QG_TYPE_F16 && out_type != QG_TYPE_BF16)))
        return QG_ERR_FORMAT;
    if (style != QG_ROPE_HALVES && style != QG_ROPE_NEIGHBOURS) return QG_ERR_FORMAT;
    if (!q || !k || !cu || !lens || !q_out || !k_out || !d_status || (R > 0 && !freq)) return QG_ERR_NULL;
    if (n < 1 || n > QG_MAX_ATTN_TOKENS || B < 1 || B > QG_MAX_SEQS || H < 1 || H > QG_MAX_HEADS || Hkv < 1 ||
        Hkv > QG_MAX_HEADS || (Dh != 64 && Dh != 128 && Dh != 256) || R < 0 || R > Dh || R % 16 != 0 ||
        !(eps >= 0x1p-100f && eps <= 0x1p100f))
        return QG_ERR_SHAPE;
    if (!row_stride_ok(type, ldq, H * Dh) || !row_stride_ok(type, ldk, Hkv * Dh) ||
        !row_stride_ok(out_type, ldq_out, H * Dh) || !row_stride_ok(out_type, ldk_out, Hkv * Dh))
        return QG_ERR_SHAPE;
    if ((long long)n * ((((long long)H + Hkv) * Dh + 1023) / 1024) > 4 * kMaxGroups) return QG_ERR_SHAPE;
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)q_out | (uintptr_t)k_out | (uintptr_t)wq | (uintptr_t)wk) & 15)
        return QG_ERR_ALIGN;
    if (((uintptr_t)cu | (uintptr_t)lens | (uintptr_t)freq | (uintptr_t)d_status) & 3) return QG_ERR_ALIGN;
    // in place, but rows of another type or stride would land on heads that other waves still read
    if ((q_out == q && (out_type != type || ldq_out != ldq)) || (k_out == k && (out_type != type || ldk_out != ldk)))
        return QG_ERR_SHAPE;
    RopeArgs a{{q, k}, {q_out, k_out}, {wq, wk}, freq, cu, lens, d_status, {ldq, ldk}, {ldq_out, ldk_out},
               n, B, H, H + Hkv, R, 0, eps};
    const bool neighbours = style == QG_ROPE_NEIGHBOURS;
    hipStream_t s = (hipStream_t)stream;
    clear_stale_error();
    if (type == QG_TYPE_BF16) return launch_rope_types<QG_TYPE_BF16, QG_TYPE_BF16>(a, Dh, neighbours, s);
    if (type == QG_TYPE_F16) return launch_rope_types<QG_TYPE_F16, QG_TYPE_F16>(a, Dh, neighbours, s);
    switch (out_type) {
        case QG_TYPE_F32: return launch_rope_types<QG_TYPE_F32, QG_TYPE_F32>(a, Dh, neighbours, s);
        case QG_TYPE_F16: return launch_rope_types<QG_TYPE_F32, QG_TYPE_F16>(a, Dh, neighbours, s);
        default: return launch_rope_types<QG_TYPE_F32, QG_TYPE_BF16>(a, Dh, neighbours, s);
    }
}
