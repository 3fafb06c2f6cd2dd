// Writing and reading the paged FP4 key/value cache.
//
// kv4_append quantizes each 32 channels of a token's key or value to E2M1
// codes with one power-of-two scale: e = least integer >= -120 with
// max|x| <= 6 * 2^e, so nothing saturates, and x * 2^-e is exact in fp32, so
// codes and scales are the same on every machine.  kv4_gather is the inverse;
// an E2M1 value times 2^e is exact in bf16 and fp32.
//
// Both move (sizeof(type) + 17/32) bytes per element and compute little: bound
// by memory.  One wave takes four neighbouring positions (aligned to four in
// their page) of 16 chunks of 8 channels: its reads of a token are runs of 256
// bytes (16-bit types, Dh = 128), and the codes it writes are one run of 256
// bytes in either half of the page.
#include "common.h"
#include "kv4_device.h"

namespace qg {

struct Kv4Move {
    Kv4Cache c;
    void *k, *v;
    const int32_t *cu;
    int n, ldk, ldv;
    int units;  // pieces of a group of four positions
    int parts;  // waves that share a group
    int run;    // groups that a wave takes after each other
};

// Scale byte of a block with largest magnitude amax: e + 127.
__device__ __forceinline__ uint32_t kv4_scale_byte(float amax) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, amax) & 0x7fffffffu;
    const int s = (int)(bits >> 23) - 2 + ((bits & 0x7fffffu) > 0x400000u ? 1 : 0);  // 6 = 1.5 * 2^2
    return (uint32_t)min(max(s, 7), 254);
}

// E2M1 code of x * inv, |x * inv| <= 6: steps of 1/2 up to 2, 1 up to 4, then 2,
// ties to the even code.
__device__ __forceinline__ uint32_t e2m1_code(float x, float inv) {
    const float a = __builtin_fabsf(x * inv);
    const float lo = __builtin_rintf(a * 2.f), mid = __builtin_rintf(a) + 2.f, hi = __builtin_rintf(a * 0.5f) + 4.f;
    const float r = a <= 2.f ? lo : a <= 4.f ? mid : hi;
    const uint32_t code = (uint32_t)__builtin_fminf(r, 7.f);  // a NaN ends as 7
    return code | (__builtin_bit_cast(uint32_t, x) >> 31 << 3);
}

__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    *(f32x4 *)p = f32x4{x[0], x[1], x[2], x[3]};
    *(f32x4 *)(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}
__device__ __forceinline__ void store8(_Float16 *p, const float (&x)[8]) {
    f16x8 a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = (_Float16)x[i];
    *(f16x8 *)p = a;
}
__device__ __forceinline__ void store8(bf16_t *p, const float (&x)[8]) {
    bf16x8 a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = (bf16_t)x[i];
    *(bf16x8 *)p = a;
}

__device__ __forceinline__ bool kv4_lengths_ok(const Kv4Move &a, int c0, int c1, int len) {
    return c0 >= 0 && c1 >= c0 && c1 <= a.n && len >= c1 - c0 && len <= a.c.max_pages << a.c.page_log2;
}

// The packed tokens of sequence b are positions [len - (c1 - c0), len).  Groups
// of four aligned positions are numbered so that sequence b's begin at
// cu[b] / 4 + 2b: enough room for any lengths, found without a prefix sum.
struct Kv4Group {
    int b, from, upto;  // the sequence, its first group and the next sequence's
    bool ok;
    int c0, start, len;  // its first token, that token's position, and its end
};

__device__ __forceinline__ Kv4Group kv4_group(const Kv4Move &a, int group) {
    Kv4Group g;
    g.b = wave_find_last(a.c.B, group, [&](int s) { return (a.cu[s] >> 2) + 2 * s; });
    const int c0 = load_uniform(a.cu + g.b), c1 = load_uniform(a.cu + g.b + 1);
    g.len = load_uniform(a.c.lens + g.b);
    g.ok = kv4_lengths_ok(a, c0, c1, g.len);
    g.from = (c0 >> 2) + 2 * g.b;
    g.upto = g.b + 1 < a.c.B ? (c1 >> 2) + 2 * g.b + 2 : 0x7fffffff;
    g.c0 = c0;
    g.start = g.len - (c1 - c0);
    return g;
}

// A wave takes `run` groups after each other, UPW pieces of each: a piece is 16
// chunks of 8 channels of the four positions, keys and values (one head of 128
// channels, two of 64, half of one of 256).  A piece's head is the same for the
// whole wave, so a lane's offsets are computed once a group and a piece adds a
// scalar: with offsets per piece (290 instructions for each) the kernel was bound
// by them, 152 us for 107 k positions of 8 heads of 128 to bf16.  All loads of a
// group are issued before the first is used.
template <int TYPE, int DH, bool APPEND, int UPW>
__global__ __launch_bounds__(256) void kv4_move_kernel(Kv4Move a) {
    typedef typename ElemOf<TYPE>::type T;
    constexpr int PH = DH >= 128 ? DH / 128 : 1;  // pieces of a head
    const Kv4Cache &c = a.c;
    const int lane = lane_id(), t = lane & 3;
    const int wave = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (blockIdx.x == 0)  // every length once: one out of order may otherwise go unseen
        for (int b = threadIdx.x; b < c.B; b += 256)
            if (!kv4_lengths_ok(a, a.cu[b], a.cu[b + 1], c.lens[b])) kv4_report(c.status, QG_DEV_BAD_LENGTH);
    const int page = 1 << c.page_log2;
    const size_t region = kv4_region_bytes(page, DH);
    const int u0 = wave % a.parts * UPW;  // the wave's first piece
    // the lane's part of a piece: a head beside the piece's (64 channels), and a chunk
    const int lh = DH == 64 ? lane >> 5 : 0, lc = DH == 64 ? lane >> 2 & 7 : lane >> 2;
    const int first = wave / a.parts * a.run;
    Kv4Group g;
    for (int group = first; group < first + a.run; ++group) {
        if (group == first || group >= g.upto) g = kv4_group(a, group);
        const int pos0 = ((g.start >> 2) + (group - g.from)) * 4;
        if (!g.ok || pos0 >= g.len || pos0 + 3 < g.start) continue;
        const int id = kv4_page_of(c, g.b, pos0 >> c.page_log2);
        if (id < 0) continue;
        const int off0 = pos0 & (page - 1);
        const bool there = pos0 + t >= g.start && pos0 + t < g.len;
        const size_t tok = (size_t)(there ? g.c0 + pos0 + t - g.start : 0);
        T *krow = (T *)a.k + tok * a.ldk + lh * DH + lc * 8, *vrow = (T *)a.v + tok * a.ldv + lh * DH + lc * 8;
        uint8_t *kv = c.kv + (size_t)id * c.Hkv * region;
        // offsets in a head's region, of the piece that begins with chunk 0
        const uint32_t lr = DH == 64 ? (uint32_t)lh * (uint32_t)region : 0;
        const uint32_t ko = lr + (uint32_t)((off0 + t) * (DH / 2) + lc * 4);
        const uint32_t vo = lr + (uint32_t)(page * (DH / 2) + ((off0 >> 2) * (DH / 8) + lc) * 16 + t * 4);
        const uint32_t kso = lr + (uint32_t)(page * DH + (off0 + t) * (DH / 32) + lc / 4);
        const uint32_t vso = lr + (uint32_t)(page * (DH + DH / 32) + ((off0 >> 2) * (DH / 32) + lc / 4) * 4 + t);
        int h[UPW], ch[UPW];  // of each piece: head, first chunk
        bool mine[UPW];
#pragma unroll
        for (int u = 0; u < UPW; ++u) {
            h[u] = DH == 64 ? 2 * (u0 + u) : (u0 + u) / PH;
            ch[u] = DH == 256 ? (u0 + u) % PH * 16 : 0;
            mine[u] = there && h[u] + lh < c.Hkv;
            if (u0 + u >= a.units) h[u] = 0;  // no such piece: nothing is read or written for it
        }
        if constexpr (APPEND) {
            Raw8<T> x[UPW][2];
#pragma unroll
            for (int u = 0; u < UPW; ++u) {
                x[u][0] = x[u][1] = Raw8<T>{};
                if (mine[u]) {
                    x[u][0] = load8(krow + h[u] * DH + ch[u] * 8);
                    x[u][1] = load8(vrow + h[u] * DH + ch[u] * 8);
                }
            }
#pragma unroll
            for (int u = 0; u < UPW; ++u) {
                uint32_t w[2] = {0, 0}, s[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float m = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) m = __builtin_fmaxf(m, __builtin_fabsf(elem(x[u][i], j)));
                    m = __builtin_fmaxf(m, shfl_xor(m, 4));  // the block's four chunks are four lanes apart
                    m = __builtin_fmaxf(m, shfl_xor(m, 8));
                    s[i] = kv4_scale_byte(m);
                    const float inv = __builtin_bit_cast(float, (254u - s[i]) << 23);  // 2^-e, s <= 253 for finite input
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[i] |= e2m1_code(elem(x[u][i], j), inv) << (4 * j);
                }
                uint8_t *r = kv + (size_t)h[u] * region;
                if (mine[u]) {
                    *(uint32_t *)(r + ko + ch[u] * 4) = w[0];
                    *(uint32_t *)(r + vo + ch[u] * 16) = w[1];
                    if ((lc & 3) == 0) {
                        r[kso + ch[u] / 4] = (uint8_t)s[0];
                        r[vso + ch[u]] = (uint8_t)s[1];
                    }
                }
            }
        } else {
            uint32_t w[UPW][2], s[UPW][2];
#pragma unroll
            for (int u = 0; u < UPW; ++u) {
                const uint8_t *r = kv + (size_t)h[u] * region;
                w[u][0] = w[u][1] = s[u][0] = s[u][1] = 0;
                if (mine[u]) {
                    w[u][0] = *(const uint32_t *)(r + ko + ch[u] * 4);
                    w[u][1] = *(const uint32_t *)(r + vo + ch[u] * 16);
                    s[u][0] = r[kso + ch[u] / 4];
                    s[u][1] = r[vso + ch[u]];
                }
            }
#pragma unroll
            for (int u = 0; u < UPW; ++u) {
                if (!mine[u]) continue;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float sc = __builtin_bit_cast(float, s[u][i] << 23);
                    const f32x2 y0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u][i], sc, 0);
                    const f32x2 y1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u][i], sc, 1);
                    const f32x2 y2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u][i], sc, 2);
                    const f32x2 y3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u][i], sc, 3);
                    store8((i ? vrow : krow) + h[u] * DH + ch[u] * 8,
                           {y0[0], y0[1], y1[0], y1[1], y2[0], y2[1], y3[0], y3[1]});
                }
            }
        }
    }
}

template <int TYPE, int DH, bool APPEND, int UPW>
static int launch_move_upw(Kv4Move a, long long groups, hipStream_t stream) {
    a.parts = (a.units + UPW - 1) / UPW;
    // gathering many positions: two groups a wave (122 against 128 us for 107 k positions); appending: 73 against 76
    a.run = !APPEND && groups * a.parts >= 16384 ? 2 : 1;
    const long long waves = (groups + a.run - 1) / a.run * a.parts;
    hipLaunchKernelGGL((kv4_move_kernel<TYPE, DH, APPEND, UPW>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0,
                       stream, a);
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

template <int TYPE, int DH, bool APPEND>
static int launch_move(Kv4Move a, hipStream_t stream) {
    const long long groups = (long long)(a.n >> 2) + 2LL * a.c.B + 1;
    a.units = (a.c.Hkv * DH + 127) / 128;
    // two pieces a wave where that leaves enough waves: 127 against 152 us for 107 k positions of 8 heads, but
    // 8.4 against 7.0 us for 32 positions (four pieces: 125 and 11.4)
    if (a.units >= 2 && groups * a.units >= 8192) return launch_move_upw<TYPE, DH, APPEND, 2>(a, groups, stream);
    return launch_move_upw<TYPE, DH, APPEND, 1>(a, groups, stream);
}

template <bool APPEND>
static int kv4_move(int type, void *k, int ldk, void *v, int ldv, int n, const int32_t *cu, const int32_t *lens, int B,
                    int Hkv, int Dh, const int32_t *pages, int max_pages, int page, int num_pages, void *kv,
                    int32_t *d_status, void *stream) {
    if (type != QG_TYPE_F32 && type != QG_TYPE_F16 && type != QG_TYPE_BF16) return QG_ERR_FORMAT;
    if (!k || !v || !cu || !lens || !pages || !kv || !d_status) return QG_ERR_NULL;
    if (!kv4_cache_shape_ok(B, Hkv, Dh, max_pages, page, num_pages)) return QG_ERR_SHAPE;
    if (n < 1 || n > QG_MAX_ATTN_TOKENS || !row_stride_ok(type, ldk, Hkv * Dh) || !row_stride_ok(type, ldv, Hkv * Dh))
        return QG_ERR_SHAPE;
    if (((long long)(n >> 2) + 2LL * B + 1) * (Hkv * Dh / 64) > 0x7fffff00LL) return QG_ERR_SHAPE;
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)kv) & 15) return QG_ERR_ALIGN;
    if (((uintptr_t)cu | (uintptr_t)lens | (uintptr_t)pages | (uintptr_t)d_status) & 3) return QG_ERR_ALIGN;
    Kv4Move a{};
    a.c.kv = (uint8_t *)kv;
    a.c.pages = pages;
    a.c.lens = lens;
    a.c.max_pages = max_pages;
    a.c.num_pages = num_pages;
    a.c.page_log2 = __builtin_ctz((unsigned)page);
    a.c.B = B;
    a.c.Hkv = Hkv;
    a.c.status = d_status;
    a.k = k;
    a.v = v;
    a.cu = cu;
    a.n = n;
    a.ldk = ldk;
    a.ldv = ldv;
    hipStream_t s = (hipStream_t)stream;
    clear_stale_error();
#define QG_MOVE(T)                                              \
    switch (Dh) {                                               \
        case 64: return launch_move<T, 64, APPEND>(a, s);       \
        case 128: return launch_move<T, 128, APPEND>(a, s);     \
        default: return launch_move<T, 256, APPEND>(a, s);      \
    }
    switch (type) {
        case QG_TYPE_F32: QG_MOVE(QG_TYPE_F32)
        case QG_TYPE_F16: QG_MOVE(QG_TYPE_F16)
        default: QG_MOVE(QG_TYPE_BF16)
    }
#undef QG_MOVE
}

}  // namespace qg

extern "C" size_t kv4_page_bytes(int page, int Hkv, int Dh) {
    if (!qg::kv4_cache_shape_ok(1, Hkv, Dh, 1, page, 1)) return 0;
    return (size_t)Hkv * qg::kv4_region_bytes(page, Dh);
}

extern "C" int kv4_append(int type, const void *k, int ldk, const void *v, int ldv, int n, const int32_t *cu,
                          const int32_t *lens, int B, int Hkv, int Dh, const int32_t *pages, int max_pages, int page,
                          int num_pages, void *kv, int32_t *d_status, void *stream) {
    return qg::kv4_move<true>(type, const_cast<void *>(k), ldk, const_cast<void *>(v), ldv, n, cu, lens, B, Hkv, Dh,
                              pages, max_pages, page, num_pages, kv, d_status, stream);
}

extern "C" int kv4_gather(int type, void *k, int ldk, void *v, int ldv, int n, const int32_t *cu, const int32_t *lens,
                          int B, int Hkv, int Dh, const int32_t *pages, int max_pages, int page, int num_pages,
                          const void *kv, int32_t *d_status, void *stream) {
    return qg::kv4_move<false>(type, k, ldk, v, ldv, n, cu, lens, B, Hkv, Dh, pages, max_pages, page, num_pages,
                               const_cast<void *>(kv), d_status, stream);
}
