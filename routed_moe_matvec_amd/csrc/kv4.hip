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
    int units;  // waves' pieces per group of four positions: Hkv * Dh / 64
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

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
}
__device__ __forceinline__ void load8(const _Float16 *p, float (&x)[8]) {
    const f16x8 a = *(const f16x8 *)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)a[i];
}
__device__ __forceinline__ void load8(const bf16_t *p, float (&x)[8]) {
    const bf16x8 a = *(const bf16x8 *)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)a[i];
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

// The packed tokens of sequence b are positions [len - (c1 - c0), len).  Groups
// of four aligned positions are numbered so that sequence b's begin at
// cu[b] / 4 + 2b: enough room for any lengths, found without a prefix sum.
struct Kv4Group {
    int b, first, tok0, lo, hi;  // positions first .. first+3, of which [lo, hi) are given; token of `first`
};

__device__ __forceinline__ bool kv4_group(const Kv4Move &a, int group, int lane0, Kv4Group *g) {
    const Kv4Cache &c = a.c;
    const int b = wave_find_last(c.B, group, [&](int s) { return (a.cu[s] >> 2) + 2 * s; });
    const int c0 = a.cu[b], c1 = a.cu[b + 1], len = c.lens[b];
    if (c0 < 0 || c1 < c0 || c1 > a.n || len < c1 - c0 || len > c.max_pages << c.page_log2) {
        if (lane0) kv4_report(c.status, QG_DEV_BAD_LENGTH);
        return false;
    }
    const int start = len - (c1 - c0);
    g->b = b;
    g->first = ((start >> 2) + (group - ((c0 >> 2) + 2 * b))) * 4;
    g->lo = start;
    g->hi = len;
    g->tok0 = c0 + g->first - start;
    return g->first < len && g->first + 3 >= start;
}

// Every cu and len, looked at once by the first workgroup: an entry out of
// order may otherwise go unseen.
__device__ __forceinline__ void kv4_check_lengths(const Kv4Move &a) {
    for (int b = threadIdx.x; b < a.c.B; b += blockDim.x) {
        const int c0 = a.cu[b], c1 = a.cu[b + 1], len = a.c.lens[b];
        if (c0 < 0 || c1 < c0 || c1 > a.n || len < c1 - c0 || len > a.c.max_pages << a.c.page_log2)
            kv4_report(a.c.status, QG_DEV_BAD_LENGTH);
    }
}

template <int TYPE, int DH, bool APPEND, int UPW>
__global__ __launch_bounds__(256) void kv4_move_kernel(Kv4Move a) {
    typedef typename ElemOf<TYPE>::type T;
    constexpr int kChunks = DH / 8;
    const int wave = (int)(blockIdx.x * 4 + threadIdx.x / kWave), lane = lane_id();
    if (blockIdx.x == 0) kv4_check_lengths(a);
    const int per = a.units / UPW;
    const int group = wave / per;
    Kv4Group g;
    if (!kv4_group(a, group, lane == 0, &g)) return;
    const Kv4Cache &c = a.c;
    const int page = 1 << c.page_log2;
    const int id = kv4_page_of(c, g.b, g.first >> c.page_log2);
    if (id < 0) return;
    const int off = g.first & (page - 1);
    const size_t region = kv4_region_bytes(page, DH);
    uint8_t *base = c.kv + (size_t)id * c.Hkv * region;
    const int t = lane & 3;  // which of the four positions
    const bool there = g.first + t >= g.lo && g.first + t < g.hi;
    const size_t tok = (size_t)(there ? g.tok0 + t : 0);
    float x[UPW][8];
#pragma unroll
    for (int u = 0; u < UPW; ++u) {
        const int item = ((wave - group * per) * UPW + u) * 16 + (lane >> 2);  // chunk of K, then of V
        const bool isv = item >= c.Hkv * kChunks;
        const int hc = isv ? item - c.Hkv * kChunks : item;
        const int h = hc / kChunks, ch = hc % kChunks;
        if (APPEND) {
            const T *src = isv ? (const T *)a.v + tok * a.ldv : (const T *)a.k + tok * a.ldk;
            if (there) load8(src + h * DH + ch * 8, x[u]);
        } else {
            const uint8_t *r = base + h * region;
            uint32_t w = 0, s = 0;
            if (there) {
                if (isv) {
                    w = *(const uint32_t *)(r + (size_t)page * (DH / 2) + ((size_t)(off >> 2) * kChunks + ch) * 16 + t * 4);
                    s = r[(size_t)page * (DH + DH / 32) + ((off >> 2) * (DH / 32) + ch / 4) * 4 + t];
                } else {
                    w = *(const uint32_t *)(r + (size_t)(off + t) * (DH / 2) + ch * 4);
                    s = r[(size_t)page * DH + (off + t) * (DH / 32) + ch / 4];
                }
            }
            const float sc = __builtin_bit_cast(float, s << 23);
            f32x2 y;
#define QG_FP4_PAIR(i)                                                \
    y = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, i);           \
    x[u][2 * i] = y[0];                                               \
    x[u][2 * i + 1] = y[1];
            QG_FP4_PAIR(0)
            QG_FP4_PAIR(1)
            QG_FP4_PAIR(2)
            QG_FP4_PAIR(3)
#undef QG_FP4_PAIR
        }
    }
#pragma unroll
    for (int u = 0; u < UPW; ++u) {
        const int item = ((wave - group * per) * UPW + u) * 16 + (lane >> 2);
        const bool isv = item >= c.Hkv * kChunks;
        const int hc = isv ? item - c.Hkv * kChunks : item;
        const int h = hc / kChunks, ch = hc % kChunks;
        if (!APPEND) {
            T *dst = isv ? (T *)a.v + tok * a.ldv : (T *)a.k + tok * a.ldk;
            if (there) store8(dst + h * DH + ch * 8, x[u]);
            continue;
        }
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(there ? x[u][i] : 0.f));
        m = __builtin_fmaxf(m, shfl_xor(m, 4));  // the block's four chunks are four lanes apart
        m = __builtin_fmaxf(m, shfl_xor(m, 8));
        const uint32_t s = kv4_scale_byte(m);
        const float inv = __builtin_bit_cast(float, (254u - s) << 23);  // 2^-e, s <= 253 for finite input
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= e2m1_code(x[u][i], inv) << (4 * i);
        if (!there) continue;
        uint8_t *r = base + h * region;
        if (isv) {
            *(uint32_t *)(r + (size_t)page * (DH / 2) + ((size_t)(off >> 2) * kChunks + ch) * 16 + t * 4) = w;
            if ((ch & 3) == 0) r[(size_t)page * (DH + DH / 32) + ((off >> 2) * (DH / 32) + ch / 4) * 4 + t] = (uint8_t)s;
        } else {
            *(uint32_t *)(r + (size_t)(off + t) * (DH / 2) + ch * 4) = w;
            if ((ch & 3) == 0) r[(size_t)page * DH + (off + t) * (DH / 32) + ch / 4] = (uint8_t)s;
        }
    }
}

template <int TYPE, int DH, bool APPEND>
static int launch_move(const Kv4Move &a, hipStream_t stream) {
    const long long waves = ((long long)(a.n >> 2) + 2LL * a.c.B + 1) * a.units;
    const int grid = (int)((waves + 3) / 4);
    hipLaunchKernelGGL((kv4_move_kernel<TYPE, DH, APPEND, 1>), dim3(grid), dim3(256), 0, stream, a);
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
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
    if (((long long)(n >> 2) + 2LL * B + 1) * (Hkv * Dh / 64) > 0x7ffffff0LL) return QG_ERR_SHAPE;
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
    a.units = Hkv * Dh / 64;
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
