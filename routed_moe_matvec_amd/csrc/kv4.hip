// Writing and reading the paged FP4 key/value cache.
//
// kv4_append quantizes each 32 channels of a token's key or value to E2M1
// codes with one power-of-two scale: e = least integer >= -120 with
// max|x| <= 6 * 2^e, so nothing saturates, and x * 2^-e is exact in fp32, so
// codes and scales are the same on every machine.  kv4_gather is the inverse;
// an E2M1 value times 2^e is exact in bf16 and fp32.
//
// Both move (sizeof(type) + 17/32) bytes per element and compute little: bound
// by memory.  A lane has one chunk of 8 channels of four neighbouring
// positions, aligned to four in their page, of the keys and of the values: the
// wave's reads or writes of one token's row are one run of 1 KiB (16-bit types,
// 512 channels and more), and four positions of a value chunk are one 16-byte
// piece of the page.  Measured: 107 k positions of 8 heads of 128 read back to
// bf16 in 107 us (5.1 TB/s; a copy reaches 6.2), where four lanes with one
// position each took 120 and had half again as many loads; 39 k appended from
// bf16 in 38 us (4.2 TB/s, 27 of them for the reads alone; 34 when the rows are
// still cached), and 46 with the codes found by comparisons instead of the
// conversion instruction, bound by them.  Non-temporal reads and writes of the
// rows would take 9 and 6 us off these, but the prompt attention that reads the
// same rows next loses more: 40000 tokens written, appended and attended to
// 406 -> 602 us, 16384 positions read back and attended to by 128 queries 145 -> 226.
#include <type_traits>

#include "common.h"
#include "kv4_device.h"

namespace qg {

struct Kv4Move {
    Kv4Cache c;
    void *k, *v;
    const int32_t *cu;
    int n, ldk, ldv;
    int pieces;  // waves that share a group of positions, 64 chunks each
};

// Scale byte of a block with largest magnitude amax: e + 127.
__device__ __forceinline__ uint32_t kv4_scale_byte(float amax) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, amax) & 0x7fffffffu;
    const int s = (int)(bits >> 23) - 2 + ((bits & 0x7fffffu) > 0x400000u ? 1 : 0);  // 6 = 1.5 * 2^2
    return (uint32_t)min(max(s, 7), 254);
}

// The codes of 8 elements.  The conversion divides by the scale, exactly, and
// rounds to the nearest value, the even code on a tie; nothing here is above 6.
template <class R>
__device__ __forceinline__ uint32_t e2m1_codes(const R &x, uint32_t scale_byte) {
    const float s = __builtin_bit_cast(float, scale_byte << 23);
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, elem(x, 0), elem(x, 1), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, elem(x, 2), elem(x, 3), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, elem(x, 4), elem(x, 5), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, elem(x, 6), elem(x, 7), s, 3);
}
// and what 8 codes stand for.
__device__ __forceinline__ void e2m1_values(uint32_t w, uint32_t scale_byte, float (&x)[8]) {
    const float s = __builtin_bit_cast(float, scale_byte << 23);
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1),
                c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
    x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1], x[4] = c[0], x[5] = c[1], x[6] = d[0], x[7] = d[1];
}

// Largest of the four lanes that share a block.
__device__ __forceinline__ float quad_max(float x) {
    auto swap = [](float v, auto ctrl) {
        return __builtin_bit_cast(
            float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    x = __builtin_fmaxf(x, swap(x, std::integral_constant<int, 0xb1>{}));      // lane ^ 1
    return __builtin_fmaxf(x, swap(x, std::integral_constant<int, 0x4e>{}));  // lane ^ 2
}

__device__ __forceinline__ bool kv4_lengths_ok(const Kv4Move &a, int c0, int c1, int len) {
    return c0 >= 0 && c1 >= c0 && c1 <= a.n && len >= c1 - c0 && len <= a.c.max_pages << a.c.page_log2;
}

// The packed tokens of sequence b are positions [len - (c1 - c0), len).  Groups
// of 2^lg aligned positions are numbered so that sequence b's begin at
// (cu[b] >> lg) + 2b: enough room for any lengths, found without a prefix sum.
struct Kv4Group {
    bool ok;
    int b, pos;          // the sequence, and the group's first position
    int c0, start, len;  // its first token, that token's position, and its end
};

__device__ __forceinline__ Kv4Group kv4_group(const Kv4Move &a, int group, int lg) {
    Kv4Group g;
    g.b = wave_find_last(a.c.B, group, [&](int s) { return (a.cu[s] >> lg) + 2 * s; });
    const int c0 = load_uniform(a.cu + g.b), c1 = load_uniform(a.cu + g.b + 1);
    g.len = load_uniform(a.c.lens + g.b);
    g.ok = kv4_lengths_ok(a, c0, c1, g.len);
    g.c0 = c0;
    g.start = g.len - (c1 - c0);
    g.pos = ((g.start >> lg) + (group - ((c0 >> lg) + 2 * g.b))) << lg;
    g.ok = g.ok && g.pos < g.len && g.pos + (1 << lg) > g.start;
    return g;
}

// QUADS: where a row has few chunks, a wave takes 2 or 4 times four positions
// (at most 16, which are always in one page).
template <int TYPE, int DH, bool APPEND, int QUADS>
__global__ __launch_bounds__(256) void kv4_move_kernel(Kv4Move a) {
    typedef typename ElemOf<TYPE>::type T;
    constexpr int LG = QUADS == 1 ? 2 : QUADS == 2 ? 3 : 4, LANES = kWave / QUADS;
    const Kv4Cache &c = a.c;
    const int lane = lane_id();
    // Workgroups are dealt to the 8 XCDs in turn: eight neighbours go to one, whose
    // L2 then holds whole lines of the scales (append of 100 k positions of 8 heads
    // of 128 in bf16 105.6 -> 101.5 us, read back 107 -> 105).
    int group = blockIdx.x;
    if (group < (int)gridDim.x / 64 * 64) group = group / 64 * 64 + group % 8 * 8 + group / 8 % 8;
    const int wave = group * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (blockIdx.x == 0)  // every length once: one out of order may otherwise go unseen
        for (int b = threadIdx.x; b < c.B; b += 256)
            if (!kv4_lengths_ok(a, a.cu[b], a.cu[b + 1], c.lens[b])) kv4_report(c.status, QG_DEV_BAD_LENGTH);
    const Kv4Group g = kv4_group(a, wave / a.pieces, LG);
    if (!g.ok) return;
    const int id = kv4_page_of(c, g.b, g.pos >> c.page_log2);
    if (id < 0) return;

    const int page = 1 << c.page_log2;
    const int chunk = wave % a.pieces * kWave + lane % LANES, h = chunk / (DH / 8), ch = chunk % (DH / 8);
    const int pos = g.pos + 4 * (lane / LANES), off = pos & (page - 1);
    const bool mine = h < c.Hkv;
    bool there[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) there[t] = mine && pos + t >= g.start && pos + t < g.len;
    const long long tok = g.c0 + (long long)(pos - g.start);  // of position 0; only those that are there are used
    T *krow = (T *)a.k + tok * a.ldk + h * DH + ch * 8, *vrow = (T *)a.v + tok * a.ldv + h * DH + ch * 8;
    uint8_t *r = c.kv + ((size_t)id * c.Hkv + (mine ? h : 0)) * kv4_region_bytes(page, DH);
    uint8_t *kc = r + (size_t)off * (DH / 2) + ch * 4;
    uint8_t *vc = r + (size_t)page * (DH / 2) + ((size_t)(off >> 2) * (DH / 8) + ch) * 16;
    uint8_t *kscale = r + (size_t)page * DH + (size_t)off * (DH / 32) + ch / 4;
    uint8_t *vscale = r + (size_t)page * (DH + DH / 32) + ((size_t)(off >> 2) * (DH / 32) + ch / 4) * 4;

    if constexpr (APPEND) {
        Raw8<T> x[2][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            x[0][t] = x[1][t] = Raw8<T>{};
            if (there[t]) {
                x[0][t] = load8(krow + (long long)t * a.ldk);
                x[1][t] = load8(vrow + (long long)t * a.ldv);
            }
        }
        u32x4 w[2];
        uint32_t s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = __builtin_fmaxf(m, __builtin_fabsf(elem(x[i][t], j)));
                s[i][t] = kv4_scale_byte(quad_max(m));
                w[i][t] = e2m1_codes(x[i][t], s[i][t]);
            }
        const bool scales = (ch & 3) == 0;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (there[t]) {
                *(uint32_t *)(kc + t * (DH / 2)) = w[0][t];
                if (scales) kscale[t * (DH / 32)] = (uint8_t)s[0][t];
            }
        if (there[0] && there[3]) {
            *(u32x4 *)vc = w[1];
            if (scales) *(uint32_t *)vscale = s[1][0] | s[1][1] << 8 | s[1][2] << 16 | s[1][3] << 24;
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (there[t]) {
                    ((uint32_t *)vc)[t] = w[1][t];
                    if (scales) vscale[t] = (uint8_t)s[1][t];
                }
        }
    } else {
        if (!mine) return;
        uint32_t w[4], s[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            w[t] = *(const uint32_t *)(kc + t * (DH / 2));
            s[t] = kscale[t * (DH / 32)];
        }
        const u32x4 vw = *(const u32x4 *)vc;
        const uint32_t vs = *(const uint32_t *)vscale;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (!there[t]) continue;
            float x[8];
            e2m1_values(w[t], s[t], x);
            store8(krow + (long long)t * a.ldk, x);
            e2m1_values(vw[t], vs >> (8 * t) & 255u, x);
            store8(vrow + (long long)t * a.ldv, x);
        }
    }
}

template <int TYPE, int DH, bool APPEND, int QUADS>
static int launch_move_quads(Kv4Move a, hipStream_t stream) {
    a.pieces = QUADS > 1 ? 1 : (a.c.Hkv * (DH / 8) + kWave - 1) / kWave;
    const long long waves = ((long long)(a.n / (4 * QUADS)) + 2LL * a.c.B + 1) * a.pieces;
    hipLaunchKernelGGL((kv4_move_kernel<TYPE, DH, APPEND, QUADS>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0,
                       stream, a);
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

template <int TYPE, int DH, bool APPEND>
static int launch_move(const Kv4Move &a, hipStream_t stream) {
    const int chunks = a.c.Hkv * (DH / 8);
    if (DH <= 128 && chunks <= 16) return launch_move_quads<TYPE, DH, APPEND, DH <= 128 ? 4 : 1>(a, stream);
    if (chunks <= 32) return launch_move_quads<TYPE, DH, APPEND, 2>(a, stream);
    return launch_move_quads<TYPE, DH, APPEND, 1>(a, stream);
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
    if (((long long)(n >> 2) + 2LL * B + 1) * ((Hkv * Dh + 511) / 512) > 4 * kMaxGroups) return QG_ERR_SHAPE;
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
