// The paged FP4 key/value cache: its layout, its element types and the device
// helpers that the cache writer, the reader and the attention over it share.
//
// One page holds `page` consecutive positions of one sequence, for every
// key/value head; head h of page p is the region of kv4_region_bytes bytes at
// (p * Hkv + h) * region:
//   key codes    [page][Dh/2]           byte i of a row: channels 2i (low nibble), 2i+1
//   value codes  [page/4][Dh/8][4][4]   position t, channel c: byte ((t/4 * Dh/8 + c/8) * 4 + t%4) * 4 + (c%8)/2
//   key scales   [page][Dh/32]          UE8M0 of each 32 channels
//   value scales [page/4][Dh/32][4]     position t innermost
// Keys are rows, since a score sums over channels: a lane's 16 bytes are 32
// channels of one key.  Values sum over positions, so four positions lie side
// by side: a lane's 16 bytes are 8 channels of four positions, which it pairs
// into matrix operands in registers, and a single position still owns whole
// bytes (no read-modify-write when one token is appended).
#pragma once

#include "common.h"

namespace qg {

typedef __bf16 bf16_t;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <int TYPE>
struct ElemOf;
template <>
struct ElemOf<QG_TYPE_F32> {
    typedef float type;
};
template <>
struct ElemOf<QG_TYPE_F16> {
    typedef _Float16 type;
};
template <>
struct ElemOf<QG_TYPE_BF16> {
    typedef bf16_t type;
};

__host__ __device__ inline size_t kv4_region_bytes(int page, int Dh) { return (size_t)page * (Dh / 16) * 17; }

// What every call over the cache is given.
struct Kv4Cache {
    uint8_t *kv;
    const int32_t *pages;  // [B, max_pages]
    const int32_t *lens;   // [B]
    int max_pages, num_pages;
    int page_log2;
    int B, Hkv;
    int32_t *status;
};

__device__ __forceinline__ void kv4_report(int32_t *status, int what) { atomicMax(status, what); }

// Page of position block `pg` of sequence b, or -1 (reported) when its id is
// outside the cache.  pg is inside [0, max_pages).
__device__ __forceinline__ int kv4_page_of(const Kv4Cache &c, int b, int pg) {
    const int id = c.pages[(size_t)b * c.max_pages + pg];
    if ((unsigned)id < (unsigned)c.num_pages) return id;
    kv4_report(c.status, QG_DEV_BAD_PAGE);
    return -1;
}

// Eight elements as they lie in memory, and as fp32.
template <class T>
struct Raw8 {
    u32x4 w[sizeof(T) / 2];
};
template <class T>
__device__ __forceinline__ Raw8<T> load8(const T *p) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = *(const u32x4 *)((const char *)p + 16 * i);
    return r;
}
__device__ __forceinline__ float elem(const Raw8<float> &r, int i) { return __builtin_bit_cast(float, (uint32_t)r.w[i / 4][i % 4]); }
__device__ __forceinline__ float elem(const Raw8<_Float16> &r, int i) {
    return (float)__builtin_bit_cast(f16x2, (uint32_t)r.w[0][i / 2])[i % 2];
}
__device__ __forceinline__ float elem(const Raw8<bf16_t> &r, int i) {
    return (float)__builtin_bit_cast(bf16x2, (uint32_t)r.w[0][i / 2])[i % 2];
}

// Index of the last b in [0, B) with key(b) <= x (0 if none), searched 64 ways
// at a time by the whole wave: one memory round trip for up to 64 sequences,
// two for 4096.  x is wave-uniform, key(0) is not read.
template <class F>
__device__ __forceinline__ int wave_find_last(int B, int x, F key) {
    int lo = 0, n = B;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + kWave - 1) / kWave;
        const int b = lo + lane_id() * step;
        const bool le = b < lo + n && (b == lo || key(b) <= x);
        const int last = 63 - __builtin_clzll(__ballot(le) | 1ull);
        const int next = lo + last * step;
        n = min(step, lo + n - next);
        lo = next;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The running maximum of a softmax, of scores q . k that are not scaled yet.  A
// score s has the weight 2^((s - raw) * scale - muse).  Up to 2^16 (scaled) raw is 0
// and muse the scaled maximum less `shift`, so that a weight takes one fused
// multiply-add: the maximum's own rounding moves all weights of the row alike, by
// at most 2^-8 in the exponent.  A larger maximum would move them out of range (at
// 1e10 by 2^440): it is raw itself, taken off the scores first (far rows).
struct RunningMax {
    float m = -INFINITY, muse = 0.f;
    unsigned long long far = 0;  // the lanes of the wave whose rows are far

    __device__ __forceinline__ bool is_far(float x, float scale) const {
        return __builtin_fabsf(x * scale) > 65536.f && x > -INFINITY;
    }
    // To the maximum with mt; returns the factor that this means for the row's sums.
    __device__ __forceinline__ float raise(float mt, float scale, float shift) {
        const float mn = __builtin_fmaxf(m, mt);
        float to = mn == -INFINITY ? 0.f : mn * scale - shift, e = m * scale - shift - to;
        const unsigned long long now = __ballot(is_far(mn, scale));
        if (far | now) {
            const float from_raw = is_far(m, scale) ? m : 0.f, to_raw = is_far(mn, scale) ? mn : 0.f;
            if (to_raw != 0.f) to = -shift;
            e = m == -INFINITY ? m : __builtin_fmaf(from_raw - to_raw, scale, muse - to);
            far = now;
        }
        m = mn;
        muse = to;
        return __builtin_amdgcn_exp2f(e);
    }
    // What is to be taken off the scores (far != 0).
    __device__ __forceinline__ float raw(float scale) const { return is_far(m, scale) ? m : 0.f; }
    // The factor that makes the row's sums relative to m * scale - shift exactly, so that
    // rows are joined by the difference of their maxima (0 where nothing was seen).
    __device__ __forceinline__ float exact(float scale, float shift) const {
        const float at = far && is_far(m, scale) ? 0.f : m;
        return m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(shift - __builtin_fmaf(at, scale, -muse));
    }
};

inline bool kv4_cache_shape_ok(int B, int Hkv, int Dh, int max_pages, int page, int num_pages) {
    return B >= 1 && B <= QG_MAX_SEQS && Hkv >= 1 && Hkv <= QG_MAX_HEADS && (Dh == 64 || Dh == 128 || Dh == 256) &&
           max_pages >= 1 && num_pages >= 1 && page >= 16 && page <= QG_MAX_PAGE && (page & (page - 1)) == 0 &&
           (long long)max_pages * page <= 0x7fffffffLL / 2;
}

inline size_t elem_bytes(int type) { return type == QG_TYPE_F32 ? 4 : 2; }

// Most workgroups of 256 threads: a launch holds fewer than 2^32 threads.
constexpr long long kMaxGroups = (1 << 24) - 1;

// Rows of `width` elements every `ld` elements, each 16-byte aligned.
inline bool row_stride_ok(int type, int ld, int width) {
    return ld >= width && (size_t)ld * elem_bytes(type) % 16 == 0;
}

}  // namespace qg
