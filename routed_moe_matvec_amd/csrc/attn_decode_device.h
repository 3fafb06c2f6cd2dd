// What the kernels of attention of new tokens over the paged FP4 cache share:
// their arguments, the parts of a sequence's positions, and how operands are made.
#pragma once

#include "common.h"
#include "kv4_device.h"

namespace qg {

constexpr int kDecWaves = 4;
constexpr int kDecStep = 32;                      // positions a wave takes at a time
constexpr int kDecChunkMax = 8192;                // most positions of a workgroup (4096 times 128 / 64)
constexpr float kDecSlack = 8.f;                  // a weight may reach 2^8 before the sums are rescaled

// Positions per workgroup, as a power of two, of a sequence of which n are
// visible: about 8 sqrt(n) at 128 channels (as many bytes at 64 and 256), so
// that short sequences still spread over the card and long ones do not spend
// their time joining; and 64 a query row, up to 1024, since every row adds
// Dh sums to what a chunk writes and the join reads (32 sequences with 16 rows
// of 256 channels: 100 us with 1024, 112 with 512; one such sequence of 8000: 22
// and 17 us).  Up to 640 positions (of 128 channels) are one chunk, which needs no
// join (32 query and 8 key heads, one sequence of 640: 8.0 -> 7.6 us, 32 of them 12.6
// -> 8.8; one of 1024 would go from 8.0 to 10.0).  A function of the sequence and
// the heads alone: a sequence's result is the same in any batch.
struct DecSplit {
    int dh_log2, least;  // log2 of the channels, least log2 of a chunk
    __host__ __device__ int chunk_log2(int n) const {
        int lg = n <= 5 << (7 + 7 - dh_log2) ? 10 : 8;
        while (lg < 12 && n >= grows_at(lg)) ++lg;
        lg += 7 - dh_log2;
        return lg < least ? least : lg;
    }
    __host__ __device__ int grows_at(int lg) const { return 1 << (2 * lg - 5 + 7 - dh_log2); }
    __host__ __device__ int chunks(int n) const {
        const int lg = chunk_log2(n);
        return (n + (1 << lg) - 1) >> lg;
    }
    // Most chunks of any n up to `most`: at `most` or just before a chunk grows.
    int chunks_max(int most) const {
        int best = chunks(most);
        for (int lg = 8; lg < 12; ++lg)
            if (grows_at(lg) - 1 <= most && chunks(grows_at(lg) - 1) > best) best = chunks(grows_at(lg) - 1);
        return best < 1 ? 1 : best;
    }
};

inline DecSplit dec_split(int rows, int Dh) {
    int least = 8;
    while (least < 10 && 1 << least < 64 * rows) ++least;
    return DecSplit{Dh == 64 ? 6 : Dh == 128 ? 7 : 8, least};
}

// What the positions of a call are:
//  PLAIN   those up to a query's own, or the last `window` of them
//  SINKS   the last `window` of them, and the first `sinks`
//  TAIL    those from `prefix` on, of sequences that share what lies before
enum DecMode { PLAIN, SINKS, TAIL };

struct DecodeArgs {
    Kv4Cache c;
    const void *q;
    float *y;
    float *po;   // [B, H * Tq, chunks, Dh] partial sums
    f32x2 *pml;  // [B, H * Tq, chunks] largest q . k and sum
    int ldq, Tq, H, G, window, max_len, chunks;
    int sinks;
    int prefix, prefix_each, prefix_chunks;  // positions, those of a chunk, and the chunks
    const int32_t *prefix_pages;
    float scale;  // times log2(e), not negative
    float qsign;  // 1, -1 (a negative scale) or 0 (scale 0)
    DecSplit split;
};

// Where the visible positions of sequence b's queries are.  A kernel counts the
// places that it walks from 0: places before `edge` are positions 0.., those
// behind it are `gap` further on.  Both are multiples of 16 (a tile), and the
// places are all of [0, n); n is negative for a length out of range.
struct DecRange {
    int len, edge, gap, n;
};
template <int MODE>
__device__ __forceinline__ DecRange dec_range(const DecodeArgs &a, int b) {
    DecRange r{load_uniform(a.c.lens + b), 0, 0, -1};
    if (r.len < 0 || r.len > a.max_len) return r;
    if (MODE == TAIL) {
        r.n = 0;
        if (r.len <= a.prefix) return r;
        r.gap = a.prefix & ~15;
    } else if (a.window && r.len - a.Tq - a.window + 1 > 0) {
        r.gap = (r.len - a.Tq - a.window + 1) & ~15;
        if (MODE == SINKS) {
            r.edge = (min(a.sinks, r.len) + 15) & ~15;
            if (r.gap <= r.edge) r.edge = r.gap = 0;
            r.gap -= r.edge;
        }
    }
    r.n = r.len - r.gap;
    return r;
}

// 8 elements of q as PARTS bf16 vectors whose sum they are.  The first part of
// fp32's largest numbers is bf16's largest, not Inf.
template <int PARTS, class T>
__device__ __forceinline__ void split8(const Raw8<T> &r, float sign, bf16x8 (&out)[PARTS]) {
    constexpr float kMost = 0x1.fep127f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float x = elem(r, i) * sign;
#pragma unroll
        for (int s = 0; s < PARTS; ++s) {
            const bf16_t h = (bf16_t)(PARTS == 3 && s == 0 ? __builtin_amdgcn_fmed3f(x, -kMost, kMost) : x);
            out[s][i] = h;
            x -= (float)h;
        }
    }
}

// Scale byte i where the conversion takes its exponent from, bits 23..30 (it
// reads no others).
__device__ __forceinline__ float scale_of(uint32_t bytes, int i) {
    return __builtin_bit_cast(float, i < 3 ? bytes << (23 - 8 * i) : bytes >> 1);
}

template <int B>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, B));
}

// Keeps the loads before it where they are: they would sink to their use.
__device__ __forceinline__ void stay() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

template <int TYPE>
constexpr int kQParts = TYPE == QG_TYPE_F32 ? 3 : TYPE == QG_TYPE_F16 ? 2 : 1;


// attn_prefix.hip: the part of attn_decode_kv4_prefix that the sequences share, `rows`
// query rows of a key/value head in tiles of prefix_tile_rows, and how it is cut.
inline int prefix_tile_rows(long long rows, int Dh) { return rows > 64 ? 128 : rows > 32 || Dh == 256 ? 64 : 32; }
struct PrefixSplit {
    int each, chunks;  // positions of a chunk, a multiple of 128, and the chunks
};
PrefixSplit prefix_split(long long rows, int Hkv, int Dh, int prefix);
int launch_attn_prefix(int type, int Dh, const DecodeArgs &a, hipStream_t stream);

}  // namespace qg
