// What the kernels of attention of new tokens over the paged FP4 cache share:
// their arguments, the parts of a sequence's positions, and how operands are made.
#pragma once

#include <type_traits>

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
//  FUSED   those before `prefix`, which all sequences share, and the sequence's own
enum DecMode { PLAIN, SINKS, TAIL, FUSED };

struct DecodeArgs {
    Kv4Cache c;
    const void *q;
    float *y;
    float *po;   // [B, H * Tq, chunks, Dh] partial sums
    f32x2 *pml;  // [B, H * Tq, chunks] largest q . k and sum
    int ldq, Tq, H, G, window, max_len, chunks;
    int sinks;
    int prefix, prefix_each, prefix_chunks;  // positions, those of a chunk, and the chunks (0: FUSED)
    int prefix_rows;
    bool wide;  // one chunk, of eight waves
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
    } else if (MODE == FUSED) {
        r.edge = (a.prefix + 15) & ~15;
        if (r.len > a.prefix) r.gap = (a.prefix & ~15) - r.edge;
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

// A lane's part of one 16-position tile.
template <int DH>
struct DecTile {
    static constexpr int KW = DH / 32, VC = DH / 128 < 1 ? 1 : DH / 128;  // dwords of a key, 16-byte pieces of values
    static constexpr int KS = VC;  // scales of a key
    uint32_t k[KW];
    u32x4 v[VC];
    uint32_t ks[KS];  // scale bytes of the lane's channels (DH / 4 of them)
    uint32_t vs[VC];  // scale bytes of four positions
};

// Offsets of a lane's parts in a tile; what depends on the tile is uniform.
template <int DH>
struct DecLane {
    uint32_t k, ks, v, vs;
    __device__ DecLane(int lane) {
        const int c = lane & 15, g = lane >> 4, chunk = DH == 64 ? c >> 1 : c;
        k = c * (DH / 2) + (DH == 64 ? g * 8 : g * 16);
        ks = c * (DH / 32) + (DH == 64 ? g >> 1 : g);  // 64 channels: two lanes a byte
        v = (g * (DH / 8) + chunk) * 16;
        vs = (g * (DH / 32) + (chunk >> 2)) * 4;
    }
};

// Through buffer instructions: the base and the tile's offsets are scalars, so
// that a load costs no vector arithmetic for its address.
template <int DH>
__device__ __forceinline__ void dec_load_k(DecTile<DH> &t, uint8_t *r, int page, int off, const DecLane<DH> &ln) {
    const auto rs = __builtin_amdgcn_make_buffer_rsrc(r, 0, (uint32_t)page * (DH / 16 * 17), 0x00027000);
    const int ko = off * (DH / 2), so = page * DH + off * (DH / 32);
    if constexpr (DH == 64) {
        const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(rs, ln.k, ko, 0);
        t.k[0] = w[0], t.k[1] = w[1];
    } else {
#pragma unroll
        for (int i = 0; i < DH / 32; i += 4) {
            const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(rs, ln.k + i * 16, ko, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) t.k[i + j] = w[j];
        }
    }
#pragma unroll
    for (int i = 0; i < DecTile<DH>::KS; ++i) t.ks[i] = __builtin_amdgcn_raw_buffer_load_b8(rs, ln.ks + 4 * i, so, 0);
}
template <int DH>
__device__ __forceinline__ void dec_load_v(DecTile<DH> &t, uint8_t *r, int page, int off, const DecLane<DH> &ln) {
    const auto rs = __builtin_amdgcn_make_buffer_rsrc(r, 0, (uint32_t)page * (DH / 16 * 17), 0x00027000);
    const int vo = page * (DH / 2) + off * (DH / 2), so = page * (DH + DH / 32) + off * (DH / 32);
#pragma unroll
    for (int x = 0; x < DecTile<DH>::VC; ++x) {
        t.v[x] = __builtin_amdgcn_raw_buffer_load_b128(rs, ln.v + x * 256, vo, 0);
        t.vs[x] = __builtin_amdgcn_raw_buffer_load_b32(rs, ln.vs + x * 16, so, 0);
    }
}

__device__ __forceinline__ f32x4 mfma16(const u32x4 &a, const u32x4 &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// Maximum over the four lanes that hold one row (16 apart).
__device__ __forceinline__ float row_max(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float y = __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
    const uint32_t w = __builtin_bit_cast(uint32_t, y);
    const auto q = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)q[0]), __builtin_bit_cast(float, (uint32_t)q[1]));
}
__device__ __forceinline__ float row_sum(float x) {
    x += shfl_xor(x, 16);
    return x + shfl_xor(x, 32);
}

// Values of two tiles as the A operands of channel pair (2 B, 2 B + 1) of a
// 16-byte piece: eight positions of either channel.
template <int B>
__device__ __forceinline__ void dec_values(const u32x4 &v0, const u32x4 &v1, const float (&s0)[4], const float (&s1)[4],
                                           u32x4 *lo, u32x4 *hi) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = fp4_pair<B>(v0[i], s0[i]);
        w[4 + i] = fp4_pair<B>(v1[i], s1[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        (*lo)[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x05040100u);
        (*hi)[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x07060302u);
    }
}

// The value of the lane 8 columns further on, of 16.
__device__ __forceinline__ float across8(float x) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x128, 0xf, 0xf, true));  // row_ror:8
}

// SLOTS: 2 with fp32 queries and 8 rows or fewer, else 1.  Then the 16 columns
// of an operand hold each row twice, with two parts of its queries or weights:
// two products do the work of three.  A score is the sum over a row's two
// columns (both get it), and so are the sums over values, once, at the end.
// Matrix units are busy 18 to 42% of this kernel's cycles, more than half of that
// beside no vector work, so fewer products pay: one sequence of 131001 positions, 8
// rows a head, 40.1 -> 37.8 us.  With one or two parts of the queries, and only the
// weights to gain on, it did not: 32 sequences of 4 rows in bf16 18.6 -> 18.9 us, of
// 2 rows in fp16 34.6 -> 34.9.
template <int DH, int WAVES>
struct DecShared {
    static constexpr int PER = DH == 64 ? 4 : 8;  // channel tiles joined at a time
    f32x4 sums[WAVES * PER * kWave];
    f32x2 ml[WAVES][16];
    int page[kDecChunkMax / 16 + 2];
};

// One workgroup: chunk group / (B Hkv) of a sequence and key/value head, rows from tile * 16 / SLOTS on.
template <int TYPE, int DH, int SLOTS, int MODE, int WAVES>
__device__ __forceinline__ void attn_decode_group(const DecodeArgs &a, DecShared<DH, WAVES> &sh, const int group, const int tile) {
    typedef typename ElemOf<TYPE>::type T;
    constexpr int QP = kQParts<TYPE>, KC = DH / 32, MT = DH / 16;  // parts of q, key products, channel tiles
    constexpr int ROWS = 16 / SLOTS, QO = (QP + SLOTS - 1) / SLOTS, PO = (3 + SLOTS - 1) / SLOTS;  // operands
    // queries of more than 16 registers stay in LDS, in the room that the join uses at the end: more waves fit
    constexpr bool QLDS = QO * KC > 4;
    constexpr int PER = DecShared<DH, WAVES>::PER;
    f32x4(&so)[WAVES * PER * kWave] = sh.sums;
    u32x4 *sq = reinterpret_cast<u32x4 *>(&so[0]);
    static_assert(!QLDS || sizeof(so) >= sizeof(u32x4) * QO * KC * kWave, "queries fit the join's room");
    f32x2(&sml)[WAVES][16] = sh.ml;
    int(&spage)[kDecChunkMax / 16 + 2] = sh.page;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    // sequence by sequence within a chunk number: the workgroups of chunks that a
    // sequence does not have come last
    const int hk = group % a.c.Hkv, bi = group / a.c.Hkv;
    const int b = bi % a.c.B, ci = bi / a.c.B;
    const int row0 = tile * ROWS;
    const int R = a.G * a.Tq;
    if (MODE == TAIL && ci > 0) {  // before anything is asked for: max_len may be far above the lengths
        const int n = dec_range<TAIL>(a, b).n;
        if (n <= 0 || ci >= a.split.chunks(n)) return;
    }
    const int c = lane & 15, g = lane >> 4;
    const int row = row0 + c % ROWS;
    const uint32_t second = c / ROWS ? ~0u : 0u;  // columns of the second, or no, part
    const bool live = row < R;
    auto token_of = [&](int r) {
        int x = 0;
        for (int i = 1; i < a.Tq; ++i) x += r >= i * a.G;
        return x;
    };
    const int t = live ? token_of(row) : 0;
    const int h = hk * a.G + (live ? row - t * a.G : 0);
    const size_t out_row = (size_t)(b * a.Tq + t) * a.H + h;

    // queries as the B operand: column c, for product i channels 8 i + 0..7 of the
    // lane's (16 g.. of 64, 32 g.. of each 128); requested first, used once the first keys are on their way
    constexpr int QN = QLDS ? (KC + WAVES - 1) / WAVES : KC;
    Raw8<T> qraw[QN];
    {
        const T *qp = (const T *)a.q + (size_t)(b * a.Tq + t) * a.ldq + (size_t)h * DH + g * (DH == 64 ? 16 : 32);
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int at = QLDS ? min(i * WAVES + wave, KC - 1) : i;
            qraw[i] = load8(qp + at / 4 * 128 + at % 4 * 8);
        }
    }

    const DecRange r = dec_range<MODE>(a, b);
    if (r.n < 0 && ci == 0 && threadIdx.x == 0) kv4_report(a.c.status, QG_DEV_BAD_LENGTH);
    const int nchunks = r.n > 0 ? a.split.chunks(r.n) : 0;
    if ((ci > 0 || MODE == TAIL) && ci >= nchunks) return;
    if (nchunks == 0) {
        if (live && wave == 0)
            for (int i = g * 4; i < DH; i += 16) *(f32x4 *)(a.y + out_row * DH + i) = f32x4{0.f, 0.f, 0.f, 0.f};
        return;
    }
    const int lg = a.split.chunk_log2(r.n);
    const int first = ci << lg, last = min(r.n, first + (1 << lg));  // this workgroup's places
    const int page = 1 << a.c.page_log2;
    // the places that this row sees: [see_lo, see_hi), and with two ranges those before `sinks`
    constexpr bool TWO = MODE == SINKS || MODE == FUSED;
    const int pos = r.len - a.Tq + t, own = MODE == TAIL || MODE == FUSED ? a.prefix - r.gap : 0;
    const int see_hi = live ? pos + 1 - r.gap : 0;
    const int see_lo = max(a.window ? pos - a.window + 1 - r.gap : 0, MODE == SINKS ? r.edge : own);
    const uint32_t seen_here = (uint32_t)max(min(see_hi, last) - see_lo, 0);  // places from see_lo on
    // the first place, behind the sinks, that a row sees, and the first that all do
    const int seen = a.window ? r.n - a.Tq - a.window + 1 : own, all_lo = a.window ? r.n - a.window : own;
    const int sinks = TWO ? min(MODE == SINKS ? a.sinks : a.prefix, r.len) : 0;
    const int sink_hi = live ? min(sinks, pos + 1) : 0, all_sinks = min(sinks, r.len - a.Tq + 1);
    const size_t region = kv4_region_bytes(page, DH);
    const DecLane<DH> ln(lane);

    // the chunk's page ids, through LDS (read by scalar loads a step ahead they made the kernel 5 to 15% slower):
    // those of places before the edge, which begin with page pg_sink, then the others, from pg0 on
    const int pg_sink = first >> a.c.page_log2;
    Kv4Cache prefix = a.c;
    prefix.pages = a.prefix_pages;
    const int n_sink = TWO && first < r.edge ? ((min(last, r.edge) - 1) >> a.c.page_log2) - pg_sink + 1 : 0;
    const int pg0 = ((TWO ? max(first, r.edge) : first) + r.gap) >> a.c.page_log2;
    const int n_pages = TWO && last <= r.edge ? n_sink : n_sink + ((last - 1 + r.gap) >> a.c.page_log2) - pg0 + 1;
    for (int i = threadIdx.x; i < n_pages; i += WAVES * kWave)
        spage[i] = MODE == FUSED && i < n_sink ? kv4_page_of(prefix, 0, pg_sink + i)
                                               : kv4_page_of(a.c, b, i < n_sink ? pg_sink + i : pg0 + i - n_sink);
    __syncthreads();

    // Where a step's two tiles lie; a tile behind the end or on a bad page
    // reads the chunk's first place, or page 0, instead and is masked.
    DecTile<DH> cur[2];
    uint8_t *at_region[2];
    int at_off[2];
    bool next_ok[2];
    auto locate = [&](int j) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int j0 = j + 16 * x, at = j0 < last ? j0 : first;
            const bool behind = !TWO || at >= r.edge;
            const int at_pos = behind ? at + r.gap : at, pg = at_pos >> a.c.page_log2;
            const int id = __builtin_amdgcn_readfirstlane(spage[behind ? pg - pg0 + n_sink : pg - pg_sink]);
            next_ok[x] = j0 < last && id >= 0;
            at_region[x] = a.c.kv + ((size_t)max(id, 0) * a.c.Hkv + hk) * region;
            at_off[x] = at_pos & (page - 1);
        }
    };
    auto load_k = [&] {
#pragma unroll
        for (int x = 0; x < 2; ++x) dec_load_k<DH>(cur[x], at_region[x], page, at_off[x], ln);
        stay();
    };
    auto load_v = [&] {
#pragma unroll
        for (int x = 0; x < 2; ++x) dec_load_v<DH>(cur[x], at_region[x], page, at_off[x], ln);
        stay();
    };
    constexpr int kStride = WAVES * kDecStep;
    const int j_first = first + wave * kDecStep;
    locate(j_first);
    load_k();
    load_v();

    u32x4 qf[QO][QLDS ? 1 : KC];
#pragma unroll
    for (int i = 0; i < QN; ++i) {
        const int at = QLDS ? i * WAVES + wave : i;
        bf16x8 parts[QP];
        split8<QP>(qraw[i], a.qsign, parts);
#pragma unroll
        for (int y = 0; y < QO; ++y) {
            u32x4 w = __builtin_bit_cast(u32x4, parts[y * SLOTS]);
            if (SLOTS == 2) {
                w &= ~second;
                if (2 * y + 1 < QP) w |= __builtin_bit_cast(u32x4, parts[2 * y + 1]) & second;
            }
            if (!QLDS)
                qf[y][QLDS ? 0 : i] = w;
            else if (at < KC)
                sq[(y * KC + at) * kWave + lane] = w;
        }
    }
    if (QLDS) lds_barrier();  // keys and values stay in flight

    f32x4 o[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    RunningMax most;
    float l = 0.f;

    // A step's keys are loaded again as soon as its scores are there, its
    // values when they are summed: the loads of the next step run beside the
    // rest of this one, in the same registers.
    auto step = [&](int j, auto more) {
        const bool cur_ok[2] = {next_ok[0], next_ok[1]};
        f32x4 s[2];
        int ql = lane;
        if (QLDS) asm volatile("" : "+v"(ql));  // or the reads below move out of the loop, into registers
#pragma unroll
        for (int x = 0; x < 2; ++x) s[x] = f32x4{0.f, 0.f, 0.f, 0.f};
        __builtin_amdgcn_s_setprio(1);  // scores before another wave's weights: its loads start earlier (101.7 -> 100.6 us)
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            u32x4 qi[QO];
#pragma unroll
            for (int y = 0; y < QO; ++y) qi[y] = QLDS ? sq[(y * KC + i) * kWave + ql] : qf[y][QLDS ? 0 : i];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float sc = scale_of(cur[x].ks[i / 4], 0);
                const uint32_t w = cur[x].k[i];
                const u32x4 kf = {fp4_pair<0>(w, sc), fp4_pair<1>(w, sc), fp4_pair<2>(w, sc), fp4_pair<3>(w, sc)};
#pragma unroll
                for (int y = 0; y < QO; ++y) s[x] = mfma16(kf, qi[y], s[x]);
            }
        }
        __builtin_amdgcn_s_setprio(0);
        if constexpr (more.value) {
            locate(j + kStride);
            load_k();
        }
        if constexpr (SLOTS == 2)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i / 4][i % 4] += across8(s[i / 4][i % 4]);
        // what a row does not see is -inf
        const bool whole = j + kDecStep <= min(last, r.n - a.Tq + 1) && cur_ok[0] && cur_ok[1] &&
                           (j >= all_lo || (TWO && j + kDecStep <= all_sinks));
        if (!whole) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t span = cur_ok[x] ? seen_here : 0u;
                const int upto = cur_ok[x] ? min(sink_hi, last) : 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = j + 16 * x + 4 * g + i;
                    if ((uint32_t)(at - see_lo) >= span && (!TWO || at >= upto)) s[x][i] = -INFINITY;
                }
            }
        }
        float mt = s[0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mt = __builtin_fmaxf(mt, s[i / 4][i % 4]);
        mt = row_max(mt);
        if (__ballot((mt - most.m) * a.scale > kDecSlack) | most.far) {
            const float keep = most.raise(mt, a.scale, 0.f);
            if (most.far) {
                const float raw = most.raw(a.scale);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i / 4][i % 4] -= raw;
            }
            l *= keep;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i] *= keep;
        }
        u32x4 pf[PO];
        {
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i / 4][i % 4], a.scale, -most.muse));
                l += p[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x0 = p[2 * i], x1 = p[2 * i + 1];
                uint32_t part[3];
#pragma unroll
                for (int y = 0; y < 3; ++y) {  // eight bits at a time, cut off: no rounding
                    const uint32_t b0 = __builtin_bit_cast(uint32_t, x0), b1 = __builtin_bit_cast(uint32_t, x1);
                    part[y] = __builtin_amdgcn_perm(b1, b0, 0x07060302u);
                    x0 -= __builtin_bit_cast(float, b0 & 0xffff0000u);
                    x1 -= __builtin_bit_cast(float, b1 & 0xffff0000u);
                }
#pragma unroll
                for (int y = 0; y < PO; ++y) {
                    pf[y][i] = part[y * SLOTS];
                    if (SLOTS == 2) {
                        pf[y][i] &= ~second;
                        if (2 * y + 1 < 3) pf[y][i] |= part[2 * y + 1] & second;
                    }
                }
            }
        }
        // what no row sees may be anything, also its scales: 0 * NaN
        if (!(j + kDecStep <= last && (j >= seen || (TWO && j + kDecStep <= sinks)) && cur_ok[0] && cur_ok[1])) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int at = j + 16 * x + 4 * g, left = cur_ok[x] ? last - at : 0, skip = seen - at;
                uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
                if (TWO) {  // of what is skipped, the sinks stay
                    auto below = [](int x) { return x >= 4 ? ~0u : x <= 0 ? 0u : (1u << (8 * x)) - 1u; };
                    keep &= ~below(skip) | below(sinks - at);
                } else if (skip > 0) {
                    keep = skip >= 4 ? 0u : keep & ~0u << (8 * skip);
                }
#pragma unroll
                for (int y = 0; y < DecTile<DH>::VC; ++y) cur[x].vs[y] &= keep;
            }
        }
#pragma unroll
        for (int y = 0; y < DecTile<DH>::VC; ++y) {
            float s0[4], s1[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) s0[i] = scale_of(cur[0].vs[y], i), s1[i] = scale_of(cur[1].vs[y], i);
            u32x4 v0 = cur[0].v[y], v1 = cur[1].v[y];
            if (DH == 64) {  // two lanes share a piece: this one takes 4 of its 8 channels
                v0 >>= (c & 1) * 16;
                v1 >>= (c & 1) * 16;
            }
            u32x4 lo, hi;
#define QG_PAIR(B)                                                                                       \
    dec_values<B>(v0, v1, s0, s1, &lo, &hi);                                                             \
    for (int w = 0; w < PO; ++w) {                                                                       \
        o[8 * y + 2 * B] = mfma16(lo, pf[w], o[8 * y + 2 * B]);                                          \
        o[8 * y + 2 * B + 1] = mfma16(hi, pf[w], o[8 * y + 2 * B + 1]);                                  \
    }
            QG_PAIR(0)
            QG_PAIR(1)
            if constexpr (DH > 64) {
                QG_PAIR(2)
                QG_PAIR(3)
            }
#undef QG_PAIR
        }
        if constexpr (more.value) load_v();
    };
    // The last step, which loads nothing, apart: loads behind a condition would
    // make every wait one for all of them.
    if (j_first < last) {
        int j = j_first;
        for (; j + kStride < last; j += kStride) step(j, std::true_type{});
        step(j, std::false_type{});
    }

    // join the waves: maxima first, then the sums of PER channel tiles at a
    // time through LDS, added and written by all threads (one wave writing
    // alone cost 22 of 117 us with 16 rows of 256 channels a workgroup)
    const float exact = most.exact(a.scale, 0.f);
    l = row_sum(l) * exact;
    if (g == 0) sml[wave][c] = f32x2{most.m, l};
    __syncthreads();  // and every wave is done with the queries
    auto joined = [&](int r) {  // maximum and sum of a row
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) top = __builtin_fmaxf(top, sml[w][r][0]);
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            sum += sml[w][r][1] * __builtin_amdgcn_exp2f((sml[w][r][0] - (top == -INFINITY ? 0.f : top)) * a.scale);
        return f32x2{top, sum};
    };
    const float top = joined(c)[0];
    const float keep = exact * __builtin_amdgcn_exp2f((most.m - (top == -INFINITY ? 0.f : top)) * a.scale);
    // o[8 y + i][k]: channel ((16 y + 4 g + k) * 8 + i), or (4 g + k) * 4 + i for 64 channels
    // what this thread adds and writes: a row's PART tiles from tile wi on, register wk of lane group wg
    constexpr int PART = PER / SLOTS;
    const int wk = threadIdx.x & 3, wc = (threadIdx.x >> 2) % ROWS, wg = threadIdx.x >> 6;
    const int wi = (threadIdx.x >> 2) % 16 / ROWS * PART;
    const bool adds = WAVES == 4 || threadIdx.x < 256;
    const int busy = (last - first + kDecStep - 1) / kDecStep;  // waves that had positions, or more
    const int wrow = row0 + wc;
    const int wt = token_of(wrow);
    const size_t wout = (size_t)(b * a.Tq + wt) * a.H + hk * a.G + wrow - wt * a.G;
    const f32x2 ml = joined(wc);
    float *dst = a.y + wout * DH;
    float f = ml[1] > 0.f ? 1.f / ml[1] : 0.f;
    if (MODE == TAIL || nchunks > 1) {
        const int chunk = MODE == TAIL ? a.prefix_chunks + ci : ci;
        dst = a.po + (wout * a.chunks + chunk) * DH;
        f = 1.f;
        if (adds && wrow < R && wg == 0 && wk == 0 && wi == 0) a.pml[wout * a.chunks + chunk] = ml;
    }
#pragma unroll
    for (int y = 0; y < DecTile<DH>::VC; ++y) {
        if (y) __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (WAVES == 4 || wave < 4 || busy > 4) so[(wave * PER + i) * kWave + lane] = o[8 * y + i] * keep;
        __syncthreads();
        if (!adds) continue;
        float acc[PART];
#pragma unroll
        for (int i = 0; i < PART; ++i) acc[i] = 0.f;
        auto add_waves = [&](int from, int to) {
#pragma unroll
            for (int i = 0; i < PART; ++i)
#pragma unroll
                for (int w = from; w < to; ++w)
#pragma unroll
                    for (int x = 0; x < SLOTS; ++x)
                        acc[i] += reinterpret_cast<const float *>(
                            &so[(w * PER + wi + i) * kWave + 16 * wg + wc + x * ROWS])[wk];
        };
        add_waves(0, 4);
        if (WAVES > 4 && busy > 4) add_waves(4, WAVES);
#pragma unroll
        for (int i = 0; i < PART; ++i) acc[i] *= f;
        if (wrow < R) {
            float *at = dst + (16 * y + 4 * wg + wk) * PER + wi;
            if constexpr (PART >= 4) {
#pragma unroll
                for (int i = 0; i < PART; i += 4)
                    *(f32x4 *)(at + i) = f32x4{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
            } else {
                *(f32x2 *)at = f32x2{acc[0], acc[1]};
            }
        }
    }
}

// attn_prefix.hip: the positions that the sequences share, for `rows` query rows of a
// key/value head, and how they are cut (no chunks: each sequence walks them by itself, FUSED);
// the launch takes the sequences' own positions along.
struct PrefixSplit {
    int rows;          // of a workgroup: 128, 64 or 32
    int each, chunks;  // positions of a chunk, a multiple of 128, and the chunks
};
PrefixSplit prefix_split(int B, long long rows, int Hkv, int Dh, int prefix);
int launch_attn_prefix(int type, int Dh, const DecodeArgs &a, hipStream_t stream);

}  // namespace qg
