// Attention over the positions that all sequences of a batch share.
//
// The query rows of all sequences (tokens and heads that read one key/value head) are
// one matrix against the shared keys.  A workgroup takes up to 128 rows and a chunk of the
// positions, a tile of them at a time, with the running maximum and sum of a softmax:
//   S^T = K Q^T    (positions x rows),  O^T += V^T P^T   (channels x rows),
// as v_mfma_f32_32x32x16.  The cache's bytes are loaded two tiles ahead and become 16-bit
// operands in one of two LDS stages once for all rows: K is read from there by rows, V by columns
// (the transposing read), pieces of 16 bytes permuted by the row's number.  A lane keeps
// one query row throughout, and the scores that it receives are the weights that it supplies.
//
// Operands are fp16 where a chunk's scales span no more than fp16 holds exactly, 36 binades, with
// one power of two taken off all keys and one off all values; a weight, times 2^11, is then two
// parts (22 bits, or 2^-36 of the row's largest), an fp32 query two and an fp16 one itself.  The second
// part of a query is taken 2^12 times as large, or fp16's least step would cut it, and its products are summed
// first: an element is off by 2^-23 of itself at most if it is within 2^26 of the row's largest; where one is not, the chunk
// is not taken so.  (The same sum for both parts lost bits from 2^17 on, at 134 us in place of 138 for the case below.)  Other
// chunks, and the keys of bf16 queries, take bf16, which holds every value exactly, and
// three parts for 24 bits: fp32, fp16, bf16 queries need 4, 3, 3 products so, and 6, 5, 4 there
// (fp32 and fp16 queries are read and split again at every tile).  48 sequences of 8 rows a head of
// fp32 queries over 40001 positions, 63 GFLOP, 127 with the parts, take 130 to 150 us by the run: the
// matrix cores are busy 51% of the cycles, the vector units 49% (without the issue of matrix
// instructions), both at once 19%, at 2.1 GHz, and neither another order of the instructions nor wave
// priorities changed that.  Few positions are bound by latency.  32 sequences of 4 rows over 6001: 4.3
// us to the first tile, 2.8 for it, 1.7 for each further one of 128, 2 for the sums.
#include <type_traits>

#include "attn_decode_device.h"

namespace qg {

// Sixteen-bit operands from codes, and their products.
template <bool F16>
struct PfxOps {
    __device__ static f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
        if constexpr (F16)
            return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                          0, 0, 0);
        else
            return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                           c, 0, 0, 0);
    }
    template <int B>
    __device__ static uint32_t pair(uint32_t w, float scale) {
        if constexpr (F16)
            return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, B));
        else
            return fp4_pair<B>(w, scale);
    }
    // eight codes of one scale byte
    __device__ static u32x4 eight(uint32_t w, uint32_t byte) {
        const float s = __builtin_bit_cast(float, byte << 23);
        return u32x4{pair<0>(w, s), pair<1>(w, s), pair<2>(w, s), pair<3>(w, s)};
    }
};

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Of the scale bytes seen so far the largest, and 255 less the least, both twice (in the halves).
struct ByteRange {
    u16x2 hi = {0, 0}, lo = {0, 0};
    __device__ void add(uint32_t w) {
        const uint32_t n = ~w;
        auto top = [](uint32_t x) {
            return __builtin_elementwise_max(__builtin_bit_cast(u16x2, x & 0x00ff00ffu), __builtin_bit_cast(u16x2, (x >> 8) & 0x00ff00ffu));
        };
        hi = __builtin_elementwise_max(hi, top(w));
        lo = __builtin_elementwise_max(lo, top(n));
    }
    __device__ u16x2 both() const { return u16x2{hi[0] > hi[1] ? hi[0] : hi[1], lo[0] > lo[1] ? lo[0] : lo[1]}; }
};

// Maxima over the wave of two numbers a lane, in the last lane.
__device__ __forceinline__ u16x2 wave_max2(u16x2 x) {
#define QG_DPP_MAX(ctrl, rows)                                                                                   \
    x = __builtin_elementwise_max(                                                                               \
        x, __builtin_bit_cast(u16x2, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl, rows, 0xf, false)))
    QG_DPP_MAX(0x111, 0xf);  // lane shifts by 1, 2, 4, 8 within rows of 16
    QG_DPP_MAX(0x112, 0xf);
    QG_DPP_MAX(0x114, 0xf);
    QG_DPP_MAX(0x118, 0xf);
    QG_DPP_MAX(0x142, 0xa);  // lane 15 of a row to the next
    QG_DPP_MAX(0x143, 0xc);  // lane 31 to the upper half
#undef QG_DPP_MAX
    return x;
}

// A workgroup's shape: KS waves share 32 rows, each with its own positions of a tile.
template <int DH, int KS>
struct PfxTile {
    static constexpr int RW = kDecWaves / KS, ROWS = 32 * RW;
    static constexpr int N = KS == 4 || DH == 64 ? 128 : KS == 1 && DH == 256 ? 32 : 64;  // positions
    static constexpr int CH = DH / 8, BYTES = N * DH * 2;
    static constexpr int PER = N * DH / 8192;                   // 16-byte pieces that a thread loads of K, and of V
    static constexpr int STAGES = BYTES <= 16384 ? 2 : 1;       // so that two workgroups share a compute unit
    __device__ static int k_piece(int r, int p) { return p ^ (r & (CH < 16 ? CH - 1 : 15)); }
    __device__ static int v_piece(int r, int p) { return p ^ (DH == 64 ? (r >> 1 & 1) << 2 : (r & 3) << 2); }
};

template <int DH, int KS>
struct PfxShared {
    char stage[PfxTile<DH, KS>::STAGES][2][PfxTile<DH, KS>::BYTES];
    f32x2 ml[KS][kDecWaves][32];
    u16x2 bytes[2][kDecWaves];  // of the chunk's key and value scales: the largest, and 255 less the least
    int bad[kDecWaves], wide[kDecWaves], seen[kDecWaves];
    int page[kDecChunkMax / 16];
};

template <int TYPE, int DH, int KS>
__device__ __forceinline__ void attn_prefix_group(const DecodeArgs &a, PfxShared<DH, KS> &sh, const int id) {
    typedef typename ElemOf<TYPE>::type T;
    typedef PfxTile<DH, KS> L;
    constexpr int N = L::N, NT = N / 32 / KS, KC = DH / 16, MT = DH / 32, PER = L::PER;
    constexpr int QS = kQParts<TYPE>, QF = QS == 3 ? 2 : 1;  // parts of q in bf16 and in fp16
    auto &stage = sh.stage;
    auto &sml = sh.ml;
    auto &sbytes = sh.bytes;
    auto &spage = sh.page;
    Kv4Cache prefix = a.c;
    prefix.pages = a.prefix_pages;
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int c = lane & 31, hf = lane >> 5, rw = wave % L::RW, ks = KS == 1 ? 0 : wave / L::RW;

    // workgroups are dealt to the 8 XCDs in turn: the row tiles of one chunk go to one XCD
    const int R = a.G * a.Tq * a.c.B, tiles = (R + L::ROWS - 1) / L::ROWS, units = a.c.Hkv * a.prefix_chunks;
    int u, rt;
    {
        const int whole = units / 8 * 8 * tiles;
        if (id < whole) {
            rt = (id >> 3) % tiles;
            u = (id >> 3) / tiles * 8 + (id & 7);
        } else {
            rt = (id - whole) % tiles;
            u = units / 8 * 8 + (id - whole) / tiles;
        }
    }
    const int hk = u % a.c.Hkv, ci = u / a.c.Hkv;
    const int first = ci * a.prefix_each, end = min(a.prefix, first + a.prefix_each);
    const int page = 1 << a.c.page_log2, pg0 = first >> a.c.page_log2;
    const size_t region = kv4_region_bytes(page, DH);

    bool bad = false;
    for (int i = tid; i <= ((end - 1) >> a.c.page_log2) - pg0; i += kDecWaves * kWave) {
        spage[i] = kv4_page_of(prefix, 0, pg0 + i);
        bad |= spage[i] < 0;
    }
    const bool wave_bad = __ballot(bad) != 0;
    if (lane == 0) sh.bad[wave] = wave_bad;
    // the lane's row, and what it sees
    const int row = rt * L::ROWS + 32 * rw + c;
    const bool live = row < R;
    const int t = live ? row / a.G : 0, h = hk * a.G + (live ? row - t * a.G : 0), len = a.c.lens[t / a.Tq];
    const T *qp = (const T *)a.q + (size_t)t * a.ldq + (size_t)h * DH + 8 * hf;
    Raw8<T> qraw[KC];
#pragma unroll
    for (int i = 0; i < KC; ++i) qraw[i] = load8(qp + 16 * i);
    const int see_hi = live && len >= 0 && len <= a.max_len ? max(min(len - a.Tq + t % a.Tq + 1, end), 0) : 0;
    int all_hi = live ? see_hi : end;  // where what all of the wave's rows see ends
    if (__ballot(all_hi != end))
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) all_hi = min(all_hi, shfl_xor(all_hi, x));
    all_hi = __builtin_amdgcn_readfirstlane(all_hi);
    int any_hi = see_hi;  // and what any of them sees
    if (!__ballot(any_hi == end))
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) any_hi = max(any_hi, shfl_xor(any_hi, x));
    else
        any_hi = end;
    if (lane == 0) sh.seen[wave] = any_hi;
    lds_barrier();
    bool any_bad = false;
#pragma unroll
    for (int w = 0; w < kDecWaves; ++w) any_bad |= sh.bad[w] != 0;
    any_bad = __builtin_amdgcn_readfirstlane(any_bad);
    // behind what any row sees there may be anything, also scales that are NaN: 0 * NaN
    int last = first;
#pragma unroll
    for (int w = 0; w < kDecWaves; ++w) last = max(last, sh.seen[w]);
    last = __builtin_amdgcn_readfirstlane(last);

    // A tile's bytes: keys by 32 channels of a position, values by 8 channels of four.  What lies
    // behind the end or on a bad page is read at the chunk's first place, or page 0, and has the scale 0.
    u32x4 kraw[PER], vraw[PER];
    uint32_t kbyte[PER], vbytes[PER];
    auto place = [&](int at, int *off) {
        const int id = spage[(at >> a.c.page_log2) - pg0];
        *off = at & (page - 1);
        return a.c.kv + ((size_t)max(id, 0) * a.c.Hkv + hk) * region;
    };
    auto load = [&](int j) {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int x = tid + p * kDecWaves * kWave;
            int off;
            {
                const int at = j + x / (DH / 32), ch = x % (DH / 32);
                const uint8_t *r = place(at < last ? at : first, &off);
                kraw[p] = *(const u32x4 *)(r + (size_t)off * (DH / 2) + ch * 16);
                kbyte[p] = r[(size_t)page * DH + (size_t)off * (DH / 32) + ch];
            }
            const int at = j + x / (DH / 8) * 4, ch = x % (DH / 8);
            const uint8_t *r = place(at < last ? at : first, &off);
            vraw[p] = *(const u32x4 *)(r + (size_t)page * (DH / 2) + ((size_t)(off >> 2) * (DH / 8) + ch) * 16);
            vbytes[p] = *(const uint32_t *)(r + (size_t)page * (DH + DH / 32) + ((size_t)(off >> 2) * (DH / 32) + (ch >> 2)) * 4);
        }
        stay();
    };
    const bool whole_pages = !any_bad;
    int dk = 0, dv = 0;  // powers of two on keys and values
    auto store = [&](int j, char *sk, char *sv, auto is_fast) {
        constexpr bool F = is_fast.value, KF = F && TYPE != QG_TYPE_BF16;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int x = tid + p * kDecWaves * kWave;
            {
                const int r = x / (DH / 32), ch = x % (DH / 32);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *(u32x4 *)(sk + r * DH * 2 + 16 * L::k_piece(r, 4 * ch + i)) =
                        PfxOps<KF>::eight(kraw[p][i], KF ? kbyte[p] + dk : kbyte[p]);
            }
            const int r = x / (DH / 8) * 4, ch = x % (DH / 8);
            int there = last - (j + r);  // of the four
            if (!whole_pages && there > 0 && spage[((j + r) >> a.c.page_log2) - pg0] < 0) there = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t byte = vbytes[p] >> (8 * i) & 255u;
                *(u32x4 *)(sv + (r + i) * DH * 2 + 16 * L::v_piece(r + i, ch)) =
                    PfxOps<F>::eight(vraw[p][i], i < there ? (F ? byte + dv : byte) : 0u);
            }
        }
    };
    load(first);

    // the range of the chunk's scales
    {
        ByteRange k, v;
        constexpr int QUADS = DH / 32;  // 16-byte pieces of 16 positions' scales
        const int n = (last - first + 15) / 16 * QUADS;
        for (int i = tid; i < 2 * n; i += kDecWaves * kWave) {
            const bool val = i >= n;
            const int x = val ? i - n : i, j = first + x / QUADS * 16, piece = x % QUADS;
            const int id = spage[(j >> a.c.page_log2) - pg0];
            if (id < 0) continue;
            const uint8_t *p = a.c.kv + ((size_t)id * a.c.Hkv + hk) * region + (size_t)page * (val ? DH + DH / 32 : DH) +
                               (size_t)(j & (page - 1)) * (DH / 32) + piece * 16;
            const u32x4 w = *(const u32x4 *)p;
            ByteRange &r = val ? v : k;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                if (j + 16 <= last) {
                    r.add(w[d]);
                    continue;
                }
                const int at = piece * 4 + d;  // dword of the tile's scales; only those of positions before the end
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (j + (val ? at / (DH / 32) * 4 + b : (4 * at + b) / (DH / 32)) < last)
                        r.add((w[d] >> (8 * b) & 255u) * 0x01010101u);
            }
        }
        const u16x2 kr = wave_max2(k.both()), vr = wave_max2(v.both());
        if (lane == kWave - 1) sbytes[0][wave] = kr, sbytes[1][wave] = vr;
    }
    int qexp = 0;  // power of two off the row's queries
    if constexpr (TYPE == QG_TYPE_F32) {
        uint32_t most_q = 0, least_q = ~0u;  // magnitudes, as bits; the least that is not 0, less 1
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t x = __builtin_bit_cast(uint32_t, elem(qraw[i], e)) & 0x7fffffffu;
                most_q = max(most_q, x);
                least_q = min(least_q, x - 1);
            }
        const float most = half_max(__builtin_bit_cast(float, most_q));
        const float least = least_q == ~0u ? INFINITY : __builtin_bit_cast(float, least_q + 1);
        if (most > 0.f) qexp = __builtin_amdgcn_frexp_expf(most) - 15;
        // the first part of what is within 2^26 of the row's largest is a normal number: two parts are off by 2^-23 of it
        const bool wide = __ballot(least * 0x1p26f < most || qexp < -60 || qexp > 60) != 0;
        if (lane == 0) sh.wide[wave] = wide;
    }
    bool fast;
    {
        lds_barrier();  // the first tile's loads stay in flight
        u16x2 k = {0, 0}, v = {0, 0};
        fast = true;
#pragma unroll
        for (int w = 0; w < kDecWaves; ++w) {
            k = __builtin_elementwise_max(k, sbytes[0][w]);
            v = __builtin_elementwise_max(v, sbytes[1][w]);
            if (TYPE == QG_TYPE_F32) fast = fast && !sh.wide[w];
        }
        // the largest becomes 2^13 (6 * 2^13 < 65504), the least 2^-23 (half of it is fp16's least)
        fast = fast && v[0] + v[1] <= 255 + 36 && v[0] > 0;
        dv = 140 - v[0];
        if (TYPE != QG_TYPE_BF16) {
            fast = fast && k[0] + k[1] <= 255 + 36 && k[0] > 0;
            dk = 140 - k[0];
        }
        const int e = __builtin_amdgcn_frexp_expf(a.scale) - dk;  // scores' factor, but for qexp: far from fp32's ends
        fast = __builtin_amdgcn_readfirstlane(fast && e >= -60 && e <= 60);
        dk = __builtin_amdgcn_readfirstlane(fast ? dk : 0);
        dv = __builtin_amdgcn_readfirstlane(fast ? dv : 0);
        if (!fast) qexp = 0;
    }
    const float scale = __builtin_ldexpf(a.scale, qexp - dk);  // of a row's scores as they are computed

    u32x4 qf[QF][KC];
    constexpr float kRest = 0x1p12f;  // on the second part of a query: at most 2^3 without
    if constexpr (TYPE == QG_TYPE_F32) {
        const float factor = a.qsign * __builtin_ldexpf(1.f, -qexp);
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x0 = elem(qraw[i], 2 * e) * factor, x1 = elem(qraw[i], 2 * e + 1) * factor;
                const f16x2 hi = __builtin_convertvector((f32x2{x0, x1}), f16x2);
                const f32x2 rest = {__builtin_fmaf((float)hi[0], -1.f, x0), __builtin_fmaf((float)hi[1], -1.f, x1)};
                qf[0][i][e] = __builtin_bit_cast(uint32_t, hi);
                qf[1][i][e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest * kRest, f16x2));
            }
    } else {
        const uint32_t flip = a.qsign < 0.f ? 0x80008000u : 0u, keep = a.qsign == 0.f ? 0u : ~0u;
#pragma unroll
        for (int i = 0; i < KC; ++i) qf[0][i] = (qraw[i].w[0] ^ flip) & keep;
    }

    f32x16 o[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int x = 0; x < 16; ++x) o[i][x] = 0.f;
    RunningMax most;
    float l = 0.f;

    constexpr int OWN = 32 * NT;  // positions of a tile that are this wave's, from r0 on
    const int r0 = ks * OWN;
    auto step = [&](int j, const char *sk, const char *sv, auto is_fast) {
        constexpr bool F = is_fast.value, KF = F && TYPE != QG_TYPE_BF16;
        constexpr int PP = F ? 2 : 3;  // parts of weights
        constexpr float kShift = F ? 11.f : 0.f, kSlack = F ? 4.f : kDecSlack;
        f32x16 s[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 16; ++x) s[n][x] = 0.f;
        auto key = [&](int n, int i) {
            const int r = r0 + 32 * n + c;
            return *(const u32x4 *)(sk + r * DH * 2 + 16 * L::k_piece(r, 2 * i + hf));
        };
        if constexpr (F && QF == 2) {  // the second parts first, then what was on them taken off
#pragma unroll
            for (int i = 0; i < KC; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n] = PfxOps<KF>::mfma(key(n, i), qf[1][i], s[n]);
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n] *= 1 / kRest;
            asm volatile("" ::: "memory");  // or the keys stay in registers for the products below, which spill
        }
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            bf16x8 slow[QS];  // rare: read and split again at each tile, no registers kept
            if constexpr (!F && QS > 1) split8<QS>(load8(qp + 16 * i), a.qsign, slow);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const u32x4 kf = key(n, i);
                if constexpr (!F && QS > 1) {
#pragma unroll
                    for (int p = 0; p < QS; ++p) s[n] = PfxOps<false>::mfma(kf, __builtin_bit_cast(u32x4, slow[p]), s[n]);
                } else {
                    s[n] = PfxOps<KF>::mfma(kf, qf[0][i], s[n]);
                }
            }
        }
        // register 4 x + y of tile n: position 32 n + 8 x + 4 hf + y
        const int j0 = j + r0;
        if (j0 + OWN > all_hi || any_bad) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 16; ++x)
                    if (j0 + 32 * n + 8 * (x / 4) + 4 * hf + x % 4 >= see_hi) s[n][x] = -INFINITY;
            if (any_bad)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int at = j0 + 32 * n + 16 * y;
                        if (at < last && spage[(at >> a.c.page_log2) - pg0] < 0)
#pragma unroll
                            for (int x = 0; x < 8; ++x) s[n][8 * y + x] = -INFINITY;
                    }
        }
        float mt = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 16; ++x) mt = __builtin_fmaxf(mt, s[n][x]);
        mt = half_max(mt);
        if (__ballot((mt - most.m) * scale > kSlack) | most.far) {
            const float keep = most.raise(mt, scale, kShift);
            if (most.far) {
                const float raw = most.raw(scale);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 16; ++x) s[n][x] -= raw;
            }
            l *= keep;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i] *= keep;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int kc = 0; kc < 2; ++kc) {
                u32x4 pf[PP];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][8 * kc + 2 * e], scale, -most.muse));
                    float x1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][8 * kc + 2 * e + 1], scale, -most.muse));
                    l += x0;
                    l += x1;
                    if constexpr (F) {
                        const f16x2 hi = __builtin_convertvector((f32x2{x0, x1}), f16x2);
                        const f32x2 rest = {__builtin_fmaf((float)hi[0], -1.f, x0), __builtin_fmaf((float)hi[1], -1.f, x1)};
                        pf[0][e] = __builtin_bit_cast(uint32_t, hi);
                        pf[1][e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, f16x2));
                    } else {
#pragma unroll
                        for (int p = 0; p < PP; ++p) {  // eight bits at a time, cut off: no rounding
                            const uint32_t b0 = __builtin_bit_cast(uint32_t, x0), b1 = __builtin_bit_cast(uint32_t, x1);
                            pf[p][e] = __builtin_amdgcn_perm(b1, b0, 0x07060302u);
                            x0 -= __builtin_bit_cast(float, b0 & 0xffff0000u);
                            x1 -= __builtin_bit_cast(float, b1 & 0xffff0000u);
                        }
                    }
                }
                const int r = r0 + 32 * n + 16 * kc + 4 * hf + (lane & 15) / 4;  // and r + 8
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int p = 4 * i + 2 * (c >> 4) + (lane & 3) / 2;
                    const int at = r * DH * 2 + 16 * L::v_piece(r, p) + 8 * (lane & 1);
                    const u32x2 x = lds_read_column4(sv + at), y = lds_read_column4(sv + (at + 8 * DH * 2));
#pragma unroll
                    for (int w = 0; w < PP; ++w) o[i] = PfxOps<F>::mfma(u32x4{x[0], x[1], y[0], y[1]}, pf[w], o[i]);
                }
            }
    };
    auto walk = [&](auto is_fast) {
        if constexpr (L::STAGES == 2) {  // a tile's operands are made while the last one's are used
            int s = 1;
            for (int j = first - N; j < last; j += N) {
                lds_barrier();  // all are done with the stage, and the other one is complete
                if (j + N < last) {
                    store(j + N, stage[s ^ 1][0], stage[s ^ 1][1], is_fast);
                    if (j + 2 * N < last) load(j + 2 * N);
                }
                if (j >= first) step(j, stage[s][0], stage[s][1], is_fast);
                s ^= 1;
            }
        } else {
            for (int j = first; j < last; j += N) {
                lds_barrier();
                store(j, stage[0][0], stage[0][1], is_fast);
                if (j + N < last) load(j + N);
                lds_barrier();
                step(j, stage[0][0], stage[0][1], is_fast);
            }
        }
    };
    if (fast)
        walk(std::true_type{});
    else
        walk(std::false_type{});

    const float exact = most.exact(scale, fast ? 11.f : 0.f), unshift = fast ? 0x1p-11f : 1.f;
    float top = most.m, keep = exact * unshift;
    l = (l + shfl_xor(l, 32)) * exact;
    if constexpr (KS > 1) {  // maximum and sum of the waves that share rows
        if (hf == 0) sml[ks][rw][c] = f32x2{most.m, l};
        __syncthreads();  // and all are done with the stages
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < KS; ++x) top = __builtin_fmaxf(top, sml[x][rw][c][0]);
        const float use = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int x = 0; x < KS; ++x) sum += sml[x][rw][c][1] * __builtin_amdgcn_exp2f((sml[x][rw][c][0] - use) * scale);
        keep *= __builtin_amdgcn_exp2f((most.m - use) * scale);
        l = sum;
    }
    const size_t at = ((size_t)t * a.H + h) * a.chunks + ci;
    if (live && ks == 0 && hf == 0) a.pml[at] = f32x2{__builtin_ldexpf(top, qexp - dk), l * unshift};
    // the sums: each of those waves adds and writes a part of the registers, the others' through the stages
    constexpr int QX = 4 / KS;  // quarters of a tile's registers that are this wave's
    f32x4 *room = reinterpret_cast<f32x4 *>(&stage[0][0][0]);
    auto place_of = [&](int from, int to) {  // [rw][from][to, but for from][quarter][tile][lane]
        return room + ((((rw * KS + from) * (KS - 1) + (to > from ? to - 1 : to)) * QX) * MT) * kWave + lane;
    };
    static_assert(KS == 1 || sizeof(sh.stage) >= L::RW * KS * (KS - 1) * QX * MT * kWave * 16, "the waves' sums fit the stages");
    f32x4 mine[QX][MT];
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const f32x4 v = f32x4{o[i][4 * x], o[i][4 * x + 1], o[i][4 * x + 2], o[i][4 * x + 3]} * keep;
            if (KS == 1 || x / QX == ks)
                mine[x % QX][i] = v;
            else
                place_of(ks, x / QX)[(x % QX * MT + i) * kWave] = v;
        }
    if constexpr (KS > 1) {
        __syncthreads();
#pragma unroll
        for (int y = 1; y < KS; ++y) {
            const f32x4 *from = place_of((ks + y) % KS, ks);
#pragma unroll
            for (int x = 0; x < QX; ++x)
#pragma unroll
                for (int i = 0; i < MT; ++i) mine[x][i] += from[(x * MT + i) * kWave];
        }
    }
    if (!live) return;
    const float back = __builtin_ldexpf(1.f, -dv);  // dv is between -113 and 133: not 0
    float *dst = a.po + at * DH + 8 * QX * ks + 4 * hf;  // register 4 x + y of tile i: channel 32 i + 8 x + 4 hf + y
#pragma unroll
    for (int x = 0; x < QX; ++x)
#pragma unroll
        for (int i = 0; i < MT; ++i) *(f32x4 *)(dst + 32 * i + 8 * x) = mine[x][i] * back;
}

// The shared positions' workgroups, then those of the sequences' own positions, which
// are shorter and fill what is left of the card.
template <int TYPE, int DH, int KS>
__global__ __launch_bounds__(kDecWaves *kWave, DH == 256 && TYPE == QG_TYPE_F32 ? 1 : 2) void attn_prefix_kernel(
    DecodeArgs a, int shared_groups, int own_groups) {
    constexpr size_t P = sizeof(PfxShared<DH, KS>), D = sizeof(DecShared<DH, kDecWaves>);
    __shared__ __attribute__((aligned(16))) char room[P > D ? P : D];
    const int id = blockIdx.x;
    if (id < shared_groups)
        attn_prefix_group<TYPE, DH, KS>(a, *reinterpret_cast<PfxShared<DH, KS> *>(room), id);
    else
        attn_decode_group<TYPE, DH, 1, TAIL, kDecWaves>(a, *reinterpret_cast<DecShared<DH, kDecWaves> *>(room), (id - shared_groups) % own_groups,
                                             (id - shared_groups) / own_groups);
}

template <int TYPE, int DH, int KS>
static int launch_prefix_ks(const DecodeArgs &a, hipStream_t stream) {
    constexpr int ROWS = PfxTile<DH, KS>::ROWS;
    const long long rows = (long long)a.G * a.Tq * a.c.B, shared = (rows + ROWS - 1) / ROWS * a.c.Hkv * a.prefix_chunks;
    const long long own = (long long)a.c.Hkv * a.c.B * (a.chunks - a.prefix_chunks), tiles = (a.G * a.Tq + 15) / 16;
    if (shared + own * tiles > kMaxGroups) return QG_ERR_SHAPE;
    hipLaunchKernelGGL((attn_prefix_kernel<TYPE, DH, KS>), dim3((unsigned)(shared + own * tiles)),
                       dim3(kDecWaves * kWave), 0, stream, a, (int)shared, (int)own);
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

template <int TYPE, int DH>
static int launch_prefix_dh(const DecodeArgs &a, hipStream_t stream) {
    switch (a.prefix_rows) {
        case 128: return launch_prefix_ks<TYPE, DH, 1>(a, stream);
        case 64: return launch_prefix_ks<TYPE, DH, 2>(a, stream);
        default: return launch_prefix_ks<TYPE, DH, DH == 256 ? 2 : 4>(a, stream);
    }
}

template <int TYPE>
static int launch_prefix(const DecodeArgs &a, int Dh, hipStream_t stream) {
    switch (Dh) {
        case 64: return launch_prefix_dh<TYPE, 64>(a, stream);
        case 128: return launch_prefix_dh<TYPE, 128>(a, stream);
        default: return launch_prefix_dh<TYPE, 256>(a, stream);
    }
}

// Rows of a workgroup and chunks that take the least time by what was measured (us, fp32
// queries, 128 channels): 128 positions of 128, 64, 32 rows take a workgroup 5.2, 2.5, 1.5 alone
// on a compute unit, 7.4, 4.2, 2.5 beside another; a second one leaves no room for the sequences' own
// positions, which then come behind (8); a chunk's sums, written and read, 0.4 a megabyte.  48
// sequences of 8 rows a head over 40001: 128 rows in 21 chunks 128, in 11 168, 64 rows 145, 32
// rows 173; 32 of 4 rows over 6001: 128 rows in 32 chunks 27, 64 in 16 26, 32 in 8 24, in 16 31.
// Each sequence by itself (no chunks) takes about 22 for 10^6 times 16 rows' positions, and
// 3 less to begin with: 4 sequences over 300 8.6 and 13.9, 2 over 30000 20 and 28, 48 of 16 rows
// over 1500 28 and 34, 16 of 4 rows over 4000 22 and 18, 8 of 2 over 16000 27 and 18.
PrefixSplit prefix_split(int B, long long rows, int Hkv, int Dh, int prefix) {
    PrefixSplit best{0, 0, 0};
    double least = (double)((rows / B + 15) / 16) * B * Hkv * prefix * Dh / 128 * 22e-6 - 3;
    for (int tile = 128; tile >= (Dh == 256 ? 64 : 32); tile /= 2)
        for (int fit = 256; fit <= 512; fit *= 2) {
            const long long groups = (rows + tile - 1) / tile * Hkv;
            long long chunks = groups < fit ? fit / groups : 1;
            long long each = ((prefix + chunks - 1) / chunks + 127) / 128 * 128;
            if (each > kDecChunkMax) each = kDecChunkMax;
            chunks = (prefix + each - 1) / each;
            const bool beside = groups * chunks > 256;
            const double step = tile == 128 ? (beside ? 7.4 : 5.2) : tile == 64 ? (beside ? 4.2 : 2.5) : beside ? 2.5 : 1.5;
            const double rounds = (double)((groups * chunks + 511) / 512);
            const double us = rounds * each / 128 * step * Dh / 128 + (beside ? 8 : 0) + rows * Hkv * chunks * Dh * 4 * 0.4e-6;
            if (us < least) best = PrefixSplit{tile, (int)each, (int)chunks}, least = us;
        }
    return best;
}

int launch_attn_prefix(int type, int Dh, const DecodeArgs &a, hipStream_t stream) {
    switch (type) {
        case QG_TYPE_F32: return launch_prefix<QG_TYPE_F32>(a, Dh, stream);
        case QG_TYPE_F16: return launch_prefix<QG_TYPE_F16>(a, Dh, stream);
        default: return launch_prefix<QG_TYPE_BF16>(a, Dh, stream);
    }
}

}  // namespace qg
