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
// parts (22 bits, or 2^-36 of the row's largest), an fp32 query two (24 bits of what is
// within 2^26 of the row's largest, else the chunk is not taken so) and an fp16 one itself.  Other
// chunks, and the keys of bf16 queries, take bf16, which holds every value exactly, and
// three parts for 24 bits: five and three products in place of four and three, and six.
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

// Least and largest of the scale bytes seen so far, in the halves of two dwords.
struct ByteRange {
    u16x2 lo = {255, 255}, hi = {0, 0};
    __device__ void add(uint32_t w) {
        const u16x2 e = __builtin_bit_cast(u16x2, w & 0x00ff00ffu), o = __builtin_bit_cast(u16x2, (w >> 8) & 0x00ff00ffu);
        lo = __builtin_elementwise_min(lo, __builtin_elementwise_min(e, o));
        hi = __builtin_elementwise_max(hi, __builtin_elementwise_max(e, o));
    }
    // least and largest of the wave's bytes, as least + 256 * largest
    __device__ uint32_t of_wave() const {
        int l = min((int)lo[0], (int)lo[1]), h = max((int)hi[0], (int)hi[1]);
#pragma unroll
        for (int x = 1; x < kWave; x <<= 1) {
            l = min(l, shfl_xor(l, x));
            h = max(h, shfl_xor(h, x));
        }
        return (uint32_t)(l | h << 8);
    }
};

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
    uint32_t bytes[2][kDecWaves];
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
    const int first = ci * a.prefix_each, last = min(a.prefix, first + a.prefix_each);
    const int page = 1 << a.c.page_log2, pg0 = first >> a.c.page_log2;
    const size_t region = kv4_region_bytes(page, DH);

    bool bad = false;
    for (int i = tid; i <= ((last - 1) >> a.c.page_log2) - pg0; i += kDecWaves * kWave) {
        spage[i] = kv4_page_of(prefix, 0, pg0 + i);
        bad |= spage[i] < 0;
    }
    // the lane's row, and what it sees
    const int row = rt * L::ROWS + 32 * rw + c;
    const bool live = row < R;
    const int t = live ? row / a.G : 0, h = hk * a.G + (live ? row - t * a.G : 0), len = a.c.lens[t / a.Tq];
    const T *qp = (const T *)a.q + (size_t)t * a.ldq + (size_t)h * DH + 8 * hf;
    Raw8<T> qraw[KC];
#pragma unroll
    for (int i = 0; i < KC; ++i) qraw[i] = load8(qp + 16 * i);
    const int see_hi = live && len >= 0 && len <= a.max_len ? max(min(len - a.Tq + t % a.Tq + 1, last), 0) : 0;
    int all_hi = live ? see_hi : last;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) all_hi = min(all_hi, shfl_xor(all_hi, x));
    all_hi = __builtin_amdgcn_readfirstlane(all_hi);
    const bool any_bad = __syncthreads_or(bad);

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
        const uint32_t kr = k.of_wave(), vr = v.of_wave();
        if (lane == 0) sbytes[0][wave] = kr, sbytes[1][wave] = vr;
    }
    float most_q = 0.f, least_q = INFINITY;  // of the row
    if constexpr (TYPE == QG_TYPE_F32) {
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = __builtin_fabsf(elem(qraw[i], e) * a.qsign);
                most_q = __builtin_fmaxf(most_q, x);
                least_q = __builtin_fminf(least_q, x > 0.f ? x : INFINITY);
            }
        most_q = half_max(most_q);
        least_q = -half_max(-least_q);
    }
    int qexp = 0;  // power of two off the row's queries
    bool fast;
    {
        const int qe = most_q > 0.f ? __builtin_amdgcn_frexp_expf(most_q) - 15 : 0;
        bool wide = TYPE == QG_TYPE_F32 && least_q * 0x1p26f < most_q;
        lds_barrier();  // the first tile's loads stay in flight
        int kl = 255, kh = 0, vl = 255, vh = 0;
#pragma unroll
        for (int w = 0; w < kDecWaves; ++w) {
            kl = min(kl, (int)(sbytes[0][w] & 255u)), kh = max(kh, (int)(sbytes[0][w] >> 8));
            vl = min(vl, (int)(sbytes[1][w] & 255u)), vh = max(vh, (int)(sbytes[1][w] >> 8));
        }
        // the largest becomes 2^13 (6 * 2^13 < 65504), the least 2^-23 (half of it is fp16's least)
        fast = vh - vl <= 36 && vh > 0;
        dv = 140 - vh;
        if (TYPE != QG_TYPE_BF16) {
            fast = fast && kh - kl <= 36 && kh > 0;
            dk = 140 - kh;
        }
        const int e = __builtin_amdgcn_frexp_expf(a.scale) + qe - dk;
        wide |= e < -100 || e > 100;
        fast = !__syncthreads_or(wide || !fast);
        qexp = fast ? qe : 0;
        dk = __builtin_amdgcn_readfirstlane(fast ? dk : 0);
        dv = __builtin_amdgcn_readfirstlane(fast ? dv : 0);
    }
    const float scale = __builtin_ldexpf(a.scale, qexp - dk);  // of a row's scores as they are computed

    u32x4 qf[QF][KC];
#pragma unroll
    for (int i = 0; i < KC; ++i) {
        if constexpr (TYPE == QG_TYPE_BF16) {
            bf16x8 part[1];
            split8<1>(qraw[i], a.qsign, part);
            qf[0][i] = __builtin_bit_cast(u32x4, part[0]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x0 = __builtin_ldexpf(elem(qraw[i], 2 * e) * a.qsign, -qexp);
                const float x1 = __builtin_ldexpf(elem(qraw[i], 2 * e + 1) * a.qsign, -qexp);
                const f16x2 hi = __builtin_convertvector((f32x2{x0, x1}), f16x2);
                qf[0][i][e] = __builtin_bit_cast(uint32_t, hi);
                if constexpr (QF == 2) {
                    const f32x2 rest = {x0 - (float)hi[0], x1 - (float)hi[1]};
                    qf[1][i][e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, f16x2));
                }
            }
        }
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
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            bf16x8 slow[QS];  // rare: read and split again at each tile, no registers kept
            if constexpr (!F && QS > 1) split8<QS>(load8(qp + 16 * i), a.qsign, slow);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = r0 + 32 * n + c;
                const u32x4 kf = *(const u32x4 *)(sk + r * DH * 2 + 16 * L::k_piece(r, 2 * i + hf));
                if constexpr (!F && QS > 1) {
#pragma unroll
                    for (int p = 0; p < QS; ++p) s[n] = PfxOps<false>::mfma(kf, __builtin_bit_cast(u32x4, slow[p]), s[n]);
                } else {
#pragma unroll
                    for (int p = 0; p < QF; ++p) s[n] = PfxOps<KF>::mfma(kf, qf[p][i], s[n]);
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
        if constexpr (L::STAGES == 2) {
            store(first, stage[0][0], stage[0][1], is_fast);
            if (first + N < last) load(first + N);
        }
        int s = 0;
        for (int j = first; j < last; j += N) {
            // this tile's operands are there for all waves, and all are done with the other stage
            lds_barrier();
            if constexpr (L::STAGES == 2) {
                if (j + N < last) {
                    store(j + N, stage[s ^ 1][0], stage[s ^ 1][1], is_fast);
                    if (j + 2 * N < last) load(j + 2 * N);
                }
            } else {
                store(j, stage[0][0], stage[0][1], is_fast);
                if (j + N < last) load(j + N);
                lds_barrier();
            }
            step(j, stage[s][0], stage[s][1], is_fast);
            if (L::STAGES == 2) s ^= 1;
        }
    };
    if (fast)
        walk(std::true_type{});
    else
        walk(std::false_type{});

    const float exact = most.exact(scale, fast ? 11.f : 0.f), unshift = fast ? 0x1p-11f : 1.f;
    float top = most.m, keep = exact * unshift;
    l = (l + shfl_xor(l, 32)) * exact;
    if constexpr (KS > 1) {  // join the waves that share rows, through the stages
        if (hf == 0) sml[ks][rw][c] = f32x2{most.m, l};
        __syncthreads();
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < KS; ++x) top = __builtin_fmaxf(top, sml[x][rw][c][0]);
        const float use = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int x = 0; x < KS; ++x) sum += sml[x][rw][c][1] * __builtin_amdgcn_exp2f((sml[x][rw][c][0] - use) * scale);
        keep *= __builtin_amdgcn_exp2f((most.m - use) * scale);
        l = sum;
        static_assert(sizeof(stage) >= (KS - 1) * L::RW * 32 * DH * 4, "the waves' sums fit the stages");
        f32x4 *room = reinterpret_cast<f32x4 *>(&stage[0][0][0]);
#pragma unroll
        for (int i = 0; i < MT; ++i) o[i] *= keep;
        keep = 1.f;
        if (ks > 0)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    room[(((ks - 1) * L::RW + rw) * MT * 4 + 4 * i + x) * kWave + lane] =
                        f32x4{o[i][4 * x], o[i][4 * x + 1], o[i][4 * x + 2], o[i][4 * x + 3]};
        __syncthreads();
        if (ks > 0) return;
        for (int y = 1; y < KS; ++y)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const f32x4 v = room[(((y - 1) * L::RW + rw) * MT * 4 + 4 * i + x) * kWave + lane];
#pragma unroll
                    for (int z = 0; z < 4; ++z) o[i][4 * x + z] += v[z];
                }
    }
    if (!live) return;
    const size_t at = ((size_t)t * a.H + h) * a.chunks + ci;
    if (hf == 0) a.pml[at] = f32x2{__builtin_ldexpf(top, qexp - dk), l * unshift};
    float *dst = a.po + at * DH + 4 * hf;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            f32x4 v;
#pragma unroll
            for (int z = 0; z < 4; ++z) v[z] = __builtin_ldexpf(o[i][4 * x + z] * keep, -dv);
            *(f32x4 *)(dst + 32 * i + 8 * x) = v;
        }
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
// 3 less to begin with: 4 sequences over 300 8.4 and 13.9, 2 over 30000 20 and 28, 48 of 16 rows
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
