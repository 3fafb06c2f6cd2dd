// Attention over the positions that all sequences of a batch share.
//
// The query rows of all sequences (tokens and heads that read one key/value head) are
// one matrix against the shared keys.  A workgroup takes 32 NR rows and a chunk of the
// positions, its four waves 32 positions each at a time, with the running maximum and sum
// of a softmax:
//   S^T = K Q^T    (positions x rows),  O^T += V^T P^T   (channels x rows),
// as v_mfma_f32_32x32x16.  A lane keeps one query row (of each 32) throughout, and the scores
// that it receives are the weights that it supplies.  Keys and values go from the cache's
// bytes to operands in registers, once for all rows.
#include <type_traits>

#include "attn_decode_device.h"

namespace qg {

constexpr int kPfxStride = kDecWaves * kDecStep;

// Operands: fp16 where a chunk's scales span no more than fp16 holds exactly, with one
// power of two taken off all keys and off all values; bf16 else.
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

template <int TYPE, int DH, int NR>
__global__ __launch_bounds__(kDecWaves *kWave, 2) void attn_prefix_kernel(DecodeArgs a) {
    typedef typename ElemOf<TYPE>::type T;
    constexpr int KC = DH / 16, MT = DH / 32, ROWS = 32 * NR;   // key products, channel tiles
    constexpr int QS = kQParts<TYPE>, QF = QS == 3 ? 2 : 1;      // parts of q in bf16 and in fp16
    constexpr int JT = MT < 4 ? MT : 4;                          // channel tiles joined at a time
    constexpr int QBYTES = QS * NR * KC * 1024, JBYTES = 12 * JT * 1024;
    __shared__ __attribute__((aligned(16))) char room[QBYTES > JBYTES ? QBYTES : JBYTES];
    u32x4 *sq = reinterpret_cast<u32x4 *>(room);
    __shared__ f32x2 sml[kDecWaves][NR][32];
    __shared__ f32x2 sqr[kDecWaves][NR][32];  // largest and least |q| of a row
    __shared__ uint32_t sbytes[2][kDecWaves];
    __shared__ int spage[kDecChunkMax / 16];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int c = lane & 31, hf = lane >> 5;

    // workgroups are dealt to the 8 XCDs in turn: the row tiles of one chunk go to one XCD
    const int R = a.G * a.Tq * a.c.B, tiles = (R + ROWS - 1) / ROWS, units = a.c.Hkv * a.prefix_chunks;
    int u, rt;
    {
        const int id = blockIdx.x, whole = units / 8 * 8 * tiles;
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
    const int page = 1 << a.c.page_log2;
    const size_t region = kv4_region_bytes(page, DH);

    // the wave's pieces of q: of row tile and key product (n, i), every fourth
    constexpr int QN = NR * KC / kDecWaves;
    Raw8<T> qraw[QN];
    int see_hi[NR], all_hi = a.prefix;
    size_t out_row[NR];
    bool live[NR];
    {
        const T *qp[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int row = rt * ROWS + 32 * n + c;
            live[n] = row < R;
            const int t = live[n] ? row / a.G : 0, h = hk * a.G + (live[n] ? row - t * a.G : 0), len = a.c.lens[t / a.Tq];
            out_row[n] = (size_t)t * a.H + h;
            qp[n] = (const T *)a.q + (size_t)t * a.ldq + (size_t)h * DH + hf * (DH / 2);
            see_hi[n] = 0;
            if (live[n]) {
                if (len >= 0 && len <= a.max_len) see_hi[n] = max(min(len - a.Tq + t % a.Tq + 1, a.prefix), 0);
                all_hi = min(all_hi, see_hi[n]);
            }
        }
#pragma unroll
        for (int k = 0; k < QN; ++k) qraw[k] = load8(qp[k * kDecWaves / KC] + (k * kDecWaves % KC + wave) * 8);
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) all_hi = min(all_hi, shfl_xor(all_hi, x));
        all_hi = __builtin_amdgcn_readfirstlane(all_hi);
    }
    for (int i = threadIdx.x; i <= ((last - 1) >> a.c.page_log2) - (first >> a.c.page_log2); i += kDecWaves * kWave)
        spage[i] = kv4_page_of(a.c, 0, (first >> a.c.page_log2) + i);
    __syncthreads();

    // A step's two tiles of 16 positions; one behind the end or on a bad page reads the
    // chunk's first place, or page 0, instead and is masked.
    uint32_t kraw[KC], kscale;
    u32x4 vraw[2][2];
    uint32_t vscale[2][2];
    const uint8_t *at_tile[2];  // the region
    int at_off[2];
    bool next_ok[2];
    auto locate = [&](int j) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int j0 = j + 16 * x, at = j0 < last ? j0 : first;
            const int id = __builtin_amdgcn_readfirstlane(spage[(at >> a.c.page_log2) - (first >> a.c.page_log2)]);
            next_ok[x] = j0 < last && id >= 0;
            at_tile[x] = a.c.kv + ((size_t)max(id, 0) * a.c.Hkv + hk) * region;
            at_off[x] = at & (page - 1);
        }
    };
    auto load_k = [&] {  // of position c, half of the channels
        const uint8_t *t = c < 16 ? at_tile[0] : at_tile[1];
        const int off = (c < 16 ? at_off[0] : at_off[1]) + (c & 15);
        const uint8_t *k = t + (size_t)off * (DH / 2) + hf * (DH / 4);
        const uint8_t *s = t + (size_t)page * DH + (size_t)off * (DH / 32) + hf * (DH / 64);
#pragma unroll
        for (int i = 0; i < KC; i += 4) {
            const u32x4 w = *(const u32x4 *)(k + 4 * i);
#pragma unroll
            for (int x = 0; x < 4; ++x) kraw[i + x] = w[x];
        }
        if constexpr (DH == 64)
            kscale = *s;
        else if constexpr (DH == 128)
            kscale = *(const uint16_t *)s;
        else
            kscale = *(const uint32_t *)s;
        stay();
    };
    auto load_v = [&] {  // channels MT c.. of positions 4 hf.. and 8 + 4 hf.. of each tile
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint8_t *v = at_tile[x] + (size_t)page * (DH / 2) + (size_t)at_off[x] * (DH / 2);
                const uint8_t *s = at_tile[x] + (size_t)page * (DH + DH / 32) + (size_t)at_off[x] * (DH / 32);
                vraw[x][y] = *(const u32x4 *)(v + ((2 * y + hf) * (DH / 8) + c * MT / 8) * 16);
                vscale[x][y] = *(const uint32_t *)(s + ((2 * y + hf) * (DH / 32) + c * MT / 32) * 4);
            }
        stay();
    };
    const int j_first = first + wave * kDecStep;
    locate(j_first);
    load_k();
    load_v();

    // the range of the chunk's scales, and of each row's queries
    {
        ByteRange k, v;
        constexpr int QUADS = DH / 32;  // 16-byte pieces of a tile's scales
        const int n = (last - first + 15) / 16 * QUADS;
        for (int i = threadIdx.x; i < 2 * n; i += kDecWaves * kWave) {
            const bool val = i >= n;
            const int x = val ? i - n : i, j = first + x / QUADS * 16, piece = x % QUADS;
            const int id = spage[(j >> a.c.page_log2) - (first >> a.c.page_log2)];
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
    if constexpr (TYPE == QG_TYPE_F32) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            float most = 0.f, least = INFINITY;
#pragma unroll
            for (int k = n * QN / NR; k < (n + 1) * QN / NR; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = __builtin_fabsf(elem(qraw[k], e) * a.qsign);
                    most = __builtin_fmaxf(most, x);
                    least = __builtin_fminf(least, x > 0.f ? x : INFINITY);
                }
            most = half_max(most);
            least = -half_max(-least);
            if (hf == 0) sqr[wave][n][c] = f32x2{most, least};
        }
    }
    __syncthreads();
    int dk = 0, dv = 0, qexp[NR];  // powers of two on keys and values, off each row's queries
    bool fast;
    {
        int kl = 255, kh = 0, vl = 255, vh = 0;
#pragma unroll
        for (int w = 0; w < kDecWaves; ++w) {
            kl = min(kl, (int)(sbytes[0][w] & 255u)), kh = max(kh, (int)(sbytes[0][w] >> 8));
            vl = min(vl, (int)(sbytes[1][w] & 255u)), vh = max(vh, (int)(sbytes[1][w] >> 8));
        }
        // 6 * 2^13 < 65504, and half of 2^-23 is fp16's least: 36 binades
        fast = vh - vl <= 36 && vh > 0;
        dv = 140 - vh;
        if (TYPE != QG_TYPE_BF16) {
            fast = fast && kh - kl <= 36 && kh > 0;
            dk = 140 - kh;
        }
        const int sexp = __builtin_amdgcn_frexp_expf(a.scale);
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            qexp[n] = 0;
            if (TYPE == QG_TYPE_F32) {
                float most = 0.f, least = INFINITY;
#pragma unroll
                for (int w = 0; w < kDecWaves; ++w) {
                    most = __builtin_fmaxf(most, sqr[w][n][c][0]);
                    least = __builtin_fminf(least, sqr[w][n][c][1]);
                }
                // two parts hold 24 bits of what is within 2^26 of the row's largest
                if (__ballot(least * 0x1p26f < most)) fast = false;
                if (most > 0.f) qexp[n] = __builtin_amdgcn_frexp_expf(most) - 15;
            }
            const int e = sexp + qexp[n] - dk;
            if (__ballot(e < -100 || e > 100)) fast = false;
        }
        fast = __builtin_amdgcn_readfirstlane(fast);
        if (!fast) {
            dk = dv = 0;
#pragma unroll
            for (int n = 0; n < NR; ++n) qexp[n] = 0;
        }
        dk = __builtin_amdgcn_readfirstlane(dk);
        dv = __builtin_amdgcn_readfirstlane(dv);
    }
    float scale[NR];  // of a row's scores as they are computed
#pragma unroll
    for (int n = 0; n < NR; ++n) scale[n] = __builtin_ldexpf(a.scale, qexp[n] - dk);

    // queries as the B operands: column c of row tile n, channels 8 i + 0..7 of the lane's half
#pragma unroll
    for (int k = 0; k < QN; ++k) {
        const int n = k * kDecWaves / KC, i = k * kDecWaves % KC + wave;
        u32x4 *to = sq + (n * KC + i) * kWave + lane;
        if (TYPE != QG_TYPE_BF16 && fast) {
            u32x4 part[2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x0 = __builtin_ldexpf(elem(qraw[k], 2 * e) * a.qsign, -qexp[n]);
                const float x1 = __builtin_ldexpf(elem(qraw[k], 2 * e + 1) * a.qsign, -qexp[n]);
                const f16x2 h = __builtin_convertvector((f32x2{x0, x1}), f16x2);
                const f32x2 rest = {x0 - (float)h[0], x1 - (float)h[1]};
                part[0][e] = __builtin_bit_cast(uint32_t, h);
                part[1][e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, f16x2));
            }
#pragma unroll
            for (int p = 0; p < QF; ++p) to[p * NR * KC * kWave] = part[p];
        } else {
            bf16x8 part[QS];
            split8<QS>(qraw[k], a.qsign, part);
#pragma unroll
            for (int p = 0; p < QS; ++p) to[p * NR * KC * kWave] = __builtin_bit_cast(u32x4, part[p]);
        }
    }
    lds_barrier();  // keys and values stay in flight

    f32x16 o[NR][MT];
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int x = 0; x < 16; ++x) o[n][i][x] = 0.f;
    RunningMax most[NR];
    float l[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) l[n] = 0.f;

    auto step = [&](int j, auto more, auto is_fast) {
        constexpr bool F = is_fast.value, KF = F && TYPE != QG_TYPE_BF16;
        constexpr int QP = KF ? QF : QS, PP = F ? 2 : 3;  // parts of queries and weights
        constexpr float kShift = F ? 11.f : 0.f, kSlack = F ? 4.f : kDecSlack;
        typedef PfxOps<KF> KOps;
        typedef PfxOps<F> VOps;
        const bool cur_ok[2] = {next_ok[0], next_ok[1]};
        f32x16 s[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int x = 0; x < 16; ++x) s[n][x] = 0.f;
        int ql = lane;
        asm volatile("" : "+v"(ql));  // or the reads below move out of the loop, into registers
        const uint32_t ks = KF ? kscale + (uint32_t)(dk * 0x01010101) : kscale;
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            const float sc = scale_of(ks, i / 4);
            const uint32_t w = kraw[i];
            const u32x4 kf = {KOps::template pair<0>(w, sc), KOps::template pair<1>(w, sc), KOps::template pair<2>(w, sc),
                              KOps::template pair<3>(w, sc)};
#pragma unroll
            for (int p = 0; p < QP; ++p)
#pragma unroll
                for (int n = 0; n < NR; ++n) s[n] = KOps::mfma(kf, sq[((p * NR + n) * KC + i) * kWave + ql], s[n]);
        }
        if constexpr (more.value) {
            locate(j + kPfxStride);
            load_k();
        }
        // register 4 x + y: position j + 8 x + 4 hf + y
        const bool whole = j + kDecStep <= min(last, all_hi) && cur_ok[0] && cur_ok[1];
        if (!whole) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int x = 0; x < 16; ++x)
                    if (j + 8 * (x / 4) + 4 * hf + x % 4 >= (cur_ok[x / 8] ? min(see_hi[n], last) : 0)) s[n][x] = -INFINITY;
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            float mt = s[n][0];
#pragma unroll
            for (int x = 1; x < 16; ++x) mt = __builtin_fmaxf(mt, s[n][x]);
            mt = half_max(mt);
            if (__ballot((mt - most[n].m) * scale[n] > kSlack) | most[n].far) {
                const float keep = most[n].raise(mt, scale[n], kShift);
                if (most[n].far) {
                    const float raw = most[n].raw(scale[n]);
#pragma unroll
                    for (int x = 0; x < 16; ++x) s[n][x] -= raw;
                }
                l[n] *= keep;
#pragma unroll
                for (int i = 0; i < MT; ++i) o[n][i] *= keep;
            }
        }
        const bool all_there = j + kDecStep <= last && cur_ok[0] && cur_ok[1];
#pragma unroll
        for (int kc = 0; kc < 2; ++kc) {
            u32x4 pf[NR][PP];
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][8 * kc + 2 * e], scale[n], -most[n].muse));
                    float x1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][8 * kc + 2 * e + 1], scale[n], -most[n].muse));
                    l[n] += x0;
                    l[n] += x1;
                    if constexpr (F) {
                        const f16x2 h = __builtin_convertvector((f32x2{x0, x1}), f16x2);
                        const f32x2 rest = {__builtin_fmaf((float)h[0], -1.f, x0), __builtin_fmaf((float)h[1], -1.f, x1)};
                        pf[n][0][e] = __builtin_bit_cast(uint32_t, h);
                        pf[n][1][e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, f16x2));
                    } else {
#pragma unroll
                        for (int p = 0; p < PP; ++p) {  // eight bits at a time, cut off: no rounding
                            const uint32_t b0 = __builtin_bit_cast(uint32_t, x0), b1 = __builtin_bit_cast(uint32_t, x1);
                            pf[n][p][e] = __builtin_amdgcn_perm(b1, b0, 0x07060302u);
                            x0 -= __builtin_bit_cast(float, b0 & 0xffff0000u);
                            x1 -= __builtin_bit_cast(float, b1 & 0xffff0000u);
                        }
                    }
                }
            float vs[2][4];
            u32x4 v[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t w = vscale[kc][y], keep = ~0u;
                if (!all_there) {  // what no row sees may be anything, also its scales: 0 * NaN
                    const int left = cur_ok[kc] ? last - (j + 16 * kc + 8 * y + 4 * hf) : 0;
                    keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
                    if (F) w = (w & keep) | (~keep & (uint32_t)((140 - dv) * 0x01010101));
                }
                if (F) w += (uint32_t)(dv * 0x01010101);
                w &= keep;
#pragma unroll
                for (int t = 0; t < 4; ++t) vs[y][t] = scale_of(w, t);
                v[y] = vraw[kc][y];
                if (DH == 64) v[y] >>= (c & 3) * 8;
                if (DH == 128) v[y] >>= (c & 1) * 16;
            }
            auto values = [&](auto pair) {  // channels 2 B, 2 B + 1 of the lane's
                constexpr int B = pair.value;
                uint32_t w[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) w[x] = VOps::template pair<B>(v[x / 4][x % 4], vs[x / 4][x % 4]);
                u32x4 lo, hi;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    lo[x] = __builtin_amdgcn_perm(w[2 * x + 1], w[2 * x], 0x05040100u);
                    hi[x] = __builtin_amdgcn_perm(w[2 * x + 1], w[2 * x], 0x07060302u);
                }
#pragma unroll
                for (int p = 0; p < PP; ++p)
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        o[n][2 * B] = VOps::mfma(lo, pf[n][p], o[n][2 * B]);
                        o[n][2 * B + 1] = VOps::mfma(hi, pf[n][p], o[n][2 * B + 1]);
                    }
            };
            values(std::integral_constant<int, 0>{});
            if constexpr (MT > 2) values(std::integral_constant<int, 1>{});
            if constexpr (MT > 4) {
                values(std::integral_constant<int, 2>{});
                values(std::integral_constant<int, 3>{});
            }
        }
        if constexpr (more.value) load_v();
    };
    // The last step, which loads nothing, apart: loads behind a condition would
    // make every wait one for all of them.
    auto walk = [&](auto is_fast) {
        int j = j_first;
        for (; j + kPfxStride < last; j += kPfxStride) step(j, std::true_type{}, is_fast);
        step(j, std::false_type{}, is_fast);
    };
    if (j_first < last) {
        if (fast)
            walk(std::true_type{});
        else
            walk(std::false_type{});
    }

    // join the waves: maxima first, then the sums through LDS, a quarter of a tile's registers each
    const float shift = fast ? 11.f : 0.f, unshift = fast ? 0x1p-11f : 1.f;
    float keep[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const float exact = most[n].exact(scale[n], shift);
        l[n] = (l[n] + shfl_xor(l[n], 32)) * exact;
        keep[n] = exact;
        if (hf == 0) sml[wave][n][c] = f32x2{most[n].m, l[n]};
    }
    __syncthreads();  // and every wave is done with the queries
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kDecWaves; ++w) top = __builtin_fmaxf(top, sml[w][n][c][0]);
        const float use = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kDecWaves; ++w)
            sum += sml[w][n][c][1] * __builtin_amdgcn_exp2f((sml[w][n][c][0] - use) * scale[n]);
        keep[n] *= __builtin_amdgcn_exp2f((most[n].m - use) * scale[n]);
        const size_t at = out_row[n] * a.chunks + ci;
        if (wave == 0 && hf == 0 && live[n]) a.pml[at] = f32x2{__builtin_ldexpf(top, qexp[n] - dk), sum * unshift};
        f32x4 *part = reinterpret_cast<f32x4 *>(room);  // [wave][quarter - 1 or quarter][tile][lane]
#pragma unroll
        for (int i0 = 0; i0 < MT; i0 += JT) {
            if (n || i0) __syncthreads();
            f32x4 mine[JT];
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < JT; ++i) {
                    f32x4 v;
#pragma unroll
                    for (int y = 0; y < 4; ++y) v[y] = o[n][i0 + i][4 * x + y] * keep[n];
                    if (x == wave)
                        mine[i] = v;
                    else
                        part[((wave * 3 + (x > wave ? x - 1 : x)) * JT + i) * kWave + lane] = v;
                }
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kDecWaves; ++w)
                if (w != wave)
#pragma unroll
                    for (int i = 0; i < JT; ++i)
                        mine[i] += part[((w * 3 + (wave > w ? wave - 1 : wave)) * JT + i) * kWave + lane];
            if (live[n]) {  // register y of tile i: channel (8 wave + 4 hf + y) * MT + i
                float *dst = a.po + at * DH + (8 * wave + 4 * hf) * MT + i0;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    float v[JT];
#pragma unroll
                    for (int i = 0; i < JT; ++i) v[i] = __builtin_ldexpf(mine[i][y] * unshift, -dv);
                    if constexpr (JT == 4)
                        *(f32x4 *)(dst + y * MT) = f32x4{v[0], v[1], v[2], v[3]};
                    else
                        *(f32x2 *)(dst + y * MT) = f32x2{v[0], v[1]};
                }
            }
        }
    }
}

template <int TYPE, int DH, int NR>
static int launch_prefix_nr(const DecodeArgs &a, hipStream_t stream) {
    const long long rows = (long long)a.G * a.Tq * a.c.B, grid = (rows + 32 * NR - 1) / (32 * NR) * a.c.Hkv * a.prefix_chunks;
    if (grid > kMaxGroups) return QG_ERR_SHAPE;
    hipLaunchKernelGGL((attn_prefix_kernel<TYPE, DH, NR>), dim3((unsigned)grid), dim3(kDecWaves * kWave), 0, stream, a);
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

template <int TYPE>
static int launch_prefix(const DecodeArgs &a, int Dh, hipStream_t stream) {
    const bool few = prefix_tile_rows((long long)a.G * a.Tq * a.c.B, Dh) == 32;
    switch (Dh) {
        case 64: return few ? launch_prefix_nr<TYPE, 64, 1>(a, stream) : launch_prefix_nr<TYPE, 64, 2>(a, stream);
        case 128: return few ? launch_prefix_nr<TYPE, 128, 1>(a, stream) : launch_prefix_nr<TYPE, 128, 2>(a, stream);
        default: return launch_prefix_nr<TYPE, 256, 1>(a, stream);
    }
}

// Chunks that fill the card once, two workgroups a compute unit.
PrefixSplit prefix_split(long long rows, int Hkv, int Dh, int prefix) {
    const int tile = prefix_tile_rows(rows, Dh);
    const long long groups = (rows + tile - 1) / tile * Hkv;
    long long chunks = groups < 512 ? 512 / groups : 1;
    long long each = (prefix + chunks - 1) / chunks;
    each = (each + kPfxStride - 1) / kPfxStride * kPfxStride;
    if (each > kDecChunkMax) each = kDecChunkMax;
    return PrefixSplit{(int)each, (int)((prefix + each - 1) / each)};
}

int launch_attn_prefix(int type, int Dh, const DecodeArgs &a, hipStream_t stream) {
    switch (type) {
        case QG_TYPE_F32: return launch_prefix<QG_TYPE_F32>(a, Dh, stream);
        case QG_TYPE_F16: return launch_prefix<QG_TYPE_F16>(a, Dh, stream);
        default: return launch_prefix<QG_TYPE_BF16>(a, Dh, stream);
    }
}

}  // namespace qg
