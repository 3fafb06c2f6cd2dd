// Attention of new tokens over the paged FP4 cache.
//
// One pass over the cache with the running maximum and sum of a softmax, its
// keys split into chunks that workgroups take independently and a second
// launch joins.  A wave takes 32 positions at a time for 16 query rows (the
// query heads and tokens that share a key/value head) on the matrix cores:
//   S^T = K Q^T    (positions x rows),  O^T += V^T P^T   (channels x rows).
// With both products transposed a lane keeps one query row throughout: the
// scores it receives are the weights it has to supply (two 16-position tiles
// fill the 32-deep product; only the order of the positions differs, and V is
// paired to match), and the running maximum, sum and rescaling need no
// exchange with other rows.
// Operands are bf16: every E2M1 value times a power of two is exact there (the
// hardware conversion takes the UE8M0 scale along), fp32 queries go in as
// three bf16 parts (24 bits, exact) and fp16 ones as two, weights as two parts
// (16 bits).  Products and sums are fp32.
#include "common.h"
#include "kv4_device.h"

namespace qg {

constexpr int kDecWaves = 4;
constexpr int kDecStep = 32;                      // positions a wave takes at a time
constexpr int kDecChunkMin = 256, kDecChunkMax = 4096;  // positions a workgroup takes
constexpr int kDecMaxPages = kDecChunkMax / 16 + 1;
constexpr float kDecSlack = 8.f;                  // a weight may reach 2^8 before the sums are rescaled

// Positions per workgroup of a sequence of which n are visible: about
// 8 sqrt(n), so that short sequences still spread over the card and long ones
// do not spend their time joining.  A function of the sequence alone: its
// result is the same in any batch.
__host__ __device__ inline int dec_chunk(int n) {
    int c = kDecChunkMin;
    while (c < kDecChunkMax && n >= c / 16 * c) c *= 2;
    return c;
}
__host__ __device__ inline int dec_chunks(int n) { return (n + dec_chunk(n) - 1) / dec_chunk(n); }

// Most chunks of any n up to `most`: at `most` or just before a chunk grows.
inline int dec_chunks_max(int most) {
    int best = dec_chunks(most);
    for (int c = kDecChunkMin; c < kDecChunkMax; c *= 2)
        if (c / 16 * c - 1 <= most && dec_chunks(c / 16 * c - 1) > best) best = dec_chunks(c / 16 * c - 1);
    return best < 1 ? 1 : best;
}

struct DecodeArgs {
    Kv4Cache c;
    const void *q;
    float *y;
    float *po;   // [B, H * Tq, chunks, Dh] partial sums
    f32x2 *pml;  // [B, H * Tq, chunks] maximum (base 2) and sum
    int ldq, Tq, H, G, window, max_len, chunks;
    float scale_log2;
};

// The visible positions of sequence b's queries are inside [begin, len), begin
// a multiple of 16; returns their count (0: nothing, or a length out of range).
__device__ __forceinline__ int dec_range(const DecodeArgs &a, int b, int *len, int *begin) {
    const int n = load_uniform(a.c.lens + b);
    *len = n;
    *begin = 0;
    if (n < 0 || n > a.max_len) return -1;
    if (a.window && n - a.Tq - a.window + 1 > 0) *begin = (n - a.Tq - a.window + 1) & ~15;
    return n - *begin;
}

// 8 elements of q as PARTS bf16 vectors whose sum they are.
template <int PARTS, class T>
__device__ __forceinline__ void split8(const T *p, bf16x8 (&out)[PARTS]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float x = (float)p[i];
#pragma unroll
        for (int s = 0; s < PARTS; ++s) {
            const bf16_t h = (bf16_t)x;
            out[s][i] = h;
            x -= (float)h;
        }
    }
}

// A lane's part of one 16-position tile.
template <int DH>
struct DecTile {
    static constexpr int KW = DH / 32, VC = DH / 128 < 1 ? 1 : DH / 128;  // dwords of a key, 16-byte pieces of values
    uint32_t k[KW];
    u32x4 v[VC];
    uint32_t ks;      // scale bytes of the lane's channels (DH / 4 of them)
    uint32_t vs[VC];  // scale bytes of four positions
};

template <int DH>
__device__ __forceinline__ void dec_load(DecTile<DH> &t, const uint8_t *r, int page, int off, int lane) {
    const int c = lane & 15, g = lane >> 4;
    const uint8_t *kp = r + (size_t)(off + c) * (DH / 2) + g * (DH / 8);
#pragma unroll
    for (int i = 0; i < DH / 32; i += (DH == 64 ? 2 : 4)) {
        if constexpr (DH == 64) {
            const u32x2 w = *as_global<u32x2>(kp);
            t.k[0] = w[0], t.k[1] = w[1];
        } else {
            const u32x4 w = *as_global<u32x4>(kp + i * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) t.k[i + j] = w[j];
        }
    }
    const uint8_t *ksp = r + (size_t)page * DH + (size_t)(off + c) * (DH / 32);
    if constexpr (DH == 64) t.ks = *as_global<uint8_t>(ksp + (g >> 1));
    if constexpr (DH == 128) t.ks = *as_global<uint8_t>(ksp + g);
    if constexpr (DH == 256) t.ks = *as_global<uint16_t>(ksp + 2 * g);
#pragma unroll
    for (int x = 0; x < DecTile<DH>::VC; ++x) {
        const int chunk = DH == 64 ? c >> 1 : c + 16 * x;
        t.v[x] = *as_global<u32x4>(r + (size_t)page * (DH / 2) + ((size_t)((off >> 2) + g) * (DH / 8) + chunk) * 16);
        t.vs[x] = *as_global<uint32_t>(r + (size_t)page * (DH + DH / 32) +
                                       (((off >> 2) + g) * (DH / 32) + (chunk >> 2)) * 4);
    }
}

__device__ __forceinline__ float scale_of(uint32_t bytes, int i) {
    return __builtin_bit_cast(float, (bytes >> (8 * i) & 0xffu) << 23);
}

template <int B>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, B));
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

template <int TYPE>
constexpr int kQParts = TYPE == QG_TYPE_F32 ? 3 : TYPE == QG_TYPE_F16 ? 2 : 1;

template <int TYPE, int DH>
__global__ __launch_bounds__(kDecWaves *kWave, 2) void attn_decode_kernel(DecodeArgs a) {
    typedef typename ElemOf<TYPE>::type T;
    constexpr int QP = kQParts<TYPE>, KC = DH / 32, MT = DH / 16;  // parts of q, key products, channel tiles
    // 256 channels: the queries' parts (up to 96 registers) stay in LDS, in the room that the join uses at the end
    constexpr bool QLDS = DH == 256;
    __shared__ __attribute__((aligned(16))) float so[2][16 * DH];
    u32x4 *sq = reinterpret_cast<u32x4 *>(&so[0][0]);
    static_assert(!QLDS || sizeof(so) >= sizeof(u32x4) * QP * KC * kWave, "queries fit the join's room");
    __shared__ f32x2 sml[kDecWaves][16];
    __shared__ int spage[kDecMaxPages];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int hk = blockIdx.x % a.c.Hkv, ci = blockIdx.x / a.c.Hkv, b = blockIdx.z, row0 = blockIdx.y * 16;
    const int R = a.G * a.Tq;
    int len, begin;
    int n = dec_range(a, b, &len, &begin);
    if (n < 0 && ci == 0 && threadIdx.x == 0) kv4_report(a.c.status, QG_DEV_BAD_LENGTH);
    const int nchunks = n > 0 ? dec_chunks(n) : 0;
    if (ci > 0 && ci >= nchunks) return;

    const int c = lane & 15, g = lane >> 4;
    const int row = row0 + c;
    const bool live = row < R;
    const int t = live ? row / a.G : 0, h = hk * a.G + (live ? row - t * a.G : 0);
    const size_t out_row = (size_t)(b * a.Tq + t) * a.H + h;
    if (nchunks == 0) {
        if (live && wave == 0)
            for (int i = g * 4; i < DH; i += 16) *(f32x4 *)(a.y + out_row * DH + i) = f32x4{0.f, 0.f, 0.f, 0.f};
        return;
    }
    const int chunk = dec_chunk(n);
    const int first = begin + ci * chunk, last = min(len, first + chunk);  // this workgroup's positions
    const int page = 1 << a.c.page_log2, pg0 = first >> a.c.page_log2;
    for (int i = threadIdx.x; i <= ((last - 1) >> a.c.page_log2) - pg0; i += kDecWaves * kWave)
        spage[i] = kv4_page_of(a.c, b, pg0 + i);

    // queries as the B operand: row c, channels g * DH/4 + 8 i + 0..7 for product i
    u32x4 qf[QP][QLDS ? 1 : KC];
    {
        const T *qp = (const T *)a.q + (size_t)(b * a.Tq + t) * a.ldq + (size_t)h * DH + g * (DH / 4);
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            if (QLDS && i % kDecWaves != wave) continue;
            bf16x8 parts[QP];
            split8<QP>(qp + 8 * i, parts);
#pragma unroll
            for (int s = 0; s < QP; ++s) {
                if (QLDS)
                    sq[(s * KC + i) * kWave + lane] = __builtin_bit_cast(u32x4, parts[s]);
                else
                    qf[s][i] = __builtin_bit_cast(u32x4, parts[s]);
            }
        }
    }
    const int pos = len - a.Tq + t;                       // this row's position
    const int see_hi = live ? pos + 1 : 0, see_lo = a.window ? pos - a.window + 1 : 0;
    __syncthreads();

    f32x4 o[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, muse = 0.f, l = 0.f;
    const size_t region = kv4_region_bytes(page, DH);

    // Loads of a step's two tiles; a tile behind the end or on a bad page
    // reads the step's (or chunk's) first place instead and is masked.
    auto load = [&](int j, DecTile<DH> (&tile)[2], bool (&ok)[2]) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int j0 = j + 16 * x;
            const int at = j0 < last ? j0 : first;
            const int id = __builtin_amdgcn_readfirstlane(spage[(at >> a.c.page_log2) - pg0]);
            ok[x] = j0 < last && id >= 0;
            dec_load<DH>(tile[x], a.c.kv + ((size_t)max(id, 0) * a.c.Hkv + hk) * region, page, at & (page - 1), lane);
        }
    };
    DecTile<DH> cur[2];
    bool cur_ok[2];
    const int j_first = first + wave * kDecStep;
    if (j_first < last) load(j_first, cur, cur_ok);
    for (int j = j_first; j < last; j += kDecWaves * kDecStep) {
        DecTile<DH> next[2];
        bool next_ok[2] = {false, false};
        const bool more = j + kDecWaves * kDecStep < last;
        if (more) load(j + kDecWaves * kDecStep, next, next_ok);

        f32x4 s[2];
        int ql = lane;
        if (QLDS) asm volatile("" : "+v"(ql));  // or the reads below move out of the loop, into registers
#pragma unroll
        for (int x = 0; x < 2; ++x) s[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            u32x4 qi[QP];
#pragma unroll
            for (int p = 0; p < QP; ++p) qi[p] = QLDS ? sq[(p * KC + i) * kWave + ql] : qf[p][QLDS ? 0 : i];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float sc = scale_of(cur[x].ks, DH == 256 ? i / 4 : 0);
                const uint32_t w = cur[x].k[i];
                const u32x4 kf = {fp4_pair<0>(w, sc), fp4_pair<1>(w, sc), fp4_pair<2>(w, sc), fp4_pair<3>(w, sc)};
#pragma unroll
                for (int p = 0; p < QP; ++p) s[x] = mfma16(kf, qi[p], s[x]);
            }
        }
        // base-2 scores; what a row does not see is -inf
        float sv[8];
        const bool whole = j + kDecStep <= min(last, len - a.Tq + 1) && cur_ok[0] && cur_ok[1] && !a.window;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int jj = j + 16 * x + 4 * g + i;
                const float v = s[x][i] * a.scale_log2;
                sv[4 * x + i] = whole || (cur_ok[x] && jj < min(see_hi, last) && jj >= see_lo) ? v : -INFINITY;
            }
        float mt = sv[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mt = __builtin_fmaxf(mt, sv[i]);
        mt = row_max(mt);
        if (__ballot(mt > m + kDecSlack)) {
            const float mn = __builtin_fmaxf(m, mt);
            const float use = mn == -INFINITY ? 0.f : mn;
            const float keep = __builtin_amdgcn_exp2f(m - use);
            m = mn;
            muse = use;
            l *= keep;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i] *= keep;
        }
        u32x4 pf[2];
        {
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = __builtin_amdgcn_exp2f(sv[i] - muse);
                l += p[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bf16x2 hi = {(bf16_t)p[2 * i], (bf16_t)p[2 * i + 1]};
                const bf16x2 lo = {(bf16_t)(p[2 * i] - (float)hi[0]), (bf16_t)(p[2 * i + 1] - (float)hi[1])};
                pf[0][i] = __builtin_bit_cast(uint32_t, hi);
                pf[1][i] = __builtin_bit_cast(uint32_t, lo);
            }
        }
        if (!(j + kDecStep <= last && cur_ok[0] && cur_ok[1])) {  // scales behind the end may be anything: 0 * NaN
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int left = cur_ok[x] ? last - (j + 16 * x + 4 * g) : 0;
                const uint32_t keep = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
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
#define QG_PAIR(B)                                                   \
    dec_values<B>(v0, v1, s0, s1, &lo, &hi);                         \
    o[8 * y + 2 * B] = mfma16(lo, pf[0], o[8 * y + 2 * B]);          \
    o[8 * y + 2 * B] = mfma16(lo, pf[1], o[8 * y + 2 * B]);          \
    o[8 * y + 2 * B + 1] = mfma16(hi, pf[0], o[8 * y + 2 * B + 1]);  \
    o[8 * y + 2 * B + 1] = mfma16(hi, pf[1], o[8 * y + 2 * B + 1]);
            QG_PAIR(0)
            QG_PAIR(1)
            if constexpr (DH > 64) {
                QG_PAIR(2)
                QG_PAIR(3)
            }
#undef QG_PAIR
        }
        if (more) {
#pragma unroll
            for (int x = 0; x < 2; ++x) cur[x] = next[x], cur_ok[x] = next_ok[x];
        }
    }

    // join the waves: maxima first, then sums pairwise through LDS
    l = row_sum(l);
    if (g == 0) sml[wave][c] = f32x2{m, l};
    __syncthreads();  // and every wave is done with the queries
    float mall = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDecWaves; ++w) mall = __builtin_fmaxf(mall, sml[w][c][0]);
    const float use = mall == -INFINITY ? 0.f : mall;
    float lall = 0.f;
#pragma unroll
    for (int w = 0; w < kDecWaves; ++w) lall += sml[w][c][1] * __builtin_amdgcn_exp2f(sml[w][c][0] - use);
    const float keep = __builtin_amdgcn_exp2f(m - use);
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i] *= keep;
#pragma unroll
    for (int half = kDecWaves / 2; half; half /= 2) {
        if (wave >= half && wave < 2 * half)
#pragma unroll
            for (int i = 0; i < MT; ++i) *(f32x4 *)&so[wave - half][(i * kWave + lane) * 4] = o[i];
        __syncthreads();
        if (wave < half)
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i] += *(const f32x4 *)&so[wave][(i * kWave + lane) * 4];
        __syncthreads();
    }
    if (wave != 0 || !live) return;
    // o[8 y + i][k]: channel ((16 y + 4 g + k) * 8 + i), or (4 g + k) * 4 + i for 64 channels
    constexpr int PER = DH == 64 ? 4 : 8;
    float *dst = a.y + out_row * DH;
    float f = lall > 0.f ? 1.f / lall : 0.f;
    if (nchunks > 1) {
        const size_t at = ((size_t)b * a.H * a.Tq + (size_t)t * a.H + h) * a.chunks + ci;
        dst = a.po + at * DH;
        f = 1.f;
        if (g == 0) a.pml[at] = f32x2{mall, lall};
    }
#pragma unroll
    for (int y = 0; y < DecTile<DH>::VC; ++y)
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < PER; i += 4)
                *(f32x4 *)(dst + (16 * y + 4 * g + k) * PER + i) =
                    f32x4{o[8 * y + i][k], o[8 * y + i + 1][k], o[8 * y + i + 2][k], o[8 * y + i + 3][k]} * f;
}

// Joins the chunks of sequences that have several: one wave per query row.
template <int DH>
__global__ __launch_bounds__(256) void attn_decode_join_kernel(DecodeArgs a) {
    const int rows = a.H * a.Tq, b = blockIdx.y, lane = lane_id();
    const int row = blockIdx.x * 4 + threadIdx.x / kWave;
    int len, begin;
    const int n = dec_range(a, b, &len, &begin);
    const int nchunks = n > 0 ? dec_chunks(n) : 0;
    if (nchunks < 2 || row >= rows) return;
    const size_t at = ((size_t)b * rows + row) * a.chunks;
    float top = -INFINITY;
    for (int i = lane; i < nchunks; i += kWave) top = __builtin_fmaxf(top, a.pml[at + i][0]);
    for (int x = 32; x; x >>= 1) top = __builtin_fmaxf(top, shfl_xor(top, x));
    const float use = top == -INFINITY ? 0.f : top;
    float l = 0.f, acc[DH / 64] = {};
    for (int i = 0; i < nchunks; ++i) {
        const f32x2 ml = a.pml[at + i];
        const float w = __builtin_amdgcn_exp2f(ml[0] - use);
        l += ml[1] * w;
        const float *o = a.po + (at + i) * DH + lane * (DH / 64);
#pragma unroll
        for (int x = 0; x < DH / 64; ++x) acc[x] += o[x] * w;
    }
    float *y = a.y + ((size_t)b * rows + row) * DH + lane * (DH / 64);
#pragma unroll
    for (int x = 0; x < DH / 64; ++x) y[x] = l > 0.f ? acc[x] / l : 0.f;
}

template <int TYPE, int DH>
static int launch_decode_dh(const DecodeArgs &a, hipStream_t stream) {
    const dim3 grid(a.c.Hkv * a.chunks, (a.G * a.Tq + 15) / 16, a.c.B);
    hipLaunchKernelGGL((attn_decode_kernel<TYPE, DH>), grid, dim3(kDecWaves * kWave), 0, stream, a);
    if (hipGetLastError() != hipSuccess) return QG_ERR_LAUNCH;
    if (a.chunks == 1) return QG_OK;
    hipLaunchKernelGGL(attn_decode_join_kernel<DH>, dim3((a.H * a.Tq + 3) / 4, a.c.B), dim3(256), 0, stream, a);
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

template <int TYPE>
static int launch_decode(const DecodeArgs &a, int Dh, hipStream_t stream) {
    switch (Dh) {
        case 64: return launch_decode_dh<TYPE, 64>(a, stream);
        case 128: return launch_decode_dh<TYPE, 128>(a, stream);
        default: return launch_decode_dh<TYPE, 256>(a, stream);
    }
}

// The workspace: partial sums, then maxima and sums, of every row and chunk.
static int decode_chunks(int Tq, int max_len, int window) {
    long long most = max_len;
    if (window && (long long)window + Tq - 1 + 15 < most) most = (long long)window + Tq - 1 + 15;
    return dec_chunks_max((int)most);
}
static size_t decode_sums_bytes(int B, int Tq, int H, int Dh, int chunks) {
    return (size_t)B * Tq * H * chunks * Dh * sizeof(float);
}

static bool decode_shape_ok(int B, int Tq, int H, int Hkv, int Dh, int max_len, int window) {
    return B >= 1 && B <= QG_MAX_SEQS && Tq >= 1 && Tq <= QG_MAX_DECODE_TOKENS && H >= 1 && H <= QG_MAX_HEADS &&
           Hkv >= 1 && H % Hkv == 0 && (Dh == 64 || Dh == 128 || Dh == 256) && max_len >= 1 &&
           max_len <= 0x3fffffff && window >= 0;
}

}  // namespace qg

extern "C" size_t attn_decode_workspace_bytes(int B, int Tq, int H, int Hkv, int Dh, int max_len, int window) {
    if (!qg::decode_shape_ok(B, Tq, H, Hkv, Dh, max_len, window)) return 0;
    const int chunks = qg::decode_chunks(Tq, max_len, window);
    if (chunks == 1) return 256;
    return qg::decode_sums_bytes(B, Tq, H, Dh, chunks) + (size_t)B * Tq * H * chunks * 2 * sizeof(float);
}

extern "C" int attn_decode_kv4(int type, const void *q, int ldq, const int32_t *lens, int B, int Tq, int H, int Hkv,
                               int Dh, float scale, int window, int max_len, const int32_t *pages, int max_pages,
                               int page, int num_pages, const void *kv, float *y, void *ws, size_t ws_bytes,
                               int32_t *d_status, void *stream) {
    using namespace qg;
    if (type != QG_TYPE_F32 && type != QG_TYPE_F16 && type != QG_TYPE_BF16) return QG_ERR_FORMAT;
    if (!q || !lens || !pages || !kv || !y || !ws || !d_status) return QG_ERR_NULL;
    if (!decode_shape_ok(B, Tq, H, Hkv, Dh, max_len, window)) return QG_ERR_SHAPE;
    if (!kv4_cache_shape_ok(B, Hkv, Dh, max_pages, page, num_pages) || max_len > (long long)max_pages * page)
        return QG_ERR_SHAPE;
    if (!row_stride_ok(type, ldq, H * Dh) || !__builtin_isfinite(2.f * scale)) return QG_ERR_SHAPE;
    if (((uintptr_t)q | (uintptr_t)kv | (uintptr_t)y | (uintptr_t)ws) & 15) return QG_ERR_ALIGN;
    if (((uintptr_t)lens | (uintptr_t)pages | (uintptr_t)d_status) & 3) return QG_ERR_ALIGN;
    if (ws_bytes < attn_decode_workspace_bytes(B, Tq, H, Hkv, Dh, max_len, window)) return QG_ERR_WORKSPACE;
    DecodeArgs a{};
    a.c.kv = (uint8_t *)const_cast<void *>(kv);
    a.c.pages = pages;
    a.c.lens = lens;
    a.c.max_pages = max_pages;
    a.c.num_pages = num_pages;
    a.c.page_log2 = __builtin_ctz((unsigned)page);
    a.c.B = B;
    a.c.Hkv = Hkv;
    a.c.status = d_status;
    a.q = q;
    a.y = y;
    a.ldq = ldq;
    a.Tq = Tq;
    a.H = H;
    a.G = H / Hkv;
    a.window = window;
    a.max_len = max_len;
    a.scale_log2 = scale * 1.44269504088896340736f;
    a.chunks = decode_chunks(Tq, max_len, window);
    a.po = (float *)ws;
    a.pml = (f32x2 *)((uint8_t *)ws + (a.chunks == 1 ? 0 : decode_sums_bytes(B, Tq, H, Dh, a.chunks)));
    if ((long long)Hkv * a.chunks > 0x7fffffffLL) return QG_ERR_SHAPE;
    clear_stale_error();
    switch (type) {
        case QG_TYPE_F32: return launch_decode<QG_TYPE_F32>(a, Dh, (hipStream_t)stream);
        case QG_TYPE_F16: return launch_decode<QG_TYPE_F16>(a, Dh, (hipStream_t)stream);
        default: return launch_decode<QG_TYPE_BF16>(a, Dh, (hipStream_t)stream);
    }
}
