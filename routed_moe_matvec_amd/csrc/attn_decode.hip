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
// three bf16 parts (24 bits, exact) and fp16 ones as two, weights as three: with
// two, they alone put the result off by 2e-6 to 1.5e-5 of its norm, with three by
// 1e-8, and fp32's own roundings by 2e-7 to 1.3e-6 up to 40000 positions.
// Products and sums are fp32.  The running maximum is one of q . k, not
// scaled, and is taken off the scores themselves where it is large (RunningMax; 0
// to 3% of the time).
//
// The same walk serves windows with first positions that stay visible (SINKS) and short
// shared prefixes (FUSED): places are counted over two ranges of positions, each from a
// multiple of 16, and a tile lies in one of them.  32 sequences of up to 20000 positions with a window
// of 1024 and 4 sinks, 32 heads of 128: 10.9 us, 35 MB; 24 of up to 60000 with a window of
// 8192 and 100 sinks, 3 tokens, 16 heads of 64: 55 to 60 us, 196 MB, bound by vector
// instructions (75% of the cycles, without the issue of matrix instructions).  Of a step's about 80 are the softmax and the
// weights' parts, on 16 columns of which 3 are rows (its 8 exponentials take four times as long as others), and about 65
// the conversion and pairing of keys and values.
#include <type_traits>

#include "attn_decode_device.h"

namespace qg {

template <int TYPE, int DH, int SLOTS, int MODE, int WAVES>
__global__ __launch_bounds__(WAVES *kWave, DH == 256 ? 3 : 4) void attn_decode_kernel(DecodeArgs a) {
    __shared__ DecShared<DH, WAVES> sh;
    attn_decode_group<TYPE, DH, SLOTS, MODE, WAVES>(a, sh, blockIdx.x, blockIdx.y);
}

// Joins the chunks of sequences that have several: one workgroup per query
// row, Dh / 4 lanes a chunk, so that 8 to 16 chunks are read at once (one wave
// per row with a chunk at a time took 20 us for 64 rows of 64 chunks).
template <int DH, int MODE>
__global__ __launch_bounds__(256) void attn_decode_join_kernel(DecodeArgs a) {
    constexpr int LN = DH / 4, NG = 256 / LN;
    __shared__ __attribute__((aligned(16))) f32x4 so[256];
    __shared__ float sl[NG];
    const int rows = a.H * a.Tq, b = blockIdx.y, row = blockIdx.x, tid = threadIdx.x, lane = lane_id();
    const int n = dec_range<MODE>(a, b).n, grp = tid / LN, ch = tid % LN;
    int nchunks = n > 0 ? a.split.chunks(n) : 0;
    if (MODE == TAIL) {
        if (n >= 0) nchunks += a.prefix_chunks;
        if (n < 0 && grp == 0) *(f32x4 *)(a.y + ((size_t)b * rows + row) * DH + ch * 4) = f32x4{0.f, 0.f, 0.f, 0.f};
        if (n < 0) {
            if (row == 0 && tid == 0) kv4_report(a.c.status, QG_DEV_BAD_LENGTH);
            return;
        }
    } else if (nchunks < 2) {
        return;
    }
    const size_t at = ((size_t)b * rows + row) * a.chunks;
    // the first pieces are requested before the maximum is known
    constexpr int PRE = 4;
    const float *po = a.po + at * DH + ch * 4;
    f32x4 pre[PRE];
#pragma unroll
    for (int x = 0; x < PRE; ++x) pre[x] = *(const f32x4 *)(po + (size_t)min(grp + x * NG, nchunks - 1) * DH);
    float top = -INFINITY;
    for (int i = lane; i < nchunks; i += kWave) top = __builtin_fmaxf(top, a.pml[at + i][0]);
#pragma unroll
    for (int x = 32; x; x >>= 1) top = __builtin_fmaxf(top, shfl_xor(top, x));
    const float use = top == -INFINITY ? 0.f : top;
    float l = 0.f;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](int i, f32x4 o) {
        const f32x2 ml = a.pml[at + i];
        const float w = __builtin_amdgcn_exp2f((ml[0] - use) * a.scale);
        l += ml[1] * w;
        acc += o * w;
    };
#pragma unroll
    for (int x = 0; x < PRE; ++x)
        if (grp + x * NG < nchunks) add(grp + x * NG, pre[x]);
#pragma unroll 4
    for (int i = grp + PRE * NG; i < nchunks; i += NG) add(i, *(const f32x4 *)(po + (size_t)i * DH));
    so[tid] = acc;
    if (ch == 0) sl[grp] = l;
    __syncthreads();
    if (tid >= LN) return;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i) l += sl[i];
#pragma unroll
    for (int i = 1; i < NG; ++i) acc += so[i * LN + ch];
    *(f32x4 *)(a.y + ((size_t)b * rows + row) * DH + ch * 4) = acc * (l > 0.f ? 1.f / l : 0.f);
}

template <int TYPE, int DH, int MODE, int WAVES = kDecWaves>
static int launch_decode_mode(const DecodeArgs &a, hipStream_t stream) {
    constexpr int SLOTS = kQParts<TYPE> == 3 ? 2 : 1;
    const int rows = a.G * a.Tq;
    const dim3 grid((unsigned)((long long)a.c.Hkv * a.c.B * a.chunks), (rows + 15) / 16), block(WAVES * kWave);
    if (rows <= 16 / SLOTS)
        hipLaunchKernelGGL((attn_decode_kernel<TYPE, DH, SLOTS, MODE, WAVES>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((attn_decode_kernel<TYPE, DH, 1, MODE, WAVES>), grid, block, 0, stream, a);
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

// One chunk a sequence, of eight waves.  A launch holds fewer than 2^32 threads, so half of the workgroups that a
// call may need: the sequences then go in two launches.
template <int TYPE, int DH>
static int launch_decode_wide(const DecodeArgs &a, hipStream_t stream) {
    const int B = a.c.B, each = (int)(kMaxGroups / 2 / ((long long)a.c.Hkv * ((a.G * a.Tq + 15) / 16)));
    for (int b = 0; b < B; b += each) {
        DecodeArgs part = a;
        const size_t rows = (size_t)b * a.Tq;
        part.c.B = B - b < each ? B - b : each;
        part.c.lens += b;
        part.c.pages += (size_t)b * a.c.max_pages;
        part.q = (const uint8_t *)a.q + rows * a.ldq * elem_bytes(TYPE);
        part.y += rows * a.H * DH;
        const int rc = launch_decode_mode<TYPE, DH, SINKS, 8>(part, stream);
        if (rc != QG_OK) return rc;
    }
    return QG_OK;
}

template <int DH, int MODE>
static int launch_join(const DecodeArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL((attn_decode_join_kernel<DH, MODE>), dim3(a.H * a.Tq, a.c.B), dim3(256), 0, stream, a);
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

template <int TYPE, int DH>
static int launch_decode_dh(const DecodeArgs &a, hipStream_t stream) {
    if (a.prefix_chunks) {
        const int rc = launch_attn_prefix(TYPE, DH, a, stream);
        return rc == QG_OK ? launch_join<DH, TAIL>(a, stream) : rc;
    }
    int rc;
    if constexpr (DH <= 128)
        if (a.wide) return launch_decode_wide<TYPE, DH>(a, stream);
    if (a.prefix)
        rc = launch_decode_mode<TYPE, DH, FUSED>(a, stream);
    else
        rc = a.sinks ? launch_decode_mode<TYPE, DH, SINKS>(a, stream) : launch_decode_mode<TYPE, DH, PLAIN>(a, stream);
    if (rc != QG_OK || a.chunks == 1) return rc;
    if (a.prefix) return launch_join<DH, FUSED>(a, stream);
    return a.sinks ? launch_join<DH, SINKS>(a, stream) : launch_join<DH, PLAIN>(a, stream);
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
struct DecodeChunks {
    PrefixSplit prefix;  // no chunks: each sequence walks it by itself
    DecSplit own;
    bool wide;  // one chunk, of eight waves
    int all;    // chunks of the prefix and a sequence
};
// With sinks and up to 1280 positions of 128 channels a sequence is one chunk, which eight waves
// share: no join.  us with that, and with chunks of four waves: 1024 positions and 4 sinks of 1, 16, 32,
// 64 sequences with 8 key heads 9.9, 10.4, 11.5, 18.5 and 8.8, 11.6, 16.7, 26; 2048 15, 16, 17.5,
// 29 and 10.5, 14.6, 21.9, 35; 500 7.8, 7.9, 8.3, 12.3 and 8.7, 8.8, 9.1, 12.2.  A rule of the call's
// window and sinks: a sequence's result does not depend on max_len.  A walk over a short shared prefix knows no other
// bound than that, and so takes four waves at any length (us with four, and with eight in one chunk: 4 sequences of 301
// to 431 positions 8.6, 7.9, of 1100 9.3, 10.5, 16 of 1100 12.1, 11.0, 64 channels: 4 of 2000 10.3, 13.0, 16 of 1300
// 15.2, 10.0).
static DecodeChunks decode_chunks(int B, int Tq, int G, int Hkv, int Dh, int max_len, int window, int sinks, int prefix) {
    DecodeChunks n{{0, 0, 0}, dec_split(G * Tq, Dh), false, 0};
    long long most = max_len, held = 1LL << 40;
    if (prefix) n.prefix = prefix_split(B, (long long)B * Tq * G, Hkv, Dh, prefix);
    if (n.prefix.chunks) {
        n.own.least = 11 + 7 - n.own.dh_log2;
        most = max_len > prefix ? max_len - (prefix & ~15) : 0;
    } else if (prefix) {
        most = max_len + 16LL;
    } else if (window) {
        held = (long long)window + Tq - 1 + 15 + (sinks + 15LL) / 16 * 16;
        if (held < most) most = held;
    }
    if (sinks && held * Dh <= 1280 * 128 && Dh <= 128) {
        n.wide = true;
        n.own.least = 13;
    }
    n.all = n.prefix.chunks + (most ? n.own.chunks_max((int)most) : 0);
    return n;
}
static size_t decode_sums_bytes(int B, int Tq, int H, int Dh, int chunks) {
    return (size_t)B * Tq * H * chunks * Dh * sizeof(float);
}

static bool decode_shape_ok(int B, int Tq, int H, int Hkv, int Dh, int max_len, int window, int sinks, int prefix) {
    return B >= 1 && B <= QG_MAX_SEQS && Tq >= 1 && Tq <= QG_MAX_DECODE_TOKENS && H >= 1 && H <= QG_MAX_HEADS &&
           Hkv >= 1 && H % Hkv == 0 && (Dh == 64 || Dh == 128 || Dh == 256) && max_len >= 1 &&
           max_len <= 0x3fffffff && window >= 0 && sinks >= 0 && prefix >= 0 && prefix <= max_len;
}

static size_t decode_workspace_bytes(int B, int Tq, int H, int Hkv, int Dh, int max_len, int window, int sinks,
                                     int prefix) {
    if (!decode_shape_ok(B, Tq, H, Hkv, Dh, max_len, window, sinks, prefix)) return 0;
    const DecodeChunks chunks = decode_chunks(B, Tq, H / Hkv, Hkv, Dh, max_len, window, sinks, prefix);
    if (chunks.all == 1 && !chunks.prefix.chunks) return 256;
    return decode_sums_bytes(B, Tq, H, Dh, chunks.all) + (size_t)B * Tq * H * chunks.all * 2 * sizeof(float);
}

static int decode(int type, const void *q, int ldq, const int32_t *lens, int B, int Tq, int H, int Hkv, int Dh,
                  float scale, int window, int sinks, int max_len, int prefix, const int32_t *prefix_pages,
                  const int32_t *pages, int max_pages, int page, int num_pages, const void *kv, float *y, void *ws,
                  size_t ws_bytes, int32_t *d_status, void *stream) {
    if (type != QG_TYPE_F32 && type != QG_TYPE_F16 && type != QG_TYPE_BF16) return QG_ERR_FORMAT;
    if (!q || !lens || !pages || !kv || !y || !ws || !d_status) return QG_ERR_NULL;
    if (!decode_shape_ok(B, Tq, H, Hkv, Dh, max_len, window, sinks, prefix)) return QG_ERR_SHAPE;
    if (!kv4_cache_shape_ok(B, Hkv, Dh, max_pages, page, num_pages) || max_len > (long long)max_pages * page)
        return QG_ERR_SHAPE;
    if (prefix && !prefix_pages) return QG_ERR_NULL;
    if (!row_stride_ok(type, ldq, H * Dh) || !__builtin_isfinite(2.f * scale)) return QG_ERR_SHAPE;
    if (((uintptr_t)q | (uintptr_t)kv | (uintptr_t)y | (uintptr_t)ws) & 15) return QG_ERR_ALIGN;
    if (((uintptr_t)lens | (uintptr_t)pages | (uintptr_t)prefix_pages | (uintptr_t)d_status) & 3) return QG_ERR_ALIGN;
    if (ws_bytes < decode_workspace_bytes(B, Tq, H, Hkv, Dh, max_len, window, sinks, prefix)) return QG_ERR_WORKSPACE;
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
    // a window that reaches, with the sinks, over a whole sequence hides nothing
    a.window = (long long)window + sinks < max_len ? window : 0;
    a.sinks = a.window ? sinks : 0;
    a.max_len = max_len;
    a.prefix = prefix;
    a.prefix_pages = prefix_pages;
    a.scale = scale == 0.f ? 1.f : __builtin_fabsf(scale) * 1.44269504088896340736f;
    a.qsign = scale > 0.f ? 1.f : scale < 0.f ? -1.f : 0.f;
    const DecodeChunks n = decode_chunks(B, Tq, a.G, Hkv, Dh, max_len, window, sinks, prefix);
    a.chunks = n.all;
    a.wide = n.wide;
    a.prefix_chunks = n.prefix.chunks;
    a.prefix_each = n.prefix.each;
    a.prefix_rows = n.prefix.rows;
    a.split = n.own;
    a.po = (float *)ws;
    a.pml = (f32x2 *)((uint8_t *)ws + (a.chunks == 1 && !a.prefix_chunks ? 0 : decode_sums_bytes(B, Tq, H, Dh, a.chunks)));
    if ((!n.prefix.chunks && (long long)Hkv * B * a.chunks * ((a.G * Tq + 15) / 16) > kMaxGroups) ||
        (long long)H * Tq * B > kMaxGroups)
        return QG_ERR_SHAPE;
    clear_stale_error();
    switch (type) {
        case QG_TYPE_F32: return launch_decode<QG_TYPE_F32>(a, Dh, (hipStream_t)stream);
        case QG_TYPE_F16: return launch_decode<QG_TYPE_F16>(a, Dh, (hipStream_t)stream);
        default: return launch_decode<QG_TYPE_BF16>(a, Dh, (hipStream_t)stream);
    }
}

}  // namespace qg

extern "C" size_t attn_decode_workspace_bytes(int B, int Tq, int H, int Hkv, int Dh, int max_len, int window) {
    return qg::decode_workspace_bytes(B, Tq, H, Hkv, Dh, max_len, window, 0, 0);
}

extern "C" int attn_decode_kv4(int type, const void *q, int ldq, const int32_t *lens, int B, int Tq, int H, int Hkv,
                               int Dh, float scale, int window, int max_len, const int32_t *pages, int max_pages,
                               int page, int num_pages, const void *kv, float *y, void *ws, size_t ws_bytes,
                               int32_t *d_status, void *stream) {
    return qg::decode(type, q, ldq, lens, B, Tq, H, Hkv, Dh, scale, window, 0, max_len, 0, nullptr, pages, max_pages,
                      page, num_pages, kv, y, ws, ws_bytes, d_status, stream);
}

extern "C" size_t attn_decode_sinks_workspace_bytes(int B, int Tq, int H, int Hkv, int Dh, int max_len, int window,
                                                    int sinks) {
    return qg::decode_workspace_bytes(B, Tq, H, Hkv, Dh, max_len, window, sinks, 0);
}

extern "C" int attn_decode_kv4_sinks(int type, const void *q, int ldq, const int32_t *lens, int B, int Tq, int H,
                                     int Hkv, int Dh, float scale, int window, int sinks, int max_len,
                                     const int32_t *pages, int max_pages, int page, int num_pages, const void *kv,
                                     float *y, void *ws, size_t ws_bytes, int32_t *d_status, void *stream) {
    return qg::decode(type, q, ldq, lens, B, Tq, H, Hkv, Dh, scale, window, sinks, max_len, 0, nullptr, pages,
                      max_pages, page, num_pages, kv, y, ws, ws_bytes, d_status, stream);
}

extern "C" size_t attn_decode_prefix_workspace_bytes(int B, int Tq, int H, int Hkv, int Dh, int max_len, int prefix) {
    return qg::decode_workspace_bytes(B, Tq, H, Hkv, Dh, max_len, 0, 0, prefix);
}

extern "C" int attn_decode_kv4_prefix(int type, const void *q, int ldq, const int32_t *lens, int B, int Tq, int H,
                                      int Hkv, int Dh, float scale, int max_len, int prefix,
                                      const int32_t *prefix_pages, const int32_t *pages, int max_pages, int page,
                                      int num_pages, const void *kv, float *y, void *ws, size_t ws_bytes,
                                      int32_t *d_status, void *stream) {
    return qg::decode(type, q, ldq, lens, B, Tq, H, Hkv, Dh, scale, 0, 0, max_len, prefix, prefix_pages, pages,
                      max_pages, page, num_pages, kv, y, ws, ws_bytes, d_status, stream);
}
