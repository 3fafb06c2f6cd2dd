// Attention of new tokens over the paged FP4 cache.  The simple form: one
// workgroup per query row, 256 keys at a time, fp32 throughout.
#include "common.h"
#include "kv4_device.h"

namespace qg {

struct DecodeArgs {
    Kv4Cache c;
    const void *q;
    float *y;
    int ldq, Tq, H, G, window, max_len;
    float scale;
};

__device__ __forceinline__ float e2m1_value(uint32_t code) {
    const uint32_t m = code & 7;
    const float v = m < 4 ? 0.5f * (float)m : m < 6 ? (float)m - 2.f : 2.f * (float)m - 8.f;
    return code & 8 ? -v : v;
}

template <int TYPE, int DH>
__global__ __launch_bounds__(256) void attn_decode_simple_kernel(DecodeArgs a) {
    typedef typename ElemOf<TYPE>::type T;
    __shared__ float sq[DH], sp[256], sm[256];
    const Kv4Cache &c = a.c;
    const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, hk = h / a.G;
    const int len = c.lens[b], page = 1 << c.page_log2;
    float *y = a.y + ((size_t)(b * a.Tq + t) * a.H + h) * DH;
    const bool ok = len >= 0 && len <= a.max_len;
    if (!ok && tid == 0) kv4_report(c.status, QG_DEV_BAD_LENGTH);
    const int pos = len - a.Tq + t;
    const int end = ok ? pos + 1 : 0, begin = a.window ? max(0, end - a.window) : 0;
    const T *q = (const T *)a.q + (size_t)(b * a.Tq + t) * a.ldq + h * DH;
    for (int i = tid; i < DH; i += 256) sq[i] = (float)q[i];
    const size_t region = kv4_region_bytes(page, DH);
    float mx = -INFINITY, l = 0.f, acc = 0.f;
    for (int j0 = begin; j0 < end; j0 += 256) {
        __syncthreads();
        const int j = j0 + tid;
        float s = -INFINITY;
        if (j < end) {
            const int id = kv4_page_of(c, b, j >> c.page_log2);
            if (id >= 0) {
                const uint8_t *r = c.kv + ((size_t)id * c.Hkv + hk) * region;
                const int o = j & (page - 1);
                s = 0.f;
                for (int i = 0; i < DH; ++i) {
                    const uint32_t w = r[(size_t)o * (DH / 2) + i / 2] >> (4 * (i & 1)) & 15u;
                    const uint32_t e = r[(size_t)page * DH + o * (DH / 32) + i / 32];
                    s += sq[i] * e2m1_value(w) * __builtin_bit_cast(float, e << 23);
                }
                s *= a.scale;
            }
        }
        sm[tid] = s;
        __syncthreads();
        float top = mx;
        for (int i = 0; i < 256; ++i) top = __builtin_fmaxf(top, sm[i]);
        const float use = top == -INFINITY ? 0.f : top;
        sp[tid] = s == -INFINITY ? 0.f : expf(s - use);
        __syncthreads();
        const float keep = mx == -INFINITY ? 0.f : expf(mx - use);
        l *= keep;
        acc *= keep;
        mx = top;
        for (int i = 0; i < 256 && j0 + i < end; ++i) {
            l += sp[i];
            if (tid < DH && sp[i] != 0.f) {
                const int jj = j0 + i, o = jj & (page - 1);
                const int id = c.pages[(size_t)b * c.max_pages + (jj >> c.page_log2)];
                const uint8_t *r = c.kv + ((size_t)id * c.Hkv + hk) * region;
                const uint32_t w = r[(size_t)page * (DH / 2) + ((o / 4) * (DH / 8) + tid / 8) * 16 + (o % 4) * 4 + tid % 8 / 2] >>
                                       (4 * (tid & 1)) & 15u;
                const uint32_t e = r[(size_t)page * (DH + DH / 32) + ((o / 4) * (DH / 32) + tid / 32) * 4 + o % 4];
                acc += sp[i] * e2m1_value(w) * __builtin_bit_cast(float, e << 23);
            }
        }
    }
    if (tid < DH) y[tid] = l > 0.f ? acc / l : 0.f;
}

template <int TYPE>
static int launch_decode(const DecodeArgs &a, int Dh, hipStream_t stream) {
    const dim3 grid(a.H, a.Tq, a.c.B);
    switch (Dh) {
        case 64: hipLaunchKernelGGL((attn_decode_simple_kernel<TYPE, 64>), grid, dim3(256), 0, stream, a); break;
        case 128: hipLaunchKernelGGL((attn_decode_simple_kernel<TYPE, 128>), grid, dim3(256), 0, stream, a); break;
        default: hipLaunchKernelGGL((attn_decode_simple_kernel<TYPE, 256>), grid, dim3(256), 0, stream, a); break;
    }
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

static bool decode_shape_ok(int B, int Tq, int H, int Hkv, int Dh, int max_len, int window) {
    return B >= 1 && B <= QG_MAX_SEQS && Tq >= 1 && Tq <= QG_MAX_DECODE_TOKENS && H >= 1 && H <= QG_MAX_HEADS &&
           Hkv >= 1 && H % Hkv == 0 && (Dh == 64 || Dh == 128 || Dh == 256) && max_len >= 1 &&
           max_len <= 0x3fffffff && window >= 0;
}

}  // namespace qg

extern "C" size_t attn_decode_workspace_bytes(int B, int Tq, int H, int Hkv, int Dh, int max_len, int window) {
    if (!qg::decode_shape_ok(B, Tq, H, Hkv, Dh, max_len, window)) return 0;
    return 256;
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
    if (!row_stride_ok(type, ldq, H * Dh) || !__builtin_isfinite(scale)) return QG_ERR_SHAPE;
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
    a.scale = scale;
    clear_stale_error();
    switch (type) {
        case QG_TYPE_F32: return launch_decode<QG_TYPE_F32>(a, Dh, (hipStream_t)stream);
        case QG_TYPE_F16: return launch_decode<QG_TYPE_F16>(a, Dh, (hipStream_t)stream);
        default: return launch_decode<QG_TYPE_BF16>(a, Dh, (hipStream_t)stream);
    }
}
