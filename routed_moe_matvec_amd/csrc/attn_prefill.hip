// Causal attention of packed prompts.  The simple form: one wave per query row
// and head, 64 keys at a time, fp32 throughout.
#include "common.h"
#include "kv4_device.h"

namespace qg {

struct PrefillArgs {
    const void *q, *k, *v;
    void *y;
    const int32_t *cu_q, *cu_k;
    int32_t *status;
    int ldq, ldk, ldv, nq, nk, B, H, G, window;
    float scale;
};

template <int TYPE, int DH>
__global__ __launch_bounds__(64) void attn_prefill_simple_kernel(PrefillArgs a) {
    typedef typename ElemOf<TYPE>::type T;
    constexpr int C = DH / 64;
    const int row = blockIdx.x, h = blockIdx.y, hk = h / a.G, lane = threadIdx.x;
    if (row == 0 && h == 0)
        for (int b = lane; b < a.B; b += 64)
            if (a.cu_q[b] < 0 || a.cu_q[b + 1] < a.cu_q[b] || a.cu_q[b + 1] > a.nq || a.cu_k[b] < 0 ||
                a.cu_k[b + 1] < a.cu_k[b] || a.cu_k[b + 1] > a.nk)
                kv4_report(a.status, QG_DEV_BAD_LENGTH);
    const int b = wave_find_last(a.B, row, [&](int s) { return a.cu_q[s]; });
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
    if (q0 < 0 || q1 > a.nq || k0 < 0 || k1 < k0 || k1 > a.nk || row < q0 || row >= q1) return;
    const int end = min(k1 - k0, row - q0 + (k1 - k0) - (q1 - q0) + 1);
    const int begin = a.window ? max(0, end - a.window) : 0;
    const T *q = (const T *)a.q + (size_t)row * a.ldq + h * DH;
    float mx = -INFINITY, l = 0.f, acc[C] = {};
    for (int j0 = begin; j0 < end; j0 += 64) {
        const int j = j0 + lane;
        float s = -INFINITY;
        if (j < end) {
            const T *k = (const T *)a.k + (size_t)(k0 + j) * a.ldk + hk * DH;
            s = 0.f;
            for (int i = 0; i < DH; ++i) s += (float)q[i] * (float)k[i];
            s *= a.scale;
        }
        float top = s;
        for (int o = 32; o; o >>= 1) top = __builtin_fmaxf(top, shfl_xor(top, o));
        top = __builtin_fmaxf(top, mx);
        const float p = s == -INFINITY ? 0.f : expf(s - top), keep = mx == -INFINITY ? 0.f : expf(mx - top);
        mx = top;
        l *= keep;
        for (int i = 0; i < C; ++i) acc[i] *= keep;
        for (int i = 0; i < 64 && j0 + i < end; ++i) {
            const float w = __shfl(p, i);
            const T *v = (const T *)a.v + (size_t)(k0 + j0 + i) * a.ldv + hk * DH;
            l += w;
            for (int x = 0; x < C; ++x) acc[x] += w * (float)v[lane + 64 * x];
        }
    }
    T *y = (T *)a.y + ((size_t)row * a.H + h) * DH;
    for (int x = 0; x < C; ++x) y[lane + 64 * x] = (T)(l > 0.f ? acc[x] / l : 0.f);
}

template <int TYPE>
static int launch_prefill(const PrefillArgs &a, int Dh, hipStream_t stream) {
    const dim3 grid(a.nq, a.H);
    switch (Dh) {
        case 64: hipLaunchKernelGGL((attn_prefill_simple_kernel<TYPE, 64>), grid, dim3(64), 0, stream, a); break;
        case 128: hipLaunchKernelGGL((attn_prefill_simple_kernel<TYPE, 128>), grid, dim3(64), 0, stream, a); break;
        default: hipLaunchKernelGGL((attn_prefill_simple_kernel<TYPE, 256>), grid, dim3(64), 0, stream, a); break;
    }
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

}  // namespace qg

extern "C" int attn_prefill(int type, const void *q, int ldq, const void *k, int ldk, const void *v, int ldv, int nq,
                            int nk, const int32_t *cu_q, const int32_t *cu_k, int B, int H, int Hkv, int Dh,
                            float scale, int window, void *y, int32_t *d_status, void *stream) {
    using namespace qg;
    if (type != QG_TYPE_F16 && type != QG_TYPE_BF16) return QG_ERR_FORMAT;
    if (!q || !k || !v || !cu_q || !cu_k || !y || !d_status) return QG_ERR_NULL;
    if (B < 1 || B > QG_MAX_SEQS || H < 1 || H > QG_MAX_HEADS || Hkv < 1 || H % Hkv != 0 ||
        (Dh != 64 && Dh != 128 && Dh != 256) || nq < 1 || nq > QG_MAX_ATTN_TOKENS || nk < 1 ||
        nk > QG_MAX_ATTN_TOKENS || window < 0 || !__builtin_isfinite(2.f * scale))
        return QG_ERR_SHAPE;
    if (!row_stride_ok(type, ldq, H * Dh) || !row_stride_ok(type, ldk, Hkv * Dh) || !row_stride_ok(type, ldv, Hkv * Dh))
        return QG_ERR_SHAPE;
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)y) & 15) return QG_ERR_ALIGN;
    if (((uintptr_t)cu_q | (uintptr_t)cu_k | (uintptr_t)d_status) & 3) return QG_ERR_ALIGN;
    const PrefillArgs a{q, k, v, y, cu_q, cu_k, d_status, ldq, ldk, ldv, nq, nk, B, H, H / Hkv, window, scale};
    clear_stale_error();
    if (type == QG_TYPE_F16) return launch_prefill<QG_TYPE_F16>(a, Dh, (hipStream_t)stream);
    return launch_prefill<QG_TYPE_BF16>(a, Dh, (hipStream_t)stream);
}
