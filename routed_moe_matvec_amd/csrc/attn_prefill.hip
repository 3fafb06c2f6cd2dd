// Causal attention of packed prompts on the matrix cores.
//
// One pass over the keys with the running maximum and sum of a softmax.  A
// workgroup takes 128 queries of one head, 32 a wave, and walks its keys in
// tiles that it copies into two LDS stages, the copies of the next tiles in
// flight while the current ones are used:
//   S^T = K Q^T    (keys x queries),  O^T += V^T P^T   (channels x queries),
// both as v_mfma_f32_32x32x16.  With the products transposed a lane keeps one
// query throughout, and the scores that it receives are the weights that it
// has to supply: P never leaves the registers.  K is read from LDS by rows, V
// by columns (the transposing LDS read); 16-byte pieces of a row are stored
// permuted by the row's number so that neither read meets a bank twice
// (SQ_LDS_BANK_CONFLICT 0).  A step computes the next tile's scores beside this
// tile's weights and sums, which are independent of them (256 channels, one
// wave a SIMD: 776 -> 604 us for 8192 tokens of 16 heads; 512 queries of 16384
// keys 233 -> 193; 128 channels with full tiles, where two waves share a SIMD
// anyway: 2110 -> 2087).
// Weights are rounded to the 16-bit type for their product with V, as is
// y: the two roundings are of one size, and scores, maxima and sums are fp32.
// fp16 weights are 2^11 times as large, below 2^15: those of a long prompt's
// many far keys would otherwise be subnormal, or 0.  The running maximum is one
// of q . k, not scaled, and is taken off the scores themselves where it is large
// (RunningMax; 0 to 2% of the time, 3 for 512 queries of 16384 keys).
//
// One prompt of 16384 tokens, 32 heads of 128 with 8 key heads, bf16: 1.98 to 2.13
// ms by the card, 1033 to 1111 TFLOP/s (a large library product reaches 1219).  The
// matrix cores are busy 57% of the cycles, the vector units 47%, both at once 22%, at
// a clock that falls as the cycles do (1.9 to 1.7 GHz): the card's power is the limit.
#include <type_traits>

#include "common.h"
#include "kv4_device.h"

namespace qg {

constexpr int kPreWaves = 4;

struct PrefillArgs {
    const void *q, *k, *v;
    void *y;
    const int32_t *cu_q, *cu_k;
    int32_t *status;
    int ldq, ldk, ldv, nq, nk, B, H, G, window;
    float scale;  // times log2(e), not negative
    int flip;     // queries change sign (a negative scale) or vanish (scale 0)
    int slots;    // query tiles, over all sequences, with room to spare
};

template <int TYPE>
struct PreElem;
template <>
struct PreElem<QG_TYPE_F16> {
    static constexpr float kShift = 11.f, kSlack = 4.f;  // weights are 2^kShift, up to 2^(kShift + kSlack) before the sums are rescaled
    __device__ static f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    }
    __device__ static uint32_t pack(float a, float b) {
        return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
    }
};
template <>
struct PreElem<QG_TYPE_BF16> {
    static constexpr float kShift = 0.f, kSlack = 8.f;
    __device__ static f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    }
    __device__ static uint32_t pack(float a, float b) {
        return __builtin_bit_cast(uint32_t, bf16x2{(bf16_t)a, (bf16_t)b});
    }
};

// A workgroup's shape: KS waves share 32 queries, each with its own keys of a
// tile, so ROWS = 128 / KS queries a workgroup; and where the 16-byte piece p
// of row r of a tile is held: reads of one piece of many rows (keys) or of four
// pieces of four rows (values) then fall into different banks.
template <int DH, int KS>
struct PreTile {
    static constexpr int RW = kPreWaves / KS, ROWS = 32 * RW;
    static constexpr int N = KS == 4 ? 128 : KS == 1 && DH == 256 ? 32 : 64;  // keys
    static constexpr int CH = DH / 8, BYTES = N * DH * 2;
    __device__ static int k_piece(int r, int p) { return p ^ (r & (CH < 16 ? CH - 1 : 15)); }
    __device__ static int v_piece(int r, int p) { return p ^ (DH == 64 ? (r >> 1 & 1) << 2 : (r & 3) << 2); }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Four rows of one column each, out of LDS.
__device__ __forceinline__ u32x2 lds_read_column4(const char *p) {
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4 *)const_cast<char *>(p));
    return __builtin_bit_cast(u32x2, x);
}

__device__ __forceinline__ float half_max(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
}

__device__ __forceinline__ bool pre_lengths_ok(const PrefillArgs &a, int q0, int q1, int k0, int k1) {
    return q0 >= 0 && q1 >= q0 && q1 <= a.nq && k0 >= 0 && k1 >= k0 && k1 <= a.nk;
}

// Sum over the wave, the same in every lane.
__device__ __forceinline__ int wave_sum(int x) {
#define QG_DPP_ADD(ctrl, rows) x += __builtin_amdgcn_update_dpp(0, x, ctrl, rows, 0xf, false)
    QG_DPP_ADD(0x111, 0xf);  // lane shifts by 1, 2, 4, 8 within rows of 16
    QG_DPP_ADD(0x112, 0xf);
    QG_DPP_ADD(0x114, 0xf);
    QG_DPP_ADD(0x118, 0xf);
    QG_DPP_ADD(0x142, 0xa);  // lane 15 of a row to the next
    QG_DPP_ADD(0x143, 0xc);  // lane 31 to the upper half
#undef QG_DPP_ADD
    return __builtin_amdgcn_readlane(x, 63);
}

// One workgroup's queries: sequence b's tile t, or nothing.
struct PreWork {
    bool any;
    int q0, q1, k0, k1, t;
};

// Up to 64 sequences: the tile of the given rank when all are ordered by the
// keys they see, most first, so that the longest do not start last (six
// prompts of 1 to 3301 keys: 154 us, and 160 in the order of the sequences).
// A lane looks after one sequence, whose tiles see one more bucket of ROWS
// keys each; a bisection over the buckets finds the rank's.
template <int ROWS>
__device__ __forceinline__ PreWork pre_by_rank(const PrefillArgs &a, int rank) {
    const int b = min(lane_id(), a.B - 1);
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
    int tiles = 0, base = 0;
    if (lane_id() < a.B && pre_lengths_ok(a, q0, q1, k0, k1)) {
        tiles = (q1 - q0 + ROWS - 1) / ROWS;
        base = ((k1 - k0) - (q1 - q0) + QG_MAX_ATTN_TOKENS) / ROWS;  // bucket of tile 0, not negative
    }
    PreWork w{false, 0, 0, 0, 0, 0};
    if (rank >= wave_sum(tiles)) return w;
    auto at_least = [&](int x) { return wave_sum(min(max(tiles + min(base - x, 0), 0), tiles)); };
    int lo = 0, hi = 2 * (QG_MAX_ATTN_TOKENS / ROWS) + 2;  // at_least(lo) > rank >= at_least(hi)
    // mostly among the first sequence's buckets
    const int own = __builtin_amdgcn_readfirstlane(base), top = own + __builtin_amdgcn_readfirstlane(tiles);
    if (own > 0) {
        if (at_least(own) > rank)
            lo = own;
        else
            hi = own;
        if (top > lo && top < hi) {
            if (at_least(top) > rank)
                lo = top;
            else
                hi = top;
        }
    }
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (at_least(mid) > rank)
            lo = mid;
        else
            hi = mid;
    }
    const int nth = rank - at_least(lo + 1);
    const bool has = lo >= base && lo - base < tiles;
    const unsigned long long mask = __ballot(has);
    const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
    const int src = __builtin_ctzll(__ballot(has && before == nth) | 1ull << 63);
    w.any = true;
    w.q0 = __builtin_amdgcn_readlane(q0, src);
    w.q1 = __builtin_amdgcn_readlane(q1, src);
    w.k0 = __builtin_amdgcn_readlane(k0, src);
    w.k1 = __builtin_amdgcn_readlane(k1, src);
    w.t = lo - __builtin_amdgcn_readlane(base, src);
    return w;
}

// More sequences: numbered so that sequence b's tiles begin at cu_q[b] / ROWS +
// b (room for any lengths), the last queries first.
template <int ROWS>
__device__ __forceinline__ PreWork pre_by_slot(const PrefillArgs &a, int slot) {
    const int b = wave_find_last(a.B, slot, [&](int s) { return a.cu_q[s] / ROWS + s; });
    PreWork w;
    w.q0 = load_uniform(a.cu_q + b);
    w.q1 = load_uniform(a.cu_q + b + 1);
    w.k0 = load_uniform(a.cu_k + b);
    w.k1 = load_uniform(a.cu_k + b + 1);
    w.t = slot - (w.q0 / ROWS + b);
    w.any = pre_lengths_ok(a, w.q0, w.q1, w.k0, w.k1) && w.t >= 0 && w.t * ROWS < w.q1 - w.q0;
    return w;
}

// 64 channels with the keys split in two: 128 registers, or a compute unit holds
// three workgroups in place of four.
template <int TYPE, int DH, int KS>
__global__ __launch_bounds__(kPreWaves *kWave, DH == 256 || KS == 4 ? 1 : DH == 64 && KS == 2 ? 4 : 2) void attn_prefill_kernel(PrefillArgs a) {
    typedef typename ElemOf<TYPE>::type T;
    typedef PreElem<TYPE> E;
    typedef PreTile<DH, KS> L;
    constexpr int N = L::N, NT = N / 32 / KS, KC = DH / 16, MT = DH / 32;
    // four objects: the compiler tells the copies in flight into one from the reads of another
    __shared__ __attribute__((aligned(16))) char sk0[L::BYTES], sk1[L::BYTES], sv0[L::BYTES], sv1[L::BYTES];
    __shared__ f32x2 sml[KS][kPreWaves][32];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int c = lane & 31, hf = lane >> 5, rw = KS == 1 ? wave : wave % L::RW;
    const int ks = KS == 1 ? 0 : wave / L::RW;

    // Workgroups are dealt to the 8 XCDs in turn: where the heads divide by 8,
    // each XCD takes its own heads, so a key/value head's tiles are fetched
    // into one L2.
    const int id = blockIdx.x;
    int h, rank;
    if (a.H % 8 == 0) {
        const int per = a.H / 8, i = id >> 3;
        h = (id & 7) * per + i % per;
        rank = i / per;
    } else {
        h = id % a.H;
        rank = id / a.H;
    }
    if (id == 0)
        for (int b = threadIdx.x; b < a.B; b += kPreWaves * kWave)
            if (!pre_lengths_ok(a, a.cu_q[b], a.cu_q[b + 1], a.cu_k[b], a.cu_k[b + 1]))
                kv4_report(a.status, QG_DEV_BAD_LENGTH);

    const PreWork w = a.B <= kWave ? pre_by_rank<L::ROWS>(a, rank) : pre_by_slot<L::ROWS>(a, a.slots - 1 - rank);
    if (!w.any) return;
    const int q0 = w.q0, k0 = w.k0, lq = w.q1 - q0, lk = w.k1 - k0;
    const int i0 = w.t * L::ROWS;  // first query of the workgroup, within the sequence
    const int hk = h / a.G;

    // positions: the workgroup's, the wave's and the lane's queries
    const int shift = lk - lq;
    const int wg_hi = min(i0 + L::ROWS, lq) + shift;  // first key that no query sees
    const int wg_lo = a.window ? max(0, i0 + shift - a.window + 1) : 0;
    const int wi0 = i0 + 32 * rw;
    const int w_hi = min(wi0 + 32, lq) + shift;
    const int qi = min(wi0 + c, lq - 1);
    const int see_hi = qi + shift + 1, see_lo = a.window ? see_hi - a.window : 0;

    u32x4 qf[KC];
    {
        const uint32_t flip = a.flip > 0 ? 0x80008000u : 0u, keep = a.flip < 0 ? 0u : ~0u;
        const T *qp = (const T *)a.q + (size_t)(q0 + qi) * a.ldq + (size_t)h * DH + 8 * hf;
#pragma unroll
        for (int i = 0; i < KC; ++i) qf[i] = (*(const u32x4 *)(qp + 16 * i) ^ flip) & keep;
    }
    f32x16 o[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
    RunningMax top;
    float l = 0.f;

    // A tile's copy: each wave takes every fourth KiB; rows behind the last key repeat it.
    constexpr int RPK = 1024 / (DH * 2), KIB = L::BYTES / 1024;  // rows of a KiB
    auto copy_k = [&](int j0, char *sk) {
#pragma unroll
        for (int i = 0; i < KIB / kPreWaves; ++i) {
            const int kib = i * kPreWaves + wave, r = kib * RPK + lane / L::CH, p = lane % L::CH;
            global_to_lds16((const T *)a.k + (size_t)(k0 + min(j0 + r, lk - 1)) * a.ldk + hk * DH + 8 * L::k_piece(r, p),
                            sk + kib * 1024);
        }
    };
    auto copy_v = [&](int j0, char *sv) {
#pragma unroll
        for (int i = 0; i < KIB / kPreWaves; ++i) {
            const int kib = i * kPreWaves + wave, r = kib * RPK + lane / L::CH, p = lane % L::CH;
            global_to_lds16((const T *)a.v + (size_t)(k0 + min(j0 + r, lk - 1)) * a.ldv + hk * DH + 8 * L::v_piece(r, p),
                            sv + kib * 1024);
        }
    };

    constexpr int OWN = 32 * NT;  // keys of a tile that are this wave's, from r0 on
    const int r0 = ks * OWN;

    // One step: the scores `t` of the next tile (keys in sk) beside the weights
    // and sums of this one (scores `s`, values in sv).  The two are independent, so matrix
    // and vector instructions interleave.
    auto step = [&](int next, f32x16 (&s)[NT], f32x16 (&t)[NT], const char *sk, const char *sv, auto do_s, auto do_v) {
        if constexpr (do_s.value) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 16; ++j) t[n][j] = 0.f;
#pragma unroll
            for (int i = 0; i < KC; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int r = r0 + 32 * n + c;
                    const int at = r * DH * 2 + 16 * L::k_piece(r, 2 * i + hf);
                    t[n] = E::mfma(*(const u32x4 *)(sk + at), qf[i], t[n]);
                }
        }
        u32x4 pf[NT][2];
        if constexpr (do_v.value) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    s[n][j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][j], a.scale, -top.muse));
                    l += s[n][j];
                }
#pragma unroll
                for (int kc = 0; kc < 2; ++kc)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        pf[n][kc][j] = E::pack(s[n][8 * kc + 2 * j], s[n][8 * kc + 2 * j + 1]);
            }
        }
        const int j0 = next + r0;
        if constexpr (do_s.value) {
            // register 4 x + y of tile n: key 32 n + 8 x + 4 hf + y
            if (j0 + OWN > wi0 + shift + 1 || (a.window && j0 < w_hi - a.window)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int key = j0 + 32 * n + 8 * (j / 4) + 4 * hf + j % 4;
                        if (key >= see_hi || key < see_lo) t[n][j] = -INFINITY;
                    }
            }
        }
        float mt = -INFINITY;
        if constexpr (do_s.value) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 16; ++j) mt = __builtin_fmaxf(mt, t[n][j]);
            mt = half_max(mt);
        }
        if constexpr (do_v.value) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int kc = 0; kc < 2; ++kc) {
                    const int r = r0 + 32 * n + 16 * kc + 4 * hf + (lane & 15) / 4;  // and r + 8
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const int p = 4 * i + 2 * (c >> 4) + (lane & 3) / 2;
                        const int at = r * DH * 2 + 16 * L::v_piece(r, p) + 8 * (lane & 1);
                        const u32x2 x = lds_read_column4(sv + at), y = lds_read_column4(sv + (at + 8 * DH * 2));
                        o[i] = E::mfma(u32x4{x[0], x[1], y[0], y[1]}, pf[n][kc], o[i]);
                    }
                }
        }
        if constexpr (do_s.value) {
            if (__ballot((mt - top.m) * a.scale > E::kSlack) | top.far) {
                const float keep = top.raise(mt, a.scale, E::kShift);
                if (top.far) {
                    const float raw = top.raw(a.scale);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 16; ++j) t[n][j] -= raw;
                }
                l *= keep;
#pragma unroll
                for (int i = 0; i < MT; ++i) o[i] *= keep;
            }
        }
    };
    f32x16 sa[NT], sb[NT];
    const int first = wg_lo;  // no key that the first query does not see, so none that no query sees
    if (wg_hi > first) {
        // Before a step its keys (of the next tile) and values have arrived for
        // all waves, and all are done with what the copies begun now replace.
        auto begin = [&](int j, char *sk, char *sv) {
            wait_vmem_all();
            __syncthreads();
            if (j + 2 * N < wg_hi) copy_k(j + 2 * N, sk);
            if (j + N < wg_hi) copy_v(j + N, sv);
        };
        copy_k(first, sk0);
        begin(first - N, sk1, sv0);
        using yes = std::true_type;
        using no = std::false_type;
        step(first, sb, sa, sk0, sv0, yes{}, no{});
        int j = first;
        for (; j + 2 * N < wg_hi; j += 2 * N) {
            begin(j, sk0, sv1);
            step(j + N, sa, sb, sk1, sv0, yes{}, yes{});
            begin(j + N, sk1, sv0);
            step(j + 2 * N, sb, sa, sk0, sv1, yes{}, yes{});
        }
        begin(j, sk0, sv1);
        const char *sv = sv0;
        if (j + N < wg_hi) {
            step(j + N, sa, sb, sk1, sv0, yes{}, yes{});
#pragma unroll
            for (int n = 0; n < NT; ++n) sa[n] = sb[n];
            begin(j + N, sk1, sv0);
            sv = sv1;
        }
        step(j, sa, sb, sk0, sv, no{}, yes{});
    }
    l += shfl_xor(l, 32);
    if constexpr (KS > 1) {  // join the waves that share queries, through the stages
        const float exact = top.exact(a.scale, E::kShift);
        if (hf == 0) sml[ks][rw][c] = f32x2{top.m, l * exact};
        __syncthreads();
        float most = -INFINITY, sum = 0.f;
#pragma unroll
        for (int x = 0; x < KS; ++x) most = __builtin_fmaxf(most, sml[x][rw][c][0]);
        if (most == -INFINITY) most = 0.f;
#pragma unroll
        for (int x = 0; x < KS; ++x)
            sum += sml[x][rw][c][1] * __builtin_amdgcn_exp2f((sml[x][rw][c][0] - most) * a.scale);
        const float keep = exact * __builtin_amdgcn_exp2f((top.m - most) * a.scale);
        l = sum;
        static_assert(L::BYTES >= 32 * DH * 4 && (KS - 1) * L::RW <= 4, "a wave's sums fit one object");
        auto room = [&](int i) { return (f32x4 *)(i == 0 ? sk0 : i == 1 ? sk1 : i == 2 ? sv0 : sv1); };
#pragma unroll
        for (int i = 0; i < MT; ++i) o[i] *= keep;
        if (ks > 0)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    room((ks - 1) * L::RW + rw)[(4 * i + x) * kWave + lane] =
                        f32x4{o[i][4 * x], o[i][4 * x + 1], o[i][4 * x + 2], o[i][4 * x + 3]};
        __syncthreads();
        if (ks > 0) return;
        for (int y = 1; y < KS; ++y)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const f32x4 v = room((y - 1) * L::RW + rw)[(4 * i + x) * kWave + lane];
#pragma unroll
                    for (int z = 0; z < 4; ++z) o[i][4 * x + z] += v[z];
                }
    }
    if (wi0 + c >= lq) return;
    const float f = l > 0.f ? 1.f / l : 0.f;
    T *y = (T *)a.y + ((size_t)(q0 + wi0 + c) * a.H + h) * DH;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const u32x2 w = {E::pack(o[i][4 * x] * f, o[i][4 * x + 1] * f),
                             E::pack(o[i][4 * x + 2] * f, o[i][4 * x + 3] * f)};
            *(u32x2 *)(y + 32 * i + 8 * x + 4 * hf) = w;
        }
}

template <int TYPE, int DH, int KS>
static int launch_prefill_ks(PrefillArgs a, hipStream_t stream) {
    a.slots = a.nq / PreTile<DH, KS>::ROWS + a.B;
    const long long grid = (long long)a.slots * a.H;
    if (grid > kMaxGroups) return QG_ERR_SHAPE;
    hipLaunchKernelGGL((attn_prefill_kernel<TYPE, DH, KS>), dim3((unsigned)grid), dim3(kPreWaves * kWave), 0, stream, a);
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

// Where tiles of 128 queries would fill the card at most once (two workgroups a
// compute unit, one with 256 channels), the waves of a workgroup share 64 or, where
// those leave compute units without work, 32 queries and split the keys: smaller
// tiles also spread the triangle of a prompt more evenly.  us with 128, 64, 32 queries
// a workgroup, 32 heads of 128: 128 of 32768 keys 588, 363, 247; 512 of 16384 keys 296,
// 204, 259; 3 and 20 of 8000 keys 147, 92, 66; prompts of 768 tokens 21.4, 16.5, 27.8; 1024
// 26.3, 20.6, 39.7; 3000 92, 99, 198; 16384 2117, 2436.  32 heads of 64: 512 tokens 11.7,
// 8.7, 8.4; 1024 18.3, 13.7, 18.3; 2048 33.4, 30.5, 47.4.  16 heads of 256: 1024 tokens 44.2,
// 31.5; 2048 78.5, 64.8; 2500 92, 100.  One round exactly is the border: tiles of one
// length are even as they are, a prompt's are not.  128 channels, us with 128, 64
// queries: 2048 of 16384 keys 500, 561; 2048 tokens 52.5, 52.2, with a window of 600
// 34.3, 35.7; 8192 of 8 heads 180, 166: tiles of 128.  64 channels: 311, 331; 34.8, 30.9;
// 22.9, 19.6; 114, 100, and 256: 562, 646; 78, 64; 42, 51; 273, 198: prompts gain more
// than the others lose.
template <int TYPE, int DH>
static int launch_prefill_dh(const PrefillArgs &a, hipStream_t stream) {
    const long long cus = device_cu_count(), round = DH == 256 ? cus : 2 * cus;
    const long long tiles = (long long)(a.nq / 128 + a.B / 2) * a.H;  // a sequence's last tile counted half
    if (tiles > round || (DH == 128 && tiles == round)) return launch_prefill_ks<TYPE, DH, 1>(a, stream);
    if (DH == 256 || (long long)(a.nq / 64 + a.B) * a.H >= cus) return launch_prefill_ks<TYPE, DH, 2>(a, stream);
    return launch_prefill_ks<TYPE, DH, DH == 256 ? 2 : 4>(a, stream);
}

template <int TYPE>
static int launch_prefill(const PrefillArgs &a, int Dh, hipStream_t stream) {
    switch (Dh) {
        case 64: return launch_prefill_dh<TYPE, 64>(a, stream);
        case 128: return launch_prefill_dh<TYPE, 128>(a, stream);
        default: return launch_prefill_dh<TYPE, 256>(a, stream);
    }
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
    PrefillArgs a{q, k, v, y, cu_q, cu_k, d_status, ldq, ldk, ldv, nq, nk, B, H, H / Hkv,
                  window < nk ? window : 0};  // a window as long as a sequence hides nothing
    a.scale = scale == 0.f ? 1.f : __builtin_fabsf(scale) * 1.44269504088896340736f;
    a.flip = scale == 0.f ? -1 : scale < 0.f;
    clear_stale_error();
    if (type == QG_TYPE_F16) return launch_prefill<QG_TYPE_F16>(a, Dh, (hipStream_t)stream);
    return launch_prefill<QG_TYPE_BF16>(a, Dh, (hipStream_t)stream);
}
