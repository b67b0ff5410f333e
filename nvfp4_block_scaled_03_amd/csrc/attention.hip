// Attention of a batch of single query tokens over the paged FP8 cache, with a prefix that every
// sequence shares read once for the whole batch.
//
// For a K/V head the queries of all sequences that use it form one matrix of batch * group rows against
// the prefix (a matrix product per 32 tokens), and group rows per sequence against its own tokens.  Both
// are walked in one launch by workgroups over (row tile, head, token range); each keeps a running
// maximum m and sum l of its rows' softmax and the unnormalised output, and a second launch joins the
// ranges: out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i.
//
// Matrix instructions, 16 rows at a time, S^T = K Q^T then O^T = V^T P^T, so that a score's lane (column
// = query row) is the lane that feeds it to the second product, with no move between lanes: score
// register i of lane group g is token 4g + i of its 16-token tile, and two tiles make the 32 tokens of
// one second product, in that order.  V's bytes take the same order by loading each lane group's own
// eight tokens (a run of head_dim/16 bytes of each) and transposing 4 x 4 bytes in registers.
// K's codes widen to bf16, exactly; the queries stay bf16.  With a scale per tensor or head V's codes widen to FP16,
// exactly too, and the probabilities are rounded to FP16, scaled by 2^7: a relative step of 2^-11 down to 2^-21 of the
// row's largest, below the bf16 output's own 2^-8.  With a scale per slot a probability carries its token's scale into
// the second product.  FP16 cannot hold such products: a row of zeros has the scale 1 where its neighbours may have
// 2^-30, and any unit that keeps the one in range loses the others.  They enter in two bf16 parts (2^-17 of each, with
// FP32's exponents, so that no token's precision depends on another's scale) against V's codes in bf16, one matrix
// instruction more per fragment.
//
// What bounds it: with few rows per head the cache's bytes, with many the matrix instructions and the widening
// of the codes, which rows_panel does once for 128 rows; with little of either the latency of a range (first
// pages, first codes, the join).  Measured, heads of 128 (a large copy moves 4.7 TB/s, a large bf16 product makes
// 1138 TFLOP/s): 64 sequences of 64 heads on 8, a prefix of 65536 and 2048 own tokens, a scale per slot: 254 us,
// 555 TFLOP/s in all (the prefix alone 585, with a scale per head 795; the own tokens alone 3.9 to 4.3 TB/s); 64 of
// 32 heads, 4096 and 512, a scale per head: 28 us, 5 of them the join.
#include "mixers.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 32;              // tokens per second product
// log2 of the probabilities' scale.  They exceed it by 2^8 at most: FP16 ends at 2^16, and with a scale per slot none is
// larger than 1, so that a product with the scale overflows only where the scale does.
template <bool kTok> constexpr float kOffset = kTok ? -8.0f : 7.0f;
constexpr float kNegInf = -__builtin_inff();

struct Params {
    AttentionArgs a;
    float scale2;                       // softmax scale * log2(e), times nothing else
    int page_shift;
    int prefix_blocks, prefix_blocks8;  // workgroups over the prefix, and rounded up to 8 XCDs
    int prefix_tiles, prefix_splits;    // row tiles per head, token ranges
    int64_t prefix_range;               // tokens per range
    int seq_tiles, seq_splits;
    int64_t seq_range;
    int joint;                          // every sequence walks the prefix itself (a short one)
    int n_part;                         // ranges per output row
    float* acc;                         // [row][n_part][D]
    float2* ml;                         // [row][n_part]
};

template <int D> struct Raw {           // one block's codes as loaded
    uint4 k[2][D / 64];
    uint32_t v[2][4][D / 64];
};

// One wavefront's state over NQ tiles of 16 query rows.
template <int D, int NQ> struct Rows {
    float4v o[NQ][D / 16];
    float4v ones[NQ];                   // l as a matrix instruction sums it (a row of ones for V), where it does
    float m[NQ], l[NQ];                 // m: the maximum so far, as far as it was moved
    float base[NQ];                     // what is added to a score: offset - m (offset before the first token)
    float limit[NQ];                    // above this a score with its base moves the maximum
    __device__ __forceinline__ void clear(float offset) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            m[n] = limit[n] = kNegInf;
            base[n] = offset;
            l[n] = 0.0f;
            ones[n] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[n][i] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }
};

// The tokens of a walk: a list of pages, then a second one that begins at the next multiple of 16.
struct Tokens {
    const int32_t* a;
    int64_t a_len, a16;                 // tokens of the first list; the same rounded up to 16
    const int32_t* b;
    int64_t b_len;
    __device__ __forceinline__ int64_t end() const { return b_len > 0 ? a16 + b_len : a_len; }
};
__device__ __forceinline__ Tokens one_list(const int32_t* pages, int64_t len) { return Tokens{pages, len, (len + 15) & ~int64_t(15), pages, 0}; }

// Where one 16-token half block lies (wave-uniform): its first slot, and how many of its tokens count.
struct Half {
    int64_t slot0;
    int live;
};

template <int D>
__device__ __forceinline__ void load_k(const Params& p, int head, int64_t slot0, int l16, int kg, uint4 (&k)[D / 64]) {
    const uint8_t* base = p.a.cache.k_codes + (slot0 * p.a.cache.heads + head) * D;
    const uint32_t at = (uint32_t)l16 * (uint32_t)(p.a.cache.heads * D) + kg * 16;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) k[i] = *reinterpret_cast<const uint4*>(base + at + i * 64);
}

template <int D>
__device__ __forceinline__ void load_v(const Params& p, int head, int64_t slot0, int l16, int kg, uint32_t (&v)[4][D / 64]) {
    const uint8_t* base = p.a.cache.v_codes + (slot0 * p.a.cache.heads + head) * D;
    const uint32_t ld = (uint32_t)(p.a.cache.heads * D), at = 4 * kg * ld + l16 * (D / 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint8_t* q = base + (at + i * ld);
        if constexpr (D == 64) {
            v[i][0] = *reinterpret_cast<const uint32_t*>(q);
        } else if constexpr (D == 128) {
            const uint2 u = *reinterpret_cast<const uint2*>(q);
            v[i][0] = u.x;
            v[i][1] = u.y;
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(q);
            v[i][0] = u.x;
            v[i][1] = u.y;
            v[i][2] = u.z;
            v[i][3] = u.w;
        }
    }
}

__device__ __forceinline__ bf16x8 widen_bf16(uint32_t lo, uint32_t hi) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ half8 widen_f16(uint32_t lo, uint32_t hi) {
    const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const half2v b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const half2v c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const half2v d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Bytes b of x[0..3] -> y[b] (a 4 x 4 byte transpose).
__device__ __forceinline__ void transpose4(uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3, uint32_t y[4]) {
    const uint32_t a = __builtin_amdgcn_perm(x1, x0, 0x05010400u), b = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
    const uint32_t c = __builtin_amdgcn_perm(x3, x2, 0x05010400u), d = __builtin_amdgcn_perm(x3, x2, 0x07030602u);
    y[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
    y[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
    y[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
    y[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

__device__ __forceinline__ float group_max(float v) {   // over the four lane groups of a column
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float group_sum(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// V's fragments and the probabilities that meet them: FP16, or with a scale per slot (in the probabilities) bf16, those in
// two parts.
template <bool kTok> struct Second;
template <> struct Second<false> {
    typedef half8 Values;
    struct Probs {
        half8 p;
        __device__ __forceinline__ void put(int i, float x0, float x1) {
            p[i] = (_Float16)x0;
            p[i + 1] = (_Float16)x1;
        }
    };
    static __device__ __forceinline__ Values widen(uint32_t lo, uint32_t hi) { return widen_f16(lo, hi); }
    static __device__ __forceinline__ uint2 widen4(uint32_t x) {
        return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, false)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, true)));
    }
    static __device__ __forceinline__ float4v product(Values v, const Probs& p, float4v o) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p.p, o, 0, 0, 0);
    }
};
template <> struct Second<true> {
    typedef bf16x8 Values;
    struct Probs {
        bf16x8 hi, lo;                  // the upper 16 bits as they are, and the nearest bf16 of the rest
        __device__ __forceinline__ void put(int i, float x0, float x1) {
            const uint32_t u0 = __float_as_uint(x0), u1 = __float_as_uint(x1);
            const bf16x2 h = __builtin_bit_cast(bf16x2, __builtin_amdgcn_perm(u1, u0, 0x07060302u));
            const bf16x2 l = __builtin_convertvector((float2v{x0 - __uint_as_float(u0 & 0xFFFF0000u),
                                                              x1 - __uint_as_float(u1 & 0xFFFF0000u)}), bf16x2);
            hi[i] = h[0];
            hi[i + 1] = h[1];
            lo[i] = l[0];
            lo[i + 1] = l[1];
        }
    };
    static __device__ __forceinline__ Values widen(uint32_t lo, uint32_t hi) { return widen_bf16(lo, hi); }
    static __device__ __forceinline__ uint2 widen4(uint32_t x) {
        return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, false)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, true)));
    }
    static __device__ __forceinline__ float4v product(Values v, const Probs& p, float4v o) {
        o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p.lo, o, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p.hi, o, 0, 0, 0);
    }
};

// One block's probabilities out of its scores (base 2, with their base added; -inf where nothing counts).  The
// running maximum is moved only when some score exceeds it by more than 2^8: until then no lane has to ask the others
// for its row's maximum.
// kTok: the probabilities of the second product carry the values' scales vs.  kSum: l is summed here.
template <int D, int NQ, bool kTok, bool kSum>
__device__ __forceinline__ void softmax_step(Rows<D, NQ>& s, float4v (&sc)[NQ][2], const float4v* vs,
                                             typename Second<kTok>::Probs (&pf)[NQ]) {
    bool move = false;
    float mx[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        mx[n] = fmaxf(fmaxf(fmaxf(sc[n][0][0], sc[n][0][1]), fmaxf(sc[n][0][2], sc[n][0][3])),
                      fmaxf(fmaxf(sc[n][1][0], sc[n][1][1]), fmaxf(sc[n][1][2], sc[n][1][3])));
        move |= mx[n] > s.limit[n];
    }
    if (__builtin_amdgcn_ballot_w64(move)) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const float top = group_max(mx[n]) - s.base[n], m_new = fmaxf(s.m[n], top);
            if (m_new > kNegInf) {           // the same for all lanes of a row
                const float f = __builtin_amdgcn_exp2f(s.m[n] - m_new), base = kOffset<kTok> - m_new, d = base - s.base[n];
                s.m[n] = m_new;
                s.base[n] = base;
                s.limit[n] = kOffset<kTok> + 8.0f;
                if (kSum) s.l[n] *= f;
                else s.ones[n] *= f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) s.o[n][i] *= f;
#pragma unroll
                for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[n][tt][i] += d;
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        float sum = 0.0f;
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float e0 = __builtin_amdgcn_exp2f(sc[n][tt][i]), e1 = __builtin_amdgcn_exp2f(sc[n][tt][i + 1]);
                if (kSum) sum += e0 + e1;
                pf[n].put(4 * tt + i, kTok ? e0 * vs[tt][i] : e0, kTok ? e1 * vs[tt][i + 1] : e1);
            }
        if (kSum) s.l[n] += sum;
    }
}

// Walks positions [t0, t_end) of `list` in blocks of 32, `step` tokens apart, for NQ tiles of 16 rows
// whose query fragments are qf.  t0 is a multiple of 16, so each half block lies in one page.
//
// The next block's codes are loaded right behind the last use of this one's, from addresses that always name a
// page of the pool (what does not count is masked), so that no branch stands around a load and the waits are for
// what is needed only.
template <int D, int NQ, bool kTok>
__device__ __forceinline__ void walk(const Params& p, int head, const Tokens& list, int64_t t0, int64_t t_end,
                                     int64_t step, const bf16x8 (&qf)[NQ][D / 32], Rows<D, NQ>& s,
                                     float (*scales)[2][kBlock]) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t page_mask = (int64_t(1) << p.page_shift) - 1;
    const int per_head = p.a.cache.scale_mode == NVFP4_KV_SCALE_HEAD ? head : 0;
    const float k_fixed = kTok ? p.scale2 : p.scale2 * p.a.cache.k_scale[per_head];
    s.clear(kOffset<kTok>);
    if (t0 < t_end) {
    const int64_t last = (t_end - 1) & ~int64_t(15);
    // A table entry is loaded a block before the codes it leads to and looked at only then: its own latency, and the
    // wait for all older loads that looking at it means, are over by that time.
    auto entry = [&](int64_t b) {
        const int64_t c = b < last ? b : last;
        return (c < list.a16 ? list.a : list.b)[(c < list.a16 ? c : c - list.a16) >> p.page_shift];
    };
    auto find = [&](int64_t b, int32_t e) {
        const int64_t c = b < last ? b : last;
        const bool first = c < list.a16;
        const int64_t at = first ? c : c - list.a16, left = (first ? list.a_len : list.b_len) - at;
        const int32_t page = __builtin_amdgcn_readfirstlane(e);
        const bool ok = page >= 0 && page < p.a.cache.pages;
        Half h;
        h.slot0 = ((int64_t)(ok ? page : 0) << p.page_shift) + (at & page_mask);
        h.live = !ok || b >= t_end ? 0 : (left < 16 ? (int)left : 16);
        return h;
    };
    float next_ks = 0.0f, next_vs = 0.0f;    // per-slot scales of token lane mod 32 of the next block
    auto load_scales = [&](const Half (&h)[2]) {
        if constexpr (kTok) {
            const int64_t s0 = h[0].slot0, s1 = h[1].slot0;
            const int n0 = h[0].live, n1 = h[1].live;
            const int64_t at = ((lane & 16 ? s1 : s0) + l16) * p.a.cache.heads + head;
            const bool there = l16 < (lane & 16 ? n1 : n0);
            next_ks = p.a.cache.k_scale[at];
            next_vs = p.a.cache.v_scale[at];
            next_ks = there ? next_ks : 0.0f;
            next_vs = there ? next_vs : 0.0f;
        }
    };
    Raw<D> raw;
    int32_t ahead[2] = {entry(t0 + step), entry(t0 + step + 16)};
    Half now[2] = {find(t0, entry(t0)), find(t0 + 16, entry(t0 + 16))};
#pragma unroll
    for (int tt = 0; tt < 2; ++tt) {
        load_k<D>(p, head, now[tt].slot0, l16, kg, raw.k[tt]);
        load_v<D>(p, head, now[tt].slot0, l16, kg, raw.v[tt]);
    }
    load_scales(now);
    for (int64_t t = t0; t < t_end; t += step) {
        const Half next[2] = {find(t + step, ahead[0]), find(t + step + 16, ahead[1])};
        ahead[0] = entry(t + 2 * step);
        ahead[1] = entry(t + 2 * step + 16);
        const bool whole = now[0].live + now[1].live == kBlock;
        float4v ks[2], vs[2];
        if constexpr (kTok) {
            if (lane < kBlock) {
                scales[wave][0][lane] = next_ks * p.scale2;
                scales[wave][1][lane] = next_vs;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                ks[tt] = *reinterpret_cast<const float4v*>(&scales[wave][0][tt * 16 + kg * 4]);
                vs[tt] = *reinterpret_cast<const float4v*>(&scales[wave][1][tt * 16 + kg * 4]);
            }
            load_scales(next);
        }
        // S^T tiles: 16 tokens x 16 query rows each
        float4v sc[NQ][2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) sc[n][tt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const bf16x8 k0 = widen_bf16(raw.k[tt][i].x, raw.k[tt][i].y);
                const bf16x8 k1 = widen_bf16(raw.k[tt][i].z, raw.k[tt][i].w);
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    sc[n][tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, qf[n][2 * i], sc[n][tt], 0, 0, 0);
                    sc[n][tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, qf[n][2 * i + 1], sc[n][tt], 0, 0, 0);
                }
            }
            load_k<D>(p, head, next[tt].slot0, l16, kg, raw.k[tt]);
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[n][tt][i] = sc[n][tt][i] * (kTok ? ks[tt][i] : k_fixed) + s.base[n];
        if (!whole) {                        // what a page holds behind the last token is anything: drop it
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool there = 4 * kg + i < now[tt].live;
#pragma unroll
                    for (int n = 0; n < NQ; ++n) sc[n][tt][i] = there ? sc[n][tt][i] : kNegInf;
#pragma unroll
                    for (int j = 0; j < D / 64; ++j) raw.v[tt][i][j] = there ? raw.v[tt][i][j] : 0u;
                }
        }
        typename Second<kTok>::Probs pf[NQ];
        softmax_step<D, NQ, kTok, true>(s, sc, vs, pf);
        // O^T += V^T P^T: tile 4 j + b holds the elements d = row * (D / 16) + 4 j + b
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            uint32_t lo[4], hi[4];
            transpose4(raw.v[0][0][j], raw.v[0][1][j], raw.v[0][2][j], raw.v[0][3][j], lo);
            transpose4(raw.v[1][0][j], raw.v[1][1][j], raw.v[1][2][j], raw.v[1][3][j], hi);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const auto vf = Second<kTok>::widen(lo[b], hi[b]);
#pragma unroll
                for (int n = 0; n < NQ; ++n) s.o[n][4 * j + b] = Second<kTok>::product(vf, pf[n], s.o[n][4 * j + b]);
            }
        }
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            load_v<D>(p, head, next[tt].slot0, l16, kg, raw.v[tt]);
            now[tt] = next[tt];
        }
    }
    }
    const float unit = kTok ? 1.0f : p.a.cache.v_scale[per_head];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        s.l[n] = group_sum(s.l[n]);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) s.o[n][i] *= unit;
    }
}

// Where the result of row (b, hq) over range i goes: a partial, or the output when it is the only one.
template <int D>
__device__ __forceinline__ void put(const Params& p, int b, int hq, int range, int d, float4v x, float l) {
    if (p.n_part == 1) {
        const float r = l > 0.0f ? 1.0f / l : 0.0f;
        uint16_t* o = p.a.out + b * p.a.out_batch + hq * p.a.out_head + d;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = f32_to_bf16_rne(x[i] * r);
    } else {
        const int64_t row = (int64_t)b * p.a.cache.heads * p.a.group + hq;
        *reinterpret_cast<float4v*>(p.acc + (row * p.n_part + range) * D + d) = x;
    }
}
__device__ __forceinline__ void put_ml(const Params& p, int b, int hq, int range, float m, float l) {
    if (p.n_part > 1)
        p.ml[((int64_t)b * p.a.cache.heads * p.a.group + hq) * p.n_part + range] = make_float2(m, l);
}

// Query fragments of 16 rows from row0 on of a head's rows_total (row = b * group + g from base_b on).
template <int D, bool kNatural = false>
__device__ __forceinline__ void load_queries(const Params& p, int head, int base_b, int row0, int rows_total,
                                             bf16x8 (&qf)[D / 32]) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, kg = lane >> 4;
    int row = row0 + l16;
    row = row < rows_total ? row : rows_total - 1;
    const int b = base_b + row / p.a.group, g = row % p.a.group;
    const uint16_t* q = p.a.q + b * p.a.q_batch + (int64_t)(head * p.a.group + g) * p.a.q_head;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)         // d in natural order, or as a lane's 16-byte loads of codes hold it
        qf[i] = *reinterpret_cast<const bf16x8*>(q + (kNatural ? i * 32 + kg * 8 : (i >> 1) * 64 + kg * 16 + (i & 1) * 8));
}

// A workgroup whose four wavefronts take the same 16 rows and every fourth block of tokens.
template <int D> struct Joint {
    alignas(16) float4v part[4][16][D / 4 + 1];
    alignas(16) float scales[4][2][kBlock];
    float2 ml[4][16];
};

template <int D, bool kTok>
__device__ __forceinline__ void rows_shared(const Params& p, int head, int base_b, int row0, int rows_total,
                                            const Tokens& list, int64_t t0, int64_t t_end, int range, void* lds) {
    auto& sh = *reinterpret_cast<Joint<D>*>(lds);
    auto& part = sh.part;
    auto& part_ml = sh.ml;
    const int lane = threadIdx.x & 63, l16 = lane & 15, kg = lane >> 4, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (t0 < t_end) {
        bf16x8 qf[1][D / 32];
        load_queries<D>(p, head, base_b, row0, rows_total, qf[0]);
        Rows<D, 1> s;
        walk<D, 1, kTok>(p, head, list, t0 + kBlock * wave, t_end, 4 * kBlock, qf, s, sh.scales);
        if (kg == 0) part_ml[wave][l16] = make_float2(s.m[0], s.l[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                part[wave][l16][(4 * kg + i) * (D / 64) + j] =
                    float4v{s.o[0][4 * j][i], s.o[0][4 * j + 1][i], s.o[0][4 * j + 2][i], s.o[0][4 * j + 3][i]};
    } else {
        if (kg == 0) part_ml[wave][l16] = make_float2(kNegInf, 0.0f);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) part[wave][l16][kg * (D / 16) + j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __syncthreads();
    for (int u = threadIdx.x; u < 16 * (D / 4); u += kThreads) {
        const int r = u / (D / 4), c = u % (D / 4);
        if (row0 + r >= rows_total) continue;
        float m = kNegInf;
#pragma unroll
        for (int w = 0; w < 4; ++w) m = fmaxf(m, part_ml[w][r].x);
        const float m_use = m == kNegInf ? 0.0f : m;
        float l = 0.0f;
        float4v x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = __builtin_amdgcn_exp2f(part_ml[w][r].x - m_use);
            l += f * part_ml[w][r].y;
            x += part[w][r][c] * f;
        }
        const int b = base_b + (row0 + r) / p.a.group, hq = head * p.a.group + (row0 + r) % p.a.group;
        if (c == 0) put_ml(p, b, hq, range, m, l);
        put<D>(p, b, hq, range, 4 * c, x, l);
    }
}

// Many rows over a long prefix (head_dim 64 and 128): a workgroup whose wavefronts take 16 NQ rows each, all over the
// same tokens.  The codes of 64 tokens are widened once for the four wavefronts, into LDS in the order of the
// fragments: K [token][d] in bf16, V [d][token] (FP16, or bf16 with a scale per slot) with each 32 tokens in the order of
// the scores' registers and the 16-byte units of a row exchanged by its number, so that neither the writes (eight rows
// apart) nor the reads (neighbouring rows) meet on a bank.  Two blocks in LDS, one barrier per block.
constexpr int kPanel = 64;

template <int D> struct Panels {
    alignas(16) __bf16 k[2][kPanel][D + 8];
    alignas(16) uint16_t v[2][D][kPanel];
    alignas(16) float scales[2][2][kPanel];  // the per-slot scales of K and V
};

__device__ __forceinline__ int panel_unit(int d, int unit) { return (unit ^ d ^ (d >> 3)) & 7; }

template <int D, int NQ, bool kTok>
__device__ __forceinline__ void rows_panel(const Params& p, int head, int row0, int rows_total,
                                           const int32_t* __restrict__ pages, int64_t t0, int64_t t_end, int range,
                                           void* lds) {
    auto& sh = *reinterpret_cast<Panels<D>*>(lds);
    const int lane = threadIdx.x & 63, l16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    row0 += wave * 16 * NQ;
    const bool any = row0 < rows_total;      // a wavefront without rows still brings its tokens
    bf16x8 qf[NQ][D / 32];
#pragma unroll
    for (int n = 0; n < NQ; ++n)             // in the natural order of d here
        load_queries<D, true>(p, head, 0, row0 + 16 * n, rows_total, qf[n]);
    Rows<D, NQ> s;
    s.clear(kOffset<kTok>);
    const int64_t page_mask = (int64_t(1) << p.page_shift) - 1;
    const int per_head = p.a.cache.scale_mode == NVFP4_KV_SCALE_HEAD ? head : 0;
    const float k_fixed = kTok ? 1.0f : p.scale2 * p.a.cache.k_scale[per_head];
    const float unit = kTok ? 1.0f : p.a.cache.v_scale[per_head];
    const int64_t last = (t_end - 1) & ~int64_t(15);
    // this wavefront's 16 tokens of a block
    uint4 rk[D / 64];
    uint32_t rv[4][D / 64];
    float rks = 0.0f, rvs = 0.0f;
    int live = 0;
    auto entry = [&](int64_t b) { return pages[(b < last ? b : last) >> p.page_shift]; };
    auto find = [&](int64_t b, int32_t e, int& n) {      // as in walk
        const int64_t c = b < last ? b : last;
        const int32_t page = __builtin_amdgcn_readfirstlane(e);
        const bool ok = page >= 0 && page < p.a.cache.pages;
        n = !ok || b >= t_end ? 0 : (t_end - b < 16 ? (int)(t_end - b) : 16);
        return ((int64_t)(ok ? page : 0) << p.page_shift) + (c & page_mask);
    };
    int32_t ahead = entry(t0 + kPanel + 16 * wave);
    auto load = [&](int64_t slot0) {
        load_k<D>(p, head, slot0, l16, kg, rk);
        load_v<D>(p, head, slot0, l16, kg, rv);
        if constexpr (kTok) {
            const int64_t at = (slot0 + l16) * p.a.cache.heads + head;
            rks = p.a.cache.k_scale[at];
            rvs = p.a.cache.v_scale[at];
        }
    };
    load(find(t0 + 16 * wave, entry(t0 + 16 * wave), live));
    for (int64_t t = t0; t < t_end; t += kPanel) {
        const int buf = (int)((t - t0) / kPanel) & 1;
        int next_live;
        const int64_t next_slot = find(t + kPanel + 16 * wave, ahead, next_live);
        ahead = entry(t + 2 * kPanel + 16 * wave);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            *reinterpret_cast<bf16x8*>(&sh.k[buf][wave * 16 + l16][i * 64 + kg * 16]) = widen_bf16(rk[i].x, rk[i].y);
            *reinterpret_cast<bf16x8*>(&sh.k[buf][wave * 16 + l16][i * 64 + kg * 16 + 8]) = widen_bf16(rk[i].z, rk[i].w);
        }
        if (live < 16) {                     // what a page holds behind the last token is anything: drop it
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < D / 64; ++j) rv[i][j] = 4 * kg + i < live ? rv[i][j] : 0u;
        }
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            uint32_t y[4];
            transpose4(rv[0][j], rv[1][j], rv[2][j], rv[3][j], y);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int d = l16 * (D / 16) + 4 * j + b;
                *reinterpret_cast<uint2*>(&sh.v[buf][d][panel_unit(d, (wave >> 1) * 4 + kg) * 8 + (wave & 1) * 4]) =
                    Second<kTok>::widen4(y[b]);
            }
        }
        if constexpr (kTok) {
            if (kg == 0) {
                sh.scales[buf][0][wave * 16 + l16] = l16 < live ? rks * p.scale2 : 0.0f;
                sh.scales[buf][1][wave * 16 + l16] = l16 < live ? rvs : 0.0f;
            }
        }
        // tokens that do not count: at the end of the range, or a page outside the pool (whose half block says so)
        if (lane == 0) reinterpret_cast<int*>(&sh.k[buf][wave * 16][D])[0] = live;
        load(next_slot);
        live = next_live;
        __syncthreads();
        // Scores of the whole block first, then its probabilities, then the second product: the matrix pipe works on
        // one while the other wavefront of the SIMD takes exponentials.
        float4v sc[2][NQ][2];
#pragma unroll
        for (int tile = 0; tile < 4; ++tile) {
            float4v(&x)[NQ][2] = sc[tile >> 1];
            const int tt = tile & 1;
#pragma unroll
            for (int n = 0; n < NQ; ++n) x[n][tt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const bf16x8 kf = *reinterpret_cast<const bf16x8*>(&sh.k[buf][tile * 16 + l16][i * 32 + kg * 8]);
#pragma unroll
                for (int n = 0; n < NQ; ++n) x[n][tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[n][i], x[n][tt], 0, 0, 0);
            }
        }
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            float4v vs[2];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                const int tile = st * 2 + tt;
                float4v ks;
                if constexpr (kTok) {
                    ks = *reinterpret_cast<const float4v*>(&sh.scales[buf][0][tile * 16 + kg * 4]);
                    vs[tt] = *reinterpret_cast<const float4v*>(&sh.scales[buf][1][tile * 16 + kg * 4]);
                }
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[st][n][tt][i] = sc[st][n][tt][i] * (kTok ? ks[i] : k_fixed) + s.base[n];
                const int count = __builtin_amdgcn_readfirstlane(reinterpret_cast<const int*>(&sh.k[buf][tile * 16][D])[0]);
                if (count < 16) {
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sc[st][n][tt][i] = 4 * kg + i < count ? sc[st][n][tt][i] : kNegInf;
                }
            }
            typename Second<kTok>::Probs pf[NQ];
            softmax_step<D, NQ, kTok, kTok>(s, sc[st], vs, pf);
            if constexpr (!kTok) {
                const _Float16 one = (_Float16)1.0f;
                const half8 ones = {one, one, one, one, one, one, one, one};
#pragma unroll
                for (int n = 0; n < NQ; ++n) s.ones[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pf[n].p, s.ones[n], 0, 0, 0);
            }
#pragma unroll
            for (int m = 0; m < D / 16; ++m) {
                const int d = m * 16 + l16;
                const auto vf = *reinterpret_cast<const typename Second<kTok>::Values*>(&sh.v[buf][d][panel_unit(d, st * 4 + kg) * 8]);
#pragma unroll
                for (int n = 0; n < NQ; ++n) s.o[n][m] = Second<kTok>::product(vf, pf[n], s.o[n][m]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        s.l[n] = kTok ? group_sum(s.l[n]) : s.ones[n][0];
        const int row = row0 + 16 * n + l16;
        if (!any || row >= rows_total) continue;
        const int b = row / p.a.group, hq = head * p.a.group + row % p.a.group;
        if (kg == 0) put_ml(p, b, hq, range, s.m[n], s.l[n]);
#pragma unroll
        for (int m = 0; m < D / 16; ++m) put<D>(p, b, hq, range, m * 16 + kg * 4, s.o[n][m] * unit, s.l[n]);
    }
}

constexpr int kWideTiles = 2;                // 16-row tiles per wavefront of rows_panel
constexpr int kWideRows = 4 * 16 * kWideTiles;

template <int D, bool kTok, bool kWide>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2))) void attention_kernel(Params p) {
    constexpr size_t kPanels = kWide ? sizeof(Panels<D>) : 0;
    __shared__ alignas(16) uint8_t lds[sizeof(Joint<D>) > kPanels ? sizeof(Joint<D>) : kPanels];
    const int id = blockIdx.x;
    if (id < p.prefix_blocks8) {
        // consecutive items (the row tiles of one head and range) on one XCD, whose L2 then reads K and V once
        const int item = (id & 7) * (p.prefix_blocks8 >> 3) + (id >> 3);
        if (item >= p.prefix_blocks) return;
        const int tile = item % p.prefix_tiles, rest = item / p.prefix_tiles;
        const int head = rest % p.a.cache.heads, range = rest / p.a.cache.heads;
        const int64_t t0 = range * p.prefix_range;
        const int64_t t1 = t0 + p.prefix_range < p.a.prefix_len ? t0 + p.prefix_range : p.a.prefix_len;
        const int rows = p.a.batch * p.a.group;
        if constexpr (kWide)
            rows_panel<D, kWideTiles, kTok>(p, head, tile * kWideRows, rows, p.a.prefix_pages, t0, t1, range, lds);
        else
            rows_shared<D, kTok>(p, head, 0, tile * 16, rows, one_list(p.a.prefix_pages, p.a.prefix_len), t0, t1, range, lds);
        return;
    }
    const int item = id - p.prefix_blocks8;
    const int head = item % p.a.cache.heads, r1 = item / p.a.cache.heads;
    const int tile = r1 % p.seq_tiles, r2 = r1 / p.seq_tiles;
    const int b = r2 % p.a.batch, range = r2 / p.a.batch;
    int64_t len = 0;
    if (p.a.max_len > 0) {                   // no table and no lengths otherwise
        len = p.a.lens[b];
        len = len < p.a.max_len ? len : p.a.max_len;
    }
    const int32_t* own = p.a.pages + b * p.a.pages_ld;
    if (p.joint) {                           // the prefix, then the sequence's own tokens, in one go
        Tokens list = one_list(p.a.prefix_pages, p.a.prefix_len);
        list.b = own;
        list.b_len = len > 0 ? len : 0;
        rows_shared<D, kTok>(p, head, b, tile * 16, p.a.group, list, 0, list.end(), 0, lds);
        return;
    }
    const int64_t t0 = range * p.seq_range;
    const int64_t t1 = t0 + p.seq_range < len ? t0 + p.seq_range : len;
    rows_shared<D, kTok>(p, head, b, tile * 16, p.a.group, one_list(own, len > 0 ? len : 0), t0, t1, p.prefix_splits + range,
                         lds);
}

// Joins the ranges of an output row, one workgroup a row: D / 4 lanes take a range at a time, four columns a lane.
template <int D>
__global__ __launch_bounds__(kThreads) void join_kernel(Params p) {
    constexpr int G = D / 4, kSlots = kThreads / G;
    __shared__ alignas(16) float4v part[4][G];
    __shared__ float part_l[4];
    const int heads = p.a.cache.heads * p.a.group, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int slot = threadIdx.x / G, c = threadIdx.x % G, n = p.n_part;
    const int64_t row = blockIdx.x;
    const float2* ml = p.ml + row * p.n_part;
    const float4v* acc = reinterpret_cast<const float4v*>(p.acc + row * p.n_part * D) + c;
    float m = kNegInf;
    for (int i = lane; i < n; i += 64) m = fmaxf(m, ml[i].x);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    const float m_use = m == kNegInf ? 0.0f : m;
    float l = 0.0f;
    float4v x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = slot; i < n; i += kSlots) {
        const float f = __builtin_amdgcn_exp2f(ml[i].x - m_use);
        l += f * ml[i].y;
        x += f * acc[(int64_t)i * G];
    }
#pragma unroll
    for (int off = G; off < 64; off <<= 1) {
        l += __shfl_xor(l, off, 64);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] += __shfl_xor(x[j], off, 64);
    }
    if (lane < G) part[wave][c] = x;
    if (lane == 0) part_l[wave] = l;
    __syncthreads();
    if (threadIdx.x >= G) return;
    l = (part_l[0] + part_l[1]) + (part_l[2] + part_l[3]);
    x = (part[0][c] + part[1][c]) + (part[2][c] + part[3][c]);
    x *= l > 0.0f ? 1.0f / l : 0.0f;
    const int b = (int)(row / heads), hq = (int)(row % heads);
    uint16_t* o = p.a.out + b * p.a.out_batch + hq * p.a.out_head + c * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = f32_to_bf16_rne(x[j]);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Token ranges so that about `want` workgroups run, none shorter than `least` tokens.  For a prefix 512: of 65536 for 64
// sequences of 8 heads of 4 rows it takes 96 us, with 256 128, with 1024 104; of 16384 for 16 24.6, 25.5, 25.0 (shorter
// ranges would cost the join what they save).  For own tokens 1024: 2048 of 64 sequences 41.6 us, with 512 39, with
// 2048 46; of 4 12.4, 13.6, 14.7.
void split(int64_t tokens, int64_t units, int64_t want, int64_t least, int& splits, int64_t& range) {
    int64_t n = want / (units > 0 ? units : 1);
    const int64_t most = ceil_div(tokens, least);
    n = n < most ? n : most;
    n = n < 1 ? 1 : n;
    range = ceil_div(ceil_div(tokens, n), kBlock) * kBlock;
    splits = (int)ceil_div(tokens, range);
}

constexpr int64_t kJointTokens = 1024;

struct Plan {
    bool wide, joint;
    int prefix_tiles, prefix_splits, seq_tiles, seq_splits;
    int64_t prefix_range, seq_range;
};

Plan plan(int heads, int dim, int64_t batch, int64_t group, int64_t prefix_len, int64_t max_len) {
    Plan q{};
    const int64_t rows = batch * group;
    // Panels widen a code once for 128 rows instead of once for 16, but fill the chip with an eighth of the workgroups
    // and cost a start of their own, which workgroups over own tokens can fill.  So the products (rows * heads *
    // prefix_len) decide, from three quarters of a panel on, earlier with own tokens.  Time of panels over that of tiles,
    // 96 to 512 rows of 2 and 8 heads of 128 and 8 of 64, a scale per head (per slot):
    //   without own tokens  8 << 20: +1 to +24% (-2 to +22);  12 << 20: -9 to +17 (-16 to +16);  16 << 20: -14 to +6
    //                       (-22 to +2);  32 << 20: -31 to -14 (-35 to -18)
    //   with 128            8 << 20: -10 to +22 (-16 to +15)
    //   with 512            6 << 20: -16 to +6 (-15 to +5);  8 << 20: -14 to +11 (-18 to +2)
    //   with 2048           6 << 20: -10 to +12 (-9 to +2);  8 << 20: -20 to +8 (-12 to +4)
    // 64 rows: 0 to +31% (-5 to +27) at 8 and 16 << 20.  head_dim 256 has no panels: two blocks of
    // K and V would take 134 of a compute unit's 160 KB of LDS, one workgroup of four wavefronts; not built or measured.
    q.wide = dim != 256 && rows >= kWideRows * 3 / 4 &&
             rows * heads * prefix_len >= (max_len >= 256 ? int64_t(7) << 20 : int64_t(12) << 20);
    q.prefix_tiles = (int)ceil_div(rows, q.wide ? kWideRows : 16);
    q.prefix_range = q.seq_range = kBlock;
    // A prefix so short that each sequence walks it itself, eight blocks of 32 per wavefront at most: one launch and
    // no partial sums.  8 heads of 4 rows, 256 own tokens (joint, by ranges): prefix of 512 for 1 sequence 8.7, 13.5 us,
    // for 64 13.4, 16.8; 700 for 64 15.8, 16.7; 1500 for 1 14.5, 13.9, for 64 23.2, 18.8.
    q.joint = prefix_len > 0 && prefix_len + max_len <= kJointTokens;
    if (q.joint) {
        q.seq_tiles = (int)ceil_div(group, 16);
        q.seq_splits = 1;
        return q;
    }
    if (prefix_len > 0)
        split(prefix_len, (int64_t)heads * q.prefix_tiles, 512, q.wide ? 256 : 512, q.prefix_splits, q.prefix_range);
    q.seq_tiles = (int)ceil_div(group, 16);
    if (max_len > 0)
        split(max_len, (int64_t)heads * q.seq_tiles * batch, 1024, 512, q.seq_splits, q.seq_range);
    else if (prefix_len == 0)
        q.seq_splits = 1;     // nothing to attend to: the rows still get their zeros
    return q;
}

size_t ml_bytes(int64_t rows, int64_t parts) { return (size_t)(rows * parts * 8 + 255) / 256 * 256; }

template <int D>
hipError_t launch_d(const Params& p, const Plan& q, hipStream_t stream) {
    const int64_t seq = (int64_t)q.seq_splits * q.seq_tiles * p.a.cache.heads * p.a.batch;
    const dim3 grid((unsigned)(p.prefix_blocks8 + seq)), block(kThreads);
    const bool tok = p.a.cache.scale_mode == NVFP4_KV_SCALE_TOKEN;
    const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, p); };
    if constexpr (D != 256)
        if (q.wide) tok ? go(attention_kernel<D, true, true>) : go(attention_kernel<D, false, true>);
    if (!q.wide) tok ? go(attention_kernel<D, true, false>) : go(attention_kernel<D, false, false>);
    if (p.n_part > 1) {
        const int64_t rows = (int64_t)p.a.batch * p.a.cache.heads * p.a.group;
        hipLaunchKernelGGL(join_kernel<D>, dim3((unsigned)rows), block, 0, stream, p);
    }
    return hipGetLastError();
}

}  // namespace

size_t attention_workspace_bytes(const nvfp4_kv_cache& c, int64_t batch, int64_t heads, int64_t prefix_len,
                                 int64_t max_len) {
    const Plan q = plan(c.heads, c.head_dim, batch, heads / c.heads, prefix_len, max_len);
    const int64_t parts = q.prefix_splits + q.seq_splits, rows = batch * heads;
    return parts <= 1 ? 0 : ml_bytes(rows, parts) + (size_t)(rows * parts * c.head_dim) * 4;
}

hipError_t launch_attention(const AttentionArgs& a, void* workspace, hipStream_t stream) {
    Params p{};
    p.a = a;
    if (a.cache.pages == 0) p.a.prefix_len = p.a.max_len = 0;      // no page number is one of the pool's
    const Plan q = plan(a.cache.heads, a.cache.head_dim, a.batch, a.group, p.a.prefix_len, p.a.max_len);
    p.scale2 = a.scale * 1.4426950408889634f;
    while ((1 << p.page_shift) < a.cache.page_size) ++p.page_shift;
    p.prefix_tiles = q.prefix_tiles;
    p.prefix_splits = q.prefix_splits;
    p.prefix_range = q.prefix_range;
    p.prefix_blocks = q.prefix_splits * q.prefix_tiles * a.cache.heads;
    p.prefix_blocks8 = (p.prefix_blocks + 7) / 8 * 8;
    p.seq_tiles = q.seq_tiles;
    p.seq_splits = q.seq_splits;
    p.seq_range = q.seq_range;
    p.joint = q.joint;
    p.n_part = q.prefix_splits + q.seq_splits;
    const int64_t rows = (int64_t)a.batch * a.cache.heads * a.group;
    p.ml = static_cast<float2*>(workspace);
    if (p.n_part > 1) p.acc = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ml_bytes(rows, p.n_part));
    switch (a.cache.head_dim) {
        case 64: return launch_d<64>(p, q, stream);
        case 128: return launch_d<128>(p, q, stream);
        default: return launch_d<256>(p, q, stream);
    }
}

}  // namespace nvfp4
