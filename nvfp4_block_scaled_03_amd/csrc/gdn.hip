// The gated delta recurrence of a Gated DeltaNet layer, per batch row and value head:
//     S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,     o_t = scale S_t^T q_t,
// with S [k_dim][v_dim] in FP32, forward and backward.
//
// A few tokens are walked one by one (gdn_step_kernel).  Longer sequences go by chunks of 64 tokens.  With
// Gam_ij = prod_{j<l<=i} alpha_l and gam_i = prod_{l<=i} alpha_l inside a chunk that starts from S0,
//     S_i = gam_i S0 + sum_{j<=i} Gam_ij k_j u_j^T
// where the rows u solve (I + A) U = beta (V - gam K S0), A_ij = beta_i Gam_ij k_i.k_j for j < i.  So
//     T = (I + A)^-1,  R = beta V - beta gam K S0,  U = T R,
//     O = scale gam Q S0 + P U,  P_ij = scale Gam_ij q_i.k_j (j <= i),
//     S' = gam_63 S0 + K^T diag(Gam_63) U.
// W = K^T diag(Gam_63) T and N = P T depend on no state: gdn_prep_kernel makes them for all chunks at once, and
// what is left to do in order is two products per chunk,
//     R = beta V - beta gam K S0,  S' = gam_63 S0 + W R      (and O = scale gam Q S0 + N R beside them).
// gdn_scan_kernel walks the chunks of one head, a workgroup per 16 or 32 columns of the state (which are
// independent).  Backward, with D the gradient of a chunk's last state,
//     dR = N^T dO + W^T D,  D' = gam_63 D + (scale gam Q)^T dO - (beta gam K)^T dR,  dV = beta dR
// is again two products in order (gdn_scan_back_kernel); the gradients of q, k and the gates follow chunk by
// chunk, all at once (gdn_grad_kernel).
//
// Precision: states, gates, sums and the triangular inverse are FP32.  The matrix instructions take bf16
// operands, so every FP32 operand is split into three bf16 parts (24 significant bits, what FP32 holds): a
// product with q, k, v or dO, exact in bf16, takes three instructions, one of two FP32 operands the six
// whose parts reach 2^-24; gfx950's FP32 matrix instruction would take the time of sixteen.
// The products of decays and T stand apart from the state, so this holds where they are no larger than 1 or so: for
// |alpha| <= 1 and 0 <= beta |k|^2 <= 2, where no factor alpha (I - beta k k^T) lengthens what it acts on.
#include "mixers.h"

namespace nvfp4 {
namespace {

constexpr int kC = 64;                  // tokens per chunk
constexpr int kThreads = 256;
// Up to this many tokens are walked one by one.  32 heads of 128 x 128, 64 sequences of 2, 8, 12, 16 tokens: 70, 152,
// 210, 270 us, by chunks 193, 197, 199, 200; 4 sequences 11, 18, 25, 32 and 22, 23, 23, 23.
constexpr int kStepTokens = 8;

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

struct Shape {
    int64_t tokens;
    int32_t batch, hk, hv, group, dk, dv, chunks;
    float scale;
    const int32_t* lens;
};

// Tokens of batch row b (wave-uniform; at most 2^28).
__device__ __forceinline__ int seq_len(const Shape& s, int b) {
    int n = (int)s.tokens;
    if (s.lens != nullptr) {
        const int m = s.lens[b];
        n = m < 0 ? 0 : (m < n ? m : n);
    }
    return __builtin_amdgcn_readfirstlane(n);
}

template <typename T> __device__ __forceinline__ T* row_ptr(const nvfp4_rows& v, int64_t b, int64_t t, int64_t h) {
    return static_cast<T*>(v.data) + b * v.batch_stride + t * v.token_stride + h * v.head_stride;
}

__device__ __forceinline__ float bf16_f32(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

__device__ __forceinline__ float4v mfma(bf16x8 a, bf16x8 b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// x = p[0] + p[1] + p[2], each part the nearest bf16 of what the earlier ones leave.
__device__ __forceinline__ void split3(float4v x, bf16x4 p[3]) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        p[k] = __builtin_convertvector(x, bf16x4);
        x = x - __builtin_convertvector(p[k], float4v);
    }
}

// Sums of products by parts.  A dependent matrix instruction waits for the one before it, so the parts accumulate
// apart and are added at the end, smallest first.
struct Acc3 {
    float4v x[3] = {};
    __device__ __forceinline__ float4v sum() const { return (x[2] + x[1]) + x[0]; }
};

// ---------------------------------------------------------------------------
// A few tokens, one by one.  A workgroup holds 32 columns of one head's
// state: a thread four columns of every 32nd row, so that a wavefront's loads
// are whole 128-byte lines.  One pass over the state's registers gives both
// k^T S and q^T S (o = scale (alpha q^T S + (q.k) u)), so a token costs one
// reduction.  Bound by the state's bytes (read and written once per call):
// 64 sequences of 32 heads of 128 x 128 take 50 us, 5.4 TB/s.  With 16 or 64
// columns per workgroup 63 and 77 us.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kThreads) void gdn_step_kernel(Shape s, nvfp4_rows q, nvfp4_rows k, nvfp4_rows v,
                                                            nvfp4_rows alpha, nvfp4_rows beta, const float* state,
                                                            nvfp4_rows o, float* state_out) {
    constexpr int CG = 8, RG = kThreads / CG, RT = 128 / RG;
    __shared__ float red[2][4][CG][9];
    const int cg = threadIdx.x % CG, rg = threadIdx.x / CG, wave = threadIdx.x >> 6;
    const int b = blockIdx.z, h = blockIdx.y, hk = h / s.group;
    const int col = blockIdx.x * 4 * CG + 4 * cg;
    const bool in = col < s.dv;
    const int64_t base = ((int64_t)b * s.hv + h) * s.dk * s.dv + col;
    float4v S[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int row = i * RG + rg;
        S[i] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
        if (state != nullptr && in && row < s.dk)
            S[i] = *reinterpret_cast<const float4v*>(state + base + (int64_t)row * s.dv);
    }
    const int n = seq_len(s, b);
    for (int t = 0; t < n; ++t) {
        const uint16_t* kp = row_ptr<const uint16_t>(k, b, t, hk);
        const uint16_t* qp = row_ptr<const uint16_t>(q, b, t, hk);
        const float al = *row_ptr<const float>(alpha, b, t, h), be = *row_ptr<const float>(beta, b, t, h);
        float kr[RT], qk = 0.0f;
        float4v ks = {0.0f, 0.0f, 0.0f, 0.0f}, qs = ks, vv = ks;
        if (in) {
            const uint16_t* vp = row_ptr<const uint16_t>(v, b, t, h) + col;
            vv = float4v{bf16_f32(vp[0]), bf16_f32(vp[1]), bf16_f32(vp[2]), bf16_f32(vp[3])};
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int row = i * RG + rg;
            kr[i] = row < s.dk ? bf16_f32(kp[row]) : 0.0f;
            const float qr = row < s.dk ? bf16_f32(qp[row]) : 0.0f;
            ks += S[i] * kr[i];
            qs += S[i] * qr;
            qk += kr[i] * qr;
        }
#pragma unroll
        for (int off = CG; off < 64; off <<= 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ks[j] += __shfl_xor(ks[j], off, 64);
                qs[j] += __shfl_xor(qs[j], off, 64);
            }
            qk += __shfl_xor(qk, off, 64);
        }
        float* mine = red[t & 1][wave][cg];
        if ((threadIdx.x & 63) < CG) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mine[j] = ks[j];
                mine[4 + j] = qs[j];
            }
            mine[8] = qk;
        }
        __syncthreads();
        float sum[9];
#pragma unroll
        for (int j = 0; j < 9; ++j)
            sum[j] = (red[t & 1][0][cg][j] + red[t & 1][1][cg][j]) + (red[t & 1][2][cg][j] + red[t & 1][3][cg][j]);
        float4v u;
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = be * (vv[j] - al * sum[j]);
        if (rg == 0 && in) {
            uint16_t* op = row_ptr<uint16_t>(o, b, t, h) + col;
#pragma unroll
            for (int j = 0; j < 4; ++j) op[j] = f32_to_bf16_rne(s.scale * (al * sum[4 + j] + sum[8] * u[j]));
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) S[i] = S[i] * al + u * kr[i];
    }
    if (state_out != nullptr && in) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int row = i * RG + rg;
            if (row < s.dk) *reinterpret_cast<float4v*>(state_out + base + (int64_t)row * s.dv) = S[i];
        }
    }
}

// ---------------------------------------------------------------------------
// What a chunk needs that depends on no state.
//
// Matrices are kept as the operand fragments the scans feed to the matrix
// instructions: [part][row tile of 16][k-step of 32][lane][8], lane = row +
// 16 * (group of 8 along k), so a fragment is one 16-byte load per lane and
// 1 KB per wavefront.
//
// Measured, 8192 tokens of 32 heads of 128 x 128: 94 to 99 us, 322 MB written
// (3.4 TB/s).  A workgroup's time is the latency of its steps one after the
// other (decays, the inverse's block diagonals), so what counts is how many
// share a compute unit: four with 35 KB of LDS (three for the backward pass, by
// its registers), with 52 KB three and 104 us, with 71 KB two and 148.
// ---------------------------------------------------------------------------
constexpr int kFrag = 64 * 8;                       // bf16 elements of one fragment
constexpr int kSquare = 8 * kFrag;                  // of a 64 x 64 matrix (one part)

struct Prep {                                       // per (batch, value head, chunk), and per key head where said
    __bf16* w;                                      // W [dk][64], three parts
    __bf16* n;                                      // N, two parts (forward)
    __bf16* wt;                                     // W^T in the state's order, three parts (backward)
    __bf16* nt;                                     // N^T, three parts (backward)
    __bf16* t;                                      // T, three parts (backward)
    __bf16* kt;                                     // per key head: K^T [dk][64] (exact; backward)
    __bf16* qt;                                     // per key head: Q^T (backward)
    __bf16* kx;                                     // per key head: K in the state's order (see put_rows_in_order)
    __bf16* qx;                                     // per key head: Q in the state's order (forward)
    float* g;                                       // gam_i [64], Gam_63,i [64], beta_i [64]
};

constexpr int kGates = 3 * kC;                      // floats of g per chunk
constexpr int kLd = kC + 4;                         // row stride of a square in LDS: rows stay on 16 bytes

__device__ __forceinline__ bf16x8 load_row8(const uint16_t* row, bool valid, int at) {
    bf16x8 z = {};
    return valid ? *reinterpret_cast<const bf16x8*>(row + at) : z;
}

__device__ __forceinline__ void split3(const float x[8], bf16x8 p[3]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float y = x[j];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            p[k][j] = (__bf16)y;
            y -= (float)p[k][j];
        }
    }
}

// Eight entries of row r of a square in LDS from column c on, or of column r from row c on.
__device__ __forceinline__ void row8(const float (*m)[kLd], int r, int c, float x[8]) {
    *reinterpret_cast<float4v*>(x) = *reinterpret_cast<const float4v*>(&m[r][c]);
    *reinterpret_cast<float4v*>(x + 4) = *reinterpret_cast<const float4v*>(&m[r][c + 4]);
}
__device__ __forceinline__ void col8(const float (*m)[kLd], int r, int c, float x[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = m[c + j][r];
}

// Writes the fragments of a lower triangular 64 x 64 FP32 matrix in LDS, three parts; the fragments above the
// diagonal are neither written nor read.
__device__ __forceinline__ void put_square(const float (*m)[kLd], __bf16* out) {
    for (int f = threadIdx.x; f < 6 * 64; f += kThreads) {
        const int lane = f & 63, i = f >> 6, l16 = lane & 15, kg = lane >> 4;
        const int tile = i < 4 ? i : i - 2, step = i < 4 ? 0 : 1;
        alignas(16) float x[8];
        row8(m, tile * 16 + l16, step * 32 + kg * 8, x);
        bf16x8 part[3];
        split3(x, part);
#pragma unroll
        for (int k = 0; k < 3; ++k)
            *reinterpret_cast<bf16x8*>(out + k * kSquare + (tile * 2 + step) * kFrag + lane * 8) = part[k];
    }
}

// Four values of column l16 of a 16 x 16 tile, rows 16 rt + 4 g + 0..3, as half of a left-hand fragment whose rows
// are the tile's columns (row tile ct) and whose k are the tile's rows.
template <int kParts>
__device__ __forceinline__ void put_turned(__bf16* out, int part_size, int ct, int rt, int l16, int kg, float4v x) {
    bf16x4 part[3];
    split3(x, part);
    const int at = (ct * 2 + (rt >> 1)) * kFrag + (l16 + 16 * ((rt & 1) * 2 + (kg >> 1))) * 8 + (kg & 1) * 4;
#pragma unroll
    for (int a = 0; a < kParts; ++a) *reinterpret_cast<bf16x4*>(out + a * part_size + at) = part[a];
}

// K^T or Q^T in LDS: 8 tokens of a row are 16 bytes, the eight such pieces of row d at places turned by d.
__device__ __forceinline__ int turned_at(int d, int t8) { return d * kC + ((t8 ^ d) & 7) * 8; }

// A row's eight entries from column 32 i + 8 kg on, of each slice i of 32, into the transposed matrix.
template <int KS>
__device__ __forceinline__ void scatter_turned(const bf16x8 (&x)[KS], uint16_t* out, int row, int kg) {
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const uint4 v = __builtin_bit_cast(uint4, x[i]);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            out[turned_at(i * 32 + kg * 8 + j, row >> 3) + (row & 7)] = (uint16_t)(u[j >> 1] >> (j & 1) * 16);
    }
}

// Fragments [column tile][step][lane][8] of a transposed matrix in LDS.
template <int KS>
__device__ __forceinline__ void put_turned_fragments(const uint16_t* m, __bf16* out) {
    for (int f = threadIdx.x; f < KS * 4 * 64; f += kThreads) {
        const int lane = f & 63, fr = f >> 6;
        *reinterpret_cast<bf16x8*>(out + fr * kFrag + lane * 8) =
            *reinterpret_cast<const bf16x8*>(m + turned_at((fr >> 1) * 16 + (lane & 15), (fr & 1) * 4 + (lane >> 4)));
    }
}

// The chunk's rows of K or Q as left-hand fragments [slice of 32 along dk][row tile][lane][8] whose eight entries
// of lane group g are k = 4 g + 0..3 and 16 + 4 g + 0..3 of the slice: the rows that a lane's accumulators of two
// neighbouring 16-row tiles hold, so that a wavefront's own state registers are the right-hand operand as they are.
// Lane group kg holds columns 8 kg + 0..7, that is halves of two fragments' entries.
template <int KS>
__device__ __forceinline__ void put_rows_in_order(const bf16x8 (&x)[KS], __bf16* out, int tile, int l16, int kg) {
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const uint4 v = __builtin_bit_cast(uint4, x[i]);
        __bf16* o = out + (i * 4 + tile) * kFrag + (l16 + 16 * (2 * kg & 3)) * 8 + (kg >> 1) * 4;
        *reinterpret_cast<uint2*>(o) = make_uint2(v.x, v.y);
        *reinterpret_cast<uint2*>(o + 16 * 8) = make_uint2(v.z, v.w);
    }
}

// Gam of a chunk into LDS, rows 16 w .. 16 w + 15 by one wavefront whose lane j holds alpha_j: lane j starts with
// the product of alpha_{j+1} .. alpha_{16 w - 1} (a suffix product by lane shifts) and runs down its column, so no
// logarithm is taken and no quotient formed (a decay of 0 is as good as any).
__device__ __forceinline__ void chunk_decays(const float* al, float (*gam)[kLd], float* since, int w) {
    const int j = threadIdx.x & 63;
    float a[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<float4v*>(a + 4 * i) = *reinterpret_cast<const float4v*>(&al[16 * w + 4 * i]);
    float r = j + 1 < 16 * w ? al[j + 1] : 1.0f;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const float o = __shfl_down(r, off, 64);
        r *= j + off < 64 ? o : 1.0f;
    }
    const float first = al[0];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int row = 16 * w + i;
        r = row == j ? 1.0f : r * a[i];
        gam[row][j] = row >= j ? r : 0.0f;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (j < 16) since[16 * w + j] = gam[16 * w + j][0] * first;
}

template <int KS, bool kBackward>
__global__ __launch_bounds__(kThreads) void gdn_prep_kernel(Shape s, nvfp4_rows q, nvfp4_rows k, nvfp4_rows alpha,
                                                            nvfp4_rows beta, Prep out) {
    // Two squares, 35 KB in all, so that four workgroups share a compute unit: Gam, then A in its place, then P; the rows of
    // K, then T, then K^T and Q^T.
    __shared__ alignas(16) float gam[kC][kLd], tm[kC][kLd];
    __shared__ alignas(16) float al[kC];
    __shared__ float be[kC], since[kC], until[kC];
    static_assert(sizeof(uint16_t[kC][KS * 32 + 8]) <= sizeof(tm), "rows and K^T fit over T");
    uint16_t(*rows)[KS * 32 + 8] = reinterpret_cast<uint16_t(*)[KS * 32 + 8]>(tm);
    float(*am)[kLd] = gam;
    uint16_t* turned = reinterpret_cast<uint16_t*>(tm);
    const int c = blockIdx.x, h = blockIdx.y, b = blockIdx.z, hk = h / s.group;
    const int64_t t0 = (int64_t)c * kC;
    const int left = seq_len(s, b) - c * kC;
    if (left <= 0) return;
    const int n = left < kC ? left : kC;
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, kg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t ch = ((int64_t)b * s.hv + h) * s.chunks + c, ck = ((int64_t)b * s.hk + hk) * s.chunks + c;
    if (tid < kC) {
        al[tid] = tid < n ? *row_ptr<const float>(alpha, b, t0 + tid, h) : 1.0f;
        be[tid] = tid < n ? *row_ptr<const float>(beta, b, t0 + tid, h) : 0.0f;
    }
    // this wavefront's rows of K and Q
    bf16x8 kw[KS], qw[KS];
    const int frow = w * 16 + l16;
    {
        const uint16_t* kp = row_ptr<const uint16_t>(k, b, t0 + frow, hk);
        const uint16_t* qp = row_ptr<const uint16_t>(q, b, t0 + frow, hk);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            kw[i] = load_row8(kp, frow < n, i * 32 + kg * 8);
            qw[i] = load_row8(qp, frow < n, i * 32 + kg * 8);
        }
    }
#pragma unroll
    for (int i = 0; i < KS; ++i) *reinterpret_cast<bf16x8*>(&rows[frow][i * 32 + kg * 8]) = kw[i];
    __syncthreads();
    const bool first = h % s.group == 0;    // the key head's own operands, by its first value head
    if (first) {
        put_rows_in_order<KS>(kw, out.kx + ck * KS * 32 * kC, w, l16, kg);
        if (!kBackward) put_rows_in_order<KS>(qw, out.qx + ck * KS * 32 * kC, w, l16, kg);
    }
    chunk_decays(al, gam, since, w);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // gam rows 16 w .. are this wavefront's own: no barrier
    if (w == 3) until[lane] = gam[kC - 1][lane];
    // (K K^T)^T and (Q K^T)^T tiles of row tile w: lane = row i, registers = four neighbouring columns j
    float4v g[4], z[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        g[m] = z[m] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
        if (m > w) continue;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const bf16x8 x = *reinterpret_cast<const bf16x8*>(&rows[m * 16 + l16][i * 32 + kg * 8]);
            g[m] = mfma(x, kw[i], g[m]);
            z[m] = mfma(x, qw[i], z[m]);
        }
    }
    __syncthreads();                        // T goes where the rows were
    float4v pw[4];                          // P until A is done with
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int j0 = m * 16 + kg * 4;
        const float4v d = *reinterpret_cast<const float4v*>(&gam[frow][j0]);
        float4v a4;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            a4[r] = j0 + r < frow ? be[frow] * (d[r] * g[m][r]) : 0.0f;
            pw[m][r] = s.scale * (d[r] * z[m][r]);
        }
        *reinterpret_cast<float4v*>(&am[frow][j0]) = a4;
        if (m > w) *reinterpret_cast<float4v*>(&tm[frow][j0]) = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // (I + A)^-1: the 16 x 16 blocks on the diagonal (each by its own wavefront) by substitution, a column per lane
    {
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float x = i == l16 ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < i; ++j) x -= am[w * 16 + i][w * 16 + j] * t[j];
            t[i] = x;
        }
        if (kg == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) tm[w * 16 + i][w * 16 + l16] = t[i];
        }
    }
    __syncthreads();
    if (tid < kC) {
        out.g[ch * kGates + tid] = since[tid];
        out.g[ch * kGates + kC + tid] = until[tid];
        out.g[ch * kGates + 2 * kC + tid] = be[tid];
    }
    // then diagonal by diagonal below: T_ij = -T_ii sum_{j<=l<i} A_il T_lj, in FP32 matrix instructions
#pragma unroll
    for (int d = 1; d < 4; ++d) {
        if (w >= d) {
            const int bi = w, bj = w - d;
            float4v x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
            for (int l = bj; l < bi; ++l)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    x = __builtin_amdgcn_mfma_f32_16x16x4f32(am[bi * 16 + l16][l * 16 + kg * 4 + r],
                                                             tm[l * 16 + kg * 4 + r][bj * 16 + l16], x, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                y = __builtin_amdgcn_mfma_f32_16x16x4f32(tm[bi * 16 + l16][bi * 16 + kg * 4 + r], x[r], y, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) tm[bi * 16 + kg * 4 + r][bj * 16 + l16] = -y[r];
        }
        __syncthreads();
    }
    if constexpr (kBackward) put_square(tm, out.t + ch * 3 * kSquare);
    // column tile w of T (row tile w of T^T), plain and times Gam_63; above row 16 w it is zero
    bf16x8 tt[2][3], tg[2][3];
#pragma unroll
    for (int st = 0; st < 2; ++st) {
        alignas(16) float x[8];
        col8(tm, frow, st * 32 + kg * 8, x);
        split3(x, tt[st]);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= until[st * 32 + kg * 8 + j];
        split3(x, tg[st]);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) *reinterpret_cast<float4v*>(&gam[frow][m * 16 + kg * 4]) = pw[m];
    __syncthreads();
    scatter_turned<KS>(kw, turned, frow, kg);
    __syncthreads();
    // W = K^T diag(Gam_63) T, columns 16 w ..
    __bf16* wo = out.w + ch * 3 * KS * 32 * kC;
#pragma unroll
    for (int m = 0; m < KS * 2; ++m) {
        Acc3 x, y;
#pragma unroll
        for (int st = 0; st < 2; ++st)
            if (st == 1 || w < 2) {
                const bf16x8 kt = *reinterpret_cast<const bf16x8*>(turned + turned_at(m * 16 + l16, st * 4 + kg));
#pragma unroll
                for (int a = 0; a < 3; ++a) {
                    x.x[a] = mfma(tg[st][a], kt, x.x[a]);                    // W^T: lane = row of W
                    if (kBackward) y.x[a] = mfma(kt, tg[st][a], y.x[a]);     // W: lane = column of W
                }
            }
        put_turned<3>(wo, KS * 32 * kC, m, w, l16, kg, x.sum());
        if constexpr (kBackward) {
            bf16x4 part[3];
            split3(y.sum(), part);
            __bf16* o = out.wt + ch * 3 * KS * 32 * kC + ((m >> 1) * 4 + w) * kFrag + lane * 8 + (m & 1) * 4;
#pragma unroll
            for (int a = 0; a < 3; ++a) *reinterpret_cast<bf16x4*>(o + a * KS * 32 * kC) = part[a];
        }
    }
    // N = P T, columns 16 w ..
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if (m < w) {
            if (!kBackward && m >> 1 == w >> 1)              // inside a fragment that is read, above the diagonal
                put_turned<2>(out.n + ch * 2 * kSquare, kSquare, m, w, l16, kg, float4v{0.0f, 0.0f, 0.0f, 0.0f});
            if (kBackward && m >> 1 == w >> 1)
                put_turned<3>(out.nt + ch * 3 * kSquare, kSquare, w, m, l16, kg, float4v{0.0f, 0.0f, 0.0f, 0.0f});
            continue;
        }
        Acc3 x;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            if ((st == 0 && w >= 2) || (st == 1 && m < 2)) continue;
            alignas(16) float p8[8];
            bf16x8 p[3];
            row8(gam, m * 16 + l16, st * 32 + kg * 8, p8);
            split3(p8, p);
            const bf16x8(&t)[3] = tt[st];
            if constexpr (kBackward) {                       // N: lane = column of N
                x.x[0] = mfma(p[0], t[0], x.x[0]);
                x.x[1] = mfma(p[1], t[0], x.x[1]);
                x.x[2] = mfma(p[2], t[0], x.x[2]);
                x.x[1] = mfma(p[0], t[1], x.x[1]);
                x.x[2] = mfma(p[1], t[1], x.x[2]);
                x.x[2] = mfma(p[0], t[2], x.x[2]);
            } else {                                         // N^T: lane = row of N
                x.x[0] = mfma(t[0], p[0], x.x[0]);
                x.x[1] = mfma(t[0], p[1], x.x[1]);
                x.x[2] = mfma(t[1], p[0], x.x[2]);
            }
        }
        if constexpr (kBackward) put_turned<3>(out.nt + ch * 3 * kSquare, kSquare, w, m, l16, kg, x.sum());
        else put_turned<2>(out.n + ch * 2 * kSquare, kSquare, m, w, l16, kg, x.sum());
    }
    if constexpr (kBackward) {
        if (!first) return;
        put_turned_fragments<KS>(turned, out.kt + ck * KS * 32 * kC);
        __syncthreads();
        scatter_turned<KS>(qw, turned, frow, kg);
        __syncthreads();
        put_turned_fragments<KS>(turned, out.qt + ck * KS * 32 * kC);
    }
}

// ---------------------------------------------------------------------------
// The scan over chunks.  A workgroup owns 16 NT columns of one head's state;
// wavefronts 0..3 a slice of 32 state rows each, in FP32 registers, and of R one
// row tile of 16 tokens each.  State and R pass through LDS already split, in
// the order of right-hand fragments, so a fragment is one 16-byte read.
// ---------------------------------------------------------------------------
template <int NT, int K> struct Panel {              // [part][column][k], three bf16 parts
    alignas(16) __bf16 x[3][NT * 16][K + 8];
};

template <int NT, int K>
__device__ __forceinline__ void put_panel(Panel<NT, K>& p, int nt, int k4, int l16, float4v v) {
    bf16x4 part[3];
    split3(v, part);
#pragma unroll
    for (int a = 0; a < 3; ++a) *reinterpret_cast<bf16x4*>(&p.x[a][nt * 16 + l16][k4]) = part[a];
}
template <int NT, int K>
__device__ __forceinline__ bf16x8 get_panel(const Panel<NT, K>& p, int part, int nt, int step, int l16, int kg) {
    return *reinterpret_cast<const bf16x8*>(&p.x[part][nt * 16 + l16][step * 32 + kg * 8]);
}

__device__ __forceinline__ bf16x8 frag(const __bf16* m, int tile, int step, int lane) {
    return *reinterpret_cast<const bf16x8*>(m + (tile * 2 + step) * kFrag + lane * 8);
}

// The rows of a view that a chunk has, as a buffer: what lies behind the last one reads as zeros and is not
// written, so loads and stores need no condition.  Token strides are at most 2^23 elements, so 64 rows fit 2 GiB.
template <int kSize>
__device__ __forceinline__ rsrc_t chunk_rows(const nvfp4_rows& v, int b, int64_t t0, int h, int left, int dim) {
    const int64_t at = b * v.batch_stride + t0 * v.token_stride + h * v.head_stride;
    return make_rsrc(static_cast<uint8_t*>(v.data) + at * kSize, (uint64_t)(((left - 1) * v.token_stride + dim) * kSize));
}

// Four FP32 rows of a [64][dv] or [dk][dv] matrix (wave-uniform), one column per lane.
__device__ __forceinline__ void put_rows(float* m, int at, int dv, float4v x) {
#pragma unroll
    for (int r = 0; r < 4; ++r) m[(uint32_t)(at + r * dv)] = x[r];
}

constexpr int kScanThreads = 512;

// Workgroup ids go round-robin over the eight XCDs, each with its own L2.  All column slices of one head read the
// same keys, queries, T and P, so they take ids of one XCD: id = (head group * slices + slice) * 8 + head mod 8.
struct Place {
    int b, h, slice;
    bool any;
};
__device__ __forceinline__ Place place_of(const Shape& s, int slices) {
    const int id = blockIdx.x, at = id >> 3, head = at / slices * 8 + (id & 7);
    return Place{head / s.hv, head % s.hv, at % slices, head < s.batch * s.hv};
}

// The state as right-hand fragments [slice][part][column tile][lane][8], in the state's order.
template <int KS, int NT> struct StatePanel {
    alignas(16) __bf16 x[KS][3][NT][kFrag];
    __device__ __forceinline__ void put(const float4v (&S)[2][NT], int slice, int lane) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float v[8] = {S[0][n][0], S[0][n][1], S[0][n][2], S[0][n][3], S[1][n][0], S[1][n][1], S[1][n][2], S[1][n][3]};
            bf16x8 p[3];
            split3(v, p);
#pragma unroll
            for (int a = 0; a < 3; ++a) *reinterpret_cast<bf16x8*>(&x[slice][a][n][lane * 8]) = p[a];
        }
    }
    __device__ __forceinline__ bf16x8 get(int slice, int part, int n, int lane) const {
        return *reinterpret_cast<const bf16x8*>(&x[slice][part][n][lane * 8]);
    }
    // The FP32 values again (the three parts hold all of their bits), stored to a [dk][dv] matrix.
    __device__ __forceinline__ void store(float* m, int slice, int n, int lane, int cell, int dv) const {
        float v[8];
        const bf16x8 p0 = get(slice, 0, n, lane), p1 = get(slice, 1, n, lane), p2 = get(slice, 2, n, lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (float)p0[j] + ((float)p1[j] + (float)p2[j]);
#pragma unroll
        for (int j = 0; j < 8; ++j) m[(uint32_t)(cell + ((j & 4) * 4 + (j & 3)) * dv)] = v[j];
    }
};

// Wavefronts 0..3 carry the chain S0 -> R -> S'; wavefronts 4..7 bring V, finish the outputs, and store what the
// backward pass keeps, beside it.  Two barriers per chunk.  Every operand of the next chunk is loaded right behind
// its last use in this one, so that the chain waits for LDS and the matrix pipe only; for that the loads carry no
// condition (a branch around one makes the compiler wait for every younger load as well) and their addresses no
// arithmetic but a scalar step per chunk.  The two roles run loops of their own for the same reason.
// The outputs, rounded to bf16 in the end, take two parts of S0, N and R (2^-16).
//
// Measured, one sequence of 8192 tokens, 32 heads of 128 x 128 (256 workgroups of 16 columns): 252 us, 2.0 us a chunk,
// in which a workgroup reads 96 KB of operands (25 bytes a clock; a plain read out of the L2 gets 52).  Without the
// reads of W it would be 180 us, without any of the operands' 145: the chain's own products, LDS round trips and
// barriers.  Looking ahead into the L2 by a wavefront of its own, operands a chunk further ahead in a second set of
// registers, loads between the products and outputs stored a chunk later changed nothing or cost 3 to 5%.
//
// With 16 columns two workgroups may share a compute unit: 7 x 1001 tokens of 12 heads of 64 x 96 34 us, one alone 38.
//
// kSave: the forward pass inside the backward one, which keeps every chunk's first state and its R and computes no
// outputs.
template <int KS, int NT, bool kSave>
__global__ __launch_bounds__(kScanThreads) __attribute__((amdgpu_waves_per_eu(2, NT == 1 ? 4 : 2))) void gdn_scan_kernel(
    Shape s, nvfp4_rows v, const float* state, Prep prep, nvfp4_rows o, float* state_out, float* states, float* rs) {
    __shared__ StatePanel<KS, NT> ps;
    __shared__ Panel<NT, kC> pr;
    __shared__ alignas(16) float bv[2][NT * 16][kC + 4];      // beta V, two chunks
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3, row4 = w * 16 + kg * 4;
    const Place at = place_of(s, (s.dv + 16 * NT - 1) / (16 * NT));
    if (!at.any) return;
    const int h = at.h, b = at.b, hk = h / s.group, col0 = at.slice * 16 * NT + l16;
    const int len = seq_len(s, b), chunks = (len + kC - 1) / kC;
    const int64_t bh = (int64_t)b * s.hv + h, ch0 = bh * s.chunks, ck0 = ((int64_t)b * s.hk + hk) * s.chunks;
    const bool mine = w < KS;                        // a slice of the state
    const int slice = mine ? w : 0, scell = (slice * 32 + kg * 4) * s.dv + col0;
    bool in[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) in[n] = col0 + 16 * n < s.dv;
    const float* gates = prep.g + ch0 * kGates;
    if (wave < 4) {
        __builtin_amdgcn_s_setprio(2);
        float4v S[2][NT];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                S[i][n] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
                if (mine && state != nullptr && in[n]) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        S[i][n][r] = state[bh * s.dk * s.dv + scell + 16 * n + (16 * i + r) * s.dv];
                }
            }
        bf16x8 kx[KS], wf[2][2][3];
        float4v be, since;
        float whole;
        auto load_rows = [&](int c) {
#pragma unroll
            for (int i = 0; i < KS; ++i)
                kx[i] = *reinterpret_cast<const bf16x8*>(prep.kx + (ck0 + c) * KS * 32 * kC + (i * 4 + w) * kFrag + lane * 8);
            since = *reinterpret_cast<const float4v*>(gates + (int64_t)c * kGates + row4);
            be = *reinterpret_cast<const float4v*>(gates + (int64_t)c * kGates + 2 * kC + row4);
        };
        auto load_state = [&](int c) {
            whole = gates[(int64_t)c * kGates + kC - 1];
#pragma unroll
            for (int a = 0; a < 3; ++a)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int st = 0; st < 2; ++st)
                        wf[i][st][a] = frag(prep.w + ((ch0 + c) * 3 + a) * KS * 32 * kC, slice * 2 + i, st, lane);
        };
        if (chunks > 0) {
            load_rows(0);
            load_state(0);
        }
        for (int c = 0; c < chunks; ++c) {
            const int next = c + 1 < chunks ? c + 1 : c;
            if (mine) ps.put(S, slice, lane);
            __syncthreads();
            Acc3 x[NT];                              // R = beta V - beta gam K S0; beta is 0 behind the last token
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int a = 0; a < 3; ++a) x[n].x[a] = mfma(kx[i], ps.get(i, a, n, lane), x[n].x[a]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                put_panel(pr, n, row4, l16,
                          *reinterpret_cast<const float4v*>(&bv[c & 1][n * 16 + l16][row4]) - (be * since) * x[n].sum());
            load_rows(next);
            __syncthreads();
            if (mine) {                              // S' = gam_63 S0 + W R
                Acc3 acc[2][NT];
#pragma unroll
                for (int st = 0; st < 2; ++st)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const bf16x8 r0 = get_panel(pr, 0, n, st, l16, kg), r1 = get_panel(pr, 1, n, st, l16, kg),
                                     r2 = get_panel(pr, 2, n, st, l16, kg);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            Acc3& y = acc[i][n];
                            y.x[0] = mfma(wf[i][st][0], r0, y.x[0]);
                            y.x[1] = mfma(wf[i][st][1], r0, y.x[1]);
                            y.x[2] = mfma(wf[i][st][2], r0, y.x[2]);
                            y.x[1] = mfma(wf[i][st][0], r1, y.x[1]);
                            y.x[2] = mfma(wf[i][st][1], r1, y.x[2]);
                            y.x[2] = mfma(wf[i][st][0], r2, y.x[2]);
                        }
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n) S[i][n] = S[i][n] * whole + acc[i][n].sum();
            }
            load_state(next);
        }
        if (mine && state_out != nullptr) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (in[n]) put_rows(state_out + bh * s.dk * s.dv, scell + 16 * n + 16 * i * s.dv, s.dv, S[i][n]);
        }
    } else {
        bf16x8 qx[KS], nf[2][2];
        float4v since, be;
        uint16_t vv[NT][4];
        const uint32_t ostep = (uint32_t)o.token_stride * 2, ooff = (uint32_t)row4 * ostep + col0 * 2;
        const uint32_t vstep = (uint32_t)v.token_stride * 2, voff = (uint32_t)row4 * vstep + col0 * 2;
        auto load_values = [&](int c) {
            const int left = len - c * kC < kC ? len - c * kC : kC;
            const rsrc_t rv = chunk_rows<2>(v, b, (int64_t)c * kC, h, left, s.dv);
            be = *reinterpret_cast<const float4v*>(gates + (int64_t)c * kGates + 2 * kC + row4);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n) vv[n][r] = (uint16_t)bload2(rv, voff + 32 * n, r * vstep);
        };
        auto stage_values = [&](int c) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4v x = {bf16_f32(vv[n][0]), bf16_f32(vv[n][1]), bf16_f32(vv[n][2]), bf16_f32(vv[n][3])};
                *reinterpret_cast<float4v*>(&bv[c & 1][n * 16 + l16][row4]) = be * x;
            }
        };
        auto load_rows = [&](int c) {
            if (!kSave) {
                since = *reinterpret_cast<const float4v*>(gates + (int64_t)c * kGates + row4);
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    qx[i] = *reinterpret_cast<const bf16x8*>(prep.qx + (ck0 + c) * KS * 32 * kC + (i * 4 + w) * kFrag + lane * 8);
            }
        };
        auto load_square = [&](int c) {              // row tiles 0 and 1 end before the second k-step
            if (!kSave) {
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    nf[0][a] = frag(prep.n + ((ch0 + c) * 2 + a) * kSquare, w, 0, lane);
                    nf[1][a] = frag(prep.n + ((ch0 + c) * 2 + a) * kSquare, w, w >> 1, lane);
                }
            }
        };
        if (chunks > 0) {
            load_values(0);
            stage_values(0);
            load_values(chunks > 1 ? 1 : 0);
            load_rows(0);
            load_square(0);
        }
        for (int c = 0; c < chunks; ++c) {
            const int next = c + 1 < chunks ? c + 1 : c;
            __syncthreads();
            Acc3 y[NT];
            if (kSave) {
                if (mine) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (in[n]) ps.store(states + (ch0 + c) * s.dk * s.dv, slice, n, lane, scell + 16 * n, s.dv);
                }
            } else {                                 // scale gam Q S0
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int i = 0; i < KS; ++i)
#pragma unroll
                        for (int a = 0; a < 2; ++a) y[n].x[a] = mfma(qx[i], ps.get(i, a, n, lane), y[n].x[a]);
#pragma unroll
                    for (int a = 0; a < 2; ++a) y[n].x[a] *= since * s.scale;
                }
                load_rows(next);
            }
            __syncthreads();
            if (c + 1 < chunks) stage_values(c + 1);
            load_values(c + 2 < chunks ? c + 2 : chunks - 1);
            if (kSave) {                             // R^T, columns major, out of its parts
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float4v x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int a = 2; a >= 0; --a)
                        x += __builtin_convertvector(*reinterpret_cast<const bf16x4*>(&pr.x[a][n * 16 + l16][row4]), float4v);
                    if (in[n]) *reinterpret_cast<float4v*>(rs + ((ch0 + c) * s.dv + col0 + 16 * n) * kC + row4) = x;
                }
                continue;
            }
            const int left = len - c * kC < kC ? len - c * kC : kC;
            const rsrc_t ro = chunk_rows<2>(o, b, (int64_t)c * kC, h, left, s.dv);
#pragma unroll
            for (int n = 0; n < NT; ++n) {           // + N R
#pragma unroll
                for (int st = 0; st < 2; ++st)
                    if (st == 0 || w >= 2) {
                        const bf16x8 r0 = get_panel(pr, 0, n, st, l16, kg), r1 = get_panel(pr, 1, n, st, l16, kg);
                        y[n].x[0] = mfma(nf[st][0], r0, y[n].x[0]);
                        y[n].x[1] = mfma(nf[st][1], r0, y[n].x[1]);
                        y[n].x[2] = mfma(nf[st][0], r1, y[n].x[2]);
                    }
                const float4v z = y[n].sum();
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    __builtin_amdgcn_raw_buffer_store_b16((short)f32_to_bf16_rne(z[r]), ro,
                                                          (int)(in[n] ? ooff + 32 * n : kOutOfBounds), (int)(r * ostep), 0);
            }
            load_square(next);
        }
    }
}

// ---------------------------------------------------------------------------
// The scan back over the chunks: D, the gradient of a chunk's last state, from
// the last chunk to the first.  Keeps every chunk's D and dR for the gradients
// of q, k and the gates.  Wavefronts 0..3 carry the chain D -> dR -> D' as in
// the forward scan; wavefronts 4..7 add N^T dO, bring the next chunk's dO, and
// store D, dR and dV.  Measured, 4 x 2048 tokens of 16 heads of 128 x 128: 158 us
// with 32 columns (239 MB written, 245 read), 235 with 16; bound as the forward
// scan is.
// ---------------------------------------------------------------------------
template <int KS, int NT>
__global__ __launch_bounds__(kScanThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void gdn_scan_back_kernel(
    Shape s, Prep prep, nvfp4_rows d_o, const float* d_state_out, nvfp4_rows d_v, float* d_state, float* ds, float* drs) {
    __shared__ StatePanel<KS, NT> pd;
    __shared__ Panel<NT, kC> pe, po[2];                       // -beta gam dR; scale gam dO, two chunks
    __shared__ alignas(16) __bf16 dox[2][NT * 16][kC + 8];    // dO itself, exact
    __shared__ alignas(16) float pz[2][NT * 16][kC + 4];      // N^T dO
    __shared__ alignas(16) float pdr[NT * 16][kC + 4];        // dR
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3, row4 = w * 16 + kg * 4;
    const Place at = place_of(s, (s.dv + 16 * NT - 1) / (16 * NT));
    if (!at.any) return;
    const int h = at.h, b = at.b, hk = h / s.group, col0 = at.slice * 16 * NT + l16;
    const int len = seq_len(s, b), chunks = (len + kC - 1) / kC;
    const int64_t bh = (int64_t)b * s.hv + h, ch0 = bh * s.chunks, ck0 = ((int64_t)b * s.hk + hk) * s.chunks;
    const bool mine = w < KS;
    const int slice = mine ? w : 0, scell = (slice * 32 + kg * 4) * s.dv + col0;
    bool in[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) in[n] = col0 + 16 * n < s.dv;
    const float* gates = prep.g + ch0 * kGates;
    if (wave < 4) {
        __builtin_amdgcn_s_setprio(2);
        float4v D[2][NT];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                D[i][n] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
                if (mine && d_state_out != nullptr && in[n]) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        D[i][n][r] = d_state_out[bh * s.dk * s.dv + scell + 16 * n + (16 * i + r) * s.dv];
                }
            }
        bf16x8 wt[KS][3], kt[2][2], qt[2][2];
        float4v be, since;
        float whole;
        auto load_rows = [&](int c) {
#pragma unroll
            for (int a = 0; a < 3; ++a)
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    wt[i][a] = *reinterpret_cast<const bf16x8*>(prep.wt + ((ch0 + c) * 3 + a) * KS * 32 * kC + (i * 4 + w) * kFrag + lane * 8);
            since = *reinterpret_cast<const float4v*>(gates + (int64_t)c * kGates + row4);
            be = *reinterpret_cast<const float4v*>(gates + (int64_t)c * kGates + 2 * kC + row4);
        };
        auto load_state = [&](int c) {
            whole = gates[(int64_t)c * kGates + kC - 1];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    kt[i][st] = frag(prep.kt + (ck0 + c) * KS * 32 * kC, slice * 2 + i, st, lane);
                    qt[i][st] = frag(prep.qt + (ck0 + c) * KS * 32 * kC, slice * 2 + i, st, lane);
                }
        };
        if (chunks > 0) {
            load_rows(chunks - 1);
            load_state(chunks - 1);
        }
        __syncthreads();
        for (int c = chunks - 1; c >= 0; --c) {
            const int next = c > 0 ? c - 1 : 0;
            if (mine) pd.put(D, slice, lane);
            __syncthreads();
            Acc3 x[NT];                                       // dR
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const bf16x8 d0 = pd.get(i, 0, n, lane), d1 = pd.get(i, 1, n, lane), d2 = pd.get(i, 2, n, lane);
                    x[n].x[0] = mfma(wt[i][0], d0, x[n].x[0]);
                    x[n].x[1] = mfma(wt[i][1], d0, x[n].x[1]);
                    x[n].x[2] = mfma(wt[i][2], d0, x[n].x[2]);
                    x[n].x[1] = mfma(wt[i][0], d1, x[n].x[1]);
                    x[n].x[2] = mfma(wt[i][1], d1, x[n].x[2]);
                    x[n].x[2] = mfma(wt[i][0], d2, x[n].x[2]);
                }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4v y = x[n].sum() + *reinterpret_cast<const float4v*>(&pz[c & 1][n * 16 + l16][row4]);
                put_panel(pe, n, row4, l16, y * (be * since) * -1.0f);
                *reinterpret_cast<float4v*>(&pdr[n * 16 + l16][row4]) = y;
            }
            load_rows(next);
            __syncthreads();
            if (mine) {
                Acc3 acc[2][NT];
#pragma unroll
                for (int st = 0; st < 2; ++st)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int a = 0; a < 3; ++a) {
                            const bf16x8 e = get_panel(pe, a, n, st, l16, kg), d = get_panel(po[c & 1], a, n, st, l16, kg);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                acc[i][n].x[a] = mfma(qt[i][st], d, acc[i][n].x[a]);
                                acc[i][n].x[a] = mfma(kt[i][st], e, acc[i][n].x[a]);
                            }
                        }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n) D[i][n] = D[i][n] * whole + acc[i][n].sum();
            }
            load_state(next);
        }
        if (mine && d_state != nullptr) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (in[n]) put_rows(d_state + bh * s.dk * s.dv, scell + 16 * n + 16 * i * s.dv, s.dv, D[i][n]);
        }
    } else {
        float4v since, be;
        uint16_t d4[NT][4];
        bf16x8 nf[2][3];
        const uint32_t dstep = (uint32_t)d_o.token_stride * 2, doff = (uint32_t)row4 * dstep + col0 * 2;
        const uint32_t vstep = (uint32_t)d_v.token_stride * 2, voff = (uint32_t)row4 * vstep + col0 * 2;
        auto load_do = [&](int c) {
            const int left = len - c * kC < kC ? len - c * kC : kC;
            const rsrc_t rd = chunk_rows<2>(d_o, b, (int64_t)c * kC, h, left, s.dv);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n) d4[n][r] = (uint16_t)bload2(rd, doff + 32 * n, r * dstep);
            since = *reinterpret_cast<const float4v*>(gates + (int64_t)c * kGates + row4);
        };
        auto stage_do = [&](int c) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4v x = {bf16_f32(d4[n][0]), bf16_f32(d4[n][1]), bf16_f32(d4[n][2]), bf16_f32(d4[n][3])};
                *reinterpret_cast<bf16x4*>(&dox[c & 1][n * 16 + l16][row4]) = __builtin_convertvector(x, bf16x4);
                put_panel(po[c & 1], n, row4, l16, x * since * s.scale);
            }
        };
        auto load_square = [&](int c) {                       // N^T is upper triangular: row tiles 2 and 3 begin late
#pragma unroll
            for (int a = 0; a < 3; ++a) {
                nf[0][a] = frag(prep.nt + ((ch0 + c) * 3 + a) * kSquare, w, w >> 1, lane);
                nf[1][a] = frag(prep.nt + ((ch0 + c) * 3 + a) * kSquare, w, 1, lane);
            }
        };
        auto outer = [&](int c) {                             // N^T dO
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                Acc3 x;
#pragma unroll
                for (int st = 0; st < 2; ++st)
                    if (st == 1 || w < 2) {
                        const bf16x8 d = *reinterpret_cast<const bf16x8*>(&dox[c & 1][n * 16 + l16][st * 32 + kg * 8]);
#pragma unroll
                        for (int a = 0; a < 3; ++a) x.x[a] = mfma(nf[st][a], d, x.x[a]);
                    }
                *reinterpret_cast<float4v*>(&pz[c & 1][n * 16 + l16][row4]) = x.sum();
            }
        };
        if (chunks > 0) {
            load_do(chunks - 1);
            stage_do(chunks - 1);
            load_do(chunks > 1 ? chunks - 2 : 0);
            load_square(chunks - 1);
        }
        __syncthreads();                                      // dO of the last chunk is there for all of them
        if (chunks > 0) {
            outer(chunks - 1);
            load_square(chunks > 1 ? chunks - 2 : 0);
        }
        for (int c = chunks - 1; c >= 0; --c) {
            __syncthreads();
            if (mine) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (in[n]) pd.store(ds + (ch0 + c) * s.dk * s.dv, slice, n, lane, scell + 16 * n, s.dv);
            }
            if (c > 0) stage_do(c - 1);
            load_do(c > 1 ? c - 2 : 0);
            be = *reinterpret_cast<const float4v*>(gates + (int64_t)c * kGates + 2 * kC + row4);
            __syncthreads();
            if (c > 0) {
                outer(c - 1);
                load_square(c > 1 ? c - 2 : 0);
            }
            const int left = len - c * kC < kC ? len - c * kC : kC;
            const rsrc_t rv = chunk_rows<2>(d_v, b, (int64_t)c * kC, h, left, s.dv);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4v y = *reinterpret_cast<const float4v*>(&pdr[n * 16 + l16][row4]);
                if (in[n]) put_rows(drs + (ch0 + c) * kC * s.dv, row4 * s.dv + col0 + 16 * n, s.dv, y);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    __builtin_amdgcn_raw_buffer_store_b16((short)f32_to_bf16_rne(be[r] * y[r]), rv,
                                                          (int)(in[n] ? voff + 32 * n : kOutOfBounds), (int)(r * vstep), 0);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Gradients of q, k and the gates, chunk by chunk and all at once.  With
// U = T R, E = dR S0^T, F = dO S0^T, H = U D^T, dP = dO U^T, dA = -dR U^T:
//     Y_ij  = scale Gam_ij dP_ij (j <= i),   X_ij = beta_i Gam_ij dA_ij (j < i)
//     dQ    = scale gam F + Y K
//     dK    = Y^T Q + (X + X^T) K - beta gam E + Gam_63 H
//     dbeta = dR.V - gam k.E + sum_j Gam_ij dA_ij (k_i.k_j)
//     dlog alpha_t = sum over pairs j < t <= i of M_ij, the products of each decay with its gradient:
//         inside the chunk M = dP . P + dA . A, from the first state M_i0 = scale gam q.F - beta gam k.E,
//         to the last one M_Cj = Gam_63 k.H and M_C0 = gam_63 <D, S0>
// (sums of terms, no differences of long sums).  A workgroup of eight wavefronts takes a chunk of one key head
// and adds up its value heads in registers, so shared heads need no atomics and no second pass.  The products
// over v_dim go by slabs of 32: S0, D, dR, R and dO of a slab are split into LDS once for all wavefronts
// (wavefront w the row tile w mod 4 of the chunk and half of the columns of k_dim), while the next slab's
// values are on their way into registers.  Measured, 4 x 2048 tokens of 16 heads of 128 x 128: 255 to 280 us, 73
// thousand cycles a workgroup and chunk, 12 of them the first loads, 42 the slabs (products 12, the rest splitting,
// LDS and its barriers) and 17 the squares at the end; 676 MB read, 98 written.  Sixteen wavefronts instead of
// eight spill and take 700.
// ---------------------------------------------------------------------------
constexpr int kGradThreads = 512;
constexpr int kSlab = 32;

template <int kRows, int kCols> struct Slab {            // [part][row][k], three bf16 parts of an FP32 matrix
    alignas(16) __bf16 x[3][kRows][kCols + 8];
    __device__ __forceinline__ void put(int row, int k4, float4v v) {
        bf16x4 p[3];
        split3(v, p);
#pragma unroll
        for (int a = 0; a < 3; ++a) *reinterpret_cast<bf16x4*>(&x[a][row][k4]) = p[a];
    }
    __device__ __forceinline__ bf16x8 get(int part, int row, int k8) const {
        return *reinterpret_cast<const bf16x8*>(&x[part][row][k8]);
    }
    __device__ __forceinline__ void get3(int row, int k8, bf16x8 (&p)[3]) const {
#pragma unroll
        for (int a = 0; a < 3; ++a) p[a] = get(a, row, k8);
    }
};

// acc + A B over one k-step, both FP32 matrices in three parts: the six products of parts that reach 2^-24, smallest
// first; or A exact in bf16.
__device__ __forceinline__ float4v mfma6(const bf16x8 (&a)[3], const bf16x8 (&b)[3], float4v x) {
    x = mfma(a[0], b[2], x);
    x = mfma(a[1], b[1], x);
    x = mfma(a[2], b[0], x);
    x = mfma(a[0], b[1], x);
    x = mfma(a[1], b[0], x);
    return mfma(a[0], b[0], x);
}
__device__ __forceinline__ float4v mfma3(bf16x8 a, const bf16x8 (&b)[3], float4v x) {
    x = mfma(a, b[2], x);
    x = mfma(a, b[1], x);
    return mfma(a, b[0], x);
}
template <int kCtrl> __device__ __forceinline__ float lane_move(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), kCtrl, 0xf, 0xf, true));
}
// The sum over the 16 lanes of a group, in every lane: neighbours, pairs, then the mirrored half and row.
__device__ __forceinline__ float sum16(float x) {
    x += lane_move<0xB1>(x);                              // quad_perm [1,0,3,2]
    x += lane_move<0x4E>(x);                              // quad_perm [2,3,0,1]
    x += lane_move<0x141>(x);                             // row_half_mirror
    return x + lane_move<0x140>(x);                       // row_mirror
}

// Four bf16 of a row, from an 8-byte aligned place if `wide`, else a 2-byte aligned one.
__device__ __forceinline__ uint2 load_row4(rsrc_t r, uint32_t at, bool wide) {
    if (wide) return bload8(r, at, 0);
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = bload2(r, at == kOutOfBounds ? at : at + 2 * i, 0);
    return make_uint2(x[0] | x[1] << 16, x[2] | x[3] << 16);
}

// One buffer load that writes LDS: lane l's 16 bytes land at lds + 16 l; lds is the wavefront's.
__device__ __forceinline__ void load_lds16(rsrc_t r, void* lds, uint32_t at) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, (int)at, 0, 0, 0);
}

template <int KS>
__global__ __launch_bounds__(kGradThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void gdn_grad_kernel(
    Shape s, nvfp4_rows q, nvfp4_rows k, nvfp4_rows v, nvfp4_rows alpha, nvfp4_rows beta, Prep prep, const float* states,
    const float* rs, const float* ds, const float* drs, nvfp4_rows d_o, nvfp4_rows d_q, nvfp4_rows d_k,
    nvfp4_rows d_log_alpha, nvfp4_rows d_beta, int wide) {
    constexpr int DK = KS * 32;
    struct Slabs {
        Slab<DK, kSlab> s0, d;
        Slab<kC, kSlab> dr, u;
        Slab<kSlab, kC> rt;                               // R^T
        alignas(16) __bf16 dox[kC][kSlab + 8];
    };
    struct Squares {
        alignas(16) float y[kC][kLd], x[kC][kLd], m[kC][kLd];
        alignas(16) __bf16 k[kC][DK + 8], q[kC][DK + 8];
        alignas(16) __bf16 turned[2][KS * 4 * kFrag];     // fragments of K^T and Q^T
    };
    union Shared {
        Slabs a;
        Squares b;
    };
    __shared__ Shared sh;
    __shared__ alignas(16) float gam[kC][kLd];
    __shared__ alignas(16) float be[kC], since[kC];
    __shared__ alignas(16) float al[kC], db[2][kC], m_in[2][kC], m_out[2][kC];
    __shared__ float vdot[kC], corner[8], pair_sum[8][kC];
    const int c = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
    const int64_t t0 = (int64_t)c * kC;
    const int len = seq_len(s, b) - c * kC;
    if (len <= 0) return;
    const int left = len < kC ? len : kC;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave & 3, half = wave >> 2;
    const int64_t ck = ((int64_t)b * s.hk + hk) * s.chunks + c;
    const rsrc_t rkt = make_rsrc(prep.kt + ck * DK * kC, DK * kC * 2), rqt = make_rsrc(prep.qt + ck * DK * kC, DK * kC * 2);
    // K and Q rows behind the last token read as zeros
    const rsrc_t rk = chunk_rows<2>(k, b, t0, hk, left, DK), rq = chunk_rows<2>(q, b, t0, hk, left, DK);
    const uint32_t kstep = (uint32_t)k.token_stride * 2, qstep = (uint32_t)q.token_stride * 2;
    float4v dq[KS], dk[KS];                               // column tiles half * KS ..
#pragma unroll
    for (int i = 0; i < KS; ++i) dq[i] = dk[i] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    const int slabs = (s.dv + kSlab - 1) / kSlab;
    for (int head = 0; head < s.group; ++head) {
        // the places that follow from the thread's number are worked out anew for each head: kept over the loop they
        // take more registers than there are
        int tid = threadIdx.x;
        asm("" : "+v"(tid));
        const int lane = tid & 63, l16 = lane & 15, kg = lane >> 4, row4 = w * 16 + kg * 4, frow = w * 16 + l16;
        const int h = hk * s.group + head;
        const int64_t ch = ((int64_t)b * s.hv + h) * s.chunks + c;
        const uint32_t sbytes = DK * s.dv * 4, rbytes = kC * s.dv * 4;
        const rsrc_t rs0 = make_rsrc(states + ch * DK * s.dv, sbytes), rdd = make_rsrc(ds + ch * DK * s.dv, sbytes);
        const rsrc_t rr = make_rsrc(rs + ch * kC * s.dv, rbytes), rdr = make_rsrc(drs + ch * kC * s.dv, rbytes);   // [dv][64], [64][dv]
        const rsrc_t rv = chunk_rows<2>(v, b, t0, h, left, s.dv), rd = chunk_rows<2>(d_o, b, t0, h, left, s.dv);
        __syncthreads();
        if (tid < kC) {
            al[tid] = tid < left ? *row_ptr<const float>(alpha, b, t0 + tid, h) : 1.0f;
            be[tid] = tid < left ? *row_ptr<const float>(beta, b, t0 + tid, h) : 0.0f;
        }
        // what a thread brings of a slab: 4 columns of rows tid / 8 (+ 64) of S0 and D, of dR, dO and V; 4 tokens of
        // row tid / 16 of R^T
        constexpr int SR = (DK + 63) / 64;
        float4v gs[SR], gd[SR], gr, gt;
        uint2 go, gv;
        const int r8 = tid >> 3, c4 = (tid & 7) * 4, r16 = tid >> 4, k4 = (tid & 15) * 4;
        const uint32_t orow = (uint32_t)r8 * (uint32_t)d_o.token_stride * 2, vrow = (uint32_t)r8 * (uint32_t)v.token_stride * 2;
        auto load_slab = [&](int j) {
            const int col = j * kSlab + c4, rrow = j * kSlab + r16;
            const bool there = col < s.dv;                // v_dim is a multiple of 16
#pragma unroll
            for (int i = 0; i < SR; ++i) {                // rows behind DK read as zeros
                const uint32_t at = there ? ((r8 + 64 * i) * s.dv + col) * 4 : kOutOfBounds;
                gs[i] = __builtin_bit_cast(float4v, bload16(rs0, at, 0));
                gd[i] = __builtin_bit_cast(float4v, bload16(rdd, at, 0));
            }
            gr = __builtin_bit_cast(float4v, bload16(rdr, there ? (r8 * s.dv + col) * 4 : kOutOfBounds, 0));
            gt = __builtin_bit_cast(float4v, bload16(rr, rrow < s.dv ? (rrow * kC + k4) * 4 : kOutOfBounds, 0));
            go = load_row4(rd, there ? orow + col * 2 : kOutOfBounds, wide);
            gv = load_row4(rv, there ? vrow + col * 2 : kOutOfBounds, wide);
        };
        load_slab(0);
        bf16x8 t3[2][3];                                  // T, row tile w
#pragma unroll
        for (int a = 0; a < 3; ++a) {
            t3[0][a] = frag(prep.t + (ch * 3 + a) * kSquare, w, 0, lane);
            if (w >= 2) t3[1][a] = frag(prep.t + (ch * 3 + a) * kSquare, w, 1, lane);
            else t3[1][a] = bf16x8{};
        }
        // pieces of 16 bytes of the rows of K and Q
        constexpr int kPieces = kC * DK / 8, PT = (kPieces + kGradThreads - 1) / kGradThreads;
        uint4 pk[PT], pq[PT];
        __syncthreads();
        if (half == 0) chunk_decays(al, gam, since, w);
        float4v dp[2] = {}, da[2] = {};                   // column tiles 2 half, 2 half + 1
        float4v e[KS], f[KS], hh[KS];
#pragma unroll
        for (int i = 0; i < KS; ++i) e[i] = f[i] = hh[i] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
        float vsum = 0.0f, csum = 0.0f;
        for (int j = 0; j < slabs; ++j) {
            __syncthreads();                              // the slab before this one is done with
#pragma unroll
            for (int i = 0; i < SR; ++i)
                if (r8 + 64 * i < DK) {
                    sh.a.s0.put(r8 + 64 * i, c4, gs[i]);
                    sh.a.d.put(r8 + 64 * i, c4, gd[i]);
                    csum += (gs[i][0] * gd[i][0] + gs[i][1] * gd[i][1]) + (gs[i][2] * gd[i][2] + gs[i][3] * gd[i][3]);
                }
            sh.a.dr.put(r8, c4, gr);
            sh.a.rt.put(r16, k4, gt);
            *reinterpret_cast<uint2*>(&sh.a.dox[r8][c4]) = go;
            vsum += (gr[0] * bf16_f32((uint16_t)gv.x) + gr[1] * bf16_f32((uint16_t)(gv.x >> 16))) +
                    (gr[2] * bf16_f32((uint16_t)gv.y) + gr[3] * bf16_f32((uint16_t)(gv.y >> 16)));
            if (j + 1 < slabs) load_slab(j + 1);
            else {
#pragma unroll
                for (int i = 0; i < PT; ++i) {
                    const int at = tid + i * kGradThreads;
                    const uint32_t row = at / (DK / 8), col = at % (DK / 8) * 16;
                    pk[i] = bload16(rk, at < kPieces ? row * kstep + col : kOutOfBounds, 0);
                    pq[i] = bload16(rq, at < kPieces ? row * qstep + col : kOutOfBounds, 0);
                }
            }
            __syncthreads();
            {                                             // U^T: rows 16 half .. of the slab, tokens of row tile w
                float4v u = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int st = 0; st < 2; ++st)
                    if (st == 0 || w >= 2) {
                        bf16x8 r3[3];
                        sh.a.rt.get3(half * 16 + l16, st * 32 + kg * 8, r3);
                        u = mfma6(r3, t3[st], u);
                    }
                sh.a.u.put(frow, half * 16 + kg * 4, u);
            }
            bf16x8 r3[3];
            sh.a.dr.get3(frow, kg * 8, r3);
            const bf16x8 o1 = *reinterpret_cast<const bf16x8*>(&sh.a.dox[frow][kg * 8]);
#pragma unroll
            for (int n = 0; n < KS; ++n) {                // E and F
                bf16x8 s3[3];
                sh.a.s0.get3((half * KS + n) * 16 + l16, kg * 8, s3);
                e[n] = mfma6(r3, s3, e[n]);
                f[n] = mfma3(o1, s3, f[n]);
            }
            __syncthreads();
            bf16x8 u3[3];
            sh.a.u.get3(frow, kg * 8, u3);
#pragma unroll
            for (int n = 0; n < KS; ++n) {                // H
                bf16x8 d3[3];
                sh.a.d.get3((half * KS + n) * 16 + l16, kg * 8, d3);
                hh[n] = mfma6(u3, d3, hh[n]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {                 // dP and dR U^T
                const int m = half * 2 + i;
                if (m <= w) {
                    sh.a.u.get3(m * 16 + l16, kg * 8, u3);
                    dp[i] = mfma3(o1, u3, dp[i]);
                    da[i] = mfma6(r3, u3, da[i]);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KS; ++i) {                    // for the last products
            const int f = w * KS + i;
            load_lds16(half == 0 ? rkt : rqt, sh.b.turned[half] + f * kFrag, f * kFrag * 2 + lane * 16);
        }
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            const int at = tid + i * kGradThreads;
            if (at < kPieces) {
                *reinterpret_cast<uint4*>(&sh.b.k[at / (DK / 8)][at % (DK / 8) * 8]) = pk[i];
                *reinterpret_cast<uint4*>(&sh.b.q[at / (DK / 8)][at % (DK / 8) * 8]) = pq[i];
            }
        }
        __syncthreads();
        // <D, S0> and dR . V
        csum = sum16(csum);
        csum += __shfl_xor(csum, 16, 64);
        csum += __shfl_xor(csum, 32, 64);
        if (lane == 0) corner[wave] = csum;
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) vsum += __shfl_xor(vsum, off, 64);
        if ((tid & 7) == 0) vdot[r8] = vsum;
        const float4v sn = *reinterpret_cast<const float4v*>(&since[row4]);
        const float4v bt = *reinterpret_cast<const float4v*>(&be[row4]);
        const float4v un = *reinterpret_cast<const float4v*>(&gam[kC - 1][row4]);
        float4v beta_sum = {0.0f, 0.0f, 0.0f, 0.0f}, in_sum = beta_sum, out_sum = beta_sum;
        // Y, X and M: the 16 x 16 tiles of row tile w
        bf16x8 kf[KS], qf[KS];
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            kf[i] = *reinterpret_cast<const bf16x8*>(&sh.b.k[frow][i * 32 + kg * 8]);
            qf[i] = *reinterpret_cast<const bf16x8*>(&sh.b.q[frow][i * 32 + kg * 8]);
        }
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
            const int m = half * 2 + i2;
            float4v gg = {0.0f, 0.0f, 0.0f, 0.0f}, zz = gg;
            if (m <= w) {
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    const bf16x8 x = *reinterpret_cast<const bf16x8*>(&sh.b.k[m * 16 + l16][i * 32 + kg * 8]);
                    gg = mfma(kf[i], x, gg);
                    zz = mfma(qf[i], x, zz);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = row4 + r, j = m * 16 + l16;
                const float d = j <= i ? gam[i][j] : 0.0f, lower = j < i ? d : 0.0f;
                const float yij = s.scale * (d * dp[i2][r]);
                const float a = -da[i2][r] * lower;          // Gam dA
                sh.b.y[i][j] = yij;
                sh.b.x[i][j] = bt[r] * a;
                sh.b.m[i][j] = j < i ? yij * zz[r] + bt[r] * (a * gg[r]) : 0.0f;
                beta_sum[r] += a * gg[r];
            }
        }
        // what E, F and H add
#pragma unroll
        for (int n = 0; n < KS; ++n) {
            const int col = (half * KS + n) * 16 + l16;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float kv = (float)sh.b.k[row4 + r][col];
                const float qv = (float)sh.b.q[row4 + r][col];
                const float ge = sn[r] * e[n][r], gf = s.scale * sn[r] * f[n][r], gh = un[r] * hh[n][r];
                dq[n][r] += gf;
                dk[n][r] += gh - bt[r] * ge;
                beta_sum[r] -= ge * kv;
                in_sum[r] += gf * qv - bt[r] * ge * kv;
                out_sum[r] += gh * kv;
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            beta_sum[r] = sum16(beta_sum[r]);
            in_sum[r] = sum16(in_sum[r]);
            out_sum[r] = sum16(out_sum[r]);
        }
        if (l16 == 0) {
            *reinterpret_cast<float4v*>(&db[half][row4]) = beta_sum;
            *reinterpret_cast<float4v*>(&m_in[half][row4]) = in_sum;
            *reinterpret_cast<float4v*>(&m_out[half][row4]) = out_sum;
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);               // vmcnt(0): the loads into LDS
        __syncthreads();
        // sums over the pairs j < t <= i: prefixes along the rows of M (eight threads a row), then down a column
        {
            const int j8 = (tid & 7) * 8;
            float x[8], sum = 0.0f;
            row8(sh.b.m, r8, j8, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float y = x[j];
                x[j] = sum;
                sum += y;
            }
            float before = sum;                           // of the segments up to this one
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) {
                const float o = __shfl_up(before, off, 64);
                before += (tid & 7) >= off ? o : 0.0f;
            }
            before = __shfl_up(before, 1, 64);
            if ((tid & 7) == 0) before = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] += before;
            *reinterpret_cast<float4v*>(&sh.b.m[r8][j8]) = float4v{x[0], x[1], x[2], x[3]};
            *reinterpret_cast<float4v*>(&sh.b.m[r8][j8 + 4]) = float4v{x[4], x[5], x[6], x[7]};
        }
        // dQ += Y K;  dK += Y^T Q + (X + X^T) K
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            bf16x8 fy[3], ft[3], fx[3];
            alignas(16) float a8[8], t8[8], x8[8], c8[8];
            row8(sh.b.y, frow, st * 32 + kg * 8, a8);
            col8(sh.b.y, frow, st * 32 + kg * 8, t8);
            row8(sh.b.x, frow, st * 32 + kg * 8, x8);
            col8(sh.b.x, frow, st * 32 + kg * 8, c8);
#pragma unroll
            for (int j = 0; j < 8; ++j) x8[j] += c8[j];
            split3(a8, fy);
            split3(t8, ft);
            split3(x8, fx);
#pragma unroll
            for (int n = 0; n < KS; ++n) {
                const bf16x8 kt = frag(sh.b.turned[0], half * KS + n, st, lane);
                const bf16x8 qt = frag(sh.b.turned[1], half * KS + n, st, lane);
#pragma unroll
                for (int p = 2; p >= 0; --p) {
                    dq[n] = mfma(fy[p], kt, dq[n]);
                    dk[n] = mfma(ft[p], qt, dk[n]);
                    dk[n] = mfma(fx[p], kt, dk[n]);
                }
            }
        }
        __syncthreads();
        {                                                 // rows 8 wave .., column `lane`
            float t = 0.0f;
            alignas(16) float in0[8], in1[8], out0[8], out1[8];
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                *reinterpret_cast<float4v*>(in0 + i) = *reinterpret_cast<const float4v*>(&m_in[0][wave * 8 + i]);
                *reinterpret_cast<float4v*>(in1 + i) = *reinterpret_cast<const float4v*>(&m_in[1][wave * 8 + i]);
                *reinterpret_cast<float4v*>(out0 + i) = *reinterpret_cast<const float4v*>(&m_out[0][wave * 8 + i]);
                *reinterpret_cast<float4v*>(out1 + i) = *reinterpret_cast<const float4v*>(&m_out[1][wave * 8 + i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                t += wave * 8 + i >= lane ? sh.b.m[wave * 8 + i][lane] + (in0[i] + in1[i]) : out0[i] + out1[i];
            pair_sum[wave][lane] = t;
        }
        __syncthreads();
        if (wave == 0 && lane < left) {
            float t = since[kC - 1] * (((corner[0] + corner[1]) + (corner[2] + corner[3])) +
                                       ((corner[4] + corner[5]) + (corner[6] + corner[7])));
#pragma unroll
            for (int i = 0; i < 8; ++i) t += pair_sum[i][lane];
            *row_ptr<float>(d_log_alpha, b, t0 + lane, h) = t;
            *row_ptr<float>(d_beta, b, t0 + lane, h) = vdot[lane] + (db[0][lane] + db[1][lane]);
        }
    }
    const int l16 = threadIdx.x & 15, row4 = w * 16 + (threadIdx.x >> 4 & 3) * 4;
    const rsrc_t oq = chunk_rows<2>(d_q, b, t0, hk, left, DK), ok = chunk_rows<2>(d_k, b, t0, hk, left, DK);
    const uint32_t dqs = (uint32_t)d_q.token_stride * 2, dks = (uint32_t)d_k.token_stride * 2;
#pragma unroll
    for (int n = 0; n < KS; ++n) {
        const uint32_t col = ((half * KS + n) * 16 + l16) * 2;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            __builtin_amdgcn_raw_buffer_store_b16((short)f32_to_bf16_rne(dq[n][r]), oq, (int)((row4 + r) * dqs + col), 0, 0);
            __builtin_amdgcn_raw_buffer_store_b16((short)f32_to_bf16_rne(dk[n][r]), ok, (int)((row4 + r) * dks + col), 0, 0);
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

Shape shape_of(const nvfp4_gdn& g) {
    Shape s{};
    s.tokens = g.tokens;
    s.batch = (int32_t)g.batch;
    s.hk = g.k_heads;
    s.hv = g.v_heads;
    s.group = g.v_heads / g.k_heads;
    s.dk = g.k_dim;
    s.dv = g.v_dim;
    s.chunks = (int32_t)((g.tokens + kC - 1) / kC);
    s.scale = g.scale;
    s.lens = g.lens;
    return s;
}

// The parts of a workspace, each 256-byte aligned.
struct Layout {
    size_t bytes = 0;
    size_t take(size_t n) {
        const size_t at = bytes;
        bytes += (n + 255) / 256 * 256;
        return at;
    }
};
struct Work {
    Prep prep;
    float *states, *rs, *ds, *drs;
    size_t bytes;
};

Work work_of(const Shape& s, bool backward, void* base) {
    Layout l;
    const size_t ch = (size_t)s.batch * s.hv * s.chunks, ck = (size_t)s.batch * s.hk * s.chunks;
    const size_t state = ch * s.dk * s.dv * 4, rows = ch * kC * s.dv * 4, key = ck * s.dk * kC * 2;
    const uintptr_t p = reinterpret_cast<uintptr_t>(base);           // NULL where only the size is asked for
    Work w{};
    auto part = [&](size_t n) { return reinterpret_cast<__bf16*>(p + l.take(n)); };
    auto real = [&](size_t n) { return reinterpret_cast<float*>(p + l.take(n)); };
    w.prep.w = part(ch * 3 * s.dk * kC * 2);
    w.prep.kx = part(key);
    w.prep.g = real(ch * kGates * 4);
    if (!backward) {
        w.prep.qx = part(key);
        w.prep.n = part(ch * 2 * kSquare * 2);
    } else {
        w.prep.wt = part(ch * 3 * s.dk * kC * 2);
        w.prep.nt = part(ch * 3 * kSquare * 2);
        w.prep.t = part(ch * 3 * kSquare * 2);
        w.prep.kt = part(key);
        w.prep.qt = part(key);
        w.states = real(state);
        w.rs = real(rows);
        w.ds = real(state);
        w.drs = real(rows);
    }
    w.bytes = l.bytes;
    return w;
}

// Whether the rows of a bf16 view start on 8-byte boundaries: then the gradients read v and dO four at a time (backward
// pass of 4 x 2048 tokens of 16 heads of 128 x 128 609 us, one at a time 641).
bool on8(const nvfp4_rows& r) {
    return reinterpret_cast<uintptr_t>(r.data) % 8 == 0 && r.batch_stride % 4 == 0 && r.token_stride % 4 == 0 &&
           r.head_stride % 4 == 0;
}

dim3 scan_grid(const Shape& s, int columns) {
    return dim3((unsigned)(((int64_t)s.batch * s.hv + 7) / 8 * 8 * ((s.dv + columns - 1) / columns)));
}

// 32 state columns per workgroup where that still gives every compute unit one, else 16.  Forward, 32 heads of
// 128 x 128: 4 sequences of 2048 tokens 271 us with 32 columns, 315 with 16; one of 8192 409 and 343.
bool wide_columns(const Shape& s) {
    return (int64_t)s.batch * s.hv * ((s.dv + 31) / 32) >= kComputeUnits;
}

template <int KS>
void forward_chunks(const nvfp4_gdn& g, const Shape& s, const Work& w, const nvfp4_rows& o, float* state_out,
                    hipStream_t stream) {
    hipLaunchKernelGGL((gdn_prep_kernel<KS, false>), dim3(s.chunks, s.hv, s.batch), dim3(kThreads), 0, stream, s, g.q,
                       g.k, g.alpha, g.beta, w.prep);
    if (wide_columns(s))
        hipLaunchKernelGGL((gdn_scan_kernel<KS, 2, false>), scan_grid(s, 32), dim3(kScanThreads), 0,
                           stream, s, g.v, g.state, w.prep, o, state_out, nullptr, nullptr);
    else
        hipLaunchKernelGGL((gdn_scan_kernel<KS, 1, false>), scan_grid(s, 16), dim3(kScanThreads), 0,
                           stream, s, g.v, g.state, w.prep, o, state_out, nullptr, nullptr);
}

template <int KS>
void backward_chunks(const nvfp4_gdn& g, const Shape& s, const Work& w, const GdnGrads& d, hipStream_t stream) {
    const dim3 block(kThreads);
    if (s.chunks > 0)                     // no tokens: the scans still carry the state's gradient through
        hipLaunchKernelGGL((gdn_prep_kernel<KS, true>), dim3(s.chunks, s.hv, s.batch), block, 0, stream, s, g.q, g.k,
                       g.alpha, g.beta, w.prep);
    if (wide_columns(s)) {
        const dim3 grid = scan_grid(s, 32);
        hipLaunchKernelGGL((gdn_scan_kernel<KS, 2, true>), grid, dim3(kScanThreads), 0, stream, s, g.v, g.state,
                           w.prep, nvfp4_rows{}, nullptr, w.states, w.rs);
        hipLaunchKernelGGL((gdn_scan_back_kernel<KS, 2>), grid, dim3(kScanThreads), 0, stream, s, w.prep, d.d_o,
                           d.d_state_out, d.d_v, d.d_state, w.ds, w.drs);
    } else {
        const dim3 grid = scan_grid(s, 16);
        hipLaunchKernelGGL((gdn_scan_kernel<KS, 1, true>), grid, dim3(kScanThreads), 0, stream, s, g.v, g.state,
                           w.prep, nvfp4_rows{}, nullptr, w.states, w.rs);
        hipLaunchKernelGGL((gdn_scan_back_kernel<KS, 1>), grid, dim3(kScanThreads), 0, stream, s, w.prep, d.d_o,
                           d.d_state_out, d.d_v, d.d_state, w.ds, w.drs);
    }
    if (s.chunks > 0)
        hipLaunchKernelGGL((gdn_grad_kernel<KS>), dim3(s.chunks, s.hk, s.batch), dim3(kGradThreads), 0, stream, s, g.q, g.k,
                           g.v, g.alpha, g.beta, w.prep, w.states, w.rs, w.ds, w.drs, d.d_o, d.d_q, d.d_k, d.d_log_alpha,
                           d.d_beta, on8(g.v) && on8(d.d_o));
}

bool by_steps(const nvfp4_gdn& g) { return g.tokens <= kStepTokens; }

}  // namespace

size_t gdn_forward_workspace_bytes(const nvfp4_gdn& g) {
    return by_steps(g) ? 0 : work_of(shape_of(g), false, nullptr).bytes;
}
size_t gdn_backward_workspace_bytes(const nvfp4_gdn& g) { return work_of(shape_of(g), true, nullptr).bytes; }

hipError_t launch_gdn_forward(const nvfp4_gdn& g, const nvfp4_rows& o, float* state_out, void* workspace,
                              hipStream_t stream) {
    const Shape s = shape_of(g);
    if (by_steps(g)) {
        hipLaunchKernelGGL(gdn_step_kernel, dim3((s.dv + 31) / 32, s.hv, s.batch), dim3(kThreads), 0, stream, s,
                           g.q, g.k, g.v, g.alpha, g.beta, g.state, o, state_out);
        return hipGetLastError();
    }
    const Work w = work_of(s, false, workspace);
    switch (s.dk / 32) {
        case 1: forward_chunks<1>(g, s, w, o, state_out, stream); break;
        case 2: forward_chunks<2>(g, s, w, o, state_out, stream); break;
        case 3: forward_chunks<3>(g, s, w, o, state_out, stream); break;
        default: forward_chunks<4>(g, s, w, o, state_out, stream); break;
    }
    return hipGetLastError();
}

hipError_t launch_gdn_backward(const nvfp4_gdn& g, const GdnGrads& d, void* workspace, hipStream_t stream) {
    const Shape s = shape_of(g);
    const Work w = work_of(s, true, workspace);
    switch (s.dk / 32) {
        case 1: backward_chunks<1>(g, s, w, d, stream); break;
        case 2: backward_chunks<2>(g, s, w, d, stream); break;
        case 3: backward_chunks<3>(g, s, w, d, stream); break;
        default: backward_chunks<4>(g, s, w, d, stream); break;
    }
    return hipGetLastError();
}

}  // namespace nvfp4
