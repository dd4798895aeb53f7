// Layers with 4-bit weights and group scales (sm_100a): launchers and the product of packed
// rows with activation columns that the matrix product and the expert layer share.
//
// Format.  Row i of W (m x n) holds its codes q in ld = 4 ceil(n / 32) 32-bit words, code of
// column k in nibble k % 8 (lowest first) of word k / 8, and per group of g consecutive
// columns (g = 32, 64, 128) a BF16 scale s and, where the layer has them, a zero point z
// (else z = 8):  W^_ik = s (q_ik - z).  Rows are 16-byte aligned whatever n is.
#pragma once
#include "common.cuh"

namespace nq {
namespace w4 {

constexpr int64_t kMaxRows = 1 << 24;   // rows of one packed array (stacked experts included)

inline int64_t row_words(int64_t n) { return 4 * ceil_div(n, 32); }
inline int64_t row_groups(int64_t n, int g) { return ceil_div(n, g); }

// One packed matrix (or a stack of them, rows one after the other).
struct Mat {
    const uint32_t *q;
    const __nv_bfloat16 *s;
    const uint8_t *z;      // or null: every zero point is 8
    int n, ld, ng;         // columns, words and groups of a row
};

// Activation columns of the product: BF16 vectors of length n, ``stride`` elements apart.
// FP32 activations are carried as kTerms BF16 columns each, x = x_0 + x_1 + x_2 exactly
// (3 x 8 significant bits), so that their products with the integers q - z are exact.
constexpr int kTerms = 3;

// ---------------------------------------------------------------------------------
// Device: rows x columns product on mma.sync.m16n8k16 (BF16, FP32 accumulation)
// ---------------------------------------------------------------------------------
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes i and i + 4 of a word as BF16 pair (q_i - z, q_{i+4} - z).  A code in the low bits
// of the mantissa of 128.0 (ulp 1) is 128 + q; ``bias`` holds 128 + z twice.  Exact.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i, uint32_t bias) {
    uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&bias));
    return *reinterpret_cast<const uint32_t *>(&d);
}

__device__ __forceinline__ uint32_t zero_bias(uint32_t z) { return (0x4300u | (z & 15u)) * 0x10001u; }

template <int VW>
__device__ __forceinline__ void load_words(uint32_t (&w)[VW], const uint32_t *p) {
    if constexpr (VW == 1) {
        w[0] = __ldg(p);
    } else if constexpr (VW == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x, w[1] = v.y;
    } else {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
}

// Eight consecutive activations x[k .. k + 7] of one column, zero from n on.
__device__ __forceinline__ uint4 load_x8(const __nv_bfloat16 *x, int k, int n, bool vec) {
    if (vec) return k < n ? *reinterpret_cast<const uint4 *>(x + k) : make_uint4(0, 0, 0, 0);
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        h[i] = k + i < n ? reinterpret_cast<const unsigned short *>(x)[k + i] : 0;
    return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}

// acc[mt][nt] += W^ rows x columns over groups grp0, grp0 + step, ... < ng, for one warp.
// The A fragment of an MMA is 16 rows of W (lane: rows lane/4 and lane/4 + 8), the B
// fragment 8 columns (lane: column lane/4), so any order of the k axis serves as long as
// both sides use it: lane%4 = t takes VW = g/32 consecutive words of a row, words
// t VW .. t VW + VW - 1 of a group, so a group is 2 VW MMAs of exactly its own columns and
// its sum is scaled once, in FP32.  Integers and BF16 activations multiply exactly.
// row[mt][h]: row (lane/4 + 8h of tile mt) as a row index of M, clamped by the caller;
// col[nt]: the lane's column of n-tile nt, or null for a column that is not there.
template <int VW, int MT, int NT>
__device__ __forceinline__ void group_products(float (&acc)[MT][NT][4], const Mat &M,
                                               const int64_t (&row)[MT][2],
                                               const __nv_bfloat16 *const (&col)[NT], bool xvec,
                                               int grp0, int step) {
    const int t = threadIdx.x & 3;
    constexpr int U = VW == 4 ? 2 : 4;     // groups in flight per lane
    for (int gr = grp0; gr < M.ng; gr += U * step) {
        uint32_t w[U][MT][2][VW];
        float s[U][MT][2];
        uint32_t bias[U][MT][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int grp = gr + u * step;
            const int word = (4 * grp + t) * VW;
            const bool in = grp < M.ng && word < M.ld;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int v = 0; v < VW; ++v) w[u][i][h][v] = 0;
                    if (in) load_words<VW>(w[u][i][h], M.q + row[i][h] * M.ld + word);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int grp = gr + u * step;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s[u][i][h] = 0.f;
                    bias[u][i][h] = zero_bias(8);
                    if (grp < M.ng) {
                        const int64_t at = row[i][h] * M.ng + grp;
                        s[u][i][h] = __bfloat162float(M.s[at]);
                        if (M.z) bias[u][i][h] = zero_bias(__ldg(M.z + at));
                    }
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int grp = gr + u * step;
            if (grp >= M.ng) break;
            float c[MT][NT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[i][j][e] = 0.f;
#pragma unroll
            for (int v = 0; v < VW; ++v) {
                const int k = ((4 * grp + t) * VW + v) * 8;
                uint32_t b[NT][4];      // (x0,x4) (x1,x5) (x2,x6) (x3,x7): the code pairs' order
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint4 x = col[j] ? load_x8(col[j], k, M.n, xvec) : make_uint4(0, 0, 0, 0);
                    b[j][0] = __byte_perm(x.x, x.z, 0x5410);
                    b[j][1] = __byte_perm(x.x, x.z, 0x7632);
                    b[j][2] = __byte_perm(x.y, x.w, 0x5410);
                    b[j][3] = __byte_perm(x.y, x.w, 0x7632);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const uint32_t a[4] = {
                            code_pair(w[u][i][0][v], 2 * p, bias[u][i][0]),
                            code_pair(w[u][i][1][v], 2 * p, bias[u][i][1]),
                            code_pair(w[u][i][0][v], 2 * p + 1, bias[u][i][0]),
                            code_pair(w[u][i][1][v], 2 * p + 1, bias[u][i][1])};
#pragma unroll
                        for (int j = 0; j < NT; ++j) mma16816(c[i][j], a, b[j][2 * p], b[j][2 * p + 1]);
                    }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    acc[i][j][0] += s[u][i][0] * c[i][j][0];
                    acc[i][j][1] += s[u][i][0] * c[i][j][1];
                    acc[i][j][2] += s[u][i][1] * c[i][j][2];
                    acc[i][j][3] += s[u][i][1] * c[i][j][3];
                }
        }
    }
}

// The three BF16 terms of an FP32 value, each the leading 8 bits of what is left (rounded
// towards zero, so a finite x never overflows): x = t[0] + t[1] + t[2] exactly.  An
// infinite or NaN x is t[0] alone.
__device__ __forceinline__ void split_terms(float x, __nv_bfloat16 (&t)[kTerms]) {
    t[0] = __float2bfloat16_rz(x);
    const float r1 = isfinite(x) ? x - __bfloat162float(t[0]) : 0.f;
    t[1] = __float2bfloat16_rz(r1);
    t[2] = __float2bfloat16_rz(r1 - __bfloat162float(t[1]));
}

// ---------------------------------------------------------------------------------
// Host: launchers
// ---------------------------------------------------------------------------------
cudaError_t quantize(const void *W, int w_bf16, int64_t m, int64_t n, const float *d_in, int group,
                     int grid, uint32_t *q, __nv_bfloat16 *s, uint8_t *z, cudaStream_t st);
cudaError_t dequantize(const Mat &M, int64_t m, int group, void *out, int out_bf16,
                       cudaStream_t st);
// xt: the split columns of FP32 X ([B][kTerms][ldx], ldx = split_ld(n)), unused for BF16.
NQ_HD int64_t split_ld(int64_t n) { return round_up(n, 8); }
cudaError_t matmul(const Mat &M, int64_t m, int group, const void *X, int x_bf16, int64_t B,
                   float *Y, __nv_bfloat16 *xt, cudaStream_t st);


// Expert layer for a few tokens (moe.cu).
struct MoeArgs {
    const void *X;             // [B][d], FP32 or BF16
    int x_bf16;
    int B, d, f, E, top_k, renormalise;
    const void *router;        // [E][d], of X's type
    Mat gate_up;               // E matrices of 2f x d, one after the other
    Mat down;                  // E matrices of d x f
    int group;
    float *Y;                  // [B][d]
    int32_t *ids;              // [B][top_k]
    float *weights;            // [B][top_k]
    __nv_bfloat16 *xt;         // [B][kTerms][split_ld(d)] (FP32 X)
    __nv_bfloat16 *h;          // [B top_k][kTerms][split_ld(f)]
};
cudaError_t moe(const MoeArgs &a, cudaStream_t st);

}  // namespace w4
}  // namespace nq
