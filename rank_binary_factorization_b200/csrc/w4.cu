// Layers with 4-bit weights and group scales (sm_100a): quantiser, read-back, matrix product.
#include "w4.cuh"

namespace nq {
namespace w4 {

// ---------------------------------------------------------------------------------
// Quantiser.  Per (row, group) and candidate c of ``grid``, alpha = 1 - c / (2 grid):
//   symmetric:  s = bf16(alpha max|w| / 7), z = 8
//   zeros:      lo = min(0, min w), hi = max(0, max w), s = bf16(alpha (hi - lo) / 15),
//               z = clamp(rint(-alpha lo / s), 0, 15)
//   q = clamp(rint(w / s) + z, 0, 15),  E = sum_j d_j^2 (w_j - s (q_j - z))^2
// and the lowest candidate with the least E is kept.  A lane holds 16 consecutive columns,
// g / 16 lanes a group; the scale and z are formed in FP64 (the scale then rounded to FP32
// and to BF16), rint(w / s) is that of the exact quotient (ties to even) and E is summed in
// FP64, so that neither a border case nor the choice depends on the order of operations.
// ---------------------------------------------------------------------------------
constexpr int kPer = 16;   // columns per lane

// rint(w / s) of the exact quotient, ties to even, exact for |w / s| <= 16 (larger
// magnitudes come out beyond +-15).  w - a s is exact in FP32 for the nearest integers a
// (s has 8 significant bits), so the remainder settles which side of the half it is on.
__device__ __forceinline__ float exact_rint(float w, float s, float inv) {
    float a = rintf(fminf(fmaxf(w * inv, -16.f), 16.f));
    const float rem = fmaf(-a, s, w), half = 0.5f * s;
    const bool odd = ((int)a) & 1;
    if (rem > half || (rem == half && odd)) a += 1.f;
    if (rem < -half || (rem == -half && odd)) a -= 1.f;
    return a;
}

template <int LPG>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = LPG / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int LPG>
__device__ __forceinline__ double group_sum(double v) {
#pragma unroll
    for (int o = LPG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Scale (a BF16 value) and zero point of a candidate.
__device__ __forceinline__ void candidate(double alpha, float lo, float hi, bool zeros, float &s,
                                          float &z) {
    if (zeros) {
        s = bf16_round((float)(alpha * ((double)hi - (double)lo) / 15.0));
        z = s > 0.f ? (float)fmin(fmax(rint(-alpha * (double)lo / (double)s), 0.0), 15.0) : 0.f;
    } else {
        s = bf16_round((float)(alpha * (double)hi / 7.0));
        z = 8.f;
    }
}

// Codes of the lane's columns for scale s: v[i] = q - z (so W^ = s v).
__device__ __forceinline__ void round_codes(const float (&w)[kPer], float s, float z,
                                            float (&v)[kPer]) {
    // a scale next to the least normal number: both sides moved up by 2^100, exactly
    const float up = s < 0x1p-100f ? 0x1p100f : 1.f;
    const float su = s * up, inv = 1.f / su;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        v[i] = s > 0.f ? fminf(fmaxf(exact_rint(w[i] * up, su, inv), -z), 15.f - z) : 0.f;
}

template <int LPG, typename T>
__global__ void __launch_bounds__(256)
    quantize_kernel(const T *__restrict__ W, int64_t m, int n, const float *__restrict__ d_in,
                    int grid, int vec, int ld, int ng, uint32_t *__restrict__ q,
                    __nv_bfloat16 *__restrict__ sc, uint8_t *__restrict__ zp) {
    const int64_t unit = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int per_row = ng * LPG;
    const int64_t row = unit / per_row;
    const int u = (int)(unit % per_row);
    const bool live = row < m;          // whole groups: a group's lanes share a row
    const int k0 = u * kPer;
    const bool zeros = zp != nullptr;
    float w[kPer];
    const T *src = W + (live ? row : 0) * n + k0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) w[i] = 0.f;
    if (live && vec && k0 + kPer <= n) {
        constexpr int NV = kPer * sizeof(T) / 16;
        uint4 raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
        const T *h = reinterpret_cast<const T *>(raw);
#pragma unroll
        for (int i = 0; i < kPer; ++i) w[i] = (float)h[i];
    } else if (live) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (k0 + i < n) w[i] = (float)src[i];
    }
    float lo = 0.f, hi = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        bad |= !isfinite(w[i]);
        lo = fminf(lo, w[i]);
        hi = fmaxf(hi, w[i]);
    }
    if (!zeros) hi = fmaxf(hi, -lo);
    hi = group_max<LPG>(hi);
    lo = -group_max<LPG>(-lo);
    bad = group_max<LPG>(bad ? 1.f : 0.f) > 0.f;

    float s, z;
    candidate(1.0, lo, hi, zeros, s, z);
    if (grid > 1) {
        double best = 0.0;
        int pick = 0;
        for (int c = 0; c < grid; ++c) {
            float cs, cz, v[kPer];
            candidate(1.0 - c / (2.0 * grid), lo, hi, zeros, cs, cz);
            round_codes(w, cs, cz, v);
            double e = 0.0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const double d = d_in && k0 + i < n ? (double)d_in[k0 + i] : 1.0;
                const double t = ((double)w[i] - (double)cs * (double)v[i]) * d;
                e += t * t;
            }
            e = group_sum<LPG>(e);
            if (c == 0 || e < best) best = e, pick = c;
        }
        candidate(1.0 - pick / (2.0 * grid), lo, hi, zeros, s, z);
    }
    // a group with a weight that is not finite reads back as NaN
    if (bad) s = __int_as_float(0x7fc00000), z = zeros ? 0.f : 8.f;
    float v[kPer];
    round_codes(w, s, z, v);
    if (!live) return;
    uint32_t word[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (k0 + i < n) word[i / 8] |= (uint32_t)(int)(v[i] + z) << (4 * (i % 8));
    const int wi = u * 2;
    if (wi < ld) *reinterpret_cast<uint2 *>(q + row * ld + wi) = make_uint2(word[0], word[1]);
    if (u % LPG == 0) {
        const int64_t at = row * ng + u / LPG;
        sc[at] = __float2bfloat16_rn(s);
        if (zeros) zp[at] = (uint8_t)(int)z;
    }
}

template <int LPG>
static cudaError_t quantize_t(const void *W, int w_bf16, int64_t m, int64_t n, const float *d_in,
                              int group, int grid, uint32_t *q, __nv_bfloat16 *s, uint8_t *z,
                              cudaStream_t st) {
    const int ld = (int)row_words(n), ng = (int)row_groups(n, group);
    const int64_t blocks = ceil_div(m * (int64_t)ng * LPG, 256);
    const int vec = n % (w_bf16 ? 8 : 4) == 0 && reinterpret_cast<uintptr_t>(W) % 16 == 0;
    if (w_bf16)
        quantize_kernel<LPG, __nv_bfloat16><<<(unsigned)blocks, 256, 0, st>>>(
            static_cast<const __nv_bfloat16 *>(W), m, (int)n, d_in, grid, vec, ld, ng, q, s, z);
    else
        quantize_kernel<LPG, float><<<(unsigned)blocks, 256, 0, st>>>(
            static_cast<const float *>(W), m, (int)n, d_in, grid, vec, ld, ng, q, s, z);
    count_launch();
    return cudaGetLastError();
}

cudaError_t quantize(const void *W, int w_bf16, int64_t m, int64_t n, const float *d_in, int group,
                     int grid, uint32_t *q, __nv_bfloat16 *s, uint8_t *z, cudaStream_t st) {
    if (group == 32) return quantize_t<2>(W, w_bf16, m, n, d_in, group, grid, q, s, z, st);
    if (group == 64) return quantize_t<4>(W, w_bf16, m, n, d_in, group, grid, q, s, z, st);
    return quantize_t<8>(W, w_bf16, m, n, d_in, group, grid, q, s, z, st);
}

// ---------------------------------------------------------------------------------
// Read-back: W^ = s (q - z), exact in FP32 (12 significant bits), rounded once for BF16.
// One lane per word (8 columns).
// ---------------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256)
    dequantize_kernel(const Mat M, int64_t m, int wpg, int vec, T *__restrict__ out) {
    const int nw = (M.n + 7) / 8;
    const int64_t unit = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t row = unit / nw;
    const int word = (int)(unit % nw);
    if (row >= m) return;
    const uint32_t w = __ldcs(M.q + row * M.ld + word);
    const int64_t at = row * M.ng + word / wpg;
    const float s = __bfloat162float(M.s[at]);
    const float z = M.z ? (float)(__ldg(M.z + at) & 15) : 8.f;
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (T)(s * ((float)((w >> (4 * i)) & 15u) - z));
    T *dst = out + row * M.n + word * 8;
    if (vec) {
        constexpr int NV = 8 * sizeof(T) / 16;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            __stcs(reinterpret_cast<uint4 *>(dst) + i, reinterpret_cast<const uint4 *>(v)[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (word * 8 + i < M.n) dst[i] = v[i];
    }
}

cudaError_t dequantize(const Mat &M, int64_t m, int group, void *out, int out_bf16,
                       cudaStream_t st) {
    const int64_t blocks = ceil_div(m * ceil_div(M.n, 8), 256);
    const int vec = M.n % 8 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
    if (out_bf16)
        dequantize_kernel<<<(unsigned)blocks, 256, 0, st>>>(M, m, group / 8, vec,
                                                           static_cast<__nv_bfloat16 *>(out));
    else
        dequantize_kernel<<<(unsigned)blocks, 256, 0, st>>>(M, m, group / 8, vec,
                                                           static_cast<float *>(out));
    count_launch();
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------------
// Matrix product for few columns: one CTA per 16 MT rows and chunk of NT x 8 columns, its
// 8 warps interleaved over the groups of the k axis, joined in shared memory in a fixed
// order.
// ---------------------------------------------------------------------------------
constexpr int kWarps = 8;

// FP32 X (B x n) into kTerms BF16 columns per row, zero padded to ldx.
__global__ void __launch_bounds__(256)
    split_x_kernel(const float *__restrict__ X, int64_t B, int n, int ldx,
                   __nv_bfloat16 *__restrict__ xt) {
    const int64_t b = blockIdx.x;
    const int k = blockIdx.y * blockDim.x + threadIdx.x;
    if (k >= ldx) return;
    __nv_bfloat16 t[kTerms];
    split_terms(k < n ? X[b * n + k] : 0.f, t);
#pragma unroll
    for (int i = 0; i < kTerms; ++i) xt[(b * kTerms + i) * ldx + k] = t[i];
}

template <int VW, int MT, int NT>
__global__ void __launch_bounds__(32 * kWarps)
    gemv_kernel(const Mat M, int64_t m, const __nv_bfloat16 *__restrict__ x, int64_t ldx, int xvec,
                int terms, int64_t B, float *__restrict__ Y) {
    constexpr int R = 16 * MT, C = 8 * NT;
    __shared__ float red[kWarps][R][C + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = (int64_t)blockIdx.x * R;
    const int per = C / terms;                       // rows of X in a chunk
    const int64_t b0 = (int64_t)blockIdx.y * per;
    const int nb = (int)min((int64_t)per, B - b0);
    int64_t row[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) row[i][h] = min(r0 + 16 * i + 8 * h + (lane >> 2), m - 1);
    const __nv_bfloat16 *col[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int c = 8 * j + (lane >> 2);
        col[j] = c < nb * terms ? x + (b0 * terms + c) * ldx : nullptr;
    }
    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
    group_products<VW, MT, NT>(acc, M, row, col, xvec, warp, kWarps);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[warp][16 * i + 8 * (e >> 1) + (lane >> 2)][8 * j + 2 * (lane & 3) + (e & 1)] =
                    acc[i][j][e];
    __syncthreads();
    for (int o = threadIdx.x; o < R * nb; o += 32 * kWarps) {
        const int r = o % R, b = o / R;
        if (r0 + r >= m) continue;
        float v = 0.f;
        for (int t = terms - 1; t >= 0; --t)
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += red[w][r][b * terms + t];
        Y[(b0 + b) * m + r0 + r] = v;
    }
}

template <int VW>
static cudaError_t gemv(const Mat &M, int64_t m, const __nv_bfloat16 *x, int64_t ldx, int xvec,
                        int terms, int64_t B, float *Y, cudaStream_t st) {
    if (B * terms <= 8) {
        const dim3 grid((unsigned)ceil_div(m, 16), (unsigned)ceil_div(B, 8 / terms));
        gemv_kernel<VW, 1, 1><<<grid, 32 * kWarps, 0, st>>>(M, m, x, ldx, xvec, terms, B, Y);
    } else {
        const dim3 grid((unsigned)ceil_div(m, 32), (unsigned)ceil_div(B, 16 / terms));
        gemv_kernel<VW, 2, 2><<<grid, 32 * kWarps, 0, st>>>(M, m, x, ldx, xvec, terms, B, Y);
    }
    count_launch();
    return cudaGetLastError();
}

cudaError_t matmul(const Mat &M, int64_t m, int group, const void *X, int x_bf16, int64_t B,
                   float *Y, __nv_bfloat16 *xt, cudaStream_t st) {
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(X);
    int64_t ldx = M.n;
    int xvec = M.n % 8 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0;
    if (!x_bf16) {
        ldx = split_ld(M.n);
        split_x_kernel<<<dim3((unsigned)B, (unsigned)ceil_div(ldx, 256)), 256, 0, st>>>(
            static_cast<const float *>(X), B, M.n, (int)ldx, xt);
        count_launch();
        x = xt;
        xvec = 1;
    }
    const int terms = x_bf16 ? 1 : kTerms;
    Mat Mx = M;
    if (xvec) Mx.n = (int)split_ld(M.n);     // the padding of a split column is zero
    if (group == 32) return gemv<1>(Mx, m, x, ldx, xvec, terms, B, Y, st);
    if (group == 64) return gemv<2>(Mx, m, x, ldx, xvec, terms, B, Y, st);
    return gemv<4>(Mx, m, x, ldx, xvec, terms, B, Y, st);
}

}  // namespace w4
}  // namespace nq
