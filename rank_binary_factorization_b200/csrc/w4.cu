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
// Matrix product for few columns: persistent CTAs walk the row tiles (run_products).
// ---------------------------------------------------------------------------------
template <int MT, int NT, bool XS>
struct GemvProb {
    int jobs, WK;
    int terms, nb, cols;                   // columns per row of X; rows of X, columns of this CTA
    int m, lrows;                          // rows of W; log2 of the rows of a job
    int64_t b0;                            // its first row of X
    const __nv_bfloat16 *xw;               // its columns (global memory), ldx apart
    int64_t ldx;
    uint32_t xs, half_stride;              // its columns (shared memory)
    float *Y;
    Red<MT, NT> *red;                      // two, used in turn: one barrier per job

    // job k of a CTA is row block blockIdx.x + k gridDim.x of 16 MT (8 / WK) rows
    __device__ __forceinline__ int block_row(int job) const {
        return (int)(blockIdx.x + (unsigned)job * gridDim.x) << lrows;
    }
    __device__ __forceinline__ int first_row(int job, int wr, int i) const {
        return block_row(job) + 16 * (MT * wr + i);
    }
    __device__ __forceinline__ int last_row(int, int) const { return m - 1; }
    __device__ __forceinline__ void ready() const { if constexpr (XS) __syncthreads(); }
    __device__ __forceinline__ void begin(int) {}
    __device__ __forceinline__ const char *col(int j) const {
        const int c = min(8 * j + (((int)threadIdx.x & 31) >> 2), cols - 1);
        if constexpr (XS) return reinterpret_cast<const char *>((uintptr_t)(xs + c * 256));
        return reinterpret_cast<const char *>(xw + c * ldx);
    }
    __device__ __forceinline__ void end(int job, const float (&acc)[MT][NT][4]) {
        Red<MT, NT> &R = red[job & 1];
        R.put(acc);
        __syncthreads();
        const int r0 = block_row(job);
        for (int o = threadIdx.x; o < nb << lrows; o += 32 * kWarps) {
            const int r = o & ((1 << lrows) - 1), b = o >> lrows;
            if (r0 + r < m)
                Y[(b0 + b) * m + r0 + r] = R.sum(r / (16 * MT), WK, r % (16 * MT), b * terms, terms);
        }
    }
};

// Whether the columns of a CTA are kept in shared memory: up to this many bytes of them leave
// two CTAs an SM.
constexpr int kXsBytes = 48 * 1024;

template <int VW, bool Z, bool XS, int MT, int NT>
__global__ void __launch_bounds__(32 * kWarps, 2)
    gemv_kernel(const Mat M, int m, const void *X, int x_bf16, const __nv_bfloat16 *xw, int svec,
                int WK, int64_t B, int blocks, float *__restrict__ Y) {
    extern __shared__ __align__(1024) char sm[];
    GemvProb<MT, NT, XS> P;
    P.jobs = (int)((blocks - blockIdx.x + gridDim.x - 1) / gridDim.x);
    P.WK = WK;
    P.terms = x_bf16 ? 1 : kTerms;
    const int per = 8 * NT / P.terms;
    P.b0 = (int64_t)blockIdx.y * per;
    P.nb = (int)min((int64_t)per, B - P.b0);
    P.cols = P.nb * P.terms;
    P.m = m, P.Y = Y;
    P.lrows = 31 - __clz(16 * MT * (kWarps / WK));
    P.ldx = padded(M.n);
    P.xw = XS ? nullptr : xw + P.b0 * P.terms * P.ldx;
    P.red = reinterpret_cast<Red<MT, NT> *>(sm + ring_bytes<MT>());
    uint4 *xs = reinterpret_cast<uint4 *>(P.red + 2);
    P.xs = (uint32_t)__cvta_generic_to_shared(xs);
    P.half_stride = P.cols * 256;
    if constexpr (XS) {
        const int words = (int)(P.ldx / 8);
        for (int o = threadIdx.x; o < words * P.nb; o += 32 * kWarps) {
            const int b = o / words, wd = o % words;
            const int64_t row = (P.b0 + b) * M.n;
            if (x_bf16) {
                xs[x_entry<VW>(wd / 16, wd % 16, b, P.cols)] =
                    x_word(static_cast<const __nv_bfloat16 *>(X) + row, wd * 8, M.n);
            } else {
                uint4 w[kTerms];
                x_words(static_cast<const float *>(X) + row, wd * 8, M.n, w);
#pragma unroll
                for (int t = 0; t < kTerms; ++t)
                    xs[x_entry<VW>(wd / 16, wd % 16, b * kTerms + t, P.cols)] = w[t];
            }
        }
    }
    run_products<VW, Z, XS, MT, NT>(P, M, svec, WK, sm);
}

// X (B x n) as columns in word order: [B][1 or kTerms][padded(n)].
__global__ void __launch_bounds__(256)
    x_words_kernel(const void *X, int x_bf16, int64_t B, int n, uint4 *__restrict__ xw) {
    const int words = (int)(padded(n) / 8);
    const int64_t b = blockIdx.x;
    const int wd = blockIdx.y * blockDim.x + threadIdx.x;
    if (wd >= words) return;
    if (x_bf16) {
        xw[b * words + wd] = x_word(static_cast<const __nv_bfloat16 *>(X) + b * n, wd * 8, n);
    } else {
        uint4 w[kTerms];
        x_words(static_cast<const float *>(X) + b * n, wd * 8, n, w);
#pragma unroll
        for (int t = 0; t < kTerms; ++t) xw[(b * kTerms + t) * words + wd] = w[t];
    }
}

// Columns of X in the call, and whether a CTA keeps its own in shared memory.
static bool x_shared(int64_t n, int x_bf16, int64_t B) {
    const int64_t cols = B * (x_bf16 ? 1 : kTerms);
    return cols <= 8 && cols * padded(n) * 2 <= kXsBytes;
}

size_t x_workspace(int64_t n, int x_bf16, int64_t B) {
    if (x_shared(n, x_bf16, B)) return 0;
    return (size_t)B * (x_bf16 ? 1 : kTerms) * padded(n) * 2;
}

template <int VW, bool Z, bool XS, int MT, int NT>
static cudaError_t gemv_t(const Mat &M, int64_t m, const void *X, int x_bf16, const __nv_bfloat16 *xw,
                          int64_t B, float *Y, cudaStream_t st) {
    const int terms = x_bf16 ? 1 : kTerms;
    constexpr int fixed = ring_bytes<MT>() + 2 * sizeof(Red<MT, NT>);
    const int smem = fixed + (XS ? (int)(B * terms * padded(M.n) * 2) : 0);
    auto kern = gemv_kernel<VW, Z, XS, MT, NT>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_smem_limit((const void *)kern, fixed + (XS ? kXsBytes : 0), configured);
    if (e != cudaSuccess) return e;
    const int WK = k_ranges(M.n);
    const int64_t blocks = ceil_div(m, 16 * MT * (kWarps / WK)), chunks = ceil_div(B, 8 * NT / terms);
    int64_t ctas = 2 * (int64_t)device_sm_count() / chunks;
    ctas = ctas < 1 ? 1 : ctas > blocks ? blocks : ctas;
    kern<<<dim3((unsigned)ctas, (unsigned)chunks), 32 * kWarps, smem, st>>>(
        M, (int)m, X, x_bf16, xw, scales_vec(M, 32 * VW), WK, B, (int)blocks, Y);
    count_launch();
    return cudaGetLastError();
}

template <int VW, bool Z>
static cudaError_t gemv(const Mat &M, int64_t m, const void *X, int x_bf16, const __nv_bfloat16 *xw,
                        int64_t B, float *Y, cudaStream_t st) {
    if (x_shared(M.n, x_bf16, B)) return gemv_t<VW, Z, true, 1, 1>(M, m, X, x_bf16, xw, B, Y, st);
    if (B * (x_bf16 ? 1 : kTerms) <= 8)
        return gemv_t<VW, Z, false, 1, 1>(M, m, X, x_bf16, xw, B, Y, st);
    return gemv_t<VW, Z, false, 2, 2>(M, m, X, x_bf16, xw, B, Y, st);
}

cudaError_t matmul(const Mat &M, int64_t m, int group, const void *X, int x_bf16, int64_t B,
                   float *Y, __nv_bfloat16 *xw, cudaStream_t st) {
    if (!x_shared(M.n, x_bf16, B)) {
        x_words_kernel<<<dim3((unsigned)B, (unsigned)ceil_div(padded(M.n) / 8, 256)), 256, 0, st>>>(
            X, x_bf16, B, M.n, reinterpret_cast<uint4 *>(xw));
        count_launch();
    }
    auto run = M.z ? (group == 32 ? gemv<1, true> : group == 64 ? gemv<2, true> : gemv<4, true>)
                   : (group == 32 ? gemv<1, false> : group == 64 ? gemv<2, false> : gemv<4, false>);
    return run(M, m, X, x_bf16, xw, B, Y, st);
}

}  // namespace w4
}  // namespace nq
