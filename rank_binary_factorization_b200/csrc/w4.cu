// Layers with 4-bit weights and group scales (sm_100a): quantiser, read-back, matrix product.
#include "w4.cuh"

namespace nq {
namespace w4 {

static std::atomic<int> g_wait_polls{-1};
uint32_t wait_polls(uint32_t most) {
    const int p = g_wait_polls.load(std::memory_order_relaxed);
    return p < 0 || (uint32_t)p > most ? most : (uint32_t)p;
}
void set_wait_polls(int polls) { g_wait_polls.store(polls, std::memory_order_relaxed); }

// ---------------------------------------------------------------------------------
// Quantiser.  Per (row, group) and candidate c of ``grid``, alpha = 1 - c / (2 grid):
//   symmetric:  s = bf16(alpha max|w| / 7), z = 8
//   zeros:      lo = min(0, min w), hi = max(0, max w), s = bf16(alpha (hi - lo) / 15),
//               z = clamp(rint(-alpha lo / s), 0, 15)
//   q = clamp(rint(w / s) + z, 0, 15),  E = sum_j d_j^2 (w_j - s (q_j - z))^2
// and the lowest candidate with the least E is kept.  A lane holds 16 consecutive columns,
// g / 16 lanes a group; the scale and z are formed in FP64 (the scale then rounded to FP32
// and to BF16), rint(w / s) is that of the exact quotient (ties to even) and E is summed in
// FP64 where it matters, so that neither a border case nor the choice depends on the order of
// operations.
//
// The search runs in FP32 (six FMA-pipe operations a column and candidate: the clamp is the
// saturation of an FMA in units of 15 steps) and is off by less than 4.5e-5 of E (16 roundings of
// a term and of the sum, 1e-6; a column within 5.4e-6 steps of a half that rounds the other way,
// 4.4e-5 of its term); a candidate within kNear of the best so far is settled in FP64, both of
// them anew (about one comparison in 10000).
//
// Measured: 4096x4096 BF16, g = 128, 16 candidates 93 us, twice the 44 us that the search's FMA-pipe
// operations take at full rate: the rest is latency and issue (shuffles, sums across a group's lanes,
// the settled pairs; 24 bytes of spills at the 64 registers of four CTAs an SM).  28672x8192 BF16,
// g = 64, zero points, one candidate: 137 us, 598 MB, 68 % of the copy rate at 68 % of the issue slots
// (a rounded quotient for every column): neither is used up; FP32, g = 32: 186 us, 90 %, bound by
// memory.  The correction of the quotient instead of a settled remainder for every column:
// 614 -> 190 us; two columns an operation and 32 a lane: 184 -> 137 us.
// ---------------------------------------------------------------------------------
constexpr int kPer = 16;            // columns per lane (kWide: BF16 without a search)
constexpr int kWide = 32;
constexpr float kNear = 1e-4f;
constexpr float kMagic = 12582912.f;   // 1.5 2^23: adding it leaves rint(x) in the low bits

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

// 1 / x to a unit in the last place or so, for normal x.
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two FP32 values in one operation each, rounded as apart: the FMA pipe takes as long, but half
// the issue slots.
struct Two {
    uint64_t v;
};
__device__ __forceinline__ Two two(float a, float b) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 apart(Two a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// Maxima that hand on a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
template <int LPG>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = LPG / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int LPG, typename T>
__device__ __forceinline__ T group_sum(T v) {
#pragma unroll
    for (int o = LPG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// x / c in FP64 for a quotient far from the ends of its range, r about 1 / c: the residual of
// the first quotient is exact and corrects it to the rounded one (Markstein's correction: P. W.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34, 1990).
__device__ __forceinline__ double quotient(double x, double c, double r) {
    const double q = x * r;
    return fma(fma(-q, c, x), r, q);
}

// Scale (a BF16 value) and zero point of a candidate.
__device__ __forceinline__ void candidate(double alpha, float lo, float hi, bool zeros, float &s,
                                          float &z) {
    if (zeros) {
        s = bf16_round((float)quotient(alpha * ((double)hi - (double)lo), 15.0, 1.0 / 15.0));
        const double x = -alpha * (double)lo, c = (double)s;
        double v;
        if (s > 0x1p-100f && s < 0x1p100f) {
            const double r0 = (double)rcp(s);
            v = quotient(x, c, fma(fma(-c, r0, 1.0), r0, r0));
        } else {
            v = x / c;
        }
        z = s > 0.f ? (float)fmin(fmax(rint(v), 0.0), 15.0) : 0.f;
    } else {
        s = bf16_round((float)quotient(alpha * (double)hi, 7.0, 1.0 / 7.0));
        z = 8.f;
    }
}

// Exact q - z of one column (so w^ = s (q - z)).  ``up`` moves a scale next to the least normal
// number away from it, exactly, together with w.
__device__ __forceinline__ float scale_up(float s) { return s < 0x1p-100f ? 0x1p100f : 1.f; }
__device__ __forceinline__ float exact_code(float w, float s, float z, float up) {
    const float su = s * up;
    return s > 0.f ? fminf(fmaxf(exact_rint(w * up, su, 1.f / su), -z), 15.f - z) : 0.f;
}

// The lane's part of E in FP64.  Rare, so its columns go through local memory in a loop that leaves
// the registers to the search (two CTAs an SM with it unrolled, four so: 116 -> 93 us).
__device__ __forceinline__ double exact_error(const float (&w)[kPer], const float (&d)[kPer], float s,
                                           float z) {
    float wl[kPer], dl[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) wl[i] = w[i], dl[i] = d[i];
    const float up = scale_up(s);
    double e = 0.0;
#pragma unroll 2
    for (int i = 0; i < kPer; ++i) {
        const double t = ((double)wl[i] - (double)s * (double)exact_code(wl[i], s, z, up)) * (double)dl[i];
        e += t * t;
    }
    return e;
}

template <int PER, typename T>
__device__ __forceinline__ void load_per(const T *src, int k0, int n, bool vec, float (&v)[PER]) {
    if (vec && k0 + PER <= n) {
        constexpr int NV = PER * sizeof(T) / 16;
        uint4 raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) raw[i] = __ldg(reinterpret_cast<const uint4 *>(src + k0) + i);
        const T *h = reinterpret_cast<const T *>(raw);
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = (float)h[i];
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = k0 + i < n ? (float)src[k0 + i] : 0.f;
    }
}

// lo = min(0, min w) and hi = max(0, max w) (without zeros: hi = max |w|); NaN in hi if in w.
template <int PER>
__device__ __forceinline__ void range_of(const float (&w)[PER], bool zeros, float &lo, float &hi) {
    lo = hi = 0.f;
    if (zeros) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            lo = fminf(lo, w[i]);
            hi = max_nan(hi, w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) hi = max_nan(hi, fabsf(w[i]));
    }
}

// A row is worked on by 2^ltpr lanes (LPG to a group) side by side, blockIdx.y of them after one
// another along the row.
template <int PER, int LPG, bool SEARCH, typename T>
__global__ void __launch_bounds__(256, SEARCH ? 4 : PER == 32 ? 4 : 5)
    quantize_kernel(const T *__restrict__ W, int64_t m, int n, const float *__restrict__ d_in,
                    int grid, int vec, int dvec, int ltpr, int ld, int ng, uint32_t *__restrict__ q,
                    __nv_bfloat16 *__restrict__ sc, uint8_t *__restrict__ zp) {
    const int64_t row = ((int64_t)blockIdx.x << (8 - ltpr)) + (threadIdx.x >> ltpr);
    const int u = ((int)blockIdx.y << ltpr) + (threadIdx.x & ((1 << ltpr) - 1));
    const bool live = row < m && u < ng * LPG;          // whole groups
    const int k0 = u * PER;
    const bool zeros = zp != nullptr;
    float w[PER], lo, hi;
    load_per(W + (live ? row * n : 0), live ? k0 : n, n, vec, w);
    range_of(w, zeros, lo, hi);
    hi = group_max<LPG>(hi);
    lo = -group_max<LPG>(-lo);
    // a weight that is not finite
    const bool nan = !(hi < __int_as_float(0x7f800000)) || !(lo > __int_as_float(0xff800000));

    float s, z;
    if constexpr (!SEARCH) {
        candidate(1.0, lo, hi, zeros, s, z);
    } else {
        float d[PER];
        if (d_in) {
            load_per(d_in, live ? k0 : n, n, dvec, d);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) d[i] = 1.f;
        }
        // outside this range of weights and errors every candidate is settled in FP64
        const bool plain = hi - lo > 1e-25f && hi - lo < 1e25f;
        float best = 0.f, bs = 0.f, bz = 0.f;
        double best64 = -1.0;                           // E of the best in FP64 once needed
        const int sub = threadIdx.x & (LPG - 1);
        for (int c0 = 0; c0 < grid; c0 += LPG) {
            float ms, mz;                               // lane ``sub`` forms candidate c0 + sub
            candidate(1.0 - (c0 + sub) / (2.0 * grid), lo, hi, zeros, ms, mz);
            const float minv = rcp(15.f * ms);
            for (int j = 0; j < min(LPG, grid - c0); ++j) {
                const int from = (threadIdx.x & 31 & ~(LPG - 1)) | j;
                const float cs = __shfl_sync(0xffffffffu, ms, from),
                            cz = __shfl_sync(0xffffffffu, mz, from),
                            inv = __shfl_sync(0xffffffffu, minv, from);
                const float z15 = cz * (1.f / 15.f), off = kMagic + cz;
                const Two m2 = two(kMagic, kMagic), n2 = two(-off, -off), s2 = two(-cs, -cs);
                Two e2 = two(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < PER; i += 2) {
                    const Two u = two(__saturatef(fmaf(w[i], inv, z15)),
                                      __saturatef(fmaf(w[i + 1], inv, z15)));
                    const Two v = add2(fma2(u, two(15.f, 15.f), m2), n2);
                    const Two t = mul2(fma2(s2, v, two(w[i], w[i + 1])), two(d[i], d[i + 1]));
                    e2 = fma2(t, t, e2);
                }
                const float2 ea = apart(e2);
                const float e = group_sum<LPG>(ea.x + ea.y);
                const bool first = c0 + j == 0;
                const bool safe = plain && e > 1e-30f && best > 1e-30f && best < 1e30f;
                bool less = first || (safe && e < best * (1.f - kNear));
                const bool near = !first && !less && !(safe && e > best * (1.f + kNear));
                if (__any_sync(0xffffffffu, near)) {
                    const double a = group_sum<LPG>(exact_error(w, d, bs, bz));
                    const double b = group_sum<LPG>(exact_error(w, d, cs, cz));
                    if (near) {
                        if (best64 < 0.0) best64 = a;
                        less = b < best64;
                        if (less) best64 = b;
                    } else if (less) {
                        best64 = -1.0;
                    }
                } else if (less) {
                    best64 = -1.0;
                }
                if (less) best = e, bs = cs, bz = cz;
            }
        }
        s = bs, z = bz;
    }
    // a group with a weight that is not finite reads back as NaN
    if (nan) s = __int_as_float(0x7fc00000), z = zeros ? 0.f : 8.f;
    uint32_t word[PER / 8];
    {
        // t = w / s, rounded correctly (quotient and one correction, so a half comes out as the
        // half and goes to even); a = rint(t) from the low bits of + kMagic.  The remainder
        // w - a s is exact: beyond half a step t was off a half by less than its last bit, and
        // the lane settles its columns one by one.
        const float inv = rcp(s), z15 = z * (1.f / 15.f);
        const Two i2 = two(inv, inv), s2 = two(-s, -s), m2 = two(kMagic, kMagic);
        float dev = 0.f;
        uint32_t acc[PER / 8] = {};
#pragma unroll
        for (int i = PER - 2; i >= 0; i -= 2) {
            const Two w2 = two(w[i], w[i + 1]);
            const Two t0 = mul2(w2, i2);
            const Two t = fma2(fma2(t0, s2, w2), i2, t0);
            const Two a2 = add2(add2(t, m2), two(-kMagic, -kMagic));
            const float2 rem = apart(fma2(a2, s2, w2)), a = apart(a2);
            dev = fmaxf(dev, fmaxf(fabsf(rem.x), fabsf(rem.y)));
            // clamped to 0 .. 15 in units of 15, and back
            const float2 c = apart(fma2(two(__saturatef(fmaf(a.x, 1.f / 15.f, z15)),
                                            __saturatef(fmaf(a.y, 1.f / 15.f, z15))),
                                        two(15.f, 15.f), m2));
            acc[i / 8] = acc[i / 8] * 16u + __float_as_uint(c.y);
            acc[i / 8] = acc[i / 8] * 16u + __float_as_uint(c.x);
        }
        // the eight codes carry the bits of kMagic each
#pragma unroll
        for (int i = 0; i < PER / 8; ++i) word[i] = acc[i] - 0x4b400000u * 0x11111111u;
        // (also where s is 0, NaN, or so small that 1 / s or a remainder is not exact)
        if (!(s > 0x1p-100f) || !(dev <= 0.5f * s)) {
            const float up = scale_up(s);
#pragma unroll 1
            for (int i = 0; i < PER; ++i) {
                float wi = 0.f;
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (j == i) wi = w[j];
                const uint32_t c = (uint32_t)(int)(exact_code(wi, s, z, up) + z);
#pragma unroll
                for (int j = 0; j < PER / 8; ++j)
                    if (j == i >> 3) word[j] = i & 7 ? word[j] | c << (4 * (i & 7)) : c;
            }
        }
    }
    if (!live) return;
    if (k0 + PER > n) {                                // codes past the last column are 0
#pragma unroll
        for (int i = 0; i < PER / 8; ++i) {
            const int left = n - k0 - 8 * i;
            word[i] = left <= 0 ? 0 : left < 8 ? word[i] & ((1u << 4 * left) - 1) : word[i];
        }
    }
    const int wi = u * (PER / 8);
    if (wi < ld) {                                      // (ld is a multiple of 4)
        uint32_t *dst = q + row * ld + wi;
        if constexpr (PER == 32)
            *reinterpret_cast<uint4 *>(dst) = make_uint4(word[0], word[1], word[2], word[3]);
        else
            *reinterpret_cast<uint2 *>(dst) = make_uint2(word[0], word[1]);
    }
    if (u % LPG == 0) {
        const int64_t at = row * ng + u / LPG;
        sc[at] = __float2bfloat16_rn(s);
        if (zeros) zp[at] = (uint8_t)(int)z;
    }
}

// log2 of the lanes of a row: a power of two that covers ``units``, at least ``least``, at most 256.
static int row_lanes(int64_t units, int least) {
    int l = least;
    while (l < 8 && (1 << l) < units) ++l;
    return l;
}

// W by lanes of PER columns; a search takes kPer.
template <int PER, bool SEARCH, typename T>
static void quantize_launch(const T *W, int64_t m, int64_t n, const float *d_in, int group, int grid,
                            uint32_t *q, __nv_bfloat16 *s, uint8_t *z, cudaStream_t st) {
    const int ld = (int)row_words(n), ng = (int)row_groups(n, group), lpg = group / PER;
    const int ltpr = row_lanes(ng * lpg, lpg == 8 ? 3 : lpg == 4 ? 2 : lpg == 2 ? 1 : 0);
    const dim3 blocks((unsigned)ceil_div(m, 256 >> ltpr), (unsigned)ceil_div(ng * lpg, 1 << ltpr));
    const int vec = n % (16 / sizeof(T)) == 0 && reinterpret_cast<uintptr_t>(W) % 16 == 0;
    const int dvec = reinterpret_cast<uintptr_t>(d_in) % 16 == 0;
    auto kern = group == 32   ? quantize_kernel<PER, 32 / PER, SEARCH, T>
                : group == 64 ? quantize_kernel<PER, 64 / PER, SEARCH, T>
                              : quantize_kernel<PER, 128 / PER, SEARCH, T>;
    kern<<<blocks, 256, 0, st>>>(W, m, (int)n, d_in, grid, vec, dvec, ltpr, ld, ng, q, s, z);
    count_launch();
}

cudaError_t quantize(const void *W, int w_bf16, int64_t m, int64_t n, const float *d_in, int group,
                     int grid, uint32_t *q, __nv_bfloat16 *s, uint8_t *z, cudaStream_t st) {
    const __nv_bfloat16 *wb = static_cast<const __nv_bfloat16 *>(W);
    const float *wf = static_cast<const float *>(W);
    // BF16 without a search: the scale's arithmetic bounds it, shared by twice the columns in a
    // lane; FP32 is bound by memory, and 128 bytes a lane would be by the loads.
    if (w_bf16)
        grid > 1 ? quantize_launch<kPer, true>(wb, m, n, d_in, group, grid, q, s, z, st)
                 : quantize_launch<kWide, false>(wb, m, n, d_in, group, grid, q, s, z, st);
    else
        grid > 1 ? quantize_launch<kPer, true>(wf, m, n, d_in, group, grid, q, s, z, st)
                 : quantize_launch<kPer, false>(wf, m, n, d_in, group, grid, q, s, z, st);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------------
// Read-back: W^ = s (q - z), exact in FP32 (12 significant bits), rounded once for BF16.
// A lane reads two words (16 columns of one group).  Memory bounds it: 28672x8192 to BF16 111 us,
// 5.4 TB/s (83 % of the copy rate; streaming loads and stores).
// ---------------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256)
    dequantize_kernel(const Mat M, int64_t m, int upg, int vec, int ltpr, T *__restrict__ out) {
    const int64_t row = ((int64_t)blockIdx.x << (8 - ltpr)) + (threadIdx.x >> ltpr);
    const int u = ((int)blockIdx.y << ltpr) + (threadIdx.x & ((1 << ltpr) - 1));
    const int k0 = u * kPer;
    if (row >= m || k0 >= M.n) return;
    const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(M.q + row * M.ld + 2 * u));
    const int64_t at = row * M.ng + u / upg;
    const float s = __bfloat162float(M.s[at]);
    // the code in the low mantissa bits of 2^23
    const float off = 8388608.f + (M.z ? (float)(__ldg(M.z + at) & 15) : 8.f);
    __align__(16) T v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t c = ((i < 8 ? w.x : w.y) >> (4 * (i & 7))) & 15u;
        v[i] = (T)(s * (__uint_as_float(0x4b000000u | c) - off));
    }
    T *dst = out + row * M.n + k0;
    if (vec && k0 + kPer <= M.n) {
        constexpr int NV = kPer * sizeof(T) / 16;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            __stcs(reinterpret_cast<uint4 *>(dst) + i, reinterpret_cast<const uint4 *>(v)[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (k0 + i < M.n) dst[i] = v[i];
    }
}

template <typename T>
static cudaError_t dequantize_t(const Mat &M, int64_t m, int group, T *out, cudaStream_t st) {
    const int64_t units = ceil_div(M.n, kPer);
    const int ltpr = row_lanes(units, 0);
    const dim3 blocks((unsigned)ceil_div(m, 256 >> ltpr), (unsigned)ceil_div(units, 1 << ltpr));
    const int vec = (M.n * sizeof(T)) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
    dequantize_kernel<T><<<blocks, 256, 0, st>>>(M, m, group / kPer, vec, ltpr, out);
    count_launch();
    return cudaGetLastError();
}

cudaError_t dequantize(const Mat &M, int64_t m, int group, void *out, int out_bf16,
                       cudaStream_t st) {
    if (out_bf16) return dequantize_t(M, m, group, static_cast<__nv_bfloat16 *>(out), st);
    return dequantize_t(M, m, group, static_cast<float *>(out), st);
}

// ---------------------------------------------------------------------------------
// Matrix product for few columns: persistent CTAs, two an SM, walk the row tiles (run_products).
// Measured: 4096x4096 g = 128, one BF16 row of X 6.4 us (latency: prologue, one job a CTA, the
// join); 11008x4096 g = 64 with zero points 11.5 us; 28672x8192 g = 128, 16 rows of X 51-53 us (the
// columns, 256 KB, come through L1 and L2 for every job, and the variant spills).  Above n = 9216 for
// one BF16 row the columns are laid out in global memory by a launch of their own: 4096x11008 12 us,
// 8192x28672 33 us.
// ---------------------------------------------------------------------------------
template <int VW, int MT, int NT, bool XS>
struct GemvProb {
    int jobs, WK;
    int terms, nb, cols;                   // columns per row of X; rows of X, their columns
    int m, lrows;                          // rows of W; log2 of the rows of a job
    const __nv_bfloat16 *xw;               // the columns (global memory), ldx apart
    int64_t ldx;
    uint32_t xs, half_stride;              // the columns (shared memory)
    uint4 *xs_words;
    const void *X;                         // what they are made from
    int x_bf16, n;
    float *Y;
    Red<MT, NT> *red;                      // two, used in turn: one barrier per job

    // job k of a CTA is row block blockIdx.x + k gridDim.x of 16 MT (8 / WK) rows
    struct Cursor {
        int row;
    };
    __device__ __forceinline__ Cursor first() const { return {(int)blockIdx.x << lrows}; }
    __device__ __forceinline__ void next(Cursor &c) const { c.row += gridDim.x << lrows; }
    __device__ __forceinline__ int first_row(const Cursor &c, int wr, int i) const {
        return c.row + 16 * (MT * wr + i);
    }
    __device__ __forceinline__ int last_row(const Cursor &, int) const { return m - 1; }
    // XS: the CTA's columns into shared memory, while the first codes are on their way
    __device__ __forceinline__ void ready() const {
        if constexpr (XS) {
            // words of all columns one after another, a few of a thread under way at a time
            const int words = (int)(ldx / 8);
            constexpr int AHEAD = 4;
            int b = threadIdx.x / words, wd = threadIdx.x % words;
            while (b < nb) {
                int bs[AHEAD], ws[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    bs[i] = b, ws[i] = wd;
                    wd += 32 * kWarps;
                    while (wd >= words) wd -= words, ++b;
                }
                if (x_bf16) {
                    uint4 v[AHEAD];
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i)
                        if (bs[i] < nb)
                            v[i] = x_word(static_cast<const __nv_bfloat16 *>(X) + (int64_t)bs[i] * n,
                                          ws[i] * 8, n);
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i)
                        if (bs[i] < nb)
                            xs_words[(ws[i] / 16 * cols + bs[i]) * 16 + x_place<VW>(ws[i] % 16, bs[i] & 1)] =
                                v[i];
                } else {
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) {
                        if (bs[i] >= nb) break;
                        uint4 w[kTerms];
                        x_words(static_cast<const float *>(X) + (int64_t)bs[i] * n, ws[i] * 8, n, w);
#pragma unroll
                        for (int t = 0; t < kTerms; ++t) {
                            const int c = bs[i] * kTerms + t;
                            xs_words[(ws[i] / 16 * cols + c) * 16 + x_place<VW>(ws[i] % 16, c & 1)] = w[t];
                        }
                    }
                }
            }
            __syncthreads();
        }
    }
    __device__ __forceinline__ int tiles(const Cursor &) const { return (cols + 7) / 8; }
    __device__ __forceinline__ const char *col(const Cursor &, int j, bool &odd) const {
        const int c = min(8 * j + (((int)threadIdx.x & 31) >> 2), cols - 1);
        odd = c & 1;
        if constexpr (XS) return reinterpret_cast<const char *>((uintptr_t)(xs + c * 256));
        return reinterpret_cast<const char *>(xw + c * ldx);
    }
    __device__ __forceinline__ void end(const Cursor &c, int job, const float (&acc)[MT][NT][4]) {
        Red<MT, NT> &R = red[job & 1];
        R.put(acc);
        const int wr = (threadIdx.x >> 5) / WK;
        group_sync(wr, WK);
        const int r0 = first_row(c, wr, 0);
        for (int o = threadIdx.x - wr * 32 * WK; o < 16 * MT * nb; o += 32 * WK) {
            const int r = o % (16 * MT), b = o / (16 * MT);
            if (r0 + r < m) Y[(int64_t)b * m + r0 + r] = R.sum(wr, WK, r, b * terms, terms);
        }
    }
};

// Columns of a CTA that are kept in shared memory, bytes at most: what leaves two CTAs an SM
// (4096x4096, 4 columns of 8 KB: 8.0 us from global memory with two, 11.4 us with one).
constexpr int kXsBytes = 18 * 1024;
static_assert(2 * (kRingBytes + 2 * (int)sizeof(Red<1, 2>) + kXsBytes + 1024) <= 228 * 1024, "two CTAs");

template <int VW, bool Z, bool SV, bool XS, int MT, int NT>
__global__ void __launch_bounds__(32 * kWarps, 2)
    gemv_kernel(const Mat M, int m, const void *X, int x_bf16, const __nv_bfloat16 *xw, int WK,
                int64_t B, int blocks, float *__restrict__ Y) {
    extern __shared__ __align__(1024) char sm[];
    GemvProb<VW, MT, NT, XS> P;
    P.jobs = (int)((blocks - blockIdx.x + gridDim.x - 1) / gridDim.x);
    P.WK = WK;
    P.terms = x_bf16 ? 1 : kTerms;
    P.nb = B;
    P.cols = P.nb * P.terms;
    P.m = m, P.Y = Y;
    P.lrows = 31 - __clz(16 * MT * (kWarps / WK));
    P.ldx = padded(M.n);
    P.xw = xw;
    P.red = reinterpret_cast<Red<MT, NT> *>(sm + kRingBytes);
    P.X = X, P.x_bf16 = x_bf16, P.n = M.n;
    P.xs_words = reinterpret_cast<uint4 *>(P.red + 2);
    P.xs = (uint32_t)__cvta_generic_to_shared(P.xs_words);
    P.half_stride = P.cols * 256;
    run_products<VW, Z, SV, XS, MT, NT>(P, M, WK, sm);
}

// X (B x n) as columns: [B][1 or kTerms][padded(n)], the words of a half placed for VW.
// err: an error word to clear, or null.
template <int VW>
__global__ void __launch_bounds__(256)
    x_words_kernel(const void *X, int x_bf16, int64_t B, int n, uint4 *__restrict__ xw, int *err) {
    if (err && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *err = 0;
    const int words = (int)(padded(n) / 8);
    const int64_t b = blockIdx.x;
    const int wd = blockIdx.y * blockDim.x + threadIdx.x;
    if (wd >= words) return;
    if (x_bf16) {
        xw[b * words + x_word_place<VW>(wd, b)] =
            x_word(static_cast<const __nv_bfloat16 *>(X) + b * n, wd * 8, n);
    } else {
        uint4 w[kTerms];
        x_words(static_cast<const float *>(X) + b * n, wd * 8, n, w);
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {
            const int64_t c = b * kTerms + t;
            xw[c * words + x_word_place<VW>(wd, c)] = w[t];
        }
    }
}

// Columns of the call above which the tensor-memory path (w4_tc.cu) takes it: the most that this
// one holds at a time, whatever m and n are.  28672x8192: 16 BF16 rows 51-53 us here, 17 there 57; 8
// FP32 rows (24 columns, the codes twice) 85 us here, 67 there.  4096x4096: 16 BF16 rows 9.7 us here, 17
// there 12.1; 8 FP32 rows 12.1 here, 11.7 there.
constexpr int kMaxColumns = 16;
static bool on_tensor_memory(int x_bf16, int64_t B) {
    return B * (x_bf16 ? 1 : kTerms) > kMaxColumns;
}

// Columns of X in the call, and whether a CTA keeps its own in shared memory.
static bool x_shared(int64_t n, int x_bf16, int64_t B) {
    const int64_t cols = B * (x_bf16 ? 1 : kTerms);
    return cols <= kMaxColumns && cols * padded(n) * 2 <= kXsBytes;
}

static size_t x_bytes(int64_t n, int x_bf16, int64_t B) {
    const size_t b = (size_t)B * (x_bf16 ? 1 : kTerms) * padded(n) * 2;
    return (b + 255) / 256 * 256;
}

// Workspace: the columns of X and, on the tensor-memory path, the parts' sums and the error word.
size_t matmul_workspace(int64_t m, int64_t n, int x_bf16, int64_t B) {
    if (x_shared(n, x_bf16, B)) return 0;
    if (!on_tensor_memory(x_bf16, B)) return x_bytes(n, x_bf16, B);
    return matmul_error_word(m, n, x_bf16, B) + sizeof(int);
}

size_t matmul_error_word(int64_t m, int64_t n, int x_bf16, int64_t B) {
    if (!on_tensor_memory(x_bf16, B)) return 0;
    const size_t b = x_bytes(n, x_bf16, B) + tc_plan(m, n, x_bf16 ? 1 : kTerms, B).partial_bytes;
    return (b + 255) / 256 * 256;
}

template <int VW, bool Z, bool SV, bool XS, int MT, int NT>
static cudaError_t gemv_t(const Mat &M, int64_t m, const void *X, int x_bf16, const __nv_bfloat16 *xw,
                          int64_t B, float *Y, cudaStream_t st) {
    const int terms = x_bf16 ? 1 : kTerms;
    constexpr int fixed = kRingBytes + 2 * sizeof(Red<MT, NT>);
    const int smem = fixed + (XS ? (int)(B * terms * padded(M.n) * 2) : 0);
    auto kern = gemv_kernel<VW, Z, SV, XS, MT, NT>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_smem_limit((const void *)kern, fixed + (XS ? kXsBytes : 0), configured);
    if (e != cudaSuccess) return e;
    // fewer rows a job where the layer has too few of them to keep two CTAs an SM busy
    int WK = k_ranges(M.n);
    while (2 * WK <= kWarps && 2 * WK <= ceil_div(M.n, kUnit) &&
           ceil_div(m, 16 * MT * (kWarps / WK)) < 2 * kNumSMsB200)
        WK *= 2;
    const int64_t blocks = ceil_div(m, 16 * MT * (kWarps / WK)), slots = 2 * (int64_t)device_sm_count();
    kern<<<(unsigned)(blocks < slots ? blocks : slots), 32 * kWarps, smem, st>>>(
        M, (int)m, X, x_bf16, xw, WK, (int)B, (int)blocks, Y);
    count_launch();
    return cudaGetLastError();
}

template <int VW, bool Z, bool SV>
static cudaError_t gemv_n(const Mat &M, int64_t m, const void *X, int x_bf16, const __nv_bfloat16 *xw,
                        int64_t B, float *Y, cudaStream_t st) {
    const int64_t cols = B * (x_bf16 ? 1 : kTerms);
    if (x_shared(M.n, x_bf16, B))
        return cols <= 8 ? gemv_t<VW, Z, SV, true, 1, 1>(M, m, X, x_bf16, xw, B, Y, st)
                         : gemv_t<VW, Z, SV, true, 1, 2>(M, m, X, x_bf16, xw, B, Y, st);
    return cols <= 8 ? gemv_t<VW, Z, SV, false, 2, 1>(M, m, X, x_bf16, xw, B, Y, st)
                     : gemv_t<VW, Z, SV, false, 2, 2>(M, m, X, x_bf16, xw, B, Y, st);
}

template <int VW, bool Z>
static cudaError_t gemv(const Mat &M, int64_t m, const void *X, int x_bf16, const __nv_bfloat16 *xw,
                        int64_t B, float *Y, cudaStream_t st) {
    return scales_vec(M, 32 * VW) ? gemv_n<VW, Z, true>(M, m, X, x_bf16, xw, B, Y, st)
                                  : gemv_n<VW, Z, false>(M, m, X, x_bf16, xw, B, Y, st);
}

cudaError_t matmul(const Mat &M, int64_t m, int group, const void *X, int x_bf16, int64_t B,
                   float *Y, __nv_bfloat16 *xw, cudaStream_t st) {
    char *ws = reinterpret_cast<char *>(xw);
    int *err = on_tensor_memory(x_bf16, B)
                   ? reinterpret_cast<int *>(ws + matmul_error_word(m, M.n, x_bf16, B)) : nullptr;
    if (!x_shared(M.n, x_bf16, B)) {
        auto words = on_tensor_memory(x_bf16, B) ? x_words_kernel<0>
                     : group == 32 ? x_words_kernel<1>
                     : group == 64 ? x_words_kernel<2>
                                   : x_words_kernel<4>;
        words<<<dim3((unsigned)B, (unsigned)ceil_div(padded(M.n) / 8, 256)), 256, 0, st>>>(
            X, x_bf16, B, M.n, reinterpret_cast<uint4 *>(xw), err);
        count_launch();
    }
    if (on_tensor_memory(x_bf16, B))
        return tc_matmul(M, m, group, xw, x_bf16 ? 1 : kTerms, B, Y,
                         reinterpret_cast<float *>(ws + x_bytes(M.n, x_bf16, B)), err, st);
    auto run = M.z ? (group == 32 ? gemv<1, true> : group == 64 ? gemv<2, true> : gemv<4, true>)
                   : (group == 32 ? gemv<1, false> : group == 64 ? gemv<2, false> : gemv<4, false>);
    return run(M, m, X, x_bf16, xw, B, Y, st);
}

}  // namespace w4
}  // namespace nq
