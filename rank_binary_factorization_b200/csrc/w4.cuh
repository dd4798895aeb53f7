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

// Codes i and i + 4 of a word as the BF16 pair ((q_i - z) / 2048, (q_{i+4} - z) / 2048), exactly,
// for i = 0, 1 (i = 2, 3: the word shifted right by 8).  Bits 0..3 of a half: the low mantissa
// bits of 128.0 (ulp 1) make 128 + q.  Bits 4..7 of a half alone are the BF16 number
// q 2^-129 for every q (subnormals and the first binade are one line), which 2^118 brings to
// q / 2048.  So four pairs cost one shift, four logical operations and four FMAs.
// The unit of 1 / 2048 costs nothing and keeps the sums in range: 128 (the longest group) x 15 / 2048
// is below 1, so no product and no group's sum of finite activations overflows, and the sum of
// the groups does so only where the result itself is near the range's end.  At the other end, sums
// below 2^-126 in this unit (results below 2^-115) lose their last bits.
struct ZeroPoint {
    uint32_t lo, hi;      // -(128 + z) / 2048 and -z / 2048, twice each
};
// -1/16 has ulp 1/2048: its low mantissa bits make -(128 + z) / 2048.
__device__ __forceinline__ ZeroPoint zero_point(uint32_t z) {
    const uint32_t lo = (0xbd80u | z) * 0x10001u, c16 = 0x3d803d80u;
    const __nv_bfloat162 hi = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&lo),
                                      *reinterpret_cast<const __nv_bfloat162 *>(&c16));
    return {lo, *reinterpret_cast<const uint32_t *>(&hi)};
}
__device__ __forceinline__ uint32_t fma_pair(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t code_pair0(uint32_t w, const ZeroPoint &z) {
    return fma_pair((w & 0x000f000fu) | 0x43004300u, 0x3a003a00u /* 1/2048 */, z.lo);
}
__device__ __forceinline__ uint32_t code_pair1(uint32_t w, const ZeroPoint &z) {
    return fma_pair(w & 0x00f000f0u, 0x7a807a80u /* 2^118 */, z.hi);
}
constexpr float kCodeUnit = 2048.f;   // the pairs hold codes in units of 1/2048

// 16 bytes global -> shared, asynchronously; zeros where ``in`` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 16 : 0)
                 : "memory");
}
// 4 or 8 bytes (aligned), of which the first ``size`` are read.
template <int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void *src, int size = N) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(size)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- activations -----------------------------------------------------------------------
// The product reads a column of activations as BF16 words of 8 values in the order of the
// code pairs, (0,4) (1,5) (2,6) (3,7), zero from n up to a multiple of kUnit; the 16 words of a
// half unit (128 columns) in the order of x_place.
constexpr int kUnit = 256;                       // columns of W in a unit of work
NQ_HD int64_t padded(int64_t n) { return round_up(n, kUnit); }

__device__ __forceinline__ uint4 pair_order(const uint4 v) {
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                      __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
}

// Values x[k .. k + 7] of a BF16 vector of length n as a word; zero from n on.
__device__ __forceinline__ uint4 x_word(const __nv_bfloat16 *x, int64_t k, int n) {
    if (k + 8 <= n && (reinterpret_cast<uintptr_t>(x + k) & 15) == 0)
        return pair_order(*reinterpret_cast<const uint4 *>(x + k));
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        h[i] = k + i < n ? reinterpret_cast<const unsigned short *>(x)[k + i] : 0;
    return make_uint4(h[0] | h[4] << 16, h[1] | h[5] << 16, h[2] | h[6] << 16, h[3] | h[7] << 16);
}

// The three BF16 terms of an FP32 value, each the leading 8 bits of what is left (rounded
// towards zero, so a finite x never overflows): x = t[0] + t[1] + t[2], exactly from
// 2^-110 on and to 2^-133 below.  An infinite or NaN x is t[0] alone.
__device__ __forceinline__ void split_terms(float x, __nv_bfloat16 (&t)[kTerms]) {
    t[0] = __float2bfloat16_rz(x);
    const float r1 = isfinite(x) ? x - __bfloat162float(t[0]) : 0.f;
    t[1] = __float2bfloat16_rz(r1);
    t[2] = __float2bfloat16_rz(r1 - __bfloat162float(t[1]));
}

// The same of an FP32 vector: the words of its kTerms columns.
__device__ __forceinline__ void x_words(const float *x, int64_t k, int n, uint4 (&w)[kTerms]) {
    __nv_bfloat16 t[8][kTerms];
    __align__(16) float v[8];
    if (k + 8 <= n && (reinterpret_cast<uintptr_t>(x + k) & 15) == 0) {
        *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(x + k);
        *reinterpret_cast<float4 *>(v + 4) = *reinterpret_cast<const float4 *>(x + k + 4);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = k + i < n ? x[k + i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) split_terms(v[i], t[i]);
#pragma unroll
    for (int j = 0; j < kTerms; ++j) {
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = __bfloat16_as_ushort(t[i][j]);
        w[j] = make_uint4(h[0] | h[4] << 16, h[1] | h[5] << 16, h[2] | h[6] << 16, h[3] | h[7] << 16);
    }
}

// Place of value k of a column in that order, within its word.
NQ_HD int in_word(int k) { return (k & ~7) | (k & 3) << 1 | (k >> 2 & 1); }

// ---- rows x columns -----------------------------------------------------------------------
// One CTA's products of packed rows with activation columns, job after job.
//
// A job is MT tiles of 16 rows, WR times over, against NT x 8 columns and the whole k axis.
// The 8 warps are WR row groups of WK; the warps of a group split the k axis into contiguous
// ranges of units and join in shared memory at the end of the job, apart from the other groups
// (WK = 8 where the axis has units enough: the fewest rows a job, the most even spread of jobs
// over the SMs).  Every warp runs its own ring of kRowStages / MT asynchronous copies (one unit
// of its rows: 128 bytes of codes a row) that carries on across jobs, so 64 KB a CTA are on their
// way from memory at any time and no warp waits for another within a job.  Where the rows' scales
// and zero points allow it (scales_vec) they come with the codes of their unit: loaded to
// registers half a unit ahead, as they are for layers that do not, their latency took a quarter
// of the time (11008x4096 g = 64 with zero points, one column: 15.0 us against 10.3 without the
// loads).
//
// The A fragment of an MMA is 16 rows of W (lane: rows lane/4 and lane/4 + 8), the B
// fragment 8 columns (lane: column lane/4), so any order of the k axis serves as long as
// both sides use it: lane%4 = t takes VW = g/32 consecutive words of a row, words t VW ..
// t VW + VW - 1 of a group, so a group is 2 VW MMAs of exactly its own columns, and its sum
// is scaled once, in FP32.
//
// Shared memory of a unit: 128 bytes a row, its eight 16-byte chunks permuted with the row so
// that the fragment loads (16, 8 or 4 bytes a lane for g = 128, 64, 32) meet every bank once.
//
// Columns past the last one repeat it: an MMA column reaches no other, and nobody reads its
// sums.  SV: scales_vec holds.  XS: the CTA's columns lie in shared memory (Prob's ready() puts
// them there), else in global memory.
//
// Measured, 28672x8192 g = 128, one BF16 column: 32 us, 3.8 TB/s (58 % of the copy rate); 162
// instructions for 16 rows x 128 columns, 57 % of the issue slots, 100 registers, two CTAs an SM.
// Neither memory nor issue is used up: of 3.6 warps a scheduler 1.2 are eligible, too few in flight
// for a warp's own chain (copy, decode, MMA, scale).  Two row tiles by two column tiles, for 9 to 16
// columns that do not fit shared memory, need more than the 128 registers that two CTAs leave: their
// variants spill 28 to 708 bytes of stores (28672x8192, 16 rows: 28 bytes, 0.9 warps eligible).
//
// Prob supplies: jobs, a Cursor over them with first() and next(cursor), first_row(cursor, group,
// tile) and last_row(cursor, tile) -> rows of M, col(cursor, j, odd) -> the lane's column of n-tile
// j (XS: byte offset of its first word in shared memory, else address) and whether it is an odd
// one (x_place), tiles(cursor) -> n-tiles that have a column, ready() (called once, with the first
// copies under way) and end(cursor, job, acc) (every warp calls it once per job; acc is in units of
// 1 / kCodeUnit).
constexpr int kWarps = 8;
constexpr int kRowStages = 4;                    // stages times row tiles of a ring
constexpr int kTileScales = 2048;                // in a stage of a tile: codes, then 16 bytes of
constexpr int kTileZeros = 2048 + 256;           // scales and 8 of zero points a row
constexpr int kTileBytes = 2048 + 256 + 128;
constexpr int kRingBytes = kWarps * kRowStages * kTileBytes;
// K-axis ranges of a row group for n columns: two units a warp where the axis has them, so that
// a job's fixed cost (joining the warps, its first loads) is shared by some work.  By n alone: a
// result does not depend on what else is in the call.
NQ_HD int k_ranges(int64_t n) {
    const int64_t u = ceil_div(n, kUnit);
    return u >= 16 ? 8 : u >= 8 ? 4 : u >= 4 ? 2 : 1;
}

// Place of word wi of a half of a column (one of its 16 words of 16 bytes): word c of lane t lies
// at 4 c + t, so that the lanes of a column read 64 consecutive bytes, and two neighbouring
// columns ("odd") read different halves of the banks.
template <int VW>
__device__ __forceinline__ int x_place(int wi, int odd) {
    const int c = VW == 4 ? wi & 3 : VW == 2 ? (wi >> 3) * 2 + (wi & 1) : wi >> 2;
    const int t = VW == 4 ? wi >> 2 : VW == 2 ? (wi >> 1) & 3 : wi & 3;
    return ((c ^ odd) << 2) + t;
}
// The same for word ``wd`` of a whole column (natural order for VW = 0, the tensor-memory path).
template <int VW>
__device__ __forceinline__ int x_word_place(int wd, int64_t col) {
    if constexpr (VW == 0) return wd;
    else return (wd & ~15) + x_place<VW>(wd & 15, (int)(col & 1));
}

// G scales (and zero points) of a row's unit, as registers.
template <int G, bool Z>
struct Scales {
    static constexpr int NS = (G + 1) / 2, NZ = (G + 3) / 4;
    uint32_t s[NS], z[NZ];
    // one by one from global memory; grp: the unit's first group, at: its place
    __device__ __forceinline__ void load(const Mat &M, int64_t at, int grp) {
#pragma unroll
        for (int i = 0; i < NS; ++i) s[i] = 0;
#pragma unroll
        for (int i = 0; i < NZ; ++i) z[i] = 0;
#pragma unroll
        for (int i = 0; i < G; ++i)
            if (grp + i < M.ng) {
                s[i / 2] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short *>(M.s) + at + i)
                            << (16 * (i & 1));
                if constexpr (Z) z[i / 4] |= (M.z ? (uint32_t)__ldg(M.z + at + i) : 8u) << (8 * (i & 3));
            }
    }
    // from a stage of the ring: row r of a tile
    __device__ __forceinline__ void load(uint32_t tile, int r, bool zeros) {
        const uint32_t ps = tile + kTileScales + r * 16, pz = tile + kTileZeros + r * 8;
        if constexpr (G == 2) {
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(s[0]) : "r"(ps));
        } else if constexpr (G == 4) {
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(s[0]), "=r"(s[1]) : "r"(ps));
        } else {
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3])
                         : "r"(ps));
        }
        if constexpr (Z) {
            if (!zeros) {
#pragma unroll
                for (int i = 0; i < NZ; ++i) z[i] = 0x08080808u;
            } else if constexpr (G == 8) {
                asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(z[0]), "=r"(z[1]) : "r"(pz));
            } else {
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(z[0]) : "r"(pz));
            }
        }
    }
    __device__ __forceinline__ float scale(int i) const {
        return __uint_as_float(i & 1 ? s[i / 2] & 0xffff0000u : s[i / 2] << 16);
    }
    __device__ __forceinline__ ZeroPoint zero(int i) const {
        if constexpr (Z) return zero_point(z[i / 4] >> (8 * (i & 3)) & 15u);
        return zero_point(8);
    }
};
// Whether the scales and zero points of a unit can be copied with its codes: every row's units
// are whole and start on a multiple of their size (zero points at least 4 bytes).
inline bool scales_vec(const Mat &M, int group) {
    const int G = kUnit / group, GZ = G < 4 ? 4 : G;
    return M.ng % G == 0 && reinterpret_cast<uintptr_t>(M.s) % (2 * G) == 0 &&
           reinterpret_cast<uintptr_t>(M.z) % GZ == 0;
}

template <int VW, bool Z, bool SV, bool XS, int MT, int NT, class Prob>
__device__ __forceinline__ void run_products(Prob &P, const Mat &M, int WK, char *ring) {
    constexpr int G = kUnit / (32 * VW);         // groups of a unit
    constexpr int kStage = MT * kTileBytes, kStages = kRowStages / MT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int wr = warp / WK, wk = warp % WK;
    const int units = (M.n + kUnit - 1) / kUnit;
    const int u0 = units * wk / WK, u1 = units * (wk + 1) / WK;      // never empty
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring) + warp * kStages * kStage;
    const int swz = VW == 4 ? (g & 1) << 2 : VW == 2 ? (g & 3) << 1 : g;

    // Producer cursor: job pj, its units from pu on.  A lane copies chunk pc of rows pr, pr + 4,
    // pr + 8, pr + 12 of a tile, each held to the last row that the tile may reach.
    const int pr = lane >> 3, pc = lane & 7;
    uint32_t put[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = pr + 4 * i;
        const int sw = VW == 4 ? (r & 1) << 2 : VW == 2 ? (r & 3) << 1 : r & 7;
        put[i] = r * 128 + ((pc ^ sw) << 4);
    }
    int pj = 0, pu = u0;
    typename Prob::Cursor pcur = P.first();
    const uint32_t *src[MT][4];
    int64_t gat[MT];                             // lanes 0..15: the unit's first scale of that row
    auto enter = [&]() {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int first = P.first_row(pcur, wr, m), last = P.last_row(pcur, m);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                src[m][i] = M.q + u0 * 32 + 4 * pc + (int64_t)min(first + pr + 4 * i, last) * M.ld;
            gat[m] = (int64_t)min(first + (lane & 15), last) * M.ng + u0 * G;
        }
    };
    auto issue = [&](uint32_t stage) {
        if (pj < P.jobs) {
            const bool in = pu * 32 + 4 * pc < M.ld;         // the row's words end here
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint32_t tile = stage + m * kTileBytes;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    copy16(tile + put[i], src[m][i], in);
                    src[m][i] += 32;
                }
                // lanes 0..15 the rows' scales, lanes 16..31 their zero points (G = 2: the
                // aligned word that holds the two)
                if constexpr (SV) {
                    if (lane < 16) {
                        if constexpr (G == 8)
                            copy16(tile + kTileScales + lane * 16, M.s + gat[m], true);
                        else
                            copy_small<2 * G>(tile + kTileScales + lane * 16, M.s + gat[m]);
                    } else if (Z && M.z) {
                        if constexpr (G == 2)
                            copy_small<4>(tile + kTileZeros + (lane & 15) * 8,
                                          M.z + (gat[m] & ~int64_t(3)), 2 + (int)(gat[m] & 2));
                        else
                            copy_small<G>(tile + kTileZeros + (lane & 15) * 8, M.z + gat[m]);
                    }
                }
                gat[m] += G;
            }
            if (++pu == u1) {
                pu = u0;
                if (++pj < P.jobs) {
                    P.next(pcur);
                    enter();
                }
            }
        }
        copy_commit();
    };

    // Consumer: scales of a unit that do not come with the ring, activations of a half, one step
    // ahead of their use.
    int64_t at[MT][2];                           // the unit's first scale of rows g and g + 8
    Scales<G, Z> sc[MT][2];
    int zrow[MT][2];                             // place of a row's first zero point in its word
    auto load_scales = [&](int unit) {
        if constexpr (!SV) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sc[m][h].load(M, at[m][h], unit * G);
                    at[m][h] += G;
                }
        }
    };
    const char *col[NT];                         // XS: shared-memory offsets
    int odd[NT];                                 // 64 for an odd column (x_place)
    int nt = NT;
    uint4 x[NT][4];
    auto load_x = [&](int half) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (j > 0 && j >= nt) break;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int off = t * 16 + (c & 2) * 64 + ((c & 1) ? 64 - odd[j] : odd[j]);
                if constexpr (XS) {
                    const uint32_t a = (uint32_t)reinterpret_cast<uintptr_t>(col[j]) +
                                       half * P.half_stride + off;
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(x[j][c].x), "=r"(x[j][c].y), "=r"(x[j][c].z), "=r"(x[j][c].w)
                                 : "r"(a));
                } else {
                    x[j][c] = *reinterpret_cast<const uint4 *>(col[j] + half * 256 + off);
                }
            }
        }
    };
    auto columns_of = [&](const typename Prob::Cursor &cur) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            bool is_odd;
            col[j] = P.col(cur, j, is_odd);
            odd[j] = is_odd ? 64 : 0;
        }
        nt = P.tiles(cur);
    };
    typename Prob::Cursor cur = pcur, after = pcur;      // the running job, the one after it
    auto start = [&]() {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t first = (int64_t)min(P.first_row(cur, wr, m) + g + 8 * h, P.last_row(cur, m)) *
                                      M.ng;
                if constexpr (!SV) at[m][h] = first + u0 * G;
                zrow[m][h] = (int)first & 2;
            }
        load_scales(u0);
    };

    enter();
    uint32_t stage = base;
#pragma unroll
    for (int s = 0; s < kStages; ++s) issue(base + s * kStage);
    P.ready();
    columns_of(cur);
    if constexpr (!XS) load_x(2 * u0);
    start();
    P.next(after);
    float acc[MT][NT][4] = {};
    for (int job = 0, unit = u0;;) {
        copy_wait<kStages - 1>();
        __syncwarp();
        Scales<G, Z> now[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (SV) {
                    now[m][h].load(stage + m * kTileBytes, g + 8 * h, M.z != nullptr);
                    // the two zero points of a unit in their aligned word
                    if (Z && G == 2 && M.z) now[m][h].z[0] >>= 8 * ((zrow[m][h] + unit * G) & 2);
                } else {
                    now[m][h] = sc[m][h];
                }
            }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t w[MT][2][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t row = stage + m * kTileBytes + (8 * h + g) * 128;
                    if constexpr (VW == 4) {
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(w[m][h][0]), "=r"(w[m][h][1]), "=r"(w[m][h][2]),
                                       "=r"(w[m][h][3])
                                     : "r"(row + (((half * 4 + t) ^ swz) << 4)));
                    } else if constexpr (VW == 2) {
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                                         : "=r"(w[m][h][2 * q]), "=r"(w[m][h][2 * q + 1])
                                         : "r"(row + (((half * 4 + 2 * q + (t >> 1)) ^ swz) << 4) +
                                               (t & 1) * 8));
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            asm volatile("ld.shared.u32 %0, [%1];"
                                         : "=r"(w[m][h][q])
                                         : "r"(row + (((half * 4 + q) ^ swz) << 4) + t * 4));
                    }
                }
            if constexpr (XS) load_x(2 * unit + half);
            if (half == 1) {
                __syncwarp();
                issue(stage);
                stage = stage == base + (kStages - 1) * kStage ? base : stage + kStage;
                if (unit + 1 < u1) load_scales(unit + 1);
            }
#pragma unroll
            for (int gi = 0; gi < G / 2; ++gi) {
                float c[MT][NT][4] = {};
#pragma unroll
                for (int v = 0; v < VW; ++v)
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const ZeroPoint z0 = now[m][0].zero(half * (G / 2) + gi),
                                        z1 = now[m][1].zero(half * (G / 2) + gi);
                        const uint32_t w0 = w[m][0][gi * VW + v], w1 = w[m][1][gi * VW + v];
                        const uint32_t a0[4] = {code_pair0(w0, z0), code_pair0(w1, z1),
                                                code_pair1(w0, z0), code_pair1(w1, z1)};
                        const uint32_t a1[4] = {code_pair0(w0 >> 8, z0), code_pair0(w1 >> 8, z1),
                                                code_pair1(w0 >> 8, z0), code_pair1(w1 >> 8, z1)};
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            if (j > 0 && j >= nt) break;
                            const uint4 b = x[j][gi * VW + v];
                            mma16816(c[m][j], a0, b.x, b.y);
                            mma16816(c[m][j], a1, b.z, b.w);
                        }
                    }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const float s0 = now[m][0].scale(half * (G / 2) + gi),
                                s1 = now[m][1].scale(half * (G / 2) + gi);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        acc[m][j][0] += s0 * c[m][j][0];
                        acc[m][j][1] += s0 * c[m][j][1];
                        acc[m][j][2] += s1 * c[m][j][2];
                        acc[m][j][3] += s1 * c[m][j][3];
                    }
                }
            }
            if constexpr (!XS) {
                if (half == 0 || unit + 1 < u1) {
                    load_x(2 * unit + half + 1);
                } else if (job + 1 < P.jobs) {   // the next job's first, while this one is joined
                    columns_of(after);
                    load_x(2 * u0);
                }
            }
        }
        if (++unit < u1) continue;
        P.end(cur, job, acc);
        unit = u0;
        if (++job == P.jobs) return;
        cur = after;
        P.next(after);
        start();
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
    }
}

// The WK warps of row group wr wait for one another.
__device__ __forceinline__ void group_sync(int wr, int WK) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + wr), "r"(32 * WK) : "memory");
}

// The warps' sums of a job side by side in shared memory: v[warp][row][column].
template <int MT, int NT>
struct Red {
    float v[kWarps][16 * MT][8 * NT + 1];
    __device__ __forceinline__ void put(const float (&acc)[MT][NT][4]) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[warp][16 * i + 8 * (e >> 1) + (lane >> 2)][8 * j + 2 * (lane & 3) + (e & 1)] =
                        acc[i][j][e];
    }
    // Sum over the WK warps of row group wr of columns c .. c + terms - 1 (the terms of one
    // value, small first).
    __device__ __forceinline__ float sum(int wr, int WK, int r, int c, int terms) const {
        float s = 0.f;
        for (int t = terms - 1; t >= 0; --t) {
            const float *p = &v[wr * WK][r][c + t];
            for (int w = 0; w < WK; ++w) s += p[w * (16 * MT) * (8 * NT + 1)];
        }
        return kCodeUnit * s;
    }
};

// ---------------------------------------------------------------------------------
// Host: launchers
// ---------------------------------------------------------------------------------
cudaError_t quantize(const void *W, int w_bf16, int64_t m, int64_t n, const float *d_in, int group,
                     int grid, uint32_t *q, __nv_bfloat16 *s, uint8_t *z, cudaStream_t st);
cudaError_t dequantize(const Mat &M, int64_t m, int group, void *out, int out_bf16,
                       cudaStream_t st);
// xw: workspace (matmul_workspace bytes) for the columns of X in word order, the parts of a split k
// axis and an error word.
size_t matmul_workspace(int64_t m, int64_t n, int x_bf16, int64_t B);
// Place of the error word in it; 0 where the call has none (no waits).
size_t matmul_error_word(int64_t m, int64_t n, int x_bf16, int64_t B);
cudaError_t matmul(const Mat &M, int64_t m, int group, const void *X, int x_bf16, int64_t B,
                   float *Y, __nv_bfloat16 *xw, cudaStream_t st);


// Polls of a device-side wait of the products and of the expert layer: ``most``, or fewer where
// nq_set_w4_wait_polls set so.
uint32_t wait_polls(uint32_t most);
void set_wait_polls(int polls);

// Many rows of X on tcgen05 (w4_tc.cu).
struct TcPlan {
    int BN;                    // rows of X of a tile
    int parts, part_units;     // parts of the k axis, units of kUnit columns of a part
    size_t partial_bytes;      // their sums ([parts][B][m]) if there is more than one
};
TcPlan tc_plan(int64_t m, int64_t n, int terms, int64_t B);
cudaError_t tc_matmul(const Mat &M, int64_t m, int group, const __nv_bfloat16 *xw, int terms, int64_t B,
                      float *Y, float *partial, int *err, cudaStream_t st);

// Expert layer for a few tokens (moe.cu).
struct MoeArgs {
    const void *X;             // [B][d], FP32 or BF16
    int x_bf16;
    int B, d, f, E, top_k, renormalise;
    const void *router;        // [E][d], of X's type
    Mat gate_up;               // E matrices of 2f x d, one after the other
    Mat down;                  // E matrices of d x f
    int group;
    uint32_t polls;            // of a wait for the other CTAs
    float *Y;                  // [B][d]
    int32_t *ids;              // [B][top_k] or null
    float *weights;            // [B][top_k] or null
    // workspace
    unsigned int *bar;         // two arrival counts
    int *err;                  // error word (behind the counts)
    double *logits;            // [ceil(d / 1024)][B][E]: parts of a logit
    uint4 *xw;                 // [B][1 or kTerms][padded(d) / 8], word order
    __nv_bfloat16 *h;          // [B top_k][kTerms][padded(f)], word order
    float *part;               // [B top_k][d]: an expert's output for a pair, not weighted
};
cudaError_t moe(const MoeArgs &a, cudaStream_t st);

}  // namespace w4
}  // namespace nq
