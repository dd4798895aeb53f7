// Product of a 4-bit layer with many rows of X on tcgen05 (sm_100a): Y^T = W^ X^T in tiles of
// 128 rows of W and BN rows of X.
//
// D = sum over k of (q - z) x is formed per group of g columns on the tensor cores, from exact
// operands (small integers in BF16; X in BF16, or FP32 as kTerms BF16 terms that share one
// operand), and drained group by group into FP32 registers as acc += s D: the scale of a row
// is one FMA of the drain, no product is rounded before the sum, and a sum in the tensor core
// never runs longer than a group.
//
// Persistent, one CTA an SM, nineteen warps around a ring of kRing stages of 128 columns of k:
//   warp 0      TMA: X (BN rows, kTerms times for FP32) into shared memory (128-byte swizzle)
//   warp 1      MMA issuer (M = 128, N = BN, K = 16, A from TMEM, B from shared memory)
//   warps 2-9   drain: thread = row of W, half of its BN sums in registers; stores
//   warps 10-17 decode: thread = row of W; codes go from shared memory through registers into
//               the A operand in TMEM (lane = row, two columns of k a word)
//   warp 18     TMA: the codes, 64 bytes a row and stage, into a ring of their own (64-byte
//               swizzle: a warp's 16-byte loads down its rows meet every bank once)
// One barrier says that a stage is full (the bytes of X and the four warps that decoded it), one
// that it is empty.  The A operand never touches shared memory, so the MMA reads only X there.
// The codes' pair order along k ((0,4) (1,5) (2,6) (3,7) of every 8) is that of the columns of X.
// Every mbarrier wait is bounded, and its outcome is one for the whole warp.  A role whose wait ran
// out ends and issues nothing more; the others then run out or end in turn, and the tiles that a
// drain did not get whole are stored as NaN.  Before such a CTA returns it waits for the copies and
// MMAs that are still under way.
//
// Measured, 11008x4096 g = 128, 2048 BF16 rows: 191 us, 964 TFLOP/s in a graph of 24 calls after a
// pause; 216 us in a run of seconds, under the power cap at a median of 1690 MHz.  The tensor pipe
// is active 51 % of the time and 63 % of the issue slots are used, the polls of waits among them; no
// unit is used up, and what is left is the hand-over of stages between the roles and the decoding of
// a row tile's codes for every 128 rows of X.  Decoding was a good part while one warp a quarter of the
// rows did it (239 us; 204 us in a copy with the decoding left out), two of them, stages in turn,
// brought it to 207 us.  Before: 64 columns a stage and a ring for each operand 549 us, four drain
// warps instead of eight 271 us.  g = 64: 277 us, g = 32: 474 us, with two and four drains a stage.
// FP32, 512 rows: 119 us (64 rows of X a tile, three terms each).
#include "gemm_tc.cuh"
#include "tc_ptx.cuh"
#include "w4.cuh"

#include <algorithm>

namespace nq {
namespace w4 {

using namespace tc;

constexpr int kDrainWarps = 8;                   // two to a quarter of the tile's rows, half the columns each
constexpr int kDecodeWarps = 8;                  // two to a quarter of the rows, stages in turn
constexpr int kTcThreads = 32 * (2 + kDrainWarps + kDecodeWarps + 1);
constexpr int kRing = 4;                         // stages
constexpr int kStageK = 128;                     // columns of k of a stage
constexpr int kStageA = kStageK / 2;             // TMEM columns of a stage of the A operand
constexpr int kCodeBytes = BM * kStageK / 2;     // codes of a stage: 64 bytes a row
constexpr int kSplitUnit = kUnit / kStageK;      // stages of the least part of a split k axis

struct TcArgs {
    Mat M;
    int m, B;
    int stages, parts, part_stages;              // stages of k; parts of the k axis; stages of a part
    int ntiles, units;                           // tiles of X; (row tile, tile of X, part) units
    float *out;                                  // [parts][B][m]
    float out_scale;
    uint32_t polls;                              // of a wait
    int *err;                                    // NQ_ERR_TIMEOUT where one ran out
};
struct TcMaps {
    CUtensorMap x[kTerms];
    CUtensorMap codes;         // [m][ld] words, 16 x 128 a box, 64-byte swizzle
};

// 32 words a lane into TMEM.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
        "%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
        "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
        "r"(r[30]), "r"(r[31])
        : "memory");
}

// 16 or 32 columns of a lane's TMEM row, asynchronously.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
// The registers may be read from here on.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
// The registers may be read from here on.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// D (TMEM) += A (TMEM) B (shared memory).
__device__ __forceinline__ void mma_bf16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// acc (two columns) += s v.
__device__ __forceinline__ void fma2(float2 &acc, float s, uint32_t v0, uint32_t v1) {
    uint64_t a = *reinterpret_cast<uint64_t *>(&acc), v, ss;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(v0), "r"(v1));
    asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(v), "l"(ss));
    acc = *reinterpret_cast<float2 *>(&a);
}

// All lanes of the warp wait, and agree on the outcome.  Each sees the phase itself: what one lane saw,
// handed on by a shuffle, would not order the others' reads behind the wait.  (Faster, too: 11008x4096
// g = 32, 2048 rows 543 -> 474 us, 28672x8192, 32 rows 66 -> 58 us.)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint32_t polls) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, nullptr, polls));
}

// Stages of the ring of codes: it runs ahead of the other one, so that codes come from memory
// well before they are decoded.
NQ_HD constexpr int tc_code_stages(int BN, int T) { return BN * T > 128 ? 4 : 8; }
template <int BN, int T>
constexpr int tc_smem() {
    return kRing * T * BN * kStageK * 2 + tc_code_stages(BN, T) * kCodeBytes + 1024 + 512;
}
// What the roles leave behind for a CTA in which a wait ran out.
struct Unfinished {
    int lost;                                    // a wait ran out
    uint32_t mma_groups;                         // groups whose MMAs were issued
    uint32_t x_issued, c_issued;                 // stages of X and of codes asked for
    uint32_t decoded[kDecodeWarps];              // stages before this one (of its turn) are decoded
};

// GS: MMA steps (16 columns of k) of a group.
template <int BN, int T, int GS>
__global__ void __launch_bounds__(kTcThreads, 1)
    w4_tc_kernel(const __grid_constant__ TcMaps maps, const TcArgs a) {
    constexpr int HALF = BN * BK * 2;            // bytes of 64 columns of BN rows of X
    constexpr int STAGE = T * 2 * HALF;
    constexpr int GROUP = 16 * GS, GROUPS = kStageK / GROUP;
    constexpr int CODES = tc_code_stages(BN, T);
    constexpr uint32_t TMEM_COLS = 512;          // two accumulators of BN columns, the A ring
    static_assert(2 * BN + kRing * kStageA <= 512, "tensor memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *codes = smem + kRing * STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(codes + CODES * kCodeBytes);
    uint64_t *empty = full + kRing, *d_full = empty + kRing, *d_empty = d_full + 2,
             *c_full = d_empty + 2, *c_empty = c_full + CODES;
    uint64_t *rest = c_empty + CODES;            // the MMAs of a CTA in which a wait ran out
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(rest + 1);
    Unfinished *un = reinterpret_cast<Unfinished *>(tmem_slot + 1);
    static_assert((2 * kRing + 4 + 2 * CODES + 1) * 8 + 4 + sizeof(Unfinished) <= 512, "barriers");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kRing; ++s) mbar_init(&full[s], 5), mbar_init(&empty[s], 1);
        for (int s = 0; s < 2; ++s) mbar_init(&d_full[s], 1), mbar_init(&d_empty[s], kDrainWarps);
        for (int s = 0; s < CODES; ++s) mbar_init(&c_full[s], 1), mbar_init(&c_empty[s], 4);
        mbar_init(rest, 1);
        un->lost = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot, tmem_a = tmem + 2 * BN;

    // unit u: part u % parts of tile u / parts; its stages of k
    auto stages_of = [&](int unit, int &k0, int &k1) {
        k0 = unit % a.parts * a.part_stages;
        k1 = min(a.stages, k0 + a.part_stages);
    };

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int unit = blockIdx.x; unit < a.units && ok; unit += gridDim.x) {
                int k0, k1;
                stages_of(unit, k0, k1);
                const int n0 = unit / a.parts % a.ntiles * BN;
                for (int k = k0; k < k1; ++k, ++it) {
                    const int s = it % kRing;
                    if (it >= kRing && !mbar_wait(&empty[s], (it / kRing - 1) & 1, nullptr, a.polls)) {
                        ok = false;
                        break;
                    }
                    mbar_expect_tx(&full[s], STAGE);
#pragma unroll
                    for (int t = 0; t < T; ++t)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            tma_load_2d(smem + s * STAGE + (2 * t + h) * HALF, &maps.x[t],
                                        k * kStageK + h * BK, n0, &full[s]);
                }
            }
            un->x_issued = it;
            if (!ok) un->lost = 1;
        }
    } else if (warp == 1) {
        // the whole warp walks the loop, so that the operands' addresses are uniform; one lane
        // issues
        constexpr uint32_t idesc = instr_desc_bf16(BM, BN);
        const bool leader = elect_one();
        const uint64_t desc0 = smem_desc_sw128(smem);
        uint32_t it = 0, grp = 0;
        bool ok = true;
        for (int unit = blockIdx.x; unit < a.units && ok; unit += gridDim.x) {
            int k0, k1;
            stages_of(unit, k0, k1);
            for (int k = k0; k < k1 && ok; ++k, ++it) {
                const uint32_t s = it % kRing;
                ok = warp_wait(&full[s], it / kRing & 1, a.polls);
                if (!ok) break;
                const uint64_t desc = desc0 + s * (STAGE / 16);
                const uint32_t at = tmem_a + s * kStageA;
#pragma unroll
                for (int g = 0; g < GROUPS; ++g, ++grp) {
                    const uint32_t d = tmem + (grp & 1) * BN;
                    if (grp >= 2) ok = warp_wait(&d_empty[grp & 1], (grp / 2 - 1) & 1, a.polls);
                    if (!ok) break;              // (the drain may still be reading this accumulator)
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int i = 0; i < GS; ++i) {
                            const int step = g * GS + i;     // 16 columns of k of the stage
#pragma unroll
                            for (int t = 0; t < T; ++t)
                                mma_bf16_ts(d, at + 8 * step,
                                            desc + ((2 * t + step / 4) * HALF / 16 + step % 4 * 2), idesc,
                                            i != 0 || t != 0);
                        }
                        // the stage's release comes before its last group's: the drain's wait
                        // for the unit's last group then covers every commit of the unit
                        if (g == GROUPS - 1) mma_commit(&empty[s]);
                        mma_commit(&d_full[grp & 1]);
                    }
                    __syncwarp();
                }
            }
        }
        if (leader) {
            un->mma_groups = grp;
            if (!ok) un->lost = 1;
        }
    } else if (warp < 2 + kDrainWarps) {
        // drain: rows of quarter q, columns c0 .. c0 + COLS - 1
        constexpr int COLS = BN / 2, LD = COLS == 32 ? 32 : 16;
        const int q = warp & 3, c0 = (warp - 2) / 4 * COLS;
        uint32_t grp = 0;
        bool dead = false;
        for (int unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
            int k0, k1;
            stages_of(unit, k0, k1);
            const int tile = unit / a.parts, n0 = tile % a.ntiles * BN + c0;
            const int row = tile / a.ntiles * BM + 32 * q + lane;
            const unsigned short *scales = reinterpret_cast<const unsigned short *>(a.M.s) +
                                           (int64_t)min(row, a.m - 1) * a.M.ng;
            const int g1 = k1 * GROUPS;
            float2 acc[COLS / 2];
#pragma unroll
            for (int j = 0; j < COLS / 2; ++j) acc[j] = make_float2(0.f, 0.f);
            // scales are asked for a group ahead, as they are (past the last group: any; those
            // groups' columns are zero)
            uint32_t s_next = __ldg(scales + k0 * GROUPS);
            for (int g = k0 * GROUPS; g < g1 && !dead; ++g, ++grp) {
                const float s = __uint_as_float(s_next << 16);
                s_next = __ldg(scales + min(g + 1, a.M.ng - 1));
                if (!warp_wait(&d_full[grp & 1], grp / 2 & 1, a.polls)) {
                    dead = true;
                    break;
                }
                tc_fence_after();
                const uint32_t base = tmem + (grp & 1) * BN + c0 + ((uint32_t)(32 * q) << 16);
#pragma unroll
                for (int c = 0; c < COLS; c += LD) {
                    uint32_t v[LD];
                    tmem_ld(base + c, v);
                    tmem_ld_wait(v);
#pragma unroll
                    for (int j = 0; j < LD; j += 2) fma2(acc[(c + j) / 2], s, v[j], v[j + 1]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&d_empty[grp & 1]);
            }
            if (row < a.m) {
                float *dst = a.out + ((int64_t)(unit % a.parts) * a.B + n0) * a.m + row;
                const float f = dead ? __int_as_float(0x7fc00000) : a.out_scale;
#pragma unroll
                for (int j = 0; j < COLS; ++j)
                    if (n0 + j < a.B) dst[(int64_t)j * a.m] = f * (j & 1 ? acc[j / 2].y : acc[j / 2].x);
            }
        }
        if (dead && lane == 0) un->lost = 1;
    } else if (warp == 2 + kDrainWarps + kDecodeWarps) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int unit = blockIdx.x; unit < a.units && ok; unit += gridDim.x) {
                int k0, k1;
                stages_of(unit, k0, k1);
                const int r0 = unit / a.parts / a.ntiles * BM;
                for (int k = k0; k < k1; ++k, ++it) {
                    const int s = it % CODES;
                    if (it >= CODES && !mbar_wait(&c_empty[s], (it / CODES - 1) & 1, nullptr, a.polls)) {
                        ok = false;
                        break;
                    }
                    mbar_expect_tx(&c_full[s], kCodeBytes);
                    tma_load_2d(codes + s * kCodeBytes, &maps.codes, k * (kStageK / 8), r0, &c_full[s]);
                }
            }
            un->c_issued = it;
            if (!ok) un->lost = 1;
        }
    } else {
        // decode: the warps of a quarter take its stages in turn
        const int q = warp & 3, r = 32 * q + lane;
        const uint32_t turn = (warp - 2 - kDrainWarps) / 4;
        uint32_t it = 0;
        bool ok = true;
        for (int unit = blockIdx.x; unit < a.units && ok; unit += gridDim.x) {
            int k0, k1;
            stages_of(unit, k0, k1);
            const int row = min(unit / a.parts / a.ntiles * BM + r, a.m - 1);
            const uint8_t *zeros = a.M.z + (int64_t)row * a.M.ng;
#pragma unroll 1
            for (int k = k0; k < k1; ++k, ++it) {
                if ((it & 1) != turn) continue;
                uint32_t zv[GROUPS];
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
                    zv[g] = a.M.z ? __ldg(zeros + min(k * GROUPS + g, a.M.ng - 1)) : 8u;
                const uint32_t cs = it % CODES, s = it % kRing;
                if (!warp_wait(&c_full[cs], it / CODES & 1, a.polls) ||
                    (it >= kRing && !warp_wait(&empty[s], (it / kRing - 1) & 1, a.polls))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // 16 words of the row, in chunks of 16 bytes that the copy permuted with it
                const uint32_t base = smem_u32(codes + cs * kCodeBytes) + r * 64;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[8], v[32];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(w[4 * c]), "=r"(w[4 * c + 1]), "=r"(w[4 * c + 2]),
                                       "=r"(w[4 * c + 3])
                                     : "r"(base + (((2 * h + c) ^ (r >> 1 & 3)) << 4)));
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const ZeroPoint z = zero_point(zv[(8 * h + c) * 8 / GROUP] & 15u);
                        v[4 * c] = code_pair0(w[c], z);
                        v[4 * c + 1] = code_pair1(w[c], z);
                        v[4 * c + 2] = code_pair0(w[c] >> 8, z);
                        v[4 * c + 3] = code_pair1(w[c] >> 8, z);
                    }
                    tmem_st32(tmem_a + s * kStageA + 32 * h + ((uint32_t)(32 * q) << 16), v);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&c_empty[cs]);
                    mbar_arrive(&full[s]);
                }
            }
        }
        if (lane == 0) {
            un->decoded[warp - 2 - kDrainWarps] = it;
            if (!ok) un->lost = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (un->lost) {
        if (threadIdx.x == 0) raise_error(a.err, NQ_ERR_TIMEOUT);
        // copies and MMAs that nobody waits for any more end by themselves, and their shared and
        // tensor memory is given back after that
        if (warp == 1) {
            if (elect_one() && un->mma_groups > 0) {
                mma_commit(rest);
                mbar_wait(rest, 0, nullptr);
            }
            __syncwarp();
        } else if (threadIdx.x == 0) {
            // the last phase of each stage; decode warps that ended before it owe their arrivals
            for (uint32_t it = un->x_issued > kRing ? un->x_issued - kRing : 0; it < un->x_issued; ++it) {
                for (int w = 0; w < 4; ++w)
                    if (un->decoded[4 * (it & 1) + w] <= it) mbar_arrive(&full[it % kRing]);
                mbar_wait(&full[it % kRing], it / kRing & 1, nullptr);
            }
            for (uint32_t it = un->c_issued > CODES ? un->c_issued - CODES : 0; it < un->c_issued; ++it)
                mbar_wait(&c_full[it % CODES], it / CODES & 1, nullptr);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(TMEM_COLS)
                     : "memory");
    }
}

// Y = sum over the parts, in their order (in the unit of the codes until then, which keeps them in
// range where Y is).
__global__ void __launch_bounds__(256)
    w4_sum_parts_kernel(const float *__restrict__ part, int parts, int64_t count,
                        float *__restrict__ Y) {
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < count;
         i += (int64_t)gridDim.x * blockDim.x) {
        float v = 0.f;
        for (int p = 0; p < parts; ++p) v += part[p * count + i];
        Y[i] = kCodeUnit * v;
    }
}

TcPlan tc_plan(int64_t m, int64_t n, int terms, int64_t B) {
    TcPlan p;
    p.BN = B <= 32 ? 32 : B <= 64 || terms > 1 ? 64 : 128;
    const int64_t tiles = ceil_div(m, BM) * ceil_div(B, p.BN), axis = ceil_div(n, kUnit);
    int64_t parts = tiles >= kNumSMsB200 ? 1 : kNumSMsB200 / tiles;
    if (parts > axis / 2) parts = axis / 2;      // at least two units of k a part
    if (parts < 1) parts = 1;
    p.part_units = (int)ceil_div(axis, parts);
    p.parts = (int)ceil_div(axis, p.part_units); // none of them empty
    p.partial_bytes = p.parts > 1 ? (size_t)p.parts * B * m * 4 : 0;
    return p;
}

template <int BN, int T, int GS>
static cudaError_t tc_launch_g(const TcMaps &maps, const TcArgs &a, cudaStream_t st) {
    auto kern = w4_tc_kernel<BN, T, GS>;
    constexpr int smem = tc_smem<BN, T>();
    static_assert(smem <= 227 * 1024, "shared memory of the ring of X");
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_smem_limit((const void *)kern, smem, configured);
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count();
    kern<<<(unsigned)(a.units < sms ? a.units : sms), kTcThreads, smem, st>>>(maps, a);
    count_launch();
    return cudaGetLastError();
}

template <int BN, int T>
static cudaError_t tc_launch(const TcMaps &maps, const TcArgs &a, int group, cudaStream_t st) {
    return group == 32   ? tc_launch_g<BN, T, 2>(maps, a, st)
           : group == 64 ? tc_launch_g<BN, T, 4>(maps, a, st)
                         : tc_launch_g<BN, T, 8>(maps, a, st);
}

cudaError_t tc_matmul(const Mat &M, int64_t m, int group, const __nv_bfloat16 *xw, int terms, int64_t B,
                      float *Y, float *partial, int *err, cudaStream_t st) {
    const TcPlan p = tc_plan(m, M.n, terms, B);
    const int64_t ldx = padded(M.n);
    TcMaps maps;
    for (int t = 0; t < terms; ++t)
        if (!make_map_bf16(&maps.x[t], xw + t * ldx, B, ldx, terms * ldx, p.BN))
            return cudaErrorInvalidValue;
    if (!make_map_u32(&maps.codes, M.q, m, M.ld, kStageK / 8, BM)) return cudaErrorInvalidValue;
    TcArgs a;
    a.M = M;
    a.m = (int)m, a.B = (int)B;
    a.stages = (int)ceil_div(M.n, kStageK);
    a.parts = p.parts;
    a.part_stages = p.part_units * kSplitUnit;
    a.ntiles = (int)ceil_div(B, p.BN);
    a.units = (int)ceil_div(m, BM) * a.ntiles * p.parts;
    a.out = p.parts > 1 ? partial : Y;
    a.out_scale = p.parts > 1 ? 1.f : kCodeUnit;
    a.polls = wait_polls(kMbarSpinLimit);
    a.err = err;
    cudaError_t e;
    if (terms == 1)
        e = p.BN == 32    ? tc_launch<32, 1>(maps, a, group, st)
            : p.BN == 64  ? tc_launch<64, 1>(maps, a, group, st)
                          : tc_launch<128, 1>(maps, a, group, st);
    else
        e = p.BN == 32 ? tc_launch<32, kTerms>(maps, a, group, st)
                       : tc_launch<64, kTerms>(maps, a, group, st);
    if (e != cudaSuccess || p.parts == 1) return e;
    const int64_t count = B * m;
    w4_sum_parts_kernel<<<(unsigned)std::min<int64_t>(ceil_div(count, 256), 4 * kNumSMsB200), 256, 0, st>>>(
        partial, p.parts, count, Y);
    count_launch();
    return cudaGetLastError();
}

}  // namespace w4
}  // namespace nq
