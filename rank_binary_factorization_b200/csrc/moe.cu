// Mixture-of-experts layer on 4-bit experts for a few tokens (sm_100a):
//   l_e = x . R_e;  the top_k largest (ties: the lowest expert);  p = softmax(l) over all
//   experts, or over the chosen ones (renormalise)
//   y = sum over the chosen e of p_e D_e (silu(G_e x) * (U_e x)),  silu(v) = v / (1 + exp(-v))
//
// Two launches: the logits, then one cooperative kernel for the choice, both products and the
// sum, whose CTAs wait for one another twice (the down product needs all of h, the sum all parts).
// An expert's rows are read once for all tokens that chose it (FP32: for every five).  Measured, bf16
// unless said: one token, 64 experts, top 6, 2048 x 1408: 27 us (latency: the choice, two grid waits,
// about one job a CTA in each product); 8 tokens, 64 experts, top 8, 4096 x 1024, g = 64 with zero
// points: 115 us, 290 MB (39 % of the copy rate, 59 % of the issue slots, 1.2 warps eligible a
// scheduler, so neither is used up: a warp's chain of copy, decode, MMA, and the joins of jobs);
// 16 tokens, 8 experts, top 2, 4096 x 11008, FP32: 278 us (three columns a token to multiply; every
// FP32 variant spills, 76 to 704 bytes of stores at 128 registers, and 0.8 warps are eligible).
// With a launch for each step: 84, 315, 580 us.  Gate and up jobs go up to padded(f) rows: the blocks
// past f (4 of 48 at f = 1408) work on the last row again and store the zeros of h's padding.
#include "w4.cuh"

namespace nq {
namespace w4 {

constexpr int kMoeMaxPairs = NQ_MOE_MAX_TOKENS * NQ_MOE_MAX_TOP_K;
constexpr int kRouterTokens = 8;       // tokens and columns of a CTA of the router: a thread
constexpr int kRouterThreads = 128;    // holds 8 columns of its expert and of each token
constexpr int kRouterColumns = 8 * kRouterThreads;

// ---- router logits, columns of X --------------------------------------------------------
// CTA: one expert, up to 8 tokens, 1024 columns; the sums are in FP64 (the parts of a logit are
// added up by ``choose``), so that which experts are chosen does not depend on their order.  The
// CTAs together also write X's columns in word order and clear the arrival counts and the error
// word of the kernel that follows.
template <typename T>
__device__ __forceinline__ void load8(const T *p, int left, bool vec, T (&v)[8]) {
    if (vec && left >= 8) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            reinterpret_cast<uint4 *>(v)[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : (T)0.f;
    }
}

template <typename T, int VW>
__global__ void __launch_bounds__(kRouterThreads) moe_logits_kernel(const MoeArgs a, int vec) {
    __shared__ double red[kRouterThreads / 32][kRouterTokens];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.x, b0 = blockIdx.y * kRouterTokens;
    const int nb = min(kRouterTokens, a.B - b0);
    const int k = blockIdx.z * kRouterColumns + threadIdx.x * 8, left = a.d - k;
    const T *X = static_cast<const T *>(a.X);
    __align__(16) T r[8], x[kRouterTokens][8];
    load8(static_cast<const T *>(a.router) + (int64_t)e * a.d + k, left, vec, r);
#pragma unroll
    for (int b = 0; b < kRouterTokens; ++b)
        if (b < nb) load8(X + (int64_t)(b0 + b) * a.d + k, left, vec, x[b]);
    if (e == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
        if (threadIdx.x < 2) a.bar[threadIdx.x] = 0;
        if (threadIdx.x == 2) *a.err = 0;
    }
    const int words = (int)(padded(a.d) / 8);
    const int ctas = gridDim.x * gridDim.y * gridDim.z,
              cta = (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
    for (int o = cta * kRouterThreads + threadIdx.x; o < a.B * words; o += ctas * kRouterThreads) {
        const int b = o / words, wd = o % words;
        if constexpr (sizeof(T) == 2) {
            a.xw[(int64_t)b * words + x_word_place<VW>(wd, b)] = x_word(X + (int64_t)b * a.d, wd * 8, a.d);
        } else {
            uint4 w[kTerms];
            x_words(X + (int64_t)b * a.d, wd * 8, a.d, w);
#pragma unroll
            for (int t = 0; t < kTerms; ++t) {
                const int64_t c = (int64_t)b * kTerms + t;
                a.xw[c * words + x_word_place<VW>(wd, c)] = w[t];
            }
        }
    }
    double rd[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rd[i] = (double)(float)r[i];
#pragma unroll
    for (int b = 0; b < kRouterTokens; ++b) {
        if (b >= nb) break;
        double v = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += rd[i] * (double)(float)x[b][i];
        v = warp_sum(v);
        if (lane == 0) red[warp][b] = v;
    }
    __syncthreads();
    if (threadIdx.x < nb) {
        double v = 0.0;
#pragma unroll
        for (int w = 0; w < kRouterThreads / 32; ++w) v += red[w][threadIdx.x];
        a.logits[((int64_t)blockIdx.z * a.B + b0 + threadIdx.x) * a.E + e] = v;
    }
}

// ---- choice of experts --------------------------------------------------------------------
// One warp, one token: the top_k largest logits (ties: the lowest expert) and their weights.
// logit: scratch of the warp, E values.
__device__ void choose(const MoeArgs &a, int b, double *logit, short *ids, float *weights) {
    const int lane = threadIdx.x & 31;
    const int slices = (a.d + kRouterColumns - 1) / kRouterColumns;
    for (int e = lane; e < a.E; e += 32) {
        double v = 0.0;
        for (int s = 0; s < slices; ++s) v += a.logits[((int64_t)s * a.B + b) * a.E + e];
        logit[e] = v;
    }
    __syncwarp();
    // Logits as whole numbers of the same order (NaNs above all others, or below); lane l looks
    // after experts l, l + 32, ...; the winner of each round leaves.
    unsigned int gone = 0;
    double mine = 0.0;     // lane j: the j-th chosen logit
    int chosen = 0;
    for (int j = 0; j < a.top_k; ++j) {
        unsigned long long best = 0;
        int at = 0x7fffffff;
        for (int e = lane, i = 0; e < a.E; e += 32, ++i) {
            if (gone >> i & 1) continue;
            const long long v = __double_as_longlong(logit[e] + 0.0);      // -0 counts as 0
            const unsigned long long key = v < 0 ? ~v : v | 1ll << 63;
            if (at == 0x7fffffff || key > best) best = key, at = e;
        }
        bool in = at != 0x7fffffff;
        const unsigned int hi = __reduce_max_sync(0xffffffffu, in ? (unsigned int)(best >> 32) : 0u);
        in = in && (unsigned int)(best >> 32) == hi;
        const unsigned int lo = __reduce_max_sync(0xffffffffu, in ? (unsigned int)best : 0u);
        in = in && (unsigned int)best == lo;
        at = (int)__reduce_min_sync(0xffffffffu, in ? (unsigned int)at : 0x7fffffffu);
        if ((at & 31) == lane) gone |= 1u << (at >> 5);
        if (lane == j) mine = logit[at], chosen = at;
    }
    const double top = __shfl_sync(0xffffffffu, mine, 0);
    const double p = lane < a.top_k ? exp(mine - top) : 0.0;
    double sum = p;
    if (!a.renormalise) {
        sum = 0.0;
        for (int e = lane; e < a.E; e += 32) sum += exp(logit[e] - top);
    }
    sum = warp_sum(sum);
    if (lane < a.top_k) {
        ids[b * a.top_k + lane] = (short)chosen;
        weights[b * a.top_k + lane] = (float)(p / sum);
    }
}

// ---- (token, expert) pairs by expert -------------------------------------------------
// Experts that some token chose, in ascending order, and their pairs (pair = token top_k +
// choice) by token: the same lists in every CTA.
struct Lists {
    short expert[NQ_MOE_MAX_EXPERTS];        // active expert a
    short first[NQ_MOE_MAX_EXPERTS + 1];     // its first place in pairs[]
    short pairs[kMoeMaxPairs];
    float weights[kMoeMaxPairs];
    int active, chunks;
    union {
        short at[NQ_MOE_MAX_EXPERTS];        // expert -> a, while the lists are built
        short chunk_first[kMoeMaxPairs];     // later: chunks of an expert's pairs, as many as one
    };                                       // job takes
    union {
        short ids[kMoeMaxPairs];             // chosen experts, pair by pair; likewise
        short chunk_active[kMoeMaxPairs];
    };
};

// users: scratch, two words of tokens an expert.
__device__ void build_lists(Lists &L, unsigned int (*users)[2], int npairs, int top_k, int E) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) users[e][0] = users[e][1] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < npairs; p += blockDim.x) {
        const int b = p / top_k;
        atomicOr(&users[L.ids[p]][b >> 5], 1u << (b & 31));
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int na = 0, np = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < E ? __popc(users[e][0]) + __popc(users[e][1]) : 0;
            const unsigned int used = __ballot_sync(0xffffffffu, c > 0);
            int incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (c > 0) {
                const int i = na + __popc(used & ((1u << lane) - 1));
                L.expert[i] = (short)e;
                L.first[i] = (short)(np + incl - c);
                L.at[e] = (short)i;
            }
            na += __popc(used);
            np += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) L.first[na] = (short)np, L.active = na;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < npairs; p += blockDim.x) {
        const int e = L.ids[p], b = p / top_k;
        const unsigned int below = (1u << (b & 31)) - 1;
        const int rank = b < 32 ? __popc(users[e][0] & below)
                                : __popc(users[e][0]) + __popc(users[e][1] & below);
        L.pairs[L.first[L.at[e]] + rank] = (short)p;
    }
    __syncthreads();
}

// Chunks of up to ``per`` pairs, expert by expert (all threads).
__device__ void build_chunks(Lists &L, int per) {
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int n = 0;
        for (int i0 = 0; i0 < L.active; i0 += 32) {
            const int i = i0 + lane;
            const int p0 = i < L.active ? L.first[i] : 0, p1 = i < L.active ? L.first[i + 1] : 0;
            const int c = (p1 - p0 + per - 1) / per;
            int incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            for (int k = 0; k < c; ++k) {
                L.chunk_active[n + incl - c + k] = (short)i;
                L.chunk_first[n + incl - c + k] = (short)(p0 + k * per);
            }
            n += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) L.chunks = n;
    }
    __syncthreads();
}

// ---- the experts ----------------------------------------------------------------------------
// Arrival of all CTAs (launched together): bounded.
__device__ __forceinline__ void arrive(unsigned int *bar) {
    __syncthreads();
    if (threadIdx.x == 0) release_add(bar, 1);
}
__device__ __forceinline__ bool all_arrived(unsigned int *bar, const MoeArgs &a) {
    bool ok = true;
    if (threadIdx.x == 0) {
        ok = wait_geq(bar, gridDim.x, a.polls);
        if (!ok) raise_error(a.err, NQ_ERR_TIMEOUT);
    }
    return __syncthreads_and(ok);
}

// The jobs of both projections: job k of a CTA is number blockIdx.x + k gridDim.x of (chunk of an
// expert's pairs, block of its rows).
struct ExpertJobs {
    int jobs, WK;
    static constexpr uint32_t half_stride = 0;
    const MoeArgs &a;
    const Lists &L;
    int terms, per, lrows, blocks;         // columns of a pair, pairs of a chunk, log2 rows of a block
    int chunk_step, block_step;            // from one job of a CTA to the next
    int64_t ld;                            // 16-byte words of a column
    struct Cursor {
        int chunk, block;
    };

    __device__ ExpertJobs(const MoeArgs &a_, const Lists &L_, int n, int rows, int terms_, int per_)
        : WK(k_ranges(n)), a(a_), L(L_), terms(terms_), per(per_) {
        lrows = 31 - __clz(16 * (kWarps / WK));
        blocks = (rows + (1 << lrows) - 1) >> lrows;
        chunk_step = gridDim.x / blocks;
        block_step = gridDim.x % blocks;
        ld = padded(n) / 8;
        const int all = L.chunks * blocks;
        jobs = ((int)blockIdx.x < all) ? (all - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    }
    __device__ __forceinline__ Cursor first() const {
        return {(int)blockIdx.x / blocks, (int)blockIdx.x % blocks};
    }
    __device__ __forceinline__ void next(Cursor &c) const {
        c.chunk += chunk_step;
        c.block += block_step;
        if (c.block >= blocks) c.block -= blocks, ++c.chunk;
    }
    // (a cursor past the last job is not looked at)
    __device__ __forceinline__ int expert(const Cursor &c) const {
        return L.expert[L.chunk_active[c.chunk]];
    }
    __device__ __forceinline__ int pairs(const Cursor &c) const {
        return min(per, L.first[L.chunk_active[c.chunk] + 1] - L.chunk_first[c.chunk]);
    }
    __device__ __forceinline__ int tiles(const Cursor &c) const { return (pairs(c) * terms + 7) / 8; }
    // the lane's column of n-tile j of a job as (pair, term)
    __device__ __forceinline__ void column(const Cursor &cur, int j, int &pair, int &term) const {
        const int c = min(8 * j + (((int)threadIdx.x & 31) >> 2), pairs(cur) * terms - 1);
        pair = L.pairs[L.chunk_first[cur.chunk] + c / terms];
        term = c % terms;
    }
};

// Gate and up projections: 16 rows of each side by side (two row tiles of a warp).  h leaves in
// kTerms BF16 columns, its padding past f as zeros.
template <int VW, int NT>
struct GateUpProb : ExpertJobs {
    Red<2, NT> *red;
    int64_t ldh;
    __device__ GateUpProb(const MoeArgs &a, const Lists &L, int terms, int per, Red<2, NT> *red_)
        : ExpertJobs(a, L, a.d, (int)padded(a.f), terms, per), red(red_), ldh(padded(a.f)) {}
    __device__ __forceinline__ int first_row(const Cursor &c, int wr, int i) const {
        return (expert(c) * 2 + i) * a.f + (c.block << lrows) + wr * 16;
    }
    __device__ __forceinline__ int last_row(const Cursor &c, int i) const {
        return (expert(c) * 2 + i + 1) * a.f - 1;
    }
    __device__ __forceinline__ void ready() const {}
    __device__ __forceinline__ const char *col(const Cursor &cur, int j, bool &odd) const {
        int pair, term;
        column(cur, j, pair, term);
        const int64_t c = (int64_t)(pair / a.top_k) * terms + term;
        odd = c & 1;
        return reinterpret_cast<const char *>(a.xw + c * ld);
    }
    __device__ __forceinline__ void end(const Cursor &cur, int job, const float (&acc)[2][NT][4]) {
        // two of them used in turn, or one where they are large (two barriers a job)
        const int wr = (threadIdx.x >> 5) / WK;
        Red<2, NT> &R = red[NT == 1 ? job & 1 : 0];
        if (NT > 1) group_sync(wr, WK);
        R.put(acc);
        group_sync(wr, WK);
        const int r0 = (cur.block << lrows) + 16 * wr, np = pairs(cur), p0 = L.chunk_first[cur.chunk];
        for (int o = threadIdx.x - wr * 32 * WK; o < 16 * np; o += 32 * WK) {
            const int r = o % 16, p = o / 16, k = r0 + r;
            if (k >= ldh) continue;              // (never: blocks divide it; without, one variant spills more)
            const float g = R.sum(wr, WK, r, p * terms, terms),
                        u = R.sum(wr, WK, 16 + r, p * terms, terms);
            __nv_bfloat16 ht[kTerms];
            split_terms(k < a.f ? g / (1.f + expf(-g)) * u : 0.f, ht);
#pragma unroll
            for (int t = 0; t < kTerms; ++t) {
                const int64_t c = (int64_t)L.pairs[p0 + p] * kTerms + t;
                a.h[c * ldh + x_word_place<VW>(k >> 3, c) * 8 + in_word(k & 7)] = ht[t];
            }
        }
    }
};

// Down projection, pair by pair.
template <int NT>
struct DownProb : ExpertJobs {
    Red<1, NT> *red;
    bool ok = true;                        // all of h was there (else its parts are NaN)
    __device__ DownProb(const MoeArgs &a, const Lists &L, int per, Red<1, NT> *red_)
        : ExpertJobs(a, L, a.f, a.d, kTerms, per), red(red_) {}
    __device__ __forceinline__ int first_row(const Cursor &c, int wr, int) const {
        return expert(c) * a.d + (c.block << lrows) + wr * 16;
    }
    __device__ __forceinline__ int last_row(const Cursor &c, int) const {
        return (expert(c) + 1) * a.d - 1;
    }
    // the first copies of the weights are under way; h is complete when all CTAs have arrived
    __device__ __forceinline__ void ready() { ok = all_arrived(a.bar, a); }
    __device__ __forceinline__ const char *col(const Cursor &cur, int j, bool &odd) const {
        int pair, term;
        column(cur, j, pair, term);
        const int64_t c = (int64_t)pair * kTerms + term;
        odd = c & 1;
        return reinterpret_cast<const char *>(reinterpret_cast<const uint4 *>(a.h) + c * ld);
    }
    __device__ __forceinline__ void end(const Cursor &cur, int job, const float (&acc)[1][NT][4]) {
        Red<1, NT> &R = red[job & 1];
        R.put(acc);
        const int wr = (threadIdx.x >> 5) / WK;
        group_sync(wr, WK);
        const int r0 = (cur.block << lrows) + 16 * wr, np = pairs(cur), p0 = L.chunk_first[cur.chunk];
        for (int o = threadIdx.x - wr * 32 * WK; o < 16 * np; o += 32 * WK) {
            const int r = o % 16, p = o / 16;
            if (r0 + r < a.d)
                a.part[(int64_t)L.pairs[p0 + p] * a.d + r0 + r] =
                    ok ? R.sum(wr, WK, r, p * kTerms, kTerms) : __int_as_float(0x7fc00000);
        }
    }
};

// n-tiles of a job: BF16 tokens of an expert in eights, FP32 ones (three columns each) in fives, as
// are the pairs of the down projection; a tile without columns costs nothing.
constexpr int kDownTiles = 2;
NQ_HD constexpr int moe_up_tiles(int terms) { return terms == 1 ? 1 : 2; }
NQ_HD constexpr int moe_red_bytes(int terms) {
    return terms == 1 ? 2 * (int)sizeof(Red<2, 1>) : (int)sizeof(Red<2, 2>);
}
static_assert(2 * sizeof(Red<1, kDownTiles>) <= 2 * sizeof(Red<2, 1>) &&
                  2 * sizeof(Red<1, kDownTiles>) <= sizeof(Red<2, 2>),
              "the down projection's sums fit where the others were");

// All CTAs of the launch are resident together (cooperative launch): choice and lists in every
// CTA, gate and up jobs, arrival, down jobs, arrival, and y = sum over a token's choices of p times
// the pair's output, in the order of the choices.
template <int VW, bool Z, bool SV, int TERMS>
__global__ void __launch_bounds__(32 * kWarps, 2) moe_experts_kernel(const MoeArgs a) {
    constexpr int NU = moe_up_tiles(TERMS), ND = kDownTiles;
    extern __shared__ __align__(1024) char sm[];
    void *red = sm + kRingBytes;
    constexpr int kRed = moe_red_bytes(TERMS);
    Lists &L = *reinterpret_cast<Lists *>(sm + kRingBytes + kRed);
    const int pairs = a.B * a.top_k;
    // (the ring of copies is not in use yet: scratch)
    for (int b = threadIdx.x >> 5; b < a.B; b += kWarps) {
        choose(a, b, reinterpret_cast<double *>(sm) + (threadIdx.x >> 5) * NQ_MOE_MAX_EXPERTS, L.ids,
               L.weights);
        __syncwarp();
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int p = threadIdx.x; p < pairs; p += 32 * kWarps) {
            if (a.ids) a.ids[p] = L.ids[p];
            if (a.weights) a.weights[p] = L.weights[p];
        }
    build_lists(L, reinterpret_cast<unsigned int(*)[2]>(sm), pairs, a.top_k, a.E);
    build_chunks(L, 8 * NU / TERMS);
    {
        GateUpProb<VW, NU> P(a, L, TERMS, 8 * NU / TERMS, static_cast<Red<2, NU> *>(red));
        if (P.jobs > 0) run_products<VW, Z, SV, false, 2, NU>(P, a.gate_up, P.WK, sm);
    }
    __threadfence();
    arrive(a.bar);
    build_chunks(L, 8 * ND / kTerms);
    bool ok = true;
    {
        DownProb<ND> P(a, L, 8 * ND / kTerms, static_cast<Red<1, ND> *>(red));
        if (P.jobs > 0) {
            run_products<VW, Z, SV, false, 1, ND>(P, a.down, P.WK, sm);
            ok = P.ok;
        }
    }
    __threadfence();
    arrive(a.bar + 1);
    ok = all_arrived(a.bar + 1, a) && ok;
    const int64_t count = (int64_t)a.B * a.d;
    for (int64_t o = (int64_t)blockIdx.x * 32 * kWarps + threadIdx.x; o < count;
         o += (int64_t)gridDim.x * 32 * kWarps) {
        const int b = (int)(o / a.d), r = (int)(o % a.d);
        float y = 0.f;
        for (int j = 0; j < a.top_k; ++j)
            y += L.weights[b * a.top_k + j] * __ldcg(a.part + (int64_t)(b * a.top_k + j) * a.d + r);
        a.Y[o] = ok ? y : __int_as_float(0x7fc00000);       // a wait ran out
    }
}

template <int VW, bool Z, bool SV, int TERMS>
static cudaError_t moe_launch(const MoeArgs &a, cudaStream_t st) {
    constexpr int smem = kRingBytes + moe_red_bytes(TERMS) + (int)sizeof(Lists);
    auto kern = moe_experts_kernel<VW, Z, SV, TERMS>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_smem_limit((const void *)kern, smem, configured);
    if (e != cudaSuccess) return e;
    // CTAs an SM, per device (0: not asked yet)
    static std::atomic<int> fit[kMaxDevices];
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    int n = fit[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, 32 * kWarps, smem);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        fit[dev].store(n, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n * device_sm_count()));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int VW, bool Z>
static cudaError_t moe_experts(const MoeArgs &a, cudaStream_t st) {
    const bool sv = scales_vec(a.gate_up, a.group) && scales_vec(a.down, a.group);
    if (a.x_bf16) return sv ? moe_launch<VW, Z, true, 1>(a, st) : moe_launch<VW, Z, false, 1>(a, st);
    return sv ? moe_launch<VW, Z, true, kTerms>(a, st) : moe_launch<VW, Z, false, kTerms>(a, st);
}

cudaError_t moe(const MoeArgs &a, cudaStream_t st) {
    const dim3 grid((unsigned)a.E, (unsigned)ceil_div(a.B, kRouterTokens),
                    (unsigned)ceil_div(a.d, kRouterColumns));
    const int vec = (a.d * (a.x_bf16 ? 2 : 4)) % 16 == 0 && reinterpret_cast<uintptr_t>(a.X) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(a.router) % 16 == 0;
    using bf16 = __nv_bfloat16;
    auto logits = a.x_bf16 ? (a.group == 32   ? moe_logits_kernel<bf16, 1>
                              : a.group == 64 ? moe_logits_kernel<bf16, 2>
                                              : moe_logits_kernel<bf16, 4>)
                           : (a.group == 32   ? moe_logits_kernel<float, 1>
                              : a.group == 64 ? moe_logits_kernel<float, 2>
                                              : moe_logits_kernel<float, 4>);
    logits<<<grid, kRouterThreads, 0, st>>>(a, vec);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    auto run = a.gate_up.z || a.down.z
                   ? (a.group == 32   ? moe_experts<1, true>
                      : a.group == 64 ? moe_experts<2, true>
                                      : moe_experts<4, true>)
                   : (a.group == 32   ? moe_experts<1, false>
                      : a.group == 64 ? moe_experts<2, false>
                                      : moe_experts<4, false>);
    return run(a, st);
}

}  // namespace w4
}  // namespace nq
