// Mixture-of-experts layer on 4-bit experts for a few tokens (sm_100a):
//   l_e = x . R_e;  the top_k largest (ties: the lowest expert);  p = softmax(l) over all
//   experts, or over the chosen ones (renormalise)
//   y = sum over the chosen e of p_e D_e (silu(G_e x) * (U_e x)),  silu(v) = v / (1 + exp(-v))
#include "w4.cuh"

namespace nq {
namespace w4 {

constexpr int kMoeWarps = 8;
constexpr int kMoeMaxPairs = NQ_MOE_MAX_TOKENS * NQ_MOE_MAX_TOP_K;

// ---- router -------------------------------------------------------------------------
// One CTA per token.  The logits are summed in FP64: which experts are chosen must not
// depend on the order of the sum.
template <typename T>
__global__ void __launch_bounds__(32 * kMoeWarps) moe_router_kernel(const MoeArgs a) {
    __shared__ double logit[NQ_MOE_MAX_EXPERTS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x;
    const T *x = static_cast<const T *>(a.X) + (int64_t)b * a.d;
    for (int e = warp; e < a.E; e += kMoeWarps) {
        const T *r = static_cast<const T *>(a.router) + (int64_t)e * a.d;
        double v = 0.0;
        for (int k = lane; k < a.d; k += 32) v += (double)(float)x[k] * (double)(float)r[k];
        v = warp_sum(v);
        if (lane == 0) logit[e] = v;
    }
    const int words = (int)(padded(a.d) / 8);
    for (int wd = threadIdx.x; wd < words; wd += blockDim.x) {
        uint4 *dst = reinterpret_cast<uint4 *>(a.xw);
        if constexpr (sizeof(T) == 2) {
            dst[(int64_t)b * words + wd] = x_word(x, wd * 8, a.d);
        } else {
            uint4 w[kTerms];
            x_words(x, wd * 8, a.d, w);
#pragma unroll
            for (int t = 0; t < kTerms; ++t) dst[((int64_t)b * kTerms + t) * words + wd] = w[t];
        }
    }
    __syncthreads();
    if (warp != 0) return;
    // lane l looks after experts l, l + 32, ...; the winner of each round leaves
    unsigned int gone = 0;
    double top = 0.0, sum = 0.0;
    double mine = 0.0;     // lane j: the j-th chosen logit
    int chosen = 0;
    for (int j = 0; j < a.top_k; ++j) {
        double best = 0.0;
        int at = -1;
        for (int e = lane, i = 0; e < a.E; e += 32, ++i)
            if (!(gone >> i & 1) && (at < 0 || logit[e] > best)) best = logit[e], at = e;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double ob = __shfl_xor_sync(0xffffffffu, best, o);
            const int oa = __shfl_xor_sync(0xffffffffu, at, o);
            if (oa >= 0 && (at < 0 || ob > best || (!(best > ob) && oa < at))) best = ob, at = oa;
        }
        at = __shfl_sync(0xffffffffu, at, 0);   // one choice, also among NaNs
        best = logit[at];
        if ((at & 31) == lane) gone |= 1u << (at >> 5);
        if (j == 0) top = best;
        sum += exp(best - top);
        if (lane == j) mine = best, chosen = at;
    }
    if (!a.renormalise) {
        sum = 0.0;
        for (int e = lane; e < a.E; e += 32) sum += exp(logit[e] - top);
        sum = warp_sum(sum);
    }
    if (lane < a.top_k) {
        a.ids[b * a.top_k + lane] = chosen;
        a.weights[b * a.top_k + lane] = (float)(exp(mine - top) / sum);
    }
}

// ---- (token, expert) pairs by expert -------------------------------------------------
// Experts that some token chose, in ascending order, and their pairs (pair = token top_k +
// choice).  The order of an expert's pairs does not reach any result: every pair is a
// column of its own.
struct Lists {
    int count[NQ_MOE_MAX_EXPERTS];
    short expert[NQ_MOE_MAX_EXPERTS];        // active expert a
    short first[NQ_MOE_MAX_EXPERTS + 1];     // its first place in pairs[]
    short at[NQ_MOE_MAX_EXPERTS];            // expert -> a
    short pairs[kMoeMaxPairs];
    int active;
};

__device__ void build_lists(Lists &L, const int32_t *ids, int npairs, int E) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) L.count[e] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < npairs; p += blockDim.x) atomicAdd(&L.count[ids[p]], 1);
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int na = 0, np = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < E ? L.count[e] : 0;
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
                L.count[e] = 0;
            }
            na += __popc(used);
            np += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) L.first[na] = (short)np, L.active = na;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < npairs; p += blockDim.x) {
        const int e = ids[p];
        L.pairs[L.first[L.at[e]] + atomicAdd(&L.count[e], 1)] = (short)p;
    }
    __syncthreads();
}

// ---- gate and up projections, activation ----------------------------------------------
// Job: 16 of an expert's f rows, gate and up side by side (two row tiles), against up to 8
// columns of its pairs.  h leaves in kTerms BF16 columns.  A CTA does one expert's jobs.
struct GateUpProb {
    int jobs, WK;
    static constexpr uint32_t half_stride = 0;
    const MoeArgs &a;
    const Lists &L;
    Red<2, 1> *red;
    int terms, per, e, first, pairs, r0, p0 = 0, np = 0;
    int64_t ldx, ldh;

    __device__ __forceinline__ int first_row(int, int wr, int i) const {
        return (e * 2 + i) * a.f + r0 + wr * 16;
    }
    __device__ __forceinline__ int last_row(int, int i) const { return (e * 2 + i + 1) * a.f - 1; }
    __device__ __forceinline__ void ready() const {}
    __device__ __forceinline__ void begin(int job) {
        p0 = first + job * per;
        np = min(per, first + pairs - p0);
    }
    __device__ __forceinline__ const char *col(int) const {
        const int c = min(((int)threadIdx.x & 31) >> 2, np * terms - 1);
        return reinterpret_cast<const char *>(
            a.xw + ((int64_t)(L.pairs[p0 + c / terms] / a.top_k) * terms + c % terms) * ldx);
    }
    __device__ __forceinline__ void end(int job, const float (&acc)[2][1][4]) {
        Red<2, 1> &R = red[job & 1];
        R.put(acc);
        __syncthreads();
        const int rows = 16 * (kWarps / WK);
        for (int o = threadIdx.x; o < rows * np; o += 32 * kWarps) {
            const int r = o % rows, p = o / rows, k = r0 + r;
            if (k >= ldh) continue;
            const float g = R.sum(r / 16, WK, r % 16, p * terms, terms),
                        u = R.sum(r / 16, WK, 16 + r % 16, p * terms, terms);
            __nv_bfloat16 ht[kTerms];
            split_terms(k < a.f ? g / (1.f + expf(-g)) * u : 0.f, ht);
#pragma unroll
            for (int t = 0; t < kTerms; ++t)
                a.h[((int64_t)L.pairs[p0 + p] * kTerms + t) * ldh + in_word(k)] = ht[t];
        }
    }
};

template <int VW, bool Z>
__global__ void __launch_bounds__(32 * kWarps, 2) moe_gate_up_kernel(const MoeArgs a) {
    extern __shared__ __align__(1024) char sm[];
    Red<2, 1> *red = reinterpret_cast<Red<2, 1> *>(sm + ring_bytes<2>());
    Lists &L = *reinterpret_cast<Lists *>(red + 2);
    build_lists(L, a.ids, a.B * a.top_k, a.E);
    if ((int)blockIdx.y >= L.active) return;
    const int WK = k_ranges(a.d);
    GateUpProb P{0, WK, a, L, red};
    P.terms = a.x_bf16 ? 1 : kTerms;
    P.per = 8 / P.terms;
    P.e = L.expert[blockIdx.y];
    P.first = L.first[blockIdx.y];
    P.pairs = L.first[blockIdx.y + 1] - P.first;
    P.r0 = blockIdx.x * 16 * (kWarps / WK);
    P.jobs = (P.pairs + P.per - 1) / P.per;
    P.ldx = padded(a.d);
    P.ldh = padded(a.f);
    run_products<VW, Z, false, 2, 1>(P, a.gate_up, a.svec_gate_up, WK, sm);
}

// ---- down projection and combination ---------------------------------------------------
// CTA: one block of rows of d, all active experts in ascending order (jobs: chunks of an
// expert's pairs); y is summed in shared memory.
struct DownProb {
    int jobs, WK;
    static constexpr uint32_t half_stride = 0;
    const MoeArgs &a;
    const Lists &L;
    Red<1, 1> *red;
    float *y;                              // [B][rows]
    const short *job_expert, *job_pair;    // active expert and first pair of a job
    int r0;
    int64_t ldh;
    int p0 = 0, np = 0;

    __device__ __forceinline__ int first_row(int job, int wr, int) const {
        return L.expert[job_expert[job]] * a.d + r0 + wr * 16;
    }
    __device__ __forceinline__ int last_row(int job, int) const {
        return (L.expert[job_expert[job]] + 1) * a.d - 1;
    }
    __device__ __forceinline__ void ready() const {}
    __device__ __forceinline__ void begin(int job) {
        p0 = job_pair[job];
        np = min(8 / kTerms, L.first[job_expert[job] + 1] - p0);
    }
    __device__ __forceinline__ const char *col(int) const {
        const int c = min(((int)threadIdx.x & 31) >> 2, np * kTerms - 1);
        return reinterpret_cast<const char *>(
            a.h + ((int64_t)L.pairs[p0 + c / kTerms] * kTerms + c % kTerms) * ldh);
    }
    __device__ __forceinline__ void end(int job, const float (&acc)[1][1][4]) {
        Red<1, 1> &R = red[job & 1];
        R.put(acc);
        __syncthreads();
        // one pair of a token per expert, and a barrier between two jobs: fixed order
        const int rows = 16 * (kWarps / WK);
        for (int o = threadIdx.x; o < rows * np; o += 32 * kWarps) {
            const int r = o % rows, p = o / rows, pair = L.pairs[p0 + p];
            y[pair / a.top_k * rows + r] +=
                a.weights[pair] * R.sum(r / 16, WK, r % 16, p * kTerms, kTerms);
        }
    }
};

template <int VW, bool Z>
__global__ void __launch_bounds__(32 * kWarps, 2) moe_down_kernel(const MoeArgs a) {
    extern __shared__ __align__(1024) char sm[];
    Red<1, 1> *red = reinterpret_cast<Red<1, 1> *>(sm + ring_bytes<1>());
    Lists &L = *reinterpret_cast<Lists *>(red + 2);
    short *job_expert = reinterpret_cast<short *>(&L + 1);
    short *job_pair = job_expert + kMoeMaxPairs;
    float *y = reinterpret_cast<float *>(job_pair + kMoeMaxPairs);
    __shared__ int njobs;
    const int WK = k_ranges(a.f), rows = 16 * (kWarps / WK);
    build_lists(L, a.ids, a.B * a.top_k, a.E);
    for (int o = threadIdx.x; o < rows * a.B; o += blockDim.x) y[o] = 0.f;
    if (threadIdx.x == 0) {
        int n = 0;
        for (int i = 0; i < L.active; ++i)
            for (int p = L.first[i]; p < L.first[i + 1]; p += 8 / kTerms, ++n)
                job_expert[n] = (short)i, job_pair[n] = (short)p;
        njobs = n;
    }
    __syncthreads();
    DownProb P{njobs, WK, a, L, red, y, job_expert, job_pair, (int)blockIdx.x * rows, padded(a.f)};
    run_products<VW, Z, false, 1, 1>(P, a.down, a.svec_down, WK, sm);
    __syncthreads();
    for (int o = threadIdx.x; o < rows * a.B; o += blockDim.x)
        if (P.r0 + o % rows < a.d) a.Y[(int64_t)(o / rows) * a.d + P.r0 + o % rows] = y[o];
}

template <class K>
static cudaError_t moe_launch(K kern, dim3 grid, int smem, const MoeArgs &a, cudaStream_t st,
                              std::atomic<uint64_t> &configured) {
    cudaError_t e = ensure_smem_limit((const void *)kern, smem, configured);
    if (e != cudaSuccess) return e;
    kern<<<grid, 32 * kWarps, smem, st>>>(a);
    count_launch();
    return cudaGetLastError();
}

template <int VW>
static cudaError_t moe_experts(const MoeArgs &a, cudaStream_t st) {
    static std::atomic<uint64_t> c0[2], c1[2];
    const int pairs = a.B * a.top_k;
    constexpr int s0 = ring_bytes<2>() + 2 * sizeof(Red<2, 1>) + sizeof(Lists);
    constexpr int s1 = ring_bytes<1>() + 2 * sizeof(Red<1, 1>) + sizeof(Lists) + 4 * kMoeMaxPairs +
                       NQ_MOE_MAX_TOKENS * 16 * kWarps * 4;
    const int zu = a.gate_up.z != nullptr, zd = a.down.z != nullptr;
    const int ru = 16 * (kWarps / k_ranges(a.d)), rd = 16 * (kWarps / k_ranges(a.f));
    // the columns of h past f are written by the blocks that cover them
    cudaError_t e = moe_launch(zu ? moe_gate_up_kernel<VW, true> : moe_gate_up_kernel<VW, false>,
                               dim3((unsigned)ceil_div(padded(a.f), ru),
                                    (unsigned)(pairs < a.E ? pairs : a.E)),
                               s0, a, st, c0[zu]);
    if (e != cudaSuccess) return e;
    return moe_launch(zd ? moe_down_kernel<VW, true> : moe_down_kernel<VW, false>,
                      dim3((unsigned)ceil_div(a.d, rd)), s1, a, st, c1[zd]);
}

cudaError_t moe(const MoeArgs &args, cudaStream_t st) {
    MoeArgs a = args;
    a.svec_gate_up = scales_vec(a.gate_up, a.group);
    a.svec_down = scales_vec(a.down, a.group);
    if (a.x_bf16)
        moe_router_kernel<__nv_bfloat16><<<(unsigned)a.B, 32 * kMoeWarps, 0, st>>>(a);
    else
        moe_router_kernel<float><<<(unsigned)a.B, 32 * kMoeWarps, 0, st>>>(a);
    count_launch();
    auto run = a.group == 32 ? moe_experts<1> : a.group == 64 ? moe_experts<2> : moe_experts<4>;
    return run(a, st);
}

}  // namespace w4
}  // namespace nq
