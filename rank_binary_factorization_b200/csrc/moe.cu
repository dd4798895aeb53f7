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
    if constexpr (sizeof(T) == 4) {
        const int ldx = (int)round_up(a.d, 8);
        for (int k = threadIdx.x; k < ldx; k += blockDim.x) {
            __nv_bfloat16 t[kTerms];
            split_terms(k < a.d ? (float)x[k] : 0.f, t);
#pragma unroll
            for (int i = 0; i < kTerms; ++i) a.xt[((int64_t)b * kTerms + i) * ldx + k] = t[i];
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
// CTA: 16 of an expert's f rows, gate and up side by side (two row tiles of a warp), for the
// expert's pairs, 8 columns at a time.  h leaves in kTerms BF16 columns.
template <int VW>
__global__ void __launch_bounds__(32 * kMoeWarps) moe_gate_up_kernel(const MoeArgs a) {
    __shared__ Lists L;
    __shared__ float red[kMoeWarps][32][9];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    build_lists(L, a.ids, a.B * a.top_k, a.E);
    if ((int)blockIdx.y >= L.active) return;
    const int e = L.expert[blockIdx.y];
    const int r0 = blockIdx.x * 16;
    int64_t row[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            row[i][h] = ((int64_t)e * 2 + i) * a.f + min(r0 + 8 * h + (lane >> 2), a.f - 1);
    const int terms = a.x_bf16 ? 1 : kTerms;
    const int64_t ldx = a.x_bf16 ? a.d : split_ld(a.d);
    const __nv_bfloat16 *x = a.x_bf16 ? static_cast<const __nv_bfloat16 *>(a.X) : a.xt;
    Mat M = a.gate_up;
    const bool xvec = !a.x_bf16 || (a.d % 8 == 0 && reinterpret_cast<uintptr_t>(a.X) % 16 == 0);
    if (xvec) M.n = (int)split_ld(a.d);
    const int64_t ldh = split_ld(a.f);
    const int per = 8 / terms;
    const int p1 = L.first[blockIdx.y + 1];
    for (int p0 = L.first[blockIdx.y]; p0 < p1; p0 += per) {
        const int np = min(per, p1 - p0);
        const int c = lane >> 2;
        const __nv_bfloat16 *col[1] = {nullptr};
        if (c < np * terms)
            col[0] = x + ((int64_t)(L.pairs[p0 + c / terms] / a.top_k) * terms + c % terms) * ldx;
        float acc[2][1][4] = {};
        group_products<VW, 2, 1>(acc, M, row, col, xvec, warp, kMoeWarps);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                red[warp][16 * i + 8 * (q >> 1) + (lane >> 2)][2 * (lane & 3) + (q & 1)] =
                    acc[i][0][q];
        __syncthreads();
        for (int o = threadIdx.x; o < 16 * np; o += blockDim.x) {
            const int r = o % 16, p = o / 16;
            if (r0 + r >= ldh) continue;
            float g = 0.f, u = 0.f;
            for (int t = terms - 1; t >= 0; --t)
#pragma unroll
                for (int w = 0; w < kMoeWarps; ++w) {
                    g += red[w][r][p * terms + t];
                    u += red[w][16 + r][p * terms + t];
                }
            __nv_bfloat16 ht[kTerms];
            split_terms(r0 + r < a.f ? g / (1.f + expf(-g)) * u : 0.f, ht);
#pragma unroll
            for (int t = 0; t < kTerms; ++t)
                a.h[((int64_t)L.pairs[p0 + p] * kTerms + t) * ldh + r0 + r] = ht[t];
        }
    }
}

// ---- down projection and combination ---------------------------------------------------
// CTA: 16 rows of d, all active experts in ascending order; y is summed in shared memory.
template <int VW>
__global__ void __launch_bounds__(32 * kMoeWarps) moe_down_kernel(const MoeArgs a) {
    __shared__ Lists L;
    __shared__ float red[kMoeWarps][16][9];
    __shared__ float y[NQ_MOE_MAX_TOKENS][16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    build_lists(L, a.ids, a.B * a.top_k, a.E);
    for (int o = threadIdx.x; o < 16 * a.B; o += blockDim.x) y[o / 16][o % 16] = 0.f;
    const int r0 = blockIdx.x * 16;
    const int64_t ldh = split_ld(a.f);
    Mat M = a.down;
    M.n = (int)ldh;
    constexpr int per = 8 / kTerms;
    for (int i = 0; i < L.active; ++i) {
        int64_t row[1][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            row[0][h] = (int64_t)L.expert[i] * a.d + min(r0 + 8 * h + (lane >> 2), a.d - 1);
        const int p1 = L.first[i + 1];
        for (int p0 = L.first[i]; p0 < p1; p0 += per) {
            const int np = min(per, p1 - p0);
            const int c = lane >> 2;
            const __nv_bfloat16 *col[1] = {nullptr};
            if (c < np * kTerms)
                col[0] = a.h + ((int64_t)L.pairs[p0 + c / kTerms] * kTerms + c % kTerms) * ldh;
            float acc[1][1][4] = {};
            group_products<VW, 1, 1>(acc, M, row, col, true, warp, kMoeWarps);
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 4; ++q)
                red[warp][8 * (q >> 1) + (lane >> 2)][2 * (lane & 3) + (q & 1)] = acc[0][0][q];
            __syncthreads();
            for (int o = threadIdx.x; o < 16 * np; o += blockDim.x) {
                const int r = o % 16, p = o / 16, pair = L.pairs[p0 + p];
                float v = 0.f;
#pragma unroll
                for (int t = kTerms - 1; t >= 0; --t)
#pragma unroll
                    for (int w = 0; w < kMoeWarps; ++w) v += red[w][r][p * kTerms + t];
                y[pair / a.top_k][r] += a.weights[pair] * v;
            }
        }
    }
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * a.B; o += blockDim.x)
        if (r0 + o % 16 < a.d) a.Y[(int64_t)(o / 16) * a.d + r0 + o % 16] = y[o / 16][o % 16];
}

template <int VW>
static void moe_experts(const MoeArgs &a, cudaStream_t st) {
    const int pairs = a.B * a.top_k;
    moe_gate_up_kernel<VW><<<dim3((unsigned)ceil_div(a.f, 16), (unsigned)(pairs < a.E ? pairs : a.E)),
                             32 * kMoeWarps, 0, st>>>(a);
    count_launch();
    moe_down_kernel<VW><<<(unsigned)ceil_div(a.d, 16), 32 * kMoeWarps, 0, st>>>(a);
    count_launch();
}

cudaError_t moe(const MoeArgs &a, cudaStream_t st) {
    if (a.x_bf16)
        moe_router_kernel<__nv_bfloat16><<<(unsigned)a.B, 32 * kMoeWarps, 0, st>>>(a);
    else
        moe_router_kernel<float><<<(unsigned)a.B, 32 * kMoeWarps, 0, st>>>(a);
    count_launch();
    if (a.group == 32)
        moe_experts<1>(a, st);
    else if (a.group == 64)
        moe_experts<2>(a, st);
    else
        moe_experts<4>(a, st);
    return cudaGetLastError();
}

}  // namespace w4
}  // namespace nq
