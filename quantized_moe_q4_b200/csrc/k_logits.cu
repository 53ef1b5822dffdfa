// k_logits.cu -- logit rules: penalties for repeated tokens, biases and
// grammar masks on the logits of the LM head, and the greedy token and
// log-sum-exp of what is left.
//
// The page has no counterpart; its LM head ("A 35B Hybrid-Attention
// Mixture-of-Experts Model on a 6GB 2011 GPU", Dutch technical summary,
// Resultaten) is moe_q4_gemv here, and this is what follows it.
//
// One pass over the logits: a row is the work of one cluster, whose CTAs own
// consecutive slices of the vocabulary.  The sparse parts become dense in
// shared memory first -- a 32-bit word per token of the slice that counts its
// occurrences in the row's history -- while the slice's logits are already on
// their way into registers; then every logit is read once, ruled, written
// once if asked for, and enters a running (maximum, lowest index, sum of
// exponentials), which the cluster joins through distributed shared memory.
#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace moeq4 {

namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_CL = 8;           // CTAs per cluster (the portable limit)
constexpr int VEC = 4;              // logits per access
constexpr int BATCH = 8;            // accesses in flight per thread
constexpr int STEP = THREADS * VEC * BATCH;  // logits a CTA holds at a time
constexpr int MAX_SLICE = 32768;    // logits whose words fit the shared memory (128 KB)

// History word of a token: bit 31: it occurs in the prompt; low bits: times generated.
constexpr uint32_t IN_PROMPT = 0x80000000u;

struct Best {
    float m;   // largest processed logit (-inf: none)
    int i;     // its lowest token
    float s;   // sum of exp(l - m); NaN where a logit is NaN
};

// exp(v - m) with m >= v; equal infinities give 1, -inf gives 0.
__device__ __forceinline__ float exp_below(float v, float m) { return v == m ? 1.0f : __expf(v - m); }

__device__ __forceinline__ Best join(Best a, Best b) {
    const bool take = b.m > a.m || (b.m == a.m && b.i < a.i);
    Best r;
    r.m = fmaxf(a.m, b.m);
    r.i = take ? b.i : a.i;
    // a side without anything has s = 0 (or NaN, which has to stay)
    r.s = (a.m == r.m ? a.s : a.s * exp_below(a.m, r.m)) + (b.m == r.m ? b.s : b.s * exp_below(b.m, r.m));
    return r;
}

struct Row {
    float rep, pres, freq;
};

// The penalties of one logit; word = its history word.
__device__ __forceinline__ float penalise(float l, uint32_t word, const Row& r) {
    if (word) {
        l = l > 0.0f ? __fdiv_rn(l, r.rep) : __fmul_rn(l, r.rep);
        const uint32_t c = word & ~IN_PROMPT;
        if (c) l = __fsub_rn(__fsub_rn(l, __fmul_rn(r.freq, (float)c)), r.pres);
    }
    return l;
}

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

// f(token, position) for the entries [lo, hi) of an int32 list.
template <class F>
__device__ __forceinline__ void each_token(const int32_t* list, int64_t lo, int64_t hi, F f) {
    // 16-byte loads from the last aligned position at or before lo
    for (int64_t i = (lo & ~int64_t(3)) + 4 * threadIdx.x; i < hi; i += 4 * THREADS) {
        if (i >= lo && i + 4 <= hi) {
            const int4 q = __ldg(reinterpret_cast<const int4*>(list + i));
            f(q.x, i); f(q.y, i + 1); f(q.z, i + 2); f(q.w, i + 3);
        } else {
            for (int k = 0; k < 4; ++k)
                if (i + k >= lo && i + k < hi) f(__ldg(list + i + k), i + k);
        }
    }
}

// Dynamic shared memory: words[slice] (history word, or for a biased token
// the bits of its logit after penalties and bias), then biased[slice / 32]
// (bit set: the word is such a logit).  `slice` is a multiple of 32.
__global__ void __launch_bounds__(THREADS, 2) logits_kernel(const __grid_constant__ LogitArgs p, int slice) {
    extern __shared__ __align__(16) uint32_t s_mem[];
    __shared__ Best s_best[WARPS];
    __shared__ Best s_cl[MAX_CL];
    __shared__ int s_dup;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t rank, ncl;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncl));
    const int64_t t = blockIdx.x / ncl;
    const bool pick = p.token || p.lse;
    const float NEG = __int_as_float(0xff800000);
    if (pick) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    uint32_t* words = s_mem;
    uint32_t* biased = s_mem + slice;

    Row row;
    row.rep = p.rep ? __ldg(p.rep + t) : 1.0f;
    row.pres = p.pres ? __ldg(p.pres + t) : 0.0f;
    row.freq = p.freq ? __ldg(p.freq + t) : 0.0f;
    int64_t h0 = 0, h1 = 0, hg = 0, b0 = 0, b1 = 0;
    if (p.row_start) {
        h0 = clamp64(__ldg(p.row_start + t), 0, p.n_tokens);
        h1 = clamp64(__ldg(p.row_start + t + 1), h0, p.n_tokens);
        hg = p.generated ? __ldg(p.generated + t) : h0;
    }
    if (p.bias_start) {
        b0 = clamp64(__ldg(p.bias_start + t), 0, p.n_bias);
        b1 = clamp64(__ldg(p.bias_start + t + 1), b0, p.n_bias);
    }
    const bool dense = h1 > h0 || b1 > b0;
    // the row's mask: none, or a row of words; an index outside the masks
    // allows nothing
    const uint32_t* mask = nullptr;
    bool nothing = false;
    if (p.mask) {
        const int64_t m = p.mask_row ? (int64_t)__ldg(p.mask_row + t) : t;
        if (m >= 0 && m < p.n_masks)
            mask = p.mask + m * ((p.V + 31) / 32);
        else if (m != -1) {
            nothing = true;
            if (tid == 0 && rank == 0 && p.status) atomicOr(p.status, STATUS_BAD_MASK_INDEX);
        }
    }
    const float* in = p.logits + t * p.ld;
    float* out = p.out ? p.out + t * p.ldo : nullptr;
    const bool vec = (reinterpret_cast<uintptr_t>(in) & 15) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    Best best{NEG, 0x7fffffff, 0.0f};

    for (int64_t v0 = (int64_t)rank * slice; v0 < p.V; v0 += (int64_t)ncl * slice) {
        const int len = (int)min((int64_t)slice, p.V - v0);
        for (int s0 = 0; s0 < len; s0 += STEP) {
            // logits of this step: access j of thread tid covers tokens
            // s0 + (j * THREADS + tid) * VEC + 0..3 of the slice
            float l[BATCH][VEC];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int i = s0 + (j * THREADS + tid) * VEC;
                if (vec && i + VEC <= len) {
                    const float4 q = *reinterpret_cast<const float4*>(in + v0 + i);
                    l[j][0] = q.x; l[j][1] = q.y; l[j][2] = q.z; l[j][3] = q.w;
                } else {
#pragma unroll
                    for (int k = 0; k < VEC; ++k) l[j][k] = i + k < len ? in[v0 + i + k] : NEG;
                }
            }
            if (s0 == 0 && dense) {
                __syncthreads();  // (an earlier slice's words are done with)
                for (int i = tid; i < (len + 3) / 4; i += THREADS) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
                if (b1 > b0)
                    for (int i = tid; i < (len + 31) / 32; i += THREADS) biased[i] = 0;
                if (tid == 0) s_dup = 0;
                __syncthreads();
                each_token(p.tokens, h0, h1, [&](int v, int64_t at) {
                    const int64_t i = (int64_t)v - v0;
                    if (i < 0 || i >= len || v < 0) return;
                    if (at >= hg) atomicAdd(&words[i], 1u);
                    else atomicOr(&words[i], IN_PROMPT);
                });
                if (b1 > b0) {
                    for (int64_t e = b0 + tid; e < b1; e += THREADS) {
                        const int64_t i = (int64_t)__ldg(p.bias_token + e) - v0;
                        if (i < 0 || i >= len) continue;
                        const uint32_t bit = 1u << (i & 31);
                        if (atomicOr(&biased[i >> 5], bit) & bit) s_dup = 1;
                    }
                    __syncthreads();
                    for (int64_t e = b0 + tid; e < b1; e += THREADS) {
                        const int v = __ldg(p.bias_token + e);
                        const int64_t i = (int64_t)v - v0;
                        if (i < 0 || i >= len) continue;
                        bool last = true;  // the later entry of a token listed twice counts
                        if (s_dup)
                            for (int64_t f = e + 1; f < b1 && last; ++f) last = __ldg(p.bias_token + f) != v;
                        if (last)
                            words[i] = __float_as_uint(__fadd_rn(penalise(in[v0 + i], words[i], row), __ldg(p.bias_value + e)));
                    }
                }
                __syncthreads();  // (with outputs in place, nothing is written before this)
            }
            float top = NEG;
            bool nan = false;
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int i = s0 + (j * THREADS + tid) * VEC;
                if (i >= len) continue;
                uint32_t allowed = 0xfu;
                if (mask) allowed = __ldg(mask + ((v0 + i) >> 5)) >> (i & 31);
                if (nothing) allowed = 0;
                if (dense) {
                    const uint4 q = *reinterpret_cast<const uint4*>(words + i);
                    const uint32_t w[VEC] = {q.x, q.y, q.z, q.w};
                    const uint32_t over = b1 > b0 ? biased[i >> 5] >> (i & 31) : 0u;
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        l[j][k] = (over >> k) & 1u ? __uint_as_float(w[k]) : penalise(l[j][k], w[k], row);
                }
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    if (!((allowed >> k) & 1u)) l[j][k] = NEG;
                    if (i + k < len) {
                        top = fmaxf(top, l[j][k]);
                        nan |= l[j][k] != l[j][k];
                    }
                }
                if (out) {
                    if (vec && i + VEC <= len) {
                        *reinterpret_cast<float4*>(out + v0 + i) = make_float4(l[j][0], l[j][1], l[j][2], l[j][3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            if (i + k < len) out[v0 + i + k] = l[j][k];
                    }
                }
            }
            if (!pick) continue;
            if (nan) best.s = __int_as_float(0x7fffffff);
            if (top == NEG) continue;
            Best b{top, 0x7fffffff, 0.0f};
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int i = s0 + (j * THREADS + tid) * VEC;
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    if (i + k < len && l[j][k] == l[j][k]) {
                        b.s += exp_below(l[j][k], top);
                        if (l[j][k] == top) b.i = min(b.i, (int)(v0 + i + k));
                    }
            }
            best = join(best, b);
        }
    }
    if (!pick) return;
    // warp, CTA, cluster: always in the same order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Best b;
        b.m = __shfl_down_sync(0xffffffffu, best.m, o);
        b.i = __shfl_down_sync(0xffffffffu, best.i, o);
        b.s = __shfl_down_sync(0xffffffffu, best.s, o);
        best = join(best, b);
    }
    if (lane == 0) s_best[warp] = best;
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (tid == 0) {
        for (int w = 1; w < WARPS; ++w) best = join(best, s_best[w]);
        uint32_t a;
        asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(&s_cl[rank])));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(best.m) : "memory");
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a + 4), "r"(best.i) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 8), "f"(best.s) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank == 0 && tid == 0) {
        best = s_cl[0];
        for (uint32_t c = 1; c < ncl; ++c) best = join(best, s_cl[c]);
        const bool nan = best.s != best.s;
        if (p.token) p.token[t] = best.m == NEG ? -1 : best.i;
        if (p.lse) p.lse[t] = nan ? best.s : best.m == NEG ? NEG : best.m + logf(best.s);
        if (nan && p.status) atomicOr(p.status, STATUS_NAN_LOGIT);
    }
}

}  // namespace

cudaError_t launch_logits(const LogitArgs& p, const DeviceInfo& dev, cudaStream_t s) {
    // As many CTAs a row as the portable cluster has, fewer where a slice
    // would be under a thousand logits, or where rows alone fill the GPU and
    // the wider slice still fits one step.
    int ncl = MAX_CL;
    while (ncl > 1 && ((int64_t)(ncl / 2) * 1024 >= p.V ||
                       (p.T * (ncl / 2) >= 4 * dev.sm_count && (int64_t)(ncl / 2) * STEP >= p.V)))
        ncl /= 2;
    int64_t slice = ceil_div(ceil_div(p.V, ncl), 32) * 32;
    if (slice > MAX_SLICE) slice = MAX_SLICE;
    const bool dense = p.row_start || p.bias_start;
    const size_t smem = dense ? 4 * (size_t)slice + (size_t)slice / 8 : 0;
    int per_sm = 0;
    cudaError_t e = kernel_occupancy(reinterpret_cast<const void*>(logits_kernel), THREADS, smem, &per_sm);
    if (e != cudaSuccess) return e;
    const int64_t grid = p.T * ncl;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)ncl;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logits_kernel, p, (int)slice);
}

}  // namespace moeq4
