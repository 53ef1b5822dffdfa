// k_logits.cu -- logit rules: penalties for repeated tokens, biases and
// grammar masks on the logits of the LM head, and the greedy token and
// log-sum-exp of what is left.
//
// The page has no counterpart; its LM head ("A 35B Hybrid-Attention
// Mixture-of-Experts Model on a 6GB 2011 GPU", Dutch technical summary,
// Resultaten) is moe_q4_gemv here, and this is what follows it.
//
// A row is the work of one cluster.  Its CTAs own the vocabulary's groups of 32
// tokens in turn (the tokens that histories are full of have low numbers, and
// would all fall to one CTA if each owned a range).  While the logits are on
// their way to L2, the few that penalties and biases change are worked out in
// shared memory: a 32-bit word per token counts its occurrences in the row's
// history and a bit says that there is one (two shared atomics a token, nothing
// that waits for them, so that long histories scan fast), the set bits become a
// list, and all threads fetch and rule the logits on it.  Then the logits are
// streamed once: four of them cost one test of four bits, the mask, a running
// maximum and, relative to the warp's maximum, one exponential each.  The
// CTAs' (maximum, lowest token, sum) are joined through distributed shared
// memory.  Bound by the logits' bytes (read, and written if asked for) without
// rules; with them a CTA spends half its time in the chain of dependent loads
// (row, tokens, their logits), which two CTAs an SM cover in part.
//
// Device times, one B200, 131072 tokens:
//   1 row with a history of 1000: 9.2 us (latency); 64 rows, histories of 2000,
//   64 biases, masks: 34 us; 32 rows, histories of 16384: 23 us; 256 rows,
//   histories of 1000, masks: 105 us, 2.6 TB/s (token and log-sum-exp only:
//   98 us); 256 rows without rules: all outputs 63 us, logits only 44 us, 6.1
//   TB/s, token and log-sum-exp only 49 us.
// Past 131072 tokens a CTA of eight holds more than STEP logits, so its stream
// takes a second turn, and from about 141,000 on (with a mask) its tables leave
// room for one CTA an SM only: the 64 rows above take 39 us at 131104 tokens, 69
// at 151936 and 82 at 248320.
#include <algorithm>
#include <type_traits>

#include "cluster.cuh"
#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace moeq4 {

namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_CL = 8;           // CTAs per cluster (the portable limit)
constexpr int BATCH = 8;            // 16-byte accesses in flight per thread
constexpr int STEP = THREADS * 4 * BATCH;  // logits a CTA holds at a time
constexpr int MAX_SLICE = 2 * STEP;  // logits whose words fit the shared memory (128 KB)

// History word of a token: bit 31: it occurs in the prompt; low bits: times generated.
constexpr uint32_t IN_PROMPT = 0x80000000u;

struct Best {
    float m;   // largest processed logit (-inf: none)
    int i;     // its lowest token
    float s;   // sum of exp(l - m); NaN where a logit is NaN
};

// exp(d) for d <= 0 (relative error 2^-22 + |d| 2^-23; below 2^-126: 0).
__device__ __forceinline__ float exp_neg(float d) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(d * 1.4426950408889634f));
    return e;
}

// exp(v - m) for m >= v, equal infinities included.
__device__ __forceinline__ float exp_below(float v, float m) { return v == m ? 1.0f : exp_neg(v - m); }

// (a side without anything has s = 0, or NaN, which has to stay)
__device__ __forceinline__ Best join(Best a, Best b) {
    Best r;
    r.m = fmaxf(a.m, b.m);
    r.i = b.m > a.m ? b.i : b.m < a.m ? a.i : min(a.i, b.i);
    r.s = a.s * exp_below(a.m, r.m) + b.s * exp_below(b.m, r.m);
    return r;
}

// Joins the first n (a power of two) lanes' values into lane 0, in a fixed order.
__device__ __forceinline__ Best join_lanes(Best b, int n) {
    for (int o = n / 2; o > 0; o >>= 1) {
        Best c;
        c.m = __shfl_down_sync(0xffffffffu, b.m, o);
        c.i = __shfl_down_sync(0xffffffffu, b.i, o);
        c.s = __shfl_down_sync(0xffffffffu, b.s, o);
        b = join(b, c);
    }
    return b;
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

// f(token, position) for the entries [lo, hi) of an int32 list, 16-byte loads
// from the last aligned position at or before lo, four of them in flight.
template <class F>
__device__ __forceinline__ void each_token(const int32_t* list, int64_t lo, int64_t hi, F f) {
    constexpr int FLY = 4;
    for (int64_t i0 = (lo & ~int64_t(3)) + 4 * threadIdx.x; i0 < hi; i0 += 4 * THREADS * FLY) {
        int4 q[FLY];
#pragma unroll
        for (int j = 0; j < FLY; ++j) {
            const int64_t i = i0 + 4 * THREADS * j;
            if (i >= lo && i + 4 <= hi) {
                q[j] = __ldg(reinterpret_cast<const int4*>(list + i));
            } else {  // (-1 is no token)
                q[j].x = i >= lo && i < hi ? __ldg(list + i) : -1;
                q[j].y = i + 1 >= lo && i + 1 < hi ? __ldg(list + i + 1) : -1;
                q[j].z = i + 2 >= lo && i + 2 < hi ? __ldg(list + i + 2) : -1;
                q[j].w = i + 3 >= lo && i + 3 < hi ? __ldg(list + i + 3) : -1;
            }
        }
#pragma unroll
        for (int j = 0; j < FLY; ++j) {
            const int64_t i = i0 + 4 * THREADS * j;
            f(q[j].x, i); f(q[j].y, i + 1); f(q[j].z, i + 2); f(q[j].w, i + 3);
        }
    }
}

// Dynamic shared memory: allowed[slice / 32] (the mask's words), and for rows
// with histories or biases words[slice] (history word, or for a ruled token
// the bits of its logit), ruled[slice / 32] (bit set: the word is such a
// logit), listed[slice / 32] (bit set: a bias lists the token), twice[slice /
// 32] (bit set: more than once), seen[slice] (16-bit: the places of the
// history's tokens).  Place i of a CTA's `slice`
// (a multiple of 32) is token base + 32 * (i / 32 * ncl + rank) + i % 32, with
// ncl = 1 << lg CTAs in the cluster.
__global__ void __launch_bounds__(THREADS, 2) logits_kernel(const __grid_constant__ LogitArgs p, int slice, int lg) {
    extern __shared__ __align__(16) uint32_t s_mem[];
    __shared__ Best s_best[WARPS];
    __shared__ Best s_cl[MAX_CL];
    __shared__ int s_seen;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int64_t t = blockIdx.x >> lg;
    const bool pick = p.token || p.lse;
    const float NEG = __int_as_float(0xff800000);
    if (pick) cluster_arrive();
    uint32_t* words = s_mem + (p.mask ? (slice / 32 + 3) / 4 * 4 : 0);
    uint32_t* ruled = words + slice;
    uint32_t* listed = ruled + slice / 32;
    uint32_t* twice = listed + slice / 32;
    uint16_t* seen = reinterpret_cast<uint16_t*>(twice + slice / 32);
    const float* in = p.logits + t * p.ld;
    float* out = p.out ? p.out + t * p.ldo : nullptr;
    const auto token_at = [&](uint32_t i) { return (((i >> 5 << lg) + rank) << 5) + (i & 31); };  // less base

    // What the rules need comes through a chain of dependent loads: the logits
    // are asked for before it begins.
    if (p.row_start || p.bias_start || p.mask)
        for (int g = tid; g < slice / 32; g += THREADS) {
            const uint32_t v = token_at(32 * g);
            if (v < p.V) prefetch_l2(in + v);
        }

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
    const bool vec = (reinterpret_cast<uintptr_t>(in) & 15) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    Best best{NEG, 0x7fffffff, 0.0f};

    for (int64_t base = 0; base < p.V; base += (int64_t)slice << lg) {
        const int left = (int)min(p.V - base, (int64_t)slice << lg);  // tokens of this turn, of all CTAs
        // this CTA's places: `len` with all of its last group; the group may end early
        const int groups = (left + 31) / 32, len = max(0, groups - (int)rank + (1 << lg) - 1 >> lg) * 32;
        const float* src = in + base;
        float* dst = out + base;
        const bool sparse = h1 > h0 || b1 > b0;
        if (sparse || mask) {
            // ---- the mask's words, and what penalties and biases change: worked
            // out before anything is written (outputs may be in place)
            const auto inside = [&](int v, uint32_t& i) {  // (vocabularies end at 2^30)
                const uint32_t u = (uint32_t)v - (uint32_t)base, g = u >> 5;
                i = (g >> lg << 5) + (u & 31);
                return u < (uint32_t)left && (g & ((1u << lg) - 1)) == rank;
            };
            if (base) __syncthreads();  // (an earlier turn's words are done with)
            if (mask)
                for (int g = tid; g < len / 32; g += THREADS) s_mem[g] = __ldg(mask + (base >> 5) + (((uint32_t)g << lg) + rank));
            if (sparse) {
                Row row;
                row.rep = p.rep ? __ldg(p.rep + t) : 1.0f;
                row.pres = p.pres ? __ldg(p.pres + t) : 0.0f;
                row.freq = p.freq ? __ldg(p.freq + t) : 0.0f;
                if (h1 > h0)
                    for (int i = tid; i < len / 4; i += THREADS) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
                for (int i = tid; i < len / 32; i += THREADS) ruled[i] = listed[i] = twice[i] = 0;
                if (tid == 0) s_seen = 0;
                __syncthreads();
                each_token(p.tokens, h0, h1, [&](int v, int64_t at) {
                    uint32_t i;
                    if (!inside(v, i)) return;
                    if (at >= hg) atomicAdd(&words[i], 1u);
                    else atomicOr(&words[i], IN_PROMPT);
                    atomicOr(&ruled[i >> 5], 1u << (i & 31));
                });
                // (a thread's first bias entry stays in registers, its logit on the way)
                uint32_t bias_at = ~0u;
                float bias_logit = 0.0f, bias_add = 0.0f;
                for (int64_t e = b0 + tid; e < b1; e += THREADS) {
                    uint32_t i;
                    if (!inside(__ldg(p.bias_token + e), i)) continue;
                    const uint32_t bit = 1u << (i & 31);
                    if (atomicOr(&listed[i >> 5], bit) & bit) atomicOr(&twice[i >> 5], bit);
                    if (e == b0 + tid) {
                        bias_at = i;
                        bias_logit = src[token_at(i)];
                        bias_add = __ldg(p.bias_value + e);
                    }
                }
                __syncthreads();
                // the places whose bits are set, as a list; their logits are fetched
                // and ruled by all threads alike
                if (h1 > h0) {
                    for (int g0 = 0; g0 < len / 32; g0 += THREADS) {
                        uint32_t bits = g0 + tid < len / 32 ? ruled[g0 + tid] : 0u;
                        const int mine = __popc(bits);
                        int before = mine;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int q = __shfl_up_sync(0xffffffffu, before, o);
                            if (lane >= o) before += q;
                        }
                        int at = 0;
                        if (lane == 31 && before) at = atomicAdd(&s_seen, before);
                        at = __shfl_sync(0xffffffffu, at, 31) + before - mine;
                        for (; bits; bits &= bits - 1) seen[at++] = (uint16_t)(32 * (g0 + tid) + __ffs(bits) - 1);
                    }
                    __syncthreads();
                    const int n = s_seen;
#pragma unroll 2
                    for (int e = tid; e < n; e += THREADS) {
                        const int i = seen[e];
                        words[i] = __float_as_uint(penalise(src[token_at(i)], words[i], row));
                    }
                }
                if (b1 > b0) {
                    __syncthreads();
                    for (int64_t e = b0 + tid; e < b1; e += THREADS) {
                        const bool kept = e == b0 + tid;
                        if (kept && bias_at == ~0u) continue;
                        const int v = __ldg(p.bias_token + e);
                        uint32_t i;
                        if (!inside(v, i)) continue;
                        const uint32_t bit = 1u << (i & 31);
                        bool last = true;  // the later entry of a token listed twice counts
                        if (twice[i >> 5] & bit)
                            for (int64_t f = e + 1; f < b1 && last; ++f) last = __ldg(p.bias_token + f) != v;
                        if (!last) continue;
                        const bool set = atomicOr(&ruled[i >> 5], bit) & bit;
                        const float l = set ? __uint_as_float(words[i]) : kept ? bias_logit : src[token_at(i)];
                        words[i] = __float_as_uint(__fadd_rn(l, kept ? bias_add : __ldg(p.bias_value + e)));
                    }
                }
            }
            __syncthreads();
        }

        // ---- Up to STEP logits from place s0 on.  Vectors: access j of a thread
        // covers its places s0 + (j * THREADS + tid) * 4 + 0 .. 3; else places
        // s0 + (4 j + k) * THREADS + tid, so that a warp's 32 are one group.
        // FULL: all of them exist.
        const auto stream = [&](auto vector, auto full, int s0) {
            constexpr bool VECTOR = decltype(vector)::value, FULL = decltype(full)::value;
            const int i0 = s0 + (VECTOR ? 4 * tid : tid);
            // its first logit's token (less base), and how much further the next access's is
            const int v0 = (int)token_at(i0), step = (VECTOR ? 4 * THREADS : THREADS) << lg;
            const auto exist = [&](int j) { return left - (v0 + j * step); };  // (vectors) of access j's logits; may be <= 0 or > 4
            const float* q0 = src + v0;
            float* d0 = dst + v0;
            float l[BATCH][4];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                if constexpr (VECTOR) {
                    const float* q = q0 + (int64_t)j * step;
                    if (FULL || exist(j) >= 4) {
                        const float4 f = *reinterpret_cast<const float4*>(q);
                        l[j][0] = f.x; l[j][1] = f.y; l[j][2] = f.z; l[j][3] = f.w;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) l[j][k] = k < exist(j) ? q[k] : NEG;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) l[j][k] = FULL || exist(4 * j + k) > 0 ? q0[(int64_t)(4 * j + k) * step] : NEG;
                }
            }
            float top = NEG;
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                if (!FULL && exist(VECTOR ? j : 4 * j) <= 0) continue;
                if constexpr (VECTOR) {
                    const int i = i0 + j * 4 * THREADS;
                    if (sparse) {
                        const uint32_t over = ruled[i >> 5] >> (i & 31) & 0xfu;
                        if (over) {
                            const uint4 q = *reinterpret_cast<const uint4*>(words + i);
                            if (over & 1u) l[j][0] = __uint_as_float(q.x);
                            if (over & 2u) l[j][1] = __uint_as_float(q.y);
                            if (over & 4u) l[j][2] = __uint_as_float(q.z);
                            if (over & 8u) l[j][3] = __uint_as_float(q.w);
                        }
                    }
                    if (mask) {
                        const uint32_t allowed = s_mem[i >> 5] >> (i & 31);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (!(allowed & (1u << k))) l[j][k] = NEG;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int i = i0 + (4 * j + k) * THREADS;
                        if (!FULL && exist(4 * j + k) <= 0) continue;
                        if (sparse && (ruled[i >> 5] >> lane) & 1u) l[j][k] = __uint_as_float(words[i]);
                        if (mask && !((s_mem[i >> 5] >> lane) & 1u)) l[j][k] = NEG;
                    }
                }
                if (nothing)
#pragma unroll
                    for (int k = 0; k < 4; ++k) l[j][k] = NEG;
#pragma unroll
                for (int k = 0; k < 4; ++k) top = fmaxf(top, l[j][k]);  // (ignores NaN; what does not exist is -inf)
                if (out) {
                    if constexpr (VECTOR) {
                        float* q = d0 + (int64_t)j * step;
                        if (FULL || exist(j) >= 4) {
                            *reinterpret_cast<float4*>(q) = make_float4(l[j][0], l[j][1], l[j][2], l[j][3]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (k < exist(j)) q[k] = l[j][k];
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (FULL || exist(4 * j + k) > 0) d0[(int64_t)(4 * j + k) * step] = l[j][k];
                    }
                }
            }
            if (!pick) return;
            // the warp's maximum, then sums relative to it
            float m = top;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            Best b{m, 0x7fffffff, 0.0f};
            if (fabsf(m) != __int_as_float(0x7f800000)) {
                float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < BATCH; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[k] += exp_neg(l[j][k] - m);
                b.s = (s[0] + s[1]) + (s[2] + s[3]);
            } else {
                // nothing (every logit -inf or NaN), or an infinite maximum
#pragma unroll
                for (int j = 0; j < BATCH; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) b.s += l[j][k] == m ? (m > 0.0f ? 1.0f : 0.0f) : l[j][k] != l[j][k] ? l[j][k] : 0.0f;
            }
            if (top == m && m != NEG) {
#pragma unroll
                for (int j = 0; j < BATCH; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (l[j][k] == m) b.i = min(b.i, (int)base + v0 + (VECTOR ? j * step + k : (4 * j + k) * step));
            }
            best = join(best, b);
        };
        // (a turn's groups are complete but for its very last)
        const int whole = left & 31 ? len - 32 : len;
        for (int s0 = 0; s0 < len; s0 += STEP) {
            if (vec && s0 + STEP <= whole)
                stream(std::true_type{}, std::true_type{}, s0);
            else if (vec)
                stream(std::true_type{}, std::false_type{}, s0);
            else if (s0 + STEP <= whole)
                stream(std::false_type{}, std::true_type{}, s0);
            else
                stream(std::false_type{}, std::false_type{}, s0);
        }
    }
    if (!pick) return;
    // warp (all lanes have the same maximum here), CTA, cluster: always in the
    // same order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        best.s += __shfl_xor_sync(0xffffffffu, best.s, o);
        best.i = min(best.i, __shfl_xor_sync(0xffffffffu, best.i, o));
    }
    if (lane == 0) s_best[warp] = best;
    __syncthreads();
    cluster_wait();
    if (warp == 0) {
        best = join_lanes(s_best[lane & (WARPS - 1)], WARPS);
        if (lane == 0) {
            const uint32_t a = map_rank(smem_u32(&s_cl[rank]), 0);
            st_cluster(a, best.m);
            st_cluster(a + 4, __int_as_float(best.i));
            st_cluster(a + 8, best.s);
        }
        __syncwarp();
    }
    cluster_arrive();
    if (rank != 0) return;  // (nobody reads this CTA's memory)
    cluster_wait();
    if (warp == 0) {
        best = lane < (1 << lg) ? s_cl[lane] : Best{NEG, 0x7fffffff, 0.0f};
        best = join_lanes(best, MAX_CL);
        if (lane == 0) {
            const bool nan = best.s != best.s;
            if (p.token) p.token[t] = best.m == NEG ? -1 : best.i;
            if (p.lse) p.lse[t] = nan ? best.s : best.m == NEG ? NEG : best.m + logf(best.s);
            if (nan && p.status) atomicOr(p.status, STATUS_NAN_LOGIT);
        }
    }
}

}  // namespace

cudaError_t launch_logits(const LogitArgs& p, const DeviceInfo& dev, cudaStream_t s) {
    // CTAs a row, two an SM at a time (counted so for large vocabularies too,
    // where one fits): a CTA takes about 6 us for the rules (3
    // without) and 3 us for STEP logits, so as many as make the fewest turns,
    // each with at most STEP logits where 8 CTAs allow that.  (16 CTAs of 256
    // threads a row: 8.2 us for one row of 131072 instead of 9.2, but 39 for 64
    // rows with histories instead of 34, and 30 for 32 rows of 16384 tokens each
    // instead of 23.)
    int ncl = 1;
    double best = 0.0;
    for (int c = 1; c <= MAX_CL; c *= 2) {
        const int64_t part = ceil_div(p.V, c);
        if (part > STEP && c < MAX_CL) continue;
        const double us = (double)ceil_div(p.T * c, 2 * dev.sm_count) * ((p.row_start || p.bias_start ? 6.0 : 3.0) + 3.0 * part / STEP);
        if (best == 0.0 || us < best) {
            best = us;
            ncl = c;
        }
    }
    int64_t slice = ceil_div(ceil_div(p.V, ncl), 32) * 32;
    if (slice > MAX_SLICE) slice = MAX_SLICE;
    const bool sparse = p.row_start || p.bias_start;
    const size_t smem = (p.mask ? ((size_t)slice / 32 + 3) / 4 * 16 : 0) + (sparse ? 6 * (size_t)slice + 3 * (size_t)slice / 8 : 0);
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
    int lg = 0;
    while ((1 << lg) < ncl) ++lg;
    return cudaLaunchKernelEx(&cfg, logits_kernel, p, (int)slice, lg);
}

}  // namespace moeq4
