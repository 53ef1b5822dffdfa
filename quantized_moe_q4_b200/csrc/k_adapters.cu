// k_adapters.cu -- low-rank adapters of many requests beside a shared
// projection:  y[t] = base[t] + scale[a] * B_a (A_a x[t]),  a = adapter[t].
//
// The frozen 4-bit matrices ("A 35B Hybrid-Attention Mixture-of-Experts Model
// on a 6GB 2011 GPU", Dutch technical summary, Methodologie 2) stay shared;
// the page has no counterpart of the per-request corrections.
//
// Work per row is 2 r (H + N) operations on 4 (H + 2 N) bytes of x, base and
// y, and r (H + N) elements of its adapter: batches of up to about 1000 rows
// are bound by latency, larger ones by DRAM and, where x passes through the
// shared memory as two parts, by that.  What matters is that the rank-r middle
// vector u = A x never leaves the chip and that nothing is launched twice.
//   - rows are grouped by adapter into tiles, on the device; the host never
//     reads the counts.  Every CTA finds its tile by itself while that is
//     cheaper than grouping kernels before it (one launch then);
//   - a tile is the work of a cluster of CTAs, several clusters if there are
//     many columns: they share u through distributed shared memory, then each
//     takes its own columns of y;
//   - tiles of 8 rows are computed with FMAs (rows kernel), tiles of 128 rows
//     on the tensor cores (tile kernel); launch_typed says when.
//
// Device times, one B200 (hidden size 2048; calls one after another, inputs of
// the smaller ones in L2; from DRAM those take 2 us more):
//   rows kernel   1 row, 2048 outputs, rank 16                 4.0 us
//                 64 rows of 64 adapters, the same              6.3 us
//                 8 rows of 8 adapters, 131072 outputs         13.5 us
//   tile kernel   947 rows in runs of 4 adapters, 2048 outputs, rank 64, 16-bit
//                 weights 21 us, binary32 25 us
//                 16384 rows of 8 adapters, the same           108 and 136 us
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "cluster.cuh"
#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace moeq4 {

namespace {

constexpr int CL = 8;             // CTAs per cluster
constexpr int THREADS = 256;
constexpr int ROWS = 8;           // rows per tile of the rows kernel
constexpr int INLINE_T = 256;     // up to this many rows are grouped inside the kernel (a thread each)
constexpr int SCAN_T = 2048;      // up to this many rows of up to SCAN_N adapters, every CTA of either kernel can find
constexpr int SCAN_N = 255;       // its tile by itself
constexpr int COLS = CL * THREADS;  // columns of y that a cluster covers at a time
constexpr int GROUP_THREADS = 1024;
constexpr int GROUP_IDS = 16;     // ids per thread of the grouping kernels
constexpr int GROUP_CHUNK = GROUP_THREADS * GROUP_IDS;
constexpr int MAX_ADAPTERS = 1024;

// ------------------------------------------------------------------ weights

// Eight consecutive elements (16-byte aligned) as binary32, exactly.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void unpack8(uint4 q, float (&v)[8], const __half*) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = half_bits_to_float(w[i]);
        v[2 * i + 1] = half_bits_to_float(w[i] >> 16);
    }
}
__device__ __forceinline__ void unpack8(uint4 q, float (&v)[8], const __nv_bfloat16*) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <class W>
__device__ __forceinline__ void load8(const W* p, float (&v)[8]) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(p)), v, p);
}

// The same in two steps, so that several loads can be in flight.
template <class W>
struct Raw8 {
    uint4 q;
    __device__ __forceinline__ void load(const W* p) { q = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void unpack(float (&v)[8]) const { unpack8(q, v, (const W*)nullptr); }
};
template <>
struct Raw8<float> {
    float v_[8];
    __device__ __forceinline__ void load(const float* p) { load8(p, v_); }
    __device__ __forceinline__ void unpack(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v_[i];
    }
};

// ------------------------------------------------------------------ finding a tile
//
// Tile g of up to `tile_rows` rows, found by all NT threads of a CTA: counts of
// the adapters' rows, their tiles' offsets, and the rows of the one adapter in
// their order.  False: there is no tile g.  (p.T <= SCAN_T, p.n <= SCAN_N.)
template <int NT>
struct TileFinder {
    static constexpr int K = (SCAN_T + NT - 1) / NT, WARPS = NT / 32;
    int cnt[SCAN_N + 1], sums[WARPS], some[K * WARPS], found[3];

    __device__ bool find(const AdapterArgs& p, int tile_rows, int g, int* tok, int& id, int& rows) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = (int)p.T;
        for (int i = tid; i <= p.n; i += NT) cnt[i] = 0;
        if (tid == 0) found[0] = -1;
        int grp[K];
        bool bad = false;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int t = j * NT + tid;
            grp[j] = -1;
            if (t < T) {
                const int e = __ldg(p.ids + t);
                const bool ok = (unsigned)e < (unsigned)p.n;
                grp[j] = ok ? e : p.n;
                bad |= !ok && e != -1;
            }
        }
        const int any = __syncthreads_or(bad);
        if (blockIdx.x + blockIdx.y == 0 && tid == 0) *p.status = any ? STATUS_BAD_ADAPTER_INDEX : 0u;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (j * NT >= T) break;  // uniform
            const unsigned peers = __match_any_sync(0xffffffffu, grp[j]);
            if (grp[j] >= 0 && lane == __ffs(peers) - 1) atomicAdd(&cnt[grp[j]], __popc(peers));
        }
        __syncthreads();
        // (in place, rows without an adapter need no tile)
        const int c = tid <= p.n && !(tid == p.n && p.base == p.y) ? cnt[tid] : 0;
        const int tiles = (c + tile_rows - 1) / tile_rows;
        int incl = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int q = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += q;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        for (int w = 0; w < warp; ++w) incl += sums[w];
        if (g >= incl - tiles && g < incl) {
            found[0] = tid;
            found[1] = (g - (incl - tiles)) * tile_rows;
            found[2] = min(tile_rows, c - found[1]);
        }
        __syncthreads();
        if (found[0] < 0) return false;
        const int first = found[1];
        id = found[0] < p.n ? found[0] : -1;
        rows = found[2];
        unsigned mine[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            mine[j] = __ballot_sync(0xffffffffu, grp[j] == found[0]);
            if (lane == 0) some[j * WARPS + warp] = __popc(mine[j]);
        }
        __syncthreads();
        int before = 0, at = 0;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            for (; at < j * WARPS + warp; ++at) before += some[at];
            const int pos = before + __popc(mine[j] & ((1u << lane) - 1u)) - first;
            if (grp[j] == found[0] && pos >= 0 && pos < rows) tok[pos] = j * NT + tid;
        }
        __syncthreads();
        return true;
    }
};

// ------------------------------------------------------------------ rows kernel

// u of NT rows of x, this CTA's share: H comes in pieces of 256 columns, piece p
// the work of CTA p % CL; with fewer pieces than CTAs, `sharing` CTAs take the
// rows of A of one piece in turn, eight at a time.  A lane keeps its eight
// columns of the NT rows in registers over all rows of A; a warp's row of A is
// one product, whose sums over the lanes go to part[row][k] of this CTA (added
// to what is there).  KF rows of A are in flight at a time.
template <class W, int NT>
__device__ __forceinline__ void shrink(const W* a, const AdapterArgs& p, const int* tok, int cnt, int rank, float* part) {
    constexpr int KF = sizeof(W) == 4 ? 2 : 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pieces = p.H / 256;
    const int sharing = pieces < CL ? CL / pieces : 1, turn = pieces < CL ? rank / pieces : 0;
    if (turn >= sharing) return;
    for (int piece = pieces < CL ? rank % pieces : rank; piece < pieces; piece += CL) {
        float v[NT][8];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[t][i] = 0.0f;
            if (t < cnt) load8(p.x + (int64_t)tok[t] * p.ldx + piece * 256 + 8 * lane, v[t]);
        }
        const W* ar = a + piece * 256 + 8 * lane;
        for (int k0 = turn * 8 + warp; k0 < p.r; k0 += 8 * sharing * KF) {
            Raw8<W> raw[KF];
#pragma unroll
            for (int j = 0; j < KF; ++j) raw[j].load(ar + (int64_t)min(k0 + 8 * sharing * j, p.r - 1) * p.H);
            float acc[KF * NT];  // row t, k0 + 8 sharing j at NT j + t
#pragma unroll
            for (int j = 0; j < KF; ++j) {
                float w[8];
                raw[j].unpack(w);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    acc[NT * j + t] = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[NT * j + t] = fmaf(w[i], v[t][i], acc[NT * j + t]);
                }
            }
            // transposing reduction: after it, lane l holds sum l * KF * NT / 32
            constexpr int S = KF * NT;
#pragma unroll
            for (int o = 16, m = S / 2; m > 0; o >>= 1, m >>= 1)
#pragma unroll
                for (int i = 0; i < m; ++i) {
                    const bool up = (lane & o) != 0;
                    const float keep = up ? acc[i + m] : acc[i], send = up ? acc[i] : acc[i + m];
                    acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
#pragma unroll
            for (int o = 16 / S; o > 0; o >>= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
            const int mine = lane / (32 / S), t = mine % NT, k = k0 + 8 * sharing * (mine / NT);
            if (lane % (32 / S) == 0 && t < cnt && k < p.r) part[t * p.r + k] += acc[0];
        }
    }
}

// y[t][n] for NT rows and this thread's columns n0, n0 + COLS, ...
template <class W, int NT>
__device__ __forceinline__ void expand_columns(const W* b, const AdapterArgs& p, const int* tok, int cnt,
                                               const float* u, int64_t n0, int64_t n1) {
    const float* br[NT];
    float* yr[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t row = tok[t < cnt ? t : 0];
        br[t] = p.base ? p.base + row * p.ldb : nullptr;
        yr[t] = p.y + row * p.ldy;
    }
    constexpr int KF = sizeof(W) == 4 ? 2 : 4;
    for (int64_t n = n0; n < n1; n += COLS) {
        const W* row = b + n * p.r;
        float acc[NT], bv[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            acc[t] = 0.0f;
            bv[t] = (t < cnt && p.base) ? br[t][n] : 0.0f;
        }
        for (int k0 = 0; k0 < p.r; k0 += 8 * KF) {
            Raw8<W> raw[KF];
#pragma unroll
            for (int j = 0; j < KF; ++j)
                if (k0 + 8 * j < p.r) raw[j].load(row + k0 + 8 * j);  // (uniform)
#pragma unroll
            for (int j = 0; j < KF; ++j) {
                const int k = k0 + 8 * j;
                if (k >= p.r) break;  // uniform
                float w[8];
                raw[j].unpack(w);
#pragma unroll
                for (int t = 0; t < NT; ++t) {  // (u of rows from cnt on is zero)
                    const float4 c = *reinterpret_cast<const float4*>(u + t * p.r + k);
                    const float4 d = *reinterpret_cast<const float4*>(u + t * p.r + k + 4);
                    acc[t] = fmaf(w[0], c.x, acc[t]); acc[t] = fmaf(w[1], c.y, acc[t]);
                    acc[t] = fmaf(w[2], c.z, acc[t]); acc[t] = fmaf(w[3], c.w, acc[t]);
                    acc[t] = fmaf(w[4], d.x, acc[t]); acc[t] = fmaf(w[5], d.y, acc[t]);
                    acc[t] = fmaf(w[6], d.z, acc[t]); acc[t] = fmaf(w[7], d.w, acc[t]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (t < cnt) yr[t][n] = bv[t] + acc[t];
    }
}

// A cluster's work: tile g of up to ROWS rows with one adapter, and columns
// [chunk * iters * COLS, + iters * COLS) of y.  Each CTA computes its part of
// u; after one cluster barrier every CTA adds all parts, always in the same
// order, and produces its own columns, a column per thread.  A is thus read
// once per chunk (from L2 after the first time).
template <class W, bool INLINE>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(THREADS, 4)
    adapters_rows_kernel(const __grid_constant__ AdapterArgs p, int chunks, int iters) {
    __shared__ __align__(16) int s_ids[THREADS];
    __shared__ int s_starts[THREADS / 32];
    __shared__ int s_tok[ROWS];
    __shared__ int s_group[3];  // adapter, rank of its first row among its adapter's rows, rows
    __shared__ __align__(16) float s_part[ROWS * 128];
    __shared__ __align__(16) float s_u[ROWS * 128];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int unit = (int)(blockIdx.x / CL), g = unit / chunks, chunk = unit % chunks;
    int id, cnt;
    if constexpr (INLINE) {
        // group g of the rows: rows of one adapter in runs of ROWS, the
        // groups in the order of their first rows
        const int T = (int)p.T;
        if (tid < 3) s_group[tid] = 0;
        static_assert(INLINE_T <= THREADS);
        int e = -2;
        bool bad = false;
        if (tid < T) {
            e = __ldg(p.ids + tid);
            bad = e < -1 || e >= p.n;
            if (bad) e = -1;
        }
        s_ids[tid] = e;
        const int any = __syncthreads_or(bad);
        // the status word is written, not OR-ed, by one CTA
        if (blockIdx.x == 0 && tid == 0) *p.status = any ? STATUS_BAD_ADAPTER_INDEX : 0u;
        // this row's rank among the rows of its adapter: in its warp, and in the warps before
        int r = __popc(__match_any_sync(0xffffffffu, e) & ((1u << lane) - 1u));
        for (int w = 0; w < warp && tid - lane < T; ++w)
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const int4 q = *reinterpret_cast<const int4*>(s_ids + 32 * w + i);
                r += (q.x == e) + (q.y == e) + (q.z == e) + (q.w == e);
            }
        const bool start = tid < T && r % ROWS == 0;
        const unsigned starts = __ballot_sync(0xffffffffu, start);
        if (lane == 0) s_starts[warp] = __popc(starts);
        __syncthreads();
        int before = 0, groups = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            before += w < warp ? s_starts[w] : 0;
            groups += s_starts[w];
        }
        if (g >= groups) return;  // uniform over the cluster
        if (start && before + __popc(starts & ((1u << lane) - 1u)) == g) {
            s_group[0] = e;
            s_group[1] = r;
        }
        __syncthreads();
        const int r0 = s_group[1];
        if (tid < T && e == s_group[0] && r >= r0 && r < r0 + ROWS) {
            s_tok[r - r0] = tid;
            atomicAdd(&s_group[2], 1);
        }
        __syncthreads();
        id = s_group[0];
        cnt = s_group[2];
    } else if (p.scan) {
        __shared__ TileFinder<THREADS> finder;
        if (!finder.find(p, ROWS, g, s_tok, id, cnt)) return;  // uniform over the cluster
    } else {
        pdl_wait();
        const int n_tiles = *p.n_tiles;
        const int4 tile = p.tiles[g];  // (not one of them, perhaps, but in the workspace; both loads at once)
        if (g >= n_tiles) return;
        id = tile.x;
        cnt = tile.z;
        if (tid < cnt) s_tok[tid] = p.perm[tile.y + tid];
        __syncthreads();
    }
    const int64_t n0 = (int64_t)chunk * iters * COLS + rank * THREADS + tid;
    const int64_t n1 = min(p.N, (int64_t)(chunk + 1) * iters * COLS);
    if (id < 0) {  // no adapter: the base, unless it is there already
        if (p.base == p.y) return;
        for (int t = 0; t < cnt; ++t) {
            const float* br = p.base ? p.base + (int64_t)s_tok[t] * p.ldb : nullptr;
            float* yr = p.y + (int64_t)s_tok[t] * p.ldy;
            for (int64_t n = n0; n < n1; n += COLS) yr[n] = br ? br[n] : 0.0f;
        }
        return;
    }
    const W* a = static_cast<const W*>(p.a) + (int64_t)id * p.r * p.H;
    const W* b = static_cast<const W*>(p.b) + (int64_t)id * p.N * p.r;
    // this thread's first rows of B are on their way to L2 while u is computed
    for (int64_t n = n0; n < n1 && n < n0 + 2 * COLS; n += COLS)
        for (int o = 0; o < p.r * (int)sizeof(W); o += 128) prefetch_l2(reinterpret_cast<const char*>(b + n * p.r) + o);
    // (parts of u that nobody computes are zero: fewer pieces than CTAs, shared rows)
    for (int i = tid; i < cnt * p.r; i += THREADS) s_part[i] = 0.0f;
    __syncthreads();
    if (cnt == 1)
        shrink<W, 1>(a, p, s_tok, cnt, (int)rank, s_part);
    else
        for (int t = 0; t < cnt; t += 4) shrink<W, 4>(a, p, s_tok + t, min(4, cnt - t), (int)rank, s_part + t * p.r);
    cluster_arrive();
    cluster_wait();
    const float scale = p.scale ? __ldg(p.scale + id) : 1.0f;
    for (int i = tid; i < cnt * p.r / 4; i += THREADS) {
        float4 part[CL];
#pragma unroll
        for (int c = 0; c < CL; ++c) part[c] = ld_cluster4(map_rank(smem_u32(s_part + 4 * i), (uint32_t)c));
        float4 v = part[0];
#pragma unroll
        for (int c = 1; c < CL; ++c) {
            v.x += part[c].x; v.y += part[c].y; v.z += part[c].z; v.w += part[c].w;
        }
        reinterpret_cast<float4*>(s_u)[i] = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
    }
    if (cnt > 1)
        for (int i = cnt * p.r + tid; i < ROWS * p.r; i += THREADS) s_u[i] = 0.0f;
    cluster_arrive();  // (this CTA has read the others' parts)
    __syncthreads();
    if (cnt == 1)
        expand_columns<W, 1>(b, p, s_tok, cnt, s_u, n0, n1);
    else if (cnt == 2)
        expand_columns<W, 2>(b, p, s_tok, cnt, s_u, n0, n1);
    else if (cnt <= 4)
        expand_columns<W, 4>(b, p, s_tok, cnt, s_u, n0, n1);
    else
        expand_columns<W, 8>(b, p, s_tok, cnt, s_u, n0, n1);
    cluster_wait();  // (the others have read this CTA's part)
}

// ------------------------------------------------------------------ tile kernel
//
// Many rows: tiles of 128 rows of one adapter on the tensor cores, tf32 with
// binary32 accumulators.  A binary32 value is split into two tf32 parts of 11
// significant bits, v = hi + lo up to 2^-21 |v|; binary16 and bfloat16 weights
// are tf32 values already, so a product with them takes two MMAs, and one of
// two binary32 values three (lo * lo, 2^-22 of the product, is left out).
//   1. u' = x A^T: each CTA of the cluster (of CLT = 1, 2, 4 or 8) sums over
//      its part of H.  M = the tile's rows, N = r, operands K-major in
//      32-column panels with 128-byte rows swizzled in 16-byte units
//      (SWIZZLE_128B).  The tensor core truncates each sum, so a long chain of
//      additions drifts: the panels take turns on several accumulators, the lo
//      products have one of their own, and all are added in binary32.  (Error
//      of y - base at H = 2048, r = 64, bfloat16 weights: 7.2e-7 of its norm
//      with CLT = 1 and 3.6e-7 with 8; a plain binary32 product has 8.2e-7.)
//   2. the partial sums are joined through distributed shared memory: each CTA
//      adds its share of the rows in rank order and hands them to all.
//   3. d^T = B u^T over the CTA's blocks of 128 columns of y: M = columns of y,
//      N = the tile's rows, so that a TMEM lane is a column and every access
//      of base and y is 32 consecutive floats, whatever their alignment.
// TMEM is held inside steps 1 and 3 only, never across a cluster barrier: a
// CTA that holds some waits for nothing but its own MMAs, so CTAs that wait
// for TMEM on other SMs cannot block each other in a ring.
//
// A kernel that uses TMEM gets one CTA an SM here, so the CTA is wide and its
// parts run apart: 16 warps in two groups convert the panels of x and A in
// turn, join u and later read base and write y; 3 warps (binary32: 2) bring the
// panels of B without waiting for u, a panel a warp; one issues the MMAs.  They
// meet on mbarriers only.
//
// What bounds it: a panel of step 1 takes 0.6 us, near the shared memory's
// bandwidth (loads 256, stores 320 and the MMAs' reads 384 clocks); a block of
// step 3 takes 2 to 2.5 us, base and y through DRAM.  With many tiles the two
// alternate on an SM instead of overlapping: 16384 rows (386 MB through DRAM)
// at 46% of the DRAM's rate, tensor pipe 19% active.  With few, the two cluster
// barriers and the join add 4 to 5 us.

constexpr int TM = 128;                 // rows of a tile; columns of y in a block
constexpr int PK = 32;                  // columns of a panel (128 bytes of binary32)
constexpr uint32_t PANEL = TM * 128;    // bytes of a panel of 128 rows
constexpr int ROW_WARPS = 16, WEIGHT_WARPS = 3;  // (20 warps with the one of the MMAs: 96 registers a thread)
constexpr int ROW_THREADS = 32 * ROW_WARPS;
constexpr int TT = ROW_THREADS + 32 * WEIGHT_WARPS + 32;
constexpr int AHEAD = 8;                // panels of x asked for ahead of the loads
constexpr uint32_t COLS_TMEM = 512;
constexpr int MAX_ACCS = 16;            // accumulators of the hi products in step 1, at most

__device__ __forceinline__ uint32_t swizzled(int row, int c16) { return (uint32_t)(row * 128 + ((c16 ^ (row & 7)) << 4)); }

// Descriptor of a K-major operand in a swizzled panel (8-row groups of 1024
// bytes): the low word; the high word is the same for all.
__device__ __forceinline__ uint32_t panel_desc(uint32_t smem_addr) { return ((smem_addr >> 4) & 0x3fffu) | (1u << 16); }
constexpr uint32_t PANEL_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);

// kind::tf32, binary32 accumulator, both operands K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_tf32(int M, int N) {
    return (1u << 4) | (2u << 7) | (2u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_tf32(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::tf32 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(PANEL_DESC_HI)
        : "memory");
}

// One lane of a converged warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void sync_rows() { asm volatile("bar.sync 1, %0;" ::"n"(ROW_THREADS) : "memory"); }

// The finite tf32 value nearest to v (ties away from zero), as binary32.  (Its
// magnitude is at most the largest tf32 value, (2 - 2^-10) 2^127: a binary32
// value above the middle between that and 2^128 would become infinite, its lo
// part too, and their products NaN.)
__device__ __forceinline__ float tf32_near(float v) {
    float h;
    asm("min.xorsign.abs.f32 %0, %1, %2;"
        : "=f"(h)
        : "f"(__uint_as_float((__float_as_uint(v) + 0x1000u) & 0xffffe000u)), "f"(__uint_as_float(0x7f7fe000u)));
    return h;
}

// Four values as two tf32 parts, into the same place of two panels.  The lo
// part (exact as a binary32 value, at most 2^-11 of v, 2^-10 beside the largest
// tf32 value) is not rounded: the MMA drops its low 13 bits, at most 2^-21 of v,
// or 2^-136 where it is subnormal.
__device__ __forceinline__ void store_split(char* hi, char* lo, uint32_t at, float4 v) {
    const float4 h = make_float4(tf32_near(v.x), tf32_near(v.y), tf32_near(v.z), tf32_near(v.w));
    *reinterpret_cast<float4*>(hi + at) = h;
    *reinterpret_cast<float4*>(lo + at) = make_float4(v.x - h.x, v.y - h.y, v.z - h.z, v.w - h.w);
}

// Panels of B, the work of one warp: 16-byte units of a panel's rows are copied
// as they are into a buffer of the warp's own (cp.async, so that a load's
// latency passes under the panel before), and converted from there to tf32
// values in the panel.  A lane reads the units that it copied itself.
template <class W>
struct Panel {
    static constexpr bool SPLIT = sizeof(W) == 4;
    static constexpr int EPU = 16 / (int)sizeof(W), UPR = PK / EPU;  // elements per unit, units per row
    static constexpr int STEP = 32 / UPR;                            // rows that a warp covers at a time
    static constexpr int BATCH = 512;                                // units per copy: a whole panel, or half of one
    static constexpr int PARTS = TM * UPR / BATCH;
    static constexpr uint32_t BYTES = 16 * BATCH;

    // Start copying part `h` of a panel; rows from `have` and elements from
    // `cols` on do not exist and are zeros.
    __device__ __forceinline__ static void copy(const W* src, int64_t pitch, int have, int cols, int h, uint32_t raw) {
        const int lane = threadIdx.x & 31, row0 = h * (BATCH / UPR) + lane / UPR, c = lane % UPR;
        const bool col = c * EPU < cols;
        const W* s = src + row0 * pitch + c * EPU;
#pragma unroll
        for (int j = 0; j < BATCH / 32; ++j, s += STEP * pitch) {
            const bool there = col && row0 + j * STEP < have;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(raw + 16u * (32 * j + lane)),
                         "l"(there ? s : src), "r"(there ? 16 : 0)
                         : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // Convert it (its copies have landed).
    __device__ __forceinline__ static void convert(const char* raw, int h, char* hi) {
        const int lane = threadIdx.x & 31, row0 = h * (BATCH / UPR) + lane / UPR, c = lane % UPR;
#pragma unroll
        for (int j = 0; j < BATCH / 32; ++j) {
            const uint4 q = *reinterpret_cast<const uint4*>(raw + 16 * (32 * j + lane));
            // (eight rows on is 1024 bytes on: the swizzle repeats)
            store(q, swizzled(row0 + (j * STEP & 7), SPLIT ? c : 2 * c) + (uint32_t)(j * STEP / 8) * 1024u,
                  swizzled(row0 + (j * STEP & 7), 2 * c + 1) + (uint32_t)(j * STEP / 8) * 1024u, hi);
        }
    }
    // One unit as tf32 values: at `at` of the hi and lo panels (binary32), or
    // at `at` and `at2` of the panel.
    __device__ __forceinline__ static void store(uint4 q, uint32_t at, uint32_t at2, char* hi) {
        if constexpr (SPLIT) {
            store_split(hi, hi + PANEL, at,
                        make_float4(__uint_as_float(q.x), __uint_as_float(q.y), __uint_as_float(q.z), __uint_as_float(q.w)));
        } else {
            float v[8];
            unpack8(q, v, (const W*)nullptr);
            *reinterpret_cast<float4*>(hi + at) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(hi + at2) = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
};

// Stages of step 1 (x and A) and slots of step 3 (panels of B).
constexpr int stages_of(bool split) { return split ? 2 : 3; }

// Shared memory of the tile kernel, from a 1024-byte aligned start: the slots
// of B, at `raw` the weight warps' copies, then at `x`
//   step 1: the stages: x (hi, lo panel) and A (binary32: hi, lo)
//   step 2: partial sums at x, u at x + u
//   step 3: panels of u (all hi, then all lo)
struct TileSmem {
    uint32_t slot, raw, x, u, total;
    __host__ __device__ TileSmem(int r, bool split) {
        slot = split ? 2 * PANEL : PANEL;
        raw = stages_of(split) * slot;
        x = raw + stages_of(split) * Panel<float>::BYTES;
        u = TM * (uint32_t)(r + 4) * 4;
        const uint32_t panels = (uint32_t)(r + PK - 1) / PK, stages = stages_of(split) * (2 * PANEL + slot);
        uint32_t most = 2 * panels * PANEL > 2 * u ? 2 * panels * PANEL : 2 * u;
        if (stages > most) most = stages;
        total = x + most;
    }
};

template <class W, int CLT>
__global__ void __launch_bounds__(TT, 1) adapters_tile_kernel(const __grid_constant__ AdapterArgs p) {
    constexpr bool SPLIT = sizeof(W) == 4;
    constexpr uint32_t RING = stages_of(SPLIT);
    extern __shared__ char s_raw[];
    __shared__ int s_tok[TM];
    __shared__ __align__(16) int64_t s_off[2][TM];  // byte offsets of the rows of base and y (32-bit unless p.wide)
    // stages full and empty again; slots of B full and empty again; blocks of y
    // computed and read; the sums of step 1; u
    __shared__ uint64_t s_full[RING], s_empty[RING], s_wfull[RING], s_wempty[RING], s_dfull[2], s_dempty[2], s_sums, s_u;
    __shared__ uint32_t s_tmem;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = CLT == 1 ? 0u : cluster_rank();
    char* sm = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);
    const uint32_t sa = smem_u32(sm);
    const int r = p.r;
    const TileSmem lay(r, SPLIT);

    if (tid == 0) {
        for (int i = 0; i < (int)RING; ++i) {
            mbar_init(&s_full[i], ROW_WARPS / 2);
            mbar_init(&s_empty[i], 1);
            mbar_init(&s_wfull[i], 1);
            mbar_init(&s_wempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_dfull[i], 1);
            mbar_init(&s_dempty[i], ROW_WARPS);
        }
        mbar_init(&s_sums, 1);
        mbar_init(&s_u, ROW_WARPS);
        mbar_fence_init();
    }
    const int g = (int)(blockIdx.x / CLT);
    // the blocks of y of a tile go around the CTAs of all its clusters
    const int first_n = (int)blockIdx.y * CLT + (int)rank, step_n = (int)gridDim.y * CLT;
    int id, cnt;
    if (p.scan) {
        __shared__ TileFinder<TT> finder;
        if (!finder.find(p, TM, g, s_tok, id, cnt)) return;  // uniform over the cluster
    } else {
        pdl_wait();
        const int n_tiles = *p.n_tiles;
        const int4 tile = p.tiles[g];  // (not one of them, perhaps, but in the workspace; both loads at once)
        if (g >= n_tiles) return;      // uniform over the cluster
        id = tile.x;
        cnt = tile.z;
        if (tid < cnt) s_tok[tid] = p.perm[tile.y + tid];
    }
    if (tid < TM) {
        const int t = tid < cnt ? s_tok[tid] : -1;
        s_tok[tid] = t;
        if (p.wide) {
            s_off[0][tid] = 4 * (int64_t)t * p.ldb;
            s_off[1][tid] = 4 * (int64_t)t * p.ldy;
        } else {
            reinterpret_cast<uint32_t*>(s_off[0])[tid] = 4u * (uint32_t)t * (uint32_t)p.ldb;
            reinterpret_cast<uint32_t*>(s_off[1])[tid] = 4u * (uint32_t)t * (uint32_t)p.ldy;
        }
    }
    __syncthreads();
    if (id < 0) {  // no adapter (never in place: such rows have no tile then)
        constexpr int FLY = 16;
        const int parts = (int)((p.N + 32 * FLY - 1) / (32 * FLY));  // of a row; a warp has one at a time
        for (int64_t i = first_n + (int64_t)step_n * warp; i < (int64_t)cnt * parts; i += (int64_t)step_n * (TT / 32)) {
            const int64_t t = s_tok[i % cnt], n = i / cnt * (32 * FLY) + lane;
            const float* base = p.base + t * p.ldb + n;
            float* y = p.y + t * p.ldy + n;
            float v[FLY];
#pragma unroll
            for (int j = 0; j < FLY; ++j) v[j] = (p.base && n + 32 * j < p.N) ? base[32 * j] : 0.0f;
#pragma unroll
            for (int j = 0; j < FLY; ++j)
                if (n + 32 * j < p.N) y[32 * j] = v[j];
        }
        return;
    }
    if (warp == 0) tmem_alloc(&s_tmem, COLS_TMEM);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // Every wait on an mbarrier is bounded; one that gives up (after about 2 s)
    // is reported and not repeated.  (The status word was stored when the rows
    // were grouped, or by CTA (0, 0) as it started: long before, though nothing
    // but the CTAs' usual order of starting puts that store first.)
    bool alive = true;
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (alive && !mbar_wait_bounded(bar, parity, 1u << 22)) {
            alive = false;
            atomicOr(p.status, STATUS_SPIN_TIMEOUT);
        }
    };
    const auto both_barriers = [&]() {  // of the roles that take no part in joining u
        if constexpr (CLT > 1) {
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            cluster_arrive();
            cluster_wait();
        }
    };
    const int chunks = p.H / CLT / PK, h0 = (int)rank * (p.H / CLT);  // this CTA's part of H
    const int blocks = (int)((p.N + TM - 1) / TM);                       // its blocks of y: first_n, first_n + step_n, ...
    const int mine = first_n < blocks ? (blocks - first_n + step_n - 1) / step_n : 0;
    const int panels = (r + PK - 1) / PK, half = (panels + 1) / 2;       // of B; from `half` on a second accumulator
    const int n16 = (r + 15) / 16 * 16;
    // accumulators of the hi products (one for every four panels, as far as TMEM has them); the lo ones' comes after them
    const int accs = min(min(MAX_ACCS, (int)COLS_TMEM / n16 - 1), (chunks + 3) / 4);

    if (warp >= ROW_WARPS + WEIGHT_WARPS) {
        // ---------------- MMA (the whole warp waits, one lane issues)
        const uint32_t xa = sa + lay.x;
        const bool leader = elect_one();
        uint32_t st = 0, ph = 0;  // stage or slot, and its phase
        {
            const uint32_t tmem = s_tmem, idesc = idesc_tf32(TM, n16), dl = tmem + (uint32_t)(accs * n16);
            uint32_t dh = tmem;
            for (int c = 0; c < chunks; ++c) {
                wait(&s_full[st], ph);
                tc_fence_after_sync();
                const uint32_t xh = panel_desc(xa + st * (2 * PANEL + lay.slot)), xl = xh + (PANEL >> 4), wh = xl + (PANEL >> 4),
                               wl = wh + (PANEL >> 4);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < PK / 8; ++k) {
                        mma_tf32(dh, xh + 2 * k, wh + 2 * k, idesc, c >= accs || k > 0);
                        mma_tf32(dl, xl + 2 * k, wh + 2 * k, idesc, c + k > 0);
                        if (SPLIT) mma_tf32(dl, xh + 2 * k, wl + 2 * k, idesc, true);
                    }
                    mma_commit(&s_empty[st]);
                }
                __syncwarp();
                dh = dh + n16 == dl ? tmem : dh + n16;
                if (++st == RING) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (leader) mma_commit(&s_sums);
        }
        both_barriers();
        if (mine) {
            wait(&s_u, 0);
            tc_fence_after_sync();
            const uint32_t tmem = s_tmem;
            st = ph = 0;
            for (int i = 0; i < mine; ++i) {
                const uint32_t buf = (uint32_t)i & 1;
                if (i >= 2) wait(&s_dempty[buf], (uint32_t)((i >> 1) - 1) & 1);
                for (int k = 0; k < panels; ++k) {
                    wait(&s_wfull[st], ph);
                    tc_fence_after_sync();
                    const uint32_t bh = panel_desc(sa + st * lay.slot), bl = bh + (PANEL >> 4), uh = panel_desc(xa + k * PANEL),
                                   ul = panel_desc(xa + (panels + k) * PANEL);
                    if (leader) {
                        const int steps = min(PK, r - k * PK) / 8;
                        const uint32_t d = tmem + buf * 2 * TM + (k >= half ? TM : 0);
                        for (int j = 0; j < steps; ++j) {  // the small products first
                            mma_tf32(d, bh + 2 * j, ul + 2 * j, idesc_tf32(TM, TM), (k != 0 && k != half) || j > 0);
                            if (SPLIT) mma_tf32(d, bl + 2 * j, uh + 2 * j, idesc_tf32(TM, TM), true);
                        }
                        for (int j = 0; j < steps; ++j) mma_tf32(d, bh + 2 * j, uh + 2 * j, idesc_tf32(TM, TM), true);
                        mma_commit(&s_wempty[st]);
                        if (k == panels - 1) mma_commit(&s_dfull[buf]);
                    }
                    __syncwarp();
                    if (++st == RING) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
        }
        return;
    }
    if (warp >= ROW_WARPS) {
        // ---------------- panels of B for each block of y, in the order of their
        // use; panel q is warp q % RING's, so that a warp has a slot of its own
        const uint32_t w = (uint32_t)(warp - ROW_WARPS);
        if (w < RING) {
            const W* b = static_cast<const W*>(p.b) + (int64_t)id * p.N * r;
            char* slot = sm + w * lay.slot;
            char* raw = sm + lay.raw + w * Panel<W>::BYTES;
            struct Cursor {
                int i, k, h;  // block of y, its panel, part of the panel
            };
            const auto step = [&](Cursor& c) {
                if (++c.h < Panel<W>::PARTS) return;
                c.h = 0;
                for (c.k += (int)RING; c.k >= panels; c.k -= panels) ++c.i;
            };
            const auto copy = [&](const Cursor& c) {
                if (c.i >= mine) return;
                const int64_t n0 = (int64_t)(first_n + c.i * step_n) * TM;
                Panel<W>::copy(b + n0 * r + c.k * PK, r, (int)min((int64_t)TM, p.N - n0), r - c.k * PK, c.h, smem_u32(raw));
                // the base under the block is needed soon after
                if (c.k == 0 && c.h == 0 && p.base)
                    for (int t = lane; t < cnt; t += 32) {
                        const float* row = p.base + (int64_t)s_tok[t] * p.ldb + n0;
#pragma unroll
                        for (int o = 0; o < TM; o += 32)
                            if (n0 + o < p.N) prefetch_l2(row + o);
                    }
            };
            Cursor at = {0, (int)w, 0};
            for (; at.k >= panels; at.k -= panels) ++at.i;
            copy(at);
            uint32_t n = 0;  // panels that this warp has brought
            for (; at.i < mine; ++n) {
                if (n == 1) both_barriers();  // (the slot's first panel waits for u; so must this warp)
                if (n > 0) wait(&s_wempty[w], (n - 1) & 1);
#pragma unroll
                for (int h = 0; h < Panel<W>::PARTS; ++h) {
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    Panel<W>::convert(raw, h, slot);
                    step(at);
                    copy(at);  // over what was just read, by the same lanes
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive(&s_wfull[w]);
            }
            if (n < 2) both_barriers();
        } else {
            both_barriers();
        }
        return;
    }

    // ---------------- rows
    // 1: x as two tf32 parts.  Two groups of 8 warps take the chunks in turn (a
    // warp's own chain of instructions is what takes its time, not the SM's
    // rates); thread t of a group has 16 bytes of rows t / 8 + 32 i of a panel.
    constexpr int GROUP = ROW_THREADS / 2, PER = TM * 8 / GROUP, FLY = 2;
    const int gt = tid % GROUP, first = tid / GROUP;
    const float* xr[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int t = s_tok[i * (GROUP / 8) + (gt >> 3)];
        xr[i] = t < 0 ? nullptr : p.x + (int64_t)t * p.ldx + h0 + 4 * (gt & 7);
    }
    // thread i of a group asks for the line of row i of its panels
    const float* xp = gt < TM && s_tok[gt] >= 0 ? p.x + (int64_t)s_tok[gt] * p.ldx + h0 : nullptr;
    if (xp)
        for (int c = first; c < AHEAD && c < chunks; c += 2) prefetch_l2(xp + c * PK);
    // ... and units gt + GROUP i of the panel of A
    constexpr int UPR = Panel<W>::UPR, EPU = Panel<W>::EPU, WPER = TM * UPR / GROUP;
    const W* wr = static_cast<const W*>(p.a) + ((int64_t)id * r + gt / UPR) * p.H + h0 + gt % UPR * EPU;
    const uint32_t wrows = (uint32_t)(GROUP / UPR);
    float4 xv[FLY][PER];
    uint4 wv[FLY][WPER];
    const auto load_x = [&](int c, float4 (&v)[PER], uint4 (&w)[WPER]) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            v[i] = xr[i] ? __ldg(reinterpret_cast<const float4*>(xr[i] + c * PK)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < WPER; ++i)
            if (gt / UPR + i * wrows < (uint32_t)r) w[i] = __ldg(reinterpret_cast<const uint4*>(wr + (int64_t)i * wrows * p.H + c * PK));
    };
    uint32_t st = (uint32_t)first, ph = 1;  // (a stage is empty at first)
    const uint32_t at0 = swizzled(gt >> 3, gt & 7);  // (32 rows on: the same swizzle)
    const uint32_t wat = swizzled(gt / UPR, gt % UPR * (Panel<W>::SPLIT ? 1 : 2)), wat2 = swizzled(gt / UPR, gt % UPR * 2 + 1);
    const auto put_x = [&](int c, float4 (&v)[PER], uint4 (&w)[WPER]) {
        if (c >= (int)RING) wait(&s_empty[st], ph);
        char* s = sm + lay.x + st * (2 * PANEL + lay.slot);
#pragma unroll
        for (int i = 0; i < PER; ++i) store_split(s, s + PANEL, at0 + i * (GROUP / 8) * 128, v[i]);
#pragma unroll
        for (int i = 0; i < WPER; ++i)
            if (gt / UPR + i * wrows < (uint32_t)r)
                Panel<W>::store(w[i], wat + i * wrows * 128, wat2 + i * wrows * 128, s + 2 * PANEL);
        if (c + 2 * FLY < chunks) load_x(c + 2 * FLY, v, w);
        if (xp && c + AHEAD < chunks) prefetch_l2(xp + (c + AHEAD) * PK);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive(&s_full[st]);
        st += 2;
        if (st >= RING) {
            st -= RING;
            ph ^= 1;
        }
    };
#pragma unroll
    for (int j = 0; j < FLY; ++j)
        if (first + 2 * j < chunks) load_x(first + 2 * j, xv[j], wv[j]);
    for (int c = first; c < chunks; c += 2 * FLY) {
#pragma unroll
        for (int j = 0; j < FLY; ++j)
            if (c + 2 * j < chunks) put_x(c + 2 * j, xv[j], wv[j]);
    }

    // 2: u
    const float scale = p.scale ? __ldg(p.scale + id) : 1.0f;
    const int pitch = (r + 4) * 4;  // bytes of a row of partial sums and of u
    char* xs = sm + lay.x;
    const int quad = warp & 3;      // the TMEM lanes that this warp reads are 32 quad .. + 31
    wait(&s_sums, 0);
    tc_fence_after_sync();
    __syncwarp();  // (lanes may leave the wait apart; tcgen05.ld takes a converged warp)
    for (int c = warp >> 2; c < r / 8; c += ROW_WARPS / 4) {
        const uint32_t at = s_tmem + (uint32_t)((quad * 32) << 16) + 8u * c;
        float sum[8];
        uint32_t v[3][8];
        tmem_ld8(at + (uint32_t)(accs * n16), v[0]);  // the small products first
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = __uint_as_float(v[0][j]);
        for (int q = 0; q < accs; q += 3) {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (q + i < accs) tmem_ld8(at + (uint32_t)((q + i) * n16), v[i]);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (q + i < accs)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] += __uint_as_float(v[i][j]);
        }
        const int row = quad * 32 + lane;
        const float4 lo4 = make_float4(sum[0], sum[1], sum[2], sum[3]), hi4 = make_float4(sum[4], sum[5], sum[6], sum[7]);
        if constexpr (CLT == 1) {
            char* h = xs + (c / 4) * PANEL;
            char* l = xs + (panels + c / 4) * PANEL;
            store_split(h, l, swizzled(row, c % 4 * 2), make_float4(lo4.x * scale, lo4.y * scale, lo4.z * scale, lo4.w * scale));
            store_split(h, l, swizzled(row, c % 4 * 2 + 1), make_float4(hi4.x * scale, hi4.y * scale, hi4.z * scale, hi4.w * scale));
        } else {
            float4* dst = reinterpret_cast<float4*>(xs + row * pitch + 32 * c);
            dst[0] = lo4;
            dst[1] = hi4;
        }
    }
    if constexpr (CLT > 1) {
        tc_fence_before_sync();
        sync_rows();
        tc_fence_after_sync();
        if (warp == 0) tmem_dealloc(s_tmem, COLS_TMEM);
        cluster_arrive();
        cluster_wait();
        const uint32_t xa = sa + lay.x;
        for (int i = tid; i < TM / CLT * (r / 4); i += ROW_THREADS) {
            const uint32_t at = (uint32_t)(((int)rank * (TM / CLT) + i / (r / 4)) * pitch + i % (r / 4) * 16);
            float4 part[CLT];
#pragma unroll
            for (int c = 0; c < CLT; ++c) part[c] = ld_cluster4(map_rank(xa + at, c));
            float4 v = part[0];
#pragma unroll
            for (int c = 1; c < CLT; ++c) {
                v.x += part[c].x; v.y += part[c].y; v.z += part[c].z; v.w += part[c].w;
            }
            v.x *= scale; v.y *= scale; v.z *= scale; v.w *= scale;
#pragma unroll
            for (int c = 0; c < CLT; ++c) st_cluster4(map_rank(xa + lay.u + at, c), v);
        }
        cluster_arrive();
        cluster_wait();
        if (!mine) return;  // (no CTA reads or writes another's memory from here on)
        if (warp == 0) tmem_alloc(&s_tmem, COLS_TMEM);
        // from rows of u to panels, which lie over them
        constexpr int MOST = TM * (128 / 4) / ROW_THREADS;
        float4 v[MOST];
#pragma unroll
        for (int j = 0; j < MOST; ++j) {
            const int i = j * ROW_THREADS + tid, row = i / (r / 4), c = i % (r / 4);
            if (row < TM) v[j] = *reinterpret_cast<const float4*>(xs + lay.u + row * pitch + 16 * c);
        }
        sync_rows();
#pragma unroll
        for (int j = 0; j < MOST; ++j) {
            const int i = j * ROW_THREADS + tid, row = i / (r / 4), c = i % (r / 4);
            if (row < TM) store_split(xs + (c / 8) * PANEL, xs + (panels + c / 8) * PANEL, swizzled(row, c % 8), v[j]);
        }
    }
    fence_proxy_async_smem();
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) arrive(&s_u);

    // 3: y = base + d.  Warp w has columns 32 (w % 4) .. + 31 of a block, a lane
    // a column, and rows 32 (w / 4) .. + 31, in two halves: while one is added
    // and written, the base of the other and of the next block is on its way.
    // Offsets of rows are 32-bit byte offsets unless the buffers are larger
    // (one add an access instead of three), and a full half is done without
    // predicates.
    const int t0 = (warp >> 2) * 32;
    const int rows = cnt - t0;  // may be <= 0 or > 32
    const auto finish = [&](auto wide) {
        using Off = std::conditional_t<decltype(wide)::value, int64_t, uint32_t>;
        const Off* boff = reinterpret_cast<const Off*>(s_off[0]) + t0;
        const Off* yoff = reinterpret_cast<const Off*>(s_off[1]) + t0;
        const char* base = reinterpret_cast<const char*>(p.base);
        char* y = reinterpret_cast<char*>(p.y);
        float bv[2][16];
        const auto load_base = [&](int i, int h) {
            const int n = (first_n + i * step_n) * TM + quad * 32 + lane;
            if (!base) {
#pragma unroll
                for (int j = 0; j < 16; ++j) bv[h][j] = 0.0f;
            } else if (rows >= 16 * h + 16 && n - lane + 32 <= p.N) {
#pragma unroll
                for (int j = 0; j < 16; ++j) bv[h][j] = *reinterpret_cast<const float*>(base + (Off)(boff[16 * h + j] + 4 * (Off)n));
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (16 * h + j < rows && n < p.N)
                        bv[h][j] = *reinterpret_cast<const float*>(base + (Off)(boff[16 * h + j] + 4 * (Off)n));
            }
        };
        load_base(0, 0);
        load_base(0, 1);
        for (int i = 0; i < mine; ++i) {
            const uint32_t buf = (uint32_t)i & 1;
            const int n = (first_n + i * step_n) * TM + quad * 32 + lane;
            wait(&s_dfull[buf], (uint32_t)(i >> 1) & 1);
            tc_fence_after_sync();
            __syncwarp();
            const uint32_t at = s_tmem + (uint32_t)((quad * 32) << 16) + buf * 2 * TM + t0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v[16];
                tmem_ld16(at + 16 * h, v);
                tmem_wait_ld();
                if (panels > 1) {
                    uint32_t v2[16];
                    tmem_ld16(at + TM + 16 * h, v2);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(v2[j]));
                }
                if (h == 1) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) arrive(&s_dempty[buf]);
                }
                if (rows >= 16 * h + 16 && n - lane + 32 <= p.N) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        *reinterpret_cast<float*>(y + (Off)(yoff[16 * h + j] + 4 * (Off)n)) = bv[h][j] + __uint_as_float(v[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (16 * h + j < rows && n < p.N)
                            *reinterpret_cast<float*>(y + (Off)(yoff[16 * h + j] + 4 * (Off)n)) = bv[h][j] + __uint_as_float(v[j]);
                }
                if (i + 1 < mine) load_base(i + 1, h);
                __syncwarp();
            }
        }
    };
    if (p.wide)
        finish(std::true_type{});
    else
        finish(std::false_type{});
    tc_fence_before_sync();
    sync_rows();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(s_tmem, COLS_TMEM);
}

// ------------------------------------------------------------------ grouping

// Group of id e: its adapter, or n for rows without one.
__device__ __forceinline__ int group_of(int e, int n, bool& bad) {
    if ((unsigned)e < (unsigned)n) return e;
    if (e != -1) bad = true;
    return n;
}

// Rank of each of this thread's ids among equal ids of the CTA, counting in
// cnt (zeroed); -1 for positions past the end.  The order within a group is
// arbitrary: a row's result does not depend on its place in a tile.
__device__ __forceinline__ void rank_ids(const int32_t* ids, int64_t first, int64_t T, int n, int* cnt, int (&grp)[GROUP_IDS],
                                         int (&rnk)[GROUP_IDS], bool& bad) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < GROUP_IDS; ++i) {
        const int64_t t = first + i * GROUP_THREADS + threadIdx.x;
        grp[i] = t < T ? group_of(__ldg(ids + t), n, bad) : -1;
    }
#pragma unroll
    for (int i = 0; i < GROUP_IDS; ++i) {
        rnk[i] = 0;
        if (first + i * GROUP_THREADS >= T) continue;  // uniform
        const unsigned peers = __match_any_sync(0xffffffffu, grp[i]);
        const int lead = __ffs(peers) - 1;
        int at = 0;
        if (lane == lead && grp[i] >= 0) at = atomicAdd(&cnt[grp[i]], __popc(peers));
        at = __shfl_sync(0xffffffffu, at, lead);
        rnk[i] = at + __popc(peers & ((1u << lane) - 1u));
    }
}

// Offsets of the groups in perm and of their tiles in the tile list
// (exclusive sums over n + 1 groups, the rows without an adapter last), and
// this CTA's share (part of parts) of the tile list.  cnt, off, toff: shared
// arrays of MAX_ADAPTERS + 2.
__device__ __forceinline__ void scan_groups(const AdapterArgs& p, int tile_rows, const int* cnt, int* off, int* toff, int part,
                                            int parts) {
    __shared__ unsigned long long s_warp[GROUP_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = tid < p.n ? cnt[tid] : 0;
    const unsigned long long v = ((unsigned long long)c << 32) | (unsigned)((c + tile_rows - 1) / tile_rows);
    unsigned long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long q = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += q;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const unsigned long long own = s_warp[lane];
        unsigned long long sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long q = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += q;
        }
        s_warp[lane] = sum - own;
    }
    __syncthreads();
    incl += s_warp[warp];
    const unsigned long long excl = incl - v;
    if (tid < p.n) {
        off[tid] = (int)(excl >> 32);
        toff[tid] = (int)(excl & 0xffffffffu);
    }
    if (tid == p.n - 1) {
        // in place, rows without an adapter need no tile
        const int none = p.base == p.y ? 0 : (cnt[p.n] + tile_rows - 1) / tile_rows;
        off[p.n] = (int)(incl >> 32);
        toff[p.n] = (int)(incl & 0xffffffffu);
        toff[p.n + 1] = toff[p.n] + none;
        if (part == 0) *p.n_tiles = toff[p.n + 1];
    }
    __syncthreads();
    const int tiles = toff[p.n + 1];
    for (int i = part * GROUP_THREADS + tid; i < tiles; i += parts * GROUP_THREADS) {
        int lo = 0, hi = p.n;  // the last group whose tiles start at or before i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (toff[mid] <= i) lo = mid; else hi = mid - 1;
        }
        const int first = (i - toff[lo]) * tile_rows;
        p.tiles[i] = make_int4(lo < p.n ? lo : -1, off[lo] + first, min(tile_rows, cnt[lo] - first), 0);
    }
}

// Up to CLG * GROUP_CHUNK rows in one launch of one cluster: each CTA counts
// `per` rows, the counts are added through distributed shared memory, each
// CTA places its own rows.
template <int CLG>
__global__ void __launch_bounds__(GROUP_THREADS)
    adapters_group_kernel(const __grid_constant__ AdapterArgs p, int tile_rows, int per) {
    __shared__ int cnt[MAX_ADAPTERS + 2], all[MAX_ADAPTERS + 2], pre[MAX_ADAPTERS + 2], off[MAX_ADAPTERS + 2], toff[MAX_ADAPTERS + 2];
    pdl_launch_dependents();
    const int rank = CLG == 1 ? 0 : (int)cluster_rank();
    const int64_t first = (int64_t)rank * per, last = CLG == 1 ? p.T : min(p.T, first + per);
    for (int i = threadIdx.x; i < p.n + 2; i += GROUP_THREADS) cnt[i] = 0;
    __syncthreads();
    int grp[GROUP_IDS], rnk[GROUP_IDS];
    bool bad = false;
    rank_ids(p.ids, first, last, p.n, cnt, grp, rnk, bad);
    if (bad) cnt[p.n + 1] = 1;
    if constexpr (CLG == 1) {
        __syncthreads();
        scan_groups(p, tile_rows, cnt, off, toff, 0, 1);
    } else {
        cluster_arrive();
        cluster_wait();
        // totals; and this CTA's rows of a group come after those of the CTAs before it
        for (int i = threadIdx.x; i < p.n + 2; i += GROUP_THREADS) {
            int sum = 0, before = 0;
#pragma unroll
            for (int c = 0; c < CLG; ++c) {
                const int v = ld_cluster1(map_rank(smem_u32(&cnt[i]), c));
                before += c < rank ? v : 0;
                sum += v;
            }
            all[i] = sum;
            pre[i] = before;
        }
        cluster_arrive();  // (this CTA has read the others' counts)
        __syncthreads();
        scan_groups(p, tile_rows, all, off, toff, rank, CLG);
    }
#pragma unroll
    for (int i = 0; i < GROUP_IDS; ++i)
        if (grp[i] >= 0)
            p.perm[off[grp[i]] + (CLG == 1 ? 0 : pre[grp[i]]) + rnk[i]] = (int32_t)(first + i * GROUP_THREADS + threadIdx.x);
    const int* total = CLG == 1 ? cnt : all;
    if (rank == 0 && threadIdx.x == 0) *p.status = total[p.n + 1] ? STATUS_BAD_ADAPTER_INDEX : 0u;
    if constexpr (CLG > 1) cluster_wait();  // (the others have read this CTA's counts)
}

// More rows: counts per chunk, offsets of every (chunk, group), placement.
__global__ void __launch_bounds__(GROUP_THREADS) adapters_count_kernel(const __grid_constant__ AdapterArgs p) {
    __shared__ int cnt[MAX_ADAPTERS + 2];
    for (int i = threadIdx.x; i < p.n + 2; i += GROUP_THREADS) cnt[i] = 0;
    __syncthreads();
    int grp[GROUP_IDS], rnk[GROUP_IDS];
    bool bad = false;
    rank_ids(p.ids, (int64_t)blockIdx.x * GROUP_CHUNK, p.T, p.n, cnt, grp, rnk, bad);
    const int any = __syncthreads_or(bad);
    int32_t* out = p.chunk_cnt + (int64_t)blockIdx.x * (p.n + 2);
    for (int i = threadIdx.x; i < p.n + 1; i += GROUP_THREADS) out[i] = cnt[i];
    if (threadIdx.x == 0) out[p.n + 1] = any;
}

__global__ void __launch_bounds__(GROUP_THREADS)
    adapters_scan_kernel(const __grid_constant__ AdapterArgs p, int nchunks, int tile_rows) {
    __shared__ int cnt[MAX_ADAPTERS + 2], off[MAX_ADAPTERS + 2], toff[MAX_ADAPTERS + 2];
    for (int i = threadIdx.x; i < p.n + 2; i += GROUP_THREADS) {
        int c = 0;
        for (int k = 0; k < nchunks; ++k) c += p.chunk_cnt[(int64_t)k * (p.n + 2) + i];
        cnt[i] = c;
    }
    __syncthreads();
    scan_groups(p, tile_rows, cnt, off, toff, 0, 1);
    for (int i = threadIdx.x; i < p.n + 1; i += GROUP_THREADS) {
        int at = off[i];
        for (int k = 0; k < nchunks; ++k) {
            p.chunk_base[(int64_t)k * (p.n + 1) + i] = at;
            at += p.chunk_cnt[(int64_t)k * (p.n + 2) + i];
        }
    }
    if (threadIdx.x == 0) *p.status = cnt[p.n + 1] ? STATUS_BAD_ADAPTER_INDEX : 0u;
}

__global__ void __launch_bounds__(GROUP_THREADS) adapters_place_kernel(const __grid_constant__ AdapterArgs p) {
    __shared__ int cnt[MAX_ADAPTERS + 2];
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < p.n + 2; i += GROUP_THREADS) cnt[i] = 0;
    __syncthreads();
    int grp[GROUP_IDS], rnk[GROUP_IDS];
    bool bad = false;
    const int64_t first = (int64_t)blockIdx.x * GROUP_CHUNK;
    rank_ids(p.ids, first, p.T, p.n, cnt, grp, rnk, bad);
    const int32_t* at = p.chunk_base + (int64_t)blockIdx.x * (p.n + 1);
#pragma unroll
    for (int i = 0; i < GROUP_IDS; ++i)
        if (grp[i] >= 0) p.perm[at[grp[i]] + rnk[i]] = (int32_t)(first + i * GROUP_THREADS + threadIdx.x);
}

// A launch of clusters of `cluster` CTAs; dependent: it may begin while the
// kernel before it drains (its kernels wait with pdl_wait before they read
// anything).
template <class... A>
cudaError_t launch_clusters(void (*kernel)(A...), dim3 grid, int cluster, int threads, size_t smem, bool dependent,
                            cudaStream_t s, A... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_group(const AdapterArgs& p, int tile_rows, cudaStream_t s) {
    if (p.T <= 2 * GROUP_THREADS) {
        adapters_group_kernel<1><<<1, GROUP_THREADS, 0, s>>>(p, tile_rows, 0);
        return cudaGetLastError();
    }
    if (p.T <= (int64_t)CL * GROUP_CHUNK) {
        const int per = (int)ceil_div(ceil_div(p.T, CL), GROUP_THREADS) * GROUP_THREADS;
        return launch_clusters(adapters_group_kernel<CL>, CL, CL, GROUP_THREADS, 0, false, s, p, tile_rows, per);
    }
    const int nchunks = (int)ceil_div(p.T, GROUP_CHUNK);
    adapters_count_kernel<<<nchunks, GROUP_THREADS, 0, s>>>(p);
    adapters_scan_kernel<<<1, GROUP_THREADS, 0, s>>>(p, nchunks, tile_rows);
    adapters_place_kernel<<<nchunks, GROUP_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

template <class W>
cudaError_t launch_rows(const AdapterArgs& p, const DeviceInfo& dev, cudaStream_t s) {
    const bool in = p.T <= INLINE_T;
    const int64_t groups = in ? std::min<int64_t>(p.T, (p.n + 1) + p.T / ROWS) : p.T / ROWS + p.n + 1;
    // columns per cluster: as many steps of COLS as leave four CTAs an SM; u is
    // computed once per cluster (8 adapters, rank 16, on 131072 columns: two
    // CTAs an SM 23.6 us, four 16.3, eight 18.0)
    const int64_t steps = ceil_div(p.N, COLS);
    const int64_t iters = std::max<int64_t>(1, std::min<int64_t>(steps, groups * steps / (4 * dev.sm_count / CL)));
    const int64_t chunks = ceil_div(steps, iters);
    const int64_t grid = groups * chunks * CL;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    if (in) {
        adapters_rows_kernel<W, true><<<(unsigned)grid, THREADS, 0, s>>>(p, (int)chunks, (int)iters);
        return cudaGetLastError();
    }
    cudaError_t e = p.scan ? cudaSuccess : launch_group(p, ROWS, s);
    if (e != cudaSuccess) return e;
    return launch_clusters(adapters_rows_kernel<W, false>, (unsigned)grid, CL, THREADS, 0, !p.scan, s, p, (int)chunks, (int)iters);
}

template <class W, int CLT>
cudaError_t launch_tiles(const AdapterArgs& p, int shares, cudaStream_t s) {
    const TileSmem lay(p.r, sizeof(W) == 4);
    const size_t smem = lay.total + 1024;
    int per_sm = 0;  // (raises the kernel's shared-memory limit)
    cudaError_t e = kernel_occupancy(reinterpret_cast<const void*>(adapters_tile_kernel<W, CLT>), TT, smem, &per_sm);
    if (e != cudaSuccess) return e;
    e = p.scan ? cudaSuccess : launch_group(p, TM, s);
    if (e != cudaSuccess) return e;
    const int64_t tiles = p.T / TM + std::min<int64_t>(p.n + 1, p.T);
    return launch_clusters(adapters_tile_kernel<W, CLT>, dim3((unsigned)(tiles * CLT), (unsigned)shares), CLT, TT, smem, !p.scan, s, p);
}

// The choice of kernel and of the tile kernel's cluster, by what the steps of
// either were measured to take (us; H = 256 .. 2048, N = 300 .. 16384):
//   rows: 9 (grouped inside: 5) + 0.04 + 2.3e-5 N + 0.9e-6 r (H + N) a tile of 8;
//   tiles: 4 + waves * (4 + 0.05 r + 0.6 a panel of H + 2 a block of y, per CTA),
//   one CTA an SM (about 12 of 13 SMs can hold clusters of 4, and 15 clusters of
//   8 fit).
// (2048 -> 2048, 4 adapters, rank 16: 512 rows 15.6 us as rows, 18.8 as tiles;
// 1024 rows 25.9 and 19.8.  Rank 64: 256 rows 18.3 and 21.5; 512 rows 26.1 and
// 22.3.)  A cluster must be wide enough that an accumulator of step 1 sums no
// more than CHAIN panels: each addition truncates, and 4 CHAIN of them drift by
// about 1e-6 of the sum.  Where 8 CTAs are too few for that, the rows kernel is
// left, at any T: above H = 7680 at ranks 104 to 128, 10240 at 88 and 96, 12800 at
// 72 and 80 (2048 rows, 2048 outputs, rank 128: H = 7680 83 us, 7936 244 us).
// CTAs that find their tiles by themselves save the grouping kernel and the start
// of a second one, but do that work once a wave, 2 to 3 us each time: so the rows
// kernel does while all its clusters can be resident at once, the tile kernel for
// up to two waves (a grouping kernel before it -> by itself: 257 rows 12.4 -> 10.9
// us, 947 rows 22.6 -> 20.7, 2048 rows in two waves 31.2 -> 29.1; in more waves
// 512 rows of 64 adapters 19.6 -> 22.2, 2048 rows of 200 adapters 59 -> 97).
template <class W>
cudaError_t launch_typed(AdapterArgs p, const DeviceInfo& dev, cudaStream_t s) {
    constexpr int CHAIN = 10;
    const bool scans = p.T <= SCAN_T && p.n <= SCAN_N;
    const int n16 = (p.r + 15) / 16 * 16, accs = std::min(MAX_ACCS, (int)COLS_TMEM / n16 - 1), chunks = p.H / PK;
    // tiles of `rows` rows: one an adapter while adapters see fewer, else half a tile too many each
    const auto tiles = [&](int rows) {
        return (double)(p.T < (int64_t)rows * (p.n + 1) ? std::min<int64_t>(p.T, p.n + 1) : p.T / rows + (p.n + 1) / 2);
    };
    const double small = std::min<double>((double)p.T, (double)(p.T / ROWS + (p.n + 1) / 2));
    double best = (p.T <= INLINE_T ? 5.0 : 9.0) + small * (0.04 + 0.9e-6 * p.r * (double)(p.H + p.N) + 2.3e-5 * (double)p.N);
    int cl = 0, shares = 1;
    p.scan = scans && small * CL <= 3.0 * dev.sm_count;
    for (int c = 1; c <= CL; c *= 2) {
        if (chunks > c * accs * CHAIN || (p.T <= INLINE_T && !scans)) continue;  // (few rows have no workspace to be grouped in)
        const int slots = c <= 2 ? dev.sm_count : c == 4 ? dev.sm_count * 12 / 13 : 15 * CL * dev.sm_count / 148;
        const int64_t blocks = ceil_div(p.N, (int64_t)TM * c);
        const int q = (int)std::max(1.0, std::min({(double)blocks, std::floor(slots / (tiles(TM) * c)), 65535.0}));
        const double waves = std::ceil(tiles(TM) * c * q / slots);
        const double t = 4.0 + waves * (4.0 + 0.05 * p.r + 0.6 * chunks / c + 2.0 * (double)ceil_div(blocks, q));
        if (t < best) {
            best = t;
            cl = c;
            shares = q;
            p.scan = scans && (waves <= 2.0 || p.T <= INLINE_T);
        }
    }
    switch (cl) {
        case 1: return launch_tiles<W, 1>(p, shares, s);
        case 2: return launch_tiles<W, 2>(p, shares, s);
        case 4: return launch_tiles<W, 4>(p, shares, s);
        case 8: return launch_tiles<W, 8>(p, shares, s);
        default: return launch_rows<W>(p, dev, s);
    }
}

}  // namespace

size_t adapters_layout(int n, int64_t T, char* base, AdapterArgs* p) {
    const auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    const bool grouped = T > INLINE_T;
    const size_t chunks = (size_t)ceil_div(T, GROUP_CHUNK);
    const size_t tiles = (size_t)(T / ROWS + n + 1);
    const size_t sz[5] = {256, grouped ? 4 * (size_t)T : 0, grouped ? sizeof(int4) * tiles : 0,
                          chunks > 1 ? 4 * chunks * (size_t)(n + 2) : 0, chunks > 1 ? 4 * chunks * (size_t)(n + 1) : 0};
    size_t off[6] = {0};
    for (int i = 0; i < 5; ++i) off[i + 1] = off[i] + up(sz[i]);
    if (p) {
        p->status = reinterpret_cast<uint32_t*>(base);
        p->n_tiles = reinterpret_cast<int32_t*>(base + 16);
        p->perm = reinterpret_cast<int32_t*>(base + off[1]);
        p->tiles = reinterpret_cast<int4*>(base + off[2]);
        p->chunk_cnt = reinterpret_cast<int32_t*>(base + off[3]);
        p->chunk_base = reinterpret_cast<int32_t*>(base + off[4]);
    }
    return off[5];
}

cudaError_t launch_adapters(const AdapterArgs& args, int dtype, const DeviceInfo& dev, cudaStream_t s) {
    AdapterArgs p = args;
    p.wide = 4 * (p.T * std::max(p.ldb, p.ldy) + p.N) > 0xffffffffll;
    if (dtype == 0) return launch_typed<float>(p, dev, s);
    if (dtype == 1) return launch_typed<__half>(p, dev, s);
    return launch_typed<__nv_bfloat16>(p, dev, s);
}

}  // namespace moeq4
