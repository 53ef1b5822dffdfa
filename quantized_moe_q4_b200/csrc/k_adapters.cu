// k_adapters.cu -- low-rank adapters of many requests beside a shared
// projection:  y[t] = base[t] + scale[a] * B_a (A_a x[t]),  a = adapter[t].
//
// The frozen 4-bit matrices ("A 35B Hybrid-Attention Mixture-of-Experts Model
// on a 6GB 2011 GPU", Dutch technical summary, Methodologie 2) stay shared;
// the page has no counterpart of the per-request corrections.
//
// Work per row is 2 r (H + N) operations on 4 (H + 2 N) bytes of x, base and
// y, and r (H + N) elements of its adapter, so every kernel here is bound by
// memory or latency; what matters is that the rank-r middle vector u = A x
// never leaves the chip and that nothing is launched twice.
//   - rows are grouped by adapter into tiles: inside the kernel up to
//     INLINE_T rows (one launch), else by the grouping kernels (device only;
//     the host never reads the counts);
//   - a tile is the work of a cluster of 8 CTAs: they share A x through
//     distributed shared memory, then each takes its own columns of y.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace moeq4 {

namespace {

constexpr int CL = 8;             // CTAs per cluster
constexpr int THREADS = 256;
constexpr int ROWS = 8;           // rows per tile of the rows kernel
constexpr int INLINE_T = 64;      // up to this many rows are grouped inside the kernel
constexpr int COLS = CL * THREADS;  // columns of y that a cluster covers at a time
constexpr int GROUP_THREADS = 1024;
constexpr int GROUP_IDS = 16;     // ids per thread of the grouping kernels
constexpr int GROUP_CHUNK = GROUP_THREADS * GROUP_IDS;
constexpr int MAX_ADAPTERS = 1024;

// ------------------------------------------------------------------ clusters

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Address of the same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t smem_addr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr), "r"(rank));
    return a;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// ------------------------------------------------------------------ weights

// Eight consecutive elements (16-byte aligned) as binary32, exactly.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = half_bits_to_float(w[i]);
        v[2 * i + 1] = half_bits_to_float(w[i] >> 16);
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ------------------------------------------------------------------ rows kernel

// Where a CTA's shrink work lies: the cluster's 8 CTAs split the r rows of A
// into blocks of 8 rows (a row per warp) and, where fewer than 8 blocks
// exist, H into `splits` interleaved parts.
struct ShrinkPart {
    int splits;
    __device__ explicit ShrinkPart(int r) : splits(r > 32 ? 1 : CL / (r / 8)) {}
};

// u[row] of NT rows of x with one row of A (this warp's), over the 256-wide
// pieces `piece`, piece + step, ... of H; the sums of all lanes go to every
// CTA's part[][row][k].
template <class W, int NT>
__device__ __forceinline__ void shrink_row(const W* arow, const AdapterArgs& p, const int* tok, int cnt, int piece,
                                           int step, float* part, int k) {
    const int lane = threadIdx.x & 31;
    float acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = 0.0f;
    const float* xr[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xr[t] = p.x + (int64_t)tok[t < cnt ? t : 0] * p.ldx + 8 * lane;
#pragma unroll 2
    for (int h = piece * 256; h < p.H; h += step * 256) {
        float w[8];
        load8(arow + h + 8 * lane, w);
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (t < cnt) {
                float v[8];
                load8(xr[t] + h, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[t] = fmaf(w[i], v[i], acc[t]);
            }
    }
    const uint32_t dst = smem_u32(part);
    if constexpr (NT == 1) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
        if (lane < CL) st_cluster(map_rank(dst + 4u * (uint32_t)k, (uint32_t)lane), acc[0]);
    } else {
        // transposing reduction: after it, lane l holds row l / 4's sum
        static_assert(NT == 8);
#pragma unroll
        for (int o = 16, m = 4; m > 0; o >>= 1, m >>= 1)
#pragma unroll
            for (int i = 0; i < m; ++i) {
                const bool up = (lane & o) != 0;
                const float keep = up ? acc[i + m] : acc[i], send = up ? acc[i] : acc[i + m];
                acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], 2);
        acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], 1);
        const int t = lane >> 2;
        if (t < cnt) {
            const uint32_t a = dst + 4u * (uint32_t)(t * p.r + k);
            st_cluster(map_rank(a, (uint32_t)(lane & 3) * 2), acc[0]);
            st_cluster(map_rank(a, (uint32_t)(lane & 3) * 2 + 1), acc[0]);
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
    for (int64_t n = n0; n < n1; n += COLS) {
        const W* row = b + n * p.r;
        float acc[NT], bv[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            acc[t] = 0.0f;
            bv[t] = (t < cnt && p.base) ? br[t][n] : 0.0f;
        }
#pragma unroll 4
        for (int k = 0; k < p.r; k += 8) {
            float w[8];
            load8(row + k, w);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (t < cnt) {
                    const float4 c = *reinterpret_cast<const float4*>(u + t * p.r + k);
                    const float4 d = *reinterpret_cast<const float4*>(u + t * p.r + k + 4);
                    acc[t] = fmaf(w[0], c.x, acc[t]); acc[t] = fmaf(w[1], c.y, acc[t]);
                    acc[t] = fmaf(w[2], c.z, acc[t]); acc[t] = fmaf(w[3], c.w, acc[t]);
                    acc[t] = fmaf(w[4], d.x, acc[t]); acc[t] = fmaf(w[5], d.y, acc[t]);
                    acc[t] = fmaf(w[6], d.z, acc[t]); acc[t] = fmaf(w[7], d.w, acc[t]);
                }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (t < cnt) yr[t][n] = bv[t] + acc[t];
    }
}

// A cluster's work: tile g of up to ROWS rows with one adapter, and columns
// [chunk * iters * COLS, + iters * COLS) of y.  Each CTA computes its part of
// u (8 rows of A x a part of H) and stores it to all 8 CTAs; after one
// cluster barrier every CTA has u and produces its own columns, a column per
// thread.  A is thus read once per chunk (from L2 after the first time).
template <class W, bool INLINE>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(THREADS)
    adapters_rows_kernel(const __grid_constant__ AdapterArgs p, int chunks, int iters) {
    __shared__ int s_ids[INLINE_T];
    __shared__ int s_starts[2];
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
        int e = -2;
        bool bad = false;
        if (tid < INLINE_T) {
            if (tid < T) {
                e = __ldg(p.ids + tid);
                bad = e < -1 || e >= p.n;
                if (bad) e = -1;
            }
            s_ids[tid] = e;
        }
        const int any = __syncthreads_or(bad);
        // the status word is written, not OR-ed, by one CTA
        if (blockIdx.x == 0 && tid == 0) *p.status = any ? STATUS_BAD_ADAPTER_INDEX : 0u;
        int r = 0;
        bool start = false;
        unsigned starts = 0;
        if (tid < INLINE_T) {
            for (int i = 0; i < INLINE_T; ++i) r += (i < tid && s_ids[i] == e) ? 1 : 0;
            start = tid < T && r % ROWS == 0;
            starts = __ballot_sync(0xffffffffu, start);
            if (lane == 0) s_starts[warp] = __popc(starts);
        }
        __syncthreads();
        if (g >= s_starts[0] + s_starts[1]) return;  // uniform over the cluster
        if (start && (warp ? s_starts[0] : 0) + __popc(starts & ((1u << lane) - 1u)) == g) {
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
    } else {
        pdl_wait();
        if (g >= *p.n_tiles) return;
        const int4 tile = p.tiles[g];
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
    cluster_arrive();  // (every CTA of the cluster has started once this completes)
    const W* a = static_cast<const W*>(p.a) + (int64_t)id * p.r * p.H;
    const W* b = static_cast<const W*>(p.b) + (int64_t)id * p.N * p.r;
    // this thread's first rows of B are on their way to L2 while u is computed
    for (int64_t n = n0; n < n1 && n < n0 + 2 * COLS; n += COLS)
        for (int o = 0; o < p.r * (int)sizeof(W); o += 128) prefetch_l2(reinterpret_cast<const char*>(b + n * p.r) + o);
    const int splits = ShrinkPart(p.r).splits, blocks = p.r / 8;
    cluster_wait();
    for (int rb = rank / splits; rb < blocks; rb += CL / splits) {
        const int k = rb * 8 + warp, piece = rank % splits;
        float* part = s_part + piece * ROWS * p.r;
        if (cnt == 1)
            shrink_row<W, 1>(a + (int64_t)k * p.H, p, s_tok, cnt, piece, splits, part, k);
        else
            shrink_row<W, 8>(a + (int64_t)k * p.H, p, s_tok, cnt, piece, splits, part, k);
    }
    cluster_arrive();
    cluster_wait();
    const float scale = p.scale ? __ldg(p.scale + id) : 1.0f;
    for (int i = tid; i < cnt * p.r; i += THREADS) {
        float v = 0.0f;
        for (int s = 0; s < splits; ++s) v += s_part[s * ROWS * p.r + i];
        s_u[i] = v * scale;
    }
    __syncthreads();
    if (cnt == 1)
        expand_columns<W, 1>(b, p, s_tok, cnt, s_u, n0, n1);
    else
        expand_columns<W, 8>(b, p, s_tok, cnt, s_u, n0, n1);
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
// the tile list itself.  cnt, off, toff: shared arrays of MAX_ADAPTERS + 2.
__device__ __forceinline__ void scan_groups(const AdapterArgs& p, int tile_rows, const int* cnt, int* off, int* toff) {
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
        *p.n_tiles = toff[p.n + 1];
    }
    __syncthreads();
    const int tiles = toff[p.n + 1];
    for (int i = tid; i < tiles; i += GROUP_THREADS) {
        int lo = 0, hi = p.n;  // the last group whose tiles start at or before i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (toff[mid] <= i) lo = mid; else hi = mid - 1;
        }
        const int first = (i - toff[lo]) * tile_rows;
        p.tiles[i] = make_int4(lo < p.n ? lo : -1, off[lo] + first, min(tile_rows, cnt[lo] - first), 0);
    }
}

// Up to GROUP_CHUNK rows: one CTA does it all.
__global__ void __launch_bounds__(GROUP_THREADS) adapters_group_kernel(const __grid_constant__ AdapterArgs p, int tile_rows) {
    __shared__ int cnt[MAX_ADAPTERS + 2], off[MAX_ADAPTERS + 2], toff[MAX_ADAPTERS + 2];
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < p.n + 2; i += GROUP_THREADS) cnt[i] = 0;
    __syncthreads();
    int grp[GROUP_IDS], rnk[GROUP_IDS];
    bool bad = false;
    rank_ids(p.ids, 0, p.T, p.n, cnt, grp, rnk, bad);
    const int any = __syncthreads_or(bad);
    scan_groups(p, tile_rows, cnt, off, toff);
#pragma unroll
    for (int i = 0; i < GROUP_IDS; ++i)
        if (grp[i] >= 0) p.perm[off[grp[i]] + rnk[i]] = i * GROUP_THREADS + threadIdx.x;
    if (threadIdx.x == 0) *p.status = any ? STATUS_BAD_ADAPTER_INDEX : 0u;
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
    scan_groups(p, tile_rows, cnt, off, toff);
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

cudaError_t launch_group(const AdapterArgs& p, int tile_rows, cudaStream_t s) {
    const int nchunks = (int)ceil_div(p.T, GROUP_CHUNK);
    if (nchunks == 1) {
        adapters_group_kernel<<<1, GROUP_THREADS, 0, s>>>(p, tile_rows);
        return cudaGetLastError();
    }
    adapters_count_kernel<<<nchunks, GROUP_THREADS, 0, s>>>(p);
    adapters_scan_kernel<<<1, GROUP_THREADS, 0, s>>>(p, nchunks, tile_rows);
    adapters_place_kernel<<<nchunks, GROUP_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

// A launch that may begin while the kernel before it drains (its kernels wait
// with pdl_wait before they read anything).
template <class... A>
cudaError_t launch_dependent(void (*kernel)(A...), unsigned grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class W>
cudaError_t launch_rows(const AdapterArgs& p, const DeviceInfo& dev, cudaStream_t s) {
    const bool in = p.T <= INLINE_T;
    const int64_t groups = in ? std::min<int64_t>(p.T, (p.n + 1) + p.T / ROWS) : p.T / ROWS + p.n + 1;
    // columns per cluster: as many steps of COLS as leave two clusters' worth
    // of CTAs for every 8 SMs; u is computed once per cluster
    const int64_t steps = ceil_div(p.N, COLS);
    const int64_t iters = std::max<int64_t>(1, std::min<int64_t>(steps, groups * steps / (2 * dev.sm_count / CL)));
    const int64_t chunks = ceil_div(steps, iters);
    const int64_t grid = groups * chunks * CL;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    if (in) {
        adapters_rows_kernel<W, true><<<(unsigned)grid, THREADS, 0, s>>>(p, (int)chunks, (int)iters);
        return cudaGetLastError();
    }
    cudaError_t e = launch_group(p, ROWS, s);
    if (e != cudaSuccess) return e;
    return launch_dependent(adapters_rows_kernel<W, false>, (unsigned)grid, THREADS, 0, s, p, (int)chunks, (int)iters);
}

template <class W>
cudaError_t launch_typed(const AdapterArgs& p, const DeviceInfo& dev, cudaStream_t s) {
    return launch_rows<W>(p, dev, s);
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

cudaError_t launch_adapters(const AdapterArgs& p, int dtype, const DeviceInfo& dev, cudaStream_t s) {
    if (dtype == 0) return launch_typed<float>(p, dev, s);
    if (dtype == 1) return launch_typed<__half>(p, dev, s);
    return launch_typed<__nv_bfloat16>(p, dev, s);
}

}  // namespace moeq4
