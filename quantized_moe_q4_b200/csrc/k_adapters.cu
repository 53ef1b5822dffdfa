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
#include "tc.cuh"

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
constexpr int TILE_MIN_ROWS = 16; // rows per adapter from which the tile kernel is used

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

__device__ __forceinline__ void st_cluster4(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

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

// ------------------------------------------------------------------ tile kernel
//
// Many rows: tiles of 128 rows of one adapter on the tensor cores, tf32 with
// binary32 accumulators.  A binary32 value is split into two tf32 parts of 11
// significant bits, v = hi + lo up to 2^-22 |v|; binary16 and bfloat16 weights
// are tf32 values already, so a product with them takes two MMAs, and one of
// two binary32 values three (lo * lo, 2^-22 of the product, is left out).
//   1. u' = x A^T: each CTA of the cluster sums over its eighth of H.
//      M = the tile's rows, N = r, operands K-major in 32-column panels with
//      128-byte rows swizzled in 16-byte units (SWIZZLE_128B).
//   2. the eight partial sums are joined through distributed shared memory:
//      CTA c adds rows 16 c .. 16 c + 15 in rank order and hands them to all.
//   3. d^T = B u^T over the CTA's blocks of 128 columns of y: M = columns of y,
//      N = the tile's rows, so that a TMEM lane is a column and every access
//      of base and y is 32 consecutive floats, whatever their alignment.
// TMEM is held inside steps 1 and 3 only, never across a cluster barrier: a
// CTA that holds some waits for nothing but its own MMAs, so CTAs that wait
// for TMEM on other SMs cannot block each other in a ring.

constexpr int TM = 128;                 // rows of a tile; columns of y in a block
constexpr int PK = 32;                  // columns of a panel (128 bytes of binary32)
constexpr uint32_t PANEL = TM * 128;    // bytes of a panel of 128 rows

__device__ __forceinline__ uint32_t swizzled(int row, int c16) { return (uint32_t)(row * 128 + ((c16 ^ (row & 7)) << 4)); }

// Descriptor of a K-major operand in a swizzled panel: 8-row groups of 1024 bytes.
__device__ __forceinline__ uint64_t panel_desc(uint32_t smem_addr) {
    return (uint64_t)((smem_addr >> 4) & 0x3fffu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// kind::tf32, binary32 accumulator, both operands K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_tf32(int M, int N) {
    return (1u << 4) | (2u << 7) | (2u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_tf32(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// The tf32 value nearest to v (ties away from zero), as binary32.
__device__ __forceinline__ float tf32_near(float v) { return __uint_as_float((__float_as_uint(v) + 0x1000u) & 0xffffe000u); }

// Four values as two tf32 parts, into the same place of two panels.
__device__ __forceinline__ void store_split(char* hi, char* lo, uint32_t at, float4 v) {
    const float4 h = make_float4(tf32_near(v.x), tf32_near(v.y), tf32_near(v.z), tf32_near(v.w));
    *reinterpret_cast<float4*>(hi + at) = h;
    *reinterpret_cast<float4*>(lo + at) =
        make_float4(tf32_near(v.x - h.x), tf32_near(v.y - h.y), tf32_near(v.z - h.z), tf32_near(v.w - h.w));
}

// A thread's share of a panel of weights in flight: rows of 32 elements at a
// pitch, 16 bytes at a time.
template <class W>
struct WeightPanel {
    static constexpr bool SPLIT = sizeof(W) == 4;
    static constexpr int EPU = 16 / (int)sizeof(W), UPR = PK / EPU, N = TM * UPR / THREADS;
    uint4 q[N];
    // rows and columns past the given ones are zeros
    __device__ __forceinline__ void load(const W* src, int64_t pitch, int rows, int cols) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = i * THREADS + threadIdx.x, row = u / UPR, c = u % UPR;
            q[i] = make_uint4(0, 0, 0, 0);
            if (row < rows && c * EPU < cols) q[i] = __ldg(reinterpret_cast<const uint4*>(src + row * pitch + c * EPU));
        }
    }
    // rows < `rows` (a multiple of 8) into the panel(s); lo: binary32 only
    __device__ __forceinline__ void store(char* hi, char* lo, int rows) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = i * THREADS + threadIdx.x, row = u / UPR, c = u % UPR;
            if (row >= rows) continue;
            if constexpr (SPLIT) {
                store_split(hi, lo, swizzled(row, c),
                            make_float4(__uint_as_float(q[i].x), __uint_as_float(q[i].y), __uint_as_float(q[i].z),
                                        __uint_as_float(q[i].w)));
            } else {
                float v[8];
                unpack8(q[i], v, (const W*)nullptr);
                *reinterpret_cast<float4*>(hi + swizzled(row, 2 * c)) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4*>(hi + swizzled(row, 2 * c + 1)) = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
    }
};

// Shared memory of the tile kernel, from a 1024-byte aligned start.
//   step 1: two stages of x panel (hi, lo) and A panel (hi, and lo of binary32)
//   step 2: partial sums at 0, u at `mid`
//   step 3: panels of u (all hi, then all lo) at 0, two slots of B panel at `mid`
struct TileSmem {
    uint32_t wpanel, stage, mid, slot, total;
    __host__ __device__ TileSmem(int r, bool split) {
        const uint32_t panels = (uint32_t)(r + PK - 1) / PK;
        wpanel = (uint32_t)((r + 15) / 16 * 16) * 128;
        stage = 2 * PANEL + wpanel * (split ? 2 : 1);
        mid = 2 * panels * PANEL;
        slot = PANEL * (split ? 2 : 1);
        const uint32_t u = TM * (uint32_t)(r + 4) * 4, tail = u > 2 * slot ? u : 2 * slot;
        total = 2 * stage > mid + tail ? 2 * stage : mid + tail;
    }
};

template <class W>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(THREADS, 2)
    adapters_tile_kernel(const __grid_constant__ AdapterArgs p) {
    constexpr bool SPLIT = WeightPanel<W>::SPLIT;
    extern __shared__ char s_raw[];
    __shared__ int s_tok[TM];
    __shared__ int64_t s_off[2][TM];  // offsets of the rows of base and y
    __shared__ uint64_t s_full[2], s_dfull[2];
    __shared__ uint32_t s_tmem;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    char* sm = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);
    const uint32_t sa = smem_u32(sm);
    const int r = p.r;
    const TileSmem lay(r, SPLIT);

    pdl_wait();
    const int g = (int)(blockIdx.x / CL);
    if (g >= *p.n_tiles) return;  // uniform over the cluster
    const int4 tile = p.tiles[g];
    const int id = tile.x, cnt = tile.z;
    for (int i = tid; i < TM; i += THREADS) {
        const int t = i < cnt ? p.perm[tile.y + i] : -1;
        s_tok[i] = t;
        s_off[0][i] = (int64_t)t * p.ldb;
        s_off[1][i] = (int64_t)t * p.ldy;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_dfull[i], 1);
        }
        mbar_fence_init();
    }
    __syncthreads();
    if (id < 0) {  // no adapter (never in place: such rows have no tile then)
        for (int t = (int)rank; t < cnt; t += CL)
            for (int64_t n = tid; n < p.N; n += THREADS) p.y[s_off[1][t] + n] = p.base ? p.base[s_off[0][t] + n] : 0.0f;
        return;
    }
    const W* a = static_cast<const W*>(p.a) + (int64_t)id * r * p.H;
    const W* b = static_cast<const W*>(p.b) + (int64_t)id * p.N * r;
    // every wait is bounded; one that gives up is reported and not repeated
    bool alive = true;
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (alive && !mbar_wait_bounded(bar, parity, 1u << 22)) {
            alive = false;
            atomicOr(p.status, STATUS_SPIN_TIMEOUT);
        }
        tc_fence_after_sync();
    };

    // ---- 1: this CTA's part of u' over columns [h0, h0 + H / CL)
    const uint32_t cols1 = r <= 32 ? 32u : r <= 64 ? 64u : 128u;
    if (warp == 0) tmem_alloc(&s_tmem, cols1);
    const int chunks = p.H / CL / PK, h0 = (int)rank * (p.H / CL);
    const float* xr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = s_tok[i * 32 + (tid >> 3)];
        xr[i] = t < 0 ? nullptr : p.x + (int64_t)t * p.ldx + h0 + 4 * (tid & 7);
    }
    float4 xv[4];
    WeightPanel<W> wv;
    const auto load1 = [&](int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            xv[i] = xr[i] ? __ldg(reinterpret_cast<const float4*>(xr[i] + c * PK)) : make_float4(0.f, 0.f, 0.f, 0.f);
        wv.load(a + h0 + c * PK, p.H, r, PK);
    };
    load1(0);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    uint32_t it = 0;  // panels handed to the tensor core so far, over steps 1 and 3
    const int n16 = (r + 15) / 16 * 16;
    for (int c = 0; c < chunks; ++c, ++it) {
        const uint32_t st = it & 1;
        if (it >= 2) wait(&s_full[st], ((it - 2) >> 1) & 1);
        char* s = sm + st * lay.stage;
#pragma unroll
        for (int i = 0; i < 4; ++i) store_split(s, s + PANEL, swizzled(i * 32 + (tid >> 3), tid & 7), xv[i]);
        wv.store(s + 2 * PANEL, s + 2 * PANEL + lay.wpanel, r);
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after_sync();
            const uint32_t s0 = sa + st * lay.stage;
            const uint64_t xh = panel_desc(s0), xl = panel_desc(s0 + PANEL), wh = panel_desc(s0 + 2 * PANEL),
                           wl = panel_desc(s0 + 2 * PANEL + lay.wpanel);
#pragma unroll
            for (int k = 0; k < PK / 8; ++k) {
                mma_tf32(s_tmem, xh + 2 * k, wh + 2 * k, idesc_tf32(TM, n16), c + k > 0);
                mma_tf32(s_tmem, xl + 2 * k, wh + 2 * k, idesc_tf32(TM, n16), true);
                if (SPLIT) mma_tf32(s_tmem, xh + 2 * k, wl + 2 * k, idesc_tf32(TM, n16), true);
            }
            mma_commit(&s_full[st]);
        }
        if (c + 1 < chunks) load1(c + 1);
    }
    // this CTA's blocks of columns of y; the first panel of B travels while u is joined
    const int64_t blocks = (p.N + TM - 1) / TM;
    const int panels = (r + PK - 1) / PK;
    const auto load3 = [&](int64_t nb, int k) {
        wv.load(b + nb * TM * r + k * PK, r, (int)min((int64_t)TM, p.N - nb * TM), r - k * PK);
    };
    if ((int64_t)rank < blocks) load3(rank, 0);

    // ---- 2: join the partial sums
    wait(&s_full[(it - 1) & 1], ((it - 1) >> 1) & 1);
    const int pitch = (r + 4) * 4;  // bytes of a row of partial sums and of u
    for (int c = warp >> 2; c < r / 8; c += 2) {
        uint32_t v[8];
        tmem_ld8(s_tmem + (uint32_t)(((warp & 3) * 32) << 16) + 8u * c, v);
        tmem_wait_ld();
        float4* dst = reinterpret_cast<float4*>(sm + ((warp & 3) * 32 + lane) * pitch + 32 * c);
        dst[0] = make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3]));
        dst[1] = make_float4(__uint_as_float(v[4]), __uint_as_float(v[5]), __uint_as_float(v[6]), __uint_as_float(v[7]));
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(s_tmem, cols1);
    cluster_arrive();
    cluster_wait();
    const float scale = p.scale ? __ldg(p.scale + id) : 1.0f;
    for (int i = tid; i < TM / CL * (r / 4); i += THREADS) {
        const uint32_t at = (uint32_t)(((int)rank * (TM / CL) + i / (r / 4)) * pitch + i % (r / 4) * 16);
        float4 part[CL];
#pragma unroll
        for (int c = 0; c < CL; ++c) part[c] = ld_cluster4(map_rank(sa + at, c));
        float4 v = part[0];
#pragma unroll
        for (int c = 1; c < CL; ++c) {
            v.x += part[c].x; v.y += part[c].y; v.z += part[c].z; v.w += part[c].w;
        }
        v.x *= scale; v.y *= scale; v.z *= scale; v.w *= scale;
#pragma unroll
        for (int c = 0; c < CL; ++c) st_cluster4(map_rank(sa + lay.mid + at, c), v);
    }
    cluster_arrive();
    cluster_wait();
    if ((int64_t)rank >= blocks) return;  // (no CTA reads or writes another's memory from here on)
    // u as two tf32 parts in panels; row = row of the tile
    if (warp == 0) tmem_alloc(&s_tmem, 2 * TM);
    for (int i = tid; i < TM * (r / 4); i += THREADS) {
        const int row = i / (r / 4), c = i % (r / 4);
        store_split(sm + (c / 8) * PANEL, sm + (panels + c / 8) * PANEL, swizzled(row, c % 8),
                    *reinterpret_cast<const float4*>(sm + lay.mid + row * pitch + 16 * c));
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();

    // ---- 3: y = base + (B u^T)^T, block by block; MMAs of a block run under
    // the epilogue of the block before it
    const auto epilogue = [&](int64_t nb, uint32_t buf) {
        const int64_t n = nb * TM + (warp & 3) * 32 + lane;
        const uint32_t taddr = s_tmem + (uint32_t)(((warp & 3) * 32) << 16) + buf * TM;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            const int t0 = (warp >> 2) * 64 + h * 32;
            if (t0 >= cnt) break;
            float bv[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
                bv[j] = (t0 + j < cnt && n < p.N && p.base) ? p.base[s_off[0][t0 + j] + n] : 0.0f;
            uint32_t v[32];
            __syncwarp();
            tmem_ld32(taddr + t0, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (t0 + j < cnt && n < p.N) p.y[s_off[1][t0 + j] + n] = bv[j] + __uint_as_float(v[j]);
        }
    };
    uint32_t nd = 0;
    for (int64_t nb = rank; nb < blocks; nb += CL, ++nd) {
        for (int k = 0; k < panels; ++k, ++it) {
            const uint32_t st = it & 1;
            if (it >= 2) wait(&s_full[st], ((it - 2) >> 1) & 1);
            char* s = sm + lay.mid + st * lay.slot;
            wv.store(s, s + PANEL, TM);
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncthreads();
            if (tid == 0) {
                tc_fence_after_sync();
                const uint32_t s0 = sa + lay.mid + st * lay.slot;
                const uint64_t bh = panel_desc(s0), bl = panel_desc(s0 + PANEL), uh = panel_desc(sa + k * PANEL),
                               ul = panel_desc(sa + (panels + k) * PANEL);
                const uint32_t d = s_tmem + (nd & 1) * TM;
                const int steps = min(PK, r - k * PK) / 8;
                for (int j = 0; j < steps; ++j) {
                    mma_tf32(d, bh + 2 * j, uh + 2 * j, idesc_tf32(TM, TM), k + j > 0);
                    mma_tf32(d, bh + 2 * j, ul + 2 * j, idesc_tf32(TM, TM), true);
                    if (SPLIT) mma_tf32(d, bl + 2 * j, uh + 2 * j, idesc_tf32(TM, TM), true);
                }
                mma_commit(&s_full[st]);
                if (k == panels - 1) mma_commit(&s_dfull[nd & 1]);
            }
            if (k + 1 < panels)
                load3(nb, k + 1);
            else if (nb + CL < blocks)
                load3(nb + CL, 0);
        }
        if (nd > 0) {
            wait(&s_dfull[(nd - 1) & 1], ((nd - 1) >> 1) & 1);
            epilogue(nb - CL, (nd - 1) & 1);
        }
    }
    wait(&s_dfull[(nd - 1) & 1], ((nd - 1) >> 1) & 1);
    epilogue((int64_t)rank + (int64_t)(nd - 1) * CL, (nd - 1) & 1);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(s_tmem, 2 * TM);
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
cudaError_t launch_tiles(const AdapterArgs& p, cudaStream_t s) {
    const TileSmem lay(p.r, sizeof(W) == 4);
    const size_t smem = lay.total + 1024;
    int per_sm = 0;  // (raises the kernel's shared-memory limit)
    cudaError_t e = kernel_occupancy(reinterpret_cast<const void*>(adapters_tile_kernel<W>), THREADS, smem, &per_sm);
    if (e != cudaSuccess) return e;
    e = launch_group(p, TM, s);
    if (e != cudaSuccess) return e;
    const int64_t tiles = p.T / TM + std::min<int64_t>(p.n + 1, p.T);
    return launch_dependent(adapters_tile_kernel<W>, (unsigned)(tiles * CL), THREADS, smem, s, p);
}

// Tensor cores once adapters see enough rows to fill a good part of a tile.
template <class W>
cudaError_t launch_typed(const AdapterArgs& p, const DeviceInfo& dev, cudaStream_t s) {
    if (p.T > INLINE_T && p.T >= (int64_t)TILE_MIN_ROWS * p.n) return launch_tiles<W>(p, s);
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
