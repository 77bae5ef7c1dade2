// hq_paged.h -- argument blocks, launchers and shared device code of the
// serving operators: rotary positions, the append to a paged KV cache,
// attention over it and the join of two partial attention results (not part
// of the public ABI).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "hq_internal.h"

namespace hq {

constexpr int kStatusIndex = 32;

// A [tokens][heads][head_dim] array; strides in elements.
struct Rows {
    void *p;
    int64_t ts, hs;
    int f32;  // binary32 elements (else bf16)
};

// ------------------------------------------------------------ positions
// Rotation and append: `heads` rows of `x` (queries) go to `y`; if kvh > 0,
// kvh rows of k (rotated) and v (copied) go to the page pool.
struct PosArgs {
    Rows x, y, k, v;
    int64_t tokens;
    int heads, kvh, head_dim, rotary;  // rotary: rotated elements per head (0: none)
    int interleaved, inverse;
    float amplitude;
    const int64_t *positions;
    const uint64_t *turns;             // theta / 2 pi in 2^-64 turns, rotary / 2 entries
    const int64_t *slots;              // null: no append
    uint16_t *pk, *pv;
    int64_t page_stride, head_stride, slot_stride, nslots;
    int page_shift;
    int tokens_per_block;
    FastDiv items_div, unit_div;       // by items per token, by items per head
    int32_t *status;
};

cudaError_t launch_positions(const PosArgs &a, cudaStream_t s);

// ------------------------------------------------------------ join
struct MergeArgs {
    Rows a, b, out;
    const float *lse_a, *lse_b;  // [tokens][heads]
    float *lse;                  // may be null
    int64_t tokens;
    int heads, head_dim;
    FastDiv heads_div;
};

cudaError_t launch_merge(const MergeArgs &a, cudaStream_t s);

// ------------------------------------------------------------ attention
// Where a block's share of the tiles begins (written by the plan kernel).
struct PagedStart {
    int32_t b, h, rt, tile;  // sequence, KV head, row tile, tile within the job
    int64_t job;             // the job's first unit of work
};

struct PagedArgs {
    Rows q, out;
    float *lse;              // [tokens][heads * group]; may be null
    const int32_t *q_start, *kv_len, *table;
    int64_t table_stride;
    int64_t tokens;
    int batch, max_q, max_tokens;  // max_tokens: tokens a row of the table can hold
    int heads, group;
    FastDiv group_div;
    const uint16_t *k, *v;
    int64_t page_stride, head_stride, slot_stride;
    uint32_t pages;
    int page_shift;
    float scale_log2;        // |scale| log2 e
    int q_mode;              // 0: q, 1: -q (negative scale), 2: zeros (scale 0)
    int causal;
    int window;              // positions a query sees, itself included (0: all)
    int row_lo, row_hi;      // sequences with row_lo < q_len * group <= row_hi
    // plan (workspace)
    int64_t *prefix;         // [batch + 1] units of work before each sequence
    PagedStart *start;       // [grid]
    uint32_t *counter;       // [grid] finished parts of the job whose first tile block c holds
    float *part;             // [2 grid] partial results
    int grid, min_units;     // blocks; least units of work a block takes
    int job_cost;            // what a job costs beside its tiles, in tiles
    int split, row_tiles;    // clusters (no plan): blocks of a job, row tiles of the longest sequence
    int stall_kind, stall;   // test hook: what block 0 withholds: this copy, or the products' notices from this tile on
    int32_t *status;
};
constexpr int kStallNone = 0, kStallCopy = 1, kStallProduct = 2;

// What a launch of one of the kernels needs of the workspace.
struct PagedShare {
    int grid, rows;                // blocks (0: not launched), rows per row tile
    int row_lo, row_hi;            // the sequences it takes (rows: new tokens x group)
    int split, row_tiles;          // clusters of `split` blocks, one job each (0: planned shares)
    uint64_t prefix, start, counter, part;  // offsets
};

struct PagedPlan {
    PagedShare few, many;          // mma.sync and tcgen05 kernels
    uint64_t total;
};

PagedPlan paged_plan(int64_t batch, int64_t tokens, int64_t max_q, int64_t max_kv, int heads, int group, int head_dim,
                     int64_t window);
cudaError_t launch_paged(const PagedArgs &a, const PagedPlan &p, int head_dim, void *workspace, cudaStream_t s);
// The tcgen05 kernel (planned before), and its row tile.
cudaError_t launch_paged_many(const PagedArgs &a, int head_dim, cudaStream_t s);
int paged_many_rows(int head_dim);

#ifdef __CUDACC__
// ------------------------------------------------------------ device side
// One sequence as a kernel sees it.
struct Seq {
    int q0, nq, kv, rows;
};

// Sequence b; rows = 0 if it is not this kernel's, empty, or inconsistent
// (offsets out of order or past the rows, more new tokens than max_q, more
// cached tokens than its row of the table holds: `bad`).
__device__ __forceinline__ Seq load_seq(const PagedArgs &a, int b, bool &bad)
{
    Seq s;
    s.q0 = a.q_start[b];
    const int q1 = a.q_start[b + 1];
    s.kv = a.kv_len[b];
    bad = s.q0 < 0 || q1 < s.q0 || q1 > a.tokens || q1 - s.q0 > a.max_q || s.kv < 0 || s.kv > a.max_tokens;
    s.nq = bad ? 0 : q1 - s.q0;
    s.rows = s.nq * a.group;
    if (s.rows <= a.row_lo || s.rows > a.row_hi) s.rows = 0;
    return s;
}

// First and last + 1 cached token that any of the new tokens j0 .. j1 of a
// sequence sees.
__device__ __forceinline__ void seen_range(const PagedArgs &a, const Seq &s, int j0, int j1, int &lo, int &hi)
{
    const int64_t first = (int64_t)s.kv - s.nq;
    int64_t l = a.window ? first + j0 + 1 - a.window : 0, h = a.causal ? first + j1 + 1 : s.kv;
    if (l < 0) l = 0;
    if (h > s.kv) h = s.kv;
    if (h < 0) h = 0;
    if (l > h) l = h;
    lo = (int)l;
    hi = (int)h;
}

// Tiles [t0, t0 + n) of T tokens that row tile rt (RT packed rows) reads; a
// job always has one tile at least (it writes its rows even if they see nothing).
template <int T, int RT>
__device__ __forceinline__ void job_tiles(const PagedArgs &a, const Seq &s, int rt, int &t0, int &n, int &lo, int &hi)
{
    const int r0 = rt * RT, r1 = min(r0 + RT, s.rows) - 1;
    seen_range(a, s, (int)fast_div((uint32_t)r0, a.group_div), (int)fast_div((uint32_t)r1, a.group_div), lo, hi);
    t0 = lo / T;
    n = (hi + T - 1) / T - t0;
    if (n < 1) n = 1;
}

// The block's walk over its share of the work: segments of jobs (sequence, KV
// head, row tile), in the order sequence, KV head, row tile, tile.  A job is
// job_cost units (queries in, results out) and then a unit for each of its
// tiles; block c takes units total c / grid .. total (c + 1) / grid, of which
// only tiles count as work to do (a share that begins within a job's own units
// begins with its first tile).
template <int T, int RT>
struct SegWalk {
    Seq s;
    int b, h, rt, nrt;
    int t0, n, lo, hi;    // the job's tiles and cached range
    int first, count;     // the segment: tiles t0 + first .. + count
    int grid;
    int64_t job, end, total;  // the job's first unit, the end of the share

    __device__ __forceinline__ bool begin(const PagedArgs &a)
    {
        total = a.prefix[a.batch];
        const int64_t most = (total + a.min_units - 1) / a.min_units;
        grid = (int)min((int64_t)a.grid, most);
        const int c = blockIdx.x;
        if (c >= grid) return false;
        end = total * (c + 1) / grid;
        const PagedStart st = a.start[c];
        b = st.b;
        h = st.h;
        rt = st.rt;
        first = st.tile;
        job = st.job;
        bool bad;
        s = load_seq(a, b, bad);
        nrt = (s.rows + RT - 1) / RT;
        job_tiles<T, RT>(a, s, rt, t0, n, lo, hi);
        return cut(a);
    }

    // the segment's tiles, from `first`
    __device__ __forceinline__ bool cut(const PagedArgs &a)
    {
        count = (int)min((int64_t)(n - first), end - (job + a.job_cost + first));
        return count > 0;
    }

    __device__ __forceinline__ bool next(const PagedArgs &a)
    {
        job += a.job_cost + n;
        if (job + a.job_cost >= end) return false;
        first = 0;
        if (++rt == nrt) {
            rt = 0;
            if (++h == a.heads) {
                h = 0;
                bool bad;
                if (++b >= a.batch) return false;
                s = load_seq(a, b, bad);
                if (s.rows == 0) {
                    // the sequence with work in it that begins at this unit: the last
                    // that begins here (one by one, millions of empty ones would
                    // outlast the other warps' waits)
                    int above = a.batch - 1;
                    while (b < above) {
                        const int mid = (int)(((int64_t)b + above + 1) >> 1);
                        if (a.prefix[mid] <= job) b = mid;
                        else above = mid - 1;
                    }
                    s = load_seq(a, b, bad);
                }
                nrt = (s.rows + RT - 1) / RT;
            }
        }
        job_tiles<T, RT>(a, s, rt, t0, n, lo, hi);
        return cut(a);
    }

    // Without a plan: a cluster of `split` blocks takes one job, each an equal
    // share of its tokens (possibly none).
    __device__ __forceinline__ bool begin_cluster(const PagedArgs &a)
    {
        const int job = (int)blockIdx.x / a.split, rank = (int)blockIdx.x - job * a.split;
        const int bh = job / a.row_tiles;
        rt = job - bh * a.row_tiles;
        b = bh / a.heads;
        h = bh - b * a.heads;
        bool bad;
        s = load_seq(a, b, bad);
        if (bad && rank == 0 && h == 0 && rt == 0 && threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusIndex);
        if (rt * RT >= s.rows) return false;
        job_tiles<T, RT>(a, s, rt, t0, n, lo, hi);
        first = (int)((int64_t)n * rank / a.split);
        count = (int)((int64_t)n * (rank + 1) / a.split) - first;
        return true;
    }

    __device__ __forceinline__ bool whole() const { return count == n; }
    __device__ __forceinline__ int block_of(int64_t unit) const { return (int)(((unit + 1) * grid - 1) / total); }
    // blocks that hold the first and the last tile of this job
    __device__ __forceinline__ int owner(const PagedArgs &a) const { return block_of(job + a.job_cost); }
    __device__ __forceinline__ int last(const PagedArgs &a) const { return block_of(job + a.job_cost + n - 1); }
    // a block's parts: one that begins inside a job, one that begins with it
    __device__ __forceinline__ int slot() const { return 2 * (int)blockIdx.x + (first == 0 ? 1 : 0); }
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------ results
// Elements 4 c .. 4 c + 3 of packed row r of a job, from its unnormalised sum,
// maximum (powers of two) and weight sum; a row that saw nothing is zero.
__device__ __forceinline__ void finish_row(const PagedArgs &a, int q0, int h, int r, int c, float4 v, float m, float l)
{
    const int j = (int)fast_div((uint32_t)r, a.group_div), head = h * a.group + r - j * a.group;
    const int64_t tok = q0 + j, off = tok * a.out.ts + head * a.out.hs + 4 * c;
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    if (l == 0.0f) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (a.out.f32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out.p) + off) =
            make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * f, v.y * f), hi = __floats2bfloat162_rn(v.z * f, v.w * f);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out.p) + off) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
    if (c == 0 && a.lse)
        a.lse[tok * (a.heads * a.group) + head] = l == 0.0f ? -INFINITY : fmaf(m, 0.693147180559945309f, logf(l));
}

// A part: m of RT rows, l of RT rows, then RT x D sums.
template <int RT, int D>
__device__ __forceinline__ const float *part_of(const PagedArgs &a, int c, int c0)
{
    return a.part + (int64_t)(2 * c + (c == c0 ? 1 : 0)) * (RT * (D + 2));
}

// Join parts k0 .. k1 of a job's nr rows (packed rows r0 ..) in order: load(k, r,
// c, m, l, v) gives part k's maximum, weight sum and columns 4 c .. of row r.
// Thread e0 of `threads` takes N groups of 4 columns at once, G parts' loads in
// flight.
template <int D, int N, int G, typename F>
__device__ __forceinline__ void join_some(const PagedArgs &a, int q0, int h, int r0, int nr, int e0, int threads, int k0, int k1,
                                          F load)
{
    constexpr int C4 = D / 4;
    for (; e0 < nr * C4; e0 += N * threads) {
        int r[N], c[N];
        float mt[N], l[N];
        float4 acc[N];
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int e = min(e0 + i * threads, nr * C4 - 1);  // (past the last: the last again, not written)
            r[i] = e / C4;
            c[i] = e % C4;
            mt[i] = -INFINITY;
            l[i] = 0.0f;
            acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        for (int k = k0; k <= k1; k += G) {
            float m[G][N], s[G][N];
            float4 v[G][N];
#pragma unroll
            for (int g = 0; g < G; g++)
#pragma unroll
                for (int i = 0; i < N; i++) {
                    m[g][i] = -INFINITY;
                    s[g][i] = 0.0f;
                    v[g][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (k + g <= k1) load(k + g, r[i], c[i], m[g][i], s[g][i], v[g][i]);
                }
#pragma unroll
            for (int i = 0; i < N; i++) {
                float top = mt[i];
#pragma unroll
                for (int g = 0; g < G; g++) top = fmaxf(top, m[g][i]);
                const float base = top == -INFINITY ? 0.0f : top, f = ex2(mt[i] - base);
                mt[i] = top;
                l[i] *= f;
                acc[i] = make_float4(acc[i].x * f, acc[i].y * f, acc[i].z * f, acc[i].w * f);
#pragma unroll
                for (int g = 0; g < G; g++) {
                    const float w = ex2(m[g][i] - base);
                    l[i] = fmaf(w, s[g][i], l[i]);
                    acc[i].x = fmaf(w, v[g][i].x, acc[i].x);
                    acc[i].y = fmaf(w, v[g][i].y, acc[i].y);
                    acc[i].z = fmaf(w, v[g][i].z, acc[i].z);
                    acc[i].w = fmaf(w, v[g][i].w, acc[i].w);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; i++)
            if (e0 + i * threads < nr * C4) finish_row(a, q0, h, r0 + r[i], c[i], acc[i], mt[i], l[i]);
    }
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------ clusters
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// the address in block `rank`'s shared memory that corresponds to `addr` here
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, int rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float cluster_ld(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Launch a kernel that may become resident before the one in front of it ends
// (it waits for that one's results with pdl_wait).
template <typename... P>
inline cudaError_t launch_dependent(void (*kern)(P...), int grid, int threads, size_t smem, cudaStream_t s, P... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Launch a kernel in clusters of `size` blocks.
template <typename... P>
inline cudaError_t launch_clusters(void (*kern)(P...), int grid, int size, int threads, size_t smem, cudaStream_t s, P... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)size;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}
#endif

}  // namespace hq
