// hq_paged.cu -- attention over a paged KV cache for few new tokens per
// sequence (decoding, drafts), its work plan, and the join of two partial
// attention results (sm_100a).  Longer chunks: hq_paged_tc.cu.
//
// The new tokens of a sequence and the `group` query heads that share a KV
// head are packed into rows (row r: token r / group, head r % group), so each
// cached vector is read once for all of them.  A job is one (sequence, KV
// head, row tile); its tokens come in tiles of 64.  The tiles of all jobs form
// one list that the blocks of a single wave cut into equal shares: lengths may
// be as uneven as they like.  A block writes a job it holds whole; a job cut
// between blocks leaves partial results (running maximum m, sum l,
// unnormalised output), and the last block to finish it -- found with a
// counter, no waiting -- adds them in block order, so results do not depend on
// which block that was.
#include "hq_paged.h"

namespace hq {

namespace {

constexpr int kFewThreads = 128, kFewT = 64;
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes global -> shared; nothing is read where !valid (zeros are stored)
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool valid)
{
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// byte offset of 16-byte chunk c of row r in a [rows][D] bf16 tile; chunks
// are swizzled by row so that 8 consecutive rows meet 8 bank groups
template <int D>
__device__ __forceinline__ uint32_t tile_off(int r, int c) { return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4)); }

// bf16 stages of K and V tiles: about 64 KB in flight per SM keep HBM busy
template <int D>
constexpr int few_stages() { return D == 64 ? 4 : 3; }
template <int D, int WM>
constexpr size_t few_smem() { return (size_t)16 * WM * D * 2 + (size_t)few_stages<D>() * 2 * kFewT * D * 2; }

}  // namespace

// ------------------------------------------------------------ plan
// Tiles before each sequence, the place where each block's share begins, and
// cleared counters.  One block; a warp counts a sequence's row tiles.
template <int T, int RT>
__device__ __forceinline__ void plan_share(const PagedArgs &a, const int parts)
{
    __shared__ int64_t w[kPlanThreads];
    __shared__ int64_t wsum[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int c = tid; c < a.grid * parts; c += kPlanThreads) a.counter[c] = 0u;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        for (int i = warp; i < kPlanThreads; i += kPlanThreads / 32) {
            const int b = b0 + i;
            int64_t tiles = 0;
            if (b < a.batch) {
                bool bad;
                const Seq s = load_seq(a, b, bad);
                if (bad && lane == 0 && a.status) atomicOr(a.status, kStatusIndex);
                const int nrt = (s.rows + RT - 1) / RT;
                for (int rt = lane; rt < nrt; rt += 32) {
                    int t0, n, lo, hi;
                    job_tiles<T, RT>(a, s, rt, t0, n, lo, hi);
                    tiles += n;
                }
            }
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) tiles += __shfl_xor_sync(FULL, tiles, m);
            if (lane == 0) w[i] = tiles * a.heads;
            if (b0 + i + kPlanThreads / 32 >= a.batch) {  // the rest of the chunk is past the last sequence
                for (int k = i + kPlanThreads / 32; k < kPlanThreads; k += kPlanThreads / 32)
                    if (lane == 0) w[k] = 0;
                break;
            }
        }
        __syncthreads();
        const int64_t mine = w[tid];
        int64_t incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(FULL, incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int64_t base = before, all = before;
        for (int k = 0; k < kPlanThreads / 32; k++) {
            if (k < warp) base += wsum[k];
            all += wsum[k];
        }
        if (b0 + tid < a.batch) a.prefix[b0 + tid] = base + incl - mine;
        before = all;
        __syncthreads();
    }
    if (tid == 0) a.prefix[a.batch] = before;
    __syncthreads();
    const int64_t total = before;
    if (total == 0) return;
    const int grid = (int)min((int64_t)a.grid, (total + a.min_tiles - 1) / a.min_tiles);
    for (int c = tid; c < grid; c += kPlanThreads) {
        const int64_t at = total * c / grid;
        int lo = 0, hi = a.batch - 1;  // the last sequence that begins at or before `at` and has tiles
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.prefix[mid] <= at) lo = mid;
            else hi = mid - 1;
        }
        const int64_t per_head = (a.prefix[lo + 1] - a.prefix[lo]) / a.heads;
        int64_t rest = at - a.prefix[lo];
        PagedStart st;
        st.b = lo;
        st.h = (int)(rest / per_head);
        rest -= st.h * per_head;
        bool bad;
        const Seq s = load_seq(a, lo, bad);
        for (st.rt = 0;; st.rt++) {
            int t0, n, l, h;
            job_tiles<T, RT>(a, s, st.rt, t0, n, l, h);
            if (rest < n || (st.rt + 1) * RT >= s.rows) break;
            rest -= n;
        }
        st.tile = (int)rest;
        a.start[c] = st;
    }
}

// Block 0 plans the first kernel's share, block 1 (if launched) the other's.
template <int T, int RT, int T2, int RT2>
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PagedArgs a, const int parts, const PagedArgs a2,
                                                                  const int parts2)
{
    pdl_launch();
    if (blockIdx.x == 0) plan_share<T, RT>(a, parts);
    else plan_share<T2, RT2>(a2, parts2);
}

// ------------------------------------------------------------ few rows
// Four warps; a row tile has 16 WM rows.  Warp (wm, wn) multiplies rows
// 16 wm .. with its share of each tile's tokens and keeps its own running
// softmax; the 4 / WM warps of the same rows are joined after the last tile.
template <int D, int WM>
__global__ void __launch_bounds__(kFewThreads) paged_few_kernel(const PagedArgs a)
{
    constexpr int T = kFewT, RT = 16 * WM, WN = 4 / WM, NC = T / WN / 16;  // NC: 16-token chunks per warp and tile
    constexpr int STAGES = few_stages<D>(), CH = D / 8, KS = D / 16;
    constexpr uint32_t TILE = T * D * 2;
    constexpr bool QREG = D <= 128;  // q fragments stay in registers
    extern __shared__ __align__(128) uint8_t sm[];
    uint8_t *sq = sm, *ring = sm + RT * D * 2;
    __shared__ float s_m[4][16], s_l[4][16];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wm = warp / WN, wn = warp % WN;

    pdl_wait();
    SegWalk<T, RT> w;
    if (!w.begin(a)) return;
    do {
        const int r0 = w.rt * RT, nr = min(RT, w.s.rows - r0);
        const int32_t *table = a.table + (int64_t)w.b * a.table_stride;

        // ---- queries (rows past the last are zero)
        for (int e = tid; e < RT * CH; e += kFewThreads) {
            const int r = e / CH, c = e % CH;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r < nr && a.q_mode != 2) {
                const int j = (int)fast_div((uint32_t)(r0 + r), a.group_div), g = r0 + r - j * a.group;
                v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q.p) + (w.s.q0 + j) * a.q.ts +
                                                     (w.h * a.group + g) * a.q.hs + 8 * c);
                if (a.q_mode == 1) {
                    v.x ^= 0x80008000u;
                    v.y ^= 0x80008000u;
                    v.z ^= 0x80008000u;
                    v.w ^= 0x80008000u;
                }
            }
            *reinterpret_cast<uint4 *>(sq + tile_off<D>(r, c)) = v;
        }

        // ---- K and V tiles into the ring: thread (row, chunk); a page's rows
        // lie anywhere, tokens outside the job's range are zeros
        const uint16_t *kb = a.k + w.h * a.head_stride, *vb = a.v + w.h * a.head_stride;
        const int lr = tid / CH, lc = tid % CH;
        constexpr int RSTEP = kFewThreads / CH;
        const int pmask = (1 << a.page_shift) - 1;
        const int ppt = T >> a.page_shift;  // pages per tile (0: a page holds several tiles)
        auto page_of = [&](int tile) -> int {  // lane l: l-th page of the tile
            const int tok = (w.t0 + tile) * T + (lane << a.page_shift);
            if (tile >= w.first + w.count || lane >= (ppt > 0 ? ppt : 1) || tok >= w.hi) return 0;
            if (tok + (1 << a.page_shift) <= w.lo) return 0;  // behind the window: its entry may be stale
            const int p = table[tok >> a.page_shift];
            if ((uint32_t)p >= a.pages && a.status) atomicOr(a.status, kStatusIndex);
            return p;
        };
        int next_page = page_of(w.first);
        auto load = [&](int tile) {
            if (tile < w.first + w.count) {
                const int stage = (tile - w.first) % STAGES;
                const uint32_t dk = smem_u32(ring + stage * 2 * TILE), dv = dk + TILE;
                const int tok0 = (w.t0 + tile) * T;
#pragma unroll
                for (int i = 0; i < T / RSTEP; i++) {
                    const int r = lr + i * RSTEP, tok = tok0 + r;
                    const int page = __shfl_sync(FULL, next_page, r >> a.page_shift);
                    const bool ok = tok >= w.lo && tok < w.hi && (uint32_t)page < a.pages;
                    const int64_t off = ok ? page * a.page_stride + (tok & pmask) * a.slot_stride + 8 * lc : 0;
                    cp16(dk + tile_off<D>(r, lc), kb + off, ok);
                    cp16(dv + tile_off<D>(r, lc), vb + off, ok);
                }
                next_page = page_of(tile + 1);
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < STAGES - 1; i++) load(w.first + i);
        __syncthreads();

        uint32_t qf[QREG ? KS : 1][4];
        const int arow = 16 * wm + (lane & 15), ach = lane >> 4;
        if constexpr (QREG) {
#pragma unroll
            for (int k = 0; k < KS; k++) ldsm4(smem_u32(sq) + tile_off<D>(arow, 2 * k + ach), qf[k]);
        }
        // the tokens each of this thread's two rows sees
        int rlo[2], rhi[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int r = 16 * wm + (lane >> 2) + 8 * i;
            rlo[i] = rhi[i] = 0;
            if (r < nr) {
                const int j = (int)fast_div((uint32_t)(r0 + r), a.group_div);
                seen_range(a, w.s, j, j, rlo[i], rhi[i]);
            }
        }
        float o[D / 8][4], m[2] = { -INFINITY, -INFINITY }, l[2] = { 0.0f, 0.0f };
#pragma unroll
        for (int i = 0; i < D / 8; i++)
#pragma unroll
            for (int k = 0; k < 4; k++) o[i][k] = 0.0f;

        for (int tile = w.first; tile < w.first + w.count; tile++) {
            cp_wait<STAGES - 2>();
            __syncthreads();  // the tile has landed for all; the stage before it is free
            load(tile + STAGES - 1);
            const uint32_t sk = smem_u32(ring + ((tile - w.first) % STAGES) * 2 * TILE), sv = sk + TILE;
            const int tok0 = (w.t0 + tile) * T + wn * (NC * 16);
            float s[NC][2][4];
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int n = 0; n < 2; n++)
#pragma unroll
                    for (int k = 0; k < 4; k++) s[c][n][k] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; k++) {
                uint32_t qk[4];
                if constexpr (!QREG) ldsm4(smem_u32(sq) + tile_off<D>(arow, 2 * k + ach), qk);
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    uint32_t b[4];
                    const int row = wn * (NC * 16) + c * 16 + (lane & 7) + ((lane >> 4) << 3);
                    ldsm4(sk + tile_off<D>(row, 2 * k + ((lane >> 3) & 1)), b);
                    if constexpr (QREG) {
                        mma16816(s[c][0], qf[k], b[0], b[1]);
                        mma16816(s[c][1], qf[k], b[2], b[3]);
                    } else {
                        mma16816(s[c][0], qk, b[0], b[1]);
                        mma16816(s[c][1], qk, b[2], b[3]);
                    }
                }
            }
            // ---- running softmax in powers of two
            float mx[2] = { m[0], m[1] };
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int n = 0; n < 2; n++)
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const int tok = tok0 + c * 16 + n * 8 + (lane & 3) * 2 + (k & 1), i = k >> 1;
                        const float x = s[c][n][k] * a.scale_log2;
                        s[c][n][k] = tok >= rlo[i] && tok < rhi[i] ? x : -INFINITY;
                        mx[i] = fmaxf(mx[i], s[c][n][k]);
                    }
            float base[2];
            bool grow = false;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(FULL, mx[i], 1));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(FULL, mx[i], 2));
                grow |= mx[i] > m[i];
                base[i] = mx[i] == -INFINITY ? 0.0f : mx[i];  // nothing seen yet: every weight is 0
            }
            if (__any_sync(FULL, grow)) {
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const float f = ex2(m[i] - base[i]);
                    l[i] *= f;
                    m[i] = mx[i];
#pragma unroll
                    for (int n = 0; n < D / 8; n++) {
                        o[n][2 * i] *= f;
                        o[n][2 * i + 1] *= f;
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < NC; c++) {
                // weights are rounded to bf16 for the product with V (2^-8 of
                // each, independent); their sum keeps binary32
#pragma unroll
                for (int n = 0; n < 2; n++)
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        s[c][n][k] = ex2(s[c][n][k] - base[k >> 1]);
                        l[k >> 1] += s[c][n][k];
                    }
                const uint32_t p[4] = { pack2(s[c][0][0], s[c][0][1]), pack2(s[c][0][2], s[c][0][3]),
                                        pack2(s[c][1][0], s[c][1][1]), pack2(s[c][1][2], s[c][1][3]) };
                const int row = wn * (NC * 16) + c * 16 + (lane & 15);
#pragma unroll
                for (int n = 0; n < D / 16; n++) {
                    uint32_t b[4];
                    ldsm4t(sv + tile_off<D>(row, 2 * n + (lane >> 4)), b);
                    mma16816(o[2 * n], p, b[0], b[1]);
                    mma16816(o[2 * n + 1], p, b[2], b[3]);
                }
            }
        }
        cp_wait<0>();
        __syncthreads();  // the ring is free: it takes the warps' outputs

        // ---- join the warps of the same rows
        float *so = reinterpret_cast<float *>(ring);  // [WN][RT][D]
#pragma unroll
        for (int i = 0; i < 2; i++) {
            l[i] += __shfl_xor_sync(FULL, l[i], 1);
            l[i] += __shfl_xor_sync(FULL, l[i], 2);
            const int r = (lane >> 2) + 8 * i;
            if ((lane & 3) == 0) {
                s_m[warp][r] = m[i];
                s_l[warp][r] = l[i];
            }
#pragma unroll
            for (int n = 0; n < D / 8; n++)
                *reinterpret_cast<float2 *>(so + ((wn * RT + 16 * wm + r) * D + ((8 * n) ^ ((r & 7) << 3)) + (lane & 3) * 2)) =
                    make_float2(o[n][2 * i], o[n][2 * i + 1]);
        }
        __syncthreads();
        const bool whole = w.whole();
        float *mine = a.part + (int64_t)w.slot() * (RT * (D + 2));
        constexpr int C4 = D / 4;
        for (int e = tid; e < nr * C4; e += kFewThreads) {
            const int r = e / C4, c = e % C4;
            float mt = -INFINITY, lt = 0.0f;
#pragma unroll
            for (int k = 0; k < WN; k++) mt = fmaxf(mt, s_m[(r >> 4) * WN + k][r & 15]);
            const float bs = mt == -INFINITY ? 0.0f : mt;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < WN; k++) {
                const int ww = (r >> 4) * WN + k;
                const float f = ex2(s_m[ww][r & 15] - bs);
                lt += f * s_l[ww][r & 15];
                const float4 v = *reinterpret_cast<const float4 *>(so + (k * RT + r) * D + ((4 * c) ^ ((r & 7) << 3)));
                acc.x += f * v.x;
                acc.y += f * v.y;
                acc.z += f * v.z;
                acc.w += f * v.w;
            }
            if (whole) {
                finish_row(a, w.s.q0, w.h, r0 + r, c, acc, mt, lt);
            } else {
                *reinterpret_cast<float4 *>(mine + 2 * RT + r * D + 4 * c) = acc;
                if (c == 0) {
                    mine[r] = mt;
                    mine[RT + r] = lt;
                }
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            const int c0 = w.owner(), c1 = w.last();
            if (tid == 0) s_last = atomicAdd(a.counter + c0, 1u) == (unsigned)(c1 - c0);
            __syncthreads();
            if (s_last) {
                __threadfence();
                for (int e = tid; e < nr * C4; e += kFewThreads) {
                    const int r = e / C4, c = e % C4;
                    join_parts<RT, D>(a, w.s.q0, w.h, r0 + r, r, c, c0, c1);
                }
            }
        }
        __syncthreads();  // shared memory is free for the next segment
    } while (w.next(a));
}

// ------------------------------------------------------------ join
namespace {

__device__ __forceinline__ void load8(const Rows &r, int64_t tok, int64_t h, int u, bool used, float (&v)[8])
{
    const int64_t off = tok * r.ts + h * r.hs + 8 * u;
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = 0.0f;
    if (!used) return;
    if (r.f32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(r.p) + off);
        const float4 x = p[0], y = p[1];
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(r.p) + off);
        const uint32_t ww[4] = { w.x, w.y, w.z, w.w };
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(ww[i] << 16);
            v[2 * i + 1] = __uint_as_float(ww[i] & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ void store8(const Rows &r, int64_t tok, int64_t h, int u, const float (&v)[8])
{
    const int64_t off = tok * r.ts + h * r.hs + 8 * u;
    if (r.f32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(r.p) + off);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(r.p) + off) =
            make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    }
}

}  // namespace

// out = (wa a + wb b) / (wa + wb), w = exp(lse - max), 8 elements per thread.
// A part that saw nothing (lse -inf) has weight 0 and its row is not used,
// whatever it holds.  HBM-bound: three rows per (token, head).
__global__ void __launch_bounds__(256) merge_kernel(const MergeArgs a)
{
    const int units = a.head_dim / 8;
    const int64_t n = a.tokens * a.heads * units;
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x) {
        const uint32_t row = (uint32_t)(e / units);
        const int u = (int)(e - (int64_t)row * units);
        const uint32_t tok = fast_div(row, a.heads_div), h = row - tok * (uint32_t)a.heads;
        const float la = a.lse_a[row], lb = a.lse_b[row];
        const float top = (la != la || lb != lb) ? la + lb : fmaxf(la, lb);
        const float ea = la == -INFINITY ? 0.0f : expf(la - top), eb = lb == -INFINITY ? 0.0f : expf(lb - top);
        const float sum = ea + eb;
        const float wa = ea == 0.0f ? 0.0f : ea / sum, wb = eb == 0.0f ? 0.0f : eb / sum;
        float x[8], y[8];
        load8(a.a, tok, h, u, la != -INFINITY, x);
        load8(a.b, tok, h, u, lb != -INFINITY, y);
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = wa * x[i] + wb * y[i];
        store8(a.out, tok, h, u, x);
        if (u == 0 && a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : top + logf(sum);
    }
}

// ------------------------------------------------------------ launch
namespace {

template <int D, int WM>
cudaError_t launch_few(const PagedArgs &a, cudaStream_t s)
{
    constexpr int smem = (int)few_smem<D, WM>();
    const cudaError_t e = cudaFuncSetAttribute(paged_few_kernel<D, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(paged_few_kernel<D, WM>, a.grid, kFewThreads, smem, s, a);
}

template <int D>
cudaError_t launch_few_d(const PagedArgs &a, int rows, cudaStream_t s)
{
    switch (rows) {
    case 16: return launch_few<D, 1>(a, s);
    case 32: return launch_few<D, 2>(a, s);
    default: return launch_few<D, 4>(a, s);
    }
}

cudaError_t launch_plan_few(const PagedArgs &a, int rows, cudaStream_t s)
{
    switch (rows) {
    case 16: paged_plan_kernel<kFewT, 16, kFewT, 16><<<1, kPlanThreads, 0, s>>>(a, 1, a, 1); break;
    case 32: paged_plan_kernel<kFewT, 32, kFewT, 32><<<1, kPlanThreads, 0, s>>>(a, 1, a, 1); break;
    default: paged_plan_kernel<kFewT, 64, kFewT, 64><<<1, kPlanThreads, 0, s>>>(a, 1, a, 1); break;
    }
    return cudaGetLastError();
}

// the tcgen05 kernel's share, and beside it the mma.sync kernel's of 16 rows per tile
cudaError_t launch_plan_many(const PagedArgs &many, const PagedArgs &few, int head_dim, bool both, cudaStream_t s)
{
    const int rows = paged_many_rows(head_dim);
    if (rows == 256) paged_plan_kernel<128, 256, kFewT, 16><<<both ? 2 : 1, kPlanThreads, 0, s>>>(many, 2, few, 1);
    else paged_plan_kernel<64, 128, kFewT, 16><<<both ? 2 : 1, kPlanThreads, 0, s>>>(many, 1, few, 1);
    return cudaGetLastError();
}

}  // namespace

// Which kernel takes which sequences.  Up to 64 rows per sequence (new tokens x
// group) the mma.sync kernel keeps pace with HBM: 16, 32 or 64 rows per tile,
// the fewest that hold the longest sequence's rows.  Beyond, the tcgen05
// kernel; in a batch, sequences of at most 16 rows (tokens being decoded
// beside a prompt) still go to the other one.  Blocks: as many as are resident
// at once (shared memory allows 3, 2 and 1 of the mma.sync kernel per SM at
// head_dim 64, 128 and 256, one of the tcgen05 kernel).
PagedPlan paged_plan(int64_t batch, int64_t tokens, int64_t max_q, int64_t max_kv, int heads, int group, int head_dim)
{
    PagedPlan p{};
    const int64_t rows = max_q * group;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    auto place = [&](PagedShare &k, int parts) {
        k.prefix = take(8 * (uint64_t)(batch + 1));
        k.start = take(sizeof(PagedStart) * (uint64_t)k.grid);
        k.counter = take(4 * (uint64_t)k.grid * parts);
        k.part = take(2 * (uint64_t)k.grid * k.rows * (head_dim + 2) * 4);
    };
    const bool many = rows > 64;
    if (!many || batch > 1) {
        p.few.rows = many || rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
        p.few.row_hi = many ? 16 : INT32_MAX;
        p.few.grid = sm_count() * (head_dim == 64 ? 3 : head_dim == 128 ? 2 : 1);
        place(p.few, 1);
    }
    if (many) {
        p.many.rows = paged_many_rows(head_dim);
        p.many.row_lo = batch > 1 ? 16 : 0;
        p.many.row_hi = INT32_MAX;
        p.many.grid = sm_count();
        place(p.many, p.many.rows / 128);
    }
    p.total = at;
    return p;
}

cudaError_t launch_paged(const PagedArgs &args, const PagedPlan &p, int head_dim, void *workspace, cudaStream_t s)
{
    auto share = [&](const PagedShare &k) {
        PagedArgs a = args;
        char *w = static_cast<char *>(workspace);
        a.prefix = reinterpret_cast<int64_t *>(w + k.prefix);
        a.start = reinterpret_cast<PagedStart *>(w + k.start);
        a.counter = reinterpret_cast<uint32_t *>(w + k.counter);
        a.part = reinterpret_cast<float *>(w + k.part);
        a.grid = k.grid;
        a.row_lo = k.row_lo;
        a.row_hi = k.row_hi;
        return a;
    };
    PagedArgs a = share(p.few);
    a.min_tiles = 2;
    cudaError_t e;
    if (p.many.grid) {
        PagedArgs b = share(p.many);
        b.min_tiles = 4;
        e = launch_plan_many(b, a, head_dim, p.few.grid > 0, s);
        if (e == cudaSuccess) e = launch_paged_many(b, head_dim, s);
        if (!p.few.grid) return e;
    } else {
        e = launch_plan_few(a, p.few.rows, s);
    }
    if (e != cudaSuccess) return e;
    switch (head_dim) {
    case 64: return launch_few_d<64>(a, p.few.rows, s);
    case 128: return launch_few_d<128>(a, p.few.rows, s);
    default: return launch_few_d<256>(a, p.few.rows, s);
    }
}

cudaError_t launch_merge(const MergeArgs &args, cudaStream_t s)
{
    MergeArgs a = args;
    a.heads_div = make_fastdiv((uint32_t)a.heads);
    const int64_t n = a.tokens * a.heads * (a.head_dim / 8);
    const int64_t blocks = (n + 255) / 256;
    const int64_t most = (int64_t)sm_count() * 8;
    merge_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace hq
