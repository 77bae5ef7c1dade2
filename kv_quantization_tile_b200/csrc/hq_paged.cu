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
#include "hq_paged_tma.cuh"

namespace hq {

namespace {

constexpr int kFewT = 64;          // tokens per tile
constexpr int kPlanThreads = 1024;
// A job's own cost in tiles (prologue and results), for equal shares
constexpr int kJobCostFew = 2, kJobCostMany = 5;
constexpr int kClusterTiles = 32;  // most tiles a block takes of an uneven batch without a plan

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
template <int THREADS>
__device__ __forceinline__ void named_sync1() { asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory"); }

// Four consumer warps and one that loads; a row tile of 16 WM rows
template <int D, int WM>
struct Few {
    static constexpr int T = kFewT, RT = 16 * WM, ROWS = 128, THREADS = ROWS + 32;
    // stages of K and V tiles: about 64 KB in flight per SM keep HBM busy
    static constexpr int STAGES = D == 64 ? 4 : 3;
    // blocks per SM that shared memory and registers allow
    static constexpr int BLOCKS = D == 64 ? 3 : D == 128 ? 2 : 1;
    static constexpr uint32_t TILE = T * D * 2;
    static constexpr size_t SMEM = 1024 + (D == 256 ? RT * D * 2 : 0) + (size_t)STAGES * 2 * TILE;
};

}  // namespace

// ------------------------------------------------------------ plan
// Units of work (tiles, and each job's own cost) before each sequence, the place where each block's share begins, and
// cleared counters.  One block, a chunk of 1024 sequences at a time: a thread
// counts a sequence's units (a warp, where sequences have many row tiles).
template <int T, int RT>
__device__ __forceinline__ void plan_share(const PagedArgs &a, const int parts)
{
    __shared__ int64_t pre[kPlanThreads];      // units of each sequence of the chunk, then before it
    __shared__ int64_t wsum[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int c = tid; c < a.grid * parts; c += kPlanThreads) a.counter[c] = 0u;
    const bool by_warp = a.max_q * (int64_t)a.group > 8 * RT;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        const int nb = min(kPlanThreads, a.batch - b0);
        auto count = [&](int i, int rt0, int step) -> int64_t {
            bool bad;
            const Seq s = load_seq(a, b0 + i, bad);
            if (bad && rt0 == 0 && a.status) atomicOr(a.status, kStatusIndex);
            int64_t tiles = 0;
            for (int rt = rt0; rt * RT < s.rows; rt += step) {
                int t0, n, lo, hi;
                job_tiles<T, RT>(a, s, rt, t0, n, lo, hi);
                tiles += n + a.job_cost;
            }
            return tiles * a.heads;
        };
        int64_t mine = 0;
        if (by_warp) {
            for (int i = warp; i < nb; i += kPlanThreads / 32) {
                int64_t tiles = count(i, lane, 32);
#pragma unroll
                for (int m = 16; m >= 1; m >>= 1) tiles += __shfl_xor_sync(FULL, tiles, m);
                if (lane == 0) pre[i] = tiles;
            }
            __syncthreads();
            if (tid < nb) mine = pre[tid];
        } else if (tid < nb) {
            mine = count(tid, 0, 1);
        }
        int64_t incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(FULL, incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int64_t sums = wsum[lane];  // every warp scans the warps' sums
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(FULL, sums, d);
            if (lane >= d) sums += o;
        }
        const int64_t base = before + (warp ? __shfl_sync(FULL, sums, warp - 1) : 0);
        pre[tid] = base + incl - mine;
        if (tid < nb) a.prefix[b0 + tid] = pre[tid];
        before += __shfl_sync(FULL, sums, 31);
        __syncthreads();
    }
    const int64_t total = before;
    if (tid == 0) a.prefix[a.batch] = total;
    if (total == 0) return;
    if (a.batch > kPlanThreads) __syncthreads();  // prefix is read back
    const int grid = (int)min((int64_t)a.grid, (total + a.min_units - 1) / a.min_units);
    auto prefix = [&](int b) -> int64_t {
        if (b == a.batch) return total;
        return a.batch <= kPlanThreads ? pre[b] : a.prefix[b];
    };
    for (int c = tid; c < grid; c += kPlanThreads) {
        const int64_t at = total * c / grid;
        int lo = 0, hi = a.batch - 1;  // the last sequence that begins at or before `at` and has units
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix(mid) <= at) lo = mid;
            else hi = mid - 1;
        }
        const int64_t per_head = (prefix(lo + 1) - prefix(lo)) / a.heads;
        int64_t rest = at - prefix(lo);
        PagedStart st;
        st.b = lo;
        st.h = (int)(rest / per_head);
        rest -= st.h * per_head;
        bool bad;
        const Seq s = load_seq(a, lo, bad);
        for (st.rt = 0;; st.rt++) {
            int t0, n, l, h;
            job_tiles<T, RT>(a, s, st.rt, t0, n, l, h);
            if (rest < n + a.job_cost || (st.rt + 1) * RT >= s.rows) break;
            rest -= n + a.job_cost;
        }
        st.job = at - rest;
        st.tile = rest > a.job_cost ? (int)rest - a.job_cost : 0;
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
// Four consumer warps; a row tile has 16 WM rows.  Warp (wm, wn) multiplies rows
// 16 wm .. with its share of each tile's tokens and keeps its own running
// softmax; the 4 / WM warps of the same rows are joined after the last tile.  One
// more warp copies the tiles' pages with TMA into a ring of stages, so the
// consumers meet no one else between tiles: each waits for a stage's bytes and
// reports when it has read them.  (With the tiles copied by the consumers
// themselves, 16 bytes a thread, and a block barrier per tile, a tile took 2500
// clocks, most of them addresses and waiting.)
// CLUSTER: no plan; the blocks of a cluster share one job, and join their
// results through each other's shared memory.
template <int D, int WM, bool CLUSTER>
__global__ void __launch_bounds__(Few<D, WM>::THREADS, Few<D, WM>::BLOCKS)
paged_few_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using F = Few<D, WM>;
    constexpr int T = F::T, RT = F::RT, ROWS = F::ROWS, STAGES = F::STAGES, KS = D / 16;
    constexpr int W = 4, WN = W / WM, NC = T / WN / 16;  // NC: 16-token chunks per warp and tile
    constexpr uint32_t TILE = F::TILE;
    constexpr bool QREG = D <= 128;  // q fragments stay in registers
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t s_bar[2 * STAGES];
    __shared__ float s_m[W][16], s_l[W][16];
    __shared__ float s_fm[CLUSTER ? RT : 1], s_fl[CLUSTER ? RT : 1];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wm = warp / WN, wn = warp % WN;
    uint8_t *ring = raw + (((smem_u32(raw) + 1023u) & ~1023u) - smem_u32(raw)), *sq = ring + STAGES * 2 * TILE;
    const uint32_t bar0 = smem_u32(s_bar), ring0 = smem_u32(ring), sq0 = smem_u32(sq);
    auto full = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty = [&](uint32_t s) { return bar0 + 8u * (STAGES + s); };
    if (tid == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), W);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W && lane == 0) {
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    SegWalk<T, RT> w;
    bool work;
    if constexpr (CLUSTER) {
        work = w.begin_cluster(a);
    } else {
        pdl_wait();
        work = w.begin(a);
    }
    if (!work) return;
    __syncthreads();
    uint32_t stage = 0, phase = 0;
    int left = blockIdx.x == 0 && a.stall_kind == kStallCopy ? a.stall : -1;  // tiles before the withheld one
    bool ok = true;  // a wait that gave up ends the loops; results are invalid then
    auto advance = [&]() {
        if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
        }
    };
    auto land = [&]() {  // (the load warp) no copy is left in flight
        for (uint32_t s = 0; s < STAGES; s++) mbar_wait(full(s), s < stage ? phase : phase ^ 1u);
    };
    do {
        const int r0 = w.rt * RT, nr = min(RT, w.s.rows - r0);
        const int end = w.first + w.count;
        if (warp == W) {
            // -------------------------------------------- loads
            const int page_rows = 1 << a.page_shift, box = page_rows < T ? page_rows : T;
            const int col = lane % (D / 64), pg = lane / (D / 64);
            // this lane's page of a tile (past the pool, where TMA fills zeros,
            // for a number outside it); read a tile ahead of its use
            auto page_of = [&](int tile) -> uint32_t {
                const int tok = (w.t0 + tile) * T + pg * box;
                if (tile >= end || pg * box >= T || tok >= w.hi || tok + box <= w.lo) return 0;
                const uint32_t page = (uint32_t)a.table[(int64_t)w.b * a.table_stride + (tok >> a.page_shift)];
                if (page >= a.pages) {
                    if (a.status) atomicOr(a.status, kStatusIndex);
                    return max(a.pages, 1u);
                }
                return page;
            };
            uint32_t page = page_of(w.first);
            for (int tile = w.first; tile < end && ok; tile++) {
                const uint32_t next = page_of(tile + 1);
                ok = __all_sync(FULL, mbar_wait(empty(stage), phase ^ 1u));
                if (!ok) break;
                const int tok = (w.t0 + tile) * T + pg * box;
                const bool mine = pg * box < T && tok < w.hi && tok + box > w.lo;
                const uint32_t n = __popc(__ballot_sync(FULL, mine));
                if (lane == 0) mbar_expect(full(stage), n * (uint32_t)box * 256u);
                __syncwarp();
                if (mine && left != 0) {
                    const uint32_t dst = ring0 + stage * 2 * TILE + (uint32_t)(col * T * 128 + pg * box * 128);
                    const int at = tok & (page_rows - 1);
                    tma_page(dst, &kmap, full(stage), col * 64, at, w.h, (int)page);
                    tma_page(dst + TILE, &vmap, full(stage), col * 64, at, w.h, (int)page);
                }
                if (left >= 0) left--;
                page = next;
                advance();
            }
            // before another use of the ring, where the consumers may have given up
            if (CLUSTER || !ok) land();
            __syncthreads();  // (A) the ring holds the consumers' outputs until (B)
            if constexpr (!CLUSTER) ok = !__syncthreads_or(!ok);
        } else {
        // ------------------------------------------------ consumers
        // ---- queries (rows past the last are zero): fragments straight into
        // registers, or a tile in shared memory (head_dim 256, whose outputs
        // leave no registers for them)
        const uint32_t flip = a.q_mode == 1 ? 0x80008000u : 0u;
        auto query = [&](int r) -> const uint16_t * {  // row r of the tile, null past the last
            if (r >= nr || a.q_mode == 2) return nullptr;
            const int j = (int)fast_div((uint32_t)(r0 + r), a.group_div), g = r0 + r - j * a.group;
            return static_cast<const uint16_t *>(a.q.p) + (w.s.q0 + j) * a.q.ts + (w.h * a.group + g) * a.q.hs;
        };
        uint32_t qf[QREG ? KS : 1][4];
        const int arow = 16 * wm + (lane & 15), ach = lane >> 4;
        if constexpr (QREG) {
            const uint16_t *q[2] = { query(16 * wm + (lane >> 2)), query(16 * wm + (lane >> 2) + 8) };
#pragma unroll
            for (int k = 0; k < KS; k++)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    qf[k][i] = q[i & 1] ? *reinterpret_cast<const uint32_t *>(q[i & 1] + 16 * k + 8 * (i >> 1) + 2 * (lane & 3)) ^ flip : 0u;
        } else {
            for (int e = tid; e < RT * (D / 8); e += ROWS) {
                const int r = e / (D / 8), c = e % (D / 8);
                const uint16_t *q = query(r);
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (q) {
                    v = *reinterpret_cast<const uint4 *>(q + 8 * c);
                    v = make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
                }
                *reinterpret_cast<uint4 *>(sq + swizzled_off(RT, r, c)) = v;
            }
            named_sync1<ROWS>();
        }
        // the tokens each of this thread's two rows sees, and those all of the
        // warp's rows see
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
        // rows past the last compute what nobody reads
        int all_lo = rlo[0], all_hi = rhi[0];
        {
            const int r = 16 * wm + (lane >> 2);
            if (r >= nr) all_lo = 0, all_hi = INT32_MAX;
            if (r + 8 < nr) {
                all_lo = max(all_lo, rlo[1]);
                all_hi = min(all_hi, rhi[1]);
            }
            all_lo = __reduce_max_sync(FULL, all_lo);
            all_hi = __reduce_min_sync(FULL, all_hi);
        }
        float o[D / 8][4], m[2] = { -INFINITY, -INFINITY }, l[2] = { 0.0f, 0.0f };
#pragma unroll
        for (int i = 0; i < D / 8; i++)
#pragma unroll
            for (int k = 0; k < 4; k++) o[i][k] = 0.0f;

        for (int tile = w.first; tile < end; tile++) {
            ok = __all_sync(FULL, mbar_wait(full(stage), phase));
            if (!ok) break;
            const uint32_t sk = ring0 + stage * 2 * TILE, sv = sk + TILE;
            const int tok0 = (w.t0 + tile) * T + wn * (NC * 16);
            // two chains per chunk of 16 tokens shorten the wait on the sums
            float s[NC][2][2][4];
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int n = 0; n < 2; n++)
#pragma unroll
                    for (int k = 0; k < 4; k++) s[c][n][0][k] = s[c][n][1][k] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; k++) {
                uint32_t qk[4];
                if constexpr (!QREG) ldsm4(sq0 + swizzled_off(RT, arow, 2 * k + ach), qk);
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    uint32_t b[4];
                    const int row = wn * (NC * 16) + c * 16 + (lane & 7) + ((lane >> 4) << 3);
                    ldsm4(sk + swizzled_off(T, row, 2 * k + ((lane >> 3) & 1)), b);
                    mma16816(s[c][0][k & 1], QREG ? qf[QREG ? k : 0] : qk, b[0], b[1]);
                    mma16816(s[c][1][k & 1], QREG ? qf[QREG ? k : 0] : qk, b[2], b[3]);
                }
            }
            // ---- running softmax in powers of two
            const bool edge = tok0 < all_lo || tok0 + NC * 16 > all_hi;
            float mx[2] = { m[0], m[1] };
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int n = 0; n < 2; n++)
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const int i = k >> 1;
                        float x = (s[c][n][0][k] + s[c][n][1][k]) * a.scale_log2;
                        if (edge) {
                            const int tok = tok0 + c * 16 + n * 8 + (lane & 3) * 2 + (k & 1);
                            x = tok >= rlo[i] && tok < rhi[i] ? x : -INFINITY;
                        }
                        s[c][n][0][k] = x;
                        mx[i] = fmaxf(mx[i], x);
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
            if (edge) {
                // rows of V outside the job's tokens meet weight 0, whatever
                // the slots (or the ring, where nothing was copied) hold
                const int from = max(w.lo - tok0, 0), to = w.hi - tok0;
                if (from > 0 || to < NC * 16) {
                    for (int e = lane; e < NC * 16 * (D / 8); e += 32) {
                        const int r = e / (D / 8), c = e % (D / 8);
                        if (r < from || r >= to)
                            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(sv + swizzled_off(T, wn * (NC * 16) + r, c)),
                                         "r"(0u) : "memory");
                    }
                    fence_async_smem();  // before the next copy into this stage
                    __syncwarp();
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
                        s[c][n][0][k] = ex2(s[c][n][0][k] - base[k >> 1]);
                        l[k >> 1] += s[c][n][0][k];
                    }
                const uint32_t p[4] = { pack2(s[c][0][0][0], s[c][0][0][1]), pack2(s[c][0][0][2], s[c][0][0][3]),
                                        pack2(s[c][1][0][0], s[c][1][0][1]), pack2(s[c][1][0][2], s[c][1][0][3]) };
                const int row = wn * (NC * 16) + c * 16 + (lane & 15);
#pragma unroll
                for (int n = 0; n < D / 16; n++) {
                    uint32_t b[4];
                    ldsm4t(sv + swizzled_off(T, row, 2 * n + (lane >> 4)), b);
                    mma16816(o[2 * n], p, b[0], b[1]);
                    mma16816(o[2 * n + 1], p, b[2], b[3]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(stage));
            advance();
        }
        if (!ok && lane == 0 && a.status) atomicOr(a.status, kStatusTimeout);
        __syncthreads();  // (A) every tile is read: the ring takes the warps' outputs

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
        named_sync1<ROWS>();
        const bool whole = CLUSTER || w.whole();
        float *mine = CLUSTER ? nullptr : a.part + (int64_t)w.slot() * (RT * (D + 2));
        constexpr int C4 = D / 4;
        for (int e = tid; e < nr * C4; e += ROWS) {
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
            if (CLUSTER) {  // in place, over the first warp's share
                *reinterpret_cast<float4 *>(so + r * D + ((4 * c) ^ ((r & 7) << 3))) = acc;
                if (c == 0) {
                    s_fm[r] = mt;
                    s_fl[r] = lt;
                }
            } else if (whole) {
                finish_row(a, w.s.q0, w.h, r0 + r, c, acc, mt, lt);
            } else {
                *reinterpret_cast<float4 *>(mine + 2 * RT + r * D + 4 * c) = acc;
                if (c == 0) {
                    mine[r] = mt;
                    mine[RT + r] = lt;
                }
            }
        }
        if constexpr (CLUSTER) {
            const int rank = (int)blockIdx.x % a.split;
            cluster_sync();
            auto load = [&](int k, int r, int c, float &m, float &l, float4 &v) {
                m = cluster_ld(cluster_map(smem_u32(s_fm + r), k));
                l = cluster_ld(cluster_map(smem_u32(s_fl + r), k));
                v = cluster_ld4(cluster_map(smem_u32(so + r * D + ((4 * c) ^ ((r & 7) << 3))), k));
            };
            join_some<D, 1, 8>(a, w.s.q0, w.h, r0, nr, rank * ROWS + tid, a.split * ROWS, 0, a.split - 1, load);
        } else if (!whole) {
            __threadfence();
            named_sync1<ROWS>();
            const int c0 = w.owner(a), c1 = w.last(a);
            if (tid == 0) s_last = atomicAdd(a.counter + c0, 1u) == (unsigned)(c1 - c0);
            named_sync1<ROWS>();
            if (s_last) {
                __threadfence();
                auto load = [&](int k, int r, int c, float &m, float &l, float4 &v) {
                    const float *p = part_of<RT, D>(a, k, c0);
                    m = __ldcg(p + r);
                    l = __ldcg(p + RT + r);
                    v = __ldcg(reinterpret_cast<const float4 *>(p + 2 * RT + r * D + 4 * c));
                };
                if (nr * C4 <= ROWS) join_some<D, 1, 8>(a, w.s.q0, w.h, r0, nr, tid, ROWS, c0, c1, load);
                else join_some<D, 4, 2>(a, w.s.q0, w.h, r0, nr, tid, ROWS, c0, c1, load);
            }
        }
        if constexpr (!CLUSTER) {
            fence_async_smem();
            ok = !__syncthreads_or(!ok);  // (B) the ring is free for the next segment's copies
        }
        }
        if constexpr (CLUSTER) {
            if (warp == W) cluster_sync();
            cluster_sync();  // no block leaves while another reads its shared memory
            return;
        }
    } while (ok && w.next(a));
    if constexpr (!CLUSTER)
        if (warp == W && !ok) land();
}

// ------------------------------------------------------------ join
namespace {

// 8 elements as they lie: 32 bytes of binary32, 16 of bf16
template <bool F32>
struct Raw8 {
    uint32_t w[F32 ? 8 : 4];
};

// The thread's two quads of a row of d elements: adjacent (16-byte accesses of
// bf16), or half a row apart (QUADS), which keeps a warp's binary32 stores
// contiguous.
template <bool F32, bool QUADS>
__device__ __forceinline__ Raw8<F32> load_raw(const Rows &r, int64_t tok, int64_t h, int u, int d)
{
    const int64_t off = tok * r.ts + h * r.hs + (QUADS ? 4 : 8) * u;
    Raw8<F32> x;
    if constexpr (F32) {
        const float *p = static_cast<const float *>(r.p) + off;
        const uint4 a = *reinterpret_cast<const uint4 *>(p), b = *reinterpret_cast<const uint4 *>(p + (QUADS ? d / 2 : 4));
        x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w;
        x.w[4] = b.x, x.w[5] = b.y, x.w[6] = b.z, x.w[7] = b.w;
    } else if constexpr (QUADS) {
        const uint16_t *p = static_cast<const uint16_t *>(r.p) + off;
        const uint2 a = *reinterpret_cast<const uint2 *>(p), b = *reinterpret_cast<const uint2 *>(p + d / 2);
        x.w[0] = a.x, x.w[1] = a.y, x.w[2] = b.x, x.w[3] = b.y;
    } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(r.p) + off);
        x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w;
    }
    return x;
}

template <bool F32>
__device__ __forceinline__ float element(const Raw8<F32> &x, int i)
{
    if constexpr (F32) return __uint_as_float(x.w[i]);
    else return __uint_as_float(i & 1 ? x.w[i / 2] & 0xffff0000u : x.w[i / 2] << 16);
}

template <bool F32>
__device__ __forceinline__ void store8(const Rows &r, int64_t tok, int64_t h, int u, int d, const float (&v)[8])
{
    const int64_t off = tok * r.ts + h * r.hs + (F32 ? 4 : 8) * u;
    if constexpr (F32) {
        float *p = static_cast<float *>(r.p) + off;
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + d / 2) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(r.p) + off) =
            make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    }
}

}  // namespace

// out = (wa a + wb b) / (wa + wb), w = exp(lse - max).  A part that saw nothing
// (lse -inf) has weight 0 and what its row holds is not used.  HBM-bound: three
// rows per (token, head).  A thread takes the same 8 elements of kMergeRows rows
// at once, all loads ahead of the first use (4099 x 32 x 128, two bf16 parts and
// a binary32 result: 25.7 us; four rows 29.3; one row, its loads after its lse,
// 37).
constexpr int kMergeRows = 2;

// A32, B32, O32: binary32 parts and output
template <bool A32, bool B32, bool O32>
__global__ void __launch_bounds__(256) merge_kernel(const MergeArgs a)
{
    const int units = a.head_dim / 8, per = 256 / units;  // units of a row, rows of a block's pass
    const int lr = (int)threadIdx.x / units, u = (int)threadIdx.x - lr * units;
    if (lr >= per) return;
    const int64_t rows = a.tokens * a.heads;
    for (int64_t r0 = (int64_t)blockIdx.x * per * kMergeRows + lr; r0 < rows; r0 += (int64_t)gridDim.x * per * kMergeRows) {
        float la[kMergeRows], lb[kMergeRows];
        Raw8<A32> x[kMergeRows];
        Raw8<B32> y[kMergeRows];
        uint32_t tok[kMergeRows], h[kMergeRows];
#pragma unroll
        for (int i = 0; i < kMergeRows; i++) {
            const int64_t row = r0 + (int64_t)i * per;
            if (row >= rows) break;
            tok[i] = fast_div((uint32_t)row, a.heads_div);
            h[i] = (uint32_t)row - tok[i] * (uint32_t)a.heads;
            la[i] = a.lse_a[row];
            lb[i] = a.lse_b[row];
            x[i] = load_raw<A32, O32>(a.a, tok[i], h[i], u, a.head_dim);
            y[i] = load_raw<B32, O32>(a.b, tok[i], h[i], u, a.head_dim);
        }
#pragma unroll
        for (int i = 0; i < kMergeRows; i++) {
            const int64_t row = r0 + (int64_t)i * per;
            if (row >= rows) break;
            const float top = (la[i] != la[i] || lb[i] != lb[i]) ? la[i] + lb[i] : fmaxf(la[i], lb[i]);
            const float ea = la[i] == -INFINITY ? 0.0f : expf(la[i] - top), eb = lb[i] == -INFINITY ? 0.0f : expf(lb[i] - top);
            const float sum = ea + eb;
            const float wa = ea == 0.0f ? 0.0f : ea / sum, wb = eb == 0.0f ? 0.0f : eb / sum;
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; k++)
                v[k] = wa * (la[i] == -INFINITY ? 0.0f : element(x[i], k)) + wb * (lb[i] == -INFINITY ? 0.0f : element(y[i], k));
            store8<O32>(a.out, tok[i], h[i], u, a.head_dim, v);
            if (u == 0 && a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : top + logf(sum);
        }
    }
}

// ------------------------------------------------------------ launch
namespace {

template <int D, int WM, bool CLUSTER>
cudaError_t launch_few(const PagedArgs &a, cudaStream_t s)
{
    using F = Few<D, WM>;
    CUtensorMap kmap, vmap;
    const int box = (1 << a.page_shift) < F::T ? 1 << a.page_shift : F::T;
    const auto kern = paged_few_kernel<D, WM, CLUSTER>;
    cudaError_t e = page_map(&kmap, a, a.k, D, box);
    if (e == cudaSuccess) e = page_map(&vmap, a, a.v, D, box);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)F::SMEM);
    if (e == cudaSuccess && CLUSTER && a.split > 8)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (CLUSTER) return launch_clusters(kern, a.grid, a.split, F::THREADS, F::SMEM, s, a, kmap, vmap);
    return launch_dependent(kern, a.grid, F::THREADS, F::SMEM, s, a, kmap, vmap);
}

template <int D>
cudaError_t launch_few_d(const PagedArgs &a, int rows, cudaStream_t s)
{
    const bool c = a.split > 0;
    switch (rows) {
    case 16: return c ? launch_few<D, 1, true>(a, s) : launch_few<D, 1, false>(a, s);
    case 32: return c ? launch_few<D, 2, true>(a, s) : launch_few<D, 2, false>(a, s);
    default: return c ? launch_few<D, 4, true>(a, s) : launch_few<D, 4, false>(a, s);
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

// Which kernel takes which sequences, by the rows (new tokens x group) of the
// longest.  The mma.sync kernel: 16, 32 or 64 rows per tile, the fewest that hold
// them, or two tiles of 64.  It takes all calls of up to 64 rows (32 at head_dim
// 256), and of up to 128 where the cache a job reads is short: the tcgen05 kernel
// has the dearer start, the cheaper tile.  Measured (us; 8 KV heads, 8 sequences,
// mma.sync / tcgen05), head_dim 128, 64 rows: 22 / 45 at 1024 tokens, 190 / 201 at
// 16384; 128 rows: 33 / 43, 79 / 80 at 4096, 339 / 199; head_dim 64, 128 rows: 21 /
// 35, 55 / 66, 202 / 176; head_dim 256, 4 KV heads, 4 sequences, 32 rows: 25 / 37,
// 108 / 95; 128 rows: 29 / 36, 59 / 53 at 4096.  In a batch for the tcgen05 kernel,
// sequences of at most 16 rows (tokens being decoded beside a prompt) still go to
// the other one.  Blocks: as many as are resident at once (shared memory allows 3,
// 2 and 1 of the mma.sync kernel per SM at head_dim 64, 128 and 256, one of the
// tcgen05 kernel).
PagedPlan paged_plan(int64_t batch, int64_t tokens, int64_t max_q, int64_t max_kv, int heads, int group, int head_dim,
                     int64_t window)
{
    PagedPlan p{};
    const int64_t rows = max_q * group;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    auto place = [&](PagedShare &k, int parts, int sums) {  // sums: floats of a row of a part beside its output
        k.prefix = take(8 * (uint64_t)(batch + 1));
        k.start = take(sizeof(PagedStart) * (uint64_t)k.grid);
        k.counter = take(4 * (uint64_t)k.grid * parts);
        k.part = take(2 * (uint64_t)k.grid * k.rows * (head_dim + sums) * 4);
    };
    // tokens a job reads (any window up to INT64_MAX; max_q <= 2^30)
    const int64_t reach = window > 0 && window < max_kv - max_q ? window + max_q : max_kv;
    const bool wide = head_dim == 256;
    const bool many = rows > (wide ? 32 : 64) && (rows > 128 || reach > (wide ? 1024 : 4096));
    if (!many || batch > 1) {
        p.few.rows = many || rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
        p.few.row_hi = many ? 16 : INT32_MAX;
        p.few.grid = sm_count() * (head_dim == 64 ? 3 : head_dim == 128 ? 2 : 1);
        // One launch in clusters where the blocks of all jobs fit at once and
        // uneven lengths cannot make one cluster late: a single sequence (its
        // jobs are alike), or few tiles per block.  Clusters of 16 fill a GPC, of
        // which there are eight (half of them, where an SM holds one block): not
        // for more jobs.  Measured, 8 KV heads of 128: one sequence of 4096 / 32768
        // tokens 10.3 / 32.8 us, by shares 16.4 / 47.2; eight of 4096 to 8192
        // tokens 40.6 us, by shares 48.7.
        const int64_t row_tiles = (rows + p.few.rows - 1) / p.few.rows;
        // a window cuts one tile more than its length, but never more than there
        // are: a plan with a window then fits the workspace of one without
        const int64_t all = (max_kv + kFewT - 1) / kFewT, cut = (reach + kFewT - 1) / kFewT + 1;
        const int64_t tiles = cut < all ? cut : all;
        const int64_t jobs = many ? 0 : batch * heads * row_tiles, most = jobs <= (wide ? 4 : 8) ? 16 : 8;
        if (!many && jobs > 0 && jobs <= p.few.grid) {
            int split = 1;
            while (split < most && 2 * split * jobs <= p.few.grid && split < tiles) split *= 2;
            if ((tiles + split - 1) / split <= kClusterTiles || (batch == 1 && jobs <= 16)) {
                p.few.split = split;
                p.few.row_tiles = (int)row_tiles;
                p.few.grid = (int)(jobs * split);
            }
        }
        // by shares: at most 32 parts of a job on average, which one block joins
        if (!many && !p.few.split && 32 * jobs < p.few.grid) p.few.grid = (int)(32 * jobs > 0 ? 32 * jobs : 1);
        if (!p.few.split) place(p.few, 1, 2);
    }
    if (many) {
        p.many.rows = paged_many_rows(head_dim);
        p.many.row_lo = batch > 1 ? 16 : 0;
        p.many.row_hi = INT32_MAX;
        p.many.grid = sm_count();
        place(p.many, p.many.rows / 128, 3);
    }
    p.total = at > 256 ? at : 256;
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
        a.split = k.split;
        a.row_tiles = k.row_tiles;
        return a;
    };
    PagedArgs a = share(p.few);
    a.job_cost = kJobCostFew;
    a.min_units = 2;
    cudaError_t e;
    if (p.many.grid) {
        PagedArgs b = share(p.many);
        b.job_cost = kJobCostMany;
        b.min_units = 3;
        e = launch_plan_many(b, a, head_dim, p.few.grid > 0, s);
        if (e == cudaSuccess) e = launch_paged_many(b, head_dim, s);
        if (!p.few.grid) return e;
    } else {
        e = a.split ? cudaSuccess : launch_plan_few(a, p.few.rows, s);
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
    const int64_t per = 256 / (a.head_dim / 8) * kMergeRows, rows = a.tokens * a.heads;
    const int64_t blocks = (rows + per - 1) / per, most = (int64_t)sm_count() * 8;
    using Kernel = void (*)(const MergeArgs);
    const Kernel kernels[8] = { merge_kernel<false, false, false>, merge_kernel<false, false, true>,
                                merge_kernel<false, true, false>,  merge_kernel<false, true, true>,
                                merge_kernel<true, false, false>,  merge_kernel<true, false, true>,
                                merge_kernel<true, true, false>,   merge_kernel<true, true, true> };
    kernels[4 * a.a.f32 + 2 * a.b.f32 + a.out.f32]<<<(unsigned)(blocks < most ? blocks : most), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace hq
