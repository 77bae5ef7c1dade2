// hq_paged_tc.cu -- attention over a paged KV cache for many new tokens per
// sequence (chunks of a prompt), on the 5th-generation tensor cores (sm_100a).
//
// Rows, jobs, tiles and the blocks' equal shares are those of hq_paged.cu,
// with row tiles of 256 packed rows (two MMA tiles of 128; one of 128 at
// head_dim 256, whose output fills the tensor memory) and token tiles of 128
// (64).  One block per SM, its warps in roles:
//   * the job warp walks the block's share and describes each segment (a job or
//     a part of one) to the others, through a ring in shared memory;
//   * the load warp copies K and V tiles page by page with TMA (128-byte
//     swizzle, one copy per page and 64 columns) into a ring of buffers;
//   * the product warp issues S = Q K^T (both operands in shared memory) and
//     O += P V (P in tensor memory, V as it lies, token-major) with
//     tcgen05.mma; while one MMA tile's softmax runs, the other's products do;
//   * two warpgroups per MMA tile, a thread of each for every row and each
//     with half of the tile's tokens, read S from tensor memory, keep the
//     running softmax and write P over S in bf16.  (With one warpgroup per
//     MMA tile two warps share a scheduler; alone there, a warp keeps the
//     exponential unit two thirds busy, and a tile pair took 3350 clocks.)
// The running maximum is raised, and O rescaled, only where a tile exceeds it
// by more than 24 powers of two: weights then stay below 2^24, sums of 2^30 of
// them times values up to 2^70 inside binary32, every value keeps its relative
// precision, and the final division by the weights' sum cancels the stale
// maximum.  (Rescaling at 8 powers of two, some row of the 256 asked for it in
// a third of the tiles of a cache with uneven channels, at 1900 clocks each.)
//
// Bound: the products are 4 d flops per (row, token), the exponentials one per
// (row, token) on a unit with 16 per clock and SM: at head_dim 128 a tile pair
// takes 2048 clocks of tensor pipe and 2048 of exponentials.  Measured: 3300, as
// a tile's softmax (2000), the rest of its product with V and its next scores
// (768) follow one another; 2048 new tokens over 32768, 32 query heads of 128 in
// 1.1 ms, 970 TFLOP/s, with the clock at 1.47 GHz (power).
#include <atomic>

#include "hq_fast.cuh"
#include "hq_paged_tma.cuh"

namespace hq {

namespace {

constexpr float kGrow = 24.0f;  // powers of two by which a tile may exceed the running maximum

template <int D>
struct Many {
    static constexpr int NT = D == 256 ? 1 : 2;        // MMA tiles of 128 rows
    static constexpr int RT = 128 * NT;
    static constexpr int T = D == 256 ? 64 : 128;      // tokens per tile
    static constexpr int THREADS = 256 * NT + 96;
    static constexpr uint32_t TILE = T * D * 2;        // one K or V tile
    static constexpr uint32_t QTILE = 128 * D * 2;
    static constexpr int STAGES = D == 64 ? 8 : 5;
    static constexpr size_t SMEM = 1024 + NT * QTILE + STAGES * TILE;
    // tensor memory: O of each MMA tile, then two score buffers
    static constexpr uint32_t O_COL = 0, S_COL = 256;
};

// A segment of the block's share, as the job warp describes it.
struct Segment {
    int valid;            // 0: the share has ended
    int b, h, q0, rows;   // sequence, KV head, first query row, rows of the sequence
    int r0;               // first packed row of the row tile
    int nq, kv;           // new and cached tokens
    int tile, count;      // first tile (of T tokens), tiles
    int lo, hi;           // cached tokens that any row of the job sees
    int whole;            // the job is not cut
    int slot, c0, c1;     // if it is: this part's slot, the blocks of the first and the last part
};
constexpr int kSegments = 4;

// Shared-memory descriptor of a 128-byte-swizzled operand: 8-row groups of 128
// bytes `sbo` apart; `lbo` is the distance between blocks of 64 elements along
// the contiguous axis when that axis is not K.
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return make_smem_desc(addr, lbo, sbo) | ((uint64_t)2 << 61);
}

// O += P V with P (bf16) in tensor memory
__device__ __forceinline__ void umma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
        :
        : "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// true in one lane of the (converged) warp, the same one every time
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(one));
    return one;
}

// 32 consecutive columns of this thread's tensor-memory lane
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
        "%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
        "%30,%31};"
        :
        : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
          "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
          "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        :
        : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Weights of 32 columns of scores: 2^(s scale - off), packed to bf16 pairs,
// their binary32 sum added to `sum`.
__device__ __forceinline__ void weights32(const uint32_t (&s)[32], float scale, float off, float2 (&sum)[2], uint32_t (&p)[16])
{
    const float2 sc = splat2(scale), no = splat2(-off);
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const float2 x = fma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sc, no);
        const float2 y = make_float2(ex2(x.x), ex2(x.y));
        sum[i & 1] = add2(sum[i & 1], y);
        p[i] = pack2(y.x, y.y);
    }
}

__device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// the same, and whether `v` holds for any of the threads
__device__ __forceinline__ bool named_any(int id, int threads, bool v)
{
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %3, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(any)
        : "r"(id), "r"(threads), "r"((uint32_t)v)
        : "memory");
    return any;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(Many<D>::THREADS, 1)
paged_many_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using C = Many<D>;
    constexpr int NT = C::NT, RT = C::RT, T = C::T, STAGES = C::STAGES;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t s_bar[2 * STAGES + NT * 2 + 6 + 2 + 2 * kSegments];
    __shared__ Segment s_seg[kSegments];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_fail;
    __shared__ int s_last[NT];
    __shared__ float s_row[NT][128];  // a value of each row, from one half to the other
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = warp >> 2;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t sq = base, ring = base + NT * C::QTILE;
    const uint32_t bar0 = smem_u32(s_bar);
    auto kv_full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
    auto kv_empty = [&](int s) { return bar0 + 8u * (uint32_t)(STAGES + s); };
    auto q_full = [&](int t) { return bar0 + 8u * (uint32_t)(2 * STAGES + t); };
    auto o_full = [&](int t) { return bar0 + 8u * (uint32_t)(2 * STAGES + NT + t); };
    auto s_full = [&](int b) { return bar0 + 8u * (uint32_t)(2 * STAGES + 2 * NT + b); };
    auto p_full = [&](int b) { return bar0 + 8u * (uint32_t)(2 * STAGES + 2 * NT + 2 + b); };
    auto p_half = [&](int b) { return bar0 + 8u * (uint32_t)(2 * STAGES + 2 * NT + 4 + b); };  // the first 32 weights of either half
    const uint32_t fix_bar = bar0 + 8u * (uint32_t)(2 * STAGES + 2 * NT + 6);
    const uint32_t done_bar = fix_bar + 8u;  // the block's last product
    auto seg_full = [&](uint32_t k) { return fix_bar + 8u * (2 + k); };
    auto seg_empty = [&](uint32_t k) { return fix_bar + 8u * (2 + kSegments + k); };

    if (warp == 0) tmem_alloc(smem_u32(&s_tmem), 512);
    if (tid == 0) {
        s_fail = 0;
        for (int s = 0; s < STAGES; s++) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int t = 0; t < NT; t++) {
            mbar_init(q_full(t), 8);
            mbar_init(o_full(t), 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(s_full(b), 1);
            mbar_init(p_full(b), 8);
            mbar_init(p_half(b), 8);
        }
        mbar_init(fix_bar, 1);
        mbar_init(done_bar, 1);
        for (int k = 0; k < kSegments; k++) {
            mbar_init(seg_full(k), 1);
            mbar_init(seg_empty(k), 8 * NT + 2);  // the softmax warps, products, loads
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // a wait that gave up: every role leaves its loops at its next check
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        if (mbar_wait(bar, parity)) return true;
        s_fail = 1;
        return false;
    };
    // the same for a warp that walks as one: its lanes go on together or not at
    // all (the clocks by which a wait gives up are read lane by lane)
    auto wait_as_one = [&](uint32_t bar, uint32_t parity) -> bool { return __all_sync(FULL, wait(bar, parity)); };

    if (warp == 2 && lane == 0) {
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    pdl_wait();
    // segment i (whether there is one; `ok` turns false if the wait gave up),
    // and this warp's leave of it
    auto segment = [&](uint32_t i, bool &ok) -> bool {
        if (!wait_as_one(seg_full(i % kSegments), (i / kSegments) & 1u)) ok = false;
        return ok && s_seg[i % kSegments].valid;
    };
    auto leave = [&](uint32_t i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty(i % kSegments));
    };

    if (wg < 2 * NT) {
        // ------------------------------------------------ softmax
        const int t = wg >> 1, hf = wg & 1, wl = warp & 3;  // MMA tile, half of the tokens, 32 rows
        const uint32_t lanes = (uint32_t)(wl * 32) << 16;
        const uint32_t to = tmem + lanes + C::O_COL + (uint32_t)(t * D + hf * (D / 2));  // this half's columns of O
        const int pair = 1 + t * 4 + wl;  // barrier of the two warps of the same rows
        uint32_t g = 0;  // tiles so far
        // This warp's half of 32 query rows of a segment, copied on the side (zeros
        // past the last row), then handed over.
        constexpr int CH = D / 16;  // chunks per half row, copies per lane
        auto copy_queries = [&](const Segment &x) {
#pragma unroll 1
            for (int e = lane; e < 32 * CH; e += 32) {
                const int rr = wl * 32 + e / CH, c = hf * CH + e % CH, r = x.r0 + t * 128 + rr;
                const bool valid = r < x.rows && a.q_mode != 2;
                const int j = (int)fast_div((uint32_t)r, a.group_div), gg = r - j * a.group;
                const uint16_t *q = static_cast<const uint16_t *>(a.q.p);
                if (valid) q += (x.q0 + j) * a.q.ts + (x.h * a.group + gg) * a.q.hs + 8 * c;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sq + t * C::QTILE + swizzled_off(128, rr, c)),
                             "l"(q), "r"(valid ? 16 : 0) : "memory");
            }
        };
        auto hand_queries = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (a.q_mode == 1)  // a negative scale: -q
                for (int e = lane; e < 32 * CH; e += 32) {
                    const uint32_t at = sq + t * C::QTILE + swizzled_off(128, wl * 32 + e / CH, hf * CH + e % CH);
                    uint32_t v[4];
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0] ^ 0x80008000u), "r"(v[1] ^ 0x80008000u),
                                 "r"(v[2] ^ 0x80008000u), "r"(v[3] ^ 0x80008000u) : "memory");
                }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full(t));
        };
        uint32_t i = 0;
        bool ok = true, more = segment(0, ok);
        if (named_any(9 + t, 256, !ok)) more = false;  // the MMA tile's warps go on together or not at all
        if (more) {
            copy_queries(s_seg[0]);
            hand_queries();
        }
        for (; more; i++) {
            const Segment &x = s_seg[i % kSegments];
            const int r = x.r0 + t * 128 + wl * 32 + lane, rows = x.rows, count = x.count;
            int rlo = 0, rhi = 0;
            if (r < rows) {
                const int j = (int)fast_div((uint32_t)r, a.group_div);
                const Seq s{ x.q0, x.nq, x.kv, rows };
                seen_range(a, s, j, j, rlo, rhi);
            }
            float m = -INFINITY, l = 0.0f;
            float near = 0.0f;  // what rounding added to the greatest weight of each tile (of this half)
            for (int n = 0; n < count; n++, g++) {
                const int b = NT == 2 ? t : (int)(g & 1u);
                const uint32_t par = NT == 2 ? g & 1u : (g >> 1) & 1u;
                const uint32_t ts = tmem + lanes + C::S_COL + (uint32_t)(b * T);
                constexpr int NC = T / 64;  // chunks of 32 columns of this half
                ok = wait(s_full(b), par) && ok;  // (a wait for O that gave up in the tile before counts)
                // Every product with V is waited for in turn (a barrier's phase can
                // only be told from the one before it).  With two MMA tiles S comes
                // after that product anyway; with one, S runs ahead of it.
                if (NT == 1 && n > 0) ok = wait(o_full(t), (g - 1u) & 1u) && ok;
                ok = __all_sync(FULL, ok);
                tc_fence_after();
                // the last scores are there, so the queries are free: the next
                // segment's take their place
                if (n + 1 == count) {
                    more = segment(i + 1, ok);
                    if (more && ok) copy_queries(s_seg[(i + 1) % kSegments]);
                }
                const uint32_t mine = ts + (uint32_t)(hf * (T / 2));  // this half's scores, then its weights
                const int tok0 = (x.tile + n) * T + hf * (T / 2);
                const bool edge = !__all_sync(FULL, rlo <= tok0 && rhi >= tok0 + T / 2);
                auto mask = [&](int c, uint32_t (&s)[32]) {
                    const int from = rlo - tok0 - 32 * c, to_ = rhi - tok0 - 32 * c;
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        if (i < from || i >= to_) s[i] = 0xff800000u;
                };
                // Weights are rounded to bf16 for the product with V (2^-8 of
                // each, independent); their sum keeps binary32.  The sum that
                // divides the product takes a tile's greatest weight as rounded:
                // where one token dominates a row, both then err alike and cancel
                // (against an exact maximum its weight would be 1, but the maximum
                // may be stale).  Measured against binary64 on prompts of peaked
                // rows: 0.0023 -> 0.0020 of the output (0.0017 is its own rounding),
                // for 1 % of time; with every weight as rounded, the same for 6 %.
                float2 sum[2] = { make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f) };
                uint32_t s[32], p[16];
                auto weights = [&]() {
                    const float off = m == -INFINITY ? 0.0f : m;  // nothing seen yet: every weight is 0
                    weights32(s, a.scale_log2, off, sum, p);
                };
                auto hand_over = [&](int c, uint32_t bar) {  // over scores already read
                    tmem_st16(mine + (uint32_t)(16 * c), p);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar);
                };
                // the maximum of the half's scores (its second 32 columns are
                // read again below, which keeps a thread within 96 registers)
                float mx[4] = { -INFINITY, -INFINITY, -INFINITY, -INFINITY };
                auto maxima = [&](const uint32_t (&x)[32]) {
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                };
                tmem_ld32(mine, s);
                if constexpr (NC == 2) {
                    uint32_t s1[32];
                    tmem_ld32(mine + 32, s1);
                    tmem_wait_ld();
                    if (edge) mask(1, s1);
                    maxima(s1);
                } else {
                    tmem_wait_ld();
                }
                if (edge) mask(0, s);
                maxima(s);
                const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                float top = most * a.scale_log2;
                // The first weights are taken against the running maximum as it
                // stands, while the other warp gets here, and again in the rare
                // tile that raises it.
                weights();
                if (NC == 2) tmem_ld32(mine + 32, s);
                if (named_any(pair, 64, n == 0 || top > m + kGrow || !ok)) {
                    float *row = &s_row[t][wl * 32 + lane];
                    if (hf) *row = top;
                    if (named_any(pair, 64, !ok)) {  // a wait gave up: both warps leave
                        ok = false;
                        tmem_wait_ld();
                        break;
                    }
                    if (!hf) *row = top = fmaxf(top, *row);
                    named_sync(pair, 64);
                    top = *row;
                    const bool grow = n == 0 || top > m + kGrow;
                    const float f = grow && n > 0 ? ex2(m - top) : 1.0f;
                    if (grow) m = top;
                    l *= f;
                    near *= f;
                    if (n > 0) {  // rescale O: the product before this one is complete
                        ok = wait(o_full(t), (g - 1u) & 1u);  // (a failure is met at the next tile's vote)
                        ok = __all_sync(FULL, ok);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 64; c++) {
                            uint32_t o[32];
                            tmem_ld32(to + 32 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(to + 32 * c, o);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                    named_sync(pair, 64);  // both halves of O are rescaled before either hands P over
                    tc_fence_after();
                    tmem_ld32(mine, s);
                    tmem_wait_ld();
                    if (edge) mask(0, s);
                    sum[0] = sum[1] = make_float2(0.0f, 0.0f);
                    weights();
                    if (NC == 2) tmem_ld32(mine + 32, s);
                }
                if constexpr (NC == 2) {
                    tmem_wait_ld();
                    hand_over(0, p_half(b));
                    if (edge) mask(1, s);
                    weights();
                    hand_over(1, p_full(b));
                } else {
                    hand_over(0, p_full(b));
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                const float w = ex2(fmaf(most, a.scale_log2, m == -INFINITY ? 0.0f : -m));
                near += __bfloat162float(__float2bfloat16_rn(w)) - w;
            }
            // ---- the segment's end (the MMA tile's warps leave together)
            ok = ok && wait(o_full(t), (g - 1u) & 1u);
            if (named_any(9 + t, 256, !ok)) break;
            tc_fence_after();
            const bool whole = x.whole;
            if (more) hand_queries();  // its first scores come while O is written out
            const int rr = wl * 32 + lane;  // row of this MMA tile
            auto both = [&](float v) -> float {  // of the two halves
                if (hf) s_row[t][rr] = v;
                named_sync(pair, 64);
                if (!hf) s_row[t][rr] = v += s_row[t][rr];
                named_sync(pair, 64);
                return s_row[t][rr];
            };
            l = both(l);
            named_sync(pair, 64);
            const float ld = l + both(near);
            // partial results by MMA tile: m, l and ld of its rows, then [D / 4][128] float4
            float *part = a.part + ((int64_t)x.slot * NT + t) * (128 * (D + 3));
            if (!whole && hf == 0) {
                part[rr] = m;
                part[128 + rr] = l;
                part[256 + rr] = ld;
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / ld;
            int64_t tok = 0;
            int head = 0;
            if (r < rows) {
                const int j = (int)fast_div((uint32_t)r, a.group_div);
                tok = x.q0 + j;
                head = x.h * a.group + r - j * a.group;
            }
            const int64_t at = tok * a.out.ts + head * a.out.hs + hf * (D / 2);
            auto put = [&](int c, const float (&v)[32], float f, bool zero) {  // 32 of this half's columns of the row
                if (r >= rows) return;
                if (a.out.f32) {
                    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(a.out.p) + at + 32 * c);
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        p[i] = zero ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                    : make_float4(v[4 * i] * f, v[4 * i + 1] * f, v[4 * i + 2] * f, v[4 * i + 3] * f);
                } else {
                    uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out.p) + at + 32 * c);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        p[i] = zero ? make_uint4(0u, 0u, 0u, 0u)
                                    : make_uint4(pack2(v[8 * i] * f, v[8 * i + 1] * f), pack2(v[8 * i + 2] * f, v[8 * i + 3] * f),
                                                 pack2(v[8 * i + 4] * f, v[8 * i + 5] * f), pack2(v[8 * i + 6] * f, v[8 * i + 7] * f));
                }
            };
#pragma unroll 1
            for (int c = 0; c < D / 64; c++) {
                uint32_t o[32];
                tmem_ld32(to + 32 * c, o);
                tmem_wait_ld();
                if (whole) {
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; i++) v[i] = __uint_as_float(o[i]);
                    put(c, v, inv, l == 0.0f);
                } else {
                    float4 *p = reinterpret_cast<float4 *>(part + 384) + (hf * (D / 8) + 8 * c) * 128 + rr;
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        p[i * 128] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                 __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                }
            }
            tc_fence_before();
            float mt = m, lt = l;
            bool write = whole;
            if (!whole) {
                __threadfence();
                const int c0 = x.c0, c1 = x.c1;
                named_sync(9 + t, 256);
                if (hf == 0 && rr == 0) s_last[t] = atomicAdd(a.counter + c0 * NT + t, 1u) == (unsigned)(c1 - c0);
                named_sync(9 + t, 256);
                write = s_last[t];
                if (write) {
                    __threadfence();
                    auto part_at = [&](int k) {
                        return a.part + ((int64_t)(2 * k + (k == c0 ? 1 : 0)) * NT + t) * (128 * (D + 3));
                    };
                    // the parts' factors, those of the first four kept
                    float f4[4];
                    mt = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        f4[k] = c0 + k <= c1 ? __ldcg(part_at(c0 + k) + rr) : -INFINITY;
                        mt = fmaxf(mt, f4[k]);
                    }
                    for (int k = c0 + 4; k <= c1; k++) mt = fmaxf(mt, __ldcg(part_at(k) + rr));
                    const float from = mt == -INFINITY ? 0.0f : mt;
                    lt = 0.0f;
                    float ldt = 0.0f;
                    auto sums = [&](int k, float e) {
                        lt = fmaf(e, __ldcg(part_at(k) + 128 + rr), lt);
                        ldt = fmaf(e, __ldcg(part_at(k) + 256 + rr), ldt);
                    };
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        f4[k] = ex2(f4[k] - from);
                        if (c0 + k <= c1) sums(c0 + k, f4[k]);
                    }
                    for (int k = c0 + 4; k <= c1; k++) sums(k, ex2(__ldcg(part_at(k) + rr) - from));
                    const float f = lt == 0.0f ? 0.0f : 1.0f / ldt;
#pragma unroll 1
                    for (int c = 0; c < D / 64; c++) {
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; i++) v[i] = 0.0f;
                        auto add = [&](int k, float e) {
                            const float4 *p = reinterpret_cast<const float4 *>(part_at(k) + 384) + (hf * (D / 8) + 8 * c) * 128 + rr;
#pragma unroll
                            for (int i = 0; i < 8; i++) {
                                const float4 x = __ldcg(p + i * 128);
                                v[4 * i] = fmaf(e, x.x, v[4 * i]);
                                v[4 * i + 1] = fmaf(e, x.y, v[4 * i + 1]);
                                v[4 * i + 2] = fmaf(e, x.z, v[4 * i + 2]);
                                v[4 * i + 3] = fmaf(e, x.w, v[4 * i + 3]);
                            }
                        };
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            if (c0 + k <= c1) add(c0 + k, f4[k]);
#pragma unroll 1
                        for (int k = c0 + 4; k <= c1; k++) add(k, ex2(__ldcg(part_at(k) + rr) - from));
                        put(c, v, f, lt == 0.0f);
                    }
                }
            }
            if (write && hf == 0 && a.lse && r < rows)
                a.lse[tok * (a.heads * a.group) + head] = lt == 0.0f ? -INFINITY : fmaf(mt, 0.693147180559945309f, logf(lt));
            leave(i);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");  // queries copied ahead for a segment that was given up
    } else {
        if ((warp & 3) == 0) {
            // -------------------------------------------- products
            // The warp walks as one, so addresses stay in uniform registers;
            // one elected lane issues (always the same one: a commit covers
            // the products of its own thread).
            bool ok = true;
            if (segment(0, ok)) {
                constexpr uint32_t ID_S = make_idesc_bf16(128, T);
                constexpr uint32_t ID_O = make_idesc_bf16(128, D) | (1u << 16);  // V is token-major: B not K-major
                const bool one = elect_one();
                const uint64_t qd = swizzled_desc(sq, 16, 1024), kd = swizzled_desc(ring, 16, 1024),
                               vd = swizzled_desc(ring, T * 128, 1024);
                uint32_t slot = 0, phase = 0, g = 0, seg = 0;
                auto take = [&]() -> uint32_t {  // the next tile of the ring, landed
                    ok = ok && wait_as_one(kv_full(slot), phase);
                    const uint32_t s = slot;
                    if (++slot == STAGES) {
                        slot = 0;
                        phase ^= 1u;
                    }
                    return s;
                };
                auto commit = [&](uint32_t bar) {
                    if (one) umma_commit(bar);
                };
                auto scores = [&](int t, int b, uint32_t s) {
                    const uint64_t q = qd + (uint32_t)t * (C::QTILE >> 4), k = kd + s * (C::TILE >> 4);
                    const uint32_t d = tmem + C::S_COL + (uint32_t)(b * T);
                    if (one) {
#pragma unroll
                        for (int i = 0; i < D / 16; i++)
                            umma_bf16(d, q + (i >> 2) * 1024 + (i & 3) * 2, k + (i >> 2) * (T * 8) + (i & 3) * 2, ID_S, i > 0);
                        umma_commit(s_full(b));
                    }
                };
                // 16-token steps i0, i0 + 1, .. i1 - 1 of either half of the tile; 16
                // weights fill 8 columns, a half's begin where its scores did
                auto outputs = [&](int t, int b, uint32_t s, int i0, int i1, bool add, bool last) {
                    const uint32_t p = tmem + C::S_COL + (uint32_t)(b * T), d = tmem + C::O_COL + (uint32_t)(t * D);
                    const uint64_t v = vd + s * (C::TILE >> 4);
                    if (one) {
#pragma unroll
                        for (int h = 0; h < 2; h++)
#pragma unroll
                            for (int i = i0; i < i1; i++)
                                umma_bf16_ts(d, p + h * (T / 2) + 8 * i, v + (h * (T / 32) + i) * 128, ID_O, add || h + i > 0);
                        if (last && !(blockIdx.x == 0 && a.stall_kind == kStallProduct && (int)g >= a.stall)) umma_commit(o_full(t));
                    }
                };
                do {
                    const uint32_t k0 = take();
                    for (int t = 0; t < NT && ok; t++) {
                        ok = wait_as_one(q_full(t), seg & 1u);
                        if (!ok) break;
                        tc_fence_after();
                        scores(t, NT == 2 ? t : (int)(g & 1u), k0);
                    }
                    if (!ok) break;
                    commit(kv_empty(k0));
                    const int count = s_seg[seg % kSegments].count;
                    leave(seg);
                    for (int j = 0; j < count && ok; j++, g++) {
                        const bool more = j + 1 < count;
                        const uint32_t k = more ? take() : 0u;
                        if (NT == 1 && more && ok) {
                            scores(0, (int)((g + 1) & 1u), k);
                            commit(kv_empty(k));
                        }
                        const uint32_t v = take();
#pragma unroll
                        for (int t = 0; t < NT; t++) {
                            if (!ok) break;
                            const int b = NT == 2 ? t : (int)(g & 1u);
                            const uint32_t par = NT == 2 ? g & 1u : (g >> 1) & 1u;
                            if (T == 128) {  // the first 32 weights of either half
                                ok = wait_as_one(p_half(b), par);
                                if (!ok) break;
                                tc_fence_after();
                                outputs(t, b, v, 0, 2, j > 0, false);
                            }
                            ok = wait_as_one(p_full(b), par);
                            if (!ok) break;
                            tc_fence_after();
                            if (T == 128) outputs(t, b, v, 2, 4, true, true);
                            else outputs(t, b, v, 0, 2, j > 0, true);
                            if (NT == 2 && more) scores(t, t, k);
                        }
                        if (!ok) break;
                        commit(kv_empty(v));
                        if (NT == 2 && more) commit(kv_empty(k));
                    }
                    seg++;
                } while (ok && segment(seg, ok));
                // no product is left running, whoever gave up
                commit(done_bar);
                wait_as_one(done_bar, 0);
            }
        } else if ((warp & 3) == 1) {
            // -------------------------------------------- loads
            const int page_rows = 1 << a.page_shift, box = page_rows < T ? page_rows : T;
            const int col = lane % (D / 64), pg = lane / (D / 64);
            uint32_t slot = 0, phase = 0, fixes = 0;
            int left = blockIdx.x == 0 && a.stall_kind == kStallCopy ? a.stall : -1;  // copies before the withheld one
            bool ok = true;
            // this lane's page of a tile (past the pool, where TMA fills zeros,
            // for a number outside it); read a tile ahead of its use
            Segment x{};
            auto page_of = [&](int n) -> uint32_t {
                const int tok = (x.tile + n) * T + pg * box;
                if (n >= x.count || pg * box >= T || tok >= x.hi || tok + box <= x.lo) return 0;
                const uint32_t page = (uint32_t)a.table[(int64_t)x.b * a.table_stride + (tok >> a.page_shift)];
                if (page >= a.pages) {
                    if (a.status) atomicOr(a.status, kStatusIndex);
                    return max(a.pages, 1u);
                }
                return page;
            };
            auto load = [&](int n, bool is_v, uint32_t page) {
                ok = ok && wait_as_one(kv_empty(slot), phase ^ 1u);
                if (!ok) return;
                const int tok0 = (x.tile + n) * T, tok = tok0 + pg * box;
                const uint32_t dst = ring + slot * C::TILE;
                // rows of V outside the job's tokens meet weight 0: they must be finite
                const bool fix = is_v && (tok0 < x.lo || tok0 + T > x.hi);
                const uint32_t bar = fix ? fix_bar : kv_full((int)slot);
                const bool mine = pg * box < T && tok < x.hi && tok + box > x.lo;
                const uint32_t boxes = __popc(__ballot_sync(FULL, mine));
                if (lane == 0) mbar_expect(bar, boxes * (uint32_t)box * 128u);
                __syncwarp();
                if (mine && left != 0)
                    tma_page(dst + (uint32_t)(col * T * 128 + pg * box * 128), is_v ? &vmap : &kmap, bar, col * 64,
                             tok & (page_rows - 1), x.h, (int)page);
                if (left >= 0) left--;
                if (fix) {
                    ok = wait_as_one(fix_bar, fixes & 1u);
                    fixes++;
                    if (!ok) return;
                    for (int e = lane; e < T * (D / 8); e += 32) {
                        const int r = e / (D / 8), c = e % (D / 8);
                        if (tok0 + r < x.lo || tok0 + r >= x.hi)
                            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(dst + swizzled_off(T, r, c)), "r"(0u) : "memory");
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(kv_full((int)slot));
                }
                if (++slot == STAGES) {
                    slot = 0;
                    phase ^= 1u;
                }
            };
            for (uint32_t i = 0; ok && segment(i, ok); i++) {
                x = s_seg[i % kSegments];
                leave(i);
                uint32_t here = page_of(0), next = page_of(1);
                load(0, false, here);
                for (int n = 0; n < x.count && ok; n++) {
                    const uint32_t after = page_of(n + 2);
                    if (n + 1 < x.count) load(n + 1, false, next);
                    load(n, true, here);
                    here = next;
                    next = after;
                }
            }
            // no copy is left in flight, whoever gave up
            for (int s = 0; s < STAGES; s++) mbar_wait(kv_full(s), s < (int)slot ? phase : phase ^ 1u);
            if (!ok && fixes) mbar_wait(fix_bar, (fixes - 1u) & 1u);
        } else {
            // -------------------------------------------- jobs
            SegWalk<T, RT> w;
            bool go = w.begin(a);
            int64_t tiles = 0;  // of the segments so far
            // The place of the segment four back: that one may last longer than any
            // one wait, so this one gives up where another role has (each waits for
            // a tile at most), and after as many limits as there were tiles.
            auto place = [&](uint32_t i) -> bool {
                for (int64_t left = tiles;; left--) {
                    if (__all_sync(FULL, mbar_wait(seg_empty(i % kSegments), ((i / kSegments) & 1u) ^ 1u))) return true;
                    if (left <= 0 || __any_sync(FULL, s_fail)) break;
                }
                s_fail = 1;
                return false;
            };
            for (uint32_t i = 0; place(i); i++) {
                if (lane == 0) {
                    Segment x{};
                    x.valid = go;
                    if (go) {
                        x.b = w.b;
                        x.h = w.h;
                        x.q0 = w.s.q0;
                        x.rows = w.s.rows;
                        x.r0 = w.rt * RT;
                        x.nq = w.s.nq;
                        x.kv = w.s.kv;
                        x.tile = w.t0 + w.first;
                        x.count = w.count;
                        x.lo = w.lo;
                        x.hi = w.hi;
                        x.whole = w.whole();
                        if (!x.whole) {
                            x.slot = w.slot();
                            x.c0 = w.owner(a);
                            x.c1 = w.last(a);
                        }
                    }
                    s_seg[i % kSegments] = x;
                    mbar_arrive(seg_full(i % kSegments));
                }
                __syncwarp();
                if (!go) break;
                tiles += w.count;
                go = w.next(a);
            }
        }
    }
    __syncthreads();
    if (tid == 0 && s_fail && a.status) atomicOr(a.status, kStatusTimeout);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------ launch
namespace {

// cuTensorMapEncodeTiled of the driver (looked up once; the library does not
// link against it)
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static std::atomic<EncodeTiled> cached{ nullptr };
    EncodeTiled f = cached.load(std::memory_order_acquire);
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            return nullptr;
        f = reinterpret_cast<EncodeTiled>(p);
        cached.store(f, std::memory_order_release);
    }
    return f;
}

}  // namespace

cudaError_t page_map(CUtensorMap *m, const PagedArgs &a, const void *pool, int d, int box)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = { (cuuint64_t)d, (cuuint64_t)1 << a.page_shift, (cuuint64_t)a.heads, a.pages ? a.pages : 1u };
    const cuuint64_t strides[3] = { 2ull * a.slot_stride, 2ull * (a.heads > 1 ? a.head_stride : d),
                                    2ull * (a.pages > 1 ? a.page_stride : d) };
    const cuuint32_t boxes[4] = { 64, (cuuint32_t)box, 1, 1 }, steps[4] = { 1, 1, 1, 1 };
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(pool), dims, strides, boxes, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {

template <int D>
cudaError_t launch_many_d(const PagedArgs &a, cudaStream_t s)
{
    using C = Many<D>;
    CUtensorMap kmap, vmap;
    const int box = (1 << a.page_shift) < C::T ? 1 << a.page_shift : C::T;
    cudaError_t e = page_map(&kmap, a, a.k, D, box);
    if (e == cudaSuccess) e = page_map(&vmap, a, a.v, D, box);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(paged_many_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_dependent(paged_many_kernel<D>, a.grid, C::THREADS, C::SMEM, s, a, kmap, vmap);
}

}  // namespace

int paged_many_rows(int head_dim) { return head_dim == 256 ? Many<256>::RT : Many<128>::RT; }

cudaError_t launch_paged_many(const PagedArgs &a, int head_dim, cudaStream_t s)
{
    switch (head_dim) {
    case 64: return launch_many_d<64>(a, s);
    case 128: return launch_many_d<128>(a, s);
    default: return launch_many_d<256>(a, s);
    }
}

}  // namespace hq
