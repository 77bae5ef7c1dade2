// hq_paged_tc.cu -- attention over a paged KV cache for many new tokens per
// sequence (chunks of a prompt), on the 5th-generation tensor cores (sm_100a).
//
// Rows, jobs, tiles and the blocks' equal shares are those of hq_paged.cu,
// with row tiles of 256 packed rows (two MMA tiles of 128; one of 128 at
// head_dim 256, whose output fills the tensor memory) and token tiles of 128
// (64).  One block per SM, its warps in roles:
//   * the load warp copies K and V tiles page by page with TMA (128-byte
//     swizzle, one copy per page and 64 columns) into a ring of buffers;
//   * the product warp issues S = Q K^T (both operands in shared memory) and
//     O += P V (P in tensor memory, V as it lies, token-major) with
//     tcgen05.mma; while one MMA tile's softmax runs, the other's products do;
//   * a warpgroup per MMA tile (its threads one row each, so a row's maximum
//     and sum need no exchange) reads S from tensor memory, keeps the running
//     softmax and writes P over S in bf16.
// The running maximum is raised, and O rescaled, only where a tile exceeds it
// by more than 2^8: weights then stay below 2^8, far inside bf16 and binary32,
// and the final division by their sum cancels the stale maximum exactly
// ("FlashAttention-4" describes this rule).
//
// Bound: the products are 4 d flops per (row, token), the exponentials one per
// (row, token) on a unit with 16 per clock and SM: at head_dim 128 a tile pair
// takes 1024 clocks of tensor pipe and 2048 of exponentials.
#include <atomic>

#include <cuda.h>

#include "hq_paged.h"
#include "hq_tcgen05.cuh"

namespace hq {

namespace {

constexpr float kGrow = 8.0f;  // powers of two by which a tile may exceed the running maximum

template <int D>
struct Many {
    static constexpr int NT = D == 256 ? 1 : 2;        // MMA tiles of 128 rows
    static constexpr int RT = 128 * NT;
    static constexpr int T = D == 256 ? 64 : 128;      // tokens per tile
    static constexpr int THREADS = 128 * (NT + 1);
    static constexpr uint32_t TILE = T * D * 2;        // one K or V tile
    static constexpr uint32_t QTILE = 128 * D * 2;
    static constexpr int STAGES = D == 64 ? 8 : 5;
    static constexpr size_t SMEM = 1024 + NT * QTILE + STAGES * TILE;
    // tensor memory: O of each MMA tile, then two score buffers
    static constexpr uint32_t O_COL = 0, S_COL = 256;
};

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
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done;
}
// bounded (mbar_wait); the first poll reads no timer
__device__ __forceinline__ bool await(uint32_t bar, uint32_t parity) { return mbar_try(bar, parity) || mbar_wait(bar, parity); }

__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap *map, uint32_t bar, int col, int slot, int head, int page)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(dst), "l"(map), "r"(bar), "r"(col), "r"(slot), "r"(head), "r"(page)
        : "memory");
}

__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// byte offset of 16-byte chunk c of row r in a 128-byte-swizzled operand of
// `rows` rows: blocks of 64 columns, each [rows][128 bytes]
__device__ __forceinline__ uint32_t swizzled_off(int rows, int r, int c)
{
    return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(Many<D>::THREADS, 1)
paged_many_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using C = Many<D>;
    constexpr int NT = C::NT, RT = C::RT, T = C::T, STAGES = C::STAGES;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t s_bar[2 * STAGES + NT * 2 + 4 + 1];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_fail;
    __shared__ int s_last[NT];
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
    const uint32_t fix_bar = bar0 + 8u * (uint32_t)(2 * STAGES + 2 * NT + 4);

    if (warp == 0) tmem_alloc(smem_u32(&s_tmem), 512);
    if (tid == 0) {
        s_fail = 0;
        for (int s = 0; s < STAGES; s++) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int t = 0; t < NT; t++) {
            mbar_init(q_full(t), 4);
            mbar_init(o_full(t), 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(s_full(b), 1);
            mbar_init(p_full(b), 4);
        }
        mbar_init(fix_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // a wait that gave up: every role leaves its loops at its next check
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        if (await(bar, parity)) return true;
        s_fail = 1;
        return false;
    };

    pdl_wait();
    SegWalk<T, RT> w;
    const bool work = w.begin(a);

    if (wg < NT) {
        // ------------------------------------------------ softmax
        if constexpr (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int t = wg, wl = warp & 3;
        const uint32_t lanes = (uint32_t)(wl * 32) << 16;
        const uint32_t to = tmem + lanes + C::O_COL + (uint32_t)(t * D);
        uint32_t g = 0;  // tiles so far
        if (work) do {
            const int r0 = w.rt * RT + t * 128;
            // ---- this warp's 32 query rows
            constexpr int CH = D / 8;
            for (int e = lane; e < 32 * CH; e += 32) {
                const int rr = wl * 32 + e / CH, c = e % CH, r = r0 + rr;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (r < w.s.rows && a.q_mode != 2) {
                    const int j = (int)fast_div((uint32_t)r, a.group_div), gg = r - j * a.group;
                    v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q.p) + (w.s.q0 + j) * a.q.ts +
                                                         (w.h * a.group + gg) * a.q.hs + 8 * c);
                    if (a.q_mode == 1) {
                        v.x ^= 0x80008000u;
                        v.y ^= 0x80008000u;
                        v.z ^= 0x80008000u;
                        v.w ^= 0x80008000u;
                    }
                }
                const uint32_t dst = sq + t * C::QTILE + swizzled_off(128, rr, c);
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full(t));

            const int r = r0 + wl * 32 + lane;
            int rlo = 0, rhi = 0;
            if (r < w.s.rows) {
                const int j = (int)fast_div((uint32_t)r, a.group_div);
                seen_range(a, w.s, j, j, rlo, rhi);
            }
            float m = -INFINITY, l = 0.0f;
            bool ok = true;
            for (int tile = w.first; tile < w.first + w.count; tile++, g++) {
                const int b = NT == 2 ? t : (int)(g & 1u);
                const uint32_t par = NT == 2 ? g & 1u : (g >> 1) & 1u;
                const uint32_t ts = tmem + lanes + C::S_COL + (uint32_t)(b * T);
                ok = wait(s_full(b), par) && !s_fail;
                if (!__all_sync(FULL, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t s[T / 32][32];
#pragma unroll
                for (int c = 0; c < T / 32; c++) tmem_ld32(ts + 32 * c, s[c]);
                tmem_wait_ld();
                const int tok0 = (w.t0 + tile) * T;
                if (!__all_sync(FULL, rlo <= tok0 && rhi >= tok0 + T)) {
                    const int from = rlo - tok0, to_ = rhi - tok0;
#pragma unroll
                    for (int c = 0; c < T / 32; c++)
#pragma unroll
                        for (int i = 0; i < 32; i++)
                            if (32 * c + i < from || 32 * c + i >= to_) s[c][i] = 0xff800000u;
                }
                float mx[4] = { -INFINITY, -INFINITY, -INFINITY, -INFINITY };
#pragma unroll
                for (int c = 0; c < T / 32; c++)
#pragma unroll
                    for (int i = 0; i < 32; i++) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[c][i]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
                if (tile == w.first) {
                    m = top;
                } else {
                    // Every product with V is waited for in turn (a barrier's
                    // phase can only be told from the one before it).  With two
                    // MMA tiles S comes after that product anyway; with one, S
                    // runs ahead of it.
                    if (NT == 1) {
                        ok = wait(o_full(t), (g - 1u) & 1u);
                        if (!__all_sync(FULL, ok)) {
                            ok = false;
                            break;
                        }
                    }
                    const bool grow = top > m + kGrow;
                    if (__any_sync(FULL, grow)) {  // rescale O: the product before this one is complete
                        const float f = grow ? ex2(m - top) : 1.0f;
                        if (grow) m = top;
                        l *= f;
                        ok = wait(o_full(t), (g - 1u) & 1u);
                        if (!__all_sync(FULL, ok)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 32; c++) {
                            uint32_t o[32];
                            tmem_ld32(to + 32 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(to + 32 * c, o);
                        }
                    }
                }
                const float off = m == -INFINITY ? 0.0f : m;  // nothing seen yet: every weight is 0
                // weights are rounded to bf16 for the product with V (2^-8 of
                // each, independent); their sum keeps binary32
                float sum[4] = { 0.0f, 0.0f, 0.0f, 0.0f };
#pragma unroll
                for (int c = 0; c < T / 64; c++) {
                    uint32_t p[32];
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        const float x = ex2(fmaf(__uint_as_float(s[2 * c + i / 16][2 * (i & 15)]), a.scale_log2, -off));
                        const float y = ex2(fmaf(__uint_as_float(s[2 * c + i / 16][2 * (i & 15) + 1]), a.scale_log2, -off));
                        sum[2 * (i & 1)] += x;
                        sum[2 * (i & 1) + 1] += y;
                        p[i] = pack2(x, y);
                    }
                    tmem_st32(ts + 32 * c, p);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(b));
            }
            if (!ok) break;
            // ---- the segment's end
            ok = wait(o_full(t), (g - 1u) & 1u);
            if (!__all_sync(FULL, ok)) break;
            tc_fence_after();
            const bool whole = w.whole();
            const int rr = wl * 32 + lane;  // row of this MMA tile
            // partial results by MMA tile: m and l of its rows, then [D / 4][128] float4
            float *part = a.part + ((int64_t)w.slot() * NT + t) * (128 * (D + 2));
            if (!whole) {
                part[rr] = m;
                part[128 + rr] = l;
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            int64_t tok = 0;
            int head = 0;
            if (r < w.s.rows) {
                const int j = (int)fast_div((uint32_t)r, a.group_div);
                tok = w.s.q0 + j;
                head = w.h * a.group + r - j * a.group;
            }
            const int64_t at = tok * a.out.ts + head * a.out.hs;
            auto put = [&](int c, const float (&v)[32], float f, bool zero) {  // 32 columns of the row
                if (r >= w.s.rows) return;
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
            for (int c = 0; c < D / 32; c++) {
                uint32_t o[32];
                tmem_ld32(to + 32 * c, o);
                tmem_wait_ld();
                if (whole) {
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; i++) v[i] = __uint_as_float(o[i]);
                    put(c, v, inv, l == 0.0f);
                } else {
                    float4 *p = reinterpret_cast<float4 *>(part + 256) + (8 * c) * 128 + rr;
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
                group_sync(1 + t);
                const int c0 = w.owner(), c1 = w.last();
                if (wl == 0 && lane == 0) s_last[t] = atomicAdd(a.counter + c0 * NT + t, 1u) == (unsigned)(c1 - c0);
                group_sync(1 + t);
                write = s_last[t];
                if (write) {
                    __threadfence();
                    auto part_at = [&](int k) {
                        return a.part + ((int64_t)(2 * k + (k == c0 ? 1 : 0)) * NT + t) * (128 * (D + 2));
                    };
                    mt = -INFINITY;
                    for (int k = c0; k <= c1; k++) mt = fmaxf(mt, __ldcg(part_at(k) + rr));
                    const float from = mt == -INFINITY ? 0.0f : mt;
                    lt = 0.0f;
                    for (int k = c0; k <= c1; k++) lt = fmaf(ex2(__ldcg(part_at(k) + rr) - from), __ldcg(part_at(k) + 128 + rr), lt);
                    const float f = lt == 0.0f ? 0.0f : 1.0f / lt;
#pragma unroll 1
                    for (int c = 0; c < D / 32; c++) {
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; i++) v[i] = 0.0f;
                        for (int k = c0; k <= c1; k++) {
                            const float e = ex2(__ldcg(part_at(k) + rr) - from);
                            const float4 *p = reinterpret_cast<const float4 *>(part_at(k) + 256) + (8 * c) * 128 + rr;
#pragma unroll
                            for (int i = 0; i < 8; i++) {
                                const float4 x = __ldcg(p + i * 128);
                                v[4 * i] = fmaf(e, x.x, v[4 * i]);
                                v[4 * i + 1] = fmaf(e, x.y, v[4 * i + 1]);
                                v[4 * i + 2] = fmaf(e, x.z, v[4 * i + 2]);
                                v[4 * i + 3] = fmaf(e, x.w, v[4 * i + 3]);
                            }
                        }
                        put(c, v, f, lt == 0.0f);
                    }
                }
            }
            if (write && a.lse && r < w.s.rows)
                a.lse[tok * (a.heads * a.group) + head] = lt == 0.0f ? -INFINITY : fmaf(mt, 0.693147180559945309f, logf(lt));
        } while (w.next(a));
    } else {
        if constexpr (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if ((warp & 3) == 0) {
            // -------------------------------------------- products
            if (lane == 0 && work) {
                constexpr uint32_t ID_S = make_idesc_bf16(128, T);
                constexpr uint32_t ID_O = make_idesc_bf16(128, D) | (1u << 16);  // V is token-major: B not K-major
                uint32_t slot = 0, phase = 0, g = 0, seg = 0;
                bool ok = true;
                auto take = [&]() -> uint32_t {  // the next tile of the ring, landed
                    ok = ok && wait(kv_full(slot), phase) && !s_fail;
                    const uint32_t s = slot;
                    if (++slot == STAGES) {
                        slot = 0;
                        phase ^= 1u;
                    }
                    return s;
                };
                auto scores = [&](int t, int b, uint32_t s) {
                    const uint32_t q = sq + t * C::QTILE, k = ring + s * C::TILE, d = tmem + C::S_COL + (uint32_t)(b * T);
#pragma unroll
                    for (int i = 0; i < D / 16; i++)
                        umma_bf16(d, swizzled_desc(q + (i >> 2) * 16384 + (i & 3) * 32, 16, 1024),
                                  swizzled_desc(k + (i >> 2) * (T * 128) + (i & 3) * 32, 16, 1024), ID_S, i > 0);
                    umma_commit(s_full(b));
                };
                auto outputs = [&](int t, int b, uint32_t s, bool add) {
                    const uint32_t p = tmem + C::S_COL + (uint32_t)(b * T), v = ring + s * C::TILE;
#pragma unroll
                    for (int i = 0; i < T / 16; i++)
                        umma_bf16_ts(tmem + C::O_COL + (uint32_t)(t * D), p + 8 * i, swizzled_desc(v + i * 2048, T * 128, 1024), ID_O,
                                     add || i > 0);
                    umma_commit(o_full(t));
                };
                do {
                    const uint32_t k0 = take();
                    for (int t = 0; t < NT && ok; t++) {
                        ok = wait(q_full(t), seg & 1u);
                        if (!ok) break;
                        tc_fence_after();
                        scores(t, NT == 2 ? t : (int)(g & 1u), k0);
                    }
                    if (!ok) break;
                    umma_commit(kv_empty(k0));
                    for (int j = 0; j < w.count && ok; j++, g++) {
                        const bool more = j + 1 < w.count;
                        const uint32_t k = more ? take() : 0u;
                        if (NT == 1 && more && ok) {
                            scores(0, (int)((g + 1) & 1u), k);
                            umma_commit(kv_empty(k));
                        }
                        const uint32_t v = take();
                        for (int t = 0; t < NT && ok; t++) {
                            const int b = NT == 2 ? t : (int)(g & 1u);
                            ok = wait(p_full(b), NT == 2 ? g & 1u : (g >> 1) & 1u) && !s_fail;
                            if (!ok) break;
                            tc_fence_after();
                            outputs(t, b, v, j > 0);
                            if (NT == 2 && more) scores(t, t, k);
                        }
                        if (!ok) break;
                        umma_commit(kv_empty(v));
                        if (NT == 2 && more) umma_commit(kv_empty(k));
                    }
                    seg++;
                } while (ok && w.next(a));
            }
            __syncwarp();
        } else if ((warp & 3) == 1 && work) {
            // -------------------------------------------- loads
            const int page_rows = 1 << a.page_shift, box = page_rows < T ? page_rows : T;
            const int col = lane % (D / 64), pg = lane / (D / 64);
            uint32_t slot = 0, phase = 0, fixes = 0;
            bool ok = true;
            auto load = [&](int tile, bool is_v) {
                ok = ok && wait(kv_empty(slot), phase ^ 1u) && !s_fail;
                ok = __all_sync(FULL, ok);
                if (!ok) return;
                const int tok0 = (w.t0 + tile) * T, tok = tok0 + pg * box;
                const uint32_t dst = ring + slot * C::TILE;
                // rows of V outside the job's tokens meet weight 0: they must be finite
                const bool fix = is_v && (tok0 < w.lo || tok0 + T > w.hi);
                const uint32_t bar = fix ? fix_bar : kv_full((int)slot);
                const bool mine = pg * box < T && tok < w.hi && tok + box > w.lo;
                uint32_t page = 0;
                if (mine) {
                    page = (uint32_t)a.table[(int64_t)w.b * a.table_stride + (tok >> a.page_shift)];
                    if (page >= a.pages) {
                        page = a.pages;  // past the pool: TMA fills zeros
                        if (a.status) atomicOr(a.status, kStatusIndex);
                    }
                }
                const uint32_t n = __popc(__ballot_sync(FULL, mine));
                if (lane == 0) mbar_expect(bar, n * (uint32_t)box * 128u);
                __syncwarp();
                if (mine)
                    tma_page(dst + (uint32_t)(col * T * 128 + pg * box * 128), is_v ? &vmap : &kmap, bar, col * 64,
                             tok & (page_rows - 1), w.h, (int)page);
                if (fix) {
                    ok = wait(fix_bar, fixes & 1u);
                    fixes++;
                    for (int e = lane; e < T * (D / 8); e += 32) {
                        const int r = e / (D / 8), c = e % (D / 8);
                        if (tok0 + r < w.lo || tok0 + r >= w.hi)
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
            do {
                const int e = w.first + w.count;
                load(w.first, false);
                for (int tile = w.first; tile < e && ok; tile++) {
                    if (tile + 1 < e) load(tile + 1, false);
                    load(tile, true);
                }
            } while (ok && w.next(a));
            // after a wait that gave up, let the copies in flight land
            if (!ok)
                for (int s = 0; s < STAGES; s++) mbar_wait(kv_full(s), s < (int)slot ? phase : phase ^ 1u);
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

// A pool as [page][head][slot][d]: one copy takes up to `box` slots of 64
// columns; a page past the pool reads zeros.
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
    if (e == cudaSuccess) e = launch_paged_plan(a, C::T, C::RT, C::NT, s);
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
