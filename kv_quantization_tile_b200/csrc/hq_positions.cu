// hq_positions.cu -- rotary positions, and the append of keys and values to a
// paged cache with the rotation on the way (sm_100a).
//
// Pair i of a head at position p turns by a = p theta_i:
//   y1 = A (x1 cos a - x2 sin a),  y2 = A (x2 cos a + x1 sin a),
// pairs being elements (i, i + r/2) (half) or (2i, 2i + 1) (interleaved) of
// the head's first r elements; the others are copied.  theta_i / 2 pi comes as
// a 64-bit fraction of a turn, so p theta_i mod one turn is one wrapping
// integer product: exact for every position (2^-65 p turns from theta's own
// rounding), where a binary32 angle would lose 2^-24 p radians.  What is left
// of the nearest quarter turn goes to sincospif, and the quarter swaps and
// negates: the values keep binary32's relative accuracy near every axis.
//
// Bound by HBM: every element is read and written once.  A block turns a few
// tokens: it computes each token's rotary / 2 cosines and sines once into
// shared memory, then every thread moves 16 elements of one head at a time
// (two 8-element units, 16-byte accesses), all heads of q, k and v alike.
#include "hq_paged.h"

namespace hq {

namespace {

constexpr int kPosThreads = 256;

struct Unit {
    float v[8];
};

__device__ __forceinline__ Unit load_unit(const Rows &r, int64_t off)
{
    Unit u;
    if (r.f32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(r.p) + off);
        const float4 a = p[0], b = p[1];
        u.v[0] = a.x; u.v[1] = a.y; u.v[2] = a.z; u.v[3] = a.w;
        u.v[4] = b.x; u.v[5] = b.y; u.v[6] = b.z; u.v[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(r.p) + off);
        const uint32_t ww[4] = { w.x, w.y, w.z, w.w };
#pragma unroll
        for (int i = 0; i < 4; i++) {
            u.v[2 * i] = __uint_as_float(ww[i] << 16);
            u.v[2 * i + 1] = __uint_as_float(ww[i] & 0xffff0000u);
        }
    }
    return u;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ void store_unit(void *p, int f32, int64_t off, const Unit &u)
{
    if (f32) {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p) + off);
        o[0] = make_float4(u.v[0], u.v[1], u.v[2], u.v[3]);
        o[1] = make_float4(u.v[4], u.v[5], u.v[6], u.v[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + off) =
            make_uint4(pack2(u.v[0], u.v[1]), pack2(u.v[2], u.v[3]), pack2(u.v[4], u.v[5]), pack2(u.v[6], u.v[7]));
    }
}

// cos and sin of `phase` (2^-64 turns), each within a rounding or two of its
// own size: q the nearest quarter turn, the rest (at most an eighth of a turn)
// in half turns for sincospif.
__device__ __forceinline__ float2 cos_sin(uint64_t phase)
{
    const uint64_t q = (phase + (1ull << 61)) >> 62;
    const int64_t rest = (int64_t)(phase - (q << 62));
    float s, c;
    sincospif((float)rest * 0x1p-63f, &s, &c);
    const float x = (q & 1) ? s : c, y = (q & 1) ? c : s;  // cos and sin up to sign
    const bool nc = ((q + 1) & 2) != 0, ns = (q & 2) != 0;
    return make_float2(nc ? -x : x, ns ? -y : y);
}

}  // namespace

// Item i of a token: 16 elements of head i / (head_dim / 16) (q heads, then k,
// then v).  Shared table: pair 8 j + 2 c + e of a token at float4 c * units + j.
__global__ void __launch_bounds__(kPosThreads) positions_kernel(const PosArgs a)
{
    extern __shared__ float4 sm_cs[];
    const int tid = threadIdx.x;
    const int units = a.head_dim / 16, runits = a.rotary / 16, pairs = a.rotary / 2;
    const int items = (a.heads + 2 * a.kvh) * units;
    const int64_t tok0 = (int64_t)blockIdx.x * a.tokens_per_block;
    const int nt = (int)min((int64_t)a.tokens_per_block, a.tokens - tok0);

    for (int e = tid; e < nt * pairs; e += kPosThreads) {
        const int t = e / pairs, i = e - t * pairs;
        const uint64_t phase = (uint64_t)a.positions[tok0 + t] * a.turns[i];
        float2 cs = cos_sin(phase);
        cs.x *= a.amplitude;
        cs.y *= a.inverse ? -a.amplitude : a.amplitude;
        const int j = i >> 3, c = (i >> 1) & 3;
        reinterpret_cast<float2 *>(sm_cs + (t * 4 + c) * runits + j)[i & 1] = cs;
    }
    __syncthreads();

    for (int e = tid; e < nt * items; e += kPosThreads) {
        const int t = (int)fast_div((uint32_t)e, a.items_div);
        const int w = e - t * items;
        int head = (int)fast_div((uint32_t)w, a.unit_div);
        const int j = w - head * units;
        const int64_t tok = tok0 + t;
        const bool rotated = j < runits && head < a.heads + a.kvh;
        const int half = rotated && !a.interleaved;
        const int e0 = half ? 8 * j : 16 * j, e1 = half ? a.rotary / 2 + 8 * j : 16 * j + 8;
        int64_t slot = 0;
        if (a.slots) {
            slot = a.slots[tok];
            if (slot < 0) continue;  // a padding token
            if (slot >= a.nslots) {
                if (w == 0 && a.status) atomicOr(a.status, kStatusIndex);
                continue;
            }
        }
        // where the row comes from and goes to
        Rows src;
        void *dst;
        int f32 = 0;
        int64_t from, to;
        if (head < a.heads) {
            src = a.x;
            dst = a.y.p;
            f32 = a.y.f32;
            from = tok * a.x.ts + head * a.x.hs;
            to = tok * a.y.ts + head * a.y.hs;
        } else {
            head -= a.heads;
            const bool is_v = head >= a.kvh;
            if (is_v) head -= a.kvh;
            src = is_v ? a.v : a.k;
            dst = is_v ? a.pv : a.pk;
            from = tok * src.ts + head * src.hs;
            to = (slot >> a.page_shift) * a.page_stride + head * a.head_stride +
                 (slot & ((1 << a.page_shift) - 1)) * a.slot_stride;
        }
        Unit u0 = load_unit(src, from + e0), u1 = load_unit(src, from + e1);
        if (rotated) {
            float cs[16];
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const float4 f = sm_cs[(t * 4 + c) * runits + j];
                cs[4 * c] = f.x;
                cs[4 * c + 1] = f.y;
                cs[4 * c + 2] = f.z;
                cs[4 * c + 3] = f.w;
            }
            if (half) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float x1 = u0.v[i], x2 = u1.v[i], co = cs[2 * i], si = cs[2 * i + 1];
                    u0.v[i] = x1 * co - x2 * si;
                    u1.v[i] = x2 * co + x1 * si;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    Unit &u = i < 4 ? u0 : u1;
                    const int k = 2 * (i & 3);
                    const float x1 = u.v[k], x2 = u.v[k + 1], co = cs[2 * i], si = cs[2 * i + 1];
                    u.v[k] = x1 * co - x2 * si;
                    u.v[k + 1] = x2 * co + x1 * si;
                }
            }
        }
        store_unit(dst, f32, to + e0, u0);
        store_unit(dst, f32, to + e1, u1);
    }
}

// One token per block while that leaves SMs idle, four at most: a block then
// computes 256 cosine pairs at once (one per thread, head_dim 128).
cudaError_t launch_positions(const PosArgs &args, cudaStream_t s)
{
    PosArgs a = args;
    const int units = a.head_dim / 16;
    a.items_div = make_fastdiv((uint32_t)((a.heads + 2 * a.kvh) * units));
    a.unit_div = make_fastdiv((uint32_t)units);
    a.tokens_per_block = a.tokens >= 16 * (int64_t)sm_count() ? 4 : 1;
    const int64_t blocks = (a.tokens + a.tokens_per_block - 1) / a.tokens_per_block;
    const size_t smem = (size_t)a.tokens_per_block * a.rotary / 2 * sizeof(float2);
    positions_kernel<<<(unsigned)blocks, kPosThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace hq
