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
// shared memory, then every thread moves 16 elements of one head at a time, all
// heads of q, k and v alike.  The 16 are four quads of 4 elements so placed
// that a warp's stores are contiguous: pairs of adjacent quads, 16 bytes, where
// the output is bf16; quads on their own, 16 bytes, where it is binary32 (8191 x
// 32 x 128 in binary32: 45.5 us, with adjacent quads, half a sector per store,
// 53.1; 8192 tokens of 48 heads from binary32 to bf16 the other way round, 55.2
// against 51.2).  The two pairs of adjacent quads lie 8 elements apart, a whole
// item in a row, unless they have to hold pairs half the rotated part apart: half
// a head apart everywhere, and with the addresses that takes, the same 8192
// tokens take 53.3 us, from bf16 to bf16 45.2 against 40.1.
#include "hq_paged.h"

namespace hq {

namespace {

constexpr int kPosThreads = 256;

__device__ __forceinline__ void unpack(uint32_t w, float &lo, float &hi)
{
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
}

// The quads of item j of a span of n elements that begins at `base`, a quarter apart
__device__ __forceinline__ void quarters(int base, int n, int j, int (&at)[4])
{
#pragma unroll
    for (int q = 0; q < 4; q++) at[q] = base + q * (n / 4) + 4 * j;
}

template <bool QUADS>
__device__ __forceinline__ void load16(const Rows &r, int64_t off, const int (&at)[4], float (&v)[16])
{
    const uint16_t *b = static_cast<const uint16_t *>(r.p) + off;
    if (r.f32) {
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const float4 x = *reinterpret_cast<const float4 *>(static_cast<const float *>(r.p) + off + at[q]);
            v[4 * q] = x.x;
            v[4 * q + 1] = x.y;
            v[4 * q + 2] = x.z;
            v[4 * q + 3] = x.w;
        }
    } else if constexpr (QUADS) {
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const uint2 x = *reinterpret_cast<const uint2 *>(b + at[q]);
            unpack(x.x, v[4 * q], v[4 * q + 1]);
            unpack(x.y, v[4 * q + 2], v[4 * q + 3]);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
            const uint4 x = *reinterpret_cast<const uint4 *>(b + at[q]);
            unpack(x.x, v[4 * q], v[4 * q + 1]);
            unpack(x.y, v[4 * q + 2], v[4 * q + 3]);
            unpack(x.z, v[4 * q + 4], v[4 * q + 5]);
            unpack(x.w, v[4 * q + 6], v[4 * q + 7]);
        }
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

template <bool QUADS>
__device__ __forceinline__ void store16(void *p, int f32, int64_t off, const int (&at)[4], const float (&v)[16])
{
    uint16_t *b = static_cast<uint16_t *>(p) + off;
    if (f32) {
#pragma unroll
        for (int q = 0; q < 4; q++)
            *reinterpret_cast<float4 *>(static_cast<float *>(p) + off + at[q]) =
                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    } else if constexpr (QUADS) {
#pragma unroll
        for (int q = 0; q < 4; q++)
            *reinterpret_cast<uint2 *>(b + at[q]) = make_uint2(pack2(v[4 * q], v[4 * q + 1]), pack2(v[4 * q + 2], v[4 * q + 3]));
    } else {
#pragma unroll
        for (int q = 0; q < 4; q += 2)
            *reinterpret_cast<uint4 *>(b + at[q]) = make_uint4(pack2(v[4 * q], v[4 * q + 1]), pack2(v[4 * q + 2], v[4 * q + 3]),
                                                               pack2(v[4 * q + 4], v[4 * q + 5]), pack2(v[4 * q + 6], v[4 * q + 7]));
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
// then v).  The shared table holds each item's 8 pairs in the order of its
// elements, two to a float4: float4 c of item j at c * items of the head + j.
// An item's pairs are `groups` runs of 8 / groups consecutive ones.
template <bool QUADS>
__global__ void __launch_bounds__(kPosThreads) positions_kernel(const PosArgs a)
{
    extern __shared__ float4 sm_cs[];
    const int tid = threadIdx.x;
    const int units = a.head_dim / 16, runits = a.rotary / 16, pairs = a.rotary / 2;
    const int items = (a.heads + 2 * a.kvh) * units;
    const int64_t tok0 = (int64_t)blockIdx.x * a.tokens_per_block;
    const int nt = (int)min((int64_t)a.tokens_per_block, a.tokens - tok0);
    const int gshift = !QUADS ? 0 : a.interleaved ? 2 : 1;  // log2 of the groups

    for (int e = tid; e < nt * pairs; e += kPosThreads) {
        const int t = e / pairs, i = e - t * pairs;
        const uint64_t phase = (uint64_t)a.positions[tok0 + t] * a.turns[i];
        float2 cs = cos_sin(phase);
        cs.x *= a.amplitude;
        cs.y *= a.inverse ? -a.amplitude : a.amplitude;
        const int run = pairs >> gshift, g = i / run, k = i - g * run;  // pair k of group g
        const int j = k >> (3 - gshift), c = (g << (2 - gshift)) + ((k >> 1) & ((4 >> gshift) - 1));
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
        int at[4];
        if constexpr (QUADS) {  // the rotated span of a head, or the rest of it (no append)
            if (rotated) quarters(0, a.rotary, j, at);
            else quarters(a.rotary, a.head_dim - a.rotary, j - runits, at);
        } else {
            const bool half = rotated && !a.interleaved;
            at[0] = half ? 8 * j : 16 * j;
            at[2] = half ? a.rotary / 2 + 8 * j : 16 * j + 8;
            at[1] = at[0] + 4;
            at[3] = at[2] + 4;
        }
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
        float v[16];
        load16<QUADS>(src, from, at, v);
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
#pragma unroll
            for (int i = 0; i < 8; i++) {
                if (a.interleaved) {
                    const float x1 = v[2 * i], x2 = v[2 * i + 1], co = cs[2 * i], si = cs[2 * i + 1];
                    v[2 * i] = x1 * co - x2 * si;
                    v[2 * i + 1] = x2 * co + x1 * si;
                } else {
                    const float x1 = v[i], x2 = v[8 + i], co = cs[2 * i], si = cs[2 * i + 1];
                    v[i] = x1 * co - x2 * si;
                    v[8 + i] = x2 * co + x1 * si;
                }
            }
        }
        store16<QUADS>(dst, f32, to, at, v);
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
    const bool quads = a.kvh == 0 && a.y.f32;
    (quads ? positions_kernel<true> : positions_kernel<false>)<<<(unsigned)blocks, kPosThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace hq
