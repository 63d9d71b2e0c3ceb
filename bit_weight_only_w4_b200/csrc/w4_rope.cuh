// w4_rope.cuh -- rotary positions on the heads of a projection's output.
//
//   pair (a, b) number i of a head at position t:  phi = t * inv_freq[i]
//     a' = m (a cos phi - b sin phi)      b' = m (b cos phi + a sin phi)
//   pairs: (x[i], x[i + rot/2]) (halves) or (x[2i], x[2i+1]) (interleaved), i < rot/2; the
//   elements behind rot are copied.
// Bound by memory: every element is read and written once.  The rot/2 angles of a token
// serve all its heads: a block takes whole tokens (as many as fill it), computes their cosines
// and sines into shared memory, and each thread takes one piece of the head (E consecutive
// pairs, their cosines and sines in registers) through every heads_lanes-th head.  Its first
// loads of x go out before the angles, whose latency they hide, kBatch heads at a time.  (One
// head a thread read shared memory as often as x: 8192 tokens x 40 heads of 128, bf16, 43.4 us
// against 29.0, 5.8 TB/s.)  The angle is reduced in fp64 to a fraction of a turn (position 2^20 times a
// frequency of 1 leaves fp32 with 4 bits of the fraction), sine and cosine are then taken in
// fp32.
// A piece is two 16-byte words (E = 8 16-bit or 4 32-bit elements), or single elements (E = 1)
// when a stride, a pointer or rot does not allow it.
#pragma once
#include "w4_common.cuh"

namespace w4r {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 256;          // rot / 2
constexpr int kMaxTokens = 16;          // tokens of one block
constexpr int kBatch = 4;               // heads of a thread in flight

struct RopeParams {
    const void* X;
    void* Y;
    const int32_t* positions;   // [tokens]
    const double* inv_freq;     // [rot / 2]
    long long ldx, hsx, ldy, hsy;   // elements between tokens and between heads
    int tokens, heads, dim, rot, interleaved;
    int per_head;               // pieces of a head: rot/2/E rotated, then ceil((dim-rot)/2E) copied
    int heads_per_block, tokens_per_block;
    int head_lanes;             // threads that share a token's heads
    int copy_tail;              // 0: in place, the tail stays where it is
    float mscale;
};

// DT: 0 fp16, 1 bf16, 2 fp32 (as w4_dtype)
template <int DT>
W4_DEV float to_f32(uint32_t bits) {
    if constexpr (DT == 2) return __uint_as_float(bits);
    else if constexpr (DT == 1) return __uint_as_float(bits << 16);
    else return __half2float(__ushort_as_half((unsigned short)bits));
}

// E elements, as they lie in memory.
template <int E>
struct Raw {
    uint32_t w[E == 1 ? 1 : 4];
};

template <int DT, int E>
W4_DEV Raw<E> load_raw(const void* base, size_t i) {
    Raw<E> r;
    if constexpr (E == 1) {
        if constexpr (DT == 2) r.w[0] = reinterpret_cast<const uint32_t*>(base)[i];
        else r.w[0] = reinterpret_cast<const unsigned short*>(base)[i];
    } else {
        const uint4 v = DT == 2 ? *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(base) + i)
                                : *reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned short*>(base) + i);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    }
    return r;
}

template <int DT, int E>
W4_DEV void store_raw(void* base, size_t i, const Raw<E>& r) {
    if constexpr (E == 1) {
        if constexpr (DT == 2) reinterpret_cast<uint32_t*>(base)[i] = r.w[0];
        else reinterpret_cast<unsigned short*>(base)[i] = (unsigned short)r.w[0];
    } else {
        const uint4 v = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        if constexpr (DT == 2) *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(base) + i) = v;
        else *reinterpret_cast<uint4*>(reinterpret_cast<unsigned short*>(base) + i) = v;
    }
}

template <int DT, int E>
W4_DEV void to_floats(const Raw<E>& r, float (&v)[E]) {
    if constexpr (E == 1) {
        v[0] = to_f32<DT>(r.w[0]);
    } else if constexpr (DT == 2) {
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = __uint_as_float(r.w[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = unpack2<DT == 1>(r.w[k]);
            v[2 * k] = f.x;
            v[2 * k + 1] = f.y;
        }
    }
}

template <int DT, int E>
W4_DEV Raw<E> from_floats(const float (&v)[E]) {
    Raw<E> r;
    if constexpr (DT == 2) {
#pragma unroll
        for (int k = 0; k < E; ++k) r.w[k] = __float_as_uint(v[k]);
    } else if constexpr (E == 1) {
        r.w[0] = DT == 1 ? __bfloat16_as_ushort(__float2bfloat16_rn(v[0])) : __half_as_ushort(__float2half_rn(v[0]));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) r.w[k] = pack2<DT == 1>(v[2 * k], v[2 * k + 1]);
    }
    return r;
}

template <int DT, int E>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
    extern __shared__ float2 turn[];   // [tokens_per_block][rot / 2] (m cos, m sin)
    pdl_launch_dependents();
    pdl_wait();   // X may come from the preceding kernel
    const int t0 = blockIdx.x * p.tokens_per_block, nt = min(p.tokens_per_block, p.tokens - t0);
    const int h0 = blockIdx.y * p.heads_per_block, h1 = min(p.heads, h0 + p.heads_per_block);
    const int half = p.rot / 2;
    // this thread's piece, head lane and token
    const int rest = threadIdx.x / p.per_head, k = threadIdx.x - rest * p.per_head;
    const int tok = rest / p.head_lanes, lane = rest - tok * p.head_lanes;
    const bool on = tok < nt;
    const int pair = E * k;
    const bool rotated = pair < half;
    const int o0 = !rotated ? p.rot + 2 * (pair - half) : p.interleaved ? 2 * pair : pair;
    const int o1 = rotated && !p.interleaved ? o0 + half : o0 + E;
    const bool two = o1 < p.dim;   // (a tail's last piece may be one word)
    const void* X = p.X;
    const size_t x0 = (size_t)(t0 + tok) * p.ldx, y0 = (size_t)(t0 + tok) * p.ldy;
    const bool moves = on && (rotated || p.copy_tail);
    Raw<E> a[kBatch], b[kBatch];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int hh = h + i * p.head_lanes;
            if (!moves || hh >= h1) continue;
            const size_t x = x0 + (size_t)hh * p.hsx;
            a[i] = load_raw<DT, E>(X, x + o0);
            if (two) b[i] = load_raw<DT, E>(X, x + o1);
        }
    };
    load(h0 + lane);
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half;
        const double turns = (double)p.positions[t0 + t] * p.inv_freq[i - t * half] * 0.15915494309189533577;
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        turn[i] = make_float2(p.mscale * c, p.mscale * s);
    }
    __syncthreads();
    if (!moves) return;
    float2 cs[E];
    if (rotated) {
#pragma unroll
        for (int i = 0; i < E; ++i) cs[i] = turn[tok * half + pair + i];
    }
    for (int h = h0 + lane; h < h1; h += kBatch * p.head_lanes) {
        if (h != h0 + lane) load(h);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int hh = h + i * p.head_lanes;
            if (hh >= h1) continue;
            const size_t y = y0 + (size_t)hh * p.hsy;
            if (rotated) {
                float u[E], v[E];
                to_floats<DT, E>(a[i], u);
                to_floats<DT, E>(b[i], v);
                if (E > 1 && p.interleaved) {
                    // words hold pairs (2j, 2j+1): E/2 pairs each
#pragma unroll
                    for (int j = 0; j < E / 2; ++j) {
                        const float2 c = cs[j], d = cs[E / 2 + j];
                        const float u0 = u[2 * j], u1 = u[2 * j + 1], v0 = v[2 * j], v1 = v[2 * j + 1];
                        u[2 * j] = u0 * c.x - u1 * c.y;
                        u[2 * j + 1] = u1 * c.x + u0 * c.y;
                        v[2 * j] = v0 * d.x - v1 * d.y;
                        v[2 * j + 1] = v1 * d.x + v0 * d.y;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        const float u0 = u[j], v0 = v[j];
                        u[j] = u0 * cs[j].x - v0 * cs[j].y;
                        v[j] = v0 * cs[j].x + u0 * cs[j].y;
                    }
                }
                a[i] = from_floats<DT, E>(u);
                b[i] = from_floats<DT, E>(v);
            }
            store_raw<DT, E>(p.Y, y + o0, a[i]);
            if (two) store_raw<DT, E>(p.Y, y + o1, b[i]);
        }
    }
}

}  // namespace w4r
