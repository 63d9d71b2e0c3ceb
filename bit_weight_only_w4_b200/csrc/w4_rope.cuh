// w4_rope.cuh -- rotary positions on the heads of a projection's output.
//
//   pair (a, b) number i of a head at position t:  phi = t * inv_freq[i]
//     a' = m (a cos phi - b sin phi)      b' = m (b cos phi + a sin phi)
//   pairs: (x[i], x[i + rot/2]) (halves) or (x[2i], x[2i+1]) (interleaved), i < rot/2; the
//   elements behind rot are copied.
// Bound by memory: every element is read and written once.  The rot/2 angles of a token
// serve all its heads, so a block takes whole tokens (as many as fill it), computes their
// cosines and sines into shared memory and then rotates; its threads issue the first loads
// of x before the angles, whose latency the loads hide.  The angle is reduced in fp64 to a
// fraction of a turn (position 2^20 times a frequency of 1 leaves fp32 with 4 bits of the
// fraction), sine and cosine are then taken in fp32.
// A thread's item is E consecutive pairs: two 16-byte pieces (E = 8 16-bit or 4 32-bit
// elements), or single elements (E = 1) when a stride, a pointer or rot does not allow it.
#pragma once
#include "w4_common.cuh"

namespace w4r {

constexpr int kMaxThreads = 512;
constexpr int kMaxPairs = 256;          // rot / 2
constexpr int kMaxTokens = 16;          // tokens of one block

struct RopeParams {
    const void* X;
    void* Y;
    const int32_t* positions;   // [tokens]
    const double* inv_freq;     // [rot / 2]
    long long ldx, hsx, ldy, hsy;   // elements between tokens and between heads
    int tokens, heads, dim, rot, interleaved;
    int per_head;               // items of a head: rot/2/E rotated, then ceil((dim-rot)/2E) copied
    int heads_per_block, tokens_per_block;
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

// E elements as fp32.
template <int DT, int E>
W4_DEV void load_piece(const void* base, size_t i, float (&v)[E]) {
    if constexpr (E == 1) {
        if constexpr (DT == 2) v[0] = reinterpret_cast<const float*>(base)[i];
        else v[0] = to_f32<DT>(reinterpret_cast<const unsigned short*>(base)[i]);
    } else if constexpr (DT == 2) {
        const float4 r = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + i);
        v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
    } else {
        const uint4 r = *reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned short*>(base) + i);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = unpack2<DT == 1>(w[k]);
            v[2 * k] = f.x;
            v[2 * k + 1] = f.y;
        }
    }
}

template <int DT, int E>
W4_DEV void store_piece(void* base, size_t i, const float (&v)[E]) {
    if constexpr (E == 1) {
        if constexpr (DT == 2) reinterpret_cast<float*>(base)[i] = v[0];
        else if constexpr (DT == 1) reinterpret_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v[0]);
        else reinterpret_cast<__half*>(base)[i] = __float2half_rn(v[0]);
    } else if constexpr (DT == 2) {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        constexpr bool B = DT == 1;
        *reinterpret_cast<uint4*>(reinterpret_cast<unsigned short*>(base) + i) =
            make_uint4(pack2<B>(v[0], v[1]), pack2<B>(v[2], v[3]), pack2<B>(v[4], v[5]), pack2<B>(v[6], v[7]));
    }
}

// What one item touches: its two pieces' offsets in a head, and its first pair.
struct Item {
    int tok, head, pair, o0, o1;
    bool rotated, two;
};

template <int E>
W4_DEV Item item_at(const RopeParams& p, int it, int t0, int h0, int nh) {
    Item r;
    const int per_tok = nh * p.per_head;
    r.tok = it / per_tok;
    const int rest = it - r.tok * per_tok;
    r.head = rest / p.per_head;
    const int k = rest - r.head * p.per_head;
    r.head += h0;
    const int half = p.rot / 2;
    r.pair = E * k;
    r.rotated = r.pair < half;
    r.two = true;
    if (r.rotated) {
        r.o0 = p.interleaved ? 2 * r.pair : r.pair;
        r.o1 = p.interleaved ? r.o0 + E : r.pair + half;
    } else {
        r.o0 = p.rot + 2 * (r.pair - half);
        r.o1 = r.o0 + E;
        r.two = r.o1 < p.dim;
    }
    r.tok += t0;
    return r;
}

template <int DT, int E>
__global__ void __launch_bounds__(kMaxThreads) rope_kernel(const RopeParams p) {
    extern __shared__ float2 turn[];   // [tokens_per_block][rot / 2] (m cos, m sin)
    pdl_launch_dependents();
    pdl_wait();   // X may come from the preceding kernel
    const int t0 = blockIdx.x * p.tokens_per_block, nt = min(p.tokens_per_block, p.tokens - t0);
    const int h0 = blockIdx.y * p.heads_per_block, nh = min(p.heads_per_block, p.heads - h0);
    const int items = nt * nh * p.per_head, half = p.rot / 2;
    const int it0 = threadIdx.x;
    float a[E], b[E];
    Item r = {};
    if (it0 < items) {
        r = item_at<E>(p, it0, t0, h0, nh);
        const size_t x = (size_t)r.tok * p.ldx + (size_t)r.head * p.hsx;
        if (r.rotated || p.copy_tail) {
            load_piece<DT, E>(p.X, x + r.o0, a);
            if (r.two) load_piece<DT, E>(p.X, x + r.o1, b);
        }
    }
    for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
        const int t = i / half;
        const double turns = (double)p.positions[t0 + t] * p.inv_freq[i - t * half] * 0.15915494309189533577;
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        turn[i] = make_float2(p.mscale * c, p.mscale * s);
    }
    __syncthreads();
    for (int it = it0; it < items; it += blockDim.x) {
        if (it != it0) {
            r = item_at<E>(p, it, t0, h0, nh);
            const size_t x = (size_t)r.tok * p.ldx + (size_t)r.head * p.hsx;
            if (r.rotated || p.copy_tail) {
                load_piece<DT, E>(p.X, x + r.o0, a);
                if (r.two) load_piece<DT, E>(p.X, x + r.o1, b);
            }
        }
        const size_t y = (size_t)r.tok * p.ldy + (size_t)r.head * p.hsy;
        if (r.rotated) {
            const float2* cs = turn + (r.tok - t0) * half + r.pair;
            if (E > 1 && p.interleaved) {
                // pieces hold pairs (2k, 2k+1): E/2 pairs each
#pragma unroll
                for (int k = 0; k < E / 2; ++k) {
                    const float2 u = cs[k], w = cs[E / 2 + k];
                    const float a0 = a[2 * k], a1 = a[2 * k + 1], b0 = b[2 * k], b1 = b[2 * k + 1];
                    a[2 * k] = a0 * u.x - a1 * u.y;
                    a[2 * k + 1] = a1 * u.x + a0 * u.y;
                    b[2 * k] = b0 * w.x - b1 * w.y;
                    b[2 * k + 1] = b1 * w.x + b0 * w.y;
                }
            } else {
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const float2 u = cs[k];
                    const float a0 = a[k], b0 = b[k];
                    a[k] = a0 * u.x - b0 * u.y;
                    b[k] = b0 * u.x + a0 * u.y;
                }
            }
        } else if (!p.copy_tail) {
            continue;
        }
        store_piece<DT, E>(p.Y, y + r.o0, a);
        if (r.two) store_piece<DT, E>(p.Y, y + r.o1, b);
    }
}

}  // namespace w4r
