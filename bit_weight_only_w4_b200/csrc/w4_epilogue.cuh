// w4_epilogue.cuh -- epilogue arithmetic of the W4A16 product: bias, activation, gate and
// residual applied to the fp32 sums before their one rounding to the output type.
//
//   t[m,n] = sum_k X'[m,k] What[n,k] + bias[n]
//   plain:  Y[m,n] = act(t[m,n]) + residual[m,n]
//   gated:  packed rows alternate in blocks of 8 gate rows and 8 up rows, so output column
//           f = 8 b + r has its gate in packed row 16 b + r and its up in row 16 b + 8 + r:
//           Y[m,f] = act(t[m, 16 b + r]) * t[m, 16 b + 8 + r] + residual[m,f]
// Blocks of 8 rows, because both matrix paths hold rows r and r + 8 of a 16-row tile in
// one place: the two row halves of a warp MMA's accumulator are registers of one thread
// (decode), and 16 consecutive staged rows are one thread's 16-byte output piece
// (prefill).  Halves [gate; up] would put the two values into different CTAs.
#pragma once
#include "w4_common.cuh"

namespace w4e {

enum : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

struct Epilogue {
    const void* bias;       // [N] in packed row order, or null
    const void* residual;   // [M, N_out], rows ldr apart, or null
    long long ldr, ldy;     // elements between rows of the residual and of Y
    int bias_dtype, res_dtype;
    int act, gated;
};

// Plain loads, not the read-only path: the residual may be Y itself, or the output of a
// kernel that this one overlaps up to griddepcontrol.wait.
W4_DEV float load_elem(const void* p, int dtype, size_t i) {
    if (dtype == 2) return reinterpret_cast<const float*>(p)[i];
    if (dtype == 1) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(reinterpret_cast<const __half*>(p)[i]);
}

// One fp32 activation.
//   none, relu  x, not below `low` (-inf, 0; NaN stays NaN)
//   silu        x / (1 + e^-x)
//   gelu_tanh   x/2 (1 + tanh w) = x / (1 + e^-2w),  2w = sqrt(8/pi) (x + 0.044715 x^3): the
//               same form as silu with another argument u
//   gelu        x Phi(x) = x/2 erfc(-x / sqrt 2)      (erfc keeps the negative tail's digits)
// Two forms of the second kind.  Short: the hardware's 2^x of u log2 e rounded, whose error
// grows with |u| to 2^-17 of the result, still far below the rounding to a 16-bit Y; for prompts
// with a 16-bit Y, where every instruction of the drain counts.  Full: what the rounding of
// u log2 e left out (of the product, by fma, and of the constant) is multiplied back in, so the
// exponential is within a few ulp for every u; for an fp32 Y, and for decode, where outputs are
// few.
enum : int { kKindClamp = 0, kKindSigmoid = 1, kKindErf = 2, kKindSigmoidFull = 3 };
template <int K>
struct KindOf {
    static constexpr int value = K;
};

struct Act {
    int kind;
    float a, c;   // clamp: a = low; sigmoid: argument x (a + c x^2)
    W4_DEV explicit Act(int act) {
        kind = act == kActNone || act == kActRelu ? kKindClamp : act == kActGelu ? kKindErf : kKindSigmoid;
        a = act == kActNone ? -INFINITY : act == kActRelu ? 0.0f : act == kActSilu ? 1.0f : 1.5957691216057308f;
        c = act == kActGeluTanh ? 1.5957691216057308f * 0.044715f : 0.0f;
    }
    template <int K>
    W4_DEV float apply(float x) const {
        if constexpr (K == kKindClamp) return x < a ? a : x;
        else if constexpr (K == kKindErf) return 0.5f * x * erfcf(-0.70710678118654752f * x);
        // for e^-u beyond 2^126 the quotient is below 2^-100: __fdividef's zero there is right
        // (fminf: with c = 0 an infinite x makes the argument's factor NaN; activate(inf) is inf)
        else if constexpr (K == kKindSigmoid)
            return __fdividef(x, 1.0f + __expf(-x * fminf(fmaf(c * x, x, a), 3.0e38f)));
        else return __fdividef(x, 1.0f + exp_of_argument(x));
    }
    // e^-u, u the argument of x; x beyond 104 either way counts as 104, where e^-u is already
    // infinite, or nothing beside 1
    W4_DEV float exp_of_argument(float x) const {
        constexpr float kLog2e = 1.44269502f, kRest = 1.925963e-8f, kLn2 = 0.693147182f;   // log2 e = kLog2e + kRest
        const float y = fminf(fmaxf(x, -104.0f), 104.0f);
        const float v = -y * fmaf(c * y, y, a);
        const float t = v * kLog2e, rest = fmaf(v, kRest, fmaf(v, kLog2e, -t));
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
        return e * fmaf(rest, kLn2, 1.0f);
    }
};
W4_DEV float activate(const Act& act, float x) {
    if (act.kind == kKindSigmoid) return act.apply<kKindSigmoidFull>(x);
    if (act.kind == kKindErf) return act.apply<kKindErf>(x);
    return act.apply<kKindClamp>(x);
}

}  // namespace w4e
