// w4_attention.cuh -- attention of packed prompts (or of their next tokens over earlier
// keys) on the 5th-generation tensor cores.
//
//   O[t,h] = sum_j p_j V[j,hk] / sum_j p_j,   p_j = exp(scale Q[t,h] . K[j,hk]),  hk = h / G
// over the keys j of the token's own sequence that its position sees.  Query i of a
// sequence with nq queries and nk keys sees, when causal, keys j <= i + nk - nq (positions
// aligned at the sequence's end), else all nk.  One pass over the keys with the running
// maximum and sum of the softmax; all statistics and sums in fp32.
//
// A tile's 128 rows are tokens x the G query heads that share a key head (row = token * G +
// head in the group), so a K or V tile in shared memory serves G heads, the causal
// diagonal is only 128 / G tokens wide, and one token of many sequences still fills rows.
// A CTA (one per SM) takes a pair of tiles, 384 threads:
//   warps 0-3, 4-7  softmax of tile A, B: a thread owns one row of S (tensor memory lane);
//   warp 8          TMA: Q of both tiles, then K and V tiles of 128 keys through a ring;
//   warp 9          issues tcgen05.mma: S = Q K^T (128 x 128), O += P V; the two tiles take
//                   turns, so one tile's softmax runs beside the other's products;
//   warps 10-11     make the V tiles of masked key blocks finite (below).
// P (16-bit) replaces the first half of S in tensor memory and is the A operand of P V.
// The running maximum used in the exponent is only raised when the row's maximum passes it
// by 8 (in powers of two): sums grow by at most 2^8, nothing is lost in fp32, and O is
// rescaled a few times a row instead of once a key block.
//
// Masked keys: their scores are replaced (not shifted) before the maximum.  A masked key's
// P is 0, but 0 * V is NaN for an infinite or NaN V, so in key blocks that hold a masked
// key the spare warps zero V's rows behind the sequence's end and its other non-finite
// values, and rows that do see such a value get it added in the epilogue.
#pragma once
#include "w4_common.cuh"
#include "w4_prefill.cuh"

namespace w4t {

constexpr int kRows = 128;      // rows of a tile (tensor memory lanes)
constexpr int kKeys = 128;      // keys of a block
constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 208, kRegsOther = 88, kLaunchRegs = 168;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * kLaunchRegs, "register split");
constexpr float kLazy = 8.0f;   // powers of two by which a row may pass its reference maximum

template <int DP>
struct Cfg {
    static constexpr int q_tile = kRows * DP * 2;
    static constexpr int kv_tile = kKeys * DP * 2;
    static constexpr int stages = DP == 128 ? 5 : 10;
    static constexpr int q = 0;
    static constexpr int ring = 2 * q_tile;
    static constexpr int bars = ring + stages * kv_tile;
    // full, empty, raw, fixed (per stage); q full; per tile: s full, p full, o done; all done
    static constexpr int nbars = 4 * stages + 1 + 3 * 2 + 1;
    static constexpr int misc = bars + nbars * 8;
    static constexpr int bytes = misc + 64 + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory");
};

struct AttnParams {
    const int32_t* cu_q;     // [batch + 1]
    const int32_t* cu_k;     // [batch + 1]
    const void* V;           // for the epilogue's repair only
    void* O;
    float* lse;              // [total_q, heads] or null
    long long ldv, hsv, ldo, hso;
    int batch, heads, kv_heads, group, dim;
    int total_q, total_k;
    int tpt;                 // tokens of a tile: 128 / group
    int causal;
    float scale, scale_log2; // scale, scale * log2 e
};

// One CTA's work: a pair of tiles of one sequence and key head.
struct Work {
    int valid;
    int q0, nq;      // first token of the sequence, its tokens
    int k0, nk;      // first key of the sequence, its keys
    int tok;         // first token (in the sequence) of the pair
    int hk;          // key head
};

// First element and length of sequence b; bounds outside [0, total] are clamped (bad).  A
// null cu is one sequence of everything.
W4_DEV void seq_bounds(const int32_t* cu, int total, int b, int& s, int& n, bool& bad) {
    if (!cu) {
        s = 0;
        n = total;
        return;
    }
    const int a = __ldg(cu + b), e = __ldg(cu + b + 1);
    s = max(0, min(a, total));
    const int t = max(s, min(e, total));
    n = t - s;
    bad |= a < 0 || e < a || e > total;
}

// Pairs of all sequences in descending order of their index in the sequence (with causal
// masks, of their cost), so the long ones start first: pair `idx` by a search for the
// level p with f(p) > idx >= f(p + 1), f(p) = sum_b max(0, pairs of b - p).  Run by one warp.
W4_DEV Work find_work(const AttnParams& p, int idx, int hk, int lane) {
    const int tp = 2 * p.tpt;
    auto count = [&](int level) {
        int c = 0;
        for (int b = lane; b < p.batch; b += 32) {
            int s, n;
            bool bad = false;
            seq_bounds(p.cu_q, p.total_q, b, s, n, bad);
            c += max(0, (n + tp - 1) / tp - level);
        }
        return __reduce_add_sync(0xffffffffu, c);
    };
    Work w = {};
    if (count(0) <= idx) return w;
    int lo = 0, hi = p.total_q / tp + 1;   // f(lo) > idx >= f(hi)
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (count(mid) > idx) lo = mid;
        else hi = mid;
    }
    int rank = idx - count(lo + 1);   // among the sequences with more than lo pairs
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const int b = b0 + lane;
        int s = 0, n = 0;
        bool bad = false;
        if (b < p.batch) seq_bounds(p.cu_q, p.total_q, b, s, n, bad);
        const unsigned has = __ballot_sync(0xffffffffu, (n + tp - 1) / tp > lo);
        const int c = __popc(has);
        if (rank >= c) {
            rank -= c;
            continue;
        }
        const int src = __fns(has, 0, rank + 1);
        w.valid = 1;
        w.q0 = __shfl_sync(0xffffffffu, s, src);
        w.nq = __shfl_sync(0xffffffffu, n, src);
        bad = false;
        seq_bounds(p.cu_k, p.total_k, b0 + src, w.k0, w.nk, bad);
        w.tok = lo * tp;
        w.hk = hk;
        break;
    }
    return w;
}

// Keys (from the sequence's first) that some row of tile x sees, and that every row sees.
W4_DEV int tile_keys(const AttnParams& p, const Work& w, int x) {
    const int t0 = w.tok + x * p.tpt, t1 = min(t0 + p.tpt, w.nq);
    if (t0 >= w.nq) return 0;
    return p.causal ? max(0, min(w.nk, t1 + w.nk - w.nq)) : w.nk;
}
W4_DEV int common_keys(const AttnParams& p, const Work& w) {
    return p.causal ? max(0, min(w.nk, w.tok + 1 + w.nk - w.nq)) : w.nk;
}

// The row of this softmax thread.
struct Row {
    int tok, head, limit;   // token in the sequence, query head, keys the row sees
    bool live;              // the row is a token of the sequence
};
W4_DEV Row row_of(const AttnParams& p, const Work& w, int x) {
    const int row = threadIdx.x & (kRows - 1);
    Row r;
    r.tok = w.tok + x * p.tpt + row / p.group;
    r.head = w.hk * p.group + row % p.group;
    r.live = w.valid && row < p.tpt * p.group && r.tok < w.nq;
    r.limit = !r.live ? 0 : p.causal ? max(0, min(w.nk, r.tok + 1 + w.nk - w.nq)) : w.nk;
    return r;
}
W4_DEV Work reload(const volatile Work* s) {
    Work w;
    w.valid = s->valid;
    w.q0 = s->q0;
    w.nq = s->nq;
    w.k0 = s->k0;
    w.nk = s->nk;
    w.tok = s->tok;
    w.hk = s->hk;
    return w;
}

// ---------------------------------------------------------------- tensor memory
W4_DEV void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
W4_DEV void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
W4_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
W4_DEV void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
W4_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory descriptors are passed as their two 32-bit words: the upper one (strides,
// version, swizzle) is a constant, the lower one holds the address.
// D[tmem] (+)= A[smem desc] * B[smem desc]^T, kind::f16.
W4_DEV void tc_mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16.
W4_DEV void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// V tile as the N x K operand with N (the head dimension) contiguous: chunks of 64 columns
// (128-byte swizzled lines, one a key) lie kKeys * 128 bytes apart (leading offset), groups
// of 8 keys 1024 bytes apart (stride offset).
W4_DEV uint64_t sw128_desc_mn(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((kKeys * 128) >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// fp32 accumulator, fp16 or bf16 operands, 128 x n; b_mn: the B operand's N is contiguous.
W4_DEV uint32_t attn_idesc(bool bf16, int n, bool b_mn) {
    const uint32_t fmt = bf16 ? 1u : 0u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kRows >> 4) << 24);
}

W4_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

using w4p::wait_or_abort;

template <bool BF16, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const AttnParams p) {
    using C = Cfg<DP>;
    constexpr int NC = DP / 64;    // 64-column chunks of a head
    constexpr int S = C::stages;
    // fp16 keeps 2^-14 as its smallest normal: P is scaled by 2^6 so that weights down to
    // 2^-20 of the row's largest keep all their digits (at most 2^(6 + 8) < 65504)
    constexpr float kShift = BF16 ? 0.0f : 6.0f;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = align_smem_1024(smem_raw);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bars);
    uint64_t* empty = full + S;
    uint64_t* raw = empty + S;       // a V tile of a masked block has landed,
    uint64_t* fixed = raw + S;       // ... and is finite (these tiles do not signal `full`)
    uint64_t* q_full = fixed + S;
    uint64_t* s_full = q_full + 1;      // [2]
    uint64_t* p_full = s_full + 2;      // [2]
    uint64_t* o_done = p_full + 2;      // [2]
    uint64_t* all_done = o_done + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc + 4);
    volatile int* poison = reinterpret_cast<volatile int*>(smem + C::misc + 8);
    Work* s_work = reinterpret_cast<Work*>(smem + C::misc + 16);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&raw[s], 1);
            mbar_init(&fixed[s], 64);
        }
        mbar_init(q_full, 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 128);
            mbar_init(&o_done[x], 1);
        }
        mbar_init(all_done, 1);
        *abort_flag = 0;
        *poison = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        w4p::tmem_alloc(tmem_slot, 512);
        w4p::tmem_relinquish();
    }
    if (warp == 8 && lane == 0) {
        prefetch_tensormap(&tmap_q);
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    pdl_launch_dependents();
    pdl_wait();   // everything read below may come from the preceding kernel
    if (warp == 0) {
        const Work w = find_work(p, blockIdx.x / p.kv_heads, blockIdx.x % p.kv_heads, lane);
        if (lane == 0) *s_work = w;
        if (blockIdx.x == 0) {
            bool bad = false;
            for (int b = lane; b < p.batch; b += 32) {
                int s, n;
                seq_bounds(p.cu_q, p.total_q, b, s, n, bad);
                seq_bounds(p.cu_k, p.total_k, b, s, n, bad);
            }
            if (bad) atomicOr(&g_w4_error_word, W4_DEVERR_GIDX);
        }
    }
    w4p::tc_fence_before();
    __syncthreads();
    w4p::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Work w = *s_work;
    const int nkeys[2] = {tile_keys(p, w, 0), tile_keys(p, w, 1)};
    const int nb0 = w.valid ? (nkeys[0] + kKeys - 1) / kKeys : 0;
    const int nb1 = w.valid ? (nkeys[1] + kKeys - 1) / kKeys : 0;
    const int nb = max(nb0, nb1);
    // blocks from mfirst on hold a key that some row of the pair does not see
    const int mfirst = common_keys(p, w) / kKeys;

    if (warp >= 8) {
        w4p::setmaxnreg_dec<kRegsOther>();
        if (warp == 8) {
            // ---------------------------------------------------------- TMA producer
            if (lane == 0 && nb > 0) {
                const int nq = (nb0 > 0 ? 1 : 0) + (nb1 > 0 ? 1 : 0);
                mbar_arrive_expect_tx(q_full, nq * NC * 128 * p.group * p.tpt);
                for (int x = 0; x < 2; ++x) {
                    if ((x ? nb1 : nb0) == 0) continue;
                    for (int c = 0; c < NC; ++c)
                        tma_load_3d(smem + C::q + x * C::q_tile + c * kRows * 128, &tmap_q, 64 * c, w.hk * p.group,
                                    w.q0 + w.tok + x * p.tpt, q_full);
                }
                // ring order: K_0, V_0, K_1, V_1, ...  Each barrier completes once a use, so
                // its parity is a bit that its users flip at each use.
                uint32_t full_ph = 0, raw_ph = 0, last_raw = 0;   // a bit a stage
                int i = 0;
                for (; i < 2 * nb; ++i) {
                    const int s = i % S;
                    if (i >= S && !wait_or_abort(&empty[s], ((i / S) & 1) ^ 1, abort_flag)) break;
                    const bool is_raw = (i & 1) && i / 2 >= mfirst;
                    uint64_t* bar = is_raw ? &raw[s] : &full[s];
                    if (is_raw) raw_ph ^= 1u << s;
                    else full_ph ^= 1u << s;
                    last_raw = (last_raw & ~(1u << s)) | ((is_raw ? 1u : 0u) << s);
                    mbar_arrive_expect_tx(bar, C::kv_tile);
                    for (int c = 0; c < NC; ++c)
                        tma_load_3d(smem + C::ring + s * C::kv_tile + c * kKeys * 128, (i & 1) ? &tmap_v : &tmap_k, 64 * c,
                                    w.hk, w.k0 + (i / 2) * kKeys, bar);
                }
                if (*abort_flag) {
                    // the copies in flight land before the block ends
                    (void)mbar_wait(q_full, 0);
                    for (int s = 0; s < min(S, i); ++s) {
                        const bool r = (last_raw >> s) & 1u;
                        (void)mbar_wait(r ? &raw[s] : &full[s], (((r ? raw_ph : full_ph) >> s) & 1u) ^ 1u);
                    }
                }
            }
            __syncwarp();
        } else if (warp == 9) {
            // ---------------------------------------------------------- MMA issuer
            const bool leader = elect_one();
            const uint32_t idesc_s = attn_idesc(BF16, kKeys, false), idesc_o = attn_idesc(BF16, DP, true);
            // descriptors: K-major tiles and V differ in the lower word's leading offset only
            const uint32_t hi = (uint32_t)(w4p::sw128_desc(0) >> 32);
            const uint32_t qd0 = (uint32_t)w4p::sw128_desc(smem_u32(smem + C::q));
            const uint32_t kd0 = (uint32_t)w4p::sw128_desc(smem_u32(smem + C::ring));
            const uint32_t vd0 = (uint32_t)sw128_desc_mn(smem_u32(smem + C::ring));
            uint32_t full_ph = 0, fixed_ph = 0;   // a bit a stage
            auto wait_bit = [&](uint64_t* bars, uint32_t& ph, int s) {
                const bool r = wait_or_abort(&bars[s], (ph >> s) & 1u, abort_flag);
                ph ^= 1u << s;
                return __all_sync(0xffffffffu, r) != 0;
            };
            auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
            // S_x = Q_x K^T with the K tile of ring position i
            auto issue_s = [&](int x, int i) {
                if (!leader) return;
                const uint32_t qd = qd0 + ((x * C::q_tile) >> 4);
                const uint32_t kd = kd0 + (((i % S) * C::kv_tile) >> 4);
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_ss(tmem + 128 * x, qd + ((c * kRows * 128 + 32 * k) >> 4),
                                  kd + ((c * kKeys * 128 + 32 * k) >> 4), hi, idesc_s, (c | k) ? 1u : 0u);
                w4p::tc_commit(&s_full[x]);
            };
            bool ok = nb > 0;
            if (ok) {
                ok = all(wait_or_abort(q_full, 0, abort_flag)) && wait_bit(full, full_ph, 0);
                w4p::tc_fence_after();
                if (ok) {
                    if (nb0 > 0) issue_s(0, 0);
                    if (nb1 > 0) issue_s(1, 0);
                    if (leader) w4p::tc_commit(&empty[0]);
                }
            }
            for (int j = 0; j < nb && ok; ++j) {
                const int iv = 2 * j + 1, ik = 2 * j + 2;   // ring positions of V_j and K_{j+1}
                const int sv = iv % S;
                ok = j >= mfirst ? wait_bit(fixed, fixed_ph, sv) : wait_bit(full, full_ph, sv);
                if (!ok) break;
                if (j + 1 < nb) ok = wait_bit(full, full_ph, ik % S);
                if (!ok) break;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int n = x ? nb1 : nb0;
                    if (j < n) {
                        ok = ok && all(wait_or_abort(&p_full[x], j & 1, abort_flag));
                        if (!ok) break;
                        w4p::tc_fence_after();
                        if (leader) {
                            const uint32_t vd = vd0 + ((sv * C::kv_tile) >> 4);
#pragma unroll
                            for (int k = 0; k < kKeys / 16; ++k)
                                tc_mma_ts(tmem + 256 + DP * x, tmem + 128 * x + 8 * k, vd + ((2048 * k) >> 4), hi, idesc_o,
                                          (j | k) ? 1u : 0u);
                            w4p::tc_commit(&o_done[x]);
                        }
                    }
                    if (j + 1 < n) issue_s(x, ik);
                }
                if (!ok) break;
                if (leader) {
                    w4p::tc_commit(&empty[sv]);
                    if (j + 1 < nb) w4p::tc_commit(&empty[ik % S]);
                }
            }
            if (leader) w4p::tc_commit(all_done);
            (void)mbar_wait(all_done, 0);
            __syncwarp();
        } else {
            // ---------------------------------------------------------- V of masked blocks
            const int t = (warp - 10) * 32 + lane;
            uint32_t raw_ph = 0;
            for (int j = mfirst; j < nb; ++j) {
                const int s = (2 * j + 1) % S;
                if (!wait_or_abort(&raw[s], (raw_ph >> s) & 1u, abort_flag)) break;
                raw_ph ^= 1u << s;
                const int left = w.nk - j * kKeys;   // keys of the block that belong to the sequence
                unsigned char* v = smem + C::ring + s * C::kv_tile;
                bool any = false, wrote = false;
                for (int q = t; q < NC * kKeys * 8; q += 64) {
                    uint4* at = reinterpret_cast<uint4*>(v + q * 16);
                    uint4 d = *at;
                    if (((q >> 3) & (kKeys - 1)) >= left) {
                        *at = make_uint4(0u, 0u, 0u, 0u);
                        wrote = true;
                        continue;
                    }
                    uint32_t e[4] = {d.x, d.y, d.z, d.w};
                    constexpr uint32_t kExp = BF16 ? 0x7F80u : 0x7C00u;
                    bool hit = false;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if ((e[k] & kExp) == kExp) {
                            e[k] &= 0xFFFF0000u;
                            hit = true;
                        }
                        if (((e[k] >> 16) & kExp) == kExp) {
                            e[k] &= 0x0000FFFFu;
                            hit = true;
                        }
                    }
                    if (hit) {
                        *at = make_uint4(e[0], e[1], e[2], e[3]);
                        any = wrote = true;
                    }
                }
                if (any) *poison = 1;
                if (wrote) fence_proxy_async_smem();
                mbar_arrive(&fixed[s]);
            }
        }
    } else {
        // -------------------------------------------------------------- softmax, one row a thread
        w4p::setmaxnreg_inc<kRegsSoftmax>();
        const int x = warp >> 2;
        const int n = x ? nb1 : nb0;
        const int limit = row_of(p, w, x).limit;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + 128 * x, to = tmem + lanes + 256 + DP * x;
        float m = -INFINITY, l = 0.0f;   // reference maximum of the raw scores, sum of the weights
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            ok = __all_sync(0xffffffffu, wait_or_abort(&s_full[x], j & 1, abort_flag));
            if (!ok) break;
            w4p::tc_fence_after();
            uint32_t sr[8][16];
#pragma unroll
            for (int c = 0; c < 8; ++c) tmem_ld16_async(ts + 16 * c, sr[c]);
            tmem_wait_ld();
            if (j >= mfirst) {
                const int lim = limit - j * kKeys;
#pragma unroll
                for (int c = 0; c < 8; ++c)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (16 * c + i >= lim) sr[c][i] = 0xFF800000u;
            }
            float bm = -INFINITY;
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) bm = fmaxf(bm, __uint_as_float(sr[c][i]));
            // (NaN compares false: such a row keeps its reference and ends as NaN)
            const bool raise = m == -INFINITY ? bm > m : (bm - m) * p.scale_log2 > kLazy;
            if (__any_sync(0xffffffffu, raise)) {
                const float nm = raise ? bm : m;
                const float f = raise ? ex2((m - nm) * p.scale_log2) : 1.0f;
                if (j > 0) {
                    // O is complete up to block j - 1 (its P V must be done), then rescaled
                    ok = __all_sync(0xffffffffu, wait_or_abort(&o_done[x], (j - 1) & 1, abort_flag));
                    if (!ok) break;
                    w4p::tc_fence_after();
#pragma unroll
                    for (int c = 0; c < DP / 16; ++c) {
                        uint32_t o[16];
                        tmem_ld16_async(to + 16 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st16(to + 16 * c, o);
                    }
                    tmem_wait_st();
                }
                l *= f;
                m = nm;
            }
            const float base = m == -INFINITY ? 0.0f : kShift - m * p.scale_log2;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t pr[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float a = ex2(fmaf(__uint_as_float(sr[2 * c + (i >> 3)][2 * (i & 7)]), p.scale_log2, base));
                    const float b = ex2(fmaf(__uint_as_float(sr[2 * c + (i >> 3)][2 * (i & 7) + 1]), p.scale_log2, base));
                    sum[2 * (i & 1)] += a;
                    sum[2 * (i & 1) + 1] += b;
                    pr[i] = pack2<BF16>(a, b);
                }
                tmem_st16(ts + 16 * c, pr);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_wait_st();
            w4p::tc_fence_before();
            mbar_arrive(&p_full[x]);
        }
        // epilogue
        if (n > 0 && ok) ok = __all_sync(0xffffffffu, wait_or_abort(&o_done[x], (n - 1) & 1, abort_flag));
        w4p::tc_fence_after();
        if (ok) {
            // read again: kept in registers through the loop, these would not fit
            const Work w = reload(s_work);
            const Row r = row_of(p, w, x);
            const int tok = r.tok, head = r.head, limit = r.limit;
            const bool live = r.live;
            const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
            const size_t at = (size_t)(w.q0 + tok) * p.ldo + (size_t)head * p.hso;
            unsigned short* O = reinterpret_cast<unsigned short*>(p.O);
            const int bad = *poison;
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
                uint32_t o[32];
                __syncwarp();
                if (n > 0) {
                    tmem_ld32_async(to + 32 * c, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
                if (live) {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(l == 0.0f ? 0.0f : __uint_as_float(o[i]) * inv);
                if (bad) {
                    // non-finite values that the spare warps took out of V, for the rows that see them
                    for (int j = mfirst * kKeys; j < limit; ++j) {
                        const unsigned short* v = reinterpret_cast<const unsigned short*>(p.V) +
                                                  (size_t)(w.k0 + j) * p.ldv + (size_t)w.hk * p.hsv + 32 * c;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (32 * c + i >= p.dim) break;
                            const uint32_t b = v[i];
                            const float f = BF16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((unsigned short)b));
                            if (!isfinite(f)) o[i] = __float_as_uint(__uint_as_float(o[i]) + f);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (32 * c + 8 * i >= p.dim) break;
                    uint32_t e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        e[k] = pack2<BF16>(__uint_as_float(o[8 * i + 2 * k]), __uint_as_float(o[8 * i + 2 * k + 1]));
                    *reinterpret_cast<uint4*>(O + at + 32 * c + 8 * i) = make_uint4(e[0], e[1], e[2], e[3]);
                }
                }
            }
            if (live && p.lse) {
                const float v = l == 0.0f ? -INFINITY : m * p.scale + (logf(l) - kShift * 0.69314718055994531f);
                p.lse[(size_t)(w.q0 + tok) * p.heads + head] = v;
            }
        }
    }
    w4p::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        w4p::tc_fence_after();
        w4p::tmem_dealloc(tmem, 512);
    }
}

}  // namespace w4t
