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
// An item of work is a pair of tiles A, B of one sequence and key head over the same key
// blocks, or (when pairs would leave SMs idle) one tile, whose even key blocks are A's and
// odd ones B's: two partial softmaxes of the same rows, joined at the item's end straight
// from tensor memory.  One CTA an SM, 384 threads, takes items until there are none; the
// roles run ahead of one another through barriers, so the loads and the first products of
// the next item overlap the end of this one:
//   warps 0-3, 4-7  softmax of A, B: a thread owns one row of S (tensor memory lane), then the
//                   item's output;
//   warp 8          loads Q, then K and V tiles of 128 keys through a ring;
//   warp 9          issues tcgen05.mma: S = Q K^T (128 x 128), O += P V; the two tiles take
//                   turns, so one tile's softmax runs beside the other's products;
//   warp 10         finds the items, one ahead (warp 11 only fills the warpgroup).
// P (16-bit) replaces the first half of S in tensor memory and is the A operand of P V.
// The running maximum used in the exponent is only raised when the row's maximum passes it
// by 8 (in powers of two): sums grow by at most 2^8, nothing is lost in fp32, and O is
// rescaled a few times a row instead of once a key block.
//
// What bounds it: a pair of 128 x 128 blocks takes 4 x 512 cycles of the tensor cores and
// 32768 exponentials, 2048 cycles at 16 a cycle and SM; but a tile's next S waits for its P V
// (tensor memory holds two S and two O tiles, no third S), so a block's softmax is also part
// of the loop's latency.  Handing P on by halves takes a quarter of P V out of that latency
// (8192 tokens, 32/8 heads: 461 -> 447 us).  Tried and slower: half-size S tiles, two a
// tile (540 us: a 128 x 64 product costs as much as a 128 x 128 one), and an eighth, a quarter
// or a third of the exponentials as a polynomial on the FMA units (456, 467, 472 us); a fourth
// warpgroup for the output beside softmax warps of 184 registers (457 us, and packed prompts
// 187 against 173).  As it stands: 436 us (1261 TFLOP/s) in a few calls on a cool board, 500 to 510 us
// (1090) in a long run, which the board's power bounds.
//
// Two ways to share the work:
//   items    by their place in the sequence, last ones first, one CTA an item; a running CTA takes
//            the place of one that has not started (cluster launch control), so the hardware
//            balances their lengths.  Under a causal mask without earlier keys that is longest
//            first.  A sequence of few tokens over many earlier keys comes late, and its keys are
//            not cut: 2000 tokens packed with 15 next tokens over 60,000 keys each (64/8 heads)
//            take 820 us, in calls of their own 76 and 569;
//   ranges   (few tokens over many keys) all key blocks of all items in one list, cut into
//            equal runs, one a CTA: every SM reads the same number of keys whatever the
//            sequences' lengths.  An item that a cut divides is written as partial outputs
//            (at most two a CTA) and joined by combine_kernel.
//
// Masked keys: their scores are replaced (not shifted) before the maximum.  A masked key's
// P is 0, but 0 * V is NaN for an infinite or NaN V.  So before the P V of a block that holds
// a masked key the softmax warps, while they wait for its S, look through the V rows of the
// keys that not every row sees: rows that no row sees become zero, other non-finite values
// zero too, and the rows that do see such a value get it added to their output.
#pragma once
#include <climits>

#include "w4_common.cuh"
#include "w4_prefill.cuh"

namespace w4t {

constexpr int kRows = 128;      // rows of a tile (tensor memory lanes)
constexpr int kKeys = 128;      // keys of a block (a K or V tile of the ring)
constexpr int kSub = 64;        // keys of half a block: P is handed on, and masked keys left out, by halves
constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 216, kRegsOther = 72, kLaunchRegs = 168;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * kLaunchRegs, "register split");
constexpr float kLazy = 8.0f;   // powers of two by which a row may pass its reference maximum

constexpr int kItems = 2;       // the item at work and the next one

template <int DP>
struct Cfg {
    static constexpr int q_tile = kRows * DP * 2;
    static constexpr int kv_tile = kKeys * DP * 2;
    static constexpr int stages = DP == 128 ? 4 : 8;
    static constexpr int q = 0;
    static constexpr int ring = 2 * q_tile;
    static constexpr int out = ring + stages * kv_tile;     // 4 KB a softmax warp
    static constexpr int bars = out + 8 * 4096;
    // full, empty, raw, fixed (per stage); item full, empty; q full, empty; of A and B: s full,
    // p full (per half of a block), o done; next item, its wish; all done; both ready, read
    static constexpr int nbars = 4 * stages + 2 * kItems + 2 + 2 + 4 + 2 + 5;
    static constexpr int next = (bars + nbars * 8 + 15) / 16 * 16;   // cluster launch control's answer
    static constexpr int items = next + 16;
    static constexpr int misc = items + kItems * 64;
    static constexpr int stats = q + q_tile;   // one tile: (m, l) of A's and B's rows, where Q of tile B would be
    static constexpr int bytes = misc + 16 + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory");
};

struct AttnParams {
    const int32_t* cu_q;     // [batch + 1]
    const int32_t* cu_k;     // [batch + 1]
    const void* V;           // for the output's repair only
    void* O;
    float* lse;              // [total_q, heads] or null
    float* part_o;           // ranges: partial outputs [2 a CTA][128 rows][dim] fp32; null for items
    float* part_lse;         // [2 a CTA][128 rows]
    long long ldv, hsv, ldo, hso;
    int batch, heads, kv_heads, group, dim;
    int total_q, total_k;
    int tpt;                 // tokens of a tile: 128 / group
    int tiles;               // tiles of an item: 1 or 2
    int ctas;                // ranges: their number
    int causal;
    int tma_out;             // a warp's 32 rows are whole tokens: O goes out by TMA
    float scale, scale_log2; // scale, scale * log2 e
};

// An item (or the part of one in a CTA's range): tiles of one sequence and key head.
struct Work {
    int valid;
    int q0, nq;      // first token of the sequence, its tokens
    int k0, nk;      // first key of the sequence, its keys
    int tok;         // first token (in the sequence) of the item
    int hk;          // key head
    int part;        // partial output it writes, or -1: the output itself
    int b0;          // first key block
    int sub0, sub1;  // half blocks of A, of B (one tile: blocks alternate, only the last may be half)
    int common;      // keys (from block b0) that every row sees
    int seen;        // keys (from block b0) that some row sees
    int poison;      // set when a non-finite value was taken out of V
};
static_assert(sizeof(Work) <= 64, "item slot");

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

// Tiles x rows of an item, as tokens.
W4_DEV int item_tokens(const AttnParams& p) { return p.tiles * p.tpt; }

// Fills in what tile `tok` of a sequence does over its key blocks [from, to).
W4_DEV void fill_work(const AttnParams& p, Work& w, int from, int to) {
    // keys that a row sees whose token is `last`
    auto sees = [&](int last) { return p.causal ? max(0, min(w.nk, last + 1 + w.nk - w.nq)) : w.nk; };
    auto subs = [&](int t0) {   // of the tile that starts at token t0, in [from, to)
        const int keys = t0 >= w.nq ? 0 : min(sees(min(t0 + p.tpt, w.nq) - 1), to * kKeys);
        return max(0, keys - from * kKeys + kSub - 1) / kSub;
    };
    const int n0 = subs(w.tok);
    w.valid = 1;
    w.b0 = from;
    if (p.tiles == 2) {
        w.sub0 = n0;
        w.sub1 = subs(w.tok + p.tpt);
    } else {
        const int nb = (n0 + 1) / 2, short_last = n0 & 1;
        w.sub0 = 2 * ((nb + 1) / 2) - (nb & 1 ? short_last : 0);
        w.sub1 = 2 * (nb / 2) - (nb & 1 ? 0 : short_last);
    }
    w.common = max(0, sees(w.tok) - from * kKeys);
    w.seen = sees(min(w.tok + item_tokens(p), w.nq) - 1) - from * kKeys;
}
W4_DEV int blocks_of_subs(int sub) { return (sub + 1) / 2; }

// 32 sequences, one a lane: read once, then handed around by shuffles.
struct Seqs {
    int q0, nq, k0, nk;
    W4_DEV void load(const AttnParams& p, int b) {
        q0 = nq = k0 = nk = 0;
        bool bad = false;
        if (b < p.batch) {
            seq_bounds(p.cu_q, p.total_q, b, q0, nq, bad);
            seq_bounds(p.cu_k, p.total_k, b, k0, nk, bad);
        }
    }
    W4_DEV void give(Work& w, int src) const {
        w.q0 = __shfl_sync(0xffffffffu, q0, src);
        w.nq = __shfl_sync(0xffffffffu, nq, src);
        w.k0 = __shfl_sync(0xffffffffu, k0, src);
        w.nk = __shfl_sync(0xffffffffu, nk, src);
    }
};

// Finds items, by one warp.  The items of all sequences are taken in descending index in
// their sequence (with causal masks and no earlier keys, descending cost): item `idx` is at the level v with
// f(v) > idx >= f(v + 1), f(v) = sum_b max(0, items of b - v), found by bisection.
struct Finder {
    Seqs seqs;       // the first 32
    int mine;        // items of this lane's first sequence
    int top, total;  // the most items of any sequence, all items
    W4_DEV static int items_of(const AttnParams& p, int b) {
        int s, n;
        bool bad = false;
        seq_bounds(p.cu_q, p.total_q, b, s, n, bad);
        return (n + item_tokens(p) - 1) / item_tokens(p);
    }
    W4_DEV void start(const AttnParams& p, int lane) {
        seqs.load(p, lane);
        int most = mine = (seqs.nq + item_tokens(p) - 1) / item_tokens(p);
        total = mine;
        for (int b = lane + 32; b < p.batch; b += 32) {
            const int n = items_of(p, b);
            most = max(most, n);
            total += n;
        }
        top = __reduce_max_sync(0xffffffffu, most);
        total = __reduce_add_sync(0xffffffffu, total);
    }
    W4_DEV int count(const AttnParams& p, int level, int lane) const {
        int c = max(0, mine - level);
        for (int b = lane + 32; b < p.batch; b += 32) c += max(0, items_of(p, b) - level);
        return __reduce_add_sync(0xffffffffu, c);
    }
    W4_DEV Work find(const AttnParams& p, int item, int lane) const {
        Work w = {};
        const int idx = item / p.kv_heads;
        if (total <= idx) return w;
        int lo = 0, hi = top;   // f(lo) > idx >= f(hi)
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            if (count(p, mid, lane) > idx) lo = mid;
            else hi = mid;
        }
        int rank = idx - (hi < top ? count(p, hi, lane) : 0);   // among the sequences with more than lo items
        Seqs at = seqs;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            if (b0 > 0) at.load(p, b0 + lane);
            unsigned has = __ballot_sync(0xffffffffu, (at.nq + item_tokens(p) - 1) / item_tokens(p) > lo);
            const int c = __popc(has);
            if (rank >= c) {
                rank -= c;
                continue;
            }
            for (; rank > 0; --rank) has &= has - 1;
            at.give(w, __ffs(has) - 1);
            break;
        }
        w.tok = lo * item_tokens(p);
        w.hk = item - idx * p.kv_heads;
        w.part = -1;
        fill_work(p, w, 0, INT_MAX / kKeys);
        return w;
    }
};

// The list of all key blocks, for ranges: sequences in order; in each the tiles, in each the
// key heads, in each the sequence's key blocks (at least one, so that every row is written).
struct List {
    W4_DEV static int blocks_of(int nk) { return max(1, (nk + kKeys - 1) / kKeys); }
    W4_DEV static long long size(const AttnParams& p, const Seqs& s) {
        return (long long)((s.nq + p.tpt - 1) / p.tpt) * p.kv_heads * blocks_of(s.nk);
    }
    W4_DEV static long long sum(long long n) {
#pragma unroll
        for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
        return n;
    }
    // First block of CTA c's range, and the CTA of a block.
    W4_DEV static long long begin(const AttnParams& p, long long total, int c) {
        return total / p.ctas * c + min((long long)c, total % p.ctas);
    }
    W4_DEV static int cta_of(const AttnParams& p, long long total, long long u) {
        const long long base = total / p.ctas, rem = total % p.ctas;
        return u < rem * (base + 1) ? (int)(u / (base + 1)) : (int)(rem + (u - rem * (base + 1)) / max(1ll, base));
    }
};

// The items of a CTA's range, one after the other, by one warp.
struct Walker {
    long long total;       // blocks of the list
    long long at, end;     // next block of the list, end of the range
    long long ends;        // list index behind this lane's sequence
    Seqs seqs;             // 32 sequences, from b0 on
    int b0;
    // the sequences from b on; `before`: blocks of those before them
    W4_DEV void load(const AttnParams& p, int b, long long before, int lane) {
        b0 = b;
        seqs.load(p, b + lane);
        ends = b + lane < p.batch ? List::size(p, seqs) : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, ends, d);
            if (lane >= d) ends += up;
        }
        ends += before;
    }
    W4_DEV void start(const AttnParams& p, int lane) {
        load(p, 0, 0, lane);
        total = __shfl_sync(0xffffffffu, ends, 31);
        for (int b = 32; b < p.batch; b += 32) {
            Seqs s;
            s.load(p, b + lane);
            total += List::sum(b + lane < p.batch ? List::size(p, s) : 0);
        }
        at = List::begin(p, total, blockIdx.x);
        end = List::begin(p, total, blockIdx.x + 1);
    }
    W4_DEV Work next(const AttnParams& p, int lane) {
        Work w = {};
        if (at >= end) return w;
        long long last = __shfl_sync(0xffffffffu, ends, 31);
        while (at >= last) {   // (at < total, so some sequence holds it)
            load(p, b0 + 32, last, lane);
            last = __shfl_sync(0xffffffffu, ends, 31);
        }
        const int src = __popc(__ballot_sync(0xffffffffu, ends <= at));
        seqs.give(w, src);
        const long long first = __shfl_sync(0xffffffffu, ends - List::size(p, seqs), src);
        const int nb = List::blocks_of(w.nk);
        const int run = (int)((at - first) / nb), from = (int)((at - first) - (long long)run * nb);
        const int to = (int)min((long long)nb, from + (end - at));
        w.tok = run / p.kv_heads * p.tpt;
        w.hk = run % p.kv_heads;
        // a part that starts inside its item is the CTA's first, one that starts the item and
        // does not end it the last: two places a CTA
        w.part = from == 0 && to == nb ? -1 : 2 * (int)blockIdx.x + (from == 0 ? 1 : 0);
        fill_work(p, w, from, to);
        at += to - from;
        return w;
    }
};

// The row of this softmax thread: token in its tile and head in its group (rg, rh) are the same
// for every item.
struct Row {
    int tok, limit;   // token in the sequence, keys the row sees
    bool live;        // the row is a token of the sequence
};
W4_DEV Row row_of(const AttnParams& p, const volatile Work* w, int x, int rg) {
    Row r;
    const int nq = w->nq, nk = w->nk;
    r.tok = w->tok + (p.tiles == 2 ? x * p.tpt : 0) + rg;
    r.live = rg < p.tpt && r.tok < nq;
    r.limit = !r.live ? 0 : p.causal ? max(0, min(nk, r.tok + 1 + nk - nq)) : nk;
    return r;
}

// Add to a row's staged output (16-byte pieces swizzled by the row's lane; columns c0 ..) the
// non-finite values of V that were taken out of the product, for the keys [first, last) that
// the row sees.  Rare: not worth registers or instructions of the common path.
template <bool BF16>
__device__ __noinline__ void repair_row(unsigned char* row, int lane, bool fp32, int c0, int cols, const unsigned short* v,
                                        long long ldv, int keys) {
    for (int j = 0; j < keys; ++j, v += ldv)
        for (int c = 0; c < cols; ++c) {
            const uint32_t b = v[c0 + c];
            const float f = BF16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((unsigned short)b));
            if (isfinite(f)) continue;
            const int byte = c * (fp32 ? 4 : 2);
            unsigned char* at = row + ((((byte >> 4) ^ lane) & 7) << 4) + (byte & 15);
            if (fp32) *reinterpret_cast<float*>(at) += f;
            else if (BF16) *reinterpret_cast<__nv_bfloat16*>(at) = __float2bfloat16_rn(__bfloat162float(*reinterpret_cast<__nv_bfloat16*>(at)) + f);
            else *reinterpret_cast<__half*>(at) = __float2half_rn(__half2float(*reinterpret_cast<__half*>(at)) + f);
        }
}

// Store 64 columns x one warp's rows from swizzled shared memory (box given by the tensor map).
W4_DEV void tma_store_3d(const CUtensorMap* map, const void* src, int32_t c0, int32_t c1, int32_t c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
W4_DEV void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
W4_DEV void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ---------------------------------------------------------------- next item
// Ask for a CTA that has not started yet, in whose place this one carries on; the answer
// (16 bytes) completes on the barrier.
W4_DEV void ask_next(void* answer, uint64_t* bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_u32(answer)),
        "r"(smem_u32(bar))
        : "memory");
}
// Its block index, or -1 when every CTA has started.
W4_DEV int answered(const void* answer) {
    uint32_t x = 0, ok = 0;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\tld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %1, 1, 0, p;\n\tmov.u32 %0, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, _, _, _}, h;\n\t}"
        : "=r"(x), "=r"(ok)
        : "r"(smem_u32(answer))
        : "memory");
    return ok ? (int)x : -1;
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

// max of three, NaN if one of them is (one instruction)
W4_DEV float max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// (x, y) = (x, y) * a + b and (s, t) += (x, y): two fp32 lanes an instruction
W4_DEV void fma2_to(float& x, float& y, float a, float b) {
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %3};\n\t"
        "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}
W4_DEV void add2_to(float& s, float& t, float x, float y) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
        "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(s), "+f"(t)
        : "f"(x), "f"(y));
}

using w4p::wait_or_abort;

template <bool BF16, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_o,
                     const AttnParams p) {
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
    uint64_t* item_full = fixed + S;          // [kItems]
    uint64_t* item_empty = item_full + kItems;
    uint64_t* q_full = item_empty + kItems;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_empty + 1;     // [A, B]
    uint64_t* p_full = s_full + 2;      // [A, B][half of the block]
    uint64_t* o_done = p_full + 4;      // [A, B]: the item's O
    uint64_t* next_bar = o_done + 2;
    uint64_t* all_done = next_bar + 1;
    uint64_t* both_ready = all_done + 1;   // one tile: A's and B's O and statistics are there,
    uint64_t* both_read = both_ready + 1;  // ... and have been read
    uint64_t* want = both_read + 1;        // the loads of the item at work near their end
    float2* stats = reinterpret_cast<float2*>(smem + C::stats);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc + 4);
    auto slot = [&](int i) { return reinterpret_cast<Work*>(smem + C::items + (i % kItems) * 64); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&raw[s], 1);
            mbar_init(&fixed[s], 8);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], 8 + 1 + 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[2 * x], 4);
            mbar_init(&p_full[2 * x + 1], 4);
            mbar_init(&o_done[x], 1);
        }
        mbar_init(next_bar, 1);
        mbar_init(all_done, 1);
        mbar_init(both_ready, 8);
        mbar_init(both_read, 8);
        mbar_init(want, 1);
        *abort_flag = 0;
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
        prefetch_tensormap(&tmap_o);
    }
    w4p::tc_fence_before();
    __syncthreads();
    w4p::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();
    auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
    // the item in slot n % kItems, for consumer warps; false at the end
    auto take = [&](int n, bool& ok) {
        ok = all(wait_or_abort(&item_full[n % kItems], (n / kItems) & 1, abort_flag));
        return ok && slot(n)->valid != 0;
    };
    auto release = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[n % kItems]);
    };

    if (warp >= 8) {
        w4p::setmaxnreg_dec<kRegsOther>();
        if (warp == 10) {
            // ---------------------------------------------------------- items
            pdl_wait();   // the bounds may come from the preceding kernel
            const bool ranges = p.part_o != nullptr;
            Finder finder = {};
            Walker walker = {};
            if (ranges) walker.start(p, lane);
            else finder.start(p, lane);
            int item = blockIdx.x, n = 0;
            bool asked = false;
            for (;; ++n) {
                const Work w = ranges ? walker.next(p, lane) : finder.find(p, item, lane);
                if (n >= kItems && !all(wait_or_abort(&item_empty[n % kItems], ((n / kItems) & 1) ^ 1, abort_flag))) break;
                if (lane == 0) {
                    *slot(n) = w;
                    mbar_arrive(&item_full[n % kItems]);
                }
                __syncwarp();
                if (!w.valid) break;
                if (ranges) continue;
                // no earlier: an item that waits here is one that no idle SM can take
                if (!all(wait_or_abort(want, n & 1, abort_flag))) break;
                asked = true;
                if (lane == 0) {
                    mbar_arrive_expect_tx(next_bar, 16);
                    ask_next(smem + C::next, next_bar);
                }
                if (!all(wait_or_abort(next_bar, n & 1, abort_flag))) break;
                asked = false;
                item = answered(smem + C::next);
                fence_proxy_async_smem();   // the answer is read before it is written again
                __syncwarp();
                if (item < 0) item = INT_MAX;   // found as the end
            }
            if (asked) (void)mbar_wait(next_bar, n & 1);   // an answer in flight lands before the block ends
            if (blockIdx.x == 0) {
                bool bad = false;
                for (int b = lane; b < p.batch; b += 32) {
                    int s, c;
                    seq_bounds(p.cu_q, p.total_q, b, s, c, bad);
                    seq_bounds(p.cu_k, p.total_k, b, s, c, bad);
                }
                if (bad) atomicOr(&g_w4_error_word, W4_DEVERR_GIDX);
            }
            __syncwarp();
        } else if (warp == 8) {
            // ---------------------------------------------------------- TMA
            pdl_wait();   // Q, K and V may come from the preceding kernel
            int i = 0, nq = 0;   // ring position, Q loads so far
            // Each barrier completes once a use, so its parity is a bit that its users flip
            // at each use (a bit a stage).
            uint32_t full_ph = 0, raw_ph = 0, last_raw = 0;
            bool ok = true;
            for (int n = 0; ok && take(n, ok); ++n) {
                const Work* w = slot(n);
                const int nb0 = blocks_of_subs(w->sub0), nb1 = blocks_of_subs(w->sub1), mfirst = w->common / kKeys, hk = w->hk;
                const int key0 = w->k0 + w->b0 * kKeys, tok0 = w->q0 + w->tok;
                release(n);
                const bool pair = p.tiles == 2;
                const int nb = pair ? max(nb0, nb1) : nb0 + nb1;
                if (lane == 0 && nb == 0) mbar_arrive(want);
                if (lane == 0 && nb > 0) {
                    // Q, then through the ring, in the order the products take them: K_0, V_0, K_1,
                    // V_1, ... (pair) or K_0, K_1, V_0, K_2, V_1, K_3, ... (one tile)
                    if (nq > 0) ok = wait_or_abort(q_empty, (nq - 1) & 1, abort_flag);
                    if (ok) {
                        const int tiles = pair ? (nb0 > 0 ? 1 : 0) + (nb1 > 0 ? 1 : 0) : 1;
                        mbar_arrive_expect_tx(q_full, tiles * NC * 128 * p.group * p.tpt);
                        ++nq;
                        for (int x = 0; x < p.tiles; ++x) {
                            if ((x ? nb1 : nb0) == 0) continue;
                            for (int c = 0; c < NC; ++c)
                                tma_load_3d(smem + C::q + x * C::q_tile + c * kRows * 128, &tmap_q, 64 * c,
                                            hk * p.group, tok0 + x * p.tpt, q_full);
                        }
                    }
                    const int lead = pair ? 1 : min(2, nb);   // K tiles ahead of the first V
                    for (int k = 0, nk = 0, nv = 0; k < 2 * nb && ok; ++k, ++i) {
                        const int s = i % S;
                        if (k == max(0, 2 * nb - 6)) mbar_arrive(want);   // about three blocks before the item's end
                        const bool is_v = nk == nb || nk - nv == lead;
                        const int blk = is_v ? nv++ : nk++;
                        if (i >= S) ok = wait_or_abort(&empty[s], ((i / S) & 1) ^ 1, abort_flag);
                        if (!ok) break;
                        const bool is_raw = is_v && blk >= mfirst;
                        uint64_t* bar = is_raw ? &raw[s] : &full[s];
                        if (is_raw) raw_ph ^= 1u << s;
                        else full_ph ^= 1u << s;
                        last_raw = (last_raw & ~(1u << s)) | ((is_raw ? 1u : 0u) << s);
                        mbar_arrive_expect_tx(bar, C::kv_tile);
                        for (int c = 0; c < NC; ++c)
                            tma_load_3d(smem + C::ring + s * C::kv_tile + c * kKeys * 128, is_v ? &tmap_v : &tmap_k,
                                        64 * c, hk, key0 + blk * kKeys, bar);
                    }
                }
                ok = all(ok);
            }
            if (*abort_flag && lane == 0) {
                // what is in flight lands before the block ends
                if (nq > 0) (void)mbar_wait(q_full, (nq - 1) & 1);
                for (int s = 0; s < min(S, i); ++s) {
                    const bool r = (last_raw >> s) & 1u;
                    (void)mbar_wait(r ? &raw[s] : &full[s], (((r ? raw_ph : full_ph) >> s) & 1u) ^ 1u);
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
                return all(r);
            };
            // S_x = Q_q K^T with the K tile of ring position i
            auto issue_s = [&](int x, int q, int i) {
                if (!leader) return;
                const uint32_t qd = qd0 + ((q * C::q_tile) >> 4);
                const uint32_t kd = kd0 + (((i % S) * C::kv_tile) >> 4);
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_ss(tmem + 128 * x, qd + ((c * kRows * 128 + 32 * k) >> 4),
                                  kd + ((c * kKeys * 128 + 32 * k) >> 4), hi, idesc_s, (c | k) ? 1u : 0u);
                w4p::tc_commit(&s_full[x]);
            };
            // O_x (+)= P_x V over half h of the block, with the V tile of ring position i
            auto issue_o = [&](int x, int h, int i, bool first) {
                if (!leader) return;
                const uint32_t vd = vd0 + (((i % S) * C::kv_tile + h * kSub * 128) >> 4);
#pragma unroll
                for (int k = 0; k < kSub / 16; ++k)
                    tc_mma_ts(tmem + 256 + DP * x, tmem + 128 * x + 32 * h + 8 * k, vd + ((2048 * k) >> 4), hi, idesc_o,
                              (first && k == 0) ? 0u : 1u);
            };
            int pos = 0, nq = 0;       // ring position, Q loads so far
            uint32_t p_ph = 0;         // parities of the next P halves, bit 2 x + h
            bool ok = true;
            auto wait_p = [&](int x, int h) {
                const bool r = wait_or_abort(&p_full[2 * x + h], (p_ph >> (2 * x + h)) & 1u, abort_flag);
                p_ph ^= 1u << (2 * x + h);
                return all(r);
            };
            auto free_slot = [&](int i) {
                if (leader) w4p::tc_commit(&empty[i % S]);
            };
            for (int n = 0; ok && take(n, ok); ++n) {
                const Work* w = slot(n);
                const int sub0 = w->sub0, sub1 = w->sub1, mfirst = w->common / kKeys;
                const int nb0 = blocks_of_subs(sub0), nb1 = blocks_of_subs(sub1);
                if (sub0 + sub1 == 0) {
                    release(n);
                    continue;
                }
                ok = all(wait_or_abort(q_full, nq & 1, abort_flag));
                ++nq;
                if (p.tiles == 2) {
                    // both tiles over the same blocks: K_0, then V_j and K_{j+1}
                    const int nb = max(nb0, nb1);
                    ok = ok && wait_bit(full, full_ph, pos % S);
                    if (!ok) break;
                    w4p::tc_fence_after();
                    if (nb0 > 0) issue_s(0, 0, pos);
                    if (nb1 > 0) issue_s(1, 1, pos);
                    free_slot(pos);
                    if (leader && nb == 1) w4p::tc_commit(q_empty);
                    ++pos;
                    for (int j = 0; j < nb && ok; ++j) {
                        const int iv = pos, ik = pos + 1;
                        ok = j >= mfirst ? wait_bit(fixed, fixed_ph, iv % S) : wait_bit(full, full_ph, iv % S);
                        if (ok && j + 1 < nb) ok = wait_bit(full, full_ph, ik % S);
                        if (!ok) break;
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int sub = x ? sub1 : sub0;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (!ok || 2 * j + h >= sub) continue;
                                ok = wait_p(x, h);
                                if (!ok) continue;
                                w4p::tc_fence_after();
                                issue_o(x, h, iv, j == 0 && h == 0);
                            }
                            if (!ok || 2 * j >= sub) continue;
                            if (2 * j + 2 < sub) issue_s(x, x, ik);
                            else if (leader) w4p::tc_commit(&o_done[x]);
                        }
                        if (!ok) break;
                        free_slot(iv);
                        ++pos;
                        if (j + 1 < nb) {
                            free_slot(ik);
                            ++pos;
                        }
                        if (leader && j + 2 == nb) w4p::tc_commit(q_empty);   // the item's last S is issued
                    }
                } else {
                    // one tile: A takes the even blocks, B the odd ones
                    const int nb = nb0 + nb1, subs = sub0 + sub1;
                    for (int k = 0; k < min(2, nb) && ok; ++k) {
                        ok = wait_bit(full, full_ph, pos % S);
                        if (!ok) break;
                        w4p::tc_fence_after();
                        issue_s(k, 0, pos);
                        free_slot(pos);
                        ++pos;
                    }
                    if (leader && nb <= 2) w4p::tc_commit(q_empty);
                    for (int k = 0; k < nb && ok; ++k) {
                        const int x = k & 1, iv = pos, ik = pos + 1;
                        ok = k >= mfirst ? wait_bit(fixed, fixed_ph, iv % S) : wait_bit(full, full_ph, iv % S);
                        if (ok && k + 2 < nb) ok = wait_bit(full, full_ph, ik % S);
                        if (!ok) break;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!ok || 2 * k + h >= subs) continue;
                            ok = wait_p(x, h);
                            if (!ok) continue;
                            w4p::tc_fence_after();
                            issue_o(x, h, iv, k < 2 && h == 0);
                        }
                        if (!ok) break;
                        if (k + 2 < nb) issue_s(x, 0, ik);
                        else if (leader) w4p::tc_commit(&o_done[x]);
                        if (!ok) break;
                        free_slot(iv);
                        ++pos;
                        if (k + 2 < nb) {
                            free_slot(ik);
                            ++pos;
                            if (leader && k + 3 == nb) w4p::tc_commit(q_empty);
                        }
                    }
                }
                if (ok) release(n);
            }
            if (leader) w4p::tc_commit(all_done);
            (void)mbar_wait(all_done, 0);
            __syncwarp();
        }
    } else {
        // -------------------------------------------------------------- softmax, one row a thread
        w4p::setmaxnreg_inc<kRegsSoftmax>();
        pdl_wait();   // before any store
        const int x = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + 128 * x, to = tmem + lanes + 256 + DP * x;
        int ones = 0;                    // one-tile items so far
        const int rg = (threadIdx.x & (kRows - 1)) / p.group;
        int base = 0;                    // ring position of the item's K_0
        uint32_t raw_ph = 0;             // a bit a stage
        uint32_t s_ph = 0, o_ph = 0;     // parities of the next S, of the next item's O
        bool ok = true;
        const bool pair = p.tiles == 2;
        for (int item = 0; ok && take(item, ok); ++item) {
        volatile Work* const ws = slot(item);
        float m = -INFINITY, l = 0.0f;   // reference maximum of the raw scores, sum of the weights
        const int n = x ? ws->sub1 : ws->sub0;
        const int common = ws->common;
        const Row mine = row_of(p, ws, x, rg);
        const int limit = mine.limit - ws->b0 * kKeys;   // in the item's keys
        const bool busy = __any_sync(0xffffffffu, mine.live);
        // blocks of the item (of both tiles), the next one whose V may need a look
        const int nb = pair ? blocks_of_subs(max(ws->sub0, ws->sub1)) : blocks_of_subs(ws->sub0) + blocks_of_subs(ws->sub1);
        int look = common / kKeys;
        auto look_until = [&](int j) {   // V of all blocks up to j
            for (; look <= j && look < nb && ok; ++look) {
                const int s = (base + look + min(look + (pair ? 1 : min(2, nb)), nb)) % S;
                ok = all(wait_or_abort(&raw[s], (raw_ph >> s) & 1u, abort_flag));
                raw_ph ^= 1u << s;
                if (!ok) break;
                // rows from `from` on are not seen by every row, rows from `left` on by none
                const int from = max(0, common - look * kKeys), left = ws->seen - look * kKeys;
                unsigned char* v = smem + C::ring + s * C::kv_tile;
                constexpr uint32_t kExp = BF16 ? 0x7F807F80u : 0x7C007C00u;
                constexpr uint32_t kOne = BF16 ? 0x00800080u : 0x04000400u;
                bool any = false;
                for (int q = 8 * from + threadIdx.x; q < 8 * kKeys; q += 256) {
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        uint4* at = reinterpret_cast<uint4*>(v + c * kKeys * 128 + q * 16);
                        if (q >= 8 * left) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                            continue;
                        }
                        const uint4 d = *at;
                        uint32_t e[4] = {d.x, d.y, d.z, d.w}, hit = 0;
                        // an exponent of all ones carries into the sign's place
#pragma unroll
                        for (int k = 0; k < 4; ++k) hit |= (e[k] & kExp) + kOne;
                        if (!(hit & 0x80008000u)) continue;
#pragma unroll
                        for (int k = 0; k < 4; ++k) e[k] &= ~(((((e[k] & kExp) + kOne) & 0x80008000u) >> 15) * 0xFFFFu);
                        *at = make_uint4(e[0], e[1], e[2], e[3]);
                        any = true;
                    }
                }
                if (any) ws->poison = 1;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&fixed[s]);
            }
        };
        for (int u = 0; u < n; u += 2) {
            const int key = pair ? kSub * u : kKeys * (u + x);   // first key of the block
            look_until(key / kKeys);
            if (!ok) break;
            ok = all(wait_or_abort(&s_full[x], s_ph, abort_flag));
            if (!ok) break;
            s_ph ^= 1u;
            if (!busy) {   // (P of rows that are no tokens may be anything)
                if (lane == 0) {
                    mbar_arrive(&p_full[2 * x]);
                    if (u + 1 < n) mbar_arrive(&p_full[2 * x + 1]);
                }
                continue;
            }
            w4p::tc_fence_after();
            uint32_t sr[8][16];
#pragma unroll
            for (int c = 0; c < 8; ++c) tmem_ld16_async(ts + 16 * c, sr[c]);
            tmem_wait_ld();
            if (key + kKeys > common) {
                const int lim = limit - key;
#pragma unroll
                for (int c = 0; c < 8; ++c)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (16 * c + i >= lim) sr[c][i] = 0xFF800000u;
            }
            // four chains: one would be 64 dependent instructions long
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    mx[i & 3] = max3(mx[i & 3], __uint_as_float(sr[c][2 * i]), __uint_as_float(sr[c][2 * i + 1]));
            const float bm = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]);
            // A NaN or +infinity among the scores makes the row NaN.  NaN compares false below:
            // the row keeps its reference.
            if (!(bm < INFINITY)) l = NAN;
            const bool raise = m == -INFINITY ? bm > m : (bm - m) * p.scale_log2 > kLazy;
            if (__any_sync(0xffffffffu, raise)) {
                const float nm = raise ? bm : m;
                const float f = raise ? ex2((m - nm) * p.scale_log2) : 1.0f;
                if (u > 0) {
                    // (O is complete up to the last block: this S was issued behind its P V)
#pragma unroll
                    for (int c = 0; c < DP / 16; ++c) {
                        uint32_t o[16];
                        tmem_ld16_async(to + 16 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st16(to + 16 * c, o);
                    }
                }
                l *= f;   // (NaN stays NaN)
                m = nm;
            }
            const float shift = m == -INFINITY ? 0.0f : kShift - m * p.scale_log2;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 1 && u + 1 >= n) break;   // the item's last block may be half
#pragma unroll
                for (int c = 2 * h; c < 2 * h + 2; ++c) {
                    uint32_t pr[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float a = __uint_as_float(sr[2 * c + (i >> 3)][2 * (i & 7)]);
                        float b = __uint_as_float(sr[2 * c + (i >> 3)][2 * (i & 7) + 1]);
                        fma2_to(a, b, p.scale_log2, shift);
                        a = ex2(a);
                        b = ex2(b);
                        add2_to(sum[2 * (i & 1)], sum[2 * (i & 1) + 1], a, b);
                        pr[i] = pack2<BF16>(a, b);
                    }
                    tmem_st16(ts + 16 * c, pr);
                }
                tmem_wait_st();
                w4p::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * x + h]);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        if (ok) look_until(nb);
        base += 2 * nb;
        // the item's output
        if (n > 0 && ok) {
            ok = all(wait_or_abort(&o_done[x], o_ph, abort_flag));
            o_ph ^= 1u;
        }
        if (!ok) break;
        // weights of this warp's O and, with one tile, of the other's O of the same rows
        float own = 1.0f, other = 0.0f;
        if (!pair) {
            stats[x * kRows + (threadIdx.x & (kRows - 1))] = make_float2(m, l);
            w4p::tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(both_ready);
            ok = all(wait_or_abort(both_ready, ones & 1, abort_flag));
            if (!ok) break;
            const float2 o = stats[(1 - x) * kRows + (threadIdx.x & (kRows - 1))];
            const float top = fmaxf(m, o.x);
            own = m == -INFINITY ? 0.0f : ex2((m - top) * p.scale_log2);
            other = o.x == -INFINITY ? 0.0f : ex2((o.x - top) * p.scale_log2);
            l = own * l + other * o.y;
            m = top;
        }
        w4p::tc_fence_after();
        if (busy) {
            // read again: kept in registers through the loop, these would not fit
            const Row r = row_of(p, ws, x, rg);
            const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
            own *= inv;
            other *= inv;
            const int n_other = pair ? 0 : x ? ws->sub0 : ws->sub1;
            const int head = ws->hk * p.group + (threadIdx.x & (kRows - 1)) - rg * p.group;
            const bool part = ws->part >= 0;
            // Of the keys that this warp's rows see, every one has been looked at (`fixed`, then the
            // products, then `o_done`); for later keys other warps may still be setting the mark.  One
            // read for the whole warp: what follows it is warp-wide.
            const bool poison = __any_sync(0xffffffffu, ws->poison != 0);
            // row offsets in the output, and where the rows of this warp that are tokens lie
            const size_t tok = (size_t)(ws->q0 + r.tok);
            const size_t prow = (size_t)ws->part * kRows + (threadIdx.x & (kRows - 1));
            const size_t at = part ? prow * p.dim : tok * p.ldo + (size_t)head * p.hso;
            const unsigned live = __ballot_sync(0xffffffffu, r.live);
            unsigned char* st = smem + C::out + warp * 4096;
            // O columns [c, c + 32) of this row, weighted
            auto load_o = [&](int c, uint32_t (&o)[2][16]) {
                if (n > 0) {
                    tmem_ld16_async(to + c, o[0]);
                    tmem_ld16_async(to + c + 16, o[1]);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i >> 4][i & 15] = __float_as_uint(__uint_as_float(o[i >> 4][i & 15]) * own);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i >> 4][i & 15] = 0u;
                }
                if (n_other > 0) {
                    uint32_t o2[2][16];
                    tmem_ld16_async(to + (x ? -DP : DP) + c, o2[0]);
                    tmem_ld16_async(to + (x ? -DP : DP) + c + 16, o2[1]);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        o[i >> 4][i & 15] = __float_as_uint(
                            fmaf(__uint_as_float(o2[i >> 4][i & 15]), other, __uint_as_float(o[i >> 4][i & 15])));
                }
            };
            // 128 bytes of each row at a time (64 16-bit or 32 fp32 columns) through shared
            // memory, 16-byte pieces swizzled by row: from there the tensor store takes 32 whole
            // rows, or the warp writes whole 128-byte lines of four rows at a time.
            const int cols = part ? 32 : 64;
            const bool whole = p.tma_out && !part && live == 0xffffffffu;
            size_t to_row[8];
            if (!whole) {
#pragma unroll
                for (int k = 0; k < 8; ++k) to_row[k] = __shfl_sync(0xffffffffu, (unsigned long long)at, 4 * k + (lane >> 3));
            }
            auto make_room = [&] {
                if (lane == 0) tma_store_read();   // the last store has read its bytes
                __syncwarp();
            };
            auto send = [&](int c0) {   // the staged columns from c0 on
                if (whole) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) tma_store_3d(&tmap_o, st, c0, ws->hk * p.group, (int)tok);
                    return;
                }
                __syncwarp();
                const int col = c0 + (part ? 4 : 8) * (lane & 7);
                uint4 d[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    d[k] = *reinterpret_cast<const uint4*>(st + (4 * k + (lane >> 3)) * 128 +
                                                           (((lane & 7) ^ ((4 * k + (lane >> 3)) & 7)) << 4));
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (!((live >> (4 * k + (lane >> 3))) & 1u) || col >= p.dim) continue;
                    if (part) *reinterpret_cast<uint4*>(p.part_o + to_row[k] + col) = d[k];
                    else *reinterpret_cast<uint4*>(reinterpret_cast<unsigned short*>(p.O) + to_row[k] + col) = d[k];
                }
                __syncwarp();
            };
            if (pair && !part && n > 0 && !poison) {
                // the common case, O's columns all at once (8 prompts of 1024 tokens, 32/8 heads:
                // 113 -> 106 us against 32 columns at a time)
                uint32_t o[DP / 16][16];
#pragma unroll
                for (int c = 0; c < DP / 16; ++c) tmem_ld16_async(to + 16 * c, o[c]);
                tmem_wait_ld();
#pragma unroll
                for (int c0 = 0; c0 < DP; c0 += 64) {
                    if (c0 >= p.dim) break;
                    make_room();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const uint32_t* v = &o[(c0 + 8 * q) / 16][(8 * q) % 16];
                        uint32_t e[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            e[k] = pack2<BF16>(__uint_as_float(v[2 * k]) * own, __uint_as_float(v[2 * k + 1]) * own);
                        *reinterpret_cast<uint4*>(st + lane * 128 + ((q ^ (lane & 7)) << 4)) = make_uint4(e[0], e[1], e[2], e[3]);
                    }
                    send(c0);
                }
            } else {
#pragma unroll 1
            for (int c0 = 0; c0 < p.dim; c0 += cols) {
                if (!pair && (c0 / cols & 1) != x) continue;   // one tile: the two warps of a row take turns
                make_room();
                uint32_t o[2][16];
                if (part) {
                    load_o(c0, o);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        *reinterpret_cast<uint4*>(st + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                            make_uint4(o[q >> 2][4 * (q & 3)], o[q >> 2][4 * (q & 3) + 1], o[q >> 2][4 * (q & 3) + 2],
                                       o[q >> 2][4 * (q & 3) + 3]);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        load_o(c0 + 32 * h, o);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t e[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                e[k] = pack2<BF16>(__uint_as_float(o[q >> 1][8 * (q & 1) + 2 * k]),
                                                   __uint_as_float(o[q >> 1][8 * (q & 1) + 2 * k + 1]));
                            *reinterpret_cast<uint4*>(st + lane * 128 + (((4 * h + q) ^ (lane & 7)) << 4)) =
                                make_uint4(e[0], e[1], e[2], e[3]);
                        }
                    }
                }
                if (poison) {
                    const int first = ws->b0 * kKeys + common, last = min(r.limit, ws->b0 * kKeys + (n + n_other) * kSub);
                    repair_row<BF16>(st + lane * 128, lane, part, c0, min(cols, p.dim - c0),
                                     reinterpret_cast<const unsigned short*>(p.V) + (size_t)(ws->k0 + first) * p.ldv +
                                         (size_t)ws->hk * p.hsv, p.ldv, last - first);
                    __syncwarp();
                }
                send(c0);
            }
            }
            const float v = l == 0.0f ? -INFINITY : m * p.scale + (logf(l) - kShift * 0.69314718055994531f);
            if (r.live && (pair || x == 0)) {
                if (part) p.part_lse[prow] = v;
                else if (p.lse) p.lse[tok * p.heads + head] = v;
            }
        }
        if (!pair) {
            // neither half writes its O or its statistics again before the other has read them
            w4p::tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(both_read);
            ok = all(wait_or_abort(both_read, ones & 1, abort_flag));
            w4p::tc_fence_after();
            ++ones;
        }
        release(item);
        }
        if (lane == 0) tma_store_done();
    }
    w4p::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        w4p::tc_fence_after();
        w4p::tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of an item that ranges cut: O = sum_s e^(lse_s - lse) O_s, lse = log sum_s
// e^lse_s over its parts s.  Block (c, y) joins rows 16 y .. of the item that CTA c's range
// starts and does not end, if there is one (items that no range cuts are already there): two
// rows a warp, four columns a lane.
constexpr int kJoinRows = 16;
template <bool BF16>
__global__ void __launch_bounds__(256) combine_kernel(const AttnParams p) {
    __shared__ Work s_work;
    __shared__ int s_last;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = blockIdx.x;
    if (warp == 0) {
        Work w = {};
        int last = first;
        Walker walker;
        walker.start(p, lane);
        const long long total = walker.total, at = walker.end;   // first block of the next range
        if (at < total && walker.at < at) {
            walker.at = at;
            walker.end = at + 1;
            w = walker.next(p, lane);   // the item of that block
            const long long start = at - w.b0;
            if (w.b0 > 0 && start >= List::begin(p, total, first))
                last = List::cta_of(p, total, start + List::blocks_of(w.nk) - 1);
        }
        if (lane == 0) {
            s_work = w;
            s_last = last;
        }
    }
    __syncthreads();
    const int last = s_last;
    if (last == first) return;
    const Work& w = s_work;
    for (int in_tile = kJoinRows * blockIdx.y + warp; in_tile < kJoinRows * (blockIdx.y + 1); in_tile += 8) {
    const int rg = in_tile / p.group, tok_in = w.tok + rg;
    if (rg >= p.tpt || tok_in >= w.nq) continue;
    const size_t tok = (size_t)(w.q0 + tok_in);
    const int head = w.hk * p.group + in_tile - rg * p.group;
    // part of CTA c: its last (place 1) where it starts the item, its first (place 0) otherwise
    auto place = [&](int c) {
        return (size_t)(2 * c + (c == first ? 1 : 0)) * kRows + in_tile;
    };
    float top = -INFINITY;
    bool nan = false;
    for (int c = first + lane; c <= last; c += 32) {
        const float v = p.part_lse[place(c)];
        top = fmaxf(top, v);
        nan |= v != v;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    nan = __any_sync(0xffffffffu, nan);
    float a[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f;
    const bool on = 4 * lane < p.dim;
#pragma unroll 4
    for (int c = first; c <= last; ++c) {
        const float v = p.part_lse[place(c)];
        const float f = v == -INFINITY ? 0.0f : expf(v - top);
        sum += f;
        const float4 o = on ? *reinterpret_cast<const float4*>(p.part_o + place(c) * p.dim + 4 * lane)
                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        a[0] = fmaf(f, o.x, a[0]);
        a[1] = fmaf(f, o.y, a[1]);
        a[2] = fmaf(f, o.z, a[2]);
        a[3] = fmaf(f, o.w, a[3]);
    }
    const float inv = nan ? NAN : sum > 0.0f ? 1.0f / sum : 0.0f;
    if (on)
        *reinterpret_cast<uint2*>(reinterpret_cast<unsigned short*>(p.O) + tok * p.ldo + (size_t)head * p.hso + 4 * lane) =
            make_uint2(pack2<BF16>(a[0] * inv, a[1] * inv), pack2<BF16>(a[2] * inv, a[3] * inv));
    if (lane == 0 && p.lse) p.lse[tok * p.heads + head] = nan ? NAN : sum > 0.0f ? top + logf(sum) : -INFINITY;
    }
}

}  // namespace w4t
