// Softmax attention of the new tokens over a paged key/value cache
// (include/gdn2_attn.h).
//
// Rows.  The query heads that share a key head are packed into the rows of one
// matrix product: row r of a 128-row tile is token r / G, head r % G of the
// group (G = HQ / HKV), so that a decode step's G rows share the keys they
// read.  An item is (sequence, key head, up to two row tiles) with its range of
// 128-key tiles (after the causal and window masks).
//
// Work.  The items' key tiles, laid end to end (with an allowance per item), are
// cut into equal shares, one per CTA (one CTA per SM), wherever the cuts fall: a
// share is a run of segments (item, key tiles).  An item cut into several segments
// leaves unnormalised sums and their maxima in the workspace, and the combine
// kernel joins them in the order of the segments.  So one long sequence, many
// short ones and any mixture fill the GPU alike, and the result does not depend on
// timing.  Every CTA finds its own share from the lengths (a sum over the
// sequences), which takes about two microseconds; a separate planning kernel cost 4
// to 25.
//
// A CTA (384 threads):
//   warps 0-3, 4-7  two softmax groups, a thread per row
//   warp 8          issues the products (tcgen05): S = Q K^T into Tensor Memory
//                   (fp32), O += P V with P from Tensor Memory (16 bits)
//   warp 9          walks the share, hands the segments out through a ring in
//                   shared memory, and loads the keys by TMA, straight from their
//                   pages, into a ring of 128-key stages
//   warp 10         loads the values into the same ring (lanes that issue TMA
//                   copies take turns, 50 cycles each: with small pages one warp
//                   for both bound decode to 79 % of the bandwidth)
//   warp 11         loads the queries as soon as the last scores of the segment
//                   before are in
// With two row tiles in an item, group x has tile x and both read every stage;
// with one (decode), group x has every second key tile, with statistics and
// outputs of its own that are merged at the end of the segment.  Either way one
// group's softmax runs while the tensor cores work for the other.
//
// The value rows of an item's first and last tile that none of its rows attends to
// (before the window, past the causal range) are zeroed in shared memory: the
// cache may hold anything there, and 0 x NaN is NaN.  The keys' scores are masked.
// Pages wholly before the window are not read, nor their table entries.
//
// Bounds, measured on a GB300 (bf16):
//   long chunks     the tensor cores under the power limit: 2048 tokens over 32768 keys,
//                   32 query and 8 key heads of 128, 660 to 695 us, 1.53 to 1.61 PFLOP/s;
//                   tensor pipe active 78 %.  Two row tiles of 128 keys take 2.55 k
//                   cycles, their products 2.05 k, a softmax 1.5 k
//   short chunks    the items' ends, when the tensor cores wait: 8 of 396 .. 3235 tokens,
//                   16 heads, pages of 16, 216 to 230 us, 1.15 to 1.22 PFLOP/s
//   D = 64          the softmax's latency, 2.2 k cycles a tile: 16384 tokens, 16 heads,
//                   536 us, 1.03 PFLOP/s
//   decode          memory: 128 sequences of up to 8192 keys, 8 key heads of 128, 355 to
//                   366 us, 6.5 to 6.7 TB/s of the 6.78 that a copy reaches
//   one token       12 us: a chain of loads and of code that is fetched as it runs
#include <cudaTypedefs.h>

#include <type_traits>

#include "gdn2_attn_internal.h"
#include "gdn2_tc.cuh"

namespace gdn2 {
namespace {

using namespace tc;

constexpr int kMaxCtas = 152;   // shares at most (SMs of a GB300)
constexpr int kTile = 128;      // rows of a tile, keys of a tile
constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kKeyWarp = 9, kValueWarp = 10, kQueryWarp = 11;
// What an item of two row tiles costs beside its key tiles, in key tiles: its
// queries, its first softmax and its epilogue, when the tensor cores wait.
// Measured with D = 128 on 8 chunks of 396 .. 3235 tokens (16 heads; 4 to 13 items per
// CTA): 229 us with 1, 219 with 2, 221 with 3, 224 with 4 (and 286 without against 267 with
// 2 before the loaders' divisions went); with D = 64 on 16384 tokens of one sequence (16
// heads) 553 us without, 536 with 1, 548 with 2.  An item of one row tile hides it
// behind its loads.
constexpr int lead_tiles(int D) { return D == 128 ? 2 : 1; }
constexpr int kSegRing = 8;     // segments in flight between the warps
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The softmax's weights are 2^(score - reference + bias) (scores times log2 e), rounded to
// the call's type, since a product has one 16-bit type for both operands: a relative
// error of up to 2^-8 (bf16) or 2^-11 (fp16) per weight, as the output has from its own
// rounding, and less where they average out.  The reference is a maximum of the row's
// keys so far, moved when a tile's maximum is more than kLag above it: the outputs are
// then seldom rescaled.
// bf16 has fp32's exponents and needs no bias.  fp16 ends at 2^16, holds 2^-14 in full
// and has nothing below 2^-25: with the weights up to 2^(kLag + kBias) = 2^15, one that
// is 2^-25 of its reference still is held in full.  Many small weights beside a few
// large ones may be what the output consists of (a key that takes nearly all weight and
// whose value is next to nothing), so in fp16 the reference also moves down to a tile that
// stays kDrop below it: tiles of small weights are held to their own maximum.  The
// sums then grow instead, in fp32, to at most kMost.  Looking for such tiles costs 4 % with
// D = 64 (16384 tokens of 16 heads 538 -> 560 us; kLag 4, 6 and 8 alike), nothing with D = 128.
template <bool F16>
struct Weights {
    static constexpr float kLag = F16 ? 4.f : 8.f, kBias = F16 ? 11.f : 0.f, kDrop = 12.f;
    static constexpr float kMost = 7.9e28f;  // 2^96; times values to 2^16 and pieces to 2^8 within fp32
};
// Registers: three warpgroups of 168 at launch, 64512 in all; the two softmax
// groups, which hold a row of scores, take 192 and the third keeps 120
// (2 x 128 x 192 + 128 x 120 = 64512).
constexpr int kSoftmaxRegs = 192, kOtherRegs = 120;

// A share's piece of an item: new tokens tok0 .. tok0 + ntok (rows of q), key
// head h, key tiles lo .. hi; slot of its partial result, -1 if it is whole.
struct __align__(16) Segment {
    int tok0, h, ntok, slot;
    int lo, hi;
    int begin, end;  // no row of the item attends to a key outside
    int place;  // of the first new token in its cached sequence
    int seq, pad[2];
};
// The item whose pieces the combine kernel joins: the first in slot `slot`,
// then `more` in slots 2 (cta + 1), 2 (cta + 2), ...
struct __align__(16) Joint {
    int tok0, h, ntok, slot;
    int more, pad[3];
};
enum Flag { kBadCu = 1, kBadPages = 2, kTimeout = 4 };

struct KernelParams {
    AttnParams a;
    int *flags;                  // [kMaxCtas]
    Joint *joint;                // [kMaxCtas]
    float *part_o;               // [2 kMaxCtas][256][D]
    float2 *part_ml;             // [2 kMaxCtas][256] (log2-scaled maximum, sum)
    float scale_log2;
    int tt;                      // tokens per row tile: 128 / G
    int granule, granule_log2;   // keys per TMA box
    Divisor page;                // page_size
    int kpos[3], vpos[3];        // coordinate (1 .. 3) of page, token, head in the tensor maps
    int ctas;                    // of the main kernel
    int q_map;                   // tq is set: the queries come by TMA
    CUtensorMap tk, tv, tq;
};

struct Layout {
    size_t flags, joint, part_ml, part_o, total;
};
Layout layout_of(const gdn2_attn_dims &d) {
    Layout l;
    size_t off = 256;  // the status words
    auto take = [&](size_t bytes) { const size_t o = off; off += (bytes + 255) & ~static_cast<size_t>(255); return o; };
    l.flags = take(kMaxCtas * 4);
    l.joint = take(kMaxCtas * sizeof(Joint));
    l.part_ml = take(4ull * kMaxCtas * kTile * sizeof(float2));
    l.part_o = take(4ull * kMaxCtas * kTile * d.D * sizeof(float));
    l.total = off;
    return l;
}

// ------------------------------------------------------------- the shares
struct Span {
    int lo, hi, begin, end;  // key tiles, keys
};
// Key tiles of the new tokens j0 .. j1 of a sequence of `len` cached tokens.
__device__ __forceinline__ Span key_span(const AttnParams &a, int len, int fresh, int j0, int j1) {
    Span s;
    s.end = a.causal ? max(0, len - fresh + j1) : len;
    s.begin = a.window >= 0 ? max(0, max(0, len - fresh + j0) - a.window) : 0;
    s.lo = s.begin / kTile;
    s.hi = (s.end + kTile - 1) / kTile;
    if (s.hi < s.lo) s.hi = s.lo;
    return s;
}
// What an item costs beside its key tiles (the items have `tokens` new tokens but for
// the last of a sequence; more than half of that makes two row tiles).
__device__ __forceinline__ int lead_of(const AttnParams &a, int fresh, int tokens, int m) {
    return min(fresh - m * tokens, tokens) > tokens / 2 ? a.lead : 0;
}
// What an item costs: its key tiles, at least 1 (an item without keys writes zeros),
// after the lead.
__device__ __forceinline__ int item_cost(const AttnParams &a, int len, int fresh, int tokens, int m) {
    const Span s = key_span(a, len, fresh, m * tokens, min(fresh, (m + 1) * tokens));
    return max(1, s.hi - s.lo) + lead_of(a, fresh, tokens, m);
}

// sum over i < n of floor((a i + b) / 128); a n + b < 2^32.
__device__ long long floor_sum(uint32_t n, uint32_t a, uint32_t b) {
    uint32_t m = 128;
    long long sum = 0;
    while (n > 0) {
        if (a >= m) {
            const uint32_t q = a / m;
            sum += static_cast<long long>(n - 1) * n / 2 * q;
            a -= q * m;
        }
        if (b >= m) {
            const uint32_t q = b / m;
            sum += static_cast<long long>(n) * q;
            b -= q * m;
        }
        const uint32_t top = a * n + b;
        if (top < m) break;
        n = top / m;
        b = top - n * m;
        const uint32_t t = m;
        m = a;
        a = t;
    }
    return sum;
}
// Whether the costs of a sequence's items add up in closed form.
__device__ __forceinline__ bool closed_form(const AttnParams &a, int len, int fresh) {
    return !a.causal || (a.window < 0 && len >= fresh);
}
// The cost of a sequence's first `items` items.
__device__ long long cost_of(const AttnParams &a, int len, int fresh, int tokens, int items) {
    if (items <= 0) return 0;
    const long long lead = static_cast<long long>(items - 1) * a.lead + lead_of(a, fresh, tokens, items - 1);
    if (!a.causal) return lead + static_cast<long long>(items) * max(1, (len + kTile - 1) / kTile);
    // item m: ceil((len - fresh + min(fresh, (m + 1) tokens)) / 128); the last one apart
    const long long last = (len - fresh + min(static_cast<long long>(fresh), static_cast<long long>(items) * tokens) + kTile - 1) / kTile;
    return lead + last + floor_sum(items - 1, tokens, static_cast<uint32_t>(len - fresh) + tokens + kTile - 1);
}

__device__ __forceinline__ long long div_by(long long x, long long y) {
    return (x | y) >> 32 ? x / y : static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
}

// A sequence as the shares see it; bad lengths count as no new tokens.
struct Seq {
    int t0, fresh, len;
};
__device__ __forceinline__ Seq seq_at(const AttnParams &a, int n, int *flags) {
    Seq q = {0, 0, 0};
    if (n >= a.N) return q;
    const int64_t c0 = cu_of(a.cu, a.cu64, n), c1 = cu_of(a.cu, a.cu64, n + 1);
    const int len = a.kv_lens[n];
    if (c0 > c1 || c0 < 0 || c1 > a.T) {
        if (flags) *flags |= kBadCu;
    } else if (len < 0 || len > static_cast<int64_t>(a.max_pages) * a.page_size) {
        if (flags) *flags |= kBadPages;
    } else {
        q.t0 = static_cast<int>(c0);
        q.fresh = static_cast<int>(c1 - c0);
        q.len = len;
    }
    return q;
}

// Cost of a sequence per key head; called by whole warps, a sequence per lane.
__device__ long long seq_cost(const AttnParams &a, const Seq &q, int tokens) {
    const int lane = threadIdx.x & 31;
    long long cost = q.fresh == 0 ? 0 : q.fresh <= tokens ? item_cost(a, q.len, q.fresh, tokens, 0)
                     : closed_form(a, q.len, q.fresh) ? cost_of(a, q.len, q.fresh, tokens, (q.fresh + tokens - 1) / tokens)
                                                      : -1;
    for (uint32_t more = __ballot_sync(0xffffffffu, cost < 0); more; more &= more - 1) {
        const int src = __ffs(more) - 1;
        const int len = __shfl_sync(0xffffffffu, q.len, src), fresh = __shfl_sync(0xffffffffu, q.fresh, src);
        long long sum = 0;
        for (int m = lane; m * static_cast<int64_t>(tokens) < fresh; m += 32) sum += item_cost(a, len, fresh, tokens, m);
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == src) cost = sum;
    }
    return cost;
}

struct Share {
    long long begin, left;   // first key tile, key tiles
    long long total, shares;
    long long in_seq, cost;  // offset of the first tile in its sequence, the sequence's cost per head
    int n, flags;            // sequence of the first tile
    Seq q;
    long long part[kThreads / 32];
};

// The share of this CTA; every thread of the block calls it, s is in shared memory
// (flags and left zero).
__device__ void find_share(const AttnParams &a, int tokens, Share &s) {
    const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
    const int parts = min(kThreads / 32, (a.N + 31) / 32);  // warps with sequences
    int flags = 0;
    if (tid == 0 && (a.N > 0 ? cu_of(a.cu, a.cu64, 0) != 0 || cu_of(a.cu, a.cu64, a.N) != a.T : a.T != 0)) flags = kBadCu;
    // cost of the sequence, and its inclusive sum over the warp
    auto scan = [&](int n, Seq &q, long long &c, int *f) {
        q = seq_at(a, n, f);
        c = seq_cost(a, q, tokens);
        long long x = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    Seq q;
    long long c, x, total = 0, before = 0;
    for (int base = 0; base < a.N || base == 0; base += kThreads) {  // the rounds before the last only add up
        x = scan(base + tid, q, c, &flags);
        if (lane == 31) s.part[wp] = x;
        if (flags) atomicOr(&s.flags, flags);
        __syncthreads();
        before = total;
#pragma unroll 1
        for (int i = 0; i < parts; ++i) total += s.part[i];
        if (base + kThreads < a.N) __syncthreads();
    }
    const bool one_round = a.N <= kThreads;
    total *= a.HKV;
    if (s.flags || total == 0) return;
    const long long shares = min(total, static_cast<long long>(gridDim.x));
    if (blockIdx.x >= shares) return;
    // (a tile each needs no division, which takes 200 cycles)
    long long begin = blockIdx.x, end = begin + 1;
    if (total > shares) {
        begin = div_by(total * begin, shares);
        end = div_by(total * end, shares);
    }
    before = 0;
    for (int base = 0; base < a.N; base += kThreads) {
        if (!one_round) {
            __syncthreads();
            x = scan(base + tid, q, c, nullptr);
            if (lane == 31) s.part[wp] = x;
            __syncthreads();
        }
        long long from = before;
#pragma unroll 1
        for (int i = 0; i < parts; ++i) {
            if (i < wp) from += s.part[i];
            before += s.part[i];
        }
        from = (from + x - c) * a.HKV;
        if (begin >= from && begin < from + c * a.HKV) {
            s.begin = begin;
            s.left = end - begin;
            s.total = total;
            s.shares = shares;
            s.n = base + tid;
            s.q = q;
            s.in_seq = begin - from;
            s.cost = c;
        }
        if (before * a.HKV > begin) break;
    }
}

// The segments of a share, one after the other; a warp walks together.
struct Walk {
    const AttnParams &a;
    int tokens;
    int n, h, m, off;       // item, how much of its cost has been given out
    int items;              // row-tile groups of the sequence
    long long left;
    bool first;
    Seq q;                  // this sequence
    int64_t end_ahead;      // and the next one's numbers, read ahead
    int len_ahead;

    __device__ void read_ahead() {
        end_ahead = 0;
        len_ahead = 0;
        if (n + 1 < a.N) {
            end_ahead = cu_of(a.cu, a.cu64, n + 2);
            len_ahead = a.kv_lens[n + 1];
        }
    }

    __device__ void enter() { items = q.fresh <= tokens ? 1 : (q.fresh + tokens - 1) / tokens; }
    __device__ Walk(const AttnParams &a_, int tokens_, const Share &s) : a(a_), tokens(tokens_) {
        left = s.left;
        first = true;
        h = m = off = items = n = 0;
        q = {0, 0, 0};
        if (left <= 0) return;
        n = s.n;
        q = s.q;
        read_ahead();
        enter();
        h = static_cast<int>(div_by(s.in_seq, s.cost));
        long long at = s.in_seq - h * s.cost;
        if (items == 1) {
            off = static_cast<int>(at);
            return;
        }
        // the item that holds tile `at` of the head
        const int lane = threadIdx.x & 31;
        if (items > 32 && closed_form(a, q.len, q.fresh)) {
            // narrow down to 32 items: lanes try as many places at once
            int lo = 0, hi = items;
            while (hi - lo > 32) {
                const int step = (hi - lo + 31) / 32, i = lo + lane * step;
                const uint32_t before = __ballot_sync(0xffffffffu, i < hi && cost_of(a, q.len, q.fresh, tokens, i) <= at);
                const int k = 31 - __clz(before | 1);
                lo += k * step;
                hi = min(hi, lo + step);
            }
            at -= cost_of(a, q.len, q.fresh, tokens, lo);
            m = lo;
        }
        for (;; m += 32) {
            const int cost = m + lane < items ? item_cost(a, q.len, q.fresh, tokens, m + lane) : 0;
            int sum = cost;
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += x;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, sum > at);
            if (past || m + 32 >= items) {
                const int k = past ? __ffs(past) - 1 : 0;
                at -= __shfl_sync(0xffffffffu, sum - cost, k);
                m += k;
                break;
            }
            at -= __shfl_sync(0xffffffffu, sum, 31);
        }
        off = static_cast<int>(at);
    }
    // The next segment; false at the end.  `cut`: it ends before its item does,
    // by `rest` key tiles.
    __device__ bool next(Segment &g, int &rest) {
        rest = 0;
        if (left <= 0) return false;
        const int j0 = m * tokens;
        const Span s = key_span(a, q.len, q.fresh, j0, min(q.fresh, j0 + tokens));
        const int lead = lead_of(a, q.fresh, tokens, m), tiles = max(1, s.hi - s.lo), cost = lead + tiles;
        const int take = static_cast<int>(min(static_cast<long long>(cost - off), left));
        const int from = max(0, off - lead), to = max(0, off + take - lead);  // key tiles
        left -= take;
        if (to == from) return false;  // the share ends in the item's lead: the next one has it all
        g.seq = n;
        g.tok0 = q.t0 + j0;
        g.h = h;
        g.ntok = min(tokens, q.fresh - j0);
        g.slot = from > 0 || to < tiles ? 2 * static_cast<int>(blockIdx.x) + (first ? 0 : 1) : -1;
        g.lo = s.lo + from;
        g.hi = s.hi == s.lo ? g.lo : s.lo + to;
        g.begin = s.begin;
        g.end = s.end;
        g.place = q.len - q.fresh + j0;
        rest = cost - off - take;
        if (from > 0) rest = -rest;  // only the piece that begins the item reports the cut
        first = false;
        off = 0;
        if (++m == items) {
            m = 0;
            if (++h == a.HKV) {
                h = 0;
                // (the lengths have been checked)
                do {
                    ++n;
                    q.t0 += q.fresh;
                    q.fresh = n < a.N ? static_cast<int>(end_ahead) - q.t0 : 0;
                    q.len = len_ahead;
                    read_ahead();
                } while (q.fresh == 0 && n < a.N);
                enter();
            }
        }
        return true;
    }
};

// ------------------------------------------------------------------- main
// What the warps share besides the tiles.
template <int STAGES>
struct Small {
    uint64_t full[STAGES], empty[STAGES], tail, drain;
    uint64_t seg_full[kSegRing], seg_empty[kSegRing];
    uint64_t q_full[2], q_free[2];                     // of row tile t
    uint64_t s_full[2], p_half[2], p_full[2], o_full[2];  // of stream x
    uint64_t s_free[2], p_free[2];  // and with weights apart: scores read, weights used
    uint64_t ml_full, o_free;  // one row tile: group 1's statistics are in; group 0 has read the outputs
    Segment seg[kSegRing];
    Share share;
    float2 ml[kTile];
    uint32_t tmem;
};

template <int D>
struct Cfg {
    static constexpr int kStageBytes = kTile * D * 2;
    static constexpr int kQBytes = kTile * D * 2;
    static constexpr int kStages = D == 128 ? 5 : 10;  // what fits beside the query tiles
    static constexpr int kRing = 2 * kQBytes;
    // Weights apart: they have Tensor Memory of their own, so that the next scores
    // are computed while the softmax works on these (it holds them in registers).
    // With D = 128 scores and outputs take it all and the weights replace the scores.
    static constexpr bool kApart = D == 64;
    static constexpr int kShared = kRing + kStages * kStageBytes;  // the barriers and small arrays
    static constexpr int kSmem = kShared + static_cast<int>(sizeof(Small<kStages>));
    static_assert(kSmem <= 232448, "shared memory of a block");
};

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, const int (&c)[4], uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c[0]), "r"(c[1]), "r"(c[2]), "r"(c[3]), "r"(smem_u32(bar))
        : "memory");
}

// Tensor Memory in the shape of 16 lanes, 64 columns: thread t has lanes t / 4 (h =
// 0) and t / 4 + 8 (h = 1) of the 16 from the address's lane on, r[4 n + 2 h + e] =
// column 8 n + 2 (t % 4) + e.
__device__ __forceinline__ void tmem_ld_rows(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
// Thread q of a quad gives w[k] to thread k and gets thread k's w[q] as w[k].
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int q) {
    const bool odd = q & 1, high = q & 2;
    uint32_t a = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1), b = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
    // pairs of group q & 1 and of group 2 + (q & 1)
    uint32_t lo0 = odd ? a : w[0], lo1 = odd ? w[1] : a, hi0 = odd ? b : w[2], hi1 = odd ? w[3] : b;
    a = __shfl_xor_sync(0xffffffffu, high ? lo0 : hi0, 2);
    b = __shfl_xor_sync(0xffffffffu, high ? lo1 : hi1, 2);
    w[0] = high ? a : lo0;
    w[1] = high ? b : lo1;
    w[2] = high ? hi0 : a;
    w[3] = high ? hi1 : b;
}

// One thread of the warp, the same each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// Shared-memory descriptors as two words: the low one (address, leading-dimension
// offset) changes by a constant from step to step, the high one (stride of the
// 8-row groups, version, 128-byte swizzle) never does.  Building them from a
// base per stage keeps the issuing thread's work per product to an addition.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | (lbo >> 4) << 16; }
// products of 16 keys or channels (see mma_f16, mma_f16_ta)
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\n.reg .b64 a, b;\n"
        "mov.b64 a, {%1, %4};\nmov.b64 b, {%2, %4};\n"
        "setp.ne.b32 p, %5, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kDescHi), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\n.reg .b64 b;\n"
        "mov.b64 b, {%2, %4};\n"
        "setp.ne.b32 p, %5, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "n"(kDescHi), "r"(acc)
        : "memory");
}

// Two fp32 values in a 64-bit register pair, and the packed operations on them.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// The same, and 2^x, kept in the order in which they are written.
__device__ __forceinline__ uint64_t fma2_here(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm volatile("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float ex2_here(float x) {
    float r;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return r;
}

// The lowest n bits set (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0 : (1u << n) - 1;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1) gdn2_paged_attn_kernel(const __grid_constant__ KernelParams p) {
    using C = Cfg<D>;
    constexpr int NB = D / 64;  // 64-channel blocks of a row
    extern __shared__ __align__(1024) uint8_t smem[];
    Small<C::kStages> &sh = *reinterpret_cast<Small<C::kStages> *>(smem + C::kShared);
    uint64_t *const full = sh.full, *const empty = sh.empty;
    const AttnParams &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
    // The 128-byte swizzle goes by address: the dynamic shared memory, the only
    // one of this kernel, has to begin on a 1024-byte boundary, as it does (the
    // room left does not allow for slack).  Checked all the same.
    if (smem_u32(smem) & 1023) {
        if (tid == 0) {
            p.flags[blockIdx.x] = kTimeout;
            p.joint[blockIdx.x].more = 0;
        }
        return;
    }

    if (wp == 0) {
        if (lane < C::kStages) {
            mbar_init(&full[lane], 1);
            mbar_init(&empty[lane], 1);
        }
        if (lane < kSegRing) {
            mbar_init(&sh.seg_full[lane], 1);
            mbar_init(&sh.seg_empty[lane], 11);  // the warps but the one that hands them out
        }
        if (lane < 2) {
            mbar_init(&sh.q_full[lane], 1);
            mbar_init(&sh.q_free[lane], 1);
            mbar_init(&sh.s_full[lane], 1);
            mbar_init(&sh.p_half[lane], 4);
            mbar_init(&sh.p_full[lane], 4);
            mbar_init(&sh.o_full[lane], 1);
            mbar_init(&sh.s_free[lane], 4);
            mbar_init(&sh.p_free[lane], 1);
        }
        if (lane == 0) {
            mbar_init(&sh.tail, 1);
            mbar_init(&sh.drain, 1);
            mbar_init(&sh.ml_full, 4);
            mbar_init(&sh.o_free, 4);
            sh.share.flags = 0;
            sh.share.left = 0;
        }
        fence_mbar_init();
    }
    if (wp == kMmaWarp) tmem_alloc(&sh.tmem, 512);
    if (tid == 32 * kKeyWarp && a.T > 0) {
        prefetch_map(&p.tk);
        prefetch_map(&p.tv);
        if (p.q_map) prefetch_map(&p.tq);
    }
    pdl_trigger();
    __syncthreads();
    find_share(a, 2 * p.tt, sh.share);
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sh.tmem;
    const uint32_t sQ = smem_u32(smem), sRing = smem_u32(smem + C::kRing);
    // Tensor Memory columns: scores of stream x at 128 x, the outputs after them, the
    // weights (16 bits, 64 columns) after those or in the scores' place
    auto tS = [&](int x) { return tm + 128 * x; };
    auto tO = [&](int x) { return tm + 256 + D * x; };
    auto tP = [&](int x) { return C::kApart ? tm + 256 + 2 * D + 64 * x : tS(x); };
    auto fail = [&]() { atomicOr(&sh.share.flags, kTimeout); };
    auto few_regs = [] { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs)); };
    // the i-th segment of the share; its last reader in a warp releases it
    auto seg_wait = [&](uint32_t i) { return warp_wait(&sh.seg_full[i % kSegRing], (i / kSegRing) & 1); };
    auto seg_done = [&](uint32_t i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[i % kSegRing]);
    };

    // Keys or values of a segment's tiles into the ring, by one warp.  `at`: the
    // place of tile i's load among the segment's 2 x tiles, in the order in which
    // the products take them: first n keys' tiles, then values and keys in turn.  The
    // releases come in the same order, so that a stage's emptiness is never
    // mistaken for an earlier one's.
    auto keys_ahead = [](bool two) { return (two ? 1 : 2) + (C::kApart ? 1 : 0); };
    auto key_at = [&](int i, bool two) { return i < keys_ahead(two) ? i : 2 * i - keys_ahead(two) + 1; };
    auto value_at = [&](int i, int tiles, bool two) { return min(2 * i + keys_ahead(two), tiles + i); };
    struct Loader {
        uint32_t base = 0, used = 0;  // loads of the segments before; one past this warp's last
        int tail_ph = 0;
        bool ok = true;
    };
    auto load_tiles = [&](Loader &ld, const Segment &g, bool is_v, auto at, auto ahead) {
        // (a division takes 100 to 200 cycles, and these stand before the first copy)
        const int gran = p.granule, per_log2 = 7 - p.granule_log2, per = 1 << per_log2;  // granules of a tile
        const int batch = 32 >> per_log2;                   // tiles whose table entries one load fetches
        const int my_gr = lane / NB, my_cb = lane % NB;     // this lane's granule and channel block
        const int tiles = g.hi - g.lo;
        const int *row = a.table + static_cast<int64_t>(g.seq) * a.table_stride;
        const int *pos = is_v ? p.vpos : p.kpos;
        // page and slot of this lane's granule of the batch that starts at tile t
        auto fetch = [&](int t) {
            t += lane >> per_log2;
            int2 e = make_int2(0, 0);
            const int key = t * kTile + (lane & (per - 1)) * gran;
            if (t < g.hi && key + gran <= g.begin) {
                e.x = static_cast<int>(a.num_pages);  // before the window, where the page may be gone: zeros
            } else if (t < g.hi && key < g.end) {
                const int col = quotient(key, p.page);
                e = make_int2(row[col], key - col * a.page_size);
                if (e.x < 0 || e.x >= a.num_pages) {
                    e.x = static_cast<int>(a.num_pages);  // past the tensor: the box reads zeros
                    atomicOr(&sh.share.flags, kBadPages);
                }
            }
            return e;
        };
        int skip = max(0, g.begin - g.lo * kTile);          // first rows of the first tile that do not count
        int2 now = fetch(g.lo), next = fetch(g.lo + batch);
        if (ld.base > 0) ahead();
        for (int i = 0, in = 0; i < tiles && ld.ok; ++i) {
            if (i == 1 && ld.base == 0) ahead();
            const uint32_t load = ld.base + at(i);
            const int st = static_cast<int>(load % C::kStages);
            const int left = min(kTile, g.end - (g.lo + i) * kTile);  // rows that count
            const int grans = (left + gran - 1) >> p.granule_log2;
            ld.ok = ld.ok && warp_wait(&empty[st], ((load / C::kStages) & 1) ^ 1);
            if (!ld.ok) return;
            const bool patch = is_v && (left < kTile || skip > 0);
            uint64_t *bar = patch ? &sh.tail : &full[st];
            uint8_t *dst = smem + C::kRing + st * C::kStageBytes;
            if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(grans * gran * 128 * NB));
            __syncwarp();
            const int from = in * per + min(my_gr, per - 1);
            const int page = __shfl_sync(0xffffffffu, now.x, from), slot = __shfl_sync(0xffffffffu, now.y, from);
            if (my_gr < grans) {
                int c[4] = {my_cb * 64, 0, 0, 0};
#pragma unroll
                for (int k = 1; k < 4; ++k) c[k] = pos[0] == k ? page : pos[1] == k ? slot : g.h;
                tma_load_4d(dst + my_cb * (kTile * 128) + my_gr * gran * 128, is_v ? &p.tv : &p.tk, c, bar);
            }
            ld.used = load + 1;
            if (patch) {  // zero the rows outside the range, once the copies are in
                ld.ok = warp_wait(&sh.tail, ld.tail_ph);
                if (!ld.ok) return;
                ld.tail_ph ^= 1;
                for (int k = lane; k < (skip + kTile - left) * NB * 8; k += 32) {
                    const int n = k / (NB * 8), r = n < skip ? n : left + n - skip, q = k % (NB * 8);
                    *reinterpret_cast<uint4 *>(dst + (q >> 3) * (kTile * 128) + r * 128 + (q & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[st]);
                skip = 0;
            }
            if (++in == batch) {
                in = 0;
                now = next;
                next = fetch(g.lo + i + 1 + batch);
            }
        }
        if (tiles == 1 && ld.base == 0) ahead();
        ld.base += 2 * tiles;
    };
    // a loader that gave up lets its copies in flight land before the block ends
    auto settle = [&](const Loader &ld) {
        if (ld.ok) return;
        if (lane == 0) fail();
        for (uint32_t i = ld.used > C::kStages ? ld.used - C::kStages : 0; i < ld.used; ++i)
            warp_wait(&full[i % C::kStages], (i / C::kStages) & 1);
    };

    if (wp == kKeyWarp) {
        // ----------------------------------------------- segments and keys
        few_regs();
        uint32_t pushed = 0;  // segments handed out
        Joint joint = {};
        Loader ld;
        Walk walk(a, 2 * p.tt, sh.share);
        // The next segment that has keys, handed out; the others' rows are
        // written here.  tok0 = -1 ends the share.
        Segment g;
        auto hand_out = [&]() {
            for (;;) {
                int rest;
                if (!walk.next(g, rest)) {
                    g.tok0 = -1;
                    break;
                }
                if (rest > 0) {
                    // the item goes on in the shares that its last tile reaches
                    joint = {g.tok0, g.h, g.ntok, g.slot, 0, {0, 0, 0}};
                    const long long last = sh.share.begin + sh.share.left + rest - 1;
                    joint.more = static_cast<int>(div_by((last + 1) * sh.share.shares - 1, sh.share.total)) - static_cast<int>(blockIdx.x);
                }
                if (g.hi > g.lo) break;
                for (int i = lane; i < g.ntok * a.G; i += 32) {
                    const int64_t tok = g.tok0 + i / a.G;
                    const int head = g.h * a.G + i % a.G;
                    bf16 *o = a.out + tok * a.so_t + head * a.so_h;
                    for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4 *>(o + c) = make_uint4(0, 0, 0, 0);
                    if (a.lse) a.lse[tok * a.HQ + head] = -INFINITY;
                }
            }
            ld.ok = ld.ok && warp_wait(&sh.seg_empty[pushed % kSegRing], ((pushed / kSegRing) & 1) ^ 1);
            if (!ld.ok) return;
            if (lane == 0) {
                sh.seg[pushed % kSegRing] = g;
                mbar_arrive(&sh.seg_full[pushed % kSegRing]);
            }
            __syncwarp();
            ++pushed;
        };
        hand_out();
        while (ld.ok && g.tok0 >= 0) {
            const Segment cur = g;
            const bool two = cur.ntok > p.tt;
            // (the next one is handed out before this one's copies, so that its
            // queries can be loaded early; after the first copy at the very start)
            load_tiles(ld, cur, false, [&](int i) { return key_at(i, two); }, hand_out);
        }
        if (lane == 0) p.joint[blockIdx.x] = joint;
        settle(ld);
    } else if (wp == kValueWarp) {
        // ---------------------------------------------------------- values
        few_regs();
        Loader ld;
        for (uint32_t s = 0; ld.ok; ++s) {
            ld.ok = seg_wait(s);
            if (!ld.ok || sh.seg[s % kSegRing].tok0 < 0) break;
            const Segment cur = sh.seg[s % kSegRing];
            seg_done(s);
            const bool two = cur.ntok > p.tt;
            load_tiles(ld, cur, true, [&](int i) { return value_at(i, cur.hi - cur.lo, two); }, [] {});
        }
        settle(ld);
    } else if (wp == kQueryWarp) {
        // --------------------------------------------------------- queries
        few_regs();
        uint32_t uses[2] = {0, 0};  // of row tile t so far
        const uint32_t inv_g = 65536u / a.G + 1;  // r / G for r < 128
        bool ok = true;
        for (uint32_t s = 0; ok; ++s) {
            ok = seg_wait(s);
            if (!ok || sh.seg[s % kSegRing].tok0 < 0) break;
            const Segment g = sh.seg[s % kSegRing];
            seg_done(s);
            const int nt = g.ntok > p.tt ? 2 : 1;
            for (int t = 0; t < nt && ok; ++t) {
                // the scores of the tile's last use are in
                ok = warp_wait(&sh.q_free[t], (uses[t] & 1) ^ 1);
                ++uses[t];
                if (!ok) break;
                uint8_t *dst = smem + t * C::kQBytes;
                if (p.q_map) {
                    // one box per 64 channels: G heads of tt tokens, in the order of
                    // the tile's rows.  Rows past the item's (or the tile's) tokens
                    // hold what is there: no row depends on another.
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&sh.q_full[t], static_cast<uint32_t>(a.G * p.tt * 128 * NB));
                        for (int cb = 0; cb < NB; ++cb)
                            tma_load_3d(dst + cb * (kTile * 128), &p.tq, 64 * cb, g.h * a.G, g.tok0 + t * p.tt, &sh.q_full[t]);
                    }
                    __syncwarp();
                    continue;
                }
                // a layout that the map cannot describe: copies of 16 bytes
                const int rows = min(p.tt, g.ntok - t * p.tt) * a.G;
                const bf16 *q = a.q + (static_cast<int64_t>(g.tok0) + t * p.tt) * a.sq_t + static_cast<int64_t>(g.h) * a.G * a.sq_h;
                constexpr int L = D / 8;  // lanes per row
                const int ch = lane % L;
                dst += (ch >> 3) * (kTile * 128);
#pragma unroll 4
                for (int r = lane / L; r < rows; r += 32 / L) {
                    const int tok = static_cast<int>((r * inv_g) >> 16), hd = r - tok * a.G;
                    cp_async16(dst + swz(r, ch & 7), q + tok * a.sq_t + hd * a.sq_h + 8 * ch, 16);
                }
                cp_async_wait_all();
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_full[t]);
            }
        }
        if (!ok && lane == 0) fail();
        // (a copy that is in flight when the warp gives up is one whose barrier the
        // issuing warp waits for; let it land)
        for (int t = 0; t < 2 && !ok; ++t)
            if (uses[t] > 0) warp_wait(&sh.q_full[t], (uses[t] - 1) & 1);
    } else if (wp == kMmaWarp) {
        // ------------------------------------------- tensor cores: one thread
        // One elected thread does it all.  With elect.sync the compiler keeps
        // descriptors and addresses in uniform registers, and a product of 16 keys
        // costs 23 cycles to issue; under `lane == 0` it moves them there one by
        // one, 54 cycles, which the 64 cycles that the product takes do not hide
        // once waits come between.  Waits, votes and elections by the whole warp
        // cost another 350 of 2800 cycles per two tiles beside busy softmax warps.
        few_regs();
        if (elect_one()) {
            constexpr uint32_t kIdS = idesc_f16kind(kTile, kTile, false, false, !F16);
            constexpr uint32_t kIdO = idesc_f16kind(kTile, D, false, true, !F16);
            uint32_t taken = 0;                  // stages taken so far
            uint32_t q_ph[2] = {0, 0}, p_ph[2] = {0, 0};
            uint32_t s_ph[2] = {1, 1};           // of s_free; the first wait passes
            bool ok = true;
            const uint32_t dq = desc_lo(sQ, 16);
            auto stage = [&](uint32_t i) { return sRing + (i % C::kStages) * C::kStageBytes; };
            auto wait_stage = [&](uint32_t i) { ok = ok && mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1); };
            // S of stream x = Q K^T with row tile t; then the stage is free if `last`, and
        // the queries' tile if `q_last`
            auto scores = [&](int x, int t, uint32_t k, bool last, bool q_last) {
                if (C::kApart) {
                    ok = ok && mbar_wait(&sh.s_free[x], s_ph[x]);
                    s_ph[x] ^= 1;
                }
                if (!ok) return;
                tc_fence_after();
                const uint32_t dk = desc_lo(stage(k), 16);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    constexpr uint32_t kBlock = kTile * 128 / 16;  // 64 channels of a tile
                    const uint32_t step = (kk >> 2) * kBlock + (kk & 3) * 2;
                    mma_ss(tS(x), dq + t * (C::kQBytes / 16) + step, dk + step, kIdS, kk > 0);
                }
                mma_commit(&sh.s_full[x]);
                if (last) mma_commit(&empty[k % C::kStages]);
                if (q_last) mma_commit(&sh.q_free[t]);
            };
            // O of stream x (+)= P V, each half of the keys as soon as its weights are
            // in; then the stage is free if `free`, and the outputs complete if `done`
            auto output = [&](int x, uint32_t v, bool first, bool free, bool done) {
                const uint32_t dv = desc_lo(stage(v), kTile * 128);
                ok = ok && mbar_wait(&sh.p_half[x], p_ph[x]);
                if (!ok) return;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kTile / 32; ++kk)
                    mma_ts(tO(x), tP(x) + 8 * kk, dv + 128 * kk, kIdO, kk > 0 || !first);
                ok = mbar_wait(&sh.p_full[x], p_ph[x]);
                p_ph[x] ^= 1;
                if (!ok) return;
                tc_fence_after();
#pragma unroll
                for (int kk = kTile / 32; kk < kTile / 16; ++kk)
                    mma_ts(tO(x), tP(x) + 8 * kk, dv + 128 * kk, kIdO, 1);
                if (C::kApart) mma_commit(&sh.p_free[x]);
                if (free) mma_commit(&empty[v % C::kStages]);
                if (done) mma_commit(&sh.o_full[x]);
            };
            auto wait_q = [&](int t) {
                ok = ok && mbar_wait(&sh.q_full[t], q_ph[t]);
                q_ph[t] ^= 1;
            };
            for (uint32_t s = 0; ok; ++s) {
                ok = mbar_wait(&sh.seg_full[s % kSegRing], (s / kSegRing) & 1);
                if (!ok) break;
                const Segment &g = sh.seg[s % kSegRing];
                if (g.tok0 < 0) break;
                const int tiles = g.hi - g.lo;
                const bool two = g.ntok > p.tt;
                mbar_arrive(&sh.seg_empty[s % kSegRing]);
                uint32_t k = taken++;
                wait_stage(k);
                wait_q(0);
                scores(0, 0, k, !two, tiles == 1);
                if (two) {
                    wait_q(1);
                    scores(1, 1, k, true, tiles == 1);
                    for (int i = 0; i < tiles && ok; ++i) {
                        const bool more = i + 1 < tiles;
                        if (C::kApart) {
                            if (more) {
                                k = taken++;
                                wait_stage(k);
                                scores(0, 0, k, false, i + 2 == tiles);
                                scores(1, 1, k, true, i + 2 == tiles);
                            }
                            const uint32_t v = taken++;
                            wait_stage(v);
                            output(0, v, i == 0, false, !more);
                            output(1, v, i == 0, true, !more);
                            continue;
                        }
                        const uint32_t v = taken++;
                        if (more) k = taken++;
                        wait_stage(v);
                        output(0, v, i == 0, false, !more);
                        if (more) {
                            wait_stage(k);
                            scores(0, 0, k, false, i + 2 == tiles);
                        }
                        output(1, v, i == 0, true, !more);
                        if (more) scores(1, 1, k, true, i + 2 == tiles);
                    }
                } else {
                    if (tiles > 1) {
                        k = taken++;
                        wait_stage(k);
                        scores(1, 0, k, true, tiles == 2);
                    }
                    for (int i = 0; i < tiles && ok; ++i) {
                        auto next = [&] {
                            if (i + 2 >= tiles) return;
                            k = taken++;
                            wait_stage(k);
                            scores(i & 1, 0, k, true, i + 3 == tiles);
                        };
                        if (C::kApart) next();
                        const uint32_t v = taken++;
                        wait_stage(v);
                        output(i & 1, v, i < 2, true, i + 2 >= tiles);
                        if (!C::kApart) next();
                    }
                }
            }
            // nothing may run on in Tensor Memory once it is released
            mma_commit(&sh.drain);
            if (!mbar_wait(&sh.drain, 0) || !ok) fail();
        }
        __syncwarp();
    } else if (wp < 8) {
        // ------------------------------------------- softmax: a thread per row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int x = wp >> 2, row = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(wp & 3) << 21;  // TMEM lane of the warp's first row
        const uint32_t inv_g = 65536u / a.G + 1;                     // r / G for r < 128
        using W = Weights<F16>;
        const float sl2 = p.scale_log2, slack = fminf(W::kLag / sl2, 1e38f), drop = fminf(W::kDrop / sl2, 1e38f);
        const int my_tok = static_cast<int>((row * inv_g) >> 16), my_head = row - my_tok * a.G;
        // A group signals with one arrival per warp: 128 arrivals on one barrier
        // take their turns, which the products waited for.
        auto arrive = [&](uint64_t *bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        bool ok = seg_wait(0);
        uint32_t steps = 0;              // tiles of this stream so far
        uint32_t o_ph[2] = {0, 0};       // segments in which stream 0, 1 had tiles
        uint32_t merges = 0;             // segments that were merged
        // One segment; compiled once for two row tiles and once for one (a common
        // loop ran 8 % slower on the former).
        auto segment = [&](uint32_t s, auto two_tiles) {
            constexpr bool TWO = decltype(two_tiles)::value;
            const Segment &g = sh.seg[s % kSegRing];
            const int tiles = g.hi - g.lo;
            const bool merged = !TWO && tiles > 1;
            // the row's token in the segment, -1 if it has none
            const int tile = TWO ? x : 0;
            const int tok = my_tok < p.tt && tile * p.tt + my_tok < g.ntok ? tile * p.tt + my_tok : -1;
            // keys [from, upto) for this row; rows without a token take what they get
            const int place = g.place + (tok < 0 ? 0 : tok);
            const int upto = tok < 0 ? 0x7fffffff : a.causal ? place + 1 : g.end;
            const int from = tok >= 0 && a.window >= 0 ? max(0, max(0, place) - a.window) : 0;
            const bool idle = !__any_sync(0xffffffffu, tok >= 0);  // no row of the warp has a token
            constexpr int stride = TWO ? 1 : 2;
            const int begin = TWO ? 0 : x;
            float m = -INFINITY, l = 0.f;
            // the first key of the tile, and the row's keys relative to it
            int lo = from - (g.lo + begin) * kTile, hi = upto - (g.lo + begin) * kTile;
            for (int i = begin; i < tiles && ok; i += stride, ++steps, lo -= stride * kTile, hi -= stride * kTile) {
                ok = warp_wait(&sh.s_full[x], steps & 1);
                if (!ok) break;
                // group 1's outputs of the last merged segment have to be read
                if (x == 1 && i == begin && merges > 0) ok = ok && warp_wait(&sh.o_free, (merges - 1) & 1);
                if (!ok) break;
                // Waits until the stream's last product is in and weights and outputs may
                // be written.  (With the weights in the scores' place it is: these
                // scores followed it.)
                auto used = [&] {
                    if (!C::kApart || steps == 0) return;
                    ok = warp_wait(&sh.p_free[x], (steps - 1) & 1);
                    tc_fence_after();
                };
                if (!idle) {
                    tc_fence_after();
                    uint32_t u[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(tS(x) + lanes + 32 * c, u[c]);
                    tmem_ld_wait();
                    if (C::kApart) {
                        tc_fence_before();
                        arrive(&sh.s_free[x]);
                    }
                    if (__any_sync(0xffffffffu, lo > 0 || hi < kTile)) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            // bit e: key 32 c + e is one of the row's
                            const uint32_t bits = low_bits(hi - 32 * c) & ~low_bits(lo - 32 * c);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(bits >> e & 1)) u[c][e] = 0xff800000u;
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 128; c += 2)
                        mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], u[c >> 5][c & 31], u[c >> 5][(c & 31) + 1]);
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if (i == begin) {
                        m = top;
                    } else {
                        const bool grow = top > m + slack, fall = F16 && top < m - drop && top > -INFINITY;
                        if (__any_sync(0xffffffffu, grow || fall)) {
                            float f = 1.f;
                            if (grow || fall) {
                                f = ex2((m - top) * sl2);
                                if (!fall || l * f < W::kMost) m = top;
                                else f = 1.f;
                            }
                            l *= f;
                            used();
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t o[32];
                                tmem_ld32(tO(x) + lanes + c, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st32(tO(x) + lanes + c, o);
                            }
                        }
                    }
                    const float base = m == -INFINITY ? 0.f : m * sl2 - W::kBias;
                    const uint64_t scale2 = pair(sl2, sl2), base2 = pair(-base, -base);
                    uint64_t sum2[4] = {0, 0, 0, 0};
                    // The weights in groups of 8 scores, three of them under way: the
                    // arguments of the next, the exponentials of this and the sums
                    // and conversions of the last.  The order is written out (and
                    // kept by `volatile`): left to the compiler, a tile took 1.6 k to
                    // 2.1 k cycles alone and two tiles 2.1 k to 2.4 k on the same
                    // schedulers, against 0.9 k and 1.3 k this way; the
                    // special-function unit's own time is 0.5 k a tile.
                    uint64_t arg[2][4];
                    float ex[2][8] = {};
                    uint32_t w[16];
                    auto args = [&](int n) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int c = 8 * n + 2 * e;
                            arg[n & 1][e] = fma2_here(pair(__uint_as_float(u[c >> 5][c & 31]), __uint_as_float(u[c >> 5][(c & 31) + 1])), scale2, base2);
                        }
                    };
                    auto finish = [&](int n, int e) {
                        const float a0 = ex[n & 1][2 * e], a1 = ex[n & 1][2 * e + 1];
                        sum2[e] = add2(sum2[e], pair(a0, a1));
                        w[4 * (n & 3) + e] = F16 ? pack_f16_rn(a0, a1) : pack_bf2(a0, a1);
                    };
                    args(0);
#pragma unroll
                    for (int n = 0; n <= 16; ++n) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (n < 16) {
                                const float2 z = unpair(arg[n & 1][e]);
                                ex[n & 1][2 * e] = ex2_here(z.x);
                                if (e == 1 && n < 15) args(n + 1);
                                ex[n & 1][2 * e + 1] = ex2_here(z.y);
                            }
                            if (n > 0) finish(n - 1, e);
                        }
                        if (n == 4) used();
                        if (n > 0 && n % 4 == 0) tmem_st16(tP(x) + lanes + 4 * (n - 4), w);
                        if (n == 9) {  // the first half of the keys: their product may begin
                            tmem_st_wait();
                            tc_fence_before();
                            arrive(&sh.p_half[x]);
                        }
                    }
                    const float2 t = unpair(add2(add2(sum2[0], sum2[1]), add2(sum2[2], sum2[3])));
                    l += t.x + t.y;
                    tmem_st_wait();
                    tc_fence_before();
                } else {
                    if (C::kApart) arrive(&sh.s_free[x]);
                    used();  // each phase is awaited, so that none is taken for another
                    arrive(&sh.p_half[x]);
                }
                arrive(&sh.p_full[x]);
            }
            if (!ok) return;
            if (merged && x == 1) {  // group 0 merges
                sh.ml[row] = make_float2(m, l);
                arrive(&sh.ml_full);
            }
            if (TWO || x == 0) {
                // where the row goes, while the last product runs
                const bool whole = g.slot < 0;
                const int head = g.h * a.G + my_head;
                const int64_t tok_row = static_cast<int64_t>(g.tok0) + max(tok, 0);
                const int64_t part = static_cast<int64_t>(max(g.slot, 0)) * 2 * kTile + tile * kTile + row;
                const uint64_t dst = tok < 0 ? 0
                                     : whole ? reinterpret_cast<uint64_t>(a.out + tok_row * a.so_t + head * a.so_h)
                                             : reinterpret_cast<uint64_t>(p.part_o + part * D);
                float f0 = 1.f, f1 = 0.f;
                if (merged) {
                    ok = warp_wait(&sh.ml_full, merges & 1);
                    const float2 ml = sh.ml[row];
                    const float peak = fmaxf(m, ml.x), base = peak == -INFINITY ? 0.f : peak * sl2;
                    f0 = ex2(fmaf(m, sl2, -base));
                    f1 = ex2(fmaf(ml.x, sl2, -base));
                    m = peak;
                    l = f0 * l + f1 * ml.y;
                }
                if (tok >= 0) {
                    const float base = m == -INFINITY ? -INFINITY : m * sl2 - W::kBias;
                    if (!whole)
                        p.part_ml[part] = make_float2(base, l);
                    else if (a.lse)
                        a.lse[tok_row * a.HQ + head] = l == 0.f ? -INFINITY : (base + log2f(l)) * kLn2;
                }
                if (whole) {
                    const float inv = l == 0.f ? 0.f : __frcp_rn(l);
                    f0 *= inv;
                    f1 *= inv;
                }
                ok = ok && warp_wait(&sh.o_full[x], o_ph[x] & 1) && (!merged || warp_wait(&sh.o_full[1], o_ph[1] & 1));
                if (!ok) return;
                tc_fence_after();
                if (!idle) {
                    // The rows out: the outputs are read in the shape of 16 lanes, a
                    // quad of threads per row, and exchanged within the quad so that
                    // it stores 64 consecutive bytes of the row (16 per thread): a
                    // store then touches 8 lines instead of the 32 of a thread per
                    // row, which took 4 k cycles an item.
                    const int q = lane & 3;
                    const uint32_t rows_in = __ballot_sync(0xffffffffu, tok >= 0);
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        if (!(rows_in >> (16 * half) & 0xffffu)) continue;
                        const uint32_t at = lanes + (static_cast<uint32_t>(16 * half) << 16);
                        uint32_t u[32];  // [4 n + 2 h + e]: row h, column c + 8 n + 2 q + e
                        __syncwarp();
                        tmem_ld_rows(tO(x) + at, u);
                        float g0[2], g1[2];
                        uint64_t o[2];  // 0: no row
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int src = 16 * half + 8 * h + (lane >> 2);  // the thread that has the row
                            g0[h] = __shfl_sync(0xffffffffu, f0, src);
                            g1[h] = merged ? __shfl_sync(0xffffffffu, f1, src) : 0.f;
                            o[h] = __shfl_sync(0xffffffffu, dst, src);
                        }
#pragma unroll 1
                        for (int c = 0; c < D; c += 64) {
                            if (c > 0) tmem_ld_rows(tO(x) + at + c, u);
                            tmem_ld_wait();
                            if (merged) {
                                uint32_t v[32];
                                tmem_ld_rows(tO(1) + at + c, v);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    u[e] = __float_as_uint(__uint_as_float(u[e]) * g0[(e >> 1) & 1] + __uint_as_float(v[e]) * g1[(e >> 1) & 1]);
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * g0[(e >> 1) & 1]);
                            }
                            if (whole) {
#pragma unroll
                                for (int n = 0; n < 8; n += 4)
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        uint32_t w[4];  // columns 8 (n + k) + 2 q, + 1
#pragma unroll
                                        for (int k = 0; k < 4; ++k) {
                                            const float y0 = __uint_as_float(u[4 * (n + k) + 2 * h]), y1 = __uint_as_float(u[4 * (n + k) + 2 * h + 1]);
                                            w[k] = F16 ? pack_f16_rn(y0, y1) : pack_bf2(y0, y1);
                                        }
                                        quad_transpose(w, q);
                                        if (o[h]) reinterpret_cast<uint4 *>(o[h])[c / 8 + n + q] = make_uint4(w[0], w[1], w[2], w[3]);
                                    }
                            } else {
#pragma unroll
                                for (int n = 0; n < 8; n += 2)
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        // an even thread keeps group n, an odd one group n + 1
                                        const bool odd = q & 1;
                                        const uint32_t a0 = u[4 * n + 2 * h], a1 = u[4 * n + 2 * h + 1], b0 = u[4 * n + 4 + 2 * h], b1 = u[4 * n + 5 + 2 * h];
                                        const uint32_t r0 = __shfl_xor_sync(0xffffffffu, odd ? a0 : b0, 1), r1 = __shfl_xor_sync(0xffffffffu, odd ? a1 : b1, 1);
                                        if (o[h])
                                            reinterpret_cast<uint4 *>(o[h])[(c + 8 * n) / 4 + 2 * (q & 1) + (q >> 1)] =
                                                odd ? make_uint4(r0, r1, b0, b1) : make_uint4(a0, a1, r0, r1);
                                    }
                            }
                        }
                    }
                }
                tc_fence_before();
                if (merged) arrive(&sh.o_free);
            }
            o_ph[0] += 1;
            o_ph[1] += TWO || merged;
            merges += merged;
        };
        for (uint32_t s = 0; ok; ++s) {
            const Segment &g = sh.seg[s % kSegRing];
            if (g.tok0 < 0) break;
            if (g.ntok > p.tt)
                segment(s, std::true_type());
            else
                segment(s, std::false_type());
            seg_done(s);
            // the next segment's description, for a group that had no tiles here
            ok = ok && seg_wait(s + 1);
        }
        if (!ok) fail();
    }
    __syncthreads();
    if (wp == kMmaWarp) {
        tmem_relinquish();
        tmem_dealloc(tm, 512);
    }
    if (tid == 0) p.flags[blockIdx.x] = sh.share.flags;
}

// ---------------------------------------------------------------- combine
// Rows of the items that were cut, pieces in order, kPieces at a time:
//   M' = max(M, m_i),  (L, o) <- 2^(M - M') (L, o) + sum_i 2^(m_i - M') (l_i, o_i);  o / L.
// Bound by latency: joints, pieces and store are a chain of loads, in code that runs
// once or twice, so at the rate of instruction fetch.  So: every block reads all
// joints and finds its rows, in a grid that is resident at once, and the code is
// one row of D / 4 lanes with four pieces under way.  Measured on 7 windowed chunks
// (1200 rows cut), one token, and one token over 131072 keys, whole call: 26.3,
// 13.0 and 90.6 us; four rows of two pieces side by side 26.3, 13.4 and 91.5; two
// rows 27.1, 13.7 and 93.2; a block per 16 rows, before, 30.1, 13.1 and 91.9.
constexpr int kJoinWarps = 8, kJoinBlocks = 4;  // warps of a block, blocks per SM
constexpr int kPieces = 4;

// The first block also gathers the CTAs' flags into the status words.
template <int D, bool F16>
__global__ void __launch_bounds__(32 * kJoinWarps, kJoinBlocks) gdn2_attn_combine_kernel(const __grid_constant__ KernelParams p) {
    constexpr int RW = 128 / D;  // rows of a warp
    __shared__ Joint joints[kMaxCtas];
    __shared__ int upto[kMaxCtas];  // tasks of the joints up to each, a task per warp
    __shared__ int sums[kJoinWarps];
    const AttnParams &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
    const int sub = lane / (D / 4), ch = lane % (D / 4) * 4;  // row and channels of this lane
    const uint32_t inv_g = 65536u / a.G + 1;
    static_assert(kMaxCtas <= 32 * kJoinWarps, "a joint per thread");
    pdl_wait();
    Joint j = {};
    if (tid < p.ctas) j = p.joint[tid];
    int tasks = 0;
    if (j.more > 0) {
        const int rows = j.ntok > p.tt ? kTile + (j.ntok - p.tt) * a.G : j.ntok * a.G;
        tasks = (rows + RW - 1) / RW;
    }
    int x = tasks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[wp] = x;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) {
        if (i < wp) x += sums[i];
        total += sums[i];
    }
    if (tid < kMaxCtas) {
        joints[tid] = j;
        upto[tid] = x;
    }
    __syncthreads();
    for (int task = blockIdx.x * kJoinWarps + wp; task < total; task += gridDim.x * kJoinWarps) {
        int cta = 0;  // the first joint whose tasks end past this one
        for (int base = 0; base < kMaxCtas; base += 32) {
            const int i = base + lane;
            cta += __popc(__ballot_sync(0xffffffffu, i < kMaxCtas && upto[i] <= task));
        }
        const Joint &g = joints[cta];
        const int row = (task - (cta > 0 ? upto[cta - 1] : 0)) * RW + sub;
        // the row's token, if it has one, and head
        const int tile = row / kTile, in = row % kTile, tk = static_cast<int>((in * inv_g) >> 16), tok = tile * p.tt + tk;
        if (tk >= p.tt || tok >= g.ntok) continue;  // (no collective operation follows before the next task)
        float M = -INFINITY, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 <= g.more; k0 += kPieces) {
            float2 ml[kPieces];
            float4 o[kPieces];
            float top = M;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                ml[i] = make_float2(-INFINITY, 0.f);
                o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + i > g.more) continue;
                const int64_t at = static_cast<int64_t>(k0 + i == 0 ? g.slot : 2 * (cta + k0 + i)) * 2 * kTile + row;
                ml[i] = p.part_ml[at];
                o[i] = *reinterpret_cast<const float4 *>(p.part_o + at * D + ch);
            }
#pragma unroll
            for (int i = 0; i < kPieces; ++i) top = fmaxf(top, ml[i].x);
            const float base = top == -INFINITY ? 0.f : top, f = ex2(M - base);
            M = top;
            L *= f;
            acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const float w = ex2(ml[i].x - base);
                L += w * ml[i].y;
                acc.x += w * o[i].x;
                acc.y += w * o[i].y;
                acc.z += w * o[i].z;
                acc.w += w * o[i].w;
            }
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int64_t at = static_cast<int64_t>(g.tok0) + tok;
        const int head = g.h * a.G + in - tk * a.G;
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(a.out + at * a.so_t + head * a.so_h + ch) =
            F16 ? make_uint2(pack_f16_rn(acc.x, acc.y), pack_f16_rn(acc.z, acc.w))
                : make_uint2(pack_bf2(acc.x, acc.y), pack_bf2(acc.z, acc.w));
        if (a.lse && ch == 0) a.lse[at * a.HQ + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
    if (blockIdx.x == 0 && wp == kJoinWarps - 1) {
        int f = 0;
        for (int c = lane; c < p.ctas; c += 32) f |= p.flags[c];
        f = __reduce_or_sync(0xffffffffu, f);
        if (lane < 8)
            a.status[lane] = lane == 0   ? f & kBadCu ? GDN2_ERR_CU_SEQLENS : f & kBadPages ? GDN2_ERR_PAGES : GDN2_OK
                               : lane == 2 ? f & kTimeout ? GDN2_ERR_TIMEOUT : GDN2_OK
                                           : 0;
    }
}

// ------------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// Tensor map over a cache [pages, page_size, heads, D]: a box is `gran` tokens
// of one page and head and 64 channels, stored with the 128-byte swizzle.  The
// three outer dimensions go in the order of their strides; pos[] says where
// page, token and head went.
bool encode_cache(CUtensorMap *map, int (&pos)[3], const void *base, const AttnParams &a, const int64_t (&st)[3], int D,
                  bool f16, int gran) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return false;
    const int64_t size[3] = {a.num_pages, a.page_size, a.HKV};
    int order[3] = {1, 2, 0};  // token, head, page
    auto key = [&](int i) { return size[i] > 1 ? st[i] : 0; };
    for (int i = 0; i < 3; ++i)
        for (int k = i + 1; k < 3; ++k)
            if (key(order[k]) < key(order[i])) {
                const int x = order[i];
                order[i] = order[k];
                order[k] = x;
            }
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(D)}, strides[3];
    cuuint32_t box[4] = {64}, estr[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        const int d = order[i];
        pos[d] = i + 1;
        dims[i + 1] = static_cast<cuuint64_t>(size[d]);
        strides[i] = static_cast<cuuint64_t>((size[d] > 1 ? st[d] : D) * 2);
        box[i + 1] = d == 1 ? static_cast<cuuint32_t>(gran) : 1;
    }
    return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base),
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over the queries [T, HQ, D]: a box is G heads of `tt` tokens and 64
// channels.  False where the driver rejects the layout (or a stride is zero).
bool encode_queries(CUtensorMap *map, const AttnParams &a, int D, bool f16, int tt) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc || (a.HQ > 1 && a.sq_h == 0) || (a.T > 1 && a.sq_t == 0)) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(a.HQ), static_cast<cuuint64_t>(a.T)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>((a.HQ > 1 ? a.sq_h : D) * 2),
                                   static_cast<cuuint64_t>((a.T > 1 ? a.sq_t : D) * 2)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(tt)}, estr[3] = {1, 1, 1};
    return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf16 *>(a.q),
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool F16>
cudaError_t launch(const KernelParams &p, int ctas, cudaStream_t s) {
    auto kern = gdn2_paged_attn_kernel<D, F16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    kern<<<ctas, kThreads, Cfg<D>::kSmem, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_chained(gdn2_attn_combine_kernel<D, F16>, dim3(kJoinBlocks * ctas), dim3(32 * kJoinWarps), 0, s, p);
}

}  // namespace

size_t paged_attn_workspace(const gdn2_attn_dims &d) { return layout_of(d).total; }

cudaError_t launch_paged_attn(const AttnParams &a, const gdn2_attn_dims &d, int sms, void *workspace, cudaStream_t s) {
    const bool f16 = d.dtype == GDN2_DTYPE_F16;
    const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
    const Layout l = layout_of(d);
    char *ws = static_cast<char *>(workspace);
    KernelParams p;
    p.a = a;
    p.flags = reinterpret_cast<int *>(ws + l.flags);
    p.joint = reinterpret_cast<Joint *>(ws + l.joint);
    p.part_o = reinterpret_cast<float *>(ws + l.part_o);
    p.part_ml = reinterpret_cast<float2 *>(ws + l.part_ml);
    p.scale_log2 = a.scale * kLog2e;
    p.a.lead = lead_tiles(d.D);
    p.ctas = ctas;
    p.tt = kTile / a.G;
    p.granule = 8;
    p.granule_log2 = 3;
    while (p.granule < kTile && a.page_size % (2 * p.granule) == 0) p.granule *= 2, ++p.granule_log2;
    p.page = divisor(a.page_size);
    if (a.T > 0 && (!encode_cache(&p.tk, p.kpos, a.k_cache, a, a.skc, d.D, f16, p.granule) ||
                    !encode_cache(&p.tv, p.vpos, a.v_cache, a, a.svc, d.D, f16, p.granule)))
        return cudaErrorInvalidValue;
    p.q_map = a.T > 0 && encode_queries(&p.tq, a, d.D, f16, p.tt);
    if (d.D == 64) return f16 ? launch<64, true>(p, ctas, s) : launch<64, false>(p, ctas, s);
    return f16 ? launch<128, true>(p, ctas, s) : launch<128, false>(p, ctas, s);
}

}  // namespace gdn2
