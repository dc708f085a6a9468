// Softmax attention of the new tokens over a paged key/value cache
// (include/gdn2_attn.h).
//
// Rows.  The query heads that share a key head are packed into the rows of one
// matrix product: row r of a 128-row tile is token r / G, head r % G of the
// group (G = HQ / HKV), so that a decode step's G rows share the keys they
// read.  A CTA holds one tile (few rows per sequence: decode, bound by the
// keys' and values' bytes) or two (chunks: bound by the tensor cores; the two
// tiles share the keys and values in shared memory, and one tile's softmax
// runs while the tensor cores work on the other's).
//
// Work.  An item is (sequence, key head, row tiles) with its range of 128-key
// tiles (after the causal and window masks).  The items' key tiles, laid end to
// end, are cut into equal shares, one per CTA (one CTA per SM), wherever the
// cuts fall: a share is a list of segments (item, key tiles).  An item cut into
// several segments leaves unnormalised sums and their maxima in the workspace
// and the combine kernel joins them, in the order of the segments.  So one long
// sequence, many short ones and any mixture fill the GPU alike, and the result
// does not depend on timing.
//
//   plan     one block: checks the lengths, cuts the shares, writes segments
//   main     per segment: S = Q K^T (tcgen05, fp32 in Tensor Memory), softmax
//            in registers with a running maximum and sum, P back to Tensor
//            Memory in 16 bits, O += P V (tcgen05, P from Tensor Memory)
//   combine  joins the items that were cut
//
// Keys and values arrive by TMA, straight from their pages, into a ring of
// 128-key stages; the last tile's value rows past the range are zeroed (the
// cache may hold anything there, and 0 x NaN is NaN), the keys' scores masked.
#include <cudaTypedefs.h>

#include "gdn2_attn_internal.cuh"
#include "gdn2_tc.cuh"

namespace gdn2 {
namespace {

using namespace tc;

constexpr int kMaxCtas = 152;   // shares at most (SMs of a GB300)
constexpr int kTile = 128;      // rows of a tile, keys of a tile
constexpr int kPlanThreads = 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A share's piece of an item: new tokens j0 .. j0 + ntok of sequence n, key
// head h, key tiles lo .. hi; slot of its partial result, -1 if it is whole.
struct __align__(16) Segment {
    int n, h, j0, ntok;
    int lo, hi, slot, end;  // end: keys from `end` on are not attended to
};
// The item whose pieces the combine kernel joins: the first in slot `slot`,
// then `more` in slots 2 (cta + 1), 2 (cta + 2), ...
struct __align__(16) Joint {
    int n, h, j0, ntok;
    int slot, more, pad0, pad1;
};
struct SeqPlan {
    long long cost, base, item;  // key tiles per head; first tile, first item
};

struct PlanPtrs {
    int *first, *last;           // [kMaxCtas] segment ids of a share
    Joint *joint;                // [kMaxCtas]
    SeqPlan *seq;                // [N]
    Segment *seg;                // [items + kMaxCtas]; segment of item i in share c: i + c
    float *part_o;               // [2 kMaxCtas][NT * 128][D]
    float2 *part_ml;             // [2 kMaxCtas][NT * 128] (log2-scaled maximum, sum)
};

struct KernelParams {
    AttnParams a;
    PlanPtrs w;
    float scale_log2;
    int tt;                      // tokens per row tile: 128 / G
    int granule;                 // keys per TMA box
    int kpos[3], vpos[3];        // coordinate (1 .. 3) of page, token, head in the tensor maps
    CUtensorMap tk, tv;
};

// One row tile per CTA while the sequences have at most one tile of rows on
// average (decode, short continuations), else two.  Measured at both ends:
// see the table of cases.
int row_tiles(const gdn2_attn_dims &d) {
    return d.T_tot * (d.HQ / d.HKV) <= static_cast<int64_t>(kTile) * d.N ? 1 : 2;
}

struct Layout {
    size_t first, last, joint, seq, seg, part_o, part_ml, total;
};
Layout layout_of(const gdn2_attn_dims &d) {
    const int G = d.HQ / d.HKV, nt = row_tiles(d);
    const size_t tokens = static_cast<size_t>(kTile / G) * nt;
    const size_t items = (static_cast<size_t>(d.T_tot) / tokens + d.N) * d.HKV;
    Layout l;
    size_t off = 256;  // the status words
    auto take = [&](size_t bytes) { const size_t o = off; off += (bytes + 255) & ~static_cast<size_t>(255); return o; };
    l.first = take(kMaxCtas * 4);
    l.last = take(kMaxCtas * 4);
    l.joint = take(kMaxCtas * sizeof(Joint));
    l.seq = take(static_cast<size_t>(d.N) * sizeof(SeqPlan));
    l.seg = take((items + kMaxCtas) * sizeof(Segment));
    l.part_ml = take(2ull * kMaxCtas * nt * kTile * sizeof(float2));
    l.part_o = take(2ull * kMaxCtas * nt * kTile * d.D * sizeof(float));
    l.total = off;
    return l;
}

// ------------------------------------------------------------------- plan
struct Span {
    int lo, hi, end;  // key tiles, first key past the range
};
// Key tiles of the new tokens j0 .. j1 of a sequence of `len` cached tokens.
__device__ __forceinline__ Span key_span(const AttnParams &a, int len, int fresh, int j0, int j1) {
    Span s;
    s.end = a.causal ? max(0, len - fresh + j1) : len;
    const int begin = a.window >= 0 ? max(0, len - fresh + j0 - a.window) : 0;
    s.lo = begin / kTile;
    s.hi = (s.end + kTile - 1) / kTile;
    if (s.hi < s.lo) s.hi = s.lo;
    return s;
}

__device__ __forceinline__ long long div_by(long long x, long long total) {
    return (x | total) >> 32 ? x / total : static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(total));
}

__global__ void __launch_bounds__(kPlanThreads) gdn2_attn_plan_kernel(const __grid_constant__ KernelParams p, int ctas, int nt) {
    __shared__ long long s_cost[33], s_item[33];
    __shared__ int s_bad_cu, s_bad_len;
    const AttnParams &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
    const int tokens = p.tt * nt;
    pdl_trigger();
    if (tid == 0) {
        s_bad_len = 0;
        s_bad_cu = a.N > 0 ? cu_of(a.cu, a.cu64, 0) != 0 || cu_of(a.cu, a.cu64, a.N) != a.T : a.T != 0;
    }
    if (tid < kMaxCtas) {
        p.w.first[tid] = 0;
        p.w.last[tid] = -1;
        p.w.joint[tid].more = 0;
    }
    __syncthreads();

    // costs of the sequences, and their running sums
    long long run_cost = 0, run_item = 0;
    for (int base = 0; base < a.N; base += kPlanThreads) {
        const int n = base + tid;
        int len = 0, fresh = 0, tiles = 0;
        long long cost = 0;
        if (n < a.N) {
            const int64_t c0 = cu_of(a.cu, a.cu64, n), c1 = cu_of(a.cu, a.cu64, n + 1);
            len = a.kv_lens[n];
            if (c0 > c1 || c0 < 0 || c1 > a.T)
                s_bad_cu = 1;
            else
                fresh = static_cast<int>(c1 - c0);
            if (len < 0 || len > static_cast<int64_t>(a.max_pages) * a.page_size) {
                s_bad_len = 1;
                fresh = 0;
            }
            tiles = (fresh + tokens - 1) / tokens;
            if (tiles == 1) {
                const Span s = key_span(a, len, fresh, 0, fresh);
                cost = max(1, s.hi - s.lo);
            }
        }
        for (uint32_t more = __ballot_sync(0xffffffffu, tiles > 1); more; more &= more - 1) {
            const int src = __ffs(more) - 1;
            const int l = __shfl_sync(0xffffffffu, len, src), f = __shfl_sync(0xffffffffu, fresh, src);
            const int m = __shfl_sync(0xffffffffu, tiles, src);
            long long sum = 0;
            for (int i = lane; i < m; i += 32) {
                const Span s = key_span(a, l, f, i * tokens, min(f, (i + 1) * tokens));
                sum += max(1, s.hi - s.lo);
            }
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == src) cost = sum;
        }
        // block scan of (cost, tiles)
        long long ic = cost, it = tiles;
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, ic, o), y = __shfl_up_sync(0xffffffffu, it, o);
            if (lane >= o) { ic += x; it += y; }
        }
        __syncthreads();
        if (lane == 31) { s_cost[wp] = ic; s_item[wp] = it; }
        __syncthreads();
        if (wp == 0) {
            long long x = s_cost[lane], y = s_item[lane];
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) { x += u; y += v; }
            }
            s_cost[lane] = x;
            s_item[lane] = y;
        }
        __syncthreads();
        const long long bc = run_cost + (wp ? s_cost[wp - 1] : 0) + ic - cost;
        const long long bi = run_item + (wp ? s_item[wp - 1] : 0) + it - tiles;
        if (n < a.N) p.w.seq[n] = {cost, bc * a.HKV, bi * a.HKV};
        run_cost += s_cost[31];
        run_item += s_item[31];
    }
    __syncthreads();
    const bool bad = s_bad_cu || s_bad_len;
    if (tid < 8) a.status[tid] = tid ? 0 : s_bad_cu ? GDN2_ERR_CU_SEQLENS : s_bad_len ? GDN2_ERR_PAGES : GDN2_OK;
    const long long total = run_cost * a.HKV;
    if (bad || total == 0) return;
    const long long shares = total < ctas ? total : ctas;

    // the segments of one item: tiles [o, o + cost) of the whole row of tiles
    auto emit = [&](int n, int h, int j0, int ntok, const Span &s, long long item, long long o) {
        const int cost = max(1, s.hi - s.lo);
        const bool none = s.hi == s.lo;
        const int c0 = static_cast<int>(div_by((o + 1) * shares - 1, total));
        const int c1 = static_cast<int>(div_by((o + cost) * shares - 1, total));
        for (int c = c0; c <= c1; ++c) {
            const long long b0 = div_by(total * c, shares), b1 = div_by(total * (c + 1), shares);
            const bool is_first = o <= b0;
            Segment g;
            g.n = n; g.h = h; g.j0 = j0; g.ntok = ntok;
            g.lo = s.lo + static_cast<int>(max(o, b0) - o);
            g.hi = none ? s.lo : s.lo + static_cast<int>(min(o + cost, b1) - o);
            g.slot = c0 == c1 ? -1 : 2 * c + (is_first ? 0 : 1);
            g.end = s.end;
            const long long id = item + c;
            p.w.seg[id] = g;
            if (is_first) p.w.first[c] = static_cast<int>(id);
            if (o + cost >= b1) p.w.last[c] = static_cast<int>(id);
            if (c == c0 && c1 > c0) p.w.joint[c] = {n, h, j0, ntok, g.slot, c1 - c0, 0, 0};
        }
    };
    // sequences of one row tile: a thread per (sequence, head)
    for (long long i = tid; i < static_cast<long long>(a.N) * a.HKV; i += kPlanThreads) {
        const int n = static_cast<int>(i / a.HKV), h = static_cast<int>(i - static_cast<long long>(n) * a.HKV);
        const int fresh = static_cast<int>(cu_of(a.cu, a.cu64, n + 1) - cu_of(a.cu, a.cu64, n));
        if (fresh == 0 || fresh > tokens) continue;
        const SeqPlan q = p.w.seq[n];
        emit(n, h, 0, fresh, key_span(a, a.kv_lens[n], fresh, 0, fresh), q.item + h, q.base + h * q.cost);
    }
    // longer ones: a warp per head, a lane per tile
    for (int n = 0; n < a.N; ++n) {
        const int fresh = static_cast<int>(cu_of(a.cu, a.cu64, n + 1) - cu_of(a.cu, a.cu64, n));
        if (fresh <= tokens) continue;
        const int len = a.kv_lens[n], tiles = (fresh + tokens - 1) / tokens;
        const SeqPlan q = p.w.seq[n];
        for (int h = wp; h < a.HKV; h += kPlanThreads / 32) {
            long long at = q.base + h * q.cost;
            for (int m0 = 0; m0 < tiles; m0 += 32) {
                const int m = m0 + lane, j0 = m * tokens;
                Span s = {0, 0, 0};
                int cost = 0;
                if (m < tiles) {
                    s = key_span(a, len, fresh, j0, min(fresh, j0 + tokens));
                    cost = max(1, s.hi - s.lo);
                }
                int sum = cost;
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += x;
                }
                if (m < tiles)
                    emit(n, h, j0, min(tokens, fresh - j0), s, q.item + static_cast<long long>(h) * tiles + m,
                         at + sum - cost);
                at += __shfl_sync(0xffffffffu, sum, 31);
            }
        }
    }
}

// ------------------------------------------------------------------- main
template <int D, int NT>
struct Cfg {
    static constexpr int kStageBytes = kTile * D * 2;
    static constexpr int kQBytes = kTile * D * 2;
    // as many stages as fit beside the query tiles
    static constexpr int kStages = D == 128 ? (NT == 2 ? 5 : 6) : (NT == 2 ? 10 : 12);
    static constexpr int kQ = 0;
    static constexpr int kRing = NT * kQBytes;
    static constexpr int kSmem = kRing + kStages * kStageBytes + 1024;  // + alignment slack
    static constexpr int kMmaWarp = 4 * NT, kTmaWarp = 4 * NT + 1;
    static constexpr int kThreads = NT == 2 ? 384 : 192;
    // NT = 2: three warpgroups of 168 registers at launch, 64512 in all; the two
    // softmax groups, which hold a row of scores, take 192 and the third keeps
    // 120 (2 x 128 x 192 + 128 x 120 = 64512)
    static constexpr int kSoftmaxRegs = 192, kOtherRegs = 120;
};

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, const int (&c)[4], uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c[0]), "r"(c[1]), "r"(c[2]), "r"(c[3]), "r"(smem_u32(bar))
        : "memory");
}

// One thread of the warp, the same each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return r;
}

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1)
    gdn2_paged_attn_kernel(const __grid_constant__ KernelParams p) {
    using C = Cfg<D, NT>;
    constexpr int NB = D / 64;  // 64-channel blocks of a row
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ uint64_t full[C::kStages], empty[C::kStages], tail, q_full[2], s_full[2], p_half[2], p_full[2], o_full[2], drain;
    __shared__ uint32_t s_tmem;
    const AttnParams &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&tail, 1);
        mbar_init(&drain, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 128);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_half[i], 128);
            mbar_init(&p_full[i], 128);
            mbar_init(&o_full[i], 1);
        }
        fence_mbar_init();
    }
    if (wp == C::kMmaWarp) tmem_alloc(&s_tmem, 512);
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;
    pdl_trigger();
    pdl_wait();  // the plan is complete
    const int seg0 = p.w.first[blockIdx.x], seg1 = p.w.last[blockIdx.x] + 1;
    const uint32_t sQ = smem_u32(smem + C::kQ), sRing = smem_u32(smem + C::kRing);
    // Tensor Memory columns: scores of tile (or buffer) x at 128 x, outputs after them
    auto tS = [&](int x) { return tm + 128 * x; };
    auto tO = [&](int x) { return tm + 256 + 128 * x; };
    auto fail = [&]() {
        atomicExch(a.status + 2, static_cast<int>(GDN2_ERR_TIMEOUT));
    };

    auto few_regs = [] {
        if (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    };
    if (wp == C::kTmaWarp) {
        few_regs();
        // ------------------------------------------- keys and values: TMA
        const int gran = p.granule, per = kTile / gran;     // granules of a tile
        const int batch = 32 / per;                         // tiles whose table entries one load fetches
        const int my_gr = lane / NB, my_cb = lane % NB;     // this lane's granule and channel block
        uint32_t loads = 0;                                 // tiles loaded so far
        int tail_ph = 0;
        bool ok = true;
        for (int s = seg0; s < seg1 && ok; ++s) {
            const Segment g = p.w.seg[s];
            const int tiles = g.hi - g.lo;
            if (tiles == 0) continue;
            const int *row = a.table + static_cast<int64_t>(g.n) * a.table_stride;
            // page and slot of this lane's granule of the batch that starts at tile t
            auto fetch = [&](int t) {
                t += lane / per;
                int2 e = make_int2(0, 0);
                const int64_t key = static_cast<int64_t>(t) * kTile + (lane % per) * gran;
                if (t < g.hi && key < g.end) {
                    const int col = static_cast<int>(key) / a.page_size;
                    e = make_int2(row[col], static_cast<int>(key) - col * a.page_size);
                    if (e.x < 0 || e.x >= a.num_pages) {
                        e.x = static_cast<int>(a.num_pages);  // past the tensor: the box reads zeros
                        atomicCAS(a.status, 0, static_cast<int>(GDN2_ERR_PAGES));
                    }
                }
                return e;
            };
            // entries of the batch that the values are in, and of the next
            int at = 0;
            int2 now = fetch(g.lo), next = fetch(g.lo + batch);
            // keys or values of tile g.lo + i into the next stage
            auto load = [&](int i, bool is_v) {
                const int st = static_cast<int>(loads % C::kStages);
                const int left = min(kTile, g.end - (g.lo + i) * kTile);  // rows that count
                const int grans = (left + gran - 1) / gran;
                ok = warp_wait(&empty[st], ((loads / C::kStages) & 1) ^ 1);
                if (!ok) return;
                const bool patch = is_v && left < kTile;
                uint64_t *bar = patch ? &tail : &full[st];
                uint8_t *dst = smem + C::kRing + st * C::kStageBytes;
                if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(grans * gran * 128 * NB));
                __syncwarp();
                const int2 e = i / batch == at ? now : next;
                const int from = i % batch * per + min(my_gr, per - 1);
                const int page = __shfl_sync(0xffffffffu, e.x, from), slot = __shfl_sync(0xffffffffu, e.y, from);
                if (my_gr < grans) {
                    const int *pos = is_v ? p.vpos : p.kpos;
                    int c[4] = {my_cb * 64, 0, 0, 0};
#pragma unroll
                    for (int k = 1; k < 4; ++k) c[k] = pos[0] == k ? page : pos[1] == k ? slot : g.h;
                    tma_load_4d(dst + my_cb * (kTile * 128) + my_gr * gran * 128, is_v ? &p.tv : &p.tk, c, bar);
                }
                ++loads;
                if (patch) {  // zero the rows past the range, once the copies are in
                    ok = warp_wait(&tail, tail_ph);
                    if (!ok) return;
                    tail_ph ^= 1;
                    for (int k = lane; k < (kTile - left) * NB * 8; k += 32) {
                        const int r = left + k / (NB * 8), q = k % (NB * 8);
                        *reinterpret_cast<uint4 *>(dst + (q >> 3) * (kTile * 128) + r * 128 + (q & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[st]);
                }
                if (is_v && (i + 1) % batch == 0) {
                    now = next;
                    next = fetch(g.lo + (++at + 1) * batch);
                }
            };
            // in the order in which the products take them: with one row tile
            // the keys run one tile ahead of the values
            if (NT == 1) load(0, false);
            for (int i = 0; i < tiles && ok; ++i) {
                if (NT == 2)
                    load(i, false);
                else if (i + 1 < tiles)
                    load(i + 1, false);
                if (ok) load(i, true);
            }
        }
        if (!ok) {
            if (lane == 0) fail();
            // let the copies in flight land before the block ends
            for (uint32_t i = loads > C::kStages ? loads - C::kStages : 0; i < loads; ++i)
                warp_wait(&full[i % C::kStages], (i / C::kStages) & 1);
        }
    } else if (wp == C::kMmaWarp) {
        few_regs();
        // ------------------------------------------- tensor cores: one thread
        // The warp goes through the steps together and one elected thread issues:
        // with elect.sync the compiler keeps descriptors and addresses in uniform
        // registers, and a product of 16 keys costs 23 cycles to issue; under
        // `lane == 0` it moves them there one by one, 54 cycles, which the 64
        // cycles that the product takes do not hide once waits come between.
        constexpr uint32_t kIdS = idesc_f16kind(kTile, kTile, false, false, !F16);
        constexpr uint32_t kIdO = idesc_f16kind(kTile, D, false, true, !F16);
        uint32_t taken = 0;                  // stages taken so far
        uint32_t steps = 0;                  // key tiles done (NT = 1)
        uint32_t q_ph[2] = {0, 0}, p_ph[2] = {0, 0};
        bool ok = true;
        auto stage = [&](uint32_t i) { return sRing + (i % C::kStages) * C::kStageBytes; };
        auto wait_stage = [&](uint32_t i) { ok = ok && warp_wait(&full[i % C::kStages], (i / C::kStages) & 1); };
        // S of tile x = Q_x K^T; then the stage is free if `last`
        auto scores = [&](int x, int buf, uint32_t k, bool last) {
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_f16(tS(buf), desc_kmajor(sQ + x * C::kQBytes, kTile, kk), desc_kmajor(stage(k), kTile, kk),
                            kIdS, kk > 0);
                mma_commit(&s_full[buf]);
                if (last) mma_commit(&empty[k % C::kStages]);
            }
            __syncwarp();
        };
        // O_x (+)= P V, each half of the keys as soon as its weights are in; then
        // the stage is free if `last`, and the product is reported on `done`
        auto output = [&](int x, int buf, uint32_t v, bool first, bool last, uint64_t *done) {
            ok = ok && warp_wait(&p_half[buf], p_ph[buf]);
            if (!ok) return;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kTile / 32; ++kk)
                    mma_f16_ta(tO(x), tS(buf) + 8 * kk, desc_mnmajor(stage(v), kTile, kk), kIdO, kk > 0 || !first);
            }
            __syncwarp();
            ok = warp_wait(&p_full[buf], p_ph[buf]);
            p_ph[buf] ^= 1;
            if (!ok) return;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = kTile / 32; kk < kTile / 16; ++kk)
                    mma_f16_ta(tO(x), tS(buf) + 8 * kk, desc_mnmajor(stage(v), kTile, kk), kIdO, 1);
                if (last) mma_commit(&empty[v % C::kStages]);
                if (done) mma_commit(done);
            }
            __syncwarp();
        };
        auto wait_q = [&](int x) {
            ok = ok && warp_wait(&q_full[x], q_ph[x]);
            q_ph[x] ^= 1;
        };
        for (int s = seg0; s < seg1 && ok; ++s) {
            const Segment g = p.w.seg[s];
            const int tiles = g.hi - g.lo;
            if (tiles == 0) continue;
            uint32_t k = taken++;
            wait_stage(k);
            if (NT == 2) {
                const int nx = g.ntok > p.tt ? 2 : 1;
                for (int x = 0; x < nx && ok; ++x) {
                    wait_q(x);
                    if (ok) scores(x, x, k, x == nx - 1);
                }
                for (int i = 0; i < tiles && ok; ++i) {
                    const uint32_t v = taken++;
                    const bool more = i + 1 < tiles;
                    if (more) k = taken++;
                    wait_stage(v);
                    for (int x = 0; x < nx && ok; ++x) {
                        output(x, x, v, i == 0, x == nx - 1, more ? nullptr : &o_full[x]);
                        if (more && x == 0) wait_stage(k);
                        if (more && ok) scores(x, x, k, x == nx - 1);
                    }
                }
            } else {
                wait_q(0);
                if (ok) scores(0, steps & 1, k, true);
                for (int i = 0; i < tiles && ok; ++i, ++steps) {
                    if (i + 1 < tiles) {
                        k = taken++;
                        wait_stage(k);
                        if (ok) scores(0, (steps + 1) & 1, k, true);
                    }
                    const uint32_t v = taken++;
                    wait_stage(v);
                    output(0, steps & 1, v, i == 0, true, &o_full[steps & 1]);
                }
            }
        }
        if (!ok && lane == 0) fail();
        // nothing may run on in Tensor Memory once it is released
        if (elect_one()) mma_commit(&drain);
        __syncwarp();
        if (!warp_wait(&drain, 0) && lane == 0) fail();
    } else if (wp < 4 * NT) {
        // ------------------------------------------- softmax: a thread per row
        if (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
        const int x = NT == 2 ? wp >> 2 : 0, row = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(wp & 3) << 21;  // TMEM lane of the warp's first row
        const uint32_t inv_g = 65536u / a.G + 1;                     // r / G for r < 128
        const float sl2 = p.scale_log2, slack = 8.f / sl2;
        const int my_tok = static_cast<int>((row * inv_g) >> 16), my_head = row - my_tok * a.G;
        // the row's token of a segment, -1 if it has none
        auto token = [&](const Segment &g) { return my_tok < p.tt && x * p.tt + my_tok < g.ntok ? x * p.tt + my_tok : -1; };
        auto next_seg = [&](int s) {  // the next segment with work for this tile
            while (s < seg1 && (p.w.seg[s].hi == p.w.seg[s].lo || p.w.seg[s].ntok <= x * p.tt)) ++s;
            return s;
        };
        auto load_q = [&](const Segment &g) {
            const int rows = min(p.tt, g.ntok - x * p.tt) * a.G;
            const bf16 *q = a.q + (cu_of(a.cu, a.cu64, g.n) + g.j0 + x * p.tt) * a.sq_t + static_cast<int64_t>(g.h) * a.G * a.sq_h;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const int at = row + 128 * i, r = at / (D / 8), ch = at % (D / 8);
                const int tok = static_cast<int>((r * inv_g) >> 16), hd = r - tok * a.G;
                const bool in = r < rows;
                cp_async16(smem + C::kQ + x * C::kQBytes + (ch >> 3) * (kTile * 128) + swz(r, ch & 7),
                           in ? q + tok * a.sq_t + hd * a.sq_h + 8 * ch : a.q, in ? 16 : 0);
            }
        };
        auto q_ready = [&]() {
            cp_async_wait_all();
            fence_proxy_async();
            mbar_arrive(&q_full[x]);
        };
        auto out_row = [&](const Segment &g, int tok) {
            return a.out + (cu_of(a.cu, a.cu64, g.n) + g.j0 + tok) * a.so_t + static_cast<int64_t>(g.h * a.G + my_head) * a.so_h;
        };
        auto put_lse = [&](const Segment &g, int tok, float v) {
            if (a.lse) a.lse[(cu_of(a.cu, a.cu64, g.n) + g.j0 + tok) * a.HQ + g.h * a.G + my_head] = v;
        };
        // items without a key
        for (int s = seg0; s < seg1; ++s) {
            const Segment g = p.w.seg[s];
            if (g.hi > g.lo) continue;
            const int tok = token(g);
            if (tok < 0) continue;
            bf16 *o = out_row(g, tok);
            for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4 *>(o + c) = make_uint4(0, 0, 0, 0);
            put_lse(g, tok, -INFINITY);
        }
        // NT = 1: the product of step i is in.  Its barrier alternates, and S of
        // step i, which the warp has seen, followed the product of step i - 2:
        // the barrier is in the phase waited for or just past it.
        auto product_done = [&](uint32_t i) { return warp_wait(&o_full[i & 1], (i >> 1) & 1); };
        bool ok = true;
        uint32_t steps = 0, o_ph = 0;
        int s = next_seg(seg0);
        if (s < seg1) {
            load_q(p.w.seg[s]);
            q_ready();
        }
        while (s < seg1 && ok) {
            const Segment g = p.w.seg[s];
            const int after = next_seg(s + 1), tiles = g.hi - g.lo;
            const int tok = token(g);
            const int len = a.kv_lens[g.n];
            const int fresh = static_cast<int>(cu_of(a.cu, a.cu64, g.n + 1) - cu_of(a.cu, a.cu64, g.n));
            // keys [from, upto) for this row; rows without a token take what they get
            const int place = len - fresh + g.j0 + (tok < 0 ? 0 : tok);
            const int upto = tok < 0 ? 0x7fffffff : a.causal ? place + 1 : len;
            const int from = tok >= 0 && a.window >= 0 ? place - a.window : 0;
            const bool idle = !__any_sync(0xffffffffu, tok >= 0);  // no row of the warp has a token
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < tiles; ++i, ++steps) {
                const int buf = NT == 2 ? x : steps & 1;
                const uint32_t par = NT == 2 ? steps & 1 : (steps >> 1) & 1;
                ok = warp_wait(&s_full[buf], par);
                if (!ok) break;
                if (i == tiles - 1 && after < seg1) load_q(p.w.seg[after]);
                if (!idle) {
                    tc_fence_after();
                    uint32_t u[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(tS(buf) + lanes + 32 * c, u[c]);
                    tmem_ld_wait();
                    const int k0 = (g.lo + i) * kTile;
                    if (__any_sync(0xffffffffu, k0 < from || upto - k0 < kTile)) {
                        const int lo = from - k0, hi = upto - k0;
#pragma unroll
                        for (int c = 0; c < 128; ++c)
                            if (c < lo || c >= hi) u[c >> 5][c & 31] = 0xff800000u;
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 128; c += 2) mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], u[c >> 5][c & 31], u[c >> 5][(c & 31) + 1]);
                    const float top = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                    if (i == 0) {
                        m = top;
                    } else {
                        // The maximum in use may lag behind the true one by a
                        // factor of 2^8 (weights to 256 lose nothing in 16-bit
                        // floating point): the outputs are then seldom rescaled.
                        const bool grow = top > m + slack;
                        if (__any_sync(0xffffffffu, grow)) {
                            const float f = grow ? ex2((m - top) * sl2) : 1.f;
                            if (grow) m = top;
                            l *= f;
                            if (NT == 1) {  // the previous product has to be in (NT = 2: S follows it)
                                ok = product_done(steps - 1);
                                if (!ok) break;
                                tc_fence_after();
                            }
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
                    const float base = m == -INFINITY ? 0.f : m * sl2;
                    const uint64_t scale2 = pair(sl2, sl2), base2 = pair(-base, -base);
                    uint64_t sum2[2] = {0, 0};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 y = unpair(fma2(pair(__uint_as_float(u[c][2 * e]), __uint_as_float(u[c][2 * e + 1])), scale2, base2));
                            const float a0 = ex2(y.x), a1 = ex2(y.y);
                            sum2[e & 1] = add2(sum2[e & 1], pair(a0, a1));
                            w[e] = F16 ? pack_f16_rn(a0, a1) : pack_bf2(a0, a1);
                        }
                        tmem_st16(tS(buf) + lanes + 16 * c, w);
                        if (c == 1) {  // the first half of the keys: their product may begin
                            tmem_st_wait();
                            tc_fence_before();
                            mbar_arrive(&p_half[buf]);
                        }
                    }
                    const float2 t = unpair(add2(sum2[0], sum2[1]));
                    l += t.x + t.y;
                    tmem_st_wait();
                    tc_fence_before();
                } else {
                    mbar_arrive(&p_half[buf]);
                }
                mbar_arrive(&p_full[buf]);
            }
            if (!ok) break;
            if (after < seg1) q_ready();
            ok = NT == 2 ? warp_wait(&o_full[x], o_ph) : product_done(steps - 1);
            if (!ok) break;
            o_ph ^= 1;
            tc_fence_after();
            if (!idle) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                bf16 *o = tok >= 0 && g.slot < 0 ? out_row(g, tok) : nullptr;
                float *po = p.w.part_o + (static_cast<int64_t>(g.slot) * NT * kTile + x * kTile + row) * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t u[32];
                    tmem_ld32(tO(x) + lanes + c, u);
                    tmem_ld_wait();
                    if (tok >= 0 && g.slot < 0) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float y = __uint_as_float(u[e + 2 * k]) * inv, z = __uint_as_float(u[e + 2 * k + 1]) * inv;
                                w[k] = F16 ? pack_f16_rn(y, z) : pack_bf2(y, z);
                            }
                            *reinterpret_cast<uint4 *>(o + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else if (tok >= 0) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4 *>(po + c + e) = make_uint4(u[e], u[e + 1], u[e + 2], u[e + 3]);
                    }
                }
                const float base = m == -INFINITY ? -INFINITY : m * sl2;
                if (tok >= 0 && g.slot < 0)
                    put_lse(g, tok, l == 0.f ? -INFINITY : (base + log2f(l)) * kLn2);
                else if (tok >= 0)
                    p.w.part_ml[static_cast<int64_t>(g.slot) * NT * kTile + x * kTile + row] = make_float2(base, l);
            }
            tc_fence_before();
            s = after;
        }
        if (!ok) fail();
        cp_async_wait_all();
    } else {
        few_regs();
    }
    __syncthreads();
    if (wp == C::kMmaWarp) {
        tmem_relinquish();
        tmem_dealloc(tm, 512);
    }
}

// ---------------------------------------------------------------- combine
// Rows of the items that were cut: a warp per row,
//   M = max_i m_i,  L = sum_i 2^(m_i - M) l_i,  o = sum_i 2^(m_i - M) o_i / L.
constexpr int kJoinRows = 16;  // rows of a block: 4 warps, 4 rows each

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(128) gdn2_attn_combine_kernel(const __grid_constant__ KernelParams p) {
    constexpr int E = D / 32;  // channels of a lane
    const AttnParams &a = p.a;
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    pdl_wait();
    const Joint j = p.w.joint[blockIdx.x];
    if (j.more <= 0) return;
    const int64_t t0 = cu_of(a.cu, a.cu64, j.n) + j.j0;
    for (int i = wp; i < kJoinRows; i += 4) {
        const int r = blockIdx.y * kJoinRows + i, x = r / kTile, rr = r % kTile;
        const int tk = rr / a.G, tok = x * p.tt + tk, hd = rr - tk * a.G;
        if (tk >= p.tt || tok >= j.ntok) continue;
        auto slot = [&](int k) { return k == 0 ? j.slot : 2 * (static_cast<int>(blockIdx.x) + k); };
        auto at = [&](int k) { return static_cast<int64_t>(slot(k)) * NT * kTile + r; };
        float M = -INFINITY;
        for (int k = lane; k <= j.more; k += 32) M = fmaxf(M, p.w.part_ml[at(k)].x);
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float base = M == -INFINITY ? 0.f : M;
        float L = 0.f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        for (int k0 = 0; k0 <= j.more; k0 += 32) {
            float w = 0.f, l = 0.f;
            if (k0 + lane <= j.more) {
                const float2 ml = p.w.part_ml[at(k0 + lane)];
                w = ex2(ml.x - base);
                l = w * ml.y;
            }
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            L += l;
            const int cnt = min(32, j.more + 1 - k0);
#pragma unroll 4
            for (int k = 0; k < cnt; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, k);
                const float *o = p.w.part_o + at(k0 + k) * D + lane * E;
                if (E == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(o);
                    acc[0] += wk * v.x; acc[1] += wk * v.y; acc[E - 2] += wk * v.z; acc[E - 1] += wk * v.w;
                } else {
                    const float2 v = *reinterpret_cast<const float2 *>(o);
                    acc[0] += wk * v.x; acc[1] += wk * v.y;
                }
            }
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int h = j.h * a.G + hd;
        bf16 *o = a.out + (t0 + tok) * a.so_t + h * a.so_h + lane * E;
        uint32_t w[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e)
            w[e] = F16 ? pack_f16_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv) : pack_bf2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
        if (E == 4)
            *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[E / 2 - 1]);
        else
            *reinterpret_cast<uint32_t *>(o) = w[0];
        if (a.lse && lane == 0) a.lse[(t0 + tok) * a.HQ + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
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
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT, bool F16>
cudaError_t launch(const KernelParams &p, int ctas, cudaStream_t s) {
    using C = Cfg<D, NT>;
    auto kern = gdn2_paged_attn_kernel<D, NT, F16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_chained(kern, dim3(ctas), dim3(C::kThreads), C::kSmem, s, p);
    if (e != cudaSuccess) return e;
    return launch_chained(gdn2_attn_combine_kernel<D, NT, F16>, dim3(ctas, NT * kTile / kJoinRows), dim3(128), 0, s, p);
}

}  // namespace

size_t paged_attn_workspace(const gdn2_attn_dims &d) { return layout_of(d).total; }

cudaError_t launch_paged_attn(const AttnParams &a, const gdn2_attn_dims &d, int sms, void *workspace, cudaStream_t s) {
    const bool f16 = d.dtype == GDN2_DTYPE_F16;
    const int nt = row_tiles(d), ctas = sms < kMaxCtas ? sms : kMaxCtas;
    const Layout l = layout_of(d);
    char *ws = static_cast<char *>(workspace);
    KernelParams p;
    p.a = a;
    p.w.first = reinterpret_cast<int *>(ws + l.first);
    p.w.last = reinterpret_cast<int *>(ws + l.last);
    p.w.joint = reinterpret_cast<Joint *>(ws + l.joint);
    p.w.seq = reinterpret_cast<SeqPlan *>(ws + l.seq);
    p.w.seg = reinterpret_cast<Segment *>(ws + l.seg);
    p.w.part_o = reinterpret_cast<float *>(ws + l.part_o);
    p.w.part_ml = reinterpret_cast<float2 *>(ws + l.part_ml);
    p.scale_log2 = a.scale * kLog2e;
    p.tt = kTile / a.G;
    p.granule = 8;
    while (p.granule < kTile && a.page_size % (2 * p.granule) == 0) p.granule *= 2;
    if (a.T > 0 && (!encode_cache(&p.tk, p.kpos, a.k_cache, a, a.skc, d.D, f16, p.granule) ||
                    !encode_cache(&p.tv, p.vpos, a.v_cache, a, a.svc, d.D, f16, p.granule)))
        return cudaErrorInvalidValue;
    gdn2_attn_plan_kernel<<<1, kPlanThreads, 0, s>>>(p, ctas, nt);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.T == 0) return e;
    if (d.D == 64) {
        if (nt == 1) return f16 ? launch<64, 1, true>(p, ctas, s) : launch<64, 1, false>(p, ctas, s);
        return f16 ? launch<64, 2, true>(p, ctas, s) : launch<64, 2, false>(p, ctas, s);
    }
    if (nt == 1) return f16 ? launch<128, 1, true>(p, ctas, s) : launch<128, 1, false>(p, ctas, s);
    return f16 ? launch<128, 2, true>(p, ctas, s) : launch<128, 2, false>(p, ctas, s);
}

}  // namespace gdn2
