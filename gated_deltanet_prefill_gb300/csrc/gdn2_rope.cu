// Per-head RMS norm and rotary position embedding of queries and keys, and the
// same on the way into a paged key/value cache (include/gdn2_attn.h).
//
// Per row x of D channels with weight w, rotated pair (a, b) and angle z:
//   r = 1 / sqrt(mean(x^2) + eps)
//   y_a = m r (x_a w_a cos z - x_b w_b sin z),  y_b = m r (x_b w_b cos z + x_a w_a sin z)
// so every channel is y = r (x A + x_partner B), where A and B hold the weight,
// the sine or cosine and the factor m, and depend on the token and the channel
// but not on the head.  A half-warp (D = 128; a quarter for D = 64) holds one
// row, 8 channels per lane in one 16-byte load; a lane keeps its channels for
// all heads of its token, so A and B are formed once per token for the queries
// and once for the keys, and a row costs one load, the shuffles of the sum of
// squares, those that fetch the partner's 8 channels (half layout; in the
// interleaved one the partner is in the lane) and 16 multiply-adds.
//
// Bound by memory: 32768 tokens of 32 + 32 heads (half of each head rotated) take
// 176 us, 6.10 TB/s of the 6.78 that a copy reaches; the append of 34997 tokens of
// 32 + 32 + 32 heads to pages of 16 takes 262 us, 6.57 TB/s.  The packed fp32
// instructions keep the issue slots below what the loads need.  A warp takes all
// heads of a token when there are tokens enough to fill the GPU, and a slice of
// them otherwise, so that a decode step is one row group per warp (128 tokens of
// 40 heads: 4 us, of which the launch is most).
#include "gdn2_attn_internal.h"
#include "gdn2_tc.cuh"

namespace gdn2 {
namespace {

using namespace tc;

constexpr int kWarps = 4;    // warps per block
constexpr int kUnroll = 4;
// Blocks per SM that the registers are cut for (72 a thread; a few of the
// coefficients spill).  Measured on 32768 tokens of 64 heads and on the append of
// 34997 tokens of 96: 200 and 288 us uncut (92 registers, 5 blocks), 187 and 269
// with 6, 179 and 266 with 7, 179 and 268 with 8; 2 groups in flight at 8 blocks
// 192 and 290, 8 groups at 4 blocks 205 and 284.
constexpr int kMinBlocks = 7;
// Warps per SM that the slicing aims at: every slice of a token forms the angles
// (and finds the page) again, so not all 28 that fit.  4099 tokens of 20 heads, 128 of 40,
// the append of 4600 tokens of 20 rows and of 128 of 48: 7.9, 4.1, 9.1 and 5.7 us with
// 32; 6.3, 3.8, 7.9 and 4.9 with 16 (and with 12).
constexpr int kWarpsPerSm = 16;

// Angle per position as a fraction of a turn in units of 2^-64 turns: f / (2
// pi) * 2^64 modulo 2^64, from the double's bits (integers only: double
// arithmetic would cost more than the rest of the token).  position * fraction
// wraps modulo a turn by itself, so the angle is off by no more than the fraction is,
// times the position: less than 1.4 x 2^-64 turns per position for f <= 1 (one for the
// bits cut off, f / pi for those of C), less than 2^-31 turns at position 2^32.
// With f = M 2^(e - 63), M in [2^63, 2^64), and C = 2^66 / (2 pi):
// f 2^64 / (2 pi) = M C 2^(e - 65).
__device__ __forceinline__ uint64_t turn_fraction(double f) {
    constexpr uint64_t C = 0xA2F9836E4E441529ull;  // floor(2^66 / (2 pi)) = floor(2^64 * 2 / pi)
    const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
    const int e = static_cast<int>((bits >> 52) & 2047) - 1023;
    const uint64_t M = (bits << 11) | (1ull << 63);
    const uint64_t hi = __umul64hi(M, C), lo = M * C;
    // (hi 2^64 + lo) 2^(e - 65)
    uint64_t r;
    if (e <= 1)
        r = 1 - e < 64 ? hi >> (1 - e) : 0;
    else if (e <= 64)
        r = (hi << (e - 1)) | (lo >> (65 - e));
    else
        r = e < 129 ? lo << (e - 65) : 0;
    return bits >> 63 ? 0 - r : r;
}

// Sine and cosine of position * fraction turns.  The angle is reduced exactly,
// then one multiply-add rounds it; on [-pi, pi] the special-function unit errs
// by 2^-21, far below the outputs' 16 bits.
__device__ __forceinline__ void turn_sincos(int64_t pos, uint64_t fraction, float &s, float &c) {
    const int32_t a = static_cast<int32_t>((static_cast<uint64_t>(pos) * fraction) >> 32);
    __sincosf(static_cast<float>(a) * 1.4629180792671596e-9f, &s, &c);  // a 2^-32 turns, 2 pi / 2^32
}

// The sequence of token t, -1 if there is none; all lanes get the same.
__device__ __forceinline__ int sequence_of(const RopeParams &p, int64_t t, int lane) {
    int lo = 0, hi = p.N;
    if (hi <= 0) return -1;
    do {
        const int step = (hi - lo + 31) >> 5;
        const int i = lo + lane * step;
        const uint32_t below = __ballot_sync(0xffffffffu, i < hi && cu_of(p.cu, p.cu64, i) <= t);
        if (!below) return -1;
        lo += (31 - __clz(below)) * step;
        hi = min(hi, lo + step);
    } while (hi - lo > 1);
    return lo;
}

struct Place {
    int64_t place, page;
    int slot;
    bool ok;
};

__device__ __forceinline__ Place place_of(const RopeParams &p, int64_t t, int lane) {
    Place r = {0, 0, 0, false};
    const int n = sequence_of(p, t, lane);
    if (n < 0) return r;
    const int64_t end = cu_of(p.cu, p.cu64, n + 1);
    r.place = p.kv_lens[n] - (end - t);
    if (t >= end || r.place < 0 || r.place >= static_cast<int64_t>(p.max_pages) * p.page_size) return r;
    const int at = static_cast<int>(r.place);
    const int col = quotient(at, p.page);
    r.slot = at - col * p.page_size;
    r.page = p.table[n * p.table_stride + col];
    r.ok = r.page >= 0 && r.page < p.num_pages;
    return r;
}

// Checks cu_seqlens, the new tokens' places and their table entries, and
// writes the status words; run by one block (which alone writes them, so that
// the words need no clearing before the call).
__device__ void check_tables(const RopeParams &p) {
    __shared__ int bad_cu, bad_page;
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) bad_cu = bad_page = 0;
    __syncthreads();
    if (tid == 0 && (p.N > 0 ? cu_of(p.cu, p.cu64, 0) != 0 || cu_of(p.cu, p.cu64, p.N) != p.T : p.T != 0)) bad_cu = 1;
    auto bad_entry = [&](int n, int col) {
        const int64_t page = p.table[n * p.table_stride + col];
        return page < 0 || page >= p.num_pages;
    };
    for (int base = tid - lane; base < p.N; base += blockDim.x) {  // 32 sequences per warp
        const int n = base + lane;
        int col0 = 0, cols = 0;
        if (n < p.N) {
            const int64_t a = cu_of(p.cu, p.cu64, n), b = cu_of(p.cu, p.cu64, n + 1), len = p.kv_lens[n];
            if (a > b || a < 0 || b > p.T) {
                bad_cu = 1;
            } else if (a < b) {
                if (len < b - a || len > static_cast<int64_t>(p.max_pages) * p.page_size) {
                    bad_page = 1;
                } else {
                    col0 = quotient(static_cast<int>(len - (b - a)), p.page);
                    cols = quotient(static_cast<int>(len) - 1, p.page) + 1 - col0;
                }
            }
        }
        if (cols > 0 && bad_entry(n, col0)) bad_page = 1;
        for (uint32_t more = __ballot_sync(0xffffffffu, cols > 1); more; more &= more - 1) {
            const int src = __ffs(more) - 1;
            const int c0 = __shfl_sync(0xffffffffu, col0, src), c = __shfl_sync(0xffffffffu, cols, src);
            for (int i = 1 + lane; i < c; i += 32)
                if (bad_entry(base + src, c0 + i)) bad_page = 1;
        }
    }
    __syncthreads();
    if (tid < 8) p.status[tid] = tid ? 0 : bad_cu ? GDN2_ERR_CU_SEQLENS : bad_page ? GDN2_ERR_PAGES : GDN2_OK;
}

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
    if (F16)
        unpack8_f16(u, f);
    else
        unpack8_bf(u, f);
}
// Pairs of fp32 values in 64-bit registers, and the packed operations on them (one
// instruction for two).
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
template <bool F16>
__device__ __forceinline__ void unpack8_pairs(const uint4 &u, uint64_t (&f)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = F16 ? unpack_h2(w[i]) : unpack_bf2(w[i]);
        f[i] = pair(x.x, x.y);
    }
}

// PAGED: keys and values go to their pages, and block 0 checks the tables.
template <int D, bool F16, bool INTER, bool PAGED>
__global__ void __launch_bounds__(32 * kWarps, kMinBlocks) gdn2_rope_kernel(const __grid_constant__ RopeParams p, int slices,
                                                                int rows_per_slice) {
    constexpr int L = D / 8;    // lanes per row
    constexpr int R = 32 / L;   // rows per warp and load
    if (PAGED && blockIdx.x == 0) {
        check_tables(p);
        return;
    }
    const int lane = threadIdx.x & 31, c = lane % L, sub = lane / L;
    const uint32_t warp = (blockIdx.x - (PAGED ? 1 : 0)) * kWarps + (threadIdx.x >> 5);  // (T is below 2^31, or slices 1)
    const int64_t t = slices == 1 ? warp : warp / slices;
    if (t >= p.T) return;
    const int r0 = static_cast<int>(warp - t * slices) * rows_per_slice;
    const int r1 = min(r0 + rows_per_slice, p.HQ + p.HK + p.HV);

    // The first rows are asked for at once: what comes before their use, the place in
    // the cache and the angles, is a chain of loads of its own.
    uint4 u[kUnroll];
    auto load = [&](int h0, int hi, const bf16 *x, int64_t sx) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int h = h0 + i * R + sub;
            u[i] = make_uint4(0, 0, 0, 0);
            if (h < hi) u[i] = *reinterpret_cast<const uint4 *>(x + h * sx + 8 * c);
        }
    };
    const int k0 = p.HQ, v0 = p.HQ + p.HK;
    if (r0 < k0)
        load(r0, min(r1, k0), p.q + t * p.sq_t, p.sq_h);
    else if (r0 < v0)
        load(r0 - k0, min(r1, v0) - k0, p.k + t * p.sk_t, p.sk_h);

    Place at = {0, 0, 0, true};
    if (PAGED) {
        at = place_of(p, t, lane);
        if (!at.ok) return;
    }
    const bool turned = 8 * c < p.rot_dim;
    const int half = p.rot_dim >> 1;
    const bool second = !INTER && 8 * c >= half;
    const int partner = INTER || !turned ? c : second ? c - half / 8 : c + half / 8;
    constexpr int F = INTER ? 4 : 8;
    float cs[F], sn[F];  // times the factor; the sine signed for this lane's side of the pair
#pragma unroll
    for (int e = 0; e < F; ++e) { cs[e] = 1.f; sn[e] = 0.f; }
    if (turned) {
        const int64_t pos = PAGED && !p.positions ? at.place
                            : p.pos64             ? static_cast<const int64_t *>(p.positions)[t]
                                                  : static_cast<const int32_t *>(p.positions)[t];
        const double *f = p.inv_freq + (INTER ? 4 * c : second ? 8 * c - half : 8 * c);
#pragma unroll
        for (int e = 0; e < F; ++e) {
            turn_sincos(pos, turn_fraction(f[e]), sn[e], cs[e]);
            cs[e] *= p.factor;
            sn[e] *= second || INTER ? p.factor : -p.factor;
        }
    }

    // rows [lo, hi) of one kind: queries or keys
    auto rows = [&](int lo, int hi, const bf16 *x, int64_t sx, bf16 *y, int64_t sy, const bf16 *w, bool loaded) {
        if (lo >= hi) return;
        uint64_t A[4], B[4];  // of channels 2 e and 2 e + 1
        {
            float wa[8], wb[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) wa[e] = wb[e] = 1.f;
            if (w) {
                unpack8<F16>(*reinterpret_cast<const uint4 *>(w + 8 * c), wa);
                unpack8<F16>(*reinterpret_cast<const uint4 *>(w + 8 * partner), wb);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                A[e] = INTER ? pair(wa[2 * e] * cs[e], wa[2 * e + 1] * cs[e]) : pair(wa[2 * e] * cs[INTER ? 0 : 2 * e], wa[2 * e + 1] * cs[INTER ? 0 : 2 * e + 1]);
                B[e] = INTER ? pair(wb[2 * e + 1] * -sn[e], wb[2 * e] * sn[e]) : pair(wb[2 * e] * sn[INTER ? 0 : 2 * e], wb[2 * e + 1] * sn[INTER ? 0 : 2 * e + 1]);
                if (!turned) B[e] = 0;  // (0 x inf is NaN)
            }
        }
        const int src = lane - c + partner;
        for (int h0 = lo; h0 < hi; h0 += R * kUnroll) {
            if (!loaded) load(h0, hi, x, sx);
            loaded = false;
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                if (h0 + i * R >= hi) break;  // the same for all lanes
                uint64_t v[4], z[4];
                unpack8_pairs<F16>(u[i], v);
                float r = 1.f;
                if (p.norm) {
                    uint64_t s2 = mul2(v[0], v[0]);
#pragma unroll
                    for (int e = 1; e < 4; ++e) s2 = fma2(v[e], v[e], s2);
                    const float2 t2 = unpair(s2);
                    float sum = t2.x + t2.y;
#pragma unroll
                    for (int d = L / 2; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    r = rsqrtf(sum * (1.f / D) + p.eps);
                }
                // the partners' values; zero where nothing turns (0 x inf is NaN)
                if (INTER) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 t2 = unpair(v[e]);
                        z[e] = turned ? pair(t2.y, t2.x) : 0;
                    }
                } else {
                    uint4 q;
                    q.x = __shfl_sync(0xffffffffu, u[i].x, src);
                    q.y = __shfl_sync(0xffffffffu, u[i].y, src);
                    q.z = __shfl_sync(0xffffffffu, u[i].z, src);
                    q.w = __shfl_sync(0xffffffffu, u[i].w, src);
                    if (!turned) q = make_uint4(0, 0, 0, 0);
                    unpack8_pairs<F16>(q, z);
                }
                const uint64_t r2 = pair(r, r);
                uint4 out;
                uint32_t *o = &out.x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 t2 = unpair(mul2(r2, fma2(z[e], B[e], mul2(v[e], A[e]))));
                    o[e] = F16 ? pack_f16_rn(t2.x, t2.y) : pack_bf2(t2.x, t2.y);
                }
                const int h = h0 + i * R + sub;
                if (h < hi) *reinterpret_cast<uint4 *>(y + h * sy + 8 * c) = out;
            }
        }
    };
    rows(r0, min(r1, p.HQ), p.q + t * p.sq_t, p.sq_h, p.q_out + t * p.sqo_t, p.sqo_h, p.q_weight, true);
    rows(max(r0, k0) - k0, min(r1, v0) - k0, p.k + t * p.sk_t, p.sk_h,
         PAGED ? p.k_cache + at.page * p.skc[0] + at.slot * p.skc[1] : p.k_out + t * p.sko_t,
         PAGED ? p.skc[2] : p.sko_h, p.k_weight, r0 >= k0);
    if (PAGED) {
        const bf16 *x = p.v + t * p.sv_t;
        bf16 *y = p.v_cache + at.page * p.svc[0] + at.slot * p.svc[1];
        const int hi = r1 - v0;
        for (int h0 = max(r0, v0) - v0 + sub; h0 < hi; h0 += R * kUnroll) {
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
                if (h0 + i * R < hi) u[i] = *reinterpret_cast<const uint4 *>(x + (h0 + i * R) * p.sv_h + 8 * c);
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
                if (h0 + i * R < hi) *reinterpret_cast<uint4 *>(y + (h0 + i * R) * p.svc[2] + 8 * c) = u[i];
        }
    }
}

template <int D, bool F16, bool INTER>
cudaError_t launch(const RopeParams &p, int sms, cudaStream_t s) {
    constexpr int R = 32 / (D / 8);
    const int rows = p.HQ + p.HK + p.HV;
    int64_t slices = 1, per = rows;
    if (p.T > 0 && rows > 0) {
        const int64_t want = (static_cast<int64_t>(sms) * kWarpsPerSm + p.T - 1) / p.T;
        const int64_t most = (rows + R - 1) / R;
        slices = want < 1 ? 1 : want > most ? most : want;
        per = ((rows + slices - 1) / slices + R - 1) / R * R;
        slices = (rows + per - 1) / per;
    }
    const int64_t blocks = rows > 0 ? (p.T * slices + kWarps - 1) / kWarps : 0;
    if (p.status)
        gdn2_rope_kernel<D, F16, INTER, true><<<static_cast<unsigned>(blocks + 1), 32 * kWarps, 0, s>>>(
            p, static_cast<int>(slices), static_cast<int>(per));
    else if (blocks > 0)
        gdn2_rope_kernel<D, F16, INTER, false><<<static_cast<unsigned>(blocks), 32 * kWarps, 0, s>>>(
            p, static_cast<int>(slices), static_cast<int>(per));
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const RopeParams &p, bool f16, bool interleaved, int sms, cudaStream_t s) {
    if (f16) return interleaved ? launch<D, true, true>(p, sms, s) : launch<D, true, false>(p, sms, s);
    return interleaved ? launch<D, false, true>(p, sms, s) : launch<D, false, false>(p, sms, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int D, bool f16, bool interleaved, int sms, cudaStream_t s) {
    return D == 64 ? launch_d<64>(p, f16, interleaved, sms, s) : launch_d<128>(p, f16, interleaved, sms, s);
}

}  // namespace gdn2
