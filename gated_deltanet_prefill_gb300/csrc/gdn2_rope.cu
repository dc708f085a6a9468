// Per-head RMS norm and rotary position embedding of queries and keys, and the
// same on the way into a paged key/value cache (include/gdn2_attn.h).
//
// One warp per (token, head) row; the row's channels sit in shared memory
// between the norm and the rotation.
#include "gdn2_attn_internal.cuh"

namespace gdn2 {
namespace {

// Angle per position as a fraction of a turn, in units of 2^-64 turns: f
// radians (f >= 0, finite) times 2^64 / (2 pi), modulo a turn.  position *
// fraction wraps modulo a turn by itself, so the angle of any position is
// exact to the frequency's own rounding.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
    const double t = f * 0.15915494309189533577;
    return static_cast<uint64_t>((t - floor(t)) * 18446744073709551616.0);
}

__device__ __forceinline__ float to_f(bf16 x, bool f16) {
    return f16 ? __half2float(*reinterpret_cast<const __half *>(&x)) : __bfloat162float(x);
}
__device__ __forceinline__ void put(bf16 *p, float x, bool f16) {
    if (f16)
        *reinterpret_cast<__half *>(p) = __float2half_rn(x);
    else
        *p = __float2bfloat16_rn(x);
}

// The sequence of token t (the last n with cu[n] <= t), or -1.
__device__ int sequence_of(const RopeParams &p, int64_t t) {
    int lo = 0, hi = p.N;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cu_of(p.cu, p.cu64, mid) <= t)
            lo = mid;
        else
            hi = mid;
    }
    return p.N > 0 && cu_of(p.cu, p.cu64, lo) <= t && t < cu_of(p.cu, p.cu64, lo + 1) ? lo : -1;
}

// Page and slot of a token's place; false if the place or the entry is bad.
__device__ bool place_of(const RopeParams &p, int64_t t, int64_t &place, int64_t &page, int &slot) {
    const int n = sequence_of(p, t);
    if (n < 0) return false;
    place = p.kv_lens[n] - (cu_of(p.cu, p.cu64, n + 1) - t);
    if (place < 0 || place / p.page_size >= p.max_pages) return false;
    page = p.table[n * p.table_stride + place / p.page_size];
    slot = static_cast<int>(place % p.page_size);
    return page >= 0 && page < p.num_pages;
}

__global__ void rope_status_kernel(RopeParams p) {
    __shared__ int bad_cu, bad_page;
    if (threadIdx.x == 0) {
        bad_cu = p.N > 0 ? cu_of(p.cu, p.cu64, 0) != 0 || cu_of(p.cu, p.cu64, p.N) != p.T : p.T != 0;
        bad_page = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.N; i += blockDim.x)
        if (cu_of(p.cu, p.cu64, i) > cu_of(p.cu, p.cu64, i + 1)) bad_cu = 1;
    __syncthreads();
    if (!bad_cu)
        for (int64_t t = threadIdx.x; t < p.T; t += blockDim.x) {
            int64_t place, page;
            int slot;
            if (!place_of(p, t, place, page, slot)) bad_page = 1;
        }
    __syncthreads();
    if (threadIdx.x < 8)
        p.status[threadIdx.x] = threadIdx.x ? 0 : bad_cu ? GDN2_ERR_CU_SEQLENS : bad_page ? GDN2_ERR_PAGES : GDN2_OK;
}

template <int D>
__global__ void __launch_bounds__(128) rope_kernel(RopeParams p, bool f16, bool interleaved) {
    __shared__ float row[4][D];
    const int wp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int heads = p.HQ + p.HK + p.HV;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + wp;
    const int64_t t = r / heads;
    int h = static_cast<int>(r % heads);
    if (t >= p.T) return;
    int64_t place = 0, page = 0;
    int slot = 0;
    if (p.status && !place_of(p, t, place, page, slot)) return;
    const bool is_q = h < p.HQ, is_v = h >= p.HQ + p.HK;
    h -= is_v ? p.HQ + p.HK : is_q ? 0 : p.HQ;
    const bf16 *x = is_q ? p.q + t * p.sq_t + h * p.sq_h : is_v ? p.v + t * p.sv_t + h * p.sv_h : p.k + t * p.sk_t + h * p.sk_h;
    bf16 *y = is_q ? p.q_out + t * p.sqo_t + h * p.sqo_h
              : is_v ? p.v_cache + page * p.svc[0] + slot * p.svc[1] + h * p.svc[2]
              : p.k_out ? p.k_out + t * p.sko_t + h * p.sko_h
                        : p.k_cache + page * p.skc[0] + slot * p.skc[1] + h * p.skc[2];
    if (is_v) {
        for (int c = lane; c < D; c += 32) y[c] = x[c];
        return;
    }
    float sum = 0.f;
    for (int c = lane; c < D; c += 32) {
        row[wp][c] = to_f(x[c], f16);
        sum += row[wp][c] * row[wp][c];
    }
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (p.norm) {
        const float inv = rsqrtf(sum / D + p.eps);
        const bf16 *w = is_q ? p.q_weight : p.k_weight;
        for (int c = lane; c < D; c += 32) row[wp][c] *= inv * (w ? to_f(w[c], f16) : 1.f);
    }
    __syncwarp();
    const int64_t pos = p.rot_dim == 0 ? 0
                        : !p.positions ? place
                        : p.pos64      ? static_cast<const int64_t *>(p.positions)[t]
                                       : static_cast<const int32_t *>(p.positions)[t];
    for (int c = lane; c < D; c += 32) {
        float v = row[wp][c];
        if (c < p.rot_dim) {
            const int half = p.rot_dim / 2;
            const int i = interleaved ? c / 2 : c % half;
            const bool second = interleaved ? c & 1 : c >= half;
            const int32_t a = static_cast<int32_t>((static_cast<uint64_t>(pos) * turn_fraction(p.inv_freq[i])) >> 32);
            float sn, cs;
            sincospif(static_cast<float>(a) * 4.656612873077393e-10f, &sn, &cs);  // a / 2^31 half turns
            const float u = row[wp][interleaved ? c ^ 1 : second ? c - half : c + half];
            v = p.factor * (second ? v * cs + u * sn : v * cs - u * sn);
        }
        put(y + c, v, f16);
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int D, bool f16, bool interleaved, int, cudaStream_t s) {
    if (p.status) rope_status_kernel<<<1, 256, 0, s>>>(p);
    const int64_t rows = p.T * (p.HQ + p.HK + p.HV);
    if (rows > 0) {
        const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
        if (D == 64)
            rope_kernel<64><<<grid, 128, 0, s>>>(p, f16, interleaved);
        else
            rope_kernel<128><<<grid, 128, 0, s>>>(p, f16, interleaved);
    }
    return cudaGetLastError();
}

}  // namespace gdn2
