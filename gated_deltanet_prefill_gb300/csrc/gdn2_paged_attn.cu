// Softmax attention of the new tokens over a paged key/value cache
// (include/gdn2_attn.h).
//
// One warp per (token, query head): 32 keys at a time, a lane scores one key,
// the running maximum and sum are kept per row, and the lanes share the
// channels of the weighted sum of the values.
#include "gdn2_attn_internal.cuh"

namespace gdn2 {
namespace {

__device__ __forceinline__ float el(const bf16 *p, bool f16) {
    return f16 ? __half2float(*reinterpret_cast<const __half *>(p)) : __bfloat162float(*p);
}

__global__ void attn_status_kernel(AttnParams p) {
    __shared__ int bad_cu, bad_len;
    if (threadIdx.x == 0) {
        bad_cu = p.N > 0 ? cu_of(p.cu, p.cu64, 0) != 0 || cu_of(p.cu, p.cu64, p.N) != p.T : p.T != 0;
        bad_len = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.N; i += blockDim.x) {
        if (cu_of(p.cu, p.cu64, i) > cu_of(p.cu, p.cu64, i + 1)) bad_cu = 1;
        if (p.kv_lens[i] < 0 || p.kv_lens[i] > static_cast<int64_t>(p.max_pages) * p.page_size) bad_len = 1;
    }
    __syncthreads();
    if (threadIdx.x < 8)
        p.status[threadIdx.x] = threadIdx.x ? 0 : bad_cu ? GDN2_ERR_CU_SEQLENS : bad_len ? GDN2_ERR_PAGES : GDN2_OK;
}

template <int D>
__global__ void __launch_bounds__(128) attn_kernel(AttnParams p, bool f16) {
    __shared__ float qs[4][D];
    __shared__ float ps[4][32];
    __shared__ const bf16 *vs[4][32];
    if (p.status[0] != GDN2_OK) return;
    const int wp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + wp;
    const int64_t t = r / p.HQ;
    const int h = static_cast<int>(r % p.HQ), hk = h / p.G;
    if (t >= p.T) return;
    int n = 0, hi = p.N;
    while (hi - n > 1) {
        const int mid = (n + hi) / 2;
        if (cu_of(p.cu, p.cu64, mid) <= t)
            n = mid;
        else
            hi = mid;
    }
    const int64_t len = p.kv_lens[n], place = len - (cu_of(p.cu, p.cu64, n + 1) - t);
    const int64_t end = p.causal ? min(len, place + 1) : len;
    const int64_t begin = p.window >= 0 ? max(static_cast<int64_t>(0), place - p.window) : 0;
    for (int c = lane; c < D; c += 32) qs[wp][c] = el(p.q + t * p.sq_t + h * p.sq_h + c, f16) * p.scale;
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    for (int64_t c0 = begin; c0 < end; c0 += 32) {
        const int64_t c = c0 + lane;
        float x = -INFINITY;
        const bf16 *v = nullptr;
        if (c < end) {
            const int64_t page = p.table[n * p.table_stride + c / p.page_size], slot = c % p.page_size;
            if (page >= 0 && page < p.num_pages) {
                const bf16 *k = p.k_cache + page * p.skc[0] + slot * p.skc[1] + hk * p.skc[2];
                v = p.v_cache + page * p.svc[0] + slot * p.svc[1] + hk * p.svc[2];
                x = 0.f;
                for (int d = 0; d < D; ++d) x += qs[wp][d] * el(k + d, f16);
            } else {
                p.status[0] = GDN2_ERR_PAGES;
            }
        }
        float top = x;
        for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
        const float m1 = fmaxf(m, top), base = m1 == -INFINITY ? 0.f : m1;
        const float e = expf(x - base), fix = expf(m - base);
        float sum = e;
        for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
        l = l * fix + sum;
        m = m1;
        ps[wp][lane] = e;
        vs[wp][lane] = v;
        __syncwarp();
        for (int j = 0; j < D / 32; ++j) o[j] *= fix;
        for (int i = 0; i < 32; ++i)
            if (vs[wp][i])
                for (int j = 0; j < D / 32; ++j) o[j] += ps[wp][i] * el(vs[wp][i] + lane + 32 * j, f16);
        __syncwarp();
    }
    bf16 *y = p.out + t * p.so_t + h * p.so_h;
    for (int j = 0; j < D / 32; ++j) {
        const float x = l > 0.f ? o[j] / l : 0.f;
        if (f16)
            reinterpret_cast<__half *>(y)[lane + 32 * j] = __float2half_rn(x);
        else
            y[lane + 32 * j] = __float2bfloat16_rn(x);
    }
    if (p.lse && lane == 0) p.lse[t * p.HQ + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t paged_attn_workspace(const gdn2_attn_dims &) { return 64; }

cudaError_t launch_paged_attn(const AttnParams &p, int D, bool f16, int, void *, cudaStream_t s) {
    attn_status_kernel<<<1, 256, 0, s>>>(p);
    const int64_t rows = p.T * p.HQ;
    if (rows > 0) {
        const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
        if (D == 64)
            attn_kernel<64><<<grid, 128, 0, s>>>(p, f16);
        else
            attn_kernel<128><<<grid, 128, 0, s>>>(p, f16);
    }
    return cudaGetLastError();
}

}  // namespace gdn2
