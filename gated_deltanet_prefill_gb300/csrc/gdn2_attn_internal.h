// Internal declarations of the attention-layer operators (include/gdn2_attn.h).
// Only their own sources include it, so it is no part of the GDN-2 kernels' shared
// headers (*.cuh), by which their profiles are matched.
#pragma once

#include "gdn2_attn.h"
#include "gdn2_internal.cuh"

namespace gdn2 {

// Workspace of the append call: the status words only.
constexpr size_t kAppendWorkspaceBytes = 64;

// A division by a number fixed on the host takes two instructions: for k < 2^31,
// k / d = floor(k m / 2^(31 + l)) with 2^(l - 1) < d <= 2^l and m = ceil(2^(31 + l) / d)
// (which is below 2^32, and off by less than k / 2^(31 + l) < 1 / d).  A division of two
// variables takes 100 to 200 cycles.
struct Divisor {
    uint32_t mul;
    int shift;
};
inline Divisor divisor(int d) {  // 2 <= d
    int l = 1;
    while ((1ll << l) < d) ++l;
    return {static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d), l - 1};
}
__device__ __forceinline__ int quotient(int k, const Divisor &d) {
    return static_cast<int>(__umulhi(static_cast<uint32_t>(k), d.mul) >> d.shift);
}

// Norm and rotation, with or without the paged cache as the keys' target.
struct RopeParams {
    const bf16 *q, *k, *v;              // dtype of the call (the bits are fp16 when f16)
    const bf16 *q_weight, *k_weight;    // null: ones
    const double *inv_freq;
    const void *positions;              // null: the places in the cached sequences
    int pos64;
    bf16 *q_out, *k_out;                // k_out: null with the paged cache
    bf16 *k_cache, *v_cache;
    int64_t sq_t, sq_h, sk_t, sk_h, sv_t, sv_h, sqo_t, sqo_h, sko_t, sko_h;
    int64_t skc[3], svc[3];             // page, token in the page, head
    const void *cu;
    int cu64;
    const int *kv_lens, *table;
    int64_t table_stride;
    int64_t num_pages;
    int64_t T;
    int N, HQ, HK, HV;                  // heads of q, k and v that the call has (0: left out)
    int page_size, max_pages;
    Divisor page;                       // page_size
    int rot_dim, norm;
    float eps, factor;
    int *status;                        // null without the paged cache
};

cudaError_t launch_rope(const RopeParams &p, int D, bool f16, bool interleaved, int sms, cudaStream_t s);

struct AttnParams {
    const bf16 *q, *k_cache, *v_cache;
    bf16 *out;
    float *lse;
    int64_t sq_t, sq_h, so_t, so_h;
    int64_t skc[3], svc[3];
    const void *cu;
    int cu64;
    const int *kv_lens, *table;
    int64_t table_stride;
    int64_t num_pages;
    int64_t T;
    int N, HQ, HKV, G;                  // G = HQ / HKV query heads per key head
    int page_size, max_pages;
    int causal, window;                 // window < 0: none
    int lead;                           // of an item of two row tiles, in key tiles
    float scale;
    int *status;
};

size_t paged_attn_workspace(const gdn2_attn_dims &d);
cudaError_t launch_paged_attn(const AttnParams &p, const gdn2_attn_dims &d, int sms, void *workspace, cudaStream_t s);

__device__ __forceinline__ int64_t cu_of(const void *cu, int cu64, int i) {
    return cu64 ? static_cast<const int64_t *>(cu)[i] : static_cast<int64_t>(static_cast<const int32_t *>(cu)[i]);
}

}  // namespace gdn2
