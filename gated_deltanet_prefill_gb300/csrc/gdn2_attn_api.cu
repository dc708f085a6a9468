// C ABI of the attention-layer operators: argument checks and launches.  See
// include/gdn2_attn.h for the contract.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "gdn2_attn_internal.h"

namespace gdn2 {
namespace {

// A strided [n, heads, D] tensor of 16-bit elements, as bytes.
struct Rows {
    uintptr_t base;
    int64_t n, heads, D, st, sh;  // strides in bytes; D in bytes
    uintptr_t end() const { return base + static_cast<uintptr_t>((n - 1) * st + (heads - 1) * sh + D); }
    bool empty() const { return base == 0 || n <= 0 || heads <= 0; }
};

Rows rows(const void *p, int64_t n, int64_t heads, int64_t D, const int64_t *s) {
    return {reinterpret_cast<uintptr_t>(p), n, heads, D * 2, s[0] * 2, s[1] * 2};
}

// Whether two row tensors may share a byte.  Exact for the common layouts:
// apart as ranges, or views of one packed tensor (the same token stride, the
// heads of a token within it).
bool overlap(const Rows &a, const Rows &b) {
    if (a.empty() || b.empty() || a.end() <= b.base || b.end() <= a.base) return false;
    const int64_t wa = (a.heads - 1) * a.sh + a.D, wb = (b.heads - 1) * b.sh + b.D;
    if (a.st == b.st && a.st > 0 && wa <= a.st && wb <= b.st) {
        const int64_t d = static_cast<int64_t>(b.base) - static_cast<int64_t>(a.base);
        const int64_t off = ((d % a.st) + a.st) % a.st;  // b's first byte within a's token
        return off < wa || off + wb > a.st;
    }
    return true;
}

bool overlap(const Rows &a, const void *p, int64_t bytes) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return !a.empty() && p && bytes > 0 && a.base < b + static_cast<uintptr_t>(bytes) && b < a.end();
}

// Bytes from the cache's first to its last element.
Rows cache_rows(const void *p, const gdn2_attn_dims &d, const int64_t *s) {
    const int64_t in_page = (d.page_size - 1) * s[1] + (d.HKV - 1) * s[2] + d.D;
    const int64_t n = d.num_pages > 0 ? 1 : 0;
    return {reinterpret_cast<uintptr_t>(p), n, 1, ((d.num_pages - 1) * s[0] + in_page) * 2, 0, 0};
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

bool strides_ok(const void *p, const int64_t *s, int n) {
    if (!p) return true;
    if (!aligned16(p)) return false;
    for (int i = 0; i < n; ++i)
        if (s[i] < 0 || s[i] % 8 || s[i] > (1ll << 38)) return false;
    return true;
}

// A cache that the kernels read through tensor maps: no broadcast dimension.
bool mapped_strides_ok(const gdn2_attn_dims &d, const int64_t *s) {
    return (d.num_pages <= 1 || s[0] > 0) && (d.page_size <= 1 || s[1] > 0) && (d.HKV <= 1 || s[2] > 0);
}

// Rows of an output do not overlap one another.
bool rows_apart(const int64_t *s, int64_t n, int heads, int D) {
    if (heads > 1 && s[1] < D) return false;
    if (n <= 1) return true;
    const int64_t width = static_cast<int64_t>(heads - 1) * s[1] + D;
    return s[0] >= width || (s[0] >= D && s[1] >= (n - 1) * s[0] + D) || (heads == 1 && s[0] >= D);
}

// The same for the slots of a cache: in some order of its three strides, each
// steps over all that the smaller ones span.
bool slots_apart(const gdn2_attn_dims &d, const int64_t *s) {
    int64_t st[3] = {s[0], s[1], s[2]}, n[3] = {d.num_pages, d.page_size, d.HKV};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) {
                const int64_t a = st[i], b = n[i];
                st[i] = st[j]; n[i] = n[j];
                st[j] = a; n[j] = b;
            }
    int64_t width = d.D;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (st[i] < width) return false;
        width += (n[i] - 1) * st[i];
    }
    return true;
}

gdn2_status check_common(const gdn2_attn_dims &d) {
    if (d.dtype != GDN2_DTYPE_BF16 && d.dtype != GDN2_DTYPE_F16) return GDN2_ERR_DTYPE;
    if (d.T_tot < 0 || d.T_tot > 2147483647ll - 65536 || d.N < 0 || d.HQ < 0 || d.HKV < 0 || d.HQ > 65536 || d.HKV > 65536)
        return GDN2_ERR_SHAPE;
    if (d.D != 64 && d.D != 128) return GDN2_ERR_SHAPE;
    return GDN2_OK;
}

gdn2_status check_rope(const gdn2_attn_dims &d) {
    if (d.rot_dim < 0 || d.rot_dim > d.D || d.rot_dim % 16) return GDN2_ERR_SHAPE;
    if ((d.norm != 0 && d.norm != 1) || (d.rope_interleaved != 0 && d.rope_interleaved != 1)) return GDN2_ERR_SHAPE;
    if (!isfinite(d.norm_eps) || d.norm_eps < 0.f || !isfinite(d.rope_factor)) return GDN2_ERR_SHAPE;
    return GDN2_OK;
}

bool paged_shape_ok(const gdn2_attn_dims &d) {
    return check_common(d) == GDN2_OK && d.HKV > 0 && d.num_pages >= 1 && d.num_pages <= 2147483647ll &&
           d.page_size >= 8 && d.page_size % 8 == 0 && d.page_size <= (1 << 20) && d.max_pages >= 0 &&
           static_cast<int64_t>(d.max_pages) * d.page_size <= 2147483647ll - 65536 && d.table_stride >= d.max_pages;
}

bool attn_shape_ok(const gdn2_attn_dims &d) {
    return paged_shape_ok(d) && d.HQ > 0 && d.HQ % d.HKV == 0 && d.HQ / d.HKV <= 128 &&
           (d.causal == 0 || d.causal == 1) && d.window_left >= -1 && (d.window_left < 0 || d.causal);
}

int64_t table_bytes(const gdn2_attn_dims &d) {
    return d.N > 0 ? ((d.N - 1) * d.table_stride + d.max_pages) * 4 : 0;
}

int sm_count(int dev) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        sms = 0;
    }
    return sms > 0 ? sms : 152;
}

void fill_rope(RopeParams &p, const gdn2_attn_dims &d, const void *q, const void *k, const void *q_weight,
               const void *k_weight, const double *inv_freq, const void *positions, void *q_out) {
    memset(&p, 0, sizeof(p));
    p.q = static_cast<const bf16 *>(q);
    p.k = static_cast<const bf16 *>(k);
    p.q_weight = d.norm ? static_cast<const bf16 *>(q_weight) : nullptr;  // the weights are part of the norm
    p.k_weight = d.norm ? static_cast<const bf16 *>(k_weight) : nullptr;
    p.inv_freq = inv_freq;
    p.positions = positions;
    p.pos64 = d.positions_i64 ? 1 : 0;
    p.q_out = static_cast<bf16 *>(q_out);
    p.sq_t = d.q_stride[0]; p.sq_h = d.q_stride[1];
    p.sk_t = d.k_stride[0]; p.sk_h = d.k_stride[1];
    p.sqo_t = d.qo_stride[0]; p.sqo_h = d.qo_stride[1];
    p.sko_t = d.ko_stride[0]; p.sko_h = d.ko_stride[1];
    p.T = d.T_tot;
    p.HQ = q ? d.HQ : 0;
    p.HK = k ? d.HKV : 0;
    p.rot_dim = d.rot_dim;
    p.norm = d.norm;
    p.eps = d.norm_eps;
    p.factor = d.rope_factor;
}

// An output of the norm and rotation against an input: the input itself with
// the same strides (in place), or apart from it.
bool in_place_or_apart(const Rows &o, const Rows &in) {
    return (o.base == in.base && o.st == in.st && o.sh == in.sh && o.heads == in.heads) || !overlap(o, in);
}

}  // namespace
}  // namespace gdn2

using namespace gdn2;

extern "C" {

gdn2_status gdn2_attn_dims_init(gdn2_attn_dims *d, int64_t T_tot, int32_t N, int32_t HQ, int32_t HKV, int32_t D,
                                int64_t num_pages, int32_t page_size, int32_t max_pages) {
    if (!d) return GDN2_ERR_NULL;
    memset(d, 0, sizeof(*d));
    d->T_tot = T_tot; d->N = N; d->HQ = HQ; d->HKV = HKV; d->D = D;
    d->num_pages = num_pages; d->page_size = page_size; d->max_pages = max_pages;
    const int64_t D64 = D;
    d->q_stride[0] = d->qo_stride[0] = HQ * D64;
    d->k_stride[0] = d->ko_stride[0] = d->v_stride[0] = HKV * D64;
    d->q_stride[1] = d->qo_stride[1] = d->k_stride[1] = d->ko_stride[1] = d->v_stride[1] = D64;
    d->kc_stride[0] = d->vc_stride[0] = page_size * HKV * D64;
    d->kc_stride[1] = d->vc_stride[1] = HKV * D64;
    d->kc_stride[2] = d->vc_stride[2] = D64;
    d->table_stride = max_pages;
    d->dtype = GDN2_DTYPE_BF16;
    d->norm = 1;
    d->norm_eps = 1e-6f;
    d->rot_dim = D;
    d->rope_factor = 1.f;
    d->causal = 1;
    d->window_left = -1;
    const gdn2_status st = check_common(*d);
    return st != GDN2_OK ? st : check_rope(*d);
}

gdn2_status gdn2_qk_norm_rope(const void *q, const void *k, const void *q_weight, const void *k_weight,
                              const double *inv_freq, const void *positions, void *q_out, void *k_out,
                              const gdn2_attn_dims *dims, void *stream) {
    if (!dims) return GDN2_ERR_NULL;
    const gdn2_attn_dims &d = *dims;
    gdn2_status st = check_common(d);
    if (st == GDN2_OK) st = check_rope(d);
    if (st != GDN2_OK) return st;
    if ((q && d.HQ < 1) || (k && d.HKV < 1)) return GDN2_ERR_SHAPE;
    if ((!q && !k && d.T_tot > 0) || !q != !q_out || !k != !k_out) return GDN2_ERR_NULL;
    if (d.T_tot > 0 && d.rot_dim > 0 && (!inv_freq || !positions)) return GDN2_ERR_NULL;
    if (!strides_ok(q, d.q_stride, 2) || !strides_ok(k, d.k_stride, 2) || !strides_ok(q_out, d.qo_stride, 2) ||
        !strides_ok(k_out, d.ko_stride, 2) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(inv_freq))
        return GDN2_ERR_STRIDE;
    const Rows rq = rows(q, d.T_tot, d.HQ, d.D, d.q_stride), rk = rows(k, d.T_tot, d.HKV, d.D, d.k_stride);
    const Rows oq = rows(q_out, d.T_tot, d.HQ, d.D, d.qo_stride), ok = rows(k_out, d.T_tot, d.HKV, d.D, d.ko_stride);
    if ((q && !rows_apart(d.qo_stride, d.T_tot, d.HQ, d.D)) || (k && !rows_apart(d.ko_stride, d.T_tot, d.HKV, d.D)))
        return GDN2_ERR_ALIAS;
    if (!in_place_or_apart(oq, rq) || !in_place_or_apart(ok, rk) || overlap(oq, rk) || overlap(ok, rq) ||
        overlap(oq, ok))
        return GDN2_ERR_ALIAS;
    for (const Rows &o : {oq, ok})
        if (overlap(o, q_weight, d.D * 2) || overlap(o, k_weight, d.D * 2) || overlap(o, inv_freq, d.rot_dim * 4) ||
            overlap(o, positions, d.T_tot * (d.positions_i64 ? 8 : 4)))
            return GDN2_ERR_ALIAS;
    int dev = 0;
    if (!device_is_sm103(&dev)) return GDN2_ERR_ARCH;
    if (d.T_tot == 0) return GDN2_OK;
    RopeParams p;
    fill_rope(p, d, q, k, q_weight, k_weight, inv_freq, positions, q_out);
    p.k_out = static_cast<bf16 *>(k_out);
    cudaGetLastError();
    return launch_rope(p, d.D, d.dtype == GDN2_DTYPE_F16, d.rope_interleaved != 0, sm_count(dev),
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GDN2_OK
               : GDN2_ERR_LAUNCH;
}

size_t gdn2_kv_append_workspace_bytes(const gdn2_attn_dims *d) {
    return d && paged_shape_ok(*d) && check_rope(*d) == GDN2_OK ? kAppendWorkspaceBytes : 0;
}

gdn2_status gdn2_kv_append(const void *q, const void *k, const void *v, const void *q_weight, const void *k_weight,
                           const double *inv_freq, const void *positions, const void *cu_seqlens,
                           const int32_t *kv_lens, const int32_t *block_table, void *q_out, void *k_cache,
                           void *v_cache, const gdn2_attn_dims *dims, void *workspace, size_t workspace_bytes,
                           void *stream) {
    if (!dims) return GDN2_ERR_NULL;
    const gdn2_attn_dims &d = *dims;
    gdn2_status st = check_common(d);
    if (st == GDN2_OK) st = check_rope(d);
    if (st != GDN2_OK) return st;
    if (!paged_shape_ok(d) || (q && d.HQ < 1)) return GDN2_ERR_SHAPE;
    if (!workspace || !cu_seqlens || (d.N > 0 && (!kv_lens || (d.max_pages > 0 && !block_table))) || !q != !q_out)
        return GDN2_ERR_NULL;
    if (d.T_tot > 0 && (!k || !v || !k_cache || !v_cache || (d.rot_dim > 0 && !inv_freq)))
        return GDN2_ERR_NULL;
    if (!strides_ok(q, d.q_stride, 2) || !strides_ok(k, d.k_stride, 2) || !strides_ok(v, d.v_stride, 2) ||
        !strides_ok(q_out, d.qo_stride, 2) || !strides_ok(k_cache, d.kc_stride, 3) ||
        !strides_ok(v_cache, d.vc_stride, 3) || !aligned16(q_weight) || !aligned16(k_weight) ||
        !aligned16(inv_freq) || !aligned16(workspace))
        return GDN2_ERR_STRIDE;
    const Rows rq = rows(q, d.T_tot, d.HQ, d.D, d.q_stride), oq = rows(q_out, d.T_tot, d.HQ, d.D, d.qo_stride);
    const Rows rk = rows(k, d.T_tot, d.HKV, d.D, d.k_stride), rv = rows(v, d.T_tot, d.HKV, d.D, d.v_stride);
    const Rows kc = cache_rows(k_cache, d, d.kc_stride), vc = cache_rows(v_cache, d, d.vc_stride);
    if ((q && !rows_apart(d.qo_stride, d.T_tot, d.HQ, d.D)) || !slots_apart(d, d.kc_stride) ||
        !slots_apart(d, d.vc_stride) || (k_cache && k_cache == v_cache))
        return GDN2_ERR_ALIAS;
    if (!in_place_or_apart(oq, rq) || overlap(oq, rk) || overlap(oq, rv)) return GDN2_ERR_ALIAS;
    for (const Rows &o : {oq, kc, vc}) {
        if (overlap(o, q_weight, d.D * 2) || overlap(o, k_weight, d.D * 2) || overlap(o, inv_freq, d.rot_dim * 4) ||
            overlap(o, positions, d.T_tot * (d.positions_i64 ? 8 : 4)) ||
            overlap(o, cu_seqlens, (d.N + 1ll) * (d.cu_seqlens_i64 ? 8 : 4)) || overlap(o, kv_lens, d.N * 4ll) ||
            overlap(o, block_table, table_bytes(d)) || overlap(o, workspace, kAppendWorkspaceBytes))
            return GDN2_ERR_ALIAS;
    }
    for (const Rows &o : {kc, vc})
        if (overlap(o, rq) || overlap(o, rk) || overlap(o, rv) || overlap(o, oq)) return GDN2_ERR_ALIAS;
    if (workspace_bytes < kAppendWorkspaceBytes) return GDN2_ERR_WORKSPACE;
    int dev = 0;
    if (!device_is_sm103(&dev)) return GDN2_ERR_ARCH;
    RopeParams p;
    fill_rope(p, d, q, k, q_weight, k_weight, inv_freq, positions, q_out);
    p.v = static_cast<const bf16 *>(v);
    p.sv_t = d.v_stride[0]; p.sv_h = d.v_stride[1];
    p.HV = d.HKV;
    p.HK = d.HKV;
    p.k_cache = static_cast<bf16 *>(k_cache);
    p.v_cache = static_cast<bf16 *>(v_cache);
    for (int i = 0; i < 3; ++i) { p.skc[i] = d.kc_stride[i]; p.svc[i] = d.vc_stride[i]; }
    p.cu = cu_seqlens;
    p.cu64 = d.cu_seqlens_i64 ? 1 : 0;
    p.kv_lens = kv_lens;
    p.table = block_table;
    p.table_stride = d.table_stride;
    p.num_pages = d.num_pages;
    p.N = d.N;
    p.page_size = d.page_size;
    p.page = divisor(d.page_size);
    p.max_pages = d.max_pages;
    p.status = static_cast<int *>(workspace);
    cudaGetLastError();
    return launch_rope(p, d.D, d.dtype == GDN2_DTYPE_F16, d.rope_interleaved != 0, sm_count(dev),
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GDN2_OK
               : GDN2_ERR_LAUNCH;
}

size_t gdn2_paged_attn_workspace_bytes(const gdn2_attn_dims *d) {
    return d && attn_shape_ok(*d) ? paged_attn_workspace(*d) : 0;
}

gdn2_status gdn2_paged_attn_fwd(const void *q, const void *k_cache, const void *v_cache, const void *cu_seqlens,
                                const int32_t *kv_lens, const int32_t *block_table, float scale, void *out,
                                float *lse, const gdn2_attn_dims *dims, void *workspace, size_t workspace_bytes,
                                void *stream) {
    if (!dims) return GDN2_ERR_NULL;
    const gdn2_attn_dims &d = *dims;
    gdn2_status st = check_common(d);
    if (st != GDN2_OK) return st;
    if (!attn_shape_ok(d) || !isfinite(scale)) return GDN2_ERR_SHAPE;
    if (!workspace || !cu_seqlens || (d.N > 0 && (!kv_lens || (d.max_pages > 0 && !block_table))))
        return GDN2_ERR_NULL;
    if (d.T_tot > 0 && (!q || !out || !k_cache || !v_cache)) return GDN2_ERR_NULL;
    if (!strides_ok(q, d.q_stride, 2) || !strides_ok(out, d.qo_stride, 2) || !strides_ok(k_cache, d.kc_stride, 3) ||
        !strides_ok(v_cache, d.vc_stride, 3) || !mapped_strides_ok(d, d.kc_stride) || !mapped_strides_ok(d, d.vc_stride) ||
        !aligned16(workspace) || reinterpret_cast<uintptr_t>(lse) % 4)
        return GDN2_ERR_STRIDE;
    const Rows rq = rows(q, d.T_tot, d.HQ, d.D, d.q_stride), ro = rows(out, d.T_tot, d.HQ, d.D, d.qo_stride);
    const Rows kc = cache_rows(k_cache, d, d.kc_stride), vc = cache_rows(v_cache, d, d.vc_stride);
    if (out && !rows_apart(d.qo_stride, d.T_tot, d.HQ, d.D)) return GDN2_ERR_ALIAS;
    const int64_t lse_bytes = d.T_tot * d.HQ * 4;
    const Rows rl = {reinterpret_cast<uintptr_t>(lse), lse_bytes > 0 ? 1 : 0, 1, lse_bytes, 0, 0};
    const Rows ws = {reinterpret_cast<uintptr_t>(workspace), 1, 1, static_cast<int64_t>(workspace_bytes), 0, 0};
    for (const Rows &o : {ro, rl, ws}) {
        if (overlap(o, rq) || overlap(o, kc) || overlap(o, vc) ||
            overlap(o, cu_seqlens, (d.N + 1ll) * (d.cu_seqlens_i64 ? 8 : 4)) || overlap(o, kv_lens, d.N * 4ll) ||
            overlap(o, block_table, table_bytes(d)))
            return GDN2_ERR_ALIAS;
    }
    if (overlap(ro, rl) || overlap(ro, ws) || overlap(rl, ws)) return GDN2_ERR_ALIAS;
    if (workspace_bytes < paged_attn_workspace(d)) return GDN2_ERR_WORKSPACE;
    int dev = 0;
    if (!device_is_sm103(&dev)) return GDN2_ERR_ARCH;
    AttnParams p;
    memset(&p, 0, sizeof(p));
    p.q = static_cast<const bf16 *>(q);
    p.k_cache = static_cast<const bf16 *>(k_cache);
    p.v_cache = static_cast<const bf16 *>(v_cache);
    p.out = static_cast<bf16 *>(out);
    p.lse = lse;
    p.sq_t = d.q_stride[0]; p.sq_h = d.q_stride[1];
    p.so_t = d.qo_stride[0]; p.so_h = d.qo_stride[1];
    for (int i = 0; i < 3; ++i) { p.skc[i] = d.kc_stride[i]; p.svc[i] = d.vc_stride[i]; }
    p.cu = cu_seqlens;
    p.cu64 = d.cu_seqlens_i64 ? 1 : 0;
    p.kv_lens = kv_lens;
    p.table = block_table;
    p.table_stride = d.table_stride;
    p.num_pages = d.num_pages;
    p.T = d.T_tot;
    p.N = d.N; p.HQ = d.HQ; p.HKV = d.HKV; p.G = d.HQ / d.HKV;
    p.page_size = d.page_size;
    p.max_pages = d.max_pages;
    p.causal = d.causal;
    p.window = d.window_left;
    p.scale = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(d.D));
    p.status = static_cast<int *>(workspace);
    cudaGetLastError();
    return launch_paged_attn(p, d, sm_count(dev), workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GDN2_OK
               : GDN2_ERR_LAUNCH;
}

}  // extern "C"
