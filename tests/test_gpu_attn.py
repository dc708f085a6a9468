"""The attention-layer operators on the GPU against plain fp64 statements of
their definitions (tests/attn_reference.py).

Tolerances, fixed before the first run.  u = unit roundoff of the 16-bit type.
* norm and rotation: fp32 arithmetic (a few 2^-24 of the row's largest value,
  2^-21 for the sine and cosine) and one rounding: u |y| + 1e-5 max|row|.
* attention: the weights are rounded to 16 bits, then the output:
  u (sum p |v| + |o|); fp32 scores of |q||k| scale <= ~20 over 128 channels err
  by at most 128 * 2^-24 * 20 ~ 1.5e-4, the weights relatively by as much:
  + 2e-4 sum p |v|.  lse: 2e-4.
"""
import numpy as np
import pytest
import torch

from attn_reference import UNIT, attention, f64, norm_rope
from gated_deltanet_prefill_gb300 import attn

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=BF):
    return torch.randn(shape, device="cuda", generator=g).to(dtype)


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def close_rope(y, ref, what):
    y, u = f64(y), UNIT[str(y.dtype)]
    tol = u * np.abs(ref) + 1e-5 * np.abs(ref).max(-1, keepdims=True) + 1e-30
    worst = (np.abs(y - ref) / tol).max() if ref.size else 0.0
    assert worst <= 1.0, (what, worst)


# ------------------------------------------------------- norm and rotation
ROPE = [
    # T, HQ, HK, D, rot, interleaved, norm, weights, dtype, positions below
    (1, 1, 1, 64, 64, False, True, True, BF, 10),
    (1, 16, 16, 128, 128, False, True, True, BF, 4096),
    (3, 5, 2, 128, 128, True, True, True, FP, 1000),
    (37, 7, 3, 128, 64, False, True, False, BF, 131072),
    (70, 15, 5, 64, 32, True, False, False, FP, 32768),
    (129, 8, 1, 64, 16, False, False, False, BF, 100),
    (65, 1, 9, 128, 96, False, True, True, FP, 1 << 20),
    (33, 40, 8, 128, 112, True, True, True, BF, 1 << 30),
    (5, 4, 4, 128, 0, False, True, True, BF, 10),
    (600, 3, 3, 64, 48, False, True, True, BF, 50000),
]


@pytest.mark.parametrize("T,HQ,HK,D,rot,inter,norm,weights,dtype,top", ROPE)
def test_norm_rope(cuda_lib, T, HQ, HK, D, rot, inter, norm, weights, dtype, top):
    g = gen(T + rot)
    q, k = normal(g, T, HQ, D, dtype=dtype), normal(g, T, HK, D, dtype=dtype)
    w = [1 + normal(g, D, dtype=dtype) / 4 for _ in range(2)] if weights else [None, None]
    pos = torch.randint(0, top, (T,), device="cuda", generator=g, dtype=torch.int32)
    f, m = attn.rope_frequencies(rot, scaling="parts", factor=8.0, trained_len=4096) if rot else (None, 1.0)
    qo, ko = attn.qk_norm_rope(q, k, pos if rot else None, f, m, inter, norm, *w, eps=1e-5)
    for y, x, wt, what in ((qo, q, w[0], "q"), (ko, k, w[1], "k")):
        ref = norm_rope(f64(x), pos.tolist(), None if f is None else f.tolist(), None if wt is None else f64(wt),
                        norm, inter, m, 1e-5)
        close_rope(y, ref, what)


def test_norm_rope_int64_positions_of_any_size(cuda_lib):
    g = gen(5)
    pos = [0, 1, -1, -12345, 2 ** 31 - 1, 2 ** 31, 2 ** 40 + 12345, -(2 ** 50), 2 ** 62 + 1]
    q = normal(g, len(pos), 2, 64)
    f, _ = attn.rope_frequencies(64)
    y, none = attn.qk_norm_rope(q, None, ints(pos, torch.int64), f)
    assert none is None
    # the frequency's 64-bit fraction of a turn is off by up to 2^-54 turns
    ref = norm_rope(f64(q)[:6], pos[:6], f.tolist())
    close_rope(y[:6], ref, "positions to 2^31")
    ref = norm_rope(f64(q)[6:7], pos[6:7], f.tolist())
    tol = 2.0 ** -8 * np.abs(ref) + 2e-3 * np.abs(ref).max(-1, keepdims=True)  # 2^40 * 2 pi 2^-53
    assert (np.abs(f64(y[6:7]) - ref) <= tol).all()
    assert torch.isfinite(y.float()).all()


def test_norm_rope_frequencies_outside_the_usual(cuda_lib):
    """Zero, tiny and large angles per position."""
    g = gen(6)
    f = torch.tensor([0.0, 1e-30, 1e-9, 0.5, 3.0, 6.5, 100.0, 1e6], dtype=torch.float64, device="cuda")
    pos = [0, 1, 2, 77, 4095]
    q = normal(g, len(pos), 3, 64)
    for inter in (False, True):
        y, _ = attn.qk_norm_rope(q, None, ints(pos), f, interleaved=inter)
        close_rope(y, norm_rope(f64(q), pos, f.tolist(), interleaved=inter), "frequencies")


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_in_place_on_packed_views(cuda_lib, inter):
    g = gen(7)
    T, HQ, HK, D = 45, 6, 2, 128
    x = normal(g, T, HQ + 2 * HK + 1, D)
    before = x.clone()
    q, k = x[:, :HQ], x[:, HQ:HQ + HK]
    pos = torch.arange(T, device="cuda")
    f, _ = attn.rope_frequencies(64)
    want = attn.qk_norm_rope(q, k, pos, f, interleaved=inter)
    assert torch.equal(x, before)  # inputs are not written
    got = attn.qk_norm_rope(q, k, pos, f, interleaved=inter, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(x[:, HQ + HK:], before[:, HQ + HK:])
    close_rope(want[1], norm_rope(f64(before[:, HQ:HQ + HK]), range(T), f.tolist(), interleaved=inter), "packed")


def test_norm_rope_head_major_and_strided(cuda_lib):
    g = gen(8)
    T, H, D = 33, 5, 64
    q = normal(g, H, T, D).transpose(0, 1)
    out = torch.zeros(T, 2 * H, 2 * D, dtype=BF, device="cuda")[:, ::2, D:]
    f, _ = attn.rope_frequencies(64)
    attn.qk_norm_rope(q, None, ints(list(range(T))), f, q_out=out)
    close_rope(out, norm_rope(f64(q), range(T), f.tolist()), "strided")


def test_norm_rope_zero_row_and_nan_row(cuda_lib):
    """A zero row stays zero (eps), a NaN row stays alone."""
    g = gen(9)
    q = normal(g, 4, 3, 128)
    q[1, 1] = 0
    q[2, 0] = float("nan")
    f, _ = attn.rope_frequencies(128)
    y, _ = attn.qk_norm_rope(q, None, ints([3, 4, 5, 6]), f)
    assert (y[1, 1] == 0).all() and torch.isnan(y[2, 0]).all()
    assert torch.isfinite(y[2, 1:].float()).all() and torch.isfinite(y[[0, 1, 3]].float()).all()


# ------------------------------------------------------------- paged caches
class Cache:
    """Caches and tables for sequences with `past` cached and `new` new tokens; every slot is filled with `fill`."""

    def __init__(self, g, new, past, page, HKV, D, dtype=BF, layout="nhd", fill=None, cu_dtype=torch.int32, width=None):
        self.new, self.total = new, [n + p for n, p in zip(new, past)]
        counts = [-(-max(t, 0) // page) for t in self.total]
        pages = sum(counts) + 2
        order = torch.randperm(pages, device="cuda", generator=g).tolist()
        width = max([1] + counts) if width is None else width
        table = [[-7] * width for _ in new]  # entries out of reach are never used
        for n, c in enumerate(counts):
            for j in range(c):
                table[n][j] = order.pop()
        self.spare = order  # pages of no sequence
        self.table = ints(table).reshape(len(new), width)
        shape = (pages, HKV, page, D) if layout == "hnd" else (pages, page, HKV, D)
        self.k, self.v = normal(g, *shape, dtype=dtype), normal(g, *shape, dtype=dtype)
        if layout == "hnd":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.lens = ints(self.total)
        self.cu = ints(np.cumsum([0] + new).tolist(), cu_dtype)
        self.page = page
        if fill is not None:  # everything that no sequence holds
            held = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
            for n, t in enumerate(self.total):
                for j in range(t):
                    held[table[n][j // page], j % page] = True
            self.k[~held] = fill
            self.v[~held] = fill

    def args(self):
        return self.k, self.v, self.table, self.lens, self.cu


APPEND = [
    # new, past, page, HQ, HKV, D, rot, interleaved, norm, dtype, layout
    ([1], [0], 16, 4, 1, 64, 64, False, True, BF, "nhd"),
    ([1] * 40, list(range(0, 400, 10)), 64, 8, 2, 128, 128, False, True, BF, "nhd"),
    ([0, 5, 0, 130, 1, 0], [3, 60, 0, 17, 15, 16], 16, 6, 3, 128, 64, True, True, FP, "hnd"),
    ([33, 7, 64], [0, 1, 127], 8, 5, 5, 64, 32, False, False, BF, "hnd"),
    ([100, 300], [0, 999], 40, 0, 4, 64, 48, True, True, FP, "nhd"),
    ([257], [511], 256, 12, 4, 128, 0, False, True, BF, "nhd"),
]


@pytest.mark.parametrize("new,past,page,HQ,HKV,D,rot,inter,norm,dtype,layout", APPEND)
def test_append(cuda_lib, new, past, page, HQ, HKV, D, rot, inter, norm, dtype, layout):
    g = gen(sum(new) + page)
    c = Cache(g, new, past, page, HKV, D, dtype, layout, cu_dtype=torch.int64 if page == 16 else torch.int32)
    T = sum(new)
    q = normal(g, T, HQ, D, dtype=dtype) if HQ else None
    x = normal(g, T, 2 * HKV, D, dtype=dtype)
    k, v = x[:, :HKV], x[:, HKV:]
    w = [1 + normal(g, D, dtype=dtype) / 4 for _ in range(2)] if norm else [None, None]
    if not HQ:
        w[0] = None
    f, m = attn.rope_frequencies(rot, scaling="linear", factor=2.0) if rot else (None, 1.0)
    k0, v0 = c.k.clone(), c.v.clone()
    ws = torch.full((64,), 255, dtype=torch.uint8, device="cuda")
    qo = attn.append_kv(k, v, *c.args(), q=q, inv_freq=f, rope_factor=m, interleaved=inter, norm=norm, q_weight=w[0],
                        k_weight=w[1], workspace=ws)
    assert attn.device_status(ws) == 0
    places = [p + j for n, p in zip(new, past) for j in range(n)]
    seqs = [i for i, n in enumerate(new) for _ in range(n)]
    table = c.table.tolist()
    pages, slots = [table[s][p // page] for s, p in zip(seqs, places)], [p % page for p in places]
    freqs = None if f is None else f.tolist()
    ref = norm_rope(f64(k), places, freqs, None if w[1] is None else f64(w[1]), norm, inter, m)
    close_rope(c.k[pages, slots], ref, "k")
    assert torch.equal(c.v[pages, slots], v)
    k0[pages, slots], v0[pages, slots] = c.k[pages, slots], c.v[pages, slots]
    assert torch.equal(c.k, k0) and torch.equal(c.v, v0)  # the other slots are as they were
    if HQ:
        close_rope(qo, norm_rope(f64(q), places, freqs, None if w[0] is None else f64(w[0]), norm, inter, m), "q")
        want = qo.clone()  # the same call with q in place, explicit positions
        attn.append_kv(k, v, *c.args(), q=q, positions=ints(places, torch.int64), inv_freq=f, rope_factor=m,
                       interleaved=inter, norm=norm, q_weight=w[0], k_weight=w[1], q_out=q)
        assert torch.equal(q, want) and torch.equal(c.k, k0)
    else:
        assert qo is None


def test_append_positions_apart_from_places(cuda_lib):
    g = gen(11)
    c = Cache(g, [9, 3], [4, 0], 16, 2, 64)
    k, v = normal(g, 12, 2, 64), normal(g, 12, 2, 64)
    pos = [1000 + 3 * i for i in range(12)]
    f, _ = attn.rope_frequencies(64)
    attn.append_kv(k, v, *c.args(), positions=ints(pos), inv_freq=f)
    t = c.table.tolist()
    at = [t[0][0]] * 9 + [t[1][0]] * 3, list(range(4, 13)) + [0, 1, 2]
    close_rope(c.k[at], norm_rope(f64(k), pos, f.tolist()), "k")


def test_append_reports_and_leaves_out_what_has_no_page(cuda_lib):
    """Bad places and table entries: reported, nothing written for them, the others in place."""
    g = gen(12)
    page = 16
    for what in ("entry low", "entry high", "length past the table", "negative place"):
        c = Cache(g, [4, 4, 4], [14, 30, 0], page, 2, 64, width=3)
        if what == "entry low":
            c.table[1, 2] = -1
        elif what == "entry high":
            c.table[1, 2] = c.k.shape[0]
        elif what == "length past the table":
            c.lens[1] = 3 * page + 2
            c.table[1] = ints(c.spare + [c.spare[0]])[:3]
        else:
            c.lens[1] = 2
        k, v = normal(g, 12, 2, 64), normal(g, 12, 2, 64)
        k0, v0 = c.k.clone(), c.v.clone()
        ws = torch.zeros(64, dtype=torch.uint8, device="cuda")
        attn.append_kv(k, v, *c.args(), norm=False, workspace=ws)
        assert attn.device_status(ws) == 16, what
        t = c.table.tolist()
        ok = {"entry low": [30, 31], "entry high": [30, 31], "length past the table": [46, 47],
              "negative place": [0, 1]}[what]
        first = {"negative place": 2}.get(what, 0)  # the first of sequence 1's new tokens that has a place
        for n, toks, places in ((0, range(0, 4), range(14, 18)), (2, range(8, 12), range(0, 4)),
                                (1, range(4 + first, 4 + first + 2), ok)):
            for tok, p in zip(toks, places):
                k0[t[n][p // page], p % page], v0[t[n][p // page], p % page] = k[tok], v[tok]
        assert torch.equal(c.k, k0) and torch.equal(c.v, v0), what
        attn.append_kv(k, v, *Cache(g, [4, 4, 4], [14, 30, 0], page, 2, 64).args(), norm=False, workspace=ws)
        assert attn.device_status(ws) == 0  # the next call on the workspace starts afresh


@pytest.mark.parametrize("cu", [[1, 4, 8], [0, 5, 4], [0, 4, 9], [0, 4, 7]])
def test_bad_cu_seqlens_reported(cuda_lib, cu):
    g = gen(13)
    c = Cache(g, [4, 4], [14, 30], 16, 2, 64)
    c.cu = ints(cu)
    ws = torch.zeros(64, dtype=torch.uint8, device="cuda")
    attn.append_kv(normal(g, 8, 2, 64), normal(g, 8, 2, 64), *c.args(), norm=False, workspace=ws)
    assert attn.device_status(ws) == 9
    out = torch.full((8, 4, 64), 3.0, dtype=BF, device="cuda")
    ws = None
    q = normal(g, 8, 4, 64)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    attn.paged_attn_fwd(q, *c.args(), out=out, workspace=ws)
    assert attn.device_status(ws) == 9 and (out == 3.0).all()


# ---------------------------------------------------------------- attention
def check_attn(q, c, out, lse, causal=True, window=-1, scale=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    table, held = c.table.cpu().numpy(), c.lens.tolist()
    k, v = np.nan_to_num(f64(c.k)), np.nan_to_num(f64(c.v))
    ref, z, spread = attention(f64(q), k, v, table, held, c.cu.tolist(), scale, causal, window)
    u = UNIT[str(q.dtype)]
    tol = u * (spread + np.abs(ref)) + 2e-4 * spread + 1e-30
    worst = (np.abs(f64(out) - ref) / tol).max() if ref.size else 0.0
    assert worst <= 1.0, worst
    if lse is not None:
        x = f64(lse)
        assert (np.isneginf(x) == np.isneginf(z)).all()
        fin = np.isfinite(z)
        assert np.isfinite(x[fin]).all() and (np.abs(x[fin] - z[fin]) <= 2e-4).all()


ATTN = [
    # new, past, page, HQ, HKV, D, causal, window, dtype, layout
    ([1], [0], 16, 1, 1, 64, True, -1, BF, "nhd"),
    ([1], [776], 64, 16, 4, 128, True, -1, BF, "nhd"),
    ([1], [5000], 64, 2, 1, 128, True, -1, FP, "nhd"),
    ([1] * 9, [0, 1, 15, 16, 127, 128, 129, 300, 1000], 16, 8, 2, 128, True, -1, BF, "nhd"),
    ([0, 1, 0, 2, 0], [5, 0, 0, 7, 200], 8, 4, 4, 64, True, -1, FP, "hnd"),
    ([128], [0], 128, 2, 2, 128, True, -1, BF, "nhd"),
    ([129, 127], [0, 128], 64, 4, 2, 128, True, -1, BF, "hnd"),
    ([256], [256], 256, 1, 1, 128, False, -1, BF, "nhd"),
    ([300, 17, 1], [0, 500, 900], 48, 6, 2, 64, True, -1, FP, "nhd"),
    ([70, 200], [90, 11], 40, 5, 1, 128, False, -1, FP, "hnd"),
    ([50, 1, 300], [300, 400, 0], 16, 12, 4, 64, True, 60, FP, "nhd"),
    ([200], [700], 64, 3, 1, 128, True, 0, BF, "nhd"),
    ([40, 1, 1], [1000, 1100, 0], 32, 16, 1, 128, True, 127, BF, "hnd"),
    ([5, 9], [300, 2], 24, 128, 1, 64, True, -1, BF, "nhd"),
    ([3, 1], [40, 600], 56, 100, 1, 128, True, -1, BF, "nhd"),
    ([20, 1], [256, 129], 72, 40, 8, 128, True, 200, FP, "nhd"),
    # several items per CTA: many sequences, whole and cut
    ([1] * 300, [(37 * i) % 400 for i in range(300)], 16, 4, 2, 64, True, -1, BF, "nhd"),
    ([1, 2, 0] * 60, [(91 * i) % 700 for i in range(180)], 64, 8, 4, 128, True, -1, BF, "hnd"),
    ([140, 1, 300] * 10, [(57 * i) % 300 for i in range(30)], 32, 8, 8, 128, True, -1, FP, "nhd"),
]


@pytest.mark.parametrize("new,past,page,HQ,HKV,D,causal,window,dtype,layout", ATTN)
def test_attention(cuda_lib, new, past, page, HQ, HKV, D, causal, window, dtype, layout):
    g = gen(sum(new) + sum(past) + page)
    c = Cache(g, new, past, page, HKV, D, dtype, layout, fill=float("nan"),
              cu_dtype=torch.int64 if page == 16 else torch.int32)
    q = normal(g, sum(new), HQ, D, dtype=dtype)
    out, lse = attn.paged_attn_fwd(q, *c.args(), causal=causal, window_left=window, return_lse=True)
    check_attn(q, c, out, lse, causal, window)
    assert torch.equal(out, attn.paged_attn_fwd(q, *c.args(), causal=causal, window_left=window))  # repeatable


def test_attention_scale_and_growing_scores(cuda_lib):
    """Scores that grow along the keys (the running maximum moves at every tile), a large and a small scale."""
    g = gen(21)
    c = Cache(g, [3, 130], [900, 500], 32, 2, 128, fill=float("inf"))
    ramp = torch.linspace(0.0, 3.0, 1024, device="cuda")
    for n, t in enumerate(c.total):
        for j in range(t):
            row = c.k[c.table[n, j // 32], j % 32]
            row.copy_((row.float() * 0.1 + ramp[j] / 4).to(BF))
    q = (normal(g, 133, 4, 128).float() * 0.2 + 0.5).to(BF)
    for scale in (0.5, 1e-3, 0.088):
        out, lse = attn.paged_attn_fwd(q, *c.args(), scale=scale, return_lse=True)
        # scores to 0.5 * 128 * 0.5 * 0.75 = 24: within the tolerance's assumption on |q||k|
        check_attn(q, c, out, lse, scale=scale)


def test_attention_rows_without_keys(cuda_lib):
    """kv_lens below the new tokens: the first rows have no key; a length of zero: none has."""
    g = gen(22)
    c = Cache(g, [10, 4, 200, 3], [0, 0, 0, 0], 16, 2, 128, fill=float("nan"))
    c.lens.copy_(ints([6, 0, 150, 3]))
    q = normal(g, 217, 4, 128)
    out, lse = attn.paged_attn_fwd(q, *c.args(), return_lse=True)
    check_attn(q, c, out, lse)
    assert (out[:4] == 0).all() and (out[10:14] == 0).all() and torch.isneginf(lse[10:14]).all()
    assert torch.isneginf(lse[14:64]).all() and torch.isfinite(lse[64:]).all()


def test_attention_strides(cuda_lib):
    """q and out as views, k and v pages interleaved in one allocation, a table with a row stride."""
    g = gen(23)
    c = Cache(g, [30, 1, 90], [100, 300, 0], 16, 2, 64)
    both = torch.empty(c.k.shape[0], 2, 16, 2, 64, dtype=BF, device="cuda")
    both[:, 0], both[:, 1] = c.k, c.v
    c.k, c.v = both[:, 0], both[:, 1]
    wide = torch.full((3, c.table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide[:, :c.table.shape[1]]
    q = normal(g, 6, 121, 64).transpose(0, 1)
    out = torch.zeros(121, 12, 128, dtype=BF, device="cuda")
    o, lse = attn.paged_attn_fwd(q, *c.args(), out=out[:, ::2, 64:], return_lse=True)
    check_attn(q, c, o, lse)
    assert (out[:, 1::2] == 0).all() and (out[:, :, :64] == 0).all()


def test_attention_offsets_past_32_bits(cuda_lib):
    """Pages more than 2^31 elements apart."""
    g = gen(24)
    small = Cache(g, [4, 1], [60, 20], 32, 1, 128)
    step = 1 << 30
    pages = small.k.shape[0]
    far = torch.empty((pages - 1) * step + 2 * 32 * 128, dtype=BF, device="cuda")
    k = far.as_strided((pages, 32, 1, 128), (step, 128, 128, 1))
    v = far[32 * 128:].as_strided((pages, 32, 1, 128), (step, 128, 128, 1))
    k.copy_(small.k)
    v.copy_(small.v)
    q = normal(g, 5, 4, 128)
    want, wl = attn.paged_attn_fwd(q, *small.args(), return_lse=True)
    got, gl = attn.paged_attn_fwd(q, k, v, *small.args()[2:], return_lse=True)
    assert torch.equal(want, got) and torch.equal(wl, gl)
    nk, nv = normal(g, 5, 1, 128), normal(g, 5, 1, 128)
    attn.append_kv(nk, nv, *small.args(), norm=False)
    attn.append_kv(nk, nv, k, v, *small.args()[2:], norm=False)
    assert torch.equal(k, small.k) and torch.equal(v, small.v)


def test_attention_reports_bad_lengths_and_entries(cuda_lib):
    g = gen(25)
    for what in ("low", "high", "entry"):
        c = Cache(g, [2, 2], [14, 100], 16, 2, 64)
        if what == "entry":
            c.table[1, 3] = c.k.shape[0] + 5
        else:
            c.lens[1] = -1 if what == "low" else c.table.shape[1] * 16 + 1
        q = normal(g, 4, 2, 64)
        out = torch.full((4, 2, 64), 3.0, dtype=BF, device="cuda")
        ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
        attn.paged_attn_fwd(q, *c.args(), out=out, workspace=ws)
        assert attn.device_status(ws) == 16, what
        if what != "entry":
            assert (out == 3.0).all()
        c = Cache(g, [2, 2], [14, 100], 16, 2, 64)
        out, lse = attn.paged_attn_fwd(q, *c.args(), out=out, workspace=ws, return_lse=True)
        assert attn.device_status(ws) == 0
        check_attn(q, c, out, lse)


def test_no_tokens(cuda_lib):
    g = gen(26)
    c = Cache(g, [0, 0], [14, 100], 16, 2, 64)
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
    empty = normal(g, 0, 2, 64)
    assert attn.qk_norm_rope(empty, empty, norm=True)[0].shape == (0, 2, 64)
    attn.append_kv(empty, empty, *c.args(), workspace=ws)
    assert attn.device_status(ws) == 0
    ws.fill_(255)
    assert attn.paged_attn_fwd(empty, *c.args(), workspace=ws).shape == (0, 2, 64)
    assert attn.device_status(ws) == 0


def test_side_stream_and_graph(cuda_lib):
    """A layer's calls on a side stream, captured once and replayed on new contents."""
    g = gen(27)
    c = Cache(g, [1, 40, 1], [70, 0, 130], 16, 2, 128)
    q, k, v = normal(g, 42, 8, 128), normal(g, 42, 2, 128), normal(g, 42, 2, 128)
    f, _ = attn.rope_frequencies(128)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    aws = torch.empty(64, dtype=torch.uint8, device="cuda")
    qo, out = torch.empty_like(q), torch.empty_like(q)

    def layer():
        attn.append_kv(k, v, *c.args(), q=q, inv_freq=f, q_out=qo, workspace=aws)
        attn.paged_attn_fwd(qo, *c.args(), out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.synchronize()
    check_attn(qo, c, out, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in (1, 2):
        h = gen(seed)
        q.copy_(normal(h, 42, 8, 128))
        k.copy_(normal(h, 42, 2, 128))
        c.lens.copy_(ints([71 - seed, 40, 131 - 20 * seed]))
        graph.replay()
        torch.cuda.synchronize()
        check_attn(qo, c, out, None)


def test_chunks_then_tokens_equal_one_pass(cuda_lib):
    """Appending and attending in chunks, then token by token, gives each token what one call over all gives."""
    g = gen(28)
    lens = [150, 91]
    c = Cache(g, lens, [0, 0], 16, 2, 64, dtype=FP)
    T = sum(lens)
    q, k, v = normal(g, T, 6, 64, dtype=FP), normal(g, T, 2, 64, dtype=FP), normal(g, T, 2, 64, dtype=FP)
    f, _ = attn.rope_frequencies(64)
    qo = attn.append_kv(k, v, *c.args(), q=q, inv_freq=f)
    whole, wl = attn.paged_attn_fwd(qo, *c.args(), return_lse=True)
    check_attn(qo, c, whole, wl)
    again = Cache(gen(29), lens, [0, 0], 16, 2, 64, dtype=FP)
    again.k.fill_(float("nan"))
    again.v.fill_(float("nan"))
    done = [0, 0]
    for step in ([64, 30], [60, 59], [25, 1], [1, 1]):
        rows = torch.cat([torch.arange(150 * n + done[n], 150 * n + done[n] + step[n]) for n in range(2)]).cuda()
        done = [a + b for a, b in zip(done, step)]
        args = again.k, again.v, again.table, ints(done), ints([0, step[0], sum(step)])
        part_q = attn.append_kv(k[rows], v[rows], *args, q=q[rows], inv_freq=f)
        assert torch.equal(part_q, qo[rows])
        part, pl = attn.paged_attn_fwd(part_q, *args, return_lse=True)
        bound = 2 * UNIT["torch.float16"] * 4 + 1e-3  # both roundings of values up to 4
        assert (part.float() - whole[rows].float()).abs().max() <= bound
        assert (pl - wl[rows]).abs().max() <= 4e-4


def drop_before_window(c, window, value=float("nan")):
    """What lies before the window of each sequence's first new token: slots overwritten, pages out of the table."""
    for n, (new, total) in enumerate(zip(c.new, c.total)):
        gone = max(0, total - new - window) if new else total
        for j in range(gone):
            page = c.table[n, j // c.page]
            c.k[page, j % c.page], c.v[page, j % c.page] = value, value
        c.table[n, :gone // c.page] = -1


@pytest.mark.parametrize("new,past,page,HQ,HKV,D,window", [
    ([1], [1000], 16, 4, 2, 128, 100),
    ([1, 1, 1], [129, 640, 3000], 8, 2, 1, 64, 127),
    ([30, 2], [900, 70], 64, 4, 1, 128, 0),
    ([300], [700], 24, 8, 2, 64, 333),
    ([5, 7], [513, 511], 256, 6, 2, 128, 200),
])
def test_attention_pages_before_the_window_may_be_gone(cuda_lib, new, past, page, HQ, HKV, D, window):
    g = gen(31)
    c = Cache(g, new, past, page, HKV, D, fill=float("nan"))
    table = c.table.clone()
    drop_before_window(c, window)
    q = normal(g, sum(new), HQ, D)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    out, lse = attn.paged_attn_fwd(q, *c.args(), window_left=window, return_lse=True, workspace=ws)
    assert attn.device_status(ws) == 0
    c.table = table  # the reference's gather reads the slots that the mask then leaves out
    check_attn(q, c, out, lse, window=window)


def test_attention_widest_windows(cuda_lib):
    """Windows up to the largest integer, rows without a key among them: as without a window."""
    g = gen(32)
    c = Cache(g, [40, 9, 300], [100, 0, 0], 16, 2, 64)
    c.lens.copy_(ints([140, 4, 170]))
    q = normal(g, 349, 4, 64)
    want, wl = attn.paged_attn_fwd(q, *c.args(), return_lse=True)
    check_attn(q, c, want, wl)
    for window in (140, 2 ** 31 - 2, 2 ** 31 - 1):
        out, lse = attn.paged_attn_fwd(q, *c.args(), return_lse=True, window_left=window)
        check_attn(q, c, out, lse, window=window)


LONG = [
    # sequences past one round of the shares' sum, and items past one warp's
    ([1] * 500 + [2] * 300 + [0] * 7, [(53 * i) % 260 for i in range(807)], 16, 2, 1, 64, True, -1),
    ([3, 0, 1, 40] * 250, [(17 * i) % 90 for i in range(1000)], 8, 8, 2, 128, True, 31),
    ([1300], [0], 64, 8, 1, 64, True, -1),
    ([1100, 700, 5], [77, 1, 300], 32, 16, 1, 64, True, -1),
    ([1500], [40], 16, 8, 1, 64, True, 150),
    ([1111], [200], 16, 8, 1, 64, False, -1),
    ([20, 600, 1], [128, 500, 90], 40, 32, 1, 128, True, -1),
]


@pytest.mark.parametrize("new,past,page,HQ,HKV,D,causal,window", LONG)
def test_attention_many_sequences_and_items(cuda_lib, new, past, page, HQ, HKV, D, causal, window):
    g = gen(len(new) + sum(new))
    c = Cache(g, new, past, page, HKV, D, fill=float("nan"))
    q = normal(g, sum(new), HQ, D)
    out, lse = attn.paged_attn_fwd(q, *c.args(), causal=causal, window_left=window, return_lse=True)
    check_attn(q, c, out, lse, causal, window)


def test_attention_long_sequence_with_rows_without_keys(cuda_lib):
    """More new tokens than cached ones in a sequence of many items."""
    g = gen(33)
    c = Cache(g, [1200, 3], [0, 50], 16, 1, 64)
    c.lens.copy_(ints([700, 53]))
    q = normal(g, 1203, 8, 64)
    out, lse = attn.paged_attn_fwd(q, *c.args(), return_lse=True)
    check_attn(q, c, out, lse)
    assert (out[:500] == 0).all() and torch.isneginf(lse[:500]).all()


def test_attention_broadcast_queries(cuda_lib):
    """Queries expanded over heads or tokens (zero strides) equal their copies."""
    g = gen(34)
    c = Cache(g, [7, 150, 1], [20, 0, 400], 16, 2, 128)
    for q in (normal(g, 158, 1, 128).expand(158, 6, 128), normal(g, 1, 6, 128).expand(158, 6, 128)):
        out, lse = attn.paged_attn_fwd(q, *c.args(), return_lse=True)
        want, wl = attn.paged_attn_fwd(q.contiguous(), *c.args(), return_lse=True)
        assert torch.equal(out, want) and torch.equal(lse, wl)
        check_attn(q, c, out, lse)


def test_nothing_is_written_past_the_buffers(cuda_lib):
    """Outputs and workspaces of exactly the stated size between canaries; a used workspace changes no result."""
    g = gen(35)
    guard = 4096

    def fenced(n):
        buf = torch.full((n + 2 * guard,), 0x5A, dtype=torch.uint8, device="cuda")
        return buf, buf[guard:guard + n]

    buffers = []
    for new, past, HQ, HKV, D in (([1] * 5, [0, 9, 500, 900, 17], 8, 2, 128), ([200, 3], [0, 700], 4, 4, 64),
                                  ([1], [4000], 2, 1, 64)):
        c = Cache(g, new, past, 16, HKV, D)
        T = sum(new)
        q, k, v = normal(g, T, HQ, D), normal(g, T, HKV, D), normal(g, T, HKV, D)
        f, _ = attn.rope_frequencies(D)
        size = T * HQ * D * 2
        qo, out, lse, aws = fenced(size), fenced(size), fenced(T * HQ * 4), fenced(64)
        dims = attn.AttnDims()
        assert attn.load().gdn2_attn_dims_init(dims, T, len(new), HQ, HKV, D, c.k.shape[0], 16, c.table.shape[1]) == 0
        ws = fenced(attn.load().gdn2_paged_attn_workspace_bytes(dims))
        view = lambda b: b[1].view(BF).view(T, HQ, D)  # noqa: E731
        attn.append_kv(k, v, *c.args(), q=q, inv_freq=f, q_out=view(qo), workspace=aws[1])
        first = None
        for fill in (0, 255, None):
            if fill is not None:
                ws[1].fill_(fill)
            out[1].fill_(0x33)
            attn.paged_attn_fwd(view(qo), *c.args(), out=view(out), lse=lse[1].view(torch.float32), workspace=ws[1])
            assert attn.device_status(ws[1]) == 0 and attn.device_status(aws[1]) == 0
            first = view(out).clone() if first is None else first
            assert torch.equal(first, view(out))
        check_attn(view(qo), c, view(out), lse[1].view(torch.float32).view(T, HQ))
        buffers += [qo[0], out[0], lse[0], aws[0], ws[0]]
    for b in buffers:
        assert (b[:guard] == 0x5A).all() and (b[-guard:] == 0x5A).all()


def test_calls_of_many_shapes_and_layouts(cuda_lib):
    """More sets of metadata than are kept, repeats among them, and the same shapes in other layouts and dtypes."""
    g = gen(41)
    f, _ = attn.rope_frequencies(64)
    q = normal(g, 600, 2, 64)
    pos = torch.arange(600, device="cuda", dtype=torch.int32)
    want, _ = attn.qk_norm_rope(q, None, pos, f)
    for t in list(range(1, 600)) + [5, 599, 5]:
        y, none = attn.qk_norm_rope(q[:t], None, pos[:t], f)
        assert none is None and y.shape == (t, 2, 64) and y.is_contiguous() and torch.equal(y, want[:t])
    for other in (q.transpose(0, 1).contiguous().transpose(0, 1), q.half(), torch.nn.Parameter(q), q[::2]):
        n = other.shape[0]
        for p in (pos[:n], pos[:n].long()):
            y, _ = attn.qk_norm_rope(other, None, p, f)
            assert y.dtype == other.dtype
            close_rope(y, norm_rope(f64(other), p.tolist(), f.tolist()), "layout")
    y, _ = attn.qk_norm_rope(q[:9], None, pos[:9], f, interleaved=True, eps=1e-2, rope_factor=2)
    close_rope(y, norm_rope(f64(q[:9]), range(9), f.tolist(), None, True, True, 2.0, 1e-2), "options")


def test_refusals_of_known_and_unknown_calls(cuda_lib):
    from gated_deltanet_prefill_gb300.gdn2 import Gdn2Error
    g = gen(42)
    c = Cache(g, [4, 4], [14, 30], 16, 2, 64)
    q, k, v = normal(g, 8, 4, 64), normal(g, 8, 2, 64), normal(g, 8, 2, 64)
    f, _ = attn.rope_frequencies(64)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    for _ in range(2):  # the second time the metadata are known
        attn.paged_attn_fwd(q, *c.args(), workspace=ws)
        attn.append_kv(k, v, *c.args(), norm=False, workspace=ws)
        for status, call in (
                (8, lambda: attn.qk_norm_rope(q.float(), None)),
                (2, lambda: attn.qk_norm_rope(q[..., :32].contiguous(), None)),
                (4, lambda: attn.qk_norm_rope(q, None, q_out=torch.as_strided(q, (8, 4, 64), (0, 64, 1)))),
                (5, lambda: attn.append_kv(k, v, *c.args(), workspace=ws[:32])),
                (4, lambda: attn.append_kv(k, v, c.k, c.k, *c.args()[2:])),
                (5, lambda: attn.paged_attn_fwd(q, *c.args(), workspace=ws[:64])),
                (4, lambda: attn.paged_attn_fwd(q, *c.args(), out=q)),
                (2, lambda: attn.paged_attn_fwd(q[:, :3], *c.args())),
                (2, lambda: attn.paged_attn_fwd(q, *c.args(), causal=False, window_left=3))):
            with pytest.raises(Gdn2Error) as e:
                call()
            assert e.value.status == status
        for call in (lambda: attn.qk_norm_rope(q, k[:3]), lambda: attn.qk_norm_rope(q, None, None, f),
                     lambda: attn.qk_norm_rope(q, None, torch.arange(8), f), lambda: attn.qk_norm_rope(q.cpu(), None),
                     lambda: attn.qk_norm_rope(q, None, norm=False, q_weight=q[0, 0]),
                     lambda: attn.append_kv(k, v, c.k, c.v, c.table, c.lens[:1], c.cu),
                     lambda: attn.append_kv(k, v[:, :1], *c.args()),
                     lambda: attn.paged_attn_fwd(q, c.k, c.v, c.table.long(), c.lens, c.cu),
                     lambda: attn.paged_attn_fwd(q, c.k, c.v[:, :8], c.table, c.lens, c.cu)):
            with pytest.raises(ValueError):
                call()
        with pytest.raises((TypeError, AttributeError)):
            attn.qk_norm_rope([1.0], None)
        with pytest.raises(TypeError):
            attn.qk_norm_rope(q, None, eps="small")


def test_call_on_a_stream_other_than_the_current_one(cuda_lib):
    """Memory made for a call on a given stream is not handed out while that stream still waits."""
    g = gen(43)
    c = Cache(g, [1, 40, 1], [70, 0, 130], 16, 2, 128)
    q, k, v = normal(g, 42, 8, 128), normal(g, 42, 2, 128), normal(g, 42, 2, 128)
    f, _ = attn.rope_frequencies(128)
    qo = attn.append_kv(k, v, *c.args(), q=q, inv_freq=f)
    want, wl = attn.paged_attn_fwd(qo, *c.args(), return_lse=True)
    size = attn.load().gdn2_paged_attn_workspace_bytes
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    out, lse = attn.paged_attn_fwd(qo, *c.args(), return_lse=True, stream=side.cuda_stream)
    x, _ = attn.qk_norm_rope(q, None, norm=False, stream=side.cuda_stream)
    dims = attn._attn_dims(qo, *c.args(), None, None, True, -1)
    blocks = [torch.full((size(dims),), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl) and torch.equal(x, q)
    assert all((b == 255).all() for b in blocks)


def test_attention_smallest_scale(cuda_lib):
    """A scale near the smallest normal number: every key weighs the same."""
    g = gen(44)
    c = Cache(g, [2, 70], [300, 60], 16, 2, 64)
    q = normal(g, 72, 4, 64)
    for scale in (2e-38, 1e-30):
        out, lse = attn.paged_attn_fwd(q, *c.args(), scale=scale, return_lse=True)
        check_attn(q, c, out, lse, scale=scale)
    out, lse = attn.paged_attn_fwd(q, *c.args(), scale=2e-38, window_left=3, return_lse=True)
    check_attn(q, c, out, lse, scale=2e-38, window=3)
