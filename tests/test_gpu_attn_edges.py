"""The attention-layer operators on the GPU where the values, not the shapes,
are the hard part: scores far apart, infinite weights, a C caller's arguments.
"""
import numpy as np
import pytest
import torch

from attn_reference import UNIT, attention, f64
from gated_deltanet_prefill_gb300 import attn
from test_gpu_attn import BF, FP, Cache, gen, ints, normal

pytestmark = pytest.mark.gpu


def loud_keys(c, q, keys, gap):
    """Channel 0 of q and the cache so that the given keys of every sequence score `gap` above the others, which score
    within +-1; their values are zero, the others' lie around 1."""
    D = q.shape[-1]
    q.mul_(0.25)
    q[..., 0] = 8.0
    c.k.mul_(0.25)
    c.k[..., 0] = 0.0
    c.v.mul_(0.25).add_(1.0)
    for n, total in enumerate(c.total):
        for key in keys:
            if key < total:
                at = int(c.table[n, key // c.page]), key % c.page
                c.k[at][..., 0] = gap * D ** 0.5 / 8.0
                c.v[at] = 0.0


LOUD = [
    # new, past, page, HQ, HKV, D, causal, window, loud keys
    ([1], [20000], 64, 4, 1, 128, True, -1, [0]),
    ([1, 1], [3000, 700], 16, 4, 2, 64, True, -1, [5]),
    ([1], [8000], 64, 4, 1, 128, True, -1, [3000, 3001]),
    ([1], [6000], 32, 8, 1, 64, True, -1, [0, 300, 3000, 5900]),
    ([300], [700], 16, 2, 1, 128, True, -1, [0]),
    ([300], [400], 64, 2, 2, 64, True, -1, [130, 500]),
    ([200], [500], 16, 2, 1, 128, True, 300, list(range(0, 700, 100))),
    ([260], [100], 64, 2, 1, 64, False, -1, [359]),
]


@pytest.mark.parametrize("gap", [14.0, 17.4, 24.0, 80.0])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("new,past,page,HQ,HKV,D,causal,window,keys", LOUD)
def test_attention_beside_keys_far_above_the_rest(cuda_lib, new, past, page, HQ, HKV, D, causal, window, keys, dtype, gap):
    """A few keys whose values are zero take nearly all of the weight; the output is what the many others leave.

    Tolerance: that of the other attention tests, u (spread + |out|) + 2e-4 spread, where spread holds the quiet
    keys only, and so follows their small weights.  An fp16 output below 2^-14 is rounded to multiples of 2^-24: + 2^-25.  A weight
    may be held to 2^-36 of the largest among the 128 keys of its tile instead of to u of itself (fp16 has no
    exponents below that beside it); 128 of them with values below 2: + 2^-28.  The loud scores, gap, exceed the 20
    for which 2e-4 (lse's bound too) was derived by gap / 20.
    """
    g = gen(sum(past) + page)
    c = Cache(g, new, past, page, HKV, D, dtype)
    q = normal(g, sum(new), HQ, D, dtype=dtype)
    loud_keys(c, q, keys, gap)
    out, lse = attn.paged_attn_fwd(q, *c.args(), causal=causal, window_left=window, return_lse=True)
    ref, z, spread = attention(f64(q), f64(c.k), f64(c.v), c.table.cpu().numpy(), c.lens.tolist(), c.cu.tolist(), D ** -0.5,
                               causal, window)
    u, scores = UNIT[str(dtype)], 2e-4 * max(1.0, gap / 20.0)
    tol = u * (spread + np.abs(ref)) + scores * spread + 2.0 ** -25 + 2.0 ** -28
    worst = (np.abs(f64(out) - ref) / tol).max()
    assert worst <= 1.0, worst
    assert (np.abs(f64(lse) - z) <= scores).all()


def test_weights_without_the_norm_are_not_used(cuda_lib):
    """The weights belong to the norm: a C caller that passes them with norm = 0 gets the rows without either."""
    g = gen(51)
    lib = attn.load()
    T, HQ, HK, D, page = 9, 3, 2, 64, 16
    q, k, v = normal(g, T, HQ, D), normal(g, T, HK, D), normal(g, T, HK, D)
    w = 2 + normal(g, D).abs()
    f, _ = attn.rope_frequencies(D)
    pos = ints(list(range(T)))
    want_q, want_k = attn.qk_norm_rope(q, k, pos, f, norm=False)
    c = Cache(g, [T], [0], page, HK, D)
    dims = attn.AttnDims()
    assert lib.gdn2_attn_dims_init(dims, T, 1, HQ, HK, D, c.k.shape[0], page, c.table.shape[1]) == 0
    dims.norm = 0
    qo, ko, ws = torch.zeros_like(q), torch.zeros_like(k), torch.zeros(64, dtype=torch.uint8, device="cuda")
    p = [x.data_ptr() for x in (q, k, w, w, f, pos, qo, ko)]
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.gdn2_qk_norm_rope(*p, dims, stream) == 0
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k)
    qo.zero_()
    p = [x.data_ptr() for x in (q, k, v, w, w, f, pos, c.cu, c.lens, c.table, qo, c.k, c.v)]
    assert lib.gdn2_kv_append(*p, dims, ws.data_ptr(), 64, stream) == 0
    rows = c.k[int(c.table[0, 0]), :T]
    assert attn.device_status(ws) == 0 and torch.equal(qo, want_q) and torch.equal(rows, want_k)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_infinite_weight_of_a_channel_that_does_not_turn(cuda_lib, inter, D):
    """y = x w / rms(x) there: infinite in that channel, and of no effect on any other."""
    g = gen(52)
    q = normal(g, 5, 3, D)
    assert (q != 0).all()
    w = 1 + normal(g, D) / 4
    f, _ = attn.rope_frequencies(32)
    pos = ints([0, 1, 2, 77, 4095])
    want, _ = attn.qk_norm_rope(q, None, pos, f, interleaved=inter, q_weight=w)
    at = [32, 45, D - 1]
    w[at] = float("inf")
    y, _ = attn.qk_norm_rope(q, None, pos, f, interleaved=inter, q_weight=w)
    assert torch.equal(y[..., at], torch.sign(q[..., at]) * float("inf"))
    rest = [i for i in range(D) if i not in at]
    assert torch.equal(y[..., rest], want[..., rest])
