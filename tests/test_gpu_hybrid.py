"""examples/hybrid_block.py: GDN-2 and attention layers over one packed batch,
prefilled in chunks and continued token by token, against the same stack in fp64
(the recurrence by the oracle, attention by tests/attn_reference.py).

Tolerance, fixed before the first run: a GDN-2 layer's heads err by at most 1e-2
of their largest value (the bound of the operator's own tests), attention's by
less; each layer adds the bf16 rounding of its input, its two projections' results and the residual
sum (4 x 2^-8 of the largest value): 2.6e-2 per layer, 5.2e-2 of the largest
output over two.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from attn_reference import attention, f64, norm_rope

pytestmark = pytest.mark.gpu
TOLERANCE = 5.2e-2


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_block.py")
    spec = importlib.util.spec_from_file_location("hybrid_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_stack(model, x, lens):
    """Whole sequences through the model's layers in fp64; x [tokens, dim]."""
    cu = np.cumsum([0] + lens)
    x = f64(x)
    for layer in model.layers:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.finfo(np.float32).eps)
        y = (y @ f64(layer.w_in)).reshape(len(x), -1, layer.d)
        if hasattr(layer, "state"):
            q, k, v, w, beta, g = np.split(y, 6, axis=1)
            o, _ = oracle.gdn2_forward(q, k, v, -np.log1p(np.exp(g - 2)), 1 / (1 + np.exp(-beta)), 1 / (1 + np.exp(-w)),
                                       cu_seqlens=cu, use_qk_l2norm=True)
        else:
            q, k, v = np.split(y, [layer.hq, layer.hq + layer.hkv], axis=1)
            place = np.concatenate([np.arange(n) for n in lens])
            f = layer.inv_freq.tolist()
            q = norm_rope(q, place, f, f64(layer.q_weight), factor=layer.rope_factor)
            k = norm_rope(k, place, f, f64(layer.k_weight), factor=layer.rope_factor)
            longest = max(lens)
            pages = np.zeros((2, len(lens), longest) + k.shape[1:])
            for n, t in enumerate(lens):
                pages[0, n, :t], pages[1, n, :t] = k[cu[n]:cu[n + 1]], v[cu[n]:cu[n + 1]]
            table = np.arange(len(lens))[:, None]
            o, _, _ = attention(q, pages[0], pages[1], table, lens, cu, layer.d ** -0.5)
        x = x + np.asarray(o).reshape(len(x), -1) @ f64(layer.w_out)
    return x


@pytest.mark.parametrize("head_dim,heads,kv_heads", [(128, 4, 1), (64, 6, 3)])
def test_chunks_and_tokens_through_both_kinds_of_layer(cuda_lib, example, head_dim, heads, kv_heads):
    lens = [150, 37, 211]
    kw = dict(dim=256, layers=2, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page_size=16, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn(sum(lens), 256, device="cuda", generator=g).to(torch.bfloat16)
    whole = example.HybridModel(3, 220, **kw)
    ref = plain_stack(whole, x, lens)
    bound = TOLERANCE * np.abs(ref).max()
    assert np.abs(f64(whole(x, lens)) - ref).max() <= bound
    # the same in chunks of odd lengths, a sequence left out of one, then single tokens
    model = example.HybridModel(3, 220, **kw)
    start, done = np.cumsum([0] + lens), [0, 0, 0]
    got = np.zeros_like(ref)
    for new in ([100, 0, 64], [45, 20, 143], [3, 15, 2], [1, 1, 1], [1, 1, 1]):
        rows = np.concatenate([start[n] + done[n] + np.arange(c) for n, c in enumerate(new)])
        got[rows] = f64(model(x[torch.from_numpy(rows).cuda()], new))
        done = [a + b for a, b in zip(done, new)]
    assert done == lens and np.abs(got - ref).max() <= bound


def test_example_command(cuda_lib, example, monkeypatch, capsys):
    for more in ([], ["--graph"]):
        monkeypatch.setattr("sys.argv", ["hybrid_block.py", "--layers", "2", "--dim", "256", "--heads", "4", "--kv-heads",
                                         "2", "--seqs", "2", "--prompt", "192", "--chunk", "128", "--tokens", "5"] + more)
        example.main()
        out = capsys.readouterr().out
        assert "prefill" in out and "decode" in out
