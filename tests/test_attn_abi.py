"""The attention-layer entry points on the host: declared and exported alike,
bad arguments refused before a device is touched.  No kernel is launched."""
import ctypes
import math
import os
import re

import pytest
import torch

from gated_deltanet_prefill_gb300 import attn, gdn2
from gated_deltanet_prefill_gb300 import build as gbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, STRIDE, ALIAS, WORKSPACE, ARCH, DTYPE = 0, 1, 2, 3, 4, 5, 6, 8
NAMES = ("q", "k", "v", "q_weight", "k_weight", "inv_freq", "positions", "cu", "kv_lens", "table", "q_out", "k_out",
         "k_cache", "v_cache", "out", "lse", "ws")
# fake, well-separated, aligned device addresses: host arithmetic only
BASE, STEP = 1 << 40, 1 << 32


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return attn.load()


def dims(lib, **over):
    """100 tokens, 3 sequences, 8 query and 2 key heads of 128, 40 pages of 16, 12 table columns."""
    d = attn.AttnDims()
    assert lib.gdn2_attn_dims_init(d, 100, 3, 8, 2, 128, 40, 16, 12) == OK
    for name, value in over.items():
        if isinstance(value, tuple):
            value = type(getattr(d, name))(*value)
        setattr(d, name, value)
    return d


def ptrs(**over):
    p = {n: BASE + i * STEP for i, n in enumerate(NAMES)}
    p.update(over)
    return p


def norm_rope(lib, d, **over):
    p = ptrs(**over)
    return lib.gdn2_qk_norm_rope(p["q"], p["k"], p["q_weight"], p["k_weight"], p["inv_freq"], p["positions"],
                                 p["q_out"], p["k_out"], d, None)


def append(lib, d, ws_bytes=64, **over):
    p = ptrs(**over)
    return lib.gdn2_kv_append(p["q"], p["k"], p["v"], p["q_weight"], p["k_weight"], p["inv_freq"], p["positions"],
                              p["cu"], p["kv_lens"], p["table"], p["q_out"], p["k_cache"], p["v_cache"], d, p["ws"],
                              ws_bytes, None)


def paged(lib, d, ws_bytes=None, scale=0.0, **over):
    p = ptrs(**over)
    ws_bytes = lib.gdn2_paged_attn_workspace_bytes(d) if ws_bytes is None else ws_bytes
    return lib.gdn2_paged_attn_fwd(p["q"], p["k_cache"], p["v_cache"], p["cu"], p["kv_lens"], p["table"], scale,
                                   p["out"], p["lse"], d, p["ws"], ws_bytes, None)


def test_header_and_binding_agree(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gdn2_attn.h")).read(), flags=re.S)
    declared = set(re.findall(r"GDN2_API\s+[\w\s\*]+?\b(gdn2_\w+)\s*\(", src))
    assert declared == set(attn.EXPORTS)
    for name in declared:
        assert hasattr(lib, name), name
    assert gdn2.STATUS_NAMES[16] == "ERR_PAGES"
    assert lib.gdn2_status_string(16).decode() != "unknown status"


def test_dims_layout_matches_the_header(lib):
    """gdn2_attn_dims_init fills the fields the binding's struct names."""
    d = dims(lib)
    assert (d.T_tot, d.N, d.HQ, d.HKV, d.D) == (100, 3, 8, 2, 128)
    assert (d.num_pages, d.page_size, d.max_pages, d.table_stride) == (40, 16, 12, 12)
    assert list(d.q_stride) == [1024, 128] and list(d.ko_stride) == [256, 128]
    assert list(d.kc_stride) == [16 * 256, 256, 128] == list(d.vc_stride)
    assert (d.dtype, d.norm, d.rot_dim, d.causal, d.window_left) == (0, 1, 128, 1, -1)
    assert d.norm_eps == pytest.approx(1e-6) and d.rope_factor == 1.0
    assert lib.gdn2_attn_dims_init(d, 1, 1, 1, 1, 96, 1, 16, 1) == SHAPE
    assert lib.gdn2_attn_dims_init(None, 1, 1, 1, 1, 64, 1, 16, 1) == NULL


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="a valid call would launch on this machine's GPU")


@needs_no_gpu
def test_valid_calls_reach_the_device_check(lib):
    """Without a device a call whose arguments pass reports ERR_ARCH."""
    d = dims(lib)
    assert norm_rope(lib, d) == ARCH and append(lib, d) == ARCH and paged(lib, d) == ARCH
    assert norm_rope(lib, d, k=None, k_out=None, k_weight=None) == ARCH
    assert norm_rope(lib, d, q=None, q_out=None) == ARCH
    assert append(lib, d, q=None, q_out=None, positions=None) == ARCH
    assert paged(lib, d, lse=None) == ARCH
    p = ptrs()
    assert norm_rope(lib, d, q_out=p["q"], k_out=p["k"]) == ARCH          # in place
    assert append(lib, d, q_out=p["q"]) == ARCH
    # views of one packed projection [T, 8 + 2 + 2, 128], in place
    packed = dims(lib, q_stride=(1536, 128), k_stride=(1536, 128), v_stride=(1536, 128), qo_stride=(1536, 128),
                  ko_stride=(1536, 128))
    at = dict(q=p["q"], k=p["q"] + 8 * 256, v=p["q"] + 10 * 256)
    assert norm_rope(lib, packed, q=at["q"], k=at["k"], q_out=at["q"], k_out=at["k"]) == ARCH
    assert append(lib, packed, q_out=at["q"], **at) == ARCH
    # k and v pages interleaved in one allocation
    both = dims(lib, kc_stride=(2 * 4096, 256, 128), vc_stride=(2 * 4096, 256, 128))
    assert append(lib, both, v_cache=p["k_cache"] + 2 * 4096) == ARCH
    assert paged(lib, both, v_cache=p["k_cache"] + 2 * 4096) == ARCH
    # head-major pages, no tokens, no sequences
    assert paged(lib, dims(lib, kc_stride=(4096, 128, 2048))) == ARCH
    assert append(lib, dims(lib, T_tot=0)) == ARCH and paged(lib, dims(lib, T_tot=0)) == ARCH
    assert paged(lib, dims(lib, T_tot=0, N=0), kv_lens=None, table=None) == ARCH


@pytest.mark.parametrize("field,value,code", [
    ("dtype", 2, DTYPE), ("dtype", 7, DTYPE), ("D", 96, SHAPE), ("D", 256, SHAPE), ("T_tot", -1, SHAPE),
    ("T_tot", 1 << 31, SHAPE), ("rot_dim", 8, SHAPE), ("rot_dim", 144, SHAPE), ("rot_dim", -16, SHAPE),
    ("norm", 2, SHAPE), ("rope_interleaved", 3, SHAPE), ("norm_eps", -1.0, SHAPE), ("norm_eps", math.nan, SHAPE),
    ("rope_factor", math.inf, SHAPE), ("HQ", 0, SHAPE), ("HKV", 0, SHAPE), ("q_stride", (1028, 128), STRIDE),
    ("q_stride", (1024, -128), STRIDE), ("qo_stride", (1024, 64), ALIAS), ("qo_stride", (512, 128), ALIAS)])
def test_norm_rope_and_append_refuse(lib, field, value, code):
    assert norm_rope(lib, dims(lib, **{field: value})) == code
    assert append(lib, dims(lib, **{field: value})) == code


def test_norm_rope_refusals(lib):
    d, p = dims(lib), ptrs()
    assert lib.gdn2_qk_norm_rope(p["q"], None, None, None, p["inv_freq"], p["positions"], p["q_out"], None, None,
                                 None) == NULL
    assert norm_rope(lib, d, q=None, k=None, q_out=None, k_out=None) == NULL
    assert norm_rope(lib, d, q=None) == NULL and norm_rope(lib, d, k_out=None) == NULL
    assert norm_rope(lib, d, inv_freq=None) == NULL and norm_rope(lib, d, positions=None) == NULL
    assert norm_rope(lib, d, q=p["q"] + 2) == STRIDE and norm_rope(lib, d, q_weight=p["q_weight"] + 2) == STRIDE
    assert norm_rope(lib, d, q_out=p["q"] + 256) == ALIAS and norm_rope(lib, d, k_out=p["q"]) == ALIAS
    assert norm_rope(lib, d, k_out=p["q_out"]) == ALIAS and norm_rope(lib, d, q_out=p["positions"]) == ALIAS
    assert norm_rope(lib, dims(lib, qo_stride=(2048, 128)), q_out=p["q"]) == ALIAS  # in place, other strides


@pytest.mark.parametrize("field,value,code", [
    ("page_size", 0, SHAPE), ("page_size", 12, SHAPE), ("max_pages", -1, SHAPE), ("max_pages", 1 << 30, SHAPE),
    ("num_pages", -1, SHAPE), ("num_pages", 1 << 32, SHAPE), ("table_stride", 11, SHAPE), ("N", -1, SHAPE),
    ("HKV", 0, SHAPE), ("kc_stride", (4096, 256, 100), STRIDE), ("vc_stride", (4096, 4, 128), STRIDE)])
def test_paged_shapes_refused(lib, field, value, code):
    d = dims(lib, **{field: value})
    assert append(lib, d) == code and paged(lib, d, ws_bytes=1 << 31) == code
    if code == SHAPE:
        assert lib.gdn2_paged_attn_workspace_bytes(d) == 0 == lib.gdn2_kv_append_workspace_bytes(d)


def test_append_refusals(lib):
    d, p = dims(lib), ptrs()
    for name in ("k", "v", "inv_freq", "cu", "kv_lens", "table", "k_cache", "v_cache", "ws", "q", "q_out"):
        assert append(lib, d, **{name: None}) == NULL, name
    assert append(lib, d, ws_bytes=63) == WORKSPACE
    assert append(lib, d, k=p["k"] + 8) == STRIDE and append(lib, d, ws=p["ws"] + 4) == STRIDE
    assert append(lib, d, v_cache=p["k_cache"]) == ALIAS and append(lib, d, k_cache=p["k"]) == ALIAS
    assert append(lib, d, q_out=p["v"]) == ALIAS and append(lib, d, v_cache=p["q_out"]) == ALIAS
    assert append(lib, d, q_out=p["kv_lens"]) == ALIAS and append(lib, d, k_cache=p["ws"]) == ALIAS
    assert append(lib, dims(lib, kc_stride=(2048, 256, 128))) == ALIAS  # pages on top of one another
    assert append(lib, dims(lib, vc_stride=(4096, 256, 64))) == ALIAS


def test_paged_attn_refusals(lib):
    d, p = dims(lib), ptrs()
    for name in ("q", "cu", "kv_lens", "table", "k_cache", "v_cache", "ws", "out"):
        assert paged(lib, d, **{name: None}) == NULL, name
    need = lib.gdn2_paged_attn_workspace_bytes(d)
    assert need >= 64 and paged(lib, d, ws_bytes=need - 1) == WORKSPACE
    assert paged(lib, d, scale=math.nan) == SHAPE
    for over in (dict(HQ=9), dict(HQ=0), dict(HQ=258), dict(causal=2), dict(window_left=-2),
                 dict(causal=0, window_left=5)):
        assert paged(lib, dims(lib, **over), ws_bytes=1 << 31) == SHAPE, over
    assert paged(lib, d, q=p["q"] + 8) == STRIDE and paged(lib, d, lse=p["lse"] + 2) == STRIDE
    for over in (dict(out=p["q"]), dict(out=p["k_cache"]), dict(out=p["lse"]), dict(lse=p["q"]), dict(lse=p["ws"]),
                 dict(ws=p["v_cache"]), dict(out=p["table"])):
        assert paged(lib, d, **over) == ALIAS, over
    assert paged(lib, dims(lib, qo_stride=(1024, 64))) == ALIAS


def test_binding_refuses_cpu_tensors_and_bad_shapes(lib):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attn.qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        attn.append_kv(x, x, cache, cache, i32[None], i32[:1], i32[:2])
    with pytest.raises(ValueError):
        attn.paged_attn_fwd(x, cache, cache, i32[None], i32[:1], i32[:2])
    with pytest.raises(ValueError):
        attn.qk_norm_rope(x, x[:3])
    with pytest.raises(ValueError):
        attn.qk_norm_rope(x, norm=False, q_weight=x[0, 0])


def test_rope_frequencies():
    f, m = attn.rope_frequencies(64, device="cpu")
    assert f.dtype == torch.float64 and f.numel() == 32 and m == 1.0
    assert f[0] == 1.0 and float(f[16]) == pytest.approx(0.01, rel=1e-14)
    g, m = attn.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(g, f / 4) and m == 1.0
    g, _ = attn.rope_frequencies(64, scaling="base", factor=4.0, device="cpu")
    assert g[0] == 1.0 and float(g[-1]) == pytest.approx(float(f[-1]) / 4, rel=1e-12)
    g, m = attn.rope_frequencies(64, scaling="parts", factor=8.0, trained_len=4096, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns > 32], f[turns > 32])
    assert torch.allclose(g[turns < 1], f[turns < 1] / 8, rtol=1e-15)
    assert m == pytest.approx(0.1 * math.log(8.0) + 1.0) and (g[1:] < g[:-1]).all()
    for bad in (dict(rot_dim=0), dict(rot_dim=64, scaling="x"), dict(rot_dim=64, scaling="linear", factor=0.0),
                dict(rot_dim=64, scaling="parts", factor=2.0)):
        with pytest.raises(ValueError):
            attn.rope_frequencies(device="cpu", **bad)
