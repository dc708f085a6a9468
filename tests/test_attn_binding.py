"""What the bindings refuse before any kernel could see it.  Host only, but for
the tests marked gpu: tensors on the CPU, or metadata alone.
"""
import pytest
import torch

from gated_deltanet_prefill_gb300 import attn, gdn2


def paged_metadata(table):
    """_check_paged on `table` as if it were on the GPU, with caches and lengths that fit."""
    n = table.shape[0]
    cache = (torch.Size((40, 16, 2, 64)), (2048, 128, 64, 1), torch.bfloat16, True)
    return attn._check_paged(cache, cache, (table.shape, table.stride(), table.dtype, True), (n, torch.int32, True),
                             (n + 1, torch.int32, True))


def test_block_table_rows_keep_their_stride():
    wide = torch.zeros(4, 15, dtype=torch.int32)
    n, _, _, stride, width, _ = paged_metadata(wide[:, :10])
    assert (n, stride, width) == (4, 15, 10)
    # a single row has no stride: any that is given goes
    for table in (wide[:1, :10], torch.zeros(10, dtype=torch.int32).expand(1, 10), wide.as_strided((1, 10), (3, 1))):
        assert paged_metadata(table)[0] == 1 and paged_metadata(table)[3] >= 10
    assert paged_metadata(wide[:, :0])[4] == 0 and paged_metadata(wide[:0])[0] == 0
    assert paged_metadata(wide[:, :1])[3:5] == (15, 1)


@pytest.mark.parametrize("shape,stride", [((4, 10), (0, 1)), ((4, 10), (5, 1)), ((2, 10), (9, 1)), ((4, 1), (0, 1)),
                                          ((4, 1), (0, 7))])
def test_block_table_rows_on_top_of_one_another_are_refused(shape, stride):
    """One row expanded to all sequences, rows that overlap: the kernels would read at strides that the table does not have."""
    table = torch.zeros(100, dtype=torch.int32).as_strided(shape, stride)
    with pytest.raises(ValueError, match="block_table"):
        paged_metadata(table)


def calls(x, workspace):
    """append_kv and paged_attn_fwd on tensors like x, with the workspace."""
    i32 = torch.zeros(4, dtype=torch.int32, device=x.device)
    cache = torch.zeros(3, 16, 2, 64, dtype=x.dtype, device=x.device)
    other = torch.zeros_like(cache)
    yield lambda: attn.append_kv(x, x, cache, other, i32[None], i32[:1], i32[:2], workspace=workspace)
    yield lambda: attn.paged_attn_fwd(x, cache, other, i32[None], i32[:1], i32[:2], workspace=workspace)


def refused_workspaces(device):
    """A workspace elsewhere (the meta device stands in for the CPU beside a GPU), and one whose bytes do not lie together:
    its size in bytes passes the library's check, its memory is not its own."""
    yield torch.empty(1 << 26, dtype=torch.uint8, device="meta" if device == "cpu" else "cpu")
    yield torch.empty(1 << 12, dtype=torch.uint8, device=device)[::2]
    yield torch.empty(1, dtype=torch.uint8, device=device).expand(1 << 26)
    yield torch.empty(64, 64, dtype=torch.float32, device=device).t()


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_prefill_gb300 import build
    build.build()
    return attn.load()


def test_workspaces_that_are_not_plain_memory_beside_the_inputs_are_refused(lib):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for workspace in refused_workspaces("cpu"):
        for call in calls(x, workspace):
            with pytest.raises(ValueError, match="workspace"):
                call()


@pytest.mark.gpu
def test_workspaces_refused_on_the_gpu(cuda_lib):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    for call in calls(x, torch.empty(1 << 26, dtype=torch.uint8, device="cuda")):
        call()  # known metadata from here on
    for workspace in refused_workspaces("cuda"):
        for call in calls(x, workspace):
            with pytest.raises(ValueError, match="workspace"):
                call()


def arguments(device):
    """The tensor arguments of the three calls, by call."""
    def zeros(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=device)

    rows = zeros(4, 2, 64)
    rotary = dict(positions=zeros(4, dtype=torch.int32), inv_freq=zeros(32, dtype=torch.float64), q_weight=zeros(64),
                  k_weight=zeros(64), q_out=zeros(4, 2, 64))
    cache = dict(k_cache=zeros(3, 16, 2, 64), v_cache=zeros(3, 16, 2, 64), block_table=zeros(1, 3, dtype=torch.int32),
                 kv_lens=zeros(1, dtype=torch.int32), cu_seqlens=zeros(2, dtype=torch.int32))
    return {attn.qk_norm_rope: dict(q=rows, k=rows, k_out=zeros(4, 2, 64), **rotary),
            attn.append_kv: dict(k=rows, v=rows, q=rows, **cache, **rotary),
            attn.paged_attn_fwd: dict(q=rows, **cache, out=zeros(4, 2, 64), lse=zeros(4, 2, dtype=torch.float32))}


def test_tensors_of_two_devices_are_refused(lib):
    """One argument after the other on another device than the rest (the meta device stands in for a second GPU)."""
    for call, args in arguments("cpu").items():
        for name in args:
            with pytest.raises(ValueError, match="one device"):
                call(**{**args, name: args[name].to("meta")})


@pytest.mark.gpu
def test_tensors_of_two_devices_are_refused_on_the_gpu(cuda_lib):
    args = arguments("cuda")
    for call in args:
        call(**args[call])  # known metadata from here on
        for name in args[call]:
            with pytest.raises(ValueError, match="one device"):
                call(**{**args[call], name: args[call][name].cpu()})


class Tensor:
    """What the GDN-2 binding's checks look at, on a device that this machine need not have."""
    is_cuda, dtype, shape = True, torch.bfloat16, (4, 2, 64)

    def __init__(self, index=0, device="cuda"):
        self.device = torch.device(device, index)
        self.is_cuda = device == "cuda"

    def is_contiguous(self):
        return True


@pytest.mark.parametrize("call,more", [(gdn2.chunk_gdn2_fwd, ("workspace",)), (gdn2.recurrent_gdn2_fwd, ("workspace",)),
                                       (gdn2.chunk_gdn2_fwd_noalloc, ())])
def test_gdn2_calls_refuse_tensors_of_two_devices(lib, call, more):
    names = ("q", "k", "v", "g", "beta", "w", "initial_state", "cu_seqlens", "out", "final_state") + more
    for name in names[1:]:
        for other in (Tensor(1), Tensor(0, "cpu")):
            with pytest.raises(ValueError, match="q's device|must be a CUDA tensor"):
                call(**{n: other if n == name else Tensor() for n in names})


@pytest.mark.parametrize("scale", [0.0, 0, -0.125, -1, 1e-50, float("nan")])
def test_scales_that_are_not_positive_are_refused(lib, scale):
    """Not taken for "no scale given", which is 1/sqrt(D)."""
    args = arguments("cpu")[attn.paged_attn_fwd]
    with pytest.raises(ValueError, match="scale"):
        attn.paged_attn_fwd(**args, scale=scale)


@pytest.mark.gpu
def test_scales_refused_on_the_gpu(cuda_lib):
    args = arguments("cuda")[attn.paged_attn_fwd]
    attn.paged_attn_fwd(**args, scale=0.25)  # known metadata from here on
    for scale in (0.0, -0.125, 1e-50, float("nan")):
        with pytest.raises(ValueError, match="scale"):
            attn.paged_attn_fwd(**args, scale=scale)
    with pytest.raises(gdn2.Gdn2Error) as e:
        attn.paged_attn_fwd(**args, scale=float("inf"))
    assert e.value.status == 2
