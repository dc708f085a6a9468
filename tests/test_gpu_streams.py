"""The GDN-2 calls on a stream other than the current one: memory made for a
call (workspace, outputs) is not handed out while that stream still waits."""
import pytest
import torch

from gated_deltanet_prefill_gb300 import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["chunk", "recurrent"])
def test_call_on_a_stream_other_than_the_current_one(cuda_lib, call):
    wl = inputs.Workload("streams", (130, 70), 2, 2, 64, 64, h0_std=0.1)
    d = {k: v.cuda() if torch.is_tensor(v) else v for k, v in inputs.generate(wl).items()}
    fn = cuda_lib.chunk_gdn2_fwd if call == "chunk" else cuda_lib.recurrent_gdn2_fwd
    args, more = [d[k] for k in ("q", "k", "v", "g", "beta", "w")], dict(initial_state=d["h0"], cu_seqlens=d["cu_seqlens"])
    want = fn(*args, **more)
    size = 256
    if call == "chunk":
        dims = cuda_lib.make_dims(*args, want[0], d["cu_seqlens"])
        size = max(size, cuda_lib.workspace_bytes(dims))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    got = fn(*args, **more, stream=side.cuda_stream)
    blocks = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all((b == 255).all() for b in blocks)
    with torch.cuda.stream(side):  # the default stream given by its handle, which is zero
        again = fn(*args, **more, stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
