"""Memory of the layer's entry points on a stream that is not the current one:
a call is queued behind a wait on its stream, and the current stream allocates
and writes tensors of the same sizes meanwhile."""
import pytest

from tests.gpu_util import note, torch_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,d,dtype", [(3001, 1000, "f32"), (600, 4096, "bf16"), (260, 130, "f32")])
def test_gradients_on_another_stream_keep_their_workspace(rows, d, dtype):
    torch, dev = torch_dev()
    import retnet_scale_retention_amd as msr
    note(f"norm backward on another stream {rows}x{d} {dtype}")
    g = torch.Generator(device=dev).manual_seed(rows)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    h, dy = (torch.randn(rows, d, generator=g, device=dev).to(t) for _ in range(2))
    w = torch.randn(d, generator=g, device=dev)
    want = msr.msr_add_rmsnorm_backward(h, w, dy)  # also warms the current stream's pool with a free workspace
    assert msr.load().msr_add_rmsnorm_backward_workspace(rows, d) > 0
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(1_000_000)
    dx, dw = msr.msr_add_rmsnorm_backward(h, w, dy, stream=st)
    n = msr.load().msr_add_rmsnorm_backward_workspace(rows, d)
    for _ in range(8):
        torch.empty(n, dtype=torch.uint8, device=dev).fill_(0xFF)
        torch.empty(d, device=dev).fill_(float("nan"))
    st.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_results_on_another_stream_that_are_dropped_early():
    torch, dev = torch_dev()
    import retnet_scale_retention_amd as msr
    x = torch.randn(512, 2048, device=dev).bfloat16()
    zero = torch.zeros_like(x)
    want, _, _, _ = msr.msr_quantize(x)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    q, s, _, _ = msr.msr_quantize(x, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda._sleep(1_000_000)
    got = q.view(torch.uint8).clone()      # reads q behind the wait
    del q, s
    for _ in range(8):                     # calls on the other stream must not get q's memory before that
        msr.msr_quantize(zero, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(got, want.view(torch.uint8))
