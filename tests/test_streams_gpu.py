"""Tensors that a call on another stream makes are that stream's: memory that the
current stream's pending work may still write is not handed out for them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

B, H, L, D = 1, 8, 256, 128


def _calls(sdpa):
    g = torch.Generator("cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    q, k, v, dout = (normal(B, H, L, D) for _ in range(4))
    lse = torch.empty(B, H, L, device="cuda")
    out = sdpa.forward_ex(q, k, v, causal=True, lse=lse)
    plan = sdpa.rotary_plan(D)
    ws = torch.empty(max(16, sdpa.workspace_bytes(B, H, H, L, L, D, D, True)), dtype=torch.uint8, device="cuda")
    return {"backward": lambda **kw: sdpa.backward(q, k, v, out, lse, dout, causal=True, **kw),
            "rotary": lambda **kw: sdpa.rotary(plan, q, k, **kw),
            "forward": lambda **kw: (sdpa.forward(q, k, v, causal=True, **kw),),
            "forward_ex": lambda **kw: (sdpa.forward_ex(q, k, v, causal=True, **kw),),
            "forward_noalloc": lambda **kw: (sdpa.forward_noalloc(q, k, v, causal=True, **kw),),
            "forward_ws": lambda **kw: (sdpa.forward_ws(q, k, v, ws, causal=True, **kw),)}


@pytest.mark.parametrize("name", ["backward", "rotary", "forward", "forward_ex", "forward_noalloc", "forward_ws"])
@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_outputs_belong_to_the_stream_of_the_call(cuda_lib, name, kind):
    call = _calls(cuda_lib)[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    # the current stream: a few milliseconds of work, behind it writes to tensors of the
    # outputs' size, which are given back to the allocator before those writes run
    late = [torch.empty(B, H, L, D, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    for _ in range(20):
        busy = busy @ busy * 1e-3
    for t in late:
        t.fill_(7)
    del late, t
    got = call(stream=side if kind == "stream" else side.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["backward", "rotary", "forward", "forward_ex", "forward_noalloc", "forward_ws"])
def test_outputs_that_the_current_stream_still_reads(cuda_lib, name):
    """A result of another stream, read by the current one and released: the next call
    does not get its memory before that read is done."""
    call = _calls(cuda_lib)[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    got = call(stream=side)
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 1e-3
    read = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):  # what comes next on that stream takes released memory
        late = [torch.full((B, H, L, D), 7, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del late
    assert all(torch.equal(a, b) for a, b in zip(read, want))


def test_the_default_stream_by_its_handle(cuda_lib):
    for name, call in _calls(cuda_lib).items():
        want = call()
        got = call(stream=0)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_captured_on_the_stream_that_is_passed(cuda_lib):
    for name, call in _calls(cuda_lib).items():
        want = [t.clone() for t in call()]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = call(stream=torch.cuda.current_stream())
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_captured_on_a_stream_of_its_own(cuda_lib):
    """A branch of a captured graph: the side stream joins the capture and is joined."""
    for name, call in _calls(cuda_lib).items():
        want = [t.clone() for t in call()]
        g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g):
            side.wait_stream(torch.cuda.current_stream())
            got = call(stream=side)
            torch.cuda.current_stream().wait_stream(side)
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
