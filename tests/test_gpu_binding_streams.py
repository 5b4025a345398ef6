"""Memory of the calls with a `stream` of their own: results and workspaces that the caller does not bring.

Each test queues work on one stream behind a wait, lets go of a tensor that this work still uses, and makes a call on
another stream meanwhile: what the call allocates must not be that tensor's memory."""
import pytest
import torch

from tests.helpers import load_lib

pytestmark = pytest.mark.gpu

LONG = 100_000_000   # clocks: some 50 ms


def _calls(M, T=512, H=1024):
    """{name: (function of a stream that returns the results, ...)}: each allocates its results and workspace."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*s, dtype=torch.bfloat16):
        return torch.randn(*s, device="cuda", generator=g).to(dtype)
    lg, x, y, du, dh = normal(T, 256, dtype=torch.float32), normal(T, H), normal(T, H), normal(T, H), normal(T, H)
    w = 1 + torch.rand(H, device="cuda")
    ids, dw = torch.randint(0, 256, (T, 1), device="cuda", dtype=torch.int32), normal(T, 1, dtype=torch.float32)
    W, A, B = normal(H, H), normal(4, 16, H), normal(4, H, 16)
    ad = torch.randint(0, 4, (T,), device="cuda", dtype=torch.int32)
    return {
        "route": lambda s: M.moe_route(lg, 8, stream=s),
        "route_backward": lambda s: (M.moe_route_backward(lg, ids, dw, stream=s),),
        "block_norm": lambda s: M.moe_block_norm(x, y, w, None, 1.0, w, stream=s),
        "block_norm_backward": lambda s: M.moe_block_norm_backward(x, y, du, dh, w, w, 1.0, w, stream=s),
        "adapter_linear": lambda s: (M.moe_adapter_linear(x, W, A, B, ad, stream=s),),
    }


NAMES = ["route", "route_backward", "block_norm", "block_norm_backward", "adapter_linear"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_uses_is_not_taken(name):
    M = load_lib()
    call = _calls(M)[name]
    want = [t.clone() for t in call(None)]
    sizes = [t.nbytes for t in want] + [1 << 16, 1 << 18, 1 << 20, 1 << 21]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    used = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    read = torch.stack([u.float().mean() for u in used])   # reads them after the wait
    del used
    got = call(s)
    s.synchronize()
    torch.cuda.synchronize()
    assert (read == 7).all()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_results_let_go_of_early_are_not_overwritten_under_the_call(name):
    M = load_lib()
    call = _calls(M)[name]
    sizes = [(t.shape, t.dtype) for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        torch.cuda._sleep(LONG)
    call(s)                                                # its results are let go of at once
    mine = [torch.full(shape, 3, dtype=dtype, device="cuda") for shape, dtype in sizes]
    torch.cuda.synchronize()
    assert all((t == 3).all() for t in mine)


@pytest.mark.parametrize("name", NAMES)
def test_results_that_the_current_stream_still_reads_are_not_taken_by_the_next_call(name):
    M = load_lib()
    call = _calls(M)[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(LONG)
    read = [t.clone() for t in got]
    del got
    with torch.cuda.stream(s):
        more = [torch.zeros(t.shape, dtype=t.dtype, device="cuda") for t in want for _ in range(2)]   # same sizes, there
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read, want)) and len(more) == 2 * len(want)
