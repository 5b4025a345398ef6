"""One token taken out of a wider batch: its row starts where it has to, and how far off the next one
would be does not matter."""
import pytest
import torch

from tests.helpers import load_lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [513, 521, 512 + 8])
def test_one_token_of_a_batch_with_odd_rows(wide):
    M = load_lib()
    H, N = 512, 40
    buf = torch.randn(16, wide, device="cuda").to(torch.bfloat16)
    one = buf[8:9, :H]                     # eight rows down: on a 16-byte boundary whatever their length
    x = one.contiguous()
    W = torch.randn(N, H, device="cuda").to(torch.bfloat16)
    A, B = torch.randn(2, 8, H, device="cuda").to(torch.bfloat16), torch.randn(2, N, 8, device="cuda").to(torch.bfloat16)
    ids = torch.ones(1, dtype=torch.int32, device="cuda")
    assert torch.equal(M.moe_adapter_linear(one, W, A, B, ids), M.moe_adapter_linear(x, W, A, B, ids))
    # and a single row of W
    w = torch.zeros(8, wide, dtype=torch.bfloat16, device="cuda")
    w[0, :H] = W[3]
    assert torch.equal(M.moe_adapter_linear(x, w[:1, :H]), M.moe_adapter_linear(x, W[3:4]))
    nw = torch.rand(H, device="cuda")
    for a, b in zip(M.moe_block_norm(one, x, nw, None, 0.5, nw), M.moe_block_norm(x, x, nw, None, 0.5, nw)):
        assert torch.equal(a, b)
    assert all(torch.equal(a, b) for a, b in zip(M.moe_route(one, 8), M.moe_route(x, 8)))
    # a result into one row of a wider buffer leaves the rest of it alone
    out = torch.full((3, N + 5), 7.0, device="cuda")
    M.moe_adapter_linear(one, W, A, B, ids, out=out[1:2, 2:N + 2])
    assert torch.equal(out[1, 2:N + 2], M.moe_adapter_linear(x, W, A, B, ids, out_dtype=torch.float32)[0])
    out[1, 2:N + 2] = 7
    assert (out == 7).all()
