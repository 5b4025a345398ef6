"""The routes of sorted rows that batches of some hundred and some thousand tokens take: a warp to a token in the gradient of
the combine, blocks with several passes over a row, sorted rows of several blocks each.

Tolerances as in test_gpu_token_rows; the reference is the formula in 64 bits, all tokens at once."""
import pytest
import torch

from tests.helpers import load_lib
from tests.test_gpu_token_rows import BF16, F16, F32, half, normal, routing, sorted_on_host, tiny

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# tokens (in SMs, and more), k, H, types of rows and tokens, columns between rows.  Vectors of 8, 2 and 1 elements, rows
# that a token's threads take in several passes with a ragged last one, one to three rounds of pairs.
BACKWARDS = [
    (16, 5, 6, 520, BF16, BF16, 0), (16, 0, 9, 1032, F16, F16, 8), (16, 3, 4, 520, F32, F32, 0), (16, 1, 8, 1032, F32, BF16, 0),
    (16, 7, 3, 4104, F32, F16, 0), (16, 2, 5, 130, BF16, BF16, 0), (16, 9, 3, 1002, F16, F16, 2), (16, 4, 17, 1002, F32, BF16, 0),
    (16, 0, 6, 1001, BF16, BF16, 7), (16, 11, 2, 1001, F32, F32, 0),
    (15, 3, 6, 2056, BF16, BF16, 0), (2, 96, 9, 4104, F16, F16, 0), (2, 0, 4, 2056, BF16, BF16, 8),
    (1, 40, 8, 4104, BF16, BF16, 0), (0, 70, 9, 8200, F16, F16, 0), (2, 96, 6, 2056, F32, F32, 0), (1, 9, 5, 4104, F32, BF16, 0),
    (2, 96, 7, 1002, BF16, BF16, 0), (2, 95, 9, 1001, F32, F16, 1), (0, 33, 3, 2051, F16, F16, 0)]


@pytest.mark.parametrize("per_sm,more,k,H,rd,yd,wide", BACKWARDS)
def test_combine_rows_backward(per_sm, more, k, H, rd, yd, wide):
    M = load_lib()
    T = per_sm * sms() + more
    g = torch.Generator(device="cuda").manual_seed(T + k + H)
    off, pos, _ = sorted_on_host(routing(g, T, k, 64, 0.1).cpu().numpy(), 64)
    n = int(off[-1])
    rows, dy, w = normal(g, T * k, H, dtype=rd, wide=wide), normal(g, T, H, dtype=yd, wide=wide), normal(g, T, k)
    rows[n:] = float("nan")                                       # rows that no pair names
    p = torch.from_numpy(pos).cuda()
    d_rows = torch.full((T * k, H), 3.0, dtype=rd, device="cuda")
    _, d_w = M.moe_combine_rows_backward(dy, rows, p.to(torch.int32), w, d_rows=d_rows)
    assert (d_rows[n:] == 3).all()
    want = torch.zeros(n, H, dtype=torch.float64, device="cuda")
    for j in range(k):
        on = p[:, j] >= 0
        at, d = p[on, j], dy[on].double()
        want[at] = d * w[on, j, None].double()
        terms = d * rows[at].double()
        # a thread's share of a row one after the other, then the threads' sums: at most H / 32 + 8 + 16 additions deep
        assert ((d_w[on, j].double() - terms.sum(1)).abs() <= (H / 32 + 24) * 2.0 ** -24 * terms.abs().sum(1)).all()
        assert (d_w[~on, j] == 0).all()
    tol = (half(rd) + 2.0 ** -24) * (1 + 2.0 ** -20) * want.abs() + tiny(rd)
    assert ((d_rows[:n].double() - want).abs() <= tol).all()
    again, none = M.moe_combine_rows_backward(dy, rows, p.to(torch.int32), w, d_rows=torch.full_like(d_rows, 3.0), want_d_w=False)
    assert none is None and torch.equal(again, d_rows)
    _, d_w2 = M.moe_combine_rows_backward(dy, rows, p.to(torch.int32), w, d_rows=rows)      # in place
    assert torch.equal(rows[:n], d_rows[:n]) and torch.equal(d_w2, d_w)


# T, k, E, H, dtype, columns between rows: more than 4096 pairs (or narrow rows), rows of several blocks with a ragged last one,
# in vectors of 16, 4 and 2 bytes
SORTS = [(700, 6, 64, 8200, BF16, 0), (500, 9, 300, 4100, F32, 0), (2100, 2, 8, 12304, F16, 8), (1400, 3, 40, 2049, F32, 0),
         (900, 5, 1500, 4102, BF16, 2), (600, 7, 16, 2051, F16, 1), (4200, 1, 5, 6151, BF16, 0), (1030, 4, 256, 8192, BF16, 0)]


@pytest.mark.parametrize("T,k,E,H,dtype,wide", SORTS)
def test_sort_rows_of_several_blocks_each(T, k, E, H, dtype, wide):
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(T + H)
    # whole numbers that tell neighbouring columns and tokens apart, exact in every type
    x = ((torch.arange(H + wide, device="cuda") + 7 * torch.arange(T, device="cuda")[:, None]) % 251).to(dtype)[:, :H]
    ids = routing(g, T, k, E, 0.1)
    rows = torch.full((T * k, H + wide), -5.0, dtype=dtype, device="cuda")[:, :H]
    _, offsets, pos = M.moe_sort_rows(x, ids, E, rows=rows)
    off, want, order = sorted_on_host(ids.cpu().numpy(), E)
    n = int(off[-1])
    assert (offsets.cpu().numpy() == off).all() and (pos.cpu().numpy() == want).all()
    assert torch.equal(rows[:n], x[torch.from_numpy(order // k).cuda()]) and (rows[n:] == -5).all()
    if wide:
        assert (rows.as_strided((T * k, wide), (H + wide, 1), H) == -5).all()                # between the rows
    back = M.moe_sort_rows_backward(rows, pos)
    count = (pos >= 0).sum(1, keepdim=True).double()
    sums = x.double() * count                                      # at most 9 * 250: exact in fp32
    assert torch.equal(back, sums.to(dtype))
