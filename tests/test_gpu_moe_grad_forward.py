"""The gradients of the MoE steps against the library's own forward steps, by differences; and at sizes that only 64-bit
positions reach."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_bf16_gb300 as m
    torch.cuda.set_device(0)
    yield m
    m.check_status()


def bf(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("topk", [1, 4, 9])
def test_gradients_are_the_differences_of_the_forward_steps(nv, topk):
    """On whole numbers (at most 9 slots of 3 * 4, and the differences' one more: exact in bf16) the gradients of
    <dout, moe_combine(y, w)> and <dxs, moe_gather_rows(x)> equal their differences to the bit."""
    r = np.random.default_rng(topk)
    tokens, h, experts = 40, 64, 11
    ids = torch.from_numpy(np.stack([r.permutation(experts)[:topk] for _ in range(tokens)]).astype(np.int32)).cuda()
    ro, src, pos = nv.moe_sort_by_expert(ids, experts)
    x, y, dout = (bf(r.integers(-4, 5, s)) for s in ((tokens, h), (tokens * topk, h), (tokens, h)))
    w = torch.from_numpy(r.integers(1, 4, (tokens, topk)).astype(np.float32)).cuda()
    dropped = pos.clone()
    dropped[::7, topk - 1] = -1                             # slots that the sort leaves out

    def combined(y_, w_):
        return float((nv.moe_combine(y_, dropped, w_).double() * dout.double()).sum())

    dy = torch.zeros_like(y)
    _, dw = nv.moe_combine_backward(dout, y, dropped, w, dy=dy)
    base = combined(y, w)
    assert base == float((dy.double() * y.double()).sum()) == float((dw.double() * w.double()).sum())
    for _ in range(20):
        t, j, c = int(r.integers(tokens)), int(r.integers(topk)), int(r.integers(h))
        row = int(pos[t, j])
        y2, w2 = y.clone(), w.clone()
        y2[row, c] += 1
        w2[t, j] += 1
        assert combined(y2, w) - base == float(dy[row, c]) and combined(y, w2) - base == float(dw[t, j])

    def gathered(x_):
        return float((nv.moe_gather_rows(x_, src).double() * y.double()).sum())

    dx = nv.moe_gather_backward(y, pos)
    base = gathered(x)
    for _ in range(20):
        t, c = int(r.integers(tokens)), int(r.integers(h))
        x2 = x.clone()
        x2[t, c] += 1
        assert gathered(x2) - base == float(dx[t, c])
    nv.check_status()


def test_gather_backward_past_32_bit_positions(nv):
    """2^31 pieces of 8 channels: the form that counts them in 64 bits."""
    tokens, h, rows = 1 << 20, 1 << 14, 64
    if torch.cuda.mem_get_info()[0] < 40 * 2 ** 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device="cuda").manual_seed(1)
    dxs = torch.randint(-64, 65, (rows, h), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(-1, rows, (tokens, 2), generator=g, device="cuda", dtype=torch.int32)
    dx = nv.moe_gather_backward(dxs, pos)
    padded = torch.cat((dxs, torch.zeros_like(dxs[:1])))     # row -1
    for t in range(0, tokens, 1 << 15):
        p = pos[t: t + (1 << 15)].long()
        assert torch.equal(dx[t: t + (1 << 15)], padded[p[:, 0]] + padded[p[:, 1]])
    nv.check_status()
