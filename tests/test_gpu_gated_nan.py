"""A product that is not a number stays one in every gradient of the gated product that depends on it."""
import pytest
import torch

from cases import dev, nvfp4_operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_bf16_gb300 as m
    return m


# whole and split weight-streaming tiles, CTA pairs, 128 x 128 tiles, stream-K
@pytest.mark.parametrize("m,inter,k", [(3, 16, 4096), (16, 512, 1024), (64, 784, 2080), (40, 10240, 320), (300, 6528, 512),
                                       (640, 512, 2048), (300, 512, 16384)])
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_nan_products(nv, m, inter, k, kind):
    ops = nvfp4_operands(m, 2 * inter, k, 1)
    args = (dev(ops["qa"]), dev(ops["sfa"]), dev(ops["qb"]), dev(ops["sfb"]))
    a = float(ops["alpha"])
    dh = torch.ones(m, inter, dtype=torch.bfloat16, device="cuda")

    def backward(gate_alpha, up_alpha):
        alpha = torch.tensor([gate_alpha, up_alpha], device="cuda")
        dgu, h = nv.nvfp4_gated_gemm_backward(*args, alpha, dh, activation=kind)
        assert torch.equal(torch.isnan(nv.nvfp4_gated_gemm(*args, alpha, activation=kind)), torch.isnan(h))
        nv.check_status()
        v = dgu.view(m, -1, 2, 16)
        return torch.isnan(v[:, :, 0]), torch.isnan(v[:, :, 1]), torch.isnan(h)

    dg, du, h = backward(float("nan"), a)      # dg = dh u act'(g), du = dh act(g), h = act(g) u
    assert dg.all() and du.all() and h.all()
    dg, du, h = backward(a, float("nan"))
    assert dg.all() and not du.any() and h.all()
