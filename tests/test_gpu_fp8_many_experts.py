"""The quantiser with more experts than its CTAs have threads: it looks for a block's expert 256 at a time."""
import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [[1] * 257, [0] * 256 + [130], [2, 0, 129] * 100, [0] * 700 + [5, 128] + [0] * 322, [1, 0] * 512])
def test_quantize(counts):
    import nvfp4_block_scaled_bf16_gb300 as nv
    torch.cuda.set_device(0)
    r = np.random.default_rng(len(counts))
    ro = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    x = torch.from_numpy(r.standard_normal((50, 48)).astype(np.float32)).to(torch.bfloat16).cuda()
    idx = r.integers(0, 50, int(ro[-1])).astype(np.int32)
    xn = x.float().cpu().numpy()[idx]
    got = nv.fp8_quantize(x, src_rows=torch.from_numpy(idx).cuda(), row_offsets=torch.from_numpy(ro).cuda(), transpose=True)
    want = ofp8.quantize_rows(xn) + ofp8.quantize_columns(xn, ro)
    for g, v in zip(got, want):
        g = g.view(torch.uint8) if g.dtype == torch.float8_e4m3fn else g
        assert np.array_equal(g.cpu().numpy(), v)
    nv.check_status()
    bad = ro.copy()
    bad[len(counts) // 2 + 100] = ro[-1] + 1                # found among the later ones too
    qt, _ = nv.fp8_quantize(x, src_rows=torch.from_numpy(idx).cuda(), row_offsets=torch.from_numpy(bad).cuda(), rows=False, transpose=True)
    assert bool((qt.view(torch.uint8) == 0).all())
    with pytest.raises(nv.NVFP4Error):
        nv.check_status()
