"""Turned queries, and turned keys in the cache, bit for bit: the rotation in 64 bits, rounded once.
The kernel's cosines and sines are within 2^-51 of the reference's (a unit in the last place of
either, and of the rotation's products), so that what is rounded lies within 2^-50 of |x| + |y| of the
reference's: both ends of that are rounded, and the output is what one of them gives, or between."""
import numpy as np
import pytest

import step_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_02_amd as sv
    sv.load_library()
    return torch.device("cuda:0")


def rounded(x, dt):
    """float64 values to the nearest of dt: for bf16 over float32 with the last bit set where that is not exact."""
    import torch
    y = x.astype(np.float32)
    if dt == torch.bfloat16:
        w = y.view(np.uint32)
        w += ((y != x) & (w & 1 == 0)) * np.where(np.abs(x) > np.abs(y), 1, -1).astype(np.int32).view(np.uint32)
    return torch.from_numpy(y).to(dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rounded_once(dev, dtype, interleaved):
    import torch
    import rejection_sampling_verify_02_amd as sv
    B, N, Hq, Hkv, D, page = 8, 256, 8, 4, 128, 64
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(31)
    q, k, v = (torch.randn((B, N, H, D), generator=g).to(dt) for H in (Hq, Hkv, Hkv))
    rot = sv.Rotary.of(D, 500000.0, interleaved=interleaved, device=dev)
    lens = torch.tensor([0, 1, 7, 100, 1000, 30, 64, 511], dtype=torch.int32)
    W = (1000 + N + page - 1) // page + 1
    table = torch.arange(B * W, dtype=torch.int32).view(B, W)
    kp, vp = sv.empty_pages(1, B * W, Hkv, D, page, dt, dev)
    qo, st = sv.spec_cache_append_rotary(q.to(dev), k.to(dev), v.to(dev), kp[0], vp[0], table.to(dev), lens.to(dev), rot)
    ko, _, _ = sv.spec_cache_read(kp[0], vp[0], table.to(dev), lens.to(dev), N)
    assert not st.any()
    pos = lens.numpy()[:, None] + np.arange(N)
    for x, y in ((q, qo), (k, ko)):
        want, size = step_ref.turn(x.double().numpy(), pos, rot.inv_freq.cpu().numpy(), interleaved, 1.0)
        ends = [rounded(want + s * 2.0 ** -50 * size, dt) for s in (-1, 1)]
        y = y.cpu()
        assert ((ends[0] <= y) & (y <= ends[1])).all()
        assert (ends[0] == ends[1]).float().mean() > 0.999  # sure nearly everywhere
