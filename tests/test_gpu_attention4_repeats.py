"""Attention over a cache in 4 bits gives the same bits again, whatever its workspace, the row codes
and the output held before, for every way that a batch is cut: one part a unit, several, and shares
that run on from unit to unit."""
import pytest

from test_gpu_attention import dev  # noqa: F401  (a fixture)
from test_gpu_attention4 import Case4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,N,Hkv,group,D,page,lens,kw", [
    (1, 1, 8, 4, 128, 16, [1009], {}),
    (24, 1, 8, 4, 128, 64, [40 + 97 * i for i in range(24)], {}),
    (9, 5, 4, 4, 128, 64, [3000 - 311 * i for i in range(9)], {}),
    (6, 32, 4, 4, 128, 32, [700 + 333 * i for i in range(6)], dict(tree=True)),
    (5, 3, 2, 8, 256, 16, [17, 900, 2200, 64, 1], {}),
    (40, 2, 4, 2, 64, 16, [11 * i for i in range(40)], dict(window=150, sinks=4)),
])
def test_same_bits(dev, B, N, Hkv, group, D, page, lens, kw):  # noqa: F811
    import torch
    import rejection_sampling_verify_02_amd as sv
    t = Case4(dev, B, N, Hkv, group, D, page, lens, **kw).tensors()
    W = t["page_table"].shape[1]
    n = sv.sv_attention4_workspace_bytes(B, N, Hkv * group, Hkv, D, page, W)
    got = []
    for fill in (0, 255, 127, None):
        ws = torch.randint(0, 256, (n,), dtype=torch.uint8, device=dev) if fill is None else torch.full((n,), fill, dtype=torch.uint8, device=dev)
        out = (torch.full_like(t["q"], float("nan")), torch.full((B,), 77, dtype=torch.int32, device=dev))
        sv.spec_paged_attention(**t, workspace=ws, out=out)
        got.append((out[0].view(torch.int16).clone(), out[1].clone()))
    for o, st in got:
        assert not st.any() and torch.equal(o, got[0][0])
    assert not torch.isnan(got[0][0].view(torch.bfloat16)).any()
