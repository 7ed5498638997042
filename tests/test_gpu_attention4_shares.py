"""spec_paged_attention over a cache in 4 bits where workgroups go on from one unit (sequence, key
head, row tile) to the next.  A unit's start counts as some rounds of work there, so that shares may
also end or begin within it and hold none of the unit's slots.

`Cut4` is a copy in Python of how the device cuts a batch of more units than workgroups."""
import numpy as np
import pytest

from test_gpu_attention import check, dev  # noqa: F401  (a fixture)
from test_gpu_attention4 import Case4
from test_gpu_attention_shares import ceil, part_of

gpu = pytest.mark.gpu


class Cut4:
    def __init__(self, B, N, H, g, D, page, lens, news, tree):
        rows = N * g
        self.W = 2 + max(ceil(n + m, page) for n, m in zip(lens, news))  # as Case has it
        self.wide = rows > (32 if D <= 128 else 16)
        R = (1 if rows <= 64 else 2) if self.wide else (1 if rows <= 16 else 2)
        self.RT = 16 * R * (4 if self.wide else 1)
        self.n_rt = ceil(rows, self.RT)
        self.units = B * H * self.n_rt
        if self.wide:
            occ, self.round, lead = (2 if R * D <= 256 else 1), (2 if D <= 128 else 1), 3
        else:
            occ, self.round, lead = (2 if D > 64 else 4 if R == 1 else 3), 4, 5
        most = ceil(self.W * page, 32) + 1
        self.grid = ceil(min(256 * occ, self.units * ceil(most, self.round)), 8) * 8
        self.D = D
        rounds = []
        for b in range(B):
            per = []
            for rt in range(self.n_rt):
                i0, i1 = rt * self.RT // g, min(news[b] - 1, (rt * self.RT + self.RT - 1) // g)
                per.append(ceil(ceil(lens[b] + (news[b] if tree else i1 + 1), 32) if i0 <= i1 else 1, self.round))
            rounds += per * H
        self.runs = ceil(sum(rounds), self.grid) > 1
        parts = np.array(rounds) + lead
        self.share = ceil(int(parts.sum()), self.grid)
        ends = np.cumsum(parts)
        starts = ends - parts
        self.joined = int(((ends - 1) // self.share > starts // self.share).sum())
        cuts = np.arange(self.share, int(ends[-1]), self.share)
        unit = np.searchsorted(ends, cuts, side="right")
        self.in_lead = int(((cuts > starts[unit]) & (cuts <= starts[unit] + lead)).sum())  # shares that end before a unit's first round

    def workspace(self):
        up = lambda x: ceil(x, 256) * 256  # noqa: E731
        return up(2 * self.grid * self.RT * self.D * 4) + up(2 * self.grid * self.RT * 8) + up(self.units * 16)


CASES = {  # B, N, Hkv, group, D, page, longest, tree
    "few rows, 64": (280, 1, 4, 4, 64, 16, 500, False),
    "two row tiles, 64": (210, 5, 4, 4, 64, 32, 450, True),
    "few rows, 128": (140, 2, 4, 4, 128, 16, 500, True),
    "two row tiles, 128": (140, 7, 4, 4, 128, 32, 400, False),
    "few rows, 256": (270, 1, 2, 4, 256, 16, 400, False),
    "many rows, 64": (140, 12, 4, 4, 64, 16, 250, True),
    "many rows, two row tiles a wave, 64": (140, 20, 4, 4, 64, 16, 250, True),
    "many rows, 128": (140, 20, 4, 4, 128, 32, 250, True),
    "many rows, 256": (140, 9, 4, 4, 256, 16, 100, False),
    "many rows, two row tiles a wave, 256": (150, 20, 2, 4, 256, 16, 120, True),
}


def sizes(name):
    B, N, H, g, D, page, longest, tree = CASES[name]
    rng = np.random.default_rng(len(name))
    lens = [int(x) for x in rng.integers(0, longest + 1, B)]
    lens[4::9] = [4 * longest + x for x in lens[4::9]]
    news = [int(x) for x in rng.integers(0, N + 1, B)]
    news[::3] = [N] * len(news[::3])
    return B, N, H, g, D, page, lens, news, tree


@pytest.mark.parametrize("name", CASES)
def test_the_cases_run_on(name):
    import rejection_sampling_verify_02_amd as sv
    if not sv.LIB_PATH.exists():
        from rejection_sampling_verify_02_amd import build
        build.build()
    B, N, H, g, D, page, *_ = sizes(name)
    k = Cut4(*sizes(name))
    assert k.units > k.grid and k.runs and k.joined > 10 and k.in_lead > 10
    assert k.workspace() == sv.sv_attention4_workspace_bytes(B, N, H * g, H, D, page, k.W)


@gpu
@pytest.mark.parametrize("name", CASES)
def test_shares_that_go_on(dev, name):  # noqa: F811
    """Every row of the batch, with blocks that are not finite in some sequences and refused sequences between."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    *shape, lens, news, tree = sizes(name)
    c = Case4(dev, *shape, lens, news=news, tree=tree, seed=len(name))
    assert c.table.shape[1] == Cut4(*sizes(name)).W
    for b in range(3, c.B, 11):
        if c.news[b]:
            c.spoil(1, b, c.lens[b] + c.news[b] - 1, 1)
    t = c.tensors()
    bad = {b: i % 3 for i, b in enumerate(range(0, c.B, 6))}
    prior = torch.zeros(c.B, dtype=torch.int32, device=dev)
    for b, kind in bad.items():
        if kind == 0:
            t["cache_len"][b] = -1
        elif kind == 1:
            t["page_table"][b, 0] = t["k_pages"].scales.shape[0]
        else:
            prior[b] = -9
    codes = (-8, -7, -9)
    out, st = sv.spec_paged_attention(**t, prior=prior)
    assert st.tolist() == [(0 if bad[b] == 1 and c.lens[b] + c.news[b] == 0 else codes[bad[b]]) if b in bad else 0 for b in range(c.B)]
    again, _ = sv.spec_paged_attention(**t, prior=prior)
    assert torch.equal(out.nan_to_num(77.0), again.nan_to_num(77.0))
    good = [b for b in range(c.B) if b not in bad]
    near = {x for b in list(bad)[::3] for x in (b - 1, b + 1)} | set(range(3, c.B, 22)) | {c.B - 1, c.B - 2}
    some = [b for b in good if b in near]
    check(part_of(c, some), out[some], st[some])
