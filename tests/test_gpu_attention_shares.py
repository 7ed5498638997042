"""spec_paged_attention where workgroups go on from one unit (sequence, key head, row tile) to the
next: books, buffers, codes and partial tiles left by one segment must not reach the following one.

`Cut` is a copy in Python of how the device cuts a batch.  Each case asserts from it that shares do
run on (a change of the grid must not make the test empty), and that the copy's grid and row tile
are the library's: the workspace's size has both in it."""
import numpy as np
import pytest

import cache_ref as ref
from test_gpu_attention import Case, check

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_02_amd as sv
    sv.load_library()
    return torch.device("cuda:0")


def ceil(a, b):
    return -(-a // b)


class Cut:
    TILE, CUS, XCDS, TRY = 32, 256, 8, 4

    def __init__(self, B, N, Hkv, group, D, esz, page, W, lens, news, tree, window, sinks, refused=()):
        rows = N * group
        two = D <= 128
        self.wide = rows > (32 if two else 16)
        self.R = (1 if rows <= 64 or D * esz == 1024 else 2) if self.wide else (1 if rows <= 16 else 2)
        self.RT = 16 * self.R * (4 if self.wide else 1)
        self.n_rt = ceil(rows, self.RT)
        self.units = B * Hkv * self.n_rt
        if self.wide:
            occ = 2 if self.R * D * esz <= 512 else 1
            self.round = 2 if D * esz <= 256 else 1
        else:
            occ = 3 if self.R * D * esz <= 128 else 2 if D * esz <= 256 or (D * esz <= 512 and self.R == 1) else 1
            self.round = 4
        most_tiles = ceil(W * page, self.TILE) + 1
        self.grid = ceil(min(self.CUS * occ, self.units * ceil(most_tiles, self.round)), self.XCDS) * self.XCDS
        self.D = D
        # rounds of every unit, in the device's order
        r = []
        for b in range(B):
            per = []
            for rt in range(self.n_rt):
                i0, i1 = rt * self.RT // group, min(news[b] - 1, (rt * self.RT + self.RT - 1) // group)
                tiles = 1
                if b not in refused and i0 <= i1:
                    end, first, n_sink = lens[b] + (news[b] if tree else i1 + 1), 0, 0
                    if window:
                        first = max(0, lens[b] + ((i0 > 0) if tree else i0) - window + 1) // self.TILE
                        n_sink = min(ceil(sinks, self.TILE), first)
                    tiles = n_sink + ceil(end, self.TILE) - first
                per.append(ceil(tiles, self.round))
            r += per * Hkv
        least = max(1, self.RT * 4 // (self.round * self.TILE * esz))
        total = sum(r)
        share, most = ceil(total, self.grid), 1
        if self.units <= self.grid and W * page < 1 << 27:
            if share > 1:
                for k in range(self.TRY if self.wide else min(1 + share // 16, self.TRY)):
                    if sum(ceil(x, max(share + k, least)) for x in r) <= self.grid:
                        most = max(share + k, least)
                        break
                if most > 1:
                    share = 1
            elif least > 1:
                most = least
        self.share, self.most = share, most
        parts = [ceil(x, most) for x in r]
        ends = np.cumsum(parts)
        starts = ends - parts
        first_wg, last_wg = starts // share, (ends - 1) // share
        self.joined = int((last_wg > first_wg).sum())  # units that several workgroups stream
        count = np.zeros(ceil(int(ends[-1]), share), int)
        for f, l in zip(first_wg, last_wg):
            count[f:l + 1] += 1
        self.go_on = int((count > 1).sum())  # workgroups with several units

    def workspace(self):
        up = lambda x: ceil(x, 256) * 256  # noqa: E731
        return up(2 * self.grid * self.RT * self.D * 4) + up(2 * self.grid * self.RT * 8) + up(self.units * 16)


def cut_of(c, refused=()):
    return Cut(c.B, c.N, c.H, c.g, c.D, c.esz, c.page, c.table.shape[1], c.lens, c.news, c.parents is not None, c.window, c.sinks, refused)


def part_of(c, some):
    p = Case.__new__(Case)
    p.__dict__.update(c.__dict__)
    p.B, p.q, p.lens, p.news = len(some), c.q[some], [c.lens[b] for b in some], [c.news[b] for b in some]
    p.ks, p.vs = [c.ks[b] for b in some], [c.vs[b] for b in some]
    p.parents = c.parents[some] if c.parents is not None else None
    return p


CASES = {  # dtype, B, N, Hkv, group, D, page, longest, tree, window, sinks, wide
    "wide bf16 64, trees": ("bf16", 160, 20, 4, 4, 64, 16, 150, True, 0, 0, True),
    "wide bf16 64, trees in a window": ("bf16", 160, 20, 4, 4, 64, 32, 150, True, 25, 5, True),
    "wide bf16 64, chains in a window": ("bf16", 160, 20, 4, 4, 64, 16, 150, False, 25, 40, True),
    "wide bf16 64, one row tile a wave": ("bf16", 180, 16, 3, 4, 64, 64, 300, True, 0, 0, True),
    "wide bf16 64, several row tiles": ("bf16", 90, 70, 2, 4, 64, 16, 90, True, 0, 0, True),
    "wide bf16 128": ("bf16", 140, 24, 4, 4, 128, 16, 100, True, 0, 0, True),
    "wide bf16 256": ("bf16", 150, 20, 2, 4, 256, 16, 120, True, 0, 0, True),
    "wide bf16 256, one row tile a wave": ("bf16", 280, 9, 2, 4, 256, 16, 60, True, 50, 3, True),
    "wide f32 64": ("f32", 140, 20, 4, 4, 64, 16, 100, True, 0, 0, True),
    "wide f32 128": ("f32", 140, 9, 2, 8, 128, 16, 100, True, 33, 2, True),
    "wide f32 256": ("f32", 150, 20, 2, 1, 256, 16, 90, True, 0, 0, True),
    "few bf16 64, trees": ("bf16", 210, 4, 4, 2, 64, 16, 400, True, 0, 0, False),
    "few bf16 64, trees in a window": ("bf16", 210, 5, 4, 2, 64, 16, 400, True, 300, 20, False),
    "few bf16 128, two row tiles": ("bf16", 140, 8, 4, 4, 128, 32, 300, True, 0, 0, False),
    "few bf16 256": ("bf16", 270, 3, 2, 4, 256, 16, 200, True, 0, 0, False),
    "few f32 64": ("f32", 160, 4, 4, 4, 64, 16, 300, True, 0, 0, False),
    "few f32 128, two row tiles": ("f32", 140, 8, 2, 4, 128, 16, 200, False, 350, 7, False),
    "few f32 256": ("f32", 140, 4, 2, 4, 256, 16, 200, True, 0, 0, False),
}


def batch(dev, name):
    dtype, B, N, H, g, D, page, longest, tree, window, sinks, wide = CASES[name]
    rng = np.random.default_rng(len(name))
    lens = [int(x) for x in rng.integers(0, longest + 1, B)]
    lens[4::9] = [6 * longest + x for x in lens[4::9]]
    news = [int(x) for x in rng.integers(0, N + 1, B)]
    news[::5] = [N] * len(news[::5])
    news[7::20] = [0] * len(news[7::20])
    return Case(dev, dtype, B, N, H, g, D, page, lens, news=news, tree=tree, window=window, sinks=sinks, seed=len(name)), wide


@pytest.mark.parametrize("name", CASES)
def test_the_cases_run_on(name):
    """From the sizes alone, without a GPU: many workgroups have several units, and some units are
    joined from several workgroups."""
    import rejection_sampling_verify_02_amd as sv
    if not sv.LIB_PATH.exists():
        from rejection_sampling_verify_02_amd import build
        build.build()
    c, wide = batch("cpu", name)
    k = cut_of(c)
    assert k.wide == wide and k.units > k.grid and k.share > 1
    assert k.go_on > k.grid // 4 and k.joined > 10
    dt = sv.SV_BF16 if c.esz == 2 else sv.SV_F32
    assert k.workspace() == sv.sv_attention_workspace_bytes(c.B, c.N, c.H * c.g, c.H, c.D, c.page, c.table.shape[1], dt)


@gpu
@pytest.mark.parametrize("name", CASES)
def test_shares_that_go_on(dev, name):
    """Mixed lengths and counts (none among them), codes of every kind between sequences that are
    in order, and values that are not finite in some: each sequence's rows are its own."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    c, _ = batch(dev, name)
    t = c.tensors()
    before, st = sv.spec_paged_attention(**t)
    assert st.tolist() == [0] * c.B

    # a value that is not finite in the last new token of some sequences: in a tree few nodes see it
    odd = [b for b in range(3, c.B, 11) if c.news[b] > 1]
    for x, b in zip([np.nan, np.inf, -np.inf] * len(odd), odd):
        at = c.lens[b] + c.news[b] - 1
        c.vs[b][:, at, 5] = x
        ref.pack_v(c.vs[b][:, at], at, c.vp, c.table[b], c.page, c.E)
    t = c.tensors()
    # codes, each kind in several places
    whole = [b for b in range(c.B) if c.news[b] == c.N and b not in odd]
    kinds = ["length", "count", "page", "prior"] + (["tree"] if c.parents is not None else [])
    bad = {b: kinds[i % len(kinds)] for i, b in enumerate(whole[::2])}
    prior = torch.zeros(c.B, dtype=torch.int32, device=dev)
    for b, kind in bad.items():
        if kind == "length":
            t["cache_len"][b] = -1
        elif kind == "count":
            t["n_new"][b] = c.N + 1
        elif kind == "page":
            t["page_table"][b, (c.lens[b] + c.N - 1) // c.page] = t["k_pages"].shape[0] if b % 2 else -1
        elif kind == "prior":
            prior[b] = -9
        else:
            t["parent"][b, c.N - 1] = c.N - 1
    refused = {b for b, kind in bad.items() if kind in ("length", "count", "prior")}
    k = cut_of(c, refused)
    assert k.share > 1 and k.go_on > k.grid // 4
    codes = {"length": -8, "count": -8, "page": -7, "prior": -9, "tree": -6}
    out, st = sv.spec_paged_attention(**t, prior=prior)
    assert st.tolist() == [codes[bad[b]] if b in bad else 0 for b in range(c.B)]
    assert torch.isnan(out[list(bad)]).all()
    again, _ = sv.spec_paged_attention(**t, prior=prior)
    assert torch.equal(out.nan_to_num(77.0), again.nan_to_num(77.0))

    # the float64 reference for the sequences around codes and values that are not finite, and some others
    good = [b for b in range(c.B) if b not in bad]
    near = {x for b in [*list(bad)[:6], *odd[:6]] for x in (b - 1, b, b + 1)} | set(range(0, c.B, 17)) | {c.B - 1, c.B - 2}
    some = [b for b in good if b in near]
    check(part_of(c, some), out[some], st[some])
    # all the others: what they were in the batch without codes, which was cut otherwise.  Both are
    # off by at most cache_ref's allowance; here with sum p |v| <= max |v| and, by Cauchy and
    # Schwarz, sum |q k| <= |q| |k|, over the sequence.
    u, w = 2.0 ** -24, (2.0 ** -8 if c.esz == 2 else 2.0 ** -24)
    a, p = out.double().cpu().numpy(), before.double().cpu().numpy()
    for b in good:
        if b in odd or not c.news[b]:
            continue
        T = c.lens[b] + c.news[b]
        dz = (c.D + 4) * u * c.scale * np.linalg.norm(c.q[b], axis=-1).max() * np.linalg.norm(c.ks[b], axis=-1).max()
        A, f = np.abs(c.vs[b]).max(), 2.2 * dz + w + (2 * (T + 8) + T / 16 + 8) * u
        assert (np.abs(a[b] - p[b]) <= 2 * (f * A + w * (np.abs(p[b]) + 2 * f * A))).all(), b


@gpu
@pytest.mark.parametrize("dtype,N,g,D,n", [("bf16", 20, 4, 64, 640), ("bf16", 20, 4, 256, 330), ("f32", 20, 4, 64, 640),
                                           ("bf16", 1, 4, 64, 1900), ("f32", 4, 2, 256, 700)])
def test_fewer_units_than_workgroups_that_no_even_cut_fits(dev, dtype, N, g, D, n):
    """Units of equal length, 0.58 of the grid: two parts each are too many for it, one is far more
    than an equal share, so the shares run on."""
    import rejection_sampling_verify_02_amd as sv
    esz = 2 if dtype == "bf16" else 4
    grid = Cut(8192, N, 1, g, D, esz, 64, ceil(n + N, 64) + 2, [n] * 8192, [N] * 8192, False, 0, 0).grid
    H = 4
    B = round(0.58 * grid / H)
    c = Case(dev, dtype, B, N, H, g, D, 64, [n] * B, tree=N > 1, seed=n + D)
    k = cut_of(c)
    assert k.units <= k.grid == grid and k.share > 1 and k.most == 1 and k.go_on and k.joined
    assert k.workspace() == sv.sv_attention_workspace_bytes(B, N, H * g, H, D, 64, c.table.shape[1], sv.SV_BF16 if esz == 2 else sv.SV_F32)
    out, st = sv.spec_paged_attention(**c.tensors())
    some = sorted({0, 1, B // 3, B // 2, B - 2, B - 1})
    check(part_of(c, some), out[some], st[some])
