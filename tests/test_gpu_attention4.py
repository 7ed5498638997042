"""spec_paged_attention over a cache in 4 bits against the float64 reference of the other types
(tests/cache_ref.py), on the values that the codes stand for: they are bf16 numbers, so that the
reference's allowance for bf16 inputs holds as it is."""
import numpy as np
import pytest

import step_ref
from test_gpu_attention import Case, check, dev  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


class Case4(Case):
    """Case with its cache in 4 bits; unused slots hold any codes, in blocks that are NaN."""

    def __init__(self, dev, B, N, Hkv, group, D, page, lens, **kw):  # noqa: F811
        super().__init__(dev, "bf16", B, N, Hkv, group, D, page, lens, **kw)
        rng = np.random.default_rng(kw.get("seed", 0) + 1)
        P = self.kp.shape[0]
        self.pools = [step_ref.Pool4(rng, P, Hkv, page, D) for _ in range(2)]
        for p in self.pools:
            p.byte[:] = 255
        counts = [-(-(n + m) // page) for n, m in zip(self.lens, self.news)]
        self.ids = np.zeros((B, max(1, max(counts))), np.int64)
        used = iter(np.random.default_rng(kw.get("seed", 0) + 2).permutation(P))
        self.table = np.full_like(self.table, -1)
        for b in range(B):
            self.ids[b, :counts[b]] = [next(used) for _ in range(counts[b])]
            self.table[b, :counts[b]] = self.ids[b, :counts[b]]
            for x, p in ((self.ks, self.pools[0]), (self.vs, self.pools[1])):
                code, byte = step_ref.encode(x[b].astype(np.float32))
                x[b] = step_ref.decode(code, byte)
                for t in range(x[b].shape[1]):
                    p.set((code[:, t], byte[:, t]), t, self.ids[b])
            if self.window and kw.get("evict", True):
                first = max(0, self.lens[b] - self.window + 1)
                for i in range(counts[b]):
                    if (i + 1) * page <= first and i * page >= self.sinks:
                        self.table[b, i] = -1

    def spoil(self, which, b, t, block):
        """Block `block` of every head of slot t is not finite."""
        p, page = self.pools[which], self.page
        p.byte[self.ids[b, t // page], :, t % page, block] = 255
        (self.ks, self.vs)[which][b][:, t, 32 * block:32 * block + 32] = np.nan

    def tensors(self):
        import torch
        import rejection_sampling_verify_02_amd as sv
        t = super().tensors()
        for name, p, values in (("k_pages", self.pools[0], False), ("v_pages", self.pools[1], True)):
            t[name] = sv.Pages4(*(torch.from_numpy(x).to(self.dev) for x in p.arrays(values)))
        return t


def run(case):
    import rejection_sampling_verify_02_amd as sv
    return sv.spec_paged_attention(**case.tensors())


SHAPES = [  # B, N, Hkv, group, D, page, lens
    (1, 1, 1, 1, 64, 16, [0]),
    (1, 1, 1, 1, 64, 16, [1]),
    (3, 1, 2, 4, 128, 16, [15, 16, 17]),
    (4, 1, 2, 5, 64, 32, [31, 32, 33, 63]),
    (3, 5, 1, 3, 128, 64, [0, 60, 129]),
    (2, 2, 2, 8, 256, 16, [47, 100]),
    (2, 7, 1, 7, 64, 128, [127, 250]),
    (2, 16, 1, 8, 128, 16, [5, 70]),
    (1, 33, 2, 4, 64, 256, [40]),
    (2, 1, 1, 64, 128, 32, [33, 2]),
    (2, 3, 1, 16, 256, 32, [90, 31]),
    (2, 9, 2, 12, 256, 64, [130, 65]),
    (1, 1, 3, 2, 256, 128, [700]),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:6])))
def test_chain(dev, shape):  # noqa: F811
    B, N, Hkv, g, D, page, lens = shape
    c = Case4(dev, B, N, Hkv, g, D, page, lens, seed=sum(lens) + D)
    check(c, *run(c))


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (3, 2), (16, 0), (33, 1), (40, 50), (500, 4), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("g,D", [(2, 64), (8, 128)])
def test_window_and_sinks(dev, window, sinks, tree, g, D):  # noqa: F811
    c = Case4(dev, 5, 9, 1, g, D, 16, [0, 3, 33, 90, 200], tree=tree, window=window, sinks=sinks, seed=window + sinks)
    check(c, *run(c))


@pytest.mark.parametrize("D,page,g", [(128, 32, 4), (256, 64, 4), (64, 64, 4), (256, 16, 1), (128, 16, 1)])
def test_trees_and_ragged_counts(dev, D, page, g):  # noqa: F811
    N = 40
    c = Case4(dev, 6, N, 1, g, D, page, [0, 1, 30, 31, 64, 77], news=[N, 0, 1, 17, 33, 39], tree=True, seed=D)
    check(c, *run(c))


def test_everything_empty(dev):  # noqa: F811
    c = Case4(dev, 3, 4, 2, 2, 64, 16, [0, 5, 0], news=[0, 0, 0])
    check(c, *run(c))


@pytest.mark.parametrize("Hkv,g,D,N", [(2, 4, 128, 2), (1, 2, 64, 2), (1, 16, 256, 1), (1, 8, 128, 3), (1, 20, 128, 5), (1, 20, 256, 5), (2, 9, 64, 5)])
def test_long_contexts_split_over_workgroups(dev, Hkv, g, D, N):  # noqa: F811
    c = Case4(dev, 6, N, Hkv, g, D, 64, [6000, 1, 40, 2500, 0, 333], seed=5)
    check(c, *run(c))


@pytest.mark.parametrize("N,g,D,window", [(24, 4, 128, 0), (12, 4, 64, 0), (40, 2, 256, 300), (20, 8, 128, 777)])
def test_long_contexts_with_many_rows(dev, N, g, D, window):  # noqa: F811
    c = Case4(dev, 3, N, 1, g, D, 32, [3500, 10, 1777], tree=True, window=window, sinks=40 if window else 0, seed=N)
    check(c, *run(c))


@pytest.mark.parametrize("N,g,lens", [(1, 4, [1100] * 40), (20, 4, [1100] * 40), (3, 1, list(range(0, 2000, 50))), (1, 2, [5] * 300 + [900])])
def test_every_way_to_cut_a_batch(dev, N, g, lens):  # noqa: F811
    """Equal lengths (a part a workgroup), lengths that no such cut fits, more units than workgroups."""
    H = 4 if len(lens) <= 40 else 2
    c = Case4(dev, len(lens), N, H, g, 64, 64, lens, seed=len(lens) + N)
    t = c.tensors()
    import rejection_sampling_verify_02_amd as sv
    out, st = sv.spec_paged_attention(**t)
    assert st.tolist() == [0] * c.B
    some = sorted({0, 1, c.B // 2, c.B - 1})
    part = Case4.__new__(Case4)
    part.__dict__.update(c.__dict__)
    part.B, part.q, part.lens, part.news = len(some), c.q[some], [c.lens[b] for b in some], [c.news[b] for b in some]
    part.ks, part.vs = [c.ks[b] for b in some], [c.vs[b] for b in some]
    check(part, out[some], st[some])
    again, _ = sv.spec_paged_attention(**t)
    assert (again == out).all()


def test_many_new_tokens(dev):  # noqa: F811
    c = Case4(dev, 1, 1024, 1, 1, 64, 64, [20], tree=True, seed=9)
    check(c, *run(c))


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales_and_strides(dev, scale):  # noqa: F811
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case4(dev, 3, 5, 2, 4, 64, 16, [10, 33, 2], seed=3)
    c.scale = scale
    t = c.tensors()
    wide = torch.full((3, 7, 8 + 4, 64), float("nan"), dtype=c.dt, device=dev)  # queries in a fused projection's rows
    wide[:, 1:6, :8] = t["q"]
    t["q"] = wide[:, 1:6, :8]
    check(c, *sv.spec_paged_attention(**t, scale=scale))


@pytest.mark.parametrize("g,D,N", [(2, 64, 12), (8, 64, 12), (6, 128, 12), (1, 256, 12), (8, 256, 12)])
def test_blocks_that_are_not_finite_reach_only_rows_that_see_them(dev, g, D, N):  # noqa: F811
    n = 37
    parents = np.array([[-1, 0, 0, 1, 1, 2, 2, 3, 5, 7, 8, 10]], np.int32)
    for window, which, slots in ((0, 1, [n + 3, n + 7]), (0, 1, [n + 2, n + 6]), (8, 1, [n - 7, n - 6]), (0, 0, [n + 3]), (0, 1, [3])):
        c = Case4(dev, 1, N, 1, g, D, 16, [n], tree=True, window=window, seed=21, evict=False)
        c.parents = parents
        for t in slots:
            c.spoil(which, 0, t, D // 32 - 1)
        check(c, *run(c))


def test_codes(dev):  # noqa: F811
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case4(dev, 9, 6, 2, 2, 64, 16, [40, 41, 42, 43, 44, 45, 300, 47, 12], tree=True, news=[6] * 9, seed=12)
    good, _ = sv.spec_paged_attention(**c.tensors())
    t = c.tensors()
    t["cache_len"][0] = -1
    t["n_new"][1] = 7
    t["cache_len"][2] = 100000
    t["parent"][3, 4] = 4
    t["parent"][4, 0] = 0
    t["page_table"][5, 2] = t["k_pages"].codes.shape[0]
    t["page_table"][6, 7] = -1
    t["prior"] = torch.tensor([0] * 8 + [-9], dtype=torch.int32, device=dev)
    out, st = sv.spec_paged_attention(**t)
    assert st.tolist() == [-8, -8, -8, -6, -6, -7, -7, 0, -9]
    assert torch.isnan(out[:7]).all() and torch.isnan(out[8]).all()
    assert torch.equal(out[7], good[7])


@pytest.mark.parametrize("N", [4, 30])
def test_streams_graphs_and_lengths_that_grow(dev, N):  # noqa: F811
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case4(dev, 3, N, 2, 4, 128, 16, [700, 30, 1], seed=15)
    t = c.tensors()
    plain, _ = sv.spec_paged_attention(**t)
    torch.cuda.synchronize(dev)
    side = torch.cuda.Stream(dev)
    got = [sv.spec_paged_attention(**t, stream=side.cuda_stream)[0] for _ in range(5)]
    torch.cuda.synchronize(dev)
    assert all(torch.equal(x, plain) for x in got)
    lens, full, short = t["cache_len"], t["cache_len"].clone(), torch.tensor([13, 29, 0], dtype=torch.int32, device=dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, st = sv.spec_paged_attention(**t)
    for want in (short, full, short, full):
        lens.copy_(want)
        out.fill_(-1)
        g.replay()
        eager, _ = sv.spec_paged_attention(**t)  # eager work between the replays
        torch.cuda.synchronize(dev)
        assert torch.equal(out, eager) and st.tolist() == [0, 0, 0]
    assert torch.equal(out, plain)


def test_pool_beyond_32_bit_offsets(dev):  # noqa: F811
    """Pages behind the first 4 GiB of codes."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case4(dev, 2, 1, 8, 1, 128, 64, [150, 64], seed=17)
    t = c.tensors()
    P = (9 << 29) // (8 * 64 * 64)
    used = t["k_pages"].codes.shape[0]
    for name in ("k_pages", "v_pages"):
        big = [torch.empty((P, *x.shape[1:]), dtype=torch.uint8, device=dev) for x in t[name]]
        for b, x in zip(big, t[name]):
            b[P - used:] = x
        t[name] = sv.Pages4(*big)
    t["page_table"] = torch.where(t["page_table"] >= 0, t["page_table"] + (P - used), -1).to(torch.int32)
    check(c, *sv.spec_paged_attention(**t))


def test_outputs_workspace_and_events_may_be_given(dev):  # noqa: F811
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case4(dev, 2, 2, 1, 2, 64, 16, [400, 3], seed=18)
    t = c.tensors()
    n = sv.sv_attention4_workspace_bytes(2, 2, 2, 1, 64, 16, t["page_table"].shape[1])
    ws = torch.randint(0, 255, (n,), dtype=torch.uint8, device=dev)  # any contents
    out = (torch.empty_like(t["q"]), torch.empty(2, dtype=torch.int32, device=dev))
    got = sv.spec_paged_attention(**t, workspace=ws, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    check(c, *got)
    assert sv.spec_paged_attention(**t, events=[])[2] == 2
    with pytest.raises(sv.SpecVerifyError, match="WORKSPACE"):
        sv.spec_paged_attention(**t, workspace=ws[:-256])
    assert sv.sv_attention4_launch_plan(1, 4, 1, 128) == ["k_attn4", "k_attn_join"]
    assert sv.sv_attention4_launch_plan(33, 4, 4, 64) == ["k_attn4_wide", "k_attn_join"]
