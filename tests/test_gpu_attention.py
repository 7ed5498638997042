"""spec_paged_attention against a float64 reference (tests/cache_ref.py), at the lengths, masks,
layouts and values where it can go wrong.  Tolerances are per element and derived in cache_ref."""
import numpy as np
import pytest

import cache_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_02_amd as sv
    sv.load_library()
    return torch.device("cuda:0")


class Case:
    """A call's inputs: values that bf16 holds, a pool whose every unused slot is NaN, pages in
    random order, table entries behind (and, with a window, left of) what is needed -1."""

    def __init__(self, dev, dtype, B, N, Hkv, group, D, page, lens, news=None, tree=False, window=0, sinks=0, seed=0,
                 spread=2.0, evict=True):
        import torch
        rng = np.random.default_rng(seed)
        self.dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.esz = 2 if dtype == "bf16" else 4
        self.B, self.N, self.H, self.g, self.D, self.page, self.window, self.sinks = B, N, Hkv, group, D, page, window, sinks
        self.lens, self.news = list(lens), list(news) if news is not None else [N] * B
        self.given = news is not None
        E = self.E = 16 // self.esz

        def draw(shape, scale=1.0):  # values of the type
            x = torch.from_numpy(scale * rng.standard_normal(shape)).to(self.dt)
            return x.double().numpy()

        self.q = draw((B, N, Hkv * group, D), spread)
        self.parents = None
        if tree:
            self.parents = np.full((B, N), -1, np.int32)
            for n in range(1, N):
                self.parents[:, n] = np.maximum(0, n - 1 - rng.integers(0, 4, B))
        counts = [-(-(n + m) // page) for n, m in zip(self.lens, self.news)]
        W = max(1, max(counts)) + 2
        P = sum(counts) + 2
        ids = rng.permutation(P)
        self.table = np.full((B, W), -1, np.int32)
        self.kp = np.full((P, Hkv, D // E, page, E), np.nan)
        self.vp = np.full((P, Hkv, page // E, D, E), np.nan)
        self.ks, self.vs, at = [], [], 0
        for b in range(B):
            own = ids[at:at + counts[b]]
            at += counts[b]
            self.table[b, :counts[b]] = own
            n = self.lens[b] + self.news[b]
            k, v = draw((Hkv, n, D)), draw((Hkv, n, D))
            for t in range(n):
                ref.pack_k(k[:, t], t, self.kp, own, page, E)
                ref.pack_v(v[:, t], t, self.vp, own, page, E)
            self.ks.append(k)
            self.vs.append(v)
            if window and evict:  # pages that no node sees have been given back
                first = max(0, self.lens[b] - window + 1)
                for i in range(counts[b]):
                    if (i + 1) * page <= first and i * page >= sinks:
                        self.table[b, i] = -1
        self.scale = 1.0 / np.sqrt(D)
        self.dev = dev

    def tensors(self):
        import torch
        to = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(self.dt).to(self.dev)  # noqa: E731
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=self.dev)  # noqa: E731
        return dict(q=to(self.q), k_pages=to(self.kp), v_pages=to(self.vp), page_table=i32(self.table), cache_len=i32(self.lens),
                    n_new=i32(self.news) if self.given else None, parent=i32(self.parents) if self.parents is not None else None,
                    window=self.window, sinks=self.sinks)

    def expect(self):
        return ref.attention(self.q, self.ks, self.vs, self.lens, self.news, self.parents, self.scale, self.window, self.sinks,
                             self.esz)


def check(case, out, status):
    want, tol = case.expect()
    got = out.double().cpu().numpy()
    assert status.cpu().tolist() == [0] * case.B
    fin = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fin) and np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    err = np.abs(got[fin] - want[fin])
    over = err / np.maximum(tol[fin], 1e-300)
    assert np.all(err <= tol[fin]), (err.max(), over.max(), np.argwhere(fin)[err > tol[fin]][:4].tolist())
    for b in range(case.B):
        assert not np.any(got[b, case.news[b]:]), "rows behind n_new are zero"
    return over.max() if over.size else 0.0


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
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:6])))
def test_chain(dev, dtype, shape):
    B, N, Hkv, g, D, page, lens = shape
    c = Case(dev, dtype, B, N, Hkv, g, D, page, lens, seed=sum(lens) + D)
    check(c, *run(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (3, 2), (16, 0), (33, 1), (40, 50), (500, 4), (2 ** 31 - 1, 2 ** 31 - 1),
                                          (5, 2 ** 31 - 1)])
@pytest.mark.parametrize("tree", [False, True])
def test_window_and_sinks(dev, dtype, window, sinks, tree):
    c = Case(dev, dtype, 5, 9, 1, 2, 64, 16, [0, 3, 33, 90, 200], tree=tree, window=window, sinks=sinks, seed=window + sinks)
    check(c, *run(c))


@pytest.mark.parametrize("dtype,D,page", [("bf16", 128, 32), ("f32", 128, 16), ("bf16", 256, 64), ("f32", 64, 64)])
def test_trees_and_ragged_counts(dev, dtype, D, page):
    N = 40
    c = Case(dev, dtype, 6, N, 1, 4, D, page, [0, 1, 30, 31, 64, 77], news=[N, 0, 1, 17, 33, 39], tree=True, seed=D)
    check(c, *run(c))


def test_everything_empty(dev):
    c = Case(dev, "bf16", 3, 4, 2, 2, 64, 16, [0, 5, 0], news=[0, 0, 0])
    check(c, *run(c))


@pytest.mark.parametrize("dtype,Hkv,g,D", [("bf16", 2, 4, 128), ("f32", 1, 2, 64), ("bf16", 1, 16, 256)])
def test_long_contexts_split_over_workgroups(dev, dtype, Hkv, g, D):
    """Lengths far apart, so that a share spans several short sequences and a long one many shares."""
    c = Case(dev, dtype, 6, 2, Hkv, g, D, 64, [6000, 1, 40, 2500, 0, 333], seed=5)
    check(c, *run(c))


@pytest.mark.parametrize("dtype,N,g,D,window", [("bf16", 24, 4, 128, 0), ("bf16", 12, 4, 64, 0), ("f32", 9, 8, 64, 0),
                                                ("bf16", 40, 2, 256, 300), ("f32", 33, 2, 256, 0), ("f32", 20, 8, 128, 777)])
def test_long_contexts_with_many_rows(dev, dtype, N, g, D, window):
    """The kernel whose waves share tiles, with units cut into parts."""
    c = Case(dev, dtype, 3, N, 1, g, D, 32, [3500, 10, 1777], tree=True, window=window, sinks=40 if window else 0, seed=N)
    check(c, *run(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,g,lens", [(1, 4, [1100] * 40), (20, 4, [1100] * 40), (3, 1, list(range(0, 2000, 50))), (1, 2, [5] * 300 + [900])])
def test_every_way_to_cut_a_batch(dev, dtype, N, g, lens):
    """Equal lengths (a part a workgroup), lengths that no such cut fits (shares that run on into
    the next unit), and more units than workgroups."""
    H = 4 if len(lens) <= 40 else 2
    c = Case(dev, dtype, len(lens), N, H, g, 64, 64, lens, seed=len(lens) + N)
    t = c.tensors()
    import rejection_sampling_verify_02_amd as sv
    out, st = sv.spec_paged_attention(**t)
    assert st.tolist() == [0] * c.B
    # the float64 reference for some sequences, and for all of them the same bits when asked again
    some = sorted({0, 1, c.B // 2, c.B - 1})
    part = Case.__new__(Case)
    part.__dict__.update(c.__dict__)
    part.B, part.q, part.lens, part.news = len(some), c.q[some], [c.lens[b] for b in some], [c.news[b] for b in some]
    part.ks, part.vs = [c.ks[b] for b in some], [c.vs[b] for b in some]
    check(part, out[some], st[some])
    again, _ = sv.spec_paged_attention(**t)
    assert (again == out).all()
    # a sequence's rows do not depend on how the others cut the batch, but for the order of f32 sums
    alone = {**t, "q": t["q"][:1].contiguous(), "page_table": t["page_table"][:1].contiguous(), "cache_len": t["cache_len"][:1].contiguous()}
    one, _ = sv.spec_paged_attention(**alone)
    first = Case.__new__(Case)
    first.__dict__.update(part.__dict__)
    first.B, first.q, first.lens, first.news, first.ks, first.vs = 1, c.q[:1], c.lens[:1], c.news[:1], c.ks[:1], c.vs[:1]
    check(first, one, st[:1])


def test_many_sequences(dev):
    """More sequences than a workgroup has threads."""
    lens = [(37 * i) % 50 for i in range(530)]
    c = Case(dev, "bf16", 530, 1, 1, 1, 64, 16, lens, seed=8)
    check(c, *run(c))


def test_many_new_tokens(dev):
    c = Case(dev, "bf16", 1, 1024, 1, 1, 64, 64, [20], tree=True, seed=9)
    check(c, *run(c))
    c = Case(dev, "f32", 2, 300, 1, 2, 64, 16, [20, 0], news=[300, 257], seed=10)
    check(c, *run(c))


def test_long_chain_as_tree_is_the_chain(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case(dev, "bf16", 2, 100, 1, 2, 64, 16, [20, 50], seed=10)
    t = c.tensors()
    check(c, *sv.spec_paged_attention(**t))
    t["parent"] = torch.arange(-1, 99, dtype=torch.int32, device=dev).expand(2, 100).contiguous()
    check(c, *sv.spec_paged_attention(**t))


def test_query_strides(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case(dev, "bf16", 3, 5, 2, 4, 64, 16, [10, 33, 2], seed=3)
    t = c.tensors()
    plain, _ = sv.spec_paged_attention(**t)
    wide = torch.full((3, 7, 8 + 4, 64), float("nan"), dtype=c.dt, device=dev)  # queries in a fused projection's rows
    wide[:, 1:6, :8] = t["q"]
    t["q"] = wide[:, 1:6, :8]
    got, st = sv.spec_paged_attention(**t)
    assert torch.equal(got, plain)
    check(c, got, st)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales(dev, dtype, scale):
    import rejection_sampling_verify_02_amd as sv
    c = Case(dev, dtype, 2, 3, 1, 2, 64, 16, [70, 9], seed=4)
    c.scale = scale
    check(c, *sv.spec_paged_attention(**c.tensors(), scale=scale))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["nan", "inf", "-inf", "both"])
@pytest.mark.parametrize("g,D", [(2, 64), (8, 64), (6, 128), (8, 256)])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(dev, dtype, what, g, D):
    """A tree's nodes whose keys or values are not finite: their descendants show it, other
    branches do not.  The same for a committed token at the window's edge."""
    import rejection_sampling_verify_02_amd as sv
    bad = {"nan": [np.nan], "inf": [np.inf], "-inf": [-np.inf], "both": [np.inf, -np.inf]}[what]
    N, n = 12, 37
    parents = np.array([[-1, 0, 0, 1, 1, 2, 2, 3, 5, 7, 8, 10]], np.int32)
    for window, where, slots in ((0, "v", [n + 3, n + 7]), (0, "v", [n + 2, n + 6]), (8, "v", [n - 7, n - 6]), (0, "k", [n + 3])):
        c = Case(dev, dtype, 1, N, 1, g, D, 16, [n], tree=True, window=window, seed=21, evict=False)
        c.parents = parents
        for x, t in zip(bad * 2, slots):
            if where == "k" and not np.isnan(x):
                continue  # a key of infinities gives scores of either sign: only NaN has one answer
            (c.vs if where == "v" else c.ks)[0][:, t, 5] = x
            if where == "v":
                ref.pack_v(c.vs[0][:, t], t, c.vp, c.table[0], 16, c.E)
            else:
                ref.pack_k(c.ks[0][:, t], t, c.kp, c.table[0], 16, c.E)
        check(c, *sv.spec_paged_attention(**c.tensors()))


def test_codes(dev):
    """A sequence that does not fit its tables has a code and NaN rows; the others are untouched."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case(dev, "bf16", 8, 6, 2, 2, 64, 16, [40, 41, 42, 43, 44, 45, 300, 47], tree=True, news=[6, 6, 6, 6, 6, 6, 6, 6], seed=12)
    good, _ = sv.spec_paged_attention(**c.tensors())
    t = c.tensors()
    t["cache_len"][0] = -1
    t["n_new"][1] = 7
    t["cache_len"][2] = 100000
    t["parent"][3, 4] = 4
    t["parent"][4, 0] = 0
    t["page_table"][5, 2] = t["k_pages"].shape[0]
    t["page_table"][6, 7] = -1
    t["parent"][5, 2] = 99  # a bad tree is told before a bad page
    out, st = sv.spec_paged_attention(**t)
    assert st.tolist() == [-8, -8, -8, -6, -6, -6, -7, 0]
    assert torch.isnan(out[:7]).all()
    assert torch.equal(out[7], good[7])
    t["n_new"][:] = -1
    out, st = sv.spec_paged_attention(**t)
    assert st.tolist() == [-8] * 8 and torch.isnan(out).all()


def test_same_bits_every_time_and_on_other_streams(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case(dev, "bf16", 4, 3, 2, 4, 128, 16, [900, 30, 2000, 5], seed=13)
    d = Case(dev, "f32", 3, 6, 2, 2, 64, 16, [1000, 77, 1500], tree=True, seed=14)
    tc, td = c.tensors(), d.tensors()
    first_c, first_d = sv.spec_paged_attention(**tc)[0], sv.spec_paged_attention(**td)[0]
    check(c, first_c, torch.zeros(4, dtype=torch.int32))
    check(d, first_d, torch.zeros(3, dtype=torch.int32))
    torch.cuda.synchronize(dev)
    sa, sb = torch.cuda.Stream(dev), torch.cuda.Stream(dev)
    got = []
    for _ in range(20):
        with torch.cuda.stream(sa):
            x = sv.spec_paged_attention(**tc)[0]
        y = sv.spec_paged_attention(**td, stream=sb.cuda_stream)[0]
        got.append((x, y))
    torch.cuda.synchronize(dev)
    assert all(torch.equal(x, first_c) and torch.equal(y, first_d) for x, y in got)


@pytest.mark.parametrize("N", [4, 30])
def test_captured_and_replayed(dev, N):
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case(dev, "bf16", 3, N, 2, 4, 64, 16, [700, 30, 1], seed=15)
    t = c.tensors()
    plain, _ = sv.spec_paged_attention(**t)
    q0 = t["q"].clone()
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(s):
        sv.spec_paged_attention(**t)
    torch.cuda.current_stream(dev).wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, st = sv.spec_paged_attention(**t)
    for k in range(4):
        t["q"].copy_(q0 if k % 2 == 0 else -q0)
        out.fill_(-1)
        g.replay()
        other, _ = sv.spec_paged_attention(**t)  # eager work between the replays
        torch.cuda.synchronize(dev)
        assert torch.equal(out, other) and st.tolist() == [0, 0, 0]
        if k % 2 == 0:
            assert torch.equal(out, plain)


def test_lengths_may_grow_between_replays(dev):
    """The captured call reads lengths and tables on the device: a later step's lengths need no
    new capture."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case(dev, "bf16", 2, 1, 1, 4, 64, 16, [600, 500], seed=16)
    t = c.tensors()
    short = torch.tensor([13, 499], dtype=torch.int32, device=dev)
    g = torch.cuda.CUDAGraph()
    sv.spec_paged_attention(**t)
    torch.cuda.synchronize(dev)
    lens = t["cache_len"]
    full = lens.clone()
    with torch.cuda.graph(g):
        out, st = sv.spec_paged_attention(**t)
    for want in (short, full, short):
        lens.copy_(want)
        g.replay()
        eager, _ = sv.spec_paged_attention(**t)
        assert torch.equal(out, eager)
    check(c, sv.spec_paged_attention(**{**t, "cache_len": full})[0], torch.zeros(2, dtype=torch.int32))


def test_pool_beyond_32_bit_offsets(dev):
    """Pages behind the first 4 GiB of the pool."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case(dev, "bf16", 2, 1, 8, 1, 128, 64, [150, 64], seed=17)
    t = c.tensors()
    page_bytes = 8 * 64 * 128 * 2
    P = (5 << 30) // page_bytes
    used = t["k_pages"].shape[0]
    for name in ("k_pages", "v_pages"):
        big = torch.empty((P, *t[name].shape[1:]), dtype=c.dt, device=dev)
        big[P - used:] = t[name]
        t[name] = big
    t["page_table"] = torch.where(t["page_table"] >= 0, t["page_table"] + (P - used), -1).to(torch.int32)
    check(c, *sv.spec_paged_attention(**t))


def test_outputs_and_workspace_may_be_given(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case(dev, "f32", 2, 2, 1, 2, 64, 16, [400, 3], seed=18)
    t = c.tensors()
    n = sv.sv_attention_workspace_bytes(2, 2, 2, 1, 64, 16, t["page_table"].shape[1], sv.SV_F32)
    ws = torch.randint(0, 255, (n,), dtype=torch.uint8, device=dev)  # any contents
    out = (torch.empty_like(t["q"]), torch.empty(2, dtype=torch.int32, device=dev))
    got = sv.spec_paged_attention(**t, workspace=ws, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    check(c, *got)
    with pytest.raises(sv.SpecVerifyError, match="WORKSPACE"):
        sv.spec_paged_attention(**t, workspace=ws[:-256])


def test_default_stream_by_its_handle_and_sizes_beyond_32_bits(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case(dev, "bf16", 2, 2, 1, 2, 64, 16, [300, 40], seed=21)
    t = c.tensors()
    torch.cuda.synchronize(dev)
    with torch.cuda.stream(torch.cuda.Stream(dev)):
        got = sv.spec_paged_attention(**t, stream=torch.cuda.default_stream(dev).cuda_stream)
    torch.cuda.synchronize(dev)
    check(c, *got)
    for kw in (dict(window=2**32 + 5), dict(window=8, sinks=2**32)):  # ctypes would pass 5 and 0
        with pytest.raises(ValueError, match="32 bits"):
            sv.spec_paged_attention(**{**t, **kw})


@pytest.mark.parametrize("N", [2, 40])  # both kernels
@pytest.mark.parametrize("D", [128, 256])
def test_f32_scores_keep_their_bits(dev, N, D):
    """The error over all outputs, which the rounding of the scores decides.  With u = 2^-24 and a
    rounding's error u / sqrt(3) in the root mean square of a sum's size, products of variance 4:
    a sum lengthened by four products at a time in K = D / 16 steps gathers (u / sqrt 3) * 2 *
    sqrt(2) K, four of them twice that, and joining them (u / sqrt 3) * 2 sqrt(D) * sqrt 2; times
    the scale 1 / sqrt D that is 3.3u + 1.6u (added in squares, 3.7u) at D = 256.  Weights (one rounding of
    an argument up to 16 below, 4.6u, the power, u, sums and quotient, 2u) come to 5.1u: 6.3u =
    3.8e-7 in all, and less for D = 128.  Twice that is allowed for the orders in which an
    instruction may add its four products; a single sum of 256 is beyond it (measured 1.2e-6)."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Case(dev, "f32", 4, N, 2, 1, D, 16, [250, 300, 331, 358], seed=23)
    rng = np.random.default_rng(24)
    t = c.tensors()
    # full mantissas: values that bf16 holds too would make the products short
    c.q = torch.from_numpy(2.0 * rng.standard_normal(c.q.shape)).float().double().numpy()
    t["q"] = torch.from_numpy(c.q).float().to(dev)
    out, st = sv.spec_paged_attention(**t)
    want = c.expect()[0]
    err = np.linalg.norm(out.double().cpu().numpy() - want) / np.linalg.norm(want)
    assert st.tolist() == [0] * 4
    assert err <= 7.6e-7, err
