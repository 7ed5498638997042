"""spec_cache_append_rotary against a float64 reference (tests/step_ref.py): both pairings, parts of
heads, trees, given positions, strides, ragged counts, row codes, streams and graphs.

Tolerance of an element y = f (a c - b s): the cosine and sine are within 2^-50 of f times theirs
(argument: one rounding of the product, the same here and there; reduction and series under 2^-51;
the factor's rounding 2^-53), the rotation in 64 bits, so the value before its rounding is within
2^-49 f (|a| + |b|); then one rounding to float32 (2^-24 relative) and for bf16 a second (2^-8)."""
import numpy as np
import pytest

import cache_ref as ref
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


class Call:
    """A call's inputs in values that bf16 holds, pages in random order."""

    def __init__(self, dtype, B, N, Hq, Hkv, D, R, page, lens, news=None, tree=False, interleaved=False, factor=1.0, positions=False,
                 seed=0, base=10000.0):
        import torch
        rng = self.rng = np.random.default_rng(seed)
        self.dt, self.esz = (torch.bfloat16, 2) if dtype == "bf16" else (torch.float32, 4)
        self.B, self.N, self.Hq, self.Hkv, self.D, self.R, self.page = B, N, Hq, Hkv, D, R, page
        self.lens, self.news, self.given = list(lens), list(news) if news is not None else [N] * B, news is not None
        self.interleaved, self.factor = interleaved, float(np.float32(factor))
        self.freq = (base ** (-np.arange(0, R, 2) / max(R, 1))).astype(np.float32)
        values = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).double().numpy()  # noqa: E731
        self.q, self.k, self.v = values(B, N, Hq, D), values(B, N, Hkv, D), values(B, N, Hkv, D)
        self.parents = None
        depth = np.broadcast_to(np.arange(N), (B, N))
        if tree:
            self.parents = np.full((B, N), -1, np.int32)
            for n in range(1, N):
                self.parents[:, n] = np.maximum(0, n - 1 - rng.integers(0, 4, B))
            depth = np.array([[ref.lineage(p, i)[1] for i in range(N)] for p in self.parents])
        self.pos = np.array(self.lens)[:, None] + depth
        self.positions = None
        if positions:
            self.pos = self.positions = rng.integers(-50, 200000, (B, N)).astype(np.int32)
        counts = [-(-(n + m) // page) for n, m in zip(self.lens, self.news)]
        W, P = max(1, max(counts)) + 1, sum(counts) + 2
        ids, at = rng.permutation(P), 0
        self.table = np.full((B, W), -1, np.int32)
        for b in range(B):
            self.table[b, :counts[b]] = ids[at:at + counts[b]]
            at += counts[b]
        self.P, self.E = P, 16 // self.esz
        self.kp = rng.integers(-9, 9, (P, Hkv, D // self.E, page, self.E)).astype(np.float64)
        self.vp = rng.integers(-9, 9, (P, Hkv, page // self.E, D, self.E)).astype(np.float64)

    def tensors(self, dev):
        import torch
        import rejection_sampling_verify_02_amd as sv
        to = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(self.dt).to(dev)  # noqa: E731
        i32 = lambda x: None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
        turn = sv.Rotary(torch.from_numpy(self.freq).to(dev), self.interleaved, self.factor)
        return dict(q=to(self.q), k=to(self.k), v=to(self.v), k_pages=to(self.kp), v_pages=to(self.vp), page_table=i32(self.table),
                    cache_len=i32(self.lens), rotary=turn, parent=i32(self.parents), positions=i32(self.positions),
                    n_new=i32(self.news) if self.given else None)

    def near(self, got, x, pos):
        y, size = step_ref.turn(x, pos, self.freq, self.interleaved, self.factor)
        tol = 2.0 ** -49 * size + np.abs(y) * (2.0 ** -24 + (2.0 ** -8 if self.esz == 2 else 0.0)) * (1 + 2.0 ** -8) + 1e-38
        err = np.abs(got - y)
        rest = slice(self.R, None)
        assert np.array_equal(got[..., rest], x[..., rest])
        assert np.all(err <= tol), (err.max(), (err / tol).max())

    def check(self, t, q_out, status, only=None):
        rows = range(self.B) if only is None else only
        kp, vp = t["k_pages"].double().cpu().numpy(), t["v_pages"].double().cpu().numpy()
        got = q_out.double().cpu().numpy() if q_out is not None else None
        want_v, mask = self.vp.copy(), np.ones(self.kp.shape, bool)
        for b in rows:
            assert int(status[b]) == 0
            m = self.news[b]
            if got is not None:
                self.near(got[b, :m], self.q[b, :m], self.pos[b, :m])
                assert not got[b, m:].any()
            for i in range(m):
                s = self.lens[b] + i
                p, at = self.table[b, s // self.page], s % self.page
                self.near(kp[p, :, :, at].reshape(self.Hkv, -1), self.k[b, i], self.pos[b, i])
                mask[p, :, :, at] = False
                ref.pack_v(self.v[b, i], s, want_v, self.table[b], self.page, self.E)
        assert np.array_equal(kp[mask], self.kp[mask]) and np.array_equal(vp, want_v)  # nothing else is touched


def run(t):
    import rejection_sampling_verify_02_amd as sv
    return sv.spec_cache_append_rotary(**t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,R,page,N,lens,news", [
    (4, 2, 64, 64, 16, 1, [0, 15, 16, 100000], None),
    (8, 2, 128, 128, 64, 5, [3, 61, 130, 7, 2], [5, 0, 3, 1, 5]),
    (3, 3, 64, 32, 16, 9, [0, 7], None),
    (2, 1, 128, 34, 32, 11, [5, 31], None),      # halves that are no whole units
    (1, 1, 256, 2, 16, 3, [14], None),
    (5, 1, 48, 46, 16, 20, [30, 1], [20, 13]),
    (2, 1, 512, 512, 16, 2, [15], None),
    (9, 1, 16, 8, 256, 300, [250, 0], [299, 1]),
])
def test_rotated_append(dev, dtype, interleaved, Hq, Hkv, D, R, page, N, lens, news):
    c = Call(dtype, len(lens), N, Hq, Hkv, D, R, page, lens, news, interleaved=interleaved, factor=1.25, seed=D + N + R)
    t = c.tensors(dev)
    c.check(t, *run(t))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [64, 24])
def test_trees_and_given_positions(dev, dtype, R):
    for kw in (dict(tree=True), dict(positions=True), dict(tree=True, positions=True)):
        c = Call(dtype, 5, 33, 4, 2, 64, R, 16, [0, 3, 50, 16, 9], [33, 17, 0, 1, 32], seed=R, factor=0.75, **kw)
        t = c.tensors(dev)
        c.check(t, *run(t))


def test_far_positions_and_fast_turns(dev):
    """Angles of millions of turns: the argument is one product, rounded once in 64 bits."""
    c = Call("f32", 3, 2, 2, 1, 64, 64, 16, [0, 3, 9], positions=True, seed=1, base=1.5)
    c.pos = c.positions = np.array([[2 ** 31 - 1, -2 ** 31], [123456789, 1 << 30], [0, -1]], np.int32)
    t = c.tensors(dev)
    c.check(t, *run(t))


def test_without_queries_and_without_rotation(dev):
    import rejection_sampling_verify_02_amd as sv
    c = Call("bf16", 3, 4, 2, 2, 64, 64, 16, [10, 0, 33], seed=2)
    t = c.tensors(dev)
    q_out, st = sv.spec_cache_append_rotary(**{**t, "q": None})
    assert q_out is None
    c.check(t, None, st)
    # no rotation: what spec_cache_append writes, and the queries as they are
    t = c.tensors(dev)
    u = c.tensors(dev)
    q_out, st = sv.spec_cache_append_rotary(**{**t, "rotary": None})
    sv.spec_cache_append(u["k"], u["v"], u["k_pages"], u["v_pages"], u["page_table"], u["cache_len"])
    assert (q_out == t["q"]).all() and (t["k_pages"] == u["k_pages"]).all() and (t["v_pages"] == u["v_pages"]).all()


def test_fused_projection_rows(dev):
    import torch
    c = Call("bf16", 3, 5, 4, 2, 64, 64, 16, [10, 33, 2], seed=3)
    t = c.tensors(dev)
    qkv = torch.full((3, 7, 9, 64), float("nan"), dtype=c.dt, device=dev)
    qkv[:, 1:6, :4], qkv[:, 1:6, 4:6], qkv[:, 1:6, 6:8] = t["q"], t["k"], t["v"]
    t.update(q=qkv[:, 1:6, :4], k=qkv[:, 1:6, 4:6], v=qkv[:, 1:6, 6:8])
    c.check(t, *run(t))


def test_codes(dev):
    import torch
    c = Call("bf16", 7, 6, 4, 2, 64, 64, 16, [40, 41, 42, 43, 44, 30, 46], [6] * 7, tree=True, seed=4)
    t = c.tensors(dev)
    t["cache_len"][0] = -1
    t["n_new"][1] = 7
    t["parent"][2, 4] = 4
    t["page_table"][3, 2] = c.P
    t["page_table"][3, 3] = c.P
    t["parent"][4, 0] = 0
    t["prior"] = torch.tensor([0, 0, 0, 0, -9, -9, 3], dtype=torch.int32, device=dev)
    q_out, st = run(t)
    assert st.tolist() == [-8, -8, -6, -7, -9, -9, 0]
    assert torch.isnan(q_out[:6]).all()
    c.check(t, q_out, st, only=[6])


def test_not_finite_stays_where_it_is(dev):
    """A pair with an infinity or NaN: what the formula gives; its neighbours are untouched by it."""
    import torch
    c = Call("f32", 1, 2, 1, 1, 64, 32, 16, [5], seed=5)
    t = c.tensors(dev)
    t["q"][0, 0, 0, 3] = float("nan")
    t["k"][0, 1, 0, 20] = float("inf")
    q_out, st = run(t)
    bad = torch.isnan(q_out[0, 0, 0]).nonzero()[:, 0].tolist()
    assert bad == [3, 19] and torch.isfinite(q_out[0, 1]).all()
    k = t["k_pages"][int(c.table[0, 0]), 0, :, 6].flatten()
    assert (~torch.isfinite(k)).nonzero()[:, 0].tolist() == [4, 20]


def test_streams_graphs_and_given_outputs(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Call("bf16", 3, 4, 4, 2, 128, 128, 16, [10, 30, 64], seed=6)
    t = c.tensors(dev)
    out = (torch.empty_like(t["q"]), torch.empty(3, dtype=torch.int32, device=dev))
    got = sv.spec_cache_append_rotary(**t, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    c.check(t, *got)
    first = out[0].clone()
    torch.cuda.synchronize(dev)
    side = torch.cuda.Stream(dev)
    u = c.tensors(dev)
    torch.cuda.synchronize(dev)
    got = sv.spec_cache_append_rotary(**u, stream=side.cuda_stream)
    side.synchronize()
    c.check(u, *got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured, st = sv.spec_cache_append_rotary(**t)
    for _ in range(3):
        captured.fill_(7)
        g.replay()
        again, _ = sv.spec_cache_append_rotary(**u)
        assert torch.equal(captured, first) and torch.equal(again, first) and st.tolist() == [0, 0, 0]


def test_refusals(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    c = Call("bf16", 2, 3, 4, 2, 64, 64, 16, [10, 30], seed=7)
    t = c.tensors(dev)
    f = t["rotary"].inv_freq
    for kw, e in ((dict(rotary=sv.Rotary(f.double())), ValueError), (dict(rotary=sv.Rotary(torch.zeros(33, device=dev))), ValueError),
                  (dict(rotary=sv.Rotary(f.cpu())), ValueError), (dict(q=t["q"].float()), TypeError), (dict(q=t["q"][:1]), ValueError),
                  (dict(parent=t["cache_len"]), ValueError), (dict(positions=t["cache_len"]), ValueError), (dict(v=t["v"][..., :32]), ValueError),
                  (dict(k=t["k"].half()), TypeError), (dict(rotary=sv.Rotary(f, False, float("inf"))), sv.SpecVerifyError),
                  (dict(out=(t["q"], None)), sv.SpecVerifyError)):
        with pytest.raises(e):
            sv.spec_cache_append_rotary(**{**t, **kw})


def test_frequencies():
    import rejection_sampling_verify_02_amd as sv
    r = sv.Rotary.of(8, 100.0)
    assert np.allclose(r.inv_freq.numpy(), 100.0 ** (-np.arange(0, 8, 2) / 8), rtol=2 ** -23) and r.factor == 1.0 and not r.interleaved
    assert np.allclose(sv.Rotary.of(8, 100.0, stretch=4.0).inv_freq.numpy(), r.inv_freq.numpy() / 4, rtol=2 ** -22)
    s = sv.Rotary.of(64, 10000.0, stretch=8.0, trained=4096, interleaved=True)
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    turns = 4096 * f / (2 * np.pi)
    got = s.inv_freq.numpy()
    assert np.allclose(got[turns >= 32], f[turns >= 32], rtol=2 ** -22) and np.allclose(got[turns <= 1], f[turns <= 1] / 8, rtol=2 ** -22)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all(got[mid] < f[mid]) and np.all(got[mid] > f[mid] / 8)
    assert abs(s.factor - (1 + 0.1 * np.log(8))) < 1e-12 and s.interleaved
    for kw in (dict(rot_dim=7), dict(rot_dim=0), dict(base=0.0), dict(stretch=0.5), dict(trained=0), dict(trained=10, slow=3, fast=2)):
        with pytest.raises(ValueError):
            sv.Rotary.of(**{"rot_dim": 8, **kw})
