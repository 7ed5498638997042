"""Sampling and filtered logits under temperature, top-k, min-p and top-p against tests/step_ref.py:
tokens and kept sets are equal wherever the reference's own cuts and boundaries are 1e-10 of the
total away (weights are within 4e-11 of theirs by the series, 1.5e-11 by the fixed point, and sums
are exact), and seeds are fixed."""
import numpy as np
import pytest

import step_ref

pytestmark = pytest.mark.gpu
NEAR = 1e-10


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_02_amd as sv
    sv.load_library()
    return torch.device("cuda:0")


def logits(rng, rows, V, dtype, kind):
    import torch
    z = rng.standard_normal((rows, V)) * 1.5 - 1.1 * np.log(np.array([rng.permutation(V) for _ in range(rows)]) + 1.0)
    if kind == "peaked":
        z *= 3
    elif kind == "flat":
        z *= 0.02
    elif kind == "equal":
        z[:] = 1.25
    elif kind == "masked":
        z[rng.random((rows, V)) < 0.7] = -np.inf
        z[:, V // 2] = 0.5
    elif kind == "ties":
        z = np.round(z)
    t = torch.from_numpy(z).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t, t.double().numpy()


def checked(z, got, want, status, near):
    sure = near > NEAR
    assert sure.mean() > 0.9
    assert np.array_equal(got[sure], want[sure]), np.argwhere(got != want)[:5].tolist()
    assert not status.any()


POLICIES = [(1.0, 0, 0.9, 0.0), (0.7, 50, 1.0, 0.0), (1.3, 0, 1.0, 0.05), (0.8, 40, 0.95, 0.02), (1.0, 0, 1.0, 0.0), (2.0, 3, 0.3, 0.5),
            (1.0, 1, 1.0, 0.0), (0.05, 0, 0.99999, 0.0), (30.0, 0, 0.5, 0.0), (1.0, 0, 1e-9, 0.0), (1.0, 10 ** 9, 1.0, 1.0), (1.5, 700, 0.999, 0.0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["usual", "peaked", "flat", "equal", "masked", "ties"])
@pytest.mark.parametrize("V", [1, 2, 7, 1000, 8191, 8200, 20011])
def test_sample_and_filter(dev, dtype, kind, V):
    import torch
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(V)
    rows = 6
    t, z = logits(rng, rows, V, dtype, kind)
    t = t.to(dev)
    u = rng.random(rows).astype(np.float32)
    u[0], u[1] = 0.0, 1 - 2.0 ** -24
    du = torch.from_numpy(u).to(dev)
    for T, k, p, m in POLICIES:
        tok, st = sv.spec_sample(t, du, T, k, top_p=p, min_p=m)
        want = [step_ref.draw(z[b], u[b], T, k, p, m) for b in range(rows)]
        if (k, p, m) == (0, 1.0, 0.0):  # the other sampler's kernels: boundaries to float32
            continue
        checked(z, tok.cpu().numpy(), np.array([x for x, _ in want]), st.cpu().numpy(), np.array([x for _, x in want]) + (V < 50))
        out, st = sv.spec_filter_logits(t, T, k, top_p=p, min_p=m)
        cut = [step_ref.kept(z[b], T, k, p, m) for b in range(rows)]
        low = np.array([x for x, _ in cut])[:, None]
        want = np.where(z >= low, z, -np.inf)
        near = np.array([x for _, x in cut])
        sure = near > NEAR
        assert not st.any() and out.dtype == t.dtype and np.array_equal(out.double().cpu().numpy()[sure], want[sure])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["usual", "flat", "peaked"])
def test_large_vocabularies(dev, dtype, kind):
    """More chunks than waves have lanes, thresholds among more tokens than the list holds."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    for V, rows in ((152064, 3), (600001, 2)):
        rng = np.random.default_rng(V)
        t, z = logits(rng, rows, V, dtype, kind)
        t = t.to(dev)
        u = np.array([0.3, 0.999, 0.7], np.float32)[:rows]
        for T, k, p, m in ((1.0, 0, 0.9, 0.0), (0.8, 20000, 1.0, 0.0), (1.0, 30000, 0.8, 1e-6), (1.2, 50, 0.9, 0.1)):
            tok, st = sv.spec_sample(t, torch.from_numpy(u).to(dev), T, k, top_p=p, min_p=m)
            want = [step_ref.draw(z[b], u[b], T, k, p, m) for b in range(rows)]
            sure = np.array([x for _, x in want]) > NEAR
            assert not st.any() and np.array_equal(tok.cpu().numpy()[sure], np.array([x for x, _ in want])[sure])
            out, _ = sv.spec_filter_logits(t, T, k, top_p=p, min_p=m)
            for b in range(rows):
                low, near = step_ref.kept(z[b], T, k, p, m)
                assert near < NEAR or np.array_equal(out[b].double().cpu().numpy(), np.where(z[b] >= low, z[b], -np.inf))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0.02, 0.15, 0.6])
def test_top_k_among_tokens_of_hardly_any_weight(dev, dtype, T):
    """The k-th token lies among tens of thousands whose weights are below 2^-32 of the largest, which
    are counted together; what is kept is few again."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    rows, V = 3, 40009
    rng = np.random.default_rng(17)
    t, z = logits(rng, rows, V, dtype, "peaked")
    t = t.to(dev)
    u = np.array([0.2, 0.9, 1 - 2.0 ** -24], np.float32)
    for k, p, m in ((2, 0.9, 0.0), (72, 0.9, 0.0), (500, 1.0, 0.0), (9000, 0.999, 0.0), (9000, 1.0, 1e-30), (20000, 0.5, 1e-12)):
        tok, st = sv.spec_sample(t, torch.from_numpy(u).to(dev), T, k, top_p=p, min_p=m)
        want = [step_ref.draw(z[b], u[b], T, k, p, m) for b in range(rows)]
        sure = np.array([x for _, x in want]) > NEAR
        assert not st.any() and np.array_equal(tok.cpu().numpy()[sure], np.array([x for x, _ in want])[sure])
        out, _ = sv.spec_filter_logits(t, T, k, top_p=p, min_p=m)
        for b in range(rows):
            low, near = step_ref.kept(z[b], T, k, p, m)
            assert near < NEAR or np.array_equal(out[b].double().cpu().numpy(), np.where(z[b] >= low, z[b], -np.inf))


def test_rows_with_settings_of_their_own(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(3)
    rows, V = 64, 5003
    t, z = logits(rng, rows, V, "bf16", "usual")
    t = t.to(dev)
    T = rng.uniform(0.2, 2, rows).astype(np.float32)
    T[::7] = 0
    k, p = rng.integers(-1, 200, rows).astype(np.int32), rng.uniform(0.2, 1, rows).astype(np.float32)
    p[::3] = 1
    m = np.where(rng.random(rows) < 0.5, 0, rng.uniform(0, 0.2, rows)).astype(np.float32)
    u = rng.random(rows).astype(np.float32)
    d = [torch.from_numpy(x).to(dev) for x in (T, k, p, m, u)]
    tok, st = sv.spec_sample(t, d[4], d[0], d[1], top_p=d[2], min_p=d[3])
    want = [step_ref.draw(z[b], u[b], T[b], k[b], p[b], m[b]) for b in range(rows)]
    checked(z, tok.cpu().numpy(), np.array([x for x, _ in want]), st.cpu().numpy(), np.array([x for _, x in want]))
    # mixed with scalars, over leading dimensions
    out, st = sv.spec_filter_logits(t.view(8, 8, V), d[0].view(8, 8), 30, top_p=d[2].view(8, 8))
    out = out.view(rows, V).double().cpu().numpy()
    assert st.shape == (8, 8) and not st.any()
    for b in range(rows):
        if T[b] == 0:
            want = np.full(V, -np.inf)
            want[np.argmax(z[b])] = z[b].max()
        else:
            want = np.where(z[b] >= step_ref.kept(z[b], T[b], 30, p[b])[0], z[b], -np.inf)
        assert np.array_equal(out[b], want)
    for b, (x, y) in enumerate(zip((T, p, m), ((-1.0, np.nan, np.inf), (0.0, 1.5, np.nan), (-0.1, 1.01, np.nan)))):
        bad = torch.from_numpy(np.concatenate([np.array(y, np.float32), x[3:]])).to(dev)
        args = [bad if i == (0, 2, 3)[b] else e for i, e in enumerate(d)]
        tok, st = sv.spec_sample(t, args[4], args[0], args[1], top_p=args[2], min_p=args[3])
        assert st.tolist() == [-11] * 3 + [0] * (rows - 3) and tok[:3].tolist() == [-1] * 3
        out, st = sv.spec_filter_logits(t, args[0], args[1], top_p=args[2], min_p=args[3])
        assert st.tolist() == [-11] * 3 + [0] * (rows - 3) and torch.isnan(out[:3]).all() and not torch.isnan(out[3:]).any()


def test_row_codes(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(4)
    for dtype in ("bf16", "f32"):
        t, z = logits(rng, 8, 9000, dtype, "usual")
        t[0, 8999], t[1, 0], t[2, :] = float("nan"), float("inf"), -float("inf")
        t[6, :] = -float("inf")
        t[6, 8888] = -3.0  # one token: drawn whatever u
        u = torch.tensor([0.5, 0.5, 0.5, 1.0, -0.1, float("nan"), 0.99, 0.5], device=dev)
        tok, st = sv.spec_sample(t.to(dev), u, 1.0, top_p=0.9)
        assert st.tolist() == [-3, -3, -3, -4, -4, -4, 0, 0] and tok[:7].tolist() == [-1] * 6 + [8888]
        tok, st = sv.spec_sample(t.to(dev), None, 0.0, top_p=0.9)
        assert st.tolist() == [-3] * 3 + [0] * 5 and tok[3:].tolist() == [int(np.argmax(x)) for x in t[3:].double().numpy()]
        out, st = sv.spec_filter_logits(t.to(dev), 1.0, top_p=0.9)
        assert st.tolist() == [-3] * 3 + [0] * 5 and torch.isnan(out[:3]).all() and not torch.isnan(out[3:]).any()


def test_extreme_logits_and_temperatures(dev):
    """Weights relative to the largest, whatever the size of the logits: values near the largest float,
    temperatures down to 2^-126, zeros of either sign, subnormal logits."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    V = 300
    rng = np.random.default_rng(5)
    z = np.tile(rng.standard_normal(V), (7, 1)).astype(np.float32)
    z[0] = np.float32(3e38) * rng.uniform(-1, 1, V)
    z[1] *= np.float32(1e-38)
    z[2] = rng.integers(0, 2, V) * np.float32(-0.0) + 0
    z[2, ::2] = -0.0
    z[3] = -1e30
    z[3, 7] = -1e30 * (1 + 2.0 ** -22)
    z[4] += 1e6
    z[5] = 1e-40 * np.arange(V)
    t = torch.from_numpy(z).to(dev)
    u = np.linspace(0, 0.99, 7).astype(np.float32)
    with np.errstate(over="ignore"):
        for T in (1.0, 1e-6, 2.0 ** -126, 1e30, 3e38):
            for k, p, m in ((0, 0.9, 0.0), (20, 0.9, 0.0), (0, 1.0, 0.3)):
                tok, st = sv.spec_sample(t, torch.from_numpy(u).to(dev), T, k, top_p=p, min_p=m)
                assert not st.any()
                for b in range(7):
                    want, near = step_ref.draw(z[b], u[b], T, k, p, m)
                    assert near < 1e-9 or int(tok[b]) == want, (b, T, k, p, m, near)


def test_unaligned_rows_in_place_and_given_outputs(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(6)
    for dtype in ("bf16", "f32"):
        t, z = logits(rng, 5, 8191, dtype, "usual")
        want = np.stack([np.where(x >= step_ref.kept(x, 1.0, 0, 0.8)[0], x, -np.inf) for x in z])
        flat = torch.empty(5 * 8191 + 3, dtype=t.dtype, device=dev)
        view = flat[3:].view(5, 8191)  # rows at every offset from a 16-byte block
        view.copy_(t)
        out, _ = sv.spec_filter_logits(view, 1.0, top_p=0.8)
        assert np.array_equal(out.double().cpu().numpy(), want)
        other = torch.empty(5 * 8191 + 1, dtype=t.dtype, device=dev)[1:].view(5, 8191)
        st = torch.empty(5, dtype=torch.int32, device=dev)
        ws = torch.randint(0, 255, (sv.sv_filter_workspace_bytes(5, 8191, sv.SV_BF16 if dtype == "bf16" else sv.SV_F32),), dtype=torch.uint8, device=dev)
        got = sv.spec_filter_logits(view, 1.0, top_p=0.8, out=(other, st), workspace=ws)
        assert got[0] is other and got[1] is st and np.array_equal(other.double().cpu().numpy(), want)
        before = flat[:3].clone()
        sv.spec_filter_logits(view, 1.0, top_p=0.8, out=(view, st))
        assert np.array_equal(view.double().cpu().numpy(), want) and (flat[:3] == before).all() | torch.isnan(before).any()
        with pytest.raises(sv.SpecVerifyError, match="PARAM"):
            sv.spec_filter_logits(view[:4], 1.0, top_p=0.8, out=(view[1:], st[:4]))
        with pytest.raises(sv.SpecVerifyError, match="WORKSPACE"):
            sv.spec_filter_logits(view, 1.0, top_p=0.8, workspace=ws[:256])


def test_law(dev):
    """A hundred thousand draws from one row follow the kept distribution."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    z = np.array([2.0, 0.5, -1.0, 1.5, 0.25, -4.0, 1.5, 0.0], np.float32)
    n = 100000
    t = torch.from_numpy(np.tile(z, (n, 1))).to(dev)
    u = torch.from_numpy(np.random.default_rng(7).random(n).astype(np.float32)).to(dev)
    tok, st = sv.spec_sample(t, u, 0.8, top_p=0.85)
    low, _ = step_ref.kept(z.astype(np.float64), 0.8, 0, 0.85)
    p = np.where(z >= low, np.exp(z / 0.8), 0)
    p /= p.sum()
    got = np.bincount(tok.cpu().numpy(), minlength=8)
    assert not st.any() and not got[p == 0].any() and (p == 0).any()
    chi = ((got - n * p)[p > 0] ** 2 / (n * p[p > 0])).sum()
    assert chi < 30  # at most 7 degrees of freedom: beyond 30 once in 10^4


def test_streams_and_graphs(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    t, z = logits(np.random.default_rng(8), 9, 30000, "bf16", "usual")
    t = t.to(dev)
    u = torch.rand(9, device=dev)
    first, _ = sv.spec_sample(t, u, 0.9, 40, top_p=0.9)
    kept, _ = sv.spec_filter_logits(t, 0.9, 40, top_p=0.9)
    torch.cuda.synchronize(dev)
    side = torch.cuda.Stream(dev)
    got = [sv.spec_sample(t, u, 0.9, 40, top_p=0.9, stream=side.cuda_stream)[0] for _ in range(5)]
    torch.cuda.synchronize(dev)
    assert all(torch.equal(x, first) for x in got)
    x, g = t.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tok, st = sv.spec_sample(x, u, 0.9, 40, top_p=0.9)
        out, _ = sv.spec_filter_logits(x, 0.9, 40, top_p=0.9)
    for s in (1.0, -1.0, 1.0):
        x.copy_(t * s)
        g.replay()
        eager, _ = sv.spec_sample(x, u, 0.9, 40, top_p=0.9)
        cut, _ = sv.spec_filter_logits(x, 0.9, 40, top_p=0.9)
        assert torch.equal(tok, eager) and torch.equal(out, cut)
    assert torch.equal(tok, first) and torch.equal(out, kept)


def test_filtered_rows_through_the_verification(dev):
    """Target and draft under one policy: the oracle's verification of the same filtered logits."""
    import torch
    import oracle
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(9)
    B, G, V = 6, 4, 4001
    target = torch.from_numpy(logits(rng, B * (G + 1), V, "f32", "usual")[1]).float().view(B, G + 1, V)
    draft = target[:, :G] + torch.from_numpy(0.5 * rng.standard_normal((B, G, V))).float()
    ft, _ = sv.spec_filter_logits(target.to(dev), 0.8, 50, top_p=0.9)
    fd, _ = sv.spec_filter_logits(draft.contiguous().to(dev), 0.8, 50, top_p=0.9)
    tokens, _ = sv.spec_sample(draft.reshape(B * G, V).to(dev), torch.from_numpy(rng.random(B * G).astype(np.float32)).to(dev), 0.8, 50, top_p=0.9)
    tokens = tokens.view(B, G)
    ua, us = rng.random((B, G)).astype(np.float32), rng.random(B).astype(np.float32)
    acc, out = sv.spec_verify(ft, fd, tokens, torch.from_numpy(ua).to(dev), torch.from_numpy(us).to(dev), 0.8)
    want = oracle.spec_verify_ref(ft.cpu().numpy(), fd.cpu().numpy(), tokens.cpu().numpy(), ua, us, 0.8, 0)
    assert acc.tolist() == want[0].tolist() and out.tolist() == want[1].tolist()  # q(x) > 0: every drafted token was kept


def test_refusals_and_what_stays(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    t = torch.randn((4, 100), device=dev)
    u = torch.rand(4, device=dev)
    for kw, e in ((dict(top_p=0.0), sv.SpecVerifyError), (dict(top_p=1.1), sv.SpecVerifyError), (dict(min_p=-0.1), sv.SpecVerifyError),
                  (dict(min_p=float("nan")), sv.SpecVerifyError), (dict(top_p=float("nan")), sv.SpecVerifyError),
                  (dict(top_p=u[:3]), ValueError), (dict(top_p=u.double()), TypeError), (dict(min_p=u.cpu()), ValueError)):
        with pytest.raises(e):
            sv.spec_sample(t, u, 1.0, **kw)
        with pytest.raises(e):
            sv.spec_filter_logits(t, 1.0, **kw)
    for T in (-1.0, float("inf"), float("nan")):
        with pytest.raises(sv.SpecVerifyError, match="TEMPERATURE"):
            sv.spec_sample(t, u, T, top_p=0.9)
    with pytest.raises(sv.SpecVerifyError, match="NULL"):
        sv.spec_sample(t, None, 1.0, top_p=0.9)
    with pytest.raises(TypeError):
        sv.spec_sample(t, u, 1.0, top_p=0.9, workspace=sv.Workspace())
    with pytest.raises(TypeError):
        sv.spec_filter_logits(t.half(), 1.0)
    with pytest.raises(ValueError):
        sv.spec_filter_logits(t.t(), 1.0)
    # temperature and top-k alone go through the kernels they went through before
    a = sv.spec_sample(t, u, 1.0, 5)
    b = sv.spec_sample(t, u, np.float32(1.0), np.int64(5))
    c = sv.spec_sample(t, u, 1.0, 5, top_p=1.0, min_p=0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[0], c[0])
