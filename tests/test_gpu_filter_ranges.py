"""Filtered sampling over several chunks of a row where a row leaves the fixed point's range (logits or
temperatures at the ends of float32's), where most of a row is masked with a finite value, and where
some rows of a call have no cut at all.  References and what counts as sure as in
tests/test_gpu_filter.py."""
import numpy as np
import pytest

import step_ref

pytestmark = pytest.mark.gpu
NEAR = 1e-9  # of the references' own sums of float64 exponentials, whose arguments are up to 10^6 large


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_02_amd as sv
    sv.load_library()
    return torch.device("cuda:0")


def check(dev, z, dtype, u, T, k, p, m, least):
    """Draws and filtered rows of z against the reference; at least `least` of the rows are sure."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    rows = len(z)
    t = torch.from_numpy(z).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    z = t.double().numpy()
    t = t.to(dev)
    with np.errstate(over="ignore", under="ignore"):
        tok, st = sv.spec_sample(t, torch.from_numpy(u).to(dev), torch.full((rows,), T, device=dev), k, top_p=p, min_p=m)
        want = [step_ref.draw(z[b], u[b], T, k, p, m) for b in range(rows)]
        assert not st.any()
        sure = np.array([x for _, x in want]) > NEAR
        assert sure.sum() >= least
        assert np.array_equal(tok.cpu().numpy()[sure], np.array([x for x, _ in want])[sure]), (T, k, p, m, tok.tolist(), want)
        out, st = sv.spec_filter_logits(t, T, k, top_p=p, min_p=m)
        assert not st.any()
        out = out.double().cpu().numpy()
        for b in range(rows):
            low, near = step_ref.kept(z[b], T, k, p, m)
            assert near < NEAR or np.array_equal(out[b], np.where(z[b] >= low, z[b], -np.inf)), (b, T, k, p, m)


U = np.array([0.0, 0.3, 0.6, 0.95, 1 - 2.0 ** -24], np.float32)
POLICIES = [(0, 0.9, 0.0), (9000, 1.0, 0.0), (12000, 0.97, 0.0), (0, 1.0, 0.0), (40, 0.9, 0.0), (0, 0.47, 0.3), (0, 1.0, 0.2)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [20011, 60000])
@pytest.mark.parametrize("kind,temperatures", [("usual", (3e38, 1e32)), ("huge", (3e38, 1e36)), ("low", (1.0, 1e28)), ("high", (1.0, 1e29)), ("usual", (2.0 ** -126, 1e-20))])
def test_out_of_range_over_several_chunks(dev, dtype, V, kind, temperatures):
    """All weights alike among more tokens than the list holds; logits over the whole of float32; rows
    far below and far above zero."""
    rng = np.random.default_rng(V)
    n = rng.standard_normal((5, V))
    z = {"usual": n, "huge": 3e38 * (2 * rng.random((5, V)) - 1), "low": -1e30 * (1 + 0.01 * rng.random((5, V))),
         "high": 1e30 * (1 + 0.3 * rng.random((5, V)))}[kind].astype(np.float32)
    for T in temperatures:
        for k, p, m in POLICIES:
            check(dev, z, dtype, U, float(np.float32(T)), k, p, m, 0 if T < 1 else 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e30, "lowest"])
@pytest.mark.parametrize("kind", ["scattered", "stretches", "one left"])
def test_finite_masks(dev, dtype, mask, kind):
    """Vocabularies mostly masked with a number: whole chunks of it, and tokens left here and there."""
    import torch
    V, rng = 50021, np.random.default_rng(23)
    z = (2 * rng.standard_normal((5, V))).astype(np.float32)
    low = float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min) if mask == "lowest" else mask
    if kind == "scattered":
        z[rng.random((5, V)) < 0.95] = low
    elif kind == "stretches":
        z[:, 3000:28000] = low
        z[1, :30000] = low
        z[2, 20000:] = low
    else:
        z[:, :] = low
        z[np.arange(5), [0, 8191, 30000, 41000, V - 1]] = 0.25
    for T in (1.0, 0.3):
        for k, p, m in POLICIES:
            check(dev, z, dtype, U, float(np.float32(T)), k, p, m, 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_rows_as_if_masked_with_infinity(dev, dtype):
    """The same draws and kept logits whatever the mask's value, where it weighs nothing."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    V, rng = 128256, np.random.default_rng(24)
    t = torch.from_numpy((2 * rng.standard_normal((6, V))).astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32).to(dev)
    masked = torch.from_numpy(rng.random((6, V)) < 0.9).to(dev)
    masked[:, 40000:100000] = True
    u = torch.from_numpy(rng.random(6).astype(np.float32)).to(dev)
    T = torch.from_numpy((0.3 + rng.random(6)).astype(np.float32)).to(dev)
    first = None
    for low in (-float("inf"), -1e5, -1e9, -1e30, float(torch.finfo(t.dtype).min)):
        z = t.masked_fill(masked, low)
        got = [sv.spec_sample(z, u, T, k, top_p=p, min_p=m)[0] for k, p, m in ((0, 1.0, 0.0), (0, 0.9, 0.0), (50, 0.95, 0.0), (0, 1.0, 0.05))]
        got.append(sv.spec_filter_logits(z, T, 2000, top_p=0.97)[0])
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(got, first)), low


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_without_cuts_among_others(dev, dtype):
    """Settings of each row's own over several chunks: no cut, one cut each, all, and greedy."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    V, rng = 30011, np.random.default_rng(25)
    kinds = [(0.9, 0, 1.0, 0.0), (0.9, -1, 1.0, 0.0), (0.9, V, 1.0, 0.0), (1.1, 300, 1.0, 0.0), (0.8, 0, 1.0, 0.02), (1.2, 0, 0.9, 0.0), (0.7, 60, 0.9, 0.05), (0.0, 0, 1.0, 0.0)]
    us = [0.0, 2.0 ** -24, 0.25, 0.5, 0.77, 0.999, 1 - 2.0 ** -24]
    rows = [(*s, u) for s in kinds for u in us]
    z = (1.5 * rng.standard_normal((len(rows), V)) - 1.1 * np.log(np.array([rng.permutation(V) for _ in rows]) + 1.0)).astype(np.float32)
    t = torch.from_numpy(z).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    z = t.double().numpy()
    T, k, p, m, u = (np.array(c, d) for c, d in zip(zip(*rows), (np.float32, np.int32, np.float32, np.float32, np.float32)))
    d = [torch.from_numpy(x).to(dev) for x in (T, k, p, m, u)]
    tok, st = sv.spec_sample(t.to(dev), d[4], d[0], d[1], top_p=d[2], min_p=d[3])
    want = [step_ref.draw(z[b], u[b], T[b], k[b], p[b], m[b]) for b in range(len(rows))]
    sure = np.array([x for _, x in want]) > 1e-10
    # u = 0 has its threshold at the first token's own beginning, which is exact
    sure |= u == 0
    assert not st.any() and sure.sum() > 0.9 * len(rows)
    assert np.array_equal(tok.cpu().numpy()[sure], np.array([x for x, _ in want])[sure])
    out, st = sv.spec_filter_logits(t.to(dev), d[0], d[1], top_p=d[2], min_p=d[3])
    out = out.double().cpu().numpy()
    assert not st.any()
    for b in range(len(rows)):
        low = z[b].max() if T[b] == 0 else step_ref.kept(z[b], T[b], k[b], p[b], m[b])[0]
        keep = np.arange(V) == z[b].argmax() if T[b] == 0 else z[b] >= low
        assert np.array_equal(out[b], np.where(keep, z[b], -np.inf)), rows[b]
    # no cut by numbers alone: the rows as they are
    out, st = sv.spec_filter_logits(t.to(dev), 0.9)
    assert not st.any() and torch.equal(out.cpu(), t)


@pytest.mark.parametrize("T", [1.0, 0.01])
def test_rows_around_the_ends_of_the_range(dev, T):
    """Row maxima where |z| / T passes 1.06 * 10^7 and 1.08 * 10^7 (64 z log2(e) / T near 10^9), some
    chunks of the row a little lower, some far below."""
    V, rng = 30011, np.random.default_rng(26)
    edge = np.array([1.0613, 1.06143, 1.0616, 1.0722, 1.0724, 1.08196, 1.0821, 1.085]) * 1e7
    for sign in (-1, 1):
        z = sign * T * edge[:, None] - 0.5 * T * rng.integers(0, 40, (len(edge), V))
        z[:, 8192:16384] -= 12 * T
        z[:, 16384:24576] = sign * T * 1.09e7 - T * 2e6
        z = z.astype(np.float32)
        u = np.linspace(0.05, 0.95, len(edge)).astype(np.float32)
        for k, p, m in ((0, 0.9, 0.0), (9000, 1.0, 0.0), (0, 1.0, 0.0), (0, 1.0, 0.01)):
            check(dev, z, "f32", u, float(np.float32(T)), k, p, m, 4)
