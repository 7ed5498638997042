"""Filtered sampling where much of the weight lies in tokens of hardly any each, up to the largest
vocabulary: draws and thresholds are those of the definition wherever a cumulative weight is more than
1e-10 of the total from its threshold.

What the kernels may be off by, relative to the total: a weight is between 1.5e-11 less (half a unit of
2^-35) and 5.1e-11 more (that and the series' next term) than its own, so that a quotient of two sums is
off by at most 6.6e-11; and each of at most 2^24 tokens loses less than 2^-59 of the total in a sum,
2.9e-11 for all of them.  Together below 1e-10.  References are sums of long doubles."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
NEAR = 1e-10
LD = np.longdouble


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_02_amd as sv
    sv.load_library()
    return torch.device("cuda:0")


def one_above_a_level_tail(V, at, low):
    """cum(v): the weight of tokens 0 .. v where token `at` weighs 1 and the others exp(low) each."""
    w = np.exp(LD(low))

    def cum(v):
        v = np.asarray(v, LD)
        return (v + 1) * w + (v >= at) * (1 - w)
    return cum


def near_boundaries(cum, V, at, rng, n, near, far, from_end):
    """n numbers u = j 2^-24 whose token is known, each with its cumulative weight `near` to `far` of the
    total above its threshold: such tokens, `from_end` of a chunk's 8192 at most before its end."""
    total = cum(V - 1)
    j = rng.integers(1 << 23, 1 << 24, 1 << 21)
    u = (j * 2.0 ** -24).astype(np.float32)
    assert np.array_equal(u.astype(np.float64) * 2 ** 24, j)
    t = u.astype(LD) * total
    u, t = u[t > cum(at + 1)], t[t > cum(at + 1)]
    lo = np.floor((t - cum(V // 2)) / (cum(1) - cum(0))).astype(np.int64) + V // 2 + 1  # the first v with cum(v) > t
    assert (cum(lo) > t).all() and (cum(lo - 1) <= t).all()
    over = (cum(lo) - t) / total
    good = (over > near) & (over < far) & (lo % 8192 >= 8192 - from_end) & (lo < V - 1)
    return u[good][:n], lo[good][:n]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_draws_among_many_small_weights(dev, dtype):
    """Half of the weight on one token, the rest in equal parts on a quarter of a million: draws whose
    boundary is 1.1e-10 to 4e-10 of the total away."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    V, rng = 262144, np.random.default_rng(11)
    rows = []
    for low in (-12.375, -12.4375, -12.5, -12.625):  # all of them bf16 numbers
        u, want = near_boundaries(one_above_a_level_tail(V, 100, low), V, 100, rng, 24, 1.1e-10, 4e-10, 3000)
        assert len(u) >= 4
        rows += [(low, a, b) for a, b in zip(u, want)]
    z = torch.empty((len(rows), V), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device=dev)
    z[:] = torch.tensor([x[0] for x in rows], device=dev)[:, None]
    z[:, 100] = 0.0
    u = torch.tensor(np.array([x[1] for x in rows], np.float32), device=dev)
    T = torch.ones(len(rows), device=dev)
    want = [int(x[2]) for x in rows]
    for kw in (dict(), dict(top_k=V - 1), dict(min_p=1e-9)):  # uncut; cuts that keep every token, since equals stay together
        tok, st = sv.spec_sample(z, u, T, **kw)
        assert not st.any() and tok.tolist() == want, kw


def test_draws_at_the_largest_vocabulary(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    V, B, low = 1 << 24, 4, -16.625
    z = torch.full((B, V), low, dtype=torch.bfloat16, device=dev)
    z[:, 5] = 0.0
    cum = one_above_a_level_tail(V, 5, low)
    total = cum(V - 1)
    rng = np.random.default_rng(12)
    T = torch.ones(B, device=dev)
    for _ in range(12):
        u = rng.random(B).astype(np.float32)
        tok, st = sv.spec_sample(z, torch.from_numpy(u).to(dev), T)
        v, t = tok.cpu().numpy().astype(np.int64), u.astype(LD) * total
        assert not st.any()
        before = np.where(v > 0, cum(np.maximum(v - 1, 0)), LD(0))
        assert (before <= t + NEAR * total).all() and (cum(v) > t - NEAR * total).all(), (u, v)


def thresholds(z, out, p):
    """How far (of the total) what is kept misses top_p's definition; rows share the logits z (float64)."""
    order = np.sort(z)[::-1]
    value, count = np.unique(order, return_counts=True)
    value, count = value[::-1], count[::-1]
    upto = np.cumsum(count * np.exp((value - value[0]).astype(LD)))
    total = upto[-1]
    miss = []
    for b in range(len(p)):
        low = float(out[0][b])
        i = int(np.searchsorted(-value, -low))
        assert value[i] == low and int(out[1][b]) == int(count[:i + 1].sum())
        t = LD(p[b]) * total
        before = upto[i - 1] if i else LD(0)
        miss.append(float(max((before - t) / total, (t - upto[i]) / total)))
    return np.array(miss)


@pytest.mark.parametrize("V,rows,dtype", [(152064, 96, "f32"), (262144, 96, "f32"), (600001, 24, "bf16"), (1 << 22, 6, "f32"), (1 << 24, 3, "f32"),
                                          (1 << 24, 3, "bf16")])
@pytest.mark.parametrize("spread", [0.25, 6.0])
def test_thresholds_among_many_small_weights(dev, V, rows, dtype, spread):
    """One token with half of the weight, the rest spread over the vocabulary's others: top-p's threshold
    lies among them.  Written rows and settings of each row's own."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(V + int(spread))
    level = -np.log(V) - np.log((np.exp(spread) - 1) / spread)  # the others weigh about 1 in all
    z = (level + spread * rng.random(V)).astype(np.float32)
    z[V // 3] = 0.0
    row = torch.from_numpy(z).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    z = row.double().numpy()
    t = row.to(dev).expand(rows, V).contiguous()
    p = (0.5 + 0.5 * rng.random(rows)).astype(np.float32)
    out, st = sv.spec_filter_logits(t, 1.0, top_p=torch.from_numpy(p).to(dev), out=(t, torch.empty(rows, dtype=torch.int32, device=dev)))
    assert not st.any()
    kept = out > -float("inf")
    low = torch.where(kept, out, torch.full_like(out, float("inf"))).amin(1).double().cpu().numpy()
    miss = thresholds(z, (low, kept.sum(1).cpu().numpy()), p)
    assert (miss < NEAR).all(), miss.max()
