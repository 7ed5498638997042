"""Attention where scores are finite and huge: the largest one takes the row, ties share it.

Queries are c u and keys s_t u with u of +-1 and small whole s_t, so that every product and sum is
exact, and scores differ by 10^9 and more: weights are one or zero whatever the rounding, and the
output is the mean of the values at the largest s_t, whole numbers whose halves every type holds."""
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


def one_hot_case(dev, dtype, N, g, D, n, power, sign, seed):
    """A sequence of n committed and N new tokens whose queries are sign 2^power u, and the
    expected rows."""
    import torch
    rng = np.random.default_rng(seed)
    dt, E, page = (torch.bfloat16, 8, 16) if dtype == "bf16" else (torch.float32, 4, 16)
    u = rng.choice([-1.0, 1.0], D)
    T = n + N
    s = rng.integers(-90, 90, T).astype(np.float64)
    s[rng.choice(T, 3)] = 95.0 if sign > 0 else -95.0  # two or three that share the rows behind them
    v = rng.integers(-60, 60, (1, T, D)).astype(np.float64)
    counts = -(-T // page)
    ids = rng.permutation(counts)
    kp, vp = np.zeros((counts, 1, D // E, page, E)), np.zeros((counts, 1, page // E, D, E))
    for t in range(T):
        ref.pack_k((s[t] * u)[None], t, kp, ids, page, E)
        ref.pack_v(v[:, t], t, vp, ids, page, E)
    c = sign * 2.0 ** (power + np.arange(g))
    q = np.tile(c[None, None, :, None] * u, (1, N, 1, 1))
    want = np.zeros((1, N, g, D))
    for i in range(N):
        z = sign * s[:n + i + 1]
        want[0, i] = v[0, :n + i + 1][z == z.max()].mean(0)
    to = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dt).to(dev)  # noqa: E731
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    return dict(q=to(q), k_pages=to(kp), v_pages=to(vp), page_table=i32(ids[None]), cache_len=i32([n])), want


def expected(got, want, dtype):
    # sums of up to three whole numbers are exact, the quotient is rounded once or twice (the
    # reciprocal and the product) in f32, and the output once to the type
    tol = np.abs(want) * (3 * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24))
    nans, off = int(np.isnan(got).sum()), int((np.abs(got - want) > tol).sum())
    assert (nans, off) == (0, 0), f"{nans} of {got.size} outputs are NaN, {off} off"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,g,D,n", [(1, 4, 128, 40), (3, 2, 64, 700), (40, 2, 64, 300), (12, 4, 128, 2500), (2, 1, 256, 5000),
                                     (70, 1, 256, 100)])
@pytest.mark.parametrize("sign", [1, -1])
def test_huge_scores(dev, dtype, N, g, D, n, sign):
    import rejection_sampling_verify_02_amd as sv
    for power in (27, 31, 40, 60):
        t, want = one_hot_case(dev, dtype, N, g, D, n, power, sign, seed=n + power)
        out, st = sv.spec_paged_attention(**t)
        assert st.tolist() == [0]
        expected(out.double().cpu().numpy(), want, dtype)
        flipped, _ = sv.spec_paged_attention(**{**t, "q": -t["q"]}, scale=-1 / np.sqrt(D))
        expected(flipped.double().cpu().numpy(), want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D,n", [(2, 64, 500), (40, 128, 100)])  # both kernels
@pytest.mark.parametrize("power,scale", [(60, 0.0), (105, 0.0), (110, 2.0 ** -122), (112, -2.0 ** -124), (110, 2.0 ** -140)])
def test_scales_down_to_nothing(dev, dtype, N, D, n, power, scale):
    """Scores up to 2^126 under scales that bring them back to ordinary sizes, or to nothing."""
    import rejection_sampling_verify_02_amd as sv
    t, _ = one_hot_case(dev, dtype, N, 1, D, n, power, 1, seed=n + power)
    out, st = sv.spec_paged_attention(**t, scale=scale)
    assert st.tolist() == [0]
    # the same products at an ordinary size, which are exact: queries 2^power smaller, the scale larger
    q = t["q"].double().cpu().numpy() * 2.0 ** -power
    ks, vs = ref.unpack(t["k_pages"].double().cpu().numpy(), t["v_pages"].double().cpu().numpy(), t["page_table"][0].tolist(), n + N, 16,
                        8 if dtype == "bf16" else 4)
    want, tol = ref.attention(q, [ks], [vs], [n], [N], None, scale * 2.0 ** power, 0, 0, 2 if dtype == "bf16" else 4)
    # scales below 2^-126 are held with fewer bits: half of 2^-149, relative to the largest score
    z = abs(scale) * 2.0 ** power * 95 * D
    tol = tol + (2 * z * min(1.0, 2.0 ** -149 / abs(scale)) if scale else 0.0) * np.abs(vs).max()
    # what stands for a scale of zero: 2^-149 times the largest difference of scores
    tol = tol + (0.0 if scale else 2 * 2.0 ** (power - 149) * 190 * D) * np.abs(vs).max()
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D,n", [(2, 64, 500), (40, 128, 100)])
def test_the_largest_scale(dev, dtype, N, D, n):
    import rejection_sampling_verify_02_amd as sv
    t, want = one_hot_case(dev, dtype, N, 2, D, n, 0, 1, seed=n)
    for scale in (1e30, float(np.finfo(np.float32).max)):
        out, st = sv.spec_paged_attention(**t, scale=scale)
        assert st.tolist() == [0]
        expected(out.double().cpu().numpy(), want, dtype)
