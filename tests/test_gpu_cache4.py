"""The cache in 4 bits: append (rotated or not), read back, commit, copy on write, against
tests/step_ref.py.  Codes are whole numbers and every comparison is exact: the decisions of the
rounding are those of float32 values, which the rotation reaches from 64 bits on both sides."""
import random

import numpy as np
import pytest

import cache_ref as ref
import step_ref
from step_ref import Pool4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_02_amd as sv
    sv.load_library()
    return torch.device("cuda:0")


def i32(x, dev):
    import torch
    return None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def to_pages(pools, values, dev):
    """Pages4 of every layer."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    codes, scales = zip(*(p.arrays(values) for p in pools))
    return sv.Pages4(torch.from_numpy(np.stack(codes)).to(dev), torch.from_numpy(np.stack(scales)).to(dev))


def same(pages, pools, values):
    for layer, p in enumerate(pools):
        codes, scales = p.arrays(values)
        assert np.array_equal(pages.scales[layer].cpu().numpy(), scales)
        assert np.array_equal(pages.codes[layer].cpu().numpy(), codes)


def tables(rng, counts, extra=2):
    W, P = max(1, max(counts)) + 1, sum(counts) + extra
    ids, at = rng.permutation(P), 0
    table = np.full((len(counts), W), -1)
    for b, n in enumerate(counts):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, P


def bf16(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("rot", [None, (64, False), (24, False), (62, True)])
@pytest.mark.parametrize("H,D,page,N,lens,news", [
    (1, 64, 16, 1, [0, 15, 16], None),
    (2, 128, 32, 5, [3, 31, 64, 7], [5, 0, 3, 1]),
    (3, 64, 64, 70, [0, 60, 61], None),
    (1, 256, 16, 200, [5, 0], [200, 123]),
    (2, 256, 256, 9, [250, 300], None),
    (1, 128, 128, 1024, [1], None),
])
def test_append_and_read(dev, rot, H, D, page, N, lens, news):
    import torch
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(D + N)
    B, m = len(lens), news or [N] * len(lens)
    table, P = tables(rng, [-(-(n + x) // page) for n, x in zip(lens, m)])
    kp, vp = Pool4(rng, P, H, page, D), Pool4(rng, P, H, page, D)
    spread = np.exp(rng.standard_normal((B, N, H, D // 32, 1)) * 3)  # blocks of very different sizes
    k, v = (bf16((rng.standard_normal((B, N, H, D // 32, 32)) * spread).reshape(B, N, H, D)) for _ in range(2))
    k[0, 0, 0, :32] = 0
    v[0, 0, 0, :32] = np.tile([0.25, -0.75, 1.25, 1.75, 2.5, -3.5, 5, 6], 4)  # ties
    dk, dv = to_pages([kp], False, dev), to_pages([vp], True, dev)
    fused = torch.zeros((B, N, 2 * H + 1, D), dtype=torch.bfloat16, device=dev)  # rows of a fused projection
    fused[:, :, :H], fused[:, :, H:2 * H] = (torch.from_numpy(x).to(dev) for x in (k, v))
    args = (fused[:, :, :H], fused[:, :, H:2 * H], dk[0], dv[0], i32(table, dev), i32(lens, dev))
    want_k = k
    if rot is None:
        st = sv.spec_cache_append(*args, n_new=i32(news, dev))
    else:
        R = D * rot[0] // 64
        f = (10000.0 ** (-np.arange(0, R, 2) / R)).astype(np.float32)
        turn = sv.Rotary(torch.from_numpy(f).to(dev), rot[1], 1.5)
        _, st = sv.spec_cache_append_rotary(None, *args, turn, n_new=i32(news, dev))
        want_k, _ = step_ref.turn(k, np.array(lens)[:, None] + np.arange(N), f, rot[1], 1.5)
    for b in range(B):
        for i in range(m[b]):
            kp.put(want_k[b, i].astype(np.float32), lens[b] + i, table[b])
            vp.put(v[b, i], lens[b] + i, table[b])
    assert st.tolist() == [0] * B
    same(dk, [kp], False)
    same(dv, [vp], True)
    got_k, got_v, st = sv.spec_cache_read(dk[0], dv[0], i32(table, dev), i32(lens, dev), N, count=i32(news, dev))
    assert st.tolist() == [0] * B
    got_k, got_v = got_k.double().cpu().numpy(), got_v.double().cpu().numpy()
    for b in range(B):
        for i in range(N):
            if i < m[b]:
                assert np.array_equal(got_k[b, i], kp.value(lens[b] + i, table[b])) and np.array_equal(got_v[b, i], vp.value(lens[b] + i, table[b]))
            else:
                assert not got_k[b, i].any() and not got_v[b, i].any()


def test_every_code_and_scale(dev):
    """Values at, just under and just over every border, at every scale; zero, the smallest and the
    largest numbers; blocks that are not finite."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    one = np.concatenate([border, border * (1 + 2.0 ** -7), border * (1 - 2.0 ** -8), [6.0, 0.0, -0.0, 1.0, 4.0, 3.0, 2.0, 0.5, -6.0, -1.5, -5.0]])
    assert one.size == 32
    rows = [np.ldexp(one, e) for e in range(-125, 125)]
    rows += [np.full(32, x) for x in (0.0, 1e-39, 2.0 ** -123, 3.3e38, -3.3e38)] + [np.eye(32)[0] * x for x in (3.2e38, 2.5e38, 1e-30)]
    x = bf16(np.stack(rows))
    n = x.shape[0]
    x = np.concatenate([x, -x], -1)[None, :, None, :]  # [1, n, 1, 64]
    bad = x.copy()
    bad[0, 3, 0, 5], bad[0, 4, 0, 40], bad[0, 5, 0, 63] = np.nan, np.inf, -np.inf
    rng = np.random.default_rng(0)
    table, P = tables(rng, [-(-n // 16)])
    for y in (x, bad):
        kp, vp = Pool4(rng, P, 1, 16, 64), Pool4(rng, P, 1, 16, 64)
        dk, dv = to_pages([kp], False, dev), to_pages([vp], True, dev)
        t = torch.from_numpy(y).to(torch.bfloat16).to(dev)
        st = sv.spec_cache_append(t, t, dk[0], dv[0], i32(table, dev), i32([0], dev))
        for i in range(n):
            kp.put(y[0, i], i, table[0])
            vp.put(y[0, i], i, table[0])
        assert st.tolist() == [0]
        same(dk, [kp], False)
        same(dv, [vp], True)
        k, v, _ = sv.spec_cache_read(dk[0], dv[0], i32(table, dev), i32([0], dev), n)
        want = np.stack([kp.value(i, table[0]) for i in range(n)])
        for got in (k, v):
            assert np.array_equal(got[0].double().cpu().numpy(), want, equal_nan=True)
    assert np.isnan(want[3, 0, :32]).all() and np.isfinite(want[3, 0, 32:]).all() and np.isnan(want[4:6, 0, 32:]).all()


def test_error_of_four_bits():
    """What the format costs normal values: the root mean square of the error against the values'.
    With a block's largest of 32 between 3 and 6 scales the steps are a half below 2, one to 4 and
    two to 6; measured in float64, 0.10 to 0.13 of the values."""
    x = np.random.default_rng(0).standard_normal((2000, 128)).astype(np.float32)
    err = np.linalg.norm(step_ref.decode(*step_ref.encode(x)) - x) / np.linalg.norm(x)
    assert 0.09 < err < 0.14


def test_append_and_read_codes(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(1)
    B, N, H, D, page, P, W = 8, 5, 1, 64, 16, 30, 3
    table = np.arange(B * W).reshape(B, W) % (P - 1)
    lens, news = [0, -1, 44, 3, 14, 15, 44, 2], [5, 1, 5, 6, 5, 0, 4, 3]
    table[4, 1] = P      # the second page of 14 .. 18
    table[5, 0] = -5     # nothing is written there
    kp, vp = Pool4(rng, P, H, page, D), Pool4(rng, P, H, page, D)
    k, v = (bf16(rng.standard_normal((B, N, H, D))) for _ in range(2))
    dk, dv = to_pages([kp], False, dev), to_pages([vp], True, dev)
    t = lambda x: torch.from_numpy(x).to(torch.bfloat16).to(dev)  # noqa: E731
    st = sv.spec_cache_append(t(k), t(v), dk[0], dv[0], i32(table, dev), i32(lens, dev), n_new=i32(news, dev),
                              prior=i32([0] * 7 + [-9], dev))
    assert st.tolist() == [0, -8, -8, -8, -7, 0, 0, -9]
    for b in (0, 6):
        for i in range(news[b]):
            kp.put(k[b, i], lens[b] + i, table[b])
            vp.put(v[b, i], lens[b] + i, table[b])
    same(dk, [kp], False)
    same(dv, [vp], True)
    k, v, st = sv.spec_cache_read(dk[0], dv[0], i32(table, dev), i32(lens, dev), N, count=i32(news, dev))
    assert st.tolist() == [0, -8, -8, -8, -7, 0, 0, 0]
    assert torch.isnan(k[1:5]).all() and torch.isnan(v[1:5]).all() and not k[5].any() and torch.isfinite(k[6]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,D,page,N,lens,count", [(2, 64, 16, 20, [0, 5, 31], [20, 0, 7]), (1, 512, 64, 3, [62], None), (3, 48, 256, 9, [250, 1], None)])
def test_read_of_other_types(dev, dtype, H, D, page, N, lens, count):
    import torch
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(D)
    dt, E = (torch.bfloat16, 8) if dtype == "bf16" else (torch.float32, 4)
    m = count or [N] * len(lens)
    table, P = tables(rng, [-(-(n + x) // page) for n, x in zip(lens, m)])
    kp = rng.integers(-99, 99, (P, H, D // E, page, E)).astype(np.float64)
    vp = rng.integers(-99, 99, (P, H, page // E, D, E)).astype(np.float64)
    dk, dv = (torch.from_numpy(x).to(dt).to(dev) for x in (kp, vp))
    k, v, st = sv.spec_cache_read(dk, dv, i32(table, dev), i32(lens, dev), N, count=i32(count, dev))
    assert st.tolist() == [0] * len(lens) and k.dtype == v.dtype == dt
    for b, n in enumerate(lens):
        want_k, want_v = ref.unpack(kp, vp, table[b], n + m[b], page, E)
        assert np.array_equal(k[b, :m[b]].double().cpu().numpy(), want_k[:, n:].transpose(1, 0, 2)) and not k[b, m[b]:].any()
        assert np.array_equal(v[b, :m[b]].double().cpu().numpy(), want_v[:, n:].transpose(1, 0, 2)) and not v[b, m[b]:].any()


@pytest.mark.parametrize("L,H,D,page,N,seed", [(1, 1, 64, 16, 2, 0), (3, 2, 128, 16, 40, 1), (2, 1, 64, 32, 33, 2), (2, 3, 256, 64, 100, 3),
                                              (1, 1, 128, 16, 1024, 4)])
def test_commit(dev, L, H, D, page, N, seed):
    import rejection_sampling_verify_02_amd as sv
    pick, rng = random.Random(seed), np.random.default_rng(seed)
    B = 6
    lens = [0] + [pick.randint(0, 3 * page) for _ in range(B - 1)]
    sizes = [0, N - 1, 1, pick.randint(0, N - 1), min(9, N - 1), (N - 1) // 2]
    paths = [sorted(pick.sample(range(1, N), a)) for a in sizes]
    table, P = tables(rng, [-(-(n + N) // page) for n in lens], 1)
    kp, vp = ([Pool4(rng, P, H, page, D) for _ in range(L)] for _ in range(2))
    dk, dv = to_pages(kp, False, dev), to_pages(vp, True, dev)
    path = np.array([p + [-1] * (N - len(p)) for p in paths])
    new, st = sv.spec_cache_commit(dk, dv, i32(table, dev), i32(lens, dev), i32(sizes, dev), i32(path, dev))
    for pool in kp + vp:
        for b in range(B):
            for j, x in enumerate(paths[b]):
                pool.set(pool.get(lens[b] + x, table[b]), lens[b] + 1 + j, table[b])
    assert st.tolist() == [0] * B and new.tolist() == [n + 1 + a for n, a in zip(lens, sizes)]
    same(dk, kp, False)
    same(dv, vp, True)


def test_commit_codes_and_chains(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(3)
    B, N, H, D, page, P, W = 9, 6, 1, 64, 16, 18, 2
    kp, vp = ([Pool4(rng, P, H, page, D) for _ in range(2)] for _ in range(2))
    table = np.arange(B * W).reshape(B, W)
    lens = [3, 3, 3, 27, 3, -2, 14, 27, 5]
    acc = [6, 2, 2, 2, -6, 1, 1, 1, 1]
    path = np.full((B, N), -1)
    path[1, :2], path[2, :2], path[3, :2], path[5, 0], path[6, 0], path[7, 0], path[8, 0] = [2, 2], [3, 6], [3, 5], 1, 3, 4, 3
    table[6, 1] = P
    dk, dv = to_pages(kp, False, dev), to_pages(vp, True, dev)
    new, st = sv.spec_cache_commit(dk, dv, i32(table, dev), i32(lens, dev), i32(acc, dev), i32(path, dev), prior=i32([0] * 8 + [-9], dev))
    assert st.tolist() == [-8, -6, -6, -8, -6, -8, -7, 0, -9]
    assert new.tolist() == [3, 3, 3, 27, 3, -2, 14, 29, 5]
    for pool in kp + vp:
        pool.set(pool.get(31, table[7]), 28, table[7])
    same(dk, kp, False)
    same(dv, vp, True)
    lens, st = i32([0, 30, 7], dev), torch.empty(3, dtype=torch.int32, device=dev)
    sv.spec_cache_commit(dk, dv, i32(table[:3], dev), lens, i32([4, 0, -3], dev), max_new=5, out=(lens, st))
    assert lens.tolist() == [5, 31, 7] and st.tolist() == [0, 0, -3]


@pytest.mark.parametrize("L,H,D,page", [(2, 2, 64, 16), (1, 1, 128, 64), (3, 1, 256, 32)])
def test_forks_are_copied_on_write(dev, L, H, D, page):
    """Random growth, forks and shrinking with a pool that runs out: the books as the model says, the
    kept slots alone copied."""
    import rejection_sampling_verify_02_amd as sv
    rng, pick = np.random.default_rng(D), random.Random(D)
    P, S, W = 24, 6, 6
    pool, books = sv.PagePool.empty(P, S, W, dev), ref.Books(P, S, W, page)
    kp, vp = ([Pool4(rng, P, H, page, D) for _ in range(L)] for _ in range(2))
    dk, dv = to_pages(kp, False, dev), to_pages(vp, True, dev)
    lens, dlens, refused, copied = [0] * S, i32([0] * S, dev), 0, 0
    for step in range(33):
        free = [b for b in range(S) if not books.rows[b]]
        held = [b for b in range(S) if books.rows[b]]
        if step == 1 or (step > 2 and free and held and pick.random() < 0.5):
            s, d = pick.choice(held), pick.choice(free)
            st = sv.spec_cache_fork(pool, dlens, i32([s], dev), i32([d], dev))
            assert st.tolist() == books.fork(lens, [s], [d])
        else:
            keep = [min(n, len(r) * page) for n, r in zip(lens, books.rows)]
            want = [n + pick.randint(0, 2 * page) if pick.random() < 0.6 else pick.choice([-1, n, 0]) for n in keep]
            if step in (0, 2):  # a sequence that is forked inside a page, then both write
                want = [[page + 5 if b == 0 else -1 for b in range(S)], [n + 3 if n else -1 for n in keep]][step // 2]
            keep = [min(k, w) if w >= 0 else k for k, w in zip(keep, want)]
            want = [min(w, W * page) for w in want]
            st = sv.spec_cache_resize(pool, i32(keep, dev), i32(want, dev), dk, dv)
            status, copies = books.resize(keep, want)
            before = [(p.code.copy(), p.byte.copy()) for p in kp + vp]
            for old, new, n in copies:
                copied += 1
                for p, (code, byte) in zip(kp + vp, before):
                    p.code[new, :, :n], p.byte[new, :, :n] = code[old, :, :n], byte[old, :, :n]
            assert st.tolist() == status
            refused += -9 in status
            lens = [w if w >= 0 and s == 0 else k for k, w, s in zip(keep, want, status)]
            lens = [min(n, len(r) * page) for n, r in zip(lens, books.rows)]
            dlens = i32(lens, dev)
        assert np.array_equal(pool.page_table.cpu().numpy(), books.table()) and pool.ref_count.tolist() == books.ref
        same(dk, kp, False)
        same(dv, vp, True)
    assert copied > 0


def test_layers_are_indexed_and_layouts_checked(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    k, v = sv.empty_pages4(3, 5, 2, 128, 32, dev)
    assert k[1].codes.shape == (5, 2, 4, 32, 16) and v[1].codes.shape == (5, 2, 8, 16, 4, 4) and k[2].scales.shape == (5, 2, 4, 32)
    assert k[1].codes.data_ptr() == k.codes[1].data_ptr()
    x = torch.zeros((2, 1, 2, 128), dtype=torch.bfloat16, device=dev)
    table, lens = i32([[0], [1]], dev), i32([0, 0], dev)
    with pytest.raises(IndexError):
        k[0][0]
    for args, e in (((x, x, k, v), ValueError), ((x, x, k[0], k[0]), ValueError), ((x, x, k[0], v[0].codes), TypeError),
                    ((x.float(), x.float(), k[0], v[0]), TypeError), ((x[..., :64], x[..., :64], k[0], v[0]), ValueError),
                    ((x, x, sv.Pages4(k[0].codes.int(), k[0].scales), v[0]), TypeError)):
        with pytest.raises(e):
            sv.spec_cache_append(*args, table, lens)
    with pytest.raises(TypeError, match="bfloat16"):
        sv.spec_paged_attention(x.float(), k[0], v[0], table, lens)
    with pytest.raises(ValueError):
        sv.spec_cache_read(k[0], v[0], table, lens, 0)
    for kw in (dict(head_dim=96), dict(page_size=8), dict(page_size=48)):
        with pytest.raises(ValueError):
            sv.empty_pages4(**{**dict(layers=1, num_pages=1, kv_heads=1, head_dim=64, page_size=16, device=dev), **kw})
