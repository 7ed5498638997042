"""The paged cache's books and movements (append, commit, resize, fork) against plain references
(tests/cache_ref.py): whole numbers and copied values, so every comparison is exact.  At the end a
whole round, as a serving loop makes it, with the tree verification in the middle."""
import random

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


def i32(x, dev):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def random_cache(rng, L, P, H, D, page, esz):
    E = 16 // esz
    k = rng.integers(-99, 99, (L, P, H, D // E, page, E)).astype(np.float64)
    v = rng.integers(-99, 99, (L, P, H, page // E, D, E)).astype(np.float64)
    return k, v, E


def to_dev(x, esz, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16 if esz == 2 else torch.float32).to(dev)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("esz", [2, 4])
@pytest.mark.parametrize("H,D,page,N,lens,news", [
    (1, 64, 16, 1, [0, 15, 16], None),
    (2, 128, 32, 5, [3, 31, 64, 7], [5, 0, 3, 1]),
    (3, 64, 64, 70, [0, 60, 61], None),
    (1, 256, 16, 200, [5, 0], [200, 123]),
    (2, 16, 256, 9, [250, 300], None),
    (1, 512, 16, 3, [14, 2], None),
    (1, 64, 128, 1024, [1], None),
])
def test_append(dev, esz, H, D, page, N, lens, news):
    import torch
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(D + N)
    B, m = len(lens), news or [N] * len(lens)
    counts = [-(-(n + x) // page) for n, x in zip(lens, m)]
    W, P = max(counts) + 1, sum(counts) + 2
    kp, vp, E = random_cache(rng, 1, P, H, D, page, esz)
    kp, vp = kp[0], vp[0]
    ids, at = rng.permutation(P), 0
    table = np.full((B, W), -1)
    for b in range(B):
        table[b, :counts[b]] = ids[at:at + counts[b]]
        at += counts[b]
    k, v = (rng.integers(-99, 99, (B, N, H, D)).astype(np.float64) for _ in range(2))
    dk, dv, dkp, dvp = (to_dev(x, esz, dev) for x in (k, v, kp, vp))
    fused = torch.zeros((B, N, 2 * H + 1, D), dtype=dk.dtype, device=dev)  # rows of a fused projection
    fused[:, :, :H], fused[:, :, H:2 * H] = dk, dv
    st = sv.spec_cache_append(fused[:, :, :H], fused[:, :, H:2 * H], dkp, dvp, i32(table, dev), i32(lens, dev),
                              n_new=i32(news, dev) if news else None)
    for b in range(B):
        for i in range(m[b]):
            ref.pack_k(k[b, i], lens[b] + i, kp, table[b], page, E)
            ref.pack_v(v[b, i], lens[b] + i, vp, table[b], page, E)
    assert st.tolist() == [0] * B
    assert np.array_equal(dkp.double().cpu().numpy(), kp) and np.array_equal(dvp.double().cpu().numpy(), vp)


def test_append_codes(dev):
    """A sequence that does not fit writes nothing; the others are written."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(1)
    B, N, H, D, page, P, W = 7, 5, 1, 64, 16, 20, 3
    table = np.arange(B * W).reshape(B, W) % (P - 1)
    lens, news = [0, -1, 44, 3, 14, 15, 44], [5, 1, 5, 6, 5, 0, 4]
    table[4, 1] = P      # the second page of 14 .. 18
    table[5, 0] = -5     # nothing is written there
    kp, vp, E = random_cache(rng, 1, P, H, D, page, 2)
    kp, vp = kp[0], vp[0]
    k, v = (rng.integers(-99, 99, (B, N, H, D)).astype(np.float64) for _ in range(2))
    dkp, dvp = to_dev(kp, 2, dev), to_dev(vp, 2, dev)
    st = sv.spec_cache_append(to_dev(k, 2, dev), to_dev(v, 2, dev), dkp, dvp, i32(table, dev), i32(lens, dev), n_new=i32(news, dev))
    assert st.tolist() == [0, -8, -8, -8, -7, 0, 0]
    for b in (0, 6):
        for i in range(news[b]):
            ref.pack_k(k[b, i], lens[b] + i, kp, table[b], page, E)
            ref.pack_v(v[b, i], lens[b] + i, vp, table[b], page, E)
    assert np.array_equal(dkp.double().cpu().numpy(), kp) and np.array_equal(dvp.double().cpu().numpy(), vp)


# ------------------------------------------------------------------ commit

@pytest.mark.parametrize("esz", [2, 4])
@pytest.mark.parametrize("L,H,D,page,N,seed", [(1, 1, 64, 16, 2, 0), (3, 2, 128, 16, 40, 1), (2, 1, 64, 32, 33, 2),
                                              (2, 3, 256, 64, 100, 3), (1, 1, 16, 16, 1024, 4), (1, 1, 512, 128, 17, 5), (1, 2, 48, 16, 25, 6)])
def test_commit(dev, esz, L, H, D, page, N, seed):
    import rejection_sampling_verify_02_amd as sv
    pick, rng = random.Random(seed), np.random.default_rng(seed)
    B = 6
    lens = [pick.randint(0, 3 * page) for _ in range(B)]
    lens[0] = 0
    sizes = [0, N - 1, 1, pick.randint(0, N - 1), min(9, N - 1), (N - 1) // 2]
    paths = [sorted(pick.sample(range(1, N), a)) for a in sizes]
    counts = [-(-(n + N) // page) for n in lens]
    W, P = max(counts) + 1, sum(counts) + 1
    kp, vp, E = random_cache(rng, L, P, H, D, page, esz)
    ids, at = rng.permutation(P), 0
    table = np.full((B, W), -1)
    for b in range(B):
        table[b, :counts[b]] = ids[at:at + counts[b]]
        at += counts[b]
    dkp, dvp = to_dev(kp, esz, dev), to_dev(vp, esz, dev)
    path = np.array([p + [-1] * (N - len(p)) for p in paths])
    new, st = sv.spec_cache_commit(dkp, dvp, i32(table, dev), i32(lens, dev), i32(sizes, dev), i32(path, dev))
    for layer in range(L):
        for b in range(B):
            k, v = ref.unpack(kp[layer], vp[layer], table[b], lens[b] + N, page, E)
            for j, x in enumerate(paths[b]):
                ref.pack_k(k[:, lens[b] + x], lens[b] + 1 + j, kp[layer], table[b], page, E)
                ref.pack_v(v[:, lens[b] + x], lens[b] + 1 + j, vp[layer], table[b], page, E)
    assert st.tolist() == [0] * B and new.tolist() == [n + 1 + a for n, a in zip(lens, sizes)]
    assert np.array_equal(dkp.double().cpu().numpy(), kp) and np.array_equal(dvp.double().cpu().numpy(), vp)


def test_commit_of_chains_and_in_place(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    kp, vp = sv.empty_pages(2, 5, 1, 64, 16, torch.bfloat16, dev)
    lens, acc = i32([0, 30, 7], dev), i32([4, 0, -3], dev)
    table = i32([[0, -1], [1, 2], [3, -1]], dev)
    st = torch.empty(3, dtype=torch.int32, device=dev)
    sv.spec_cache_commit(kp, vp, table, lens, acc, max_new=5, out=(lens, st))
    assert lens.tolist() == [5, 31, 7] and st.tolist() == [0, 0, -3]


def test_commit_codes(dev):
    import rejection_sampling_verify_02_amd as sv
    rng = np.random.default_rng(3)
    B, N, H, D, page, P, W = 8, 6, 1, 64, 16, 16, 2
    kp, vp, E = random_cache(rng, 2, P, H, D, page, 2)
    table = np.arange(B * W).reshape(B, W)
    lens = [3, 3, 3, 27, 3, -2, 14, 27]
    acc = [6, 2, 2, 2, -6, 1, 1, 1]
    path = np.full((B, N), -1)
    path[1, :2], path[2, :2], path[3, :2], path[5, 0], path[6, 0], path[7, 0] = [2, 2], [3, 6], [3, 5], 1, 3, 4
    table[6, 1] = P
    dkp, dvp = to_dev(kp, 2, dev), to_dev(vp, 2, dev)
    new, st = sv.spec_cache_commit(dkp, dvp, i32(table, dev), i32(lens, dev), i32(acc, dev), i32(path, dev))
    assert st.tolist() == [-8, -6, -6, -8, -6, -8, -7, 0]
    assert new.tolist() == [3, 3, 3, 27, 3, -2, 14, 29]
    for layer in range(2):
        k, v = ref.unpack(kp[layer], vp[layer], table[7], 32, page, E)
        ref.pack_k(k[:, 31], 28, kp[layer], table[7], page, E)
        ref.pack_v(v[:, 31], 28, vp[layer], table[7], page, E)
    assert np.array_equal(dkp.double().cpu().numpy(), kp) and np.array_equal(dvp.double().cpu().numpy(), vp)


# ------------------------------------------------------------------ resize and fork

class Both:
    """A pool on the device and its books in Python, driven by the same calls."""

    def __init__(self, dev, P, S, W, page, L=2, H=2, D=64, esz=2, seed=0):
        import rejection_sampling_verify_02_amd as sv
        self.sv, self.dev, self.page, self.esz, self.S, self.P = sv, dev, page, esz, S, P
        self.pool = sv.PagePool.empty(P, S, W, dev)
        self.books = ref.Books(P, S, W, page)
        self.kp, self.vp, self.E = random_cache(np.random.default_rng(seed), L, P, H, D, page, esz)
        self.dk, self.dv = to_dev(self.kp, esz, dev), to_dev(self.vp, esz, dev)
        self.lens = [0] * S
        self.dlens = i32(self.lens, dev)

    def resize(self, keep, want):
        st = self.sv.spec_cache_resize(self.pool, i32(keep, self.dev), i32(want, self.dev), self.dk, self.dv)
        status, copies = self.books.resize(list(keep), list(want))
        k0, v0 = self.kp.copy(), self.vp.copy()
        for old, new, n in copies:
            for t in range(n):
                self.kp[:, new, :, :, t] = k0[:, old, :, :, t]
                self.vp[:, new, :, t // self.E, :, t % self.E] = v0[:, old, :, t // self.E, :, t % self.E]
        assert st.tolist() == status
        self.same()
        return status

    def fork(self, src, dst):
        st = self.sv.spec_cache_fork(self.pool, self.dlens, i32(src, self.dev), i32(dst, self.dev))
        assert st.tolist() == self.books.fork(self.lens, src, dst)
        self.same()

    def set_lens(self, lens):
        self.lens = list(lens)
        self.dlens = i32(lens, self.dev)

    def same(self):
        b = self.books
        assert np.array_equal(self.pool.page_table.cpu().numpy(), b.table())
        assert self.pool.seq_pages.tolist() == [len(r) for r in b.rows]
        assert self.pool.ref_count.tolist() == b.ref
        assert np.array_equal(self.pool.free_map.cpu().numpy(), b.free_map())
        assert self.dlens.tolist() == self.lens
        assert np.array_equal(self.dk.double().cpu().numpy(), self.kp) and np.array_equal(self.dv.double().cpu().numpy(), self.vp)


@pytest.mark.parametrize("esz,page", [(2, 16), (4, 32), (2, 128)])
def test_books_over_random_rounds(dev, esz, page):
    """Growth, truncation, forks, copy on write, refusals, whatever a serving loop does, in turn."""
    pick = random.Random(page)
    S, P, W = 23, 61, 9
    x = Both(dev, P, S, W, page, esz=esz, seed=page)
    refused = copied = 0
    for step in range(60):
        if step % 3 == 2:
            free = [b for b in range(S) if not x.books.rows[b]]
            used = [b for b in range(S) if x.books.rows[b]]
            if free and used:
                dst = pick.sample(free, min(len(free), pick.randint(1, 5)))
                x.fork([pick.choice(used) for _ in dst], dst)
            continue
        keep, want = [], []
        for b in range(S):
            n = x.lens[b]
            act = pick.random()
            if act < 0.25:
                keep.append(n)
                want.append(-1)
            elif act < 0.35:
                keep.append(0)
                want.append(0)
            elif act < 0.5:  # rolled back, maybe into pages that others hold, and written again
                keep.append(pick.randint(0, n))
                want.append(pick.randint(keep[-1], min(W * page, keep[-1] + 3 * page)))
            else:
                keep.append(n)
                want.append(min(W * page, n + pick.randint(0, 2 * page)))
        before = x.books.table()
        status = x.resize(keep, want)
        refused += sum(s == -9 for s in status)
        lens = []
        for b in range(S):
            if want[b] < 0:
                lens.append(x.lens[b])
            else:
                lens.append(want[b] if status[b] == 0 else min(keep[b], len(x.books.rows[b]) * page))
        x.set_lens(lens)
        copied += int((before != x.books.table()).any())
    assert refused and copied


def test_books_of_a_large_pool(dev):
    """More map words than the workgroup has threads, and rows longer than a wave."""
    S, P, W, page = 40, 50021, 900, 16
    x = Both(dev, P, S, W, page, L=1, H=1, D=16)
    pick = random.Random(5)
    want = [pick.randint(0, W * page) for _ in range(S)]
    x.resize([0] * S, want)
    x.set_lens(want)
    x.resize(want, [w // 2 for w in want])
    x.set_lens([w // 2 for w in want])
    x.resize(x.lens, [W * page] * S)


def test_many_sequences(dev):
    """More sequences than the workgroup has threads: as many as a call takes."""
    S, P, W, page = 4096, 6500, 3, 16
    x = Both(dev, P, S, W, page, L=1, H=1, D=16)
    want = [(7 * b) % 40 for b in range(S)]
    status = x.resize([0] * S, want)
    assert -9 in status and 0 in status
    x.set_lens([w if s == 0 else 0 for w, s in zip(want, status)])
    x.resize(x.lens, [0] * S)


def test_resize_codes(dev):
    S, P, W, page = 6, 12, 3, 16
    x = Both(dev, P, S, W, page)
    x.resize([0] * S, [16, 16, 33, 16, 16, 0])
    x.set_lens([16, 10, 33, 16, 16, 0])
    x.resize([16, 17, 33, -1, 16, 0], [17, 16, 49, 16, 49, -1])
    # entries and counts that cannot be: the sequence is left as it is
    x.pool.page_table[0, 1] = P + 7
    x.pool.ref_count[x.books.rows[3][0]] = 0
    before = [t.clone() for t in x.pool]
    st = x.sv.spec_cache_resize(x.pool, i32([16, 0, 0, 0, 0, 0], dev), i32([0, -1, -1, 16, -1, -1], dev), x.dk, x.dv)
    assert st.tolist() == [-7, 0, 0, -7, 0, 0]
    assert all((a == b).all() for a, b in zip(before, x.pool))


def test_fork_codes(dev):
    x = Both(dev, 20, 8, 4, 16)
    x.resize([0] * 8, [40, 17, 0, 0, 0, 0, 0, 5])
    x.set_lens([40, 17, 0, 0, 0, 0, 0, 5])
    #        held dst, twice the same dst, itself, out of range, a dst that is a source, an empty source
    x.fork([0, 0, 1, 0, 3, 0, -1, 8, 0, 4], [1, 2, 2, 0, 5, 8, 6, 6, 3, 6])
    x.pool.page_table[0, 0] = 20
    before = [t.clone() for t in x.pool]
    st = x.sv.spec_cache_fork(x.pool, x.dlens, i32([0], dev), i32([5], dev))
    assert st.tolist() == [-7] and all((a == b).all() for a, b in zip(before, x.pool))


def test_resize_without_pages(dev):
    """Books alone: a pool whose pages are never shared needs no cache to copy in."""
    import rejection_sampling_verify_02_amd as sv
    pool = sv.PagePool.empty(10, 3, 4, dev)
    st = sv.spec_cache_resize(pool, i32([0, 0, 0], dev), i32([20, 64, 200], dev), page_size=16)
    assert st.tolist() == [0, 0, -8]
    assert pool.page_table.tolist() == [[0, 1, -1, -1], [2, 3, 4, 5], [-1] * 4]


def test_captured_and_replayed(dev):
    """A round's books and movements in one graph, replayed against eager calls on a twin."""
    import torch
    import rejection_sampling_verify_02_amd as sv

    def make():
        pool = sv.PagePool.empty(40, 4, 6, dev)
        kp, vp = sv.empty_pages(2, 40, 1, 64, 16, torch.float32, dev)
        lens = i32([0, 0, 0, 0], dev)
        return pool, kp, vp, lens

    gen = torch.Generator(device=dev).manual_seed(3)
    k = torch.randn((4, 5, 1, 64), generator=gen, device=dev)
    acc, path = i32([2, 0, 1, 3], dev), i32([[2, 4, -1, -1, -1], [-1] * 5, [3, -1, -1, -1, -1], [1, 2, 4, -1, -1]], dev)

    def step(pool, kp, vp, lens):
        sv.spec_cache_resize(pool, lens, lens + 5, kp, vp)
        for l in range(2):
            sv.spec_cache_append(k, k + l, kp[l], vp[l], pool.page_table, lens)
        new, st = sv.spec_cache_commit(kp, vp, pool.page_table, lens, acc, path)
        lens.copy_(new)
        sv.spec_cache_resize(pool, lens, lens, kp, vp)

    a, b, c = make(), make(), make()
    step(*c)
    torch.cuda.synchronize(dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*a)
    for _ in range(5):
        g.replay()
        step(*b)
        torch.cuda.synchronize(dev)
        for x, y in zip((*a[0], *a[1:]), (*b[0], *b[1:])):
            assert torch.equal(x, y)


# ------------------------------------------------------------------ a round, as a serving loop makes it

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rounds_of_tree_verification_over_the_cache(dev, dtype):
    """Two layers of attention over a paged cache score draft trees, the tree verification picks
    paths, the commit keeps them; prompts are forked on the way.  After every round the cache must
    hold exactly the entries of each sequence's own tokens, kept here token by token, and the
    attention must be that of the reference over them."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    from test_gpu_attention import check

    tdt, esz = (torch.bfloat16, 2) if dtype == "bf16" else (torch.float32, 4)
    S, N, H, g, D, page, L, V, P, W = 6, 10, 2, 2, 64, 16, 2, 97, 60, 8
    pick, rng = random.Random(7), np.random.default_rng(7)
    E = 16 // esz

    def entry(shape):
        return torch.from_numpy(rng.standard_normal(shape)).to(tdt).to(dev)

    pool = sv.PagePool.empty(P, S, W, dev)
    kp, vp = sv.empty_pages(L, P, H, D, page, tdt, dev)
    kp.fill_(float("nan"))
    vp.fill_(float("nan"))
    lens = i32([0] * S, dev)
    kept = [[] for _ in range(S)]  # per sequence the entries [L, 2, H, D] of its tokens
    prompts = i32([13, 20, 0, 0, 0, 16], dev)
    assert sv.spec_cache_resize(pool, lens, prompts, kp, vp).tolist() == [0] * S
    new = entry((L, 2, S, 20, H, D))
    for l in range(L):
        sv.spec_cache_append(new[l, 0], new[l, 1], kp[l], vp[l], pool.page_table, lens, n_new=prompts)
    for b, n in enumerate(prompts.tolist()):
        kept[b] = [new[:, :, b, t].double().cpu().numpy() for t in range(n)]
    lens.copy_(prompts)
    assert sv.spec_cache_fork(pool, lens, i32([0, 1, 0], dev), i32([2, 3, 4], dev)).tolist() == [0, 0, 0]
    for s, d in ((0, 2), (1, 3), (0, 4)):
        kept[d] = list(kept[s])
    for _ in range(3):
        assert sv.spec_cache_resize(pool, lens, lens + N, kp, vp).tolist() == [0] * S
        parent = np.array([[-1] + [max(0, n - 1 - pick.randrange(4)) for n in range(1, N)] for _ in range(S)], np.int32)
        new, q = entry((L, 2, S, N, H, D)), entry((S, N, H * g, D))
        for l in range(L):
            assert sv.spec_cache_append(new[l, 0], new[l, 1], kp[l], vp[l], pool.page_table, lens).tolist() == [0] * S
            out, st = sv.spec_paged_attention(q, kp[l], vp[l], pool.page_table, lens, parent=i32(parent, dev))

            class C:  # the reference's view: every sequence's own tokens, then its nodes
                B, N, page = S, 10, 16
                news = [10] * S

                @staticmethod
                def expect():
                    host = new.double().cpu().numpy()
                    ks, vs = ([np.stack([t[l, x] for t in kept[b]] + [host[l, x, b, n] for n in range(N)], 1) for b in range(S)]
                              for x in (0, 1))
                    return ref.attention(q.double().cpu().numpy(), ks, vs, [len(t) for t in kept], [N] * S, parent,
                                         1 / np.sqrt(D), 0, 0, esz)

            check(C, out, st)
        logits = torch.randn((2, S, N, V), device=dev)
        tokens, u = torch.randint(0, V, (S, N), device=dev, dtype=torch.int32), torch.rand((S, N + 1), device=dev)
        logits[1] = logits[0]  # a draft that proposes well: many nodes are accepted
        acc, _, path = sv.spec_tree_verify(logits[0], logits[1], tokens, i32(parent, dev), u[:, :N].contiguous(),
                                           u[:, N].contiguous(), 1.0)
        lens, st = sv.spec_cache_commit(kp, vp, pool.page_table, lens, acc, path)
        host = new.double().cpu().numpy()
        for b, (a, p) in enumerate(zip(acc.tolist(), path.tolist())):
            assert a >= 0
            kept[b] += [host[:, :, b, n] for n in [0] + p[:a]]
        assert st.tolist() == [0] * S and lens.tolist() == [len(t) for t in kept]
        assert sv.spec_cache_resize(pool, lens, lens, kp, vp).tolist() == [0] * S
        table, hk, hv = pool.page_table.cpu().numpy(), kp.double().cpu().numpy(), vp.double().cpu().numpy()
        for b in range(S):
            for l in range(L):
                k, v = ref.unpack(hk[l], hv[l], table[b], len(kept[b]), page, E)
                assert np.array_equal(k, np.stack([t[l, 0] for t in kept[b]], 1)) and np.array_equal(v, np.stack([t[l, 1] for t in kept[b]], 1))
    assert sv.spec_cache_resize(pool, lens, i32([0] * S, dev), kp, vp).tolist() == [0] * S
    assert pool.ref_count.sum().item() == 0 and pool.free_map.tolist() == sv.PagePool.empty(P, S, W, dev).free_map.tolist()
