"""A decoding step over a paged cache in 4 bits, as a serving loop makes it: pages, rotation and append
in every layer, attention, logits, a draw under the whole policy, the new lengths; and a round with a
draft tree in the middle.  Each part against its own reference on what the part before it left."""
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


class Model:
    """Two layers' projections and an unembedding, random and fixed."""

    def __init__(self, dev, Hq, Hkv, D, V, width=96, layers=2):
        import torch
        g = torch.Generator(device=dev).manual_seed(1)
        r = lambda *s: torch.randn(s, generator=g, device=dev) / s[0] ** 0.5  # noqa: E731
        self.Hq, self.Hkv, self.D, self.V = Hq, Hkv, D, V
        self.embed = r(V, width) * V ** 0.5
        self.qkv = [r(width, (Hq + 2 * Hkv) * D) for _ in range(layers)]
        self.back = [r(Hq * D, width) for _ in range(layers)]
        self.head = r(width, V) * 2

    def step(self, sv, tokens, k_pages, v_pages, table, lens, turn, parent=None, prior=None, keep=None):
        """Logits [B, N, V] of the new tokens; keep: a list that gets what each layer saw and made."""
        import torch
        B, N = tokens.shape
        x = self.embed[tokens.long()]
        for l, (w, back) in enumerate(zip(self.qkv, self.back)):
            heads = (x @ w).to(torch.bfloat16).view(B, N, self.Hq + 2 * self.Hkv, self.D)
            q, k, v = heads.split([self.Hq, self.Hkv, self.Hkv], 2)
            turned, st = sv.spec_cache_append_rotary(q, k, v, k_pages[l], v_pages[l], table, lens, turn, parent=parent, prior=prior)
            out, st2 = sv.spec_paged_attention(turned, k_pages[l], v_pages[l], table, lens, parent=parent, prior=prior)
            if keep is not None:
                keep.append((turned, out, st, st2))
            x = x + (out.float().flatten(2) @ back).nan_to_num()
        return (x @ self.head).float()


def entries(sv, pages_k, pages_v, table, b, n):
    """What the cache holds in the first n slots of sequence b: [Hkv, n, D] float64."""
    import torch
    first = torch.zeros(table.shape[0], dtype=torch.int32, device=table.device)
    count = first.clone()
    count[b] = n
    k, v, _ = sv.spec_cache_read(pages_k, pages_v, table, first, n, count=count)
    return (x[b].double().cpu().numpy().transpose(1, 0, 2) for x in (k, v))


@pytest.mark.parametrize("D,page", [(64, 16), (128, 32)])
def test_decoding_in_four_bits(dev, D, page):
    import torch
    import rejection_sampling_verify_02_amd as sv
    B, Hq, Hkv, V, L = 3, 4, 2, 500, 2
    m = Model(dev, Hq, Hkv, D, V, layers=L)
    pool = sv.PagePool.empty(20, B, 6, dev)
    kp, vp = sv.empty_pages4(L, 20, Hkv, D, page, dev)
    turn = sv.Rotary.of(D, 10000.0, device=dev)
    rng = np.random.default_rng(0)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    lens = i32([0, 0, 0])
    prompts = i32(rng.integers(0, V, (B, 21)))
    T, k, p = torch.tensor([0.8, 0.0, 1.2], device=dev), i32([0, 0, 20]), torch.tensor([0.9, 1.0, 0.95], device=dev)
    feed, n = prompts, 21
    for step in range(5):
        room = sv.spec_cache_resize(pool, lens, lens + n, kp, vp)
        assert room.tolist() == [0] * B
        keep = []
        logits = m.step(sv, feed, kp, vp, pool.page_table, lens, turn, prior=room, keep=keep)
        for l, (q, out, st, st2) in enumerate(keep):
            assert st.tolist() == st2.tolist() == [0] * B
            held = [list(entries(sv, kp[l], vp[l], pool.page_table, b, int(lens[b]) + n)) for b in range(B)]
            want, tol = ref.attention(q.double().cpu().numpy(), [x[0] for x in held], [x[1] for x in held], lens.tolist(), [n] * B, None,
                                      D ** -0.5, 0, 0, 2)
            assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)
        u = rng.random(B).astype(np.float32)
        last = logits[:, -1].contiguous()
        tok, st = sv.spec_sample(last, torch.from_numpy(u).to(dev), T, k, top_p=p)
        z = last.double().cpu().numpy()
        want = [step_ref.draw(z[b], u[b], float(T[b]), int(k[b]), float(p[b])) for b in range(B)]
        assert not st.any() and all(near < 1e-10 or int(tok[b]) == w for b, (w, near) in enumerate(want))
        lens, st = sv.spec_cache_commit(kp, vp, pool.page_table, lens, i32([n - 1] * B), max_new=n, prior=room)
        assert st.tolist() == [0] * B
        feed, n = tok[:, None].contiguous(), 1
    assert lens.tolist() == [21 + 4] * B


def test_a_round_with_a_tree_in_four_bits(dev):
    """Trees verified by the existing operators on filtered logits, accepted paths committed in 4 bits: the
    cache then holds what appending the accepted tokens one after another would have left."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    B, N, Hq, Hkv, D, V, L, page = 4, 9, 4, 2, 64, 60, 2, 16
    m = Model(dev, Hq, Hkv, D, V, layers=L)
    rng = np.random.default_rng(3)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    turn = sv.Rotary.of(D // 2, 10000.0, interleaved=True, device=dev)
    parent = np.full((B, N), -1)
    for j in range(1, N):
        parent[:, j] = np.maximum(0, j - 1 - rng.integers(0, 3, B))
    parent, tokens = i32(parent), i32(rng.integers(0, V, (B, N)))
    lens0 = i32([0, 5, 15, 16])
    pool = sv.PagePool.empty(30, B, 4, dev)
    kp, vp = sv.empty_pages4(L, 30, Hkv, D, page, dev)
    assert sv.spec_cache_resize(pool, torch.zeros_like(lens0), lens0 + N, kp, vp).tolist() == [0] * B
    for x in (kp, vp):  # committed tokens of before
        x.codes.copy_(torch.randint(0, 256, x.codes.shape, dtype=torch.uint8, device=dev))
        x.scales.fill_(124)
    fresh = [sv.Pages4(*(t.clone() for t in x)) for x in (kp, vp)]
    logits = m.step(sv, tokens, kp, vp, pool.page_table, lens0, turn, parent=parent)
    target, st = sv.spec_filter_logits(logits, 1.0, 30, top_p=0.98)
    draft, _ = sv.spec_filter_logits(logits + 0.1, 1.0)  # some distribution with every token in it
    ua, us = torch.rand((B, N), device=dev), torch.rand(B, device=dev)
    acc, out, path = sv.spec_tree_verify(target, draft.contiguous(), tokens, parent, ua, us, 1.0)
    assert (acc >= 0).all()
    new, st = sv.spec_cache_commit(kp, vp, pool.page_table, lens0, acc, path)
    assert st.tolist() == [0] * B and new.tolist() == (lens0 + 1 + acc).tolist()
    # the same tokens as chains: node 0 and the accepted path
    for b in range(B):
        n = int(acc[b]) + 1
        chain = torch.cat([tokens[b, :1], tokens[b, path[b, :n - 1].long()]])[None].contiguous()
        m.step(sv, chain, *fresh, pool.page_table[b:b + 1].contiguous(), lens0[b:b + 1].contiguous(), turn)
        for l in range(L):
            if l == 0:  # its inputs are the tokens' own: exactly the same entries
                for x, y in zip(entries(sv, kp[l], vp[l], pool.page_table, b, int(new[b])), entries(sv, fresh[0][l], fresh[1][l], pool.page_table, b, int(new[b]))):
                    assert np.array_equal(x, y)


def test_a_captured_step_replayed(dev):
    """One graph of a step, replayed while lengths and tokens move on: every replay like the eager step."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    B, Hq, Hkv, D, V, L, page = 3, 4, 2, 64, 300, 2, 16
    m = Model(dev, Hq, Hkv, D, V, layers=L)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    turn = sv.Rotary.of(D, 10000.0, device=dev)
    state = []
    for _ in range(2):
        pool = sv.PagePool.empty(20, B, 5, dev)
        kp, vp = sv.empty_pages4(L, 20, Hkv, D, page, dev)
        lens = i32([3, 15, 30])
        assert sv.spec_cache_resize(pool, torch.zeros_like(lens), lens, kp, vp).tolist() == [0] * B
        state.append((pool, kp, vp, lens, i32([[1], [2], [3]]), torch.rand(B, device=dev)))
    state[1][5].copy_(state[0][5])

    def step(pool, kp, vp, lens, feed, u):
        room = sv.spec_cache_resize(pool, lens, lens + 1, kp, vp)
        logits = m.step(sv, feed, kp, vp, pool.page_table, lens, turn, prior=room)
        tok, st = sv.spec_sample(logits[:, 0].contiguous(), u, 0.9, 30, top_p=0.9)
        new, _ = sv.spec_cache_commit(kp, vp, pool.page_table, lens, torch.zeros_like(lens), max_new=1, prior=room)
        lens.copy_(new)
        feed.copy_(tok[:, None])
        return tok, st

    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        step(*state[0])
        step(*state[1])
    torch.cuda.current_stream(dev).wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tok, st = step(*state[0])
    for _ in range(6):
        g.replay()
        want, _ = step(*state[1])
        torch.cuda.synchronize(dev)
        assert torch.equal(tok, want) and st.tolist() == [0] * B and torch.equal(state[0][3], state[1][3])
    assert state[0][3].tolist() == [3 + 7, 15 + 7, 30 + 7]
    for x, y in zip(state[0][1] + state[0][2], state[1][1] + state[1][2]):
        assert torch.equal(x, y)
