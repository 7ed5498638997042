"""The paged cache's entry points refuse bad arguments before any HIP call, and its binding
checks shapes, types and layouts: all of it without a GPU."""
import ctypes

import pytest

import rejection_sampling_verify_02_amd as sv

FAKE = 1 << 20  # never dereferenced: argument checks reject before any launch
V_, I_, F_, Z_, Q_ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not sv.LIB_PATH.exists():
        from rejection_sampling_verify_02_amd import build
        build.build()
    return sv.load_library()


def attention(lib, **kw):
    a = dict(q=FAKE, qb=5 * 8 * 128, qn=8 * 128, k=FAKE, v=FAKE, dt=sv.SV_BF16, table=FAKE, lens=FAKE, news=None, parent=None,
             B=4, N=5, Hq=8, Hkv=2, D=128, page=16, P=10, W=7, scale=0.1, window=0, sinks=0, out=FAKE, st=FAKE, ws=FAKE,
             nbytes=1 << 40, stream=None)
    a.update(kw)
    return lib.spec_paged_attention(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), 3), (dict(dt=-1), 3),
    (dict(B=0), 2), (dict(N=0), 2), (dict(N=1025), 2), (dict(Hkv=0), 2), (dict(Hq=7), 2), (dict(Hq=1), 2), (dict(D=96), 2),
    (dict(page=8), 2), (dict(page=24), 2), (dict(page=512), 2), (dict(P=0), 2), (dict(W=0), 2), (dict(W=1 << 28), 2),
    (dict(B=1 << 30, W=1 << 20), 2),
    (dict(scale=NAN), 8), (dict(scale=INF), 8), (dict(window=-1), 8), (dict(sinks=-1, window=3), 8), (dict(sinks=2), 8),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(out=None), 1),
    (dict(st=None), 1), (dict(ws=None), 1),
    (dict(q=FAKE + 8), 6), (dict(k=FAKE + 2), 6), (dict(v=FAKE + 4), 6), (dict(out=FAKE + 8), 6), (dict(qb=100), 6), (dict(qn=1), 6),
    (dict(nbytes=100), 5), (dict(ws=FAKE + 64), 5),
])
def test_attention_refuses(lib, kw, status):
    assert attention(lib, **kw) == status


def test_attention_workspace_and_plan(lib):
    # any contents will do; more workgroups than the work has are not provided for
    small = sv.sv_attention_workspace_bytes(1, 1, 8, 8, 64, 16, 1, sv.SV_BF16)
    large = sv.sv_attention_workspace_bytes(64, 32, 32, 8, 128, 64, 1000, sv.SV_BF16)
    assert 256 < small < large and small % 256 == 0 and large % 256 == 0
    assert sv.sv_attention_workspace_bytes(64, 32, 32, 8, 100, 64, 1000, sv.SV_BF16) == 256  # a call that is refused
    assert sv.sv_attention_launch_plan(1, 32, 8, 128, sv.SV_BF16) == ["k_attn", "k_attn_join"]
    assert sv.sv_attention_launch_plan(32, 32, 8, 128, sv.SV_BF16) == ["k_attn_wide", "k_attn_join"]
    assert sv.sv_attention_launch_plan(1, 32, 8, 96, sv.SV_BF16) == []


def append(lib, **kw):
    a = dict(k=FAKE, kb=1280, kn=256, v=FAKE, vb=1280, vn=256, dt=sv.SV_BF16, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE, news=None,
             B=4, N=5, Hkv=2, D=128, page=16, P=10, W=7, st=FAKE, stream=None)
    a.update(kw)
    return lib.spec_cache_append(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), 3), (dict(B=0), 2), (dict(N=0), 2), (dict(N=1025), 2), (dict(Hkv=0), 2), (dict(D=8), 2), (dict(D=72), 2),
    (dict(D=528), 2), (dict(page=17), 2), (dict(P=0), 2), (dict(W=0), 2), (dict(B=1 << 30, Hkv=1 << 20), 2),
    (dict(k=None), 1), (dict(v=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(st=None), 1), (dict(k=FAKE + 2), 6), (dict(v=FAKE + 8), 6), (dict(kp=FAKE + 4), 6), (dict(vn=255), 6), (dict(kb=3), 6),
])
def test_append_refuses(lib, kw, status):
    assert append(lib, **kw) == status


def commit(lib, **kw):
    a = dict(kp=FAKE, vp=FAKE, dt=sv.SV_F32, table=FAKE, lens=FAKE, acc=2 * FAKE, path=FAKE, L=2, B=4, N=5, Hkv=2, D=128, page=16,
             P=10, W=7, new=4 * FAKE, st=5 * FAKE, stream=None)
    a.update(kw)
    return lib.spec_cache_commit(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dt=-1), 3), (dict(B=0), 2), (dict(L=0), 2), (dict(N=0), 2), (dict(N=1025), 2), (dict(D=24), 2), (dict(page=0), 2),
    (dict(L=1 << 20, Hkv=1 << 20), 2), (dict(kp=None), 1), (dict(vp=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(acc=None), 1), (dict(new=None), 1), (dict(st=None), 1), (dict(kp=FAKE + 8), 6),
    # lengths that several workgroups read may not be written by the same call
    (dict(new=FAKE), 8), (dict(new=FAKE + 12), 8), (dict(st=FAKE), 8), (dict(new=2 * FAKE), 8), (dict(st=2 * FAKE - 12), 8),
])
def test_commit_refuses(lib, kw, status):
    assert commit(lib, **kw) == status


def resize(lib, **kw):
    a = dict(table=FAKE, held=FAKE, ref=FAKE, free=FAKE, keep=FAKE, want=FAKE, kp=FAKE, vp=FAKE, dt=sv.SV_F32, L=2, S=4, Hkv=2,
             D=128, page=16, P=10, W=7, st=FAKE, ws=FAKE, nbytes=1 << 30, stream=None)
    a.update(kw)
    return lib.spec_cache_resize(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dt=5), 3), (dict(S=0), 2), (dict(S=4097), 2), (dict(L=-1), 2), (dict(D=0), 2), (dict(page=100), 2), (dict(P=0), 2),
    (dict(W=-3), 2), (dict(S=4096, W=1 << 19), 2), (dict(table=None), 1), (dict(held=None), 1), (dict(ref=None), 1), (dict(free=None), 1), (dict(keep=None), 1),
    (dict(want=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(st=None), 1), (dict(ws=None), 1), (dict(vp=FAKE + 8), 6),
    (dict(nbytes=256), 5), (dict(ws=FAKE + 16), 5), (dict(L=0, kp=None, vp=None, Hkv=0, D=0, nbytes=0), 5),
])
def test_resize_refuses(lib, kw, status):
    assert resize(lib, **kw) == status


def fork(lib, **kw):
    a = dict(table=FAKE, held=FAKE, ref=FAKE, lens=FAKE, src=FAKE, dst=FAKE, F=2, S=4, P=10, W=7, st=FAKE, stream=None)
    a.update(kw)
    return lib.spec_cache_fork(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(F=0), 2), (dict(F=4097), 2), (dict(S=0), 2), (dict(S=4097), 2), (dict(P=0), 2), (dict(W=0), 2), (dict(table=None), 1),
    (dict(held=None), 1), (dict(ref=None), 1), (dict(lens=None), 1), (dict(src=None), 1), (dict(dst=None), 1), (dict(st=None), 1),
])
def test_fork_refuses(lib, kw, status):
    assert fork(lib, **kw) == status


def test_binding_refuses_what_is_not_on_the_device():
    import torch
    kp, vp = sv.empty_pages(1, 4, 2, 64, 16, torch.bfloat16, "cpu")
    i32 = dict(dtype=torch.int32)
    table, lens = torch.zeros((3, 2), **i32), torch.zeros(3, **i32)
    q = torch.zeros((3, 1, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        sv.spec_paged_attention(q, kp[0], vp[0], table, lens)
    with pytest.raises(ValueError, match="device tensor"):
        sv.spec_cache_append(q, q, kp[0], vp[0], table, lens)
    with pytest.raises(ValueError, match="device tensor"):
        sv.spec_cache_commit(kp, vp, table, lens, lens, max_new=1)
    pool = sv.PagePool.empty(40, 3, 2, "cpu")
    assert pool.free_map.tolist() == [-1, 255] and pool.page_table.tolist() == [[-1, -1]] * 3
    with pytest.raises(ValueError, match="device tensor"):
        sv.spec_cache_resize(pool, lens, lens, kp, vp)
    with pytest.raises(ValueError, match="device tensor"):
        sv.spec_cache_fork(pool, lens, lens, lens)


def test_checks_of_the_binding():
    """The checks themselves, on CPU tensors (a device tensor differs in its address alone)."""
    import torch
    from rejection_sampling_verify_02_amd import cache
    cpu = -1  # what get_device() says of CPU tensors
    kp, vp = sv.empty_pages(2, 4, 3, 64, 32, torch.float32, "cpu")
    assert kp.shape == (2, 4, 3, 16, 32, 4) and vp.shape == (2, 4, 3, 8, 64, 4)
    assert cache._pages(kp, vp, 6, torch.float32, cpu) == (4, 3, 64, 32)
    assert cache._pages(kp[1], vp[1], 5, torch.float32, cpu) == (4, 3, 64, 32)
    for k, v, n, dt in ((kp, vp, 5, torch.float32), (kp, kp, 6, torch.float32), (kp[:, :, :, ::2], vp[:, :, :, :, ::2], 6, torch.float32),
                        (kp[:1], vp, 6, torch.float32), (kp[..., :2], vp[..., :2], 6, torch.float32)):
        with pytest.raises(ValueError):
            cache._pages(k, v, n, dt, cpu)
    with pytest.raises(TypeError):
        cache._pages(kp, vp, 6, torch.bfloat16, cpu)
    x = torch.zeros((2, 3, 8, 64))
    assert cache._rows(x, "x", (2, 3, 8, 64), torch.float32, cpu)[1:] == (3 * 8 * 64, 8 * 64)
    assert cache._rows(x[:, :1], "x", (2, 1, 8, 64), torch.float32, cpu)[1:] == (3 * 8 * 64, 0)
    assert cache._rows(x[:, :, 2:4], "x", (2, 3, 2, 64), torch.float32, cpu)[1:] == (3 * 8 * 64, 8 * 64)
    for bad in (x[:, :, ::2], x[..., ::2], x.transpose(1, 2)):
        with pytest.raises(ValueError):
            cache._rows(bad, "x", bad.shape, torch.float32, cpu)
    with pytest.raises(TypeError):
        cache._rows(x, "x", (2, 3, 8, 64), torch.bfloat16, cpu)
    i = torch.zeros((2, 3), dtype=torch.int32)
    assert cache._ints(i, "i", (2, 3), cpu) == i.data_ptr() and cache._ints(None, "i", (2, 3), cpu, True) is None
    for bad, e in ((i.long(), TypeError), (None, TypeError), (i[:, ::2], ValueError), (i.t().contiguous().t(), ValueError)):
        with pytest.raises(e):
            cache._ints(bad, "i", tuple(bad.shape) if bad is not None else (2, 3), cpu)
    with pytest.raises(TypeError):
        cache._code(x.half(), "x")
    with pytest.raises(ValueError):
        cache._work(torch.zeros(8), 8, cpu)


def test_sizes_that_are_refused_early():
    import torch
    from rejection_sampling_verify_02_amd import cache
    for kw, e in ((dict(dtype=torch.float16), TypeError), (dict(head_dim=100), ValueError), (dict(head_dim=0), ValueError),
                  (dict(page_size=8), ValueError), (dict(page_size=24), ValueError), (dict(page_size=512), ValueError)):
        a = dict(layers=1, num_pages=2, kv_heads=1, head_dim=64, page_size=16, dtype=torch.float32, device="cpu")
        a.update(kw)
        with pytest.raises(e):
            sv.empty_pages(**a)
    for sizes in ((0, 1, 1), (1, 0, 1), (1, 1, 0)):
        with pytest.raises(ValueError):
            sv.PagePool.empty(*sizes, "cpu")
    # ctypes passes the low 32 bits of an int: 2^32 + 5 would be a window of 5
    assert cache._int32(2**31 - 1, "window") == 2**31 - 1 and cache._int32(-2**31, "window") == -2**31
    for x in (2**31, 2**32 + 5, -2**31 - 1):
        with pytest.raises(ValueError, match="window"):
            cache._int32(x, "window")
