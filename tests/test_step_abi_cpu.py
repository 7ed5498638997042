"""The entry points of positions, of the cache in 4 bits and of filtered sampling refuse bad arguments
before any HIP call: all of it without a GPU."""
import ctypes

import pytest

import rejection_sampling_verify_02_amd as sv

FAKE = 1 << 20  # never dereferenced: argument checks reject before any launch
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not sv.LIB_PATH.exists():
        from rejection_sampling_verify_02_amd import build
        build.build()
    return sv.load_library()


class Rot(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("factor", ctypes.c_float)]


def rotary(lib, rot=(FAKE, 64, 0, 1.0), **kw):
    a = dict(q=FAKE, qb=5120, qn=1024, k=2 * FAKE, kb=1280, kn=256, v=3 * FAKE, vb=1280, vn=256, dt=sv.SV_BF16, kp=FAKE, ks=None, vp=FAKE, vs=None,
             rot=ctypes.byref(Rot(*rot)) if rot else None, table=FAKE, lens=FAKE, news=None, parent=None, pos=None, prior=None,
             B=4, N=5, Hq=8, Hkv=2, D=128, page=16, P=10, W=7, out=64 * FAKE, st=FAKE, stream=None)
    a.update(kw)
    return lib.spec_cache_append_rotary(*a.values())


FOUR = dict(ks=FAKE, vs=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), 3), (dict(dt=sv.SV_F32, **FOUR), 3), (dict(B=0), 2), (dict(N=0), 2), (dict(N=1025), 2), (dict(Hkv=0), 2), (dict(Hq=-1), 2),
    (dict(Hq=0), 2), (dict(q=None), 2), (dict(D=24), 2), (dict(D=528), 2), (dict(D=96, **FOUR), 2), (dict(page=24), 2), (dict(W=0), 2),
    (dict(rot=(FAKE, 63, 0, 1.0)), 2), (dict(rot=(FAKE, 130, 0, 1.0)), 2), (dict(rot=(FAKE, -2, 0, 1.0)), 2), (dict(B=1 << 30), 2),
    (dict(rot=(FAKE, 64, 0, NAN)), 8), (dict(rot=(FAKE, 64, 0, INF)), 8),
    (dict(k=None), 1), (dict(v=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(st=None), 1),
    (dict(out=None), 1), (dict(rot=(None, 64, 0, 1.0)), 1), (dict(ks=FAKE), 1), (dict(vs=FAKE), 1),
    (dict(q=FAKE + 8), 6), (dict(qn=1025), 6), (dict(k=FAKE + 2), 6), (dict(vb=3), 6), (dict(kp=FAKE + 8), 6), (dict(out=64 * FAKE + 4), 6),
    (dict(ks=FAKE + 4, vs=FAKE), 6), (dict(rot=(FAKE + 2, 64, 0, 1.0)), 6),
    (dict(prior=FAKE + 12), 8), (dict(out=FAKE), 8), (dict(out=FAKE + 2 * 5120 * 4 - 16), 8),
])
def test_rotary_refuses(lib, kw, status):
    assert rotary(lib, **kw) == status


def read(lib, **kw):
    a = dict(kp=FAKE, ks=None, vp=FAKE, vs=None, dt=sv.SV_F32, table=FAKE, first=FAKE, count=None, B=4, N=5, Hkv=2, D=128, page=16, P=10, W=7,
             k=FAKE, v=FAKE, st=3 * FAKE, stream=None)
    a.update(kw)
    return lib.spec_cache_read(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dt=9), 3), (dict(**FOUR), 3), (dict(B=0), 2), (dict(N=0), 2), (dict(N=113), 2), (dict(D=0), 2), (dict(dt=0, D=80, page=3), 2),
    (dict(dt=sv.SV_BF16, D=80, **FOUR), 2), (dict(Hkv=1 << 29), 2), (dict(kp=None), 1), (dict(vp=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(first=None), 1), (dict(table=None), 1), (dict(st=None), 1), (dict(dt=sv.SV_BF16, ks=FAKE), 1), (dict(k=FAKE + 4), 6), (dict(kp=FAKE + 4), 6),
    (dict(st=FAKE), 8), (dict(count=3 * FAKE), 8),
])
def test_read_refuses(lib, kw, status):
    assert read(lib, **kw) == status


def attention(lib, **kw):
    a = dict(q=FAKE, qb=5 * 8 * 128, qn=8 * 128, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, table=FAKE, lens=FAKE, news=None, parent=None, prior=None,
             B=4, N=5, Hq=8, Hkv=2, D=128, page=16, P=10, W=7, scale=0.1, window=0, sinks=0, out=FAKE, st=2 * FAKE, ws=FAKE,
             nbytes=1 << 40, stream=None, ev=None, nev=0, n=None)
    a.update(kw)
    return lib.spec_paged_attention4(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 2), (dict(N=0), 2), (dict(N=1025), 2), (dict(Hkv=0), 2), (dict(Hq=7), 2), (dict(D=96), 2), (dict(page=8), 2), (dict(P=0), 2),
    (dict(W=0), 2), (dict(W=1 << 28), 2), (dict(B=1 << 30, W=1 << 20), 2),
    (dict(scale=NAN), 8), (dict(scale=INF), 8), (dict(window=-1), 8), (dict(sinks=-1, window=3), 8), (dict(sinks=2), 8), (dict(prior=2 * FAKE), 8),
    (dict(q=None), 1), (dict(kc=None), 1), (dict(ks=None), 1), (dict(vc=None), 1), (dict(vs=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(out=None), 1), (dict(st=None), 1), (dict(ws=None), 1),
    (dict(q=FAKE + 8), 6), (dict(kc=FAKE + 8), 6), (dict(vs=FAKE + 4), 6), (dict(out=FAKE + 8), 6), (dict(qb=100), 6),
    (dict(nbytes=100), 5), (dict(ws=FAKE + 64), 5),
])
def test_attention4_refuses(lib, kw, status):
    assert attention(lib, **kw) == status


def commit(lib, **kw):
    a = dict(kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, table=FAKE, lens=FAKE, acc=2 * FAKE, path=FAKE, prior=None, L=2, B=4, N=5, Hkv=2, D=128, page=16,
             P=10, W=7, new=4 * FAKE, st=5 * FAKE, stream=None)
    a.update(kw)
    return lib.spec_cache_commit4(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 2), (dict(L=0), 2), (dict(N=0), 2), (dict(N=1025), 2), (dict(D=48), 2), (dict(page=0), 2), (dict(L=1 << 20, Hkv=1 << 20), 2),
    (dict(kc=None), 1), (dict(ks=None), 1), (dict(vc=None), 1), (dict(vs=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(acc=None), 1),
    (dict(new=None), 1), (dict(st=None), 1), (dict(kc=FAKE + 8), 6), (dict(vs=FAKE + 2), 6),
    (dict(new=FAKE), 8), (dict(st=2 * FAKE - 12), 8), (dict(prior=4 * FAKE), 8), (dict(prior=5 * FAKE + 8), 8),
])
def test_commit4_refuses(lib, kw, status):
    assert commit(lib, **kw) == status


def resize(lib, **kw):
    a = dict(table=FAKE, held=FAKE, ref=FAKE, free=FAKE, keep=FAKE, want=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, L=2, S=4, Hkv=2,
             D=128, page=16, P=10, W=7, st=FAKE, ws=FAKE, nbytes=1 << 30, stream=None)
    a.update(kw)
    return lib.spec_cache_resize4(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), 2), (dict(S=4097), 2), (dict(L=0), 2), (dict(D=0), 2), (dict(D=512), 2), (dict(page=100), 2), (dict(P=0), 2), (dict(W=-3), 2),
    (dict(L=1 << 20, Hkv=1 << 20), 2), (dict(kc=None), 1), (dict(ks=None), 1), (dict(vc=None), 1), (dict(vs=None), 1), (dict(table=None), 1),
    (dict(ref=None), 1), (dict(st=None), 1), (dict(ws=None), 1), (dict(vc=FAKE + 8), 6), (dict(ks=FAKE + 1), 6), (dict(nbytes=256), 5), (dict(ws=FAKE + 16), 5),
])
def test_resize4_refuses(lib, kw, status):
    assert resize(lib, **kw) == status


class Policy(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_k", ctypes.c_int32), ("top_p", ctypes.c_float), ("min_p", ctypes.c_float),
                ("temperatures", ctypes.c_void_p), ("top_ks", ctypes.c_void_p), ("top_ps", ctypes.c_void_p), ("min_ps", ctypes.c_void_p)]


def sample(lib, pol=(1.0, 0, 0.9, 0.0), **kw):
    a = dict(z=FAKE, dt=sv.SV_BF16, u=FAKE, B=4, V=1000, pol=ctypes.byref(Policy(*pol)) if pol else None, tok=FAKE, st=FAKE, ws=FAKE,
             nbytes=1 << 30, stream=None, ev=None, nev=0, n=None)
    a.update(kw)
    return lib.spec_sample_filtered(*a.values())


def filtered(lib, pol=(1.0, 0, 0.9, 0.0), **kw):
    a = dict(z=FAKE, dt=sv.SV_F32, rows=4, V=1000, pol=ctypes.byref(Policy(*pol)) if pol else None, out=2 * FAKE, st=FAKE, ws=FAKE,
             nbytes=1 << 30, stream=None, ev=None, nev=0, n=None)
    a.update(kw)
    return lib.spec_filter_logits(*a.values())


SHARED = [
    (dict(dt=5), 3), (dict(V=0), 2), (dict(V=(1 << 24) + 1), 2), (dict(pol=None), 1),
    (dict(pol=(-1.0, 0, 0.9, 0.0)), 4), (dict(pol=(NAN, 0, 0.9, 0.0)), 4), (dict(pol=(INF, 0, 0.9, 0.0)), 4),
    (dict(pol=(1.0, 0, 0.0, 0.0)), 8), (dict(pol=(1.0, 0, 1.01, 0.0)), 8), (dict(pol=(1.0, 0, NAN, 0.0)), 8), (dict(pol=(1.0, 0, 1.0, -0.1)), 8),
    (dict(pol=(1.0, 0, 1.0, 1.1)), 8), (dict(pol=(1.0, 0, 1.0, NAN)), 8),
    (dict(pol=(-1.0, 0, 0.0, 2.0, FAKE, None, FAKE, FAKE), nbytes=0), 5),  # rows' own settings are looked at on the device
    (dict(z=None), 1), (dict(st=None), 1), (dict(ws=None), 1), (dict(z=FAKE + 1), 6), (dict(nbytes=100), 5), (dict(ws=FAKE + 64), 5),
]


@pytest.mark.parametrize("kw,status", SHARED + [(dict(B=0), 2), (dict(tok=None), 1), (dict(u=None), 1), (dict(u=None, pol=(0.0, 0, 0.5, 0.0), nbytes=0), 5),
                                                (dict(u=None, pol=(0.0, 0, 0.5, 0.0, FAKE)), 1)])
def test_sample_refuses(lib, kw, status):
    assert sample(lib, **kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [(dict(rows=0), 2), (dict(rows=1 << 30), 2), (dict(out=None), 1), (dict(out=2 * FAKE + 2), 6),
                                                (dict(out=FAKE + 4), 8), (dict(out=FAKE - 8), 8), (dict(out=FAKE, nbytes=0), 5)])
def test_filter_refuses(lib, kw, status):
    assert filtered(lib, **kw) == status


def test_codes_apart_from_inputs(lib):
    """Row codes on what other workgroups may still have to read of a sequence: refused."""
    far = [FAKE + i * 4096 for i in range(1, 6)]
    for name, last in (("lens", 12), ("news", 12), ("parent", 76), ("pos", 76)):
        own = dict(zip(("lens", "news", "parent", "pos"), far))
        for at in (own[name], own[name] - 12, own[name] + last):
            assert rotary(lib, **{**own, "st": at}) == 8
            if name != "pos":
                assert attention(lib, **{k: v for k, v in own.items() if k != "pos"}, st=at) == 8


def test_outputs_apart_from_settings(lib):
    """An output on u, on a row's settings or on the other output would be read by later kernels: refused."""
    far = [FAKE + i * 4096 for i in range(8)]
    for i in range(4):
        pol = [None] * 4
        pol[i] = far[i]
        for at in (far[i], far[i] + 12, far[i] - 12):
            assert sample(lib, pol=(1.0, 0, 0.9, 0.0, *pol), u=far[4], tok=far[5], st=at) == 8
            assert sample(lib, pol=(1.0, 0, 0.9, 0.0, *pol), u=far[4], tok=at, st=far[5]) == 8
            assert filtered(lib, pol=(1.0, 0, 0.9, 0.0, *pol), st=at) == 8
    assert sample(lib, u=far[4], tok=far[5], st=far[4]) == 8 and sample(lib, u=far[4], tok=far[5], st=far[5] + 8) == 8


def test_sizes_and_plans(lib):
    small, large = (sv.sv_attention4_workspace_bytes(*x) for x in ((1, 1, 8, 8, 64, 16, 1), (64, 32, 32, 8, 128, 64, 1000)))
    assert 256 < small < large and small % 256 == 0 and large % 256 == 0 and sv.sv_attention4_workspace_bytes(1, 1, 8, 8, 80, 16, 1) == 256
    assert sv.sv_attention4_launch_plan(1, 32, 8, 128) == ["k_attn4", "k_attn_join"]
    assert sv.sv_attention4_launch_plan(32, 32, 8, 128) == ["k_attn4_wide", "k_attn_join"]
    assert sv.sv_attention4_launch_plan(32, 32, 8, 100) == []
    small, large = sv.sv_filter_workspace_bytes(1, 1, sv.SV_F32), sv.sv_filter_workspace_bytes(64, 128256, sv.SV_BF16)
    assert 256 < small < large and sv.sv_filter_workspace_bytes(0, 5, sv.SV_F32) == 256 and sv.sv_filter_workspace_bytes(1, 5, 9) == 256
    assert sv.sv_filter_launch_plan(True) == ["k_filter_scan", "k_filter_plan", "k_filter_gather", "k_filter_pick"]
    assert sv.sv_filter_launch_plan(False) == ["k_filter_scan", "k_filter_plan", "k_filter_gather", "k_filter_pick", "k_filter_write"]


def test_binding_refuses_what_is_not_on_the_device():
    import torch
    i32 = dict(dtype=torch.int32)
    table, lens = torch.zeros((3, 2), **i32), torch.zeros(3, **i32)
    q = torch.zeros((3, 1, 4, 64), dtype=torch.bfloat16)
    k, v = sv.empty_pages4(1, 4, 4, 64, 16, "cpu")
    z = torch.zeros((3, 10))
    for call in (lambda: sv.spec_paged_attention(q, k[0], v[0], table, lens), lambda: sv.spec_cache_append(q, q, k[0], v[0], table, lens),
                 lambda: sv.spec_cache_append_rotary(q, q, q, k[0], v[0], table, lens, sv.Rotary.of(64)), lambda: sv.spec_cache_read(k[0], v[0], table, lens, 1),
                 lambda: sv.spec_cache_commit(k, v, table, lens, lens, max_new=1), lambda: sv.spec_sample(z, z[:, 0], 1.0, top_p=0.5),
                 lambda: sv.spec_filter_logits(z, 1.0)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
