"""The calls that take an earlier call's row codes refuse what their plain forms refuse, and codes
that overlap their outputs, before any HIP call."""
import pytest

import rejection_sampling_verify_02_amd as sv

FAKE = 1 << 20  # never dereferenced: argument checks reject before any launch


@pytest.fixture(scope="module")
def lib():
    if not sv.LIB_PATH.exists():
        from rejection_sampling_verify_02_amd import build
        build.build()
    return sv.load_library()


def attention(lib, **kw):
    a = dict(q=FAKE, qb=5 * 8 * 128, qn=8 * 128, k=FAKE, v=FAKE, dt=sv.SV_BF16, table=FAKE, lens=FAKE, news=None, parent=None,
             prior=None, B=4, N=5, Hq=8, Hkv=2, D=128, page=16, P=10, W=7, scale=0.1, window=0, sinks=0, out=FAKE, st=FAKE, ws=FAKE,
             nbytes=1 << 40, stream=None, ev=None, nev=0, nl=None)
    a.update(kw)
    return lib.spec_paged_attention_after(*a.values())


def append(lib, **kw):
    a = dict(k=FAKE, kb=1280, kn=256, v=FAKE, vb=1280, vn=256, dt=sv.SV_BF16, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE, news=None,
             prior=None, B=4, N=5, Hkv=2, D=128, page=16, P=10, W=7, st=FAKE, stream=None)
    a.update(kw)
    return lib.spec_cache_append_after(*a.values())


def commit(lib, **kw):
    a = dict(kp=FAKE, vp=FAKE, dt=sv.SV_F32, table=FAKE, lens=FAKE, acc=2 * FAKE, path=FAKE, prior=None, L=2, B=4, N=5, Hkv=2, D=128,
             page=16, P=10, W=7, new=4 * FAKE, st=5 * FAKE, stream=None)
    a.update(kw)
    return lib.spec_cache_commit_after(*a.values())


@pytest.mark.parametrize("kw,status", [(dict(dt=7), 3), (dict(D=96), 2), (dict(q=None), 1), (dict(q=FAKE + 8), 6), (dict(nbytes=100), 5),
                                       (dict(sinks=2), 8), (dict(prior=FAKE), 8), (dict(prior=FAKE + 12), 8), (dict(prior=FAKE - 12), 8)])
def test_attention_refuses(lib, kw, status):
    assert attention(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(dt=2), 3), (dict(N=1025), 2), (dict(k=None), 1), (dict(kn=255), 6),
                                       (dict(prior=FAKE), 8), (dict(prior=FAKE + 12), 8), (dict(prior=FAKE - 12), 8)])
def test_append_refuses(lib, kw, status):
    assert append(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(dt=-1), 3), (dict(L=0), 2), (dict(acc=None), 1), (dict(kp=FAKE + 8), 6), (dict(new=FAKE), 8),
                                       (dict(prior=4 * FAKE), 8), (dict(prior=5 * FAKE + 12), 8), (dict(prior=5 * FAKE, path=None), 8)])
def test_commit_refuses(lib, kw, status):
    assert commit(lib, **kw) == status


def test_binding_checks_the_codes():
    import torch
    from rejection_sampling_verify_02_amd import cache
    ok = torch.zeros(3, dtype=torch.int32)
    assert cache._ints(ok, "prior", (3,), -1, True) == ok.data_ptr()
    for bad, e in ((ok.long(), TypeError), (ok[:2], ValueError), (torch.zeros(6, dtype=torch.int32)[::2], ValueError)):
        with pytest.raises(e, match="prior"):
            cache._ints(bad, "prior", (3,), -1, True)
