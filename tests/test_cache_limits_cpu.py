"""Sizes at which a launch would have 2^32 threads are refused before anything is enqueued (a launch
of that size fails, behind kernels that a call may have enqueued before it)."""
import pytest

import rejection_sampling_verify_02_amd as sv

FAKE = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not sv.LIB_PATH.exists():
        from rejection_sampling_verify_02_amd import build
        build.build()
    return sv.load_library()


# Every call below leaves a required pointer out: sizes that are taken end with SV_ERR_NULL (1),
# sizes that are not with SV_ERR_SHAPE (2).

@pytest.mark.parametrize("B,N,Hq,Hkv,D,dt,status", [
    (1024, 1024, 64, 8, 128, sv.SV_BF16, 2),   # 8192 units of 64 tiles of 128 rows: 2^26 rows, a wave each
    (1023, 1024, 64, 8, 128, sv.SV_BF16, 1),
    (1 << 22, 1, 1, 1, 64, sv.SV_BF16, 2),     # 2^22 units of 16 rows, one of them used
    ((1 << 22) - 1, 1, 1, 1, 64, sv.SV_BF16, 1),
    (1 << 20, 9, 1, 1, 256, sv.SV_F32, 1),
    (1 << 20, 17, 1, 1, 256, sv.SV_F32, 2),
])
def test_attention(lib, B, N, Hq, Hkv, D, dt, status):
    rc = lib.spec_paged_attention(FAKE, N * Hq * D, Hq * D, FAKE, FAKE, dt, FAKE, FAKE, None, None, B, N, Hq, Hkv, D, 256, 10, 4, 0.1, 0, 0,
                                  FAKE, FAKE, None, 0, None)
    assert rc == status
    assert (sv.sv_attention_workspace_bytes(B, N, Hq, Hkv, D, 256, 4, dt) == 256) == (status == 2)


@pytest.mark.parametrize("B,N,Hkv,status", [(1 << 20, 1, 16, 2), ((1 << 20) - 1, 1, 16, 1), (1 << 19, 2, 16, 2), ((1 << 19) - 1, 2, 16, 1),
                                            (1 << 24, 1, 1, 2), ((1 << 24) - 1, 1, 1, 1)])
def test_append(lib, B, N, Hkv, status):
    assert lib.spec_cache_append(None, Hkv * 64, Hkv * 64, FAKE, Hkv * 64, Hkv * 64, sv.SV_BF16, FAKE, FAKE, FAKE, FAKE, None, B, N, Hkv, 64, 16,
                                 10, 4, FAKE, None) == status


@pytest.mark.parametrize("L,B,Hkv,path,status", [(64, 1 << 14, 16, FAKE, 2), (64, (1 << 14) - 1, 16, FAKE, 1), (64, 1 << 14, 16, None, 1),
                                                 (1, 1 << 24, 1, None, 2), (1, (1 << 24) - 1, 1, None, 1), (1, 1 << 24, 1, FAKE, 2)])
def test_commit(lib, L, B, Hkv, path, status):
    assert lib.spec_cache_commit(None, FAKE, sv.SV_BF16, FAKE, FAKE, FAKE, path, L, B, 2, Hkv, 64, 16, 10, 4, FAKE, FAKE, None) == status


def test_tensors_whose_sizes_do_not_fit_32_bits():
    """Expanded tensors have any size for nothing; ctypes would pass the low 32 bits, here 3."""
    import torch
    from rejection_sampling_verify_02_amd import cache
    n, cpu = 2**32 + 3, -1
    x = torch.zeros((1, 1, 1, 64))
    for shape in ((1, n, 1, 64), (n, 1, 1, 64), (1, 1, n, 64)):
        with pytest.raises(ValueError, match="32 bits"):
            cache._rows(x.expand(shape), "k", shape, torch.float32, cpu)
    for shape in ((1, n), (n, 1)):
        with pytest.raises(ValueError, match="32 bits"):
            cache._table(torch.zeros((1, 1), dtype=torch.int32).expand(shape), cpu)
    pool = sv.PagePool.empty(8, 2, 2, "cpu")
    with pytest.raises(ValueError, match="32 bits"):
        cache._books(pool._replace(ref_count=pool.ref_count[:1].expand(n)), cpu)


def test_outputs_that_overlap_inputs_are_named():
    """In the binding by the two tensors' names, in the library's text as one of the reasons; the
    text has the scale among the parameters too."""
    import torch
    from rejection_sampling_verify_02_amd import cache
    x = torch.zeros(8, dtype=torch.int32)
    cache._apart({"new_len": x[:4]}, {"cache_len": x[4:], "prior": None})
    for a, b in ((x[:4], x[:4]), (x[:4], x[3:7]), (x[2:6], x[:3])):
        with pytest.raises(ValueError, match="new_len.*cache_len"):
            cache._apart({"row_status": torch.zeros(4, dtype=torch.int32), "new_len": a}, {"prior": None, "cache_len": b})
    assert "overlap" in sv.sv_status_string(8) and "scale" in sv.sv_status_string(8)


def test_remembered_workspace_sizes_are_bounded():
    from rejection_sampling_verify_02_amd import cache
    for f, size in ((cache._attention_bytes, lambda n: (1 + n % 7, 1, 8, 2, 64, 16, 1 + n, sv.SV_BF16)), (cache._resize_bytes, lambda n: (4, 1 + n))):
        most = f.cache_info().maxsize
        assert most is not None and most <= 4096
        for n in range(most + 50):
            f(*size(n))
        assert f.cache_info().currsize == most
        assert f(*size(0)) == getattr(sv, "sv" + f.__name__.replace("_bytes", "_workspace_bytes"))(*size(0))
