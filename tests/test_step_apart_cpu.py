"""Outputs of positions, of the cache in 4 bits and of filtered sampling that lie on what a call still
reads, or on each other, are refused before any HIP call: all of it without a GPU."""
import pytest

import rejection_sampling_verify_02_amd as sv
from test_step_abi_cpu import FAKE, attention, filtered, lib, read, rotary, sample  # noqa: F401 (lib: the fixture)

PARAM = 8
FAR = [FAKE + i * (1 << 16) for i in range(12)]  # places that nothing of one call reaches from another's


def test_filtered_rows_apart_from_codes_and_settings(lib):
    """4 rows of 1000 float32: 16000 bytes."""
    z, out, st = FAR[0], FAR[1], FAR[2]
    for at in (out, out + 15996, out - 12, out + 8000):
        assert filtered(lib, z=z, out=out, st=at) == PARAM
        for i in range(4):
            pol = [None] * 4
            pol[i] = at
            assert filtered(lib, pol=(1.0, 0, 0.9, 0.0, *pol), z=z, out=out, st=st) == PARAM
    # in place as well
    assert filtered(lib, z=z, out=z, st=z + 400) == PARAM
    assert filtered(lib, pol=(1.0, 0, 0.9, 0.0, z + 400), z=z, out=z, st=st) == PARAM
    # what is written for a row, on the logits that the other workgroups still read
    assert filtered(lib, z=z, out=out, st=z + 15996) == PARAM


@pytest.mark.parametrize("dt,size", [(sv.SV_BF16, 8000), (sv.SV_F32, 16000)])
def test_tokens_and_codes_apart_from_logits(lib, dt, size):
    for at in (FAR[0], FAR[0] + size - 4, FAR[0] - 12):
        assert sample(lib, z=FAR[0], dt=dt, u=FAR[1], tok=at, st=FAR[2]) == PARAM
        assert sample(lib, z=FAR[0], dt=dt, u=FAR[1], tok=FAR[2], st=at) == PARAM


def test_turned_queries_apart_from_what_other_workgroups_read(lib):
    """4 sequences of 5 nodes: queries of 8 heads, keys and values of 2 heads of 128, in bf16."""
    own = dict(q=FAR[0], k=FAR[1], v=FAR[2], out=FAR[3], kp=FAR[4], vp=FAR[5], table=FAR[6], lens=FAR[7], st=FAR[8])
    last = (3 * 1280 + 4 * 256 + 256) * 2 - 16  # the last 16 bytes of keys or values
    for name in ("k", "v"):
        for at in (own["out"], own["out"] + 4 * 5 * 1024 * 2 - 16, own["out"] - last):
            assert rotary(lib, **{**own, name: at}) == PARAM
            assert rotary(lib, **{**own, name: at}, ks=FAR[9], vs=FAR[10]) == PARAM


def test_codes_apart_from_page_tables(lib):
    own = dict(table=FAR[1], lens=FAR[2])
    for at in (FAR[1], FAR[1] - 12, FAR[1] + (4 * 7 - 1) * 4):
        assert rotary(lib, q=FAR[3], k=FAR[4], v=FAR[5], out=FAR[6], **own, st=at) == PARAM
        assert attention(lib, **own, st=at) == PARAM
        assert read(lib, table=FAR[1], first=FAR[2], st=at) == PARAM
