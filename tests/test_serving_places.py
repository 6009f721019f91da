"""Positions are 32-bit: a block table and a batch that could leave that range are refused
before anything is enqueued (the pointers here are made up)."""
import pytest

import exact_tiled_attention_forward_gb300 as fa
from test_serving_abi import APPEND, EXTEND, READ, _caller, lib  # noqa: F401

EDGE = ((1 << 31) - 257) // 128          # pages of a table that leaves no token past 2^31 - 256


@pytest.mark.parametrize("call", [APPEND, READ, EXTEND], ids=["append", "read", "extend"])
def test_positions_stay_in_32_bits(lib, call):  # noqa: F811
    name = {id(APPEND): "fa_cache_append", id(READ): "fa_cache_read", id(EXTEND): "fa_extend_paged"}[id(call)]
    f = _caller(getattr(lib, name), *call)
    small = dict(B=1, Hkv=1, pages=16, T=(1 << 31) - 256 - EDGE * 128)
    if call is EXTEND:
        small.update(Hq=1)
    assert f(**dict(small, max_pages=EDGE)) == fa.FA_ERR_INVALID_ARG
    # one token less is no reason to refuse: the next check (a missing pointer) answers
    assert f(**dict(small, max_pages=EDGE, T=0, cu=0)) == fa.FA_OK
