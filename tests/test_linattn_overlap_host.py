"""Host-side checks (no GPU) that what linear attention writes is apart from the small arrays it reads: decays,
lengths, slots and counts.  Addresses are fake and never dereferenced."""

import pytest

from tests.test_linattn_host import FAR, _decode, _prefill, kda  # noqa: F401

O, POOL, STATE, WS = 6 * FAR, 4 * FAR, 5 * FAR, 7 * FAR
O_BYTES = 128 * 512 * 4                       # prefill: 128 rows of 2 heads x 256
STATE_BYTES = 2 * 2 * 256 * 128 * 4
O_DECODE_BYTES, POOL_BYTES = 6 * 512 * 4, 8 * 2 * 256 * 128 * 4


@pytest.mark.parametrize("varlen", [False, True])
@pytest.mark.parametrize("at", [O, O + O_BYTES - 8, O - 4, STATE, STATE + STATE_BYTES - 4, STATE - 4])
def test_prefill_decays(kda, varlen, at):  # noqa: F811
    assert _prefill(kda, varlen, g=at) == 40003


@pytest.mark.parametrize("at", [O, O + O_BYTES - 4, O - 8, STATE + 64, STATE + STATE_BYTES - 4, STATE - 8])
def test_prefill_lengths(kda, at):  # noqa: F811
    assert _prefill(kda, True, cu=at) == 40003


@pytest.mark.parametrize("kw", [dict(g=WS), dict(g=WS + 1024), dict(cu=WS + 16), dict(cu=WS - 8)])
def test_prefill_workspace(kda, kw):  # noqa: F811
    assert _prefill(kda, True, raw=0, **kw) == 40003


@pytest.mark.parametrize("name,size", [("g", 8), ("slots", 12), ("so", 12), ("keep", 12)])
@pytest.mark.parametrize("begin,end", [(O, O + O_DECODE_BYTES), (POOL, POOL + POOL_BYTES)])
def test_decode(kda, name, size, begin, end):  # noqa: F811
    for at in (begin, end - 4, begin - size + 4):
        assert _decode(kda, **{name: at}) == 40003
