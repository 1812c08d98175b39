"""Host-side checks (no GPU) of the flag that asks linear attention for the recurrence at any length."""

import pytest
import torch

from tests.test_linattn_host import FAR, _decode, _prefill, kda  # noqa: F401


def test_flag(kda):  # noqa: F811
    lib, flag = kda.library(), kda.LINATTN_SEQ
    sizes = (2, 4096, 4, 2, 128, 256)
    assert lib.kda_linattn_workspace_bytes(*sizes, 0) > 0
    for raw in (0, 1):
        assert lib.kda_linattn_workspace_bytes(*sizes, raw | flag) == 0
        assert kda.kda_linattn_workspace_bytes(2, 4096, 4, 2, 256, (torch.float32, torch.bfloat16)[raw],
                                               algo=kda.ALGO_SEQ) == 0
        assert kda.linattn_workspace(2, 4096, 4, "cpu", 2, 256, algo=kda.ALGO_SEQ) is None
    for varlen in (False, True):
        assert _prefill(kda, varlen, raw=2 | flag) == 40007 and _prefill(kda, varlen, raw=2 * flag) == 40007
        # (types keep their rules under the flag: strides of 16 bytes, overlaps)
        assert _prefill(kda, varlen, raw=flag, vs=514) == 40005 and _prefill(kda, varlen, raw=flag, o=FAR) == 40003
    assert _decode(kda, raw=flag) == 40007


@pytest.mark.parametrize("algo", [2, 3, -1])
def test_unknown_forms(kda, algo):  # noqa: F811
    q, g, s = torch.zeros(4, 256), torch.zeros(2), torch.zeros(2, 2, 128, 128)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_linattn_prefill(q, q, q, g, s, s, q, None, N=2, T=2, H=2, algo=algo)
    assert e.value.status == 40007
