"""Refusals of the attention-layer calls that test_attention_layer_cpu.py does not have (no GPU needed)."""
import pytest

import uniform_state_text_b200 as dg
from uniform_state_text_b200 import build as dgbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    dgbuild.build()
    return dg.lib()


@pytest.mark.parametrize("limit,stall", [(-1, 0), (60_000_000_001, 0), (0, -1)])
def test_stalls_are_checked(lib, limit, stall):
    assert lib.dg_cache_attention_inject_stall(limit, stall) == dg.DG_EINVAL
    assert dg.dg_last_error(None)
    with pytest.raises(dg.DgError):
        dg.dg_cache_attention_inject_stall(limit, stall)
    assert lib.dg_cache_attention_inject_stall(0, 0) == dg.DG_OK
