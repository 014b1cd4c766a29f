"""Attention-layer operators at the edges of their contract: against the fp64 oracle with the
tolerances of test_attention_layer_gpu.py, and against themselves."""
import pytest
import torch

import uniform_state_text_b200 as dg
from test_attention_layer_gpu import MASKS, Setup, _check_attention, _tokens_q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from uniform_state_text_b200 import build
    build.build()
    dg.lib()


# ----------------------------------------------------------------------------- the plan and the first copies
@pytest.mark.parametrize("batch,D,G", [(1, 128, 2), (1024, 64, 1), (1024, 128, 2), (1024, 256, 1), (33, 128, 150)])
def test_first_tiles_over_the_plan(batch, D, G):
    """The split's sums (one per sequence) lie where the first key tiles are copied to: the largest
    batch and the smallest, pages by TMA, a hundred times the same to the bit."""
    s = Setup([(120 + b % 9, 1) for b in range(batch)], dg.DG_KV_BF16, 1, D, 128, seed=D)
    q = _tokens_q(s, G, 3)
    want, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    s.cache.check()
    _check_attention(s, q, "causal", D ** -0.5, want, lse)
    off = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        out, l = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
        off += (out.view(torch.int16) != want.view(torch.int16)).sum()
        off += (l.view(torch.int32) != lse.view(torch.int32)).sum()
    assert int(off) == 0
    s.cache.check()
