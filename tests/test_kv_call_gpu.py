"""moe_kv_call's doubles: what a float cannot hold does not turn into a default."""
import pytest
import torch

import fp4_block_scaled_gb300 as moe
from kv_setup import handle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


def test_a_factor_that_rounds_to_zero_is_refused():
    """scale 0 is 1 / sqrt(D) and softcap 0 none: neither is meant by 1e-60."""
    q = torch.ones((1, 1, 16), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros((1, 1, 16), dtype=torch.float32, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = torch.zeros((1, 1, 16, 16), dtype=torch.bfloat16, device="cuda")
    with handle(1, 1, 16) as h:
        for kw in (dict(scale=1e-60), dict(scale=-1e-60), dict(softcap=1e-60), dict(softcap=-1e-60), dict(scale=float("nan"))):
            with pytest.raises(moe.MoeError) as e:
                moe.moe_attn_decode(h, moe.kv_pool(p, p), q, n, n.view(1, 1), 1, o, **kw)
            assert e.value.code == moe.MOE_ERR_INVALID_ARG, kw
        for kw in (dict(scale=0.0), dict(scale=-0.0), dict(scale=1e-40), dict(softcap=0.0)):
            moe.moe_attn_decode(h, moe.kv_pool(p, p), q, n, n.view(1, 1), 1, o, **kw)
        assert moe.moe_kv_status(h) == moe.MOE_OK
