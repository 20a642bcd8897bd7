"""Rows whose first key tile holds none of their keys, and whose scores lie far below
zero: the running maximum has to come from the row's own scores."""
import pytest
import torch

import oracle
from gpu_util import BF16_MAX_ABS, LSE_ABS, compare
from sliding_window_attention_fwd_b200 import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import sliding_window_attention_fwd_b200 as m
    return m


@pytest.mark.parametrize("H,Hkv", [(2, 1), (1, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_windows_that_start_in_a_later_tile(swa, H, Hkv, D):
    N, L = 500, 100
    noise = inputs.normal((1, N, Hkv, D), 5, 0).float() * 0.25
    q = torch.full((1, N, H, D), 6.0 if D == 64 else 4.0).to(torch.bfloat16)
    k = (noise - (6.0 if D == 64 else 4.0)).to(torch.bfloat16)  # scores around -200
    v = inputs.normal((1, N, Hkv, D), 5, 1)
    lse = torch.empty(1, H, N, device="cuda")
    out = swa.swa_forward(q.cuda(), k.cuda(), v.cuda(), lse=lse, win_left=L, win_right=0)
    torch.cuda.synchronize()
    ro, rl = oracle.forward(q, k, v, L, 0)
    compare(out.float().cpu().numpy(), ro, BF16_MAX_ABS, what="out")
    compare(lse.cpu().numpy(), rl, LSE_ABS, what="lse")
