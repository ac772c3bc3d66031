"""What the paged-cache calls do at the edges of what a batch may hold."""
import pytest
import torch

from megatron_tensor_transformer_plan_b200 import tpl
from tests.paged_util import Case, check, outputs, plan_of
from tests.test_gpu_paged import PROMPT_P, q_bits, workspace

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def run_shared(plan, c, shared, ws=None):
    o, lse = outputs(c)
    plan.paged_attn_shared(c.kv(plan), c.batch(plan), shared, c.q, o, workspace(plan, c) if ws is None else ws, lse=lse)
    torch.cuda.synchronize()
    assert plan.last_device_error() == tpl.TPL_OK
    return o, lse


# ---- a prefix that no sequence fills ------------------------------------------

INSIDE = [
    # nq, nkv, t, page, shared, kv_len
    (8, 8, 1, 16, 48, [33]),
    (64, 8, 8, 64, 1024, [700, 650, 0, 3]),
    (40, 8, 2, 32, 992, [961] * 40),
    (32, 32, 2, 128, 1536, [1, 0, 2]),
    (16, 1, 1, 256, 512, [0, 0]),
    (4, 4, 1, 16, 4096, [130, 129]),       # whole tiles that nobody sees
    (24, 8, 1, 64, 1536, [1500] * 50),
    (16, 8, 2, 32, 1024, [10] * 33 + [801] + [5] * 3),
    (16, 8, 2, 32, 1024, [100] * 35 + [1030, 3]),   # (filled by one, the 36th)
]


@pytest.mark.parametrize("p", INSIDE)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("stale", [NAN, INF])
def test_a_prefix_that_no_sequence_fills(gpu, p, dtype, stale):
    """Slots of the prefix behind the longest sequence hold anything, and the
    table names no page where nothing is seen."""
    nq, nkv, t, page, shared, kv_len = p
    plan = plan_of(nq, nkv, t)
    c = Case(gpu, nq, nkv, t, page, kv_len, shared=shared, dtype=dtype, seed=page)
    top = max(kv_len)
    for key in range(min(top, shared), shared):
        for pool in (c.k, c.v):
            pool[:, c.pages[0][key // page], :, key % page] = stale
    c.table[:, (top + page - 1) // page:] = -3
    o, lse = run_shared(plan, c, shared)
    check(c, o, lse, 0, 0, q_bits(c, False), PROMPT_P)
