"""What the paged-cache calls do at the edges of what a batch may hold."""
import pytest
import torch

from megatron_tensor_transformer_plan_b200 import tpl
from tests.paged_util import D, Case, check, outputs, plan_of
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


# ---- starts that are out of range ------------------------------------------------

STARTS = [
    # q_start with n_tokens = 60, the rows that some sequence validly has
    ([0, 50, 20, 60], [(0, 0, 20), (2, 20, 60)]),       # (rows 20 .. 49 lie in two sequences: either may lack them)
    ([70, 75], []),
    ([-5, -2], []),
    ([0, 10, 61, 62, 70], [(0, 0, 10)]),
    ([60, 65], []),
    ([-1, 10, 30], [(1, 10, 30)]),
    ([0, 10, 10, 5], [(0, 0, 10)]),
]


@pytest.mark.parametrize("p", STARTS)
def test_append_reports_starts_out_of_range(gpu, p):
    starts, valid = p
    plan = plan_of(16, 8, 2, rope=False)
    n, tokens, page = len(starts) - 1, 60, 16
    c = Case(gpu, 16, 8, 2, page, [100] * n, [0] * n, seed=2)
    q_start = torch.tensor(starts, dtype=torch.int32, device=gpu)
    batch = plan.paged_batch(c.table, c.lens, q_start, tokens)
    k, v = (torch.randn((tokens, 8, D), device=gpu) for _ in "kv")
    want = c.k.clone(), c.v.clone()
    loose = torch.zeros((c.n_pages, page), dtype=torch.bool, device=gpu)  # slots that may or may not be written
    for b, first, end in valid:
        for r in range(first, end):
            pos = 100 - starts[b + 1] + r
            for pool, x in zip(want, (k, v)):
                pool[:, c.pages[b][pos // page], :, pos % page] = x[r].to(torch.bfloat16).unflatten(0, (2, 4))
    for b in range(n):
        if 0 <= starts[b] <= starts[b + 1] <= tokens:
            for r in range(starts[b], starts[b + 1]):
                if sum(starts[x] <= r < starts[x + 1] <= tokens and starts[x] >= 0 for x in range(n)) > 1:
                    pos = 100 - starts[b + 1] + r
                    loose[c.pages[b][pos // page], pos % page] = True
    plan.paged_append(c.kv(plan), batch, k, v)
    assert plan.last_device_error() == tpl.TPL_EDEVICE
    for pool, w in zip((c.k, c.v), want):
        same = (pool == w).permute(1, 3, 0, 2, 4).flatten(2).all(-1)
        assert (same | loose).all()
    assert plan.last_device_error() == tpl.TPL_OK
