"""Refusals of the paged-cache calls: every one is made on the host, before
anything is launched, so they are tested without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def tpl():
    from megatron_tensor_transformer_plan_b200 import build
    build.build()
    from megatron_tensor_transformer_plan_b200 import tpl as m
    return m


A = 0x10000  # addresses that nothing reads


class Call:
    def __init__(self, tpl, nq=16, nkv=8, t=2, f32=False):
        flags = tpl.TPL_NORM | tpl.TPL_ROPE | (tpl.TPL_FP32_WEIGHTS if f32 else 0)
        self.m = tpl
        self.plan = tpl.Plan(tpl.make_dims(nq * 128, nq, nkv, 128, 256 * nq, 1, 1e-5, flags, 10000.0), t)
        self.kv = tpl.tpl_paged_kv(A, A, 10, 64)
        self.batch = tpl.tpl_paged_batch(A, 8, 8, 3, A, None, 3)
        self.q = tpl.tpl_heads(A, tpl.TPL_F32, nq * 128, 128)
        self.q_out = tpl.tpl_heads(2 * A, tpl.TPL_F32, nq * 128, 128)
        self.k = tpl.tpl_heads(A, tpl.TPL_F32, nkv * 128, 128)
        self.v = tpl.tpl_heads(A, tpl.TPL_F32, nkv * 128, 128)
        self.o, self.lse, self.ws, self.ws_bytes, self.window, self.sinks, self.shared = A, None, A, 1 << 40, 0, 0, 64

    def ref(self, x):
        return None if x is None else ctypes.byref(x)

    def append(self):
        return self.m.tpl_paged_append(self.plan.handle, self.ref(self.kv), self.ref(self.batch), self.ref(self.q),
                                       self.ref(self.q_out), self.ref(self.k), self.ref(self.v), None)

    def attn(self):
        return self.m.tpl_paged_attn(self.plan.handle, self.ref(self.kv), self.ref(self.batch), self.ref(self.q),
                                     self.window, self.sinks, self.o, self.lse, self.ws, self.ws_bytes, None)

    def attn_shared(self):
        return self.m.tpl_paged_attn_shared(self.plan.handle, self.ref(self.kv), self.ref(self.batch), self.shared,
                                            self.ref(self.q), self.o, self.lse, self.ws, self.ws_bytes, None)


def every(c, want, calls=("append", "attn", "attn_shared")):
    for name in calls:
        assert getattr(c, name)() == want, name


@pytest.mark.parametrize("change", [
    ("kv", None), ("batch", None), ("kv.k", None), ("kv.v", A + 8), ("kv.n_pages", 0), ("kv.page_size", 0),
    ("batch.page_table", None), ("batch.kv_len", None), ("batch.kv_len", A + 2), ("batch.max_pages", 0),
    ("batch.table_stride", 7), ("batch.n_seqs", -1), ("batch.n_tokens", -3), ("batch.n_tokens", 4),
    ("q.data", None), ("q.data", A + 4), ("q.type", 2), ("q.token_stride", -128), ("q.head_stride", 130)])
def test_invalid(tpl, change):
    c = Call(tpl)
    path, value = change
    *outer, name = path.split(".")
    setattr(getattr(c, outer[0]) if outer else c, name, value)
    every(c, tpl.TPL_EINVAL)


@pytest.mark.parametrize("change", [("kv.page_size", 8), ("kv.page_size", 48), ("kv.page_size", 512),
                                    ("kv.n_pages", 1 << 23), ("batch.max_pages", 1 << 25), ("batch.n_seqs", 1025)])
def test_unsupported(tpl, change):
    c = Call(tpl)
    path, value = change
    outer, name = path.split(".")
    setattr(getattr(c, outer), name, value)
    if name == "max_pages":
        c.batch.table_stride = value
    if name == "n_seqs":
        c.batch.n_tokens = value
    every(c, tpl.TPL_EUNSUPPORTED)


def test_append_arguments(tpl):
    for name in ("k", "v", "q", "q_out"):
        c = Call(tpl)
        setattr(c, name, None)
        every(c, tpl.TPL_EINVAL, ["append"])
    c = Call(tpl)
    c.k = c.q = c.q_out = None
    every(c, tpl.TPL_EINVAL, ["append"])
    for name in ("k", "v", "q", "q_out"):
        c = Call(tpl)
        getattr(c, name).type = tpl.TPL_BF16
        every(c, tpl.TPL_EINVAL, ["append"])
    for ts, hs in ((0, 128), (128, 128), (2048, 64), (1920, 128), (128, 256)):  # rows of q_out that overlap
        c = Call(tpl)
        c.q_out.token_stride, c.q_out.head_stride = ts, hs
        every(c, tpl.TPL_EINVAL, ["append"])
    c = Call(tpl)
    c.q_out.data = c.q.data  # in place, but other rows
    c.q_out.token_stride = 2 * c.q.token_stride
    every(c, tpl.TPL_EINVAL, ["append"])


def test_attention_arguments(tpl):
    for name, value in (("o", None), ("o", A + 8), ("ws", None), ("ws", A + 4), ("lse", A + 2)):
        c = Call(tpl)
        setattr(c, name, value)
        every(c, tpl.TPL_EINVAL, ["attn", "attn_shared"])
    c = Call(tpl)
    c.ws_bytes = c.plan.paged_workspace_size(3, 3) - 1
    every(c, tpl.TPL_EWORKSPACE, ["attn", "attn_shared"])
    for name in ("window", "sinks"):
        c = Call(tpl)
        setattr(c, name, -1)
        every(c, tpl.TPL_EINVAL, ["attn"])
    for shared in (-64, 32, 65, 9 * 64):
        c = Call(tpl)
        c.shared = shared
        every(c, tpl.TPL_EINVAL, ["attn_shared"])
    c = Call(tpl)
    c.batch.q_start = A  # prompts
    every(c, tpl.TPL_EUNSUPPORTED, ["attn_shared"])
    c = Call(tpl, f32=True)
    every(c, tpl.TPL_EUNSUPPORTED, ["attn_shared"])
    c.batch.q_start = A
    every(c, tpl.TPL_EUNSUPPORTED, ["attn"])


def test_nothing_to_do(tpl):
    c = Call(tpl)
    c.batch = tpl.tpl_paged_batch(None, 0, 0, 0, None, None, 0)
    every(c, tpl.TPL_OK)
    c.batch = tpl.tpl_paged_batch(A, 8, 8, 3, A, A, 0)
    every(c, tpl.TPL_OK, ["append", "attn"])


def test_workspace_size(tpl):
    p = Call(tpl).plan
    out = ctypes.c_size_t()
    for n, tokens, rc in ((0, 1, tpl.TPL_EINVAL), (1, 0, tpl.TPL_EINVAL), (1025, 1025, tpl.TPL_EUNSUPPORTED),
                          (1, (1 << 22) + 1, tpl.TPL_EUNSUPPORTED)):
        assert tpl.tpl_paged_workspace_size(p.handle, n, tokens, ctypes.byref(out)) == rc
    sizes = [p.paged_workspace_size(n, tokens) for n, tokens in ((1, 1), (1, 1000), (7, 1000), (1024, 1 << 22))]
    assert sizes == sorted(sizes)
    for n in (1, 8, 9, 64, 65, 1024):  # enough for every smaller batch
        assert all(p.paged_workspace_size(m, m) <= p.paged_workspace_size(n, n) for m in range(1, n))


def test_binding_refuses(tpl):
    import torch
    p = Call(tpl).plan
    pool = torch.zeros((2, 5, 4, 64, 128), dtype=torch.bfloat16)
    for k in (pool.float(), pool[0], pool.transpose(0, 1), torch.zeros((1, 5, 8, 64, 128), dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            p.paged_kv(k, k)
    with pytest.raises(ValueError):
        p.paged_kv(pool, pool[:, :4].contiguous())
    with pytest.raises(ValueError, match="CUDA"):
        p.paged_kv(pool, pool)
    table, lens = torch.zeros((3, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for args in ((table.long(), lens), (table, lens[:2]), (table[0], lens), (table, lens, lens, 3), (table.t(), lens),
                 (table, lens, torch.zeros(4, dtype=torch.int32)), (table, lens, None, 4)):
        with pytest.raises(ValueError):
            p.paged_batch(*args)
