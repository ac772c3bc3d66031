"""The paged-cache calls as a serving loop uses them: requests of different
lengths come in as prompts, share a system prompt, and go on token by token,
between the projections of a layer.  Checked against the layer run for each
request alone on the contiguous cache, and against the oracle."""
import pytest
import torch

import oracle
from megatron_tensor_transformer_plan_b200 import synth, tpl
from tests.gpu_util import TOL, assert_close_rel, to_np
from tests.paged_util import BASE, D

pytestmark = pytest.mark.gpu


class Server:
    """A layer over a pool of pages; the pages of a request grow one by one."""

    def __init__(self, dev, H, nq, nkv, F, t, page, n_pages, seed=1):
        flags = tpl.TPL_NORM | tpl.TPL_RESIDUAL
        self.dims = (H, nq, nkv, F, t)
        self.plan = tpl.Plan(tpl.make_dims(H, nq, nkv, D, F, 1, 1e-5, flags | tpl.TPL_ROPE, BASE), t)
        self.proj = tpl.Plan(tpl.make_dims(H, nq, nkv, D, F, 1, 1e-5, flags), t)  # the same weights, no rotation
        self.w = synth.layer_weights(H, nq, nkv, D, F, seed=seed, device=dev)
        self.packed = self.proj.pack_layer(self.w)
        self.page, self.dev = page, dev
        shape = (t, n_pages, nkv // t, page, D)
        # a cache that was used before: whatever it holds must not be seen
        self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=dev)
        self.v = torch.full_like(self.k, float("nan"))
        self.kv = self.plan.paged_kv(self.k, self.v)
        self.free = list(range(n_pages - 1, -1, -1))
        self.pages, self.lens = [], []

    def grow(self, b, n):
        self.lens[b] += n
        while len(self.pages[b]) * self.page < self.lens[b]:
            self.pages[b].append(self.free.pop())

    def batch(self, news=None):
        entries = max(1, max(map(len, self.pages)))
        table = torch.tensor([p + [-1] * (entries - len(p)) for p in self.pages], dtype=torch.int32, device=self.dev)
        lens = torch.tensor(self.lens, dtype=torch.int32, device=self.dev)
        if news is None:
            return self.plan.paged_batch(table, lens)
        start = [0]
        for x in news:
            start.append(start[-1] + x)
        return self.plan.paged_batch(table, lens, torch.tensor(start, dtype=torch.int32, device=self.dev), start[-1])

    def layer(self, x, batch, shared=0, window=0, sinks=0):
        """One layer over the rows of x: (y fp32, attention output)."""
        H, nq, nkv, F, t = self.dims
        B = x.shape[0]
        new = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=self.dev)
        q, k, v = new(B, nq, D), new(B, nkv, D), new(B, nkv, D)
        slot = new(t * B * (nkv // t) * D, dt=torch.bfloat16), new(t * B * (nkv // t) * D, dt=torch.bfloat16)
        ws = self.proj.workspace(B, 0, device=self.dev)
        self.proj.qkv(self.packed, tpl.Plan.kv(*slot, B, 1), x, 0, q, ws, k, v)
        self.plan.paged_append(self.kv, batch, k, v, q)
        o = new(B, nq * D, dt=torch.bfloat16)
        pws = self.plan.paged_workspace(batch.page_table.shape[0], B, device=self.dev)
        if shared:
            self.plan.paged_attn_shared(self.kv, batch, shared, q, o, pws)
        else:
            self.plan.paged_attn(self.kv, batch, q, o, pws, window=window, sinks=sinks)
        h, act = new(B, H), new(B, F, dt=torch.bfloat16)
        y, y32 = new(B, H, dt=torch.bfloat16), new(B, H)
        self.proj.o_proj(self.packed, o, x, h=h, ws=ws)
        self.proj.gate_up(self.packed, h, act, ws)
        self.proj.down_proj(self.packed, act, h, y=y, y32=y32, ws=ws)
        torch.cuda.synchronize()
        assert self.plan.last_device_error() == tpl.TPL_OK
        return y32, o


def alone(s, xs, S):
    """The layer's output for the last token of one request, xs its tokens: the
    prompt's first S tokens by prefill, the others by decode, contiguous cache."""
    H, nq, nkv, F, t = s.dims
    n = xs.shape[0]
    packed = s.plan.pack_layer(s.w)
    kc, vc = torch.zeros((2, nkv * n * D), dtype=torch.bfloat16, device=s.dev)
    kv = tpl.Plan.kv(kc, vc, 1, n)
    out = torch.empty((n, H), dtype=torch.float32, device=s.dev)
    s.plan.prefill_layer(packed, kv, xs[:S].contiguous(), None, out[:S], s.plan.prefill_workspace(S, device=s.dev))
    for p in range(S, n):
        s.plan.decode_layer(packed, kv, xs[p:p + 1].contiguous(), p, torch.empty((1, H), dtype=torch.bfloat16, device=s.dev),
                            out[p:p + 1], s.plan.workspace(1, p, device=s.dev))
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("shape", [(1024, 16, 4, 2816, 4, 32), (1024, 8, 8, 2816, 2, 16), (1280, 10, 2, 2816, 1, 64)])
def test_prompts_then_tokens(gpu, shape):
    H, nq, nkv, F, t, page = shape
    s = Server(gpu, H, nq, nkv, F, t, page, 40)
    prompts, steps = [23, 1, 37], 4
    xs = [synth.activations(p + steps, H, seed=10 + b, device=gpu) for b, p in enumerate(prompts)]
    s.pages, s.lens = [[] for _ in prompts], [0] * len(prompts)
    got = [[] for _ in prompts]
    for b, p in enumerate(prompts):
        s.grow(b, p)
    y, _ = s.layer(torch.cat([x[:p] for x, p in zip(xs, prompts)]), s.batch(prompts))
    at = 0
    for b, p in enumerate(prompts):
        got[b].append(y[at:at + p])
        at += p
    for i in range(steps):
        for b in range(len(prompts)):
            s.grow(b, 1)
        y, _ = s.layer(torch.stack([x[p + i] for x, p in zip(xs, prompts)]), s.batch())
        for b in range(len(prompts)):
            got[b].append(y[b:b + 1])
    for b, p in enumerate(prompts):
        assert_close_rel(to_np(torch.cat(got[b])), to_np(alone(s, xs[b], p)), tol=TOL, what=f"request {b}")


def test_tokens_against_the_oracle(gpu):
    """A request's tokens one at a time: the oracle's whole layer, prompt included."""
    H, nq, nkv, F, t, page, n = 1024, 16, 4, 2816, 2, 16, 21
    s = Server(gpu, H, nq, nkv, F, t, page, 8)
    x = synth.activations(n, H, seed=5, device=gpu)
    s.pages, s.lens = [[]], [0]
    y = []
    for i in range(n):
        s.grow(0, 1)
        y.append(s.layer(x[i:i + 1].contiguous(), s.batch())[0])
    od = oracle.Dims(H, nq, nkv, D, F, flags=oracle.NORM | oracle.RESIDUAL | oracle.ROPE, rope_base=BASE)
    wb = {k: synth.bits(v) for k, v in s.w.items()}
    ref, _, _ = oracle.prefill_layer(od, wb, to_np(x))
    assert_close_rel(to_np(torch.cat(y)), ref, tol=TOL, what="tokens")


def test_shared_prompt_and_window(gpu):
    """Requests behind one system prompt: the shared call gives what plain
    attention over the same pages gives, within the rounding of P; a window
    that holds every key changes no bit."""
    H, nq, nkv, F, t, page = 1024, 16, 4, 2816, 4, 16
    s = Server(gpu, H, nq, nkv, F, t, page, 60)
    system = synth.activations(48, H, seed=1, device=gpu)
    s.pages, s.lens = [[]], [0]
    s.grow(0, 48)
    s.layer(system, s.batch([48]))
    common = s.pages[0]
    s.pages, s.lens = [list(common) for _ in range(5)], [48] * 5
    own = [3, 17, 1, 9, 30]
    for b, n in enumerate(own):
        s.grow(b, n)
    s.layer(synth.activations(sum(own), H, seed=2, device=gpu), s.batch(own))
    for b in range(5):
        s.grow(b, 1)
    x = synth.activations(5, H, seed=3, device=gpu)
    y0, o0 = s.layer(x, s.batch())
    y1, o1 = s.layer(x, s.batch(), shared=48)
    y2, o2 = s.layer(x, s.batch(), window=100, sinks=2)
    assert torch.equal(o0, o2) and torch.equal(y0, y2)
    # P as one bf16 instead of two, 2^-8 of each term; both outputs rounded to bf16
    bound = 2.0 ** -8 * (2 * o0.float().abs() + 4.0)  # (4: above any value of these caches)
    assert ((o0.float() - o1.float()).abs() <= bound).all()
    assert_close_rel(to_np(y1), to_np(y0), tol=TOL, what="shared")
