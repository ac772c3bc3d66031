"""The paged-cache operators: appending with the rotary embedding, attention
over the pages (causal, with a sliding window and sinks) and attention for a
batch that shares a prefix -- their measured cases and their plain forms.

A case is a batch of sequences over one paged cache of bf16 keys and values,
[t][n_pages][n_kv/t][page][128]; `page_table` names the pages of each
sequence, `kv_len` how many keys it has (this call's tokens included), and
`q_start` where its tokens lie among the rows of q (None: one token each).
A token at position p sees the keys j <= p with j > p - window (window 0: no
limit) or j < sinks.  Outputs of attention are o, rounded to bf16, and the
natural logarithm of the softmax denominator, fp32.
"""
import math
import random

import torch

own = False

HD = 128            # head dimension
ROPE_BASE = 500000.0
HEADS = [(32, 32), (64, 8), (32, 8), (40, 8), (16, 8), (24, 8), (16, 2), (8, 1), (48, 4)]  # (query heads, kv heads)


def _case(name, op, **kw):
    case = {"name": name, "op": op, "seqs": 1, "new": 0, "past": 0, "ragged": False, "nq": 64, "nkv": 8, "t": 1,
            "page": 64, "window": 0, "sinks": 0, "prefix": 0, "type": "f32", "mix": 1}
    case.update(kw)
    return case


def listed():
    return [
        # appending: one chat's next token on the 7B-shaped layer (32 heads, no groups)
        _case("append_one", "append", past=517, nq=32, nkv=32, page=16),
        # a full decode batch of the 70B-shaped layer, far positions
        _case("append_batch", "append", seqs=64, past=131072, ragged=True, t=4),
        # the prompts of seven requests, q/k/v as slices of one fused bf16 projection
        _case("append_prompt", "append", seqs=7, new=2341, past=6000, ragged=True, t=8, type="bf16"),
        # attention: one chat's next token, short history
        _case("attn_one", "attn", past=517, nq=32, nkv=32, page=16),
        # the 70B-shaped decode batch of 16 at 8192 cached keys
        _case("attn_batch", "attn", seqs=16, past=8192, t=4),
        # long conversations kept to a window of 4096 and four first tokens
        _case("attn_window", "attn", seqs=32, past=32768, ragged=True, window=4096, sinks=4, page=16, t=8),
        # a few short follow-up prompts in one batch, groups of five heads
        _case("prompt_short", "attn", seqs=3, new=37, past=900, ragged=True, nq=40, page=32, type="bf16"),
        # one chunk of 4096 tokens of a long prompt after 4096 cached ones
        _case("prompt_chunk", "attn", new=4096, past=4096, t=8, type="bf16"),
        # prompts of five requests with a window and sinks, fp32 queries
        _case("prompt_window", "attn", seqs=5, new=1777, past=6000, ragged=True, window=1024, sinks=16, page=128),
        # shared prefix: a handful of requests behind one system prompt
        _case("shared_few", "shared", seqs=5, prefix=1536, past=200, ragged=True, nq=32, page=16, type="bf16"),
        # a decode batch behind a prompt of 8192 tokens
        _case("shared_batch", "shared", seqs=64, prefix=8192, past=512, ragged=True, t=4),
        # many samples of one long document
        _case("shared_many", "shared", seqs=192, prefix=16384, past=1024, ragged=True, t=8, type="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    nq, nkv = rng.choice(HEADS)
    kw = {"nq": nq, "nkv": nkv, "t": rng.choice([t for t in (1, 2, 4, 8) if nkv % t == 0]),
          "page": rng.choice([16, 32, 64, 128, 256]), "ragged": rng.random() < 0.8,
          "type": rng.choice(["f32", "bf16"]), "mix": rng.randrange(1 << 30)}
    kind = rng.choice(["append", "append_prompt", "attn", "attn", "prompt", "prompt", "shared", "shared"])
    if kind == "append":
        kw.update(op="append", seqs=_log(rng, 1, 64), past=_log(rng, 1, 131072))
    elif kind == "append_prompt":
        kw.update(op="append", seqs=_log(rng, 1, 16), past=_log(rng, 1, 131072))
        kw["new"] = _log(rng, 1, 16000 // kw["seqs"])
    elif kind == "attn":
        kw.update(op="attn", seqs=_log(rng, 1, 64))
        kw["past"] = _log(rng, 1, min(65536, 1 << 20) // max(1, kw["seqs"] * nkv // 16))
        if rng.random() < 0.5:
            kw.update(window=_log(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 33, 128]))
    elif kind == "prompt":
        kw.update(op="attn", seqs=_log(rng, 1, 8))
        kw["new"] = _log(rng, 1, 2048 // kw["seqs"])
        kw["past"] = _log(rng, 1, 8192 // kw["seqs"])
        if rng.random() < 0.5:
            kw.update(window=_log(rng, 16, 4096), sinks=rng.choice([0, 1, 4, 33, 128]))
    else:
        kw.update(op="shared", seqs=_log(rng, 1, 128), past=_log(rng, 1, 1024))
        kw["prefix"] = kw["page"] * max(1, _log(rng, 256, 16384) // kw["page"])
    case = _case("", **kw) if "op" in kw else None
    del case["name"]
    return case


# ---- sizes -------------------------------------------------------------------

def _lens(case):
    """Per sequence: (keys before this call beyond the prefix, new tokens)."""
    rnd = random.Random(case["mix"])
    n, past, new = case["seqs"], case["past"], max(1, case["new"])
    if not case["ragged"]:
        return [(past, new)] * n
    out = [(rnd.randint((past + 3) // 4, past), rnd.randint(1, new) if case["new"] else 1) for _ in range(n)]
    out[0] = (past, new)
    if n >= 3:
        out[n // 2] = (0, out[n // 2][1])  # a request that has just begun
    return out


def _visible(case, past, new):
    """(keys any of the new tokens sees, (token, key) pairs) of one sequence."""
    total, w, s = past + new, case["window"], case["sinks"]
    if not w:
        return total, new * past + new * (new + 1) // 2
    first = max(0, past - w + 1)
    keys = total - first + min(s, first)
    pairs = 0
    for p in range(past, total):
        lo = max(0, p - w + 1)
        pairs += p + 1 - lo + min(s, lo)
    return keys, pairs


def work(case):
    lens = _lens(case)
    nq, nkv = case["nq"], case["nkv"]
    tokens = sum(new for _, new in lens)
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "append":
        values = tokens * (nq + 2 * nkv) * HD
        written = tokens * (nq * HD * size + 2 * nkv * HD * 2)
        return {"bytes": values * size + written, "flops": 3 * tokens * (nq + nkv) * HD}
    kv = pairs = 0
    for past, new in lens:
        a, b = _visible(case, past, new)
        kv, pairs = kv + a, pairs + b + new * case["prefix"]
    kv += case["prefix"]
    io = tokens * nq * (HD * (size + 2) + 4)
    return {"bytes": kv * nkv * HD * 4 + io, "flops": 4 * pairs * nq * HD}


# ---- inputs ------------------------------------------------------------------

def _inputs(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lens = _lens(case)
    n, page, nq, nkv, t = case["seqs"], case["page"], case["nq"], case["nkv"], case["t"]
    prefix, append = case["prefix"], case["op"] == "append"
    kv_len = [prefix + past + new for past, new in lens]
    news = [new for _, new in lens]
    entries = (max(kv_len) + page - 1) // page
    # pages: an append touches only the pages its tokens land in; the others
    # of its history are named as page 0
    first = [(kv_len[b] - news[b]) // page if append else 0 for b in range(n)]
    need = [(kv_len[b] + page - 1) // page - first[b] for b in range(n)]
    shared = prefix // page
    count = shared + sum(x - shared for x in need) if prefix else sum(need)
    n_pages = count + 1
    order = (torch.randperm(count, generator=g, device=dev) + 1).to(torch.int32)
    table = torch.zeros((n, entries), dtype=torch.int32, device=dev)
    at = shared
    for b in range(n):
        if shared:
            table[b, :shared] = order[:shared]
        k = need[b] - shared
        table[b, first[b] + shared:first[b] + need[b]] = order[at:at + k]
        at += k
    tokens = sum(news)
    dt = torch.float32 if case["type"] == "f32" else torch.bfloat16

    def normal(shape, dtype, scale=1.0):
        x = torch.empty(shape, dtype=dtype, device=dev)
        return x.normal_(0.0, scale, generator=g)

    pool = (t, n_pages, nkv // t, page, HD)
    st = {"case": case, "table": table, "kv_len": torch.tensor(kv_len, dtype=torch.int32, device=dev),
          "q_start": None, "tokens": tokens, "q_max": max(news), "l_max": max(kv_len),
          "k_pool": normal(pool, torch.bfloat16), "v_pool": normal(pool, torch.bfloat16)}
    if case["new"]:
        starts = [0]
        for x in news:
            starts.append(starts[-1] + x)
        st["q_start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    if append:
        # what a fused projection leaves: q, k and v side by side in each row
        qkv = normal((tokens, nq + 2 * nkv, HD), dt)
        st["q"], st["k"], st["v"] = qkv[:, :nq], qkv[:, nq:nq + nkv], qkv[:, nq + nkv:]
    else:
        # logits of standard deviation 2: some keys matter far more than others
        st["q"] = normal((tokens, nq, HD), dt, 2.0)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    nq, tokens = case["nq"], st["tokens"]
    if case["op"] == "append":
        st["q_out"] = torch.empty((tokens, nq, HD), dtype=st["q"].dtype, device="cuda")
        freq = torch.arange(64, dtype=torch.float64, device="cuda")
        st["theta"] = ROPE_BASE ** (-2.0 * freq / HD)
    else:
        st["o"] = torch.empty((tokens, nq * HD), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty((tokens, nq), dtype=torch.float32, device="cuda")
    if own:
        from megatron_tensor_transformer_plan_b200 import tpl
        dims = tpl.make_dims(nq * HD, nq, case["nkv"], HD, 4 * nq * HD, 1, 1e-5,
                             tpl.TPL_NORM | tpl.TPL_RESIDUAL | tpl.TPL_ROPE, ROPE_BASE)
        st["plan"] = tpl.Plan(dims, case["t"])
        st["kv"] = st["plan"].paged_kv(st["k_pool"], st["v_pool"])
        st["batch"] = st["plan"].paged_batch(st["table"], st["kv_len"], st["q_start"], tokens)
        st["ws"] = st["plan"].paged_workspace(case["seqs"], tokens)
    return st


# ---- one pass ----------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if op == "append":
        if own:
            st["plan"].paged_append(st["kv"], st["batch"], st["k"], st["v"], st["q"], st["q_out"])
        else:
            _append(st)
        return {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    if own:
        if op == "attn":
            st["plan"].paged_attn(st["kv"], st["batch"], st["q"], st["o"], st["ws"], window=st["case"]["window"],
                                  sinks=st["case"]["sinks"], lse=st["lse"])
        else:
            st["plan"].paged_attn_shared(st["kv"], st["batch"], st["case"]["prefix"], st["q"], st["o"], st["ws"],
                                         lse=st["lse"])
        return {"o": st["o"], "lse": st["lse"]}
    return _attention(st) if op == "attn" else _shared(st)


def _rows(st):
    """Of every token: its sequence, its place among the sequence's tokens and its position."""
    at = torch.arange(st["tokens"], device="cuda")
    if st["q_start"] is None:
        return at, torch.zeros_like(at), st["kv_len"].long() - 1
    start = st["q_start"].long()
    seq = torch.searchsorted(start[1:], at, right=True)
    inner = at - start[seq]
    pos = st["kv_len"].long()[seq] - (start[seq + 1] - start[seq]) + inner
    return seq, inner, pos


def _append(st):
    page, t = st["case"]["page"], st["case"]["t"]
    seq, _, pos = _rows(st)
    angle = pos.double()[:, None] * st["theta"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x):
        a, b = x.float().split(64, dim=-1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)

    st["q_out"].copy_(turned(st["q"]))
    pages, slots = st["table"].long()[seq, pos // page], pos % page
    for pool, new in ((st["k_pool"], turned(st["k"])), (st["v_pool"], st["v"])):
        rows = new.to(torch.bfloat16).unflatten(1, (t, -1))                 # [tokens][t][n_kv/t][128]
        pool.permute(1, 3, 0, 2, 4)[pages, slots] = rows


def _gather(pool, pages):
    """Pages [n][e] of the pool as fp32 [n][e * page][n_kv][128]."""
    x = pool[:, pages.long()]                                               # [t][n][e][n_kv/t][page][128]
    return x.permute(1, 2, 4, 0, 3, 5).flatten(3, 4).flatten(1, 2).float()


def _softmax(s, seen):
    """exp(s - max), its sum and the log of the denominator over the last axis, where `seen`; rows that see nothing give 0, 0, -inf."""
    s = s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return p, total, (top + total.log()).squeeze(-1)


def _attention(st):
    case = st["case"]
    nq, nkv = case["nq"], case["nkv"]
    seq, inner, pos = _rows(st)
    keys, values = _gather(st["k_pool"], st["table"]), _gather(st["v_pool"], st["table"])
    n, length = keys.shape[:2]
    q = torch.zeros((n, st["q_max"], nq, HD), device="cuda")
    where = torch.full((n, st["q_max"]), -1, dtype=torch.long, device="cuda")
    q[seq, inner], where[seq, inner] = st["q"].float(), pos
    at = torch.arange(length, device="cuda")
    seen = at <= where[..., None]
    if case["window"]:
        seen &= (at > where[..., None] - case["window"]) | (at < case["sinks"])
    grouped = q.unflatten(2, (nkv, -1)).permute(0, 2, 3, 1, 4)              # [n][n_kv][g][q_max][128]
    rows = grouped.flatten(2, 3)
    s = (rows @ keys.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(HD))
    p, total, lse = _softmax(s.unflatten(2, (-1, st["q_max"])), seen[:, None, None])
    o = (p.flatten(2, 3) @ values.permute(0, 2, 1, 3)).unflatten(2, (-1, st["q_max"])) / total
    o = torch.where(total > 0, o, torch.zeros_like(o))
    o, lse = o.permute(0, 3, 1, 2, 4).flatten(2, 4), lse.permute(0, 3, 1, 2).flatten(2, 3)
    return {"o": o[seq, inner].to(torch.bfloat16), "lse": lse[seq, inner]}


def _shared(st):
    case = st["case"]
    nkv, first = case["nkv"], case["prefix"] // case["page"]
    table = st["table"]
    pk, pv = _gather(st["k_pool"], table[:1, :first])[0], _gather(st["v_pool"], table[:1, :first])[0]
    ok, ov = _gather(st["k_pool"], table[:, first:]), _gather(st["v_pool"], table[:, first:])
    q = st["q"].float().unflatten(1, (nkv, -1)).mul(1.0 / math.sqrt(HD))    # [n][n_kv][g][128]
    heads = q.permute(1, 0, 2, 3).flatten(1, 2)                             # [n_kv][n * g][128]
    sp = (heads @ pk.permute(1, 2, 0)).unflatten(1, (case["seqs"], -1)).transpose(0, 1)
    so = q @ ok.permute(0, 2, 3, 1)
    length = so.shape[-1]
    seen = torch.arange(length, device="cuda") + case["prefix"] < st["kv_len"][:, None].long()
    seen = torch.cat([torch.ones_like(seen[:, :1]).expand(-1, case["prefix"]), seen], dim=1)
    p, total, lse = _softmax(torch.cat([sp, so], dim=-1), seen[:, None, None])
    pp = p[..., :case["prefix"]].transpose(0, 1).flatten(1, 2)
    o = (pp @ pv.permute(1, 0, 2)).unflatten(1, (case["seqs"], -1)).transpose(0, 1)
    o = (o + p[..., case["prefix"]:] @ ov.permute(0, 2, 1, 3)) / total
    return {"o": o.flatten(1, 3).to(torch.bfloat16), "lse": lse.flatten(1, 2)}


# ---- the definition in 64 bits --------------------------------------------------

def exact(case, seed):
    st = _inputs(case, seed)
    lens, page, t = _lens(case), case["page"], case["t"]
    nq, nkv = case["nq"], case["nkv"]
    group = nq // nkv
    starts, at = [], 0
    for _, new in lens:
        starts.append(at)
        at += new
    if case["op"] == "append":
        q_out = torch.empty((at, nq, HD), dtype=torch.float64, device="cuda")
        k_pool, v_pool = st["k_pool"].double(), st["v_pool"].double()
        rate = torch.exp(-math.log(ROPE_BASE) * torch.arange(64, dtype=torch.float64, device="cuda") / 64)
        for b, (past, new) in enumerate(lens):
            pos = torch.arange(past, past + new, device="cuda")
            turn = torch.polar(torch.ones((new, 64), dtype=torch.float64, device="cuda"), pos[:, None] * rate)[:, None]
            rows = slice(starts[b], starts[b] + new)

            def rotated(x):
                z = torch.complex(x[..., :64].double(), x[..., 64:].double()) * turn
                return torch.cat([z.real, z.imag], dim=-1)

            q_out[rows] = rotated(st["q"][rows])
            pages = st["table"][b].long()[pos // page]
            for h in range(nkv):
                shard, local = h // (nkv // t), h % (nkv // t)
                k_pool[shard, pages, local, pos % page] = rotated(st["k"][rows])[:, h]
                v_pool[shard, pages, local, pos % page] = st["v"][rows][:, h].double()
        return {"q": q_out, "k_pool": k_pool, "v_pool": v_pool}
    o = torch.zeros((at, nq, HD), dtype=torch.float64, device="cuda")
    lse = torch.full((at, nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, (past, new) in enumerate(lens):
        total = case["prefix"] + past + new
        key = torch.arange(total, device="cuda")
        pages = st["table"][b].long()[key // page]
        pos = torch.arange(total - new, total, device="cuda")[:, None]
        hidden = key[None] > pos
        if case["window"]:
            hidden = hidden | ((key[None] <= pos - case["window"]) & (key[None] >= case["sinks"]))
        rows = slice(starts[b], starts[b] + new)
        for h in range(nkv):
            shard, local = h // (nkv // t), h % (nkv // t)
            k = st["k_pool"][shard, pages, local, key % page].double()
            v = st["v_pool"][shard, pages, local, key % page].double()
            heads = range(h * group, (h + 1) * group)
            for part in ([[x] for x in heads] if new > 1 else [list(heads)]):
                q = st["q"][rows][:, part].double().transpose(0, 1)
                s = torch.einsum("htd,kd->htk", q, k) / math.sqrt(HD)
                s[hidden.expand_as(s)] = -math.inf
                z = torch.logsumexp(s, dim=-1)
                o[rows, part] = torch.einsum("htk,kd->thd", torch.exp(s - z[..., None]), v)
                lse[rows, part] = z.T
    return {"o": o.flatten(1, 2), "lse": lse}
