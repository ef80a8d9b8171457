"""Operators of a decode step over shared prompts, and of the sampling that ends it: inputs, plain forms and work of the
measured calls.

    shared   attention of requests that share a long prefix over the paged 8-bit cache, the prefix read once for all
    sample   tokens drawn from logits by temperature, top-k, top-p and min-p with given random numbers, or the probabilities they leave
    step     positions, slots and row lengths of a step's new tokens from the requests' lengths and block tables
    prefix   how long the prefix is that the block tables of each set of requests share

`run` computes the plain form where `own` is false and calls the package's operators where it is true.
"""
import math
import random
from fractions import Fraction

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
# 2^-f = 1 + f (C1 + f (C2 + .. f C6)) for f in [0, 1): minimax in relative error (2^-28.9), rounded to fp32. A weight is defined by this
# polynomial in separately rounded fp32 steps, a whole multiple of 2^-40, so that every implementation draws the same token.
POLY = [float.fromhex(x) for x in ("-0x1.62e42cp-1", "0x1.ebfacp-3", "-0x1.c6948ep-5", "0x1.39e3fcp-7", "-0x1.4e2aeap-10", "0x1.c946d2p-14")]
LOG2E = float(np.float32(1.44269504))


# ------------------------------------------------------------------ cases
def listed():
    return [
        # eight samples forked from one 80K prompt, a few hundred tokens in: 64 query rows to a key head, HBM counts
        dict(name="shared_fork_8", kind="shared", sets=1, set_min=8, set_max=8, pre_min=80000, pre_max=80000, own_min=100, own_max=600, pad=0.0, group=1,
             q_heads=64, kv_heads=8, dim=128, page=64, block=64, dtype="bf16", lens_seed=1),
        # a decode batch of 64 requests behind one 32K system prompt: 512 query rows to a key head, the products count
        dict(name="shared_batch_64", kind="shared", sets=1, set_min=64, set_max=64, pre_min=32768, pre_max=32768, own_min=64, own_max=4096, pad=0.0, group=1,
             q_heads=64, kv_heads=8, dim=128, page=64, block=64, dtype="bf16", lens_seed=2),
        # verify steps (a token and six drafts) of 16 requests that share a 16K prompt
        dict(name="shared_verify_16", kind="shared", sets=1, set_min=16, set_max=16, pre_min=16000, pre_max=16000, own_min=20, own_max=2000, pad=0.0, group=7,
             q_heads=64, kv_heads=8, dim=128, page=64, block=64, dtype="bf16", lens_seed=3),
        # ragged sets with few-shot prompts, padding rows among them, small blocks and pages
        dict(name="shared_sets_ragged", kind="shared", sets=6, set_min=1, set_max=24, pre_min=500, pre_max=20000, own_min=1, own_max=3000, pad=0.1, group=1,
             q_heads=16, kv_heads=4, dim=64, page=32, block=16, dtype="fp16", lens_seed=4),
        # two samples of one short prompt: the smallest step, where latency counts
        dict(name="shared_pair", kind="shared", sets=1, set_min=2, set_max=2, pre_min=339, pre_max=339, own_min=1, own_max=40, pad=0.0, group=1,
             q_heads=16, kv_heads=2, dim=128, page=64, block=64, dtype="bf16", lens_seed=5),
        # one request's next token
        dict(name="sample_1", kind="sample", rows=1, param_rows=1, vocab=131072, dtype="fp32", top_k=True, top_p=True, min_p=False, want="tokens"),
        # a decode batch with an odd vocabulary, every request with settings of its own (off, greedy, narrow, wide)
        dict(name="sample_64_mixed", kind="sample", rows=64, param_rows=1, vocab=100003, dtype="bf16", top_k=True, top_p=True, min_p=True, want="tokens"),
        # draft tokens of a large batch, and the probabilities that their verification needs
        dict(name="sample_256_drafts", kind="sample", rows=256, param_rows=1, vocab=131072, dtype="fp32", top_k=False, top_p=True, min_p=False, want="both"),
        # slots of a decode step of 64 requests
        dict(name="step_decode_64", kind="step", reqs=64, new_min=1, new_max=1, ctx=4096, page=64, spare=0, lens_seed=6),
        # chunks of a large prefill: 512 requests, about a million tokens, into a fixed number of places
        dict(name="step_prefill_1m", kind="step", reqs=512, new_min=1, new_max=8192, ctx=32768, page=64, spare=1000, lens_seed=7),
        # the samples of one 80K prompt
        dict(name="prefix_fork_8", kind="prefix", sets=1, set_min=8, set_max=8, pre_min=80000, pre_max=80000, own_max=600, pad=0.0, page=64, lens_seed=8),
        # 1024 requests in sets behind long prompts
        dict(name="prefix_sets", kind="prefix", sets=16, set_min=1, set_max=128, pre_min=2000, pre_max=131072, own_max=3000, pad=0.05, page=16, lens_seed=9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["shared", "shared", "sample", "sample", "step", "prefix"])
    seed = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 64, 128])
    if kind == "sample":
        vocab = _log_int(rng, 1000, 160000)
        group = rng.choice([1, 1, rng.randint(2, 8)])
        rows = max(1, min(_log_int(rng, 1, 256), 33000000 // vocab) // group) * group
        return dict(kind=kind, rows=rows, param_rows=group, vocab=vocab, dtype=rng.choice(["fp32", "bf16", "fp16"]), top_k=rng.random() < 0.6,
                    top_p=rng.random() < 0.6, min_p=rng.random() < 0.4, want=rng.choice(["tokens", "tokens", "probs", "both"]))
    if kind == "step":
        reqs = _log_int(rng, 1, 1024)
        top = max(1, min(_log_int(rng, 1, 8192), 1000000 // reqs))
        return dict(kind=kind, reqs=reqs, new_min=rng.choice([0, 1, top]), new_max=top, ctx=_log_int(rng, 16, 32768), page=page, spare=rng.choice([0, rng.randint(1, 500)]),
                    lens_seed=seed)
    sets = _log_int(rng, 1, 12)
    size = _log_int(rng, 1, 64)
    hi = _log_int(rng, 100, 80000)
    pad = rng.choice([0.0, 0.0, 0.2])
    if kind == "prefix":
        return dict(kind=kind, sets=sets, set_min=rng.randint(1, size), set_max=size, pre_min=max(1, int(hi * rng.uniform(0.05, 1.0))), pre_max=hi,
                    own_max=_log_int(rng, 1, 3000), pad=pad, page=page, lens_seed=seed)
    group = rng.choice([1, 1, 2, 4, 7, 8])
    kv, ratio, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 7, 8, 16]), rng.choice([64, 128])
    # no more than the largest listed step
    rows = sets * size * group * kv * ratio
    hi = max(20, min(hi, 64 * 64 * 32768 // rows))
    own_hi = max(group, min(_log_int(rng, 1, 4096), 150000 // (sets * size)))
    return dict(kind=kind, sets=sets, set_min=rng.randint(1, size), set_max=size, pre_min=max(1, int(hi * rng.uniform(0.05, 1.0))), pre_max=hi,
                own_min=group, own_max=own_hi, pad=pad, group=group, q_heads=kv * ratio, kv_heads=kv, dim=dim, page=page,
                block=rng.choice([b for b in (16, 32, 64, 128) if b <= page]), dtype=rng.choice(["bf16", "fp16"]), lens_seed=seed)


def _sets(case):
    """Per set: its prefix in whole pages' positions, and its requests' own tokens (None of a padding row)."""
    rng = random.Random(case["lens_seed"])
    out = []
    for _ in range(case["sets"]):
        size = rng.randint(case["set_min"], case["set_max"])
        pre = _log_int(rng, case["pre_min"], case["pre_max"]) // case["page"] * case["page"]
        lo = case.get("own_min", 1)
        out.append((pre, [None if rng.random() < case["pad"] else _log_int(rng, lo, case["own_max"]) for _ in range(size)]))
    return out


def _step_lens(case):
    rng = random.Random(case["lens_seed"])
    old = [rng.randint(0, case["ctx"]) for _ in range(case["reqs"])]
    lo, hi = case["new_min"], case["new_max"]
    return old, [x + (rng.randint(lo, hi) if lo < hi else hi) for x in old]


def _type(case):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["dtype"]]


def work(case):
    kind = case["kind"]
    if kind == "sample":
        n = case["rows"] * case["vocab"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": n * (size + (4 if case["want"] != "tokens" else 0)), "flops": 20 * n}
    if kind == "step":
        old, new = _step_lens(case)
        tokens = sum(new) - sum(old)
        return {"bytes": 16 * (tokens + case["spare"]) + 16 * case["reqs"] + 4 * (tokens // case["page"] + case["reqs"]), "flops": 0}
    if kind == "prefix":
        return {"bytes": sum(4 * sum(x is not None for x in mine) * (pre // case["page"] + 1) for pre, mine in _sets(case)), "flops": 0}
    d, hq, hk, g = case["dim"], case["q_heads"], case["kv_heads"], case["group"]
    keys = pairs = rows = 0
    for pre, mine in _sets(case):
        live = [x for x in mine if x is not None]
        rows += g * len(mine)
        keys += sum(live) + (pre if live else 0)
        pairs += sum(g * (pre + x) - g * (g - 1) // 2 for x in live)
    return {"bytes": int(keys * hk * (2 * d + 8 / case["block"]) + 4 * rows * hq * d), "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ inputs
def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"sample": _prepare_sample, "step": _prepare_step, "prefix": _prepare_sets, "shared": _prepare_sets}[case["kind"]](case, gen, {"case": case})


def _prepare_sample(case, gen, s):
    n, v = case["rows"], case["vocab"]
    groups = n // case["param_rows"]
    rand = lambda: torch.rand(groups, generator=gen, device="cuda")  # noqa: E731
    # some rows are sure of a few tokens, some of none
    x = (1.0 + 3.0 * torch.rand((n, 1), generator=gen, device="cuda")) * torch.randn((n, v), generator=gen, device="cuda")
    x[:, v - v // 50:] = -math.inf  # places of the vocabulary that name no token
    s["logits"] = x.to(_type(case))
    s["uniforms"] = torch.rand(n, generator=gen, device="cuda") if case["want"] != "probs" else None
    t = 0.3 + rand()
    s["temperature"] = t if groups == 1 else torch.where(rand() < 0.1, torch.zeros_like(t), t)
    off = rand()
    k = (2.0 ** (1 + 10 * rand())).to(torch.int32)
    s["top_k"] = torch.where(off < (0.0 if groups == 1 else 0.25), torch.zeros_like(k), k) if case["top_k"] else None
    off = rand()
    s["top_p"] = torch.where(off < (0.0 if groups == 1 else 0.25), torch.ones_like(t), 0.5 + 0.49 * rand()) if case["top_p"] else None
    s["min_p"] = torch.where(rand() < 0.25, torch.zeros_like(t), 0.2 * rand()) if case["min_p"] else None
    return s


def _tables(gen, need, width, pages):
    """One row of page ids per request, drawn from a shuffled pool; -1 past a request's pages."""
    perm = torch.randperm(pages, generator=gen, device="cuda")
    need = torch.tensor(need, device="cuda")
    col = torch.arange(width, device="cuda")
    at = (torch.cumsum(need, 0) - need)[:, None] + col
    return torch.where(col < need[:, None], perm[at.clamp(max=pages - 1)], -1).to(torch.int32)


def _prepare_step(case, gen, s):
    old, new = _step_lens(case)
    page = case["page"]
    need = [-(-x // page) for x in new]
    pages = sum(need) + 3
    s["table"] = _tables(gen, need, max(1, max(need)), pages)
    s["refs"] = torch.ones(pages, dtype=torch.int32, device="cuda")
    s["rows"] = torch.randperm(case["reqs"], generator=gen, device="cuda").to(torch.int32)
    at = s["rows"].long()
    s["old"], s["new"] = _ints(old)[at], _ints(new)[at]
    s["tokens"] = sum(new) - sum(old) + case["spare"]
    if own:
        from sparse_attention_indexer_gb300 import KvPages
        s["api"] = KvPages(s["table"], s["refs"], page)
    return s


def _prepare_sets(case, gen, s):
    page, sets = case["page"], _sets(case)
    reqs = sum(len(mine) for _, mine in sets)
    starts, lens, need, lead = [0], [], [], []  # lead: the request whose pages the prefix names, and how many of them
    for pre, mine in sets:
        first = None
        for x in mine:
            r = len(lens)
            lens.append(0 if x is None else pre + x)
            if x is not None and first is None:
                first = r
            need.append(0 if x is None else -(-(pre + x) // page) - (pre // page if r != first else 0))
            lead.append((r if first is None or x is None else first, pre // page if x is not None else 0))
        starts.append(len(lens))
    # every request's own pages, the prefix among those of its set's first
    width = max(1, max(-(-x // page) for x in lens)) + 1
    pages = sum(need) + 3
    table = _tables(gen, need, width, pages).long()
    col = torch.arange(width, device="cuda")
    who = torch.tensor([x for x, _ in lead], device="cuda")
    shared = torch.tensor([n for _, n in lead], device="cuda")
    mine = torch.arange(reqs, device="cuda")
    moved = torch.gather(table, 1, (col - torch.where(who == mine, 0, shared)[:, None]).clamp(min=0))
    s["table"] = torch.where(col < shared[:, None], table[who], moved).to(torch.int32).contiguous()
    s["rows"] = torch.arange(reqs, device="cuda", dtype=torch.int32)
    s["lens"] = _ints(lens)
    s["starts"] = _ints(starts)
    s["refs"] = torch.ones(pages, dtype=torch.int32, device="cuda")
    if case["kind"] == "prefix":
        # in each set one sample was rolled back into the prompt and went on from there
        for (pre, mine), a in zip(sets, starts):
            live = [a + i for i, x in enumerate(mine) if x is not None]
            if len(live) > 1 and pre:
                back = torch.randint(pre // page // 2, pre // page, (1,), generator=gen, device="cuda")
                s["table"][live[len(live) // 2], back] += 1
                s["table"][live[len(live) // 2], back] %= pages
        if own:
            from sparse_attention_indexer_gb300 import KvPages
            s["api"] = KvPages(s["table"], s["refs"], page)
        return s
    heads, dim, block, g = case["kv_heads"], case["dim"], case["block"], case["group"]
    codes = lambda: torch.randn((pages * page, heads, dim), generator=gen, device="cuda", dtype=torch.float16).mul_(100).clamp_(-448, 448).to(E4M3).view(torch.uint8)  # noqa: E731
    scales = lambda: torch.exp(0.3 * torch.randn((pages * page // block, heads), generator=gen, device="cuda")) / 100  # noqa: E731
    s["cache"] = dict(k=codes(), v=codes(), k_scale=scales(), v_scale=scales())
    s["q"] = (1.5 * torch.randn((reqs * g, case["q_heads"], dim), generator=gen, device="cuda")).to(_type(case))
    s["scale"] = 1.0 / math.sqrt(dim)
    # row i of a group of g sees all but the last g - 1 - i tokens
    back = torch.arange(g - 1, -1, -1, device="cuda", dtype=torch.int32)
    s["row_lens"] = (s["lens"][:, None] - back).clamp(min=0).view(-1)
    s["max_len"] = max(max(lens), 1)
    s["prefix"] = _ints([pre for pre, _ in sets])
    s["max_prefix"] = max(pre for pre, _ in sets)
    s["host_sets"] = [(min(pre, s["max_len"]), a, b) for (pre, _), a, b in zip(sets, starts, starts[1:])]
    if own:
        from sparse_attention_indexer_gb300 import Kv8Cache
        c = s["cache"]
        s["api"] = Kv8Cache(c["k"], c["v"], c["k_scale"], c["v_scale"], page, block)
    return s


# ------------------------------------------------------------------ the calls
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    case = s["case"]
    kind = case["kind"]
    if kind == "shared":
        return s["api"].attention_shared(s["q"], s["row_lens"], s["max_len"], s["table"], s["scale"], s["starts"], s["prefix"], s["max_prefix"], case["group"], s["rows"])
    if kind == "step":
        return tuple(s["api"].step(s["rows"], s["old"], s["new"], s["tokens"]))
    if kind == "prefix":
        return s["api"].shared(s["rows"], s["lens"], s["starts"])
    from sparse_attention_indexer_gb300 import sample_tokens, token_probs
    settings = dict(temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], param_rows=case["param_rows"])
    if case["want"] == "probs":
        return token_probs(s["logits"], **settings)
    tokens, probs = sample_tokens(s["logits"], s["uniforms"], with_probs=case["want"] == "both", **settings)
    return (tokens, probs) if case["want"] == "both" else tokens


def _run_plain(s):
    return {"shared": _plain_shared, "sample": _plain_sample, "step": _plain_step, "prefix": _plain_prefix}[s["case"]["kind"]](s)


def _keys(c, name, slots, block):
    return c[name][slots].view(E4M3).float() * c[name + "_scale"][slots // block][..., None]


def _plain_shared(s):
    """Set by set: the scores of the prefix for all its rows at once, those of the own tokens padded to the longest, one softmax over both."""
    case, c, q = s["case"], s["cache"], s["q"]
    page, block, g = case["page"], case["block"], case["group"]
    hq, hk, dim = case["q_heads"], case["kv_heads"], case["dim"]
    ratio = hq // hk
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, device="cuda")
    table = s["table"].long()
    for pre, a, b in s["host_sets"]:
        n = b - a
        t = torch.arange(s["max_len"], device="cuda")
        tail = t[pre:]
        lens = s["row_lens"][a * g:b * g].view(n, g)
        lead = (s["lens"][a:b] > 0).int().argmax()
        pslots = table[a + lead, t[:pre] // page].clamp(min=0) * page + t[:pre] % page
        oslots = table[a:b, tail // page].clamp(min=0) * page + tail % page
        x = q[a * g:b * g].float().view(n, g, hk, ratio, dim).permute(2, 0, 1, 3, 4)  # [hk, n, g, ratio, dim]
        kp, ko = _keys(c, "k", pslots, block), _keys(c, "k", oslots, block)
        sp = torch.matmul(x.reshape(hk, -1, dim), kp.permute(1, 2, 0)).view(hk, n, g, ratio, -1) * s["scale"]
        so = torch.matmul(x.reshape(hk, n, g * ratio, dim), ko.permute(2, 0, 3, 1)).view(hk, n, g, ratio, -1) * s["scale"]
        del kp, ko
        see = lens[None, :, :, None, None]
        sp = sp.masked_fill(t[:pre] >= see, -math.inf)
        so = so.masked_fill(tail >= see, -math.inf)
        top = torch.maximum(sp.amax(-1) if pre else so.amax(-1), so.amax(-1))[..., None] if len(tail) else sp.amax(-1, keepdim=True)
        safe = torch.where(top > -math.inf, top, 0.0)
        sp, so = torch.exp(sp - safe), torch.exp(so - safe)
        total = sp.sum(-1) + so.sum(-1)
        vp, vo = _keys(c, "v", pslots, block), _keys(c, "v", oslots, block)
        o = torch.matmul(sp.view(hk, -1, pre), vp.permute(1, 0, 2)).view(hk, n, g, ratio, dim)
        o = o + torch.matmul(so.view(hk, n, g * ratio, -1), vo.permute(2, 0, 1, 3)).view(hk, n, g, ratio, dim)
        o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
        out[a * g:b * g] = o.permute(1, 2, 0, 3, 4).reshape(n * g, hq, dim).to(q.dtype)
        lse[a * g:b * g] = (torch.log(total) + top[..., 0]).permute(1, 2, 0, 3).reshape(n * g, hq)
    return out, lse


def _part(frac, total, up):
    """floor (or ceil) of frac * total, exactly: frac an fp32 in [0, 1), total < 2^60."""
    m, e = torch.frexp(frac)
    m, down = (m * 2.0 ** 24).to(torch.int64), (24 - e).to(torch.int64)
    hi, lo = m * (total >> 32), m * (total & 0xFFFFFFFF)
    hi, lo = hi + (lo >> 32), lo & 0xFFFFFFFF
    near = down <= 32
    d1, d2 = down.clamp(max=32), (down - 32).clamp(0, 62)
    whole = torch.where(near, (hi << (32 - d1)) + (lo >> d1), hi >> d2)
    rest = torch.where(near, lo & ((1 << d1) - 1), (hi & ((1 << d2) - 1)) | lo)
    return whole + (rest > 0).to(torch.int64) if up else whole


def _plain_sample(s):
    case = s["case"]
    x = s["logits"].float()
    n, v = x.shape
    each = lambda t: t.repeat_interleave(case["param_rows"])[:, None]  # noqa: E731
    temp = each(s["temperature"])
    greedy = temp == 0
    top = x.amax(-1, keepdim=True)
    z = (top - x) * (torch.full_like(temp, LOG2E) / torch.where(greedy, torch.ones_like(temp), temp))
    whole = torch.floor(z).clamp(max=41.0)
    f = torch.where(whole < 41, z - whole, 0.0)
    p = torch.full_like(f, POLY[5])
    for coefficient in POLY[4::-1] + [1.0]:
        p = p * f
        p = p + coefficient
    w = ((p * 2.0 ** 24).to(torch.int64) << 16) >> whole.to(torch.int64)
    w = torch.where(whole < 41, w, 0)
    del z, f, p, whole
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    ws = torch.gather(w, 1, order)
    keep = torch.ones_like(ws, dtype=torch.bool)
    if s["top_k"] is not None:
        k = each(s["top_k"])
        keep &= (k <= 0) | (torch.arange(v, device="cuda") < k)
    if s["top_p"] is not None:
        tp = each(s["top_p"])
        run_sum = torch.cumsum(ws, -1)
        target = _part(torch.where(tp < 1, tp, 0.5), torch.where(keep, ws, 0).sum(-1, keepdim=True), True)
        keep &= (tp >= 1) | (run_sum - ws < target)
        del run_sum
    if s["min_p"] is not None:
        keep &= ws >= torch.ceil(each(s["min_p"]).double() * 2.0 ** 40).to(torch.int64)
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, 0))
    first = (x == top).int().argmax(-1, keepdim=True)
    w = torch.where(greedy, torch.zeros_like(w).scatter_(1, first, 1 << 40), w)
    del ws, keep, order
    total = w.sum(-1, keepdim=True)
    tokens = None
    if s["uniforms"] is not None:
        tokens = (torch.cumsum(w, -1) > _part(s["uniforms"][:, None], total, False)).int().argmax(-1).to(torch.int32)
    if case["want"] == "tokens":
        return tokens
    probs = w.float() / total.float()
    return probs if case["want"] == "probs" else (tokens, probs)


def _plain_step(s):
    page, n = s["case"]["page"], s["tokens"]
    count = (s["new"] - s["old"]).long()
    ends = torch.cumsum(count, 0)
    starts = torch.cat([ends.new_zeros(1), ends])
    t = torch.arange(n, device="cuda")
    r = torch.searchsorted(ends, t, right=True)
    live = t < ends[-1]
    r = r.clamp(max=len(count) - 1)
    pos = s["old"].long()[r] + t - starts[r]
    row = s["rows"].long()[r]
    page_id = s["table"][row, torch.where(live, pos // page, 0)].long()
    put = lambda x, other: torch.where(live, x, other).to(torch.int32)  # noqa: E731
    return put(pos, -1), put(row, -1), put(page_id * page + pos % page, -1), put(pos + 1, 0), starts.to(torch.int32)


def _plain_prefix(s):
    page = s["case"]["page"]
    starts = s["starts"]
    n = s["rows"].shape[0]
    of = torch.searchsorted(starts[1:], torch.arange(n, device="cuda", dtype=torch.int32), right=True)
    live = s["lens"] > 0
    sets = starts.shape[0] - 1
    at = torch.arange(n, device="cuda")
    lead = torch.full((sets,), n, device="cuda").index_reduce_(0, of, torch.where(live, at, n), "amin").clamp(max=n - 1)
    least = torch.full((sets,), 1 << 30, device="cuda").index_reduce_(0, of, torch.where(live, s["lens"].long(), 1 << 30), "amin")
    many = torch.zeros(sets, device="cuda", dtype=torch.int64).index_add_(0, of, live.long())
    mine = s["table"][s["rows"].long()]
    same = (mine == mine[lead[of]]) & (mine >= 0)
    same = torch.where(live[:, None], same, torch.ones_like(same))
    pages = torch.full((sets,), 1 << 30, device="cuda").index_reduce_(0, of, same.long().cumprod(-1).sum(-1), "amin")
    return torch.where(many > 1, torch.minimum(pages, least // page) * page, 0).to(torch.int32)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    keep = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = keep
    return {"shared": _exact_shared, "sample": _exact_sample, "step": _exact_step, "prefix": _exact_prefix}[case["kind"]](s)


def _exact_shared(s):
    """Row by row over the slots of the row's own table, the prefix no different from the rest."""
    case, c, q = s["case"], s["cache"], s["q"].double()
    page, block, g = case["page"], case["block"], case["group"]
    rows, hq, dim = q.shape
    ratio = hq // case["kv_heads"]
    lens = s["row_lens"].tolist()
    if sum(lens) * hq * dim > 2e11 or rows * case["kv_heads"] > 12000:
        return None
    out = torch.zeros((rows, hq, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device="cuda")
    off = torch.arange(page, device="cuda")
    for r in range(0, rows, g):
        n = lens[r + g - 1]
        if n == 0:
            continue
        at = (s["table"][r // g, :-(-n // page)].long()[:, None] * page + off).reshape(-1)[:n]
        t = torch.arange(n, device="cuda")
        hide = (t >= s["row_lens"][r:r + g, None])[:, None]
        for h in range(case["kv_heads"]):
            k = c["k"][at, h].view(E4M3).double() * c["k_scale"][at // block, h].double()[:, None]
            v = c["v"][at, h].view(E4M3).double() * c["v_scale"][at // block, h].double()[:, None]
            mine = slice(h * ratio, (h + 1) * ratio)
            x = (q[r:r + g, mine] @ k.T * s["scale"]).masked_fill(hide, -math.inf)
            lse[r:r + g, mine] = torch.logsumexp(x, -1)
            out[r:r + g, mine] = torch.nan_to_num(torch.softmax(x, -1)) @ v
    return out, lse


def _exact_sample(s):
    """The kept set and the token by whole numbers on the host, the probabilities by exp in 64 bits over the kept set."""
    case = s["case"]
    if case["rows"] * case["vocab"] > 40e6:
        return None
    logits = s["logits"].float().cpu().numpy()
    host = {k: None if s[k] is None else s[k].cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p", "uniforms")}
    tokens, probs = [], []
    for r, x in enumerate(logits):
        j = r // case["param_rows"]
        temp = host["temperature"][j]
        if temp == 0:
            tokens.append(int(np.argmax(x)))
            p = np.zeros(len(x))
            p[tokens[-1]] = 1.0
            probs.append(torch.from_numpy(p))
            continue
        z = (x.max() - x) * (np.float32(LOG2E) / temp)  # fp32 throughout
        n = np.minimum(np.floor(z), np.float32(63))
        f = np.where(n < 63, z, n) - n
        y = np.float32(POLY[5])
        for a in POLY[4::-1]:
            y = y * f + np.float32(a)
        y = y * f + np.float32(1)
        w = np.floor(np.ldexp(y.astype(np.float64), 40 - n.astype(np.int64))).astype(np.int64)
        by = np.argsort(-x.astype(np.float64), kind="stable")
        count = len(x)
        if host["top_k"] is not None and 0 < host["top_k"][j] < count:
            count = int(host["top_k"][j])
        if host["top_p"] is not None and host["top_p"][j] < 1:
            total = int(w[by[:count]].sum())
            need = math.ceil(Fraction(float(host["top_p"][j])) * total)
            count = min(count, int(np.searchsorted(np.cumsum(w[by]), need)) + 1)
        kept = np.zeros(len(x), bool)
        kept[by[:count]] = True
        if host["min_p"] is not None:
            kept &= w >= math.ceil(Fraction(float(host["min_p"][j])) * (1 << 40))
        w = np.where(kept, w, 0)
        if host["uniforms"] is not None:
            at = math.floor(Fraction(float(host["uniforms"][r])) * int(w.sum()))
            tokens.append(int(np.searchsorted(np.cumsum(w), at, side="right")))
        if case["want"] != "tokens":
            e = np.where(kept & (w > 0), np.exp((x.astype(np.float64) - float(x.max())) / float(temp)), 0.0)
            probs.append(torch.from_numpy(e / e.sum()))
    tokens = torch.tensor(tokens, dtype=torch.int32, device="cuda")
    if case["want"] == "tokens":
        return tokens
    probs = torch.stack(probs).cuda()
    return probs if case["want"] == "probs" else (tokens, probs)


def _exact_step(s):
    """Token by token in the order of the requests (numpy over each request's tokens)."""
    page, n = s["case"]["page"], s["tokens"]
    table, rows, old, new = (s[k].cpu().numpy() for k in ("table", "rows", "old", "new"))
    got = [np.full(n, -1, np.int32) for _ in range(3)] + [np.zeros(n, np.int32)]
    starts, t = [0], 0
    for r, a, b in zip(rows.tolist(), old.tolist(), new.tolist()):
        pos = np.arange(a, b)
        for x, y in zip(got, (pos, r, table[r, pos // page] * page + pos % page, pos + 1)):
            x[t:t + b - a] = y
        t += b - a
        starts.append(t)
    return tuple(torch.from_numpy(x).cuda() for x in got) + (_ints(starts),)


def _exact_prefix(s):
    page, starts = s["case"]["page"], s["starts"].tolist()
    table, lens, rows = s["table"].cpu().numpy(), s["lens"].tolist(), s["rows"].tolist()
    out = []
    for a, b in zip(starts, starts[1:]):
        live = [i for i in range(a, b) if lens[i] > 0]
        n = 0
        if len(live) > 1:
            first = table[rows[live[0]]]
            n = min(lens[i] for i in live) // page
            for i in live:
                wrong = np.nonzero((table[rows[i]][:n] != first[:n]) | (first[:n] < 0))[0]
                n = int(wrong[0]) if len(wrong) else n
        out.append(n * page)
    return _ints(out)
