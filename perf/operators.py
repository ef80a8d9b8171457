"""Serving operators around the paged 8-bit KV cache: inputs, plain forms and work of the measured calls.

    store      new K/V tokens quantised to e4m3 into a paged cache, one power-of-two scale per (token block, head)
    attention  decode and verify steps over that cache, through block tables
    selected   the same over the slots of a top-k selection
    pages      copying, forking with copy-on-write, and compacting the pages of a cache
    verify     drafted tokens accepted or replaced by given random numbers

`run` computes the plain form where `own` is false and calls the package's operators where it is true.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
UNIT = 2.0 ** 60  # probabilities are summed as whole multiples of 2^-60


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 requests: a token each, most of them into a block that has tokens already
        dict(name="store_decode_64", kind="store", reqs=64, new=1, ctx=4096, kv_heads=8, dim=128, page=64, block=64, dtype="bf16", lens_seed=1),
        # prefill chunks of three requests (16K tokens, 4K and a verify step's 7 near position 100K are the mix the key prologue serves)
        dict(name="store_prefill_20k", kind="store", reqs=3, new=6829, ctx=32768, kv_heads=8, dim=128, page=64, block=64, dtype="bf16", lens_seed=2),
        # one request at 80K tokens, one query token: the smallest decode step, where latency counts
        dict(name="attn_decode_80k", kind="attention", reqs=1, group=1, min_len=80000, max_len=80000, q_heads=64, kv_heads=8, dim=128, page=64, block=64, dtype="bf16", lens_seed=3),
        # the 7-row verify step (one token and six drafts) at 80K
        dict(name="attn_verify_80k", kind="attention", reqs=1, group=7, min_len=80000, max_len=80006, q_heads=64, kv_heads=8, dim=128, page=64, block=64, dtype="bf16", lens_seed=4),
        # mixed decode batch, log-uniform lengths
        dict(name="attn_mixed_32", kind="attention", reqs=32, group=1, min_len=1024, max_len=131072, q_heads=64, kv_heads=8, dim=128, page=64, block=32, dtype="fp16", lens_seed=5),
        # what top-k hands over: 2048 slots for each of 7 verify rows
        dict(name="selected_verify_7", kind="selected", reqs=1, group=7, min_len=80000, max_len=80006, k=2048, q_heads=64, kv_heads=8, dim=128, page=64, block=64, dtype="bf16", lens_seed=6),
        # 64 decode rows over their selections, some contexts shorter than k
        dict(name="selected_decode_64", kind="selected", reqs=64, group=1, min_len=1024, max_len=20000, k=2048, q_heads=32, kv_heads=8, dim=128, page=64, block=16, dtype="bf16", lens_seed=7),
        # one request, six drafts
        dict(name="verify_1", kind="verify", reqs=1, drafts=6, vocab=131072, point=False),
        # a batch with an odd vocabulary
        dict(name="verify_64_odd", kind="verify", reqs=64, drafts=6, vocab=100003, point=False),
        # eight samples forked from one 80K prompt, each about to append its next token into the shared tail page
        dict(name="pages_fork_8", kind="pages", op="fork", parents=1, children=8, ctx=80000, page=64, pages=4096, kv_heads=8, dim=128, live=0.0, lens_seed=8),
        # the pages of an 80K request copied
        dict(name="pages_copy_80k", kind="pages", op="copy", n=1251, page=64, pages=4096, kv_heads=8, dim=128, lens_seed=9),
        # a half-empty pool of 1M tokens compacted
        dict(name="pages_compact_16k", kind="pages", op="compact", page=64, pages=16384, kv_heads=8, dim=128, live=0.5, lens_seed=10),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["store", "attention", "selected", "verify", "pages"])
    seed = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= page])
    dim = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    kv = rng.choice([1, 2, 4, 8])
    if kind == "store":
        new = rng.choice([1, 1, 7, _log_int(rng, 2, 4096)])
        reqs = max(1, min(_log_int(rng, 1, 128), 20480 // new))
        return dict(kind=kind, reqs=reqs, new=new, ctx=_log_int(rng, 64, 8192), kv_heads=kv, dim=dim, page=page, block=block, dtype=dtype, lens_seed=seed)
    if kind == "verify":
        return dict(kind=kind, reqs=_log_int(rng, 1, 64), drafts=rng.randint(1, 7), vocab=_log_int(rng, 1000, 160000), point=rng.random() < 0.3)
    if kind == "pages":
        op = rng.choice(["fork", "copy", "compact"])
        pages = _log_int(rng, 1024, 8192)
        if op == "copy":
            return dict(kind=kind, op=op, n=_log_int(rng, 1, pages // 2), page=page, pages=pages, kv_heads=kv, dim=dim, lens_seed=seed)
        if op == "compact":
            return dict(kind=kind, op=op, page=page, pages=pages, kv_heads=kv, dim=dim, live=round(rng.uniform(0.1, 0.95), 3), lens_seed=seed)
        parents, children = rng.randint(1, 8), rng.randint(1, 8)
        return dict(kind=kind, op=op, parents=parents, children=children, ctx=_log_int(rng, 1, page * pages // (2 * parents)), page=page, pages=pages,
                    kv_heads=kv, dim=dim, live=round(rng.uniform(0.0, 0.2), 3), lens_seed=seed)
    ratio = rng.choice([1, 4, 7, 8, 16])
    group = rng.choice([1, 1, 2, 4, 7, 8])
    reqs = _log_int(rng, 1, 64)
    top = min(200000, 4000000 // (reqs * group))
    hi = _log_int(rng, min(200, top), top)
    lo = max(group, int(hi * rng.uniform(0.01, 1.0)))
    case = dict(kind=kind, reqs=reqs, group=group, min_len=lo, max_len=hi, q_heads=kv * ratio, kv_heads=kv, dim=dim, page=page, block=block, dtype=dtype, lens_seed=seed)
    if kind == "selected":
        case["reqs"] = reqs = min(reqs, 256 // group)
        case["max_len"] = hi = min(hi, 2000000 // reqs)
        case["min_len"] = min(lo, hi)
        case["k"] = rng.choice([64, 512, 2048, rng.randint(1, 2048)])
    return case


def _type(case):
    return torch.float16 if case["dtype"] == "fp16" else torch.bfloat16


def _lens(case):
    """Length of each request's last query row."""
    rng = random.Random(case["lens_seed"])
    lo, hi = case["min_len"], case["max_len"]
    return [min(hi, max(lo, _log_int(rng, lo, hi))) for _ in range(case["reqs"])]


def _row_lens(case):
    """Row g of a group of G sees all but the last G - 1 - g tokens."""
    g = case["group"]
    return [max(0, n - (g - 1 - i)) for n in _lens(case) for i in range(g)]


def _store_starts(case):
    rng = random.Random(case["lens_seed"])
    return [rng.randint(0, case["ctx"]) for _ in range(case["reqs"])]


def _page_bytes(case):
    """Bytes of one page: K and V codes, their scales (one per head for a block of a page), indexer keys and their scales."""
    return 2 * case["page"] * case["kv_heads"] * case["dim"] + 8 * case["kv_heads"] + case["page"] * (case["dim"] + 4)


def work(case):
    kind = case["kind"]
    if kind == "store":
        n = case["reqs"] * case["new"] * case["kv_heads"] * case["dim"]
        return {"bytes": 2 * n * 3, "flops": 4 * n}
    if kind == "verify":
        rows = case["reqs"] * (1 if case["point"] else 1.75)  # about a quarter of the requests keep every draft and need no draft row
        return {"bytes": int(rows * case["vocab"] * 4), "flops": int(rows * case["vocab"] * 2)}
    if kind == "pages":
        if case["op"] == "copy":
            moved = case["n"]
        elif case["op"] == "compact":
            moved = int(case["pages"] * case["live"] * (1 - case["live"]))
        else:
            moved = case["parents"] * case["children"]
        table = 4 * case["pages"] * 2 if case["op"] != "fork" else 8 * case["parents"] * case["children"] * -(-case["ctx"] // case["page"])
        return {"bytes": int(2 * moved * _page_bytes(case) + table), "flops": 0}
    d, hq, hk = case["dim"], case["q_heads"], case["kv_heads"]
    rows = case["reqs"] * case["group"]
    if kind == "attention":
        keys, pairs = sum(_lens(case)), sum(_row_lens(case))
    else:
        pairs = sum(min(case["k"], n) for n in _row_lens(case))
        keys = pairs
    return {"bytes": int(keys * hk * (2 * d + 8 / case["block"]) + 4 * rows * hq * d), "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _tables(gen, need, width, pages):
    """One row of page ids per request, drawn from a shuffled pool; -1 past a request's pages."""
    perm = torch.randperm(pages, generator=gen, device="cuda")
    need = torch.tensor(need, device="cuda")
    col = torch.arange(width, device="cuda")
    at = (torch.cumsum(need, 0) - need)[:, None] + col
    return torch.where(col < need[:, None], perm[at.clamp(max=pages - 1)], -1).to(torch.int32)


def _codes(gen, slots, heads, dim):
    x = torch.randn((slots, heads, dim), generator=gen, device="cuda", dtype=torch.float16)
    return x.mul_(100).clamp_(-448, 448).to(E4M3).view(torch.uint8)


def _scales(gen, blocks, heads):
    return torch.exp(0.3 * torch.randn((blocks, heads), generator=gen, device="cuda")) / 100


def prepare(case, seed):
    gen = _gen(seed)
    s = {"case": case}
    kind = case["kind"]
    if kind == "verify":
        n, d, v = case["reqs"], case["drafts"], case["vocab"]
        logits = 2.5 * torch.randn((n, d + 1, v), generator=gen, device="cuda")
        s["target"] = torch.softmax(logits, -1)
        near = logits[:, :d] + 0.4 * torch.randn((n, d, v), generator=gen, device="cuda")
        q = torch.softmax(near, -1)
        pick = torch.rand((n, d, 1), generator=gen, device="cuda", dtype=torch.float64)
        c = torch.cumsum(q.double(), -1)
        best = near.argmax(-1) if case["point"] else (c > pick * c[..., -1:]).int().argmax(-1)
        s["draft"] = None if case["point"] else q
        s["tokens"] = best.to(torch.int32)
        s["uniforms"] = torch.rand((n, d + 1), generator=gen, device="cuda")
        return s
    heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    if kind == "pages":
        return _prepare_pages(case, gen, s)
    block = case["block"]
    if kind == "store":
        starts = _store_starts(case)
        need = [-(-(x + case["new"]) // page) for x in starts]
    else:
        starts = _lens(case)
        need = [-(-x // page) for x in starts]
    pages = sum(need) + 3
    s["table"] = _tables(gen, need, max(need) + 1, pages)
    cache = dict(k=_codes(gen, pages * page, heads, dim), v=_codes(gen, pages * page, heads, dim),
                 k_scale=_scales(gen, pages * page // block, heads), v_scale=_scales(gen, pages * page // block, heads))
    s["cache"] = cache
    if kind == "store":
        n = case["reqs"] * case["new"]
        s["k_new"] = torch.randn((n, heads, dim), generator=gen, device="cuda").mul_(3).to(_type(case))
        s["v_new"] = torch.randn((n, heads, dim), generator=gen, device="cuda").to(_type(case))
        first = torch.tensor(starts, device="cuda", dtype=torch.int32)
        step = torch.arange(case["new"], device="cuda", dtype=torch.int32)
        s["positions"] = (first[:, None] + step).reshape(-1)
        s["token_table"] = torch.arange(case["reqs"], device="cuda", dtype=torch.int32).repeat_interleave(case["new"])
        s["first"] = torch.arange(case["reqs"], device="cuda") * case["new"]  # each request's first token
    else:
        rows = case["reqs"] * case["group"]
        s["q"] = (1.5 * torch.randn((rows, case["q_heads"], dim), generator=gen, device="cuda")).to(_type(case))
        s["scale"] = 1.0 / math.sqrt(dim)
        s["lens"] = torch.tensor(_row_lens(case), device="cuda", dtype=torch.int32)
        s["of"] = torch.arange(case["reqs"], device="cuda", dtype=torch.int32)  # table row of each group
        s["max_len"] = max(starts)
        if kind == "selected":
            k = case["k"]
            lens = s["lens"].long()[:, None]
            # k distinct positions of each row: an odd stride's multiples modulo the next power of two, cut to the length
            w = 1 << max(1, (max(starts) - 1).bit_length())
            j = torch.arange(w, device="cuda")
            off = torch.randint(0, w, (rows, 1), generator=gen, device="cuda")
            at = torch.cat([(off[r:r + 1] + j * 40503) % w for r in range(rows)])
            keep = at < lens
            order = torch.argsort((~keep).to(torch.int8), dim=1, stable=True)[:, :k]
            pos = torch.gather(at, 1, order)
            got = torch.gather(keep, 1, order)
            row = torch.arange(rows, device="cuda")[:, None] // case["group"]
            slot = s["table"][row, (pos // page).clamp(max=s["table"].shape[1] - 1)].long() * page + pos % page
            slots = torch.full((rows, k), -1, device="cuda", dtype=torch.int32)
            slots[:, :pos.shape[1]] = torch.where(got, slot, -1).to(torch.int32)
            s["slots"] = slots
    if own:
        from sparse_attention_indexer_gb300 import Kv8Cache
        s["api"] = Kv8Cache(cache["k"], cache["v"], cache["k_scale"], cache["v_scale"], page, block)
    return s


def _prepare_pages(case, gen, s):
    n, page, heads, dim = case["pages"], case["page"], case["kv_heads"], case["dim"]
    byte = lambda *shape: torch.randint(0, 120, shape, generator=gen, device="cuda", dtype=torch.uint8)  # noqa: E731
    s["planes"] = [byte(n, page * heads * dim), byte(n, page * heads * dim), torch.rand((n, heads), generator=gen, device="cuda"),
                   torch.rand((n, heads), generator=gen, device="cuda"), byte(n, page * dim), torch.rand((n, page), generator=gen, device="cuda")]
    op = case["op"]
    perm = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
    if op == "copy":
        s["src"], s["dst"] = perm[:case["n"]].contiguous(), perm[n - case["n"]:].contiguous()
        s["table"] = torch.full((1, 8), -1, device="cuda", dtype=torch.int32)
        s["refs"] = torch.zeros(n, device="cuda", dtype=torch.int32)
    elif op == "compact":
        # random pages of 16 requests; the rest of the pool is free
        live = int(n * case["live"])
        width = -(-live // 16)
        table = torch.full((16 * width,), -1, device="cuda", dtype=torch.int32)
        table[:live] = perm[:live]
        s["table0"] = table.view(16, width)
        s["refs0"] = torch.zeros(n, device="cuda", dtype=torch.int32)
        s["refs0"][perm[:live].long()] = 1
        s["table"], s["refs"] = s["table0"].clone(), s["refs0"].clone()
    else:
        par, kids = case["parents"], case["children"]
        used = -(-case["ctx"] // page)
        other = int(n * case["live"])
        width = -(-(case["ctx"] + 1) // page) + 1
        table = torch.full((par * (1 + kids), width), -1, device="cuda", dtype=torch.int32)
        table[:par, :used] = perm[:par * used].view(par, used)
        s["table"], s["refs"] = table, torch.zeros(n, device="cuda", dtype=torch.int32)
        s["refs"][perm[:par * used + other].long()] = 1
        ids = torch.arange(par * (1 + kids), device="cuda", dtype=torch.int32)
        s["children"] = ids[par:].contiguous()
        s["parents"] = ids[:par].repeat_interleave(kids).contiguous()
        s["old"] = torch.full((par * kids,), case["ctx"], device="cuda", dtype=torch.int32)
        s["new"] = s["old"] + 1
    if own:
        from sparse_attention_indexer_gb300 import KvPages
        s["api"] = KvPages(s["table"], s["refs"], page, s["planes"])
    return s


# ------------------------------------------------------------------ the calls
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    kind = s["case"]["kind"]
    if kind == "store":
        s["api"].store(s["k_new"], s["v_new"], s["positions"], s["token_table"], s["table"])
        return _cache_out(s["cache"])
    if kind == "attention":
        return s["api"].attention(s["q"], s["lens"], s["max_len"], s["table"], s["scale"], s["case"]["group"], s["of"])
    if kind == "selected":
        return s["api"].attention_selected(s["q"], s["slots"], s["scale"])
    if kind == "verify":
        from sparse_attention_indexer_gb300 import verify_drafts
        return verify_drafts(s["target"], s["draft"], s["tokens"], s["uniforms"])
    op = s["case"]["op"]
    api = s["api"]
    if op == "copy":
        api.copy(s["src"], s["dst"])
        return s["planes"]
    if op == "compact":
        s["table"].copy_(s["table0"])  # back to the scattered pool
        s["refs"].copy_(s["refs0"])
        moved, counts = api.compact()
        return s["planes"], s["table"], s["refs"], moved, counts
    api.free(s["children"])  # the children of the pass before
    api.fork(s["parents"], s["children"], s["old"])
    api.reserve(s["children"], s["old"], s["new"])
    return s["planes"], s["table"], s["refs"]


def _cache_out(c):
    return c["k"].view(E4M3), c["v"].view(E4M3), c["k_scale"], c["v_scale"]


def _run_plain(s):
    kind = s["case"]["kind"]
    if kind == "store":
        slots, blocks, old = _plain_slots(s)
        _plain_store(s["cache"]["k"], s["cache"]["k_scale"], s["k_new"], slots, blocks, old, s["case"]["block"])
        _plain_store(s["cache"]["v"], s["cache"]["v_scale"], s["v_new"], slots, blocks, old, s["case"]["block"])
        return _cache_out(s["cache"])
    if kind == "attention":
        page, g = s["case"]["page"], s["case"]["group"]
        t = torch.arange(s["max_len"], device="cuda")
        row = s["table"][s["of"].long()].long()
        slots = row[:, t // page].clamp(min=0) * page + t % page
        mask = t < s["lens"].view(-1, g)[:, :, None]
        return _plain_attention(s, slots, mask)
    if kind == "selected":
        return _plain_attention(s, s["slots"].long().clamp(min=0), (s["slots"] >= 0)[:, None])
    if kind == "verify":
        return _plain_verify(s["target"], s["draft"], s["tokens"], s["uniforms"])
    op = s["case"]["op"]
    if op == "copy":
        src, dst = s["src"].long(), s["dst"].long()
        [p.index_copy_(0, dst, p[src]) for p in s["planes"]]
        return s["planes"]
    if op == "compact":
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        return (s["planes"], s["table"], s["refs"]) + _plain_compact(s["table"], s["refs"], s["planes"])
    _plain_free(s["table"], s["refs"], s["children"])
    _plain_fork(s["table"], s["refs"], s["parents"], s["children"], s["old"], s["case"]["page"])
    _plain_reserve(s["table"], s["refs"], s["planes"], s["children"], s["old"], s["new"], s["case"]["page"])
    return s["planes"], s["table"], s["refs"]


def _least_scale(amax):
    """The least power of two 2^e, e >= -120, with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, -120).clamp(min=-120)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_slots(s):
    """Each token's slot and block, and how many earlier tokens the first block of each request holds."""
    page, block = s["case"]["page"], s["case"]["block"]
    pos = s["positions"].long()
    slots = s["table"][s["token_table"].long(), pos // page].long() * page + pos % page
    return slots, slots // block, (slots[s["first"]] // block, slots[s["first"]] % block)


def _plain_store(codes, scales, x, slots, blocks, old, block):
    x = x.float()
    top = torch.zeros_like(scales).index_reduce_(0, blocks, x.abs().amax(-1), "amax")
    b, n = old  # the blocks that may hold earlier tokens, and how many
    before = scales[b]
    least = _least_scale(top)
    grown = torch.where(n[:, None] > 0, torch.maximum(before, least[b]), least[b])
    least[b] = grown
    scales[blocks] = least[blocks]
    at = b[:, None] * block + torch.arange(block, device="cuda")
    held = torch.arange(block, device="cuda") < n[:, None]
    was = codes[at]
    again = was.view(E4M3).float() * (before / grown)[:, None, :, None]
    codes[at] = torch.where(held[..., None, None], again.clamp(-448, 448).to(E4M3).view(torch.uint8), was)
    codes[slots] = (x / scales[blocks][..., None]).clamp(-448, 448).to(E4M3).view(torch.uint8)


def _plain_attention(s, slots, mask):
    """slots [groups, keys], mask [groups, rows of a group, keys]."""
    c, q = s["cache"], s["q"]
    block = s["case"]["block"]
    groups, keys = slots.shape
    rows, hq, dim = q.shape
    hk, g = c["k"].shape[1], rows // groups
    kf = c["k"][slots].view(E4M3).float() * c["k_scale"][slots // block][..., None]
    qf = q.float().view(groups, g, hk, hq // hk, dim).permute(0, 2, 1, 3, 4).reshape(groups, hk, -1, dim)
    sc = torch.matmul(qf, kf.permute(0, 2, 3, 1)).view(groups, hk, g, hq // hk, keys) * s["scale"]
    del kf
    sc = sc.masked_fill_(~mask[:, None, :, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    sc = sc.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = sc.sum(-1, keepdim=True)
    vf = c["v"][slots].view(E4M3).float() * c["v_scale"][slots // block][..., None]
    out = torch.matmul(sc.view(groups, hk, -1, keys), vf.permute(0, 2, 1, 3)).view(groups, hk, g, hq // hk, dim)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (torch.log(total) + top).squeeze(-1)
    return out.permute(0, 2, 1, 3, 4).reshape(rows, hq, dim).to(q.dtype), lse.permute(0, 2, 1, 3).reshape(rows, hq)


def _plain_verify(target, draft, tokens, uniforms):
    n, d = tokens.shape
    tok = tokens.long()[..., None]
    p = target[:, :d].gather(-1, tok).squeeze(-1).double()
    q = torch.ones_like(p) if draft is None else draft.gather(-1, tok).squeeze(-1).double()
    ok = uniforms[:, :d].double() * q < p
    kept = ok.int().cumprod(-1).sum(-1)
    every = torch.arange(n, device=tokens.device)
    last = kept.clamp(max=d - 1)
    whole = (target[every, kept].double() * UNIT).to(torch.int64)
    if draft is None:
        less = torch.zeros_like(whole).scatter_(1, tokens[every, last].long()[:, None], int(UNIT))
    else:
        less = (draft[every, last].double() * UNIT).to(torch.int64)
    rest = (whole - less).clamp(min=0)
    rest = torch.where(((kept < d) & (rest.sum(-1) > 0))[:, None], rest, whole)
    run_sum = torch.cumsum(rest, -1)
    want = (uniforms[:, d].double() * run_sum[:, -1].double()).to(torch.int64)
    new = (run_sum > want[:, None]).int().argmax(-1).to(torch.int32)
    col = torch.arange(d + 1, device=tokens.device)
    padded = torch.cat([tokens, tokens[:, :1]], 1)
    out = torch.where(col < kept[:, None], padded, torch.where(col == kept[:, None], new[:, None], -1))
    return out.to(torch.int32), kept.to(torch.int32)


def _plain_free(table, refs, rows):
    row = table[rows.long()]
    refs.index_add_(0, row.clamp(min=0).long().view(-1), -(row >= 0).to(torch.int32).view(-1))
    table[rows.long()] = -1


def _plain_fork(table, refs, parents, children, lens, page):
    col = torch.arange(table.shape[1], device=table.device)
    row = torch.where(col * page < lens[:, None], table[parents.long()], -1)
    table[children.long()] = row
    refs.index_add_(0, row.clamp(min=0).long().view(-1), (row >= 0).to(torch.int32).view(-1))


def _plain_reserve(table, refs, planes, rows, old, new, page):
    col = torch.arange(table.shape[1], device=table.device)
    row = table[rows.long()].long()
    span = (col >= (old // page)[:, None]) & (col * page < new[:, None]) & (new > old)[:, None]
    shared = span & (row >= 0) & (refs[row.clamp(min=0)] > 1)
    need = span & ((row < 0) | shared)
    per_row = need.sum(-1)
    served = torch.cumsum(per_row, 0) <= (refs == 0).sum()
    need, shared = need & served[:, None], shared & served[:, None]
    free = torch.argsort((refs > 0).to(torch.int8), stable=True)
    rank = torch.cumsum(need.view(-1), 0).view(need.shape) - 1
    got = torch.where(need, free[rank.clamp(min=0)], row)
    r, c = torch.nonzero(shared & (col * page < old[:, None]), as_tuple=True)
    src, dst = row[r, c], got[r, c]
    [p.index_copy_(0, dst, p[src]) for p in planes]
    refs.index_add_(0, row.clamp(min=0).view(-1), -shared.to(torch.int32).view(-1))
    refs.index_add_(0, got.clamp(min=0).view(-1), need.to(torch.int32).view(-1))
    table[rows.long()] = got.to(torch.int32)


def _plain_compact(table, refs, planes):
    n = refs.shape[0]
    ids = torch.arange(n, device=refs.device)
    live = refs > 0
    count = live.sum()
    src = torch.nonzero(live & (ids >= count)).view(-1)
    dst = torch.nonzero(~live & (ids < count)).view(-1)
    [p.index_copy_(0, dst, p[src]) for p in planes]
    new = torch.where(live, ids, -1)
    new[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, new[table.clamp(min=0).long()], table.long()))
    return new.to(torch.int32), torch.stack([count, count.new_tensor(src.numel())]).to(torch.int32)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    kind = case["kind"]
    if kind == "pages" or kind == "verify":
        return None
    keep = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = keep
    if kind == "store":
        return _exact_store(s)
    if kind == "attention":
        page = case["page"]
        off = torch.arange(page, device="cuda")
        return _exact_attention(s, [(s["table"][r // case["group"], :-(-n // page)].long()[:, None] * page + off).reshape(-1)[:n]
                                    for r, n in enumerate(s["lens"].tolist())])
    return _exact_attention(s, [x[x >= 0].long() for x in s["slots"]])


def _exact_attention(s, lists):
    """Row by row and head by head over the list of each row's slots."""
    c, q, block = s["cache"], s["q"].double(), s["case"]["block"]
    rows, hq, dim = q.shape
    ratio = hq // c["k"].shape[1]
    out = torch.zeros((rows, hq, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device="cuda")
    for r, at in enumerate(lists):
        if len(at) == 0:
            continue
        for h in range(c["k"].shape[1]):
            k = c["k"][at, h].view(E4M3).double() * c["k_scale"][at // block, h].double()[:, None]
            v = c["v"][at, h].view(E4M3).double() * c["v_scale"][at // block, h].double()[:, None]
            x = q[r, h * ratio:(h + 1) * ratio] @ k.T * s["scale"]
            lse[r, h * ratio:(h + 1) * ratio] = torch.logsumexp(x, -1)
            out[r, h * ratio:(h + 1) * ratio] = torch.softmax(x, -1) @ v
    return out, lse


def _exact_store(s):
    """What each code stands for before its rounding, and the scales."""
    c, page, block = s["cache"], s["case"]["page"], s["case"]["block"]
    pos, row = s["positions"].tolist(), s["token_table"].tolist()
    table = s["table"].tolist()
    runs = []  # [block, earlier tokens, first new token, new tokens]
    for t, (p, r) in enumerate(zip(pos, row)):
        slot = table[r][p // page] * page + p % page
        if runs and runs[-1][0] == slot // block and row[t - 1] == r:
            runs[-1][3] += 1
        else:
            runs.append([slot // block, slot % block, t, 1])
    got = []
    for codes, scales, x in ((c["k"], c["k_scale"], s["k_new"]), (c["v"], c["v_scale"], s["v_new"])):
        val, sc = codes.view(E4M3).double(), scales.double().clone()
        for b, off, t, n in runs:
            y = x[t:t + n].double()
            top = y.abs().amax((0, 2)).tolist()
            # floats in Python: 2^e and 448 * 2^e are exact, so is the comparison
            new = torch.tensor([next(2.0 ** e for e in range(-120, 129) if a <= 448 * 2.0 ** e) for a in top], dtype=torch.float64, device="cuda")
            if off:
                new = torch.maximum(new, sc[b])
                val[b * block:b * block + off] *= (sc[b] / new)[None, :, None]
            sc[b] = new
            val[b * block + off:b * block + off + n] = y / new[None, :, None]
        got.append((val, sc))
    return got[0][0], got[1][0], got[0][1], got[1][1]
