"""What the prompt-side and drafting-side operators compute, and the sizes they are measured at.

Around the selection and the quantised cache a serving program needs four more
things: attention over whole prompts of packed sequences, whose log-sum-exps the
scoring takes (`tsel_prompt_attention`); attention of a tree of drafted tokens
over the cache (`tsel_tree_attention`); the cache rows of the tokens that stay,
moved together (`tsel_cache_compact`); and requests that start from another one's
pages, grow and end (`tsel_cache_fork`, `tsel_cache_resize`).

`run` computes a case with plain torch operations in 32 bits where `own` is
false, and with the library's calls where it is true. `exact` gives the same
outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
MOST = 5.7e12        # operations of the largest case


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one image in a small vision encoder: latency counts
        dict(name="prompt_image", op="prompt", segments=1, rows=256, context=0, causal=False, heads=4, kv_heads=4, dim=64, type="bf16"),
        # the vision encoder of a 30-image request, images of up to 4,096 tokens, no mask; the scoring reuses the log-sum-exps
        dict(name="prompt_images", op="prompt", segments=30, rows=4096, context=0, causal=False, heads=16, kv_heads=16, dim=80, type="bf16"),
        # the language model's prefill of the pruned 30-image request and its question: 36,831 + 142 tokens
        dict(name="prompt_pruned", op="prompt", segments=1, rows=36973, context=0, causal=True, heads=16, kv_heads=8, dim=128, type="bf16"),
        # prefill of 24 pruned six-view requests at once: packed, ragged
        dict(name="prompt_batch", op="prompt", segments=24, rows=1370, context=0, causal=True, heads=32, kv_heads=8, dim=128, type="fp16"),
        # a question of 142 tokens after 36,831 that are there already: few rows, many keys
        dict(name="prompt_question", op="prompt", segments=1, rows=142, context=36831, causal=True, heads=16, kv_heads=8, dim=128, type="bf16"),
        # four users of one six-view request, eight drafted tokens each: latency counts
        dict(name="tree_six_views", op="tree", requests=4, nodes=8, prefix=1228, suffix=142, heads=16, kv_heads=8, dim=128, page=16, type="bf16"),
        # 32 users of the pruned 30-image request, 16 drafted tokens each after answers of up to 1,000 tokens
        dict(name="tree_step", op="tree", requests=32, nodes=16, prefix=36831, suffix=1000, heads=32, kv_heads=8, dim=128, page=64, type="bf16"),
        # large trees over each request's own keys, one query head per cached head
        dict(name="tree_own", op="tree", requests=16, nodes=61, prefix=0, suffix=4000, heads=16, kv_heads=16, dim=80, page=32, type="fp16"),
        # the accepted path of 64 drafted trees goes to the front, in place
        dict(name="compact_accepted", op="compact", requests=64, tokens=1000, nodes=32, kept=6, inplace=True, kv_heads=8, dim=128, page=64),
        # 60% of the cached tokens of a 30-image request into pages of their own (its old pages stay with others)
        dict(name="compact_pruned", op="compact", requests=1, tokens=61385, nodes=61385, kept=36831, inplace=False, kv_heads=8, dim=128, page=64),
        # four answers sampled from each of 16 six-view requests: forked, grown by a few tokens, freed
        dict(name="fork_answers", op="fork", parents=16, children=4, tokens=1370, grow=20, kv_heads=8, dim=128, page=16, spare=700),
        # 256 answers over 8 prompts of the pruned 30-image request, a pool of some thousand large pages
        dict(name="fork_many", op="fork", parents=8, children=32, tokens=36973, grow=300, kv_heads=8, dim=128, page=128, spare=1200),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "tree", "tree", "compact", "fork"])
    dim = rng.choice([64, 80, 96, 112, 128])
    kv = rng.choice([1, 2, 4, 8])
    if op == "prompt":
        c = dict(op=op, segments=_log(rng, 1, 64), rows=_log(rng, 1, 16384), context=rng.choice([0, 0, _log(rng, 1, 40000)]),
                 causal=rng.random() < 0.6, heads=kv * rng.choice([1, 2, 4, 5, 8]), kv_heads=kv, dim=dim,
                 type=rng.choice(["bf16", "bf16", "fp16"]))
        while work(c)["flops"] > MOST / 2 or sum(_qlens(c)) > 131072 or sum(_klens(c)) > 400000:
            if c["segments"] > 1:
                c["segments"] = (c["segments"] + 1) // 2
            else:
                c["rows"] = c["rows"] // 2 + 1
        return c
    page = rng.choice([16, 32, 64, 128])
    if op == "tree":
        c = dict(op=op, requests=_log(rng, 1, 64), nodes=_log(rng, 2, 64), prefix=rng.choice([0, _log(rng, 1, 40000)]), suffix=_log(rng, 70, 4000),
                 heads=kv * rng.choice([1, 2, 4, 5, 8]), kv_heads=kv, dim=dim, page=page, type=rng.choice(["bf16", "fp16"]))
        while work(c)["flops"] > 6.0e11 or c["requests"] * c["suffix"] > 200000:
            c["prefix"] //= 2
            c["requests"] = c["requests"] // 2 + 1
        return c
    if op == "compact":
        if rng.random() < 0.5:
            nodes = _log(rng, 2, 64)
            return dict(op=op, requests=_log(rng, 1, 200), tokens=_log(rng, 100, 2000), nodes=nodes, kept=rng.randint(1, (nodes + 1) // 2),
                        inplace=True, kv_heads=kv, dim=dim, page=page)
        tokens = _log(rng, 100, 61385)
        return dict(op=op, requests=rng.choice([1, 1, 2, 3]), tokens=tokens, nodes=tokens, kept=max(1, tokens * rng.randint(30, 90) // 100), inplace=False,
                    kv_heads=kv, dim=dim, page=page)
    tokens = _log(rng, 1, 37000)
    grow = _log(rng, 1, 500)
    parents, children = _log(rng, 1, 16), _log(rng, 1, 32)
    return dict(op=op, parents=parents, children=children, tokens=tokens, grow=grow, kv_heads=kv, dim=dim, page=page,
                spare=parents * children * (1 + (grow + page) // page) + rng.randint(0, 500))


def _ragged(n, most, a, b):
    """n lengths from 1 to `most`, the first the longest."""
    return [1 + (a * i + b) % most if i else most for i in range(n)]


def _qlens(c):
    return _ragged(c["segments"], c["rows"], 7919, 3)


def _klens(c):
    before = [0] * c["segments"] if not c["context"] else _ragged(c["segments"], c["context"], 104729, 11)
    return [n + b for n, b in zip(_qlens(c), before)]


def _nodes(c):
    return _ragged(c["requests"], c["nodes"], 7919, 3)


def _lens(c):
    """Suffix keys of each request of a tree case, its drafted tokens among them."""
    return [n + (104729 * i + 11) % (c["suffix"] - n + 1) if i else c["suffix"] for i, n in enumerate(_nodes(c))]


def _kept(c):
    return _ragged(c["requests"], c["kept"], 31, 2) if c["inplace"] else [c["kept"]] * c["requests"]


def _parent_lens(c):
    return _ragged(c["parents"], c["tokens"], 6151, 5)


def _grown(c):
    return _ragged(c["parents"] * c["children"], c["grow"], 53, 7)


def _up(a, b):
    return (a + b - 1) // b


def work(c):
    d = c["dim"]
    if c["op"] == "prompt":
        nq, nk = _qlens(c), _klens(c)
        pairs = sum(a * b - (a * (a - 1) // 2 if c["causal"] else 0) for a, b in zip(nq, nk))
        bytes_ = sum(nq) * c["heads"] * (4 * d + 4) + 4 * sum(nk) * c["kv_heads"] * d
        return {"bytes": bytes_, "flops": 4 * d * c["heads"] * pairs}
    row = 2 * c["kv_heads"] * (d + 1)   # K and V of a cached token
    if c["op"] == "tree":
        n, lens = _nodes(c), _lens(c)
        keys = c["prefix"] + sum(lens)
        # a node sees the keys before the tree and about log(nodes) of the tree; counted as itself and one more
        pairs = sum(n) * c["prefix"] + sum(a * (s - a + 2) for a, s in zip(n, lens))
        return {"bytes": keys * row + sum(n) * (c["heads"] * (4 * d + 4) + 4), "flops": 4 * d * c["heads"] * pairs}
    if c["op"] == "compact":
        rows = sum(_kept(c))
        return {"bytes": rows * (2 * row + 4), "flops": rows}
    tails = sum(t % c["page"] for t in _parent_lens(c)) * c["children"]
    pages = sum(_up(t, c["page"]) for t in _parent_lens(c)) * c["children"]
    fresh = sum(_up(t + g, c["page"]) - t // c["page"] for t, g in zip([x for x in _parent_lens(c) for _ in range(c["children"])], _grown(c)))
    # shared pages: read and noted in the child's list, counted up and down again; fresh ones found and noted
    return {"bytes": 2 * tails * row + 24 * pages + 12 * fresh, "flops": 4 * (pages + fresh)}


# ------------------------------------------------------------------- the inputs

def _codes(rows, dim, g):
    """E4M3 codes and scale bytes of cached rows of varying size."""
    x = torch.randn(*rows, dim, generator=g, device=DEV)
    x *= torch.exp2(torch.randn(*rows, 1, generator=g, device=DEV))
    f, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(f <= 0.875, e - 9, e - 8).clamp(-127, 127)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _pool(c, pages, g):
    """A cache whose every row is in use."""
    shape = (pages, c["kv_heads"], c["page"])
    out = {}
    for n in "kv":
        out[n + "_pages"] = torch.empty(*shape, c["dim"], dtype=torch.uint8, device=DEV)
        out[n + "_exps"] = torch.empty(shape, dtype=torch.uint8, device=DEV)
        for a in range(0, pages, 512):
            out[n + "_pages"][a:a + 512], out[n + "_exps"][a:a + 512] = _codes((min(512, pages - a),) + shape[1:], c["dim"], g)
    return out


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    {"prompt": _prepare_prompt, "tree": _prepare_tree, "compact": _prepare_compact, "fork": _prepare_fork}[c["op"]](c, s, g)
    if own:
        import attention_score_vision_gb300 as tsel
        if "k_pages" in s:
            s["cache"] = tsel.TselCache(s["k_pages"], s["v_pages"], s["k_exps"], s["v_exps"])
        if c["op"] == "prompt":
            need = tsel.tsel_prompt_attention_workspace_size(c["segments"], s["q"].shape[0], s["max_q"], s["max_k"], c["heads"], c["kv_heads"], c["dim"])
        elif c["op"] == "tree":
            need = tsel.tsel_tree_attention_workspace_size(c["requests"], s["q"].shape[0], c["nodes"], c["heads"], c["kv_heads"], c["dim"],
                                                           c["prefix"], c["suffix"])
        elif c["op"] == "compact":
            need = tsel.tsel_cache_workspace_size()
        else:
            need = tsel.tsel_cache_resize_workspace_size(s["table"].shape[0], s["table"].shape[1])
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    return s


def _prepare_prompt(c, s, g):
    nq, nk = _qlens(c), _klens(c)
    dt, h, hk, d = TYPES[c["type"]], c["heads"], c["kv_heads"], c["dim"]
    if not c["context"]:   # views of one projection's output
        qkv = torch.randn(sum(nq), h + 2 * hk, d, generator=g, device=DEV).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    else:
        s["q"] = torch.randn(sum(nq), h, d, generator=g, device=DEV).to(dt)
        s["k"], s["v"] = (torch.randn(sum(nk), hk, d, generator=g, device=DEV).to(dt) for _ in range(2))
    s["cu_q"], s["cu_k"] = (_ints([0] + list(x)).cumsum(0).to(torch.int32) for x in (nq, nk))
    s["max_q"], s["max_k"] = max(nq), max(nk)


def _prepare_tree(c, s, g):
    n, lens, ps = _nodes(c), _lens(c), c["page"]
    np_, ns = _up(c["prefix"], ps), _up(c["suffix"], ps)
    pages = np_ + c["requests"] * ns + 3
    s.update(_pool(c, pages, g))
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    s["prefix_pages"] = order[:np_]
    s["table"] = order[np_:np_ + c["requests"] * ns].view(c["requests"], ns)
    s["q"] = torch.randn(sum(n), c["heads"], c["dim"], generator=g, device=DEV).to(TYPES[c["type"]])
    s["cu"] = _ints([0] + n).cumsum(0).to(torch.int32)
    s["lens"] = _ints(lens)
    s["prefix_len"] = _ints([c["prefix"]])
    # node i of a request hangs on one before it, or on the last key before the tree (-1)
    i = torch.cat([torch.arange(a, device=DEV) for a in n])
    s["parents"] = (torch.rand(i.numel(), generator=g, device=DEV, dtype=torch.float64) * (i + 1)).floor().to(torch.int32) - 1


def _prepare_compact(c, s, g):
    ps, r = c["page"], c["requests"]
    n = _up(c["tokens"] + c["nodes"] if c["inplace"] else c["tokens"], ps)
    m = 0 if c["inplace"] else _up(c["kept"], ps)
    pages = r * (n + m) + 3
    s.update(_pool(c, pages, g))
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    s["table"] = order[:r * n].view(r, n)
    s["to"] = None if c["inplace"] else order[r * n:r * (n + m)].view(r, m)
    kept = _kept(c)
    s["cu"] = _ints([0] + kept).cumsum(0).to(torch.int32)
    keep = []
    for a in kept:
        if c["inplace"]:   # accepted from the front, then some further behind
            front = int(torch.randint(max(0, 2 * a - c["nodes"]), a + 1, (1,), generator=g, device=DEV))
            rest = a + torch.randperm(c["nodes"] - a, generator=g, device=DEV)[:a - front].sort().values
            keep.append(torch.cat([torch.arange(front, device=DEV), rest]))
        else:
            keep.append(torch.randperm(c["tokens"], generator=g, device=DEV)[:a].sort().values)
    if c["inplace"]:
        s["starts"], s["bases"] = _ints(_ragged(r, c["tokens"], 6151, 5)), None
    else:   # indices as the selection gives them, over the tokens of all requests
        s["starts"], s["bases"] = None, _ints([i * c["tokens"] for i in range(r)])
        keep = [k + i * c["tokens"] for i, k in enumerate(keep)]
    s["keep"] = torch.cat(keep).to(torch.int32)


def _prepare_fork(c, s, g):
    ps, lens, grown = c["page"], _parent_lens(c), _grown(c)
    kids = c["parents"] * c["children"]
    width = _up(c["tokens"] + c["grow"], ps)
    used = [_up(t, ps) for t in lens]
    pages = sum(used) + c["spare"]
    s.update(_pool(c, pages, g))
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((c["parents"] + kids, width), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    refs[order[:at].long()] = 1
    s["table"], s["refs"] = table, refs
    s["lens"] = _ints(lens + [0] * kids)
    s["parents"] = _ints([i // c["children"] for i in range(kids)])
    s["children"] = _ints([c["parents"] + i for i in range(kids)])
    s["grown"] = _ints([-1] * c["parents"] + [lens[i // c["children"]] + grown[i] for i in range(kids)])   # -1: as it is
    s["ended"] = _ints([-1] * c["parents"] + [0] * kids)


# ------------------------------------------------------------------- the plain forms

def _plain_prompt(s, c):
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    group = h // hk
    q, k, v = s["q"], s["k"], s["v"]
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    lse = torch.empty(h, q.shape[0], device=DEV)
    a = b = 0
    for nq, nk in zip(_qlens(c), _klens(c)):
        kk, vv = k[b:b + nk].float().permute(1, 2, 0), v[b:b + nk].float().transpose(0, 1)
        step = max(1, 400_000_000 // (h * nk))
        for i in range(0, nq, step):
            n = min(step, nq - i)
            qq = q[a + i:a + i + n].float().view(n, hk, group, d).permute(1, 2, 0, 3).reshape(hk, group * n, d) / math.sqrt(d)
            p = torch.matmul(qq, kk).view(hk, group, n, nk)
            if c["causal"]:
                seen = torch.arange(nk, device=DEV) <= torch.arange(i, i + n, device=DEV)[:, None] + (nk - nq)
                p.masked_fill_(~seen, -math.inf)
            top = p.amax(-1, keepdim=True)
            p = p.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(hk, group * n, nk), vv).view(hk, group, n, d) / total
            out[a + i:a + i + n] = o.permute(2, 0, 1, 3).reshape(n, h, d).to(q.dtype)
            lse[:, a + i:a + i + n] = (top + total.log()).view(h, n)
        a, b = a + nq, b + nk
    return out, lse


def _plain_rows(s, page, at):
    return [torch.ldexp(s[n + "_pages"][page, :, at].view(torch.float8_e4m3fn).float(), (s[n + "_exps"][page, :, at].int() - 127)[..., None])
            for n in "kv"]


def _plain_tree(s, c):
    ps, hk, d, top_n = c["page"], c["kv_heads"], c["dim"], c["nodes"]
    group, r = c["heads"] // hk, c["requests"]
    tokens = s["q"].shape[0]
    j = torch.arange(c["suffix"], device=DEV).expand(r, -1)
    sk, sv = (x.view(r, -1, hk, d).permute(0, 2, 1, 3) for x in _plain_rows(s, s["table"].long().gather(1, j // ps).reshape(-1), (j % ps).reshape(-1)))
    cu = s["cu"].long()
    t = torch.arange(tokens, device=DEV)
    req = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[req]
    n = cu[1:] - cu[:-1]
    # which nodes of the tree each one sees: paths of any length up to the root
    sees = torch.zeros(r, top_n, top_n, device=DEV)
    sees[req, i, i] = 1.0
    hangs = s["parents"] >= 0
    sees[req[hangs], i[hangs], s["parents"].long()[hangs]] = 1.0
    reach = 1
    while reach < top_n:
        sees = (torch.matmul(sees, sees) > 0).float()
        reach *= 2
    before = s["lens"].long()[req] - n[req]
    at = torch.arange(c["suffix"], device=DEV) - before[:, None]
    inside = (at >= 0) & (at < n[req][:, None])
    seen = (at < 0) | (inside & (sees[req, i].gather(1, at.clamp(0, top_n - 1)) > 0))
    q = s["q"].float().view(tokens, hk, group, d) / math.sqrt(d)
    padded = q.new_zeros(r, top_n, hk, group, d)
    padded[req, i] = q
    ss = torch.matmul(padded.permute(0, 2, 1, 3, 4).reshape(r, hk, top_n * group, d), sk.transpose(2, 3)).view(r, hk, top_n, group, -1)
    ss = ss.permute(0, 2, 1, 3, 4)[req, i].permute(1, 0, 2, 3)     # [Hkv, T, group, S]
    ss = ss.masked_fill(~seen[None, :, None], -math.inf)
    top = ss.amax(-1)
    if c["prefix"]:
        p = torch.arange(c["prefix"], device=DEV)
        pk, pv = _plain_rows(s, s["prefix_pages"].long()[p // ps], p % ps)
        sp = torch.matmul(q.permute(1, 0, 2, 3).reshape(hk, tokens * group, d), pk.permute(1, 2, 0)).view(hk, tokens, group, -1)
        top = torch.maximum(top, sp.amax(-1))
        sp = torch.exp(sp - top[..., None])
    ss = torch.exp(ss - top[..., None])
    total = ss.sum(-1)
    padded = ss.new_zeros(r, top_n, hk, group, ss.shape[-1])
    padded[req, i] = ss.permute(1, 0, 2, 3)
    out = torch.matmul(padded.permute(0, 2, 1, 3, 4).reshape(r, hk, top_n * group, -1), sv).view(r, hk, top_n, group, d)
    out = out.permute(0, 2, 1, 3, 4)[req, i].permute(1, 0, 2, 3)
    if c["prefix"]:
        total = total + sp.sum(-1)
        out = out + torch.matmul(sp.reshape(hk, tokens * group, -1), pv.permute(1, 0, 2)).view(hk, tokens, group, d)
    lse = top + total.log()
    out = out / total[..., None]
    return out.permute(1, 0, 2, 3).reshape(tokens, c["heads"], d).to(s["q"].dtype), lse.permute(0, 2, 1).reshape(c["heads"], tokens)


def _plain_compact(s, c):
    ps = c["page"]
    cu = s["cu"].long()
    t = torch.arange(s["keep"].numel(), device=DEV)
    req = torch.searchsorted(cu, t, right=True) - 1
    start = torch.zeros(c["requests"], dtype=torch.int64, device=DEV) if s["starts"] is None else s["starts"].long()
    src = start[req] + s["keep"].long() - (0 if s["bases"] is None else s["bases"].long()[req])
    dst = start[req] + t - cu[req]
    page = s["table"].long()[req, src // ps]
    to = (s["table"] if s["to"] is None else s["to"]).long()[req, dst // ps]
    for n in ("k_pages", "v_pages", "k_exps", "v_exps"):
        s[n][to, :, dst % ps] = s[n][page, :, src % ps]
    return [*_state(s), (start + cu[1:] - cu[:-1]).to(torch.int32)]


def _plain_resize(s, c, asked):
    """Pages for rows that grow (the lowest free ones, row by row), back from rows that shrink; -1 leaves a row alone."""
    ps, table, refs = c["page"], s["table"], s["refs"]
    old = s["lens"].long()
    new = torch.where(asked < 0, old, asked.long())
    have, need = (old + ps - 1) // ps, (new + ps - 1) // ps
    at = torch.arange(table.shape[1], device=DEV)
    grows = (at >= have[:, None]) & (at < need[:, None])
    drops = (at >= need[:, None]) & (at < have[:, None])
    free = torch.nonzero(refs == 0)[:, 0].to(torch.int32)
    fresh = free[:int(grows.sum())]
    table[grows] = fresh
    refs[fresh.long()] = 1
    refs.scatter_add_(0, table[drops].long(), torch.full((int(drops.sum()),), -1, dtype=torch.int32, device=DEV))
    s["lens"].copy_(new)


def _plain_fork(s, c):
    ps, table, refs, lens = c["page"], s["table"], s["refs"], s["lens"]
    src, dst = s["parents"].long(), s["children"].long()
    n = lens[src].long()
    at = torch.arange(table.shape[1], device=DEV)
    whole = at < (n // ps)[:, None]
    rows = torch.where(at < ((n + ps - 1) // ps)[:, None], table[src], table[dst])
    table[dst] = rows
    refs.scatter_add_(0, rows[whole].long(), torch.ones(int(whole.sum()), dtype=torch.int32, device=DEV))
    cut = torch.nonzero(n % ps)[:, 0]
    fresh = torch.nonzero(refs == 0)[:, 0][:cut.numel()]
    last = (n // ps)[cut]
    page = table[src[cut], last].long()
    table[dst[cut], last] = fresh.to(torch.int32)
    refs[fresh] = 1
    keeps = torch.arange(ps, device=DEV) < (n % ps)[cut][:, None]          # rows in use of the parent's last page
    for name in ("k_pages", "v_pages", "k_exps", "v_exps"):
        mask = keeps[:, None, :, None] if name.endswith("pages") else keeps[:, None, :]
        s[name][fresh] = torch.where(mask, s[name][page], s[name][fresh])
    lens[dst] = n.to(torch.int32)


def _state(s):
    return [s["k_pages"].view(torch.float8_e4m3fn), s["v_pages"].view(torch.float8_e4m3fn), s["k_exps"], s["v_exps"]]


# ------------------------------------------------------------------- a pass

def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "prompt":
        return _plain_prompt(s, c)
    if c["op"] == "tree":
        return _plain_tree(s, c)
    if c["op"] == "compact":
        return _plain_compact(s, c)
    _plain_fork(s, c)
    _plain_resize(s, c, s["grown"])
    _plain_resize(s, c, s["ended"])
    return [*_state(s), s["table"], s["refs"], s["lens"]]


def _run_own(s, c):
    import attention_score_vision_gb300 as tsel
    if c["op"] == "prompt":
        return tsel.tsel_prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"],
                                          flags=tsel.TSEL_ATT_CAUSAL if c["causal"] else 0, workspace=s["ws"])
    if c["op"] == "tree":
        prefix = (s["prefix_pages"], s["prefix_len"]) if c["prefix"] else (None, None)
        return tsel.tsel_tree_attention(s["q"], s["cu"], c["nodes"], s["parents"], s["cache"], *prefix, c["prefix"], s["table"], s["lens"], c["suffix"],
                                        workspace=s["ws"])
    if c["op"] == "compact":
        lens = tsel.tsel_cache_compact(s["cache"], s["table"], s["keep"], s["cu"], c["kept"], starts=s["starts"], bases=s["bases"], dst_table=s["to"],
                                       workspace=s["ws"])
        return [*_state(s), lens]
    tsel.tsel_cache_fork(s["cache"], s["refs"], s["table"], s["lens"], s["parents"], s["children"], workspace=s["ws"])
    tsel.tsel_cache_resize(s["refs"], s["table"], s["lens"], s["grown"], c["page"], workspace=s["ws"])
    tsel.tsel_cache_resize(s["refs"], s["table"], s["lens"], s["ended"], c["page"], workspace=s["ws"])
    return [*_state(s), s["table"], s["refs"], s["lens"]]


# ------------------------------------------------------------------- in 64 bits, from the definitions

def _exact_softmax(x, seen, values):
    """Weighted means of `values` and log-sum-exps of the logits that are seen."""
    x = torch.where(seen, x, torch.full((), -math.inf, dtype=torch.float64, device=DEV))
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[..., None]) @ values, lse


def exact(c, seed):
    if c["op"] not in ("prompt", "tree"):
        return None        # moved, not computed
    s = prepare(c, seed)
    h, group, d = c["heads"], c["heads"] // c["kv_heads"], c["dim"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(h, s["q"].shape[0], dtype=torch.float64, device=DEV)
    if c["op"] == "prompt":
        if work(c)["flops"] * (1 if c["context"] or not c["causal"] else 1.1) > 8e12:
            return None
        q0, k0 = s["cu_q"].tolist(), s["cu_k"].tolist()
        for z in range(c["segments"]):
            nq, nk = q0[z + 1] - q0[z], k0[z + 1] - k0[z]
            for head in range(h):
                k, v = (s[n][k0[z]:k0[z + 1], head // group].double() for n in "kv")
                for i in range(0, nq, 4096):
                    e = min(nq, i + 4096)
                    last = nk - nq + e if c["causal"] else nk       # keys that the block's last row sees
                    x = s["q"][q0[z] + i:q0[z] + e, head].double() @ k[:last].T * d ** -0.5
                    row = torch.arange(i, e, device=DEV)[:, None]
                    seen = (torch.arange(last, device=DEV) - (nk - nq) <= row) if c["causal"] else torch.ones_like(x, dtype=torch.bool)
                    out[q0[z] + i:q0[z] + e, head], lse[head, q0[z] + i:q0[z] + e] = _exact_softmax(x, seen, v[:last])
        return [out, lse]
    byte = torch.arange(256, device=DEV)
    size, power = byte % 8, (byte // 8) % 16
    grid = torch.where(power == 0, size * 2.0 ** -9, (8 + size).double() * torch.exp2((power - 10).double()))
    grid = torch.where(byte < 128, grid, -grid).double()
    cu, parents, lens, ps = s["cu"].tolist(), s["parents"].tolist(), s["lens"].tolist(), c["page"]
    for r in range(c["requests"]):
        n, m = cu[r + 1] - cu[r], lens[r]
        seen = torch.zeros(n, c["prefix"] + m, dtype=torch.bool)
        seen[:, :c["prefix"] + m - n] = True
        for i in range(n):
            node = i
            while node >= 0:
                seen[i, c["prefix"] + m - n + node] = True
                node = parents[cu[r] + node]
        seen = seen.to(DEV)
        pages = torch.cat([s["prefix_pages"].long().repeat_interleave(ps)[:c["prefix"]], s["table"][r].long().repeat_interleave(ps)[:m]])
        at = torch.cat([torch.arange(c["prefix"], device=DEV) % ps, torch.arange(m, device=DEV) % ps])
        k, v = (grid[s[x + "_pages"][pages, :, at].long()] * torch.exp2(s[x + "_exps"][pages, :, at].double() - 127)[..., None] for x in "kv")
        for head in range(h):
            x = s["q"][cu[r]:cu[r + 1], head].double() @ k[:, head // group].T * d ** -0.5
            out[cu[r]:cu[r + 1], head], lse[head, cu[r]:cu[r + 1]] = _exact_softmax(x, seen, v[:, head // group])
    return [out, lse]
