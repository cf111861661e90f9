"""What the cache-side operators compute, and the sizes they are measured at.

Three operators follow the token selection: rotary positions with several axes
on Q and K (`tsel_rope`), the quantised paged cache the kept tokens are written
to and read back from (`tsel_cache_write`, `tsel_cache_read`), and attention of
a batch of requests over a prefix that all of them share plus each one's own
suffix (`tsel_prefix_attention`).

`run` computes a case with plain torch operations in 32 bits (angles in 64)
where `own` is false, and with the library's calls where it is true. `exact`
gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3_MAX = 448.0
THETA = 1.0e6


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # the new tokens of 64 requests in one decoding step: latency counts
        dict(name="rope_step", op="rope", tokens=64, heads=16, kv_heads=8, dim=128, sections="24,20,20",
             layout="interleaved", type="bf16", adjacent=False, inverse=False),
        # Q and K of the vision encoder for the 30-image request, rotated by row and column
        dict(name="rope_thirty_images", op="rope", tokens=61385, heads=16, kv_heads=16, dim=80, sections="0,20,20",
             layout="per_axis", type="bf16", adjacent=False, inverse=False),
        # the gradients of Q and K in a training step: rotated back, in 32 bits
        dict(name="rope_gradient", op="rope", tokens=16384, heads=16, kv_heads=8, dim=128, sections="16,24,24",
             layout="sectioned", type="fp32", adjacent=True, inverse=True),
        # one decoding step of 200 requests: K and V of each new token, short pages
        dict(name="write_step", op="write", tokens=200, kv_heads=16, dim=80, page=16, pages=256, type="fp16"),
        # the kept tokens of the 30-image request after prefill (60% of 61,385)
        dict(name="write_thirty_images", op="write", tokens=36831, kv_heads=8, dim=128, page=64, pages=640, type="bf16"),
        # K rotated as it is written, then the rows read back for scoring: eight requests of 16 images
        dict(name="write_read_batch", op="write_read", tokens=131072, kv_heads=8, dim=128, page=128, pages=1100,
             sections="24,20,20", layout="interleaved", type="bf16"),
        # a text query's own keys read back
        dict(name="read_query", op="read", tokens=142, kv_heads=8, dim=128, page=16, pages=64, type="bf16"),
        # a pruned request read back to be scored again against another question
        dict(name="read_thirty_images", op="read", tokens=36831, kv_heads=8, dim=128, page=64, pages=640, type="bf16"),
        # four users of one six-view request: few rows, the prefix split over the device
        dict(name="attend_six_views", op="attend", requests=4, rows=1, prefix=1228, suffix=142, heads=16, kv_heads=8,
             dim=128, page=16, type="bf16"),
        # one decoding step of 64 users of the pruned 30-image request, answers of up to 1,000 tokens
        dict(name="attend_step", op="attend", requests=64, rows=1, prefix=36831, suffix=1000, heads=32, kv_heads=8,
             dim=128, page=64, type="bf16"),
        # the questions of 16 users (up to 142 tokens) prefilled over the same images
        dict(name="attend_questions", op="attend", requests=16, rows=142, prefix=36831, suffix=142, heads=16, kv_heads=8,
             dim=128, page=64, type="bf16"),
        # many heads of 80, one query head per cached head, drafted tokens, ragged lengths
        dict(name="attend_drafts", op="attend", requests=37, rows=5, prefix=9229, suffix=777, heads=16, kv_heads=16,
             dim=80, page=32, type="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _near_equal(n, parts):
    return [n // parts + (1 if a < n % parts else 0) for a in range(parts)]


def draw(rng):
    op = rng.choice(["rope", "write", "write_read", "read", "attend", "attend"])
    if op == "rope":
        dim = rng.choice([64, 72, 80, 96, 112, 128])
        pairs = rng.choice([dim // 2, dim // 2, dim // 4])
        sec = ",".join(map(str, _near_equal(pairs, rng.choice([1, 2, 3, 4]))))
        kv = rng.choice([1, 2, 4, 8])
        kind = rng.choice(["bf16", "fp16", "fp32"])
        heads = kv * rng.choice([1, 2, 4])
        return dict(op=op, tokens=min(_log(rng, 1, 65536), 314_000_000 // ((heads + kv) * dim * BYTES[kind])), heads=heads,
                    kv_heads=kv, dim=dim, sections=sec, layout=rng.choice(["sectioned", "interleaved", "per_axis"]),
                    type=kind, adjacent=rng.random() < 0.3, inverse=rng.random() < 0.3)
    dim = rng.choice([64, 80, 96, 112, 128])
    page = rng.choice([16, 32, 64, 128])
    if op in ("write", "write_read", "read"):
        kv = rng.choice([1, 2, 4, 8])
        tokens = _log(rng, 1, 131072)
        c = dict(op=op, tokens=tokens, kv_heads=kv, dim=dim, page=page, pages=tokens // page + rng.randint(1, 60),
                 type=rng.choice(["bf16", "fp16"]))
        if op == "write_read":
            c.update(sections=",".join(map(str, _near_equal(dim // 2, 3))), layout=rng.choice(["sectioned", "interleaved"]))
        return c
    kv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, requests=_log(rng, 1, 100), rows=rng.choice([1, 1, 1, 2, 5, _log(rng, 1, 142)]), prefix=_log(rng, 1, 40000),
             suffix=_log(rng, 150, 1000), heads=kv * rng.choice([1, 2, 4, 5, 8]), kv_heads=kv, dim=dim, page=page,
             type=rng.choice(["bf16", "fp16"]))
    while work(c)["flops"] > 6.0e11:
        c["prefix"] = c["prefix"] // 2 + 1
        c["requests"] = c["requests"] // 2 + 1
    return c


def _rows(c):
    """Query rows of each request: `rows` at most, ragged."""
    return [1 + (7919 * i + 3) % c["rows"] if i else c["rows"] for i in range(c["requests"])]


def _lens(c):
    """Suffix keys of each request, its own query rows among them: `suffix` at most, ragged."""
    rows = _rows(c)
    return [min(c["suffix"], n + (104729 * i + 11) % max(1, c["suffix"] - n + 1)) if i else c["suffix"]
            for i, n in enumerate(rows)]


def work(c):
    d = c["dim"]
    if c["op"] == "rope":
        per = c["tokens"] * (c["heads"] + c["kv_heads"])
        axes = len(c["sections"].split(","))
        return {"bytes": 2 * per * d * BYTES[c["type"]] + 4 * c["tokens"] * axes, "flops": 3 * per * d}
    if c["op"] != "attend":
        rows = c["tokens"] * c["kv_heads"]
        wide, narrow = 2 * rows * d * BYTES[c["type"]], 2 * rows * (d + 1)
        n = 4 * c["tokens"]
        if c["op"] == "write_read":
            return {"bytes": 2 * (wide + narrow + n) + 12 * c["tokens"], "flops": 8 * rows * d}
        return {"bytes": wide + narrow + n, "flops": 4 * rows * d}
    rows, lens = _rows(c), _lens(c)
    keys = c["prefix"] + sum(lens)
    pairs = sum(rows) * c["prefix"] + sum(n * s - n * (n - 1) // 2 for n, s in zip(rows, lens))
    io = sum(rows) * c["heads"] * (2 * d * BYTES[c["type"]] + 4)
    return {"bytes": 2 * keys * c["kv_heads"] * (d + 1) + io, "flops": 4 * d * c["heads"] * pairs}


# ------------------------------------------------------------------- the inputs

def _frequencies(c):
    """(radians a position step, axis) of every rotated pair."""
    sec = [int(x) for x in c["sections"].split(",")]
    pairs, n = sum(sec), len(sec)
    axis, freq = [], []
    if c["layout"] == "interleaved":
        for i in range(pairs):
            axis.append(i % n if i // n < sec[i % n] else 0)
    else:
        for a, s in enumerate(sec):
            axis += [a] * s
    if c["layout"] == "per_axis":
        for s in sec:
            freq += [THETA ** (-j / s) for j in range(s)]
    else:
        freq = [THETA ** (-i / pairs) for i in range(pairs)]
    return freq, axis


def _positions(tokens, axes, g):
    """(image or time, row, column) positions of image tokens, 64 a row, at varying offsets."""
    t = torch.arange(tokens, device=DEV)
    cols = [t // 2048 + int(torch.randint(0, 5000, (1,), generator=g, device=DEV)), (t // 64) % 64, t % 64, t]
    return torch.stack(cols[:axes], 1).to(torch.int32).contiguous()


def _quantised(tokens, heads, dim, g):
    """Codes and scale exponents of rows of varying size."""
    x = torch.randn(tokens, heads, dim, generator=g, device=DEV)
    x *= torch.exp2(torch.randn(tokens, heads, 1, generator=g, device=DEV))
    return _plain_quantise(x)


def _fill(c, tokens, g):
    """A pool of pages with `tokens` cached tokens at random places; their slots."""
    hk, d, ps = c["kv_heads"], c["dim"], c["page"]
    pages = c.get("pages") or (c["prefix"] + ps - 1) // ps + c["requests"] * ((c["suffix"] + ps - 1) // ps) + 3
    pool = [torch.zeros(pages, hk, ps, d, dtype=torch.uint8, device=DEV) for _ in range(2)]
    exps = [torch.zeros(pages, hk, ps, dtype=torch.uint8, device=DEV) for _ in range(2)]
    order = torch.randperm(pages, generator=g, device=DEV)
    return pool, exps, order


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    dt = TYPES[c["type"]]
    if "sections" in c:
        freq, axis = _frequencies(c)
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device=DEV)
        s["axis"] = torch.tensor(axis, dtype=torch.int64, device=DEV)
        s["pos"] = _positions(c["tokens"], len(c["sections"].split(",")), g)
        if own:
            import attention_score_vision_gb300 as tsel
            s["table"] = tsel.tsel_rope_table(freq, axis, device=DEV)
    if c["op"] == "rope":
        s["q"] = torch.randn(c["tokens"], c["heads"], c["dim"], generator=g, device=DEV).to(dt)
        s["k"] = torch.randn(c["tokens"], c["kv_heads"], c["dim"], generator=g, device=DEV).to(dt)
    elif c["op"] != "attend":
        (s["k_pages"], s["v_pages"]), (s["k_exps"], s["v_exps"]), order = _fill(c, c["tokens"], g)
        at = torch.arange(c["tokens"], device=DEV)
        s["slots"] = (order[at // c["page"]] * c["page"] + at % c["page"]).to(torch.int32)
        if c["op"] == "read":
            for n in "kv":
                codes, exps = _quantised(c["tokens"], c["kv_heads"], c["dim"], g)
                _put(s[n + "_pages"], s[n + "_exps"], codes, exps, s["slots"].long(), c["page"])
        else:
            shape = (c["tokens"], c["kv_heads"], c["dim"])
            for n in "kv":
                x = torch.randn(*shape, generator=g, device=DEV)
                s[n] = (x * torch.exp2(torch.randn(shape[0], shape[1], 1, generator=g, device=DEV))).to(dt)
    else:
        rows, lens, ps = _rows(c), _lens(c), c["page"]
        total = c["prefix"] + sum(lens)
        (s["k_pages"], s["v_pages"]), (s["k_exps"], s["v_exps"]), order = _fill(c, total, g)
        np_, ns = (c["prefix"] + ps - 1) // ps, (c["suffix"] + ps - 1) // ps
        s["prefix_pages"] = order[:np_].to(torch.int32)
        s["page_table"] = order[np_:np_ + c["requests"] * ns].view(c["requests"], ns).to(torch.int32).contiguous()
        p = torch.arange(c["prefix"], device=DEV)
        slots = [order[:np_][p // ps] * ps + p % ps]
        length = torch.tensor(lens, device=DEV)
        j = torch.arange(ns * ps, device=DEV).expand(c["requests"], -1)
        inside = j < length[:, None]
        slots.append((s["page_table"].long().gather(1, j // ps) * ps + j % ps)[inside])
        slots = torch.cat(slots)
        for n in "kv":
            codes, exps = _quantised(total, c["kv_heads"], c["dim"], g)
            _put(s[n + "_pages"], s[n + "_exps"], codes, exps, slots, ps)
        s["q"] = torch.randn(sum(rows), c["heads"], c["dim"], generator=g, device=DEV).to(dt)
        s["cu"] = torch.tensor([0] + rows, device=DEV).cumsum(0).to(torch.int32)
        s["lens"] = length.to(torch.int32)
        s["prefix_len"] = torch.tensor([c["prefix"]], dtype=torch.int32, device=DEV)
    if own:
        import attention_score_vision_gb300 as tsel
        if "k_pages" in s:
            s["cache"] = tsel.TselCache(s["k_pages"], s["v_pages"], s["k_exps"], s["v_exps"])
        need = tsel.tsel_cache_workspace_size()
        if c["op"] == "attend":
            need = tsel.tsel_prefix_attention_workspace_size(c["requests"], sum(_rows(c)), c["rows"], c["heads"], c["kv_heads"],
                                                             c["dim"], c["prefix"], c["suffix"])
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    return s


def _put(pages, exps, codes, e, slots, ps):
    pages[slots // ps, :, slots % ps] = codes
    exps[slots // ps, :, slots % ps] = e


# ------------------------------------------------------------------- the plain forms

def _plain_rotate(x, pos, freq, axis, adjacent, inverse):
    """x [T, H, d] with its first 2 * len(freq) columns rotated by pos[axis] * freq."""
    angle = pos[:, axis].double() * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        sin = -sin
    n = freq.numel()
    y = x.float().clone()
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., first].float(), x[..., second].float()
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


def _plain_quantise(x):
    """E4M3 codes and the biased exponent of the power of two that scales them: the least with |x| <= 448 * 2^e."""
    f, e = torch.frexp(x.abs().amax(-1).float())
    e = torch.where(f <= 0.875, e - 9, e - 8)
    e = torch.where(f == 0, -127, e).clamp(-127, 127)
    codes = torch.ldexp(x.float(), -e[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _plain_dequantise(codes, exps):
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), (exps.int() - 127)[..., None])


def _plain_read(s, slots, ps):
    slots = slots.long()
    return [_plain_dequantise(s[n + "_pages"][slots // ps, :, slots % ps], s[n + "_exps"][slots // ps, :, slots % ps]) for n in "kv"]


def _plain_write(s, c):
    slots = s["slots"].long()
    k = s["k"]
    if c["op"] == "write_read":
        k = _plain_rotate(k, s["pos"], s["freq"], s["axis"], False, False)
    for n, x in (("k", k), ("v", s["v"])):
        _put(s[n + "_pages"], s[n + "_exps"], *_plain_quantise(x), slots, c["page"])


def _plain_attend(s, c):
    ps, hk, d = c["page"], c["kv_heads"], c["dim"]
    group = c["heads"] // hk
    tokens = s["q"].shape[0]
    p = torch.arange(c["prefix"], device=DEV)
    pk, pv = _plain_read(s, s["prefix_pages"][p // ps] * ps + p % ps, ps)
    j = torch.arange(c["suffix"], device=DEV).expand(c["requests"], -1)
    sk, sv = _plain_read(s, (s["page_table"].gather(1, j // ps) * ps + j % ps).reshape(-1), ps)
    sk, sv = (x.view(c["requests"], -1, hk, d).permute(0, 2, 1, 3) for x in (sk, sv))      # [R, Hkv, S, d]
    cu = s["cu"].long()
    t = torch.arange(tokens, device=DEV)
    req = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[req]
    n = cu[1:] - cu[:-1]
    q = s["q"].float().view(tokens, hk, group, d) / math.sqrt(d)
    # prefix scores [Hkv, T, group, P]; suffix scores of each request's padded rows, taken back to [Hkv, T, group, S]
    sp = torch.matmul(q.permute(1, 0, 2, 3).reshape(hk, tokens * group, d), pk.permute(1, 2, 0)).view(hk, tokens, group, -1)
    padded = q.new_zeros(c["requests"], c["rows"], hk, group, d)
    padded[req, i] = q
    qs = padded.permute(0, 2, 1, 3, 4).reshape(c["requests"], hk, c["rows"] * group, d)
    ss = torch.matmul(qs, sk.transpose(2, 3)).view(c["requests"], hk, c["rows"], group, -1)
    ss = ss.permute(0, 2, 1, 3, 4)[req, i].permute(1, 0, 2, 3)
    seen = torch.arange(c["suffix"], device=DEV) < (s["lens"].long()[req] - n[req] + i + 1)[:, None]
    ss = ss.masked_fill(~seen[None, :, None], -math.inf)
    top = torch.maximum(sp.amax(-1), ss.amax(-1))[..., None]
    sp, ss = torch.exp(sp - top), torch.exp(ss - top)
    total = sp.sum(-1) + ss.sum(-1)
    out = torch.matmul(sp.reshape(hk, tokens * group, -1), pv.permute(1, 0, 2)).view(hk, tokens, group, d)
    padded = ss.new_zeros(c["requests"], c["rows"], hk, group, ss.shape[-1])
    padded[req, i] = ss.permute(1, 0, 2, 3)
    ps_ = padded.permute(0, 2, 1, 3, 4).reshape(c["requests"], hk, c["rows"] * group, -1)
    os_ = torch.matmul(ps_, sv).view(c["requests"], hk, c["rows"], group, d).permute(0, 2, 1, 3, 4)[req, i]
    out = (out + os_.permute(1, 0, 2, 3)) / total[..., None]
    lse = top[..., 0] + total.log()
    return out.permute(1, 0, 2, 3).reshape(tokens, c["heads"], d).to(s["q"].dtype), lse.permute(0, 2, 1).reshape(c["heads"], tokens)


# ------------------------------------------------------------------- a pass

def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    dt = TYPES[c["type"]]
    if c["op"] == "rope":
        return [_plain_rotate(s[n], s["pos"], s["freq"], s["axis"], c["adjacent"], c["inverse"]).to(dt) for n in "qk"]
    if c["op"] == "read":
        return [x.to(dt) for x in _plain_read(s, s["slots"], c["page"])]
    if c["op"] == "attend":
        return _plain_attend(s, c)
    _plain_write(s, c)
    if c["op"] == "write_read":
        return [x.to(dt) for x in _plain_read(s, s["slots"], c["page"])]
    return _state(s)


def _state(s):
    return [s["k_pages"].view(torch.float8_e4m3fn), s["v_pages"].view(torch.float8_e4m3fn), s["k_exps"], s["v_exps"]]


def _run_own(s, c):
    import attention_score_vision_gb300 as tsel
    dt = TYPES[c["type"]]
    if c["op"] == "rope":
        flags = (tsel.TSEL_ROPE_ADJACENT if c["adjacent"] else 0) | (tsel.TSEL_ROPE_INVERSE if c["inverse"] else 0)
        return tsel.tsel_rope(s["q"], s["k"], s["pos"], s["table"], flags=flags, workspace=s["ws"])
    if c["op"] == "read":
        return tsel.tsel_cache_read(s["cache"], s["slots"], dtype=dt, workspace=s["ws"])
    if c["op"] == "attend":
        return tsel.tsel_prefix_attention(s["q"], s["cu"], c["rows"], s["cache"], s["prefix_pages"], s["prefix_len"], c["prefix"],
                                          s["page_table"], s["lens"], c["suffix"], workspace=s["ws"])
    if c["op"] == "write_read":
        tsel.tsel_cache_write(s["k"], s["v"], s["slots"], s["cache"], pos=s["pos"], table=s["table"], workspace=s["ws"])
        return tsel.tsel_cache_read(s["cache"], s["slots"], dtype=dt, workspace=s["ws"])
    tsel.tsel_cache_write(s["k"], s["v"], s["slots"], s["cache"], workspace=s["ws"])
    return _state(s)


# ------------------------------------------------------------------- in 64 bits, from the definitions

def _exact_round(x):
    """x on E4M3's grid scaled by a power of two for each row: (values on the grid, exponents)."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / E4M3_MAX).clamp(min=-200))
    e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e)
    e = torch.where(top <= E4M3_MAX * torch.exp2(e - 1), e - 1, e).clamp(-127, 127)
    y = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, e


def _exact_turn(x, s, c, sign):
    """Rotation as a product of complex numbers."""
    n = s["freq"].numel()
    x = x.double()
    z = torch.complex(x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if c.get("adjacent") else torch.complex(x[..., :n], x[..., n:2 * n])
    w = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), sign * s["freq"] * s["pos"].double()[:, s["axis"]])
    z = z * w[:, None]
    rest = x[..., 2 * n:]
    turned = torch.view_as_real(z).flatten(-2) if c.get("adjacent") else torch.cat([z.real, z.imag], -1)
    return torch.cat([turned, rest], -1)


def _grid(codes):
    """The values of E4M3 codes, from their bits."""
    v = torch.arange(256, device=DEV)
    m, e = v % 8, (v // 8) % 16
    values = torch.where(e == 0, m * 2.0 ** -9, (8 + m).double() * torch.exp2((e - 10).double()))
    return torch.where(v < 128, values, -values).double()[codes.long()]


def _rows_of(pages, exps, page, offset):
    return _grid(pages[page, :, offset]) * torch.exp2(exps[page, :, offset].double() - 127)[..., None]


def exact(c, seed):
    s = prepare(c, seed)
    ps = c.get("page")
    if c["op"] == "rope":
        return [_exact_turn(s[n], s, c, -1 if c["inverse"] else 1) for n in "qk"]
    if c["op"] == "read":
        at = s["slots"].long()
        return [_rows_of(s[n + "_pages"], s[n + "_exps"], at.div(ps, rounding_mode="floor"), at.remainder(ps)) for n in "kv"]
    if c["op"] == "write_read":
        return [torch.ldexp(*_exact_round(x)) for x in (_exact_turn(s["k"], s, c, 1), s["v"].double())]
    if c["op"] == "write":
        out = []
        at = s["slots"].long()
        for n in "kv":
            whole = torch.zeros(s[n + "_pages"].shape, dtype=torch.float64, device=DEV)
            whole[at.div(ps, rounding_mode="floor"), :, at.remainder(ps)] = _exact_round(s[n].double())[0]
            out.append(whole)
        return out + [None, None]
    # attention: request by request, head by head, over all of its keys at once
    cu, lens, group = s["cu"].tolist(), s["lens"].tolist(), c["heads"] // c["kv_heads"]
    p = torch.arange(c["prefix"], device=DEV)
    pk, pv = (_rows_of(s[n + "_pages"], s[n + "_exps"], s["prefix_pages"].long()[p // ps], p % ps) for n in "kv")
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(c["heads"], s["q"].shape[0], dtype=torch.float64, device=DEV)
    for r in range(c["requests"]):
        j = torch.arange(lens[r], device=DEV)
        at = s["page_table"][r].long()[j // ps]
        k, v = (torch.cat([x, _rows_of(s[n + "_pages"], s[n + "_exps"], at, j % ps)]) for n, x in (("k", pk), ("v", pv)))
        n = cu[r + 1] - cu[r]
        hidden = j[None] > lens[r] - n + torch.arange(n, device=DEV)[:, None]
        for h in range(c["heads"]):
            z = s["q"][cu[r]:cu[r + 1], h].double() @ k[:, h // group].T / math.sqrt(c["dim"])
            z[:, c["prefix"]:][hidden] = -math.inf
            lse[h, cu[r]:cu[r + 1]] = torch.logsumexp(z, -1)
            out[cu[r]:cu[r + 1], h] = torch.softmax(z, -1) @ v[:, h // group]
    return [out, lse]
