"""Measured cases of the paged 8-bit KV cache: page tables from request lengths,
writes of new rows as 8-bit codes, attention of ragged queries over the pages.

Each case is one pass through one operator.  ``run`` computes it in plain torch
operations, or, where ``own`` is set, by the library's entry points.  Pages hold
64 tokens; every page has one scale per KV head for K and one for V.
"""

import math
import random

import torch

own = False

PAGE = 64
DIM = 128


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _plan(name, batch, width, grow, ending, spread):
    return {"name": name, "op": "plan", "batch": batch, "width": width, "grow": grow, "ending": ending,
            "spread": spread}


def _append(name, batch, kv_heads, have, grow, code, dtype, fused, spread):
    return {"name": name, "op": "append", "batch": batch, "kv_heads": kv_heads, "have": have, "grow": grow,
            "code": code, "dtype": dtype, "fused": fused, "spread": spread}


def _attend(name, batch, kv_heads, group, grow, least, most, code, dtype="bf16", fused=False, cap=0.0,
            slopes=False, window=0, prefix=0, spread=1):
    return {"name": name, "op": "attend", "batch": batch, "kv_heads": kv_heads, "group": group, "grow": grow,
            "least": least, "most": most, "code": code, "dtype": dtype, "fused": fused, "cap": cap,
            "slopes": slopes, "window": window, "prefix": prefix, "spread": spread}


def listed():
    return [
        # one serving step of a running batch: a token each, a few requests end
        _plan("plan-decode-b64", 64, 512, 1, 3, 1),
        # a step that admits many prompts at once, beside ending requests
        _plan("plan-prompts-b1500", 1500, 96, 40, 100, 2),
        # the new token of each of 64 running requests, as slices of a fused projection
        _append("append-decode-b64", 64, 8, 3000, 1, "int8", "bf16", True, 3),
        # a long prompt filled at once
        _append("append-prompt-16k", 1, 8, 0, 16384, "e4m3", "bf16", False, 4),
        # ragged prompts of an fp32 model on top of partly filled pages
        _append("append-ragged-f32", 13, 5, 333, 777, "int8", "f32", False, 5),
        # one request, short context: the smallest decode step
        _attend("decode-b1-1k", 1, 8, 4, 1, 1000, 1000, "int8"),
        # the decode step of the benchmark's shape: 8 sequences, 32K tokens each
        _attend("decode-b8-32k", 8, 8, 4, 1, 32768, 32768, "int8"),
        # a ragged serving batch, capped scores, queries as slices of a fused projection
        _attend("decode-ragged-b96-cap", 96, 8, 8, 1, 1, 16000, "e4m3", fused=True, cap=30.0, spread=6),
        # a few draft tokens to verify in each request, fp32, distance bias
        _attend("verify-f32-b6-slopes", 6, 2, 3, 5, 500, 9000, "int8", dtype="f32", slopes=True, spread=7),
        # one whole prompt
        _attend("prompt-8k", 1, 8, 4, 8192, 8192, 8192, "e4m3"),
        # chunks of four prompts on top of what is cached already, ragged
        _attend("chunk-512-b4", 4, 8, 4, 512, 5000, 24000, "int8", spread=8),
        # prompts with a freely visible prefix and a sliding window
        _attend("prompt-window-prefix-b3", 3, 4, 7, 3000, 2500, 6000, "int8", window=1024, prefix=300, spread=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "append", "attend", "attend", "attend"))
    spread = rng.randrange(1 << 20)
    code = rng.choice(("int8", "e4m3"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op == "plan":
        c = _plan("", _log(rng, 1, 2048), _log(rng, 16, 512), _log(rng, 1, 60), 0, spread)
        c["ending"] = rng.randrange(0, c["batch"] // 4 + 1)
    elif op == "append":
        grow = _log(rng, 1, 8000)
        batch = max(1, min(_log(rng, 1, 128), 16000 // grow))
        c = _append("", batch, rng.randint(1, 8), rng.choice((0, _log(rng, 1, 1000))), grow, code, dtype,
                    rng.random() < 0.5, spread)
    else:
        kv_heads, group = rng.randint(1, 8), rng.randint(1, 8)
        kind = rng.choice(("decode", "decode", "few", "prompt"))
        if kind == "decode":
            grow, most = 1, _log(rng, 1, 40000)
            batch = max(1, min(_log(rng, 1, 100), 250000 // most))
        elif kind == "few":
            grow, most = rng.randint(2, 24), _log(rng, 30, 16000)
            batch = max(1, min(_log(rng, 1, 32), 100000 // most))
        else:
            dtype = "bf16"
            grow, most = _log(rng, 32, 4096), _log(rng, 4096, 8192)
            batch = max(1, min(rng.randint(1, 4), 4096 // grow))
            kv_heads = min(kv_heads, 40 // group)
        least = rng.randint(max(1, most // 8), most)
        c = _attend("", batch, kv_heads, group, grow, least, most, code, dtype, rng.random() < 0.3,
                    rng.choice((0.0, 0.0, 20.0, 50.0)), rng.random() < 0.3, rng.choice((0, 0, 0, 100, 1024)),
                    rng.choice((0, 0, 0, 77, 300)), spread)
    del c["name"]
    return c


def _plan_lengths(case):
    """(tokens held, tokens to come or -1) of every request."""
    r = random.Random(case["spread"])
    n, full = case["batch"], case["width"] * PAGE
    new = [1 if case["grow"] == 1 else r.randint(0, case["grow"]) for _ in range(n)]
    held = [r.randint(0, full - max(1, k)) for k in new]
    for b in r.sample(range(n), case["ending"]):
        new[b] = -1
    return held, new


def _append_lengths(case):
    r = random.Random(case["spread"])
    n, grow, have = case["batch"], case["grow"], case["have"]
    if n == 1 or grow == 1:
        new = [grow] * n
    else:
        new = [r.randint(1, grow) for _ in range(n)]
    held = [have if n == 1 else r.randint(0, have) for _ in range(n)]
    return held, new


def _attend_lengths(case):
    """(tokens held with the new ones, new tokens, free prefix) of every request."""
    r = random.Random(case["spread"])
    n, grow = case["batch"], case["grow"]
    ends = [case["most"]] + [r.randint(case["least"], case["most"]) for _ in range(n - 1)]
    new = [min(e, grow) if k == 0 or grow == 1 else r.randint(1, min(e, grow)) for k, e in enumerate(ends)]
    prefix = [min(e, r.randint(0, case["prefix"])) for e in ends]
    return ends, new, prefix


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def work(case):
    if case["op"] == "plan":
        held, new = _plan_lengths(case)
        n = case["batch"]
        tokens = sum(k for k in new if k > 0)
        moved = sum(_pages(h) if k < 0 else _pages(h + k) - _pages(h) for h, k in zip(held, new))
        return {"bytes": 4 * (2 * n + n + n + 1 + tokens + 2 * moved), "flops": 0}
    if case["op"] == "append":
        held, new = _append_lengths(case)
        rows = sum(new) * case["kv_heads"] * DIM * 2
        touched = sum(_pages(h + k) - h // PAGE for h, k in zip(held, new))
        return {"bytes": rows * ((2 if case["dtype"] == "bf16" else 4) + 1) + 4 * sum(new)
                + touched * case["kv_heads"] * 2 * 4, "flops": 0}
    ends, new, prefix = _attend_lengths(case)
    w, pairs, keys = case["window"], 0, 0
    for e, k, f in zip(ends, new, prefix):
        first = e - k
        for p in (range(first, e) if w or f else ()):
            lo = max(0, p - w + 1) if w else 0
            pairs += p + 1 - lo + max(0, f - (p + 1)) + min(f, lo)
        if not (w or f):
            pairs += k * first + k * (k + 1) // 2
        lo = max(0, first - w + 1) if w else 0
        keys += e - lo + min(f, lo)
    heads = case["kv_heads"] * case["group"]
    size = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": keys * case["kv_heads"] * 2 * (DIM + 4.0 / PAGE) + 2 * sum(new) * heads * DIM * size,
            "flops": 4.0 * DIM * heads * pairs}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(counts, width, pages, gen):
    """Pages of every request in the order of a running server's pool: scattered."""
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    count = _ints(counts)[:, None]
    start = torch.cumsum(count, 0) - count
    col = torch.arange(width, device="cuda", dtype=torch.int32)[None]
    place = (start + col).clamp(max=pages - 1).long()
    used = sum(counts)
    return torch.where(col < count, order[place], -1).contiguous(), order[used:].contiguous()


def _rows(shape, gen, outliers):
    """Rows as a model's projections give them; keys with a few strong channels."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if outliers:
        x[..., 5::32] *= 10.0
    return x


def _coded(x, code):
    """Pages [.., 64, 128] as codes and scales, the scale covering the page's largest value."""
    top = x.abs().amax((-1, -2))
    if code == "int8":
        s = top / 127.0
        return torch.round(x / s[..., None, None]).to(torch.int8), s
    s = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
    return (x / s[..., None, None]).to(torch.float8_e4m3fn), s


def _slices(n, heads, kv_heads, dtype, fused, gen):
    """q, k, v [n, heads, 128]; slices of one projection's result where `fused`."""
    x = _rows((n, heads + 2 * kv_heads, DIM), gen, False)
    x[:, heads:heads + kv_heads, 5::32] *= 10.0
    x = x.to(_TYPES[dtype])
    q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"op": case["op"], "case": case}
    if case["op"] == "plan":
        held, new = _plan_lengths(case)
        counts = [_pages(h) for h in held]
        need = sum(_pages(h + max(k, 0)) for h, k in zip(held, new))
        pages = need + 7
        table, free = _table(counts, case["width"], pages, gen)
        stack = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        stack[:free.numel()] = free
        s.update(lens=_ints(held), new=_ints(new), table=table, free=stack, n_free=_ints([free.numel()]),
                 pages=pages, tokens=sum(k for k in new if k > 0) + 5)
        if own:
            import online_rank_kv_b200 as ik
            s["out"] = ik.PagePlan.empty(case["batch"], s["tokens"], device="cuda")
    elif case["op"] == "append":
        held, new = _append_lengths(case)
        counts = [_pages(h + k) for h, k in zip(held, new)]
        pages = sum(counts) + 3
        table, _ = _table(counts, max(counts), pages, gen)
        k, v, ks, vs = _store(pages, case["kv_heads"], case["code"], gen)
        _, kn, vn = _slices(sum(new), case["kv_heads"], case["kv_heads"], case["dtype"], case["fused"], gen)
        who = torch.repeat_interleave(torch.arange(len(new), device="cuda"), _ints(new))
        cu = torch.cumsum(_ints(new), 0) - _ints(new)
        at = torch.arange(sum(new), device="cuda") - cu[who] + _ints(held)[who]
        slots = table[who, at // PAGE] * PAGE + (at % PAGE).to(torch.int32)
        s.update(k=k, v=v, ks=ks * 0.5, vs=vs * 0.5, kn=kn, vn=vn, slots=slots.to(torch.int32).contiguous())
    else:
        ends, new, prefix = _attend_lengths(case)
        counts = [_pages(e) for e in ends]
        pages = sum(counts) + 3
        table, _ = _table(counts, max(counts), pages, gen)
        k, v, ks, vs = _store(pages, case["kv_heads"], case["code"], gen)
        heads = case["kv_heads"] * case["group"]
        q, _, _ = _slices(sum(new), heads, case["kv_heads"], case["dtype"], case["fused"], gen)
        cu = _ints([0] + new).cumsum(0).to(torch.int32)
        slopes = torch.exp2(-8.0 * torch.arange(1, heads + 1, device="cuda") / heads) if case["slopes"] else None
        s.update(k=k, v=v, ks=ks, vs=vs, q=q, table=table, lens=_ints(ends), cu=cu, slopes=slopes,
                 prefix=_ints(prefix) if case["prefix"] else None, most=max(new))
    if own and case["op"] != "plan":
        import online_rank_kv_b200 as ik
        s["store"] = ik.Q8Pages.of(s["k"], s["v"], s["ks"], s["vs"])
    return s


def _store(pages, kv_heads, code, gen):
    k, ks = _coded(_rows((pages, kv_heads, PAGE, DIM), gen, True), code)
    v, vs = _coded(_rows((pages, kv_heads, PAGE, DIM), gen, False), code)
    return k, v, ks, vs


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["op"]
    if own:
        import online_rank_kv_b200 as ik
        if op == "plan":
            p = ik.page_plan(state["lens"], state["new"], state["table"], state["free"], state["n_free"],
                             out=state["out"])
            return {"table": state["table"], "free": state["free"], "n_free": p.n_free, "lens": p.lens,
                    "cu": p.cu, "slots": p.slots, "status": p.status}
        if op == "append":
            state["store"].append(state["kn"], state["vn"], state["slots"])
            return {"k": state["k"], "v": state["v"], "ks": state["ks"], "vs": state["vs"]}
        c = state["case"]
        return state["store"].attention(state["q"], state["table"], state["lens"], state["cu"],
                                        max_new=state["most"], cap=c["cap"], slopes=state["slopes"],
                                        window=c["window"], prefix=state["prefix"])
    if op == "plan":
        return _plain_plan(state)
    if op == "append":
        return _plain_append(state)
    return _plain_attend(state)


def _plain_plan(s):
    lens, new, table, free, n_free = s["lens"].long(), s["new"].long(), s["table"], s["free"], s["n_free"].long()
    width, pages = table.shape[1], s["pages"]
    col = torch.arange(width, device="cuda")[None]
    ended = new < 0
    grow = new.clamp(min=0)
    had = (lens + PAGE - 1) // PAGE
    has = torch.where(ended, had, (lens + grow + PAGE - 1) // PAGE)
    # pages of ended requests on top of the stack, in request order
    back = torch.where(ended, had, 0)
    put = n_free + (torch.cumsum(back, 0) - back)[:, None] + col
    away = torch.full_like(put, pages)
    stack = torch.cat([free, free[:1]])
    stack[torch.where(ended[:, None] & (col < had[:, None]), put, away)] = table
    free.copy_(stack[:pages])
    top = n_free + back.sum()
    # new blocks take pages from the top
    need = torch.where(ended, 0, has - had)
    take = top - 1 - ((torch.cumsum(need, 0) - need)[:, None] + col - had[:, None])
    fresh = (col >= had[:, None]) & (col < has[:, None]) & ~ended[:, None]
    table.copy_(torch.where(fresh, free[take.clamp(0, pages - 1)], table))
    cu = torch.cumsum(torch.cat([grow.new_zeros(1), grow]), 0)
    at = torch.arange(s["tokens"], device="cuda")
    who = torch.searchsorted(cu, at, right=True) - 1
    live = at < cu[-1]
    who = who.clamp(max=lens.numel() - 1)
    pos = torch.where(live, lens[who] + at - cu[who], 0)
    slots = torch.where(live, table[who, pos // PAGE].long() * PAGE + pos % PAGE, -1)
    return {"table": table, "free": free, "n_free": (top - need.sum()).to(torch.int32),
            "lens": torch.where(ended, 0, lens + grow).to(torch.int32), "cu": cu.to(torch.int32),
            "slots": slots.to(torch.int32), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _plain_write(store, scale, rows, slots):
    """rows [n, heads, 128] into the pages of their slots."""
    page, at = slots.long() // PAGE, slots.long() % PAGE
    touched, which = torch.unique(page, return_inverse=True)
    heads = rows.shape[1]
    x = rows.float()
    x = torch.where(torch.isfinite(x), x, 0.0)
    top = x.new_zeros(touched.numel(), heads).index_reduce(0, which, x.abs().amax(2), "amax")
    first = torch.full_like(touched, PAGE).index_reduce(0, which, at, "amin")
    before = torch.where(first[:, None] == 0, 0.0, scale[touched])
    top = torch.where(top < 2.0 ** -64, 0.0, top)
    if store.dtype == torch.int8:
        now = torch.maximum(before, top / 127.0)
    else:
        m, e = torch.frexp(top)
        e = e - 9 + (m > 0.875)
        now = torch.maximum(before, torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), 0.0))
    by = torch.where(now > 0, now, 1.0)
    bits = store.view(torch.int8)
    held = bits[touched]
    old = held.view(store.dtype).float() * (before / by)[:, :, None, None]
    code = x / by[which][:, :, None]
    if store.dtype == torch.int8:
        old, code = torch.round(old), torch.round(code).clamp(-127, 127)
    keep = torch.arange(PAGE, device="cuda")[None] < first[:, None]
    bits[touched] = torch.where(keep[:, None, :, None], old.to(store.dtype).view(torch.int8), held)
    bits[page, :, at] = torch.where((now > 0)[which][:, :, None], code.to(store.dtype).view(torch.int8), 0)
    scale[touched] = now


def _plain_append(s):
    _plain_write(s["k"], s["ks"], s["kn"], s["slots"])
    _plain_write(s["v"], s["vs"], s["vn"], s["slots"])
    return {"k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"]}


def _plain_values(store, scale, table):
    x = store.view(torch.int8)[table.long()].view(store.dtype).float() * scale[table.long()][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attend(s):
    c, q, cu, lens = s["case"], s["q"], s["cu"].long(), s["lens"].long()
    batch, hkv, g, most = c["batch"], c["kv_heads"], c["group"], s["most"]
    k, v = _plain_values(s["k"], s["ks"], s["table"]), _plain_values(s["v"], s["vs"], s["table"])
    step = torch.arange(most, device="cuda")[None]
    count = (cu[1:] - cu[:-1])[:, None]
    at = (cu[:-1, None] + step).clamp(max=q.shape[0] - 1)
    x = q[at].float().view(batch, most, hkv, g, DIM).permute(0, 2, 1, 3, 4).reshape(batch, hkv, most * g, DIM)
    score = torch.matmul(x, k.transpose(2, 3)).mul_(1.0 / math.sqrt(DIM)).view(batch, hkv, most, g, -1)
    if c["cap"]:
        score = score.div_(c["cap"]).tanh_().mul_(c["cap"])
    p = (lens[:, None] - count + step)[:, :, None]
    j = torch.arange(score.shape[-1], device="cuda")[None, None]
    if s["slopes"] is not None:
        score = score - s["slopes"].view(1, hkv, 1, g, 1) * (p - j).abs().float()[:, None, :, None]
    seen = j <= p
    if c["window"]:
        seen = seen & (j > p - c["window"])
    if s["prefix"] is not None:
        seen = seen | (j < s["prefix"][:, None, None])
    seen = (seen & (j < lens[:, None, None]))[:, None, :, None]
    score = score.masked_fill_(~seen, float("-inf"))
    w = score.sub_(score.amax(-1, keepdim=True)).exp_()
    w = w.div_(w.sum(-1, keepdim=True)).view(batch, hkv, most * g, -1)
    o = torch.matmul(w, v).view(batch, hkv, most, g, DIM).permute(0, 2, 1, 3, 4)
    return o.reshape(batch, most, hkv * g, DIM)[step.expand(batch, -1) < count].to(q.dtype)


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None
    if case["op"] == "append":
        k, ks = _exact_write(s["k"], s["ks"], s["kn"], s["slots"])
        v, vs = _exact_write(s["v"], s["vs"], s["vn"], s["slots"])
        return {"k": k, "v": v, "ks": ks, "vs": vs}
    return _exact_attend(case, s)


def _exact_write(store, scale, rows, slots):
    e4m3 = store.dtype != torch.int8
    code, scale, rows = store.to(torch.float64), scale.double(), rows.double()
    slot = slots.tolist()
    runs, i = [], 0
    while i < len(slot):
        n = 1
        while i + n < len(slot) and slot[i + n] == slot[i] + n and slot[i + n] % PAGE:
            n += 1
        runs.append((i, n))
        i += n

    def rounded(x):
        if not e4m3:
            return x.round()
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        return (x / step).round() * step

    for i, n in runs:
        page, at = divmod(slot[i], PAGE)
        x = rows[i:i + n].transpose(0, 1)
        top = x.abs().amax((1, 2))
        if e4m3:
            s = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
        else:
            s = top / 127.0
        if at:
            old = scale[page].clone()
            s = torch.maximum(s, old)
            code[page, :, :at] = rounded(code[page, :, :at] * (old / s)[:, None, None])
        code[page, :, at:at + n] = rounded(x / s[:, None, None])
        scale[page] = s
    # whole-numbered codes hang on the last bit of a 32-bit quotient: no 64-bit value
    return (code if e4m3 else None), scale


def _exact_attend(case, s):
    g, hkv = case["group"], case["kv_heads"]
    ends, new, prefix = _attend_lengths(case)
    if sum(e * n for e, n in zip(ends, new)) * g * hkv > 4e9:
        return None
    q, out, at = s["q"].double(), [], 0
    for b, (e, n, f) in enumerate(zip(ends, new, prefix)):
        pg = s["table"][b, :_pages(e)].long()
        pos = torch.arange(e - n, e, device="cuda")[:, None]
        key = torch.arange(e, device="cuda")[None]
        hide = key > pos
        if case["window"]:
            hide = hide | (pos - key >= case["window"])
        if case["prefix"]:
            hide = hide & (key >= f)
        dist = (pos - key).abs().double()
        res = torch.empty(n, hkv * g, DIM, dtype=torch.float64, device="cuda")
        for h in range(hkv):
            kk = (s["k"].view(torch.int8)[pg, h].view(s["k"].dtype).double() * s["ks"][pg, h].double()[:, None, None]).reshape(-1, DIM)[:e]
            vv = (s["v"].view(torch.int8)[pg, h].view(s["v"].dtype).double() * s["vs"][pg, h].double()[:, None, None]).reshape(-1, DIM)[:e]
            for a in range(h * g, h * g + g):
                z = q[at:at + n, a] @ kk.T / math.sqrt(DIM)
                if case["cap"]:
                    z = torch.tanh(z / case["cap"]) * case["cap"]
                if s["slopes"] is not None:
                    z = z - dist * s["slopes"][a].double()
                z[hide] = -math.inf
                res[:, a] = torch.softmax(z, 1) @ vv
        out.append(res)
        at += n
    return torch.cat(out)
