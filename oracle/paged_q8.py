"""CPU reference of the paged 8-bit cache: page tables, coded writes, ragged
attention.  Plain loops over requests and runs; attention in float64.  Codes
and scales are decided in float32, as the format states them."""

import numpy as np

PAGE = 64
INVALID_ARG, CAPACITY, RANGE = -1, -2, -9
INT8, E4M3 = 0, 1


def _blocks(n):
    return -(-n // PAGE)


def page_plan(lens, add, table, free, n_free, tokens):
    """(lens, cu, slots, n_free, status) after one step; table and free are
    updated in place unless the step is refused."""
    lens, add = [int(x) for x in lens], [int(x) for x in add]
    n_free, pages, width = int(n_free), len(free), table.shape[1]

    def refuse(code):
        return lens, [0] * (len(lens) + 1), [-1] * tokens, n_free, code

    if not 0 <= n_free <= pages or any(not 0 <= x <= width * PAGE for x in lens) or any(a < -1 for a in add):
        return refuse(INVALID_ARG)
    back = [(b, j) for b, a in enumerate(add) if a < 0 for j in range(_blocks(lens[b]))]
    if n_free + len(back) > pages:
        return refuse(INVALID_ARG)
    need = [(b, j) for b, a in enumerate(add) if a > 0 for j in range(_blocks(lens[b]), _blocks(lens[b] + a))]
    if (any(a > 0 and lens[b] + a > width * PAGE for b, a in enumerate(add)) or
            sum(max(a, 0) for a in add) > tokens or len(need) > n_free + len(back)):
        return refuse(CAPACITY)
    for i, (b, j) in enumerate(back):
        free[n_free + i] = table[b, j]
    top = n_free + len(back)
    for i, (b, j) in enumerate(need):
        table[b, j] = free[top - 1 - i]
    cu, slots = [0], []
    for b, a in enumerate(add):
        for t in range(lens[b], lens[b] + max(a, 0)):
            page = int(table[b, t // PAGE])
            slots.append(page * PAGE + t % PAGE if 0 <= page < pages else -1)
        cu.append(len(slots))
    slots += [-1] * (tokens - len(slots))
    return [0 if a < 0 else n + a for n, a in zip(lens, add)], cu, slots, top - len(need), 0


def e4m3_values():
    """The 256 e4m3 values by code (float64; NaN at 0x7f and 0xff)."""
    out = []
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out.append(np.nan if e == 15 and m == 7 else (-v if s else v))
    return np.array(out)


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]


def e4m3_encode(x):
    """Codes of x (|x| <= 448), rounded half to even."""
    a = np.abs(x).astype(np.float64)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def decode(codes, code):
    """Code values as float64; `codes` int8 (INT8) or uint8 (E4M3)."""
    return codes.astype(np.float64) if code == INT8 else _VALUES[codes]


def _scale_of(top, code):
    top = np.float32(top)
    if not top >= np.float32(2.0 ** -64):
        return np.float32(0)
    if code == INT8:
        return np.float32(top * (np.float32(1) / np.float32(127)))
    e = int(np.floor(np.log2(float(top)))) - 9
    while float(top) > 448 * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def _encode(x, code):
    return np.clip(np.rint(x), -127, 127).astype(np.int8) if code == INT8 else e4m3_encode(x)


def append(codes, scale, rows, slots, code):
    """rows [n, heads, 128] float32 into codes [pages, heads, 64, 128] and
    scale [pages, heads], in place; returns the status."""
    status, i, n = 0, 0, len(slots)
    while i < n:
        s = int(slots[i])
        if not 0 <= s < codes.shape[0] * PAGE:
            if s != -1:
                status = min(status, INVALID_ARG)
            i += 1
            continue
        m = 1
        while i + m < n and slots[i + m] == s + m and (s + m) % PAGE:
            m += 1
        page, at = divmod(s, PAGE)
        for h in range(codes.shape[1]):
            x = rows[i:i + m, h].astype(np.float32)
            if not np.isfinite(x).all():
                status = min(status, RANGE)
                x = np.where(np.isfinite(x), x, np.float32(0))
            old = scale[page, h] if at else np.float32(0)
            now = max(old, _scale_of(np.abs(x).max(), code))
            if at and now > old:
                f = np.float32(old) / np.float32(now)
                codes[page, h, :at] = _encode(decode(codes[page, h, :at], code).astype(np.float32) * f, code)
            codes[page, h, at:at + m] = _encode(x / now, code) if now > 0 else 0
            scale[page, h] = now
        i += m
    return status


def visible(length, n, window, prefix):
    """[n, length] truth values: what the last n queries of a request see."""
    p = np.arange(length - n, length)[:, None]
    t = np.arange(length)[None]
    on = t <= p
    if window > 0:
        on &= t > p - window
    return on | (t < prefix)


def attention(q, k, v, scale, cap=0.0, slopes=None, window=0, prefix=0):
    """One request: q [n, q_heads, 128], k, v [length, kv_heads, 128] (float64
    values of the codes); the queries are the last n positions.  Returns the
    output, and for error bounds sum p |v| and the largest sum |q||k| scale."""
    n, heads = q.shape[:2]
    length, kv = k.shape[:2]
    out = np.zeros((n, heads, 128))
    mass, size = np.zeros((n, heads, 128)), np.zeros((n, heads, 1))
    if length == 0:
        return out, mass, size
    on = visible(length, n, window, prefix)
    dist = np.abs(np.arange(length - n, length)[:, None] - np.arange(length)[None])
    for h in range(heads):
        kh, vh = k[:, h * kv // heads], v[:, h * kv // heads]
        x = scale * (q[:, h] @ kh.T)
        size[:, h, 0] = (scale * (np.abs(q[:, h]) @ np.abs(kh).T)).max(1)
        if cap > 0:
            x = cap * np.tanh(x / cap)
        if slopes is not None:
            x = x - float(slopes[h]) * dist
        x = np.where(on, x, -np.inf)
        top = x.max(1, keepdims=True)
        w = np.where(on, np.exp(x - np.where(np.isfinite(top), top, 0.0)), 0.0)
        tot = w.sum(1, keepdims=True)
        w = w / np.where(tot > 0, tot, 1.0)
        out[:, h] = w @ vh
        mass[:, h] = w @ np.abs(vh)
    return out, mass, size
