"""Plain 64-bit restatement of the key/value cache calls, from the text of
include/qnt.h (numpy, one request, run and head at a time).  Shares no code with
the kernels; test infrastructure, not collected."""
from __future__ import annotations

import math

import numpy as np

INT8, E4M3 = 1, 2
OK, ARG, PAGES, NONFINITE = 0, 1, 8, 6
TOP = {INT8: 127.0, E4M3: 448.0}


def e4m3_table() -> np.ndarray:
    """Value of each of the 256 E4M3 bytes, from the bit fields."""
    v = np.zeros(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            x = math.nan
        v[b] = -x if s else x
    return v


_E4M3 = e4m3_table()


def value(codes: np.ndarray, fmt: int) -> np.ndarray:
    return codes.astype(np.float64) - 128.0 if fmt == INT8 else _E4M3[codes]


def nearest(y: np.ndarray, fmt: int) -> np.ndarray:
    """Code bytes of the values nearest to y, ties to even (y in 64 bits)."""
    if fmt == INT8:
        return (np.clip(np.rint(y), -127, 127) + 128).astype(np.uint8)
    grid = _E4M3[:127]                                  # 0 .. 448; the byte is the index, its last bit the mantissa's
    mids = (grid[1:] + grid[:-1]) / 2                   # exact: five significant bits
    a = np.abs(y)
    lo = np.searchsorted(mids, a, side="left")          # a tie goes to the lower neighbour ...
    tie = (lo < 126) & (a == mids[np.minimum(lo, 125)])
    lo = np.where(tie & (lo % 2 == 1), lo + 1, lo)      # ... unless that one is odd
    return (lo | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def slots(page, pages, length, add, table, free, count, tokens):
    """Returns (table, free, len_out, cu, slots, count_out, status)."""
    table, free = table.copy(), free.copy()
    rows, width = table.shape
    room, status = width * page, OK
    if not 0 <= count <= pages:
        status = ARG
    count = min(max(count, 0), pages)
    up = lambda v: -(-v // page)  # noqa: E731
    stack = [int(x) for x in free[:count]]
    len_out, cu, out = np.array(length), np.zeros(rows + 1, np.int64), np.full(tokens, -1, np.int64)
    for b in range(rows):
        if add[b] < 0:
            len_out[b] = 0
            if 0 <= length[b] <= room:
                stack += [int(x) for x in table[b, :up(length[b])]]
            else:
                status = max(status, ARG)
    at, closed = 0, False
    for b in range(rows):
        n, begin = max(int(add[b]), 0), at
        at += n
        cu[b + 1] = min(at, tokens)
        if add[b] < 0:
            continue
        if not 0 <= length[b] <= room or length[b] + n > room or at > tokens:
            status = max(status, ARG)
            continue
        used = up(length[b])
        need = up(length[b] + n) - used
        if need and (closed or need > len(stack)):
            closed, status = True, max(status, PAGES)
            continue
        for j in range(need):
            table[b, used + j] = stack.pop()
        len_out[b] = length[b] + n
        for t in range(n):
            p = int(length[b]) + t
            pg = int(table[b, p // page])
            out[begin + t] = pg * page + p % page if 0 <= pg < pages else 2 ** 31 - 1
    left = len(stack)
    if left > count:
        free[count:left] = stack[count:]
    return table, free, len_out, cu, out, left, status


def append(fmt, page, codes, scales, x, slot):
    """One of K or V.  codes uint8 [pages][heads][page][dim], scales fp32 [pages][heads], x float64
    [tokens][heads][dim] (finite), slot [tokens]; returns new (codes, scales, status)."""
    codes, scales, status = codes.copy(), scales.copy(), OK
    pages, heads = scales.shape
    t, n, last = 0, len(slot), -1000
    while t < n:
        s = int(slot[t])
        if s >= pages * page:
            status, t = ARG, t + 1
            continue
        if s < 0:
            t += 1
            continue
        end = t + 1
        while end < n and slot[end] == s + (end - t) and (s + end - t) % page:
            end += 1
        if last // page == s // page:
            status, t, last = ARG, end, int(slot[end - 1])   # a second run of the page: not written
            continue
        last = int(slot[end - 1])
        pg, off = s // page, s % page
        for h in range(heads):
            run = x[t:end, h]
            new = np.float32(np.abs(run).max() / TOP[fmt])
            old = scales[pg, h] if off else np.float32(0)
            new = max(new, old)
            if off and new > old:
                codes[pg, h, :off] = nearest(value(codes[pg, h, :off], fmt) * np.float64(old) / np.float64(new), fmt)
            scales[pg, h] = new
            y = run / np.float64(new) if new > 0 else np.zeros_like(run)
            codes[pg, h, off:off + end - t] = nearest(y, fmt)
        t = end
    return codes, scales, status


def attn(fmt, page, kc, vc, ks, vs, q, cu, length, table, scale, window, out_eps):
    """q float64 [tokens][heads][dim].  Returns (y, bound) [tokens][heads][dim] with NaN in rows of no request: the
    exact result and how far a kernel may be off (see below)."""
    y = np.full(q.shape, np.nan)
    bound = np.full(q.shape, np.nan)
    kv_heads = ks.shape[1]
    group = q.shape[1] // kv_heads
    for b in range(len(length)):
        n = cu[b + 1] - cu[b]
        L = int(length[b])
        if n == 0:
            continue
        ids = table[b, :-(-L // page)]
        full = [(value(c[ids], fmt) * s[ids].astype(np.float64)[..., None, None]).transpose(1, 0, 2, 3)
                .reshape(kv_heads, -1, q.shape[2])[:, :L] for c, s in ((kc, ks), (vc, vs))]
        for h in range(q.shape[1]):
            k, v = full[0][h // group], full[1][h // group]
            top_ks = float(ks[ids, h // group].max()) if len(ids) else 0.0
            top_vs = float(vs[ids, h // group].max()) if len(ids) else 0.0
            for t in range(n):
                p = L - n + t
                lo = max(0, p - window + 1) if window else 0
                row = q[cu[b] + t, h]
                if p + 1 <= lo:
                    y[cu[b] + t, h] = bound[cu[b] + t, h] = 0.0
                    continue
                x = k[lo:p + 1] @ row * scale
                w = np.exp(x - x.max())
                total = w.sum()
                r = w @ v[lo:p + 1] / total
                size = w @ np.abs(v[lo:p + 1]) / total
                # Logits: fp32 sums of products of up to 255 (INT8's offset codes, its 128 taken off: 383) or 448 times
                # the scale; 16 roundings of 2^-24, and 4 of the logit itself.  Weights: half a step of fp16, in the
                # numerator and in the sum, or half its subnormal step.  Output sums: one rounding of a page's sum
                # (up to 255 or 448 codes times the scale) per 16 tokens, and the type's half step.
                dx = 2.0 ** -20 * (383 if fmt == INT8 else 448) * abs(scale) * top_ks * np.abs(row).sum() + 2.0 ** -22 * np.abs(x).max()
                steps = len(x) / 16 + 16
                vmax = np.abs(v[lo:p + 1]).max()
                bound[cu[b] + t, h] = ((2.0 ** -11 + 2 * dx) * (size + np.abs(r)) + len(x) * 2.0 ** -25 / total * (vmax + np.abs(r))
                                       + steps * 2.0 ** -23 * (383 if fmt == INT8 else 448) * top_vs + out_eps / 2 * np.abs(r) * 1.01 + 2.0 ** -25)
                y[cu[b] + t, h] = r
    return y, bound
