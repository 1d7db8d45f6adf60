"""The paged E4M3 cache in plain float64: tables, slots, codes, attention, block masses.

One power-of-two scale per page of 16 tokens and KV head, for each of K and V.  Code
values are kept as float64 numbers; a stored value is code * scale.
"""

import math

import numpy as np

PAGE = 16
MIN_EXP, MAX_EXP = -100, 119


def round_e4m3(x):
    """x to the nearest E4M3 value, ties to even, saturating at 448; NaN becomes 0."""
    x = np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=448.0, neginf=-448.0)
    a = np.minimum(np.abs(x), 448.0)
    _, e = np.frexp(a)                                    # a = f * 2^e, f in [0.5, 1)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), x)


def page_scale(absmax):
    """The smallest power of two s with absmax <= 448 s, within the exponents allowed."""
    absmax = np.asarray(absmax, np.float64)
    f, e = np.frexp(absmax / 448.0)
    e = np.where(f == 0.5, e - 1, e)
    return np.ldexp(1.0, np.clip(np.where(absmax > 0, e, MIN_EXP), MIN_EXP, MAX_EXP))


def plan(ctx, new, table, free, count, capacity):
    """dict of what kvs_paged_plan makes (table is not changed in place)."""
    table = np.array(table, np.int64)
    n, most = len(ctx), table.shape[1] * PAGE
    slots, positions = np.full(capacity, -1), np.zeros(capacity, np.int64)
    row_start, kv_len, denied = [0], [], 0
    wanted, left = 0, count
    for r in range(n):
        c, q = max(int(ctx[r]), 0), max(int(new[r]), 0)
        h = -(-c // PAGE)
        need = -(-(c + q) // PAGE) - h if c + q <= most else 0
        wanted += need
        ok = c + q <= most and (need == 0 or wanted <= count)
        if ok:
            for b in range(need):
                left -= 1
                table[r, h + b] = free[left]
        denied += not ok
        kv_len.append(c + q if ok else c)
        for i in range(q):
            row = row_start[-1] + i
            if row < capacity:
                positions[row] = c + i
                if ok:
                    slots[row] = table[r, (c + i) // PAGE] * PAGE + (c + i) % PAGE
        row_start.append(row_start[-1] + q)
    return {"table": table, "row_start": np.array(row_start), "kv_len": np.array(kv_len), "slots": slots,
            "positions": positions, "count": left, "denied": denied}


class Pages:
    """One layer's pages."""

    def __init__(self, num_pages, hkv, d):
        self.codes = [np.zeros((num_pages, PAGE, hkv, d)) for _ in range(2)]
        self.scales = [np.full((num_pages, hkv), 2.0 ** MIN_EXP) for _ in range(2)]
        self.num_pages = num_pages

    def append(self, k, v, slots):
        slots = np.asarray(slots)
        i = 0
        while i < len(slots):
            page = slots[i] // PAGE
            j = i
            while j < len(slots) and slots[i] >= 0 and slots[j] // PAGE == page:
                j += 1
            if slots[i] >= 0 and page < self.num_pages:
                for x, codes, scales in ((k, self.codes[0], self.scales[0]), (v, self.codes[1], self.scales[1])):
                    run = np.asarray(x[i:j], np.float64)
                    offs = slots[i:j] % PAGE
                    finite = np.where(np.isfinite(run), np.abs(run), 0.0)
                    old = scales[page]
                    if (offs == 0).any():
                        codes[page] = 0
                        old = np.full_like(old, 2.0 ** MIN_EXP)
                    scale = np.maximum(old, page_scale(finite.max(axis=(0, 2))))
                    codes[page] = round_e4m3(codes[page] * (old / scale)[None, :, None])
                    codes[page][offs] = round_e4m3(run / scale[None, :, None])
                    scales[page] = scale
            i = max(j, i + 1)

    def gather(self, slots):
        """(K, V) [rows, hkv, d]; zero where the slot is negative or out of range."""
        slots = np.asarray(slots)
        ok = (slots >= 0) & (slots // PAGE < self.num_pages)
        s = np.where(ok, slots, 0)
        return [np.where(ok[:, None, None], c[s // PAGE, s % PAGE] * z[s // PAGE][:, :, None], 0.0)
                for c, z in zip(self.codes, self.scales)]

    def attend(self, q, table, kv_len, row_start=None, window=0):
        """dict: out [rows, hq, d]; spread, the same with |v| (the scale of what rounding a
        probability costs); reach [rows, hq], the largest sum |q k| / sqrt(D) over a row's
        entries (the scale of a logit's error); floor, max_j(weight * V scale) * sum_j |V code|
        (the scale of what a probability's smallest step costs); mass [n, stride] for
        single-token rows."""
        q = np.asarray(q, np.float64)
        rows, hq, d = q.shape
        table = np.asarray(table)
        n, stride = table.shape
        hkv = self.codes[0].shape[2]
        g = hq // hkv
        row_start = np.arange(n + 1) if row_start is None else np.asarray(row_start)
        out, spread, reach = np.zeros((rows, hq, d)), np.zeros((rows, hq, d)), np.zeros((rows, hq))
        mass, floor = np.zeros((n, stride)), np.zeros((rows, hq, d))
        for r in range(n):
            length = min(max(int(kv_len[r]), 0), stride * PAGE)
            pages = table[r, :-(-length // PAGE)]
            held = np.repeat((pages >= 0) & (pages < self.num_pages), PAGE)[:length]
            pages = np.where((pages >= 0) & (pages < self.num_pages), pages, 0)
            k, v = ((c[pages] * z[pages][:, None, :, None]).reshape(-1, hkv, d)[:length]
                    for c, z in zip(self.codes, self.scales))
            vs = self.scales[1][pages].repeat(PAGE, axis=0)[:length]
            nq = int(row_start[r + 1] - row_start[r])
            for i in range(nq):
                t = int(row_start[r]) + i
                p = length - nq + i
                j = np.arange(length)
                seen = (j <= p) & held
                if window:
                    seen &= j > p - window
                if not seen.any():
                    continue
                kh, vh = k[seen], v[seen]                                   # [entries, hkv, d]
                qh = q[t].reshape(hkv, g, d)
                s = (qh @ kh.transpose(1, 2, 0)).reshape(hq, -1) / math.sqrt(d)
                reach[t] = (np.abs(qh) @ np.abs(kh).transpose(1, 2, 0)).max(-1).reshape(hq) / math.sqrt(d)
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                wg = w.reshape(hkv, g, -1)
                out[t] = (wg @ vh.transpose(1, 0, 2)).reshape(hq, d)
                spread[t] = (wg @ np.abs(vh).transpose(1, 0, 2)).reshape(hq, d)
                codes = np.repeat((np.abs(vh) / vs[seen][:, :, None]).sum(0), g, axis=0)       # [hq, d]
                floor[t] = (w * np.repeat(vs[seen].T, g, axis=0)).max(-1)[:, None] * codes
                if nq == 1:
                    blocks = np.zeros((hq, stride))
                    np.add.at(blocks.T, j[seen] // PAGE, w.T)
                    mass[r] = blocks.max(0)
        return {"out": out, "spread": spread, "reach": reach, "floor": floor, "mass": mass}
