"""Plain definitions, in fp64 and whole numbers, of the 8-bit paged cache, the
verification of drafted tokens and the pages' bookkeeping.  Test infrastructure only."""
import numpy as np

QMAX = {"e4m3": 448.0, "int8": 127.0}


def e4m3_values():
    """What the 256 codes stand for: sign, 4 exponent bits (bias 7), 3 of the significand;
    0x7f and 0xff are NaN."""
    out = np.zeros(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if e == 15 and m == 7 else x
        if c & 128:
            out[c] = -out[c]
    return out


E4M3 = e4m3_values()


def values(codes, fmt):
    """fp64 values of uint8 codes in units of their scale."""
    return codes.view(np.int8).astype(np.float64) if fmt == "int8" else E4M3[codes]


def encode(x, fmt):
    """uint8 codes of fp64 values in units of the scale: nearest, ties to even."""
    x = np.asarray(x, np.float64)
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    mag = E4M3[:127]  # increasing with the code
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(mag, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up = mag[hi] - a
    down = a - mag[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_for(top, fmt):
    """The least power of two >= 2^-64 at which `top` has a code."""
    e = -64
    while QMAX[fmt] * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


def append(codes, scales, rows, table_row, length, block, fmt):
    """Writes one request's new rows (n, heads, d) fp64 as its last n tokens into codes
    (pages, page, heads, d) uint8 and scales (pages, blocks, heads), in place."""
    page, n = codes.shape[1], rows.shape[0]
    start = length - n
    finite = np.isfinite(rows)
    for t0 in range(start // block * block, length, block):
        pg, at = table_row[t0 // page], t0 % page
        lo, hi = max(t0, start), min(t0 + block, length)
        for h in range(rows.shape[1]):
            x, ok = rows[lo - start:hi - start, h], finite[lo - start:hi - start, h]
            s = scale_for(np.abs(np.where(ok, x, 0.0)).max(), fmt)
            old = scales[pg, at // block, h]
            if lo > t0 and old >= s:
                s = old
            elif lo > t0:
                have = codes[pg, at:at + lo - t0, h]
                codes[pg, at:at + lo - t0, h] = encode(values(have, fmt) * (old / s), fmt)
            y = np.where(np.isnan(x), 0.0, np.clip(np.where(np.isnan(x), 0.0, x) / s, -QMAX[fmt], QMAX[fmt]))
            codes[pg, at + lo - t0:at + hi - t0, h] = encode(y, fmt)
            scales[pg, at // block, h] = s


def expand(codes, scales, fmt):
    """The whole cache's values, fp64."""
    return values(codes, fmt) * np.repeat(scales.astype(np.float64), codes.shape[1] // scales.shape[1], 1)[..., None]


def chunk_seen(length, n, first=0, last=0, causal=True):
    """(n, length): which tokens the last n of a request see."""
    pos = np.arange(length - n, length)[:, None]
    t = np.arange(length)[None]
    if not causal:
        return np.ones((n, length), bool)
    seen = t <= pos
    return seen if last <= 0 else seen & ((t < first) | (t >= pos + 1 - last))


def verify(target, draft, tokens, parents, u, u_next):
    """One request (fp64 probabilities, node 0 first): (nodes that stand, next token, weights)."""
    n = len(tokens)
    clean = lambda p: np.clip(np.nan_to_num(np.asarray(p, np.float64), nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)
    path = [0]
    while True:
        i = path[-1]
        p = clean(target[i])
        q = None if draft is None else clean(draft[i])
        w, cover, mass, took = p.copy(), 0.0, 1.0, None
        for c in range(i + 1, n):
            if parents[c] != i:
                continue
            x = tokens[c]
            inside = 0 <= x < p.size
            have = w[x] if inside else 0.0
            if (u[c] * mass * (q[x] if inside else 0.0) if q is not None else u[c] * mass) < have:
                took = c
                break
            if q is not None:
                cover += mass
                w = np.maximum(p - cover * q, 0.0)
                mass = w.sum()
            elif inside:
                mass = max(mass - w[x], 0.0)
                w[x] = 0.0
        if took is None:
            break
        path.append(took)
    if not w.sum() > 0:
        w = p
    if not w.sum() > 0:
        return path, -1, w
    cum = np.cumsum(w)
    at = min(max(float(u_next), 0.0), 1.0 - 2.0 ** -24)
    return path, int(np.searchsorted(cum, at * cum[-1], side="right")), w


class Pages:
    """Page table, lengths, reference counts; the pages' contents follow as labels."""

    def __init__(self, table, refs, lens, page, labels):
        self.table, self.refs, self.lens = np.array(table), np.array(refs), np.array(lens)
        self.page, self.labels = page, np.array(labels)

    def held(self, tokens):
        return -(-int(tokens) // self.page)

    def fork(self, src):
        table = np.full((len(src), self.table.shape[1]), -1, self.table.dtype)
        lens = np.zeros(len(src), self.lens.dtype)
        for b, n in enumerate(self.lens):
            for p in self.table[b, :self.held(n)]:
                self.refs[p] -= 1
        for b, s in enumerate(src):
            if s >= 0:
                lens[b] = self.lens[s]
                table[b, :self.held(lens[b])] = self.table[s, :self.held(lens[b])]
                for p in table[b, :self.held(lens[b])]:
                    self.refs[p] += 1
        self.table, self.lens = table, lens

    def release(self, new):
        for b, n in enumerate(new):
            for i in range(self.held(n), self.held(self.lens[b])):
                self.refs[self.table[b, i]] -= 1
                self.table[b, i] = -1
        self.lens = np.array(new)

    def reserve(self, new):
        save = self.table.copy(), self.refs.copy(), self.labels.copy()
        free = [p for p, r in enumerate(self.refs) if r == 0]
        need, moves = 0, []

        def take():
            nonlocal need
            need += 1
            return free[need - 1] if need <= len(free) else None
        for b, n in enumerate(new):
            old = int(self.lens[b])
            if n > old and old % self.page and self.refs[self.table[b, old // self.page]] > 1:
                was, p = self.table[b, old // self.page], take()
                self.refs[was] -= 1
                if p is not None:
                    moves.append((was, p))
                    self.table[b, old // self.page] = p
                    self.refs[p] = 1
            for i in range(self.held(old), self.held(n)):
                p = take()
                if p is not None:
                    self.table[b, i] = p
                    self.refs[p] = 1
        if need > len(free):
            self.table, self.refs, self.labels = save
            return need - len(free)
        for a, p in moves:
            self.labels[p] = self.labels[a]
        self.lens = np.array(new)
        return 0

    def compact(self):
        held = int((self.refs > 0).sum())
        to = [p for p in range(held) if self.refs[p] <= 0]
        out = [p for p in range(held, len(self.refs)) if self.refs[p] > 0]
        for a, p in zip(out, to):
            self.labels[p] = self.labels[a]
            self.refs[p], self.refs[a] = self.refs[a], 0
            for b, n in enumerate(self.lens):
                row = self.table[b, :self.held(n)]
                row[row == a] = p
        return held
