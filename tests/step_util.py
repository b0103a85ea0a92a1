"""Plain 64-bit implementations of the model-step operators and the batches
their tests run on.  Torch on the CPU, one sequence and one head at a time,
straight from the formulas; no code of the library."""
import math

import torch

NAN = float("nan")


class Batch:
    """A pool with a permuted block table per sequence and per shared prefix.
    Every row that no sequence holds, and every row behind a sequence's last
    token, is NaN: nothing of it may reach a result."""

    def __init__(self, seed, heads, dim, page, lens, new, prefix=(), sizes=(), layers=1, spare=3, table_room=0,
                 gain=1.0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.heads, self.dim, self.page, self.layers = g, heads, dim, page, layers
        self.lens, self.new, self.prefix, self.sizes = list(lens), list(new), list(prefix), list(sizes)
        need = [-(-n // page) for n in self.lens + self.prefix]
        room = [n + table_room for n in need]
        self.pages = sum(room) + spare
        ids = torch.randperm(self.pages, generator=g, dtype=torch.int32)
        width = max([1] + room[:len(lens)])
        pwidth = max([1] + room[len(lens):])
        self.own_table = torch.full((len(lens), width), -7, dtype=torch.int32)
        self.prefix_table = torch.full((len(self.prefix), pwidth), -7, dtype=torch.int32)
        at = 0
        for i, n in enumerate(room):
            t, j = (self.own_table, i) if i < len(lens) else (self.prefix_table, i - len(lens))
            t[j, :n] = ids[at:at + n]
            at += n
        self.pool = torch.full((layers, 2, self.pages, page, heads, dim), NAN, dtype=torch.bfloat16)
        for t, ns in ((self.own_table, self.lens), (self.prefix_table, self.prefix)):
            for i, n in enumerate(ns):
                x = torch.randn((layers, 2, n, heads, dim), generator=g) * gain
                self.flat()[:, :, self.rows(t, i, n)] = x.bfloat16()
        self.q_start = [0]
        for m in self.new:
            self.q_start.append(self.q_start[-1] + m)
        self.groups = [g for g, n in enumerate(self.sizes) for _ in range(n)]

    def flat(self):
        return self.pool.view(self.layers, 2, -1, self.heads, self.dim)

    def rows(self, table, i, n, start=0):
        t = torch.arange(start, n)
        return table[i, t // self.page].long() * self.page + t % self.page

    def normal(self, *shape, dtype=torch.bfloat16, gain=1.0):
        return (torch.randn(shape, generator=self.g) * gain).to(dtype)

    def group(self, s):
        return self.groups[s] if s < len(self.groups) else None

    def cached(self, which, s, layer=0):
        """64-bit K (0) or V (1) [tokens, heads, dim] that sequence s sees: prefix, then own."""
        g = self.group(s)
        parts = [self.flat()[layer, which, self.rows(self.own_table, s, self.lens[s])]]
        if g is not None:
            parts.insert(0, self.flat()[layer, which, self.rows(self.prefix_table, g, self.prefix[g])])
        return torch.cat(parts).double()


def attend64(b, q, scale, layer=0):
    """(out, lse, bound of out, bound of lse), 64 bits; rows of no sequence are NaN in both.

    The bounds are the errors that float32 sums and one bf16 rounding allow
    (u = 2^-24, the half step of float32):
      score: D products, exact, D rounded sums, then scale and log2 e: (D + 4) u S with S = scale sum |q_d k_d|;
      weight: e^(score error) and 4 u of the exponential; n rounded sums in l and in acc, again when pieces join;
      P as two bf16 parts: what is left is at most 2^-8 2^-8 = 2^-16 of each p (its half steps multiplied);
      out: all of these, twice (numerator and l), of sum p |v| / l, then 2^-8 |out| of the bf16 rounding (which may
      round a value that is off, hence the 1 + 2^-8), and 2^-133 where bf16 has no more bits."""
    rows, hq, D = q.shape
    u = 2.0 ** -24
    rep = hq // b.heads
    out = torch.full((rows, hq, D), NAN, dtype=torch.float64)
    lse = torch.full((rows, hq), NAN, dtype=torch.float64)
    eo, el = torch.zeros_like(out), torch.zeros_like(lse)
    for s, (n, m) in enumerate(zip(b.lens, b.new)):
        k, v = b.cached(0, s, layer), b.cached(1, s, layer)
        pre = k.shape[0] - n
        for i in range(m):
            r = b.q_start[s] + i
            see = pre + max(0, n - m + i + 1)
            for h in range(hq):
                if see == 0:
                    out[r, h], lse[r, h] = 0.0, -math.inf
                    continue
                kk, vv, x = k[:see, h // rep], v[:see, h // rep], q[r, h].double()
                sc = (kk @ x) * scale
                S = float((kk.abs() @ x.abs()).max() * scale)
                lse[r, h] = torch.logsumexp(sc, 0)
                p = torch.exp(sc - lse[r, h])
                out[r, h] = p @ vv
                rel = (D + 4) * u * S + (see + 12) * u
                if math.isfinite(rel):
                    el[r, h] = rel + 4 * u * (abs(float(lse[r, h])) + S)
                    eo[r, h] = ((2 * rel + 2.0 ** -16) * (p @ vv.abs())) * (1 + 2.0 ** -8) + 2.0 ** -8 * out[r, h].abs() + 2.0 ** -133
    return out, lse, eo, el


def weights64(b, q, lse, scale, own, prefix=None, layer=0):
    """(own sums, prefix sums, their bounds): each weight is off by its score's error (D + 4) u S, by 4 u (S + |lse|) of
    the exponent's own roundings and by 4 u of the exponential; a sum of N weights by N u of them."""
    rows, hq, D = q.shape
    u = 2.0 ** -24
    rep = hq // b.heads
    own, eo = own.double().clone(), torch.zeros_like(own, dtype=torch.float64)
    pre = prefix.double().clone() if prefix is not None else None
    ep = torch.zeros_like(pre) if pre is not None else None
    group_new = [0] * len(b.sizes)
    for g, m in zip(b.groups, b.new):
        group_new[g] += m
    for s, (n, m) in enumerate(zip(b.lens, b.new)):
        k = b.cached(0, s, layer)
        np_ = k.shape[0] - n
        g = b.group(s)
        count = rep * (m if g is None else group_new[g])
        for i in range(m):
            r = b.q_start[s] + i
            see = np_ + max(0, n - m + i + 1)
            for h in range(hq):
                L = float(lse[r, h])
                if L == -math.inf or see == 0:
                    continue
                kk, x = k[:see, h // rep], q[r, h].double()
                p = torch.exp((kk @ x) * scale - L)
                S = (kk.abs() @ x.abs()) * scale
                e = p * ((D + 4) * u * S + 4 * u * (S + abs(L)) + (4 + count) * u)
                if g is not None and pre is not None:
                    pre[g, h // rep, :np_] += p[:np_]
                    ep[g, h // rep, :np_] += e[:np_]
                own[s, h // rep, :see - np_] += p[np_:]
                eo[s, h // rep, :see - np_] += e[np_:]
    eo += u * own.abs()
    if ep is not None:
        ep += u * pre.abs()
    return own, pre, eo, ep


def rope64(x, positions, f, gain, rot, interleaved):
    """Rotated x [rows, heads, dim] in 64 bits, and |x| + |y| of each element's pair (0 where nothing rotates)."""
    y, size = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        t = positions.double() * f[j]
        c, s = torch.cos(t)[:, None] * gain, torch.sin(t)[:, None] * gain
        u, w = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = u * c - w * s, w * c + u * s
        size[..., a] = size[..., b] = (u.abs() + w.abs()) * gain
    return y, size


def evict_row(weights, positions, keep, recent):
    """One row's (weights, positions, [(to, from)]) after eviction, as Python lists."""
    n = len(weights)
    if n <= keep:
        return list(weights), list(positions), []
    newest = max(positions)

    def rank(i):
        w = weights[i]
        if positions[i] > newest - recent:
            return (0, 0.0, i)
        if w != w:
            return (2, 0.0, i)
        return (1, -w, i)
    stay = set(sorted(range(n), key=rank)[:keep])
    to = [i for i in range(keep) if i not in stay]
    src = [i for i in range(keep, n) if i in stay]
    w, p = list(weights[:keep]), list(positions[:keep])
    for a, b in zip(to, src):
        w[a], p[a] = weights[b], positions[b]
    return w, p, list(zip(to, src))
