"""Measured cases of the operators that work on the paged KV pool.

Four operators, each with a plain form in elementary torch operations
(``own = False``) and the framework's calls (``own = True``):

* ``append``   new tokens' q and k rotated, k and v written into their page rows;
* ``attend``   attention over a prefix that a group of sequences shares and over
  each sequence's own pages, for single new tokens and for prompts;
* ``weights``  every cached token's attention weight added to its running sum;
* ``evict``    the heaviest and the newest tokens kept, moved into the first slots.

The pool is bf16 ``[layers, 2, pages, page_size, heads, dim]``; a sequence's
pages are found through an int32 block table.  The shapes are the KV shapes of
``paged_kv_movement_amd.workloads`` (8 KV heads of 128, its one-head share
under 8-way tensor parallelism, 16-token pages, 10000-token contexts, a
32768-token prefix) and generic ones around them.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def _case(name, op, **k):
    c = {"op": op, "heads": 8, "rep": 4, "dim": 128, "page": 16, "seqs": 1, "seed": 11,
         "own_lo": 0, "own_hi": 0, "new_lo": 1, "new_hi": 1, "groups": 0, "prefix": 0}
    if name is not None:
        c["name"] = name
    c.update(k)
    return c


def listed():
    return [
        # one user's next token: one row of q, k and v, where the launch is all there is
        _case("append_token", "append", own_lo=10000, own_hi=10000, rot=128, interleaved=False,
              scaling="none", factor=1.0, base=500000.0, type="bf16", evicting=False),
        # a decode batch far beyond the trained length, half of each head rotated in interleaved pairs, with the
        # running sums and positions of the new slots set for a later eviction
        _case("append_batch", "append", seqs=64, own_lo=500, own_hi=10000, rot=64, interleaved=True,
              scaling="yarn", factor=8.0, base=10000.0, type="fp16", evicting=True),
        # eight prompts of up to 10000 tokens written at once
        _case("append_prompts", "append", seqs=8, own_lo=10000, own_hi=10000, new_lo=700, new_hi=10000, rot=128,
              interleaved=False, scaling="wavelength", factor=8.0, base=500000.0, type="bf16", evicting=False),
        # one user's next token over a 10000-token context, nothing shared
        _case("attend_token", "attend", own_lo=10000, own_hi=10000),
        # the same context length for eight users on one rank's share under 8-way tensor parallelism
        _case("attend_share", "attend", heads=1, seqs=8, own_lo=9001, own_hi=10000),
        # 32 conversations over one 8192-token system prompt, single tokens
        _case("attend_prefix", "attend", seqs=32, own_lo=17, own_hi=2000, groups=1, prefix=8192),
        # two 32768-token documents, 32 questions on each, single tokens
        _case("attend_documents", "attend", seqs=64, own_lo=300, own_hi=4000, groups=2, prefix=32768),
        # four ragged prompts after a shared 4096-token prefix, causal among their own tokens
        _case("attend_prompts", "attend", seqs=4, own_lo=1100, own_hi=1300, new_lo=101, new_hi=1024, groups=1,
              prefix=4096),
        # the weights of a decode step over a shared prefix and own tokens
        _case("weights_step", "weights", seqs=32, own_lo=17, own_hi=2000, groups=1, prefix=8192),
        # the weights of whole prompts, as an eviction after prefill needs them
        _case("weights_prompts", "weights", seqs=4, own_lo=1300, own_hi=2000, new_lo=1000, new_hi=1300),
        # every step once the budget is reached: one token more than is kept
        _case("evict_step", "evict", seqs=16, own_lo=2049, own_hi=2049, keep=2048, recent=256, layers=1, shared=False),
        # after prefill: 10000-token contexts brought down to 4096, several layers in one call
        _case("evict_prompts", "evict", seqs=8, own_lo=3000, own_hi=10000, keep=4096, recent=512, layers=4,
              shared=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "weights", "evict"])
    most = [work(c) for c in listed() if c["op"] == op]
    most = {k: max(w[k] for w in most) for k in ("bytes", "flops")}
    while True:
        c = _case(None, op, heads=rng.choice([1, 2, 3, 4, 8]), rep=rng.choice([1, 2, 4, 5, 8]),
                  dim=rng.choice([64, 80, 128, 128, 256]), page=rng.choice([16, 16, 16, 8, 12, 32, 256]),
                  seqs=_log(rng, 1, 64), seed=rng.randrange(1 << 30))
        hi = _log(rng, 1, 12000)
        c["own_hi"], c["own_lo"] = hi, rng.randint(max(1, hi // 20), hi)
        if op != "evict" and rng.random() < 0.4:          # prompts; else single tokens
            c["new_hi"] = _log(rng, 1, min(hi, 4000))
            c["new_lo"] = rng.randint(1, c["new_hi"])
        if op in ("attend", "weights") and rng.random() < 0.6:
            c["groups"] = rng.randint(1, min(4, c["seqs"]))
            c["prefix"] = _log(rng, 1, 32768)
        if op == "append":
            c.update(rot=2 * rng.randint(1, c["dim"] // 2), interleaved=rng.random() < 0.5,
                     scaling=rng.choice(["none", "linear", "ntk", "yarn", "wavelength"]),
                     factor=rng.choice([2.0, 4.0, 8.0]), base=rng.choice([10000.0, 500000.0]),
                     type=rng.choice(["bf16", "fp16", "fp32"]), evicting=rng.random() < 0.5)
            if c["rot"] < 4:
                c["rot"] = 4
        if op == "evict":
            c["keep"] = rng.randint(1, hi)
            c.update(recent=rng.randint(0, min(c["keep"], 1 + c["keep"] // 4)), layers=rng.randint(1, 4),
                     shared=rng.random() < 0.3)
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def _lens(c):
    """(tokens in own pages, new ones among them, sequences per group, prefix tokens per group), from the case alone."""
    r = random.Random(c["seed"])
    lens = [r.randint(c["own_lo"], c["own_hi"]) for _ in range(c["seqs"])]
    new = [min(n, r.randint(c["new_lo"], c["new_hi"])) for n in lens]
    sizes, prefix = [], []
    for g in range(c["groups"]):
        left = c["seqs"] - sum(sizes)
        sizes.append(left if g == c["groups"] - 1 else max(1, left // (c["groups"] - g)))
        prefix.append(c["prefix"] if g == 0 else r.randint(max(1, c["prefix"] // 2), c["prefix"]))
    return lens, new, sizes, prefix


def _group_of(c, sizes):
    out = []
    for g, n in enumerate(sizes):
        out += [g] * n
    return out + [None] * (c["seqs"] - len(out))


def _visible(c):
    """(query row, visible token) pairs of one query head."""
    lens, new, sizes, prefix = _lens(c)
    group = _group_of(c, sizes)
    pairs = 0
    for s, (n, m) in enumerate(zip(lens, new)):
        pairs += m * (n - m) + m * (m + 1) // 2 + m * (prefix[group[s]] if group[s] is not None else 0)
    return pairs


def work(case):
    c = case
    lens, new, sizes, prefix = _lens(c)
    H, Hq, D, rows = c["heads"], c["heads"] * c["rep"], c["dim"], sum(new)
    kv = (sum(lens) + sum(prefix)) * H * D * 2                 # one of K and V
    if c["op"] == "append":
        b = 4 if c["type"] == "fp32" else 2
        return {"bytes": rows * (Hq * D * 2 * b + 2 * H * D * (b + 2) + 4) + (rows * H * 8 if c["evicting"] else 0),
                "flops": rows * (Hq + H) * c["rot"] * 3}
    if c["op"] == "attend":
        return {"bytes": 2 * kv + rows * Hq * (4 * D + 4), "flops": 4 * D * Hq * _visible(c)}
    if c["op"] == "weights":
        return {"bytes": kv + rows * Hq * (2 * D + 4) + (sum(lens) + sum(prefix)) * H * 8,
                "flops": 2 * D * Hq * _visible(c)}
    hs = 1 if c["shared"] else H
    moved = read = kept = 0.0
    for n in lens:
        k = min(n, c["keep"])
        read, kept = read + n, kept + k
        if n > k:
            new_kept = min(c["recent"], n - k)                 # newest ones, behind the first `keep` slots
            others = (k - c["recent"]) / max(1, n - c["recent"])
            moved += min(k, new_kept + others * max(0, n - k - new_kept))
    rows = c["layers"] * hs
    return {"bytes": int(rows * (8 * read + 8 * kept) + c["layers"] * moved * H * D * 2 * 2 * 2),
            "flops": int(rows * read * 8)}


# ------------------------------------------------------------------ inputs

def _tables(lens, page, ids):
    """Block tables of consecutive runs of the page ids, one row per sequence, -1 behind each one's last page."""
    need = [-(-n // page) for n in lens]
    t = torch.full((len(lens), max([1] + need)), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = ids[at:at + n]
        at += n
    return t, at


def _inputs(case, seed):
    c = case
    lens, new, sizes, prefix = _lens(c)
    g = torch.Generator().manual_seed(seed)
    d = torch.Generator(device="cuda").manual_seed(seed)
    H, Hq, D, P, rows = c["heads"], c["heads"] * c["rep"], c["dim"], c["page"], sum(new)
    pages = sum(-(-n // P) for n in lens + prefix) + 3
    ids = torch.randperm(pages, generator=g, dtype=torch.int32)
    own_t, used = _tables(lens, P, ids)
    layers = c.get("layers", 1)
    st = {"case": c, "lens": lens, "new": new, "sizes": sizes, "prefix": prefix, "layers": layers,
          "pool": torch.randn((layers, 2, pages, P, H, D), generator=d, device="cuda", dtype=torch.bfloat16),
          "own_table": own_t.cuda(), "own_lens": torch.tensor(lens, dtype=torch.int32).cuda(),
          "prefix_table": None, "prefix_lens": None}
    if prefix:
        pre_t, _ = _tables(prefix, P, ids[used:])
        st.update(prefix_table=pre_t.cuda(), prefix_lens=torch.tensor(prefix, dtype=torch.int32).cuda())

    def normal(*shape, type=torch.bfloat16, gain=1.0):
        return (torch.randn(shape, generator=d, device="cuda") * gain).to(type)

    if c["op"] == "append":
        # one fused projection's output; q, k and v are views of its rows
        t = _TYPES[c["type"]]
        qkv = normal(rows, (Hq + 2 * H) * D, type=t)
        pos = []
        for s, (n, m) in enumerate(zip(lens, new)):
            start = int(torch.randint(0, 4, (1,), generator=g)) * 30000     # what came before the own pages
            pos += range(start + n - m, start + n)
        st.update(q=qkv[:, :Hq * D].unflatten(1, (Hq, D)), k=qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D)),
                  v=qkv[:, (Hq + H) * D:].unflatten(1, (H, D)),
                  positions=torch.tensor(pos, dtype=torch.int32).cuda())
        if c["evicting"]:
            cap = max(lens)
            st.update(weights=torch.rand((c["seqs"], H, cap), generator=d, device="cuda"),
                      slots=torch.arange(cap, dtype=torch.int32, device="cuda").expand(c["seqs"], H, cap).contiguous())
    elif c["op"] == "attend":
        st["q"] = normal(rows, Hq, D, gain=2.0)
    elif c["op"] == "weights":
        st["q"] = normal(rows, Hq, D, gain=2.0)
        pre = torch.tensor([prefix[x] if x is not None else 0 for x in _group_of(c, sizes)])
        ends = torch.cat([torch.arange(n - m + 1, n + 1) + int(p) for n, m, p in zip(lens, new, pre)]).cuda()
        # about what a row's scores sum to: log(visible tokens) + variance / 2
        st["lse"] = (ends.float().log()[:, None] + 2.0 + 0.3 * normal(rows, Hq, type=torch.float32)).contiguous()
        st["own_sums"] = torch.rand((c["seqs"], H, max(lens)), generator=d, device="cuda")
        st["own_out"] = torch.zeros_like(st["own_sums"])
        if prefix:
            st["prefix_sums"] = torch.rand((len(prefix), H, max(prefix)), generator=d, device="cuda")
            st["prefix_out"] = torch.zeros_like(st["prefix_sums"])
    else:
        hs, cap = (1 if c["shared"] else H), max(lens)
        w = (2.0 * torch.randn((layers, c["seqs"], hs, cap), generator=d, device="cuda")).exp()
        w[torch.rand(w.shape, generator=d, device="cuda") < 0.1] = 0.0      # never attended to
        st["weights"] = w
        # an earlier eviction has filled holes with later tokens: positions rise with the slot, here and there out of
        # order, and the newest token is behind the last slot
        p = 3 * torch.arange(cap, dtype=torch.int32).repeat(layers, c["seqs"], hs, 1)
        for s, n in enumerate(lens):
            for _ in range(min(n // 4, 50)):
                i, j = (int(x) for x in torch.randint(0, n, (2,), generator=g))
                p[:, s, :, [i, j]] = p[:, s, :, [j, i]]
        st["slots"] = p.cuda()
        shape = (layers, c["seqs"], hs, c["keep"])
        st["out_weights"] = torch.zeros(shape, device="cuda")
        st["out_slots"] = torch.zeros(shape, dtype=torch.int32, device="cuda")
    return st


def prepare(case, seed):
    c = case
    st = _inputs(c, seed)
    if own:
        import paged_kv_movement_amd as kvm
        st["kvm"] = kvm
        st["paged"] = kvm.Paged.from_pool(st["pool"], chunk_size=c["page"])
        tables = kvm.Tables(st["own_table"], st["own_lens"], max_len=max(st["lens"]))
        pre = None
        if st["prefix"]:
            pre = kvm.Tables(st["prefix_table"], st["prefix_lens"], max_len=max(st["prefix"]))
        st["tables"] = tables
        if c["op"] != "evict":
            st["step"] = kvm.Step(st["paged"], tables, st["new"], prefix=pre, group_sizes=st["sizes"])
        if c["op"] == "append":
            st["rope"] = kvm.Rope(c["rot"], base=c["base"], interleaved=c["interleaved"], scaling=c["scaling"],
                                  factor=c["factor"], original_length=8192)
        if c["op"] == "attend":
            st["workspace"] = st["step"].new_attend_workspace(c["heads"] * c["rep"])
        if c["op"] == "evict":
            st["workspace"] = tables.new_evict_workspace(st["paged"], c["layers"], st["weights"].shape[2], c["keep"])
    elif c["op"] == "append":
        f, m = _frequencies(c)
        st["freqs"], st["gain"] = torch.tensor(f, dtype=torch.float64).cuda(), m
    return st


# ------------------------------------------------------------------ the two sides

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_append(st):
    kvm, c = st["kvm"], st["case"]
    extra = {}
    if c["evicting"]:
        extra = {"weights": st["weights"], "slot_positions": st["slots"]}
    q = kvm.append(st["paged"], st["step"], 0, st["q"], st["k"], st["v"], st["positions"], st["rope"], **extra)
    return [q, st["pool"]] + ([st["weights"], st["slots"]] if c["evicting"] else [])


def _own_attend(st):
    out, lse = st["kvm"].attend(st["paged"], st["step"], 0, st["q"], workspace=st["workspace"])
    return [out, lse]


def _own_weights(st):
    st["kvm"].add_weights(st["paged"], st["step"], 0, st["q"], st["lse"], st["own_sums"], st.get("prefix_sums"),
                          out=st["own_out"], prefix_out=st.get("prefix_out"))
    return [st["own_out"]] + ([st["prefix_out"]] if st["prefix"] else [])


def _own_evict(st):
    c = st["case"]
    lens = st["kvm"].evict(st["paged"], st["tables"], 0, c["layers"], st["weights"], st["slots"], c["keep"],
                           recent=c["recent"], out_weights=st["out_weights"], out_positions=st["out_slots"],
                           workspace=st["workspace"])
    return [lens, st["out_weights"], st["out_slots"], st["pool"]]


_own = {"append": _own_append, "attend": _own_attend, "weights": _own_weights, "evict": _own_evict}


def _frequencies(c):
    """(radians per position of each pair, gain of the rotated values), in 64 bits."""
    R, base, s, first = c["rot"], c["base"], c["factor"], 8192
    if c["scaling"] == "ntk":
        base = base * s ** (R / (R - 2))
    f = [base ** (-2.0 * j / R) for j in range(R // 2)]
    if c["scaling"] == "linear":
        f = [x / s for x in f]
    if c["scaling"] == "yarn":
        # pairs that turn at least 32 times in the first length stay, those that turn less than once are interpolated
        def pair(turns):
            return R * math.log(first / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), R - 1)
        for j in range(R // 2):
            stay = 1.0 - min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f[j] = f[j] / s * (1.0 - stay) + f[j] * stay
        return f, 0.1 * math.log(s) + 1.0
    if c["scaling"] == "wavelength":
        # short waves stay, waves longer than the first length are interpolated, a ramp (1 to 4 turns) lies between
        for j in range(R // 2):
            turns = first * f[j] / (2 * math.pi)
            stay = min(max((turns - 1.0) / (4.0 - 1.0), 0.0), 1.0)
            f[j] = (1.0 - stay) * f[j] / s + stay * f[j]
    return f, 1.0


def _rows(st, table, i, lo, hi):
    """Rows of a layer's [pages * page_size] that tokens [lo, hi) of a table's row i are in."""
    t = torch.arange(lo, hi, device="cuda")
    P = st["case"]["page"]
    return table[i, t // P].long() * P + t % P


def _plain_append(st):
    c = st["case"]
    R, D, H = c["rot"], c["dim"], c["heads"]
    a = st["positions"].double()[:, None] * st["freqs"][None, :]
    cos, sin = (a.cos() * st["gain"]).float()[:, None], (a.sin() * st["gain"]).float()[:, None]

    def rotated(x):
        x = x.float()
        if c["interleaved"]:
            u, w = x[..., 0:R:2], x[..., 1:R:2]
            y = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)
        else:
            u, w = x[..., :R // 2], x[..., R // 2:R]
            y = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
        return torch.cat([y, x[..., R:]], -1)

    q = rotated(st["q"]).to(st["q"].dtype)
    k, v = rotated(st["k"]).bfloat16(), st["v"].float().bfloat16()
    at = 0
    for s, (n, m) in enumerate(zip(st["lens"], st["new"])):
        slots = _rows(st, st["own_table"], s, n - m, n)
        st["pool"][0, 0].view(-1, H, D)[slots] = k[at:at + m]
        st["pool"][0, 1].view(-1, H, D)[slots] = v[at:at + m]
        if c["evicting"]:
            st["weights"][s, :, n - m:n] = 0.0
            st["slots"][s, :, n - m:n] = st["positions"][at:at + m]
        at += m
    return [q, st["pool"]] + ([st["weights"], st["slots"]] if c["evicting"] else [])


def _kept(st, which, table, i, n, layer=0):
    """Cached K (0) or V (1) of a table's first n tokens: float32 [heads, n, dim]."""
    c = st["case"]
    x = st["pool"][layer, which].view(-1, c["heads"], c["dim"])[_rows(st, table, i, 0, n)]
    return x.float().transpose(0, 1).contiguous()


def _scores(st, q, k, n, m):
    """Scores of m new tokens' heads [heads, m * rep, tokens] against the cached keys; with m, causal for the last m."""
    c = st["case"]
    rows = q.float().unflatten(1, (c["heads"], c["rep"])).permute(1, 0, 2, 3).flatten(1, 2)
    s = torch.matmul(rows, k.transpose(1, 2).contiguous()) * (1.0 / math.sqrt(c["dim"]))
    if m:
        t = torch.arange(n, device="cuda")
        last = torch.arange(n - m, n, device="cuda").repeat_interleave(c["rep"])
        s.masked_fill_(t[None, None, :] > last[None, :, None], -math.inf)
    return s


def _plain_attend(st):
    c = st["case"]
    H, rep, D = c["heads"], c["rep"], c["dim"]
    group = _group_of(c, st["sizes"])
    out = torch.empty((sum(st["new"]), H * rep, D), device="cuda")
    lse = torch.empty((sum(st["new"]), H * rep), device="cuda")
    at, have = 0, None
    for s, (n, m) in enumerate(zip(st["lens"], st["new"])):
        q = st["q"][at:at + m]
        k, v = _kept(st, 0, st["own_table"], s, n), _kept(st, 1, st["own_table"], s, n)
        x = _scores(st, q, k, n, m)
        if group[s] is not None:
            if have != group[s]:
                have, np_ = group[s], st["prefix"][group[s]]
                pk = _kept(st, 0, st["prefix_table"], have, np_)
                pv = _kept(st, 1, st["prefix_table"], have, np_)
            x = torch.cat([_scores(st, q, pk, np_, 0), x], -1)
        top = x.amax(-1, keepdim=True)
        p = (x - top).exp()
        total = p.sum(-1, keepdim=True)
        y = torch.matmul(p[..., -n:], v)
        if group[s] is not None:
            y = y + torch.matmul(p[..., :-n], pv)
        out[at:at + m] = (y / total).unflatten(1, (m, rep)).transpose(0, 1).flatten(1, 2)
        lse[at:at + m] = (top + total.log()).squeeze(-1).unflatten(1, (m, rep)).transpose(0, 1).flatten(1, 2)
        at += m
    return [out.bfloat16(), lse]


def _plain_weights(st):
    c = st["case"]
    H, rep = c["heads"], c["rep"]
    group = _group_of(c, st["sizes"])
    own_out, pre_out = st["own_out"], st.get("prefix_out")
    own_out.copy_(st["own_sums"])
    if st["prefix"]:
        pre_out.copy_(st["prefix_sums"])
    for s, n in enumerate(st["lens"]):
        own_out[s, :, n:] = 0.0
    for g, n in enumerate(st["prefix"]):
        pre_out[g, :, n:] = 0.0
    at, have = 0, None
    for s, (n, m) in enumerate(zip(st["lens"], st["new"])):
        q = st["q"][at:at + m]
        lse = st["lse"][at:at + m].unflatten(1, (H, rep)).transpose(0, 1).flatten(1, 2)[..., None]
        x = _scores(st, q, _kept(st, 0, st["own_table"], s, n), n, m)
        own_out[s, :, :n] += (x - lse).exp().sum(1)
        if group[s] is not None:
            if have != group[s]:
                have = group[s]
                pk = _kept(st, 0, st["prefix_table"], have, st["prefix"][have])
            x = _scores(st, q, pk, 0, 0)
            pre_out[have, :, :st["prefix"][have]] += (x - lse).exp().sum(1)
        at += m
    return [own_out] + ([pre_out] if st["prefix"] else [])


def _plain_evict(st):
    c = st["case"]
    H, D, keep = c["heads"], c["dim"], c["keep"]
    W, S = st["weights"], st["slots"]
    layers, _, hs, _ = W.shape
    for s, n in enumerate(st["lens"]):
        k = min(n, keep)
        w, p = W[:, s, :, :n], S[:, s, :, :n]
        if n <= keep:
            st["out_weights"][:, s, :, :n], st["out_slots"][:, s, :, :n] = w, p
            continue
        rank = torch.where(p > p.amax(-1, keepdim=True) - c["recent"], math.inf, w)
        best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :k]
        keeps = torch.zeros(w.shape, dtype=torch.bool, device="cuda").scatter_(-1, best, True)
        rows = _rows(st, st["own_table"], s, 0, n)
        for l in range(layers):
            for h in range(hs):
                to = (~keeps[l, h, :k]).nonzero().squeeze(1)
                src = keeps[l, h, k:].nonzero().squeeze(1) + k
                ow, os = w[l, h, :k].clone(), p[l, h, :k].clone()
                ow[to], os[to] = w[l, h, src], p[l, h, src]
                st["out_weights"][l, s, h, :k], st["out_slots"][l, s, h, :k] = ow, os
                for kv in range(2):
                    x = st["pool"][l, kv].view(-1, hs, H // hs * D)
                    x[rows[to], h] = x[rows[src], h]
    return [st["own_lens"].clamp(max=keep), st["out_weights"], st["out_slots"], st["pool"]]


_plain = {"append": _plain_append, "attend": _plain_attend, "weights": _plain_weights, "evict": _plain_evict}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    c = case
    if c["op"] == "evict":
        return None                      # moves and comparisons: nothing is computed
    st = _inputs(c, seed)
    return {"append": _exact_append, "attend": _exact_attend, "weights": _exact_weights}[c["op"]](c, st)


def _exact_append(c, st):
    """Complex numbers: pair j of a head turned by exp(i * position * f[j])."""
    R, H, D, P = c["rot"], c["heads"], c["dim"], c["page"]
    f, gain = _frequencies(c)
    turn = torch.polar(torch.full((len(st["positions"]), R // 2), gain, dtype=torch.float64),
                       torch.outer(st["positions"].cpu().double(), torch.tensor(f, dtype=torch.float64)))[:, None]
    if c["interleaved"]:
        first, second = torch.arange(0, R, 2), torch.arange(1, R, 2)
    else:
        first, second = torch.arange(R // 2), torch.arange(R // 2, R)

    def rotated(x):
        y = x.cpu().double().clone()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k, v = rotated(st["q"]), rotated(st["k"]), st["v"].cpu().double()
    pool, table = st["pool"].cpu().double(), st["own_table"].cpu()
    page, line = [], []
    for s, (n, m) in enumerate(zip(st["lens"], st["new"])):
        for t in range(n - m, n):
            page.append(int(table[s, t // P]))
            line.append(t % P)
    pool[0, 0, page, line], pool[0, 1, page, line] = k, v
    out = [q.cuda(), pool.cuda()]
    if c["evicting"]:
        w, p = st["weights"].double(), st["slots"].clone()
        at = 0
        for s, (n, m) in enumerate(zip(st["lens"], st["new"])):
            w[s, :, n - m:n] = 0
            p[s, :, n - m:n] = st["positions"][at:at + m]
            at += m
        out += [w, p]
    return out


def _pages64(st, which, table, i, n, head):
    """One head's K or V of the first n tokens, whole pages at a time."""
    pages = table[i, :-(-n // st["case"]["page"])].long()
    return st["pool"][0, which].index_select(0, pages)[:, :, head].flatten(0, 1)[:n].double()


def _heads64(c, st):
    """For each sequence and KV head: (sequence, group, rows, own tokens, head, its query heads, scores in 64 bits of the
    new tokens' heads over [prefix, own] with -inf where a row does not see, prefix length)."""
    rep, group, at = c["rep"], _group_of(c, st["sizes"]), 0
    for s, (n, m) in enumerate(zip(st["lens"], st["new"])):
        g = group[s]
        np_ = st["prefix"][g] if g is not None else 0
        for h in range(c["heads"]):
            heads = slice(h * rep, (h + 1) * rep)
            k = _pages64(st, 0, st["own_table"], s, n, h)
            if g is not None:
                k = torch.cat([_pages64(st, 0, st["prefix_table"], g, np_, h), k])
            x = st["q"][at:at + m, heads].double().flatten(0, 1) @ k.T.contiguous() / c["dim"] ** 0.5
            x = x.view(m, rep, np_ + n)
            seen = torch.ones((m, np_ + n), dtype=torch.bool, device="cuda").tril(np_ + n - m)
            yield s, g, slice(at, at + m), n, h, heads, torch.where(seen[:, None], x, -math.inf), np_
        at += m


def _exact_attend(c, st):
    if work(c)["flops"] > 4e11:
        return None
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    for s, g, rows, n, h, heads, x, np_ in _heads64(c, st):
        v = _pages64(st, 1, st["own_table"], s, n, h)
        if g is not None:
            v = torch.cat([_pages64(st, 1, st["prefix_table"], g, np_, h), v])
        lse[rows, heads] = x.logsumexp(-1)
        out[rows, heads] = (x.softmax(-1).flatten(0, 1) @ v).view(-1, c["rep"], c["dim"])
    return [out, lse]


def _exact_weights(c, st):
    if work(c)["flops"] > 4e11:
        return None
    own_out = st["own_sums"].double()
    pre_out = st["prefix_sums"].double() if st["prefix"] else None
    for s, n in enumerate(st["lens"]):
        own_out[s, :, n:] = 0
    for g, n in enumerate(st["prefix"]):
        pre_out[g, :, n:] = 0
    for s, g, rows, n, h, heads, x, np_ in _heads64(c, st):
        p = (x - st["lse"][rows, heads].double()[..., None]).exp().sum((0, 1))
        own_out[s, h, :n] += p[np_:]
        if g is not None:
            pre_out[g, h, :np_] += p[:np_]
    return [own_out] + ([pre_out] if st["prefix"] else [])
