"""Measured cases of the operators of an 8-bit paged KV pool, of attention with
a sliding window, and of appends that normalise queries and keys.

Each has a plain form in elementary torch operations (``own = False``) and the
framework's calls (``own = True``):

* ``norm``     append with each head of q and k normalised before it is rotated;
* ``append8``  append into an 8-bit pool: e4m3 bytes, one power-of-two scale for
  each block (page) of tokens and head, blocks that a later token outgrows held
  anew; the pool's values are read back as bf16;
* ``window``   attention over the last ``window`` tokens and the first ``sinks``
  ones, over a shared prefix and own pages, in a bf16 or an 8-bit pool;
* ``attend8``  attention over an 8-bit pool;
* ``through8`` pages of a bf16 pool into an 8-bit one and back, as a cache goes
  that is stored and retrieved in bf16 and attended to in 8 bits.

A block's scale is the smallest power of two s with |x| <= 448 s for all of it
(in 2^-100 .. 2^119), its bytes are e4m3(x / s), ties to even.  The shapes are
the KV shapes of ``paged_kv_movement_amd.workloads`` (8 KV heads of 128,
16-token pages, 10000-token contexts, a 32768-token prefix) and generic ones
around them.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_E4M3 = torch.float8_e4m3fn
_LEAST, _MOST = -100, 119                # exponents of a scale


# ------------------------------------------------------------------ cases

def _case(name, op, **k):
    c = {"op": op, "heads": 8, "rep": 4, "dim": 128, "page": 16, "seqs": 1, "seed": 11, "own_lo": 0, "own_hi": 0,
         "new_lo": 1, "new_hi": 1, "groups": 0, "prefix": 0, "layers": 1, "window": 0, "sinks": 0, "bits": 16}
    if op in ("norm", "append8"):
        c.update(rot=128, interleaved=False, base=500000.0, type="bf16", norm="rms", by_head=False)
    if op in ("append8", "attend8"):
        c["bits"] = 8
    if name is not None:
        c["name"] = name
    c.update(k)
    return c


def listed():
    return [
        # one user's next token, q and k normalised for each head: the launch is all there is
        _case("norm_token", "norm", own_lo=10000, own_hi=10000),
        # eight prompts of up to 10000 tokens written at once
        _case("norm_prompts", "norm", seqs=8, own_lo=10000, own_hi=10000, new_lo=700, new_hi=10000),
        # the next tokens of 64 short conversations; most land in a page that holds tokens already
        _case("append8_batch", "append8", seqs=64, own_lo=17, own_hi=300),
        # eight prompts of up to 10000 tokens written into an 8-bit pool
        _case("append8_prompts", "append8", seqs=8, own_lo=10000, own_hi=10000, new_lo=700, new_hi=10000, norm="none"),
        # one user's next token late in a long conversation
        _case("window_token", "window", own_lo=32768, own_hi=32768, window=4096, sinks=4),
        # 32 conversations behind one system prompt, some still within a window of it, others long past it
        _case("window_prefix", "window", seqs=32, own_lo=17, own_hi=6000, groups=1, prefix=8192, window=4096, sinks=4),
        # two long prompts, each token with the 1024 before it
        _case("window_prompts", "window", seqs=2, own_lo=8192, own_hi=10000, new_lo=8000, new_hi=8192, window=1024,
              sinks=4),
        # one user's next token over a 10000-token context in 8 bits
        _case("attend8_token", "attend8", own_lo=10000, own_hi=10000),
        # two 32768-token documents, 32 questions on each, single tokens
        _case("attend8_documents", "attend8", seqs=64, own_lo=300, own_hi=4000, groups=2, prefix=32768),
        # four ragged prompts after a shared 4096-token prefix, causal among their own tokens
        _case("attend8_prompts", "attend8", seqs=4, own_lo=1100, own_hi=1300, new_lo=101, new_hi=1024, groups=1,
              prefix=4096),
        # the pages of four chunks of one layer
        _case("through8_chunks", "through8", seqs=4, own_lo=256, own_hi=256),
        # eight 10000-token contexts, four layers in one call
        _case("through8_contexts", "through8", seqs=8, own_lo=9000, own_hi=10000, layers=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append8", "append8", "window", "window", "attend8", "attend8", "through8"])
    most = [work(c) for c in listed() if c["op"] == op]
    most = {k: max(w[k] for w in most) for k in ("bytes", "flops")}
    while True:
        c = _case(None, op, heads=rng.choice([1, 2, 3, 4, 8]), rep=rng.choice([1, 2, 4, 5, 8]),
                  dim=rng.choice([64, 80, 128, 128, 256]), page=rng.choice([16, 16, 16, 8, 12, 32, 64]),
                  seqs=_log(rng, 1, 64), seed=rng.randrange(1 << 30))
        hi = _log(rng, 1, 12000)
        c["own_hi"], c["own_lo"] = hi, rng.randint(max(1, hi // 20), hi)
        if op != "through8" and rng.random() < 0.4:          # prompts; else single tokens
            c["new_hi"] = _log(rng, 1, min(hi, 4000))
            c["new_lo"] = rng.randint(1, c["new_hi"])
        if op in ("window", "attend8") and rng.random() < 0.5:
            c["groups"] = rng.randint(1, min(4, c["seqs"]))
            c["prefix"] = _log(rng, 1, 32768)
        if op == "window":
            c.update(window=_log(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 16, 130]), bits=rng.choice([16, 8]))
        if op in ("norm", "append8"):
            c.update(rot=2 * rng.randint(2, c["dim"] // 2), interleaved=rng.random() < 0.5,
                     base=rng.choice([10000.0, 500000.0]), type=rng.choice(["bf16", "fp16", "fp32"]),
                     norm=rng.choice(["rms", "centered"] if op == "norm" else ["none", "rms"]),
                     by_head=rng.random() < 0.5)
        if op == "through8":
            c["layers"] = rng.randint(1, 4)
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


def _seen(c):
    """((row, token) pairs that one query head sees, tokens that any row sees, a shared one counted once)."""
    lens, new, sizes, prefix = _lens(c)
    W, S = c["window"] or 1 << 30, c["sinks"]
    pairs = tokens = 0
    first = {}                                               # the first prefix token inside a window of its group
    for g, n, m in zip(_group_of(c, sizes), lens, new):
        np_ = prefix[g] if g is not None else 0
        total = np_ + n
        for p in (range(total - m, total) if c["window"] else ()):
            pairs += min(W, p + 1) + min(S, max(0, p + 1 - W))
        if not c["window"]:
            pairs += m * (total - m) + m * (m + 1) // 2
        lo = max(0, total - m + 1 - W)                       # of the first new token
        tokens += (total - max(lo, np_)) + max(0, min(S, lo) - np_)
        if g is not None:
            first[g] = min(first.get(g, np_), lo)
    for g, lo in first.items():
        tokens += (prefix[g] - lo) + min(S, lo, prefix[g])
    return pairs, tokens


def work(case):
    c = case
    lens, new, sizes, prefix = _lens(c)
    H, Hq, D, P, rows = c["heads"], c["heads"] * c["rep"], c["dim"], c["page"], sum(new)
    if c["op"] in ("norm", "append8"):
        b = 4 if c["type"] == "fp32" else 2
        flops = rows * (Hq + H) * (c["rot"] * 3 + (0 if c["norm"] == "none" else 4 * D))
        moved = rows * (Hq * D * 2 * b + 2 * H * D * b + 4)
        if c["op"] == "norm":
            return {"bytes": moved + rows * 2 * H * D * 2, "flops": flops}
        # k and v as bytes, old tokens of a begun page, and the values read back
        blocks = sum(-(-n // P) - (n - m) // P for n, m in zip(lens, new))
        begun = sum((n - m) % P for n, m in zip(lens, new))
        return {"bytes": moved + (rows + begun) * 2 * H * D + blocks * 2 * H * 8 + sum(lens) * 2 * H * D * 3,
                "flops": flops + (rows + sum(lens)) * 2 * H * D}
    if c["op"] == "through8":
        blocks = sum(-(-n // P) for n in lens)
        return {"bytes": c["layers"] * 2 * H * (sum(lens) * D * 6 + blocks * 8),
                "flops": c["layers"] * 2 * H * sum(lens) * D * 3}
    pairs, tokens = _seen(c)
    per = D * (c["bits"] // 8) + (4 / P if c["bits"] == 8 else 0)        # bytes of a token's K or V in one head
    return {"bytes": int(tokens * 2 * H * per) + rows * Hq * (4 * D + 4), "flops": 4 * D * Hq * pairs}


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


def _rows_of(table, i, lo, hi, page):
    """Rows of a layer's [pages * page] that tokens [lo, hi) of a table's row i are in (on the CPU)."""
    t = torch.arange(lo, hi)
    return table[i, t // page].long() * page + t % page


def _exponent(amax):
    """The scale's exponent for a block's largest magnitude: smallest e with amax <= 448 * 2^e, 448 = 0.875 * 2^9."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, _LEAST).clamp(_LEAST, _MOST)


def _to_bytes(x, scale):
    """e4m3 bytes of x / scale."""
    return (x / scale).clamp(-448.0, 448.0).to(_E4M3).view(torch.uint8)


def _inputs(case, seed):
    c = case
    lens, new, sizes, prefix = _lens(c)
    g = torch.Generator().manual_seed(seed)
    d = torch.Generator(device="cuda").manual_seed(seed)
    H, Hq, D, P, rows, L = c["heads"], c["heads"] * c["rep"], c["dim"], c["page"], sum(new), c["layers"]
    pages = sum(-(-n // P) for n in lens + prefix) + 3
    ids = torch.randperm(pages, generator=g, dtype=torch.int32)
    own_t, used = _tables(lens, P, ids)
    st = {"case": c, "lens": lens, "new": new, "sizes": sizes, "prefix": prefix,
          "own_table": own_t.cuda(), "own_lens": torch.tensor(lens, dtype=torch.int32).cuda(),
          "prefix_table": None, "prefix_lens": None}
    if prefix:
        pre_t, _ = _tables(prefix, P, ids[used:])
        st.update(prefix_table=pre_t.cuda(), prefix_lens=torch.tensor(prefix, dtype=torch.int32).cuda())

    def normal(*shape, type=torch.bfloat16, gain=1.0):
        return (torch.randn(shape, generator=d, device="cuda") * gain).to(type)

    shape = (L, 2, pages, P, H, D)
    if c["bits"] == 8:
        # what an earlier append has left: a block's scale from its own tokens
        bytes8 = torch.empty(shape, dtype=torch.uint8, device="cuda")
        scales = torch.empty((L, 2, pages, H), device="cuda")
        for l in range(L):
            for kv in range(2):
                x = torch.randn(shape[2:], generator=d, device="cuda")
                s = torch.ldexp(torch.ones(()).cuda(), _exponent(x.abs().amax((1, 3))))
                bytes8[l, kv], scales[l, kv] = _to_bytes(x, s[:, None, :, None]), s
        st.update(bytes8=bytes8, scales=scales)
    else:
        st["pool"] = torch.randn(shape, generator=d, device="cuda", dtype=torch.bfloat16)
    if c["op"] in ("norm", "append8"):
        # one fused projection's output; q, k and v are views of its rows
        t = _TYPES[c["type"]]
        qkv = normal(rows, (Hq + 2 * H) * D, type=t)
        pos = []
        for n, m in zip(lens, new):
            start = int(torch.randint(0, 4, (1,), generator=g)) * 30000     # what came before the own pages
            pos += range(start + n - m, start + n)
        st.update(q=qkv[:, :Hq * D].unflatten(1, (Hq, D)), k=qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D)),
                  v=qkv[:, (Hq + H) * D:].unflatten(1, (H, D)), positions=torch.tensor(pos, dtype=torch.int32).cuda())
        if c["norm"] != "none":
            st["q_weight"] = 1.0 + 0.3 * normal(*((Hq, D) if c["by_head"] else (D,)), type=torch.float32)
            st["k_weight"] = 1.0 + 0.3 * normal(*((H, D) if c["by_head"] else (D,)), type=torch.float32)
    elif c["op"] in ("window", "attend8"):
        st["q"] = normal(rows, Hq, D, gain=2.0)
    else:
        st["bytes8"] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.ones((L, 2, pages, H), device="cuda")
    if c["op"] in ("append8", "through8"):
        st["values"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    return st


def prepare(case, seed):
    c = case
    st = _inputs(c, seed)
    if own:
        import paged_kv_movement_amd as kvm
        st["kvm"] = kvm
        if "pool" in st:
            st["paged"] = kvm.Paged.from_pool(st["pool"], chunk_size=c["page"])
        if "bytes8" in st:
            st["paged8"] = kvm.Paged8.from_pool(st["bytes8"], st["scales"])
        if "values" in st:
            st["paged_values"] = kvm.Paged.from_pool(st["values"], chunk_size=c["page"])
        tables = kvm.Tables(st["own_table"], st["own_lens"], max_len=max(st["lens"]))
        pre = None
        if st["prefix"]:
            pre = kvm.Tables(st["prefix_table"], st["prefix_lens"], max_len=max(st["prefix"]))
        st["tables"] = tables
        st["pool_of"] = st["paged8"] if c["bits"] == 8 else st["paged"]
        if c["op"] != "through8":
            st["step"] = kvm.Step(st["pool_of"], tables, st["new"], prefix=pre, group_sizes=st["sizes"])
        if c["op"] in ("norm", "append8"):
            st["rope"] = kvm.Rope(c["rot"], base=c["base"], interleaved=c["interleaved"])
            st["norm"] = None
            if c["norm"] != "none":
                st["norm"] = kvm.Norm(st["q_weight"], st["k_weight"], eps=1e-6, centered=c["norm"] == "centered")
        if c["op"] in ("window", "attend8"):
            st["seen"] = {"window": c["window"], "sinks": c["sinks"]} if c["window"] else {}
            st["workspace"] = st["step"].new_attend_workspace(c["heads"] * c["rep"], **st["seen"])
        return st
    # the plain forms' plan: where each new token goes, which blocks are written, which rows of the pool hold tokens
    P, table = c["page"], st["own_table"].cpu()
    st["held"] = torch.zeros(_pages(st) * P, dtype=torch.bool)
    slots, block, pages, before = [torch.zeros(0, dtype=torch.long)], [], [], []
    for s, (n, m) in enumerate(zip(st["lens"], st["new"])):
        st["held"][_rows_of(table, s, 0, n, P)] = True
        slots.append(_rows_of(table, s, n - m, n, P))
        for p in range((n - m) // P, -(-n // P)):
            block += [len(pages)] * (min(n, (p + 1) * P) - max(n - m, p * P))
            pages.append(int(table[s, p]))
            before.append(max(0, n - m - p * P))             # tokens that are there already
    st["held"] = st["held"].cuda()
    st.update(slots_at=torch.cat(slots).cuda(), block=torch.tensor(block).cuda(), blocks=torch.tensor(pages).cuda(),
              before=torch.tensor(before).cuda())
    if "rot" in c:
        f = [c["base"] ** (-2.0 * j / c["rot"]) for j in range(c["rot"] // 2)]
        st["freqs"] = torch.tensor(f, dtype=torch.float64).cuda()
    return st


def _pages(st):
    return (st["bytes8"] if "bytes8" in st else st["pool"]).shape[2]


# ------------------------------------------------------------------ the framework's calls

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_norm(st):
    q = st["kvm"].append(st["paged"], st["step"], 0, st["q"], st["k"], st["v"], st["positions"], st["rope"],
                         norm=st["norm"])
    return [q, st["pool"]]


def _own_append8(st):
    kvm = st["kvm"]
    q = kvm.append(st["paged8"], st["step"], 0, st["q"], st["k"], st["v"], st["positions"], st["rope"],
                   norm=st["norm"])
    kvm.unpack8(st["paged8"], st["tables"], st["paged_values"])
    return [q, st["values"]]


def _own_attend(st):
    out, lse = st["kvm"].attend(st["pool_of"], st["step"], 0, st["q"], workspace=st["workspace"], **st["seen"])
    return [out, lse]


def _own_through8(st):
    kvm = st["kvm"]
    kvm.pack8(st["paged"], st["tables"], st["paged8"])
    kvm.unpack8(st["paged8"], st["tables"], st["paged_values"])
    return [st["values"]]


_own = {"norm": _own_norm, "append8": _own_append8, "window": _own_attend, "attend8": _own_attend,
        "through8": _own_through8}


# ------------------------------------------------------------------ plain forms

def _normed(st, x, weight):
    if st["case"]["norm"] == "none":
        return x
    if st["case"]["norm"] == "centered":
        x = x - x.mean(-1, keepdim=True)
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight


def _rotated(st, x):
    R = st["case"]["rot"]
    a = st["positions"].double()[:, None] * st["freqs"][None, :]
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    if st["case"]["interleaved"]:
        u, w = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)
    else:
        u, w = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
    return torch.cat([y, x[..., R:]], -1)


def _qkv(st):
    q = _rotated(st, _normed(st, st["q"].float(), st.get("q_weight"))).to(st["q"].dtype)
    return q, _rotated(st, _normed(st, st["k"].float(), st.get("k_weight"))), st["v"].float()


def _plain_norm(st):
    c = st["case"]
    q, k, v = _qkv(st)
    rows = st["pool"].view(2, -1, c["heads"], c["dim"])
    rows[0, st["slots_at"]], rows[1, st["slots_at"]] = k.bfloat16(), v.bfloat16()
    return [q, st["pool"]]


def _read_back(st):
    """bf16 values of every token that a sequence holds."""
    c = st["case"]
    x = st["bytes8"].view(_E4M3).float() * st["scales"][:, :, :, None, :, None]
    held = st["held"].view(-1, c["page"])[None, None, :, :, None, None]
    st["values"].copy_(torch.where(held, x, st["values"].float()))
    return st["values"]


def _plain_append8(st):
    c = st["case"]
    H, D, P = c["heads"], c["dim"], c["page"]
    q, k, v = _qkv(st)
    blocks, before = st["blocks"], st["before"]
    there = (torch.arange(P, device="cuda") < before[:, None])[:, :, None, None]
    for kv, x in ((0, k), (1, v)):
        bytes8, scales = st["bytes8"][0, kv], st["scales"][0, kv]
        amax = torch.zeros((len(blocks), H), device="cuda")
        amax.scatter_reduce_(0, st["block"][:, None].expand(-1, H), x.abs().amax(-1), "amax")
        s = torch.ldexp(torch.ones((), device="cuda"), _exponent(amax))
        was = scales[blocks]
        s = torch.where(before[:, None] > 0, torch.maximum(s, was), s)
        old = bytes8[blocks]
        held = old.view(_E4M3).float() * was[:, None, :, None]
        bytes8[blocks] = torch.where(there, _to_bytes(held, s[:, None, :, None]), old)
        bytes8.view(-1, H, D)[st["slots_at"]] = _to_bytes(x, s[st["block"]][:, :, None])
        scales[blocks] = s
    return [q, _read_back(st)]


def _plain_through8(st):
    c = st["case"]
    held = st["held"].view(-1, c["page"])[None, None, :, :, None, None]
    x = torch.where(held, st["pool"].float(), 0.0)
    s = torch.ldexp(torch.ones((), device="cuda"), _exponent(x.abs().amax((3, 5))))
    st["scales"].copy_(s)
    st["bytes8"].copy_(_to_bytes(x, s[:, :, :, None, :, None]))
    return [_read_back(st)]


def _kept(st, which, table, i, t):
    """K (0) or V (1) of tokens t of the table's rows i (of one shape), float32 [..., heads, dim]."""
    c = st["case"]
    page = table[i, t // c["page"]].long()
    if c["bits"] == 8:
        x = st["bytes8"][0, which][page, t % c["page"]].view(_E4M3).float()
        return x * st["scales"][0, which][page][..., None]
    return st["pool"][0, which][page, t % c["page"]].float()


def _scores(c, q, k, seen):
    """q [b, m, q heads, dim], k [b, n, heads, dim], seen [b, m, n]: scores [b, heads, m * rep, n]."""
    H, rep, m = c["heads"], c["rep"], q.shape[1]
    rows = q.float().unflatten(2, (H, rep)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = torch.matmul(rows, k.permute(0, 2, 3, 1).contiguous()) * (1.0 / math.sqrt(c["dim"]))
    return x.unflatten(2, (m, rep)).masked_fill_(~seen[:, None, :, None, :], -math.inf).flatten(2, 3)


def _values(p, v):
    return torch.matmul(p, v.transpose(1, 2).contiguous())


def _by_row(c, z):
    """[b, heads, m * rep, x] as [b, m, q heads, x]."""
    return z.unflatten(2, (-1, c["rep"])).permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_tokens(st):
    """One new token each: all sequences' own tokens at once, a prefix once for its group."""
    c = st["case"]
    W, S = c["window"] or 1 << 30, c["sinks"]
    B, H, q = len(st["lens"]), c["heads"], st["q"]
    ahead = torch.tensor([0 if x is None else st["prefix"][x] for x in _group_of(c, st["sizes"])], device="cuda")
    last = st["own_lens"].long() - 1
    t = last[:, None] - torch.arange(min(W, max(st["lens"])), device="cuda")       # the window, newest first
    first = torch.arange(min(S, max(st["lens"])), device="cuda").expand(B, -1)
    seen = torch.cat([t >= 0, (first <= last[:, None] - W) & (first < (S - ahead)[:, None])], 1)
    t = torch.cat([t.clamp(min=0), torch.minimum(first, last[:, None])], 1)
    s = torch.arange(B, device="cuda")[:, None].expand_as(t)
    x = _scores(c, q[:, None], _kept(st, 0, st["own_table"], s, t), seen[:, None])
    parts, lo = [(slice(0, B), x, _kept(st, 1, st["own_table"], s, t))], 0
    for g, (size, n) in enumerate(zip(st["sizes"], st["prefix"])):
        t = torch.arange(n, device="cuda")
        i = torch.full_like(t, g)
        pos = n + last[lo:lo + size, None]
        seen = (t > pos - W) | (t < S)
        y = _scores(c, q[None, lo:lo + size], _kept(st, 0, st["prefix_table"], i, t)[None], seen[None])
        parts.append((slice(lo, lo + size), _by_row(c, y)[0].unflatten(1, (H, -1)),
                      _kept(st, 1, st["prefix_table"], i, t)[None]))
        lo += size
    top = x.amax(-1, keepdim=True)
    for at, y, _ in parts[1:]:
        top[at] = torch.maximum(top[at], y.amax(-1, keepdim=True))
    total, out = torch.zeros_like(top), torch.zeros((B, H, c["rep"], c["dim"]), device="cuda")
    for k, (at, y, v) in enumerate(parts):
        p = (y - top[at]).exp()
        total[at] += p.sum(-1, keepdim=True)
        if k == 0:
            out[at] += _values(p, v)
        else:                                                            # the group's rows against one V
            out[at] += _values(p.transpose(0, 1).flatten(1, 2)[None], v)[0].unflatten(1, (-1, c["rep"])).transpose(0, 1)
    lse = (top + total.log()).flatten(1)
    return [(out / total).flatten(1, 2).bfloat16(), lse]


def _plain_attend(st):
    c = st["case"]
    if max(st["new"]) == 1:
        return _plain_tokens(st)
    W, S, at, most = c["window"] or 1 << 30, c["sinks"], 0, 1024          # rows at once
    out = torch.empty(st["q"].shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(st["q"].shape[:2], device="cuda")
    for s, (g, n, m) in enumerate(zip(_group_of(c, st["sizes"]), st["lens"], st["new"])):
        np_ = st["prefix"][g] if g is not None else 0
        for r in range(0, m, most):
            rows = slice(at + r, at + min(m, r + most))
            pos = torch.arange(np_ + n - m + r, np_ + n - m + min(m, r + most), device="cuda")
            begin = max(0, np_ + n - m + r - W + 1)                      # of the first row's window
            t = torch.cat([torch.arange(min(S, begin), device="cuda"),
                           torch.arange(begin, np_ + n - m + min(m, r + most), device="cuda")])
            before, behind = t[t < np_], t[t >= np_] - np_
            k, v = (_kept(st, w, st["own_table"], torch.full_like(behind, s), behind) for w in (0, 1))
            if np_ > 0:
                k, v = (torch.cat([_kept(st, w, st["prefix_table"], torch.full_like(before, g), before), x])
                        for w, x in ((0, k), (1, v)))
            seen = (t <= pos[:, None]) & ((t > pos[:, None] - W) | (t < S))
            x = _scores(c, st["q"][None, rows], k[None], seen[None])
            top = x.amax(-1, keepdim=True)
            p = (x - top).exp()
            total = p.sum(-1, keepdim=True)
            out[rows] = _by_row(c, _values(p, v[None]) / total)[0].bfloat16()
            lse[rows] = _by_row(c, top + total.log())[0].squeeze(-1)
        at += m
    return [out, lse]


_plain = {"norm": _plain_norm, "append8": _plain_append8, "window": _plain_attend, "attend8": _plain_attend,
          "through8": _plain_through8}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    c = case
    if c["op"] in ("window", "attend8"):
        lens, new, sizes, prefix = _lens(c)
        ahead = [0 if g is None else prefix[g] for g in _group_of(c, sizes)]
        if sum(m * (n + p) for m, n, p in zip(new, lens, ahead)) * c["heads"] * c["rep"] * c["dim"] * 4 > 4e12:
            return None
    return {"norm": _exact_append, "append8": _exact_append, "window": _exact_attend, "attend8": _exact_attend,
            "through8": _exact_through8}[c["op"]](c, _inputs(c, seed))


def _through_e4m3(x, scale):
    """x / scale rounded to four bits (fewer below 2^-6) and times the scale, in 64 bits."""
    y = (x / scale).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * scale              # round: halves to even


def _block_scale(amax):
    """Least power of two of which 448 reach amax: a logarithm, put right by one where its rounding missed."""
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448))
    e = torch.where(448 * torch.exp2(e - 1) >= amax, e - 1, e)
    e = torch.where(448 * torch.exp2(e) < amax, e + 1, e)
    return torch.exp2(e.clamp(-100, 119))


def _exact_append(c, st):
    """Complex numbers: pair j of a head turned by exp(i * position * f[j]); 8-bit blocks one after the other."""
    R, H, D, P = c["rot"], c["heads"], c["dim"], c["page"]
    f = torch.tensor([c["base"] ** (-2.0 * j / R) for j in range(R // 2)], dtype=torch.float64, device="cuda")
    angle = torch.outer(st["positions"].double(), f)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    first = torch.arange(0, R, 2) if c["interleaved"] else torch.arange(R // 2)
    second = first + (1 if c["interleaved"] else R // 2)

    def turned(x, weight):
        y = x.double()
        if c["norm"] != "none":
            mean = y.sum(-1, keepdim=True) / D if c["norm"] == "centered" else 0.0
            y = y - mean
            y = y / (torch.linalg.vector_norm(y, dim=-1, keepdim=True).square() / D + 1e-6).sqrt() * weight.double()
        y = y.clone()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k, v = turned(st["q"], st.get("q_weight")), turned(st["k"], st.get("k_weight")), st["v"].double()
    table = st["own_table"].cpu()
    if c["op"] == "norm":
        pool = st["pool"].double()
    else:
        pool = torch.zeros(st["values"].shape, dtype=torch.float64, device="cuda")
        held = st["bytes8"].view(_E4M3).double() * st["scales"].double()[:, :, :, None, :, None]
    at = 0
    for s, (n, m) in enumerate(zip(st["lens"], st["new"])):
        for p in range(-(-n // P)):
            page, lo, hi = int(table[s, p]), max(0, n - m - p * P), min(P, n - p * P)
            for kv, x in ((0, k), (1, v)):
                if c["op"] != "norm":
                    pool[0, kv, page, :min(lo, hi)] = held[0, kv, page, :min(lo, hi)]
                if lo >= hi:
                    continue
                i = at + p * P + lo - (n - m)
                y = x[i:i + hi - lo]
                if c["op"] != "norm":
                    scale = _block_scale(y.abs().amax((0, 2)))
                    if lo > 0:
                        scale = torch.maximum(scale, st["scales"][0, kv, page].double())
                        pool[0, kv, page, :lo] = _through_e4m3(pool[0, kv, page, :lo], scale[:, None])
                    y = _through_e4m3(y, scale[:, None])
                pool[0, kv, page, lo:hi] = y
        at += m
    return [q, pool]


def _exact_through8(c, st):
    P, table = c["page"], st["own_table"].cpu()
    out = torch.zeros(st["values"].shape, dtype=torch.float64, device="cuda")
    for s, n in enumerate(st["lens"]):
        whole = n // P
        for pages, tokens in ((table[s, :whole], P), (table[s, whole:whole + 1], n - whole * P)):
            if tokens == 0 or len(pages) == 0:
                continue
            pages = pages.long().cuda()
            x = st["pool"][:, :, pages, :tokens].double()
            out[:, :, pages, :tokens] = _through_e4m3(x, _block_scale(x.abs().amax((3, 5)))[:, :, :, None, :, None])
    return [out]


def _pages64(c, st, which, table, i, n, head):
    """One head's K or V of the first n tokens, whole pages at a time."""
    pages = table[i, :-(-n // c["page"])].long()
    if c["bits"] == 8:
        x = st["bytes8"][0, which].index_select(0, pages)[:, :, head].contiguous().view(_E4M3).double()
        x = x * st["scales"][0, which].index_select(0, pages)[:, head].double()[:, None, None]
    else:
        x = st["pool"][0, which].index_select(0, pages)[:, :, head].double()
    return x.flatten(0, 1)[:n]


def _exact_attend(c, st):
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for s, (g, n, m) in enumerate(zip(_group_of(c, st["sizes"]), st["lens"], st["new"])):
        np_ = st["prefix"][g] if g is not None else 0
        far = torch.arange(np_ + n - m, np_ + n, device="cuda")[:, None] - torch.arange(np_ + n, device="cuda")
        seen = far >= 0
        if c["window"]:
            seen &= (far < c["window"]) | (torch.arange(np_ + n, device="cuda") < c["sinks"])
        for h in range(c["heads"]):
            k, v = (_pages64(c, st, w, st["own_table"], s, n, h) for w in (0, 1))
            if g is not None:
                k, v = (torch.cat([_pages64(c, st, w, st["prefix_table"], g, np_, h), x]) for w, x in ((0, k), (1, v)))
            heads = slice(h * c["rep"], (h + 1) * c["rep"])
            x = st["q"][at:at + m, heads].double().flatten(0, 1) @ k.T.contiguous() / c["dim"] ** 0.5
            x = torch.where(seen[:, None], x.view(m, c["rep"], np_ + n), -math.inf)
            lse[at:at + m, heads] = x.logsumexp(-1)
            out[at:at + m, heads] = (x.softmax(-1).flatten(0, 1) @ v).view(m, c["rep"], c["dim"])
        at += m
    return [out, lse]
