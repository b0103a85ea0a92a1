"""append, attend, add_weights and evict where they can go wrong at the edges: values that are not finite in every form of
the attention, rows of many pieces, several streams.  Against plain 64-bit implementations; every pool row that no token
is in holds NaN."""
import math

import pytest
import torch

import paged_kv_movement_amd as kvm
import step_util as su
from gpu_util import say
from test_gpu_step import device, within

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
U = 2.0 ** -24


def attend64(b, q, scale, layer=0):
    """step_util.attend64 for caches whose scores may be infinite: an infinite score has no error of its own, so the
    bounds are those of the finite ones (the same count of roundings); a row whose scores are all -infinity weighs
    nothing and gets 0."""
    rows, hq, D = q.shape
    rep = hq // b.heads
    out = torch.full((rows, hq, D), NAN, dtype=torch.float64)
    lse = torch.full((rows, hq), NAN, dtype=torch.float64)
    eo, el = torch.zeros_like(out), torch.zeros_like(lse)
    for s, (n, m) in enumerate(zip(b.lens, b.new)):
        k, v = b.cached(0, s, layer), b.cached(1, s, layer)
        pre = k.shape[0] - n
        for i in range(m):
            r, see = b.q_start[s] + i, pre + max(0, n - m + i + 1)
            for h in range(hq):
                kk, vv, x = k[:see, h // rep], v[:see, h // rep], q[r, h].double()
                sc = (kk @ x) * scale
                lse[r, h] = torch.logsumexp(sc, 0) if see else -INF
                if float(lse[r, h]) == -INF:
                    out[r, h] = 0.0
                    continue
                p = torch.exp(sc - lse[r, h])
                out[r, h] = p @ vv
                size = ((kk.abs() @ x.abs()) * scale)[torch.isfinite(sc)]
                if math.isfinite(float(lse[r, h])):
                    S = float(size.max())
                    rel = (D + 4) * U * S + (see + 12) * U
                    el[r, h] = rel + 4 * U * (abs(float(lse[r, h])) + S)
                    eo[r, h] = ((2 * rel + 2.0 ** -16) * (p @ vv.abs())) * (1 + 2.0 ** -8) + 2.0 ** -8 * out[r, h].abs() + 2.0 ** -133
    return out, lse, eo, el


def weights64(b, q, lse, scale, layer=0):
    """(own, prefix) sums from zero and their bounds, step_util.weights64's count of roundings, infinite scores as above;
    a row whose lse is -infinity adds nothing."""
    rows, hq, D = q.shape
    rep = hq // b.heads
    own = torch.zeros((len(b.lens), b.heads, max(b.lens)), dtype=torch.float64)
    pre = torch.zeros((len(b.prefix), b.heads, max(b.prefix, default=0)), dtype=torch.float64)
    eo, ep = torch.zeros_like(own), torch.zeros_like(pre)
    count = rep * sum(b.new)
    for s, (n, m) in enumerate(zip(b.lens, b.new)):
        k, g = b.cached(0, s, layer), b.group(s)
        np_ = k.shape[0] - n
        for i in range(m):
            r, see = b.q_start[s] + i, np_ + max(0, n - m + i + 1)
            for h in range(hq):
                L = float(lse[r, h])
                if L == -INF or see == 0:
                    continue
                kk, x = k[:see, h // rep], q[r, h].double()
                sc = (kk @ x) * scale
                p = torch.exp(sc - L)
                S = torch.where(torch.isfinite(sc), (kk.abs() @ x.abs()) * scale, 0.0)
                e = p * ((D + 4) * U * S + 4 * U * (S + (abs(L) if math.isfinite(L) else 0.0)) + (4 + count) * U)
                if g is not None:
                    pre[g, h // rep, :np_] += p[:np_]
                    ep[g, h // rep, :np_] += e[:np_]
                own[s, h // rep, :see - np_] += p[np_:]
                eo[s, h // rep, :see - np_] += e[np_:]
    return own, pre, eo, ep


# Each form of the attention and each of its layouts (a narrow piece has at most 16 rows, a wide one 16 or 32 a wave):
# heads, rep, dim, page, lens, new, prefix, sizes, own token of sequence 0 and token of prefix 0 that is not finite
FORMS = {
    "narrow 128": (2, 4, 128, 16, [300, 170], [1, 1], [400], [1], 210, 333),
    "narrow 64": (1, 2, 64, 16, [150, 40], [1, 1], [260], [1], 149, 5),
    "narrow 80": (1, 4, 80, 12, [130, 33], [2, 1], [140], [1], 129, 139),
    "narrow 256": (1, 3, 256, 16, [90, 20], [2, 1], [70], [1], 88, 40),
    "one piece": (1, 1, 64, 16, [20, 9], [1, 1], [], [], 3, None),
    "prefix wide, own narrow": (1, 4, 128, 16, [70] + [30, 9] * 4, [1] * 9, [300], [8], 60, 250),
    "prefix wide of two blocks, own narrow": (1, 8, 128, 16, [70] + [30, 9] * 6, [1] * 13, [300], [12], 60, 250),
    "prefix wide 256, own narrow": (1, 4, 256, 16, [70] + [30, 9] * 4, [1] * 9, [130], [8], 60, 77),
    "wide 64": (1, 2, 64, 16, [120, 20], [20, 9], [90], [1], 110, 17),
    "wide 64 of two blocks": (1, 2, 64, 16, [140, 20], [70, 9], [90], [1], 100, 17),
    "wide 80": (1, 2, 80, 16, [120, 20], [20, 9], [90], [1], 110, 17),
    "wide 80 of two blocks": (1, 2, 80, 12, [140, 20], [70, 9], [90], [1], 100, 17),
    "wide 128 of two blocks": (2, 2, 128, 16, [240, 20], [70, 9], [90], [1], 200, 89),
    "wide 256": (1, 2, 256, 16, [90, 20], [40, 9], [60], [1], 70, 17),
}
VALUES = [INF, -INF, NAN]


def _form(name, place, where, value):
    H, rep, D, P, lens, new, prefix, sizes, own_tok, pre_tok = FORMS[name]
    b = su.Batch(21, H, D, P, lens, new, prefix, sizes, layers=2)
    q = b.normal(b.q_start[-1], H * rep, D)
    table, tok = (b.own_table, own_tok) if place == "own" else (b.prefix_table, pre_tok)
    b.flat()[1, where, b.rows(table, 0, tok + 1, tok)[0], 0, 3] = value
    return b, q


PLACES = [(f, p) for f in FORMS for p in ("own", "prefix") if p == "own" or FORMS[f][9] is not None]


@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("where", [0, 1], ids=["k", "v"])
@pytest.mark.parametrize("form,place", PLACES)
def test_attend_follows_the_formula_where_a_value_is_not_finite(form, place, where, value):
    """Rows that see it follow the formula (an infinite lse included), the others stay as they are without it."""
    say("not finite", form, place, where, value)
    b, q = _form(form, place, where, value)
    pool, paged, step = device(b)
    out, lse = kvm.attend(paged, step, 1, q.cuda())
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    wo, wl, eo, el = attend64(b, q, b.dim ** -0.5, layer=1)
    assert not torch.isfinite(b.cached(where, 0, layer=1)).all()
    within(lse, wl, el, "lse")
    within(out, wo, eo, "out")


@pytest.mark.parametrize("lse_of", ["its own", "another cache"])
@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("form,place", PLACES)
def test_weights_follow_the_formula_where_a_key_is_not_finite(form, place, value, lse_of):
    """With the lse of the same cache, and with a finite one (of the cache before the key was overwritten)."""
    say("weights not finite", form, place, value, lse_of)
    b, q = _form(form, place, 0, value)
    clean = _form(form, place, 0, 0.5)[0] if lse_of == "another cache" else b
    lse = attend64(clean, q, b.dim ** -0.5, layer=1)[1].float()
    pool, paged, step = device(b)
    o = torch.zeros((len(b.lens), b.heads, max(b.lens)), device="cuda")
    p = torch.zeros((len(b.prefix), b.heads, max(b.prefix)), device="cuda") if b.prefix else None
    kvm.add_weights(paged, step, 1, q.cuda(), lse.cuda(), o, p)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    wo, wp, eo, ep = weights64(b, q, lse, b.dim ** -0.5, layer=1)
    within(o, wo, eo, "own")
    if b.prefix:
        within(p, wp, ep, "prefix")


def test_a_row_whose_scores_are_all_minus_infinity_weighs_nothing():
    b = su.Batch(22, 1, 64, 16, [1, 30], [1, 1], layers=2)
    q = b.normal(2, 2, 64)
    q[0, :, 3] = q[0, :, 3].abs() + 1
    b.flat()[1, 0, b.rows(b.own_table, 0, 1)[0], 0, 3] = -INF
    pool, paged, step = device(b)
    out, lse = kvm.attend(paged, step, 1, q.cuda())
    assert torch.all(out[0] == 0) and torch.all(lse[0] == -INF)
    assert torch.isfinite(lse[1]).all()
    w = torch.zeros((2, 1, 30), device="cuda")
    kvm.add_weights(paged, step, 1, q.cuda(), lse, w)
    assert torch.all(w[0] == 0) and torch.isfinite(w[1]).all()


@pytest.mark.parametrize("lens", [[], [0, 0]], ids=["no sequences", "nothing cached"])
def test_a_batch_of_nothing(lens):
    """Every call takes a step without sequences, and one whose sequences hold nothing, and leaves all as it was."""
    H, D = 2, 64
    b = su.Batch(23, H, D, 16, lens, [0] * len(lens), layers=1)
    pool, paged, step = device(b)
    q, k = (torch.zeros((0, h, D), dtype=torch.bfloat16, device="cuda") for h in (4, H))
    w = torch.zeros((len(lens), H, 0 if lens else 5), device="cuda")
    p = torch.zeros(w.shape, dtype=torch.int32, device="cuda")
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert kvm.append(paged, step, 0, q, k, k, pos, kvm.Rope(D), weights=w, slot_positions=p).shape == q.shape
    out, lse = kvm.attend(paged, step, 0, q)
    assert out.shape == q.shape and lse.shape == (0, 4)
    assert kvm.add_weights(paged, step, 0, q, lse, w)[0] is w
    assert kvm.evict(paged, step.own, 0, 1, w[None], p[None], 3).tolist() == lens
    assert kvm.evict(paged, step.own, 0, 1, w[None], p[None], 0, out_weights=w[None, :, :, :0].contiguous(),
                     out_positions=p[None, :, :, :0].contiguous()).tolist() == lens
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0 and torch.equal(pool.cpu().view(torch.int16), b.pool.view(torch.int16))


def test_evict_to_nothing_into_empty_tensors():
    b = su.Batch(24, 2, 64, 16, [9, 3], [0, 0], layers=1)
    pool, paged, step = device(b)
    w = torch.rand((1, 2, 2, 9), generator=b.g).cuda()
    p = torch.zeros(w.shape, dtype=torch.int32, device="cuda")
    empty = {"out_weights": torch.empty((1, 2, 2, 0), device="cuda"),
             "out_positions": torch.empty((1, 2, 2, 0), dtype=torch.int32, device="cuda")}
    assert kvm.evict(paged, step.own, 0, 1, w, p, 0, **empty).tolist() == [0, 0]


@pytest.mark.parametrize("what", ["append", "attend", "evict", "store"])
def test_what_the_binding_made_outlives_calls_on_another_current_stream(what):
    """Made on the default stream, used under another one and dropped while that one is still busy: their memory goes
    to nobody else before the calls have run."""
    b = su.Batch(25, 2, 64, 16, [40, 20], [1, 1], [50], [2], layers=2)
    q, k = b.normal(2, 4, 64).cuda(), b.normal(2, 2, 64).cuda()
    pos = torch.tensor([39, 19], dtype=torch.int32, device="cuda")
    w = torch.rand((1, 2, 2, 48), device="cuda")
    p = torch.arange(48, dtype=torch.int32, device="cuda").expand(1, 2, 2, 48).contiguous()
    chunk = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    busy = torch.randn((8192, 8192), device="cuda").bfloat16()
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    pool, paged, step = device(b)
    table, rope = step.own.table, kvm.Rope(64)
    ws, es = step.new_attend_workspace(4), step.own.new_evict_workspace(paged, 1, 2, 10)
    batch = kvm.Batch(paged, [kvm.Seq(table[0].contiguous(), 0, 40, [chunk] * 3)])

    def call():
        if what == "append":
            return kvm.append(paged, step, 1, q, k, k, pos, rope)
        if what == "attend":
            return kvm.attend(paged, step, 1, q, workspace=ws)
        if what == "evict":
            return kvm.evict(paged, step.own, 0, 1, w, p, 10, workspace=es)
        return kvm.store(paged, batch)
    hidden = {"append": [step.q_start, step.group_start, paged.k_addrs, paged.v_addrs, rope.freqs],
              "attend": [step.q_start, step.group_start, paged.k_addrs, paged.v_addrs],
              "evict": [paged.k_addrs, paged.v_addrs],
              "store": [paged.k_addrs, paged.v_addrs, batch.seqs[0].chunk_addrs]}[what]
    held = {t.data_ptr() for t in hidden}
    call()                                        # loads the code
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(150):
            busy @ busy
        call()
        done.record()
    del hidden, step, rope, paged, batch, call
    new = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (2, 3, 4, 16, 64) for _ in range(300)]
    taken = {t.data_ptr() for t in new} & held
    pending = not done.query()
    torch.cuda.synchronize()
    assert pending, "the stream was not busy for long enough to tell"
    assert not taken
    assert kvm.take_faults() == 0


def test_side_streams_with_inputs_of_their_own():
    """Three streams at once, each with its own pool, inputs and workspaces, in every call; each result equals the one
    of the same call alone on the current stream, bit for bit."""
    H, rep, D = 2, 4, 128
    rope = kvm.Rope(D)

    def batch(i):
        b = su.Batch(30 + i, H, D, 16, [600 - 90 * i, 170 + i], [1, 1], [400 + 37 * i], [2], layers=1, table_room=1)
        d = dict(zip(("pool", "paged", "step"), device(b)))
        d.update(q=b.normal(2, H * rep, D).cuda(), k=b.normal(2, H, D).cuda(), v=b.normal(2, H, D).cuda(),
                 pos=torch.tensor([1000 + i, 50 * i], dtype=torch.int32).cuda(),
                 w=torch.rand((1, 2, H, 640), generator=b.g).cuda(), pw=torch.rand((1, H, 500), generator=b.g).cuda(),
                 p=torch.arange(640, dtype=torch.int32, device="cuda").expand(1, 2, H, 640).contiguous())
        d["sp"] = d["p"].clone()
        return d

    def steps(d, stream):
        d["qr"] = kvm.append(d["paged"], d["step"], 0, d["q"], d["k"], d["v"], d["pos"], rope, weights=d["w"][0],
                             slot_positions=d["sp"][0], stream=stream)
        for _ in range(4):
            d["out"], d["lse"] = kvm.attend(d["paged"], d["step"], 0, d["qr"], stream=stream)
            kvm.add_weights(d["paged"], d["step"], 0, d["qr"], d["lse"], d["w"][0], d["pw"], stream=stream)
        d["new"] = kvm.evict(d["paged"], d["step"].own, 0, 1, d["w"], d["sp"], 150, recent=9, stream=stream)

    alone, beside = [batch(i) for i in range(3)], [batch(i) for i in range(3)]
    for d in alone:
        steps(d, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in beside]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for d, st in zip(beside, streams):
        steps(d, st)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    for i, (x, y) in enumerate(zip(alone, beside)):
        for name in ("pool", "qr", "out", "lse", "w", "pw", "sp", "new"):
            a, c = x[name], y[name]
            if a.dtype == torch.bfloat16:
                a, c = a.view(torch.int16), c.view(torch.int16)
            assert torch.equal(a, c), (i, name)
    for name in ("out", "lse"):
        assert not torch.equal(alone[0][name], alone[1][name])


# Rows of many pieces: heads, rep, dim, page, lens, new, prefix, sizes, pieces a row has (of 128 tokens each)
MANY = [
    (1, 1, 64, 16, [63 * 128], [1], [], [], 63),
    (1, 4, 128, 16, [64 * 128], [1], [], [], 64),
    (1, 4, 128, 16, [64 * 128 + 1], [1], [], [], 65),
    (1, 2, 80, 16, [10200], [1], [], [], 80),
    (1, 1, 256, 256, [10001], [1], [], [], 79),
    (1, 4, 128, 16, [900], [1], [20000], [1], 157 + 8),                     # 157 of the prefix, 8 of its own
    (1, 4, 64, 16, [70] + [20, 9] * 4, [1] * 9, [20000], [9], 64),          # a wide prefix beside own pieces
    (1, 1, 64, 16, [30, 20] * 65, [1] * 130, [17000], [130], 64),           # rows enough for a join by rows
]


@pytest.mark.parametrize("case", MANY, ids=[str(i) for i in range(len(MANY))])
@pytest.mark.parametrize("value", [None, INF, NAN], ids=["finite", "inf", "nan"])
def test_attend_rows_of_many_pieces(case, value):
    """Joins of more pieces than a wave has lanes; with a value that is not finite in the last but one token, too."""
    H, rep, D, P, lens, new, prefix, sizes, pieces = case
    say("many pieces", case, value)
    b = su.Batch(26, H, D, P, lens, new, prefix, sizes, layers=2)
    q = b.normal(b.q_start[-1], H * rep, D, gain=3.0)
    if value is not None:
        b.flat()[1, 0, b.rows(b.own_table, 0, lens[0] - 1, lens[0] - 2)[0], 0, 3] = value
    pool, paged, step = device(b)
    # the workspace has a float32 pair and a float32 row for each (row, head, piece)
    assert step.attend_workspace_bytes(H * rep) // (b.q_start[-1] * H * rep * (8 + 4 * D)) >= pieces
    out, lse = kvm.attend(paged, step, 1, q.cuda(), workspace=step.new_attend_workspace(H * rep).fill_(0xFF))
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    wo, wl, eo, el = attend64(b, q, D ** -0.5, layer=1)
    within(lse, wl, el, "lse")
    within(out, wo, eo, "out")


@pytest.mark.parametrize("bound", [1, 64, 1000, 8191])
def test_attend_short_rows_under_a_long_bound(bound):
    """A capacity as the bound, as in a captured graph: rows of one token to a full one under pieces cut for 8192."""
    lens = [bound, max(1, bound // 3), 1]
    b = su.Batch(27, 1, 64, 16, lens, [1, 1, 1], [bound], [2], layers=2, table_room=512)
    q = b.normal(3, 2, 64, gain=3.0)
    pool, paged, step = device(b, max_len=8192, prefix_max=8192)
    out, lse = kvm.attend(paged, step, 1, q.cuda(), workspace=step.new_attend_workspace(2).fill_(0xFF))
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    wo, wl, eo, el = attend64(b, q, 64 ** -0.5, layer=1)
    within(lse, wl, el, "lse")
    within(out, wo, eo, "out")


# Head ratios, forms and layouts: heads, rep, dim, page, lens, new, prefix, sizes
LAYOUTS = [
    (1, 128, 64, 16, [130, 20], [2, 1], [40], [2]),                         # a KV head for 128 query heads
    (1, 64, 128, 16, [150, 3], [5, 3], [33], [1]),
    (2, 48, 80, 12, [70, 41], [1, 4], [20], [2]),
    (1, 20, 128, 16, [90], [1], [70], [1]),                                 # one token takes the wide form
    (1, 17, 256, 16, [40, 9], [1, 1], [70], [2]),
    (1, 2, 128, 16, [30, 200, 9], [1, 100, 1], [140], [1]),                 # narrow prefix beside a prompt of no group
    (2, 4, 64, 16, [30, 400], [1, 77], [300], [1]),
    (1, 1, 128, 16, [65, 64, 63, 129, 128, 127], [65, 1, 63, 2, 128, 1], [64, 63], [3, 2]),
]


@pytest.mark.parametrize("case", LAYOUTS, ids=[str(i) for i in range(len(LAYOUTS))])
@pytest.mark.parametrize("gain", [1.0, 64.0])
def test_attend_and_weights_in_more_layouts(case, gain):
    """Against 64 bits, with scores of hundreds too; tables that are views of wider ones; prefix sums alone, in place and
    from zero."""
    say("layouts", case, gain)
    H, rep, D, P, lens, new, prefix, sizes = case
    b = su.Batch(28, H, D, P, lens, new, prefix, sizes, layers=2)
    q = b.normal(b.q_start[-1], H * rep, D, gain=gain)
    pool, paged, _ = device(b)

    def view(t):
        wide = torch.full((t.shape[0], t.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
        wide[:, 2:2 + t.shape[1]] = t.cuda()
        return wide[:, 2:2 + t.shape[1]]
    own = kvm.Tables(view(b.own_table), torch.tensor(lens, dtype=torch.int32).cuda(), max(lens))
    pre = kvm.Tables(view(b.prefix_table), torch.tensor(prefix, dtype=torch.int32).cuda(), max(prefix))
    step = kvm.Step(paged, own, new, prefix=pre, group_sizes=sizes)
    out, lse = kvm.attend(paged, step, 1, q.cuda())
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    wo, wl, eo, el = su.attend64(b, q, D ** -0.5, layer=1)
    within(lse, wl, el, "lse")
    within(out, wo, eo, "out")
    w0 = torch.rand((len(lens), H, max(lens)), generator=b.g)
    p0 = torch.rand((len(prefix), H, max(prefix) + 1), generator=b.g)
    lse = wl.float()
    ww, wp, ew, ep = su.weights64(b, q, lse, D ** -0.5, w0, p0, layer=1)
    gw, gp = kvm.add_weights(paged, step, 1, q.cuda(), lse.cuda(), w0.cuda(), p0.cuda())
    within(gw, ww, ew, "weights")
    within(gp, wp, ep, "prefix weights")
    none, alone = kvm.add_weights(paged, step, 1, q.cuda(), lse.cuda(), prefix_weights=p0.cuda())
    # the same rows in the same order, but perhaps by the other form (the larger side decides it)
    assert none is None
    within(alone, wp, ep, "prefix weights alone")
    _, zero = kvm.add_weights(paged, step, 1, q.cuda(), lse.cuda(), prefix_out=torch.full(p0.shape, 9.0, device="cuda"))
    for g, n in enumerate(prefix):
        assert torch.all(zero[g, :, n:] == 9.0)
    _, z64, _, ez = su.weights64(b, q, lse, D ** -0.5, torch.zeros_like(w0), torch.zeros_like(p0), layer=1)
    # The exponential's result is 0 where it lies below float32's smallest normal number, 2^-126: each of a token's
    # weights (one per row and query head) is off by up to that, which only sums from zero show.  64 bits hold it: with
    # scores of hundreds e^(score - lse) goes down to e^-700.
    for g, n in enumerate(prefix):
        within(zero[g, :, :n], z64[g, :, :n], ez[g, :, :n] + b.q_start[-1] * rep * 2.0 ** -126, "prefix weights from zero")
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0


def test_step_calls_in_a_pool_past_4_gib():
    """Pages whose bytes lie beyond 32 bits: append, attend (narrow, wide), add_weights and evict on a slab of 4.6 GB."""
    H, rep, D, P, pages = 8, 4, 128, 16, 140000
    lens, new, prefix = [40, 90, 33], [1, 70, 1], [100]
    b = su.Batch(29, H, D, P, lens, new, prefix, [3], layers=1, table_room=1)
    # the small batch's pages, spread over the top of a large pool
    at = torch.linspace(pages - 9000, pages - 1, b.pages).long()
    pool = torch.full((1, 2, pages, P, H, D), NAN, dtype=torch.bfloat16, device="cuda")
    pool[:, :, at.cuda()] = b.pool.cuda()
    paged = kvm.Paged.from_pool(pool, chunk_size=P)

    def up(t):
        return torch.where(t >= 0, at[t.clamp(min=0).long()].int(), t).cuda()
    own = kvm.Tables(up(b.own_table), torch.tensor(lens, dtype=torch.int32).cuda(), max(lens))
    pre = kvm.Tables(up(b.prefix_table), torch.tensor(prefix, dtype=torch.int32).cuda(), max(prefix))
    small_pool, small_paged, small_step = device(b)
    step = kvm.Step(paged, own, new, prefix=pre, group_sizes=[3])
    rope = kvm.Rope(D)
    rows = b.q_start[-1]
    q, k, v = (b.normal(rows, h, D).cuda() for h in (H * rep, H, H))
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    results = []
    for pg, st, pl in ((paged, step, pool), (small_paged, small_step, small_pool)):
        w = torch.zeros((1, 3, H, max(lens)), device="cuda")
        pw = torch.zeros((1, H, 100), device="cuda")
        sp = torch.arange(max(lens), dtype=torch.int32, device="cuda").expand(1, 3, H, max(lens)).contiguous()
        qr = kvm.append(pg, st, 0, q, k, v, pos, rope, weights=w[0], slot_positions=sp[0])
        out, lse = kvm.attend(pg, st, 0, qr)
        kvm.add_weights(pg, st, 0, qr, lse, w[0], pw)
        n = kvm.evict(pg, st.own, 0, 1, w, sp, 30, recent=3)
        torch.cuda.synchronize()
        assert kvm.take_faults() == 0
        results.append([qr, out, lse, w, pw, sp, n, pl[:, :, at.cuda()] if pl is pool else pl])
    for i, (x, y) in enumerate(zip(*results)):
        if x.dtype == torch.bfloat16:
            x, y = x.view(torch.int16), y.view(torch.int16)
        assert torch.equal(x, y), i
    assert torch.isnan(pool[0, :, :pages - 9001].flatten(1)[:, ::997].float()).all()


def test_attend_of_subnormal_values_and_weights():
    """V below bf16's smallest normal number, and weights far below the largest."""
    b = su.Batch(31, 1, 128, 16, [200], [1], [50], [1], layers=2)
    f = b.flat()
    x = torch.cat([b.rows(b.own_table, 0, 200), b.rows(b.prefix_table, 0, 50)])
    f[1, 1, x] = (torch.randn((250, 1, 128), generator=b.g) * 2.0 ** -130).bfloat16()
    q = b.normal(1, 4, 128, gain=8.0)
    pool, paged, step = device(b)
    out, lse = kvm.attend(paged, step, 1, q.cuda())
    wo, wl, eo, el = su.attend64(b, q, 128 ** -0.5, layer=1)
    within(lse, wl, el, "lse")
    within(out, wo, eo, "out")


def test_two_graphs_share_a_workspace():
    """Two steps of different shapes captured with one workspace for attend and one for evict, replayed in turn with eager
    work between: each replay equals its eager calls."""
    H, rep, D = 2, 4, 128
    rope = kvm.Rope(D)
    batches = [su.Batch(33, H, D, 16, [700, 90], [1, 1], [400], [2], layers=1),
               su.Batch(34, H, D, 16, [120, 60, 33], [40, 1, 33], [90], [3], layers=1)]

    def make(b):
        pool, paged, step = device(b)
        n, cap = len(b.lens), max(b.lens)
        return {"pool": pool, "first": pool.clone(), "paged": paged, "step": step,
                "q": b.normal(b.q_start[-1], H * rep, D).cuda(), "k": b.normal(b.q_start[-1], H, D).cuda(),
                "pos": torch.arange(b.q_start[-1], dtype=torch.int32, device="cuda"),
                "qr": torch.empty((b.q_start[-1], H * rep, D), dtype=torch.bfloat16, device="cuda"),
                "out": torch.empty((b.q_start[-1], H * rep, D), dtype=torch.bfloat16, device="cuda"),
                "lse": torch.empty((b.q_start[-1], H * rep), device="cuda"),
                "w": torch.zeros((1, n, H, cap), device="cuda"),
                "p": torch.arange(cap, dtype=torch.int32, device="cuda").expand(1, n, H, cap).contiguous(),
                "ow": torch.zeros((1, n, H, 50), device="cuda"),
                "op": torch.zeros((1, n, H, 50), dtype=torch.int32, device="cuda"),
                "lens": torch.zeros(n, dtype=torch.int32, device="cuda")}

    def run(d, ws, es):
        kvm.append(d["paged"], d["step"], 0, d["q"], d["k"], d["k"], d["pos"], rope, q_out=d["qr"])
        kvm.attend(d["paged"], d["step"], 0, d["qr"], out=d["out"], lse=d["lse"], workspace=ws)
        kvm.add_weights(d["paged"], d["step"], 0, d["qr"], d["lse"], None, out=d["w"][0])
        kvm.evict(d["paged"], d["step"].own, 0, 1, d["w"], d["p"], 50, recent=5, out_weights=d["ow"], out_positions=d["op"],
                  out_lens=d["lens"], workspace=es)

    def again(d):
        d["pool"].copy_(d["first"])
        for x in ("qr", "out", "lse", "ow", "op", "lens"):
            d[x].zero_()
    sides = [make(b) for b in batches]
    ws = max((d["step"].new_attend_workspace(H * rep) for d in sides), key=lambda t: t.numel())
    es = max((d["step"].own.new_evict_workspace(d["paged"], 1, H, 50) for d in sides), key=lambda t: t.numel())
    names = ("pool", "qr", "out", "lse", "w", "ow", "op", "lens")
    want = []
    for d in sides:
        run(d, ws, es)
        want.append({x: d[x].clone() for x in names})
        again(d)
    torch.cuda.synchronize()
    graphs = []
    for d in sides:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(d, ws, es)
        graphs.append(g)
    for _ in range(4):
        for g, d, w in zip(graphs, sides, want):
            again(d)
            g.replay()
            torch.cuda.synchronize()
            for x in names:
                a, c = d[x], w[x]
                if a.dtype == torch.bfloat16:
                    a, c = a.view(torch.int16), c.view(torch.int16)
                assert torch.equal(a, c), x
            (torch.randn(512, 512, device="cuda") @ torch.randn(512, 512, device="cuda")).sum().item()
    assert kvm.take_faults() == 0
