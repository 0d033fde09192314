"""Cases of the cached-attention operators: what a pass takes, what it must give.

The operators are those of one softmax-attention layer that a hybrid model serves between
its linear layers, over a cache of keys and values in pages:

  rotary     rotary positions with one or several axes (time, height, width) on each head,
             and the turn back, which is its gradient
  append     the keys and values of new tokens to the paged cache, keys and queries rotated
             on the way
  attention  new tokens (one of each request, a few drafts, or a chunk of a prompt) over the
             paged cache

Each case runs in a plain form (elementary torch operations in 32 bits, angles in 64, rounded
once at the end) or, with ``own`` true, through the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SCORES = 1 << 29  # scores that the plain form of the attention holds at a time


def _size(name):
    return 4 if name == "f32" else 2


# ------------------------------------------------------------------------ cases ---

def listed():
    return [
        # Queries of a prompt of text and image patches, three axes in contiguous sections, a
        # slice of the fused projection of queries, keys and values.
        dict(name="rotary_image", op="rotary", N=4100, H=32, d=128, R=128, axes=3, cycle=False, pairs=False,
             inverse=False, start=0, theta=1000000.0, slack=2048, dtype="bf16"),
        # A few requests at decode, far into their texts: a part of each head, neighbouring
        # elements turn together. The smallest call, all latency.
        dict(name="rotary_decode", op="rotary", N=7, H=6, d=64, R=32, axes=1, cycle=False, pairs=True,
             inverse=False, start=1000000, theta=10000.0, slack=0, dtype="f16"),
        # The gradient of an image's keys in 32 bits, axes in turn along a head.
        dict(name="rotary_back_f32", op="rotary", N=2501, H=8, d=128, R=96, axes=3, cycle=True, pairs=False,
             inverse=True, start=100, theta=10000.0, slack=0, dtype="f32"),
        # A batch of ragged prompts into an empty cache, three axes.
        dict(name="append_prompts", op="append", B=16, lo=100, hi=600, old_lo=0, old_hi=0, Hq=32, Hk=8, d=128,
             R=128, axes=3, cycle=True, pairs=False, theta=1000000.0, page=64, dtype="bf16"),
        # One token of each request of a full batch, at the cache's own positions.
        dict(name="append_decode", op="append", B=256, lo=1, hi=1, old_lo=20, old_hi=300, Hq=16, Hk=2, d=128, R=64,
             axes=0, cycle=False, pairs=False, theta=10000000.0, page=16, dtype="f16"),
        # One decode step of one request: few rows, a long axis, all latency.
        dict(name="attention_decode_B1", op="attention", B=1, lo=1, hi=1, old_lo=5000, old_hi=5000, Hq=16, Hk=2, d=64,
             window=0, lse=False, page=16, dtype="bf16"),
        # One decode step of a full serving batch with ragged lengths.
        dict(name="attention_decode_B256", op="attention", B=256, lo=1, hi=1, old_lo=500, old_hi=1500, Hq=32, Hk=8,
             d=128, window=0, lse=False, page=16, dtype="bf16"),
        # The target's pass over four drafts and the token before them, six query heads a key head.
        dict(name="attention_verify", op="attention", B=12, lo=5, hi=5, old_lo=3000, old_hi=9000, Hq=12, Hk=2, d=128,
             window=0, lse=True, page=64, dtype="f16"),
        # A chunk of a long prompt over what the cache holds of it: the largest call.
        dict(name="attention_long", op="attention", B=1, lo=4100, hi=4100, old_lo=28000, old_hi=28000, Hq=32, Hk=8,
             d=128, window=0, lse=False, page=64, dtype="bf16"),
        # Ragged prompts of a batch from empty caches, narrow heads.
        dict(name="attention_prompts", op="attention", B=16, lo=200, hi=2000, old_lo=0, old_hi=0, Hq=32, Hk=4, d=64,
             window=0, lse=False, page=32, dtype="f16"),
        # A chunk of each of a few requests in a layer with a sliding window.
        dict(name="attention_window", op="attention", B=4, lo=512, hi=512, old_lo=1000, old_hi=7000, Hq=16, Hk=2,
             d=128, window=1024, lse=False, page=128, dtype="bf16"),
        # Everything in 32 bits, narrow heads, pages of an odd size.
        dict(name="attention_f32", op="attention", B=3, lo=1, hi=65, old_lo=0, old_hi=700, Hq=4, Hk=2, d=32,
             window=0, lse=True, page=20, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _turn(rng, d):
    """Rotation of a head: how many of its elements, on which axes, which ones turn together."""
    axes = rng.choice([1, 1, 2, 3, 3])
    R = rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)])
    return dict(R=R, axes=axes, cycle=rng.random() < 0.5, pairs=rng.random() < 0.4,
                theta=rng.choice([10000.0, 500000.0, 1000000.0, 10000000.0]))


def draw(rng):
    op = rng.choice(["rotary", "append", "attention", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "rotary":
        H, d = rng.choice([1, 2, 5, 8, 16, 32]), rng.choice([32, 64, 80, 128, 128, 256])
        return dict(op=op, N=_log(rng, 1, 4100 * 4096 // (H * d)), H=H, d=d, inverse=rng.random() < 0.3,
                    start=rng.choice([0, 0, 1000, 1000000]), slack=rng.choice([0, 0, 8, 1024, 3]), dtype=dtype,
                    **_turn(rng, d))
    Hk, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([32, 64, 128, 128])
    heads = dict(Hq=Hk * rng.choice([1, 2, 3, 4, 4, 6, 8]), Hk=Hk, d=d, page=rng.choice([8, 16, 16, 20, 32, 64, 128]),
                 dtype=dtype)
    if op == "append":
        turn = dict(_turn(rng, d))
        turn["axes"] = rng.choice([0, turn["axes"]])
        if rng.random() < 0.5:
            lo, hi, B = 1, rng.choice([1, 1, 2, 5]), _log(rng, 1, 256)
            old = _log(rng, 1, 400)
        else:
            B = _log(rng, 1, 32)
            hi = _log(rng, 1, max(1, 8000 // B))
            lo, old = max(1, hi // rng.randint(1, 5)), rng.choice([0, hi])
        return dict(op=op, B=B, lo=lo, hi=hi, old_lo=0, old_hi=old, **heads, **turn)
    kind = rng.choice(["decode", "decode", "verify", "chunk", "prompt"])
    room = (1 << 30) // (4 * _size(dtype) * Hk * d)  # keys of all rows
    if kind in ("decode", "verify"):
        lo = hi = 1 if kind == "decode" else rng.randint(2, 9)
        B = _log(rng, 1, 256)
        old = _log(rng, 1, max(1, min(60000, room // B)))
        old_lo = old // rng.randint(1, 4)
    else:
        pairs = 4e11 / (4 * heads["Hq"] * d) * (0.05 if dtype == "f32" else 1.0)
        B = _log(rng, 1, 16)
        hi = _log(rng, 10, max(10, min(8200, int(math.sqrt(pairs / B)))))
        lo = max(1, hi // rng.randint(1, 5))
        old = 0 if kind == "prompt" else _log(rng, 1, max(1, min(30000, int(pairs / B / hi), room // B)))
        old_lo = old // 2
    window = _log(rng, 8, 2000) if rng.random() < 0.25 else 0
    return dict(op=op, B=B, lo=lo, hi=hi, old_lo=old_lo, old_hi=old, window=window, lse=rng.random() < 0.3, **heads)


def _spread(B, lo, hi, step):
    """B whole numbers of lo .. hi, fixed by the case, the last one the largest."""
    return [lo + (b * step + 3) % (hi - lo + 1) for b in range(B - 1)] + [hi]


def _lengths(case):
    """New tokens of each row, and keys of each row with them."""
    new = _spread(case["B"], case["lo"], case["hi"], 7919)
    return new, [n + o for n, o in zip(new, _spread(case["B"], case["old_lo"], case["old_hi"], 5903))]


def _pairs(case):
    """Pairs of a query and a key that it sees, of one head; keys that any query sees."""
    new, length = _lengths(case)
    pairs = seen = 0
    w = case["window"]
    for n, m in zip(new, length):
        first = m - n + 1  # keys of the first query without a window
        if w == 0 or w >= m:
            pairs += n * (first + m) // 2
            seen += m
        else:
            short = max(0, min(n, w - first))  # queries with fewer keys than the window
            pairs += short * (2 * first + short - 1) // 2 + (n - short) * w
            seen += m - max(0, first - w)
    return pairs, seen


def work(case):
    op, e, d = case["op"], _size(case["dtype"]), case["d"]
    if op == "rotary":
        n = case["N"] * case["H"]
        return {"bytes": 2 * n * d * e + 4 * case["N"] * case["axes"], "flops": 3 * n * case["R"]}
    tok = sum(_lengths(case)[0])
    if op == "append":
        return {"bytes": 2 * tok * (case["Hq"] + 2 * case["Hk"]) * d * e + 4 * tok * case["axes"],
                "flops": 3 * tok * (case["Hq"] + case["Hk"]) * case["R"]}
    pairs, seen = _pairs(case)
    data = 2 * tok * case["Hq"] * d * e + 2 * seen * case["Hk"] * d * e
    return {"bytes": data + (4 * tok * case["Hq"] if case["lse"] else 0), "flops": 4 * d * case["Hq"] * pairs}


# ----------------------------------------------------------------------- inputs ---

def _frequencies(case):
    half = case["R"] // 2
    i = torch.arange(half, dtype=torch.float64)
    f = (case["theta"] ** (-i / half)).float().cuda()
    if case["axes"] < 2:
        return f, None
    i = torch.arange(half)
    a = i % case["axes"] if case["cycle"] else i * case["axes"] // max(half, 1)
    return f, a.to(torch.int32).cuda()


def _patches(n, axes, start):
    """Positions [axes, n] of text followed by images of 24 x 36 patches, and so on."""
    at, p, k = [[] for _ in range(axes)], start, 0
    while len(at[0]) < n:
        if k % 2 == 0:
            for i in range(37):
                for a in range(axes):
                    at[a].append(p + i)
            p += 37
        else:
            for i in range(24 * 36):
                for a, v in enumerate((0, i // 36, i % 36)[3 - axes:] if axes > 1 else (i,)):
                    at[a].append(p + v)
            p += 36
        k += 1
    return torch.tensor([x[:n] for x in at], dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    dev, dt, op, d = "cuda", DTYPES[case["dtype"]], case["op"], case["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": dict(case)}
    if op == "rotary":
        N, H = case["N"], case["H"]
        wide = normal(N, H * d + case["slack"]).to(dt)
        s["x"] = wide[:, :H * d].unflatten(1, (H, d))
        s["f"], s["axes"] = _frequencies(case)
        start = case["start"] + int(torch.randint(0, 1000, (1,), generator=host))
        s["pos"] = _patches(N, case["axes"], start).to(dev)
        return s
    B, Hq, Hk, page = (case[n] for n in ("B", "Hq", "Hk", "page"))
    new, length = _lengths(case)
    tok = sum(new)
    # pages of the rows in no order, a few of them nobody's
    need = [-(-m // page) for m in length]
    pages, width = sum(need) + 5, max(need) + 1
    order = torch.randperm(pages, generator=host)
    table = torch.zeros(B, width, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table.to(dev)
    s["len"] = torch.tensor(length, dtype=torch.int32, device=dev)
    s["T"] = new[0] if len(set(new)) == 1 else None
    s["cu"] = None
    if s["T"] is None:
        s["cu"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
    s["B"], s["most"], s["longest"] = B, max(new), max(length)
    s["kp"] = normal(pages, page, Hk, d).to(dt)
    s["vp"] = normal(pages, page, Hk, d).to(dt)
    if op == "append":
        # one projection gives queries, keys and values
        wide = normal(tok, (Hq + 2 * Hk) * d).to(dt)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in wide.split([Hq * d, Hk * d, Hk * d], 1))
        s["f"], s["axes"] = _frequencies(case)
        s["pos"] = None
        if case["axes"]:
            s["pos"] = torch.cat([_patches(n, case["axes"], m - n) for n, m in zip(new, length)], 1).to(dev)
    else:
        # a few keys of each query stand out, as they do in a trained model
        s["q"] = (1.5 * normal(tok, Hq, d)).to(dt)
        s["scale"] = d ** -0.5
    return s


# ------------------------------------------------------------------ plain forms ---

def _rotate(x, pos, f, axes, pairs, inverse):
    """x [N, H, d] with the first 2 f.numel() elements of each head turned, in 32 bits."""
    R = 2 * f.numel()
    p = pos[0][:, None] if axes is None else pos[axes.long()].T
    angle = p.double() * f.double()
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    s = -s if inverse else s
    x = x.float()
    t = x[..., :R]
    a, b = (t[..., 0::2], t[..., 1::2]) if pairs else (t[..., :R // 2], t[..., R // 2:])
    a, b = a * c - b * s, b * c + a * s
    t = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([t, x[..., R:]], -1)


def _places(s):
    """Row, cache position, page and slot of every new token."""
    case, dev = s["case"], s["table"].device
    B, page = s["B"], case["page"]
    tok = s["k"].shape[0] if "k" in s else s["q"].shape[0]
    cu = torch.arange(B + 1, device=dev) * s["T"] if s["cu"] is None else s["cu"].long()
    t = torch.arange(tok, device=dev)
    row = torch.searchsorted(cu, t, right=True) - 1
    at = s["len"].long()[row] - cu[row + 1] + t
    return row, at, s["table"][row, at // page].long(), at % page


def _append(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    _, at, page, slot = _places(s)
    pos = at[None] if s["pos"] is None else s["pos"]
    q = _rotate(s["q"], pos, s["f"], s["axes"], c["pairs"], False).to(dt)
    s["kp"][page, slot] = _rotate(s["k"], pos, s["f"], s["axes"], c["pairs"], False).to(dt)
    s["vp"][page, slot] = s["v"]
    return q


def _attention(s):
    """Outputs [tok, Hq, d] and logs of the sums of weights [tok, Hq], in 32 bits."""
    c = s["case"]
    B, Hk, d, w = s["B"], c["Hk"], c["d"], c["window"]
    G, dev = c["Hq"] // Hk, s["q"].device
    row, at, _, _ = _places(s)
    cu = torch.arange(B, device=dev) * s["T"] if s["cu"] is None else s["cu"][:-1].long()
    step = torch.arange(row.numel(), device=dev) - cu[row]
    L, M = s["longest"], s["most"]
    keys = torch.arange(L, device=dev)
    pages = s["table"][:, :-(-L // c["page"])].long()
    out = torch.empty(row.numel(), c["Hq"], d, device=dev)
    lse = torch.empty(row.numel(), c["Hq"], device=dev)
    some = max(1, min(B, SCORES // (Hk * G * M * L)))  # rows at a time
    heads = Hk if some > 1 else max(1, min(Hk, SCORES // (G * M * L)))
    for b0 in range(0, B, some):
        mine = (row >= b0) & (row < b0 + some)
        r, t = row[mine] - b0, step[mine]
        n = min(some, B - b0)
        where = torch.full((n, M), -1, device=dev).index_put((r, t), at[mine])  # cache position of each query
        see = keys <= where[..., None]
        if w:
            see &= keys > where[..., None] - w
        here = keys < s["len"][b0:b0 + n, None]
        for h in range(0, Hk, heads):
            k, v = (x[pages[b0:b0 + n], :, h:h + heads].flatten(1, 2)[:, :L].float() for x in (s["kp"], s["vp"]))
            v = v * here[..., None, None]
            q = torch.zeros(n, M, heads, G, d, device=dev)
            q[r, t] = s["q"][mine].unflatten(1, (Hk, G))[:, h:h + heads].float()
            x = torch.einsum("bthgd,bkhd->bhgtk", q * s["scale"], k)
            x = x.masked_fill(~see[:, None, None], -math.inf)
            top = x.amax(-1, keepdim=True).clamp(min=-1e30)
            x = torch.exp(x - top)
            total = x.sum(-1, keepdim=True)
            o = torch.einsum("bhgtk,bkhd->bthgd", x, v) / total.permute(0, 3, 1, 2, 4).clamp(min=1e-30)
            l = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2)
            out.unflatten(1, (Hk, G))[mine.nonzero().squeeze(-1), h:h + heads] = o[r, t]
            lse.unflatten(1, (Hk, G))[mine.nonzero().squeeze(-1), h:h + heads] = l[r, t]
    return out, lse


# ------------------------------------------------------------------------- run ---

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "rotary":
        return _rotate(s["x"], s["pos"], s["f"], s["axes"], c["pairs"], c["inverse"]).to(dt)
    if c["op"] == "append":
        return {"q": _append(s), "k_pages": s["kp"], "v_pages": s["vp"]}
    out, lse = _attention(s)
    return {"out": out.to(dt), "lse": lse} if c["lse"] else {"out": out.to(dt)}


def _run_own(s):
    from gated_deltanet_recurrence_02_gb300 import gdn
    c = s["case"]
    if c["op"] == "rotary":
        return gdn.gdn_rotary(s["x"], s["pos"], s["f"], axes=s["axes"], pairs=c["pairs"], inverse=c["inverse"])
    rows = dict(B=s["B"], T=s["T"], cu_seqlens=s["cu"])
    if c["op"] == "append":
        q = gdn.gdn_paged_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["len"], q=s["q"], inv_freq=s["f"],
                                 positions=s["pos"], axes=s["axes"], pairs=c["pairs"], **rows)
        return {"q": q, "k_pages": s["kp"], "v_pages": s["vp"]}
    out, lse = gdn.gdn_paged_attention(s["q"], s["kp"], s["vp"], s["table"], s["len"], scale=s["scale"],
                                       window=c["window"], want_lse=c["lse"], **rows)
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


# ----------------------------------------------------------------------- exact ---

def _exact_turn(x, pos, f, axes, pairs, inverse):
    """A turn as the product with a complex number of length one."""
    half = f.numel()
    x = x.double()
    angle = torch.stack([pos[0 if axes is None else int(axes[i])].double() * float(f[i]) for i in range(half)], 1)
    z = torch.polar(torch.ones_like(angle), -angle if inverse else angle)[:, None]
    first, second = (range(0, 2 * half, 2), range(1, 2 * half, 2)) if pairs else (range(half), range(half, 2 * half))
    y = torch.complex(x[..., list(first)], x[..., list(second)]) * z
    x = x.clone()
    x[..., list(first)], x[..., list(second)] = y.real, y.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_turn(s["x"], s["pos"], s["f"], s["axes"], case["pairs"], case["inverse"])
    new, length = _lengths(case)
    page, dev = case["page"], "cuda"
    start = [sum(new[:b]) for b in range(case["B"])]
    if case["op"] == "append":
        places = torch.cat([torch.arange(m - n, m) for n, m in zip(new, length)]).to(dev)
        pos = places[None] if s["pos"] is None else s["pos"]
        q, k = (_exact_turn(s[n], pos, s["f"], s["axes"], case["pairs"], False) for n in ("q", "k"))
        kp, vp = s["kp"].double(), s["vp"].double()
        for b, (n, m) in enumerate(zip(new, length)):
            at = places[start[b]:start[b] + n]
            kp[s["table"][b].long()[at // page], at % page] = k[start[b]:start[b] + n]
            vp[s["table"][b].long()[at // page], at % page] = s["v"][start[b]:start[b] + n].double()
        return {"q": q, "k_pages": kp, "v_pages": vp}
    if work(case)["flops"] > 4e12:
        return None
    Hk, G, d, w = case["Hk"], case["Hq"] // case["Hk"], case["d"], case["window"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=dev)
    for b, (n, m) in enumerate(zip(new, length)):
        mine = s["table"][b, :-(-m // page)].long()
        key = torch.arange(m, device=dev)
        rows = max(1, (1 << 28) // (m * G))
        for h in range(Hk):
            k = s["kp"][mine, :, h].reshape(-1, d)[:m].double()
            v = s["vp"][mine, :, h].reshape(-1, d)[:m].double()
            for t0 in range(0, n, rows):
                t1 = min(n, t0 + rows)
                at = torch.arange(m - n + t0, m - n + t1, device=dev)
                hidden = key > at[:, None]
                if w:
                    hidden |= key <= at[:, None] - w
                q = s["q"][start[b] + t0:start[b] + t1, h * G:(h + 1) * G].double().transpose(0, 1)
                x = (q @ k.T).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
                l = torch.logsumexp(x, -1)
                o = torch.exp(x.sub_(l[..., None])) @ v
                out[start[b] + t0:start[b] + t1, h * G:(h + 1) * G] = o.transpose(0, 1)
                lse[start[b] + t0:start[b] + t1, h * G:(h + 1) * G] = l.T
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
