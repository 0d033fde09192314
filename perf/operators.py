"""Cases of the linear-attention serving operators: what a pass takes, what it must give.

The operators are those of one linear-attention layer that is served next to the
gated delta rule, and of the speculative decoding step around it:

  prefill    linear attention with a decay for each head over prompts (chunked form)
  recurrent  the same attention token by token, with the compact state capture
  gated      the mixer's output norm of each head, fused with its gate
  residual   the norm after a block, its gate and residual scale, and the norm before
             the next block
  accept     verification of drafted tokens against the target's probabilities

Each case runs in a plain form (elementary torch operations in 32 bits, rounded once at
the end) or, with ``own`` true, through the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
CHUNK = 64  # tokens per chunk of the plain form


def _size(name):
    return 4 if name == "f32" else 2


# ------------------------------------------------------------------------ cases ---

def listed():
    return [
        # A short prompt pair on small heads in 32 bits: the smallest call, all latency.
        dict(name="prefill_tiny_f32", op="prefill", B=2, lo=64, hi=64, Hk=1, Hv=2, dk=32, dv=32,
             dtype="f32", gate="f32", per_head=False, state=True, shared=False),
        # One long prompt of an odd length that continues from a state: few rows, a long axis.
        dict(name="prefill_one_row", op="prefill", B=1, lo=4100, hi=4100, Hk=16, Hv=32, dk=128, dv=128,
             dtype="bf16", gate="f32", per_head=False, state=True, shared=False),
        # A batch of packed prompts of ragged lengths from empty states, one fixed decay per
        # head: the largest call.
        dict(name="prefill_packed", op="prefill", B=64, lo=500, hi=1500, Hk=16, Hv=32, dk=128, dv=128,
             dtype="bf16", gate="f32", per_head=True, state=False, shared=False),
        # Prompts that continue one shared prefix snapshot, narrow heads, three value heads per
        # key head, in fp16.
        dict(name="prefill_snapshot_f16", op="prefill", B=12, lo=200, hi=1000, Hk=2, Hv=6, dk=64, dv=64,
             dtype="f16", gate="f16", per_head=False, state=True, shared=True),
        # One decode step of a full serving batch.
        dict(name="decode_B256", op="recurrent", B=256, T=1, Hk=16, Hv=32, dk=128, dv=128,
             dtype="bf16", gate="bf16", per_head=False, capture=0),
        # The target's pass over four drafted tokens and the one before them, with capture, for
        # a few requests.
        dict(name="verify_B3_T5", op="recurrent", B=3, T=5, Hk=2, Hv=6, dk=128, dv=64,
             dtype="f16", gate="f32", per_head=True, capture=5),
        # The mixer's output norm over a whole prompt; the gate is a slice of a wider projection.
        dict(name="gated_prompt", op="gated", N=4100, H=32, D=128, dtype="bf16", weight="f32",
             act="silu", first=False, slack=4096),
        # The same at decode for a few requests, in fp16, heads of an odd size, gated before the norm.
        dict(name="gated_decode", op="gated", N=7, H=6, D=80, dtype="f16", weight="f16",
             act="sigmoid", first=True, slack=0),
        # Between two blocks over a prompt: 16-bit block output, 32-bit residual stream.
        dict(name="residual_prompt", op="residual", N=4100, D=4096, dtype="bf16", res="f32", weight="bf16",
             post=True, gate=True, scale=0.5),
        # The same at decode, without gate, an odd width, everything in 16 bits.
        dict(name="residual_decode", op="residual", N=5, D=2047, dtype="bf16", res="bf16", weight="f32",
             post=True, gate=False, scale=1.0),
        # Four drafts of each request of a serving batch; the vocabulary's size is odd.
        dict(name="accept_B128", op="accept", B=128, K=4, V=100003, dtype="f32", ragged=True, draft=True),
        # One request whose drafts come from a lookup (no draft probabilities), in bf16.
        dict(name="accept_lookup_B1", op="accept", B=1, K=7, V=32000, dtype="bf16", ragged=False, draft=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "recurrent", "gated", "residual", "accept"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    gate = rng.choice(["f32", dtype])
    if op in ("prefill", "recurrent"):
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        heads = dict(Hk=Hk, Hv=Hk * rng.choice([1, 2, 3]), dk=rng.choice([32, 64, 128, 128]),
                     dv=rng.choice([32, 64, 128, 128]), dtype=dtype, gate=gate, per_head=rng.random() < 0.4)
        if op == "recurrent":
            T = rng.choice([1, 1, 1, 2, 3, 5, 8])
            return dict(op=op, B=_log(rng, 1, 256), T=T, capture=rng.choice([0, T]), **heads)
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, min(8200, max(1, 60000 // B)))
        lo = rng.choice([hi, max(1, hi // rng.randint(2, 5))])
        state = rng.random() < 0.6
        return dict(op=op, B=B, lo=lo, hi=hi, state=state, shared=state and rng.random() < 0.3, **heads)
    if op == "gated":
        H, D = rng.choice([1, 2, 6, 16, 32]), rng.choice([32, 64, 80, 128, 128, 129, 256])
        return dict(op=op, N=_log(rng, 1, 4100 * 4096 // (H * D)), H=H, D=D, dtype=dtype, weight=gate,
                    act=rng.choice(["silu", "sigmoid"]), first=rng.random() < 0.3, slack=rng.choice([0, 8, 256, 3]))
    if op == "residual":
        D = rng.choice([_log(rng, 64, 8192), 64 * rng.randint(1, 128)])
        D = 2048 if D == 3072 else D
        return dict(op=op, N=_log(rng, 1, 4100 * 4096 // D), D=D, dtype=dtype, res=rng.choice([dtype, "f32"]),
                    weight=gate, post=rng.random() < 0.7, gate=rng.random() < 0.5, scale=rng.choice([1.0, 0.5, 0.22]))
    V = _log(rng, 1000, 200000)
    return dict(op=op, B=_log(rng, 1, max(1, min(256, 12000000 // V))), K=rng.choice([1, 2, 4, 4, 7]), V=V, dtype=dtype,
                ragged=rng.random() < 0.5, draft=rng.random() < 0.7)


def _lengths(case):
    """Tokens of each row: fixed by the case, spread over lo .. hi, the last row the longest."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [lo + (b * 7919 + 3) % (hi - lo + 1) for b in range(B - 1)] + [hi]


def work(case):
    op, e = case["op"], _size(case["dtype"])
    if op in ("prefill", "recurrent"):
        B, Hk, Hv, dk, dv = (case[n] for n in ("B", "Hk", "Hv", "dk", "dv"))
        tok = sum(_lengths(case)) if op == "prefill" else B * case["T"]
        data = tok * (2 * Hk * dk + 2 * Hv * dv) * e + (Hv if case["per_head"] else tok * Hv) * _size(case["gate"])
        st = Hv * dv * dk * 4
        if op == "prefill":
            n_in = 0 if not case["state"] else 3 if case["shared"] else B
            data += (B + min(n_in, B)) * st
        else:
            data += 2 * B * st + B * case["capture"] * (Hv + Hk * dk + Hv * dv) * 4
        return {"bytes": data, "flops": 4 * tok * Hv * dk * dv}
    if op == "gated":
        n = case["N"] * case["H"] * case["D"]
        return {"bytes": 3 * n * e, "flops": 8 * n}
    if op == "residual":
        n = case["N"] * case["D"]
        return {"bytes": n * ((3 if case["gate"] else 2) * e + 2 * _size(case["res"])), "flops": 12 * n}
    # the target's row that is sampled from, and the draft's row where there is one
    n = case["B"] * case["V"]
    return {"bytes": n * e * (2 if case["draft"] else 1), "flops": 4 * n}


# ----------------------------------------------------------------------- inputs ---

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt = "cuda", DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    op = case["op"]
    s = {"case": dict(case)}
    if op in ("prefill", "recurrent"):
        B, Hk, Hv, dk, dv = (case[n] for n in ("B", "Hk", "Hv", "dk", "dv"))
        lens = _lengths(case) if op == "prefill" else [case["T"]] * B
        tok, gt = sum(lens), DTYPES[case["gate"]]
        q, k = normal(tok, Hk, dk), normal(tok, Hk, dk)
        s["q"] = (q / (q.norm(dim=-1, keepdim=True) * dk ** 0.5)).to(dt)
        s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
        s["v"] = normal(tok, Hv, dv).to(dt)
        # a fixed decay of each head reaches from some ten tokens to some thousand; decays of
        # each token are those of the gated delta rule's layers
        s["alpha"] = (1 - 2.0 ** (-3 - 7 * uniform(Hv)) if case["per_head"]
                      else torch.exp(-(0.01 + 0.49 * uniform(tok, Hv)))).to(gt)
        s["B"], s["max_len"], s["T"] = B, max(lens), lens[0] if len(set(lens)) == 1 else None
        s["cu"] = None
        if s["T"] is None:
            s["cu"] = torch.tensor([sum(lens[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
        s["index"] = None
        if op == "prefill":
            s["state"] = None
            if case["state"]:
                s["state"] = 0.1 * normal(3 if case["shared"] else B, Hv, dv, dk)
                if case["shared"]:
                    s["index"] = torch.randint(0, 3, (B,), generator=g, device=dev, dtype=torch.int32)
        else:
            s["state"] = 0.1 * normal(B, Hv, dv, dk)
            s["count"] = torch.full((B,), case["capture"], dtype=torch.int32, device=dev)
        # the buffers that a serving program keeps for its calls
        s["final"] = torch.empty(B, Hv, dv, dk, device=dev)
        s["out"] = torch.empty_like(s["v"])
    elif op == "gated":
        N, H, D = case["N"], case["H"], case["D"]
        s["x"] = (0.3 * normal(N, H, D)).to(dt)
        wide = normal(N, H * D + case["slack"]).to(dt)
        s["z"] = wide[:, case["slack"]:].unflatten(1, (H, D))
        s["w"] = (1 + 0.1 * normal(D)).to(DTYPES[case["weight"]])
    elif op == "residual":
        N, D = case["N"], case["D"]
        s["y"] = (0.5 * normal(N, D)).to(dt)
        s["x"] = (2.0 * normal(N, D)).to(DTYPES[case["res"]])
        s["z"] = normal(N, D).to(dt) if case["gate"] else None
        s["w_post"] = (1 + 0.1 * normal(D)).to(DTYPES[case["weight"]]) if case["post"] else None
        s["w_pre"] = (1 + 0.1 * normal(D)).to(DTYPES[case["weight"]])
    else:
        B, K, V = case["B"], case["K"], case["V"]
        logits = 3 * normal(B, K + 1, V)
        s["p"] = torch.softmax(logits, -1).to(dt)
        q = torch.softmax(logits[:, :K] + 0.5 * normal(B, K, V), -1)
        # drafts drawn from the draft's distribution by its running sums
        at = torch.searchsorted(q.cumsum(-1), uniform(B, K, 1)).squeeze(-1)
        s["drafts"] = at.clamp(max=V - 1).to(torch.int32)
        s["q"] = q.to(dt) if case["draft"] else None
        s["u"] = uniform(B, K + 1)
        s["count"] = torch.randint(0, K + 1, (B,), generator=g, device=dev, dtype=torch.int32) if case["ragged"] else None
    return s


# ------------------------------------------------------------------ plain forms ---

def _segment_sums(x):
    """[..., n] -> [..., n, n]: entry (i, j) is x[j + 1] + ... + x[i] for i >= j, each sum
    formed on its own so that a short segment keeps its own precision; -inf above."""
    n = x.shape[-1]
    below = torch.ones(n, n, dtype=torch.bool, device=x.device).tril(-1)
    s = x.unsqueeze(-1).expand(*x.shape, n).masked_fill(~below, 0).cumsum(-2)
    return s.masked_fill(below.T, -math.inf)


def _linear_attention(q, k, v, alpha, cu, B, max_len, state, index):
    """S <- alpha S + v k^T, o = S q for every row, in chunks: the outputs of the packed tokens
    and the last states, in 32 bits."""
    (tok, Hk, dk), (_, Hv, dv) = q.shape, v.shape
    G, dev = Hv // Hk, q.device
    n = -(-max_len // CHUNK)
    start = torch.arange(B, device=dev) * max_len if cu is None else cu[:-1].long()
    length = torch.full((B,), max_len, device=dev) if cu is None else cu[1:].long() - start
    t = torch.arange(n * CHUNK, device=dev)
    there = t < length[:, None]
    at = (start[:, None] + t).clamp(max=tok - 1)

    def rows(x, *heads):  # [tok, heads, d] -> [B, heads, n, CHUNK, d], zeros past a row's end
        x = x.float()[at] * there[..., None, None]
        return x.unflatten(2, heads).unflatten(1, (n, CHUNK)).movedim((1, 2), (-3, -2))

    qs, ks, vs = rows(q, Hk, 1), rows(k, Hk, 1), rows(v, Hk, G)
    la = torch.log(alpha.float())
    la = la.expand(tok, Hv) if la.dim() == 1 else la
    la = torch.where(there[..., None], la[at], 0.0).unflatten(2, (Hk, G)).unflatten(1, (n, CHUNK)).movedim((1, 2), (-2, -1))
    inside = torch.exp(_segment_sums(la))
    o = (qs @ ks.transpose(-1, -2) * inside) @ vs
    added = (vs * inside[..., -1, :, None]).transpose(-1, -2) @ ks
    first = torch.zeros(B, Hv, dv, dk, device=dev) if state is None else state if index is None else state[index.long()]
    events = torch.cat([first.unflatten(1, (Hk, G)).unsqueeze(3), added], 3)
    total = torch.cat([torch.zeros_like(la[..., :1, 0]), la.sum(-1)], -1)
    carried = torch.exp(_segment_sums(total))
    states = (carried @ events.flatten(-2)).unflatten(-1, (dv, dk))
    o = o + torch.exp(la.cumsum(-1))[..., None] * (qs @ states[..., :-1, :, :].transpose(-1, -2))
    o = o.movedim((-3, -2), (1, 2)).flatten(3, 4).flatten(1, 2)
    return o[there], states[..., -1, :, :].flatten(1, 2)


def _activation(z, act):
    s = 1 / (1 + torch.exp(-z))
    return z * s if act == "silu" else s


def _rms(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _accept(p, q, drafts, u, count):
    """Tokens and their number for each request; weights in whole units of 2^-40."""
    B, K1, V = p.shape
    K, dev = K1 - 1, p.device
    count = torch.full((B,), K, device=dev) if count is None else count.long()
    step = torch.arange(K, device=dev)
    at = drafts.long().unsqueeze(-1)
    px = p[:, :K].gather(2, at).squeeze(-1).float()
    qx = torch.ones_like(px) if q is None else q.gather(2, at).squeeze(-1).float()
    good = (u[:, :K] * qx < px) & (step < count[:, None])
    n = good.long().cumprod(1).sum(1)
    rows = torch.arange(B, device=dev)
    target = p[rows, n].float()
    held = n.clamp(max=K - 1)
    other = (torch.zeros_like(target).scatter_(1, drafts[rows, held].long()[:, None], math.inf) if q is None
             else q[rows, held].float())
    other = torch.where((n < count)[:, None], other, 0.0)

    def units(x):
        return (x.clamp(0, 1) * 2.0 ** 40).to(torch.int64)

    w = units(target - other)
    w = torch.where(w.sum(1, keepdim=True) == 0, units(target), w)
    total = w.sum(1)
    # the tests' numbers are used up: given a rejection they are no longer uniform
    goal = (u[:, K].double() * total.double()).to(torch.int64).clamp(max=total - 1)
    token = (w.cumsum(1) <= goal[:, None]).sum(1)
    token = torch.where(total > 0, token, -1)
    steps = torch.arange(K1, device=dev)
    kept = torch.cat([drafts.long(), torch.full((B, 1), -1, device=dev)], 1)
    tokens = torch.where(steps < n[:, None], kept, torch.where(steps == n[:, None], token[:, None], -1))
    return tokens.to(torch.int32), (n + 1).to(torch.int32)


def _capture(s):
    """Decay, key and delta of every token as the compact capture packs them."""
    c = s["case"]
    B, T = c["B"], c["T"]
    a = s["alpha"].float().expand(B * T, c["Hv"]) if c["per_head"] else s["alpha"].float()
    return torch.cat([a, s["k"].float().flatten(1), s["v"].float().flatten(1)], 1).unflatten(0, (B, T))


# ------------------------------------------------------------------------- run ---

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(s):
    c = s["case"]
    op, dt = c["op"], DTYPES[c["dtype"]]
    if op in ("prefill", "recurrent"):
        o, last = _linear_attention(s["q"], s["k"], s["v"], s["alpha"], s["cu"], s["B"], s["max_len"], s["state"], s["index"])
        r = {"out": o.to(dt), "state": last}
        if c.get("capture"):
            r["capture"] = _capture(s)
        return r
    if op == "gated":
        x, z = s["x"].float(), _activation(s["z"].float(), c["act"])
        y = _rms(x * z) * s["w"].float() if c["first"] else _rms(x) * s["w"].float() * z
        return y.to(dt)
    if op == "residual":
        y = s["y"].float()
        if s["w_post"] is not None:
            y = _rms(y) * s["w_post"].float()
        if s["z"] is not None:
            y = y * _activation(s["z"].float(), "sigmoid")
        x = s["x"].float() + c["scale"] * y
        return {"residual": x.to(DTYPES[c["res"]]), "out": (_rms(x) * s["w_pre"].float()).to(dt)}
    tokens, emitted = _accept(s["p"], s["q"], s["drafts"], s["u"], s["count"])
    return {"tokens": tokens, "emitted": emitted}


def _run_own(s):
    from gated_deltanet_recurrence_02_gb300 import gdn
    c = s["case"]
    op = c["op"]
    if op in ("prefill", "recurrent"):
        how = gdn.GDN_ALPHA_PER_HEAD if c["per_head"] else 0
        if op == "prefill":
            o, last = gdn.gdn_linear_prefill(
                s["q"], s["k"], s["v"], s["alpha"], B=s["B"], T=s["T"], cu_seqlens=s["cu"], initial_state=s["state"],
                initial_state_indices=s["index"], final_state=s["final"], out=s["out"], conventions=how)
            return {"out": o, "state": last}
        o, last, seen = gdn.gdn_linear_recurrent(
            s["q"], s["k"], s["v"], s["alpha"], B=s["B"], T=s["T"], initial_state=s["state"], final_state=s["final"],
            out=s["out"], state_update_capacity=c["capture"], capture_count=s["count"], conventions=how)
        r = {"out": o, "state": last}
        if c["capture"]:
            r["capture"] = seen
        return r
    if op == "gated":
        act = gdn.GDN_GATE_SILU if c["act"] == "silu" else gdn.GDN_GATE_SIGMOID
        return gdn.gdn_gated_norm(s["x"], s["z"], s["w"], eps=EPS, gate=act | (gdn.GDN_GATE_FIRST if c["first"] else 0))
    if op == "residual":
        x, h = gdn.gdn_residual_norm(s["y"], s["x"], post_weight=s["w_post"], gate=s["z"], gate_act=gdn.GDN_GATE_SIGMOID,
                                     res_scale=c["scale"], pre_weight=s["w_pre"], eps=EPS)
        return {"residual": x, "out": h}
    tokens, emitted = gdn.gdn_accept_drafts(s["p"], s["q"], s["drafts"], s["u"], draft_count=s["count"])
    return {"tokens": tokens, "emitted": emitted}


# ----------------------------------------------------------------------- exact ---

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "accept":
        return None
    if op in ("prefill", "recurrent"):
        return _exact_attention(case, s)
    if op == "gated":
        out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        w = s["w"].double()
        for i in range(0, out.shape[0], 512):
            x, z = s["x"][i:i + 512].double(), s["z"][i:i + 512].double()
            a = torch.sigmoid(z) * (z if case["act"] == "silu" else 1)
            if case["first"]:
                x = x * a
            y = x * w / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["D"] + EPS)
            out[i:i + 512] = y if case["first"] else y * a
        return out
    y, x = s["y"].double(), s["x"].double()
    D = case["D"]
    if case["post"]:
        y = y * s["w_post"].double() / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / D + EPS)
    if case["gate"]:
        y = y * torch.sigmoid(s["z"].double())
    x = x + case["scale"] * y
    return {"residual": x, "out": x * s["w_pre"].double() / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)}


def _exact_attention(case, s):
    """Token after token, as the recurrence is defined, all rows at once."""
    B, Hk, Hv = case["B"], case["Hk"], case["Hv"]
    lens = _lengths(case) if case["op"] == "prefill" else [case["T"]] * B
    if max(lens) * B * Hv * case["dk"] * case["dv"] > 2e12:
        return None
    order = sorted(range(B), key=lambda b: -lens[b])  # the rows still running are the first ones
    starts = [sum(lens[:b]) for b in range(B)]
    start = torch.tensor([starts[b] for b in order], device="cuda")
    S = torch.zeros(B, Hv, case["dv"], case["dk"], dtype=torch.float64, device="cuda")
    if s["state"] is not None:
        pick = torch.tensor(order, device="cuda")
        S += s["state"].double()[pick if s["index"] is None else s["index"].long()[pick]]
    out = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    running = B
    for t in range(max(lens)):
        while running and lens[order[running - 1]] <= t:
            running -= 1
        i = start[:running] + t
        q = s["q"][i].double().repeat_interleave(Hv // Hk, 1)
        k = s["k"][i].double().repeat_interleave(Hv // Hk, 1)
        a = s["alpha"].double().expand(running, Hv) if case["per_head"] else s["alpha"][i].double()
        S[:running].mul_(a[..., None, None]).add_(s["v"][i].double()[..., None] * k[:, :, None, :])
        out[i] = (S[:running] @ q[..., None]).squeeze(-1)
    last = torch.empty_like(S)
    last[torch.tensor(order, device="cuda")] = S
    r = {"out": out, "state": last}
    if case.get("capture"):
        a = s["alpha"].double()
        a = a.expand(B * case["T"], Hv) if case["per_head"] else a
        flat = [a, s["k"].double().reshape(B * case["T"], -1), s["v"].double().reshape(B * case["T"], -1)]
        r["capture"] = torch.cat(flat, 1).reshape(B, case["T"], -1)
    return r
