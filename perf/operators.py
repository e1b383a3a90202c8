"""Cases of the packed-batch operators: what serving a SALA layer group for requests of different
lengths calls.

  qk_norm   QK-RMSNorm of packed tokens, with RoPE where positions are given
  dense     causal softmax attention over packed prompts, grouped heads, sigmoid gate
  linear    linear attention with a decay for each head over packed prompts, states in a slot pool
  step      the same for one token of each request, states updated in place
  prefix    one decode token of each request of a batch whose requests share a prefix

``run`` computes them in elementary torch operations (``own`` false) or through the library.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch of the sparse layer: 8 tokens, no RoPE; the smallest call there is
        {"name": "qk_norm_decode8", "op": "qk_norm", "tokens": 8, "hq": 32, "hk": 2, "d": 128, "rope": False},
        # q and k of a linear layer for a 32K packed prefill, RoPE at far positions
        {"name": "qk_norm_rope_32k", "op": "qk_norm", "tokens": 32768, "hq": 32, "hk": 32, "d": 128, "rope": True},
        # a handful of short prompts on the small configuration (4 heads of 64)
        {"name": "dense_short", "op": "dense", "tokens": 333, "seqs": 6, "hq": 4, "hkv": 1, "d": 64},
        # an ordinary prefill batch of the layer group's sparse layer: 16 prompts, ragged
        {"name": "dense_ragged_16k", "op": "dense", "tokens": 16384, "seqs": 16, "hq": 32, "hkv": 2, "d": 128},
        # one 32K prompt: the largest
        {"name": "dense_one_32k", "op": "dense", "tokens": 32768, "seqs": 1, "hq": 32, "hkv": 2, "d": 128},
        # ragged prompts through a linear layer, states resumed from the pool
        {"name": "linear_ragged_9k", "op": "linear", "tokens": 9001, "seqs": 13, "h": 32, "d": 128},
        # one long prompt through a linear layer, which only its heads and columns can share out
        {"name": "linear_one_64k", "op": "linear", "tokens": 65536, "seqs": 1, "h": 32, "d": 128},
        # single tokens of 4 requests on the small configuration: latency
        {"name": "step_4", "op": "step", "rows": 4, "h": 4, "d": 64},
        # single tokens of a full serving batch
        {"name": "step_256", "op": "step", "rows": 256, "h": 32, "d": 128},
        # a few requests with a short common instruction, small configuration
        {"name": "prefix_small", "op": "prefix", "rows": 5, "prefix": 700, "cap": 192, "hq": 4, "hkv": 1, "d": 64},
        # many requests over one long document
        {"name": "prefix_64x32k", "op": "prefix", "rows": 64, "prefix": 32768, "cap": 1024, "hq": 32, "hkv": 2, "d": 128},
        # few requests, shorter prefix, long histories of their own
        {"name": "prefix_own_long", "op": "prefix", "rows": 12, "prefix": 1000, "cap": 16384, "hq": 32, "hkv": 8, "d": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.5e12, w["flops"] / 1.4e15)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["qk_norm", "dense", "dense", "linear", "linear", "step", "prefix", "prefix"])
        d = rng.choice([64, 128, 128])
        hkv = rng.choice([1, 2, 3, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8, 16])
        if op == "qk_norm":
            c = {"op": op, "tokens": _log(rng, 1, 32768), "hq": hq, "hk": rng.choice([hkv, hq]), "d": d,
                 "rope": rng.random() < 0.6}
        elif op == "dense":
            c = {"op": op, "tokens": _log(rng, 1, 24000), "seqs": _log(rng, 1, 64), "hq": hq, "hkv": hkv, "d": d}
        elif op == "linear":
            c = {"op": op, "tokens": _log(rng, 1, 60000), "seqs": _log(rng, 1, 64),
                 "h": rng.choice([4, 8, 24, 32]), "d": d}
        elif op == "step":
            c = {"op": op, "rows": _log(rng, 1, 256), "h": rng.choice([4, 8, 24, 32]), "d": d}
        else:
            c = {"op": op, "rows": _log(rng, 1, 128), "prefix": _log(rng, 1, 32768), "cap": 64 * _log(rng, 1, 128),
                 "hq": hq, "hkv": hkv, "d": d}
        if _cost(c) <= most and _elements(c) <= 3.0e8:
            return c


def _elements(case):
    """Values of the largest tensor of a case (keeps drawn states well inside the card)."""
    op, d = case["op"], case["d"]
    if op == "qk_norm":
        return case["tokens"] * max(case["hq"], case["hk"]) * d
    if op == "dense":
        return case["tokens"] * case["hq"] * d
    if op == "linear":
        return max(case["tokens"] * case["h"] * d, case["seqs"] * case["h"] * d * d)
    if op == "step":
        return case["rows"] * case["h"] * d * d
    return max(case["rows"] * case["cap"] * case["hkv"] * d, case["rows"] * case["hq"] * case["prefix"])


def _lengths(tokens, seqs):
    """`seqs` lengths that sum to `tokens`: a few long ones, many short ones, an empty one and one of
    a single token where there is room."""
    r = random.Random(7919 * tokens + seqs)
    if seqs == 1:
        return [tokens]
    w = [math.exp(r.gauss(0.0, 1.2)) for _ in range(seqs)]
    if seqs >= 4:
        w[1] = 0.0
    n = [int(tokens * x / sum(w)) for x in w]
    if seqs >= 4 and n[2] > 1:
        n[0] += n[2] - 1
        n[2] = 1
    n[-1] += tokens - sum(n)
    return n


def _own_lengths(rows, cap):
    """Tokens that each request has behind the prefix already, 0 .. cap - 1 (the call adds one)."""
    r = random.Random(104729 * rows + cap)
    n = [r.randrange(cap) for _ in range(rows)]
    n[0] = cap - 1
    if rows > 1:
        n[1] = 0
    return n


def work(case):
    op, d = case["op"], case["d"]
    if op == "qk_norm":
        el = case["tokens"] * (case["hq"] + case["hk"]) * d
        return {"bytes": 4 * el + 4 * case["tokens"] * case["rope"], "flops": 10 * el}
    if op == "dense":
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        pairs = sum(n * (n + 1) // 2 for n in _lengths(t, case["seqs"]))
        return {"bytes": 2 * t * d * (3 * hq + 2 * hkv), "flops": 4 * d * hq * pairs}
    if op == "linear":
        t, h = case["tokens"], case["h"]
        return {"bytes": 10 * t * h * d + 8 * case["seqs"] * h * d * d, "flops": 4 * t * h * d * d}
    if op == "step":
        b, h = case["rows"], case["h"]
        return {"bytes": 8 * b * h * d * d + 10 * b * h * d, "flops": 5 * b * h * d * d}
    b, hq, hkv, p = case["rows"], case["hq"], case["hkv"], case["prefix"]
    held = sum(_own_lengths(b, case["cap"]))
    return {"bytes": 4 * d * hkv * (p + held) + 6 * b * hq * d + 8 * b * hkv * d,
            "flops": 4 * d * hq * (b * (p + 1) + held)}


# --------------------------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _normed(g, *shape):
    """Rows as QK-RMSNorm leaves them: root mean square 1."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True))).to(torch.bfloat16)


def _starts(lengths):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device=DEV)


def _decays(h):
    return torch.tensor([1.0 - 2.0 ** (-5.0 - i / 4.0) for i in range(h)], dtype=torch.float32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, d = case["op"], case["d"]
    s = {"op": op}
    if op == "qk_norm":
        t = case["tokens"]
        s["q"] = _normal(g, t, case["hq"], d)
        s["k"] = _normal(g, t, case["hk"], d)
        s["wq"], s["wk"] = (1.0 + 0.1 * torch.randn((d,), generator=g, device=DEV) for _ in range(2))
        s["pos"] = None
        if case["rope"]:
            first = torch.randint(0, 1 << 20, (1,), generator=g, device=DEV)
            s["pos"] = (first + torch.arange(t, device=DEV)).to(torch.int32)
        return s
    if op == "dense":
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        s["len"] = _lengths(t, case["seqs"])
        s["q"], s["k"] = _normed(g, t, hq, d), _normed(g, t, hkv, d)
        s["v"], s["gate"] = _normal(g, t, hkv, d), _normal(g, t, hq, d)
        s["cu"] = _starts(s["len"])
        return s
    if op in ("linear", "step"):
        t, h = case["tokens"] if op == "linear" else case["rows"], case["h"]
        n = case["seqs"] if op == "linear" else case["rows"]
        s["q"], s["k"] = _normed(g, t, h, d), _normed(g, t, h, d)
        s["v"], s["gate"] = _normal(g, t, h, d), _normal(g, t, h, d)
        s["lam"] = _decays(h)
        s["state"] = torch.randn((n, h, d, d), generator=g, device=DEV, dtype=torch.float32)
        s["slots"] = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
        if op == "linear":
            s["len"] = _lengths(t, n)
            s["cu"] = _starts(s["len"])
            s["state_out"] = torch.zeros_like(s["state"])
        return s
    b, hq, hkv, cap = case["rows"], case["hq"], case["hkv"], case["cap"]
    s["q"], s["k"] = _normed(g, b, hq, d), _normed(g, b, hkv, d)
    s["v"], s["gate"] = _normal(g, b, hkv, d), _normal(g, b, hq, d)
    s["pk"], s["pv"] = _normed(g, case["prefix"], hkv, d), _normal(g, case["prefix"], hkv, d)
    s["kc"], s["vc"] = _normed(g, b, cap, hkv, d), _normal(g, b, cap, hkv, d)
    s["lens"] = torch.tensor(_own_lengths(b, cap), dtype=torch.int32, device=DEV)
    s["slots"] = torch.randperm(b, generator=g, device=DEV).to(torch.int32)
    return s


# ---------------------------------------------------------------------------------- plain forms

def _gated(o, gate):
    return (o / (1.0 + torch.exp(-gate.float()))).to(torch.bfloat16)


def _plain_norm(x, w, pos):
    x = x.float()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    if pos is not None:
        d = x.shape[-1]
        theta = 10000.0 ** (-2.0 * torch.arange(d // 2, device=x.device, dtype=torch.float64) / d)
        a = pos.double()[:, None, None] * theta
        c, s = torch.cos(a).float(), torch.sin(a).float()
        lo, hi = y[..., :d // 2], y[..., d // 2:]
        y = torch.cat([lo * c - hi * s, hi * c + lo * s], -1)
    return y.to(torch.bfloat16)


def _attend(q, k, v, keep, scale):
    """q [hkv, rows, d], k and v [hkv, keys, d], keep [rows, keys] (or None): [hkv, rows, d]."""
    x = torch.matmul(q, k.transpose(-1, -2)) * scale
    if keep is not None:
        x = torch.where(keep, x, torch.full((), -math.inf, device=x.device))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return torch.matmul(p, v) / p.sum(-1, keepdim=True)


def _plain_dense(s):
    t, hq, d = s["q"].shape
    hkv = s["k"].shape[1]
    grp = hq // hkv
    o = torch.empty((t, hq, d), dtype=torch.float32, device=s["q"].device)
    at = 0
    for n in s["len"]:
        step = max(1, (1 << 28) // max(1, n * hq))       # rows at a time: the scores of all would not fit
        for r0 in range(0, n, step):
            r1 = min(n, r0 + step)
            q = s["q"][at + r0:at + r1].float().view(r1 - r0, hkv, grp, d).permute(1, 0, 2, 3)
            k, v = (s[x][at:at + r1].float().transpose(0, 1) for x in ("k", "v"))
            row = torch.arange(r0, r1, device=q.device).repeat_interleave(grp)
            keep = torch.arange(r1, device=q.device)[None, :] <= row[:, None]
            x = _attend(q.reshape(hkv, -1, d), k, v, keep, d ** -0.5)
            o[at + r0:at + r1] = x.view(hkv, r1 - r0, grp, d).permute(1, 0, 2, 3).reshape(r1 - r0, hq, d)
        at += n
    return _gated(o, s["gate"])


def _plain_linear(s):
    """Chunks of 64 tokens of all sequences at once: each chunk's own part, and its entering state as a
    decayed sum over the earlier chunks of its sequence."""
    chunk = 64
    q, lam, dev = s["q"], s["lam"].double(), s["q"].device
    t, h, d = q.shape
    n = torch.tensor(s["len"], device=dev)
    cu = s["cu"].long()
    per = torch.div(n + chunk - 1, chunk, rounding_mode="floor")
    nch = sum((x + chunk - 1) // chunk for x in s["len"])
    seq = torch.repeat_interleave(torch.arange(len(s["len"]), device=dev), per, output_size=nch)
    within = torch.arange(nch, device=dev) - (torch.cumsum(per, 0) - per)[seq]
    first = within * chunk                                             # first token, in its sequence
    size = torch.minimum(n[seq] - first, torch.full((), chunk, device=dev))
    j = torch.arange(chunk, device=dev)
    real = j[None, :] < size[:, None]                                  # [nch, chunk]
    tok = torch.where(real, (cu[seq] + first)[:, None] + j, 0)
    def take(x):
        return torch.where(real[:, None, :, None], x.float()[tok].transpose(1, 2), torch.zeros((), device=dev))
    qc, kc, vc = take(s["q"]), take(s["k"]), take(s["v"])              # [nch, h, chunk, d]
    # powers of the decays, in 64 bits: the exponents reach the sequence's length
    def power(e):
        return torch.where(e >= 0, lam[:, None, None] ** e.clamp(min=0).double(), 0.0).float()
    inner = power((j[:, None] - j[None, :])[None])                     # [h, chunk, chunk], zero above the diagonal
    o = torch.matmul(torch.matmul(qc, kc.transpose(-1, -2)) * inner, vc)
    left = power((size[:, None] - 1 - j[None, :])[None])               # [h, nch, chunk]: from token j to the chunk's end
    own_sum = torch.matmul((kc * left.transpose(0, 1)[..., None]).transpose(-1, -2), vc)   # [nch, h, d, d]
    flat = own_sum.transpose(0, 1).reshape(h, nch, d * d)
    init = s["state"][s["slots"].long()]                               # [seqs, h, d, d]
    init_flat = init.transpose(0, 1).reshape(h, -1, d * d)
    end = first + size
    gap = torch.where((seq[:, None] == seq[None, :]) & (within[:, None] > within[None, :]),
                      first[:, None] - end[None, :], -1)               # tokens between chunk b's end and chunk a
    enter = torch.matmul(power(gap[None]), flat)
    enter = enter + power(first[None, None])[:, 0, :, None] * init_flat[:, seq]
    enter = enter.view(h, nch, d, d).transpose(0, 1)
    o = o + torch.matmul(qc, enter) * power((j + 1)[None, None])[None, :, 0, :, None]
    out = torch.empty((t + 1, h, d), dtype=torch.float32, device=dev)   # the last row takes what pads the chunks
    out[torch.where(real, tok, t)] = o.transpose(1, 2)
    own_seq = torch.arange(len(s["len"]), device=dev)
    tail = torch.where(seq[None, :] == own_seq[:, None], n[:, None] - end[None, :], -1)
    final = torch.matmul(power(tail[None]), flat) + power(n[None, None])[:, 0, :, None] * init_flat
    state = s["state_out"]
    state[s["slots"].long()] = final.view(h, -1, d, d).transpose(0, 1)
    return _gated(out[:t], s["gate"]), state


def _plain_step(s):
    at = s["slots"].long()
    q, k, v = (s[x].float() for x in ("q", "k", "v"))
    new = s["state"][at] * s["lam"][None, :, None, None] + k[..., :, None] * v[..., None, :]
    s["state"][at] = new
    o = (q[..., :, None] * new).sum(-2)
    return _gated(o, s["gate"]), s["state"]


def _plain_prefix(s):
    b, hq, d = s["q"].shape
    hkv, cap = s["k"].shape[1], s["kc"].shape[1]
    grp = hq // hkv
    at, lens = s["slots"].long(), s["lens"].long()
    s["kc"][at, lens] = s["k"]
    s["vc"][at, lens] = s["v"]
    q = s["q"].float().view(b, hkv, grp, d)
    pk, pv = (s[x].float().transpose(0, 1) for x in ("pk", "pv"))       # [hkv, prefix, d]
    kc, vc = (s[x][at].float().transpose(1, 2) for x in ("kc", "vc"))   # [b, hkv, cap, d]
    x1 = torch.matmul(q.transpose(0, 1).reshape(hkv, b * grp, d), pk.transpose(-1, -2)) * d ** -0.5
    x1 = x1.view(hkv, b, grp, -1).transpose(0, 1)
    x2 = torch.matmul(q, kc.transpose(-1, -2)) * d ** -0.5
    held = torch.arange(cap, device=q.device) <= lens[:, None]
    x2 = torch.where(held[:, None, None, :], x2, torch.full((), -math.inf, device=q.device))
    m = torch.maximum(x1.amax(-1, keepdim=True), x2.amax(-1, keepdim=True))
    p1, p2 = torch.exp(x1 - m), torch.exp(x2 - m)
    o1 = torch.matmul(p1.transpose(0, 1).reshape(hkv, b * grp, -1), pv).view(hkv, b, grp, d).transpose(0, 1)
    o = (o1 + torch.matmul(p2, vc)) / (p1.sum(-1, keepdim=True) + p2.sum(-1, keepdim=True))
    return _gated(o.reshape(b, hq, d), s["gate"]), s["kc"], s["vc"]


def _plain(s):
    if s["op"] == "qk_norm":
        return _plain_norm(s["q"], s["wq"], s["pos"]), _plain_norm(s["k"], s["wk"], s["pos"])
    return {"dense": _plain_dense, "linear": _plain_linear, "step": _plain_step, "prefix": _plain_prefix}[s["op"]](s)


def _library(s):
    from hybrid_sparse_linear_lightning_b200 import sala
    op = s["op"]
    if op == "qk_norm":
        return sala.qk_norm(s["q"], s["k"], s["wq"], s["wk"], s["pos"])
    if op == "dense":
        return sala.dense_prefill(s["q"], s["k"], s["v"], s["gate"], s["cu"])
    if op == "linear":
        out = sala.linear_packed_prefill(s["q"], s["k"], s["v"], s["gate"], s["lam"], s["cu"], slots=s["slots"],
                                         state_in=s["state"], state_out=s["state_out"])
        return out, s["state_out"]
    if op == "step":
        out = sala.linear_packed_step(s["q"], s["k"], s["v"], s["gate"], s["lam"], s["state"], slots=s["slots"])
        return out, s["state"]
    out = sala.prefix_decode(s["q"], s["k"], s["v"], s["gate"], s["pk"], s["pv"], s["kc"], s["vc"], s["lens"],
                             slots=s["slots"])
    return out, s["kc"], s["vc"]


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------- exact

def _sigmoid64(x):
    return torch.sigmoid(x.double())


def _exact_norm(x, w, pos):
    x = x.double()
    d = x.shape[-1]
    y = torch.nn.functional.normalize(x, dim=-1, eps=0.0)               # x / |x|; eps folded in below
    ss = x.square().sum(-1, keepdim=True)
    y = y * (ss / (ss / d + 1e-6)).sqrt() * w.double()
    if pos is not None:
        i = torch.arange(d // 2, device=x.device, dtype=torch.float64)
        turn = torch.polar(torch.ones((), device=x.device, dtype=torch.float64).expand(pos.numel(), d // 2),
                           pos.double()[:, None] * torch.exp(i * (-2.0 / d * math.log(10000.0))))
        z = torch.complex(y[..., :d // 2].contiguous(), y[..., d // 2:].contiguous()) * turn[:, None, :]
        y = torch.cat([z.real, z.imag], -1)
    return y


def _exact_rows(q, k, v, visible):
    """One kv head: q [rows, d], k and v [keys, d], each row seeing its first `visible` keys."""
    x = (q @ k.T) / math.sqrt(q.shape[-1])
    x.masked_fill_(torch.arange(k.shape[0], device=q.device)[None, :] >= visible[:, None], -math.inf)
    return torch.softmax(x, -1) @ v


def _exact_dense(s):
    t, hq, d = s["q"].shape
    hkv = s["k"].shape[1]
    grp = hq // hkv
    out = torch.empty((t, hq, d), dtype=torch.float64, device=DEV)
    cu = s["cu"].tolist()
    for a, z in zip(cu[:-1], cu[1:]):
        rows = max(1, (1 << 27) // max(1, z - a))
        for h in range(hq):
            k, v = s["k"][a:z, h // grp].double(), s["v"][a:z, h // grp].double()
            for r in range(a, z, rows):
                e = min(z, r + rows)
                seen = torch.arange(r - a + 1, e - a + 1, device=DEV)
                out[r:e, h] = _exact_rows(s["q"][r:e, h].double(), k[:e - a], v[:e - a], seen)
    return out * _sigmoid64(s["gate"])


def _exact_linear(s):
    """The recurrence itself, token by token, all heads at once and all sequences that still have tokens."""
    t, h, d = s["q"].shape
    cu = s["cu"].tolist()
    lens = [z - a for a, z in zip(cu[:-1], cu[1:])]
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    S = s["state"][s["slots"].long()][order].double()
    start = torch.tensor([cu[i] for i in order], device=DEV)
    lam = s["lam"].double()[None, :, None, None]
    out = torch.empty((t, h, d), dtype=torch.float64, device=DEV)
    live = len(order)
    for u in range(max(lens)):
        while lens[order[live - 1]] <= u:
            live -= 1
        rows = start[:live] + u
        now = S[:live]
        now.mul_(lam)
        k, v, q = (s[x][rows].double() for x in ("k", "v", "q"))
        now.addcmul_(k[..., :, None], v[..., None, :])
        out[rows] = torch.matmul(q[..., None, :], now)[..., 0, :]
    state = torch.zeros_like(s["state"], dtype=torch.float64)
    state[s["slots"].long()[torch.tensor(order, device=DEV)]] = S
    return out * _sigmoid64(s["gate"]), state


def _exact_step(s):
    S = s["state"].double()
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for i, slot in enumerate(s["slots"].tolist()):
        S[slot] = s["lam"].double()[:, None, None] * S[slot] + torch.einsum("hi,hj->hij", s["k"][i].double(),
                                                                           s["v"][i].double())
        o[i] = torch.einsum("hi,hij->hj", s["q"][i].double(), S[slot])
    return o * _sigmoid64(s["gate"]), S


def _exact_prefix(s):
    b, hq, d = s["q"].shape
    hkv = s["k"].shape[1]
    grp = hq // hkv
    kc, vc = s["kc"].double(), s["vc"].double()
    pk, pv = s["pk"].double(), s["pv"].double()
    out = torch.empty((b, hq, d), dtype=torch.float64, device=DEV)
    for i, (slot, n) in enumerate(zip(s["slots"].tolist(), s["lens"].tolist())):
        kc[slot, n], vc[slot, n] = s["k"][i].double(), s["v"][i].double()
        for g in range(hkv):
            k = torch.cat([pk[:, g], kc[slot, :n + 1, g]])
            v = torch.cat([pv[:, g], vc[slot, :n + 1, g]])
            q = s["q"][i, g * grp:(g + 1) * grp].double()
            out[i, g * grp:(g + 1) * grp] = _exact_rows(q, k, v, torch.full((grp,), k.shape[0], device=DEV))
    return out * _sigmoid64(s["gate"]), kc, vc


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "qk_norm":
        return _exact_norm(s["q"], s["wq"], s["pos"]), _exact_norm(s["k"], s["wk"], s["pos"])
    return {"dense": _exact_dense, "linear": _exact_linear, "step": _exact_step, "prefix": _exact_prefix}[s["op"]](s)
