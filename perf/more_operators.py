"""Cases of the gated delta rule (prompts, and one token a row) and of the norms around a layer
(gated, and with the residual). Each has a plain form (elementary torch operations in 32 bits,
rounded once at the end) and the framework's call (``own``)."""

import math

import torch

own = False

W = 4            # taps of the convolution before the delta rule
L = 3            # its state: the taps before the newest input
CHUNK = 64       # tokens a block of the plain delta rule
EPS = 1e-6       # of every norm


# ---------------------------------------------------------------------------- the cases

def listed():
    return [
        # one short prompt of odd length, 2048 channels, as many query heads as value heads: latency
        dict(name="rule_one_short", op="rule", lens="37", heads=16, head=128, keys=128, groups=16, initial=False),
        # ordinary ragged batch with an empty and a one-token sequence, small heads, shared queries and keys, half of it continued
        dict(name="rule_ragged", op="rule", lens="512,1,0,129,384,77,1024,250", heads=48, head=64, keys=64, groups=8, initial=True),
        # one long document: few heads for the card, one sequence
        dict(name="rule_long", op="rule", lens="16384", heads=32, head=128, keys=128, groups=16, initial=False),
        # the prefill benchmark's batch (8 x 4096 tokens, 4096 channels)
        dict(name="rule_batch", op="rule", lens="4096,4096,4096,4096,4096,4096,4096,4096", heads=32, head=128, keys=128, groups=16, initial=False),
        # a single user's token: latency
        dict(name="step_one_row", op="step", rows=1, slots=8, heads=16, head=128, keys=128, groups=16, padding=0),
        # the strided decode batch (64 rows, 6144 channels of values) on permuted slots, eight groups
        dict(name="step_strided", op="step", rows=64, slots=64, heads=96, head=64, keys=64, groups=8, padding=0),
        # the paged decode batch (256 rows, 8192 channels of values, a tenth of the rows padding)
        dict(name="step_paged", op="step", rows=256, slots=320, heads=64, head=128, keys=128, groups=32, padding=26),
        # behind the recurrence: one token's heads, normed and gated
        dict(name="gated_one_token", op="gated", rows=1, heads=16, head=128, weights="head", first=True),
        # behind the scan, whose gate comes before the norm: 8 groups of 1024 channels, a weight a channel, a ragged batch
        dict(name="gated_groups", op="gated", rows=2377, heads=8, head=1024, weights="channel", first=False),
        # the prefill benchmark's batch, heads of 128
        dict(name="gated_batch", op="gated", rows=32768, heads=32, head=128, weights="head", first=True),
        # a decode batch's residual stream in BF16, as wide as the benchmark's
        dict(name="residual_decode", op="residual", rows=64, width=16384, wide=False, post=False, scale=1.0),
        # the prefill benchmark's batch, residual in FP32, the block's output normed too and scaled
        dict(name="residual_batch", op="residual", rows=32768, width=4096, wide=True, post=True, scale=0.5),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total):
    """Up to 24 lengths that sum to `total`, and an empty or a one-token one among them."""
    count = _spread(rng, 1, 24)
    cuts = sorted(rng.randint(0, total) for _ in range(count - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if count > 3:
        lens.insert(rng.randrange(count), rng.randint(0, 1))
    return ",".join(str(n) for n in lens)


def draw(rng):
    op = rng.choice(("rule", "rule", "step", "gated", "residual"))
    if op == "gated":
        heads, head = _spread(rng, 1, 64), rng.choice((128, 64, 256, 96, 1024, 8 * _spread(rng, 1, 512), _spread(rng, 1, 2000)))
        return dict(op=op, rows=_spread(rng, 1, max(1, min(32768, (1 << 27) // (heads * head)))), heads=heads, head=head,
                    weights=rng.choice(("head", "channel")), first=rng.random() < 0.5)
    if op == "residual":
        width = rng.choice((8 * _spread(rng, 64, 2048), 1024 * rng.choice((1, 2, 4, 8)), _spread(rng, 50, 5000)))
        return dict(op=op, rows=_spread(rng, 1, max(1, min(32768, (1 << 27) // width))), width=width, wide=rng.random() < 0.5,
                    post=rng.random() < 0.5, scale=rng.choice((1.0, 0.5, 0.22)))
    groups = rng.choice((1, 2, 8, 16))
    sizes = dict(heads=groups * max(1, _spread(rng, 4, 64) // groups), head=rng.choice((128, 128, 64, 96, 256, 40)),
                 keys=rng.choice((128, 128, 64, 32, 96, 40)), groups=groups)
    inner = sizes["heads"] * max(sizes["head"], 128) * 128
    if op == "rule":
        return dict(op=op, lens=_lens(rng, _spread(rng, 5, max(8, min(16384, (1 << 33) // inner)))), initial=rng.random() < 0.5, **sizes)
    rows = _spread(rng, 1, max(2, min(256, (1 << 28) // inner)))
    return dict(op=op, rows=rows, slots=rows + rng.randint(0, 40), padding=rng.randint(0, rows // 5), **sizes)


# ---------------------------------------------------------------------------- their inputs

def _lengths(case):
    return [int(n) for n in case["lens"].split(",")]


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _chunks(lens):
    """Blocks of up to CHUNK tokens that stay inside a sequence, the first of every sequence before all second ones, and so on: their
    sequences, first tokens and sizes, and how many sequences have an i-th block (the longest sequences come first)."""
    at = _offsets(lens)
    order = sorted(range(len(lens)), key=lambda b: -lens[b])
    table, live = [], []
    for c in range(0, max(lens), CHUNK):
        rows = [(b, at[b] + c, min(CHUNK, lens[b] - c)) for b in order if lens[b] > c]
        live.append(len(rows))
        table += rows
    return order, live, torch.tensor(table, device="cuda").t().contiguous()


def _maker(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _uniform(g, lo, hi, *shape):
    return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo


def prepare(case, seed):
    g = _maker(seed)
    op = case["op"]
    if op == "gated":
        T, H, P = case["rows"], case["heads"], case["head"]
        weight = 1 + _normal(g, *((H, P) if case["weights"] == "channel" else (P,)), scale=0.1)
        # z sits in the layer's projection, with the block's inputs beside it
        wide = _normal(g, T, 2 * H * P)
        return dict(case=case, x=_normal(g, T, H, P, scale=0.3), z=wide[:, H * P:].unflatten(1, (H, P)), weight=weight)
    if op == "residual":
        T, D = case["rows"], case["width"]
        return dict(case=case, x=_normal(g, T, D, scale=0.5), residual=_normal(g, T, D, scale=2.0, dtype=torch.float32 if case["wide"] else torch.bfloat16),
                    weight=1 + _normal(g, D, scale=0.1), post=1 + _normal(g, D, scale=0.1) if case["post"] else None)
    H, P, K, G = case["heads"], case["head"], case["keys"], case["groups"]
    rows = sum(_lengths(case)) if op == "rule" else case["rows"]
    channels = 2 * G * K + H * P
    # one row of the layer's in-projection: q k v | a b, padded to whole 16-byte vectors
    proj = _normal(g, rows, (channels + 2 * H + 7) // 8 * 8)
    # per head: A < 0, and a bias that puts softplus(a) in 0.001..0.1
    step = torch.exp(_uniform(g, math.log(1e-3), math.log(1e-1), H))
    s = dict(case=case, A=-_uniform(g, 1.0, 16.0, H), dt_bias=step + torch.log(-torch.expm1(-step)),
             a=proj[:, channels:channels + H], b=proj[:, channels + H:channels + 2 * H])
    qkv = proj[:, :channels]
    if op == "rule":
        lens = _lengths(case)
        B = len(lens)
        qkv = torch.nn.functional.silu(qkv)  # what the convolution's activation leaves
        order, live, chunks = _chunks(lens)
        s.update(q=qkv[:, :G * K].unflatten(1, (G, K)), k=qkv[:, G * K:2 * G * K].unflatten(1, (G, K)),
                 v=qkv[:, 2 * G * K:].unflatten(1, (H, P)), lens=lens, order=order, live=live, chunks=chunks,
                 cu=torch.tensor(_offsets(lens), dtype=torch.int32, device="cuda"),
                 slots=torch.randperm(B + 3, generator=g, device="cuda")[:B].to(torch.int32),
                 state=_normal(g, B + 3, H, P, K, scale=0.05, dtype=torch.float32),
                 has=(torch.arange(B, device="cuda", dtype=torch.int32) % 2 == 0).to(torch.int32) if case["initial"] else None)
        return s
    N, S = rows, case["slots"]
    slots = torch.randperm(S, generator=g, device="cuda")[:N].to(torch.int32)
    order = torch.randperm(N, generator=g, device="cuda")
    slots[order[:case["padding"]]] = -1
    s.update(qkv=qkv, weight=_normal(g, channels, W, scale=0.5), bias=_normal(g, channels, scale=0.1), slots=slots,
             live=order[case["padding"]:].sort().values,  # the rows that are not padding: a scheduler knows them
             conv=_normal(g, S, L, channels).permute(0, 2, 1),  # channel-last
             state=_normal(g, S, H, P, K, scale=0.05, dtype=torch.float32))
    return s


# ---------------------------------------------------------------------------- the plain forms

def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _unit(v):
    return v * torch.rsqrt((v * v).sum(-1, keepdim=True) + EPS)


def _between(a):
    """[..., n] -> [..., n, n]: entry (t, s) is the sum of a over s < j <= t, -inf for s > t."""
    n = a.shape[-1]
    below = torch.ones(n, n, dtype=torch.bool, device=a.device).tril(-1)
    v = torch.where(below, a[..., :, None], torch.zeros((), device=a.device)).cumsum(-2)
    return torch.where(below | torch.eye(n, dtype=torch.bool, device=a.device), v, v.new_tensor(-math.inf))


def _inverse(a):
    """(1 + a)^-1 of strictly lower triangular [..., 64, 64]: blocks of 16 by their powers, then two by two."""
    lead = a.shape[:-2]
    blocks = a.view(*lead, 4, 16, 4, 16)
    b = -torch.stack((blocks[..., 0, :, 0, :], blocks[..., 1, :, 1, :], blocks[..., 2, :, 2, :], blocks[..., 3, :, 3, :]), -3)
    one = torch.eye(16, device=a.device)
    b2 = b @ b
    b4 = b2 @ b2
    t = (one + b) @ (one + b2) @ (one + b4) @ (one + b4 @ b4)
    low = torch.stack((blocks[..., 1, :, 0, :], blocks[..., 3, :, 2, :]), -3)
    u, v = t[..., 0::2, :, :], t[..., 1::2, :, :]
    t = torch.cat((torch.cat((u, torch.zeros_like(u)), -1), torch.cat((-(v @ low @ u), v), -1)), -2)
    u, v = t[..., 0, :, :], t[..., 1, :, :]
    return torch.cat((torch.cat((u, torch.zeros_like(u)), -1), torch.cat((-(v @ a[..., 32:, :32] @ u), v), -1)), -2)


def _plain_rule(s):
    case, lens = s["case"], s["lens"]
    H, P, K, G = case["heads"], case["head"], case["keys"], case["groups"]
    T, (of, start, size) = s["v"].shape[0], s["chunks"]
    slots, state = s["slots"].long(), s["state"]
    S = state[slots]
    S = S * s["has"].float()[:, None, None, None] if s["has"] is not None else torch.zeros_like(S)
    S = S[s["order"]]
    # whole chunks; a place past its sequence's end changes nothing: no step, and no strength
    inside = torch.arange(CHUNK, device="cuda") < size[:, None]
    token = torch.where(inside, start[:, None] + torch.arange(CHUNK, device="cuda"), 0)
    mask = inside.float()[..., None]                                                         # [n, C, 1]
    q, k = (_unit(s[i].float())[token].permute(0, 2, 1, 3) for i in "qk")                     # [n, G, C, K]
    v = s["v"].float()[token].permute(0, 2, 1, 3)                                            # [n, H, C, P]
    step = (s["A"] * _softplus(s["a"].float() + s["dt_bias"]))[token] * mask
    step = step.permute(0, 2, 1)                                                             # [n, H, C]
    beta = (torch.sigmoid(s["b"].float())[token] * mask).permute(0, 2, 1)[..., None]          # [n, H, C, 1]
    decay = torch.exp(_between(step))
    since = torch.exp(step.cumsum(-1))[..., None]                                            # from the chunk's first token
    left = torch.exp(torch.flip(torch.flip(step, [-1]).cumsum(-1), [-1]) - step)[..., None]  # to its last
    each = H // G
    q, kh = q.repeat_interleave(each, 1), k.repeat_interleave(each, 1)
    t = _inverse(((k @ k.mT).repeat_interleave(each, 1) * decay * beta).tril(-1)) * beta.mT
    m = (q @ kh.mT) * decay
    u, w = t @ v, t @ (kh * since)
    q, kl, total = q * since, kh * left, since[:, :, -1:]
    y = torch.empty_like(u)
    at = 0
    for n in s["live"]:  # the i-th chunks of all sequences that have one
        now = slice(at, at + n)
        h = S[:n]
        u[now] -= w[now] @ h.mT
        y[now] = q[now] @ h.mT
        S[:n] = h * total[now] + u[now].mT @ kl[now]
        at += n
    y = (y + m @ u).permute(0, 2, 1, 3) * (K ** -0.5)
    out = y.new_zeros(T, H, P)
    out.index_add_(0, token.flatten(), (y * mask[..., None]).flatten(0, 1))
    state[slots[s["order"]]] = S
    return {"out": out.to(torch.bfloat16), "state": state}


def _plain_step(s):
    case, live = s["case"], s["live"]
    H, P, K, G = case["heads"], case["head"], case["keys"], case["groups"]
    at = s["slots"][live].long()
    new = s["qkv"][live]
    seen = torch.cat([s["conv"][at], new[..., None]], -1)
    s["conv"][at] = seen[..., 1:]
    qkv = _silu((seen[..., -W:].float() * s["weight"].float()).sum(-1) + s["bias"].float())
    q = _unit(qkv[:, :G * K].unflatten(1, (G, K))).repeat_interleave(H // G, 1)
    k = _unit(qkv[:, G * K:2 * G * K].unflatten(1, (G, K))).repeat_interleave(H // G, 1)
    v = qkv[:, 2 * G * K:].unflatten(1, (H, P))
    decay = torch.exp(s["A"] * _softplus(s["a"][live].float() + s["dt_bias"]))
    h = s["state"][at] * decay[..., None, None]
    u = torch.sigmoid(s["b"][live].float())[..., None] * (v - (h * k[:, :, None, :]).sum(-1))
    h = h + u[..., None] * k[:, :, None, :]
    s["state"][at] = h
    out = torch.zeros(case["rows"], H, P, dtype=torch.bfloat16, device="cuda")
    out[live] = ((h * q[:, :, None, :]).sum(-1) * (K ** -0.5)).to(torch.bfloat16)
    return {"out": out, "conv": s["conv"], "state": s["state"]}


def _norm(v):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _plain_gated(s):
    x, gate = s["x"].float(), _silu(s["z"].float())
    y = _norm(x) * s["weight"].float() * gate if s["case"]["first"] else _norm(x * gate) * s["weight"].float()
    return {"out": y.to(torch.bfloat16)}


def _plain_residual(s):
    x = s["x"].float()
    if s["post"] is not None:
        x = _norm(x) * s["post"].float()
    r = s["residual"].float() + s["case"]["scale"] * x
    s["residual"].copy_(r)
    return {"out": (_norm(r) * s["weight"].float()).to(torch.bfloat16), "residual": s["residual"]}


# ---------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"rule": _plain_rule, "step": _plain_step, "gated": _plain_gated, "residual": _plain_residual}[op](s)
    import depthwise_causal_conv1d_gb300 as ccu

    if op == "rule":
        out = ccu.gated_delta_rule(s["q"], s["k"], s["v"], s["a"], s["b"], s["A"], dt_bias=s["dt_bias"], cu_seqlens=s["cu"],
                                   state=s["state"], state_indices=s["slots"], has_initial_state=s["has"])
        return {"out": out, "state": s["state"]}
    if op == "step":
        out = ccu.gated_delta_update(s["qkv"], s["a"], s["b"], s["A"], s["state"], s["conv"], s["weight"], s["bias"], "silu",
                                     dt_bias=s["dt_bias"], groups=s["case"]["groups"], state_indices=s["slots"])
        return {"out": out, "conv": s["conv"], "state": s["state"]}
    if op == "gated":
        return {"out": ccu.gated_rms_norm(s["x"], s["z"], s["weight"], eps=EPS, norm_before_gate=s["case"]["first"])}
    out = ccu.residual_rms_norm(s["x"], s["residual"], s["weight"], post_weight=s["post"], scale=s["case"]["scale"], eps=EPS)
    return {"out": out, "residual": s["residual"]}


# ---------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gated":
        x, z, w = s["x"].double(), s["z"].double(), s["weight"].double()
        z = z * torch.sigmoid(z)
        if not case["first"]:
            x = x * z
        y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        return {"out": y * z if case["first"] else y}
    if op == "residual":
        x = s["x"].double()
        if s["post"] is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * s["post"].double()
        r = s["residual"].double() + case["scale"] * x
        return {"out": r / torch.sqrt(r.square().mean(-1, keepdim=True) + EPS) * s["weight"].double(), "residual": r}
    return _exact_rule(s) if op == "rule" else _exact_step(s)


def _exact_unit(x):
    return x / torch.sqrt(x.square().sum(-1, keepdim=True) + EPS)


def _exact_token(h, q, k, v, decay, beta):
    """One token of the rule: h [n, H, P, K], q and k of unit length [n, H, K], v [n, H, P], decay and beta [n, H]. Changes h."""
    h.mul_(decay[..., None, None])
    u = (v - torch.matmul(h, k[..., None])[..., 0]) * beta[..., None]
    h.addcmul_(u[..., None], k[..., None, :])
    return torch.matmul(h, q[..., None])[..., 0] / math.sqrt(q.shape[-1])


def _exact_rule(s):
    """Token by token, all sequences that are that long at once."""
    case, lens, order = s["case"], s["lens"], s["order"]
    H, G = case["heads"], case["groups"]
    state, slots = s["state"].double(), s["slots"].long()
    h = state[slots]
    h = h * s["has"].double()[:, None, None, None] if s["has"] is not None else torch.zeros_like(h)
    h = h[torch.tensor(order, device="cuda")]
    decay = torch.exp(s["A"].double() * torch.nn.functional.softplus(s["a"].double() + s["dt_bias"].double(), threshold=1e9))
    beta = torch.sigmoid(s["b"].double())
    spread = torch.arange(H, device="cuda") // (H // G)
    q, k, v = _exact_unit(s["q"].double()), _exact_unit(s["k"].double()), s["v"].double()
    out = torch.zeros_like(v)
    starts = torch.tensor([_offsets(lens)[b] for b in order], device="cuda")
    live = len(order)
    for t in range(max(lens)):
        while lens[order[live - 1]] <= t:
            live -= 1
        at = starts[:live] + t
        out[at] = _exact_token(h[:live], q[at][:, spread], k[at][:, spread], v[at], decay[at], beta[at])
    state[slots[torch.tensor(order, device="cuda")]] = h
    return {"out": out, "state": state}


def _exact_step(s):
    case = s["case"]
    H, P, K, G = case["heads"], case["head"], case["keys"], case["groups"]
    conv, state = s["conv"].double(), s["state"].double()
    out = torch.zeros(case["rows"], H, P, dtype=torch.float64, device="cuda")
    w, bias = s["weight"].double(), s["bias"].double()
    for n, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        full = torch.cat([conv[slot], s["qkv"][n].double()[:, None]], 1)
        conv[slot] = full[:, 1:]
        x = (full[:, L + 1 - W:] * w).sum(1) + bias
        x = x * torch.sigmoid(x)
        q, k = _exact_unit(x[:2 * G * K].view(2, G, 1, K)).expand(2, G, H // G, K).reshape(2, 1, H, K)
        delta = torch.nn.functional.softplus(s["a"][n].double() + s["dt_bias"].double(), threshold=1e9)
        h = state[slot][None]
        out[n] = _exact_token(h, q, k, x[2 * G * K:].view(1, H, P), torch.exp(delta * s["A"].double())[None],
                              torch.sigmoid(s["b"][n].double())[None])[0]
        state[slot] = h[0]
    return {"out": out, "conv": conv, "state": state}


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "gated":
        T, inner = case["rows"], case["heads"] * case["head"]
        return {"bytes": 6 * T * inner + 2 * (inner if case["weights"] == "channel" else case["head"]), "flops": 9 * T * inner}
    if op == "residual":
        T, D = case["rows"], case["width"]
        return {"bytes": (12 if case["wide"] else 8) * T * D + (4 if case["post"] else 2) * D, "flops": (10 if case["post"] else 6) * T * D}
    H, P, K, G = case["heads"], case["head"], case["keys"], case["groups"]
    inner, channels = H * P, 2 * G * K + H * P
    if op == "rule":
        lens = _lengths(case)
        T = sum(lens)
        kept = 4 * len(lens) * inner * K
        read = 4 * sum(1 for b in range(len(lens)) if b % 2 == 0) * inner * K if case["initial"] else 0
        return {"bytes": T * (2 * channels + 2 * inner + 4 * H) + kept + read + 8 * H, "flops": 7 * T * inner * K}
    N = case["rows"] - case["padding"]
    row = 8 * inner * K + 2 * channels * (1 + 2 * L) + 4 * H
    return {"bytes": N * row + 2 * case["rows"] * inner + 2 * channels * (W + 1) + 8 * H,
            "flops": N * (7 * inner * K + channels * (2 * W + 5))}
