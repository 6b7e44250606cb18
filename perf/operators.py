"""Cases of the state-space operators: packed causal convolution, selective scan, selective
state update, and products with 4-bit weights. Each has a plain form (elementary torch
operations in 32 bits, rounded once at the end) and the framework's call (``own``)."""

import math

import torch

own = False

W = 4            # filter taps
L = 3            # convolution state: the taps before the newest input
CHUNK = 64       # tokens a block of the plain scan


# ---------------------------------------------------------------------------- the cases

def listed():
    return [
        # one short prompt of odd length entering a layer of 2048 channels (and 2 x 128 of B, C)
        dict(name="conv_one_short", op="conv", lens="37", channels=2304, initial=False),
        # a full prefill batch of unequal prompts, 4096 channels, half of them continued
        dict(name="conv_batch", op="conv", lens="4096,4096,8192,1000,3096,5000,191,7097", channels=4352, initial=True),
        # the scan of that one short prompt: latency
        dict(name="scan_one_short", op="scan", lens="37", heads=32, head=64, states=128, groups=1, gate=True, initial=False),
        # ordinary ragged batch with an empty and a one-token sequence, wide heads, eight groups, continued
        dict(name="scan_ragged", op="scan", lens="512,1,0,129,384,77,1024,250", heads=48, head=128, states=64, groups=8, gate=False, initial=True),
        # one long document: too few heads to fill the card without a split over its length
        dict(name="scan_long", op="scan", lens="16384", heads=64, head=64, states=128, groups=1, gate=True, initial=False),
        # the prefill benchmark's batch (8 x 4096 tokens, 4096 channels)
        dict(name="scan_batch", op="scan", lens="4096,4096,4096,4096,4096,4096,4096,4096", heads=64, head=64, states=128, groups=1, gate=True, initial=False),
        # a single user's token: latency
        dict(name="step_one_row", op="step", rows=1, slots=8, heads=32, head=64, states=128, groups=1, gate=True, padding=0),
        # the strided decode batch (64 rows, 6144 channels) on permuted slots, eight groups
        dict(name="step_strided", op="step", rows=64, slots=64, heads=96, head=64, states=64, groups=8, gate=False, padding=0),
        # the paged decode batch (256 rows, 8192 channels, a tenth of the rows padding)
        dict(name="step_paged", op="step", rows=256, slots=320, heads=128, head=64, states=128, groups=1, gate=True, padding=26),
        # in-projection of one token: z, x, B, C and dt of 4096 channels from 2048
        dict(name="w4_one_token", op="w4", rows=1, inner=2048, outer=8512, group=128, zeros=False),
        # in-projection of a few tokens with zero points and short groups: 8192 channels from 4096
        dict(name="w4_few", op="w4", rows=5, inner=4096, outer=16768, group=64, zeros=True),
        # out-projection of a decode batch of 64 rows
        dict(name="w4_batch", op="w4", rows=64, inner=16384, outer=8192, group=128, zeros=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total):
    """Up to 24 lengths that sum to at most `total`, empty and one-token ones among them."""
    count = _spread(rng, 1, 24)
    cuts = sorted(rng.randint(0, total) for _ in range(count - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if count > 3:
        lens[rng.randrange(count)] = rng.randint(0, 1)
    return ",".join(str(n) for n in lens)


def draw(rng):
    op = rng.choice(("conv", "scan", "step", "w4"))
    if op == "conv":
        return dict(op=op, lens=_lens(rng, _spread(rng, 5, 16384)), channels=8 * _spread(rng, 9, 800), initial=rng.random() < 0.5)
    if op == "w4":
        group = rng.choice((32, 64, 128))
        return dict(op=op, rows=_spread(rng, 1, 64), inner=group * _spread(rng, 256 // group, 8192 // group),
                    outer=_spread(rng, 100, 16384), group=group, zeros=rng.random() < 0.5)
    groups = rng.choice((1, 1, 2, 8))
    sizes = dict(heads=groups * max(1, _spread(rng, 4, 96) // groups), head=rng.choice((64, 64, 128, 32, 40)),
                 states=rng.choice((128, 128, 64, 16, 48, 200)), groups=groups, gate=rng.random() < 0.5)
    channels = sizes["heads"] * sizes["head"]
    if op == "scan":
        total = _spread(rng, 5, max(8, min(16384, (1 << 30) // (channels * sizes["states"]))))
        return dict(op=op, lens=_lens(rng, total), initial=rng.random() < 0.5, **sizes)
    rows = _spread(rng, 1, max(2, min(256, (1 << 28) // (channels * sizes["states"]))))
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
    """Blocks of up to CHUNK tokens that stay inside a sequence: their sequences, first tokens and sizes, and each sequence's last."""
    table = [(b, at + c, min(CHUNK, n - c)) for b, (at, n) in enumerate(zip(_offsets(lens), lens)) for c in range(0, n, CHUNK)]
    ended = [i for i, row in enumerate(table) if i + 1 == len(table) or table[i + 1][0] != row[0]]
    return torch.tensor(table, device="cuda").t().contiguous(), torch.tensor(ended, device="cuda")


def _maker(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _uniform(g, lo, hi, *shape):
    return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo


def _heads(g, case):
    """What a layer has per head: A < 0, D, and a bias that puts softplus(dt) in 0.001..0.1."""
    H = case["heads"]
    step = torch.exp(_uniform(g, math.log(1e-3), math.log(1e-1), H))
    return dict(A=-_uniform(g, 1.0, 16.0, H), D=_uniform(g, 0.5, 1.5, H), dt_bias=step + torch.log(-torch.expm1(-step)))


def prepare(case, seed):
    g = _maker(seed)
    op = case["op"]
    if op == "w4":
        M, I, O, group = case["rows"], case["inner"], case["outer"], case["group"]
        s = dict(case=case, x=_normal(g, M, I), q=torch.randint(0, 256, (O, I // 2), generator=g, device="cuda", dtype=torch.uint8),
                 scales=(_uniform(g, 0.5, 1.5, O, I // group) / (4.6 * math.sqrt(I))).to(torch.bfloat16), zeros=None)
        if case["zeros"]:
            s["zeros"] = torch.randint(0, 16, (O, I // group), generator=g, device="cuda").to(torch.bfloat16)
        return s
    if op == "conv":
        lens = _lengths(case)
        T, B, C = sum(lens), len(lens), case["channels"]
        return dict(case=case, x=_normal(g, T, C), weight=_normal(g, C, W, scale=0.5), bias=_normal(g, C, scale=0.1),
                    cu=torch.tensor(_offsets(lens), dtype=torch.int32, device="cuda"),
                    slots=torch.randperm(B + 3, generator=g, device="cuda")[:B].to(torch.int32),
                    state=_normal(g, B + 3, L, C).permute(0, 2, 1),  # channel-last, as the decode update takes it
                    has=(torch.arange(B, device="cuda", dtype=torch.int32) % 2 == 0).to(torch.int32) if case["initial"] else None)
    H, P, K, G = case["heads"], case["head"], case["states"], case["groups"]
    inner, bc = H * P, G * K
    rows = sum(_lengths(case)) if op == "scan" else case["rows"]
    # one row of the layer's in-projection: z | x B C | dt, padded to whole 16-byte vectors
    wide = (2 * inner + 2 * bc + H + 7) // 8 * 8
    proj = _normal(g, rows, wide)
    s = dict(case=case, z=proj[:, :inner].unflatten(1, (H, P)) if case["gate"] else None, **_heads(g, case))
    s["dt"] = proj[:, 2 * inner + 2 * bc:2 * inner + 2 * bc + H]
    xbc = proj[:, inner:2 * inner + 2 * bc]
    if op == "scan":
        lens = _lengths(case)
        B = len(lens)
        chunks, last_chunk = _chunks(lens)
        xbc = torch.nn.functional.silu(xbc)  # what the convolution's activation leaves
        s.update(x=xbc[:, :inner].unflatten(1, (H, P)), B=xbc[:, inner:inner + bc].unflatten(1, (G, K)),
                 C=xbc[:, inner + bc:].unflatten(1, (G, K)), lens=lens, chunks=chunks, last_chunk=last_chunk,
                 cu=torch.tensor(_offsets(lens), dtype=torch.int32, device="cuda"),
                 slots=torch.randperm(B + 3, generator=g, device="cuda")[:B].to(torch.int32),
                 state=_normal(g, B + 3, H, P, K, scale=0.05, dtype=torch.float32),
                 has=(torch.arange(B, device="cuda", dtype=torch.int32) % 2 == 0).to(torch.int32) if case["initial"] else None)
        return s
    N, S = rows, case["slots"]
    slots = torch.randperm(S, generator=g, device="cuda")[:N].to(torch.int32)
    order = torch.randperm(N, generator=g, device="cuda")
    slots[order[:case["padding"]]] = -1
    C = inner + 2 * bc
    s.update(xbc=xbc, weight=_normal(g, C, W, scale=0.5), bias=_normal(g, C, scale=0.1), slots=slots,
             live=order[case["padding"]:].sort().values,  # the rows that are not padding: a scheduler knows them
             conv=_normal(g, S, L, C).permute(0, 2, 1), state=_normal(g, S, H, P, K, scale=0.05, dtype=torch.float32))
    return s


# ---------------------------------------------------------------------------- the plain forms

def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _plain_conv(s):
    x, slots, state = s["x"].float(), s["slots"].long(), s["state"]
    T, B = x.shape[0], slots.numel()
    cu = s["cu"].long()
    before = state[slots].float().permute(0, 2, 1)  # [B, L, C]
    before = before * s["has"].float()[:, None, None] if s["has"] is not None else torch.zeros_like(before)
    # every sequence with its L earlier entries in front: row t of sequence b is row t + (b + 1) L
    seq = torch.searchsorted(cu[1:], torch.arange(T, device="cuda"), right=True)
    at = torch.arange(T, device="cuda") + (seq + 1) * L
    ext = x.new_empty(T + B * L, x.shape[1])
    ext[at] = x
    ext[(cu[:-1] + torch.arange(B, device="cuda") * L)[:, None] + torch.arange(L, device="cuda")] = before
    w = s["weight"].float()
    acc = s["bias"].float() + sum(ext[at - (W - 1) + j] * w[:, j] for j in range(W))
    ends = cu[1:] + (torch.arange(B, device="cuda") + 1) * L
    last = ext[ends[:, None] - L + torch.arange(L, device="cuda")]
    state[slots] = last.permute(0, 2, 1).to(torch.bfloat16)
    return {"out": _silu(acc).to(torch.bfloat16), "state": state}


def _between(a):
    """[..., n] -> [..., n, n]: entry (t, s) is the sum of a over s < j <= t, -inf for s > t."""
    n = a.shape[-1]
    below = torch.ones(n, n, dtype=torch.bool, device=a.device).tril(-1)
    v = torch.where(below, a[..., :, None], torch.zeros((), device=a.device)).cumsum(-2)
    return torch.where(below | torch.eye(n, dtype=torch.bool, device=a.device), v, v.new_tensor(-math.inf))


def _plain_scan(s):
    case, lens = s["case"], s["lens"]
    H, P, K, G = case["heads"], case["head"], case["states"], case["groups"]
    slots, state = s["slots"].long(), s["state"]
    first = state[slots]
    first = first * s["has"].float()[:, None, None, None] if s["has"] is not None else torch.zeros_like(first)
    # whole chunks of every sequence; a place past its sequence's end counts nothing
    T, (of, start, size) = s["x"].shape[0], s["chunks"]
    inside = torch.arange(CHUNK, device="cuda") < size[:, None]
    token = torch.where(inside, start[:, None] + torch.arange(CHUNK, device="cuda"), 0)
    mask = inside.float()
    x = s["x"].float()[token] * mask[..., None, None]                       # [n, Q, H, P]
    Bm, Cm = s["B"].float()[token] * mask[..., None, None], s["C"].float()[token] * mask[..., None, None]
    d = _softplus(s["dt"].float() + s["dt_bias"])[token] * mask[..., None]   # [n, Q, H]
    a = (d * s["A"]).permute(0, 2, 1)                                       # [n, H, Q]
    dx = x * d[..., None]
    cum = a.cumsum(-1)
    within = torch.exp(_between(a)) * torch.einsum("ntgk,nsgk->ngts", Cm, Bm).repeat_interleave(H // G, 1)
    y = torch.einsum("nhts,nshp->nthp", within, dx)
    to_end = torch.exp(torch.flip(torch.flip(a, [-1]).cumsum(-1), [-1]) - a)  # decay after each token
    Bh, Ch = Bm.repeat_interleave(H // G, 2), Cm.repeat_interleave(H // G, 2)
    part = torch.einsum("nshp,nshk->nhpk", dx * to_end.permute(0, 2, 1)[..., None], Bh)
    # a chunk starts from the sequence's first state and the parts of its earlier chunks
    total = cum[..., -1].t()                                                 # [H, n]
    n = total.shape[1]
    same = of[:, None] == of[None, :]
    reach = torch.zeros_like(total)[:, :, None].repeat(1, 1, n)              # decay over the chunks in between
    reach[:, 1:] = torch.exp(_between(total)[:, :-1]) * same[1:]
    own_total = torch.where(same.tril(-1), total[:, None, :], torch.zeros((), device="cuda")).sum(-1)  # [H, n]
    carry = torch.einsum("hts,shv->thv", reach, part.flatten(2)).view_as(part) + first[of] * torch.exp(own_total).t()[..., None, None]
    y = y + torch.einsum("nthk,nhpk->nthp", Ch, carry) * torch.exp(cum).permute(0, 2, 1)[..., None]
    y = y + x * s["D"][:, None]
    flat = y.new_zeros(T, H, P)
    flat.index_add_(0, token.flatten(), (y * mask[..., None, None]).flatten(0, 1))
    if s["z"] is not None:
        flat = flat * _silu(s["z"].float())
    after = carry * torch.exp(total).t()[..., None, None] + part
    ended = s["last_chunk"]
    first[of[ended]] = after[ended]
    state[slots] = first
    return {"out": flat.to(torch.bfloat16), "state": state}


def _plain_step(s):
    case, live = s["case"], s["live"]
    H, P, K, G = case["heads"], case["head"], case["states"], case["groups"]
    at = s["slots"][live].long()
    new = s["xbc"][live]
    seen = torch.cat([s["conv"][at], new[..., None]], -1)
    s["conv"][at] = seen[..., 1:]
    w = s["weight"].float()
    xbc = _silu((seen[..., -W:].float() * w).sum(-1) + s["bias"].float())
    x = xbc[:, :H * P].unflatten(1, (H, P))
    Bm = xbc[:, H * P:H * P + G * K].unflatten(1, (G, K)).repeat_interleave(H // G, 1)
    Cm = xbc[:, H * P + G * K:].unflatten(1, (G, K)).repeat_interleave(H // G, 1)
    d = _softplus(s["dt"][live].float() + s["dt_bias"])
    h = s["state"][at] * torch.exp(d * s["A"])[..., None, None] + (x * d[..., None])[..., None] * Bm[:, :, None, :]
    s["state"][at] = h
    y = (h * Cm[:, :, None, :]).sum(-1) + x * s["D"][:, None]
    if s["z"] is not None:
        y = y * _silu(s["z"][live].float())
    out = torch.zeros(case["rows"], H, P, dtype=torch.bfloat16, device="cuda")
    out[live] = y.to(torch.bfloat16)
    return {"out": out, "conv": s["conv"], "state": s["state"]}


def _plain_w4(s):
    group = s["case"]["group"]
    q = torch.stack([s["q"] & 15, s["q"] >> 4], -1).flatten(1).float()
    zero = s["zeros"].float().repeat_interleave(group, 1) if s["zeros"] is not None else 8.0
    w = (q - zero) * s["scales"].float().repeat_interleave(group, 1)
    return {"out": (s["x"].float() @ w.t()).to(torch.bfloat16)}


# ---------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"conv": _plain_conv, "scan": _plain_scan, "step": _plain_step, "w4": _plain_w4}[op](s)
    import depthwise_causal_conv1d_gb300 as ccu

    if op == "conv":
        out = ccu.causal_conv1d_packed(s["x"], s["weight"], s["bias"], "silu", cu_seqlens=s["cu"], conv_state=s["state"],
                                       conv_state_indices=s["slots"], has_initial_state=s["has"])
        return {"out": out, "state": s["state"]}
    if op == "scan":
        out = ccu.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                                 cu_seqlens=s["cu"], ssm_state=s["state"], state_indices=s["slots"], has_initial_state=s["has"])
        return {"out": out, "state": s["state"]}
    if op == "step":
        out = ccu.selective_state_update(s["xbc"], s["dt"], s["A"], s["state"], s["conv"], s["weight"], s["bias"], "silu",
                                         D=s["D"], z=s["z"], dt_bias=s["dt_bias"], groups=s["case"]["groups"], state_indices=s["slots"])
        return {"out": out, "conv": s["conv"], "state": s["state"]}
    return {"out": ccu.w4_matmul(s["x"], s["q"], s["scales"], s["zeros"])}


# ---------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "w4":
        group, I = case["group"], case["inner"]
        q = torch.empty(case["outer"], I, dtype=torch.float64, device="cuda")
        q[:, 0::2] = (s["q"] % 16).double()
        q[:, 1::2] = (s["q"] // 16).double()
        q = q.view(case["outer"], I // group, group)
        q -= s["zeros"].double()[..., None] if s["zeros"] is not None else 8
        q *= s["scales"].double()[..., None]
        return {"out": s["x"].double() @ q.view(case["outer"], I).t()}
    if op == "conv":
        return _exact_conv(s)
    return _exact_scan(s) if op == "scan" else _exact_step(s)


def _exact_conv(s):
    state, out = s["state"].double(), []
    cu, slots = s["cu"].tolist(), s["slots"].tolist()
    has = s["has"].tolist() if s["has"] is not None else [0] * len(slots)
    w, bias = s["weight"].double(), s["bias"].double()
    for b, slot in enumerate(slots):
        before = state[slot].t() * has[b]
        full = torch.cat([before, s["x"][cu[b]:cu[b + 1]].double()])
        n = full.shape[0] - L
        acc = bias.expand(n, -1).clone()
        for j in range(W):
            acc += w[:, j] * full[L - (W - 1) + j:L - (W - 1) + j + n]
        out.append(acc * torch.sigmoid(acc))
        state[slot] = full[n:].t()
    return {"out": torch.cat(out), "state": state}


def _exact_scan(s):
    """Token by token, all sequences that are that long at once."""
    case, lens = s["case"], s["lens"]
    H, G = case["heads"], case["groups"]
    state, slots = s["state"].double(), s["slots"].long()
    h = state[slots] if s["has"] is not None else torch.zeros_like(state[slots])
    if s["has"] is not None:
        h = h * s["has"].double()[:, None, None, None]
    delta = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=1e9)
    decay = torch.exp(delta * s["A"].double())
    x = s["x"].double()
    out = torch.zeros_like(x)
    order = sorted(range(len(lens)), key=lambda b: -lens[b])
    h = h[torch.tensor(order, device="cuda")]
    starts = torch.tensor([_offsets(lens)[b] for b in order], device="cuda")
    live = len(order)
    spread = torch.arange(H, device="cuda") // (H // G)
    Bm, Cm = s["B"].double(), s["C"].double()
    for t in range(max(lens)):
        while lens[order[live - 1]] <= t:
            live -= 1
        at = starts[:live] + t
        xt = x[at]
        hv = h[:live]
        hv.mul_(decay[at][..., None, None])
        hv += (xt * delta[at][..., None])[..., None] * Bm[at][:, spread][:, :, None, :]
        out[at] = torch.matmul(hv, Cm[at][:, spread][..., None])[..., 0] + s["D"].double()[:, None] * xt
    if s["z"] is not None:
        z = s["z"].double()
        out = out * z * torch.sigmoid(z)
    state[slots[torch.tensor(order, device="cuda")]] = h
    return {"out": out, "state": state}


def _exact_step(s):
    case = s["case"]
    H, P, K, G = case["heads"], case["head"], case["states"], case["groups"]
    conv, state = s["conv"].double(), s["state"].double()
    out = torch.zeros(case["rows"], H, P, dtype=torch.float64, device="cuda")
    w, bias = s["weight"].double(), s["bias"].double()
    for n, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        full = torch.cat([conv[slot], s["xbc"][n].double()[:, None]], 1)
        conv[slot] = full[:, 1:]
        v = (full[:, L + 1 - W:] * w).sum(1) + bias
        v = v * torch.sigmoid(v)
        x, bc = v[:H * P].view(H, P), v[H * P:].view(2, G, 1, K).expand(2, G, H // G, K).reshape(2, H, 1, K)
        delta = torch.nn.functional.softplus(s["dt"][n].double() + s["dt_bias"].double(), threshold=1e9)
        h = state[slot] * torch.exp(delta * s["A"].double())[:, None, None] + (delta[:, None] * x)[..., None] * bc[0]
        state[slot] = h
        y = (h * bc[1]).sum(-1) + s["D"].double()[:, None] * x
        if s["z"] is not None:
            z = s["z"][n].double()
            y = y * z * torch.sigmoid(z)
        out[n] = y
    return {"out": out, "conv": conv, "state": state}


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "w4":
        M, I, O, group = case["rows"], case["inner"], case["outer"], case["group"]
        sets = 2 if case["zeros"] else 1
        return {"bytes": O * I / 2 + 2 * sets * O * I / group + 2 * M * (I + O), "flops": 2 * M * I * O}
    if op == "conv":
        lens = _lengths(case)
        T, C = sum(lens), case["channels"]
        kept = len(lens) * L * C * 2 + (sum(1 for b in range(len(lens)) if b % 2 == 0) * L * C * 2 if case["initial"] else 0)
        return {"bytes": 4 * T * C + 2 * C * (W + 1) + kept, "flops": (2 * W + 5) * T * C}
    H, P, K, G = case["heads"], case["head"], case["states"], case["groups"]
    inner = H * P
    if op == "scan":
        lens = _lengths(case)
        T = sum(lens)
        kept = 4 * len(lens) * inner * K
        read = 4 * sum(1 for b in range(len(lens)) if b % 2 == 0) * inner * K if case["initial"] else 0
        row = 2 * inner * (3 if case["gate"] else 2) + 4 * G * K + 2 * H
        return {"bytes": T * row + kept + read + 12 * H, "flops": T * inner * (5 * K + 6)}
    N, C = case["rows"] - case["padding"], inner + 2 * G * K
    row = 8 * inner * K + 2 * C * (1 + 2 * L) + 2 * H + 2 * inner * (1 if case["gate"] else 0)
    return {"bytes": N * row + 2 * case["rows"] * inner + 2 * C * (W + 1) + 12 * H,
            "flops": N * (inner * (5 * K + 6) + C * (2 * W + 5))}
