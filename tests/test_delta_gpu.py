"""The gated delta rule and the norms around a layer on the GPU against their definitions in 64 bits."""

import numpy as np
import pytest
import torch

import delta_reference as ref
from gpu_util import Guarded

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF = 2.0 ** -8  # a rounding to BF16, relative to the value
NEAR = 2.0 ** -19  # error of a state, 2-norm over 2-norm: some thirty roundings of 2^-24 a term, in quadrature 2^-21.5
ROUTES = ["auto", "recurrent", "chunked"]


@pytest.fixture(scope="module")
def ccu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import depthwise_causal_conv1d_gb300 as ccu

    return ccu


def bf(rng, *shape, scale=1.0):
    """BF16 values on the device (as the kernels get them) and the same in 64 bits."""
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)
    return t.to(DEV), t.double().numpy()


def f32(a):
    t = torch.from_numpy(np.asarray(a, np.float32))
    return t.to(DEV), t.double().numpy()


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def offsets(lens):
    return i32(np.concatenate([[0], np.cumsum(lens)]).tolist())


def num(t):
    return t.double().cpu().numpy()


def within(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}: "
                           f"{got[bad][0]} for {want[bad][0]}, allowed {np.broadcast_to(tol, bad.shape)[bad][0]}")


class Rule:
    """Inputs of one call; ``wide`` takes q, k, v, a and b as slices of one wider row."""

    def __init__(self, lens, H, P, K, G, seed=0, bias=True, initial=None, slots=None, spare=2, wide=False, shift=0,
                 decay=(1.0, 16.0), mean=0.0, strength=1.0):
        rng = np.random.default_rng(seed)
        T, self.lens, self.dims = sum(lens), lens, (H, P, K, G)
        sizes = (G * K, G * K, H * P, H, H)
        if wide:
            w = sum(sizes) + shift
            w = w if shift else (w + 7) // 8 * 8
            row, rown = bf(rng, max(T, 1), w)
            row, rown = row[:T], rown[:T]
            cut = np.cumsum([shift, *sizes])
            part = [(row[:, a:b], rown[:, a:b]) for a, b in zip(cut, cut[1:])]
        else:
            part = [bf(rng, T, n) for n in sizes]
        shape = [(G, K), (G, K), (H, P), (H,), (H,)]
        (self.q, self.qn), (self.k, self.kn), (self.v, self.vn), (self.a, self.an), (self.b, self.bn) = [
            (t.unflatten(1, s) if len(s) > 1 else t, a.reshape((T,) + s)) for (t, a), s in zip(part, shape)]
        if mean:  # keys that have much in common
            self.k += mean
            self.kn = num(self.k)
        if strength != 1.0:
            self.b *= strength
            self.bn = num(self.b)
        self.A, self.An = f32(-rng.uniform(*decay, H))
        step = np.exp(rng.uniform(np.log(1e-3), np.log(1e-1), H))
        self.bias, self.biasn = f32(step + np.log(-np.expm1(-step))) if bias else (None, None)
        n = len(lens)
        self.slots = list(rng.permutation(n + spare)[:n]) if slots is None else slots
        self.S = max([n + spare] + [s + 1 for s in self.slots if s < 100])
        self.state, self.staten = f32(rng.standard_normal((self.S, H, P, K)) * 0.1)
        self.has = initial

    def run(self, ccu, state=None, **kw):
        return ccu.gated_delta_rule(self.q, self.k, self.v, self.a, self.b, self.A, cu_seqlens=offsets(self.lens),
                                    state=self.state if state is None else state, dt_bias=self.bias,
                                    state_indices=i32([int(s) for s in self.slots]),
                                    has_initial_state=None if self.has is None else i32(self.has), **kw)

    def want(self, **kw):
        return ref.rule(self.qn, self.kn, self.vn, self.an, self.bn, self.An, self.biasn, self.lens, self.staten, self.slots,
                        self.has, **kw)

    def check(self, out, state, what="", near=NEAR, **kw):
        o, off, s, bound = self.want(**kw)
        within(num(out), o, HALF * np.abs(o) + off + 1e-30, f"{what} out")
        got = num(state)
        within(got, s, bound[..., None] + 1e-30, f"{what} state")
        far = np.linalg.norm(got - s) / max(np.linalg.norm(s), 1e-30)
        assert far <= near, f"{what} state: {far} of its size off"
        size = np.linalg.norm(o)
        if size:
            far = np.linalg.norm(num(out) - o) / size
            assert far <= HALF / 2 + 2.0 ** -12, f"{what} out: {far} of its size off"  # roundings of half a step at most are 2^-9 at the root mean square or less


SHAPES = [(2, 64, 128, 1), (4, 64, 64, 2), (3, 128, 128, 3), (2, 8, 16, 1), (6, 40, 24, 3), (1, 5, 7, 1), (2, 33, 200, 1),
          (2, 1, 1, 2), (1, 80, 256, 1), (8, 16, 96, 8), (2, 256, 128, 1), (2, 136, 72, 2)]
LENS = [[1], [37], [128, 129, 0, 1], [5, 0, 0, 3, 260], [300]]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("route", ROUTES)
def test_rule(ccu, shape, lens, route):
    if route == "chunked" and (shape[1] % 8 or shape[2] % 8 or shape[2] > 128):
        pytest.skip("token by token only")
    r = Rule(lens, *shape, seed=len(lens) + shape[1], initial=[i % 2 for i in range(len(lens))])
    r.check(r.run(ccu, route=route), r.state, route)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("norm,scale,bias", [(True, 0.25, False), (False, None, True), (False, -1.5, False)])
def test_rule_options(ccu, route, norm, scale, bias):
    r = Rule([70, 3, 129], 2, 64, 64, 1, seed=5, bias=bias, initial=[1, 0, 1])
    if not norm:  # keys as they are: below unit length
        r.k *= 0.1
        r.kn = num(r.k)
        assert (r.kn ** 2).sum(-1).max() < 1.3
    r.check(r.run(ccu, route=route, scale=scale, qk_norm=norm), r.state, scale=scale, qk_norm=norm)


@pytest.mark.parametrize("route", ROUTES)
def test_rule_default_slots(ccu, route):
    r = Rule([9, 20, 100], 2, 8, 16, 1, seed=6, slots=[0, 1, 2], spare=0)
    out = ccu.gated_delta_rule(r.q, r.k, r.v, r.a, r.b, r.A, cu_seqlens=offsets(r.lens), state=r.state, dt_bias=r.bias, route=route)
    r.check(out, r.state)


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("shape", [(2, 64, 128, 1), (4, 40, 24, 2)], ids=str)
def test_rule_of_slices(ccu, shape, shift):
    """Slices of one projection row; an odd shift leaves every row on a 2-byte boundary."""
    r = Rule([130, 1, 40], *shape, seed=7, wide=True, shift=shift, initial=[1, 1, 0])
    r.check(r.run(ccu), r.state)


def test_rule_out_and_slots_by_strides(ccu):
    """Outputs as a slice of wider rows, slots further apart than their size."""
    H, P, K, G = 2, 64, 64, 1
    r = Rule([70, 66], H, P, K, G, seed=8, initial=[1, 0], slots=[2, 0])
    wide = torch.full((136, H + 1, P + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    held = torch.zeros(r.S, H * P * K + 64, device=DEV)
    state = held[:, :H * P * K].unflatten(1, (H, P, K))
    state.copy_(r.state)
    r.run(ccu, state=state, out=wide[:, :H, :P])
    r.check(wide[:, :H, :P], state)
    assert (wide[:, H] == 7).all() and (wide[:, :, P:] == 7).all() and not held[:, H * P * K:].any()


@pytest.mark.parametrize("route", ROUTES)
def test_rule_padding_and_range(ccu, route):
    """Slots of -1 and out of range: outputs +0, nothing kept, the range reported."""
    r = Rule([20, 150, 3, 140], 2, 64, 64, 1, seed=8, slots=[1, -1, 1000, 0], initial=[1, 1, 1, 1])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = r.run(ccu, route=route, status=status)
    r.check(out, r.state)
    assert status.item() == ccu.CCU_DEVERR_RANGE
    assert not out.view(torch.int16)[20:173].any()


@pytest.mark.parametrize("route", ROUTES)
def test_rule_of_no_tokens(ccu, route):
    """Empty sequences: states kept or zeroed; none at all."""
    r = Rule([0, 0], 2, 64, 64, 1, seed=9, slots=[2, 0], initial=[1, 0])
    out = r.run(ccu, route=route)
    assert out.shape == (0, 2, 64)
    assert not r.state[0].any() and torch.equal(r.state[1:].cpu().double(), torch.from_numpy(r.staten[1:]))
    none = ccu.gated_delta_rule(r.q, r.k, r.v, r.a, r.b, r.A, cu_seqlens=i32([0]), state=r.state, route=route)
    assert none.shape == (0, 2, 64)


@pytest.mark.parametrize("route", ROUTES)
def test_rule_keeps_nan_and_inf_apart(ccu, route):
    """A sequence of NaN or infinities reaches neither its neighbours nor their states."""
    for bad in (float("nan"), float("inf")):
        r = Rule([100, 33, 150], 2, 64, 128, 1, seed=9, slots=[0, 1, 2], spare=0, initial=[0, 0, 1])
        for t in (r.q, r.k, r.v, r.a, r.b):
            t[100:133] = bad
        r.state[1] = bad  # not an initial state: must not be read
        for a in (r.qn, r.kn, r.vn, r.an, r.bn):
            a[100:133] = 0
        r.staten[1] = 0
        out, state = r.run(ccu, route=route), r.state
        out[100:133], state[1] = 0, 0
        o, off, s, bound = r.want()
        o[100:133], off[100:133], s[1], bound[1] = 0, 0, 0, 0
        within(num(out), o, HALF * np.abs(o) + off, "out")
        within(num(state), s, bound[..., None], "state")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")], ids=str)
@pytest.mark.parametrize("which", ["q", "k", "v", "a", "b"])
def test_rule_is_causal_for_nan_and_inf(ccu, route, bad, which):
    """One at token 150 changes no output before it; in v it stays in its channel, in q in its token. Infinite gates are
    the formula's: a decay to nothing, none at all, a full write, none."""
    r = Rule([300], 1, 64, 64, 1, seed=41, initial=[1])
    first = r.state.clone()
    clean = r.run(ccu, route=route, state=first.clone())
    t, tn = getattr(r, which), getattr(r, which + "n")
    at = (150, 0) if which in "ab" else (150, 0, 5)
    t[at] = bad
    tn[at] = bad
    out = r.run(ccu, route=route)
    assert torch.equal(out[:150], clean[:150])
    if which == "v":
        keep = [c for c in range(64) if c != 5]
        assert torch.equal(out[:, :, keep], clean[:, :, keep])
        assert not torch.isfinite(out[150:, :, 5].float()).any()
        assert torch.isfinite(r.state[r.slots[0], 0, keep]).all() and not torch.isfinite(r.state[r.slots[0], 0, 5]).any()
    if which == "q":
        assert torch.equal(out[151:], clean[151:]) and torch.isfinite(r.state).all()
        assert not torch.isfinite(out[150].float()).all()
    if which == "k":
        assert not torch.isfinite(out[150:].float()).all()
    if which in "ab" and bad != bad:
        assert torch.isnan(out[150:].float()).all() and torch.isnan(r.state[r.slots[0]]).all()
    if which in "ab" and bad == bad:
        r.an, r.bn = np.clip(r.an, -1e4, 1e4), np.clip(r.bn, -1e4, 1e4)
        r.check(out, r.state)


@pytest.mark.parametrize("route", ROUTES)
def test_rule_of_a_state_with_nan(ccu, route):
    """A NaN in a row of the initial state stays in that row."""
    r = Rule([200], 1, 64, 64, 1, seed=42, initial=[1])
    clean_state = r.state.clone()
    clean = r.run(ccu, route=route, state=clean_state)
    r.state[r.slots[0], 0, 7, 3] = float("nan")
    out = r.run(ccu, route=route)
    keep = [c for c in range(64) if c != 7]
    assert torch.equal(out[:, :, keep], clean[:, :, keep])
    assert torch.isnan(out[:, :, 7].float()).all()
    assert torch.equal(r.state[r.slots[0], 0, keep], clean_state[r.slots[0], 0, keep])


@pytest.mark.parametrize("route", ROUTES)
def test_rule_of_extreme_decays(ccu, route):
    """Steps from 1e-8 to 60 and decays from none to exp(-1000): no overflow, no NaN."""
    r = Rule([200], 4, 64, 64, 1, seed=10, bias=False, initial=[1])
    r.a = torch.linspace(-20, 60, 800, device=DEV).view(200, 4)[torch.randperm(200)].to(torch.bfloat16).contiguous()
    r.an = num(r.a)
    r.A, r.An = f32([0.0, -1e-4, -1.0, -16.0])
    r.check(r.run(ccu, route=route), r.state)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("decay", [(1e-5, 1e-4), (0.01, 0.1), (100.0, 4000.0)], ids=str)
def test_rule_of_slow_and_fast_decays(ccu, route, decay):
    r = Rule([1000], 2, 64, 64, 1, seed=40, decay=decay, initial=[1])
    r.check(r.run(ccu, route=route), r.state)


@pytest.mark.parametrize("route", ROUTES)
def test_rule_of_keys_alike(ccu, route):
    """Keys that have most of their length in common, written at nearly full strength without decay: a token takes out most of what the
    one before it wrote, the same key again and again replaces its value."""
    r = Rule([400], 2, 64, 64, 1, seed=43, decay=(1e-5, 1e-4), mean=2.0, strength=4.0, initial=[1])
    r.check(r.run(ccu, route=route), r.state)
    r = Rule([200], 1, 64, 64, 1, seed=44, decay=(1e-5, 1e-4), initial=[1])
    r.k[:] = r.k[:1].clone()
    r.b[:] = 30.0
    r.kn, r.bn = num(r.k), num(r.b)
    r.check(r.run(ccu, route=route), r.state)


@pytest.mark.parametrize("route", ROUTES)
def test_rule_of_zero_and_huge_keys(ccu, route):
    """Keys and queries of zeros write and read nothing; their lengths may be anything between 1e-18 and 1e18."""
    r = Rule([150], 2, 64, 64, 2, seed=45, initial=[1])
    r.k[10:20] = 0
    r.q[30:40] = 0
    r.k[50:60] *= 1e15
    r.q[55:65] *= 1e15
    r.k[70:80] *= 1e-15
    r.q[75:85] *= 1e-15
    r.kn, r.qn = num(r.k), num(r.q)
    r.check(r.run(ccu, route=route), r.state)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("qk_norm", [True, False])
def test_rule_is_causal_for_keys_whose_squares_overflow(ccu, route, qk_norm):
    """Several of them in a chunk, whose products overflow too, change no output before the first; queries none but their own."""
    r = Rule([200, 70], 1, 64, 64, 1, seed=46, initial=[1, 0])
    if not qk_norm:
        r.k *= 0.0625
    first = r.state.clone()
    clean = r.run(ccu, route=route, state=first.clone(), qk_norm=qk_norm)
    r.k[90:120:7] *= 1e25
    out = r.run(ccu, route=route, state=first.clone(), qk_norm=qk_norm)
    assert torch.isfinite(out[:90].float()).all() and torch.equal(out[:90], clean[:90]) and torch.equal(out[200:], clean[200:])
    if route == "chunked":
        assert torch.isnan(out[90:200].float()).all()
    r.k[90:120:7] *= 1e-25
    r.q[90:120:7] *= 1e25
    base = r.run(ccu, route=route, state=first.clone(), qk_norm=qk_norm)
    r.q[90:120:7] *= 1e-25
    other = r.run(ccu, route=route, state=first.clone(), qk_norm=qk_norm)
    keep = [t for t in range(270) if t not in range(90, 120, 7)]
    assert torch.equal(base[keep], other[keep])


@pytest.mark.parametrize("route", ROUTES)
def test_rule_in_pieces(ccu, route):
    """A prompt in three calls, then token by token, against the whole prompt's definition."""
    H, P, K, G = 4, 64, 64, 2
    r = Rule([190], H, P, K, G, seed=11, slots=[1])
    got, at = [], 0
    for n in (100, 1, 70):
        cut = slice(at, at + n)
        got.append(ccu.gated_delta_rule(r.q[cut], r.k[cut], r.v[cut], r.a[cut], r.b[cut], r.A, cu_seqlens=offsets([n]), state=r.state,
                                        dt_bias=r.bias, state_indices=i32([1]), has_initial_state=i32([1 if at else 0]), route=route))
        at += n
    for t in range(at, 190):
        qkv = torch.cat([r.q[t].flatten(), r.k[t].flatten(), r.v[t].flatten()])[None]
        got.append(ccu.gated_delta_update(qkv, r.a[t:t + 1], r.b[t:t + 1], r.A, r.state, dt_bias=r.bias, groups=G, state_indices=i32([1])))
    r.check(torch.cat(got), r.state)


@pytest.mark.parametrize("route", ROUTES)
def test_rule_guard_bands(ccu, route):
    """Nothing outside out, the used slots and the sequences' rows is written."""
    r = Rule([3, 130], 2, 24, 48, 1, seed=12, slots=[0, 3])
    H, P, K, G = r.dims
    go, gs = Guarded(140 * H * P * 2, DEV), Guarded(4 * H * P * K * 4, DEV)
    out, state = go.view(torch.bfloat16, (140, H, P)), gs.view(torch.float32, (4, H, P, K))
    state.copy_(r.state[:4])
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, 0, 0, 7), value=float("nan")) for t in (r.q, r.k, r.v))
    a, b = (torch.nn.functional.pad(t, (0, 0, 0, 7), value=float("nan")) for t in (r.a, r.b))
    before = out.clone()
    ccu.gated_delta_rule(q, k, v, a, b, r.A, cu_seqlens=offsets(r.lens), state=state, dt_bias=r.bias, state_indices=i32(r.slots),
                         out=out, route=route)
    r.staten = r.staten[:4]
    r.check(out[:133], state)
    assert torch.equal(out[133:].view(torch.int16), before[133:].view(torch.int16))
    assert go.guards_intact() and gs.guards_intact()


def test_rule_offsets_out_of_order(ccu):
    """Offsets that do not ascend, or leave the rows, reach no memory outside the tensors."""
    for cu in ([0, 90, 40, 133], [-5, 200, 100, 1000], [133, 0, 133, 0]):
        r = Rule([60, 40, 33], 2, 64, 64, 1, seed=13, initial=[1, 0, 1], slots=[0, 2, 3], spare=2)
        H, P, K, G = r.dims
        go, gs = Guarded(133 * H * P * 2, DEV), Guarded(r.S * H * P * K * 4, DEV)
        out, state = go.view(torch.bfloat16, (133, H, P)), gs.view(torch.float32, (r.S, H, P, K))
        state.copy_(r.state)
        ccu.gated_delta_rule(r.q, r.k, r.v, r.a, r.b, r.A, cu_seqlens=i32(cu), state=state, state_indices=i32(r.slots), out=out)
        torch.cuda.synchronize()
        assert go.guards_intact() and gs.guards_intact() and torch.equal(state[[1, 4]], r.state[[1, 4]])


@pytest.mark.parametrize("route", ROUTES)
def test_rule_far_slots_and_rows(ccu, route):
    """Slots and rows whose offsets pass 2^31 elements."""
    H, P, K, G = 1, 64, 64, 1
    r = Rule([70], H, P, K, G, seed=13, slots=[2], spare=0)
    stride = (1 << 30) + 4096
    far = torch.zeros(2 * stride + P * K, device=DEV)
    state = far.as_strided((3, H, P, K), (stride, P * K, K, 1))
    rows = (1 << 31) // 64
    wide = torch.zeros(69 * rows + 64, dtype=torch.bfloat16, device=DEV)
    v = wide.as_strided((70, H, P), (rows, P, 1))
    v.copy_(r.v)
    r.v = v
    r.staten[:] = 0
    out = r.run(ccu, state=state, route=route)
    r.check(out, state.clone())


def in_a_graph(call):
    """`call` captured on a side stream (it has run before)."""
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


@pytest.mark.parametrize("route", ROUTES)
def test_rule_on_another_stream_and_in_a_graph(ccu, route):
    r = Rule([300, 140], 2, 64, 128, 1, seed=14, initial=[1, 0])
    first = r.state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)  # the default stream would read before the inputs are final
        r.v.mul_(1)
        out = r.run(ccu, route=route)
    side.synchronize()
    r.check(out, r.state, "stream")
    r.state.copy_(first)
    cu, slots, has = offsets(r.lens), i32([int(v) for v in r.slots]), i32(r.has)
    held = torch.empty_like(out)
    graph = in_a_graph(lambda: ccu.gated_delta_rule(r.q, r.k, r.v, r.a, r.b, r.A, cu_seqlens=cu, state=r.state, dt_bias=r.bias,
                                                    state_indices=slots, has_initial_state=has, out=held, route=route))
    for _ in range(2):
        r.state.copy_(first)
        held.zero_()
        graph.replay()
        torch.cuda.synchronize()
        r.check(held, r.state, "graph")


SEGMENTS = [([5000], 2, [1]), ([2500, 1, 0, 700, 2048], 3, [1, 0, 1, 1, 0]), ([1024, 1025, 1536, 1600], 1, None), ([4096], 1, [0]), ([3000], 40, [1])]


@pytest.mark.parametrize("lens,heads,initial", SEGMENTS, ids=str)
@pytest.mark.parametrize("shape", [(64, 64), (40, 128), (136, 24)], ids=str)
def test_rule_cut_into_segments(ccu, lens, heads, initial, shape):
    """Too few sequences and heads to fill the card: segments, their states joined; sequences that end on,
    before and behind a segment's end, empty ones, and a padding sequence."""
    if heads > 3 and shape != (64, 64):
        pytest.skip("one shape of many heads")
    r = Rule(lens, heads, *shape, 1, seed=44, initial=initial, decay=(0.01, 4.0))
    if len(lens) > 4:
        r.slots[3] = -1
    r.check(r.run(ccu, route="chunked"), r.state)


def test_rule_workspace(ccu):
    """The caller's workspace serves as well as torch's; one that is too small is refused, and nothing is changed."""
    a, b = (Rule([4000], 2, 64, 64, 1, seed=45, slots=[0]) for _ in range(2))
    out = a.run(ccu)
    work = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    assert torch.equal(out, b.run(ccu, workspace=work)) and torch.equal(a.state, b.state)
    before = b.state.clone()
    with pytest.raises(ValueError, match="workspace"):
        b.run(ccu, workspace=work[:1024])
    assert torch.equal(b.state, before)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=str)
@pytest.mark.parametrize("which", ["q", "k", "v", "a", "b"])
def test_rule_of_segments_is_causal_for_nan_and_inf(ccu, which, bad):
    """As in one piece: what is not finite in one segment reaches the later ones, and of a value only its channel."""
    r = Rule([3000], 1, 64, 64, 1, seed=46, initial=[1], decay=(0.01, 0.1))
    clean = r.run(ccu, state=r.state.clone())
    t = getattr(r, which)
    t[(1500, 0) if which in "ab" else (1500, 0, 5)] = bad
    out = r.run(ccu)
    assert torch.equal(out[:1500], clean[:1500])
    keep = [c for c in range(64) if c != 5]
    if which == "v":
        assert torch.equal(out[:, :, keep], clean[:, :, keep]) and not torch.isfinite(out[1500:, :, 5].float()).any()
    if which == "q":
        assert torch.equal(out[1501:], clean[1501:])
    if which == "k" or bad != bad and which != "q" and which != "v":
        assert not torch.isfinite(out[1500:].float()).any() and not torch.isfinite(r.state[r.slots[0]]).any()


def test_rule_two_graphs_share_a_workspace(ccu):
    """Two captured calls on one workspace, replayed in turn, and a third with a workspace of its own."""
    rules = [Rule([4000 + 100 * i], 2, 64, 64, 1, seed=47 + i, slots=[0]) for i in range(2)]
    work = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    graphs, outs, firsts = [], [], []
    for r in rules:
        cu, slots = offsets(r.lens), i32([0])
        held = torch.empty_like(r.v)
        firsts.append(r.state.clone())
        args = dict(cu_seqlens=cu, state=r.state, dt_bias=r.bias, state_indices=slots, out=held, workspace=work)
        call = lambda r=r, args=args: ccu.gated_delta_rule(r.q, r.k, r.v, r.a, r.b, r.A, **args)  # noqa: E731
        call()
        graphs.append((in_a_graph(call), args))
        outs.append(held)
    for r, first in zip(rules, firsts):
        r.state.copy_(first)
    for _ in range(2):
        for (graph, _), r, held in zip(graphs, rules, outs):
            held.zero_()
            graph.replay()
            torch.cuda.synchronize()
            r.check(held, r.state)


def halves(ccu, r, state, ranges, **kw):
    """The calls of ``ranges`` of heads one by one: too few items each to be shared out."""
    outs = []
    for lo, hi in ranges:
        outs.append(ccu.gated_delta_rule(r.q, r.k, r.v[:, lo:hi], r.a[:, lo:hi], r.b[:, lo:hi], r.A[lo:hi].contiguous(), cu_seqlens=offsets(r.lens),
                                         state=state[:, lo:hi], dt_bias=r.bias[lo:hi].contiguous(), state_indices=i32([int(s) for s in r.slots]),
                                         has_initial_state=None if r.has is None else i32(r.has), route="chunked", **kw))
    return torch.cat(outs, 1)


SHARED = [([2000] * 5, 32, (8, 16)), ([700, 300, 2000, 0, 64, 513], 27, (16, 8)), ([6400, 64, 70, 1, 900], 33, (24, 128)), ([4100], 160, (8, 64)),
          ([1300, 1290], 27, (264, 8)), ([1300, 1290], 28, (264, 8)), ([700, 300, 2000, 0, 64, 513], 28, (16, 8)),
          ([640] * 20, 8, (128, 128))]


@pytest.mark.parametrize("lens,heads,shape", SHARED, ids=str)
def test_rule_in_even_shares(ccu, lens, heads, shape):
    """More items than SMs: cut ones give the bits of calls of fewer heads, which are not cut, and the definition's values."""
    r = Rule(lens, heads, *shape, 1, seed=60, initial=[i % 2 for i in range(len(lens))], decay=(0.01, 2.0))
    blocks = (shape[0] + 127) // 128
    calls = -(-heads // (100 // (len(lens) * blocks)))  # 50 to 100 items each: not shared out, nor cut into segments
    borders = [heads * i // calls for i in range(calls + 1)]
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        with pytest.raises(ValueError, match="workspace"):  # it has a plan: one byte is not enough
            r.run(ccu, route="chunked", workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    start = r.state.clone()
    want = start.clone()
    o = halves(ccu, r, want, list(zip(borders, borders[1:])))
    for _ in range(2):
        state = start.clone()
        out = r.run(ccu, route="chunked", state=state)
        assert torch.equal(out, o) and torch.equal(state, want)
    if sum(lens) * heads * shape[0] * shape[1] < 1 << 28:
        r.check(out, state)


@pytest.mark.parametrize("heads", [32, 33])
def test_rule_in_even_shares_of_padding_and_nan(ccu, heads):
    """A padding sequence among shared ones; a NaN in a key reaches its sequence's later tokens in whichever piece, nothing else."""
    lens = [1500, 1400, 1450, 1600, 1550]
    r = Rule(lens, heads, 8, 16, 1, seed=61, initial=[1, 0, 1, 1, 0], slots=[3, -1, 0, 4, 1], spare=1)
    start, clean_state = r.state.clone(), r.state.clone()
    clean = r.run(ccu, route="chunked", state=clean_state)
    assert not clean[1500:2900].view(torch.int16).any()
    at = 1500 + 1400 + 100
    r.k[at, 0, 3] = float("nan")
    state = start.clone()
    out = r.run(ccu, route="chunked", state=state)
    end = 1500 + 1400 + 1450
    assert torch.equal(out[:at], clean[:at]) and torch.equal(out[end:], clean[end:]) and torch.isnan(out[at:end].float()).all()
    assert torch.isnan(state[0]).all() and torch.equal(state[1:], clean_state[1:])


def test_rule_in_even_shares_in_graphs_with_one_workspace(ccu):
    """Captured calls that share a workspace, replayed in turn and again: each starts from cleared flags."""
    lens = [2000] * 5
    rules = [Rule(lens, 32, 8, 16, 1, seed=62 + i, initial=[1] * 5) for i in range(2)]
    starts = [r.state.clone() for r in rules]
    wants = [(r.run(ccu, route="chunked", state=s), s) for r, s in ((r, r.state.clone()) for r in rules)]
    work = torch.full((1 << 24,), 255, dtype=torch.uint8, device=DEV)
    states = [s.clone() for s in starts]
    outs = [torch.empty_like(w[0]) for w in wants]
    calls = [dict(cu_seqlens=offsets(lens), state=s, dt_bias=r.bias, state_indices=i32([int(x) for x in r.slots]), has_initial_state=i32(r.has),
                  workspace=work, out=o, route="chunked") for r, s, o in zip(rules, states, outs)]
    graphs = []
    for r, c in zip(rules, calls):
        ccu.gated_delta_rule(r.q, r.k, r.v, r.a, r.b, r.A, **c)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ccu.gated_delta_rule(r.q, r.k, r.v, r.a, r.b, r.A, **c)
        graphs.append(g)
    for _ in range(3):
        for s, start in zip(states, starts):
            s.copy_(start)
        for g in graphs:
            g.replay()
        for out, s, (o, t) in zip(outs, states, wants):
            assert torch.equal(out, o) and torch.equal(s, t)


def test_rule_longest_sequences_first(ccu):
    """More sequences than are put in order by length, and as many: every one keeps its own slot and rows."""
    for n in (64, 65, 130):
        rng = np.random.default_rng(n)
        lens = [int(v) for v in rng.integers(0, 90, n)]
        r = Rule(lens, 2, 64, 64, 1, seed=n, initial=[i % 2 for i in range(n)])
        r.check(r.run(ccu, route="chunked"), r.state)


@pytest.mark.parametrize("route", ROUTES)
def test_rule_gives_the_same_bits_again(ccu, route):
    r = Rule([700, 5, 64], 2, 128, 128, 1, seed=15, initial=[1, 1, 0])
    first = r.state.clone()
    out = r.run(ccu, route=route)
    again = first.clone()
    assert torch.equal(out, r.run(ccu, state=again, route=route)) and torch.equal(again, r.state)


# ------------------------------------------------------------------ one token a row

def one_token(rng, N, H, P, K, G, S, W, L, bias=True, conv=True):
    channels = 2 * G * K + H * P
    d = dict(qkv=bf(rng, N, channels), a=bf(rng, N, H), b=bf(rng, N, H), A=f32(-rng.uniform(1, 16, H)), state=f32(rng.standard_normal((S, H, P, K)) * 0.1))
    step = np.exp(rng.uniform(np.log(1e-3), np.log(1e-1), H))
    d["dt_bias"] = f32(step + np.log(-np.expm1(-step)))
    if conv:
        d.update(weight=bf(rng, channels, W, scale=0.5), cbias=bf(rng, channels, scale=0.1), conv=bf(rng, S, channels, L))
    return d


def want_token(d, slots, G, act, scale=None, qk_norm=True):
    """out, its bound before rounding, the new states and the bound, the new convolution state."""
    S, H, P, K = d["state"][1].shape
    N = len(slots)
    x, state, bound = d["qkv"][1], d["state"][1].copy(), np.zeros((S, H, P))
    out, off, conv = np.zeros((N, H, P)), np.zeros((N, H, P)), None
    slip = np.zeros(x.shape)  # error of the convolution's 32-bit sums
    if "weight" in d:
        w, cb, conv = d["weight"][1], d["cbias"][1], d["conv"][1].copy()
        W = w.shape[1]
        done = np.zeros(x.shape)
        for n, s in enumerate(slots):
            if s < 0 or s >= S:
                continue
            full = np.concatenate([d["conv"][1][s], x[n][:, None]], 1)
            conv[s] = full[:, 1:]
            acc = (full[:, -W:] * w).sum(1) + cb
            mag = (np.abs(full[:, -W:]) * np.abs(w)).sum(1) + np.abs(cb)
            done[n] = ref.silu(acc) if act == "silu" else acc
            slip[n] = (W + 1) * 2.0 ** -24 * 1.1 * mag + 2.0 ** -20 * np.abs(done[n])  # silu grows by at most 1.1, and its own error
        x = done
    q, k = (ref.unit(x[:, i * G * K:(i + 1) * G * K].reshape(N, G, K), qk_norm) for i in range(2))
    v, vs = x[:, 2 * G * K:].reshape(N, H, P), slip[:, 2 * G * K:].reshape(N, H, P)
    # a relative error of q and k (2-norm), from the convolution's sums
    length = [np.sqrt((x[:, i * G * K:(i + 1) * G * K].reshape(N, G, K) ** 2).sum(-1) + ref.UNIT * qk_norm) for i in range(2)]
    away = [np.sqrt((slip[:, i * G * K:(i + 1) * G * K].reshape(N, G, K) ** 2).sum(-1)) / np.maximum(length[i], 1e-30) for i in range(2)]
    g = np.arange(H) // (H // G)
    for n, s in enumerate(slots):
        if s < 0 or s >= S:
            continue
        decay, beta = np.exp(d["A"][1] * ref.softplus(d["a"][1][n] + d["dt_bias"][1])), ref.sigmoid(d["b"][1][n])
        size = np.sqrt((state[s] ** 2).sum(-1)) + np.abs(v[n])
        more = 3 * away[1][n][g][:, None] * size + vs[n]
        scaled = K ** -0.5 if scale is None else scale
        state[s], err, out[n], off[n] = ref.token(state[s], np.zeros((H, P)), q[n][g], k[n][g], v[n], decay, beta, scaled)
        bound[s] = err + more
        off[n] += abs(scaled) * np.sqrt((q[n][g] ** 2).sum(-1))[:, None] * (more + 2 * away[0][n][g][:, None] * size)
    return out, off, state, bound, conv


STEPS = [(3, 2, 64, 128, 1, 4, 3), (4, 4, 64, 64, 2, 4, 4), (2, 3, 33, 50, 1, 2, 1), (5, 2, 8, 32, 2, 3, 2), (2, 2, 128, 256, 1, 4, 3),
         (3, 6, 40, 24, 3, 4, 12), (2, 2, 5, 7, 1, 1, 1), (1, 4, 256, 128, 2, 4, 3), (2, 1, 20, 130, 1, 4, 3)]


@pytest.mark.parametrize("case", STEPS, ids=str)
@pytest.mark.parametrize("conv", [True, False])
@pytest.mark.parametrize("channel_last", [True, False])
def test_update(ccu, case, conv, channel_last):
    N, H, P, K, G, W, L = case
    rng = np.random.default_rng(P + K)
    S = N + 3
    d = one_token(rng, N, H, P, K, G, S, W, L, conv=conv)
    slots = [int(s) for s in rng.permutation(S)[:N]]
    if N > 2:
        slots[1] = -1
    args = {}
    if conv:
        state = d["conv"][0]
        if channel_last:
            state = state.permute(0, 2, 1).contiguous().permute(0, 2, 1)
        args = dict(conv_state=state, conv_weight=d["weight"][0], conv_bias=d["cbias"][0], activation="silu")
    out = ccu.gated_delta_update(d["qkv"][0], d["a"][0], d["b"][0], d["A"][0], d["state"][0], dt_bias=d["dt_bias"][0], groups=G,
                                 state_indices=i32(slots), **args)
    o, off, s, bound, c = want_token(d, slots, G, "silu")
    within(num(out), o, HALF * np.abs(o) + off + 1e-30, "out")
    within(num(d["state"][0]), s, bound[..., None] + 1e-30, "state")
    if conv:
        assert np.array_equal(num(args["conv_state"]), c)
    if N > 2:
        assert not out[1].view(torch.int16).any()


@pytest.mark.parametrize("scale,norm", [(0.5, True), (None, False)])
def test_update_options(ccu, scale, norm):
    N, H, P, K, G, W, L = 3, 4, 64, 64, 2, 4, 3
    d = one_token(np.random.default_rng(3), N, H, P, K, G, N, W, L, conv=False)
    d["qkv"][0].mul_(0.1)
    d["qkv"] = (d["qkv"][0], num(d["qkv"][0]))
    out = ccu.gated_delta_update(d["qkv"][0], d["a"][0], d["b"][0], d["A"][0], d["state"][0], dt_bias=d["dt_bias"][0], groups=G, scale=scale,
                                 qk_norm=norm)
    o, off, s, bound, _ = want_token(d, [0, 1, 2], G, None, scale, norm)
    within(num(out), o, HALF * np.abs(o) + off, "out")
    within(num(d["state"][0]), s, bound[..., None], "state")


def test_update_slices_strides_guards_and_range(ccu):
    """Rows of a projection, slots apart, outputs in wider rows, a slot out of range; nothing else is written."""
    N, H, P, K, G, W, L, S = 4, 2, 64, 64, 1, 4, 3, 6
    rng = np.random.default_rng(4)
    d = one_token(rng, N, H, P, K, G, S, W, L)
    channels = 2 * G * K + H * P
    wide = torch.zeros(N, channels + 2 * H + 3, dtype=torch.bfloat16, device=DEV)
    wide[:, 1:1 + channels], wide[:, 1 + channels:1 + channels + H], wide[:, 1 + channels + H:1 + channels + 2 * H] = d["qkv"][0], d["a"][0], d["b"][0]
    held, go = Guarded(S * (H * P * K + 4) * 4, DEV), Guarded(N * 3 * P * 2, DEV)
    state = held.view(torch.float32, (S, H * P * K + 4))[:, :H * P * K].unflatten(1, (H, P, K))
    state.copy_(d["state"][0])
    out = go.view(torch.bfloat16, (N, 3, P))[:, :H]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    work = torch.empty(4 * N * channels, dtype=torch.uint8, device=DEV)
    slots = [5, 99, 0, -1]
    got = ccu.gated_delta_update(wide[:, 1:1 + channels], wide[:, 1 + channels:1 + channels + H], wide[:, 1 + channels + H:1 + channels + 2 * H],
                                 d["A"][0], state, d["conv"][0], d["weight"][0], d["cbias"][0], "silu", dt_bias=d["dt_bias"][0], groups=G,
                                 state_indices=i32(slots), out=out, status=status, workspace=work)
    assert got is out and status.item() == ccu.CCU_DEVERR_RANGE
    o, off, s, bound, c = want_token(d, slots, G, "silu")
    within(num(out), o, HALF * np.abs(o) + off, "out")
    within(num(state), s, bound[..., None], "state")
    assert np.array_equal(num(d["conv"][0]), c) and held.guards_intact() and go.guards_intact()
    assert not out[[1, 3]].reshape(-1).view(torch.int16).any()
    with pytest.raises(ValueError, match="workspace"):
        ccu.gated_delta_update(wide[:, 1:1 + channels], d["a"][0], d["b"][0], d["A"][0], state, d["conv"][0], d["weight"][0], groups=G,
                               state_indices=i32(slots), workspace=work[:64])


def test_update_keeps_rows_apart(ccu):
    """NaN in one row, in a slot that nobody uses, and in a head's gate."""
    N, H, P, K, G, S = 3, 2, 64, 64, 2, 5
    d = one_token(np.random.default_rng(5), N, H, P, K, G, S, 4, 3)
    clean = {k: v[0].clone() for k, v in d.items()}
    args = lambda t: (t["qkv"], t["a"], t["b"], t["A"], t["state"], t["conv"], t["weight"], t["cbias"], "silu")  # noqa: E731
    want = ccu.gated_delta_update(*args(clean), dt_bias=d["dt_bias"][0], groups=G, state_indices=i32([4, 1, 0]))
    t = {k: v[0] for k, v in d.items()}
    t["qkv"][1] = float("nan")
    t["state"][2] = float("nan")
    t["a"][0, 1] = float("nan")
    out = ccu.gated_delta_update(*args(t), dt_bias=d["dt_bias"][0], groups=G, state_indices=i32([4, 1, 0]))
    assert torch.equal(out[2], want[2]) and torch.equal(out[0, 0], want[0, 0]) and torch.isnan(out[0, 1]).all() and torch.isnan(out[1]).all()
    assert torch.equal(t["state"][0], clean["state"][0]) and torch.equal(t["state"][4, 0], clean["state"][4, 0])
    assert torch.equal(t["state"][3], clean["state"][3]) and torch.isnan(t["state"][2]).all()


def test_update_far_slots_graph_and_stream(ccu):
    """Slots past 2^31 elements; two captured steps, replayed, on a side stream."""
    N, H, P, K, G, S = 2, 1, 64, 64, 1, 3
    d = one_token(np.random.default_rng(6), N, H, P, K, G, S, 4, 3, conv=False)
    stride = (1 << 30) + 4096
    far = torch.zeros(2 * stride + P * K, device=DEV)
    state = far.as_strided((S, H, P, K), (stride, P * K, K, 1))
    slots = i32([2, 0])
    out = torch.empty(N, H, P, dtype=torch.bfloat16, device=DEV)
    call = lambda: ccu.gated_delta_update(d["qkv"][0], d["a"][0], d["b"][0], d["A"][0], state, dt_bias=d["dt_bias"][0], groups=G,  # noqa: E731
                                          state_indices=slots, out=out)
    call()
    graph = in_a_graph(lambda: (call(), call()))
    state.copy_(d["state"][0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
    side.synchronize()
    *_, s, bound, _ = want_token(d, [2, 0], G, None)
    d["state"] = (None, s)
    o, off, s2, bound2, _ = want_token(d, [2, 0], G, None)
    within(num(state.clone()), s2, (bound + bound2)[..., None] + 1e-30, "state")
    within(num(out), o, HALF * np.abs(o) + off + np.abs(bound[[2, 0]]) + 1e-30, "out")


# ------------------------------------------------------------------ norms

# In 32 bits: squares 1 each and their sum 13 at most (8 entries a thread, 32 lanes, 32 warps) make 7 of the root, the root 2, the quotient
# and the eps 1, products 3, a gate 8: 24 units of 2^-24, relative. The long rows' kernel sums up to n / 1024 entries a thread.
NORM = 24 * 2.0 ** -24

ROWS = [(1, 16, 128), (5, 3, 64), (3, 4, 256), (2, 8, 1024), (7, 2, 40), (3, 5, 37), (2, 1, 1), (4, 3, 6), (2, 2, 2050), (1, 1, 16384),
        (1, 1, 70000), (1, 1, 8200), (1, 1, 8201), (300, 7, 96), (2, 1, 24 * 1024)]


@pytest.mark.parametrize("rows", ROWS, ids=str)
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("weight", ["head", "channel", "wide", None])
def test_gated_norm(ccu, rows, first, weight):
    T, H, P = rows
    rng = np.random.default_rng(P)
    x, xn = bf(rng, T, H, P)
    z, zn = (None, None) if weight is None else bf(rng, T, H, P)
    w, wn = (None, None) if weight is None else bf(rng, *((P,) if weight == "head" else (H, P)))
    if weight == "wide":
        w, wn = f32(wn + 2.0 ** -12)
    out = ccu.gated_rms_norm(x, z, w, norm_before_gate=first)
    want = ref.gated(xn, zn, wn, 1e-6, first)
    within(num(out), want, (HALF + NORM + P / 1024 * 2.0 ** -24) * np.abs(want), "out")


@pytest.mark.parametrize("P", [64, 37, 130])
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_gated_norm_of_slices(ccu, P, shift):
    """Slices of wider rows on 16-, 4- and 2-byte boundaries, weights too; nothing else is written."""
    T, H = 5, 3
    rng = np.random.default_rng(P + shift)
    wide, wn = bf(rng, T, 2 * H * P + 8)
    x, z = wide[:, shift:shift + H * P].unflatten(1, (H, P)), wide[:, shift + H * P:shift + 2 * H * P].unflatten(1, (H, P))
    xn, zn = wn[:, shift:shift + H * P].reshape(T, H, P), wn[:, shift + H * P:shift + 2 * H * P].reshape(T, H, P)
    w, wgt = bf(rng, H * P + shift)
    w, wgt = w[shift:].view(H, P), wgt[shift:].reshape(H, P)
    g = Guarded(T * (H + 1) * P * 2, DEV)
    full = g.view(torch.bfloat16, (T, H + 1, P))
    before = full[:, H].clone()
    ccu.gated_rms_norm(x, z, w, eps=1e-3, out=full[:, :H])
    want = ref.gated(xn, zn, wgt, 1e-3, True)
    within(num(full[:, :H]), want, (HALF + NORM) * np.abs(want), "out")
    assert g.guards_intact() and torch.equal(full[:, H].view(torch.int16), before.view(torch.int16))


def test_gated_norm_of_extremes(ccu):
    """Rows of zeros, NaN, infinities, huge and tiny entries, gates from -inf to inf: each in its own row."""
    T, H, P = 8, 1, 128
    rng = np.random.default_rng(1)
    x, _ = bf(rng, T, H, P)
    z, _ = bf(rng, T, H, P)
    x[0] = 0
    x[1, 0, 5] = float("nan")
    x[2, 0, 7] = float("inf")
    x[3] *= 1e17
    x[4] *= 1e-30
    z[5, 0, 0], z[5, 0, 1], z[5, 0, 2] = -1e4, 1e4, -100
    z[6, 0, 3] = float("nan")
    out = ccu.gated_rms_norm(x, z, None)
    want = ref.gated(num(x), num(z), None, 1e-6, True)
    assert not out[0].any() and torch.isnan(out[1].float()).all()
    assert torch.isnan(out[2, 0, 7].float()) and not out[2, 0, :7].any()  # x / infinity
    good = np.ones((T, H, P), bool)
    good[1:3], good[6, 0, 3] = False, False
    assert torch.isnan(out[6, 0, 3].float())
    # a SiLU below 2^-126 may be flushed
    within(num(out)[good], want[good], (HALF + NORM) * np.abs(want[good]) + 2.0 ** -120, "out")


@pytest.mark.parametrize("rows", [(1, 2048), (64, 16384), (5, 37), (3, 1), (200, 512), (7, 622), (2, 70000), (2, 9001), (33, 4096)], ids=str)
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("post,weight,scale", [(True, True, 0.5), (False, True, 1.0), (True, False, -2.0), (False, False, 0.0)])
def test_residual_norm(ccu, rows, wide, post, weight, scale):
    T, D = rows
    rng = np.random.default_rng(D)
    x, xn = bf(rng, T, D)
    r, rn = f32(rng.standard_normal((T, D)) * 3) if wide else bf(rng, T, D, scale=3)
    kind = f32 if wide else (lambda a: bf(rng, *a.shape))
    w, wn = kind(rng.standard_normal(D)) if weight else (None, None)
    p, pn = kind(rng.standard_normal(D)) if post else (None, None)
    out = ccu.residual_rms_norm(x, r, w, post_weight=p, scale=scale, eps=1e-5)
    want, sums = ref.residual(xn, rn, wn, pn, scale, 1e-5)
    off = (NORM + D / 1024 * 2.0 ** -24) * (np.abs(sums - rn) + np.abs(sums))  # of the sum in 32 bits
    within(num(r), sums, off + (0 if wide else HALF) * np.abs(sums), "residual")
    each = np.abs(wn) if weight else 1
    size = np.sqrt((sums * sums).mean(-1, keepdims=True) + 1e-5)
    root = np.sqrt((off * off).mean(-1, keepdims=True)) / size  # what the sums' errors make of the root
    within(num(out), want, (HALF + NORM + D / 1024 * 2.0 ** -24 + root) * np.abs(want) + 1.01 * each * off / size, "out")


@pytest.mark.parametrize("shift", [0, 1, 2])
@pytest.mark.parametrize("wide", [True, False])
def test_residual_norm_of_slices(ccu, shift, wide):
    """Rows of wider tensors on any boundary; rows and columns beside them are left as they were."""
    T, D = 6, 136
    rng = np.random.default_rng(shift)
    xw, xn = bf(rng, T, D + 8)
    g = Guarded(T * (D + 16) * (4 if wide else 2), DEV)
    r = g.view(torch.float32 if wide else torch.bfloat16, (T, D + 16))
    r.copy_(torch.from_numpy(rng.standard_normal((T, D + 16))))
    before, rn = r.clone(), num(r)
    go = Guarded(T * (D + 8) * 2, DEV)
    out = go.view(torch.bfloat16, (T, D + 8))
    out.zero_()
    cut = slice(shift, shift + D)
    ccu.residual_rms_norm(xw[:, cut], r[:, cut], None, scale=2.0, out=out[:, cut])
    want, sums = ref.residual(xn[:, cut], rn[:, cut], None, None, 2.0, 1e-6)
    within(num(out[:, cut]), want, (HALF + 2 * NORM) * np.abs(want) + 2.0 ** -22, "out")
    within(num(r[:, cut]), sums, ((0 if wide else HALF) + 2.0 ** -23) * np.abs(sums) + 2.0 ** -23 * np.abs(rn[:, cut]), "residual")
    keep = [i for i in range(D + 16) if not cut.start <= i < cut.stop]
    assert torch.equal(r[:, keep], before[:, keep]) and g.guards_intact() and go.guards_intact()
    assert not out[:, [i for i in keep if i < D + 8]].any()


def test_norms_on_a_stream_in_a_graph_and_of_nothing(ccu):
    T, H, P = 9, 4, 128
    rng = np.random.default_rng(2)
    (x, xn), (z, zn), (w, wn), (r, rn) = bf(rng, T, H, P), bf(rng, T, H, P), bf(rng, P), bf(rng, T, H * P)
    y, out = torch.empty_like(x), torch.empty_like(r)
    first = r.clone()

    def call():
        ccu.gated_rms_norm(x, z, w, out=y)
        ccu.residual_rms_norm(y.flatten(1), r, None, out=out)

    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    eager = (y.clone(), out.clone(), r.clone())
    graph = in_a_graph(call)
    with torch.cuda.stream(side):
        r.copy_(first)
        graph.replay()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, (y, out, r)))
    want = ref.gated(xn, zn, wn, 1e-6, True)
    within(num(y), want, (HALF + NORM) * np.abs(want), "gated")
    assert ccu.gated_rms_norm(x[:0], z[:0], w).shape == (0, H, P) and ccu.residual_rms_norm(r[:0], r[:0]).shape == (0, H * P)
    assert ccu.gated_rms_norm(x[..., :0], None, None).shape == (T, H, 0)


def test_refusals(ccu):
    bf16 = dict(device=DEV, dtype=torch.bfloat16)
    x, v = torch.zeros(4, 8, **bf16), torch.zeros(4, 2, 8, **bf16)
    A, state, cu = torch.zeros(2, device=DEV), torch.zeros(3, 2, 8, 8, device=DEV), i32([0, 4])
    a = torch.zeros(4, 2, **bf16)
    rule = lambda **kw: ccu.gated_delta_rule(**{**dict(q=v, k=v, v=v, a=a, b=a, A=A, cu_seqlens=cu, state=state), **kw})  # noqa: E731
    rule()
    for kw, message in ((dict(q=v.transpose(1, 2)), "q must be"), (dict(k=v[:3]), "k must be"), (dict(a=x), "a must be"),
                        (dict(A=A.double()), "A must be torch.float32"), (dict(state=state[:, :1]), "state must be"),
                        (dict(state=state.permute(0, 1, 3, 2)), "slot of state"), (dict(cu_seqlens=cu[:0]), "cu_seqlens"),
                        (dict(cu_seqlens=cu.long()), "cu_seqlens must be"), (dict(scale=0.0), "scale"),
                        (dict(v=v.requires_grad_(False).clone().requires_grad_()), "inference-only"),
                        (dict(v=torch.zeros(4, 2, 16, **bf16)[..., ::2]), "unit stride"), (dict(state_indices=i32([0, 1])), "state_indices")):
        with pytest.raises(ValueError, match=message):
            rule(**kw)
    with pytest.raises(ValueError, match="multiple of G"):
        ccu.gated_delta_rule(v, v, torch.zeros(4, 3, 8, **bf16), torch.zeros(4, 3, **bf16), torch.zeros(4, 3, **bf16), torch.zeros(3, device=DEV),
                             cu_seqlens=cu, state=torch.zeros(3, 3, 8, 8, device=DEV))
    with pytest.raises(NotImplementedError, match="K <= 256"):
        big = torch.zeros(4, 2, 264, **bf16)
        rule(q=big, k=big, state=torch.zeros(3, 2, 8, 264, device=DEV))
    with pytest.raises(ValueError, match="weight must be"):
        ccu.gated_rms_norm(v, v, x[0, :4])
    with pytest.raises(ValueError, match="torch.float16"):
        ccu.gated_rms_norm(v, v, x[0].half())
    with pytest.raises(ValueError, match="eps"):
        ccu.gated_rms_norm(v, v, x[0], eps=-1.0)
    with pytest.raises(ValueError, match="as weight is"):
        ccu.residual_rms_norm(x, x.clone(), x[0], post_weight=x[0].float())
    with pytest.raises(ValueError, match="residual must be"):
        ccu.residual_rms_norm(x, x[:3].clone())
    with pytest.raises(ValueError, match="unit stride"):
        ccu.residual_rms_norm(x, torch.zeros(8, 4, **bf16).t())


# ------------------------------------------------------------------ together

def test_a_layer_of_them(ccu):
    """Packed prompts through convolution, delta rule, gated norm and residual norm, then tokens on the slots they left,
    against the definitions in 64 bits of every step on what the step before it gave."""
    G, H, K, P, W, D = 2, 4, 64, 64, 4, 256
    rng = np.random.default_rng(20)
    lens, slots, S = [100, 1, 70], [3, 0, 2], 5
    channels, T = 2 * G * K + H * P, sum(lens)
    (weight, weightn), (cbias, cbiasn) = bf(rng, channels, W, scale=0.5), bf(rng, channels, scale=0.1)
    conv = torch.zeros(S, W - 1, channels, dtype=torch.bfloat16, device=DEV).permute(0, 2, 1)
    state = torch.zeros(S, H, P, K, device=DEV)
    A, An = f32(-rng.uniform(1, 16, H))
    w, wn = bf(rng, P)
    cu, at = offsets(lens), i32(slots)

    def norms(y, yn_shape, r, z, rn, zn):
        o = ccu.gated_rms_norm(y, z, w)
        want = ref.gated(num(y), zn, wn, 1e-6, True)
        within(num(o), want, (HALF + NORM) * np.abs(want), "gated")
        h = ccu.residual_rms_norm(o.flatten(1), r, None, scale=0.5)
        want, sums = ref.residual(num(o).reshape(yn_shape), rn, None, None, 0.5, 1e-6)
        within(num(h), want, (HALF + 2 * NORM) * np.abs(want) + 2.0 ** -22, "residual norm")

    (x, xn), (z, zn), (r, rn) = bf(rng, T, channels), bf(rng, T, H, P), bf(rng, T, D)
    (a, an), (b, bn) = bf(rng, T, H, scale=0.5), bf(rng, T, H)
    u = ccu.causal_conv1d_packed(x, weight, cbias, "silu", cu_seqlens=cu, conv_state=conv, conv_state_indices=at)
    y = ccu.gated_delta_rule(u[:, :G * K].unflatten(1, (G, K)), u[:, G * K:2 * G * K].unflatten(1, (G, K)), u[:, 2 * G * K:].unflatten(1, (H, P)),
                             a, b, A, cu_seqlens=cu, state=state, state_indices=at)
    un = num(u)
    o, off, s, bound = ref.rule(un[:, :G * K].reshape(T, G, K), un[:, G * K:2 * G * K].reshape(T, G, K), un[:, 2 * G * K:].reshape(T, H, P), an, bn,
                                An, None, lens, np.zeros((S, H, P, K)), slots, None)
    within(num(y), o, HALF * np.abs(o) + off, "prompts")
    within(num(state), s, bound[..., None], "state")
    norms(y, (T, D), r, z, rn, zn)
    d = dict(A=(A, An), weight=(weight, weightn), cbias=(cbias, cbiasn), dt_bias=(None, np.zeros(H)))
    for _ in range(3):
        d.update(qkv=bf(rng, 3, channels), a=bf(rng, 3, H, scale=0.5), b=bf(rng, 3, H), state=(state, num(state)), conv=(conv, num(conv)))
        o, off, s, bound, c = want_token(d, slots, G, "silu")
        y = ccu.gated_delta_update(d["qkv"][0], d["a"][0], d["b"][0], A, state, conv, weight, cbias, "silu", groups=G, state_indices=at)
        within(num(y), o, HALF * np.abs(o) + off, "token")
        within(num(state), s, bound[..., None], "state")
        assert np.array_equal(num(conv), c)
        (z, zn), (r, rn) = bf(rng, 3, H, P), bf(rng, 3, D)
        norms(y, (3, D), r, z, rn, zn)
