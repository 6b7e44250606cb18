"""The state-space operators on the GPU against their definitions in 64 bits."""
import itertools

import numpy as np
import pytest
import torch

import ssm_reference as ref
from gpu_util import Guarded

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 2.0 ** -22  # error of one token's decay and update, see ssm_reference


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


class Scan:
    """Inputs of one scan; ``wide`` takes x, B, C, dt and z as slices of one wider row."""

    def __init__(self, lens, H, P, K, G, seed=0, gate=True, skip=True, bias=True, initial=None, slots=None, spare=2,
                 wide=False, shift=0, decay=(1.0, 16.0)):
        rng = np.random.default_rng(seed)
        T, self.lens, self.dims = sum(lens), lens, (H, P, K, G)
        if wide:
            w = 2 * H * P + 2 * G * K + H + shift
            w = w if shift else (w + 7) // 8 * 8
            row, rown = bf(rng, max(T, 1), w)
            row, rown = row[:T], rown[:T]
            cut = np.cumsum([shift, H * P, H * P, G * K, G * K, H])
            part = [(row[:, a:b], rown[:, a:b]) for a, b in zip(cut, cut[1:])]
        else:
            part = [bf(rng, T, n) for n in (H * P, H * P, G * K, G * K, H)]
        shape = [(H, P), (H, P), (G, K), (G, K), (H,)]
        (self.z, self.zn), (self.x, self.xn), (self.B, self.Bn), (self.C, self.Cn), (self.dt, self.dtn) = [
            (t.unflatten(1, s) if len(s) > 1 else t, a.reshape((T,) + s)) for (t, a), s in zip(part, shape)]
        if not gate:
            self.z = self.zn = None
        self.A, self.An = f32(-rng.uniform(*decay, H))
        self.D, self.Dn = f32(rng.uniform(0.5, 1.5, H)) if skip else (None, None)
        step = np.exp(rng.uniform(np.log(1e-3), np.log(1e-1), H))
        self.bias, self.biasn = f32(step + np.log(-np.expm1(-step))) if bias else (None, None)
        n = len(lens)
        self.slots = list(rng.permutation(n + spare)[:n]) if slots is None else slots
        self.S = max([n + spare] + [s + 1 for s in self.slots if s < 100])
        self.state, self.staten = f32(rng.standard_normal((self.S, H, P, K)) * 0.1)
        self.has = initial

    def run(self, ccu, state=None, **kw):
        return ccu.selective_scan(self.x, self.dt, self.A, self.B, self.C, cu_seqlens=offsets(self.lens),
                                  ssm_state=self.state if state is None else state, D=self.D, z=self.z, dt_bias=self.bias,
                                  state_indices=i32([int(s) for s in self.slots]),
                                  has_initial_state=None if self.has is None else i32(self.has), **kw)

    def want(self, **kw):
        return ref.scan(self.xn, self.dtn, self.An, self.Bn, self.Cn, self.Dn, self.zn, self.biasn, self.lens, self.staten,
                        self.slots, self.has, **kw)

    def check(self, out, state, loose=0.0, what="", **kw):
        o, m, s, sm = self.want(**kw)
        n = max(max(self.lens), 1) + 4
        within(num(out), o, 2.0 ** -8 * np.abs(o) + (n * EPS + loose) * m + 1e-30, f"{what} out")
        within(num(state), s, n * EPS * sm + 1e-30, f"{what} state")


# what the chunked kernel may be off: it rounds two factors of every term to BF16 (2^-9 each)
LOOSE = {"auto": 2.0 ** -8, "recurrent": 0.0, "chunked": 2.0 ** -8}

SHAPES = [(2, 64, 128, 1), (4, 64, 64, 2), (3, 128, 128, 1), (2, 8, 16, 1), (6, 40, 24, 3), (1, 5, 7, 1), (2, 33, 200, 1),
          (2, 1, 1, 2), (1, 80, 256, 1), (8, 16, 96, 8)]
LENS = [[1], [37], [128, 129, 0, 1], [5, 0, 0, 3, 260], [300]]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("route", ["auto", "recurrent"])
def test_scan(ccu, shape, lens, route):
    H, P, K, G = shape
    s = Scan(lens, H, P, K, G, seed=len(lens) + P, initial=[i % 2 for i in range(len(lens))])
    out = s.run(ccu, route=route)
    s.check(out, s.state, LOOSE[route], route)


@pytest.mark.parametrize("gate,skip,bias", list(itertools.product([True, False], repeat=3)))
def test_scan_options(ccu, gate, skip, bias):
    s = Scan([70, 3], 2, 64, 64, 1, seed=5, gate=gate, skip=skip, bias=bias, initial=[1, 0])
    s.check(s.run(ccu), s.state, LOOSE["auto"])


def test_scan_without_softplus_and_default_slots(ccu):
    s = Scan([9, 20], 2, 8, 16, 1, seed=6, slots=[0, 1], bias=False)
    s.dt, s.dtn = s.dt.abs() * 0.1, None
    s.dtn = num(s.dt)
    out = ccu.selective_scan(s.x, s.dt, s.A, s.B, s.C, cu_seqlens=offsets(s.lens), ssm_state=s.state, D=s.D, z=s.z,
                             dt_softplus=False)
    s.check(out, s.state, LOOSE["auto"], dt_softplus=False)


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("shape", [(2, 64, 128, 1), (4, 40, 24, 2)], ids=str)
def test_scan_of_slices(ccu, shape, shift):
    """Slices of one projection row; an odd shift leaves every row on a 2-byte boundary."""
    s = Scan([130, 1, 40], *shape, seed=7, wide=True, shift=shift, initial=[1, 1, 0])
    s.check(s.run(ccu), s.state, LOOSE["auto"])


@pytest.mark.parametrize("route", ["auto", "recurrent"])
def test_scan_padding_and_range(ccu, route):
    """Slots of -1 and out of range: outputs +0, nothing kept, the range reported."""
    s = Scan([20, 150, 3, 140], 2, 64, 64, 1, seed=8, slots=[1, -1, 1000, 0], initial=[1, 1, 1, 1])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = s.run(ccu, route=route, status=status)
    s.check(out, s.state, LOOSE[route])
    assert status.item() == ccu.CCU_DEVERR_RANGE
    bits = out.view(torch.int16)[20:173]
    assert not bits.any()


@pytest.mark.parametrize("route", ["auto", "recurrent"])
def test_scan_keeps_nan_and_inf_apart(ccu, route):
    """A sequence of NaN or infinities reaches neither its neighbours nor their states."""
    for bad in (float("nan"), float("inf")):
        s = Scan([100, 33, 150], 2, 64, 128, 1, seed=9, slots=[0, 1, 2], spare=0, initial=[0, 0, 1])
        for t in (s.x, s.B, s.C, s.dt, s.z):
            t[100:133] = bad
        s.state[1] = bad  # not an initial state: must not be read
        for a in (s.xn, s.Bn, s.Cn, s.dtn, s.zn):
            a[100:133] = 0
        s.staten[1] = 0
        out, state = s.run(ccu, route=route), s.state
        out[100:133], state[1] = 0, 0
        want = s.want()
        o, m = want[0].copy(), want[1].copy()
        o[100:133], m[100:133] = 0, 0
        within(num(out), o, 2.0 ** -8 * np.abs(o) + (160 * EPS + LOOSE[route]) * m, "out")
        within(num(state)[[0, 2]], want[2][[0, 2]], 160 * EPS * want[3][[0, 2]], "state")


@pytest.mark.parametrize("route", ["auto", "recurrent"])
def test_scan_of_extreme_decays(ccu, route):
    """Steps from 1e-8 to 60 and decays from none to exp(-1000): no overflow, no NaN."""
    s = Scan([200], 4, 64, 64, 1, seed=10, bias=False, initial=[1])
    s.dt = torch.linspace(-20, 60, 800, device=DEV).view(200, 4)[torch.randperm(200)].to(torch.bfloat16).contiguous()
    s.dtn = num(s.dt)
    s.A, s.An = f32([0.0, -1e-4, -1.0, -16.0])
    s.check(s.run(ccu, route=route), s.state, LOOSE[route])


def test_scan_in_pieces(ccu):
    """A prompt in three calls, then token by token, against the whole prompt's definition."""
    H, P, K, G = 2, 64, 64, 1
    s = Scan([190], H, P, K, G, seed=11, slots=[1])
    got, at = [], 0
    for n in (100, 1, 70):
        cut = slice(at, at + n)
        got.append(ccu.selective_scan(s.x[cut], s.dt[cut], s.A, s.B[cut], s.C[cut], cu_seqlens=offsets([n]), ssm_state=s.state,
                                      D=s.D, z=s.z[cut], dt_bias=s.bias, state_indices=i32([1]),
                                      has_initial_state=i32([1 if at else 0])))
        at += n
    for t in range(at, 190):
        xbc = torch.cat([s.x[t].flatten(), s.B[t].flatten(), s.C[t].flatten()])[None]
        got.append(ccu.selective_state_update(xbc, s.dt[t:t + 1], s.A, s.state, D=s.D, z=s.z[t:t + 1], dt_bias=s.bias,
                                              groups=G, state_indices=i32([1])))
    s.check(torch.cat(got), s.state, LOOSE["auto"])


def test_scan_guard_bands(ccu):
    """Nothing outside out, the used slots and the sequences' rows is written."""
    s = Scan([3, 130], 2, 24, 48, 1, seed=12, slots=[0, 3])
    H, P, K, G = s.dims
    go, gs = Guarded(140 * H * P * 2, DEV), Guarded(4 * H * P * K * 4, DEV)
    out, state = go.view(torch.bfloat16, (140, H, P)), gs.view(torch.float32, (4, H, P, K))
    state.copy_(s.state[:4])
    full = torch.nn.functional.pad(s.x, (0, 0, 0, 0, 0, 7)), torch.nn.functional.pad(s.dt, (0, 0, 0, 7))
    B, C = (torch.nn.functional.pad(t, (0, 0, 0, 0, 0, 7)) for t in (s.B, s.C))
    before = out.clone()
    ccu.selective_scan(full[0], full[1], s.A, B, C, cu_seqlens=offsets(s.lens), ssm_state=state, D=s.D, dt_bias=s.bias,
                       state_indices=i32(s.slots), out=out)
    s.z = s.zn = None
    s.staten = s.staten[:4]
    s.check(out[:133], state, LOOSE["auto"])
    assert torch.equal(out[133:].view(torch.int16), before[133:].view(torch.int16))
    assert go.guards_intact() and gs.guards_intact()


def test_scan_far_slots_and_rows(ccu):
    """Slots and rows whose offsets pass 2^31 elements."""
    H, P, K, G = 1, 64, 64, 1
    s = Scan([70], H, P, K, G, seed=13, slots=[2], spare=0)
    stride = (1 << 30) + 4096
    far = torch.zeros(2 * stride + P * K, device=DEV)
    state = far.as_strided((3, H, P, K), (stride, P * K, K, 1))
    rows = (1 << 31) // 60
    wide = torch.zeros(69 * rows + 64, dtype=torch.bfloat16, device=DEV)
    x = wide.as_strided((70, H, P), (rows, P, 1))
    x.copy_(s.x)
    s.x = x
    s.staten[:] = 0
    out = s.run(ccu, state=state)
    s.check(out, state.clone(), LOOSE["auto"])


def test_scan_on_another_stream_and_in_a_graph(ccu):
    s = Scan([300, 140], 2, 64, 128, 1, seed=14, initial=[1, 0])
    first = s.state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)  # the default stream would read before the inputs are final
        s.x.mul_(1)
        out = s.run(ccu)
    side.synchronize()
    s.check(out, s.state, LOOSE["auto"], "stream")
    s.state.copy_(first)
    cu, slots, has = offsets(s.lens), i32([int(v) for v in s.slots]), i32(s.has)
    held = torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ccu.selective_scan(s.x, s.dt, s.A, s.B, s.C, cu_seqlens=cu, ssm_state=s.state, D=s.D, z=s.z, dt_bias=s.bias,
                           state_indices=slots, has_initial_state=has, out=held)
    for _ in range(2):
        s.state.copy_(first)
        held.zero_()
        graph.replay()
        torch.cuda.synchronize()
        s.check(held, s.state, LOOSE["auto"], "graph")


# the chunked kernel: whole and partial chunks, blocks of 64 channels and what is left, few states
CHUNKED = [(2, 64, 128, 1), (2, 8, 8, 1), (4, 72, 64, 2), (1, 136, 120, 1), (8, 64, 16, 8), (3, 48, 104, 1)]


@pytest.mark.parametrize("shape", CHUNKED, ids=str)
@pytest.mark.parametrize("lens", [[1], [31, 33], [128], [257, 0, 127, 32], [700, 5]], ids=str)
@pytest.mark.parametrize("initial", [False, True])
def test_scan_chunked(ccu, shape, lens, initial):
    H, P, K, G = shape
    s = Scan(lens, H, P, K, G, seed=sum(lens) + K, initial=[1] * len(lens) if initial else None, gate=initial, skip=not initial)
    out = s.run(ccu, route="chunked")
    s.check(out, s.state, LOOSE["chunked"])


@pytest.mark.parametrize("decay", [(1e-5, 1e-4), (0.01, 0.1), (100.0, 4000.0)], ids=str)
def test_scan_chunked_slow_and_fast_decays(ccu, decay):
    """States that live for thousands of tokens and states that are gone after one."""
    s = Scan([1500], 2, 64, 64, 1, seed=40, decay=decay, initial=[1])
    out = s.run(ccu, route="chunked")
    s.check(out, s.state, LOOSE["chunked"])


@pytest.mark.parametrize("lens,heads,initial", [([5000], 2, [1]), ([3000, 1, 0, 700, 2048], 3, [1, 0, 1, 1, 0]),
                                                ([513, 1024, 1536, 1537], 1, None), ([4096], 1, [0])], ids=str)
def test_scan_cut_into_segments(ccu, lens, heads, initial):
    """Too few sequences and heads to fill the card: segments, their states joined; sequences that end on,
    before and behind a segment's end, empty ones, and a padding sequence."""
    s = Scan(lens, heads, 64, 64, 1, seed=44, initial=initial)
    if len(lens) > 3:
        s.slots[3] = -1
    args = dict(route="chunked")
    out = s.run(ccu, **args)
    s.check(out, s.state, LOOSE["chunked"])


def test_scan_workspace(ccu):
    """The caller's workspace serves as well as torch's; one that is too small is refused."""
    a = Scan([4000], 2, 64, 64, 1, seed=45, slots=[0])
    b = Scan([4000], 2, 64, 64, 1, seed=45, slots=[0])
    out = a.run(ccu)
    work = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    assert torch.equal(out, b.run(ccu, workspace=work)) and torch.equal(a.state, b.state)
    with pytest.raises(ValueError, match="workspace"):
        b.run(ccu, workspace=work[:1024])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")], ids=str)
@pytest.mark.parametrize("which", ["x", "B", "C", "dt", "z"])
def test_scan_chunked_is_causal_for_nan_and_inf(ccu, bad, which):
    """A NaN or an infinity at token 150 changes no output before it, and only its own channel
    when it comes in x or z."""
    s = Scan([300], 1, 64, 64, 1, seed=41, initial=[1])
    clean = s.run(ccu, route="chunked", state=s.state.clone())
    t = getattr(s, which)
    if which == "dt":
        t[150] = bad
    else:
        t[150, 0, 5] = bad
    out = s.run(ccu, route="chunked")
    assert torch.equal(out[:150], clean[:150])
    if which in ("x", "z"):
        keep = [c for c in range(64) if c != 5]
        assert torch.equal(out[:, :, keep], clean[:, :, keep])
    if which == "x":
        assert not torch.isfinite(out[150:, :, 5].float()).any()
        assert not torch.isfinite(s.state[int(s.slots[0]), 0, 5]).any()
    if which in ("C", "z"):
        assert torch.equal(out[151:], clean[151:])


def test_scan_chunked_padding_and_range(ccu):
    s = Scan([20, 150, 3, 140], 2, 64, 64, 1, seed=42, slots=[1, -1, 1000, 0], initial=[1, 1, 1, 1])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = s.run(ccu, route="chunked", status=status)
    s.check(out, s.state, LOOSE["chunked"])
    assert status.item() == ccu.CCU_DEVERR_RANGE
    assert not out.view(torch.int16)[20:173].any()


def test_scan_chunked_repeats_its_bits(ccu):
    """The same call twice, alone and with other work on the card, gives the same bits."""
    s = Scan([900, 64, 333], 8, 64, 128, 2, seed=43, initial=[1, 0, 1])
    first = s.state.clone()
    a = s.run(ccu, route="chunked")
    kept = s.state.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(20):
            torch.randn(1 << 22, device=DEV).sort()
    s.state.copy_(first)
    b = s.run(ccu, route="chunked")
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(s.state, kept)
    assert ccu.ccu_conv1d_take_device_error() == (0, 0)


# ------------------------------------------------------------------ packed convolution

@pytest.mark.parametrize("D", [8, 24, 7, 136])
@pytest.mark.parametrize("W,L", [(4, 3), (4, 5), (3, 2), (2, 1), (2, 4)])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("last", [True, False], ids=["channel_last", "compact"])
def test_conv_packed(ccu, D, W, L, act, last):
    rng = np.random.default_rng(D + W)
    lens = [1, 0, 2, 3, 70, 0, 33, 200, 4]
    T, n = sum(lens), len(lens)
    x, xn = bf(rng, T, D)
    w, wn = bf(rng, D, W)
    b, bn = bf(rng, D)
    st, sn = bf(rng, n + 2, D, L)
    if last:
        st = st.permute(0, 2, 1).contiguous().permute(0, 2, 1)
    slots = rng.permutation(n + 2)[:n].astype(np.int32)
    slots[4] = -1
    has = [i % 3 != 0 for i in range(n)]
    out = ccu.causal_conv1d_packed(x, w, b, act, cu_seqlens=offsets(lens), conv_state=st, conv_state_indices=i32(slots.tolist()),
                                   has_initial_state=i32([int(v) for v in has]))
    o, m, s = ref.conv(xn, wn, bn, act is not None, lens, sn, slots, has)
    within(num(out), o, 2.0 ** -8 * np.abs(o) + 8 * 2.0 ** -23 * m, "out")
    assert np.array_equal(num(st), s)
    assert not out.view(torch.int16)[6:76].any()  # the padding sequence: +0


@pytest.mark.parametrize("D", [64, 20])
def test_conv_packed_equals_the_prefill(ccu, D):
    """Each sequence's bits are those of causal_conv1d_fwd on it alone."""
    rng = np.random.default_rng(3)
    lens = [5, 64, 131, 2]
    x, _ = bf(rng, sum(lens), D)
    w, _ = bf(rng, D, 4)
    b, _ = bf(rng, D)
    st, _ = bf(rng, 4, 3, D)
    st = st.permute(0, 2, 1)
    old = st.clone()
    out = ccu.causal_conv1d_packed(x, w, b, "silu", cu_seqlens=offsets(lens), conv_state=st, has_initial_state=i32([1] * 4))
    at = 0
    for i, n in enumerate(lens):
        y, fin = ccu.causal_conv1d_fwd(x[None, at:at + n].clone().permute(0, 2, 1), w, b, "silu", initial_states=old[i:i + 1].clone(),
                                       return_final_states=True)
        assert torch.equal(out[at:at + n].view(torch.int16), y[0].t().contiguous().view(torch.int16))
        assert torch.equal(st[i], fin[0])
        at += n


def test_conv_packed_slices_offsets_and_range(ccu):
    """Rows that are slices on odd boundaries, rows outside every sequence, a slot out of range."""
    rng = np.random.default_rng(4)
    row, rown = bf(rng, 40, 51)
    w, wn = bf(rng, 48, 4)
    g = Guarded(40 * 48 * 2, DEV)
    out = g.view(torch.bfloat16, (40, 48))
    before = out.clone()
    st, sn = bf(rng, 2, 48, 3)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ccu.causal_conv1d_packed(row[:, 3:], w, cu_seqlens=i32([2, 20, 25, 33]), conv_state=st, conv_state_indices=i32([1, 5, 0]),
                             out=out, status=status)
    o, m, s = ref.conv(rown[2:33, 3:], wn, None, False, [18, 5, 8], sn, [1, 5, 0], None)
    within(num(out)[2:33], o, 2.0 ** -8 * np.abs(o) + 8 * 2.0 ** -23 * m, "out")
    assert np.array_equal(num(st), s)
    assert status.item() == ccu.CCU_DEVERR_RANGE
    for cut in (slice(0, 2), slice(33, 40)):
        assert torch.equal(out[cut].view(torch.int16), before[cut].view(torch.int16))
    assert g.guards_intact()


def test_conv_packed_without_states(ccu):
    rng = np.random.default_rng(5)
    x, xn = bf(rng, 30, 16)
    w, wn = bf(rng, 16, 4)
    out = ccu.causal_conv1d_packed(x, w, cu_seqlens=offsets([10, 20]))
    o, m, _ = ref.conv(xn, wn, None, False, [10, 20], None, [0, 1], None)
    within(num(out), o, 2.0 ** -8 * np.abs(o) + 8 * 2.0 ** -23 * m, "out")


def test_conv_packed_many_sequences_and_wild_offsets(ccu):
    """Thousands of short sequences; offsets out of range or out of order reach no memory."""
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 4, 3000).tolist()
    x, xn = bf(rng, sum(lens), 16)
    w, wn = bf(rng, 16, 4)
    st, sn = bf(rng, 3000, 16, 3)
    out = ccu.causal_conv1d_packed(x, w, None, "silu", cu_seqlens=offsets(lens), conv_state=st, has_initial_state=i32([1] * 3000))
    o, m, s = ref.conv(xn, wn, None, True, lens, sn, list(range(3000)), [1] * 3000)
    within(num(out), o, 2.0 ** -8 * np.abs(o) + 8 * 2.0 ** -23 * m, "out")
    assert np.array_equal(num(st), s)
    g = Guarded(20 * 16 * 2, DEV)
    ccu.causal_conv1d_packed(x[:20], w, cu_seqlens=i32([-5, 12, 4, 2_000_000_000]), out=g.view(torch.bfloat16, (20, 16)))
    assert g.guards_intact()


# ------------------------------------------------------------------ single-token update

@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("N", [1, 5])
@pytest.mark.parametrize("W,L", [(4, 3), (2, 4), (0, 0), (6, 5)])
def test_update(ccu, shape, N, W, L):
    H, P, K, G = shape
    rng = np.random.default_rng(N + P + W)
    channels, S = H * P + 2 * G * K, N + 2
    xbc, xn = bf(rng, N, channels)
    dt, dtn = bf(rng, N, H)
    z, zn = bf(rng, N, H, P)
    A, An = f32(-rng.uniform(1, 16, H))
    D, Dn = f32(rng.uniform(0.5, 1.5, H))
    bias, biasn = f32(rng.uniform(-6, -2, H))
    state, sn = f32(rng.standard_normal((S, H, P, K)))
    slots = rng.permutation(S)[:N]
    if N > 1:
        slots[1] = -1
    kw, conv = {}, None
    xbcn, xmag = xn, np.abs(xn)
    if W:
        w, wn = bf(rng, channels, W, scale=0.5)
        b, bn = bf(rng, channels, scale=0.1)
        conv, cn = bf(rng, S, channels, L)
        if N == 5:
            conv = conv.permute(0, 2, 1).contiguous().permute(0, 2, 1)
        kw = dict(conv_state=conv, conv_weight=w, conv_bias=b, activation="silu")
        xbcn, xmag, cs = ref.conv(xn, wn, bn, True, [1] * N, cn, slots, [1] * N)
    out = ccu.selective_state_update(xbc, dt, A, state, D=D, z=z, dt_bias=bias, groups=G, state_indices=i32(slots.tolist()), **kw)
    cut = [H * P, H * P + G * K]
    x, B, C = (a.reshape(N, *s) for a, s in zip(np.split(xbcn, cut, 1), ((H, P), (G, K), (G, K))))
    o, m, s, sm = ref.scan(x, dtn, An, B, C, Dn, zn, biasn, [1] * N, sn, slots, [1] * N)
    # the convolution's own error (8 units of its magnitude) in x, B and C, each a factor of a term
    if W:
        xm, Bm, Cm = (a.reshape(N, *t) for a, t in zip(np.split(xmag, cut, 1), ((H, P), (G, K), (G, K))))
        m = ref.scan(xm, dtn, An, Bm, Cm, Dn, zn, biasn, [1] * N, np.abs(sn), slots, [1] * N)[0]
        m = np.abs(m)
        sm = ref.scan(xm, dtn, An, Bm, Cm, Dn, zn, biasn, [1] * N, np.abs(sn), slots, [1] * N)[2]
    within(num(out), o, 2.0 ** -8 * np.abs(o) + 24 * EPS * m + 1e-30, "out")
    within(num(state), s, 24 * EPS * sm + 1e-30, "state")
    if W:
        assert np.array_equal(num(conv), cs)
    if N > 1:
        assert not out.view(torch.int16)[1].any()


@pytest.mark.parametrize("shift", [0, 1])
def test_update_of_slices(ccu, shift):
    """Slices of one projection row (odd boundaries with a shift), no gate, slots further apart."""
    H, P, K, G, N = 4, 32, 64, 2, 9
    rng = np.random.default_rng(20 + shift)
    channels = H * P + 2 * G * K
    row, rown = bf(rng, N, channels + H + shift + 8)
    cut = shift, shift + channels, shift + channels + H
    A, An = f32(-rng.uniform(1, 16, H))
    far = torch.randn(N, 3, H, P, K, device=DEV)
    state = far[:, 1]
    sn = num(state)
    before = far.clone()
    out = ccu.selective_state_update(row[:, cut[0]:cut[1]], row[:, cut[1]:cut[2]], A, state, groups=G)
    v = rown[:, cut[0]:cut[1]]
    x, B, C = v[:, :H * P].reshape(N, H, P), v[:, H * P:H * P + G * K].reshape(N, G, K), v[:, H * P + G * K:].reshape(N, G, K)
    o, m, s, sm = ref.scan(x, rown[:, cut[1]:cut[2]], An, B, C, None, None, None, [1] * N, sn, list(range(N)), [1] * N)
    within(num(out), o, 2.0 ** -8 * np.abs(o) + 8 * EPS * m, "out")
    within(num(state), s, 8 * EPS * sm, "state")
    assert torch.equal(far[:, 0], before[:, 0]) and torch.equal(far[:, 2], before[:, 2])


def test_update_padding_and_range(ccu):
    """Rows of NaN on slots -1 and out of range: outputs +0, no state touched, the range reported."""
    H, P, K = 2, 64, 128
    C = H * P + 2 * K
    xbc = torch.full((4, C), float("nan"), dtype=torch.bfloat16, device=DEV)
    dt = torch.full((4, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    xbc[2], dt[2] = 0.5, 0.5
    state = torch.randn(2, H, P, K, device=DEV)
    conv = torch.randn(2, C, 3, device=DEV).to(torch.bfloat16)
    w = torch.randn(C, 4, device=DEV).to(torch.bfloat16)
    s0, c0 = state.clone(), conv.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = ccu.selective_state_update(xbc, dt, -torch.ones(H, device=DEV), state, conv, w, state_indices=i32([-1, 2, 0, -7]),
                                     status=status)
    assert not out.view(torch.int16)[[0, 1, 3]].any()
    assert torch.isfinite(out[2].float()).all()
    assert torch.equal(state[1], s0[1]) and torch.equal(conv[1], c0[1])
    assert not torch.equal(state[0], s0[0])
    assert status.item() == ccu.CCU_DEVERR_RANGE


def test_update_far_slot_stream_and_graph(ccu):
    H, P, K, N = 2, 64, 128, 3
    rng = np.random.default_rng(22)
    C = H * P + 2 * K
    stride = (1 << 30) + 4096
    far = torch.zeros(2 * stride + H * P * K, device=DEV)
    state = far.as_strided((3, H, P, K), (stride, P * K, K, 1))
    conv, cn = bf(rng, 3, C, 3)
    first, sn = f32(rng.standard_normal((3, H, P, K)))
    w, wn = bf(rng, C, 4)
    A, An = f32([-1, -2])
    xs = [bf(rng, N, C) for _ in range(3)]
    dts = [bf(rng, N, H) for _ in range(3)]
    state.copy_(first)
    c0 = conv.clone()
    # a chain of calls with nothing in between, then the same as one graph
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs = [ccu.selective_state_update(x[0], d[0], A, state, conv, w, None, "silu") for x, d in zip(xs, dts)]
    side.synchronize()
    s, sm, c = sn, np.abs(sn), cn
    for i, (x, d, got) in enumerate(zip(xs, dts, outs)):
        v, vm, c = ref.conv(x[1], wn, None, True, [1] * N, c, [0, 1, 2], [1] * N)
        # as in test_update: magnitudes from the convolution's, 24 units a step
        both = []
        for st, a in ((s, v), (sm, vm)):
            x_, B_, C_ = (p.reshape(N, *t) for p, t in zip(np.split(a, [H * P, H * P + K], 1), ((H, P), (1, K), (1, K))))
            both.append(ref.scan(x_, d[1], An, B_, C_, None, None, None, [1] * N, st, [0, 1, 2], [1] * N))
        (o, _, s, _), (m, _, sm, _) = both
        within(num(got), o, 2.0 ** -8 * np.abs(o) + 24 * (i + 1) * EPS * m, "out")
    within(num(state.clone()), s, 24 * 3 * EPS * sm, "state")
    assert np.array_equal(num(conv), c)
    last = state.clone()
    state.copy_(first)
    conv.copy_(c0)
    hold = [torch.empty(N, H, P, dtype=torch.bfloat16, device=DEV) for _ in xs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, d, o in zip(xs, dts, hold):
            ccu.selective_state_update(x[0], d[0], A, state, conv, w, None, "silu", out=o)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(hold, outs))
    assert torch.equal(state, last)


# ------------------------------------------------------------------ 4-bit products

@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 17, 64, 65, 130])
@pytest.mark.parametrize("I,O,group", [(128, 16, 128), (32, 1, 32), (96, 37, 32), (192, 130, 64), (2048, 40, 128), (4224, 33, 64)])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4(ccu, M, I, O, group, zeros):
    rng = np.random.default_rng(M + I)
    x, xn = bf(rng, M, I)
    q = rng.integers(0, 256, (O, I // 2), dtype=np.uint8)
    s, sn = bf(rng, O, I // group)
    z, zn = None, None
    if zeros:
        zn = rng.integers(0, 16, (O, I // group)).astype(np.float64)
        z = torch.from_numpy(zn).to(torch.bfloat16).to(DEV)
    out = ccu.w4_matmul(x, torch.from_numpy(q).to(DEV), s, z)
    o, m = ref.w4(xn, q, sn, zn, group)
    within(num(out), o, 2.0 ** -8 * np.abs(o) + I * 2.0 ** -23 * m, "out")


def test_w4_zero_points_with_fractions(ccu):
    """A zero point need not be whole: any BF16 value, also one that an integer sum would drop."""
    rng = np.random.default_rng(30)
    x, xn = bf(rng, 3, 256)
    q = rng.integers(0, 256, (24, 128), dtype=np.uint8)
    s, sn = bf(rng, 24, 2)
    z, zn = bf(rng, 24, 2, scale=5.0)
    out = ccu.w4_matmul(x, torch.from_numpy(q).to(DEV), s, z)
    o, m = ref.w4(xn, q, sn, zn, 128)
    # the sums q x and z x may be formed apart: their magnitudes add up
    far = np.abs(xn) @ (np.repeat(np.abs(zn) + 15, 128, 1) * np.repeat(np.abs(sn), 128, 1)).T
    within(num(out), o, 2.0 ** -8 * np.abs(o) + 256 * 2.0 ** -23 * far, "out")


@pytest.mark.parametrize("shift", [0, 1, 4])
def test_w4_strides_and_guards(ccu, shift):
    rng = np.random.default_rng(31)
    row, rown = bf(rng, 6, 300)
    x, xn = row[:, shift:shift + 256], rown[:, shift:shift + 256]
    q = rng.integers(0, 256, (50, 128), dtype=np.uint8)
    s, sn = bf(rng, 50, 4)
    g = Guarded(6 * 61 * 2, DEV)
    wide = g.view(torch.bfloat16, (6, 61))
    before = wide.clone()
    ccu.w4_matmul(x, torch.from_numpy(q).to(DEV), s, out=wide[:, 3:53])
    o, m = ref.w4(xn, q, sn, None, 64)
    within(num(wide)[:, 3:53], o, 2.0 ** -8 * np.abs(o) + 256 * 2.0 ** -23 * m, "out")
    for cut in (slice(0, 3), slice(53, 61)):
        assert torch.equal(wide[:, cut].contiguous().view(torch.int16), before[:, cut].contiguous().view(torch.int16))
    assert g.guards_intact()


def test_w4_unaligned_weights(ccu):
    """Weights that begin on a 4-byte boundary only."""
    rng = np.random.default_rng(32)
    x, xn = bf(rng, 4, 128)
    q = rng.integers(0, 256, (20, 64), dtype=np.uint8)
    buf = torch.zeros(20 * 64 + 4, dtype=torch.uint8, device=DEV)
    buf[4:] = torch.from_numpy(q).to(DEV).flatten()
    s, sn = bf(rng, 20, 1)
    out = ccu.w4_matmul(x, buf[4:].view(20, 64), s)
    o, m = ref.w4(xn, q, sn, None, 128)
    within(num(out), o, 2.0 ** -8 * np.abs(o) + 128 * 2.0 ** -23 * m, "out")


def test_w4_keeps_nan_rows_apart(ccu):
    """A row of NaN or infinities stays in its own outputs."""
    rng = np.random.default_rng(33)
    x, xn = bf(rng, 5, 128)
    x[2], x[4] = float("nan"), float("inf")
    q = rng.integers(0, 256, (20, 64), dtype=np.uint8)
    s, sn = bf(rng, 20, 1)
    out = num(ccu.w4_matmul(x, torch.from_numpy(q).to(DEV), s))
    o, m = ref.w4(xn, q, sn, None, 128)
    keep = [0, 1, 3]
    within(out[keep], o[keep], (2.0 ** -8 * np.abs(o) + 128 * 2.0 ** -23 * m)[keep], "out")
    assert np.isnan(out[2]).all() and not np.isfinite(out[4]).any()


@pytest.mark.parametrize("symmetric", [True, False])
def test_w4_quantize(ccu, symmetric):
    """Every weight within half a step (and the scale's own rounding) of its 4-bit form."""
    rng = np.random.default_rng(34)
    w = rng.standard_normal((40, 256)) + 0.3
    w[3] = 0
    q, s, z = ccu.w4_quantize(torch.from_numpy(w).to(DEV), 64, symmetric)
    back, _ = ref.w4(np.eye(256), q.cpu().numpy(), num(s), None if z is None else num(z), 64)
    step = np.repeat(num(s), 64, 1)
    # the scale's BF16 rounding moves the ends of the range by at most 15 steps * 2^-8
    assert (np.abs(back.T - w) <= step * (1.0 + 15 * 2.0 ** -8)).all()
    assert np.abs(back.T - w).mean() <= 0.3 * step.mean()


@pytest.mark.parametrize("M,I,O,group,zeros", [(40, 5184, 9800, 64, True), (64, 12416, 9728, 128, False), (16, 8224, 9800, 32, True),
                                               (6, 8224, 1000, 32, True), (30, 4096, 500, 128, False)])
def test_w4_long_inputs(ccu, M, I, O, group, zeros):
    """Many steps of inputs a CTA (its copies' ring goes round), and few outputs with the inputs split."""
    rng = np.random.default_rng(I)
    x, xn = bf(rng, M, I)
    q = rng.integers(0, 256, (O, I // 2), dtype=np.uint8)
    s, sn = bf(rng, O, I // group)
    z, zn = None, None
    if zeros:
        zn = rng.integers(0, 16, (O, I // group)).astype(np.float64)
        z = torch.from_numpy(zn).to(torch.bfloat16).to(DEV)
    a, b = (ccu.w4_matmul(x, torch.from_numpy(q).to(DEV), s, z) for _ in range(2))
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    some = np.unique(np.r_[0, O - 1, rng.integers(0, O, 150)])
    o, m = ref.w4(xn, q[some], sn[some], None if zn is None else zn[some], group)
    within(num(a)[:, some], o, 2.0 ** -8 * np.abs(o) + I * 2.0 ** -23 * m, "out")
    assert ccu.ccu_conv1d_take_device_error() == (0, 0)


def test_w4_tile_keeps_nan_rows_apart(ccu):
    rng = np.random.default_rng(34)
    x, xn = bf(rng, 20, 256)
    x[2], x[13] = float("nan"), float("inf")
    q = rng.integers(0, 256, (140, 128), dtype=np.uint8)
    s, sn = bf(rng, 140, 2)
    z, zn = bf(rng, 140, 2, scale=4.0)
    out = num(ccu.w4_matmul(x, torch.from_numpy(q).to(DEV), s, z))
    o, m = ref.w4(xn, q, sn, zn, 128)
    far = np.abs(xn) @ (np.repeat(np.abs(zn) + 15, 128, 1) * np.repeat(np.abs(sn), 128, 1)).T
    keep = [i for i in range(20) if i not in (2, 13)]
    within(out[keep], o[keep], (2.0 ** -8 * np.abs(o) + 256 * 2.0 ** -23 * far)[keep], "out")
    assert np.isnan(out[2]).all() and not np.isfinite(out[13]).any()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("sizes", [dict(), dict(width=256, heads=12, head=40, states=24, groups=3, lens=(140, 3), group=32),
                                   dict(width=512, heads=4, head=128, states=64, groups=2, lens=(300, 5, 1), tokens=3)], ids=str)
def test_layer_example(ccu, sizes):
    """Prompts continued token by token against whole prompts. The prompt's convolution is rounded to BF16
    before the scan and the token's is not: 2^-9 of x, B and C each, and the outputs' own rounding, through
    sums of both signs."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "ssm_layer.py")
    spec = importlib.util.spec_from_file_location("ssm_layer_example", path)
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    off, off_state = layer.main(**sizes)
    assert off < 8 * 2.0 ** -8 and off_state < 4 * 2.0 ** -8


# ------------------------------------------------------------------ precision of the chunked scan

@pytest.mark.parametrize("shape,lens", [((2, 64, 128, 1), [700]), ((3, 128, 64, 3), [300, 129, 1]), ((1, 40, 24, 1), [257]),
                                        ((1, 64, 128, 1), [2600])], ids=str)
def test_scan_chunked_outputs_err_by_their_own_rounding(ccu, shape, lens):
    """What the outputs are off is their own rounding to BF16: the root mean square of the errors is that of
    the definition's values rounded once. Factors that carry 16 bits (2^-16 of a term where the output's rounding
    takes 2^-9) add less than a hundredth even to outputs a tenth of their terms' size; factors rounded to BF16 add a quarter and more."""
    s = Scan(lens, *shape, seed=46, gate=False, skip=False, initial=[1] * len(lens))
    out = s.run(ccu, route="chunked")
    exact = s.want()[0]
    own = num(torch.from_numpy(exact).to(torch.bfloat16)) - exact
    off = num(out) - exact
    ratio = np.sqrt((off ** 2).mean() / (own ** 2).mean())
    assert ratio < 1.02, ratio


# ------------------------------------------------------------------ infinities in 4-bit products

@pytest.mark.parametrize("M", [3, 20, 40])
@pytest.mark.parametrize("shift", [0, 1], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("I,O,group", [(256, 40, 64), (4224, 130, 128), (8192, 20, 32)])
@pytest.mark.parametrize("whole", [True, False], ids=["whole", "fractions"])
def test_w4_zero_points_and_infinite_inputs(ccu, M, shift, I, O, group, whole):
    """An infinite input makes an output the infinity that (q - zero) x is, NaN only where q is the zero point or infinities
    of both signs meet; the other rows stay as they are. For operands on any boundary."""
    rng = np.random.default_rng(M + I)
    row, rown = bf(rng, M, I + 8)
    x, xn = row[:, shift:shift + I], rown[:, shift:shift + I]
    q = rng.integers(0, 256, (O, I // 2), dtype=np.uint8)
    s, sn = bf(rng, O, I // group)
    zn = rng.integers(0, 16, (O, I // group)) + (0.0 if whole else 0.5)
    z = torch.from_numpy(zn).to(torch.bfloat16).to(DEV)
    for m, i, v in ((0, 5, np.inf), (1, I - 1, -np.inf), (2, 17, np.inf), (2, I - 40, np.inf)):
        x[m, i], xn[m, i] = v, v
    out = num(ccu.w4_matmul(x, torch.from_numpy(q).to(DEV), s, z))
    with np.errstate(invalid="ignore"):
        o = ref.w4(xn, q, sn, zn, group)[0]
    assert np.isinf(o[:3]).any() and np.array_equal(np.isnan(out), np.isnan(o))
    assert np.array_equal(out[:3][~np.isnan(o[:3])], o[:3][~np.isnan(o[:3])])
    far = np.abs(xn[3:]) @ (np.repeat(np.abs(zn) + 15, group, 1) * np.repeat(np.abs(sn), group, 1)).T
    within(out[3:], o[3:], 2.0 ** -8 * np.abs(o[3:]) + I * 2.0 ** -23 * far, "out")


# ------------------------------------------------------------------ the way out of a CTA

def test_scan_chunked_ctas_leave_nothing_behind(ccu):
    """Thousands of one-chunk CTAs, one after the other on every SM: a copy, a product or a barrier's arrival that outlived its CTA
    would fall into the next one's shared memory. The same bits every time, and no wait that ran out."""
    rng = np.random.default_rng(47)
    lens = rng.integers(1, 129, 500).tolist()
    s = Scan(lens, 8, 64, 128, 1, seed=47, gate=False)
    out, state = s.run(ccu, route="chunked").clone(), s.state.clone()
    for _ in range(20):
        assert torch.equal(s.run(ccu, route="chunked").view(torch.int16), out.view(torch.int16))
        assert torch.equal(s.state, state)
    s.check(out, state, LOOSE["chunked"])
    assert ccu.ccu_conv1d_take_device_error() == (0, 0)


# ------------------------------------------------------------------ segments

def scan_args(ccu, T, n_seq, H, P, K, G=1):
    """The struct of a scan of so many tokens, its pointers aligned and never read."""
    a = 0x100000
    return ccu.SelectiveScanArgs(x=a, x_stride_t=H * P, x_stride_h=P, dt=a, dt_stride_t=H, b=a, b_stride_t=G * K, b_stride_g=K, c=a,
                                 c_stride_t=G * K, c_stride_g=K, A=a, cu_seqlens=a, state=a, state_stride_s=H * P * K, out=a,
                                 out_stride_t=H * P, out_stride_h=P, T=T, n_seq=n_seq, H=H, P=P, K=K, G=G, S=n_seq, dt_softplus=1)


@pytest.mark.parametrize("T,n_seq,H,P,K", [(1 << 18, 76, 1, 64, 128), (20000, 30, 2, 64, 128), (4096, 16, 4, 64, 64),
                                           (100000, 1, 8, 128, 128), (1 << 20, 5, 3, 72, 64)])
def test_scan_workspace_grows_with_tokens_and_sequences(ccu, T, n_seq, H, P, K):
    """A segment has 512 tokens or more: the workspace holds one state and one decay a head for every 512 tokens and every
    sequence at most, however the tokens are spread over the sequences."""
    need = ccu.ccu_selective_scan_workspace_bytes(scan_args(ccu, T, n_seq, H, P, K))
    assert 0 < need <= 4 * (T // 512 + n_seq) * (H * P * K + H)


@pytest.mark.parametrize("lens,shape,initial", [
    ([2100, 513], (2, 128, 128, 2), True),          # two blocks of channels, whose decays one of them writes; groups
    ([1, 1500, 0, 512, 1024, 3], (3, 72, 64, 3), True),   # a block of 8 channels; ends on a segment's end
    ([700] * 9, (1, 136, 120, 1), False),           # three blocks
    ([37, 0, 600, 1, 1, 555, 513, 2, 90, 1100, 0, 0, 800, 4], (2, 64, 128, 1), True),
    ([100] * 30 + [2000], (1, 64, 96, 1), True),    # one long prompt behind many short ones
    ([0, 0, 2049], (4, 64, 128, 4), False)], ids=str)
def test_scan_segments_of_all_shapes(ccu, lens, shape, initial):
    H, P, K, G = shape
    s = Scan(lens, H, P, K, G, seed=48, initial=[i % 2 for i in range(len(lens))] if initial else None)
    if len(lens) > 5:
        s.slots[4] = -1
    args = scan_args(ccu, sum(lens), len(lens), H, P, K, G)
    assert ccu.ccu_selective_scan_select_route(args) == ccu.SCAN_ROUTES["chunked"]
    assert ccu.ccu_selective_scan_workspace_bytes(args) > 0  # it is cut
    out = s.run(ccu)
    # the kernel's own error: 2^-16 a factor in two terms, differences of sums of steps 2^-13 (see the scan's rounding)
    s.check(out, s.state, 2.0 ** -12)


def test_scan_segments_of_wild_offsets(ccu):
    """Offsets out of range or out of order reach nothing outside the tensors, cut into segments too; rows before the
    first sequence and behind the last are not written."""
    H, P, K, T = 1, 64, 64, 3000
    s = Scan([T], H, P, K, 1, seed=49, slots=[0], gate=False)
    go, gs = Guarded(T * H * P * 2, DEV), Guarded(8 * H * P * K * 4, DEV)
    out, state = go.view(torch.bfloat16, (T, H, P)), gs.view(torch.float32, (8, H, P, K))

    def run(cu):
        state.zero_()
        ccu.selective_scan(s.x, s.dt, s.A, s.B, s.C, cu_seqlens=i32(cu), ssm_state=state, D=s.D, dt_bias=s.bias, out=out, route="chunked")

    for cu in ([-7, 2_000_000_000, 5, 1200, -3, 2900], [2990, 12, 2999, 2, 1, 0], [0, 3001, 3002, 3003, 3004, 3005]):
        run(cu)
        assert go.guards_intact() and gs.guards_intact()
    out.fill_(7)
    run([1100, 1100, 1700, 2900])
    assert (out[:1100] == 7).all() and (out[2900:] == 7).all()
    rows = slice(1100, 2900)
    o, m, st, sm = ref.scan(s.xn[rows], s.dtn[rows], s.An, s.Bn[rows], s.Cn[rows], s.Dn, None, s.biasn, [0, 600, 1200],
                            np.zeros((8, H, P, K)), [0, 1, 2], None)
    within(num(out[rows]), o, 2.0 ** -8 * np.abs(o) + (1204 * EPS + 2.0 ** -12) * m + 1e-30, "out")
    within(num(state), st, 1204 * EPS * sm + 1e-30, "state")


# ------------------------------------------------------------------ what is not finite

@pytest.mark.parametrize("route", ["chunked", "recurrent"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")], ids=str)
@pytest.mark.parametrize("which,token", [("x", 0), ("x", 150), ("x", 255), ("B", 127), ("C", 130), ("dt", 128), ("dt", 40), ("z", 200),
                                         ("state", 0), ("D", 0)])
def test_scan_is_not_finite_where_the_formula_is_not(ccu, route, bad, which, token):
    """Outputs and states that the formula makes NaN or infinite are not finite, in every route, and all others are what they
    are without that value's neighbours: finite and within the tolerance. Token by token an infinity is the formula's; the chunked
    kernel may give NaN for it."""
    s = Scan([300, 20], 2, 16, 16, 1, seed=50, initial=[1, 1])
    at = dict(x=(token, 1, 5), B=(token, 0, 3), C=(token, 0, 3), dt=(token, 1), z=(token, 1, 5), state=(int(s.slots[0]), 1, 5, 3), D=(1,))[which]
    getattr(s, which)[at] = bad
    getattr(s, which + "n")[at] = bad
    out = s.run(ccu, route=route)
    with np.errstate(invalid="ignore", over="ignore"):
        o, m, st, sm = s.want()
    for got, want, mag, loose, tie in ((num(out), o, m, 2.0 ** -12, 2.0 ** -8), (num(s.state), st, sm, 0.0, 0.0)):
        fine = np.isfinite(want)
        assert np.array_equal(np.isfinite(got), fine)
        within(got[fine], want[fine], tie * np.abs(want[fine]) + (304 * EPS + loose) * mag[fine] + 1e-30, which)
        if route == "recurrent":
            assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])


# ------------------------------------------------------------------ far rows, streams and graphs

@pytest.mark.parametrize("route", ["auto", "chunked", "recurrent"])
def test_scan_far_rows_and_slots_in_every_route(ccu, route):
    """Rows of x, z and out and slots whose offsets pass 2^31 elements, on boundaries that the chunked kernel serves."""
    H, P, K, G = 1, 64, 64, 1
    s = Scan([70, 69], H, P, K, G, seed=51, slots=[2, 0], spare=1, initial=[1, 0])
    rows = ((1 << 31) // 60 + 7) // 8 * 8
    assert 69 * rows > 1 << 31

    def far(t):
        held = torch.empty(138 * rows + P, dtype=torch.bfloat16, device=DEV).as_strided((139, H, P), (rows, P, 1))
        return held if t is None else held.copy_(t)

    s.x, s.z, out = far(s.x), far(s.z), far(None)
    stride = (1 << 30) + 4096
    state = torch.empty(2 * stride + P * K, device=DEV).as_strided((3, H, P, K), (stride, P * K, K, 1))
    state.copy_(s.state)
    args = scan_args(ccu, 139, 2, H, P, K, G)
    args.x_stride_t = args.out_stride_t = args.z_stride_t = rows
    args.state_stride_s, args.route, args.S = stride, ccu.SCAN_ROUTES[route], 3
    assert ccu.ccu_selective_scan_select_route(args) == ccu.SCAN_ROUTES["recurrent" if route == "recurrent" else "chunked"]
    s.run(ccu, state=state, out=out, route=route)
    s.check(out.contiguous(), state.contiguous(), 0.0 if route == "recurrent" else 2.0 ** -12)


def on_another_stream_and_in_a_graph(call, refill):
    """``call()`` on a side stream behind work that its input waits for, and twice in a graph; yields after each. ``call`` returns its
    outputs; ``refill()`` puts them and what the call changes back."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
        refill()
        call()
    side.synchronize()
    yield "stream"
    refill()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        refill()
        graph.replay()
        torch.cuda.synchronize()
        yield "graph"


@pytest.mark.parametrize("M,I,O,group,shift", [(1, 2048, 8512, 128, 0), (5, 8192, 1024, 32, 0), (64, 16384, 512, 128, 0),
                                               (20, 1024, 300, 64, 0), (3, 256, 40, 64, 1)], ids=["few", "split", "cluster", "tile", "scalar"])
def test_w4_on_another_stream_and_in_a_graph(ccu, M, I, O, group, shift):
    rng = np.random.default_rng(52)
    kept, xn = bf(rng, M, I)
    q = rng.integers(0, 256, (O, I // 2), dtype=np.uint8)
    s, sn = bf(rng, O, I // group)
    z = torch.from_numpy(rng.integers(0, 16, (O, I // group)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    qd, out = torch.from_numpy(q).to(DEV), torch.empty(M, O, dtype=torch.bfloat16, device=DEV)
    o, _ = ref.w4(xn, q, sn, num(z), group)
    far = np.abs(xn) @ (np.repeat(np.abs(num(z)) + 15, group, 1) * np.repeat(np.abs(sn), group, 1)).T
    held = torch.zeros(M, I + shift, dtype=torch.bfloat16, device=DEV)[:, shift:]  # shifted: off 16-byte boundaries

    def refill():
        out.zero_()
        held.copy_(kept)

    held.fill_(3)  # what a call that did not wait would read
    for where in on_another_stream_and_in_a_graph(lambda: ccu.w4_matmul(held, qd, s, z, out=out), refill):
        within(num(out), o, 2.0 ** -8 * np.abs(o) + I * 2.0 ** -23 * far, where)


@pytest.mark.parametrize("D", [136, 7])
def test_conv_packed_on_another_stream_and_in_a_graph(ccu, D):
    rng = np.random.default_rng(53)
    lens = [70, 0, 3, 129]
    x, xn = bf(rng, sum(lens), D)
    w, wn = bf(rng, D, 4)
    b, bn = bf(rng, D)
    st, sn = bf(rng, 6, D, 3)
    first, kept, out = st.clone(), x.clone(), torch.empty_like(x)
    cu, slots, has = offsets(lens), i32([5, 1, 0, 2]), i32([1, 0, 1, 0])
    o, m, after = ref.conv(xn, wn, bn, True, lens, sn, [5, 1, 0, 2], [1, 0, 1, 0])

    def refill():
        out.zero_()
        x.copy_(kept)
        st.copy_(first)

    x.fill_(3)
    for where in on_another_stream_and_in_a_graph(
            lambda: ccu.causal_conv1d_packed(x, w, b, "silu", cu_seqlens=cu, conv_state=st, conv_state_indices=slots, has_initial_state=has, out=out),
            refill):
        within(num(out), o, 2.0 ** -8 * np.abs(o) + 8 * 2.0 ** -23 * m, where)
        assert np.array_equal(num(st), after)


# ------------------------------------------------------------------ AUTO, held to the kernel it takes

def route_of(ccu, s):
    """The kernel that AUTO takes for these inputs."""
    H, P, K, G = s.dims
    args = scan_args(ccu, sum(s.lens), len(s.lens), H, P, K, G)
    args.S, args.x, args.b, args.c = s.S, s.x.data_ptr(), s.B.data_ptr(), s.C.data_ptr()
    args.x_stride_t, args.x_stride_h = s.x.stride()[:2]
    args.b_stride_t, args.b_stride_g = s.B.stride()[:2]
    args.c_stride_t, args.c_stride_g = s.C.stride()[:2]
    if s.z is not None:
        args.z, args.z_stride_t, args.z_stride_h = s.z.data_ptr(), *s.z.stride()[:2]
    return {v: k for k, v in ccu.SCAN_ROUTES.items()}[ccu.ccu_selective_scan_select_route(args)]


@pytest.mark.parametrize("lens,shape,wide,shift,route", [
    ([128, 129, 0, 1], (2, 64, 128, 1), False, 0, "chunked"), ([300], (6, 40, 24, 3), False, 0, "chunked"),
    ([130, 1, 40], (4, 40, 24, 2), True, 0, "chunked"), ([130, 1, 40], (4, 40, 24, 2), True, 1, "recurrent"),
    ([130, 1, 40], (2, 64, 128, 1), True, 3, "recurrent"), ([300], (1, 5, 7, 1), False, 0, "recurrent"),
    ([300], (1, 80, 256, 1), False, 0, "recurrent"), ([15, 16, 15], (2, 64, 64, 1), False, 0, "recurrent"),
    ([16, 16, 16], (2, 64, 64, 1), False, 0, "chunked")], ids=str)
def test_scan_auto_takes_the_kernel_and_its_precision(ccu, lens, shape, wide, shift, route):
    """Token by token nothing but 32-bit errors is allowed, in chunks 2^-12 of the terms (factors of 16 bits and sums of
    steps over 32 tokens)."""
    s = Scan(lens, *shape, seed=54, wide=wide, shift=shift, initial=[i % 2 for i in range(len(lens))])
    assert route_of(ccu, s) == route
    s.check(s.run(ccu), s.state, 2.0 ** -12 if route == "chunked" else 0.0, route)
