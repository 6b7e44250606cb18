"""The gated delta rule on the GPU where calls could go wrong without changing a result much: what its launches hand to each other,
and the ends of the range of its arguments."""

import numpy as np
import pytest
import torch

from gpu_util import Guarded
from test_delta_gpu import DEV, HALF, ROUTES, Rule, ccu, i32, num, offsets  # noqa: F401

pytestmark = pytest.mark.gpu


def fma(a, b, c):
    """a b + c with one rounding to 32 bits: the product is exact in 64."""
    return (a.double() * b.double() + c.double()).float()


def one_sequence(ccu, r, lo, hi, state, initial):  # noqa: F811
    """The state after tokens lo..hi - 1 of a rule of one sequence, from ``state`` [H, P, K] or from none; too short to be cut."""
    held = state.clone()[None]
    cut = slice(lo, hi)
    ccu.gated_delta_rule(r.q[cut], r.k[cut], r.v[cut], r.a[cut], r.b[cut], r.A, cu_seqlens=offsets([hi - lo]), state=held, dt_bias=r.bias,
                         has_initial_state=i32([1 if initial else 0]), route="chunked")
    return held[0]


def test_rule_joined_states_are_left_alone(ccu):  # noqa: F811
    """The states between segments are made by the join and only read after it: a CTA may read one at any time of the last launch, so
    nobody writes there again, not even the same state computed another way."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("segments of other lengths")
    H, P, K, tokens, T = 2, 64, 64, 8 * 64, 4 * 8 * 64 + 100
    r = Rule([T], H, P, K, 1, seed=70, initial=[1], slots=[0], spare=0, decay=(0.01, 1.0))
    first = r.state[0].clone()
    count = T // tokens + 1  # the least length of a segment, as there are few items
    size = 4 * count * H * K * (P + K)
    with pytest.raises(ValueError, match=f"of {size} bytes"):
        r.run(ccu, route="chunked", workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    work = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    r.check(r.run(ccu, route="chunked", workspace=work), r.state)
    states = work[:4 * count * H * P * K].view(torch.float32).view(count, H, P, K)
    maps = work[4 * count * H * P * K:].view(torch.float32).view(count, H, K, K)
    want = one_sequence(ccu, r, 0, tokens, first, True)
    assert torch.equal(states[1], want)
    for j in range(1, count - 1):
        joined = one_sequence(ccu, r, j * tokens, (j + 1) * tokens, torch.zeros_like(first), False)
        for i in range(K):
            joined = fma(want[..., i:i + 1], maps[j, :, i:i + 1, :], joined)
        assert torch.equal(states[j + 1], joined), j
        want = joined


def test_rule_of_segments_gives_the_same_bits_again(ccu):  # noqa: F811
    """A long sequence beside short ones, whose last launch has more CTAs than the card holds at a time."""
    r = Rule([4400, 100, 108], 10, 256, 16, 1, seed=71, initial=[1, 0, 1], decay=(0.01, 1.0))
    first = r.state.clone()
    out = r.run(ccu, route="chunked")
    r.check(out, r.state)
    for _ in range(20):
        state = first.clone()
        assert torch.equal(out, r.run(ccu, route="chunked", state=state)) and torch.equal(state, r.state)


@pytest.mark.parametrize("heads,blocks", [(27, 1), (28, 1), (27, 2), (160, 1)], ids=str)
def test_rule_in_even_shares_gives_the_same_bits_again(ccu, heads, blocks):  # noqa: F811
    """Even shares, whose CTAs take their pieces by a ticket, in pairs (an even number of items a sequence) and one by one: the order in which
    CTAs start changes nothing, alone and beside a kernel of another stream that holds SMs."""
    lens = [4000] if heads == 160 else [700, 300, 2000, 0, 64, 513]
    r = Rule(lens, heads, 128 * blocks, 16, 1, seed=73, initial=[i % 2 for i in range(len(lens))], decay=(0.01, 1.0))
    with pytest.raises(ValueError, match="workspace"):
        r.run(ccu, route="chunked", workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    first = r.state.clone()
    out = r.run(ccu, route="chunked")
    side, busy = torch.cuda.Stream(), torch.randn(8192, 8192, device=DEV)
    torch.cuda.synchronize()
    for i in range(20):
        if i >= 10:
            with torch.cuda.stream(side):
                busy.mul_(-1)
        state = first.clone()
        assert torch.equal(out, r.run(ccu, route="chunked", state=state)) and torch.equal(state, r.state)
    torch.cuda.synchronize()


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("size", [1.0, 256.0, 16384.0])
@pytest.mark.parametrize("tokens", [64, 200])
def test_rule_outputs_of_a_large_state(ccu, route, size, tokens):  # noqa: F811
    """One key and query throughout, written at full strength: the first token replaces what the state, much larger than the values, holds
    along the key, and every output is the small difference of two large sums. Both are sums of 32 bits, so their errors are too.

    Chunked, what cancels is of size m = |s k| (``size`` for a channel, in the mean square). It passes 24 sums of products on its way into r, 36 into u, 24 into s q and
    24 into the output, 108 in all, and some 20 more roundings in decays, lengths and factors. Each is off by less than a step, 2^-23 of m, evenly
    spread: 0.58 of that in the mean square, sqrt(128) = 11.3 times as much for independent ones, 13 units of 2^-24 m. The bound is 16, and a rounding to BF16 beside it."""
    r = Rule([tokens], 1, 64, 128, 1, seed=74, initial=[1], decay=(1e-5, 1e-4))
    r.k[:] = r.k[:1].clone()
    r.q[:] = r.k
    r.b[:] = 30.0
    r.state *= 10 * size
    r.qn, r.kn, r.bn, r.staten = num(r.q), num(r.k), num(r.b), num(r.state)
    out = r.run(ccu, route=route, scale=1.0)
    want = r.want(scale=1.0)[0]
    rms = lambda v: np.sqrt((v * v).mean())  # noqa: E731
    m = rms(r.staten[r.slots[0], 0] @ (r.kn[0, 0] / np.linalg.norm(r.kn[0, 0])))
    assert rms(num(out) - want) <= 16 * 2.0 ** -24 * m + HALF / 2 * rms(want)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("scale,size", [(3e38, 0.01), (-3e38, 1e-4), (1e-38, 1e15), (1e-42, 1.0)])
def test_rule_of_scales_at_the_ends_of_the_type(ccu, route, scale, size):  # noqa: F811
    """Scales near the largest and the smallest float beside short and long queries: outputs that the type holds are finite and right.
    A half step of BF16 below 2^-126 is 2^-134, and the products before it may lose another."""
    r = Rule([150], 2, 64, 64, 2, seed=75, initial=[1])
    r.q *= size
    r.qn = num(r.q)
    r.v *= 0.1
    r.vn = num(r.v)
    o, off, *_ = r.want(scale=scale)
    out = num(r.run(ccu, route=route, scale=scale))
    assert np.abs(o).max() < 3e38
    bad = ~(np.abs(out - o) <= HALF * np.abs(o) + off + 2.0 ** -133)
    assert not bad.any(), (bad.sum(), out[bad][0], o[bad][0])


@pytest.mark.parametrize("channel_last", [True, False])
def test_update_convolution_in_32_bits(ccu, channel_last):  # noqa: F811
    """What the convolution step's SiLU gives becomes the state, and is as exact as the state. One tap of 1 makes its sum the input, an empty
    state and a key of (30, 0, ...) make the state 30 silu(v): the exponential 2 steps of 2^-23, its product, the sum, the quotient and the product with 30
    half a step each: 8 units of 2^-24."""
    N, H, P, K = 6, 4, 256, 8
    rng = np.random.default_rng(76)
    channels = 2 * K + H * P
    qkv = torch.from_numpy(rng.uniform(-11, 11, (N, channels)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    qkv[0, 2 * K:2 * K + 8] = torch.tensor([-30.0, -60, -80, -87, 40, 88, 100, 0], device=DEV)
    qkv[:, K] = 30.0
    qkv[:, K + 1:2 * K] = 0
    weight = torch.zeros(channels, 4, dtype=torch.bfloat16, device=DEV)
    weight[:, 3] = 1
    conv = torch.zeros(N, 3, channels, dtype=torch.bfloat16, device=DEV).permute(0, 2, 1)
    state = torch.zeros(N, H, P, K, device=DEV)
    ccu.gated_delta_update(qkv, torch.zeros(N, H, dtype=torch.bfloat16, device=DEV), torch.full((N, H), 40.0, dtype=torch.bfloat16, device=DEV),
                           -torch.ones(H, device=DEV), state, conv if channel_last else conv.contiguous(), weight, None, "silu", qk_norm=False)
    v = num(qkv)[:, 2 * K:].reshape(N, H, P)
    want = 30 * np.where(v < 0, v * np.exp(-np.abs(v)), v) / (1 + np.exp(-np.abs(v)))
    off = np.abs(num(state)[..., 0] - want)
    bad = ~(off <= 8.01 * 2.0 ** -24 * np.abs(want) + 2.0 ** -145)
    assert not bad.any(), (bad.sum(), (off / np.maximum(np.abs(want), 1e-300)).max() * 2.0 ** 24)
    assert not state[..., 1:].any()


@pytest.mark.parametrize("cu", [[0, 9000, 4000, 13300], [-5, 20000, 10000, 100000], [13300, 0, 13300, 0], [13300, 13300, 0, 13300]], ids=str)
@pytest.mark.parametrize("heads", [2, 60])
def test_rule_offsets_out_of_order_in_parts(ccu, cu, heads):  # noqa: F811
    """Offsets that do not ascend, or leave the rows, in calls that are cut into segments and in ones that are shared out evenly: no
    memory outside the tensors is reached."""
    T, P, K = 13300, 8, 16
    r = Rule([6000, 4000, 3300], heads, P, K, 1, seed=72, initial=[1, 0, 1], slots=[0, 2, 3], spare=2)
    go, gs = Guarded(T * heads * P * 2, DEV), Guarded(r.S * heads * P * K * 4, DEV)
    out, state = go.view(torch.bfloat16, (T, heads, P)), gs.view(torch.float32, (r.S, heads, P, K))
    state.copy_(r.state)
    with pytest.raises(ValueError, match="workspace"):  # it is cut
        r.run(ccu, route="chunked", workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    gw = Guarded(1 << 24, DEV)
    ccu.gated_delta_rule(r.q, r.k, r.v, r.a, r.b, r.A, cu_seqlens=i32(cu), state=state, state_indices=i32(r.slots), has_initial_state=i32(r.has),
                         out=out, route="chunked", workspace=gw.view(torch.uint8, (1 << 24,)))
    torch.cuda.synchronize()
    assert go.guards_intact() and gs.guards_intact() and gw.guards_intact() and torch.equal(state[[1, 4]], r.state[[1, 4]])


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("first", [True, False])
def test_rule_of_a_long_prompt_among_single_tokens(ccu, route, first):  # noqa: F811
    """A continuous batch: one prompt beside many sequences of one token, which continue from their states."""
    lens = [1] * 120
    lens[0 if first else 77] = 1500
    r = Rule(lens, 2, 64, 64, 1, seed=77, initial=[0 if n > 1 else 1 for n in lens])
    r.check(r.run(ccu, route=route), r.state)
