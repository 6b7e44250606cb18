"""Numbers that the calls of the delta rule and of the norms pass on in 32 bits, without a GPU: those that 32 bits do not hold."""

import pytest


@pytest.fixture(scope="module")
def ccu():
    import __graft_entry__ as g

    g.build()
    import depthwise_causal_conv1d_gb300 as ccu

    return ccu


@pytest.mark.parametrize("scale", [1e-46, -1e-46, 5e-324, 3.5e38, -1e39, 1e300])
def test_scale_of_the_rule_that_32_bits_do_not_hold(ccu, scale):
    """A scale of 0 is the C struct's default, 1 / sqrt(K): one that rounds to it is refused, as 0 itself is, and so is one that overflows."""
    from depthwise_causal_conv1d_gb300 import delta

    with pytest.raises(ValueError, match="scale must be finite and not 0"):
        delta._scale(scale, 64)


@pytest.mark.parametrize("scale", [1.4e-45, -1.2e-38, 3.4e38, 0.1])
def test_scale_of_the_rule_at_the_ends_of_32_bits(ccu, scale):
    import struct

    from depthwise_causal_conv1d_gb300 import delta

    packed = struct.unpack("f", struct.pack("f", delta._scale(scale, 64)))[0]
    assert packed != 0 and abs(packed - scale) <= max(2.0 ** -24 * abs(scale), 2.0 ** -150)


def test_scale_of_the_norms_that_32_bits_do_not_hold(ccu, monkeypatch):
    """What overflows is declined as an infinity is: a ValueError that names it. A scale that rounds to 0 adds nothing, which is its product."""
    import torch

    from depthwise_causal_conv1d_gb300 import delta

    # CPU tensors in the place of the GPU's: every call here is declined, or has nothing to do
    monkeypatch.setattr(delta, "_check", lambda dev, name, t, dtype, shape, contiguous=False: t.data_ptr())
    for entry in (delta._GATED, delta._RESIDUAL):
        monkeypatch.setattr(entry, "launch", lambda dev, packed, entry=entry: ccu.raise_for_status(st) if (st := entry.call(packed, None)) else None)
    x, v = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 2, 8, dtype=torch.bfloat16)
    for big in (1e39, float("inf"), float("nan")):
        with pytest.raises(ValueError, match="scale"):
            ccu.residual_rms_norm(x, x.clone(), scale=big)
        with pytest.raises(ValueError, match="eps"):
            ccu.residual_rms_norm(x, x.clone(), eps=big)
        with pytest.raises(ValueError, match="eps"):
            ccu.gated_rms_norm(v, eps=big)
    assert ccu.residual_rms_norm(x[:0], x[:0], scale=1e-60, eps=1e-60).shape == (0, 8)
