"""Rotary positions on the GPU against the 64-bit rotation.

Tolerance: one rounding to fp16 (2^-11 of the result, 2^-25 below the normals), and
before it in fp32 the magnitude's rounding, the conversion of the angle (2^-24 of at
most pi), sincospif (2^-22) and three products and sums: 2^-20 g (|x_a| + |x_b|)."""
import numpy as np
import pytest
import torch

from mixed_precision_quantized_gb300 import build, ekv
from oracle import serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ekv.lib()


def _check(x, y, pos, rope, d, layout, kw):
    f, mag = serving.rope_freqs(kw["rot_dim"], kw.get("base", 10000.0), kw.get("scaling", "none"),
                                kw.get("factor", 1.0), kw.get("original_len", 0.0))
    xn = x.cpu().numpy().astype(np.float64)
    want = serving.rope(xn, pos.cpu().numpy(), f, mag, layout)
    r = kw["rot_dim"]
    size = np.abs(serving.rope(np.abs(xn), np.zeros(len(pos)), f, 1.0, layout))
    ia = np.arange(r // 2) if layout == "half" else np.arange(0, r, 2)
    ib = ia + (r // 2 if layout == "half" else 1)
    both = size[..., ia] + size[..., ib]
    size[..., ia] = size[..., ib] = both
    got = y.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -25 +
                  2.0 ** -20 * mag * size)
    assert np.array_equal(got[..., r:], xn[..., r:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,kw", [
    (128, dict(rot_dim=128)), (64, dict(rot_dim=64, base=500000.0)), (128, dict(rot_dim=32)),
    (128, dict(rot_dim=2)), (64, dict(rot_dim=20)), (128, dict(rot_dim=126)), (128, dict(rot_dim=24)),
    (128, dict(rot_dim=128, scaling="linear", factor=8.0)),
    (128, dict(rot_dim=128, base=500000.0, scaling="banded", factor=8.0, original_len=8192)),
    (64, dict(rot_dim=32, scaling="yarn", factor=32.0, original_len=4096))])
def test_rotation(d, kw, layout):
    g = torch.Generator(device="cuda").manual_seed(1)
    n = 37
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda").int()
    pos[:6] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131071])
    q = torch.randn(n, 6, d, generator=g, device="cuda").half()
    k = torch.randn(n, 2, d, generator=g, device="cuda").half()
    rope = ekv.Rope(d, layout=layout, **kw)
    qo, ko = rope(q, k, pos)
    _check(q, qo, pos, rope, d, layout, kw)
    _check(k, ko, pos, rope, d, layout, kw)


@pytest.mark.parametrize("n", [0, 1, 3, 2047, 2048, 2051])
def test_token_counts_views_and_places(n):
    """Odd counts around the switch of tokens per CTA; q and k as views of a fused
    projection, in place: the third part is left as it was."""
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, 12, 64, generator=g, device="cuda").half()
    pos = torch.arange(n, device="cuda", dtype=torch.int32) + 70000
    rope = ekv.Rope(64)
    old = x.clone()
    q, k = x[:, :8], x[:, 8:10]
    qo, ko = rope(q, k, pos)
    qi, ki = rope(q, k, pos, q_out=q, k_out=k)
    assert qi.data_ptr() == x.data_ptr() or n == 0
    assert torch.equal(qo, q) and torch.equal(ko, k) and torch.equal(x[:, 10:], old[:, 10:])
    if n:
        _check(old[:, :8], qo, pos, rope, 64, "half", dict(rot_dim=64))


def test_one_tensor_alone_and_wide_heads():
    x = torch.randn(5, 300, 128, device="cuda").half()
    pos = torch.tensor([3, 3, 9, 0, 100000], dtype=torch.int32, device="cuda")
    rope = ekv.Rope(128)
    qo, none = rope(x, None, pos)
    none2, ko = rope(None, x, pos)
    assert none is None and none2 is None and torch.equal(qo, ko)
    _check(x, qo, pos, rope, 128, "half", dict(rot_dim=128))


def test_subnormals_infinities_and_captured_graph_on_another_stream():
    """Values outside the rotated part pass bit for bit (infinities and NaN too); a
    captured call replays on new contents."""
    x = torch.randn(4, 2, 64, device="cuda").half()
    x[0, 0, 40:44] = torch.tensor([float("inf"), float("nan"), 6e-8, -0.0])
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    rope = ekv.Rope(64, rot_dim=32)
    out, _ = rope(x, None, pos)
    assert torch.equal(out[..., 32:].view(torch.int16), x[..., 32:].view(torch.int16))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    buf = torch.empty_like(x)
    with torch.cuda.stream(s):
        rope(x, None, pos, q_out=buf)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope(x, None, pos, q_out=buf)
    x[:, :, :32] = torch.randn(4, 2, 32, device="cuda").half()
    pos += 1000
    g.replay()
    torch.cuda.synchronize()
    want, _ = rope(x, None, pos)
    assert torch.equal(buf[..., :32], want[..., :32])


def test_refusals():
    rope = ekv.Rope(64)
    x = torch.zeros(4, 2, 64, device="cuda").half()
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: rope(x.float(), None, pos), lambda: rope(x, None, pos.long()),
                lambda: rope(x[:3], None, pos), lambda: rope(x[..., :32], None, pos),
                lambda: rope(x.transpose(0, 1), None, pos[:2]),
                lambda: rope(x, None, pos, q_out=torch.zeros(4, 3, 64, device="cuda").half()),
                lambda: rope(x, None, pos, k_out=x)):
        with pytest.raises((TypeError, ValueError)):
            bad()
