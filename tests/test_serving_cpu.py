"""Serving operators without a GPU: the rotary frequency table against the formulas,
the refusals of every entry point (bad arguments return before anything is
launched), and the oracle's own definitions against hand-worked cases."""
import ctypes
import math
import os
import shutil
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

from oracle import serving

EINVAL, EUNSUPPORTED = 1, 5


@pytest.fixture(scope="module")
def ekv():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("no CUDA toolkit on this host")
    from mixed_precision_quantized_gb300 import build
    from mixed_precision_quantized_gb300 import ekv as mod
    build.build()
    mod.lib()
    return mod


CONFIGS = [dict(rot_dim=128), dict(rot_dim=64), dict(rot_dim=20, base=500000.0), dict(rot_dim=2),
           dict(rot_dim=128, scaling="linear", factor=8.0),
           dict(rot_dim=128, base=500000.0, scaling="banded", factor=8.0, original_len=8192),
           dict(rot_dim=96, scaling="banded", factor=2.0, original_len=1000,
                low_freq_factor=2.0, high_freq_factor=16.0),
           dict(rot_dim=64, scaling="yarn", factor=32.0, original_len=4096),
           dict(rot_dim=128, scaling="yarn", factor=4.0, original_len=32768, beta_fast=16.0,
                beta_slow=2.0)]


@pytest.mark.parametrize("kw", CONFIGS, ids=lambda c: f"{c.get('scaling', 'none')}{c['rot_dim']}")
def test_rope_table_matches_the_formulas(ekv, kw):
    """Turns per position as 64-bit fractions: the table and the formula are both
    fp64, a few roundings of 2^-53 apart relative to f."""
    r = ekv.Rope(128, device="cpu", **kw)
    f, mag = serving.rope_freqs(
        kw["rot_dim"], kw.get("base", 10000.0), kw.get("scaling", "none"), kw.get("factor", 1.0),
        kw.get("original_len", 0.0), kw.get("low_freq_factor", 1.0),
        kw.get("high_freq_factor", 4.0), kw.get("beta_fast", 32.0), kw.get("beta_slow", 1.0))
    assert len(r.turns) == kw["rot_dim"] // 2
    assert abs(r.magnitude - mag) <= 2 ** -23 * mag
    for t, want in zip(r.turns, f / (2 * math.pi)):
        assert abs(t * 2.0 ** -64 - want) <= 64 * 2.0 ** -53 * want + 2.0 ** -63


@pytest.mark.parametrize("base", [1.5, 10000.0, 500000.0, 7e8])
@pytest.mark.parametrize("rot", [2, 20, 126, 128])
def test_rope_table_in_50_digits(ekv, base, rot):
    """Against decimal arithmetic: within 2^-53 turns a position.  -2i/r is rounded (2^-53),
    which moves f by f |ln f| 2^-53 <= 2^-53 / e; pow adds 2^-52 f at most, the division by
    2 pi and 2 pi itself 2^-53 f each: (1 / e + 4) 2^-53 / 2 pi < 2^-53.4; what is cut below
    2^-64 is nothing beside it."""
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582")
    with localcontext() as c:
        c.prec = 50
        for i, t in enumerate(ekv.Rope(128, rot_dim=rot, base=base, device="cpu").turns):
            want = (Decimal(base).ln() * Decimal(-2 * i) / Decimal(rot)).exp() / (2 * pi)
            assert abs(Decimal(t) / 2 ** 64 - want) <= Decimal(2) ** -53


def test_rope_magnitude_can_be_set(ekv):
    assert ekv.Rope(64, device="cpu", magnitude=0.5).magnitude == 0.5
    assert ekv.Rope(64, device="cpu", scaling="yarn", factor=0.5, original_len=64).magnitude == 1.0


@pytest.mark.parametrize("kw", [
    dict(head_dim=96), dict(head_dim=128, rot_dim=130), dict(head_dim=128, rot_dim=0),
    dict(head_dim=128, rot_dim=7), dict(head_dim=128, base=1.0), dict(head_dim=128, base=math.nan),
    dict(head_dim=128, base=math.inf), dict(head_dim=128, magnitude=-1.0),
    dict(head_dim=128, scaling="linear", factor=0.0),
    dict(head_dim=128, scaling="linear", factor=math.nan),
    dict(head_dim=128, scaling="banded", factor=2.0),
    dict(head_dim=128, scaling="banded", factor=2.0, original_len=10, low_freq_factor=4.0),
    dict(head_dim=128, scaling="yarn", factor=2.0, original_len=10, beta_fast=1.0, beta_slow=1.0),
    dict(head_dim=128, scaling="yarn", factor=2.0, original_len=10, beta_slow=0.0)])
def test_rope_refuses_bad_configurations(ekv, kw):
    with pytest.raises(ekv.EkvError) as e:
        ekv.Rope(device="cpu", **kw)
    assert e.value.code == EINVAL


@pytest.mark.parametrize("kw", [
    dict(magnitude=1e39), dict(scaling="linear", factor=1e-310),
    dict(scaling="banded", factor=5e-324, original_len=8192),
    dict(scaling="yarn", factor=1e-309, original_len=8192)])
def test_rope_refuses_what_no_float_holds(ekv, kw):
    """A magnitude past fp32; a factor whose inverse is infinite (no frequency table)."""
    with pytest.raises(ekv.EkvError) as e:
        ekv.Rope(128, device="cpu", **kw)
    assert e.value.code == EINVAL
    r = ekv.Rope(128, device="cpu", scaling="linear", factor=1e-300)
    assert all(0 <= t < 1 << 64 for t in r.turns)


def test_rope_refuses_unknown_names(ekv):
    with pytest.raises(ValueError):
        ekv.Rope(128, layout="rows", device="cpu")
    with pytest.raises(ValueError):
        ekv.Rope(128, scaling="cubic", device="cpu")


P16, P4, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 4), ctypes.c_void_p((1 << 20) + 2)


def _rope_args(ekv, **kw):
    c = ekv.Rope(128, device="cpu").cfg
    a = dict(cfg=ctypes.byref(c), turns=P16, n=4, pos=P16, hq=4, q=P16, qs=512, qo=P16, qos=512,
             hk=2, k=P16, ks=256, ko=P16, kos=256, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(cfg=None), dict(turns=None), dict(pos=None), dict(n=-1), dict(hq=-1), dict(q=None),
    dict(qo=None), dict(q=P4), dict(k=P4), dict(qs=504), dict(qs=516), dict(ks=248), dict(kos=0),
    dict(qs=520), dict(pos=ODD), dict(turns=P4), dict(n=1 << 31)])
def test_rope_refuses(ekv, kw):
    """`qs=520` is an in-place call with two strides."""
    assert ekv.lib().ekv_rope(*_rope_args(ekv, **kw)) == EINVAL


def test_rope_of_nothing_is_ok(ekv):
    assert ekv.lib().ekv_rope(*_rope_args(ekv, n=0)) == 0
    assert ekv.lib().ekv_rope(*_rope_args(ekv, hq=0, hk=0)) == 0


def _prompt_args(**kw):
    a = dict(hq=4, hk=2, d=128, scale=0.0, total=4, n=1, cu=P16, q=P16, qs=512, k=P16, ks=256,
             v=P16, vs=256, o=P16, os=512, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(hq=0), dict(hk=0), dict(hq=5), dict(hk=-2), dict(scale=-1.0), dict(scale=math.nan),
    dict(scale=math.inf), dict(total=-1), dict(n=-1), dict(cu=None), dict(q=None), dict(k=None),
    dict(v=None), dict(o=None), dict(q=P4), dict(k=P4), dict(v=P4), dict(o=P4), dict(qs=511),
    dict(qs=504), dict(ks=252), dict(vs=128), dict(os=0), dict(cu=ODD)])
def test_prompt_refuses(ekv, kw):
    assert ekv.lib().ekv_prompt_attn(*_prompt_args(**kw)) == EINVAL


def test_prompt_refuses_scales_whose_product_with_log2e_overflows(ekv):
    for scale in (2.4e38, 3.0e38):
        assert ekv.lib().ekv_prompt_attn(*_prompt_args(scale=scale)) == EINVAL


def test_prompt_head_dim_and_nothing(ekv):
    assert ekv.lib().ekv_prompt_attn(*_prompt_args(d=96)) == EUNSUPPORTED
    assert ekv.lib().ekv_prompt_attn(*_prompt_args(total=0)) == 0
    assert ekv.lib().ekv_prompt_attn(*_prompt_args(n=0)) == 0


def _verify_args(**kw):
    a = dict(n=2, m=4, V=32, p=P16, ps=128, pr=32, q=None, qs=0, qr=0, tok=P16, par=P16, cnt=None,
             u=P16, us=P16, path=P16, acc=P16, nxt=P16, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(m=0), dict(m=65), dict(V=0), dict(p=None), dict(tok=None), dict(par=None),
    dict(u=None), dict(us=None), dict(path=None), dict(acc=None), dict(nxt=None), dict(p=ODD),
    dict(q=ODD), dict(pr=31), dict(q=P16, qr=31, qs=128), dict(ps=-1), dict(tok=ODD)])
def test_verify_refuses(ekv, kw):
    assert ekv.lib().ekv_verify_tree(*_verify_args(**kw)) == EINVAL


@pytest.mark.parametrize("V", [(1 << 30) + 1, (1 << 31) - 1])
def test_verify_refuses_rows_past_its_index_arithmetic(ekv, V):
    assert ekv.lib().ekv_verify_tree(*_verify_args(V=V, ps=4 * V, pr=V)) == EINVAL


def test_verify_of_nothing_is_ok(ekv):
    assert ekv.lib().ekv_verify_tree(*_verify_args(n=0)) == 0


def test_tree_refuses_without_a_handle(ekv):
    out = ctypes.c_int64()
    assert ekv.lib().ekv_tree_attn_scratch_bytes(None, 1, 4, ctypes.byref(out)) == EINVAL
    assert ekv.lib().ekv_tree_attn(None, 0, 1, P16, 4, None, P16, P16, P16, P16, P16, P16, 0,
                                   None) == EINVAL


def test_binding_refuses_cpu_tensors_types_and_shapes(ekv):
    h = torch.zeros(4, 2, 64, dtype=torch.float16)
    cu = torch.zeros(2, dtype=torch.int32)
    for bad in (lambda: ekv.prompt_attn(h, h, h, cu),                       # not on a GPU
                lambda: ekv.prompt_attn(h[0], h, h, cu),
                lambda: ekv.Rope(64, device="cpu")(h, None, torch.zeros(4, dtype=torch.int32)),
                lambda: ekv.verify_tree(torch.zeros(1, 2, 8), *[torch.zeros(1, 2)] * 3,
                                        torch.zeros(1))):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(TypeError):
        ekv.prompt_attn(h.float(), h, h, cu)


def test_binding_refuses_a_stream_of_another_gpu(ekv):
    """The call runs where its tensors are; a stream elsewhere is not replaced by one there."""
    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    with pytest.raises(ValueError, match="stream"):
        ekv._on(0, Stream())


def test_oracle_attention_and_tree():
    """Two keys of equal logits average; a chain's node sees its prefix, a tree's only
    its ancestors; a row that sees nothing is zero."""
    q = np.zeros((3, 1, 2))
    k, v = np.zeros((3, 1, 2)), np.array([[[1.0, 0]], [[3.0, 0]], [[8.0, 1]]])
    o, _ = serving.attention(q, k, v, serving.causal(3))
    assert np.allclose(o[:, 0], [[1, 0], [2, 0], [4, 1 / 3]])
    see = serving.tree_sees([-1, 0, 0, 1], 4, 2)
    assert see[:, :2].all() and see[:, 2:].astype(int).tolist() == [
        [1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 1, 0, 1]]
    o, b = serving.attention(q, k, v, np.zeros((3, 3), dtype=bool))
    assert not o.any() and np.all(b <= 2.0 ** -24)


@pytest.mark.parametrize("draft", [False, True])
def test_oracle_walk_follows_the_target(draft):
    """Over many draws the first emitted token of a one-level tree is distributed as
    the target, whatever was drafted.  40,000 draws: a frequency is within 5 standard
    deviations sqrt(p(1-p)/n) of p (8 frequencies, probability of a miss < 5e-6)."""
    rng = np.random.default_rng(3)
    V, n = 8, 40000
    p = rng.dirichlet(np.ones(V))[None].repeat(3, 0)
    q = rng.dirichlet(np.ones(V))[None].repeat(3, 0)
    seen = np.zeros(V)
    for _ in range(n):
        x = [0, *rng.choice(V, 2, p=q[0])] if draft else [0, 2, 5]
        path, nxt = serving.verify(p, q if draft else None, x, [-1, 0, 0], rng.random(3),
                                   rng.random(), 3)
        seen[x[path[0]] if path else nxt] += 1
    assert np.all(np.abs(seen / n - p[0]) <= 5 * np.sqrt(p[0] * (1 - p[0]) / n))
