"""Attention over packed prompts on the GPU against the 64-bit definition, within the
bound that the oracle derives (one fp16 rounding of each probability and of the
output, fp32 otherwise)."""
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


def _inputs(T, hq, hkv, d, seed=0, qs=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((qs * torch.randn(T, hq, d, generator=g, device="cuda")).half(),
            torch.randn(T, hkv, d, generator=g, device="cuda").half(),
            torch.randn(T, hkv, d, generator=g, device="cuda").half())


def _check(q, k, v, o, bounds, scale=None, rows=None):
    """Compare sequence by sequence; `rows`: at most that many query rows of each, the
    first and last among them."""
    qn, kn, vn, on = (x.cpu().numpy() for x in (q, k, v, o))
    for a, b in zip(bounds, bounds[1:]):
        if a == b:
            continue
        n = b - a
        pick = np.arange(n)
        if rows and n > rows:
            pick = np.unique(np.concatenate([[0, n - 1], np.linspace(0, n - 1, rows).astype(int)]))
        see = np.arange(n)[None] <= pick[:, None]
        want, tol = serving.attention(qn[a:b][pick], kn[a:b], vn[a:b], see, scale)
        err = np.abs(on[a:b][pick].astype(np.float64) - want)
        assert np.all(err <= tol), f"sequence {a}:{b}: {np.max(err / tol):.2f} of the bound"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (5, 1), (3, 3), (16, 2)])
@pytest.mark.parametrize("lens", [[1], [2], [17], [127], [128], [129], [255, 1, 256, 257],
                                  [0, 3, 0, 64, 1, 0], [300, 129, 5]],
                         ids=lambda v: "-".join(map(str, v)))
def test_lengths_and_groups(d, hq, hkv, lens):
    T = sum(lens)
    q, k, v = _inputs(T, hq, hkv, d, seed=T)
    cu = [0, *np.cumsum(lens).tolist()]
    o = ekv.prompt_attn(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    _check(q, k, v, o, cu)


@pytest.mark.parametrize("lens,hq,hkv,d", [([4100], 4, 1, 128), ([2048, 1, 1500], 10, 2, 64),
                                           ([6001], 8, 8, 128)])
def test_long_prompts(lens, hq, hkv, d):
    T = sum(lens)
    q, k, v = _inputs(T, hq, hkv, d, seed=3)
    cu = [0, *np.cumsum(lens).tolist()]
    o = ekv.prompt_attn(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    _check(q, k, v, o, cu, rows=24)


def test_many_sequences():
    """400 sequences of 0 to 40 tokens."""
    lens = np.random.default_rng(0).integers(0, 41, 400).tolist()
    q, k, v = _inputs(sum(lens), 4, 2, 64)
    cu = [0, *np.cumsum(lens).tolist()]
    o = ekv.prompt_attn(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    _check(q, k, v, o, cu)


def test_more_sequences_than_one_launch_takes():
    """1,100 sequences of 0 to 5 tokens (a launch takes 512)."""
    lens = np.random.default_rng(1).integers(0, 6, 1100).tolist()
    q, k, v = _inputs(sum(lens), 2, 1, 64)
    cu = [0, *np.cumsum(lens).tolist()]
    o = ekv.prompt_attn(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    _check(q, k, v, o, cu)


def test_offsets_past_32_bits():
    """Token strides of 2^20 elements over 4,200 tokens: the last rows lie 4.4e9 elements
    behind the first."""
    T, step = 4200, 1 << 20
    bufs = [torch.empty(T, step, dtype=torch.float16, device="cuda") for _ in range(2)]
    q, k, v = _inputs(T, 2, 1, 64, seed=2)
    bufs[0][:, :128] = q.view(T, 128)
    bufs[0][:, 128:192] = k.view(T, 64)
    bufs[0][:, 256:320] = v.view(T, 64)
    view = lambda b, c, h: b[:, c:c + 64 * h].unflatten(1, (h, 64))  # noqa: E731
    cu = torch.tensor([0, 100, 4090, T], dtype=torch.int32, device="cuda")
    o = ekv.prompt_attn(view(bufs[0], 0, 2), view(bufs[0], 128, 1), view(bufs[0], 256, 1), cu,
                        out=view(bufs[1], 0, 2))
    want = ekv.prompt_attn(q, k, v, cu)
    assert torch.equal(o, want)
    _check(q[4090:], k[4090:], v[4090:], o[4090:], [0, T - 4090])
    rope = ekv.Rope(64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    qo, _ = rope(view(bufs[0], 0, 2), None, pos, q_out=view(bufs[1], 0, 2))
    assert torch.equal(qo, rope(q, None, pos)[0])


def test_rows_behind_and_before_the_sequences_are_left_and_never_read():
    """A padded buffer: rows outside the sequences hold NaN and infinities, and the
    output keeps what it held there."""
    q, k, v = _inputs(700, 8, 2, 128)
    bounds = [5, 135, 400]
    out = torch.full_like(q, 7.0)
    for x in (q, k, v):
        x[:5] = float("nan")
        x[400:] = float("inf")
        x[450:] = float("nan")
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    o = ekv.prompt_attn(q, k, v, cu, out=out)
    assert o.data_ptr() == out.data_ptr()
    _check(q, k, v, o, bounds)
    assert torch.all(o[:5] == 7) and torch.all(o[400:] == 7)


def test_a_neighbour_of_infinities_does_not_leak():
    q, k, v = _inputs(300, 4, 4, 64)
    for x in (k, v):
        x[100:200] = float("nan")
    cu = torch.tensor([0, 100, 200, 300], dtype=torch.int32, device="cuda")
    o = ekv.prompt_attn(q, k, v, cu)
    _check(q, k, v, o, [0, 100])
    _check(q[200:], k[200:], v[200:], o[200:], [0, 100])


def test_bad_bounds_leave_their_sequence_out():
    """Descending bounds, bounds below 0 and past the end: skipped; the others stand."""
    q, k, v = _inputs(260, 4, 2, 64)
    out = torch.full_like(q, 3.0)
    for bounds, good in (([-5, 10, 140, 10 ** 6], (10, 140)), ([-9, -2, 260], None),
                         ([260, 5, 105], (5, 105)), ([0, 100, 90], (0, 100))):
        cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        out[:] = 3.0
        o = ekv.prompt_attn(q, k, v, cu, out=out)
        torch.cuda.synchronize()
        a, b = good or (0, 0)
        assert torch.all(o[:a] == 3) and torch.all(o[b:] == 3)
        if good:
            _check(q[a:b], k[a:b], v[a:b], o[a:b], [0, b - a])


def test_views_of_a_fused_projection_and_scale():
    """Token strides of a fused projection, an output view, a given scale."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(333, 8 + 2 + 2, 128, generator=g, device="cuda").half()
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    big = torch.zeros(333, 10, 128, device="cuda").half()
    cu = torch.tensor([0, 200, 333], dtype=torch.int32, device="cuda")
    o = ekv.prompt_attn(q, k, v, cu, softmax_scale=0.2, out=big[:, :8])
    _check(q, k, v, o, [0, 200, 333], scale=0.2)
    assert not big[:, 8:].any()


@pytest.mark.parametrize("d", [64, 128])
def test_large_logits_and_equal_rows(d):
    """Logits of several hundred (one key takes all), and all-equal keys."""
    q, k, v = _inputs(400, 4, 2, d, seed=9, qs=40.0)
    cu = torch.tensor([0, 400], dtype=torch.int32, device="cuda")
    _check(q, k, v, ekv.prompt_attn(q, k, v, cu), [0, 400])
    k[:] = k[0, 0]
    _check(q, k, v, ekv.prompt_attn(q, k, v, cu), [0, 400])
    q[:] = 0
    v[:] = 65504
    assert torch.all(ekv.prompt_attn(q, k, v, cu) == 65504)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [100, 3000, 10000, 30000, 65504])
def test_largest_logits(size, d):
    """Logits up to fp16's end squared times d: equal keys give the mean of their values,
    opposite ones nothing; keys that rise by steps give each row its own value.  Equal
    scores have equal probabilities 2^(7 + e), e the reference's rounding; their rounding to
    fp16 (2^-11) is in the products and not in the row sum, so it stays: with the output's
    own rounding and n of 2^-23 for the sums, 2^-11 (|o| + mean |v|) + n 2^-23 mean |v|."""
    T = 300
    g = torch.Generator(device="cuda").manual_seed(d)
    row = torch.sign(torch.randn(1, 1, d, generator=g, device="cuda")).half() * size
    q, k = row.repeat(T, 2, 1), row.repeat(T, 1, 1)
    v = torch.randn(T, 1, d, generator=g, device="cuda").half()
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    live = torch.ones(T, 1, 1, dtype=torch.float64, device="cuda")
    for step in (None, 7):
        if step:
            k[step::step] *= -1
            live[step::step] = 0
        o = ekv.prompt_attn(q, k, v, cu).double()
        n = live.cumsum(0)
        want, size_v = (live * v.double()).cumsum(0) / n, (live * v.double().abs()).cumsum(0) / n
        assert torch.all((o - want).abs() <= 2.0 ** -11 * (want.abs() + size_v) +
                         T * 2.0 ** -23 * size_v)
    if size >= 3000:  # steps of 1 in 2^10 of the logit, far above one
        k = row * (0.5 + torch.arange(T, device="cuda").view(T, 1, 1) * 2.0 ** -10).half()
        assert torch.equal(ekv.prompt_attn(q, k, v, cu), v.expand(T, 2, d))
        assert torch.equal(ekv.prompt_attn(q, k, v, cu, softmax_scale=2.0 ** 126), v.expand(T, 2, d))


def test_rising_maximum():
    """Each key's logit is far above all before it, then far below: the running
    maximum moves at every key, and a late row's first keys vanish."""
    T, d = 513, 64
    q = torch.zeros(T, 1, d, device="cuda").half()
    k, v = torch.zeros_like(q), torch.randn(T, 1, d, device="cuda").half()
    q[:, 0, 0] = 64
    for sign in (1, -1):
        k[:, 0, 0] = sign * torch.arange(T, device="cuda").half() * 0.5
        cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        _check(q, k, v, ekv.prompt_attn(q, k, v, cu), [0, T])


def test_repeats_are_equal_and_graphs_replay():
    q, k, v = _inputs(1500, 8, 2, 128)
    cu = torch.tensor([0, 700, 701, 1500], dtype=torch.int32, device="cuda")
    a = ekv.prompt_attn(q, k, v, cu)
    for _ in range(3):
        assert torch.equal(a, ekv.prompt_attn(q, k, v, cu))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(a, _sync(ekv.prompt_attn(q, k, v, cu, stream=s), s))
    out = torch.zeros_like(q)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = [out, torch.zeros_like(q)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            ekv.prompt_attn(q, k, v, cu, out=o)
    cu[1] = 650
    cu[2] = 1200
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    want = ekv.prompt_attn(q, k, v, cu)
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def _sync(x, s):
    s.synchronize()
    return x


def test_two_calls_at_once():
    """Two streams, two calls in flight: no state is shared."""
    q, k, v = _inputs(4000, 8, 2, 128)
    cu = torch.tensor([0, 4000], dtype=torch.int32, device="cuda")
    a = ekv.prompt_attn(q, k, v, cu)
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in range(2)]
    outs = [ekv.prompt_attn(q, k, v, cu, stream=ss[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for o in outs)


def test_refusals():
    q, k, v = _inputs(8, 4, 2, 64)
    cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    for bad in (lambda: ekv.prompt_attn(q, k[:4], v, cu), lambda: ekv.prompt_attn(q, k, v.float(), cu),
                lambda: ekv.prompt_attn(q, k, v, cu.long()), lambda: ekv.prompt_attn(q, k, v, cu[:0]),
                lambda: ekv.prompt_attn(q.transpose(0, 1), k[:4], v[:4], cu),
                lambda: ekv.prompt_attn(q, k, v, cu, out=q[:, :2])):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(ekv.EkvError):
        ekv.prompt_attn(q[:, :3], k, v, cu)
    with pytest.raises(ekv.EkvError):
        ekv.prompt_attn(q, k, v, cu, softmax_scale=float("nan"))
