"""Attention of drafted trees over the quantized cache on the GPU, against the 64-bit
definition over the oracle's own quantize-dequantize of the same tokens, within the
bound that the oracle derives (one fp16 rounding of each probability times its value
row's scale, and of the output; fp32 otherwise)."""
import numpy as np
import pytest
import torch

from mixed_precision_quantized_gb300 import build, ekv
from oracle import serving
from oracle.decoder import SeqState

pytestmark = pytest.mark.gpu

EINVAL, EUNSUPPORTED, ESTATE = 1, 5, 6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ekv.lib()


class Case:
    """A one-layer cache of ragged sequences whose K widths go through `kbits` (one
    run of tokens each), and its oracle."""

    def __init__(self, lens, hq, hkv, d, kbits, vb, asym=False, seed=0, gain=8.0, slots=None,
                 max_seqs=None, v_scale=1.0, room=0):
        self.lens, self.hq, self.hkv, self.d, self.vb, self.asym = lens, hq, hkv, d, vb, asym
        self.rng = np.random.default_rng(seed)
        pages = sum(-(-max(t, room) // 16) + len(kbits) for t in lens) * hkv + 1
        self.cache = ekv.Cache(1, max_seqs or len(lens), hq, hkv, d, max(max(lens), 16, room),
                               {(b, vb): pages for b in set(kbits)}, [kbits[0]], [vb], asym=asym)
        self.order = list(range(len(lens))) if slots is None else slots
        self.slots = torch.tensor(self.order, dtype=torch.int32, device="cuda")
        self.state = []
        for z, t in enumerate(lens):
            st = SeqState(hkv, d, vb, None, None, asym)
            k = self.rng.normal(size=(t, hkv, d))
            k[:, :, 3] *= gain
            k, v = k.astype(np.float16), (v_scale * self.rng.normal(size=(t, hkv, d))).astype(np.float16)
            cut = [t * i // len(kbits) for i in range(len(kbits) + 1)]
            for b, a, e in zip(kbits, cut, cut[1:]):
                if e > a:
                    self.cache.set_tiers([b])
                    self.cache.append(0, self.slots[z:z + 1], torch.from_numpy(k[None, a:e]).cuda(),
                                      torch.from_numpy(v[None, a:e]).cuda())
                    st.append(k[a:e], v[a:e], b)
            self.state.append(st)
        self.cache.sync()

    def drafts(self, m, shape="tree", q_scale=1.0):
        n, r = len(self.lens), self.rng
        mk = lambda h: torch.from_numpy(r.normal(size=(n, m, h, self.d)).astype(np.float16)).cuda()  # noqa: E731
        par = np.full((n, m), -1, np.int32)
        for z in range(n):
            for i in range(1, m):
                par[z, i] = i - 1 if shape == "chain" else r.integers((i - 1) // 3, i)
        return (q_scale * mk(self.hq)).half(), mk(self.hkv), mk(self.hkv), par

    def check(self, o, q, k, v, par, cnt=None):
        o, q, k, v = (x.cpu().numpy() for x in (o, q, k, v))
        worst = 0.0
        for z, t in enumerate(self.lens):
            c = q.shape[1] if cnt is None else max(0, min(q.shape[1], int(cnt[z])))
            kh, vh = np.zeros((0, self.hkv, self.d)), np.zeros((0, self.hkv, self.d))
            if t:
                kh, vh = self.state[z].khat(), self.state[z].vhat()
            want, tol = serving.attention(q[z, :c], np.concatenate([kh, k[z, :c]]),
                                          np.concatenate([vh, v[z, :c]]),
                                          serving.tree_sees(par[z], c, t), rounded=self.sizes(vh, c))
            err = np.abs(o[z, :c].astype(np.float64) - want)
            assert np.all(err <= tol), f"sequence {z}: {np.max(err / tol):.2f} of the bound"
            worst = max(worst, float(np.max(err / tol)) if err.size else 0.0)
        return worst

    def sizes(self, vh, c):
        """What the rounded probability multiplies, where that is not the value: with the
        asymmetric quantizer a value is code * s + (zero point), |code| <= 2^(b-1), and the
        row's values span at least 2^b - 2 steps (its smallest and largest take the end
        codes, at most one step short), so |code| s <= span * 2^(b-1) / (2^b - 2)."""
        if not self.asym or self.vb == 16:
            return None
        span = vh.max(-1, keepdims=True) - vh.min(-1, keepdims=True) if len(vh) else vh[..., :1]
        w = span * 2.0 ** (self.vb - 1) / (2.0 ** self.vb - 2)
        return np.concatenate([w, np.zeros((c, self.hkv, 1))])

    def refill(self, k, v, kb, z=0):
        """Sequence z holds the rows k, v [T, Hkv, d] instead, K at kb bits."""
        self.cache.reset(self.order[z])
        self.cache.set_tiers([kb])
        self.state[z], self.lens[z] = SeqState(self.hkv, self.d, self.vb, None, None, self.asym), len(k)
        self.cache.append(0, self.slots[z:z + 1], torch.from_numpy(k[None]).cuda(),
                          torch.from_numpy(v[None]).cuda())
        self.state[z].append(k, v, kb)

    def attend(self, q, k, v, par):
        o = self.cache.tree_attn(0, self.slots, q, k, v, torch.from_numpy(par).cuda())
        self.cache.sync()
        self.check(o, q, k, v, par)
        return o

    def run(self, m, shape="tree", cnt=None, q_scale=1.0):
        q, k, v, par = self.drafts(m, shape, q_scale)
        out = torch.full_like(q, 9.0)
        dc = None if cnt is None else torch.tensor(cnt, dtype=torch.int32, device="cuda")
        o = self.cache.tree_attn(0, self.slots, q, k, v, torch.from_numpy(par).cuda(), n_nodes=dc,
                                 out=out)
        self.cache.sync()
        for z in range(len(self.lens)):
            if cnt is not None:
                assert torch.all(o[z, max(0, min(m, cnt[z])):] == 9.0)
        self.check(o, q, k, v, par, cnt)

    def close(self):
        self.cache.close()


@pytest.fixture
def case():
    made = []

    def make(*a, **kw):
        made.append(Case(*a, **kw))
        return made[-1]

    yield make
    for c in made:
        c.close()


@pytest.mark.parametrize("vb", [2, 4, 8, 16])
@pytest.mark.parametrize("kb", [2, 4, 8, 16])
@pytest.mark.parametrize("asym", [False, True], ids=["sym", "asym"])
def test_formats(case, kb, vb, asym):
    case([300], 4, 2, 64, [kb], vb, asym).run(5)
    case([333], 8, 1, 128, [kb], vb, asym).run(3)


@pytest.mark.parametrize("asym", [False, True], ids=["sym", "asym"])
@pytest.mark.parametrize("m", [1, 2, 7, 16, 33, 64])
def test_node_counts(case, m, asym):
    case([500, 40], 8, 2, 128, [4], 4, asym, seed=m).run(m)


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (5, 1, 128), (8, 1, 64), (12, 4, 128), (7, 7, 64)])
@pytest.mark.parametrize("m", [1, 6, 40])
def test_groups(case, hq, hkv, d, m):
    case([129, 70], hq, hkv, d, [8], 8).run(m)


@pytest.mark.parametrize("t", [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 1000, 2049])
@pytest.mark.parametrize("m", [1, 9])
def test_cached_lengths(case, t, m):
    case([t], 4, 1, 128, [4], 8).run(m)


@pytest.mark.parametrize("vb", [4, 16])
@pytest.mark.parametrize("asym", [False, True], ids=["sym", "asym"])
def test_mixed_widths(case, vb, asym):
    """K widths that change inside a sequence, every pair of neighbours; ragged lengths."""
    case([900, 64, 0, 415], 8, 2, 128, [8, 4, 2, 16, 2], vb, asym).run(12)
    case([700], 4, 2, 64, [2, 16, 4, 8], vb, asym).run(20)


def test_ragged_counts_and_slots(case):
    """Counts of 0, below 0 and above the rows; slots in another order; forests."""
    c = case([100, 33, 250, 16], 4, 2, 64, [4], 4, slots=[5, 0, 3, 1], max_seqs=6)
    c.run(8, cnt=[8, 0, 3, 100])
    c.run(8, cnt=[-4, 1, 8, 5])
    q, k, v, par = c.drafts(6)
    par[:] = [-1, -1, 1, 7, -9, 5]  # 7, -9 and a node that is its own parent read as -1
    o = c.cache.tree_attn(0, c.slots, q, k, v, torch.from_numpy(par).cuda())
    c.cache.sync()
    c.check(o, q, k, v, par)


@pytest.mark.parametrize("t,m,hq,hkv", [(5000, 4, 8, 1), (20000, 16, 8, 1), (9000, 64, 4, 1)])
def test_long_caches(case, t, m, hq, hkv):
    case([t], hq, hkv, 128, [4], 4).run(m)


def test_large_logits_and_small_values(case):
    """Logits of several hundred; values so small that their scales are subnormal, and
    values near the largest fp16."""
    case([400], 4, 2, 64, [8], 8).run(6, q_scale=60.0)
    for s in (1e-5, 12000.0):
        for vb in (2, 4, 8, 16):
            case([200], 4, 2, 64, [4], vb, v_scale=s).run(4)


def test_zero_values_beside_large_logits(case):
    """A cached token whose value row is all zero (scale 0) with by far the largest
    logit: the output is zero, not infinite."""
    c = case([32], 2, 1, 64, [16], 4)
    c.cache.reset(0)
    k = np.zeros((40, 1, 64), np.float16)
    v = np.ones((40, 1, 64), np.float16)
    k[5, 0, 0], v[5] = 200, 0
    c.state[0] = SeqState(1, 64, 4, None, None, False)
    c.lens = [20]
    c.cache.append(0, c.slots, torch.from_numpy(k[None, :20]).cuda(), torch.from_numpy(v[None, :20]).cuda())
    c.state[0].append(k[:20], v[:20], 16)
    q, kd, vd, par = c.drafts(3)
    q[:] = 0
    q[..., 0] = 100
    o = c.cache.tree_attn(0, c.slots, q, kd, vd, torch.from_numpy(par).cuda())
    c.cache.sync()
    c.check(o, q, kd, vd, par)


@pytest.mark.parametrize("asym", [False, True], ids=["sym", "asym"])
@pytest.mark.parametrize("vb", [2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("row", ["zero", "constant", "small span"])
@pytest.mark.parametrize("boost", [0.0, 60.0])
def test_value_rows_of_scale_zero(case, asym, vb, d, row, boost):
    """Value rows whose stored scale is 0 (all zero; equal entries and a span below the
    smallest scale, with the asymmetric quantizer), in sealed blocks and the open one,
    with logits as the others' and far above them.  What such a row adds is its zero
    point; a rounded probability (2^-11) times the centred code 2^(vb-1) <= 2^7 at the
    smallest fp16 scale 2^-24 is below 2^-28, inside the bound's 2^-24."""
    c = case([64], 4, 2, d, [16], vb, asym)
    T = 55
    k, v = (c.rng.normal(size=(T, 2, d)).astype(np.float16) for _ in range(2))
    at = [2, 17, 40, 50]
    v[at] = 3.5 if row == "constant" else 0.0
    if row == "small span":
        v[at, :, ::3] = 2.0 ** -24
    k[at, :, 0] = boost
    c.refill(k, v, 16)
    q, kd, vd, par = c.drafts(3)
    q[..., 0] = 1.0
    c.attend(q, kd, vd, par)


@pytest.mark.parametrize("asym", [False, True], ids=["sym", "asym"])
@pytest.mark.parametrize("vb", [2, 4, 8, 16])
@pytest.mark.parametrize("size", [0.1, 1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("nats", [0.0, 4.0, 8.0, 12.0])
@pytest.mark.parametrize("lead", ["drafts", "zero rows"])
def test_small_values_beside_rows_that_lead(case, asym, vb, size, nats, lead):
    """Values of one sign near `size` under equal logits, and drafts or zero rows whose
    logits lead by `nats`: each cached probability is small, rounds alike, and all of them
    together count.  They keep their bits, because the reference follows the probabilities
    times the values' scales, and the drafts (of scale 1) come after it.  (64 tokens a
    sequence and more units than CTAs: a CTA has the cached tile and the drafts' in turn.)"""
    n, T, h, d = (48, 64, 4, 64) if lead == "drafts" else (1, 2000, 2, 64)
    c = case([0] * n, h, h, d, [16], vb, asym, room=T)
    for z in range(n):
        k = np.zeros((T, h, d), np.float16)
        v = (size * (1 + 0.1 * c.rng.normal(size=(T, h, d)))).astype(np.float16)
        if lead == "zero rows":
            v[100:104] = 0
            k[100:104, :, 0] = nats
        c.refill(k, v, 16, z)
    q, kd, vd, par = c.drafts(3)
    q[..., 0] = 8.0
    vd = (size * vd.float()).half()
    kd[:] = 0
    kd[..., 0] = nats if lead == "drafts" else -100.0
    c.attend(q, kd, vd, par)


@pytest.mark.parametrize("asym", [False, True], ids=["sym", "asym"])
@pytest.mark.parametrize("kb", [2, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_largest_keys(case, asym, kb, d):
    """Key channels at fp16's end (what a saturated projection holds): their scales round
    up, so the largest stored values lie past 65504.  Such channels have small queries
    (2^-13), so that the other channels count too; decode attention on the same cache
    agrees (the tree's one node points away from every query)."""
    c = case([64], 4, 2, d, [kb], 16, asym)
    T = 53
    k, v = (c.rng.normal(size=(T, 2, d)).astype(np.float16) for _ in range(2))
    k[:, 0, 3] = np.where(np.arange(T) % 2, 65504, -65504)
    k[:, 1, 5] = 65504 - 32 * (np.arange(T) % 5)
    k[:16, 1, 7] = -65504
    k[3, 1, 7] = 60000
    c.refill(k, v, kb)
    q, kd, vd, par = c.drafts(3)
    q[..., [3, 5, 7]] *= 2.0 ** -13
    c.attend(q, kd, vd, par)
    q[:, :, 1], q[:, :, 3] = q[:, :, 0], q[:, :, 2]
    kd = -8 * q[:, :, ::2]
    o = c.attend(q[:, :1].contiguous(), kd[:, :1].contiguous(), vd[:, :1].contiguous(), par[:, :1])
    b = c.cache.decode_attn(0, c.slots, q[:, 0].contiguous()).float()
    c.cache.sync()
    assert torch.all((o[:, 0].float() - b).abs() <= 2e-3 + 1e-2 * b.abs())


@pytest.mark.parametrize("asym", [False, True], ids=["sym", "asym"])
@pytest.mark.parametrize("vb", [2, 4, 8, 16])
@pytest.mark.parametrize("d,m", [(64, 16), (128, 33), (64, 64)])
def test_draft_values_of_every_size(case, asym, vb, d, m):
    """Drafted value rows from zero and the smallest fp16 to the largest, one size a node
    (each node's own logit leads, so that its row shows), over cached values of 1 and of
    none: sequences without cached tokens too."""
    c = case([100, 0], 4, 2, d, [4], vb, asym)
    q, kd, vd, par = c.drafts(m)
    size = torch.logspace(-24, 15, m, base=2.0, device="cuda").view(1, m, 1, 1)
    size[0, m // 2] = 0
    vd = (size * vd.float().clamp(-1.9, 1.9)).half()
    q[:, :, 1], q[:, :, 3] = q[:, :, 0], q[:, :, 2]
    kd = (0.7 * q[:, :, ::2].float()).half()
    c.attend(q, kd, vd, par)


@pytest.mark.parametrize("vb", [4, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [40, 3000])
@pytest.mark.parametrize("size", [100, 3000, 10000, 30000, 65504])
def test_largest_logits(case, vb, d, T, size):
    """Logits up to fp16's end squared times d, in one CTA's run and in many: equal keys
    give the mean of their values, opposite ones (a third of the cached, and the node's
    own) nothing, as with decode attention; the values' scales are all one (a score of this
    size leaves no bits for them).  Equal scores have equal probabilities up to the
    exponent's rounding, whose rounding to fp16 (2^-11) is in the products and not in the
    row sum: 2^-11 (|o| + mean |v|), and T of 2^-23 for the sums."""
    rng = np.random.default_rng(d)
    c = case([0], 2, 1, d, [16], vb, room=T)
    row = np.sign(rng.normal(size=(1, 1, d))).astype(np.float16) * np.float16(size)
    k, v = np.repeat(row, T, 0), rng.uniform(-1, 1, size=(T, 1, d)).astype(np.float16)
    v[:, :, 5] = 1
    k[1::3] *= -1
    c.refill(k, v, 16)
    live = np.ones((T, 1))
    live[1::3] = 0
    vh = c.state[0].vhat().astype(np.float64)[:, 0]
    want = (live * vh).sum(0) / live.sum()
    mean = (live * np.abs(vh)).sum(0) / live.sum()
    q = torch.from_numpy(np.repeat(row[None], 2, 2)).cuda()
    kd, vd = torch.from_numpy(-row[None]).cuda(), torch.from_numpy(v[None, :1]).cuda()
    o = c.cache.tree_attn(0, c.slots, q, kd, vd, torch.full((1, 1), -1, dtype=torch.int32).cuda())
    b = c.cache.decode_attn(0, c.slots, q[:, 0].contiguous()).double().cpu().numpy()
    c.cache.sync()
    o = o[0, 0].double().cpu().numpy()
    assert np.all(np.abs(o - want) <= 2.0 ** -11 * (np.abs(want) + mean) + T * 2.0 ** -23 * mean)
    assert np.all(np.abs(b[0] - want) <= 2e-3 + 1e-2 * np.abs(want))


def test_trees_of_no_nodes_leave_everything(case):
    """Counts of 0 for every sequence (no unit, so no part to merge), then the scratch's
    memory goes to the next tensors: they hold what is written to them."""
    c = case([300, 20], 8, 2, 128, [4], 4)
    q, k, v, par = c.drafts(9)
    out = torch.full_like(q, 5.0)
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    for i in range(20):
        c.cache.tree_attn(0, c.slots, q, k, v, torch.from_numpy(par).cuda(), n_nodes=none, out=out)
        fill = [torch.full((1 << 22,), i, dtype=torch.int32, device="cuda") for _ in range(3)]
        assert all(torch.all(f == i) for f in fill)
    c.cache.sync()
    assert torch.all(out == 5.0)


def test_more_sequences_than_one_launch_takes(case):
    """300 sequences of 0 to 40 tokens (a launch takes 256)."""
    lens = np.random.default_rng(2).integers(0, 41, 300).tolist()
    c = case(lens, 2, 1, 64, [4], 8)
    c.run(3, cnt=np.random.default_rng(3).integers(0, 4, 300).tolist())


def test_the_same_sequence_twice_and_equal_bits(case):
    """A slot listed twice gives the same rows twice; repeated calls, and calls that
    overlap on two streams, give equal bits."""
    c = case([1500, 600], 8, 2, 128, [4, 2], 4)
    q, k, v, par = c.drafts(9)
    q[1], k[1], v[1], par[1] = q[0], k[0], v[0], par[0]
    dp = torch.from_numpy(par).cuda()
    twice = torch.zeros(2, dtype=torch.int32, device="cuda")
    a = c.cache.tree_attn(0, twice, q, k, v, dp)
    c.cache.sync()
    c.state[1], c.lens = c.state[0], [1500, 1500]
    c.check(a, q, k, v, par)
    ss = [torch.cuda.Stream() for _ in range(2)]
    for s in ss:
        s.wait_stream(torch.cuda.current_stream())
    outs = [c.cache.tree_attn(0, twice, q, k, v, dp, stream=ss[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for o in outs)


@pytest.mark.parametrize("scale,ok", [(1e-6, True), (0.01, True), (3.0, True), (900.0, True),
                                      (1e-9, False), (1e6, False)])
def test_softmax_scales(scale, ok):
    """The handle's own scale, from one that makes every weight equal to one that leaves
    the largest alone; outside the stated range the call is refused."""
    rng = np.random.default_rng(5)
    cache = ekv.Cache(1, 1, 4, 2, 64, 64, {(8, 8): 16}, [8], [8], softmax_scale=scale)
    st = SeqState(2, 64, 8, None, None, False)
    k, v = (rng.normal(size=(50, 2, 64)).astype(np.float16) for _ in range(2))
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.append(0, slots, torch.from_numpy(k[None]).cuda(), torch.from_numpy(v[None]).cuda())
    st.append(k, v, 8)
    q, kd, vd = (torch.from_numpy(rng.normal(size=(1, 3, h, 64)).astype(np.float16)).cuda()
                 for h in (4, 2, 2))
    par = torch.tensor([[-1, 0, 0]], dtype=torch.int32, device="cuda")
    if ok:
        o = cache.tree_attn(0, slots, q, kd, vd, par)
        cache.sync()
        want, tol = serving.attention(
            q[0].cpu().numpy(), np.concatenate([st.khat(), kd[0].cpu().numpy()]),
            np.concatenate([st.vhat(), vd[0].cpu().numpy()]),
            serving.tree_sees([-1, 0, 0], 3, 50), np.float32(scale))
        assert np.all(np.abs(o[0].double().cpu().numpy() - want) <= tol)
    else:
        with pytest.raises(ekv.EkvError) as e:
            cache.tree_attn(0, slots, q, kd, vd, par)
        assert e.value.code == EUNSUPPORTED
    cache.close()


def test_one_node_equals_the_decode_step():
    """A tree of one node over the cache is the decode step's attention: append the
    node on a twin and read it back through ekv_append_decode_attn (the newest token
    sits in the open block, whose K rows are raw)."""
    c = Case([100, 37], 8, 2, 128, [4], 16, seed=4)
    q, k, v, par = c.drafts(1)
    a = c.cache.tree_attn(0, c.slots, q, k, v, torch.from_numpy(par).cuda())
    c.cache.sync()
    b = c.cache.append_decode_attn(0, c.slots, k, v, q[:, 0].contiguous())
    c.cache.sync()
    err = (a[:, 0].float() - b.float()).abs()
    assert torch.all(err <= 2e-3 + 1e-2 * b.float().abs())
    c.close()


def test_cache_is_only_read(case):
    c = case([70, 5], 4, 2, 64, [4], 4)
    before = [c.cache.read_pages(0, s, h, 0, 1).cpu() for s in (0, 1) for h in (0, 1)]
    c.run(9)
    after = [c.cache.read_pages(0, s, h, 0, 1).cpu() for s in (0, 1) for h in (0, 1)]
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    assert [c.cache.seq_len(0, s) for s in (0, 1)] == [70, 5]


def test_graphs_streams_and_repeats(case):
    """Two graphs captured of one handle, replayed in turn after the cache has grown;
    another stream; equal results each time (decode attention runs between them)."""
    c = case([600, 90], 8, 2, 128, [4, 8], 4)
    q, k, v, par = c.drafts(10)
    dp = torch.from_numpy(par).cuda()
    outs = [torch.zeros_like(q) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    first = c.cache.tree_attn(0, c.slots, q, k, v, dp)
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            c.cache.tree_attn(0, c.slots, q, k, v, dp, out=o)
    for i in (0, 1, 0):
        graphs[i].replay()
        c.cache.decode_attn(0, c.slots, q[:, 0].contiguous())
    c.cache.sync()
    c.check(outs[0], q, k, v, par)
    c.check(outs[1], q, k, v, par)
    c.check(first, q, k, v, par)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = c.cache.tree_attn(0, c.slots, q, k, v, dp, stream=s)
    c.cache.sync(stream=s)
    c.check(other, q, k, v, par)


def test_device_errors_and_refusals(case):
    c = case([20], 4, 2, 64, [4], 4)
    q, k, v, par = c.drafts(3)
    dp = torch.from_numpy(par).cuda()
    bad = torch.tensor([7], dtype=torch.int32, device="cuda")
    c.cache.tree_attn(0, bad, q, k, v, dp)  # a slot outside the handle: device error
    with pytest.raises(ekv.EkvError) as e:
        c.cache.sync()
    assert e.value.code == EINVAL
    o = c.cache.tree_attn(0, c.slots, q, k, v, dp)
    c.cache.sync()
    c.check(o, q, k, v, par)
    for call in (lambda: c.cache.tree_attn(0, c.slots, q[:, :2], k, v, dp),
                 lambda: c.cache.tree_attn(0, c.slots, q, k, v.float(), dp),
                 lambda: c.cache.tree_attn(0, c.slots, q, k, v, dp.long()),
                 lambda: c.cache.tree_attn(0, c.slots, q, k, v, dp, n_nodes=dp),
                 lambda: c.cache.tree_attn(0, c.slots, q, k, v, dp, out=q[:, :, :2])):
        with pytest.raises((TypeError, ValueError)):
            call()
    with pytest.raises(ekv.EkvError):
        c.cache.tree_attn(1, c.slots, q, k, v, dp)
    with pytest.raises(ekv.EkvError):
        c.cache.tree_attn(0, c.slots, *(torch.zeros(1, 65, h, 64, device="cuda").half() for h in (4, 2, 2)),
                          torch.zeros(1, 65, dtype=torch.int32, device="cuda"))
    assert c.cache.tree_attn(0, c.slots[:0], q[:0], k[:0], v[:0], dp[:0]).shape[0] == 0
