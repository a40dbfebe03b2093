"""Measured cases of the serving operators around the mixed-precision KV cache: rotary
positions, attention over packed prompts, attention of drafted trees over the quantized
cache, and verification of drafted trees.

`run` computes each operator in a plain form (elementary torch operations in 32 bits, in
64 where that matters) or, with `own` set, through the library's entry points.  `exact`
gives the same outputs in 64 bits, computed apart from the plain form.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16  # tokens per cache page
DEV = "cuda"


# ---- cases ---------------------------------------------------------------------------
def listed():
    return [
        # q and k of one decode step of 32 sequences (the ragged batch-32 workload), latency
        dict(name="rope_step", op="rope", tokens=32, hq=32, hkv=8, d=128, rot=128, layout="half",
             scaling="none", base=500000.0, factor=1.0, far=8192, fused=False),
        # a long prompt's q and k read from the fused projection, long-context scaling, far
        # positions, half of the head rotated, an odd token count
        dict(name="rope_part", op="rope", tokens=4099, hq=64, hkv=8, d=128, rot=64, layout="half",
             scaling="yarn", base=10000.0, factor=32.0, far=131072, fused=True),
        # a whole 32K prompt, 40 query heads, interleaved pairs, banded scaling
        dict(name="rope_prompt", op="rope", tokens=32768, hq=40, hkv=8, d=128, rot=128,
             layout="interleaved", scaling="banded", base=500000.0, factor=8.0, far=131072,
             fused=False),
        # one short prompt of the two-layer test workload, latency
        dict(name="prompt_tiny", op="prompt", seqs=1, lo=256, hi=256, hq=4, hkv=2, d=64),
        # a batch of ragged prompts, from one token to 2K
        dict(name="prompt_packed", op="prompt", seqs=24, lo=1, hi=2047, hq=32, hkv=8, d=128),
        # one long prompt
        dict(name="prompt_long", op="prompt", seqs=1, lo=16384, hi=16384, hq=32, hkv=8, d=128),
        # short drafted chains of a batch of 8 at 4K, 8-bit pages
        dict(name="tree_chain", op="tree", seqs=8, lo=4096, hi=4096, hq=32, hkv=8, d=128, nodes=4,
             shape="chain", ragged=False, kbits="8", vbits=8),
        # one sequence at 128K, 64 query heads, 4-bit pages, a tree of 16
        dict(name="tree_long", op="tree", seqs=1, lo=131072, hi=131072, hq=64, hkv=8, d=128,
             nodes=16, shape="tree", ragged=False, kbits="4", vbits=4),
        # a ragged batch of 32 with trees of up to 64 nodes, K widths that changed on the way
        dict(name="tree_batch", op="tree", seqs=32, lo=1024, hi=8191, hq=32, hkv=8, d=128, nodes=64,
             shape="tree", ragged=True, kbits="8,4,2", vbits=4),
        # one sequence, a chain of 8 sampled drafts with their probabilities, latency
        dict(name="verify_one", op="verify", seqs=1, nodes=8, shape="chain", vocab=32768, draft=True,
             ragged=False),
        # a batch of sampled trees with their draft probabilities, an odd vocabulary
        dict(name="verify_draft", op="verify", seqs=16, nodes=16, shape="tree", vocab=100003,
             draft=True, ragged=True),
        # a batch of large top-k trees against the target's probabilities alone
        dict(name="verify_batch", op="verify", seqs=32, nodes=64, shape="tree", vocab=131072,
             draft=False, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "tree", "verify"])
    if op == "rope":
        hq, hkv = rng.choice([(32, 8), (40, 8), (64, 8), (4, 2), (7, 1)])
        d = rng.choice([64, 128])
        tokens = _log(rng, 1, 32768 * 48 // (hq + hkv))
        return dict(op=op, tokens=min(tokens, 32768), hq=hq, hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4, 20]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "banded", "yarn"]),
                    base=rng.choice([10000.0, 500000.0]), factor=rng.choice([2.0, 8.0, 32.0]),
                    far=_log(rng, 32, 1 << 20), fused=rng.random() < 0.5)
    if op == "prompt":
        hq, hkv = rng.choice([(32, 8), (40, 8), (64, 8), (4, 2), (8, 8)])
        seqs = _log(rng, 1, 32)
        hi = _log(rng, 1, min(8192, int(16384 * math.sqrt(32 / (seqs * hq)))))
        return dict(op=op, seqs=seqs, lo=rng.randint(1, hi), hi=hi, hq=hq, hkv=hkv,
                    d=rng.choice([64, 128]))
    if op == "tree":
        hq, hkv = rng.choice([(32, 8), (40, 8), (64, 8), (4, 2), (8, 8)])
        seqs = _log(rng, 1, 32)
        nodes = _log(rng, 1, 64)
        hi = _log(rng, 1, min(65536 // seqs, (1 << 27) // (seqs * nodes * hq)))
        return dict(op=op, seqs=seqs, lo=rng.randint(1, hi), hi=hi, hq=hq, hkv=hkv,
                    d=rng.choice([64, 128]), nodes=nodes,
                    shape=rng.choice(["chain", "tree"]), ragged=rng.random() < 0.5,
                    kbits=rng.choice(["2", "4", "8", "16", "8,4", "4,2", "16,8,4,2"]),
                    vbits=rng.choice([2, 4, 8, 16]))
    draft = rng.random() < 0.5
    return dict(op=op, seqs=_log(rng, 1, 16), nodes=_log(rng, 1, 16 if draft else 64),
                shape=rng.choice(["chain", "tree"]), vocab=_log(rng, 32, 100003 if draft else 131072),
                draft=draft,
                ragged=rng.random() < 0.5)


# ---- inputs --------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)


def _lengths(case, seed):
    """Lengths in [lo, hi], drawn in pairs about the middle: their sum goes by the case alone."""
    r = random.Random(int(seed) * 31 + 7)
    lens = []
    while len(lens) < case["seqs"]:
        t = r.randint(case["lo"], case["hi"])
        lens += [t, case["lo"] + case["hi"] - t]
    if case["seqs"] % 2:
        lens[-2:] = [(case["lo"] + case["hi"]) // 2]
    r.shuffle(lens)
    return lens


def _parents(case, seed):
    """Parents [seqs][nodes] (node 0 the root, -1) and node counts [seqs]."""
    r = random.Random(int(seed) * 17 + 3)
    m, par, cnt = case["nodes"], [], []
    for _ in range(case["seqs"]):
        par.append([-1] + [i - 1 if case["shape"] == "chain" else r.randint((i - 1) // 3, i - 1)
                           for i in range(1, m)])
        cnt.append(r.randint(1, m) if case["ragged"] else m)
    return par, cnt


def _freqs(case):
    """Radians per position of each rotated pair, and the magnitude of cos and sin."""
    r, base, s = case["rot"], case["base"], case["factor"]
    f = base ** (-np.arange(0, r, 2, dtype=np.float64) / r)
    kind, length = case["scaling"], 8192.0
    if kind == "linear":
        return f / s, 1.0
    if kind == "banded":  # short waves kept, long ones stretched, between them a blend
        lo, hi = 1.0, 4.0
        w = np.clip((length * f / (2 * np.pi) - lo) / (hi - lo), 0.0, 1.0)
        return f * (w + (1 - w) / s), 1.0
    if kind == "yarn":
        edge = lambda turns: r * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(edge(32.0)), 0), min(math.ceil(edge(1.0)), r - 1)
        w = np.clip((np.arange(r // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return f * (1 - w + w / s), 0.1 * math.log(s) + 1.0 if s > 1 else 1.0
    return f, 1.0


def _prepare_rope(case, seed):
    g = _gen(seed)
    n, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    if case["fused"]:  # views of one projection's output
        x = torch.randn(n, hq + 2 * hkv, d, generator=g, device=DEV).half()
        q, k = x[:, :hq], x[:, hq:hq + hkv]
    else:
        q = torch.randn(n, hq, d, generator=g, device=DEV).half()
        k = torch.randn(n, hkv, d, generator=g, device=DEV).half()
    start = random.Random(int(seed)).randint(0, max(0, case["far"] - n))
    pos = (torch.arange(n, device=DEV, dtype=torch.int32) + start
           if n > 64 else torch.randint(0, case["far"], (n,), generator=g, device=DEV).int())
    st = dict(op="rope", q=q, k=k, pos=pos, rot=case["rot"], layout=case["layout"])
    if own:
        from mixed_precision_quantized_gb300 import ekv
        st["rope"] = ekv.Rope(d, rot_dim=case["rot"], layout=case["layout"], base=case["base"],
                              scaling=case["scaling"], factor=case["factor"], original_len=8192,
                              device=DEV)
    else:
        f, mag = _freqs(case)
        st["freqs"], st["mag"] = torch.tensor(f, device=DEV), mag
    return st


def _prepare_prompt(case, seed):
    g, lens = _gen(seed), _lengths(case, seed)
    t, hq, hkv, d = sum(lens), case["hq"], case["hkv"], case["d"]
    q = (1.5 * torch.randn(t, hq, d, generator=g, device=DEV)).half()
    k = torch.randn(t, hkv, d, generator=g, device=DEV).half()
    v = torch.randn(t, hkv, d, generator=g, device=DEV).half()
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    return dict(op="prompt", q=q, k=k, v=v, cu=cu, lens=lens)


def _block_bits(case, t):
    """K bits of each 16-token block of a sequence of t tokens: the widths in turn."""
    bits, nb = [int(b) for b in case["kbits"].split(",")], -(-t // BLOCK)
    return [bits[j * len(bits) // nb] for j in range(nb)]


def _cached_kv(case, g, t):
    hkv, d = case["hkv"], case["d"]
    gain = torch.ones(hkv, d, device=DEV)
    gain[:, 3] = 8.0  # an outlier channel
    k = (torch.randn(t, hkv, d, generator=g, device=DEV) * gain).half()
    v = torch.randn(t, hkv, d, generator=g, device=DEV).half()
    return k, v


def _codes(x, bits, dim):
    """Symmetric codes and fp16 scales of x (fp16), one group along `dim`."""
    qm = float(2 ** (bits - 1) - 1)
    x = x.float()
    s = (x.abs().amax(dim, keepdim=True) / qm).half()
    sf = s.float()
    return torch.where(sf > 0, (x / sf).round().clamp(-qm, qm), torch.zeros_like(x)).to(torch.int8), s


def _prepare_tree(case, seed):
    g, lens = _gen(seed), _lengths(case, seed)
    n, m, hq, hkv, d, vb = (case[x] for x in ("seqs", "nodes", "hq", "hkv", "d", "vbits"))
    par, cnt = _parents(case, seed)
    st = dict(op="tree", lens=lens, counts=cnt, n=n, m=m, par=par,
              q=torch.randn(n, m, hq, d, generator=g, device=DEV).half(),
              k=torch.randn(n, m, hkv, d, generator=g, device=DEV).half(),
              v=torch.randn(n, m, hkv, d, generator=g, device=DEV).half(),
              parents=torch.tensor(par, dtype=torch.int32, device=DEV),
              cnt=torch.tensor(cnt, dtype=torch.int32, device=DEV),
              slots=torch.arange(n, dtype=torch.int32, device=DEV),
              o=torch.zeros(n, m, hq, d, dtype=torch.float16, device=DEV))
    widths = [_block_bits(case, t) for t in lens]
    if own:
        from mixed_precision_quantized_gb300 import ekv
        pools = {}
        for w in widths:
            for b in w:
                pools[(b, vb)] = pools.get((b, vb), 0) + hkv
        cache = ekv.Cache(1, n, hq, hkv, d, max(lens), pools, [widths[0][0]], [vb], device=DEV)
    else:
        kv = []
    for z, t in enumerate(lens):
        k, v = _cached_kv(case, g, t)
        runs, j = [], 0  # runs of blocks of one K width: (bits, first token, end)
        while j < len(widths[z]):
            e = j
            while e < len(widths[z]) and widths[z][e] == widths[z][j]:
                e += 1
            runs.append((widths[z][j], j * BLOCK, min(e * BLOCK, t)))
            j = e
        if own:
            for b, t0, t1 in runs:
                cache.set_tiers([b])
                cache.append(0, st["slots"][z:z + 1], k[None, t0:t1], v[None, t0:t1])
        else:
            parts = []  # (codes [blocks, 16, hkv, d], scales) or raw rows
            for b, t0, t1 in runs:
                full = (t1 - t0) // BLOCK * BLOCK
                x = k[t0:t0 + full].view(-1, BLOCK, hkv, d)
                if full:
                    parts.append((x, None) if b == 16 else _codes(x, b, 1))
                if full < t1 - t0:  # the open block's rows stay raw
                    parts.append((k[t0 + full:t1], None))
            kv.append((parts, (v, None) if vb == 16 else _codes(v, vb, 2)))
    if own:
        cache.sync()
        st["cache"] = cache
    else:
        st["kv"] = kv
    return st


def _prepare_verify(case, seed):
    g = _gen(seed)
    n, m, V = case["seqs"], case["nodes"], case["vocab"]
    par, cnt = _parents(case, seed)
    parents = torch.tensor(par, dtype=torch.int32, device=DEV)
    p = torch.empty(n, m, V, device=DEV)
    q = torch.empty(n, m, V, device=DEV) if case["draft"] else None
    tokens = torch.zeros(n, m, dtype=torch.int32, device=DEV)
    rank = [[sum(par[z][j] == par[z][i] for j in range(1, i)) for i in range(m)] for z in range(n)]
    for z in range(n):
        x = 3.0 * torch.randn(m, V, generator=g, device=DEV)
        peak = torch.randint(0, V, (m, 1), generator=g, device=DEV)
        x.scatter_add_(1, peak, 16.0 * torch.rand(m, 1, generator=g, device=DEV))
        p[z] = torch.softmax(x, -1)
        y = x + 0.7 * torch.randn(m, V, generator=g, device=DEV)  # the draft model's view
        up = parents[z].long().clamp(min=0)
        if case["draft"]:
            q[z] = torch.softmax(y, -1)
            tokens[z] = torch.multinomial(q[z][up], 1, generator=g)[:, 0].int()
        else:
            k = min(V, max(rank[z]) + 1)
            best = y.topk(k, -1).indices[up]
            r = torch.tensor(rank[z], device=DEV).clamp(max=k - 1)
            tokens[z] = best.gather(1, r[:, None])[:, 0].int()
    return dict(op="verify", p=p, q=q, tokens=tokens, parents=parents,
                cnt=torch.tensor(cnt, dtype=torch.int32, device=DEV),
                u=torch.rand(n, m, generator=g, device=DEV),
                us=torch.rand(n, generator=g, device=DEV))


def prepare(case, seed):
    return {"rope": _prepare_rope, "prompt": _prepare_prompt, "tree": _prepare_tree,
            "verify": _prepare_verify}[case["op"]](case, seed)


# ---- plain forms ---------------------------------------------------------------------
def _rope_plain(s):
    ang = s["pos"].double()[:, None] * s["freqs"]
    cos, sin = (s["mag"] * ang.cos()).float()[:, None], (s["mag"] * ang.sin()).float()[:, None]
    r = s["rot"]

    def turn(x):
        y = x.float()
        out = y.clone()
        if s["layout"] == "half":
            a, b = y[..., :r // 2], y[..., r // 2:r]
            out[..., :r // 2], out[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            out[..., 0:r:2], out[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
        return out.half()

    return [turn(s["q"]), turn(s["k"])]


def _softmax(x):
    e = (x - x.amax(-1, keepdim=True)).exp()
    return e / e.sum(-1, keepdim=True)


def _prompt_plain(s):
    q, k, v = s["q"], s["k"], s["v"]
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    grp, o, t0 = hq // hkv, torch.empty_like(q), 0
    for t in s["lens"]:
        kz, vz = (x[t0:t0 + t].float().transpose(0, 1) for x in (k, v))  # [hkv, t, d]
        rows = max(1, min(t, (1 << 28) // (hq * t)))
        for a in range(0, t, rows):
            b = min(t, a + rows)
            qz = q[t0 + a:t0 + b].float().view(b - a, hkv, grp, d).permute(1, 2, 0, 3)
            x = torch.matmul(qz.reshape(hkv, grp * (b - a), d), kz[:, :b].transpose(1, 2))
            x = x.view(hkv, grp, b - a, b) / math.sqrt(d)
            i = torch.arange(a, b, device=DEV)[:, None]
            x = x.masked_fill(torch.arange(b, device=DEV) > i, -math.inf)
            y = torch.matmul(_softmax(x).view(hkv, grp * (b - a), b), vz[:, :b])
            o[t0 + a:t0 + b] = y.view(hkv, grp, b - a, d).permute(2, 0, 1, 3).reshape(
                b - a, hq, d).half()
        t0 += t
    return [o]


def _ancestors(parents):
    """[n, m, m] truth: column j is row i itself or one of its ancestors."""
    n, m = parents.shape
    up = (parents[:, :, None] == torch.arange(m, device=DEV)).double()
    eye = torch.eye(m, device=DEV, dtype=torch.float64)
    return torch.linalg.matrix_power(eye + up, max(m, 1)) > 0


def _tree_plain(s):
    q, o = s["q"], s["o"]
    n, m, hq, d = q.shape
    hkv = s["k"].shape[2]
    grp, see = hq // hkv, _ancestors(s["parents"])
    for z in range(n):
        c = s["counts"][z]
        parts, (vq, vs) = s["kv"][z]
        kz = [x.float().reshape(-1, hkv, d) if sc is None else
              (x.float() * sc.float()).reshape(-1, hkv, d) for x, sc in parts]
        kz = torch.cat(kz + [s["k"][z, :c].float()]).permute(1, 2, 0)        # [hkv, d, T + c]
        vz = vq.float() if vs is None else vq.float() * vs.float()
        vz = torch.cat([vz, s["v"][z, :c].float()]).transpose(0, 1)          # [hkv, T + c, d]
        qz = q[z, :c].float().view(c, hkv, grp, d).permute(1, 2, 0, 3).reshape(hkv, grp * c, d)
        x = (torch.matmul(qz, kz) / math.sqrt(d)).view(hkv, grp, c, -1)
        x[..., x.shape[-1] - c:].masked_fill_(~see[z, :c, :c], -math.inf)
        y = torch.matmul(_softmax(x).view(hkv, grp * c, -1), vz)
        o[z, :c] = y.view(hkv, grp, c, d).permute(2, 0, 1, 3).reshape(c, hq, d).half()
    return [o]


def _verify_plain(s):
    p, q, par, u = s["p"], s["q"], s["parents"].long(), s["u"].double()
    n, m, V = p.shape
    z, idx = torch.arange(n, device=DEV)[:, None], torch.arange(m, device=DEV)
    up, tok = par.clamp(min=0), s["tokens"].long()
    live = (idx < s["cnt"][:, None]) & (idx > 0)
    same = live[:, :, None] & live[:, None] & (par[:, :, None] == par[:, None])
    before = same & (idx < idx[:, None])                    # [n, i, j]: j an earlier sibling of i
    if q is None:
        twin = (before & (tok[:, :, None] == tok[:, None])).any(-1)
        px = torch.where(twin, 0.0, p[z, up, tok].double())
        left = 1.0 - (before.double() * px[:, None]).sum(-1)
        take = live & (u * left < px)
    else:
        r, left = p.double(), torch.ones(n, m, device=DEV, dtype=torch.float64)
        rank, take = before.sum(-1), torch.zeros_like(live)
        done = torch.zeros_like(live)                       # by parent: a child was taken
        for k in range(int(rank.max()) + 1):
            now = live & (rank == k)
            qx, rx = q[z, up, tok].double(), r[z, up, tok]
            ok = now & (u * qx * left[z, up] < rx)
            take = take | ok
            has = torch.zeros(n, m, dtype=torch.long, device=DEV)
            has.scatter_add_(1, up, now.long())
            won = torch.zeros(n, m, dtype=torch.long, device=DEV)
            won.scatter_add_(1, up, ok.long())
            done = done | (won > 0)
            cut = (has > 0) & ~done
            nr = (r - left[..., None] * q.double()).clamp(min=0)
            r = torch.where(cut[..., None], nr, r)
            left = torch.where(cut, r.sum(-1), left)
    first = take & ~(before & take[:, None]).any(-1)
    root = (idx == 0) & (s["cnt"][:, None] > 0)
    see = _ancestors(s["parents"])
    reached = ~(see & ~(first | root)[:, None]).any(-1)
    last = torch.where(reached, idx, -1).amax(-1).clamp(min=0)
    taken = reached & (idx > 0)
    path = torch.full((n, m), -1, dtype=torch.int32, device=DEV)
    at = torch.where(taken, taken.cumsum(-1) - 1, m - 1)
    path.scatter_reduce_(1, at, torch.where(taken, idx, -1).int(), "amax")
    z1 = z[:, 0]
    rows = p[z1, last].double()
    if q is None:
        kids = live & (par == last[:, None])
        gone = torch.zeros(n, V, device=DEV)
        gone.scatter_add_(1, tok, kids.float())
        rest = torch.where(gone > 0, 0.0, rows)
    else:
        rest = r[z1, last]
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, rows)
    cum = rest.cumsum(-1)
    nxt = torch.searchsorted(cum, s["us"].double()[:, None] * cum[:, -1:], right=True)[:, 0]
    nxt = torch.where(s["cnt"] > 0, nxt.clamp(max=V - 1), -1).int()
    return [path, taken.sum(-1).int(), nxt]


def run(state):
    op = state["op"]
    if own:
        if op == "rope":
            return list(state["rope"](state["q"], state["k"], state["pos"]))
        if op == "prompt":
            from mixed_precision_quantized_gb300 import ekv
            return [ekv.prompt_attn(state["q"], state["k"], state["v"], state["cu"])]
        if op == "tree":
            return [state["cache"].tree_attn(0, state["slots"], state["q"], state["k"], state["v"],
                                             state["parents"], n_nodes=state["cnt"],
                                             out=state["o"])]
        from mixed_precision_quantized_gb300 import ekv
        return list(ekv.verify_tree(state["p"], state["tokens"], state["parents"], state["u"],
                                    state["us"], draft_probs=state["q"], n_nodes=state["cnt"]))
    return {"rope": _rope_plain, "prompt": _prompt_plain, "tree": _tree_plain,
            "verify": _verify_plain}[op](state)


# ---- what one pass cannot do without -------------------------------------------------
def work(case):
    op = case["op"]
    if op == "rope":
        n, h, d = case["tokens"], case["hq"] + case["hkv"], case["d"]
        return dict(bytes=4 * n * h * d + 4 * n + 4 * case["rot"], flops=3 * n * h * case["rot"])
    if op == "verify":
        return dict(bytes=case["seqs"] * (4 * case["vocab"] * (2 if case["draft"] else 1)
                                          + 20 * case["nodes"] + 12),
                    flops=case["seqs"] * case["vocab"] * (4 if case["draft"] else 1))
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    t = (case["lo"] + case["hi"]) / 2  # the mean length of a sequence
    if op == "prompt":
        pairs = ((case["hi"] ** 2 + case["hi"] * case["lo"] + case["lo"] ** 2) / 3 + t) / 2
        return dict(bytes=case["seqs"] * t * (2 * hq + 2 * hkv) * d * 2,
                    flops=case["seqs"] * 4 * pairs * hq * d)
    m = (1 + case["nodes"]) / 2 if case["ragged"] else case["nodes"]
    kb = [int(b) for b in case["kbits"].split(",")]
    page = sum(2 * BLOCK * d if b == 16 else BLOCK * d * b / 8 + 2 * d for b in kb) / len(kb)
    page += 2 * BLOCK * d if case["vbits"] == 16 else BLOCK * d * case["vbits"] / 8 + 2 * BLOCK
    return dict(bytes=case["seqs"] * (t / BLOCK * hkv * page + m * (2 * hq + 2 * hkv) * d * 2),
                flops=case["seqs"] * 4 * m * (t + 1) * hq * d)


# ---- 64 bits, apart from the plain forms ---------------------------------------------
def _exact_attention(q, k, v, allowed=None, causal_from=None):
    """q [R, d], k, v [T, d] in fp64; row i sees columns `allowed[i]`, or j <= causal_from + i."""
    x = q @ k.T
    x *= q.shape[1] ** -0.5
    if causal_from is not None:
        j = torch.arange(k.shape[0], device=x.device)
        i = causal_from + torch.arange(q.shape[0], device=x.device)
        x.masked_fill_(j[None] > i[:, None], -math.inf)
    if allowed is not None:
        x.masked_fill_(~allowed, -math.inf)
    return torch.exp(x - torch.logsumexp(x, 1, keepdim=True)) @ v


def _exact_rope(s, case):
    f, mag = _freqs(case)
    ang = torch.outer(s["pos"].double(), torch.tensor(f, device=DEV))
    w = mag * torch.polar(torch.ones_like(ang), ang)[:, None]
    r, out = case["rot"], []
    for x in (s["q"], s["k"]):
        y = x.double()
        n, h, _ = y.shape
        pairs = (y[..., :r].view(n, h, 2, r // 2).transpose(2, 3) if case["layout"] == "half"
                 else y[..., :r].view(n, h, r // 2, 2))
        t = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
        t = t.transpose(2, 3) if case["layout"] == "half" else t
        out.append(torch.cat([t.reshape(n, h, r), y[..., r:]], -1))
    return out


def _exact_prompt(s, case):
    o, t0, grp = torch.empty_like(s["q"], dtype=torch.float64), 0, case["hq"] // case["hkv"]
    for t in s["lens"]:
        for h in range(case["hq"]):
            k, v = (s[x][t0:t0 + t, h // grp].double() for x in "kv")
            for a in range(0, t, 4096):
                b = min(t, a + 4096)
                o[t0 + a:t0 + b, h] = _exact_attention(s["q"][t0 + a:t0 + b, h].double(), k[:b],
                                                       v[:b], causal_from=a)
        t0 += t
    return [o]


def _stored(x, bits, groups):
    """What a quantizer with fp16 scales holds of x [groups..., members, ...] along dim `groups`."""
    if bits == 16:
        return x.double()
    top = 2 ** (bits - 1) - 1
    step = (x.float().abs().max(groups, keepdim=True).values / torch.tensor(float(top))).half()
    code = torch.round(x.float() / step.float()).nan_to_num(0.0, 0.0, 0.0)
    return code.clamp(-top, top).double() * step.double()


def _exact_tree(case, seed):
    g, lens = _gen(seed), _lengths(case, seed)
    n, m, hq, hkv, d = (case[x] for x in ("seqs", "nodes", "hq", "hkv", "d"))
    par, cnt = _parents(case, seed)
    q, kd, vd = (torch.randn(n, m, h, d, generator=g, device=DEV).half().double()
                 for h in (hq, hkv, hkv))
    o = torch.zeros(n, m, hq, d, dtype=torch.float64, device=DEV)
    for z, t in enumerate(lens):
        k, v = _cached_kv(case, g, t)
        kk = k.double()
        for j, b in enumerate(_block_bits(case, t)):
            if (j + 1) * BLOCK <= t:
                kk[j * BLOCK:(j + 1) * BLOCK] = _stored(k[j * BLOCK:(j + 1) * BLOCK], b, 0)
        kk = torch.cat([kk, kd[z, :cnt[z]]])
        vv = torch.cat([_stored(v, case["vbits"], 2), vd[z, :cnt[z]]])
        see = np.zeros((cnt[z], t + cnt[z]), dtype=bool)
        see[:, :t] = True
        for i in range(cnt[z]):
            a = i
            while a >= 0:
                see[i, t + a] = True
                a = par[z][a]
        see = torch.tensor(see, device=DEV)
        for h in range(hq):
            o[z, :cnt[z], h] = _exact_attention(q[z, :cnt[z], h], kk[:, h * hkv // hq],
                                                vv[:, h * hkv // hq], allowed=see)
    return [o]


def _exact_verify(s, case):
    n, m, V = s["p"].shape
    path, acc, nxt = np.full((n, m), -1, np.int32), np.zeros(n, np.int32), np.full(n, -1, np.int32)
    tok, par, cnt = (s[x].cpu().numpy() for x in ("tokens", "parents", "cnt"))
    u, us = (s[x].double().cpu().numpy() for x in ("u", "us"))
    for z in range(n):
        node = 0
        while cnt[z] > 0:
            p = s["p"][z, node].double().cpu().numpy()
            r, left, moved = p.copy(), 1.0, False
            q = None if s["q"] is None else s["q"][z, node].double().cpu().numpy()
            for c in range(1, cnt[z]):
                if par[z, c] != node:
                    continue
                x = tok[z, c]
                if u[z, c] * left * (1.0 if q is None else q[x]) < r[x]:
                    path[z, acc[z]] = node = c
                    acc[z] += 1
                    moved = True
                    break
                if q is None:
                    left -= r[x]
                    r[x] = 0.0
                else:
                    r = np.maximum(r - left * q, 0.0)
                    left = r.sum()
            if not moved:
                cum = np.cumsum(r if r.sum() > 0 else p)
                nxt[z] = min(V - 1, int(np.searchsorted(cum, us[z] * cum[-1], side="right")))
                break
    return [torch.from_numpy(path), torch.from_numpy(acc), torch.from_numpy(nxt)]


def exact(case, seed):
    if case["op"] == "tree":
        return _exact_tree(case, seed)
    s = prepare(case, seed)
    return {"rope": _exact_rope, "prompt": _exact_prompt, "verify": _exact_verify}[case["op"]](s, case)
