"""The serving operators together, as a program uses them: a prompt rotated, attended
and appended; then steps that draft a tree, rotate it by depth, attend it over the
cache, verify it and append the accepted path.  The 64-bit oracle runs the same
sequence of steps on the same numbers."""
import numpy as np
import pytest
import torch

from mixed_precision_quantized_gb300 import build, ekv
from oracle import serving
from oracle.decoder import SeqState

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("draft", [False, True], ids=["target", "draft"])
def test_speculative_decoding_run(draft):
    build.build()
    rng = np.random.default_rng(7)
    hq, hkv, d, m, V, lens, steps = 8, 2, 64, 7, 97, [70, 1, 33], 5
    n = len(lens)
    kb = 8
    cache = ekv.Cache(1, n, hq, hkv, d, 256, {(kb, 8): 200}, [kb], [8])
    rope = ekv.Rope(d, base=500000.0, scaling="banded", factor=8.0, original_len=8192)
    f, mag = serving.rope_freqs(d, 500000.0, "banded", 8.0, 8192)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    states = [SeqState(hkv, d, 8, None, None, False) for _ in range(n)]
    half = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float16)).cuda()  # noqa: E731

    # the prompt
    T = sum(lens)
    q, k, v = half(T, hq, d), half(T, hkv, d), half(T, hkv, d)
    pos = np.concatenate([np.arange(t) for t in lens]).astype(np.int32)
    cu = [0, *np.cumsum(lens).tolist()]
    qr, kr = rope(q, k, torch.from_numpy(pos).cuda())
    want = serving.rope(q.cpu().numpy(), pos, f, mag, "half")
    assert np.abs(qr.cpu().numpy().astype(np.float64) - want).max() <= 2.0 ** -11 * np.abs(want).max() + 2 ** -16
    o = ekv.prompt_attn(qr, kr, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    for z, (a, b) in enumerate(zip(cu, cu[1:])):
        cache.append(0, slots[z:z + 1], kr[None, a:b], v[None, a:b])
        states[z].append(kr[a:b].cpu().numpy(), v[a:b].cpu().numpy(), kb)
        ref, tol = serving.attention(qr[a:b].cpu().numpy(), kr[a:b].cpu().numpy(),
                                     v[a:b].cpu().numpy(), serving.causal(b - a))
        assert np.all(np.abs(o[a:b].cpu().numpy() - ref) <= tol)

    # drafted steps
    accepted = 0
    for _ in range(steps):
        par = np.full((n, m), -1, np.int32)
        depth = np.zeros((n, m), np.int32)
        for z in range(n):
            for i in range(1, m):
                par[z, i] = rng.integers((i - 1) // 2, i)
                depth[z, i] = depth[z, par[z, i]] + 1
        pos = np.array([[cache.seq_len(0, z) + depth[z, i] for i in range(m)] for z in range(n)])
        q, k, v = half(n, m, hq, d), half(n, m, hkv, d), half(n, m, hkv, d)
        flat = torch.from_numpy(pos.astype(np.int32).reshape(-1)).cuda()
        qr, kr = rope(q.view(n * m, hq, d), k.view(n * m, hkv, d), flat)
        qr, kr = qr.view(n, m, hq, d), kr.view(n, m, hkv, d)
        dpar = torch.from_numpy(par).cuda()
        o = cache.tree_attn(0, slots, qr, kr, v, dpar)
        cache.sync()
        for z in range(n):
            ref, tol = serving.attention(
                qr[z].cpu().numpy(),
                np.concatenate([states[z].khat(), kr[z].cpu().numpy()]),
                np.concatenate([states[z].vhat(), v[z].cpu().numpy()]),
                serving.tree_sees(par[z], m, states[z].T))
            assert np.all(np.abs(o[z].cpu().numpy() - ref) <= tol)
        # a head of random weights on the attention output gives the target's rows
        w = torch.from_numpy(rng.normal(size=(hq * d, V)).astype(np.float32)).cuda()
        x = o.view(n, m, hq * d).float() @ w
        p = torch.softmax(x, -1)
        qd = torch.softmax(x + torch.randn_like(x), -1)
        if draft:
            up = dpar.long().clamp(min=0)
            tok = torch.multinomial(qd.gather(1, up[..., None].expand(n, m, V)).view(-1, V), 1)
            tok = tok.view(n, m).int()
        else:
            tok = p.gather(1, dpar.long().clamp(min=0)[..., None].expand(n, m, V)).argmax(-1).int()
        u = torch.from_numpy(rng.random((n, m)).astype(np.float32)).cuda()
        us = torch.from_numpy(rng.random(n).astype(np.float32)).cuda()
        path, acc, nxt = ekv.verify_tree(p, tok, dpar, u, us, draft_probs=qd if draft else None)
        path, acc, nxt = path.cpu().numpy(), acc.cpu().numpy(), nxt.cpu().numpy()
        for z in range(n):
            want, t = serving.verify(p[z].cpu().numpy(), qd[z].cpu().numpy() if draft else None,
                                     tok[z].cpu().numpy(), par[z], u[z].cpu().numpy(),
                                     us[z].item(), m)
            assert path[z, :acc[z]].tolist() == want and nxt[z] == t
            rows = torch.tensor([0, *want], device="cuda")  # the root and what was accepted
            cache.append(0, slots[z:z + 1], kr[z, rows][None], v[z, rows][None])
            states[z].append(kr[z, rows].cpu().numpy(), v[z, rows].cpu().numpy(), kb)
            accepted += len(want)
    cache.sync()
    assert accepted > 0
    assert [cache.seq_len(0, z) for z in range(n)] == [states[z].T for z in range(n)]
    cache.close()
