"""Appends of several tokens that start inside a block and end inside a later one: the
call that seals the begun block (from its staging rows) also leaves a new block's rows
in the same staging buffer.  Page bytes are bit-exact and the open rows are the last
tokens', whatever the pieces."""
import numpy as np
import pytest
import torch

from mixed_precision_quantized_gb300 import build, ekv
from oracle import pages
from oracle.decoder import SeqState

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pieces", [[15, 3], [1, 16, 17, 15, 2, 30, 1], [5, 60, 7, 100, 9], [31, 33, 2]],
                         ids=lambda p: "-".join(map(str, p)))
def test_pieces(d, pieces):
    build.build()
    n, h, T = 24, 4, sum(pieces)
    rng = np.random.default_rng(T)
    cache = ekv.Cache(1, n, h, h, d, T, {(4, 8): n * h * (T // 16 + 1)}, [4], [8])
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    for _ in range(4):  # every round starts from empty sequences
        k, v = (rng.normal(size=(n, T, h, d)).astype(np.float16) for _ in range(2))
        a = 0
        for p in pieces:
            cache.append(0, slots, torch.from_numpy(k[:, a:a + p]).cuda().contiguous(),
                         torch.from_numpy(v[:, a:a + p]).cuda().contiguous())
            a += p
        q = torch.from_numpy(rng.normal(size=(n, h, d)).astype(np.float16)).cuda()
        o = cache.decode_attn(0, slots, q)
        cache.sync()
        for z in range(n):
            st = SeqState(h, d, 8, None, None, False)
            st.append(k[z], v[z], 4)
            for i in range(h):
                raw = cache.read_pages(0, z, i, 0, (T + 15) // 16).cpu().numpy()
                for j in range((T + 15) // 16):
                    for name, want in st.page_expect(j, i).items():
                        got = pages.extract(raw[j], 4, 8, d, name, rows=want.shape[0])
                        assert np.array_equal(got, want), (z, i, j, name)
            kh, vh = st.khat().astype(np.float64), st.vhat().astype(np.float64)
            for i in range(h):  # the open block's rows are read back through attention
                x = kh[:, i] @ q[z, i].double().cpu().numpy() / np.sqrt(d)
                w = np.exp(x - x.max())
                want = (w / w.sum()) @ vh[:, i]
                err = np.abs(o[z, i].double().cpu().numpy() - want)
                assert np.all(err <= 2e-3 + 1e-2 * np.abs(want))
            cache.reset(z)
        cache.sync()
    cache.close()
