"""The paged-cache oracle against dense arithmetic without pages, and the
tables' oracle against what it must keep: every token its own slot, every page
one owner."""
import numpy as np
import pytest

from oracle import paged
from tests.paged_cases import Batch


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (5, 3), (1, 0), (100, 2)])
@pytest.mark.parametrize("lens", [[(1, 1)], [(20, 7), (0, 0), (33, 1)], [(3, 5), (0, 2), (16, 16)]])
def test_attention_is_dense_masked_softmax(lens, window, sinks):
    b = Batch(lens, H_q=4, H_kv=2, D=64, window=window, sinks=sinks, device=None, seed=3)
    out = b.oracle()[0]
    q = b.q.double().numpy()
    for r, (L, n) in enumerate(lens):
        k = np.stack([b.k[int(b.table[r, j // 16]), :, j % 16].double().numpy() for j in range(L)]) if L else np.zeros((0, 2, 64))
        v = np.stack([b.v[int(b.table[r, j // 16]), :, j % 16].double().numpy() for j in range(L)]) if L else np.zeros((0, 2, 64))
        for i in range(n):
            t, p = int(b.cu[r]) + i, L - n + i
            for h in range(4):
                num, den = np.zeros(64), 0.0
                for j in range(L):
                    if j > p or (window and j <= p - window and j >= sinks):
                        continue
                    w = np.exp(b.scale * (q[t, h] @ k[j, h // 2]))
                    num, den = num + w * v[j, h // 2], den + w
                want = num / den if den else num
                np.testing.assert_allclose(out[t, h], want, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("page", [16, 64])
def test_tables_give_every_token_its_own_slot(page):
    r = np.random.default_rng(page)
    B, width = 9, 12
    cached = r.integers(0, 5 * page, B)
    fresh = r.integers(0, 5 * page, B)
    have = [-(-int(c) // page) for c in cached]
    need = [-(-int(c + n) // page) - h for c, n, h in zip(cached, fresh, have)]
    order = r.permutation(sum(have) + sum(need) + 2)
    table = np.full((B, width), -1)
    at = 0
    for b, h in enumerate(have):
        table[b, :h] = order[at:at + h]
        at += h
    rows = int(fresh.sum()) + 4
    t2, cu, kv_len, slots, taken = paged.tables(cached, fresh, order[at:], table, page, len(order), rows)
    assert taken == sum(need) and (kv_len == cached + fresh).all() and cu[-1] == fresh.sum()
    live = slots[:cu[-1]]
    assert (slots[cu[-1]:] == -1).all() and (live >= 0).all() and len(set(live.tolist())) == len(live)
    used = [int(p) for b in range(B) for p in t2[b, :have[b] + need[b]]]
    assert len(set(used)) == len(used)
    for b in range(B):
        for i in range(int(fresh[b])):
            j = int(cached[b]) + i
            assert slots[cu[b] + i] == t2[b, j // page] * page + j % page
