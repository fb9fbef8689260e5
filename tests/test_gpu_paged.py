"""The paged-cache operators on the GPU against the oracle in 64 bits: tables,
the write into pages, and attention of decode tokens and chunks, with windows
and sinks, at the sizes and masks where they can go wrong.  The batches
(tests/paged_cases.py) hold NaN wherever no request owns a slot; the tolerance
is derived there."""
import numpy as np
import pytest
import torch

import w8a8_activation_quantized_b200 as cider
from oracle import paged
from tests.paged_cases import Batch, check

pytestmark = pytest.mark.gpu
KERNELS = [0, 1, 2]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cider.cider_device_status()
    yield
    cider.cider_device_status()


@pytest.fixture(params=KERNELS)
def kernel(request):
    cider.cider_test_set_paged_kernel(request.param)
    yield request.param
    cider.cider_test_set_paged_kernel(0)


# ---- tables ------------------------------------------------------------------------

def _i(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables_case(B, page, top, seed, rows_extra=3, width_extra=1, free_short=0):
    r = np.random.default_rng(seed)
    cached, fresh = r.integers(0, top + 1, B), r.integers(0, top + 1, B) * (r.random(B) < 0.7)
    have = -(-cached // page)
    need = -(-(cached + fresh) // page) - have
    num_pages = int(have.sum() + need.sum()) + 5
    order = r.permutation(num_pages)
    width = int((have + need).max()) + width_extra
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    free = order[at:len(order) - 5 - free_short]
    return cached, fresh, free, table, num_pages, int(fresh.sum()) + rows_extra


@pytest.mark.parametrize("B,page,top", [(1, 16, 0), (1, 16, 1), (1, 256, 5000), (7, 32, 100), (64, 16, 900), (257, 64, 70),
                                        (1000, 128, 300), (4096, 16, 40)])
def test_tables(B, page, top):
    cached, fresh, free, table, num_pages, rows = _tables_case(B, page, top, B + page)
    want = paged.tables(cached, fresh, free, table, page, num_pages, rows)
    t = _i(table)
    cu, kv_len, slots, taken = cider.cider_paged_tables(_i(cached), _i(fresh), _i(free), t, page, num_pages, rows)
    for got, w in zip((t, cu, kv_len, slots), want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    assert taken.item() == want[4]
    cider.cider_device_status()


@pytest.mark.parametrize("what", ["free pages run out", "rows too few", "table too narrow", "negative", "bad free page",
                                  "bad old page"])
def test_tables_report_what_does_not_fit(what):
    cached, fresh, free, table, num_pages, rows = _tables_case(40, 16, 100, 5)
    if what == "free pages run out":
        free = free[:len(free) // 2]
    elif what == "rows too few":
        rows = rows // 2
    elif what == "table too narrow":
        table = np.ascontiguousarray(table[:, :4])
    elif what == "negative":
        cached[3], fresh[5] = -4, -1
    elif what == "bad free page":
        free[2], free[4] = num_pages, -1
    else:
        b = int(np.argmax((cached % 16 != 0) & (fresh > 0)))
        table[b, cached[b] // 16] = num_pages + 3
    want = paged.tables(cached, fresh, free, table, 16, num_pages, rows)
    t = _i(table)
    cu, kv_len, slots, taken = cider.cider_paged_tables(_i(cached), _i(fresh), _i(free), t, 16, num_pages, rows)
    for got, w in zip((t, cu, kv_len, slots), want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    assert taken.item() == want[4]
    with pytest.raises(cider.CiderError) as e:
        cider.cider_device_status()
    assert e.value.status == 1
    cider.cider_device_status()


def test_tables_strided_and_no_rows():
    cached, fresh, free, table, num_pages, rows = _tables_case(9, 32, 60, 8)
    want = paged.tables(cached, fresh * 0, free, table, 32, num_pages, 0)
    wide = torch.full((9, table.shape[1] + 7), 77, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = _i(table)
    cu, kv_len, slots, taken = cider.cider_paged_tables(_i(cached), _i(fresh * 0), _i(free), wide[:, :table.shape[1]], 32,
                                                        num_pages, 0)
    np.testing.assert_array_equal(wide[:, :table.shape[1]].cpu().numpy(), want[0])
    assert (wide[:, table.shape[1]:] == 77).all() and slots.numel() == 0 and taken.item() == 0


# ---- the write into pages -------------------------------------------------------------

@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,H,D,page,token_major", [(1, 1, 64, 16, False), (61, 8, 128, 16, False), (1000, 3, 64, 256, True),
                                                    (513, 2, 128, 32, True), (5000, 8, 128, 64, False)])
def test_append(T, H, D, page, token_major, dt):
    g = torch.Generator(device="cuda").manual_seed(T)
    num_pages = -(-T // page) + 4
    shape = (num_pages, page, H, D) if token_major else (num_pages, H, page, D)
    k = torch.randn(shape, generator=g, device="cuda").to(dt)
    v = torch.randn(shape, generator=g, device="cuda").to(dt)
    if token_major:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    qkv = torch.randn((T, 2 * H + 3, D), generator=g, device="cuda").to(dt)
    kn, vn = qkv[:, 3:3 + H], qkv[:, 3 + H:]
    slots = torch.randperm(num_pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    slots[::7] = -1
    want = [k.clone(), v.clone()]
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want[0][s // page, :, s % page] = kn[t]
            want[1][s // page, :, s % page] = vn[t]
    cider.cider_paged_append(kn, vn, k, v, slots)
    assert torch.equal(k.contiguous().view(torch.int16), want[0].contiguous().view(torch.int16))
    assert torch.equal(v.contiguous().view(torch.int16), want[1].contiguous().view(torch.int16))
    cider.cider_device_status()


def test_append_skips_and_reports_slots_outside_the_cache():
    k, v = (torch.zeros((2, 2, 16, 64), dtype=torch.float16, device="cuda") for _ in range(2))
    x = torch.ones((4, 2, 64), dtype=torch.float16, device="cuda")
    cider.cider_paged_append(x, x.clone(), k, v, _i([32, -2, 5, 2 ** 31 - 1]))
    with pytest.raises(cider.CiderError) as e:
        cider.cider_device_status()
    assert e.value.status == 1
    assert k.sum().item() == 2 * 64 and (k[0, :, 5] == 1).all() and torch.equal(k, v)


# ---- attention ---------------------------------------------------------------------------

LENS = {
    "one key": [(1, 1)],
    "decode": [(1, 1), (15, 1), (16, 1), (17, 1), (63, 1), (64, 1), (65, 1), (300, 1), (1025, 1)],
    "decode long": [(4097, 1), (3, 1)],
    "few tokens": [(40, 2), (129, 3), (5, 5), (700, 4)],
    "chunks": [(130, 70), (33, 33), (1, 1), (260, 129), (128, 128), (400, 16)],
    "long chunk": [(900, 515)],
    "idle requests": [(0, 0), (50, 0), (20, 3), (0, 0), (64, 64), (70, 0)],
    "more new than keys": [(0, 3), (2, 7), (10, 40), (33, 1)],
}


@pytest.mark.parametrize("window,sinks", [(0, 0), (64, 0), (100, 4), (1, 1), (17, 70), (5000, 3)])
@pytest.mark.parametrize("name", list(LENS))
def test_every_seen_key_counts_once(kernel, name, window, sinks):
    """Zero queries weigh every key the same, and the values are integers, so
    the result is their exact mean: one key too many or too few shows."""
    for dt, D, page, heads in (("f16", 128, 16, (8, 2)), ("bf16", 64, 64, (6, 6)), ("bf16", 128, 256, (12, 1))):
        b = Batch(LENS[name], *heads, D=D, page=page, dt=dt, seed=len(name) + window, window=window, sinks=sinks, pad=2,
                  kind="count")
        check(b, b.run(cider), roundings_only=True)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("H_q,H_kv,D,page", [(8, 8, 128, 16), (8, 2, 64, 32), (16, 1, 128, 64), (6, 3, 128, 128),
                                             (64, 2, 64, 256), (5, 1, 64, 16), (20, 1, 128, 32)])
def test_random(kernel, H_q, H_kv, D, page, dt):
    for name, w, s in (("decode", 0, 0), ("few tokens", 50, 3), ("chunks", 0, 0), ("chunks", 60, 5), ("long chunk", 0, 0)):
        b = Batch(LENS[name], H_q, H_kv, D=D, page=page, dt=dt, seed=H_q + D, window=w, sinks=s)
        check(b, b.run(cider))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens", [[(20000, 1)], [(9000, 3), (40, 1)], [(5000, 300)]])
def test_long_contexts(kernel, lens, dt):
    b = Batch(lens, 8, 2, dt=dt, seed=7)
    check(b, b.run(cider))


@pytest.mark.parametrize("kind", ["peaked"])
def test_peaked_weights(kernel, kind):
    b = Batch([(700, 1), (300, 90)], 8, 2, dt="f16", seed=5, kind=kind)
    check(b, b.run(cider))


def test_strided_queries_outputs_and_token_major_pages(kernel):
    b = Batch(LENS["chunks"], 8, 2, dt="bf16", seed=9, token_major=True, fused=True, pad=5)
    buf = torch.full((b.T, 13, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, 2:10]
    b.run(cider, out=out)
    check(b, out)
    assert (buf[:, :2] == 3).all() and (buf[:, 10:] == 3).all()
    assert (out[int(b.cu[-1]):] == 3).all()  # rows behind the last request


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens", [[(90, 4)], [(200, 60)], [(300, 300)]])
def test_keys_that_a_query_does_not_see_have_no_effect(kernel, lens, bad):
    """K and V of later tokens, and of tokens in front of the window, hold NaN
    or infinities: the rows that must not see them stay right."""
    L, n = lens[0]
    for window, sinks in ((0, 0), (30, 2)):
        b = Batch(lens, 8, 2, dt="f16", seed=L, window=window, sinks=sinks)
        for j in {L - 1, L - n // 2, max(0, L - n - 40)}:
            p, o = int(b.table[0, j // 16]), j % 16
            b.v[p, :, o, ::3] = bad
            b.k[p, 0, o] = bad
        want, mag, smax, cnt = b.oracle()
        out = b.run(cider)
        got = out.double().cpu().numpy()
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        fine = np.isfinite(want)
        assert fine.any() and not fine.all()
        mag, smax = np.where(np.isfinite(mag), mag, 0), np.where(np.isfinite(smax), smax, 0)
        w2 = np.where(fine, want, 0)
        check(b, torch.from_numpy(np.where(fine, got, 0)), (w2, mag, smax, cnt))


def test_infinite_scores(kernel):
    b = Batch([(40, 1), (50, 20)], 4, 2, D=64, dt="bf16", seed=2)
    b.q = b.q.abs()
    p = int(b.table[0, 0])
    b.k[p, :, 3, 0] = float("-inf")  # one key of score -inf: no weight
    want = b.oracle()
    mag, smax = want[1], np.where(np.isfinite(want[2]), want[2], 60.0)
    check(b, b.run(cider), (want[0], mag, smax, want[3]))
    b.k[int(b.table[1, 0]), :, :, 0] = float("-inf")  # a request's first 16 keys
    for j in range(16, 50):
        b.k[int(b.table[1, j // 16]), :, j % 16, 0] = float("-inf")  # and all others: 0 / 0, as the formula's
    out = b.run(cider)
    assert torch.isnan(out[1:]).all() and torch.isfinite(out[:1]).all()


def test_pages_outside_the_cache_are_not_seen_and_reported(kernel):
    b = Batch([(100, 30), (40, 1), (20, 1)], 8, 2, seed=4)
    num_pages = b.k.shape[0]
    b.table[0, 2] = num_pages
    b.table[1, 0] = -1
    b.table[2, :2] = 2 ** 31 - 1  # nothing left: zeros
    out = b.run(cider)
    with pytest.raises(cider.CiderError) as e:
        cider.cider_device_status()
    assert e.value.status == 1
    check(b, out)
    assert (out[31] == 0).all()


@pytest.mark.parametrize("cu,kv", [([0, 3, 2, 9], [40, 40, 40]), ([0, 3, 5, 40], [40, 40, 40]), ([-5, 3, 5, 9], [40, 40, 40]),
                                   ([0, 3, 5, 9], [-3, 40, 10 ** 9])])
def test_lengths_outside_their_range_are_cut_and_reported(kernel, cu, kv):
    b = Batch([(40, 3), (40, 2), (40, 4)], 8, 2, seed=6)
    b.cu, b.kv_len = _i(cu), _i(kv)
    out = torch.full_like(b.q, 7.0)
    b.run(cider, out=out)
    with pytest.raises(cider.CiderError) as e:
        cider.cider_device_status()
    assert e.value.status == 1
    if kv[0] > 0:
        t = _i([min(max(c, 0), 9) for c in cu])
        t = torch.cummax(t, 0).values.to(torch.int32) if cu[2] >= cu[1] else None
        if t is not None:
            b.cu = t
            check(b, out)
    else:
        assert (out[:3] == 0).all()
    cider.cider_device_status()


def test_a_bound_on_new_tokens_that_does_not_hold_costs_no_correctness():
    b = Batch(LENS["chunks"], 8, 2, seed=3)
    for m in (0, 1, 5, 1 << 20):
        check(b, b.run(cider, max_fresh=m))


def test_offsets_past_32_bits(kernel):
    """A cache of more than 2^32 elements, the request's pages at its end."""
    H, D, page = 8, 128, 256
    num_pages = (1 << 32) // (H * D * page) + 40
    cache = torch.zeros((num_pages, H, page, D), dtype=torch.float16, device="cuda")
    small = Batch([(700, 3), (300, 200)], 8, 8, D=D, page=page, seed=1)
    n = small.k.shape[0]
    cache[-n:] = small.k
    small.v = small.k
    want = check(small, small.run(cider))
    small.k = small.v = cache
    small.table = torch.where(small.table >= 0, small.table + (num_pages - n), -1).to(torch.int32)
    out = small.run(cider)
    del cache
    small.k = small.v = small.k[-n:].clone()
    small.table = torch.where(small.table >= 0, small.table - (num_pages - n), -1).to(torch.int32)
    check(small, out)
    assert want is not None
    big = torch.zeros((num_pages, H, page, D), dtype=torch.float16, device="cuda")
    x = torch.randn((5, H, D), device="cuda").half()
    other = torch.zeros((num_pages, H, page, D), dtype=torch.float16, device="cuda")
    slots = _i([num_pages * page - 1 - i for i in range(5)])
    cider.cider_paged_append(x, 2 * x, big, other, slots)
    assert torch.equal(big[-1, :, -5:].flip(1), x.transpose(0, 1)) and torch.equal(other[-1, :, -5:], 2 * big[-1, :, -5:])
    assert big[:-1].any().item() is False


def test_same_bits_every_time(kernel):
    b = Batch([(3000, 1), (2000, 1), (777, 100), (64, 64)], 8, 2, seed=8)
    first = b.run(cider)
    for _ in range(5):
        assert torch.equal(b.run(cider), first)


def test_another_stream_and_two_at_once(kernel):
    bs = [Batch([(3000, 1), (500, 77)], 8, 2, seed=s) for s in (1, 2)]
    want = [b.run(cider) for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    got = [[], []]
    for _ in range(10):
        for i, (b, s) in enumerate(zip(bs, streams)):
            got[i].append(b.run(cider, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_captured_step_replays_with_other_lengths():
    """Tables, write and attention of a decode step in one graph; the lengths
    in device memory move on between replays."""
    H_q, H_kv, D, page, B, width = 8, 2, 128, 16, 5, 12
    g = torch.Generator(device="cuda").manual_seed(3)
    num_pages = B * width
    k, v = (torch.full((num_pages, H_kv, page, D), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    cached, fresh = _i([0] * B), _i([1, 1, 0, 1, 1])
    free = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    qkv = torch.zeros((B, H_q + 2 * H_kv, D), dtype=torch.float16, device="cuda")
    out = torch.zeros((B, H_q, D), dtype=torch.float16, device="cuda")

    def step():
        cu, kv_len, slots, taken = cider.cider_paged_tables(cached, fresh, free, table, page, num_pages, B)
        cider.cider_paged_append(qkv[:, H_q:H_q + H_kv], qkv[:, H_q + H_kv:], k, v, slots)
        cider.cider_paged_attention(qkv[:, :H_q], k, v, table, cu, kv_len, max_fresh=1, window=40, sinks=2, out=out)
        return cu, kv_len, slots, taken

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cu, kv_len, slots, taken = step()
    hist = [[[], []] for _ in range(B)]
    for n in range(60):
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        live = [b for b in range(B) if b != 2 or n >= 7]
        fresh.copy_(_i([int(b in live) for b in range(B)]))
        graph.replay()
        torch.cuda.synchronize()
        for row, b in enumerate(live):
            hist[b][0].append(qkv[row, H_q:H_q + H_kv].double().cpu())
            hist[b][1].append(qkv[row, H_q + H_kv:].double().cpu())
            kk, vv = torch.stack(hist[b][0]), torch.stack(hist[b][1])
            j = torch.arange(len(kk))
            see = (j > len(kk) - 1 - 40) | (j < 2)
            kk, vv = kk[see].repeat_interleave(4, 1), vv[see].repeat_interleave(4, 1)
            p = torch.softmax(torch.einsum("hd,jhd->hj", qkv[row, :H_q].double().cpu(), kk) * D ** -0.5, -1)
            want = torch.einsum("hj,jhd->hd", p, vv)
            # u (A + |out|) with A <= max |v|, u = 2^-11, and fp32 terms far below
            assert (out[row].double().cpu() - want).abs().max() <= 2.0 ** -11 * 2.2 * vv.abs().max()
        free = free  # the captured call keeps its list: the taken pages move to its front's end
        used = int(taken)
        free.copy_(torch.roll(free, -used))
        cached.copy_(kv_len)
    cider.cider_device_status()


def _reference(b):
    """The float64 result on the GPU, request by request, laid out as the
    oracle's (tests/test_gpu_paged.py holds the two together below)."""
    T, H_q, D = b.q.shape
    H_kv, ps = b.k.shape[1], b.page
    G = H_q // H_kv
    out = torch.full((T, H_q, D), float("nan"), dtype=torch.float64, device="cuda")
    mag, smax = torch.zeros_like(out), torch.zeros((T, H_q), dtype=torch.float64, device="cuda")
    cnt = torch.zeros(T, dtype=torch.int64, device="cuda")
    at = 0
    for r, (L, n) in enumerate(b.lens):
        if n == 0:
            continue
        ids = b.table[r, :-(-L // ps)].long()
        k = b.k[ids].transpose(1, 2).reshape(-1, H_kv, D)[:L].double()
        v = b.v[ids].transpose(1, 2).reshape(-1, H_kv, D)[:L].double()
        pos = torch.arange(L - n, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None, :]
        see = j <= pos
        if b.window:
            see &= (j > pos - b.window) | (j < b.sinks)
        for h in range(H_q):
            q = b.q[at:at + n, h].double()
            s = (b.scale * (q @ k[:, h // G].T)).masked_fill(~see, -float("inf"))
            p = torch.softmax(s, -1)
            out[at:at + n, h] = p @ v[:, h // G]
            mag[at:at + n, h] = p @ v[:, h // G].abs()
            smax[at:at + n, h] = (b.scale * (q.abs() @ k[:, h // G].abs().T)).masked_fill(~see, 0).amax(-1)
        cnt[at:at + n] = see.sum(-1)
        at += n
    return [x.cpu().numpy() for x in (out, mag, smax, cnt)]


def test_the_two_references_agree():
    b = Batch([(130, 70), (33, 33), (260, 129)], 4, 2, D=64, page=32, seed=3, window=40, sinks=3)
    for x, y in zip(_reference(b), b.oracle()):
        np.testing.assert_allclose(x, y, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("D,page,dt", [(128, 16, "f16"), (128, 64, "bf16"), (64, 128, "f16"), (64, 16, "bf16")])
@pytest.mark.parametrize("lens,window,sinks", [
    ([(6000, 2500), (5000, 1900)], 0, 0),             # more units than SMs
    ([(7001, 1500), (2000, 2000), (64, 1)], 900, 4),
    ([(30000, 130)], 0, 0),                           # few units, cut into many pieces
    ([(20000, 1), (1500, 700)], 0, 0),                # a long decode among chunks
    ([(12000, 64)] * 9, 3000, 100),
])
def test_large_chunks(lens, window, sinks, D, page, dt):
    b = Batch(lens, 16, 4, D=D, page=page, dt=dt, seed=D + page, window=window, sinks=sinks, pad=1)
    check(b, b.run(cider), _reference(b))


@pytest.mark.parametrize("lens", [[(9000, 1)] * 3, [(3000 + 37 * i, 1) for i in range(70)], [(17, 1)] * 900,
                                  [(i % 40, i % 2) for i in range(4096)]])
@pytest.mark.parametrize("H_q,H_kv,D", [(8, 1, 128), (4, 4, 64)])
def test_large_decode_batches(lens, H_q, H_kv, D):
    b = Batch(lens, H_q, H_kv, D=D, page=32, dt="bf16", seed=len(lens))
    check(b, b.run(cider), _reference(b))


@pytest.mark.parametrize("H_q,H_kv", [(130, 1), (256, 1), (34, 2), (128, 1)])
def test_groups_of_more_heads_than_a_tile(H_q, H_kv):
    b = Batch([(100, 3), (40, 33), (70, 1)], H_q, H_kv, D=64, seed=H_q)
    check(b, b.run(cider))


def test_padded_strides(kernel):
    """Caches that are slices of wider ones, with strides that do not divide one
    another, K and V interleaved page by page."""
    for order in ("head", "token"):
        b = Batch(LENS["chunks"], 6, 3, D=64, page=32, dt="f16", seed=12)
        P, H, S, D = b.k.shape
        if order == "head":
            whole = torch.full((P, 2, H + 2, S + 3, D + 8), float("nan"), dtype=torch.float16, device="cuda")
            k, v = whole[:, 0, :H, :S, :D], whole[:, 1, :H, :S, :D]
        else:
            whole = torch.full((P, 2, S + 3, H + 2, D + 8), float("nan"), dtype=torch.float16, device="cuda")
            k, v = (whole[:, i, :S, :H, :D].transpose(1, 2) for i in (0, 1))
        k.copy_(b.k)
        v.copy_(b.v)
        want = b.oracle()
        b.k, b.v = k, v
        check(b, b.run(cider), want)


def test_captured_chunk_replays_with_other_lengths():
    """A captured call whose lengths, table and queries change in place: chunks,
    decode tokens and idle requests, whole and cut work lists."""
    b = Batch([(3000, 600), (2500, 600)], 8, 2, seed=20, pad=50)
    out = torch.zeros_like(b.q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b.run(cider, out=out, max_fresh=b.T)
    for lens in ([(3000, 600), (2500, 600)], [(3000, 1), (2500, 1)], [(100, 100), (2500, 1100)], [(0, 0), (17, 3)],
                 [(0, 0), (0, 0)], [(2999, 1200), (1, 1)]):
        b.lens = lens
        b.kv_len.copy_(_i([L for L, _ in lens]))
        b.cu.copy_(_i([0, lens[0][1], lens[0][1] + lens[1][1]]))
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        check(b, out, _reference(b))
        assert (out[int(b.cu[-1]):] == 5).all()


def test_two_captured_graphs_at_once():
    """Each with its own workspace, replayed on two streams at the same time."""
    bs = [Batch([(4000, 1)] * 5, 8, 2, seed=31), Batch([(1500, 400)], 8, 2, seed=32)]
    want = [b.run(cider) for b in bs]
    outs, graphs, streams = [torch.empty_like(w) for w in want], [], [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for b, o, s in zip(bs, outs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(5):
                b.run(cider, out=o)
        graphs.append(g)
    for _ in range(10):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("L,n", [(1000, 1000), (9000, 260)])
def test_values_that_are_not_finite_reach_their_own_queries_alone(L, n):
    """A NaN in the last token's V, an infinity in one in the middle of the chunk
    (some of its dims): every query in front of them stays right, every element
    behind them is what the formula says."""
    b = Batch([(L, n)], 4, 2, D=128, page=64, seed=L)
    mid = L - n // 2
    for j, x in ((L - 1, float("nan")), (mid, float("inf"))):
        b.v[int(b.table[0, j // 64]), :, j % 64, 5::9] = x
    out = b.run(cider)
    want, mag, smax, cnt = _reference(b)
    got = out.double().cpu().numpy()
    seen_inf = np.arange(n) >= n - n // 2
    dims = np.zeros(128, dtype=bool)
    dims[5::9] = True
    # softmax in 64 bits gives 0 x inf = NaN where the mask gives weight 0: those are not the formula's
    assert np.isfinite(got[~seen_inf]).all() and np.isfinite(got[:-1][:, :, ~dims]).all()
    assert (got[seen_inf][:-1][:, :, dims] == np.inf).all() and np.isnan(got[-1][:, dims]).all()
    b.v[int(b.table[0, (L - 1) // 64]), :, (L - 1) % 64, 5::9] = 0.0
    b.v[int(b.table[0, mid // 64]), :, mid % 64, 5::9] = 0.0
    clean = b.run(cider).double().cpu().numpy()
    fine = np.isfinite(got)
    # the same scores and weights; only the products' order differs (fp32 sums), then one rounding
    assert np.abs(got - clean)[fine].max() <= 2.0 ** -10 * 2 * np.abs(clean).max() + 2 * L * 2.0 ** -24
    cider.cider_device_status()


def test_refusals_on_the_device():
    b = Batch([(40, 3)], 8, 2, seed=1)
    with pytest.raises(cider.CiderError):
        b.run(cider, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(cider.CiderError):
        b.run(cider, out=b.q)
    with pytest.raises(ValueError):
        b.run(cider, out=torch.empty_like(b.q, device="cpu"))
    out = torch.empty((0, 8, 128), dtype=torch.float16, device="cuda")
    assert cider.cider_paged_attention(out, b.k, b.v, b.table, b.cu, b.kv_len).shape == (0, 8, 128)


@pytest.mark.parametrize("D", [64, 128])
def test_workspace_at_16_bytes_and_what_lies_behind_it(kernel, D):
    """Units of several pieces, whose partial results the tensor-core kernel writes 32 bytes at a time."""
    b = Batch([(3000, 64), (700, 3)], 8, 2, D=D, seed=11)
    n = cider.cider_paged_attention_workspace_bytes(b.T, 2, 8, 2, D, b.max_fresh)
    buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 32 == 0
    for at in (0, 16, 32):
        check(b, b.run(cider, workspace=buf[at:at + n]))
        torch.cuda.synchronize()
        assert (buf[at + n:] == 0xA5).all()
        buf.fill_(0xA5)


def test_offsets_that_decrease_stay_inside_the_workspace(kernel):
    """Every other request claims all rows: 2048 times as many blocks of queries as there are."""
    T, B = 32768, 4096
    b = Batch([(32, 1)] * B, 8, 2, D=64, page=32, seed=12, pad=T - B)
    n = cider.cider_paged_attention_workspace_bytes(T, B, 8, 2, 64, T)
    buf = torch.full((n + (32 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    cu = b.cu
    b.cu = _i([0, T] * (B // 2) + [0])
    out = torch.full((T + 64, 8, 64), 7.0, dtype=torch.float16, device="cuda")
    b.run(cider, max_fresh=T, workspace=buf[:n], out=out[:T])
    with pytest.raises(cider.CiderError) as e:
        cider.cider_device_status()
    assert e.value.status == 1
    assert (buf[n:] == 0xA5).all() and (out[T:] == 7).all()
    b.cu = cu
    check(b, b.run(cider, max_fresh=T, workspace=buf[:n]))
    cider.cider_device_status()


def test_same_bits_with_blocks_beyond_the_planner_s_classes(kernel):
    """More than 255 blocks of 128 keys: units of different lengths share a class of the sorted list."""
    b = Batch([(40000, 70), (39900, 130), (39700, 64), (39500, 1), (20000, 65)], 4, 1, D=64, page=64, seed=13)
    first = b.run(cider)
    check(b, first)
    for _ in range(10):
        assert torch.equal(b.run(cider), first)


@pytest.mark.parametrize("D,H_q,H_kv", [(128, 32, 8), (64, 16, 2)])
@pytest.mark.parametrize("B,n", [(1, 5), (1, 16), (1, 40), (6, 9), (16, 5)])
def test_the_table_s_width_chooses_a_kernel_and_changes_no_result(B, n, D, H_q, H_kv):
    """A wide table is a large bound on the keys: the tensor-core tiles; a tight one may mean the 16-row tiles."""
    b = Batch([(700 + 37 * i, max(1, n - i)) for i in range(B)], H_q, H_kv, D=D, page=32, seed=14 + n)
    check(b, b.run(cider))
    wide = torch.full((B, 4096), -7, dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    check(b, b.run(cider))


@pytest.mark.parametrize("lens", [[(2048, 2048)], [(500, 500), (1200, 1200), (3000, 3000), (200, 200)], [(300, 300), (9000, 64), (70, 70), (5, 5), (0, 0)],
                                  [(60, 100), (6000, 40), (40, 200)]])
@pytest.mark.parametrize("D,H_q,H_kv", [(128, 8, 2), (64, 8, 1), (128, 4, 4)])
def test_units_of_all_lengths_on_one_line(lens, D, H_q, H_kv):
    """Short and long units side by side, cut into equal shares; some that see nothing among them."""
    cider.cider_test_set_paged_kernel(2)
    try:
        b = Batch(lens, H_q, H_kv, D=D, page=16, seed=15)
        check(b, b.run(cider))
    finally:
        cider.cider_test_set_paged_kernel(0)
