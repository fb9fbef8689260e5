"""A decoder layer's attention block over several steps of a small server, every
part through the public calls: W8A8 linears for q, k and v and for the output,
tables from the lengths, the write into the pages, paged attention.  Prompts
arrive in chunks, requests decode, finish and give their pages back.  Attention
is checked against 64 bits on the very q, k and v that the linears wrote (which
have their own tests), the output linear on the attention's result."""
import numpy as np
import pytest
import torch

import oracle
import w8a8_activation_quantized_b200 as cider
from tests.paged_cases import E, U
from w8a8_activation_quantized_b200 import synth

pytestmark = pytest.mark.gpu
HIDDEN, H_Q, H_KV, D, PAGE, WIDTH = 512, 8, 2, 64, 16, 12


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cider.cider_device_status()


def _i(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_serving_steps(window, sinks):
    g = torch.Generator(device="cuda").manual_seed(5)
    wqkv = cider.cider_quantize_weight_pc(synth.weights_device((H_Q + 2 * H_KV) * D, HIDDEN, 1, 0.05, "cuda"))
    wo_host = synth.weights(HIDDEN, H_Q * D, seed=2)
    qo, so = oracle.quantize_weight_pc(wo_host)
    wo = (torch.from_numpy(qo).cuda(), torch.from_numpy(so).cuda())
    num_pages = 40
    k, v = (torch.full((num_pages, H_KV, PAGE, D), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    B = 4
    table = torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda")
    free = list(range(num_pages))
    cached = [0] * B
    history = [[], [], [], []]
    # (new tokens of each request, requests that start anew in front of the step)
    steps = [([50, 7, 0, 33], []), ([40, 1, 90, 1], []), ([1, 1, 1, 1], []), ([0, 1, 60, 1], [0]), ([64, 1, 1, 20], [3]),
             ([1, 1, 1, 1], []), ([1, 0, 0, 1], [])]
    for n, (fresh, restart) in enumerate(steps):
        for b in restart:
            used = -(-cached[b] // PAGE)
            free += table[b, :used].tolist()
            table[b] = -1
            cached[b], history[b] = 0, []
        T, pad = sum(fresh), n % 3
        x = torch.randn((T + pad, HIDDEN), generator=g, device="cuda").half()
        qkv = cider.cider_w8a8_linear_pc(x, *wqkv).view(T + pad, H_Q + 2 * H_KV, D)
        cu, kv_len, slots, taken = cider.cider_paged_tables(_i(cached), _i(fresh), _i(free), table, PAGE, num_pages, T + pad)
        cider.cider_paged_append(qkv[:, H_Q:H_Q + H_KV], qkv[:, H_Q + H_KV:], k, v, slots)
        out = torch.zeros((T + pad, H_Q, D), dtype=torch.float16, device="cuda")
        cider.cider_paged_attention(qkv[:, :H_Q], k, v, table, cu, kv_len, max_fresh=max(fresh), window=window, sinks=sinks, out=out)
        y = cider.cider_w8a8_linear_pc(out.view(T + pad, H_Q * D), *wo)
        free = free[int(taken):]
        at = 0
        for b in range(B):
            rows = qkv[at:at + fresh[b]].double()
            history[b] += list(rows)
            cached[b] += fresh[b]
            assert int(kv_len[b]) == cached[b]
            if fresh[b]:
                h = torch.stack(history[b])
                L = len(h)
                pos, j = torch.arange(L - fresh[b], L, device="cuda")[:, None], torch.arange(L, device="cuda")[None, :]
                see = (j <= pos) & ((j > pos - window) | (j < sinks) if window else True)
                kk, vv = (h[:, H_Q + o:H_Q + o + H_KV].repeat_interleave(H_Q // H_KV, 1) for o in (0, H_KV))
                s = torch.einsum("nhd,jhd->nhj", rows[:, :H_Q], kk) * D ** -0.5
                p = torch.softmax(s.masked_fill(~see[:, None], -float("inf")), -1)
                want = torch.einsum("nhj,jhd->nhd", p, vv)
                mag = torch.einsum("nhj,jhd->nhd", p, vv.abs())
                S = (torch.einsum("nhd,jhd->nhj", rows[:, :H_Q].abs(), kk.abs()) * D ** -0.5).amax(-1, keepdim=True)
                # tests/paged_cases.py derives this bound
                w = 2 * D * E * S + 6 * E * S + 4 * E
                tol = (2 * (w + (L / 16 + 8) * (w + E) + 2 * L * E) + U["f16"] + 4 * E) * mag * (1 + U["f16"]) + \
                    U["f16"] * want.abs() + 2.0 ** -25 + L * 2.0 ** -32 * vv.abs().max()
                assert ((out[at:at + fresh[b]].double() - want).abs() <= tol).all()
            at += fresh[b]
        assert (out[T:] == 0).all()
        ref = oracle.as_float(oracle.linear_pc(out.view(T + pad, -1).cpu().numpy(), qo, so), oracle.F16)[:T]
        got = y[:T].float().cpu().numpy()
        assert np.all(np.abs(got - ref) <= 1e-3 * np.abs(ref).max(axis=1, keepdims=True))
    owned = [int(p) for b in range(B) for p in table[b, :-(-cached[b] // PAGE)]]
    assert len(set(owned + free)) == len(owned) + len(free) == num_pages
    cider.cider_device_status()
