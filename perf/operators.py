"""The paged key/value cache operators: the cases that are measured, their
plain forms and their values in 64 bits.

    tables   cider_paged_tables     block tables, slots and offsets of one
                                    step, from the requests' lengths
    append   cider_paged_append     the step's new keys and values into their
                                    pages
    attend   cider_paged_attention  attention of every request's new tokens
                                    (one, or a chunk of a prompt) over its
                                    pages, causal, with an optional sliding
                                    window and a few first tokens (sinks) that
                                    stay visible

A case is one step of a server: B requests with cached tokens, of which each
brings some new ones.  With `own` false, run() is the plain form; with `own`
true it makes the calls of the package.
"""
import math
import random

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- the cases ------------------------------------------------------------------

def _tables(name, B, chunk, cached, page, width, shape):
    """chunk = 1: every request decodes one token; else up to `chunk` new tokens."""
    return {"name": name, "op": "tables", "B": B, "chunk": chunk, "cached": cached, "page": page, "width": width,
            "shape": shape}


def _append(name, dt, T, H_kv, D, page, shape):
    return {"name": name, "op": "append", "dt": dt, "T": T, "H_kv": H_kv, "D": D, "page": page, "shape": shape}


def _attend(name, dt, B, chunk, kv, H_q, H_kv, D, page, window=0, sinks=0, idle=0, shape=1):
    """kv: the longest request's length with its new tokens; the others have
    between a quarter of it and all of it.  idle: requests without new tokens
    (a batch padded to a fixed size)."""
    return {"name": name, "op": "attend", "dt": dt, "B": B, "chunk": chunk, "kv": kv, "H_q": H_q, "H_kv": H_kv,
            "D": D, "page": page, "window": window, "sinks": sinks, "idle": idle, "shape": shape}


def listed():
    return [
        # the bookkeeping of a decode step of 64 running requests
        _tables("tables_decode_64", 64, 1, 8192, 16, 520, 1),
        # of a large mixed step: 512 requests, chunks of prompts among decodes
        _tables("tables_mixed_512", 512, 256, 16384, 16, 1056, 2),
        # the new tokens of a decode step of 61 requests, 8 KV heads
        _append("append_decode_61", "bf16", 61, 8, 128, 16, 3),
        # a prompt of 16K tokens, 8 KV heads
        _append("append_prompt_16k", "f16", 16000, 8, 128, 64, 4),
        # one user's decode: latency
        _attend("decode_1_1k", "f16", 1, 1, 1000, 32, 8, 128, 16, shape=5),
        # a server's decode step, ragged, padded to 64 requests
        _attend("decode_64_8k", "bf16", 64, 1, 8192, 32, 8, 128, 16, idle=3, shape=6),
        # few requests with long contexts, eight query heads per KV head
        _attend("decode_4_32k", "bf16", 4, 1, 32768, 32, 4, 128, 64, shape=7),
        # one head per KV head, a window over a long context and four sinks
        _attend("decode_16_window", "f16", 16, 1, 20001, 32, 32, 64, 32, window=4096, sinks=4, shape=8),
        # a fresh prompt of 2K tokens
        _attend("chunk_2k_fresh", "bf16", 1, 2048, 2048, 32, 8, 128, 16, shape=9),
        # chunks of four prompts over what is cached of them
        _attend("chunk_500_x4_16k", "f16", 4, 500, 16384, 32, 8, 128, 16, shape=10),
        # a window of 1024 with sinks over a chunk, heads of 64
        _attend("chunk_2k_window", "bf16", 2, 2048, 8000, 32, 4, 64, 128, window=1024, sinks=4, shape=11),
        # the largest chunk over a long context
        _attend("chunk_4k_16k", "bf16", 1, 4096, 16384, 32, 8, 128, 64, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend", "attend", "attend"])
    shape = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        chunk = rng.choice([1, _log(rng, 2, 512)])
        cached = _log(rng, 16, 16384)
        return {k: v for k, v in _tables("", _log(rng, 1, 512 if chunk <= 256 else 256), chunk, cached, page,
                                         (cached + chunk) // page + 2 + rng.randrange(9), shape).items() if k != "name"}
    if op == "append":
        return {k: v for k, v in _append("", rng.choice(["f16", "bf16"]), _log(rng, 1, 16000), rng.choice([1, 2, 4, 8]),
                                         rng.choice([64, 128]), page, shape).items() if k != "name"}
    H_q, H_kv = rng.choice([(32, 32), (32, 8), (32, 4), (8, 1), (6, 3), (64, 2), (16, 16)])
    B = _log(rng, 1, 64)
    kv = _log(rng, 64, 32768)
    chunk = rng.choice([1, 1, rng.randrange(2, 6), _log(rng, 8, 4096)])
    chunk = max(1, min(chunk, kv))
    while B * H_q * chunk * kv > 32 * 4096 * 16384 or B * H_kv * kv > 64 * 8 * 8192:  # no dearer than the largest
        if B > 1:
            B = (B + 1) // 2
        else:
            chunk = (chunk + 1) // 2
    window = rng.choice([0, 0, _log(rng, 16, 8192)])
    return {k: v for k, v in _attend("", rng.choice(["f16", "bf16"]), B, chunk, kv, H_q, H_kv, rng.choice([64, 128]), page,
                                     window, rng.choice([0, 4, rng.randrange(1, 100)]) if window else 0,
                                     rng.randrange(B) if rng.random() < 0.3 else 0, shape).items() if k != "name"}


def _lengths(case):
    """(cached, new) tokens of every request; they belong to the case, not to the seed."""
    r = random.Random(case["shape"])
    cached, new = [], []
    if case["op"] == "tables":
        for _ in range(case["B"]):
            c = r.randrange(case["cached"] + 1)
            n = 1 if case["chunk"] == 1 else r.choice([0, 1, 1, r.randrange(1, case["chunk"] + 1)])
            cached.append(c)
            new.append(n)
        return cached, new
    for b in range(case["B"]):
        n = case["chunk"] if b == 0 or case["chunk"] == 1 else r.randrange((case["chunk"] + 1) // 2, case["chunk"] + 1)
        total = case["kv"] if b == 0 else r.randrange(max(n, case["kv"] // 4), max(n, case["kv"]) + 1)
        if b >= case["B"] - case["idle"]:
            n = 0
        cached.append(total - n)
        new.append(n)
    return cached, new


def _ceil(a, b):
    return -(-a // b)


def _visible(case):
    """(query, key) pairs and distinct keys that the step's attention reaches, summed over the requests."""
    pairs = keys = 0
    w, s = case["window"], case["sinks"]
    for c, n in zip(*_lengths(case)):
        if n == 0:
            continue
        if not w:
            pairs += n * c + n * (n + 1) // 2
            keys += c + n
            continue
        for p in range(c, c + n):
            lo = max(0, p + 1 - w)
            pairs += p + 1 - lo + min(s, lo)
        lo = max(0, c + 1 - w)
        keys += c + n - lo + min(s, lo)
    return pairs, keys


def work(case):
    cached, new = _lengths(case) if case["op"] != "append" else ([], [])
    if case["op"] == "tables":
        pages = sum(_ceil(c + n, case["page"]) - _ceil(c, case["page"]) for c, n in zip(cached, new))
        # lengths in; free pages in, new entries out; slots, offsets and lengths out; one partly filled page's entry
        return {"bytes": 4 * (2 * len(cached) + 2 * pages + sum(new) + 2 * len(cached) + 2 + len(cached)), "flops": 0}
    if case["op"] == "append":
        return {"bytes": case["T"] * (4 + 2 * 2 * case["H_kv"] * case["D"] * 2), "flops": 0}
    pairs, keys = _visible(case)
    H_q, H_kv, D = case["H_q"], case["H_kv"], case["D"]
    pages = sum(_ceil(c + n, case["page"]) for c, n in zip(cached, new))
    return {"bytes": 2 * keys * H_kv * D * 2 + 2 * sum(new) * H_q * D * 2 + 4 * (pages + 2 * len(cached) + 1),
            "flops": 4 * pairs * H_q * D}


# ---- what a server has in hand before the call -------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    st = {"op": case["op"], "page": case["page"]}
    page = case["page"]
    if case["op"] == "tables":
        cached, new = _lengths(case)
        B, width = case["B"], case["width"]
        have = [_ceil(c, page) for c in cached]
        need = sum(_ceil(c + n, page) - h for c, n, h in zip(cached, new, have))
        num_pages = sum(have) + need + 64
        order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
        first = _ints(have).long()
        start = torch.cumsum(first, 0) - first
        j = torch.arange(width, device="cuda")
        held = j[None, :] < first[:, None]
        table = torch.where(held, order[(start[:, None] + j[None, :]).clamp(max=num_pages - 1)], -1).to(torch.int32)
        st.update(table=table, free=order[sum(have):].contiguous(), cached=_ints(cached), new=_ints(new),
                  num_pages=num_pages, rows=max(1, sum(new)) + 3)
        return st
    dt = _DT[case["dt"]]
    H_kv, D = case["H_kv"], case["D"]
    if case["op"] == "append":
        T = case["T"]
        num_pages = _ceil(T, page) + 8
        st["k_cache"] = torch.randn((num_pages, H_kv, page, D), generator=g, device="cuda").to(dt)
        st["v_cache"] = torch.randn((num_pages, H_kv, page, D), generator=g, device="cuda").to(dt)
        # k and v are slices of the fused projection's output rows
        kv = torch.randn((T, 2 * H_kv, D), generator=g, device="cuda").to(dt)
        st["k"], st["v"] = kv[:, :H_kv], kv[:, H_kv:]
        order = torch.randperm(num_pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        slots = order[t // page] * page + t % page
        slots[T - T // 32:] = -1  # the padding of the batch
        st["slots"] = slots.to(torch.int32)
        return st
    cached, new = _lengths(case)
    kv_len = [c + n for c, n in zip(cached, new)]
    have = [_ceil(n, page) for n in kv_len]
    width, num_pages = max(have) + 1, sum(have) + 2
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    first = _ints(have).long()
    start = torch.cumsum(first, 0) - first
    j = torch.arange(width, device="cuda")
    st["table"] = torch.where(j[None, :] < first[:, None], order[(start[:, None] + j[None, :]).clamp(max=num_pages - 1)],
                              -1).to(torch.int32)
    # the last page of a request ends with what an earlier owner left there
    st["k_cache"] = torch.randn((num_pages, H_kv, page, D), generator=g, device="cuda").to(dt)
    st["v_cache"] = torch.randn((num_pages, H_kv, page, D), generator=g, device="cuda").to(dt)
    T = sum(new) + case["idle"]  # rows behind the last request: the batch's padding
    st["q"] = (2.0 * torch.randn((T, case["H_q"], D), generator=g, device="cuda")).to(dt)
    st["out"] = torch.zeros_like(st["q"])
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st.update(cu=_ints(cu), kv_len=_ints(kv_len), max_new=max(new), max_kv=max(kv_len), window=case["window"],
              sinks=case["sinks"])
    if own:
        import w8a8_activation_quantized_b200 as cider
        need = cider.cider_paged_attention_workspace_bytes(T, case["B"], case["H_q"], H_kv, D, st["max_new"])
        st["workspace"] = torch.empty((max(need, 16),), dtype=torch.uint8, device="cuda")
    return st


# ---- one pass -------------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    return {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend}[st["op"]](st)


def _run_own(st):
    import w8a8_activation_quantized_b200 as cider
    if st["op"] == "tables":
        cu, kv_len, slots, taken = cider.cider_paged_tables(st["cached"], st["new"], st["free"], st["table"], st["page"],
                                                            st["num_pages"], st["rows"])
        return {"table": st["table"], "cu": cu, "kv_len": kv_len, "slots": slots, "taken": taken}
    if st["op"] == "append":
        cider.cider_paged_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"])
        return {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    return cider.cider_paged_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["cu"], st["kv_len"],
                                       max_fresh=st["max_new"], window=st["window"], sinks=st["sinks"], out=st["out"],
                                       workspace=st["workspace"])


def _plain_tables(st):
    page, table, free = st["page"], st["table"], st["free"]
    c, n = st["cached"].long(), st["new"].long()
    first = (c + page - 1) // page
    need = (c + n + page - 1) // page - first
    before = torch.cumsum(need, 0) - need
    i = torch.arange(table.shape[1], device=table.device)[None, :] - first[:, None]
    fresh = (i >= 0) & (i < need[:, None])
    table = torch.where(fresh, free[(before[:, None] + i).clamp(0, free.numel() - 1)], table)
    ends = torch.cumsum(n, 0)
    cu = torch.cat([torch.zeros_like(ends[:1]), ends])
    t = torch.arange(st["rows"], device=table.device)
    b = (t[:, None] >= ends[None, :]).sum(1).clamp(max=n.numel() - 1)
    pos = c[b] + t - cu[b]
    slot = table[b, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    slots = torch.where(t < ends[-1], slot, -1)
    return {"table": table, "cu": cu.to(torch.int32), "kv_len": (c + n).to(torch.int32), "slots": slots.to(torch.int32),
            "taken": need.sum().to(torch.int32).reshape(1)}


def _plain_append(st):
    page = st["page"]
    live = st["slots"] >= 0
    s = st["slots"][live].long()
    st["k_cache"][s // page, :, s % page] = st["k"][live]
    st["v_cache"][s // page, :, s % page] = st["v"][live]
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain_attend(st):
    """Every request padded to the longest: gather, product, mask, softmax, product."""
    q, table, cu, kv_len = st["q"], st["table"], st["cu"].long(), st["kv_len"].long()
    T, H_q, D = q.shape
    H_kv = st["k_cache"].shape[1]
    B, n_max, L = table.shape[0], st["max_new"], st["max_kv"]
    pages = table.long().clamp(min=0)
    k = st["k_cache"][pages].float().transpose(1, 2).reshape(B, H_kv, -1, D)[:, :, :L]
    v = st["v_cache"][pages].float().transpose(1, 2).reshape(B, H_kv, -1, D)[:, :, :L]
    n = cu[1:] - cu[:-1]
    i = torch.arange(n_max, device=q.device)
    live = i[None, :] < n[:, None]  # [B, n_max]
    row = (cu[:-1, None] + i[None, :]).clamp(max=T - 1)
    x = q[row].float().reshape(B, n_max, H_kv, H_q // H_kv, D).permute(0, 2, 3, 1, 4).reshape(B, H_kv, -1, D)
    s = torch.matmul(x, k.transpose(2, 3)).reshape(B, H_q, n_max, L)
    s *= 1.0 / math.sqrt(D)
    pos = (kv_len - n)[:, None] + i[None, :]  # [B, n_max]
    key = torch.arange(L, device=q.device)
    seen = key[None, None, :] <= pos[:, :, None]
    if st["window"]:
        seen &= (key[None, None, :] > pos[:, :, None] - st["window"]) | (key < st["sinks"])[None, None, :]
    s.masked_fill_(~seen[:, None], -math.inf)
    s -= s.amax(-1, keepdim=True).clamp(min=-1e30)
    s.exp_()
    s /= s.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(s.reshape(B, H_kv, -1, L), v).reshape(B, H_q, n_max, D).transpose(1, 2)
    out = torch.zeros_like(q)
    out[row[live]] = o[live].to(q.dtype)
    return out


# ---- the values in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    if case["op"] == "append":
        return None  # copies
    st = prepare(case, seed)
    q, page, w, sinks = st["q"].double(), case["page"], case["window"], case["sinks"]
    H_kv, D = case["H_kv"], case["D"]
    group = case["H_q"] // H_kv
    out = torch.zeros_like(q)
    at = 0
    for b, (c, n) in enumerate(zip(*_lengths(case))):
        if n == 0:
            continue
        ids = st["table"][b, :_ceil(c + n, page)].long()
        key = torch.arange(c + n, device="cuda")
        pos = torch.arange(c, c + n, device="cuda")[:, None]
        hidden = key[None, :] > pos
        if w:
            hidden |= (key[None, :] <= pos - w) & (key[None, :] >= sinks)
        for h in range(H_kv):
            kh = st["k_cache"][ids, h].double().reshape(-1, D)[:c + n]
            vh = st["v_cache"][ids, h].double().reshape(-1, D)[:c + n]
            for e in range(h * group, (h + 1) * group):
                s = (q[at:at + n, e] @ kh.T) / math.sqrt(D)
                s[hidden] = -math.inf
                out[at:at + n, e] = torch.softmax(s, -1) @ vh
        at += n
    return out
