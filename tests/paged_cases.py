"""Batches for the paged-cache tests: requests of given lengths over randomly
placed pages.  Everything that no request owns -- the other pages, and the last
page's slots behind a request's end -- holds NaN, so a kernel that lets any of
it into a result fails every test.

The tolerance of the attention kernels' outputs.  With u the largest relative
error of one rounding to the 16-bit format (2^-11 fp16, 2^-8 bf16), e = 2^-24
that of one to fp32, N keys seen and D dims, in the order of the arithmetic:

  score     each of the D products is exact in fp32; their sum in fp32, rounded
            toward zero at worst (2 e each): 2 D e S, S = sum |q||k| scale
  exponent  x = (s - m) scale log2 e: the scale's rounding, the product with m
            and the fma: 3 e |x|, |x| <= 2 S log2 e
  weight    2^x by ex2.approx: 4 e relative (2^-22).  The errors of x count
            times ln 2 in the weight:
            w = 2 D e S + 3 e 2 S + 4 e
  rescales  a running maximum moves at most once per step of 16 keys and
            multiplies the sums by a factor of error w + e: R (w + e),
            R = N / 16 + 8 (the joins of warps and of pieces)
  sums      O and l add N terms in fp32, rounded toward zero at worst: 2 N e each
  P         rounded to 16 bits before the product: u; in fp16, whose weights are
            made as up to 2^7 and more, those below 2^-14 by half of the smallest
            subnormal, 2^-25 / 2^7 against the largest weight: N 2^-32 max |v|
  result    O / l: the weight's, rescales' and sums' errors count twice (in O
            and in l), u of P once, each against A = sum_j p_j |v_j|; the
            division and its product 3 e; then one rounding: u |out|, or half of
            the smallest subnormal (2^-25 in fp16).
  oracle    its own sums in 64 bits: each of N + 2 operations is off by 2^-53 A
            at most (a mean that is zero comes out as 1e-16, say)
"""
import numpy as np
import torch

from oracle import paged

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
E = 2.0 ** -24


class Batch:
    """lens: (total keys, new tokens) per request."""

    def __init__(self, lens, H_q=8, H_kv=2, D=128, page=16, dt="f16", seed=0, window=0, sinks=0, pad=0, token_major=False,
                 fused=False, kind="random", device="cuda", spare=3):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.window, self.sinks, self.page, self.dt, self.D = lens, window, sinks, page, dt, D
        t = DT[dt]
        have = [-(-L // page) for L, _ in lens]
        num_pages = sum(have) + spare
        order = torch.randperm(num_pages, generator=g).to(torch.int32)
        width = max(have + [1]) + 1
        table = torch.full((len(lens), width), -7, dtype=torch.int32)  # unused entries: no valid page
        at = 0
        for b, h in enumerate(have):
            table[b, :h] = order[at:at + h]
            at += h
        shape = (num_pages, page, H_kv, D) if token_major else (num_pages, H_kv, page, D)

        def view(c):
            return c.transpose(1, 2) if token_major else c
        k, v = (torch.full(shape, float("nan"), dtype=t) for _ in range(2))
        self.k, self.v = view(k), view(v)
        for b, (L, _) in enumerate(lens):
            if kind == "count":  # integers: every sum of them is exact in fp32
                kk = torch.randint(-4, 5, (L, H_kv, D), generator=g).to(t)
                vv = torch.randint(-8, 9, (L, H_kv, D), generator=g).to(t)
            else:
                kk = torch.randn((L, H_kv, D), generator=g).to(t)
                vv = torch.randn((L, H_kv, D), generator=g).to(t)
            for j in range(0, L, page):
                n = min(page, L - j)
                p = int(table[b, j // page])
                self.k[p, :, :n] = kk[j:j + n].transpose(0, 1)
                self.v[p, :, :n] = vv[j:j + n].transpose(0, 1)
        cu = [0]
        for _, n in lens:
            cu.append(cu[-1] + n)
        T = cu[-1] + pad
        self.T = T
        row = H_q + 2 * H_kv if fused else H_q
        qq = torch.randn((T, row, D), generator=g) * (2.0 if kind != "peaked" else 8.0)
        self.q = (torch.zeros_like(qq) if kind == "count" else qq).to(t)[:, :H_q]
        self.table, self.cu, self.kv_len = table, torch.tensor(cu, dtype=torch.int32), \
            torch.tensor([L for L, _ in lens], dtype=torch.int32)
        self.max_fresh = max([n for _, n in lens] + [0])
        self.scale = D ** -0.5
        if device is not None:
            self.to(device)

    def to(self, device):
        for n in ("k", "v", "q", "table", "cu", "kv_len"):
            x = getattr(self, n)
            y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=device)
            y.copy_(x)
            setattr(self, n, y)

    def run(self, cider, **kw):
        a = dict(max_fresh=self.max_fresh, window=self.window, sinks=self.sinks)
        a.update(kw)
        return cider.cider_paged_attention(self.q, self.k, self.v, self.table, self.cu, self.kv_len, **a)

    def oracle(self):
        f = [x.double().cpu().numpy() for x in (self.q, self.k, self.v)]
        return paged.attention(*f, self.table.cpu().numpy(), self.cu.cpu().numpy(), self.kv_len.cpu().numpy(), self.window,
                               self.sinks, self.scale)


def check(batch, out, ref=None, roundings_only=False):
    """Asserts `out` within the tolerance above of the float64 result.
    roundings_only: weights that are all equal and sums that are exact, so the
    result is off by the division, its product and the last rounding alone."""
    want, mag, smax, cnt = batch.oracle() if ref is None else ref
    live = ~np.isnan(want).all(axis=(1, 2)) | (cnt > 0)
    got = out.double().cpu().numpy()
    u = U[batch.dt]
    tiny = 2.0 ** -25 if batch.dt == "f16" else 0.0
    n = cnt[:, None, None].astype(np.float64)
    if roundings_only:
        tol = u * np.abs(want) * (1 + 4 * E) + 4 * E * np.abs(want) + tiny
    else:
        S = smax[:, :, None]
        w = 2 * batch.D * E * S + 6 * E * S + 4 * E
        rel = 2 * (w + (n / 16 + 8) * (w + E) + 2 * n * E) + u + 4 * E
        tol = rel * mag * (1 + u) + u * np.abs(want) + tiny
        if batch.dt == "f16":
            tol = tol + n * 2.0 ** -32 * batch.v[batch.v.isfinite()].abs().max().item()
    tol = tol + (n + 2) * 2.0 ** -53 * mag
    err = np.abs(got - want)
    bad = live[:, None, None] & ~(err <= tol) & ~(np.isnan(want) & np.isnan(got)) & ~(want == got)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off; first at {np.argwhere(bad)[0]}: " \
        f"{got[tuple(np.argwhere(bad)[0])]} for {want[tuple(np.argwhere(bad)[0])]}"
    return err
