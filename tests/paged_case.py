"""Shared pieces of the paged KV4 tests: ragged batches over shuffled pages,
the CUDA path through the binding, and its comparison with oracle.kv4_paged.

Attention bar: |o - o*| <= 2^-10 max|v| + 2^-24 per (row, query head), o* the
binary64 value and max|v| over the tokens the row sees. A softmax weight times
its value scale is rounded to FP16 once (half a step, relative 2^-11, so at
most 2^-11 max|v| on the weighted mean; the weights are scaled so that none
that matters is subnormal), the output once (2^-11 |o| <= 2^-11 max|v|, or
2^-25 where it is subnormal); FP32 sums add some 2^-20.
"""
import numpy as np

from oracle import kv4_paged
from gpu_helpers import dev, host, torch
from w4a8_quantized_gemm_qoq_b200 import qoq


class Batch:
    """A ragged batch: ctx[b] cached and new[b] new tokens per request, pages
    in random order, two spare pages, N(0, 1) values with two outlier channels in the keys.
    Every slot that no request uses holds NaN parameters (`poison`)."""

    def __init__(self, ctx, new, Hq, Hkv, D, page, seed=0, poison=True, spare_rows=0, gain=1.0):
        rng = np.random.default_rng(seed)
        self.ctx, self.new = np.asarray(ctx), np.asarray(new)
        self.kv = (self.ctx + self.new).astype(np.int32)
        self.Hq, self.Hkv, self.D, self.page = Hq, Hkv, D, page
        B = len(ctx)
        pages = -(-self.kv // page)
        self.n_pages = int(pages.sum()) + 2
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((B, int(pages.max(initial=0)) + 1), -1, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
        self.q_start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.rows = int(self.q_start[-1])
        N = self.rows + spare_rows
        self.q = rng.standard_normal((N, Hq, D)).astype(np.float16)
        cols = rng.choice(D, 2, replace=False)
        shape = (self.n_pages, Hkv, page)
        self.k_codes, self.v_codes = (rng.integers(0, 256, shape + (D // 2,), dtype=np.uint8) for _ in "kv")
        self.k_params, self.v_params = (np.zeros(shape + (2,), np.float16) for _ in "kv")
        if poison:
            self.k_params[:], self.v_params[:] = np.nan, np.nan
        for b in range(B):
            T = int(self.kv[b])
            t = np.arange(T)
            slots = self.table[b, t // page].astype(np.int64) * page + t % page
            k = rng.standard_normal((T, Hkv, D))
            k[:, :, cols] *= 8
            v = rng.standard_normal((T, Hkv, D)) * gain
            self.k_codes, self.k_params = self._put(k, slots, self.k_codes, self.k_params)
            self.v_codes, self.v_params = self._put(v, slots, self.v_codes, self.v_params)

    def _put(self, x, slots, codes, params):
        d = kv4_paged.quantize_kv4(x.astype(np.float16))
        page, at = slots // self.page, slots % self.page
        codes[page, :, at] = kv4_paged.pack_kv4(d["q"])
        params[page, :, at] = np.stack([d["s"], d["z"]], -1)
        return codes, params

    def cache(self):
        return qoq.PagedKV4Cache.of(*(dev(x) for x in (self.k_codes, self.k_params, self.v_codes, self.v_params)))

    def oracle(self, window=0, sinks=0):
        return kv4_paged.attention(self.q, self.k_codes, self.k_params, self.v_codes, self.v_params, self.table,
                                   self.q_start, self.kv, window, sinks)


def workspace(b, max_new=None):
    max_new = max_new or max(1, int(b.new.max(initial=1)))
    return qoq.Workspace(qoq.kv4_paged_workspace_bytes(len(b.ctx), len(b.q), b.Hq, b.Hkv, b.D, max_new))


def run(b, window=0, sinks=0, max_new=None, ws=None):
    """One attention call; rows behind the last request start as 7 and must stay so."""
    max_new = max_new or max(1, int(b.new.max(initial=1)))
    ws = ws or workspace(b, max_new)
    out = torch().full(b.q.shape, 7.0, dtype=torch().float16, device="cuda")
    qoq.kv4_paged_attention(dev(b.q), b.cache(), dev(b.table), dev(b.q_start), dev(b.kv), max_new, window=window,
                            sinks=sinks, ws=ws, out=out)
    torch().cuda.synchronize()
    assert ws.status() == 0, "status %d" % ws.status()
    out = host(out)
    assert (out[b.rows:] == 7.0).all(), "rows behind the last sequence were written"
    return out


def check(b, out, window=0, sinks=0, want=None):
    """The bar above on every row; returns the worst share of it."""
    o, vmax = b.oracle(window, sinks) if want is None else want
    assert np.isfinite(out[:b.rows].astype(np.float64)).all(), "not finite"
    err = np.abs(out[:b.rows].astype(np.float64) - o[:b.rows]).max(axis=2, initial=0.0)
    tol = 2.0 ** -10 * vmax[:b.rows] + 2.0 ** -24
    worst = (err / tol).max(initial=0.0)
    assert worst <= 1.0, "%.3g of the bound at (row, head) %s" % (worst, np.unravel_index((err / tol).argmax(), err.shape))
    return worst
