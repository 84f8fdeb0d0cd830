"""Pins of the paged KV4 oracle (oracle/kv4_paged.py) by hand-worked tables,
closed forms and the contiguous oracle, and the paged calls' host-side checks,
which need no GPU."""
import ctypes

import numpy as np
import pytest

from oracle import kv4, kv4_paged
from w4a8_quantized_gemm_qoq_b200 import inputs, qoq


def test_assign_by_hand():
    """Pages of 4: request 0 fills its second page and takes one more,
    request 1 has no new tokens, request 2 starts."""
    table = np.array([[8, 3, -1], [5, -1, -1], [-1, -1, -1]], np.int32)
    r = kv4_paged.assign([6, 4, 0], [3, 0, 5], [9, 2, 7, 1, 0], 4, table, 4, 10)
    assert r["q_start"].tolist() == [0, 3, 3, 8] and r["kv_lens"].tolist() == [9, 4, 5]
    assert r["positions"].tolist() == [6, 7, 8, 0, 1, 2, 3, 4, -1, -1]
    assert r["block_table"].tolist() == [[8, 3, 1], [5, -1, -1], [7, 2, -1]] and r["free_left"] == 1
    assert r["slots"].tolist() == [14, 15, 4, 28, 29, 30, 31, 8, -1, -1]
    assert kv4_paged.assign([6, 4, 0], [3, 0, 5], [9, 2, 7, 1, 0], 2, table, 4, 10) is None
    assert kv4_paged.assign([6, 4, 0], [3, 0, 5], [9, 2, 7, 1, 0], 4, table, 4, 7) is None
    assert kv4_paged.assign([6, 4, 0], [7, 0, 5], [9, 2, 7, 1, 0], 5, table, 4, 20) is None


def test_release_by_hand():
    seq, table, free, count = kv4_paged.release([0, 1, 1], [6, 4, 5], np.array([[8, 3], [5, -1], [7, 2]]),
                                                np.array([9, 0, 0, 0]), 1, 4)
    assert seq.tolist() == [6, 0, 0] and table.tolist() == [[8, 3], [-1, -1], [-1, -1]]
    assert free.tolist() == [9, 2, 7, 5] and count == 4


def test_visible_by_hand():
    assert kv4_paged.visible(3, 6).tolist() == [1, 1, 1, 1, 0, 0]
    assert kv4_paged.visible(3, 6, window=2).tolist() == [0, 0, 1, 1, 0, 0]
    assert kv4_paged.visible(4, 6, window=2, sinks=1).tolist() == [1, 0, 0, 1, 1, 0]
    assert kv4_paged.visible(-1, 3, window=2, sinks=1).tolist() == [0, 0, 0]


def test_attention_reduces_to_the_contiguous_oracle():
    """Pages in order, one new token per request: the contiguous decode
    attention of the same tokens; a window is that of the tokens it keeps."""
    q, K, V = inputs.make_decode_attention(2, 32, 4, 2, 64, seed=3)
    Kq, Vq = kv4.quantize_kv4(K), kv4.quantize_kv4(V)

    def pages(d):   # [B][H][32] -> pages of 16
        codes = kv4.pack_kv4(d["q"]).reshape(2, 2, 2, 16, 32).transpose(0, 2, 1, 3, 4).reshape(4, 2, 16, 32)
        sz = np.stack([d["s"], d["z"]], -1).reshape(2, 2, 2, 16, 2).transpose(0, 2, 1, 3, 4).reshape(4, 2, 16, 2)
        return codes, sz

    table = np.array([[0, 1], [2, 3]])
    args = (q, *pages(Kq), *pages(Vq), table, [0, 1, 2], [32, 32])
    want = kv4.decode_attention(q, Kq, Vq)
    assert np.allclose(kv4_paged.attention(*args)[0], want, rtol=0, atol=1e-13)
    keep = np.r_[0:3, 22:32]
    some = [{k: d[k][:, :, keep] for k in d} for d in (Kq, Vq)]
    assert np.allclose(kv4_paged.attention(*args, window=10, sinks=3)[0], kv4.decode_attention(q, *some), rtol=0,
                       atol=1e-13)


def test_write_and_read_of_the_oracle():
    x = np.random.default_rng(0).standard_normal((5, 2, 64)).astype(np.float16)
    codes, params = np.zeros((3, 2, 16, 32), np.uint8), np.zeros((3, 2, 16, 2), np.float16)
    slots = np.array([40, -1, 3, 48, 17])
    codes, params = kv4_paged.write(x, slots, codes, params, 16)
    d = kv4.quantize_kv4(x)
    want = kv4.dequantize_kv4(d["q"], d["s"], d["z"]).astype(np.float64)
    want[[1, 3]] = 0
    assert np.array_equal(kv4_paged.read(slots, codes, params), want)
    assert codes.any(axis=(1, 3)).sum() == 3


# ------------------------------------------------------------ refusals

P16 = 16 * 1024   # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    from w4a8_quantized_gemm_qoq_b200 import build
    build.build()
    return qoq.lib()


def _p(a=P16):
    return ctypes.c_void_p(a)


def _assign(L, B=2, page=16, n_pages=8, max_pages=4, max_tokens=10, **at):
    names = ["seq", "new", "free", "count", "table", "kv", "q_start", "pos", "slots", "left", "status"]
    a = {n: at.get(n, _p()) for n in names}
    return L.qoq_kv4_pages_assign(a["seq"], a["new"], B, page, a["free"], a["count"], n_pages, a["table"], max_pages,
                                  max_tokens, a["kv"], a["q_start"], a["pos"], a["slots"], a["left"], a["status"], None)


def test_pages_calls_refuse(L):
    assert _assign(L, B=-1) == 1 and _assign(L, B=16385) == 2
    assert _assign(L, page=0) == 1 and _assign(L, page=48) == 2 and _assign(L, page=8) == 2 and _assign(L, page=512) == 2
    assert _assign(L, n_pages=0) == 1 and _assign(L, n_pages=2 ** 27) == 2 and _assign(L, max_pages=0) == 1
    assert _assign(L, max_pages=2 ** 27) == 2 and _assign(L, max_tokens=-1) == 1 and _assign(L, max_tokens=2 ** 31) == 2
    for name in ("seq", "new", "free", "count", "table", "kv", "q_start", "pos", "slots", "left", "status"):
        assert _assign(L, **{name: None}) == 1, name
        assert _assign(L, **{name: _p(P16 + 2)}) == 3, name
    r = L.qoq_kv4_pages_release
    assert r(_p(), 2, 16, _p(), _p(), 4, _p(), _p(), 0, _p(), None) == 1
    assert r(_p(), 2, 24, _p(), _p(), 4, _p(), _p(), 8, _p(), None) == 2
    assert r(None, 2, 16, _p(), _p(), 4, _p(), _p(), 8, _p(), None) == 1
    assert r(_p(), 2, 16, _p(), _p(), 4, _p(), _p(), 8, _p(P16 + 1), None) == 3
    assert r(None, 0, 16, None, None, 4, None, None, 8, None, None) == 0


def test_paged_cache_calls_refuse(L):
    w, r = L.qoq_kv4_paged_write, L.qoq_kv4_paged_read

    def write(k=P16, ks=1024, v=P16, vs=1024, slots=P16, N=4, H=8, D=128, n=8, page=16, c=P16, m=P16):
        return w(_p(k), ks, _p(v), vs, _p(slots), N, H, D, n, page, _p(c), _p(m), _p(c), _p(m), None)

    assert write(D=96) == 2 and write(H=0) == 1 and write(H=70000, ks=1 << 24, vs=1 << 24) == 2 and write(N=-1) == 1
    assert write(ks=1016) == 1 and write(vs=0) == 1 and write(page=20) == 2 and write(n=-3) == 1
    assert write(ks=1028) == 3 and write(k=P16 + 8) == 3 and write(c=P16 + 4) == 3 and write(m=P16 + 4) == 3
    assert write(slots=P16 + 1) == 3 and write(k=None) == 1 and write(slots=None) == 1 and write(c=None) == 1
    assert write(N=0, k=None, v=None, slots=None) == 0

    def read(slots=P16, N=4, H=8, D=128, n=8, page=16, c=P16, m=P16, o=P16):
        return r(_p(slots), N, H, D, n, page, _p(c), _p(m), _p(c), _p(m), _p(o), _p(o), None)

    assert read(D=32) == 2 and read(N=-1) == 1 and read(page=0) == 1 and read(o=None) == 1 and read(o=P16 + 8) == 3
    assert read(N=2 ** 31, H=1) == 2 and read(N=0, slots=None) == 0


def test_paged_attention_refuses(L):
    a = L.qoq_kv4_paged_attention

    def call(q=P16, qs=4096, c=P16, m=P16, table=P16, max_pages=4, q_start=P16, kv=P16, B=2, N=4, max_new=3, Hq=32,
             Hkv=8, D=128, n=8, page=16, window=0, sinks=0, out=P16, os=4096, ws=P16, size=1 << 40):
        return a(_p(q), qs, _p(c), _p(m), _p(c), _p(m), _p(table), max_pages, _p(q_start), _p(kv), B, N, max_new, Hq,
                 Hkv, D, n, page, window, sinks, _p(out), os, _p(ws), ctypes.byref(ctypes.c_size_t(size)), None)

    assert call(Hq=30) == 2 and call(Hq=72) == 2 and call(D=96) == 2 and call(Hkv=0) == 1 and call(B=-1) == 1
    assert call(B=20000) == 2 and call(N=-1) == 1 and call(N=2 ** 30) == 2 and call(max_new=0) == 1
    assert call(size=8) == 4 and call(page=100) == 2 and call(n=0) == 1 and call(max_pages=0) == 1
    assert call(window=-1) == 1 and call(sinks=-1) == 1 and call(qs=4088) == 1 and call(os=0) == 1
    for name in ("q", "c", "m", "table", "q_start", "kv", "out"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: P16 + 2}) == 3, name
    assert call(q=P16 + 8) == 3 and call(qs=4100) == 3 and call(os=4100) == 3 and call(ws=P16 + 128) == 3 and call(m=P16 + 4) == 3
    assert call(B=0, q=None) == 0 and call(N=0, q=None) == 0
    assert qoq.kv4_paged_workspace_bytes(64, 64, 32, 8, 128, 1) >= 256


def test_binding_refuses_host_tensors():
    import torch
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        qoq.PageTable.of(z, torch.zeros((4, 2), dtype=torch.int32), z, z[:1], 16)
    with pytest.raises(TypeError):
        qoq.PagedKV4Cache.of(*[torch.zeros((2, 1, 16, 32), dtype=torch.uint8)] * 4)
