"""The paged KV4 operators on the GPU against the CPU oracle
(oracle/kv4_paged.py): page tables and slot maps, the cache's bytes and the
values read back exactly; attention within the bar stated in paged_case.py."""
import numpy as np
import pytest

import oracle
from oracle import kv4, kv4_paged
from gpu_helpers import dev, host, torch
from paged_case import Batch, check, run, workspace
from w4a8_quantized_gemm_qoq_b200 import inputs, qoq

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch().cuda.is_available(), "GPU tests need a CUDA device"
    from w4a8_quantized_gemm_qoq_b200 import build
    build.build()
    yield


# ------------------------------------------------------------ page tables

def _table(ctx, page, spare, max_extra, seed):
    """A PageTable whose requests hold ctx[b] tokens, pages in random order."""
    rng = np.random.default_rng(seed)
    held = [-(-int(s) // page) for s in ctx]
    n_pages = sum(held) + spare
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(ctx), max(held, default=0) + max_extra), -1, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    free = np.full(n_pages, -5, np.int32)
    free[:spare] = order[at:]
    state = dict(seq_lens=np.asarray(ctx, np.int32), block_table=table, free_pages=free, free_count=spare)
    pt = qoq.PageTable.of(dev(state["seq_lens"]), dev(table), dev(free), dev(np.array([spare], np.int32)), page)
    return pt, state


def _state(pt):
    return dict(seq_lens=host(pt.seq_lens), block_table=host(pt.block_table), free_pages=host(pt.free_pages),
                free_count=int(host(pt.free_count)[0]))


def _same(a, b):
    return all(np.array_equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("B,page,top,max_ctx", [(1, 16, 1, 0), (1, 64, 200, 31), (3, 32, 40, 64), (64, 64, 1, 1100),
                                                (65, 16, 9, 300), (513, 16, 5, 50), (1500, 32, 3, 70), (130, 256, 700, 900)])
def test_assign_and_release(B, page, top, max_ctx):
    """Two steps in place, then some requests leave and the rest step again:
    every buffer equals the oracle's. Lengths of zero and full last pages
    are among them."""
    rng = np.random.default_rng(B + page)
    ctx = rng.integers(0, max_ctx + 1, B)
    ctx[B // 2] = max_ctx // page * page
    pt, st = _table(ctx, page, spare=4 * B * (1 + top // page) + 8, max_extra=4 * (1 + top // page) + 1, seed=B)
    for k in range(3):
        n = rng.integers(0 if B > 1 else 1, top + 1, B).astype(np.int32)
        rows = int(n.sum()) + (5 if k else 0)
        step = qoq.PagedStep(B, rows)
        want = kv4_paged.assign(st["seq_lens"], n, st["free_pages"], st["free_count"], st["block_table"], page, rows)
        if k == 0:   # into buffers of its own first: the state but for the entries taken stays
            kv, left = dev(np.zeros(B, np.int32)), dev(np.zeros(1, np.int32))
            pt.assign(dev(n), step, kv_lens=kv, free_left=left)
            assert np.array_equal(host(kv), want["kv_lens"]) and int(host(left)[0]) == want["free_left"]
            assert _same(dict(st, block_table=want["block_table"]), _state(pt))
        pt.assign(dev(n), step)
        for name in ("q_start", "positions", "slots"):
            assert np.array_equal(host(getattr(step, name)), want[name]), name
        st = dict(seq_lens=want["kv_lens"], block_table=want["block_table"], free_pages=st["free_pages"],
                  free_count=want["free_left"])
        assert _same(st, _state(pt))
        if k == 1:
            leave = (rng.random(B) < 0.4).astype(np.int32) * 7
            for _ in range(2):   # leaving twice gives the pages back once
                pt.release(dev(leave))
                r = kv4_paged.release(leave, st["seq_lens"], st["block_table"], st["free_pages"], st["free_count"], page)
                st = dict(zip(("seq_lens", "block_table", "free_pages", "free_count"), r))
                assert _same(st, _state(pt))
    assert pt.status() == 0


def test_release_restores_the_stack():
    """What one step takes, a release gives back in place: the same stack."""
    pt, st = _table([0] * 40, 16, 300, 9, 1)
    step = qoq.PagedStep(40, 4000)
    n = np.arange(40, dtype=np.int32) * 3
    for _ in range(3):
        pt.assign(dev(n), step)
        pt.release(dev(np.ones(40, np.int32)))
    assert _same(st, _state(pt)) and pt.status() == 0


@pytest.mark.parametrize("why,code", [("negative", 1), ("bad_tail_page", 1), ("bad_free_page", 1), ("bad_count", 1),
                                      ("rows", 4), ("pages", 4), ("too_long", 4), ("huge", 4)])
def test_assign_refuses_a_step_that_does_not_fit(why, code):
    """The whole step is refused: state as it was, an empty step, the status
    word set; it stays set over a good step, which works."""
    pt, st = _table([5, 16, 0, 40], 16, 6, 2, 3)
    n, rows = np.array([3, 20, 1, 0], np.int32), 24
    good, good_rows = n.copy(), rows
    if why == "negative":
        n[2] = -1
    elif why == "bad_tail_page":
        pt.block_table[0, 0] = 99
    elif why == "bad_free_page":
        pt.free_pages[4] = -7
    elif why == "bad_count":
        pt.free_count[0] = 1000
    elif why == "rows":
        rows = 23
    elif why == "pages":
        pt.free_count[0] = 2
    elif why == "too_long":
        n[3] = 100
        rows = 200
    elif why == "huge":
        n[:] = 2 ** 31 - 1
    before = _state(pt)
    step = qoq.PagedStep(4, rows)
    kv = dev(np.zeros(4, np.int32))
    pt.assign(dev(n), step, kv_lens=kv)
    assert pt.status() == code
    assert _same(before, _state(pt)) and np.array_equal(host(kv), before["seq_lens"])
    assert not host(step.q_start).any() and (host(step.slots) == -1).all() and (host(step.positions) == -1).all()
    pt.block_table.copy_(dev(st["block_table"]))
    pt.free_pages.copy_(dev(st["free_pages"]))
    pt.free_count.fill_(6)
    step = qoq.PagedStep(4, good_rows)
    pt.assign(dev(good), step)
    want = kv4_paged.assign(st["seq_lens"], good, st["free_pages"], 6, st["block_table"], 16, good_rows)
    assert np.array_equal(host(step.slots), want["slots"]) and pt.status() == code


@pytest.mark.parametrize("why,code", [("bad_page", 1), ("negative", 1), ("too_long", 1), ("full", 4)])
def test_release_refuses(why, code):
    pt, _ = _table([5, 16, 0, 40], 16, 6, 2, 3)
    if why == "bad_page":
        pt.block_table[3, 1] = -1
    elif why == "negative":
        pt.seq_lens[1] = -3
    elif why == "too_long":
        pt.seq_lens[1] = 16 * 6
    elif why == "full":
        pt.free_count[0] = 9
    before = _state(pt)
    pt.release(dev(np.ones(4, np.int32)))
    assert pt.status() == code and _same(before, _state(pt))


def test_assign_of_no_requests():
    pt = qoq.PageTable(0, 4, 8, 16)
    step = qoq.PagedStep(0, 5)
    step.slots.fill_(3)
    pt.assign(torch().zeros(0, dtype=torch().int32, device="cuda"), step)
    assert host(step.q_start).tolist() == [0] and (host(step.slots) == -1).all() and pt.status() == 0


def test_assign_in_a_graph_fills_a_sequence():
    """One captured decode step, replayed: the lengths grow in place across
    page borders until the pages run out; then it is refused and stays put."""
    t = torch()
    pt, st = _table([0, 7, 15], 16, 4, 3, 8)
    n, step = dev(np.ones(3, np.int32)), qoq.PagedStep(3, 4)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        pt.assign(n, step)
    for k in range(40):
        want = kv4_paged.assign(st["seq_lens"], [1] * 3, st["free_pages"], st["free_count"], st["block_table"], 16, 4)
        g.replay()
        if want is None:
            assert pt.status() == 4 and _same(st, _state(pt)) and (host(step.slots) == -1).all()
            break
        st = dict(seq_lens=want["kv_lens"], block_table=want["block_table"], free_pages=st["free_pages"],
                  free_count=want["free_left"])
        assert _same(st, _state(pt)) and np.array_equal(host(step.slots), want["slots"])
    assert want is None and k > 16


# ------------------------------------------------------------ cache

@pytest.mark.parametrize("N,Hkv,D,page", [(1, 1, 64, 16), (3, 8, 128, 64), (37, 4, 128, 256), (130, 5, 64, 32),
                                          (1000, 2, 128, 128)])
def test_write_and_read_are_exact(N, Hkv, D, page):
    """Codes, scales and zeros bit for bit, from strided rows, with skipped
    rows and degenerate vectors; other slots untouched; values read back
    rounded once."""
    rng = np.random.default_rng(N + D)
    n_pages = -(-N // page) + 2
    qkv = rng.standard_normal((N, 3 * Hkv + 2, D)).astype(np.float16)
    if N >= 37:
        edge = qkv[:, Hkv:2 * Hkv]
        edge[0, 0], edge[1, 0], edge[2, 0] = 0, 1.875, -1.875
        edge[3, 0], edge[3, 0, 5] = 0, -3
        edge[4, 0], edge[5, 0, ::2], edge[6, 0] = 65504, -65504, np.float16(6e-8)
        edge[7, 0] = np.linspace(-1e-5, 3e-6, D).astype(np.float16)
        edge[8, 0] = np.linspace(-65504, 65504, D).astype(np.float16)
    slots = rng.permutation(n_pages * page)[:N].astype(np.int32)
    slots[::7] = [-1, -2 ** 31, n_pages * page, 2 ** 31 - 1][N % 4]
    c = qoq.PagedKV4Cache(n_pages, Hkv, page, D)
    for x in (c.k_codes, c.v_codes):
        x.fill_(0xA5)
    for x in (c.k_params, c.v_params):
        x.fill_(3.0)
    before = [host(x).copy() for x in (c.k_codes, c.k_params, c.v_codes, c.v_params)]
    d = dev(qkv)
    c.write(d[:, Hkv:2 * Hkv], d[:, 2 * Hkv + 2:], dev(slots))
    k, v = c.read(dev(slots))
    for x, src, i in ((k, qkv[:, Hkv:2 * Hkv], 0), (v, qkv[:, 2 * Hkv + 2:], 2)):
        codes, params = kv4_paged.write(src, slots, before[i], before[i + 1], page)
        got = host((c.k_codes, c.k_params, c.v_codes, c.v_params)[i]), host((c.k_codes, c.k_params, c.v_codes, c.v_params)[i + 1])
        assert np.array_equal(got[0], codes), "codes"
        assert np.array_equal(got[1].view(np.uint16), params.view(np.uint16)), "params"
        want = kv4_paged.read(slots, codes, params).astype(np.float16)
        assert np.array_equal(host(x).view(np.uint16) & 0x7FFF | (host(x) < 0) * 0x8000,
                              want.view(np.uint16) & 0x7FFF | (want < 0) * 0x8000), "read"


@pytest.mark.parametrize("D", [64, 128])
def test_written_bytes_of_not_finite_values(D):
    """Infinities and NaN among the values: the contiguous cache's bytes."""
    x = np.random.default_rng(D).standard_normal((16, 1, D)).astype(np.float16)
    x[0, 0, 3], x[1, 0, 7], x[2, 0, 60], x[3, 0, :] = np.inf, -np.inf, np.nan, np.nan
    x[4, 0, 1], x[4, 0, 2], x[5, 0, 5], x[5, 0, 6] = np.inf, -np.inf, np.nan, np.inf
    a = qoq.KV4Cache(1, 1, 16, D).write(dev(x.reshape(1, 1, 16, D)))
    c = qoq.PagedKV4Cache(1, 1, 16, D)
    c.write(dev(x), dev(x), dev(np.arange(16, dtype=np.int32)))
    for got in (c.k_codes, c.v_codes):
        assert np.array_equal(host(got).reshape(16, D // 2), host(a.codes).reshape(16, D // 2))
    for got in (c.k_params, c.v_params):
        s, z = host(got).reshape(16, 2)[:, 0], host(got).reshape(16, 2)[:, 1]
        assert np.array_equal(np.isnan(s), np.isnan(host(a.scales).reshape(16)))
        assert np.array_equal(np.nan_to_num(s), np.nan_to_num(host(a.scales).reshape(16)))
        assert np.array_equal(z.view(np.uint16), host(a.zeros).reshape(16).view(np.uint16))


def test_paged_and_contiguous_caches_hold_the_same_bytes():
    _, K, _ = inputs.make_decode_attention(2, 48, 8, 4, 128, seed=5)
    a = qoq.KV4Cache(2, 4, 48, 128).write(dev(K))
    c = qoq.PagedKV4Cache(6, 4, 16, 128)
    rows = dev(np.ascontiguousarray(K.transpose(0, 2, 1, 3).reshape(96, 4, 128)))
    c.write(rows, rows, dev(np.arange(96, dtype=np.int32)))
    codes = host(c.k_codes).reshape(2, 3, 4, 16, 64).transpose(0, 2, 1, 3, 4).reshape(2, 4, 48, 64)
    params = host(c.v_params).reshape(2, 3, 4, 16, 2).transpose(0, 2, 1, 3, 4).reshape(2, 4, 48, 2)
    assert np.array_equal(codes, host(a.codes)) and np.array_equal(host(c.k_codes), host(c.v_codes))
    assert np.array_equal(params[..., 0], host(a.scales)) and np.array_equal(params[..., 1], host(a.zeros))


# ------------------------------------------------------------ attention

HEADS = [(32, 8, 128), (16, 2, 64), (3, 3, 128), (7, 1, 64), (10, 2, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_decode(Hq, Hkv, D, page):
    """One token per request, lengths around tile and page borders."""
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700, 1025]
    b = Batch([n - 1 for n in kv], [1] * len(kv), Hq, Hkv, D, page, seed=page + D)
    check(b, run(b))


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [16, 32, 128, 256])
def test_chunks(Hq, Hkv, D, page):
    """Ragged new tokens over ragged contexts, requests without rows or
    tokens among them; rows behind the last stay."""
    b = Batch([0, 0, 5, 0, 131, 64, 300, 1, 0, 17], [1, 0, 3, 130, 65, 257, 2, 64, 0, 400], Hq, Hkv, D, page,
              seed=page + D, spare_rows=3)
    check(b, run(b))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (64, 0), (100, 64), (129, 70), (333, 1), (100000, 4),
                                          (5, 100000)])
@pytest.mark.parametrize("page", [16, 64])
def test_window_with_sinks(window, sinks, page):
    """Windows shorter and longer than tiles, sinks that end inside a tile,
    reach into the window or beyond the sequence."""
    b = Batch([0, 700, 60, 1030, 500, 3], [300, 1, 70, 5, 129, 1], 8, 2, 128, page, seed=window + sinks)
    check(b, run(b, window, sinks), window, sinks)


def test_masked_values_do_not_matter():
    """Infinite scales at tokens that a window hides from some rows and shows
    to none: the outputs are those of clean pages."""
    b = Batch([400, 900], [40, 1], 8, 2, 128, 64, seed=9)
    want = b.oracle(50, 2)
    for r in range(2):
        for t in range(2, int(b.ctx[r]) - 49):
            b.k_params[b.table[r, t // 64], :, t % 64] = np.inf
            b.v_params[b.table[r, t // 64], :, t % 64] = np.nan
    check(b, run(b, 50, 2), want=want)


def test_partly_masked_values_stay_in_their_rows():
    """A token with an infinite value scale reaches the rows that see it and
    no others (rows before it, and rows whose window has passed it)."""
    b = Batch([0], [300], 4, 1, 128, 32, seed=10)
    want = b.oracle(60, 1)
    b.v_params[b.table[0, 150 // 32], :, 150 % 32, 0] = np.inf
    b.k_params[b.table[0, 220 // 32], :, 220 % 32, 0] = np.inf
    out = run(b, 60, 1)
    clean = [i for i in range(300) if not (150 <= i < 210 or 220 <= i < 280)]
    err = np.abs(out[clean].astype(np.float64) - want[0][clean]).max(axis=2)
    assert (err <= 2.0 ** -10 * want[1][clean] + 2.0 ** -24).all()


@pytest.mark.parametrize("gain", [2.0 ** -13, 30.0, 2.0 ** 13])
def test_value_scales_far_from_one(gain):
    b = Batch([100, 0, 800], [1, 200, 3], 8, 2, 128, 64, seed=11, gain=gain)
    check(b, run(b))


def test_value_scales_that_grow_along_the_sequence():
    """Values from 1e-5 at the start of the sequence to 1e3 at its end and back."""
    b = Batch([900, 1200], [1, 300], 8, 2, 128, 64, seed=12)
    for r in range(2):
        t = np.arange(int(b.kv[r]))
        f = 10.0 ** (3 - 8 * np.abs(2 * t / len(t) - 1)) if r else 10.0 ** (-5 + 8 * t / len(t))
        at = b.table[r, t // 64], slice(None), t % 64, 0
        b.v_params[at] = (b.v_params[at].astype(np.float64) * f[:, None]).astype(np.float16)
    check(b, run(b))


def test_scores_far_apart():
    """Keys so large that most weights vanish and the maximum rises often."""
    b = Batch([500, 0], [1, 400], 8, 2, 128, 64, seed=13)
    for r in range(2):
        t = np.arange(int(b.kv[r]))
        at = b.table[r, t // 64], slice(None), t % 64, 0
        b.k_params[at] = (b.k_params[at].astype(np.float64) * (1 + t[:, None] / 40)).astype(np.float16)
    check(b, run(b))


def test_zero_vectors():
    """Cached zeros (scale 0): uniform weights over the keys, zero outputs of
    the values; and a zero query."""
    b = Batch([70, 0], [1, 90], 4, 2, 64, 32, seed=14)
    b.q[3] = 0
    for r in range(2):
        t = np.arange(0, int(b.kv[r]), 3)
        b.k_params[b.table[r, t // 32], 0, t % 32] = 0
        b.v_params[b.table[r, t // 32], 1, t % 32] = 0
    check(b, run(b))


def test_fewer_tokens_than_rows():
    """kv_lens below the new rows: the first rows stand before the sequence,
    see nothing and give zeros."""
    b = Batch([0, 0, 9], [6, 200, 2], 8, 2, 128, 16, seed=15)
    b.kv = np.array([2, 130, 11], np.int32)
    out = run(b)
    check(b, out)
    assert (out[:4] == 0).all() and (out[6:76] == 0).all()


@pytest.mark.parametrize("new", [1, 70])
def test_lengths_are_clamped_to_the_buffers(new):
    """Negative lengths count as 0, lengths beyond the table as its capacity;
    row ranges that run backwards as empty, beyond q as its rows."""
    b = Batch([200 - new, 256 - new, 100], [new] * 3, 8, 2, 128, 16, seed=24)
    b.table[b.table < 0] = 0   # every entry of the table names some page
    table = b.table[:, :16].copy()
    lens = np.array([-5, 2 ** 31 - 1, 100 + new], np.int32)
    starts = np.array([0, new, 2 * new, 2 ** 31 - 1], np.int32)
    ws = workspace(b)
    out = host(qoq.kv4_paged_attention(dev(b.q), b.cache(), dev(table), dev(starts), dev(lens), new, ws=ws))
    assert ws.status() == 0 and (out[:new] == 0).all()
    b.table, b.kv = table, np.array([0, 256, 100 + new], np.int32)
    check(b, out)
    out = torch().full(b.q.shape, 7.0, dtype=torch().float16, device="cuda")
    back = np.array([2 * new, new, 0, -3], np.int32)
    qoq.kv4_paged_attention(dev(b.q), b.cache(), dev(table), dev(back), dev(lens), new, ws=ws, out=out)
    assert ws.status() == 0 and (host(out) == 7.0).all()


@pytest.mark.parametrize("max_new", [1, 4])
def test_more_rows_than_promised(max_new):
    """A request with more rows than max_new is refused: its rows stay, the
    status names it, the others are computed."""
    b = Batch([50, 60, 70], [1, 5, 1], 8, 2, 128, 64, seed=16)
    out = torch().full(b.q.shape, 7.0, dtype=torch().float16, device="cuda")
    ws = workspace(b, max_new)
    qoq.kv4_paged_attention(dev(b.q), b.cache(), dev(b.table), dev(b.q_start), dev(b.kv), max_new, ws=ws, out=out)
    out = host(out)
    assert ws.status() == 1 and ws.timeout_site()[0] == 1
    assert (out[1:6] == 7.0).all()
    o, vmax = b.oracle()
    for i in (0, 6):
        assert (np.abs(out[i] - o[i]).max(axis=1) <= 2.0 ** -10 * vmax[i] + 2.0 ** -24).all()


@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_bad_page(new, bad):
    """A page number outside the cache: the status names the request, its
    tokens there count as zero keys and values, the others are computed."""
    b = Batch([200, 300], [new, 1], 8, 2, 128, 64, seed=17)
    table, good = b.table.copy(), int(b.table[0, 1])
    table[0, 1] = bad
    ws = workspace(b)
    out = host(qoq.kv4_paged_attention(dev(b.q), b.cache(), dev(table), dev(b.q_start), dev(b.kv), new, ws=ws))
    assert ws.status() == 1 and ws.timeout_site()[0] == 0
    b.k_params[good] = 0
    b.v_params[good] = 0
    check(b, out)


@pytest.mark.parametrize("ctx,new,window", [([300, 40, 1000], [1, 1, 1], 0), ([0, 300, 77], [200, 1, 64], 0),
                                            ([2000], [3], 0), ([5000], [40], 0), ([900], [300], 200)])
def test_graph_replays_and_a_second_stream(ctx, new, window):
    """Captured calls replayed, and calls on two streams at once with
    workspaces of their own, give the eager call's bits."""
    t = torch()
    b = Batch(ctx, new, 32, 8, 128, 64, seed=18)
    want = run(b, window, 4).view(np.uint16)
    args = dev(b.q), b.cache(), dev(b.table), dev(b.q_start), dev(b.kv), max(new)
    ws = [workspace(b) for _ in range(3)]
    outs = [t.empty(b.q.shape, dtype=t.float16, device="cuda") for _ in range(3)]
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        qoq.kv4_paged_attention(*args, window=window, sinks=4, ws=ws[0], out=outs[0])
        qoq.kv4_paged_attention(*args, window=window, sinks=4, ws=ws[0], out=outs[0])
    streams = [t.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        g.replay()
        for i, s in enumerate(streams):
            qoq.kv4_paged_attention(*args, window=window, sinks=4, ws=ws[i + 1], out=outs[i + 1], stream=s)
    t.cuda.synchronize()
    for w, o in zip(ws, outs):
        assert np.array_equal(host(o).view(np.uint16), want) and w.status() == 0


def test_one_graph_for_growing_sequences():
    """A captured step over device-side lengths: the same graph serves batches
    whose rows and lengths change between replays."""
    t = torch()
    a = Batch([10, 0, 300], [20, 100, 1], 8, 2, 128, 64, seed=19, spare_rows=300)
    bufs = [dev(x) for x in (a.q, a.k_codes, a.k_params, a.v_codes, a.v_params)]
    cache = qoq.PagedKV4Cache.of(*bufs[1:])
    table, q_start, kv = (dev(x) for x in (a.table, a.q_start, a.kv))
    ws = workspace(a, 130)
    out = t.empty(a.q.shape, dtype=t.float16, device="cuda")
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        qoq.kv4_paged_attention(bufs[0], cache, table, q_start, kv, 130, ws=ws, out=out)
    for lens, new in (([30, 100, 301], [20, 100, 1]), ([30, 90, 301], [3, 0, 130]), ([0, 1, 200], [0, 1, 2])):
        a.kv, a.new = np.array(lens, np.int32), np.array(new)
        a.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        a.rows = int(a.q_start[-1])
        kv.copy_(dev(a.kv))
        q_start.copy_(dev(a.q_start))
        out.fill_(7.0)
        g.replay()
        o = host(out)
        assert (o[a.rows:] == 7.0).all() and ws.status() == 0
        check(a, o)


@pytest.mark.parametrize("G,Hkv,D", [(1, 2, 128), (3, 1, 64), (8, 2, 64), (7, 1, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 70)])
def test_rows_around_the_kernels_limits(G, Hkv, D, window, sinks):
    """Row counts at which a KV head's (row, head) pairs pass a multiple of 8, or 48."""
    new = sorted({max(1, n // G + d) for n in (8, 16, 24, 40, 48) for d in (0, 1)})
    b = Batch([(0, 61, 500, 3, 260, 1000)[i % 6] for i in range(len(new))], new, G * Hkv, Hkv, D, 16, seed=G)
    check(b, run(b, window, sinks), window, sinks)


@pytest.mark.parametrize("B,Hkv,D,top", [(129, 1, 64, 70), (140, 8, 64, 40), (300, 2, 128, 0), (592, 1, 64, 0),
                                         (593, 1, 64, 0), (1100, 1, 64, 50), (2100, 1, 64, 20)])
@pytest.mark.parametrize("chunks", [False, True])
def test_large_batches(B, Hkv, D, top, chunks):
    """Batches whose division is worked out by a kernel of its own, of equal
    (top 0) and ragged lengths, with and without requests of many rows."""
    rng = np.random.default_rng(B)
    ctx = rng.integers(0, top, B) if top else np.full(B, 33)
    new = np.ones(B, int)
    if chunks:
        new[::B // 7] = rng.integers(9, 50, len(new[::B // 7]))
        new[5::97] = 0
    b = Batch(ctx, new, 4 * Hkv, Hkv, D, 16, seed=B, spare_rows=2)
    check(b, run(b))


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page", [
    ([40000], [1], 1, 1, 64, 256), ([200000], [1], 2, 1, 64, 256), ([9000], [5], 8, 2, 128, 16),
    ([1] * 40 + [30000], [1] * 41, 4, 2, 64, 64), ([20000, 0, 0, 3, 5000], [1, 1, 0, 2, 1], 4, 1, 128, 32),
    ([30000, 10], [40, 90], 4, 1, 64, 128)])
def test_long_sequences_among_short_ones(ctx, new, Hq, Hkv, D, page):
    """Sequences that many CTAs share, alone and beside short ones."""
    b = Batch(ctx, new, Hq, Hkv, D, page, seed=len(ctx))
    check(b, run(b))


@pytest.mark.parametrize("seed", range(16))
def test_random_batches(seed):
    rng = np.random.default_rng(100 + seed)
    B, Hkv, D = int(rng.integers(1, 40)), int(rng.choice([1, 2, 3, 8])), int(rng.choice([64, 128]))
    G, page = int(rng.integers(1, 9)), int(rng.choice([16, 32, 64, 128, 256]))
    ctx = np.exp(rng.uniform(0, np.log(3000), B)).astype(int) - 1
    new = np.where(rng.random(B) < 0.6, 1, rng.integers(0, 70, B))
    window, sinks = ((0, 0), (int(rng.integers(1, 700)), int(rng.integers(0, 90))))[seed % 2]
    b = Batch(ctx, new, G * Hkv, Hkv, D, page, seed=seed, spare_rows=1)
    check(b, run(b, window, sinks), window, sinks)


def test_pages_beyond_four_gigabytes():
    """Codes at offsets past 32 bits: the last pages of a cache of 4.3 GB per
    tensor are written, read and attended to."""
    t = torch()
    n_pages, Hkv, P, D = 33000, 8, 256, 128
    c = qoq.PagedKV4Cache(n_pages, Hkv, P, D)
    assert c.k_codes.numel() > 2 ** 32
    rng = np.random.default_rng(22)
    ctx = [600, 300]
    table = np.array([[32999, 5, 32990], [32800, 32801, -1]], np.int32)
    kv = rng.standard_normal((2, sum(ctx), Hkv, D)).astype(np.float16)
    at = [np.arange(n) for n in ctx]
    slots = np.concatenate([table[r, a // P] * P + a % P for r, a in enumerate(at)]).astype(np.int32)
    c.write(dev(kv[0]), dev(kv[1]), dev(slots))
    k, v = c.read(dev(slots))
    for x, got in zip(kv, (k, v)):
        d = kv4_paged.quantize_kv4(x)
        want = ((d["q"].astype(np.float32) - d["z"].astype(np.float32)[..., None]) * d["s"].astype(np.float32)[..., None])
        assert (host(got) == want.astype(np.float16)).all()
    # The oracle on the same pages, renumbered.
    pages = [32999, 5, 32990, 32800, 32801]
    small = [host(x[pages]) for x in (c.k_codes, c.k_params, c.v_codes, c.v_params)]
    small_table = np.array([[0, 1, 2], [3, 4, -1]], np.int32)
    for new in ([1, 1], [70, 3]):
        q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q = rng.standard_normal((q_start[-1], 16, D)).astype(np.float16)
        out = host(qoq.kv4_paged_attention(dev(q), c, dev(table), dev(q_start), dev(np.array(ctx, np.int32)), max(new)))
        o, vmax = kv4_paged.attention(q, *small, small_table, q_start, np.array(ctx, np.int32), 0, 0)
        assert (np.abs(out - o).max(axis=2) <= 2.0 ** -10 * vmax + 2.0 ** -24).all()
    del c, k, v
    t.cuda.empty_cache()


def test_a_step_on_a_given_stream():
    """Plan, write, read, attention and release with stream=: the buffers and
    bits of the same calls on the current stream."""
    t = torch()
    rng = np.random.default_rng(23)
    new, rows = dev(np.array([70, 0, 3, 200], np.int32)), rng.standard_normal((2, 280, 2, 64)).astype(np.float16)
    q = dev(rng.standard_normal((280, 8, 64)).astype(np.float16))
    leave = dev(np.array([0, 0, 1, 1], np.int32))
    got = []
    for s in (None, t.cuda.Stream()):
        pt, c, step = qoq.PageTable(4, 20, 40, 16), qoq.PagedKV4Cache(40, 2, 16, 64), qoq.PagedStep(4, 280)
        k, v = dev(rows[0]), dev(rows[1])
        out, kr, vr = t.zeros_like(q), t.zeros_like(k), t.zeros_like(v)
        ws = qoq.Workspace(qoq.kv4_paged_workspace_bytes(4, 280, 8, 2, 64, 200))
        t.cuda.synchronize()
        pt.assign(new, step, stream=s)
        c.write(k, v, step.slots, stream=s)
        assert c.read(step.slots, kr, vr, stream=s) == (kr, vr)
        qoq.kv4_paged_attention(q, c, pt.block_table, step.q_start, pt.seq_lens, 200, ws=ws, out=out, stream=s)
        pt.release(leave, stream=s)
        t.cuda.synchronize()
        assert pt.status() == 0 and ws.status() == 0 and host(pt.seq_lens).tolist() == [70, 0, 0, 0]
        got.append([host(x) for x in (out, kr, vr, step.slots, pt.block_table, pt.free_pages)])
    assert all(np.array_equal(a, b) for a, b in zip(*got)) and (got[0][1][:273] != 0).any()


def test_strided_queries_and_outputs():
    t = torch()
    b = Batch([100, 0], [2, 150], 8, 2, 128, 32, seed=20)
    wide = t.full((b.rows, 12, 128), 7.0, dtype=t.float16, device="cuda")
    wide[:, 2:10] = dev(b.q)
    out = t.full((b.rows, 20, 128), 7.0, dtype=t.float16, device="cuda")
    qoq.kv4_paged_attention(wide[:, 2:10], b.cache(), dev(b.table), dev(b.q_start), dev(b.kv), 150, out=out[:, 5:13])
    o = host(out)
    check(b, np.ascontiguousarray(o[:, 5:13]))
    assert (o[:, :5] == 7.0).all() and (o[:, 13:] == 7.0).all()


def test_attention_equals_contiguous_decode():
    """The same tokens in the contiguous cache: both decode calls meet the bar
    around one another."""
    q, K, V = inputs.make_decode_attention(3, 500, 32, 8, 128, seed=21)
    kc, vc = (qoq.KV4Cache(3, 8, 500, 128).write(dev(x)) for x in (K, V))
    a = host(qoq.kv4_decode_attention(dev(q), kc, vc)).astype(np.float64)
    pt, c, step = qoq.PageTable(3, 32, 100, 16), qoq.PagedKV4Cache(100, 8, 16, 128), qoq.PagedStep(3, 1500)
    pt.assign(dev(np.full(3, 500, np.int32)), step)
    rows = [dev(np.ascontiguousarray(x.transpose(0, 2, 1, 3).reshape(1500, 8, 128))) for x in (K, V)]
    c.write(*rows, step.slots)
    out = host(qoq.kv4_paged_attention(dev(q), c, pt.block_table, dev(np.arange(4, dtype=np.int32)), pt.seq_lens, 1))
    vmax = np.abs(V.astype(np.float64)).max(axis=(2, 3)).repeat(4, axis=1)
    assert (np.abs(out - a).max(axis=2) <= 2 * (2.0 ** -10 * 1.1 * vmax + 2.0 ** -24)).all()


def test_a_served_batch_end_to_end():
    """A layer's path as a server runs it: hidden states through the W4A8 qkv
    projection, pages assigned, K and V written, attention, requests ending
    and joining; every step's outputs against the oracle on the cache's bytes,
    the cache's bytes against the oracle's quantiser of the projection."""
    t = torch()
    Hq, Hkv, D, P, B, K = 8, 2, 128, 16, 5, 256
    blob = qoq.quantize_weights(dev(inputs.make_weights((Hq + 2 * Hkv) * D, K, seed=1, std=0.05)), 128)
    pt, c = qoq.PageTable(B, 20, 60, P), qoq.PagedKV4Cache(60, Hkv, P, D)
    shadow = [np.zeros((60, Hkv, P, D // 2), np.uint8), np.zeros((60, Hkv, P, 2), np.float16)] * 2
    plan = [[40, 0, 7, 0, 1], [1, 90, 1, 0, 1], [1, 1, 1, 33, 64], [1, 1, 0, 1, 1], [30, 1, 1, 1, 1], [1, 1, 1, 1, 1]]
    for k, new in enumerate(plan):
        step = qoq.PagedStep(B, 160)
        pt.assign(dev(np.array(new, np.int32)), step)
        X = inputs.make_activations(160, K, seed=k)
        qkv = qoq.linear(dev(X), blob, (Hq + 2 * Hkv) * D, K).view(160, Hq + 2 * Hkv, D)
        c.write(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], step.slots)
        out = qoq.kv4_paged_attention(qkv[:, :Hq], c, pt.block_table, step.q_start, pt.seq_lens, 100, window=48, sinks=2)
        h, slots, rows = host(qkv), host(step.slots), sum(new)
        shadow[0], shadow[1] = kv4_paged.write(h[:, Hq:Hq + Hkv], slots, shadow[0], shadow[1], P)
        shadow[2], shadow[3] = kv4_paged.write(h[:, Hq + Hkv:], slots, shadow[2], shadow[3], P)
        for x, y in zip((c.k_codes, c.k_params, c.v_codes, c.v_params), shadow):
            assert np.array_equal(host(x), y)
        o, vmax = kv4_paged.attention(h[:, :Hq], *shadow, host(pt.block_table), host(step.q_start), host(pt.seq_lens),
                                      48, 2)
        err = np.abs(host(out)[:rows].astype(np.float64) - o[:rows]).max(axis=2)
        assert (err <= 2.0 ** -10 * vmax[:rows] + 2.0 ** -24).all()
        if k == 2:
            pt.release(dev(np.array([0, 1, 0, 0, 1], np.int32)))
    assert pt.status() == 0 and oracle.kv4 is kv4
