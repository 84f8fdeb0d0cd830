"""The paged KV4 calls on the GPU where little separates a right answer from a
wrong one: attention at the borders of its stated bound (the bar of
paged_case.py), and calls beside one another."""
import threading

import numpy as np
import pytest

from gpu_helpers import dev, host, torch
from oracle import kv4_paged
from paged_case import Batch, check, run, workspace
from w4a8_quantized_gemm_qoq_b200 import qoq

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch().cuda.is_available(), "GPU tests need a CUDA device"
    from w4a8_quantized_gemm_qoq_b200 import build
    build.build()
    yield


def slots_of(b, r, t):
    """Index of tokens t of request r in the cache's arrays, all heads."""
    return b.table[r, t // b.page], slice(None), t % b.page


def put(b, r, t, x, tensor):
    """Tokens t of request r: x [len(t)][Hkv][D], quantised as the cache does."""
    slots = b.table[r, t // b.page].astype(np.int64) * b.page + t % b.page
    if tensor == "k":
        b._put(x, slots, b.k_codes, b.k_params)
    else:
        b._put(x, slots, b.v_codes, b.v_params)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rise", [3.0, 7.0, 13.0])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 5)])
def test_a_maximum_that_rises_in_every_block(D, rise, window, sinks):
    """Scores that grow by 2^rise every 32 keys, so that the weights stored
    earlier in a step are rescaled in its second, third and fourth block."""
    b = Batch([700, 0], [40, 300], 8, 2, D, 64, seed=int(rise))
    b.q[:] = 1.0 + 0.125 * b.q
    for r in range(2):
        t = np.arange(int(b.kv[r]))
        level = (t // 32) * rise * np.log(2.0) / np.sqrt(D)
        put(b, r, t, np.broadcast_to(level[:, None, None], (len(t), 2, D)).copy(), "k")
    check(b, run(b, window, sinks), window, sinks)


def test_page_steps_of_several_threads():
    """Host threads with tables of different sizes above 4096 requests, each on
    its own stream: no step is refused for what another thread's needs."""
    t = torch()
    go, failed = threading.Barrier(3), []

    def serve(B):
        try:
            s = t.cuda.Stream()
            pt, step = qoq.PageTable(B, 8, B, 16), qoq.PagedStep(B, 0)
            none, leave = (t.zeros(B, dtype=t.int32, device="cuda") for _ in range(2))
            t.cuda.synchronize()
            go.wait()
            for _ in range(6000):
                pt.assign(none, step, stream=s)
                pt.release(leave, stream=s)
            s.synchronize()
            assert pt.status() == 0
        except Exception as e:
            failed.append((B, e))

    threads = [threading.Thread(target=serve, args=(B,)) for B in (16384, 4200, 12500)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not failed, failed


def test_a_captured_page_step_beside_a_smaller_one():
    """A step of 16384 requests, captured before and replayed after one of 4200."""
    t = torch()
    B = 16384
    pt, step, n = qoq.PageTable(B, 2, B, 16), qoq.PagedStep(B, B), t.ones(B, dtype=t.int32, device="cuda")
    small, small_step = qoq.PageTable(4200, 2, 4200, 16), qoq.PagedStep(4200, 4200)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        pt.assign(n, step)
    small.assign(n[:4200], small_step)
    g.replay()
    small.assign(n[:4200], small_step)
    g.replay()
    assert pt.status() == 0 and small.status() == 0
    assert (host(pt.seq_lens) == 2).all() and (host(small.seq_lens) == 2).all()


@pytest.mark.parametrize("B", [4050, 4080, 4096, 4097, 12200, 12288, 12289, 16384])
def test_page_steps_of_many_requests(B):
    """Batches around those at which a step's shared memory passes what a kernel
    gets without asking: a step in which every request begins, and its release."""
    t = torch()
    pt, step, n = qoq.PageTable(B, 2, B, 16), qoq.PagedStep(B, B), t.ones(B, dtype=t.int32, device="cuda")
    free = host(pt.free_pages)
    pt.assign(n, step)
    want = kv4_paged.assign(np.zeros(B, int), np.ones(B, int), free, B, np.full((B, 2), -1), 16, B)
    for name in ("q_start", "positions", "slots"):
        assert np.array_equal(host(getattr(step, name)), want[name]), name
    assert np.array_equal(host(pt.block_table), want["block_table"]) and int(host(pt.free_count)[0]) == 0
    pt.release(n)
    assert np.array_equal(host(pt.free_pages), free) and not host(pt.seq_lens).any() and pt.status() == 0


U = 2.0 ** -24   # the smallest FP16 number, and the step of every scale below 2^-14


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("level", [-22, -37, -217, 22])
def test_values_of_the_smallest_scales(D, page, new, level):
    """Vectors whose scale is subnormal: its rounding makes zeros of up to 22 of
    4-bit codes (-22 units: scale 1, zero 22, code 0)."""
    b = Batch([90, 0, 300], [new, 3, 1], 8, 2, D, page, seed=new)
    for r in range(3):
        t = np.arange(int(b.kv[r]))
        x = np.full((len(t), 2, D), level * U)
        x[t % 5 == 4] = 3 * U
        put(b, r, t, x, "v")
    if level < 0:
        assert (b.v_params[slots_of(b, 0, np.arange(90))][..., 1] > 15).any()
    check(b, run(b))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("level", [-22, -37, -217])
def test_keys_of_the_smallest_scales(D, page, new, level):
    """The same among the keys, under queries so large that they count: scores
    0.7 to 4 apart, and values of ordinary size that tell them apart."""
    b = Batch([90, 0, 300], [new, 3, 1], 8, 2, D, page, seed=new)
    b.q[:] = min(50000.0, 4 / (-level * U * np.sqrt(D))) * (0.9 + 0.1 * np.tanh(b.q.astype(np.float64)))
    for r in range(3):
        t = np.arange(int(b.kv[r]))
        x = np.zeros((len(t), 2, D))
        x[t % 3 == 0] = level * U
        put(b, r, t, x, "k")
    check(b, run(b))


def test_smallest_scales_equal_contiguous_decode():
    """One request of such keys and values in both caches: each decode call
    within the bar."""
    b = Batch([199], [1], 8, 2, 128, 16, seed=4)
    rng = np.random.default_rng(4)
    t = np.arange(200)
    x = {n: (rng.choice([-22, -37, -217, 0, 5], (200, 2, 1)) * U * np.ones(128)).astype(np.float16) for n in "kv"}
    for n in "kv":
        put(b, 0, t, x[n], n)
    kc, vc = (qoq.KV4Cache(1, 2, 200, 128).write(dev(np.ascontiguousarray(x[n].transpose(1, 0, 2))[None])) for n in "kv")
    for got in (run(b), host(qoq.kv4_decode_attention(dev(b.q), kc, vc))):
        check(b, got)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gain", [2.0 ** -13, 0.002, 2.0 ** -4])
@pytest.mark.parametrize("window,sinks", [(50, 2), (1, 0), (1, 1), (130, 20)])
@pytest.mark.parametrize("bad", [65504.0, np.inf, np.nan])
def test_scales_of_hidden_tokens_do_not_matter(D, gain, window, sinks, bad):
    """Tokens that no row sees hold huge, infinite or NaN scales beside small
    visible values: the bound is that of the visible ones alone."""
    b = Batch([400, 901, 130], [40, 1, 60], 8, 2, D, 16, seed=9, gain=gain)
    want = b.oracle(window, sinks)
    for r in range(3):
        t = np.arange(sinks, int(b.ctx[r]) - window + 1)
        b.k_params[slots_of(b, r, t)] = bad if bad != 65504.0 else 1.0
        b.v_params[slots_of(b, r, t)] = bad
    check(b, run(b, window, sinks), want=want)


def _hide(b, window, sinks, number):
    """Entries of pages without a visible token become `number`."""
    for r in range(len(b.ctx)):
        first = max(0, int(b.ctx[r]) - window + 1)   # of the first row's window
        for i in range(-(-int(b.kv[r]) // b.page)):
            if sinks <= i * b.page and (i + 1) * b.page <= first:
                b.table[r, i] = number


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(100, 0), (100, 4), (77, 70), (1, 1)])
@pytest.mark.parametrize("number", [-1, 10 ** 6])
def test_pages_without_visible_tokens_may_be_taken_back(D, page, window, sinks, number):
    """Pages between the sinks and the window are no longer in the table:
    no request is refused, the outputs are those of the full table."""
    b = Batch([1000, 611, 0, 2050, 333], [1, 5, 300, 90, 17], 8, 2, D, page, seed=page)
    want = b.oracle(window, sinks)
    _hide(b, window, sinks, number)
    assert (b.table[:, :2] != -1).any()
    check(b, run(b, window, sinks), want=want)


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("where", ["sinks", "window"])
def test_a_page_with_one_visible_token_is_checked(page, new, where):
    """The page that holds the first token of the window, its last one, or the last sink:
    a bad entry names the request."""
    ctx = 20 * page + 99   # the first row's window begins with the last token of page 20
    window, sinks = 100 - page + 1, 3 * page + 1
    b = Batch([50, ctx], [1, new], 8, 2, 128, page, seed=page)
    assert (ctx - window + 1) == 21 * page - 1
    entry = 3 if where == "sinks" else 20
    b.table[1, entry] = -1
    ws = workspace(b)
    qoq.kv4_paged_attention(dev(b.q), b.cache(), dev(b.table), dev(b.q_start), dev(b.kv), new, window=window, sinks=sinks,
                            ws=ws)
    assert ws.status() == 1 and ws.timeout_site()[0] == 1


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,G", [(1, 4), (5, 8), (3, 1), (100, 4)])
def test_queries_of_the_smallest_numbers(D, new, G):
    """Queries of a few units of 2^-24 under keys of 60000: scores of ordinary
    size, which an eighth of a unit lost per dim would change."""
    b = Batch([60, 0, 300], [new, new, 1], 2 * G, 2, D, 64, seed=D + new)
    rng = np.random.default_rng(D)
    b.q[:] = rng.integers(1, 40, b.q.shape) * U
    for r in range(3):
        t = np.arange(int(b.kv[r]))
        put(b, r, t, np.broadcast_to((rng.integers(-1, 2, (len(t), 2, 1)) * 60000.0), (len(t), 2, D)).copy(), "k")
    check(b, run(b))


def test_queries_of_different_sizes_side_by_side():
    """Heads and rows from 2^-24 to 2^10 in one product: each meets the bar."""
    b = Batch([70, 500], [3, 1], 16, 2, 128, 64, seed=6)
    e = np.arange(b.rows * 16).reshape(b.rows, 16)
    b.q[:] = b.q.astype(np.float64) * 2.0 ** -(e % 15)[..., None]
    b.q[0, 3], b.q[1, 5], b.q[2, 7, ::2] = 0, np.float16(U), 0
    b.q[3, 9] *= np.float16(2.0 ** 9)
    for r in range(2):
        t = np.arange(int(b.kv[r]))
        at = slots_of(b, r, t)
        b.k_params[at + (0,)] = (b.k_params[at + (0,)].astype(np.float64) / 256).astype(np.float16)
    check(b, run(b))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new", [([300, 40], [1, 1]), ([5000], [3]), ([200, 0], [100, 70]), ([4000], [60])])
@pytest.mark.parametrize("what", [np.nan, np.inf])
def test_queries_that_are_not_numbers(D, ctx, new, what):
    """A NaN or infinite component of a query: that row and head's outputs are
    not numbers, the others are as without it."""
    b = Batch(ctx, new, 8, 2, D, 64, seed=5)
    want = b.oracle()
    i, h = b.rows - 1, 5
    b.q[i, h, 17] = what
    out = run(b)
    assert np.isnan(out[i, h]).all()
    err = np.abs(out.astype(np.float64) - want[0]).max(axis=2)
    err[i, h] = 0
    assert (err <= 2.0 ** -10 * want[1] + 2.0 ** -24).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new", [([300, 40], [1, 1]), ([5000], [3]), ([200, 0], [100, 70]), ([4000], [60])])
@pytest.mark.parametrize("tensor", ["k", "v"])
@pytest.mark.parametrize("what", [np.nan, np.inf])
def test_visible_scales_that_are_not_numbers(D, ctx, new, tensor, what):
    """A token whose scale is infinite or NaN: the outputs of the rows that see
    it are not numbers, in its KV head alone; rows that do not see it are clean."""
    b = Batch(ctx, new, 8, 2, D, 64, seed=7)
    window, sinks = 90, 3
    want = b.oracle(window, sinks)
    n, kv = int(b.new[0]), int(b.kv[0])
    at = kv - 1 - n // 2
    (b.k_params if tensor == "k" else b.v_params)[b.table[0, at // 64], 1, at % 64, 0] = what
    out = run(b, window, sinks)
    seen = np.zeros((b.rows, 8), bool)
    for i in range(n):
        seen[i, 4:] = kv4_paged.visible(kv - n + i, kv, window, sinks)[at]
    assert seen.any() and np.isnan(out[seen]).all()
    err = np.abs(out.astype(np.float64) - want[0]).max(axis=2)
    assert (err[~seen] <= (2.0 ** -10 * want[1] + 2.0 ** -24)[~seen]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new", [([30], [1]), ([30], [40]), ([3000], [60])])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_infinite_query_under_keys_of_one_sign(D, ctx, new, sign):
    """Every score of the row is -infinity, or every one +infinity: a softmax of
    either has no value."""
    b = Batch(ctx, new, 8, 2, D, 64, seed=8)
    t = np.arange(int(b.kv[0]))
    x = np.random.default_rng(8).standard_normal((len(t), 2, D))
    x[:, :, 17] = sign * 4
    put(b, 0, t, x, "k")
    want = b.oracle()
    b.q[0, 2, 17] = np.inf
    out = run(b)
    assert np.isnan(out[0, 2]).all()
    err = np.abs(out.astype(np.float64) - want[0]).max(axis=2)
    err[0, 2] = 0
    assert (err <= 2.0 ** -10 * want[1] + 2.0 ** -24).all()


@pytest.mark.parametrize("B,top,window", [(8, 16, 0), (3, 100, 0), (20, 13, 200)])
def test_a_padded_batch_of_few_rows(B, top, window):
    """A step with room for `top` rows of every request serves requests of few:
    the bits are those of the step without that room."""
    b = Batch([(0, 61, 500, 3, 260)[i % 5] for i in range(B)], [1 + i % 3 for i in range(B)], 8, 2, 128, 64, seed=B)
    want = run(b, window, 4)
    b.q = np.concatenate([b.q, np.zeros((B * top - len(b.q),) + b.q.shape[1:], np.float16)])
    got = run(b, window, 4, max_new=top)
    check(b, got, window, 4)
    assert np.array_equal(got[:b.rows].view(np.uint16), want[:b.rows].view(np.uint16))


def test_one_workspace_for_calls_of_different_shapes():
    """Batches, head sizes and row bounds that lay the scratch out differently,
    one after another in one workspace: the bits of calls with their own."""
    shapes = [([300] * 200, [1] * 200, 4, 1, 64), ([5000], [1], 8, 2, 128), ([100, 0], [200, 3], 8, 2, 128),
              ([7] * 130, [30] * 130, 4, 1, 64), ([9000, 20], [1, 40], 8, 8, 128), ([20000], [2], 8, 1, 64)]
    batches = [Batch(c, n, Hq, Hkv, D, 64, seed=i) for i, (c, n, Hq, Hkv, D) in enumerate(shapes)]
    big = qoq.Workspace(max(workspace(b).buf.numel() for b in batches))
    for _ in range(2):
        for b in batches + batches[::-1]:
            got = run(b, ws=big)
            assert np.array_equal(got.view(np.uint16), run(b).view(np.uint16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new", [([300, 40], [1, 1]), ([200, 0], [100, 70])])
def test_negative_zeros_among_the_parameters(D, ctx, new):
    """A cache filled by other means may hold -0 as a zero or a scale: 0."""
    b = Batch(ctx, new, 8, 2, D, 64, seed=2)
    rng = np.random.default_rng(2)
    for r in range(2):
        t = np.arange(int(b.kv[r]))
        for name in "kv":
            put(b, r, t, np.abs(rng.standard_normal((len(t), 2, D))), name)
            put(b, r, t[::5], np.zeros((len(t[::5]), 2, D)), name)
    want = b.oracle()
    for params in (b.k_params, b.v_params):
        params[params == 0] = np.float16(-0.0)
    check(b, run(b), want=want)


@pytest.mark.parametrize("many", [False, True])
def test_the_largest_batch(many):
    """16384 requests, the most a step takes, with and without requests of many rows."""
    rng = np.random.default_rng(1)
    new = rng.integers(0, 3, 16384)
    if many:
        new[::3000] = 40
    b = Batch(rng.integers(0, 20, 16384), new, 2, 1, 64, 16, seed=1, spare_rows=1)
    check(b, run(b))


@pytest.mark.parametrize("B", [1, 7, 130, 2100])
def test_a_step_without_rows(B):
    """No request brings a token: nothing is written, nothing refused."""
    b = Batch([30] * B, [0] * B, 8, 2, 64, 16, seed=1, spare_rows=60)
    run(b, max_new=1)
    run(b, max_new=60)
    run(b, 7, 1, max_new=60)
