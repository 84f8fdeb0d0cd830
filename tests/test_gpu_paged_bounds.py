"""Paged KV4 attention on the GPU at the borders of its stated bound (the bar
of paged_case.py): inputs for which one rounding, one hidden token or one wait
too few would show."""
import numpy as np
import pytest

from gpu_helpers import torch
from paged_case import Batch, check, run

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
