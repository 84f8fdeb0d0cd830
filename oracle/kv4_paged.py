"""Plain CPU reference of the paged KV4 cache -- TEST INFRASTRUCTURE.

Page tables, slot maps, the paged cache's bytes and the attention of new
tokens over it, written from the definitions in include/qoq.h with Python
loops and binary64, sharing no code with the CUDA library. The quantiser is
oracle.kv4's.
"""
from __future__ import annotations

import numpy as np

from .kv4 import dequantize_kv4, pack_kv4, quantize_kv4


def assign(seq_lens, new_lens, free_pages, free_count, block_table, page_size, max_tokens):
    """A step's page tables, or None when it is refused for lack of room.
    Returns dict(kv_lens, q_start, positions, slots, block_table, free_left);
    the inputs are not changed."""
    table = np.array(block_table, copy=True)
    stack = [int(p) for p in free_pages[:free_count]]
    q_start, positions, slots, kv = [0], [], [], []
    for b, (s, n) in enumerate(zip(seq_lens, new_lens)):
        if s + n > table.shape[1] * page_size:
            return None
        for pos in range(s, s + n):
            if pos % page_size == 0:
                if not stack:
                    return None
                table[b, pos // page_size] = stack.pop()
            positions.append(pos)
            slots.append(int(table[b, pos // page_size]) * page_size + pos % page_size)
        q_start.append(len(positions))
        kv.append(s + n)
    if len(positions) > max_tokens:
        return None
    pad = [-1] * (max_tokens - len(positions))
    return dict(kv_lens=np.array(kv, np.int32), q_start=np.array(q_start, np.int32),
                positions=np.array(positions + pad, np.int32), slots=np.array(slots + pad, np.int32),
                block_table=table, free_left=len(stack))


def release(leave, seq_lens, block_table, free_pages, free_count, page_size):
    """Pages of the flagged requests back on the stack, the last taken first.
    Returns (seq_lens, block_table, free_pages, free_count)."""
    seq, table, free = np.array(seq_lens), np.array(block_table), np.array(free_pages)
    back = [(b, i) for b in range(len(seq)) if leave[b] for i in range(-(-int(seq[b]) // page_size))]
    for b, i in reversed(back):
        free[free_count] = table[b, i]
        free_count += 1
        table[b, i] = -1
    seq[np.asarray(leave) != 0] = 0
    return seq, table, free, free_count


def write(k, slots, codes, params, page_size):
    """Rows k FP16 [N][Hkv][D] into copies of codes and params."""
    codes, params = np.array(codes), np.array(params)
    d = quantize_kv4(k)
    packed = pack_kv4(d["q"])
    for row, slot in enumerate(slots):
        if 0 <= slot < codes.shape[0] * page_size:
            page, at = divmod(int(slot), page_size)
            codes[page, :, at] = packed[row]
            params[page, :, at, 0] = d["s"][row]
            params[page, :, at, 1] = d["z"][row]
    return codes, params


def read(slots, codes, params):
    """(q - z) * s of slots, binary64 [N][Hkv][D]; 0 outside the cache."""
    n_pages, Hkv, P, DB = codes.shape
    slots = np.asarray(slots, dtype=np.int64)
    ok = (slots >= 0) & (slots < n_pages * P)
    page, at = np.divmod(np.where(ok, slots, 0), P)
    c = codes[page, :, at]
    q = np.stack([c & 15, c >> 4], axis=-1).reshape(len(slots), Hkv, 2 * DB)
    out = dequantize_kv4(q, params[page, :, at, 0], params[page, :, at, 1]).astype(np.float64)
    out[~ok] = 0.0
    return out


def visible(position, n_tokens, window=0, sinks=0):
    """Truth values over a request's tokens: what a row at `position` sees."""
    t = np.arange(n_tokens)
    seen = t <= position
    if window:
        seen &= (position - t < window) | (t < sinks)
    return seen


def attention(q, k_codes, k_params, v_codes, v_params, block_table, q_start, kv_lens, window=0, sinks=0):
    """Binary64 outputs [N][Hq][D] (rows of no request: NaN), and per row and
    head the largest |v| over the tokens that the row sees."""
    P, Hkv = k_codes.shape[2], k_codes.shape[1]
    N, Hq, D = q.shape
    out = np.full((N, Hq, D), np.nan)
    vmax = np.zeros((N, Hq))
    for b in range(len(kv_lens)):
        a, n, T = int(q_start[b]), int(q_start[b + 1]) - int(q_start[b]), int(kv_lens[b])
        out[a:a + n] = 0.0
        if n == 0 or T == 0:
            continue
        where = np.arange(T - n, T)
        seen = np.stack([visible(p, T, window, sinks) for p in where])
        some = seen.any(axis=0)
        t = np.flatnonzero(some)
        slots = block_table[b, t // P].astype(np.int64) * P + t % P
        kk, vv = read(slots, k_codes, k_params), read(slots, v_codes, v_params)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            s = q[a:a + n, h].astype(np.float64) @ kk[:, g].T / np.sqrt(D)
            s = np.where(seen[:, some], s, -np.inf)
            m = s.max(axis=1, keepdims=True)
            e = np.exp(s - np.where(np.isfinite(m), m, 0.0))
            e = np.where(seen[:, some], e, 0.0)
            total = e.sum(axis=1, keepdims=True)
            out[a:a + n, h] = np.where(total > 0, e @ vv[:, g] / np.where(total > 0, total, 1.0), 0.0)
            big = np.abs(vv[:, g]).max(axis=1)
            vmax[a:a + n, h] = np.where(seen[:, some], big, 0.0).max(axis=1)
    return out, vmax
