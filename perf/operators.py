"""The paged KV4 operators as measured workloads: page tables and slot maps
from request lengths, the paged 4-bit cache's write and read, and attention
of new tokens over the paged cache, with and without a sliding window.

``run`` computes them in elementary torch operations (``own`` false) or by the
library's calls (``own`` true); ``exact`` in 64 bits from the definitions.
Sequence lengths follow from the case alone and only their order from the
seed, so ``work`` holds for every seed.
"""
import math

import torch

own = False

KEY_OUTLIERS, KEY_GAIN = 2, 8.0   # outlier channels of the keys, per KV head


def listed():
    heads = dict(Hq=32, Hkv=8, D=128)   # the repository's attention heads
    none = dict(window=0, sinks=0)
    return [
        # A decode step's page table update: one token for each of 64 sequences.
        dict(name="plan_decode_64", op="plan", B=64, page=64, ctx_lo=1000, ctx_hi=1100, chunks=0, new_lo=1, new_hi=1,
             release=False),
        # 256 requests enter with prompts of 1 to 1000 tokens, and all of them leave again.
        dict(name="plan_turnover_256", op="plan", B=256, page=16, ctx_lo=0, ctx_hi=0, chunks=256, new_lo=1,
             new_hi=1000, release=True),
        # A decode step's new keys and values.
        dict(name="write_decode_64", op="write", N=64, Hkv=8, D=128, Hq=32, page=64, pad=0),
        # The keys and values of a prefill step of 8187 tokens, padded to 8192 rows.
        dict(name="write_prefill_8192", op="write", N=8192, Hkv=8, D=128, Hq=32, page=64, pad=5),
        # The attention measurement shape of the repository: batch 64 x 1024 cached tokens.
        dict(name="decode_64x1024", op="attn", B=64, page=64, ctx_lo=1023, ctx_hi=1023, chunks=0, new_lo=1, new_hi=1,
             **heads, **none),
        # Decode of 24 conversations of very different lengths, in small pages.
        dict(name="decode_ragged_24", op="attn", B=24, page=16, ctx_lo=99, ctx_hi=32700, chunks=0, new_lo=1, new_hi=1,
             **heads, **none),
        # Five drafted tokens of 32 sequences verified at once.
        dict(name="verify_32x5", op="attn", B=32, page=64, ctx_lo=1500, ctx_hi=4500, chunks=32, new_lo=5, new_hi=5,
             **heads, **none),
        # A whole prompt at once.
        dict(name="prompt_4096", op="attn", B=1, page=64, ctx_lo=0, ctx_hi=0, chunks=1, new_lo=4096, new_hi=4096,
             **heads, **none),
        # One chunk of a long prompt over what is cached of it.
        dict(name="chunk_2048_of_16384", op="attn", B=1, page=64, ctx_lo=14336, ctx_hi=14336, chunks=1, new_lo=2048,
             new_hi=2048, **heads, **none),
        # A serving step: four chunks of odd lengths among decoding sequences; small heads, eight per KV head.
        dict(name="mixed_16", op="attn", B=16, page=32, ctx_lo=17, ctx_hi=5000, chunks=4, new_lo=77, new_hi=777, Hq=16,
             Hkv=2, D=64, **none),
        # Decode of 64 long streams that keep a window of 1024 tokens and four sinks.
        dict(name="window_decode_64", op="attn", B=64, page=64, ctx_lo=4000, ctx_hi=8100, chunks=0, new_lo=1, new_hi=1,
             window=1024, sinks=4, **heads),
        # Two prompts under the same window.
        dict(name="window_prompt_2x4096", op="attn", B=2, page=64, ctx_lo=2000, ctx_hi=2000, chunks=2, new_lo=4001,
             new_hi=4096, window=1024, sinks=4, **heads),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "attn", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 1000)
        release = rng.random() < 0.4
        chunks = B if release else rng.randint(0, B)
        lo = _log(rng, 1, 300)
        return dict(op=op, B=B, page=page, ctx_lo=0 if release else _log(rng, 1, 500),
                    ctx_hi=0 if release else _log(rng, 501, 9000), chunks=chunks, new_lo=lo,
                    new_hi=lo + _log(rng, 1, 300), release=release)
    Hkv, G, D = rng.choice([(8, 4, 128), (2, 8, 64), (8, 1, 128), (4, 7, 128), (1, 8, 128), (5, 3, 64)])
    if op == "write":
        N = _log(rng, 1, 8192)
        return dict(op=op, N=N, Hkv=Hkv, D=D, Hq=Hkv * G, page=page, pad=rng.randint(0, min(9, N - 1)))
    windowed = rng.random() < 0.4
    mask = dict(window=_log(rng, 100, 4000), sinks=rng.choice([0, 1, 4, 70])) if windowed else dict(window=0, sinks=0)
    kind = rng.choice(["decode", "verify", "chunk", "mixed"])
    B = _log(rng, 1, 64) if kind == "decode" else _log(rng, 1, 32) if kind == "verify" else rng.randint(1, 12)
    top = 1 if kind == "decode" else rng.randint(2, 9) if kind == "verify" else _log(rng, 100, 2500)
    hi = _log(rng, 300, 16000)
    # Scores of the padded plain form, and the work, at most those of the largest listed case.
    while B * Hkv * G * top * (hi + top) > 1 << 30 or B * Hkv * (hi + top) * D > 1 << 29:
        B, top, hi = max(1, B - 1), max(1, top - top // 8), max(200, hi - hi // 8)
    chunks = 0 if kind == "decode" else B if kind in ("verify", "chunk") else rng.randint(1, B)
    return dict(op=op, B=B, page=page, ctx_lo=rng.choice([0, 1, hi // 50, hi // 2, hi]), ctx_hi=hi, chunks=chunks,
                new_lo=top if kind == "verify" else max(1, top // 3), new_hi=top, Hq=Hkv * G, Hkv=Hkv, D=D, **mask)


# ------------------------------------------------------------------ lengths

def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spaced over their logarithm."""
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / max(1, n - 1)))) - 1 for i in range(n)]


def _lengths(c):
    """(cached, new) tokens per request: `chunks` requests bring new_lo..new_hi tokens, the others one."""
    new = _spread(c["new_lo"], c["new_hi"], c["chunks"]) + [1] * (c["B"] - c["chunks"])
    ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["B"])
    return list(zip(ctx[1::2] + ctx[0::2], new))


def _visible(ctx, new, window, sinks):
    """(keys that some query sees, visible pairs) of one request."""
    total = ctx + new
    if not window:
        return total, new * ctx + new * (new + 1) // 2
    pairs = 0
    for p in range(ctx, total):
        first = max(0, p - window + 1)
        pairs += p + 1 - first + min(sinks, first)
    first = max(0, ctx - window + 1)
    return total - first + min(sinks, first), pairs


def work(case):
    c = case
    if c["op"] == "plan":
        pairs = _lengths(c)
        tokens = sum(n for _, n in pairs)
        pages = sum(-(-(s + n) // c["page"]) - -(-s // c["page"]) for s, n in pairs)
        # lengths in and out, token ranges, positions and slots; a taken page is read from the free list and entered
        nbytes = 16 * c["B"] + 8 * tokens + 8 * pages
        if c["release"]:   # lengths and the entries read, entries cleared, pages listed as free again
            nbytes += 12 * c["B"] + 12 * pages
        return {"bytes": nbytes, "flops": 0}
    if c["op"] == "write":
        vec = 2 * (c["N"] - c["pad"]) * c["Hkv"]
        # FP16 in, codes and scale and zero out; those in again, FP16 out
        return {"bytes": vec * (2 * c["D"] + 2 * (c["D"] // 2 + 4) + 2 * c["D"]) + 8 * c["N"], "flops": 4 * vec * c["D"]}
    rows = keys = pairs = 0
    for s, n in _lengths(c):
        k, p = _visible(s, n, c["window"], c["sinks"])
        rows, keys, pairs = rows + n, keys + k, pairs + p
    return {"bytes": 4 * rows * c["Hq"] * c["D"] + 2 * keys * c["Hkv"] * (c["D"] // 2 + 4) + 4 * (keys // c["page"]),
            "flops": 4 * c["D"] * c["Hq"] * pairs}


# ------------------------------------------------------------------ the plain forms

def _scale_zero(x):
    """Scale (FP16 value) and zero of each vector along the last axis, in FP32."""
    lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
    s = ((hi - lo) / 15).half().float()
    z = torch.where(s > 0, torch.round(-lo / torch.where(s > 0, s, 1)), 0)
    return s, z


def _quantise(x):
    """FP32 [..., D] -> codes 0..15 (FP32), scales, zeros."""
    s, z = _scale_zero(x)
    safe = torch.where(s > 0, s, 1)[..., None]
    q = (torch.round(x / safe) + z[..., None]).clamp(0, 15)
    return torch.where(s[..., None] > 0, q, 0), s, z


def _pack(q, s, z):
    q = q.to(torch.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4), torch.stack([s, z], -1).half()


def _unpack(codes, params):
    """(code - zero) * scale, FP32 [..., D]."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    p = params.float()
    return (q - p[..., 1:2]) * p[..., 0:1]


def _plain_plan(st):
    P, s, n, count = st["page"], st["seq_lens"].long(), st["new_lens"].long(), st["free_count"].long()
    table, dev = st["table"], st["seq_lens"].device
    have, need = (s + P - 1) // P, (s + n + P - 1) // P
    take = need - have
    taken = torch.cumsum(take, 0)
    start = torch.cumsum(n, 0)
    col = torch.arange(table.shape[1], device=dev)
    new_page = (col >= have[:, None]) & (col < need[:, None])
    at = count - 1 - (taken - take)[:, None] - (col - have[:, None])
    filled = torch.where(new_page, st["free_pages"][at.clamp(min=0, max=st["free_pages"].numel() - 1)], table)
    tok = torch.arange(st["max_tokens"], device=dev)
    b = torch.searchsorted(start, tok, right=True).clamp(max=s.numel() - 1)
    real = tok < start[-1]
    pos = s[b] + tok - (start - n)[b]
    page = filled[b, (pos // P).clamp(max=table.shape[1] - 1)].long()
    out = dict(q_start=torch.cat([torch.zeros_like(start[:1]), start]).int(), kv_lens=(s + n).int(),
               positions=torch.where(real, pos, -1).int(), slots=torch.where(real, page * P + pos % P, -1).int())
    if not st["release"]:
        return dict(out, table=filled, free_left=(count - taken[-1]).int())
    # every request leaves: its pages go back, the last one first
    g = (taken - take)[:, None] + col
    back = count - taken[-1] + taken[-1] - 1 - g
    free = st["free_pages"].clone()
    free[back[new_page]] = filled[new_page]
    return dict(out, kv_lens=torch.zeros_like(out["kv_lens"]), table=torch.full_like(table, -1), free=free,
                free_left=count.int())


def _plain_write(st):
    slots = st["slots"].long()
    keep = slots >= 0
    page, at = slots[keep] // st["page"], slots[keep] % st["page"]
    got = []
    for name in ("k", "v"):
        codes, params = _pack(*_quantise(st[name][keep].float()))
        st[name + "_codes"][page, :, at] = codes
        st[name + "_params"][page, :, at] = params
        back = _unpack(st[name + "_codes"][page, :, at], st[name + "_params"][page, :, at])
        full = torch.zeros(st[name].shape, dtype=torch.float16, device=back.device)
        full[keep] = back.half()
        got.append(full)
    return tuple(got)


def _plain_attention(st):
    q, table, dev = st["q"], st["table"], st["q"].device
    B, Hkv, P = table.shape[0], st["k_codes"].shape[1], st["page"]
    N, Hq, D = q.shape
    new, kv = st["q_start"].diff().long(), st["kv_lens"].long()
    nmax, used = st["max_new"], st["used_pages"]
    pages = table[:, :used].long().clamp(min=0)
    T = used * P

    def cached(name):   # [B][Hkv][T][D]
        x = _unpack(st[name + "_codes"][pages], st[name + "_params"][pages])
        return x.transpose(1, 2).reshape(B, Hkv, T, D)

    i = torch.arange(nmax, device=dev)
    row = (st["q_start"][:-1].long()[:, None] + i).clamp(max=N - 1)
    real = i < new[:, None]
    qp = q[row].float().view(B, nmax, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    scores = torch.matmul(qp, cached("k").transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, Hkv, -1, nmax, T)
    pos = (kv - new)[:, None] + i
    t = torch.arange(T, device=dev)
    seen = t <= pos[..., None]
    if st["window"]:
        seen &= (pos[..., None] - t < st["window"]) | (t < st["sinks"])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    total = scores.sum(-1, keepdim=True)
    o = torch.matmul(scores.view(B, Hkv, -1, T), cached("v")).view(B, Hkv, -1, nmax, D) / total
    return o.permute(0, 3, 1, 2, 4).reshape(B, nmax, Hq, D)[real].half()


# ------------------------------------------------------------------ inputs

def _caches(st, pages, Hkv, P, D, g, dev):
    """K and V pages as a server holds them: quantised N(0, 1) values, outlier channels in the keys."""
    cols = torch.stack([torch.randperm(D, generator=g, device=dev)[:KEY_OUTLIERS] for _ in range(Hkv)])
    gain = torch.ones(Hkv, D, device=dev).scatter_(1, cols, KEY_GAIN)
    step = max(1, (1 << 27) // (Hkv * P * D))
    for name in ("k", "v"):
        parts = []
        for a in range(0, pages, step):
            x = torch.randn(min(step, pages - a), Hkv, P, D, generator=g, device=dev)
            if name == "k":
                x = x * gain[:, None]
            parts.append(_pack(*_quantise(x.half().float())))
        st[name + "_codes"] = torch.cat([p[0] for p in parts])
        st[name + "_params"] = torch.cat([p[1] for p in parts])


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    P = c["page"]
    st = dict(op=c["op"], page=P)
    if c["op"] == "write":
        N, Hq, Hkv, D = c["N"], c["Hq"], c["Hkv"], c["D"]
        n_pages = -(-N // P) + 3
        _caches(st, n_pages, Hkv, P, D, g, dev)
        qkv = torch.randn(N, Hq + 2 * Hkv, D, generator=g, device=dev).half()   # the merged projection's output
        st["k"], st["v"] = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        st["slots"] = torch.randperm(n_pages * P, generator=g, device=dev)[:N].int()
        st["slots"][N - c["pad"]:] = -1
        if own:
            from w4a8_quantized_gemm_qoq_b200 import qoq
            st["cache"] = qoq.PagedKV4Cache.of(*(st[n] for n in ("k_codes", "k_params", "v_codes", "v_params")))
        return st
    pairs = _lengths(c)
    order = torch.randperm(len(pairs), generator=g, device=dev).tolist()
    pairs = [pairs[i] for i in order]
    ctx, new = [s for s, _ in pairs], [n for _, n in pairs]
    B, N = len(pairs), sum(new)
    kv = [s + n for s, n in pairs]
    before = [-(-s // P) for s in ctx]
    after = [-(-s // P) for s in kv]
    if c["op"] == "plan":
        n_pages = sum(after) + 7
        perm = torch.randperm(n_pages, generator=g, device=dev).int()
        table = torch.full((B, max(after) + 2), -1, dtype=torch.int32, device=dev)
        held = torch.arange(table.shape[1], device=dev) < _i32(before, dev)[:, None]
        table[held] = perm[:sum(before)]
        free = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        free[:n_pages - sum(before)] = perm[sum(before):]
        st.update(seq_lens=_i32(ctx, dev), new_lens=_i32(new, dev), table=table, free_pages=free,
                  free_count=_i32([n_pages - sum(before)], dev), max_tokens=N + 3, release=c["release"])
        if own:
            from w4a8_quantized_gemm_qoq_b200 import qoq
            st["pages"] = qoq.PageTable.of(st["seq_lens"], table, free, st["free_count"], P)
            st["step"] = qoq.PagedStep(B, N + 3)
            st["leave"] = torch.ones(B, dtype=torch.int32, device=dev)
            st["kv_lens"], st["free_left"] = torch.empty_like(st["seq_lens"]), torch.empty_like(st["free_count"])
        return st
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    n_pages = sum(after) + 3
    _caches(st, n_pages, Hkv, P, D, g, dev)
    table = torch.full((B, max(after) + 1), -1, dtype=torch.int32, device=dev)
    held = torch.arange(table.shape[1], device=dev) < _i32(after, dev)[:, None]
    table[held] = torch.randperm(n_pages, generator=g, device=dev)[:sum(after)].int()
    qkv = torch.randn(N, Hq + 2 * Hkv, D, generator=g, device=dev).half()
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    st.update(q=qkv[:, :Hq], table=table, q_start=_i32(starts, dev), kv_lens=_i32(kv, dev), max_new=max(new),
              used_pages=max(after), window=c["window"], sinks=c["sinks"])
    if own:
        from w4a8_quantized_gemm_qoq_b200 import qoq
        st["cache"] = qoq.PagedKV4Cache.of(*(st[n] for n in ("k_codes", "k_params", "v_codes", "v_params")))
        st["ws"] = qoq.Workspace(qoq.kv4_paged_workspace_bytes(B, N, Hq, Hkv, D, max(new)))
        st["out"] = torch.empty(N, Hq, D, dtype=torch.float16, device=dev)
    return st


def run(state):
    st = state
    if own:
        from w4a8_quantized_gemm_qoq_b200 import qoq
        if st["op"] == "plan":
            pages, step = st["pages"], st["step"]
            if st["release"]:
                pages.assign(st["new_lens"], step)
                pages.release(st["leave"])
                return dict(q_start=step.q_start, kv_lens=pages.seq_lens, positions=step.positions,
                            slots=step.slots, table=pages.block_table, free=pages.free_pages,
                            free_left=pages.free_count)
            pages.assign(st["new_lens"], step, kv_lens=st["kv_lens"], free_left=st["free_left"])
            return dict(q_start=step.q_start, kv_lens=st["kv_lens"], positions=step.positions, slots=step.slots,
                        table=pages.block_table, free_left=st["free_left"])
        if st["op"] == "write":
            st["cache"].write(st["k"], st["v"], st["slots"])
            return st["cache"].read(st["slots"])
        return qoq.kv4_paged_attention(st["q"], st["cache"], st["table"], st["q_start"], st["kv_lens"],
                                       st["max_new"], window=st["window"], sinks=st["sinks"], ws=st["ws"],
                                       out=st["out"])
    if st["op"] == "plan":
        return _plain_plan(st)
    return _plain_write(st) if st["op"] == "write" else _plain_attention(st)


# ------------------------------------------------------------------ in 64 bits

def _exact_vectors(x):
    """What each FP16 vector stands for after quantisation: (q - z) s."""
    x = x.double()
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    low = torch.minimum(x.min(dim=-1, keepdim=True).values, zero)
    high = torch.maximum(x.max(dim=-1, keepdim=True).values, zero)
    s = ((high - low) / 15).to(torch.float16).double()
    flat = s == 0
    s1 = s.masked_fill(flat, 1.0)
    z = torch.round(-low / s1)
    q = torch.clip(torch.round(x / s1) + z, 0, 15)
    return ((q - z) * s).masked_fill(flat, 0.0)


def exact(case, seed):
    if case["op"] == "plan":
        return None
    st = prepare(case, seed)
    if case["op"] == "write":
        there = (st["slots"] >= 0).double()[:, None, None]
        return _exact_vectors(st["k"]) * there, _exact_vectors(st["v"]) * there
    P, W, sinks = case["page"], case["window"], case["sinks"]
    N, Hq, D = st["q"].shape
    G = Hq // case["Hkv"]
    out = torch.zeros(N, Hq, D, dtype=torch.float64, device=st["q"].device)
    starts, kv = st["q_start"].tolist(), st["kv_lens"].tolist()
    for b, T in enumerate(kv):
        a, n = starts[b], starts[b + 1] - starts[b]
        first = max(0, T - n - W + 1) if W else 0
        keys = torch.arange(T, device=out.device)
        keys = keys[(keys >= first) | (keys < sinks)]   # every key that some query of the request sees
        page, at = st["table"][b].long()[keys // P], keys % P
        where = torch.arange(T - n, T, device=out.device)[:, None]
        hidden = keys > where
        if W:
            hidden |= (where - keys >= W) & (keys >= sinks)
        for h in range(case["Hkv"]):
            kk, vv = (((st[x + "_codes"][page, h, at][:, :, None] >> torch.tensor([0, 4], device=out.device)) & 15)
                      .reshape(len(keys), D).double() for x in ("k", "v"))
            kp, vp = (st[x + "_params"][page, h, at].double() for x in ("k", "v"))
            kk, vv = (kk - kp[:, 1:]) * kp[:, :1], (vv - vp[:, 1:]) * vp[:, :1]
            for j in range(h * G, (h + 1) * G):
                s = (st["q"][a:a + n, j].double() @ kk.T / D ** 0.5).masked_fill(hidden, -math.inf)
                s = s - torch.logsumexp(s, 1, keepdim=True)
                out[a:a + n, j] = s.exp() @ vv
    return out
