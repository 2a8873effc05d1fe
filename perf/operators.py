"""What is measured of the operators on a paged KV cache.

The operators are the steps of a stream whose cache stays bounded: the norm
and rotation of queries and keys (alone, or storing K and V into the cache's
pages in the same pass), the attention of a chunk of new tokens over the
pages, the attention weight that every cached key has received, and the
eviction of the keys that received least.

``run`` computes a case in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, with the library's kernels; ``exact`` is the
definition in 64 bits.
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
FRAME = 1560          # tokens of a frame (30 x 52 latent positions)
FRAME_H, FRAME_W = 30, 52

# 33 streams that decode one token each: short, page-edge and long caches.
_TOKEN_SEQS = ",".join(f"1:{n}" for n in (
    1, 2, 15, 16, 17, 127, 128, 129, 255, 600, 900, 1561, 2047, 2049, 2500, 3120, 3500, 4095, 4097, 5000, 6241, 7000,
    8191, 8193, 9000, 9999, 10921, 12000, 12481, 14000, 16383, 18000, 20281))


def _case(name, op, dtype, heads, kv_heads, d, page, seqs, **kw):
    c = {"op": op, "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "d": d, "page": page, "seqs": seqs}
    if name:
        c = {"name": name, **c}
    c.update(kw)
    return c


def listed():
    video = {"axes": "44,42,42", "halves": False, "norm": True}
    text = {"axes": "128", "halves": True, "norm": True}
    return [
        # One token of one stream: what a call costs when there is next to nothing to do.
        _case("prep-one-token", "prep", BF16, 12, 12, 128, 0, "1:1", **video),
        # The frame of the single-layer workload between its projection and its attention.
        _case("prep-frame", "prep", BF16, 12, 12, 128, 0, f"{FRAME}:{FRAME}", **video),
        # Eight streams that bring chunks of several frames and odd lengths into their caches.
        _case("append-chunks", "append", BF16, 12, 12, 128, 64,
              f"{2 * FRAME}:{2 * FRAME},{4 * FRAME}:{9 * FRAME},1:777,{FRAME}:{21 * FRAME},4999:5003,129:4000,7000:7000,"
              f"{FRAME + 1}:{FRAME + 1}", **video),
        # A single new token against a one-frame cache: latency.
        _case("attend-token", "attend", BF16, 12, 12, 128, 64, f"1:{FRAME + 1}", mask=1),
        # Single tokens of many streams of very different lengths, shared key heads, small pages.
        _case("attend-tokens-ragged", "attend", BF16, 16, 2, 128, 16, _TOKEN_SEQS, mask=1),
        # A frame's query pass against 20 clean frames and itself: the KV-cache layer of the stack, paged.
        _case("attend-frame", "attend", BF16, 12, 12, 128, 128, f"{FRAME}:{21 * FRAME}", mask=FRAME),
        # Causal prompt chunks of odd lengths, some with a cache before them, shared key heads.
        _case("attend-causal-chunks", "attend", BF16, 32, 4, 128, 16, "1:4097,77:77,513:8000,1900:1900,2000:16001", mask=1),
        # The float32 path on small heads: frames of 16 tokens and longer ones.
        _case("attend-f32", "attend", F32, 4, 2, 32, 16, "16:128,16:400,100:1000,1:3000,333:333", mask=16),
        # The frame's weights after its clean pass.
        _case("weights-frame", "weights", BF16, 12, 12, 128, 128, f"{FRAME}:{21 * FRAME}", mask=FRAME, decay=1.0),
        # The weights of single tokens, fading.
        _case("weights-tokens", "weights", BF16, 16, 2, 128, 16, _TOKEN_SEQS, mask=1, decay=0.97),
        # A 21-frame cache cut back to ten and a half frames.
        _case("evict-frames", "evict", BF16, 12, 12, 128, 128, f"{FRAME}:{21 * FRAME}", budget=16380, sink=FRAME,
              recent=2 * FRAME),
        # Ragged float32 caches; some are below the budget and are kept whole.
        _case("evict-ragged-f32", "evict", F32, 4, 2, 64, 16, "1:100,1:999,1:1024,1:1025,1:2222,1:4100,1:6000,1:7777,1:9001",
              budget=1024, sink=4, recent=100),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prep", "append", "attend", "attend", "attend", "weights", "weights", "evict"])
    dtype = BF16 if rng.random() < 0.75 else F32
    heads, kv_heads = rng.choice([(12, 12), (4, 4), (6, 2), (16, 2), (32, 4), (5, 1)])
    d = 128 if dtype == BF16 else rng.choice([32, 64, 128])
    page = rng.choice([16, 24, 64, 128])
    n = _log(rng, 1, 33)
    pairs = []
    if op in ("prep", "append"):
        budget = 25000 // (1 if dtype == BF16 else 4)
        for _ in range(n):
            q = max(1, min(_log(rng, 1, 7000), budget))
            budget = max(1, budget - q)
            pairs.append((q, q + (rng.choice([0, 0, _log(rng, 1, 3000)]) if op == "append" else 0)))
        axes = rng.choice([str(d), f"{d // 2}", f"{d // 2},{d // 4},{d // 4}", f"{d // 4},{d // 4}"])
        kw = {"axes": axes, "halves": rng.random() < 0.5, "norm": rng.random() < 0.8}
    elif op in ("attend", "weights"):
        # visible pairs x heads stay below a few percent of the largest case's
        work = 2.0e9 / heads if dtype == BF16 else 1.0e8 / heads
        for _ in range(n):
            q = 1 if rng.random() < 0.5 else _log(rng, 1, 2100)
            old = _log(rng, 1, 20000)
            while q > 1 and q * (q + old) > work:
                q //= 2
            if q * (q + old) > work:
                old = max(1, int(work / q) - q)
            work -= q * (q + old)
            if work <= 0 and pairs:
                break
            pairs.append((q, q + old - 1))
        kw = {"mask": rng.choice([0, 1, 1, 16, 100])}
        if op == "weights":
            kw["decay"] = rng.choice([1.0, 0.9])
    else:
        total = 300000 // kv_heads
        for _ in range(n):
            kv = min(_log(rng, 1, 30000), total)
            total -= kv
            if kv < 1:
                break
            pairs.append((1, kv))
        b = _log(rng, 8, 12000)
        sink = rng.randrange(0, b // 2)
        kw = {"budget": b, "sink": sink, "recent": rng.randrange(0, b - sink)}
    return _case(None, op, dtype, heads, kv_heads, d, page if op != "prep" else 0,
                 ",".join(f"{q}:{k}" for q, k in pairs), **kw)


# ------------------------------------------------------------------ inputs
def _seqs(case):
    """[(new tokens, cached tokens with them)] of each stream."""
    return [tuple(int(x) for x in s.split(":")) for s in case["seqs"].split(",")]


def _tdt(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def _axes(case):
    return [int(a) for a in case["axes"].split(",")]


def _inputs(case, seed):
    """The tensors a program has in hand before the call, on the GPU."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, dt = "cuda", _tdt(case)
    H, Hk, d = case["heads"], case["kv_heads"], case["d"]
    seqs = _seqs(case)
    T = sum(q for q, _ in seqs)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    def starts(ns):
        s = [0]
        for n in ns:
            s.append(s[-1] + n)
        return s

    x = {"q_start": torch.tensor(starts([q for q, _ in seqs]), dtype=torch.int32, device=dev),
         "kv_len": torch.tensor([k for _, k in seqs], dtype=torch.int32, device=dev)}
    op = case["op"]
    if op in ("prep", "append"):
        # Q | K | V side by side in each token's row, as a fused projection writes them
        x["rows"] = randn(T, (H + 2 * Hk) * d).to(dt)
        x["w_q"] = (1.0 + 0.1 * randn(d)).to(dt)
        x["w_k"] = (1.0 + 0.1 * randn(d)).to(dt)
        axes = _axes(case)
        if len(axes) == 1:  # far positions of a long stream
            first = torch.randint(0, 1000000, (len(seqs),), generator=g, device=dev)
        else:
            first = torch.randint(0, 40 * FRAME, (len(seqs),), generator=g, device=dev)
        tok = torch.cat([first[b] + torch.arange(q, device=dev) for b, (q, _) in enumerate(seqs)])
        cols = {1: [tok], 2: [tok // FRAME_W, tok % FRAME_W],
                3: [tok // FRAME, tok % FRAME // FRAME_W, tok % FRAME_W]}[len(axes)]
        x["pos"] = torch.stack(cols, 1).to(torch.int32).contiguous()
    else:
        x["q"] = randn(T, H, d).to(dt)
    if op == "prep":
        return x
    page = case["page"]
    need = [-(-k // page) for _, k in seqs]
    kept = [-(-min(k, case["budget"]) // page) for _, k in seqs] if op == "evict" else []
    n_pages = sum(need) + sum(kept) + 3  # a few pages that belong to nobody
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    x["pages"] = torch.full((len(seqs), max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        x["pages"][b, :n] = order[at:at + n]
        at += n
    if op == "evict":
        x["dst_pages"] = torch.full((len(seqs), max(kept)), -1, dtype=torch.int32, device=dev)
        for b, n in enumerate(kept):
            x["dst_pages"][b, :n] = order[at:at + n]
            at += n
    x["k_pool"] = randn(n_pages, Hk, page, d).to(dt)
    x["v_pool"] = randn(n_pages, Hk, page, d).to(dt)
    width = max(k for _, k in seqs)
    if op == "weights":
        # the attention of the same rows has left their logarithms of the sums
        x["lse"] = torch.cat([t for t in _row_lse(case, x)])
    if op in ("weights", "evict"):
        # heavy-tailed sums of weights; those of keys that got little come in coarse steps and tie
        w = torch.exp(1.5 * randn(len(seqs), Hk, width))
        w = torch.where(w < 0.5, torch.round(w * 64) / 64, w)
        behind = torch.arange(width, device=dev)[None, None, :] >= x["kv_len"][:, None, None]
        x["w"] = torch.where(behind, torch.zeros_like(w), w).contiguous()
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    st = {"case": case, "x": x, "seqs": _seqs(case)}
    if not own:
        return st
    from hybrid_linear_attention_arl2_b200 import arl2
    dt = arl2.ARL2_BF16 if case["dtype"] == BF16 else arl2.ARL2_F32
    H, Hk, d = case["heads"], case["kv_heads"], case["d"]
    if case["op"] in ("prep", "append"):
        norm = case["norm"]
        st["prep"] = arl2.QKPrep(axis_dims=_axes(case), theta=10000.0, halves=case["halves"], eps=1e-6,
                                 w_q=x["w_q"] if norm else None, w_k=x["w_k"] if norm else None)
    if case["op"] != "prep":
        max_q = max(q for q, _ in st["seqs"])
        max_kv = max(k for _, k in st["seqs"])
        st["batch"] = arl2.PagedBatch(x["q_start"], x["kv_len"], x["pages"], tokens=sum(q for q, _ in st["seqs"]),
                                      max_q=max_q, max_kv=max_kv)
        st["layer"] = arl2.PagedKVLayer(H, Hk, d, dt, x["k_pool"], x["v_pool"])
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    case, x = state["case"], state["x"]
    if own:
        return _run_own(state, case, x)
    return {"prep": _plain_prep, "append": _plain_append, "attend": _plain_attend, "weights": _plain_weights,
            "evict": _plain_evict}[case["op"]](case, x)


def _split_rows(case, x):
    H, Hk, d = case["heads"], case["kv_heads"], case["d"]
    rows = x["rows"]
    T = rows.shape[0]
    q, k, v = rows[:, :H * d], rows[:, H * d:(H + Hk) * d], rows[:, (H + Hk) * d:]
    return q.unflatten(1, (H, d)), k.unflatten(1, (Hk, d)), v.unflatten(1, (Hk, d))


def _run_own(state, case, x):
    from hybrid_linear_attention_arl2_b200 import arl2
    op = case["op"]
    if op == "prep":
        q, k, _ = _split_rows(case, x)
        return arl2.qk_norm_rope(state["prep"], q, k, x["pos"])
    layer, batch = state["layer"], state["batch"]
    if op == "append":
        q, k, v = _split_rows(case, x)
        q_out = layer.append(batch, k, v, q=q, prep=state["prep"], pos=x["pos"])
        return q_out, x["k_pool"], x["v_pool"]
    if op == "attend":
        return layer.attend(batch, x["q"], mask_block=case["mask"])
    if op == "weights":
        return layer.weights(batch, x["q"], x["lse"], x["w"], mask_block=case["mask"], decay=case["decay"])
    n, w, kept = layer.evict(batch, x["w"], x["dst_pages"], budget=case["budget"], sink=case["sink"],
                             recent=case["recent"])
    return n, w, kept, x["k_pool"], x["v_pool"]


# ------------------------------------------------------------------ plain forms
def _plain_norm_rope(case, t, w, pos):
    """[T, heads, d] -> the same, normed and rotated, in the type of t."""
    y = t.float()
    if case["norm"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
    axes = _axes(case)
    R = sum(axes)
    ang = []
    for a, n in enumerate(axes):
        freq = 10000.0 ** (-2.0 * torch.arange(n // 2, device=t.device, dtype=torch.float64) / n)
        ang.append(pos[:, a].double()[:, None] * freq)  # far positions need the 64 bits
    ang = torch.cat(ang, 1)
    cos, sin = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    if case["halves"]:
        y0, y1 = y[..., :R // 2], y[..., R // 2:R]
        rot = torch.cat([y0 * cos - y1 * sin, y0 * sin + y1 * cos], -1)
    else:
        y0, y1 = y[..., 0:R:2], y[..., 1:R:2]
        rot = torch.stack([y0 * cos - y1 * sin, y0 * sin + y1 * cos], -1).flatten(-2)
    return torch.cat([rot, y[..., R:]], -1).to(t.dtype)


def _plain_prep(case, x):
    q, k, _ = _split_rows(case, x)
    return _plain_norm_rope(case, q, x["w_q"], x["pos"]), _plain_norm_rope(case, k, x["w_k"], x["pos"])


def _plain_append(case, x):
    q, k, v = _split_rows(case, x)
    q_out = _plain_norm_rope(case, q, x["w_q"], x["pos"])
    k_new = _plain_norm_rope(case, k, x["w_k"], x["pos"])
    page, at = case["page"], 0
    for b, (n, kv) in enumerate(_seqs(case)):
        j = torch.arange(kv - n, kv, device=k.device)
        p = x["pages"][b, j // page].long()
        x["k_pool"][p, :, j % page] = k_new[at:at + n]
        x["v_pool"][p, :, j % page] = v[at:at + n]
        at += n
    return q_out, x["k_pool"], x["v_pool"]


def _gathered(pool, table, kv, page):
    """[kv heads, kv, d] of one stream, in 32 bits."""
    p = table[:-(-kv // page)].long()
    return pool[p].float().transpose(0, 1).flatten(1, 2)[:, :kv]


def _visible(n, kv, mask, device):
    """How many cached keys each new token sees: all, or those before the chunk and the chunk's blocks up to its own."""
    if mask == 0:
        return torch.full((n,), kv, device=device)
    t = torch.arange(n, device=device)
    return (kv - n + (torch.div(t, mask, rounding_mode="floor") + 1) * mask).clamp(0, kv)


def _scores(case, x):
    """Yields (first row, rows, stream, masked scores [kv heads, rows, G, kv]) over the streams' rows, in pieces."""
    H, Hk, d, page = case["heads"], case["kv_heads"], case["d"], case["page"]
    G, at = H // Hk, 0
    for b, (n, kv) in enumerate(_seqs(case)):
        K = _gathered(x["k_pool"], x["pages"][b], kv, page)
        lim = _visible(n, kv, case["mask"], K.device)
        step = max(1, int(2 ** 28 // (H * kv)))
        for r in range(0, n, step):
            m = min(step, n - r)
            q = x["q"][at + r:at + r + m].float().unflatten(1, (Hk, G)).permute(1, 0, 2, 3).flatten(1, 2)
            s = ((q @ K.transpose(1, 2)) * d ** -0.5).unflatten(1, (m, G))
            hide = torch.arange(kv, device=K.device)[None, :] >= lim[r:r + m, None]
            yield at + r, m, b, s.masked_fill_(hide[None, :, None, :], -math.inf)
        at += n


def _row_lse(case, x):
    for _, m, _, s in _scores(case, x):
        top = s.amax(-1, keepdim=True)
        lse = (s - top).exp_().sum(-1).log_() + top[..., 0]
        yield lse.permute(1, 0, 2).flatten(1)


def _plain_attend(case, x):
    H, Hk, d = case["heads"], case["kv_heads"], case["d"]
    o, lse = torch.empty_like(x["q"]), torch.empty(x["q"].shape[:2], dtype=torch.float32, device="cuda")
    have, V = -1, None
    for r, m, b, s in _scores(case, x):
        if b != have:
            have, V = b, _gathered(x["v_pool"], x["pages"][b], _seqs(case)[b][1], case["page"])
        top = s.amax(-1, keepdim=True)
        p = s.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        out = (p.flatten(1, 2) @ V).unflatten(1, (m, H // Hk)) / total
        o[r:r + m] = out.permute(1, 0, 2, 3).flatten(1, 2).to(o.dtype)
        lse[r:r + m] = (total.log() + top)[..., 0].permute(1, 0, 2).flatten(1)
    return o, lse


def _plain_weights(case, x):
    Hk = case["kv_heads"]
    w = x["w"] * case["decay"]
    for r, m, b, s in _scores(case, x):
        lse = x["lse"][r:r + m].unflatten(1, (Hk, -1)).permute(1, 0, 2)[..., None]
        w[b, :, :s.shape[-1]] += (s - lse).exp_().sum((1, 2))
    return w


def _plain_evict(case, x):
    page, budget, sink, recent = case["page"], case["budget"], case["sink"], case["recent"]
    seqs, Hk = _seqs(case), case["kv_heads"]
    dev = x["w"].device
    kept = torch.full((len(seqs), Hk, budget), -1, dtype=torch.int32, device=dev)
    w_out = torch.zeros_like(x["w"])
    for b, (_, kv) in enumerate(seqs):
        m = min(kv, budget)
        if kv <= budget:
            idx = torch.arange(kv, device=dev).expand(Hk, kv)
        else:
            mid = x["w"][b, :, sink:kv - recent]
            best = torch.sort(mid, dim=-1, descending=True, stable=True).indices[:, :budget - sink - recent] + sink
            ends = torch.cat([torch.arange(sink, device=dev), torch.arange(kv - recent, kv, device=dev)])
            idx = torch.cat([best, ends.expand(Hk, sink + recent)], 1).sort(-1).values
        kept[b, :, :m] = idx.to(torch.int32)
        w_out[b, :, :m] = x["w"][b].gather(1, idx)
        src = x["pages"][b].long()[idx // page]
        head = torch.arange(Hk, device=dev)[:, None]
        j = torch.arange(m, device=dev)
        dst = x["dst_pages"][b].long()[j // page]
        for pool in (x["k_pool"], x["v_pool"]):
            rows = pool[src, head, idx % page]
            pool[dst[None, :], head, (j % page)[None, :]] = rows
    n_out = torch.clamp(x["kv_len"], max=budget)
    return n_out, w_out, kept, x["k_pool"], x["v_pool"]


# ------------------------------------------------------------------ work
def _pairs(case):
    total = 0
    for n, kv in _seqs(case):
        if case["mask"] == 0:
            total += n * kv
        else:
            m = case["mask"]
            total += sum(max(0, min(kv, kv - n + (t // m + 1) * m)) for t in range(n))
    return total * case["heads"]


def work(case):
    H, Hk, d = case["heads"], case["kv_heads"], case["d"]
    e = 2 if case["dtype"] == BF16 else 4
    seqs = _seqs(case)
    T, cached = sum(q for q, _ in seqs), sum(k for _, k in seqs)
    op = case["op"]
    if op == "prep":
        return {"bytes": 2 * T * (H + Hk) * d * e + T * len(_axes(case)) * 4, "flops": 8 * T * (H + Hk) * d}
    if op == "append":
        return {"bytes": 2 * T * (H + 2 * Hk) * d * e + T * len(_axes(case)) * 4, "flops": 8 * T * (H + Hk) * d}
    if op == "attend":
        return {"bytes": 2 * T * H * d * e + 4 * T * H + 2 * cached * Hk * d * e, "flops": 4 * d * _pairs(case)}
    if op == "weights":
        return {"bytes": T * H * d * e + 4 * T * H + cached * Hk * d * e + 8 * cached * Hk, "flops": 2 * d * _pairs(case)}
    kept = sum(min(k, case["budget"]) for _, k in seqs)
    return {"bytes": 4 * cached * Hk + kept * Hk * (4 * d * e + 8), "flops": cached * Hk}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_turned(case, t, w, pos):
    y = t.double()
    if case["norm"]:
        y = y / torch.sqrt(torch.sum(y ** 2, -1, keepdim=True) / y.shape[-1] + 1e-6) * w.double()
    out, at, R = y.clone(), 0, sum(_axes(case))
    for a, n in enumerate(_axes(case)):
        for i in range(n // 2):
            ang = pos[:, a].double() * math.exp(-2.0 * i / n * math.log(10000.0))
            c0, c1 = (at, at + R // 2) if case["halves"] else (2 * at, 2 * at + 1)
            z = torch.complex(y[..., c0], y[..., c1]) * torch.polar(torch.ones_like(ang), ang)[:, None]
            out[..., c0], out[..., c1] = z.real, z.imag
            at += 1
    return out


def _exact_rows(case, x, b, start, h):
    """The stream's queries of head h, keys and values it reads, scaled logits with hidden pairs at -inf; 64 bits."""
    n, kv = _seqs(case)[b]
    hk, page, d = h // (case["heads"] // case["kv_heads"]), case["page"], case["d"]
    j = torch.arange(kv, device="cuda")
    at = x["pages"][b].long()[j // page] * page + j % page
    k = x["k_pool"][:, hk].reshape(-1, d)[at].double()
    v = x["v_pool"][:, hk].reshape(-1, d)[at].double()
    logits = x["q"][start:start + n, h].double() @ k.T / math.sqrt(d)
    if case["mask"]:
        block = torch.where(j < kv - n, -1, torch.div(j - (kv - n), case["mask"], rounding_mode="floor"))
        logits[block[None, :] > block[kv - n:, None]] = -math.inf
    return logits, v


def exact(case, seed):
    x = _inputs(case, seed)
    op, H, Hk = case["op"], case["heads"], case["kv_heads"]
    seqs, page = _seqs(case), case["page"]
    if op in ("prep", "append"):
        q, k, v = _split_rows(case, x)
        q, k = _exact_turned(case, q, x["w_q"], x["pos"]), _exact_turned(case, k, x["w_k"], x["pos"])
        if op == "prep":
            return q, k
        kp, vp = x["k_pool"].double(), x["v_pool"].double()
        row = [(b, j) for b, (n, kv) in enumerate(seqs) for j in range(kv - n, kv)]
        rb = torch.tensor([r[0] for r in row], device="cuda")
        rj = torch.tensor([r[1] for r in row], device="cuda")
        p = x["pages"].long()[rb, rj // page]
        kp[p, :, rj % page], vp[p, :, rj % page] = k, v.double()
        return q, kp, vp
    if op == "attend":
        T = x["q"].shape[0]
        o = torch.zeros(T, H, case["d"], dtype=torch.float64, device="cuda")
        lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
        start = 0
        for b, (n, _) in enumerate(seqs):
            for h in range(H):
                logits, v = _exact_rows(case, x, b, start, h)
                o[start:start + n, h] = torch.softmax(logits, -1) @ v
                lse[start:start + n, h] = torch.logsumexp(logits, -1)
            start += n
        return o, lse
    if op == "weights":
        w, start = x["w"].double() * case["decay"], 0
        for b, (n, kv) in enumerate(seqs):
            for h in range(H):
                logits, _ = _exact_rows(case, x, b, start, h)
                w[b, h // (H // Hk), :kv] += torch.exp(logits - x["lse"][start:start + n, h, None].double()).sum(0)
            start += n
        return w
    budget, sink, recent = case["budget"], case["sink"], case["recent"]
    kept = torch.full((len(seqs), Hk, budget), -1, dtype=torch.int32)
    w_out, w_in = torch.zeros(x["w"].shape, dtype=torch.float64), x["w"].cpu()
    kp, vp = x["k_pool"].double(), x["v_pool"].double()
    for b, (_, kv) in enumerate(seqs):
        for h in range(Hk):
            w = w_in[b, h, :kv].tolist()
            if kv <= budget:
                ids = list(range(kv))
            else:
                mid = sorted(range(sink, kv - recent), key=lambda j: (-w[j], j))[:budget - sink - recent]
                ids = sorted(list(range(sink)) + mid + list(range(kv - recent, kv)))
            m = len(ids)
            idx = torch.tensor(ids)
            kept[b, h, :m] = idx.int()
            w_out[b, h, :m] = w_in[b, h, idx].double()
            idx, j = idx.cuda(), torch.arange(m, device="cuda")
            s, t = x["pages"][b].long()[idx // page], x["dst_pages"][b].long()[j // page]
            kp[t, h, j % page] = x["k_pool"][s, h, idx % page].double()
            vp[t, h, j % page] = x["v_pool"][s, h, idx % page].double()
    return torch.clamp(x["kv_len"], max=budget), w_out.cuda(), kept.cuda(), kp, vp
