"""The paged-cache operators on the GPU against their float64 oracle: norm and
rotation, storing into pages, attention of new tokens, attention weights,
eviction, and a run of them together.

Rows that nobody owns hold NaN throughout.  Tolerances are bounds by
arithmetic (see paged_util.attend_bounds and the comments here); half a step is
2^-24 in float32 and 2^-8 in bf16.
"""
import ctypes

import numpy as np
import pytest
import torch

from hybrid_linear_attention_arl2_b200 import arl2, build
from oracle import paged_oracle as po
from tests.paged_util import ABI, TORCH, Paged, attend_bounds, host

pytestmark = pytest.mark.gpu
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    arl2.load_library()


def ok(layer):
    assert layer.last_error() == 0


# ------------------------------------------------------------------ norm and rotation
PREPS = [  # dtype, heads, kv_heads, d, axes, halves, norm, tokens
    ("bf16", 12, 12, 128, (44, 42, 42), False, True, 1),
    ("bf16", 12, 12, 128, (44, 42, 42), False, True, 131),
    ("bf16", 16, 2, 128, (128,), True, True, 700),
    ("bf16", 5, 1, 128, (32, 32), True, False, 33),
    ("bf16", 3, 3, 8, (2, 4), False, True, 7),
    ("bf16", 4, 2, 40, (32,), True, True, 3),
    ("bf16", 2, 2, 128, (), False, True, 5),
    ("f32", 4, 2, 32, (16, 8, 8), False, True, 600),
    ("f32", 6, 2, 64, (32,), False, False, 19),
    ("f32", 1, 1, 128, (64, 64), True, True, 2),
    ("f32", 7, 7, 4, (4,), False, True, 1000),
    ("f32", 2, 1, 100, (96,), True, True, 40),
]


def prep_bound(dtype, x, w, ref):
    """Norm: the sum of squares adds d/2 + 5 roundings at most in 32 lanes' order, of which the root takes half, plus
    its own and two products: under 80 steps of 2^-24 of y.  Rotation: the angle is a float of a fraction of a turn
    (2^-25 of half a turn: under 2^-23), its sine and cosine 2 steps, two products and a sum; relative to |y0| + |y1|,
    which R channels' largest norm bounds by sqrt(2) |y|_pair <= |ref pair| sqrt 2.  Then one rounding."""
    pair = np.sqrt(2 * (ref ** 2).sum(-1, keepdims=True))  # at least any pair's length
    return HALF[dtype] * np.abs(ref) + 100 * 2.0 ** -24 * np.minimum(pair, 1e30) + 1e-30


@pytest.mark.parametrize("dtype,H,hk,d,axes,halves,norm,T", PREPS)
@pytest.mark.parametrize("layout", ["dense", "rows", "in_place"])
def test_norm_rope(dtype, H, hk, d, axes, halves, norm, T, layout):
    g = torch.Generator().manual_seed(T * 7 + d)
    rows = torch.randn(T, (H + 2 * hk) * d, generator=g).to(TORCH[dtype])
    w_q, w_k = ((1 + 0.1 * torch.randn(d, generator=g)).to(TORCH[dtype]) for _ in range(2))
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (T, max(1, len(axes))), generator=g).to(torch.int32)
    pos[: T // 2] = torch.randint(0, 2000, (T // 2, pos.shape[1]), generator=g).to(torch.int32)
    pos = pos[:, :len(axes)].contiguous()
    prep = arl2.QKPrep(axes, theta=500.0, halves=halves, eps=1e-5, w_q=w_q.cuda() if norm else None,
                       w_k=w_k.cuda() if norm else None)
    dev = rows.cuda()
    q, k = (dev[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, H), (H, H + hk)))
    if layout == "dense":
        q, k = q.contiguous(), k.contiguous()
    p = pos.cuda() if axes else None
    if layout == "in_place":
        q_out, k_out = arl2.qk_norm_rope(prep, q, k, p, q_out=q, k_out=k)
        assert torch.equal(dev[:, (H + hk) * d:].cpu(), rows[:, (H + hk) * d:])
    else:
        q_out, k_out = arl2.qk_norm_rope(prep, q, k, p)
    x = host(rows)
    for got, a, n, w in ((q_out, 0, H, w_q), (k_out, H, hk, w_k)):
        ref = po.norm_rope(x[:, a * d:(a + n) * d].reshape(T, n, d), host(w) if norm else None, pos.numpy(), axes, 500.0,
                           halves, np.float32(1e-5))
        assert (np.abs(host(got) - ref) <= prep_bound(dtype, None, None, ref)).all()


# ------------------------------------------------------------------ append
APPENDS = [
    ("bf16", 12, 12, 128, 16, [(1, 1)]),
    ("bf16", 4, 2, 128, 24, [(5, 5), (0, 3), (70, 75), (1, 24), (2, 49), (0, 0)]),
    ("f32", 4, 2, 32, 8, [(3, 3), (9, 41), (600, 601)]),
    ("bf16", 2, 1, 128, 64, [(1, k + 1) for k in range(300)]),
]


@pytest.mark.parametrize("dtype,H,hk,d,page,seqs", APPENDS)
@pytest.mark.parametrize("prepped", [True, False])
def test_append(dtype, H, hk, d, page, seqs, prepped):
    c = Paged(dtype, H, hk, d, page, seqs, 5)
    extra = 3  # token rows behind the last stream's
    rows = c.randn(c.T + extra, (H + 2 * hk) * d)
    w_q, w_k = c.randn(d), c.randn(d)
    pos = torch.randint(0, 100000, (c.T + extra, 1), generator=c.g).to(torch.int32)
    kp, vp = c.kp.clone(), c.vp.clone()
    at = 0
    x = host(rows)
    turn = lambda a, n, w: po.norm_rope(x[:, a * d:(a + n) * d].reshape(-1, n, d), host(w), pos.numpy(), (d,))
    k_ref = turn(H, hk, w_k) if prepped else x[:, H * d:(H + hk) * d].reshape(-1, hk, d)
    k_all, new = host(kp), np.zeros(kp.shape, bool)
    for b, (n, kv) in enumerate(seqs):
        for t in range(n):
            j = kv - n + t
            pg = int(c.tables[b, j // page])
            k_all[pg, :, j % page], new[pg, :, j % page] = k_ref[at + t], True
            vp[pg, :, j % page] = rows[at + t, (H + hk) * d:].reshape(hk, d)
        at += n
    c.to_gpu(rows=c.T + extra)
    dev = rows.cuda()
    q, k, v = (dev[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, H), (H, H + hk), (H + hk, H + 2 * hk)))
    if prepped:
        prep = arl2.QKPrep([d], w_q=w_q.cuda(), w_k=w_k.cuda())
        q_out = torch.full((c.T + extra, H, d), 7.0, dtype=TORCH[dtype], device="cuda")
        c.layer.append(c.batch, k, v, q=q, prep=prep, pos=pos.cuda(), q_out=q_out)
        ref = turn(0, H, w_q)[:c.T]
        assert (np.abs(host(q_out)[:c.T] - ref) <= prep_bound(dtype, None, None, ref)).all()
        assert (q_out[c.T:] == 7).all()
    else:
        c.layer.append(c.batch, k, v)
    ok(c.layer)
    got = host(c.kp)
    assert np.array_equal(got[~new], k_all[~new], equal_nan=True)
    bound = prep_bound(dtype, None, None, k_all) if prepped else 0.0
    assert (np.abs(got - k_all) <= bound)[new].all()
    assert torch.equal(c.vp.cpu().nan_to_num(9.0), vp.nan_to_num(9.0))


# ------------------------------------------------------------------ attention and weights
ATTEND = [  # dtype, H, hk, d, page, mask, seqs
    ("bf16", 12, 12, 128, 16, 1, [(1, 1)]),
    ("bf16", 12, 12, 128, 64, 1, [(1, 1561)]),
    ("bf16", 16, 2, 128, 16, 1, [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 127), (1, 128), (1, 129), (1, 600), (1, 2049)]),
    ("bf16", 2, 2, 128, 128, 0, [(300, 300), (7, 900)]),
    ("bf16", 2, 2, 128, 128, 64, [(200, 700), (129, 129), (1, 300)]),
    ("bf16", 8, 1, 128, 24, 1, [(33, 33), (0, 50), (5, 3), (200, 345), (1, 0)]),
    ("bf16", 4, 4, 128, 8, 1, [(128, 128), (127, 255), (129, 513)]),
    ("bf16", 5, 1, 128, 96, 100, [(150, 400), (3, 3)]),
    ("bf16", 64, 1, 128, 32, 1, [(1, 700), (3, 77), (2, 130)]),
    ("bf16", 6, 2, 128, 4096, 1, [(40, 5000), (2, 2)]),
    ("bf16", 4, 2, 128, 136, 0, [(17, 1000), (300, 1700)]),
    ("f32", 4, 2, 32, 16, 16, [(16, 128), (100, 300), (1, 500), (33, 33)]),
    ("f32", 12, 12, 64, 24, 1, [(5, 3), (70, 200), (0, 0), (1, 0)]),
    ("f32", 3, 1, 128, 8, 0, [(65, 129), (1, 64)]),
    ("f32", 64, 1, 4, 16, 1, [(3, 90)]),
    ("f32", 2, 1, 100, 64, 1, [(64, 64)]),
]


def logit_parts(c, q):
    k = host(c.kp)
    return q, k[~np.isnan(k).any(-1)] if (~np.isnan(k).any(-1)).any() else np.zeros((1, c.d))


@pytest.mark.parametrize("dtype,H,hk,d,page,mask,seqs", ATTEND)
@pytest.mark.parametrize("spread", [1.0, 6.0])
def test_attend_and_weights(dtype, H, hk, d, page, mask, seqs, spread):
    c = Paged(dtype, H, hk, d, page, seqs, 11)
    wide = c.randn(c.T + 2, (H + 2) * d, scale=spread)  # queries as a strided view, two rows behind the last stream
    c.to_gpu(rows=c.T + 2)
    q = wide.cuda()[:, :H * d].unflatten(1, (H, d))
    o = torch.full((c.T + 2, H, d), 5.0, dtype=TORCH[dtype], device="cuda")
    lse = torch.full((c.T + 2, H), 5.0, dtype=torch.float32, device="cuda")
    c.layer.attend(c.batch, q, mask_block=mask, o=o, lse=lse)
    ok(c.layer)
    assert (o[c.T:] == 5).all() and (lse[c.T:] == 5).all()
    qh = host(q)[:c.T]
    kp, vp, tables = np.nan_to_num(host(c.kp)), np.nan_to_num(host(c.vp)), c.tables.numpy()
    ref_o, ref_l, mag = po.attend(qh, kp, vp, seqs, tables, mask)
    bo, bl = attend_bounds(dtype, d, *logit_parts(c, qh), c.width, mag, ref_o)
    got_o, got_l = host(o)[:c.T], host(lse)[:c.T]
    none = np.isinf(ref_l)
    assert np.array_equal(np.isinf(got_l), none) and not got_o[none].any()
    assert (np.abs(got_o - ref_o) <= bo).all()
    assert (np.abs(got_l - ref_l) <= bl)[~none].all()
    # again: the same bits
    o2, lse2 = c.layer.attend(c.batch, q, mask_block=mask)
    assert torch.equal(o[:c.T], o2[:c.T]) and torch.equal(lse[:c.T], lse2[:c.T])

    # the weights, from the exact sums
    width = c.width + 5
    w = torch.rand(len(seqs), hk, width, generator=c.g)
    for b, (_, kv) in enumerate(seqs):
        w[b, :, kv:] = float("nan")
    dl = torch.tensor(ref_l, dtype=torch.float32)
    full = torch.cat([dl, torch.full((2, H), float("nan"))]).cuda()
    ref_w = po.weights(qh, kp, host(dl), w.numpy(), seqs, tables, mask, 0.75)
    got = c.layer.weights(c.batch, q, full, w.cuda(), mask_block=mask, decay=0.75)
    M = float(np.sqrt((logit_parts(c, qh)[0] ** 2).sum(-1).max() * (logit_parts(c, qh)[1] ** 2).sum(-1).max())) * d ** -0.5
    big = max(M, np.abs(ref_l[~none]).max() if (~none).any() else 0.0)
    add = 2.0 ** (-24 if dtype == "f32" else -22)
    # of a weight: the logit's d additions and its scaling, the difference's rounding, the exponential; of the sum: a step a row
    rel = d * add * M + 6 * 2.0 ** -24 * big + 2.0 ** -20 + c.T * H * 2.0 ** -24
    assert (np.abs(host(got) - ref_w) <= rel * ref_w + 1e-30).all()
    wg = w.cuda()
    c.layer.weights(c.batch, q, full, wg, mask_block=mask, decay=0.75, w_out=wg)
    assert torch.equal(wg, got)
    ok(c.layer)


@pytest.mark.parametrize("dtype,H,hk,d,seqs", [
    ("bf16", 1, 1, 128, [(1, 20001)]), ("bf16", 3, 1, 128, [(1, 9000)]), ("bf16", 16, 2, 128, [(1, 20000)]),
    ("bf16", 64, 2, 128, [(1, 9001), (2, 300)]), ("bf16", 64, 1, 128, [(1, 20000)]), ("bf16", 10, 1, 128, [(12, 12000)]),
    ("f32", 2, 1, 32, [(1, 9000)]), ("f32", 24, 1, 64, [(1, 7000)]), ("f32", 8, 1, 128, [(4, 7001), (1, 1)])])
def test_attend_few_rows_of_a_long_cache(dtype, H, hk, d, seqs):
    """Items cut into as many pieces as there are CTAs, with few and many rows to join."""
    c = Paged(dtype, H, hk, d, 16, seqs, 17)
    q = c.randn(c.T, H, d, scale=3.0)
    c.to_gpu()
    o, lse = c.layer.attend(c.batch, q.cuda(), mask_block=1)
    for _ in range(3):
        o2, lse2 = c.layer.attend(c.batch, q.cuda(), mask_block=1)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    ok(c.layer)
    qh = host(q)
    ref_o, ref_l, mag = po.attend(qh, np.nan_to_num(host(c.kp)), np.nan_to_num(host(c.vp)), seqs, c.tables.numpy(), 1)
    bo, bl = attend_bounds(dtype, d, *logit_parts(c, qh), c.width, mag, ref_o)
    assert (np.abs(host(o) - ref_o) <= bo).all()
    assert (np.abs(host(lse) - ref_l) <= bl).all()


@pytest.mark.parametrize("dtype,H,hk,d,page,mask,seqs", [
    ("f32", 8, 1, 64, 16, 1, [(600, 700), (1, 3000), (0, 40), (1, 1)]),
    ("f32", 4, 4, 128, 8, 0, [(300, 300), (257, 90), (1, 1000)]),
    ("f32", 2, 1, 36, 24, 50, [(900, 64), (130, 130)]),
    ("bf16", 16, 1, 128, 16, 1, [(500, 600), (1, 5000), (0, 30)])])
def test_attend_and_weights_of_cut_blocks(dtype, H, hk, d, page, mask, seqs):
    """Chunks whose blocks of keys several CTAs share, beside streams of one token and of none."""
    test_attend_and_weights(dtype, H, hk, d, page, mask, seqs, 2.0)


def test_attend_weights_sum_to_one_over_long_caches():
    """A cache longer than any tile or page, every CTA's range cut: equal keys give the mean of V."""
    c = Paged("bf16", 8, 2, 128, 64, [(1, 9999), (300, 5000)], 2)
    c.kp.fill_(0.25)
    c.to_gpu()
    q = c.randn(c.T, 8, 128).cuda()
    o, lse = c.layer.attend(c.batch, q)
    for b, (n, kv) in enumerate(c.seqs):
        V = po.gather(np.nan_to_num(host(c.vp)), c.tables.numpy()[b], kv)
        at = 0 if b == 0 else 1
        # P = 1 for every key: the sums are exact to 2^-22 a key, the output to half a step
        assert np.abs(host(o)[at:at + n, :4] - V[0].mean(0)).max() <= 2.0 ** -8 * np.abs(V[0].mean(0)).max() + 1e-4
    w = c.layer.weights(c.batch, q, lse, torch.zeros(2, 2, 9999, device="cuda"))
    want = torch.tensor([[4.0], [300 * 4.0]]).expand(2, 2)
    # each row's weights sum to one up to its lse's rounding (2^-20 of values near 9) and the sums'
    assert torch.allclose(w.sum(-1).cpu(), want, rtol=1e-4)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_graph_replay_with_other_lengths(dtype, d):
    """A captured step replayed after lengths, pages and rows were rewritten gives what eager calls give."""
    seqs = [(3, 40), (1, 300), (40, 90)]
    c = Paged(dtype, 4, 2, d, 16, seqs, 21).to_gpu(rows=64, max_q=64, max_kv=400)
    q = c.randn(64, 4, d).cuda()
    o, lse = torch.zeros_like(q), torch.zeros(64, 4, device="cuda")
    w = torch.zeros(3, 2, 400, device="cuda")

    def step():
        c.layer.attend(c.batch, q, mask_block=1, o=o, lse=lse)
        c.layer.weights(c.batch, q, lse, w, mask_block=1, decay=0.5, w_out=w)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n, kv in (([3, 1, 40], [40, 300, 90]), ([1, 1, 1], [39, 299, 1]), ([20, 0, 17], [33, 0, 89])):
        c.batch.q_start.copy_(torch.tensor(np.cumsum([0] + n), dtype=torch.int32))
        c.batch.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        T = sum(n)
        w.zero_(), o.zero_(), lse.zero_()
        g.replay()
        a = o.clone(), lse.clone(), w.clone()
        w.zero_(), o.zero_(), lse.zero_()
        step()
        ok(c.layer)
        for x, y in zip(a, (o, lse, w)):
            assert torch.equal(x, y)
        ref, _, mag = po.attend(host(q)[:T], np.nan_to_num(host(c.kp)), np.nan_to_num(host(c.vp)), list(zip(n, kv)),
                                c.tables.numpy(), 1)
        bo, _ = attend_bounds(dtype, d, *logit_parts(c, host(q)), 400, mag, ref)
        assert (np.abs(host(o)[:T] - ref) <= bo).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 32)])
def test_bad_pages_and_lengths_are_recorded(dtype, d):
    """Pages outside the pool read as zeros; streams that break the bounds are left out; both are errors."""
    seqs = [(2, 40), (2, 70), (150, 200)]
    c = Paged(dtype, 4, 2, d, 16, seqs, 31)
    c.tables[0, 1] = 10 ** 6
    c.tables[2, 3] = -5
    c.to_gpu()
    q = c.randn(c.T, 4, d).cuda()
    o, lse = c.layer.attend(c.batch, q)
    assert c.layer.last_error() == 9 and c.layer.last_error() == 0
    kp, vp = np.nan_to_num(host(c.kp)), np.nan_to_num(host(c.vp))
    ref, _, mag = po.attend(host(q), kp, vp, seqs, c.tables.numpy(), 0)
    bo, _ = attend_bounds(dtype, d, *logit_parts(c, host(q)), c.width, mag, ref)
    assert (np.abs(host(o) - ref) <= bo).all()
    c.layer.weights(c.batch, q, lse, torch.zeros(3, 2, c.width, device="cuda"))
    assert c.layer.last_error() == 9
    before = c.kp.clone()
    c.batch.pages[:, :] = 10 ** 6
    kv = c.randn(c.T, 2, d).cuda()
    c.layer.append(c.batch, kv, kv)
    assert c.layer.last_error() == 9 and torch.equal(c.kp.nan_to_num(3.0), before.nan_to_num(3.0))
    c.batch.pages.copy_(c.tables)
    # lengths past the bound, past the table, negative; rows past the tensors
    for kv_len, q_start in (([c.width + 1, 70, 200], [0, 2, 4, 154]), ([40, -1, 200], [0, 2, 4, 154]),
                            ([40, 70, 200], [0, 2, 4, 155]), ([40, 70, 200], [0, 2, 1, 154])):
        c.batch.kv_len.copy_(torch.tensor(kv_len, dtype=torch.int32))
        c.batch.q_start.copy_(torch.tensor(q_start, dtype=torch.int32))
        c.layer.attend(c.batch, q)
        assert c.layer.last_error() == 9
        c.layer.weights(c.batch, q, lse, torch.zeros(3, 2, c.width, device="cuda"))
        assert c.layer.last_error() == 9


def test_more_new_tokens_than_keys_append():
    c = Paged("bf16", 2, 2, 128, 16, [(5, 3)], 1).to_gpu()
    k = c.randn(5, 2, 128).cuda()
    c.layer.append(c.batch, k, k)
    assert c.layer.last_error() == 9
    pg = int(c.tables[0, 0])
    assert torch.equal(c.kp[pg, :, :3], k[2:].transpose(0, 1))
    assert c.kp[pg, :, 3:].isnan().all()


# ------------------------------------------------------------------ eviction
EVICT = [  # dtype, hk, d, page, kv lengths, budget, sink, recent
    ("bf16", 12, 128, 128, [5000], 2500, 1560, 300),
    ("bf16", 2, 128, 16, [1, 99, 100, 101, 257, 1030, 0], 100, 4, 10),
    ("f32", 3, 64, 24, [300, 64, 65, 66, 5], 64, 0, 0),
    ("f32", 1, 4, 8, [70, 10], 9, 4, 5),
    ("bf16", 1, 128, 96, [400, 130], 1, 0, 0),
    ("f32", 2, 100, 136, [3000], 2999, 1, 1),
    ("f32", 2, 32, 16, [30000], 7000, 5, 7),
]


@pytest.mark.parametrize("dtype,hk,d,page,kvs,budget,sink,recent", EVICT)
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "special"])
def test_evict(dtype, hk, d, page, kvs, budget, sink, recent, kind):
    n = len(kvs)
    c = Paged(dtype, hk, hk, d, page, [(0, kv) for kv in kvs], 17, dst=[min(kv, budget) for kv in kvs])
    width = c.width + 3
    w = torch.randn(n, hk, width, generator=c.g)
    if kind == "ties":
        w = (w * 2).round()
    elif kind == "equal":
        w = torch.full_like(w, 0.5)
    elif kind == "special":
        pick = torch.randint(0, 6, w.shape, generator=c.g)
        for i, v in enumerate((float("nan"), 0.0, -0.0, float("inf"), -float("inf"))):
            w = torch.where(pick == i, torch.tensor(v), w)
    kp, vp = c.kp.clone(), c.vp.clone()
    c.to_gpu()
    kv_len, w_out, kept = c.layer.evict(c.batch, w.cuda(), c.dst.cuda(), budget=budget, sink=sink, recent=recent)
    ok(c.layer)
    assert kv_len.tolist() == [min(kv, budget) for kv in kvs]
    want_w, want_k = torch.zeros(n, hk, width), torch.full((n, hk, budget), -1, dtype=torch.int32)
    for b, kv in enumerate(kvs):
        for h in range(hk):
            ids = torch.tensor(po.keep(w[b, h].numpy(), kv, budget, sink, recent), dtype=torch.long)
            m = len(ids)
            j = torch.arange(m)
            want_k[b, h, :m], want_w[b, h, :m] = ids.int(), w[b, h, ids]
            s, t = c.tables[b].long()[ids // page], c.dst[b].long()[j // page]
            for pool in (kp, vp):
                pool[t, h, j % page] = pool[s, h, ids % page]
    assert torch.equal(kept.cpu(), want_k)
    assert torch.equal(w_out.cpu().nan_to_num(77.0), want_w.nan_to_num(77.0))
    for got, ref in ((c.kp, kp), (c.vp, vp)):
        assert torch.equal(got.cpu().nan_to_num(77.0), ref.nan_to_num(77.0))


def test_evict_refuses_pages_that_the_stream_reads():
    for page in (16, 96):
        c = Paged("f32", 1, 1, 32, page, [(0, 300), (0, 20)], 3, dst=[200, 20])
        c.dst[0, 1] = c.tables[0, 2]
        c.dst[1, 0] = 10 ** 6
        before = c.kp.clone()
        c.to_gpu()
        w = torch.rand(2, 1, 300, generator=c.g).cuda()
        _, _, kept = c.layer.evict(c.batch, w, c.dst.cuda(), budget=200)
        assert c.layer.last_error() == 9
        for b, kv in enumerate((300, 20)):
            assert torch.equal(c.kp.cpu()[c.tables[b, :-(-kv // page)].long()].nan_to_num(7.0),
                               before[c.tables[b, :-(-kv // page)].long()].nan_to_num(7.0))
        j = torch.arange(page)
        ids = kept[0, 0, :page].long().cpu()
        assert torch.equal(c.kp[int(c.dst[0, 0]), 0].cpu(), before[c.tables[0].long()[ids // page], 0, ids % page])


# ------------------------------------------------------------------ refusals that need a handle, streams, a whole run
def test_refusals_with_a_handle():
    c = Paged("bf16", 4, 2, 128, 16, [(3, 20)], 1, dst=[8]).to_gpu()
    lib, h, b = arl2.load_library(), c.layer.handle, c.batch.struct
    st, P = 0, ctypes.addressof
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    o, f = torch.zeros_like(q), torch.zeros(4096, device="cuda")
    Q, K, O, F = (t.data_ptr() for t in (q, k, o, f))
    att = lambda q=Q, ld=0, m=1, o=O, l=F, b=b: lib.arl2_paged_attend(h, b and P(b), q, ld, m, o, l, st)
    assert att() == 0 and att(l=None) == 0
    for kw in (dict(q=None), dict(o=None), dict(o=Q), dict(o=Q + 16), dict(m=-1), dict(ld=8), dict(ld=516), dict(q=Q + 8),
               dict(l=O), dict(o=c.kp.data_ptr()), dict(l=F + 2), dict(b=None), dict(o=b.kv_len)):
        assert att(**kw) == 1, kw
    edit = lambda **kw: arl2.arl2_paged_batch(*[kw.get(n, getattr(b, n)) for n, _ in b._fields_])
    assert att(b=edit(n_seqs=0)) == 0 and att(b=edit(tokens=0)) == 0 and att(b=edit(max_q=0)) == 0
    for kw in (dict(n_seqs=-1), dict(tokens=-1), dict(max_q=-1), dict(max_kv=-1), dict(pages_ld=-1), dict(q_start=None),
               dict(kv_len=None), dict(pages=None), dict(kv_len=b.kv_len + 2)):
        assert att(b=edit(**kw)) == 1, kw
    assert att(b=edit(max_kv=2 ** 31 - 1)) == 2
    wts = lambda d=1.0, i=F, o=F, ld=20, l=F + 8192: lib.arl2_paged_weights(h, P(b), Q, 0, 1, l, d, i, o, ld, st)
    assert wts() == 0
    for kw in (dict(d=float("nan")), dict(i=None), dict(o=F + 4), dict(ld=19), dict(l=None), dict(l=F), dict(o=Q)):
        assert wts(**kw) == 1, kw
    dst = c.dst.cuda()
    ev = lambda i=F, ld=20, bud=8, s=1, r=1, dp=dst.data_ptr(), dl=1, o=F + 1024, kk=F + 2048, n=F + 4096: \
        lib.arl2_paged_evict(h, P(b), i, ld, bud, s, r, dp, dl, o, kk, n, st)
    assert ev() == 0
    for kw in (dict(bud=0), dict(s=-1), dict(s=5, r=4), dict(ld=19), dict(o=F), dict(kk=F + 1024), dict(n=b.kv_len),
               dict(n=None), dict(dp=None), dict(dl=-1), dict(o=c.vp.data_ptr())):
        assert ev(**kw) == 1, kw
    ap = lambda q=None, k=K, v=K, ld=0, qo=None, prep=None: lib.arl2_paged_append(
        h, P(b), prep and P(prep), q, k, v, ld, None, qo, st)
    assert ap() == 0
    for kw in (dict(k=None), dict(q=Q, qo=O), dict(q=Q), dict(ld=8), dict(v=c.kp.data_ptr()), dict(k=K + 8)):
        assert ap(**kw) == 1, kw
    ok(c.layer)
    assert c.layer.device_bytes() > 0
    with pytest.raises(arl2.Arl2Error):
        arl2.PagedKVLayer(4, 2, 128, ABI["bf16"], c.kp, c.kp)
    with pytest.raises(ValueError):
        c.layer.attend(c.batch, q.float())
    with pytest.raises(ValueError):
        c.layer.attend(c.batch, q[:2])


def test_other_stream_and_two_layers_at_once():
    """Two layers on two streams, interleaved, give what each gives alone."""
    cs = [Paged("bf16", 4, 2, 128, 16, [(70, 700), (1, 900)], 40 + i).to_gpu() for i in range(2)]
    qs = [c.randn(c.T, 4, 128).cuda() for c in cs]
    alone = [c.layer.attend(c.batch, q, mask_block=1) for c, q in zip(cs, qs)]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in cs]
    outs = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(ss[i]):
                outs[i].append(cs[i].layer.attend(cs[i].batch, qs[i], mask_block=1))
    torch.cuda.synchronize()
    for i in range(2):
        ok(cs[i].layer)
        for o, lse in outs[i]:
            assert torch.equal(o, alone[i][0]) and torch.equal(lse, alone[i][1])


@pytest.mark.parametrize("dtype,H,hk,d", [("bf16", 4, 2, 128), ("f32", 4, 2, 32)])
def test_bounded_stream(dtype, H, hk, d):
    """append -> attend -> weights -> evict, three rounds of two streams: the caches stay bounded, every step as the
    oracle has it on the same cache."""
    page, budget, chunk = 16, 48, 20
    c = Paged(dtype, H, hk, d, page, [(chunk, chunk), (chunk, chunk)], 8, spare=40)
    pool_pages = c.kp.shape[0]
    c.kp.fill_(float("nan")), c.vp.fill_(float("nan"))
    c.kp, c.vp = c.kp.cuda(), c.vp.cuda()
    layer = arl2.PagedKVLayer(H, hk, d, ABI[dtype], c.kp, c.vp)
    w_q, w_k = (1 + 0.1 * c.randn(d)).to(TORCH[dtype]).cuda(), c.randn(d).cuda()
    prep = arl2.QKPrep([d // 2, d // 4], w_q=w_q, w_k=w_k)
    half = pool_pages // 2
    banks = [[range(0, half // 2), range(half // 2, half)], [range(half, half + half // 2), range(half + half // 2, 2 * half)]]
    table = lambda i: torch.tensor([list(r)[:half // 2] for r in banks[i]], dtype=torch.int32).cuda()
    kv = torch.zeros(2, dtype=torch.int32, device="cuda")
    w = torch.zeros(2, hk, budget + chunk, device="cuda")
    q_start = torch.tensor([0, chunk, 2 * chunk], dtype=torch.int32).cuda()
    for rnd in range(5):
        kv = kv + chunk
        pages = table(rnd % 2)
        batch = arl2.PagedBatch(q_start, kv, pages, tokens=2 * chunk, max_q=chunk, max_kv=budget + chunk)
        rows = c.randn(2 * chunk, (H + 2 * hk) * d).cuda()
        q, k, v = (rows[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, H), (H, H + hk), (H + hk, H + 2 * hk)))
        pos = (torch.arange(chunk).repeat(2)[:, None] + torch.tensor([[100 * rnd, 7]])).int().cuda()
        qt = layer.append(batch, k, v, q=q, prep=prep, pos=pos)
        o, lse = layer.attend(batch, qt, mask_block=4)
        w2 = layer.weights(batch, qt, lse, w, mask_block=4, decay=0.9)
        seqs = [(chunk, int(x)) for x in kv]
        kp, vp, tb = np.nan_to_num(host(c.kp)), np.nan_to_num(host(c.vp)), pages.cpu().numpy()
        ref, _, mag = po.attend(host(qt), kp, vp, seqs, tb, 4)
        bo, _ = attend_bounds(dtype, d, *logit_parts(c, host(qt)), budget + chunk, mag, ref)
        assert (np.abs(host(o) - ref) <= bo).all()
        ref_w = po.weights(host(qt), kp, host(lse), host(w), seqs, tb, 4, np.float32(0.9))
        assert np.allclose(host(w2), ref_w, rtol=1e-4)
        for b in range(2):  # each of the rows hands out weight one in all (bounds of lse and of the sums above)
            gain = host(w2)[b].sum() - 0.9 * host(w)[b, :, :int(kv[b]) - chunk].sum()
            assert abs(gain - chunk * H) <= 1e-3 * chunk * H
        n, w, kept = layer.evict(batch, w2, table((rnd + 1) % 2), budget=budget, sink=2, recent=8)
        for b in range(2):
            for h in range(hk):
                ids = po.keep(w2[b, h].cpu().numpy(), int(kv[b]), budget, 2, 8)
                assert kept[b, h, :len(ids)].tolist() == ids
        kv = n
        assert kv.tolist() == [min(budget, (rnd + 1) * chunk)] * 2 if rnd < 3 else [budget] * 2
    assert layer.last_error() == 0


def test_ragged_calls_back_to_back():
    """Many launches in a row over short and long streams, single tokens and chunks, give the first one's bits."""
    seqs = [(1, n) for n in (1, 2, 17, 64, 65, 127, 129, 200, 640, 1000, 2049)] + [(40, 300), (1, 3000), (17, 17), (150, 1200)]
    c = Paged("bf16", 16, 2, 128, 16, seqs, 77).to_gpu()
    q = c.randn(c.T, 16, 128).cuda()
    first = c.layer.attend(c.batch, q, mask_block=1)
    w = torch.zeros(len(seqs), 2, c.width, device="cuda")
    w0 = c.layer.weights(c.batch, q, first[1], w, mask_block=1)
    outs = [(c.layer.attend(c.batch, q, mask_block=1), c.layer.weights(c.batch, q, first[1], w, mask_block=1))
            for _ in range(200)]
    ok(c.layer)
    for (o, lse), x in outs:
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1]) and torch.equal(x, w0)


@pytest.mark.parametrize("mask", [0, 64])
def test_chunks_on_a_pool_larger_than_l2(mask):
    """Several blocks of rows on one key head: CTAs begin inside their key ranges (the pool does not fit L2)."""
    seqs = [(700, 2500), (300, 300), (1, 500), (513, 1111)]
    c = Paged("bf16", 4, 2, 128, 64, seqs, 9, spare=2300)
    c.to_gpu()
    assert 2 * c.kp.numel() * 2 > torch.cuda.get_device_properties(0).L2_cache_size
    q = c.randn(c.T, 4, 128).cuda()
    o, lse = c.layer.attend(c.batch, q, mask_block=mask)
    ok(c.layer)
    used = torch.unique(c.tables[c.tables >= 0]).long()
    kp, vp = np.zeros(c.kp.shape, np.float32), np.zeros(c.vp.shape, np.float32)
    kp[used], vp[used] = np.nan_to_num(host(c.kp[used])), np.nan_to_num(host(c.vp[used]))
    rows = np.r_[0:2, 127:130, 255:257, 511:513, 640:645, 699:705, 999:1003, 1250:1270, c.T - 3:c.T]  # of every block's kind
    ref, ref_l, mag = po.attend(host(q), kp, vp, seqs, c.tables.numpy(), mask, rows=set(rows.tolist()))
    bo, bl = attend_bounds("bf16", 128, host(q), kp[used].astype(np.float64), c.width, mag, ref)
    assert (np.abs(host(o) - ref) <= bo)[rows].all() and (np.abs(host(lse) - ref_l) <= bl)[rows].all()
