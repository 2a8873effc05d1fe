"""The paged-cache calls at the edge of what their documentation allows: other
streams and replays, waits that run out, streams that are left out, queries
that are no numbers, bounds that are far above the work."""
import ctypes

import numpy as np
import pytest
import torch

from hybrid_linear_attention_arl2_b200 import arl2, build
from oracle import paged_oracle as po
from tests.paged_util import ABI, TORCH, Paged, attend_bounds, host

pytestmark = pytest.mark.gpu
ERR_TIMEOUT, ERR_PAGE = 5, 9
DELAY = 200_000_000  # clocks, a tenth of a second


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    arl2.load_library()


# ------------------------------------------------------------------ errors
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 32)])
def test_last_error_waits_for_a_replay_on_another_stream(dtype, d):
    """A replay runs on a stream that the handle never saw; its error is there when last_error returns."""
    c = Paged(dtype, 4, 2, d, 16, [(3, 40), (1, 300)], 3).to_gpu()
    q = c.randn(c.T, 4, d).cuda()
    o, lse = c.layer.attend(c.batch, q)
    good = o.clone(), lse.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.layer.attend(c.batch, q, o=o, lse=lse)
    side = torch.cuda.Stream()
    c.batch.pages[0, 1] = 10 ** 6
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
        g.replay()
    assert c.layer.last_error() == ERR_PAGE and c.layer.last_error() == 0
    c.batch.pages.copy_(c.tables)
    torch.cuda.synchronize()
    for _ in range(20):  # right after an error was cleared, on a stream that does not order with the default one
        with torch.cuda.stream(side):
            c.batch.pages[0, 1] = -1
            c.layer.attend(c.batch, q)
            c.batch.pages.copy_(c.tables)
            assert c.layer.last_error() == ERR_PAGE
            o2, lse2 = c.layer.attend(c.batch, q)
            assert torch.equal(o2, good[0]) and torch.equal(lse2, good[1])
    assert c.layer.last_error() == 0


def test_waits_that_run_out():
    """A batch of so many empty streams that finding a CTA's work takes far longer than the limit: the roles that wait
    for it give up, the kernels return and say so, and after last_error the handle's next results are those of a fresh
    one."""
    c = Paged("bf16", 16, 2, 128, 16, [(1, 900), (200, 700), (40, 300)], 19).to_gpu()
    empty = 20000
    q_start = torch.cat([c.q_start, c.q_start[-1:].expand(empty)]).cuda()
    kv_len = torch.cat([c.kv_len, torch.zeros(empty, dtype=torch.int32)]).cuda()
    pages = torch.cat([c.tables, torch.full((empty, c.tables.shape[1]), -1, dtype=torch.int32)]).cuda()
    long = arl2.PagedBatch(q_start, kv_len, pages, tokens=c.T, max_q=200, max_kv=900)
    q = c.randn(c.T, 16, 128).cuda()
    w = torch.zeros(3 + empty, 2, 900, device="cuda")
    o, lse = c.layer.attend(long, q, mask_block=1)
    ref = o, lse, c.layer.weights(long, q, lse, w, mask_block=1)
    assert c.layer.last_error() == 0
    for limit in (1000, 10000, 100000, 1000000):
        for call in (lambda: c.layer.attend(long, q, mask_block=1),
                     lambda: c.layer.weights(long, q, lse, w, mask_block=1)):
            arl2.arl2_paged_set_wait_limit(c.layer.handle, limit)
            call()
            status = c.layer.last_error()
            assert status in (0, ERR_TIMEOUT) and c.layer.last_error() == 0
            assert status == ERR_TIMEOUT or limit > 1000
            arl2.arl2_paged_set_wait_limit(c.layer.handle, 0)
            o, l2 = c.layer.attend(long, q, mask_block=1)
            got = o, l2, c.layer.weights(long, q, lse, w, mask_block=1)
            assert c.layer.last_error() == 0
            for x, y in zip(got, ref):
                assert torch.equal(x, y)


def test_a_new_layer_is_ready_on_any_stream():
    """What a layer's creation clears is clear when it returns: a call on another stream records its error after it."""
    c = Paged("bf16", 4, 2, 128, 16, [(3, 40), (1, 300)], 4).to_gpu()
    q = c.randn(c.T, 4, 128).cuda()
    c.batch.pages[0, 1] = 10 ** 6
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        torch.cuda._sleep(DELAY)
        layer = arl2.PagedKVLayer(4, 2, 128, arl2.ARL2_BF16, c.kp, c.vp)
    with torch.cuda.stream(b):
        layer.attend(c.batch, q)
    torch.cuda.synchronize()
    assert layer.last_error() == ERR_PAGE


# ------------------------------------------------------------------ streams that are left out
@pytest.mark.parametrize("bad", ["negative", "bound", "table"])
def test_eviction_empties_a_stream_that_it_leaves_out(bad):
    """A stream whose length breaks a bound has no keys afterwards, whatever the outputs' memory held; the others are
    cut as ever."""
    kvs, budget = [30, 90, 25], 20
    c = Paged("f32", 2, 2, 32, 16, [(0, kv) for kv in kvs], 6, dst=[20, 20, 20]).to_gpu()
    w = torch.rand(3, 2, c.width + 7, generator=c.g).cuda()
    want = [x.clone() for x in c.layer.evict(c.batch, w, c.dst.cuda(), budget=budget, sink=2, recent=3)]
    assert c.layer.last_error() == 0
    c.batch.kv_len[1] = {"negative": -3, "bound": 91, "table": 97}[bad]
    if bad == "table":
        c.batch.struct.max_kv = c.width + 7
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    dirty = [torch.full((3, 2, c.width + 7), 5.0, device="cuda"), torch.full((3, 2, budget), 5, dtype=torch.int32, device="cuda"),
             torch.full((3,), 5, dtype=torch.int32, device="cuda")]
    del dirty
    kv_len, w_out, kept = c.layer.evict(c.batch, w, c.dst.cuda(), budget=budget, sink=2, recent=3)
    assert c.layer.last_error() == ERR_PAGE
    assert kv_len.tolist() == [20, 0, 20]
    assert (kept[1] == -1).all() and not w_out[1].any()
    for got, ref in zip((kv_len, w_out, kept), want):
        assert torch.equal(got[[0, 2]], ref[[0, 2]])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 32)])
def test_fading_records_streams_that_it_leaves_out(dtype, d):
    """Weights without new tokens fade; a stream that breaks a bound is left as it was, and said so."""
    c = Paged(dtype, 4, 2, d, 16, [(0, 40), (0, 70)], 5).to_gpu(max_q=0)
    q, lse = c.randn(0, 4, d).cuda(), torch.zeros(0, 4, device="cuda")
    w = torch.rand(2, 2, c.width + 3, generator=c.g).cuda()
    want = w * 0.5
    want[0, :, 40:], want[1, :, 70:] = 0, 0
    assert torch.equal(c.layer.weights(c.batch, q, lse, w, decay=0.5), want)
    assert c.layer.last_error() == 0
    c.batch.kv_len[0] = c.width + 1
    out = torch.full_like(w, 3.0)
    c.layer.weights(c.batch, q, lse, w, decay=0.5, w_out=out)
    assert c.layer.last_error() == ERR_PAGE
    assert (out[0] == 3).all() and torch.equal(out[1], want[1])


# ------------------------------------------------------------------ an explicit stream
@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("op", ["prep", "append", "attend", "weights", "evict"])
def test_outputs_belong_to_the_stream_that_writes_them(op, raw):
    """With stream=, what a call allocates is not memory that the current stream has still to write."""
    c = Paged("bf16", 4, 2, 128, 16, [(20, 60), (1, 300)], 8, dst=[40, 40]).to_gpu()
    q, k = c.randn(c.T, 4, 128).cuda(), c.randn(c.T, 2, 128).cuda()
    w, dst = torch.rand(2, 2, 300, generator=c.g).cuda(), c.dst.cuda()
    prep, pos = arl2.QKPrep([128]), torch.arange(c.T, dtype=torch.int32)[:, None].cuda()
    lse = c.layer.attend(c.batch, q)[1]
    call = {"prep": lambda **s: arl2.qk_norm_rope(prep, q, k, pos, **s),
            "append": lambda **s: (c.layer.append(c.batch, k, k, q=q, prep=prep, pos=pos, **s),),
            "attend": lambda **s: c.layer.attend(c.batch, q, **s),
            "weights": lambda **s: (c.layer.weights(c.batch, q, lse, w, **s),),
            "evict": lambda **s: c.layer.evict(c.batch, w, dst, budget=40, **s)}[op]
    want = [x.clone() for x in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(DELAY)
    for x in [torch.empty_like(x) for x in want]:  # freed, and yet to be written by the current stream
        x.fill_(3)
    del x
    got = call(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    for x, ref in zip(got, want):
        assert torch.equal(x, ref)
    assert c.layer.last_error() == 0


# ------------------------------------------------------------------ queries that are no numbers
@pytest.mark.parametrize("dtype,H,hk,d,seqs", [
    ("bf16", 4, 2, 128, [(1, 9000), (300, 700), (3, 40), (70, 70)]),
    ("bf16", 16, 1, 128, [(1, 20000), (30, 500)]),
    ("f32", 4, 2, 64, [(1, 5000), (100, 300), (3, 40)])])
def test_rows_that_are_no_numbers(dtype, H, hk, d, seqs):
    """A query of NaN has outputs and a logarithm of NaN, not those of a row that sees no key; its neighbours keep
    their bits, whole items and cut ones."""
    c = Paged(dtype, H, hk, d, 16, seqs, 23).to_gpu()
    q = c.randn(c.T, H, d).cuda()
    o, lse = c.layer.attend(c.batch, q, mask_block=1)
    bad = torch.zeros(c.T, H, dtype=torch.bool)
    for t, h in ((0, 1), (c.T // 2, 0), (c.T // 2, H - 1), (c.T - 1, H // 2)):
        bad[t, h] = True
    bad = bad.cuda()
    q2 = q.masked_fill(bad[..., None], float("nan"))
    o2, lse2 = c.layer.attend(c.batch, q2, mask_block=1)
    assert c.layer.last_error() == 0
    assert o2[bad].isnan().all() and lse2[bad].isnan().all()
    assert torch.equal(o2[~bad], o[~bad]) and torch.equal(lse2[~bad], lse[~bad])


# ------------------------------------------------------------------ bounds far above the work
MIXED = [  # dtype, heads, kv_heads, d, chunk, its keys, streams of one token
    ("bf16", 8, 1, 128, 1500, 1700, 200),
    ("f32", 8, 2, 32, 700, 900, 150),
]


def check_rows(c, q, o, lse, mask, rows):
    used = c.tables[c.tables >= 0].long()
    kp, vp = np.nan_to_num(host(c.kp)), np.nan_to_num(host(c.vp))
    ref, ref_l, mag = po.attend(host(q)[:c.T], kp, vp, c.seqs, c.tables.numpy(), mask, rows=set(rows.tolist()))
    bo, bl = attend_bounds(c.dtype, c.d, host(q)[:c.T], kp[used.numpy()].reshape(-1, c.d), c.width, mag, ref)
    assert (np.abs(host(o)[:c.T] - ref) <= bo)[rows].all() and (np.abs(host(lse)[:c.T] - ref_l) <= bl)[rows].all()


@pytest.mark.parametrize("dtype,H,hk,d,chunk,keys,tokens", MIXED)
@pytest.mark.parametrize("place", ["first", "last", "between"])
def test_single_tokens_beside_a_chunk(dtype, H, hk, d, chunk, keys, tokens, place):
    """Many streams of one token, some of none, beside one of many blocks of rows: attention, and the weights' sums."""
    seqs = [(1 if i % 7 else 0, 1 + (37 * i) % 90) for i in range(tokens)]
    seqs.insert({"first": 0, "last": tokens, "between": tokens // 3}[place], (chunk, keys))
    c = Paged(dtype, H, hk, d, 16, seqs, 29).to_gpu()
    q = c.randn(c.T, H, d).cuda()
    o, lse = c.layer.attend(c.batch, q, mask_block=1)
    at = sum(n for n, _ in seqs[:seqs.index((chunk, keys))])
    rows = np.unique(np.clip(np.r_[0:c.T:11, at - 2:at + 40, at + chunk - 40:at + chunk + 3, at + 250:at + 262], 0, c.T - 1))
    check_rows(c, q, o, lse, 1, rows)
    w = c.layer.weights(c.batch, q, lse, torch.zeros(len(seqs), hk, c.width, device="cuda"), mask_block=1)
    # each row of a key head hands out weight one, up to its lse's rounding and the sums'
    want = torch.tensor([float(n * (H // hk)) for n, _ in seqs])[:, None].expand(-1, hk)
    assert torch.allclose(w.sum(-1).cpu(), want, rtol=1e-4)
    assert c.layer.last_error() == 0


@pytest.mark.parametrize("dtype,H,hk,d", [("bf16", 64, 8, 128), ("f32", 64, 8, 16)])
def test_bounds_far_above_the_work(dtype, H, hk, d):
    """1024 streams of at most a few tokens, with bounds that would allow each 8192 on 131072 keys (2^31 tiles of keys
    and more in all): what a graph for chunks meets when it replays single tokens."""
    seqs = [(1 + (i % 97 == 5) * 2, 3 + i % 29) for i in range(1024)]
    c = Paged(dtype, H, hk, d, 16, seqs, 31).to_gpu(max_q=8192, max_kv=131072)
    q = c.randn(c.T, H, d).cuda()
    o, lse = c.layer.attend(c.batch, q, mask_block=1)
    rows = np.r_[0:12, 500:520, c.T - 9:c.T]
    check_rows(c, q, o, lse, 1, rows)
    tight = arl2.PagedBatch(c.batch.q_start, c.batch.kv_len, c.batch.pages, tokens=c.T, max_q=3, max_kv=c.width)
    o2, lse2 = c.layer.attend(tight, q, mask_block=1)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # (no stream is long enough for its tiles to be cut)
    assert c.layer.last_error() == 0


@pytest.mark.parametrize("dtype,H,hk,d", [("bf16", 64, 8, 128), ("f32", 64, 8, 16)])
def test_weights_with_bounds_far_above_the_work(dtype, H, hk, d):
    """The weights of such a batch, whose bounds' product is past 2^31 units."""
    seqs = [(1 + (i % 97 == 5) * 2, 3 + i % 29) for i in range(256)]
    c = Paged(dtype, H, hk, d, 16, seqs, 33).to_gpu(max_q=1 << 20, max_kv=4096)
    q = c.randn(c.T, H, d).cuda()
    tight = arl2.PagedBatch(c.batch.q_start, c.batch.kv_len, c.batch.pages, tokens=c.T, max_q=3, max_kv=c.width)
    lse = c.layer.attend(tight, q, mask_block=1)[1]
    w = torch.rand(len(seqs), hk, 4096, generator=c.g).cuda()
    got = c.layer.weights(c.batch, q, lse, w, mask_block=1, decay=0.5)
    ref = c.layer.weights(tight, q, lse, w, mask_block=1, decay=0.5)
    assert torch.equal(got, ref) and c.layer.last_error() == 0
    want = torch.tensor([float(n * (H // hk)) for n, _ in seqs])[:, None].expand(-1, hk)
    faded = torch.stack([0.5 * w[b, :, :kv].sum(-1) for b, (_, kv) in enumerate(seqs)]).cpu()
    assert torch.allclose(got.sum(-1).cpu() - faded, want, rtol=1e-3)


# ------------------------------------------------------------------ runs
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 32)])
def test_a_stream_stays_at_its_budget(dtype, d):
    """Chunk after chunk through append, attention, weights and eviction: the lengths grow to the budget and stay."""
    H, hk, page, budget, chunk = 4, 2, 16, 48, 20
    c = Paged(dtype, H, hk, d, page, [(chunk, chunk), (chunk, chunk)], 8, spare=20).to_gpu(max_kv=budget + chunk)
    each = -(-(budget + chunk) // page)
    tables = [torch.arange(i * 2 * each, (i + 1) * 2 * each, dtype=torch.int32).view(2, each).cuda() for i in range(2)]
    kv, w = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, hk, budget + chunk, device="cuda")
    for rnd in range(6):
        kv += chunk
        batch = arl2.PagedBatch(c.batch.q_start, kv, tables[rnd % 2], tokens=2 * chunk, max_q=chunk, max_kv=budget + chunk)
        k, v, q = c.randn(2 * chunk, hk, d).cuda(), c.randn(2 * chunk, hk, d).cuda(), c.randn(2 * chunk, H, d).cuda()
        c.layer.append(batch, k, v)
        w = c.layer.weights(batch, q, c.layer.attend(batch, q, mask_block=1)[1], w, mask_block=1)
        kv, w, kept = c.layer.evict(batch, w, tables[(rnd + 1) % 2], budget=budget, sink=2, recent=8)
        n = min(budget, (rnd + 1) * chunk)
        assert kv.tolist() == [n, n]
        assert (kept[:, :, :n] >= 0).all() and (kept[:, :, n:] == -1).all()
        assert (kept[:, :, 1:n] > kept[:, :, :n - 1]).all()
    assert c.layer.last_error() == 0


def test_norm_and_rotation_before_a_hybrid_layer():
    """A fused row turned in place, then read by the hybrid layer through its pitch: what a block with head norms and
    positions does.  Equal to turned copies, contiguous, bit by bit."""
    from hybrid_linear_attention_arl2_b200 import workloads as W
    from tests.gpu_util import make_layer, small_config
    cfg = small_config(B=2, H=3, L=200)
    layer, _ = make_layer(cfg, W.Workload(cfg))
    B, L, H, d = cfg.batch, cfg.tokens, cfg.heads, 128
    g = torch.Generator().manual_seed(3)
    rows = torch.randn(B * L, 3 * H * d, generator=g).to(torch.bfloat16).cuda()
    w_q, w_k = ((1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    pos = torch.stack([torch.arange(B * L) // L, torch.arange(B * L) % L // 20, torch.arange(B * L) % 20], 1).int().cuda()
    prep = arl2.QKPrep([44, 42, 42], w_q=w_q, w_k=w_k)
    q, k, v = (rows[:, i * H * d:(i + 1) * H * d].unflatten(1, (H, d)) for i in range(3))
    turned = arl2.qk_norm_rope(prep, q, k, pos)
    ref = layer.query(*(x.contiguous().view(B, L, H, d) for x in (*turned, v)))
    arl2.qk_norm_rope(prep, q, k, pos, q_out=q, k_out=k)
    o = torch.empty_like(ref)
    arl2.arl2_frame_query_strided(layer.handle, q, k, v, rows.shape[1], o)
    assert layer.last_error() == 0 and torch.equal(o, ref)
    layer.close()
