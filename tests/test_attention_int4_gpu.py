"""Attention over a 4-bit KV cache against fp64 attention over the values the
cache holds; the bound of each element is derived from the kernel's roundings
(int4_util.attend)."""
import numpy as np
import pytest
import torch

import synthetic as syn
import weight_shared_looped_b200 as tl

from int4_util import Cache, attend

pytestmark = pytest.mark.gpu


def _kv(lanes, H, ctx, hd, seed):
    k = syn.normal((lanes, H, ctx, hd), 1.0, seed, "a4.k")
    k += np.where(np.abs(syn.normal((H, 1, hd), 1.0, seed, "a4.off")) > 1.8, 3.0, 0.0)
    return k.astype(np.float16), syn.normal((lanes, H, ctx, hd), 1.0, seed, "a4.v").astype(np.float16)


def _q(rows, heads, hd, seed, std=1.0):
    return syn.normal((rows, heads, hd), std, seed, "a4.q").astype(np.float16)


def _run(q, cache, lens, n_q, window, out=None):
    rows, heads, hd = q.shape
    tq = torch.from_numpy(q.reshape(rows, heads * hd)).cuda()
    if out is None:
        out = torch.full((rows, heads * hd), float("nan"), dtype=torch.float16, device="cuda")
    tl.tl_attention_int4(tq, *cache.t, torch.tensor(lens, dtype=torch.int32, device="cuda"), out,
                         n_q=n_q, window=window)
    torch.cuda.synchronize()
    return out.cpu().numpy().reshape(rows, heads, hd)


class TwoByTurns:
    """The lanes 0, 1, 0, 1, .. of a cache of two."""

    def __init__(self, two):
        self.K, self.V = lambda b: two.K(b % 2), lambda b: two.V(b % 2)


def _check(got, q, cache, lens, n_q, window):
    for b, length in enumerate(lens):
        rows = slice(b * n_q, (b + 1) * n_q)
        ref, tol = attend(q[rows].astype(np.float64), cache.K(b), cache.V(b), length, n_q, window)
        y = got[rows].astype(np.float64)
        assert np.isfinite(y).all(), (b, length)
        over = np.abs(y - ref) - tol
        assert over.max() <= 0, (b, length, over.max(), np.unravel_index(over.argmax(), over.shape))


CASES = [
    # H, group, hd, ctx, n_q, window, lens, q_std
    (1, 1, 64, 1, 1, 0, [1], 1.0),
    (1, 1, 128, 16, 1, 0, [1, 2, 15, 16], 1.0),
    (2, 1, 128, 17, 1, 0, [17, 16, 0, 1], 1.0),
    (4, 1, 64, 63, 1, 0, [63, 62, 33], 4.0),
    (16, 1, 128, 384, 1, 0, [384, 257], 1.0),
    (2, 4, 128, 130, 1, 0, [130, 128, 65], 1.0),
    (1, 8, 64, 200, 1, 0, [200, 111], 2.0),
    (2, 3, 64, 90, 5, 0, [90, 7, 5, 4, 1, 0], 1.0),       # 15 queries a head; rows that see nothing
    (1, 16, 128, 70, 8, 0, [70, 33, 8, 3], 1.0),          # 128 queries a head
    (3, 1, 128, 100, 2, 1, [100, 50, 2, 1], 1.0),         # window 1: only itself
    (2, 2, 64, 300, 3, 40, [300, 41, 40, 39, 3], 1.0),
    (2, 1, 128, 300, 8, 17, [300, 16, 160], 8.0),
    (2, 1, 64, 1000, 4, 1000, [1000, 999], 1.0),
    (1, 2, 128, 2112, 1, 0, [2112, 2049], 8.0),
    (2, 1, 128, 9000, 1, 0, [9000], 4.0),
    (1, 4, 64, 33000, 2, 20000, [33000], 2.0),
]


@pytest.mark.parametrize("H,group,hd,ctx,n_q,window,lens,q_std", CASES)
def test_matches_fp64(H, group, hd, ctx, n_q, window, lens, q_std):
    lanes = len(lens)
    cache = Cache(*_kv(lanes, H, ctx, hd, ctx))
    q = _q(lanes * n_q, H * group, hd, ctx + 1, q_std)
    got = _run(q, cache, lens, n_q, window)
    _check(got, q, cache, lens, n_q, window)
    for b, length in enumerate(lens):
        for i in range(n_q):
            if length - n_q + i < 0:
                assert (got[b * n_q + i] == 0).all()


def test_length_above_the_cache_counts_as_the_cache():
    cache = Cache(*_kv(1, 2, 20, 64, 7))
    q = _q(1, 2, 64, 8)
    assert np.array_equal(_run(q, cache, [1 << 30], 1, 0), _run(q, cache, [20], 1, 0))
    assert (_run(q, cache, [-5], 1, 0) == 0).all()


@pytest.mark.parametrize("window", [100, 101, 2 ** 31 - 1])
def test_windows_beyond_the_context_are_no_windows(window):
    """Also where some of the queries see nothing."""
    cache = Cache(*_kv(2, 2, 100, 64, 23))
    q = _q(10, 2, 64, 24)
    lens = [100, 3]
    got = _run(q, cache, lens, 5, window)
    assert np.array_equal(got, _run(q, cache, lens, 5, 0))
    _check(got, q, cache, lens, 5, 0)


@pytest.mark.parametrize("lanes,H,group,hd,ctx,n_q,window", [
    (1, 2, 1, 128, 8191, 1, 0), (1, 2, 1, 128, 8192, 1, 0), (1, 1, 8, 64, 8193, 3, 0), (2, 3, 2, 128, 9000, 5, 700),
    (1, 1, 1, 64, 40001, 1, 0),
])
def test_long_contexts_go_through_a_workspace(lanes, H, group, hd, ctx, n_q, window):
    """From 8192 positions a split may be wider than a cluster; lengths from none to
    all of the cache, a workspace given and one allocated by the binding."""
    k, v = _kv(1, H, ctx, hd, 25)
    cache = Cache(np.repeat(k, lanes, 0), np.repeat(v, lanes, 0))
    q = _q(lanes * n_q, H * group, hd, 26, 2.0)
    need = tl.tl_attention_int4_workspace_bytes(*cache.t, n_q, H * group)
    assert (need > 0) == (ctx >= 8192)
    for lens in ([ctx] * lanes, [ctx - 1, 7000][:lanes], [1, 0][:lanes], [33, 5][:lanes]):
        got = _run(q, cache, lens, n_q, window)
        _check(got, q, cache, lens, n_q, window)
        ws = torch.full((max(need, 1) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        out = torch.zeros(q.shape[0], H * group * hd, dtype=torch.float16, device="cuda")
        tl.tl_attention_int4(torch.from_numpy(q.reshape(q.shape[0], -1)).cuda(), *cache.t,
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), out, n_q=n_q, window=window,
                             workspace=ws[:max(need, 1)])
        assert np.array_equal(out.cpu().numpy().reshape(got.shape), got)
        assert (ws[max(need, 1):] == 0xFF).all()


@pytest.mark.parametrize("hd", [64, 128])
def test_equal_keys_give_the_mean(hd):
    """Constant groups have scale 0: the value is the zero point, and equal keys
    weigh equally whatever the query."""
    ctx, n = 100, 77
    k = np.full((1, 1, ctx, hd), 1.5, np.float16)
    _, v = _kv(1, 1, ctx, hd, 9)
    cache = Cache(k, v)
    assert (cache.kp[..., 0] == 0).all()
    q = _q(1, 1, hd, 10)
    _check(_run(q, cache, [n], 1, 0), q, cache, [n], 1, 0)


def _spoil(cache, lane, head, p, value):
    cache.kp[lane, head, p] = value
    cache.vp[lane, head, p] = value


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf, 65504.0])
def test_unseen_entries_have_no_effect(value):
    """Entries behind a lane's length, before its window, after a query's own
    position, or of another lane may hold anything."""
    H, hd, ctx, n_q, window = 2, 128, 90, 3, 30
    lens = [70, 35, 2]
    clean = Cache(*_kv(3, H, ctx, hd, 11))
    q = _q(9, 2 * H, hd, 12)
    want = _run(q, clean, lens, n_q, window)
    _check(want, q, clean, lens, n_q, window)
    dirty = Cache(*_kv(3, H, ctx, hd, 11))
    for b, length in enumerate(lens):
        for p in list(range(length, ctx)) + list(range(max(0, length - n_q + 1 - window))):
            _spoil(dirty, b, slice(None), p, value)
    dirty.upload()
    assert np.array_equal(_run(q, dirty, lens, n_q, window), want)
    # the last token's own entry and the oldest: seen by some of the lane's queries, not by others
    _spoil(dirty, 0, slice(None), 69, value)
    _spoil(dirty, 0, slice(None), 70 - n_q + 1 - window, value)
    dirty.upload()
    got = _run(q, dirty, lens, n_q, window)
    assert np.array_equal(got[3:], want[3:])                        # the other lanes
    assert np.array_equal(got[1], want[1])                          # query 1 sees neither
    if np.isnan(value):
        assert np.isnan(got[0]).all() and np.isnan(got[2]).all()    # query 0 the oldest, query 2 its own


def test_a_seen_nan_reaches_only_its_lane_and_head():
    H, hd, ctx = 3, 64, 50
    cache = Cache(*_kv(2, H, ctx, hd, 13))
    q = _q(2, H, hd, 14)
    want = _run(q, cache, [50, 50], 1, 0)
    _spoil(cache, 0, 1, 20, np.nan)
    cache.upload()
    got = _run(q, cache, [50, 50], 1, 0)
    assert np.isnan(got[0, 1]).all()
    got[0, 1] = want[0, 1]
    assert np.array_equal(got, want)


@pytest.mark.parametrize("ctx,lanes,H,group,hd,n_q", [
    (100, 80, 2, 1, 64, 1), (200, 90, 1, 2, 128, 3), (130, 40, 1, 1, 128, 1), (512, 100, 1, 1, 128, 1),
    (700, 80, 1, 4, 128, 1), (2112, 75, 1, 1, 64, 1), (2112, 37, 4, 1, 128, 2), (2112, 90, 1, 8, 128, 1),
    (2112, 25, 2, 3, 64, 1), (2112, 19, 2, 8, 128, 1), (1100, 300, 2, 1, 128, 1), (1100, 150, 2, 8, 64, 1),
    (8200, 80, 1, 1, 128, 1), (9000, 20, 1, 1, 64, 1), (16500, 38, 1, 16, 64, 1),
])
def test_any_number_of_lanes(ctx, lanes, H, group, hd, n_q):
    """However the work is spread (one CTA a lane and head, clusters, a workspace),
    lanes of the same cache and length give the same bits, and the right ones."""
    two = Cache(*_kv(2, H, ctx, hd, 27))
    pick = np.arange(lanes) % 2
    at = torch.from_numpy(pick).cuda()
    cache = [t[at] for t in two.t]
    base = _q(6 * n_q, H * group, hd, 28, 2.0).reshape(6, n_q, H * group, hd)
    kind = np.arange(lanes) % 6                        # lanes b and b + 6 are alike
    q = base[kind].reshape(lanes * n_q, H * group, hd)
    lens = np.array([ctx, 1, 0, ctx - 37, ctx // 2, ctx - 1], np.int32)[kind]
    x = torch.from_numpy(q.reshape(lanes * n_q, -1)).cuda()
    out = torch.full_like(x, 9.0)
    tl.tl_attention_int4(x, *cache, torch.from_numpy(lens).cuda(), out, n_q=n_q)
    got = out.cpu().numpy().reshape(lanes, n_q, H * group, hd)
    for b in range(6, lanes):
        assert np.array_equal(got[b], got[b % 6]), b
    for b in range(0, 6, 2):
        six = slice(b * n_q, (b + 2) * n_q)
        _check(got[b:b + 2].reshape(2 * n_q, H * group, hd), q[six], two, lens[b:b + 2].tolist(), n_q, 0)
    # what lies behind a lane's last entry may be anything
    behind = torch.arange(ctx, device="cuda") >= torch.from_numpy(lens).cuda()[:, None]
    for i in (1, 3):
        cache[i][behind[:, None].expand(-1, H, -1)] = float("nan")
        cache[i - 1][behind[:, None].expand(-1, H, -1)] = -1
    again = torch.full_like(x, 9.0)
    tl.tl_attention_int4(x, *cache, torch.from_numpy(lens).cuda(), again, n_q=n_q)
    assert torch.equal(again, out)
    # a window: tiles in front of it are skipped, the first one is cut
    window = max(1, ctx // 3)
    tl.tl_attention_int4(x, *cache, torch.from_numpy(lens).cuda(), again, n_q=n_q, window=window)
    got = again.cpu().numpy().reshape(lanes, n_q, H * group, hd)
    for b in range(6, lanes):
        assert np.array_equal(got[b], got[b % 6]), b
    _check(got[:4].reshape(4 * n_q, H * group, hd), q[:4 * n_q], TwoByTurns(two), lens[:4].tolist(), n_q, window)


def test_lengths_below_zero():
    """A negative length is an empty lane, down to the least 32-bit value."""
    cache = Cache(*_kv(1, 1, 70, 64, 42))
    q = _q(5, 1, 64, 43)
    for n in (-1, -6, -(1 << 31), -(1 << 31) + 3):
        assert (_run(q, cache, [n], 5, 0) == 0).all() and (_run(q, cache, [n], 5, 3) == 0).all(), n


def test_a_query_alone_and_among_others_gives_the_same_bits():
    """A query's arithmetic does not depend on the lane's other queries, its
    neighbours' contents, or the run."""
    H, hd, ctx, n_q = 2, 128, 400, 8
    cache = Cache(*_kv(1, H, ctx, hd, 15))
    q = _q(n_q, H, hd, 16, 3.0)
    many = _run(q, cache, [333], n_q, 0)
    assert np.array_equal(many, _run(q, cache, [333], n_q, 0))
    for i in range(n_q):
        assert np.array_equal(_run(q[i:i + 1], cache, [333 - n_q + 1 + i], 1, 0)[0], many[i]), i


def test_strides():
    """Queries and outputs as column slices of wider rows, lanes further apart
    than their size."""
    H, hd, ctx, lens = 2, 64, 40, [40, 13]
    k, v = _kv(2, H, ctx, hd, 17)
    cache, padded = Cache(k, v), Cache(k, v, lane_pad=3)
    q = _q(2, 2 * H, hd, 18)
    want = _run(q, cache, lens, 1, 0)
    assert padded.t[0].stride(0) == H * (ctx + 3) * hd // 8
    assert np.array_equal(_run(q, padded, lens, 1, 0), want)
    w = 2 * H * hd
    wide = torch.zeros(2, 3 * w, dtype=torch.float16, device="cuda")
    wide[:, w:2 * w] = torch.from_numpy(q.reshape(2, w)).cuda()
    out = torch.full((2, 2 * w), 5.0, dtype=torch.float16, device="cuda")
    tl.tl_attention_int4(wide[:, w:2 * w], *cache.t, torch.tensor(lens, dtype=torch.int32, device="cuda"), out[:, w:])
    got = out.cpu().numpy()
    assert (got[:, :w] == 5).all() and np.array_equal(got[:, w:].reshape(want.shape), want)


@pytest.mark.parametrize("raw", [False, True])
def test_a_workspace_for_another_stream(raw):
    """The workspace that the binding allocates for a call on another stream is none of
    the current stream's blocks: work queued there may still use them."""
    H, hd, ctx = 1, 64, 8192
    cache = Cache(*_kv(1, H, ctx, hd, 40))
    q = _q(1, H, hd, 41)
    want = _run(q, cache, [ctx], 1, 0)
    need = tl.tl_attention_int4_workspace_bytes(*cache.t, 1, H)
    tq = torch.from_numpy(q.reshape(1, -1)).cuda()
    out, lens = torch.zeros_like(tq), torch.tensor([ctx], dtype=torch.int32, device="cuda")
    block = torch.full((need,), 0xAB, dtype=torch.uint8, device="cuda")
    ptr = block.data_ptr()
    torch.cuda.synchronize()
    del block
    s = torch.cuda.Stream()
    tl.tl_attention_int4(tq, *cache.t, lens, out, stream=s.cuda_stream if raw else s)
    torch.cuda.synchronize()
    again = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() == ptr and (again == 0xAB).all()
    assert np.array_equal(out.cpu().numpy().reshape(want.shape), want)


def test_streams_graphs_and_growing_lengths():
    """Two calls at once on two streams; a captured write and attention replayed
    while the lane grows."""
    H, hd, ctx = 2, 128, 64
    k, v = _kv(1, H, ctx, hd, 19)
    ref = Cache(k, v)
    q = _q(1, H, hd, 20)
    others = [Cache(*_kv(1, H, ctx, hd, 30 + i)) for i in range(2)]
    wants = [_run(q, c, [ctx], 1, 0) for c in others]
    streams = [torch.cuda.Stream() for _ in others]
    tq = torch.from_numpy(q.reshape(1, -1)).cuda()
    full = torch.tensor([ctx], dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(tq) for _ in others]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, c, out in zip(streams, others, outs):
            tl.tl_attention_int4(tq, *c.t, full, out, stream=s)
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        assert np.array_equal(out.cpu().numpy().reshape(want.shape), want)

    cache = [torch.full_like(t, 0) for t in ref.t]
    row = [torch.zeros(1, H * hd, dtype=torch.float16, device="cuda") for _ in range(2)]
    pos, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(tq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tl.tl_kv_write_int4(row[0], row[1], *cache, pos)
        tl.tl_attention_int4(tq, *cache, lens, out)
    for p in range(40):
        row[0].copy_(torch.from_numpy(k[0, :, p].reshape(1, -1)))
        row[1].copy_(torch.from_numpy(v[0, :, p].reshape(1, -1)))
        pos.fill_(p)
        lens.fill_(p + 1)
        graph.replay()
        if p in (0, 15, 16, 39):
            torch.cuda.synchronize()
            assert np.array_equal(out.cpu().numpy().reshape(1, H, hd), _run(q, ref, [p + 1], 1, 0)), p


def test_far_offsets():
    """A cache whose last lane lies past 2^31 code words: one head of lane 2 over
    a lane stride of 2^30 words, most of it never touched."""
    hd, ctx = 128, 48
    k, v = _kv(3, 1, ctx, hd, 21)
    cache = Cache(k, v)
    stride = 1 << 30
    big = torch.empty(2 * stride + ctx * hd // 8, dtype=torch.int32, device="cuda")
    codes = [torch.as_strided(big, (3, 1, ctx, hd // 8), (stride, ctx * hd // 8, hd // 8, 1))] * 2
    # K and V share the far array here: both hold K's codes
    codes[0].copy_(cache.t[0])
    cache.vw = cache.kw
    cache.t = [codes[0], cache.t[1], codes[1], cache.t[3]]
    q = _q(3, 1, hd, 22)
    lens = [48, 47, 33]
    _check(_run(q, cache, lens, 1, 0), q, cache, lens, 1, 0)


@pytest.mark.parametrize("lanes,H,ctx,hd,gap", [
    (1, 1, 2112, 64, 26.0), (80, 1, 4096, 64, 26.0), (80, 1, 4096, 64, 30.0), (1, 2, 9000, 128, 28.0), (160, 4, 1024, 128, 24.5),
])
def test_many_keys_of_small_weight(lanes, H, ctx, hd, gap):
    """Keys of a weight 2^-gap each below some heavy ones whose values are zero: the light
    ones, of equal weight and value, are all of the output.  Every part of the split meets a
    heavy key first.  A weight is off by half of fp16's least step at most, 2^-32 of the
    heavy ones' (which weigh 2^7 or more), and by 2^-10 for the exponential of scores whose
    terms are exact; the result rounds by 2^-11, or by half of fp16's least step, 2^-25,
    where it is subnormal (1920 * 7 * 2^-30 = 1.25e-5 is)."""
    heavy = np.arange(ctx) < ctx // 8
    k = np.zeros((1, H, ctx, hd), np.float16)
    k[:, :, heavy, 0] = 15                                  # held exactly: scale 1, zero point 0
    v = np.where(heavy[None, None, :, None], 0.0, 1920.0) * np.ones((1, H, 1, hd))
    cache = Cache(np.repeat(k, lanes, 0), np.repeat(v.astype(np.float16), lanes, 0))
    q = np.zeros((lanes, H, hd), np.float16)
    q[:, :, 0] = gap / np.log2(np.e) * np.sqrt(hd) / 15
    got = _run(q, cache, [ctx] * lanes, 1, 0).astype(np.float64)
    w = np.exp(-float(q[0, 0, 0]) * 15 / np.sqrt(hd))       # of a light key
    light = ctx - heavy.sum()
    want = 1920.0 * light * w / (heavy.sum() + light * w)
    assert w * 2.0 ** 24 < 1
    assert (np.abs(got - want) <= want * (2.0 ** -32 / w + 2.0 ** -10 + 2.0 ** -11) + 2.0 ** -25).all(), (got.min(), got.max(), want)


@pytest.mark.parametrize("ctx,n_q,lens", [(90, 3, [90, 2, 0]), (2112, 1, [2112, 1, 0]), (9000, 2, [9000, 1, 0])])
def test_an_infinite_query(ctx, n_q, lens):
    """Scores that are all -inf have no distribution: NaN, not the zeros of a query that sees
    nothing.  The other head's outputs are its own."""
    H, hd = 2, 64
    k, v = _kv(3, H, ctx, hd, 50)
    k[..., 0] = -3 - np.abs(k[..., 0])                      # below zero as held, too
    cache = Cache(k, v)
    q = _q(3 * n_q, H, hd, 51)
    want = _run(q, cache, lens, n_q, 0)
    q[:, 0, 0] = np.inf
    got = _run(q, cache, lens, n_q, 0)
    assert np.array_equal(got[:, 1], want[:, 1])
    for b, length in enumerate(lens):
        for i in range(n_q):
            sees = length - n_q + i >= 0
            assert (np.isnan(got[b * n_q + i, 0]) if sees else got[b * n_q + i, 0] == 0).all(), (b, i)


def test_refusals_on_the_device():
    """What is refused before any launch, with tensors where they belong."""
    H, hd = 2, 64
    cache = Cache(*_kv(1, H, 8, hd, 52))
    q = torch.zeros(1, H * hd, dtype=torch.float16, device="cuda")
    lens, out = torch.ones(1, dtype=torch.int32, device="cuda"), torch.full_like(q, 5.0)
    none = [t[..., :0].contiguous() if i % 2 == 0 else t[..., :0, :].contiguous() for i, t in enumerate(cache.t)]
    with pytest.raises(tl.TLError, match="no values"):
        tl.tl_attention_int4(q, *none, lens, out)
    with pytest.raises(tl.TLError, match="no values"):
        tl.tl_kv_write_int4(q, q, *none, lens)
    assert (out == 5).all()


@pytest.mark.parametrize("window", [1 << 31, (1 << 32) + 3, -(1 << 32), -(1 << 32) + 3, -1])
def test_windows_out_of_range_are_refused(window):
    """They are not cut to a window of another size."""
    cache = Cache(*_kv(1, 1, 8, 64, 53))
    q = torch.zeros(1, 64, dtype=torch.float16, device="cuda")
    lens, out = torch.full((1,), 8, dtype=torch.int32, device="cuda"), torch.full_like(q, 5.0)
    with pytest.raises(tl.TLError, match="window"):
        tl.tl_attention_int4(q, *cache.t, lens, out, window=window)
    torch.cuda.synchronize()
    assert (out == 5).all()


@pytest.mark.parametrize("ctx,lanes,H,group,hd,n_q", [
    (129, 38, 1, 1, 64, 1), (520, 40, 1, 1, 128, 1), (1024, 74, 1, 1, 64, 1), (1025, 48, 1, 1, 64, 1), (4064, 40, 1, 1, 64, 1),
    (4095, 75, 1, 1, 64, 1), (4096, 65, 1, 1, 64, 1), (4097, 40, 1, 2, 128, 1), (4100, 75, 1, 1, 64, 1), (8192, 38, 1, 1, 64, 1),
    (8193, 65, 1, 1, 64, 1), (8300, 22, 4, 1, 64, 2), (8200, 130, 1, 1, 64, 1),
])
def test_both_sides_of_the_split(ctx, lanes, H, group, hd, n_q):
    """Contexts and unit counts around those where the split changes."""
    test_any_number_of_lanes(ctx, lanes, H, group, hd, n_q)


@pytest.mark.parametrize("lanes,H,group,ctx,same", [
    (1, 2, 1, 400, True), (2, 2, 2, 2112, True), (20, 2, 4, 2112, False), (6, 8, 2, 9000, False), (2, 1, 4, 9000, False),
])
def test_a_query_alone_and_with_others_of_its_lane(lanes, H, group, ctx, same):
    """The last of eight queries as a call of its own: right in both; the same bits where the
    number of column tiles leaves the split as it is, else the split may differ."""
    hd, n_q = 64, 8
    cache = Cache(*_kv(lanes, H, ctx, hd, 54))
    q = _q(lanes * n_q, H * group, hd, 55, 2.0)
    lens = [ctx - 5 * b for b in range(lanes)]
    many = _run(q, cache, lens, n_q, 0)
    _check(many, q, cache, lens, n_q, 0)
    alone = _run(q[n_q - 1::n_q], cache, lens, 1, 0)
    _check(alone, q[n_q - 1::n_q], cache, lens, 1, 0)
    if same:
        assert np.array_equal(alone, many[n_q - 1::n_q])
