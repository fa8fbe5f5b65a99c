"""Writing rows into a 4-bit KV cache and reading them back, against the
oracle's quantiser: codes, scales and zero points bit for bit, read-back values
equal to the held value rounded once to fp16 (exact: the value has few enough
bits for fp64)."""
import numpy as np
import pytest
import torch

import synthetic as syn
import weight_shared_looped_b200 as tl
from oracle import tinyloop_oracle as o

from int4_util import held_bound, narrow_groups, pack, quantise, values

pytestmark = pytest.mark.gpu


def _rows(n, H, hd, seed):
    """K-like rows, then rows where the format can go wrong."""
    x = syn.normal((n, H, hd), 1.0, seed, "int4.rows").astype(np.float16)
    special = [
        np.zeros(32), np.full(32, -0.0), np.full(32, 3.5), np.linspace(-1, 1, 32),
        np.where(np.arange(32) == 7, 100.0, 0.01), np.linspace(-65504, 65504, 32),
        np.full(32, 65504.0), np.where(np.arange(32) % 2, 6e-8, 0.0), np.arange(32) * 2.0 ** -24,
        np.arange(32) / 2.0, np.concatenate([[-0.0, 0.0], np.full(30, 1.0)]),
        np.concatenate([[0.0, 15.0], np.arange(30) * 0.5]),
    ]
    flat = x.reshape(-1, 32)
    for i, g in enumerate(special):
        if i < len(flat):
            flat[-1 - i] = g.astype(np.float16)
    return x


def _empty(lanes, H, ctx, hd):
    """Caches full of a pattern that no test writes, and that pattern."""
    return [torch.full((lanes, H, ctx, hd // 8), 0x5A5A5A5A, dtype=torch.int32, device="cuda"),
            torch.full((lanes, H, ctx, hd // 32, 2), 77.0, dtype=torch.float16, device="cuda"),
            torch.full((lanes, H, ctx, hd // 8), 0x5A5A5A5A, dtype=torch.int32, device="cuda"),
            torch.full((lanes, H, ctx, hd // 32, 2), 77.0, dtype=torch.float16, device="cuda")]


def _expect(cache, k, v, place):
    """The host copy of `cache` with rows r of k, v [n, H, hd] at place[r] = (lane, pos)."""
    want = [t.cpu().numpy().copy() for t in cache]
    for x, wi, pi in ((k, 0, 1), (v, 2, 3)):
        w, p = quantise(x)
        for r, at in enumerate(place):
            if at is not None:
                want[wi][at[0], :, at[1]] = w[r]
                want[pi][at[0], :, at[1]] = p[r]
    return want


def _same(cache, want):
    for t, w, name in zip(cache, want, ("k codes", "k params", "v codes", "v params")):
        got = t.cpu().numpy()
        view = np.int32 if got.dtype == np.int32 else np.uint16
        bad = np.argwhere(got.view(view) != w.view(view))
        assert bad.size == 0, (name, bad[:5])


def _place(cu, pos, ctx, n):
    place = [None] * n
    for b in range(len(pos)):
        for r in range(max(0, cu[b]), min(n, cu[b + 1])):
            p = pos[b] + r - cu[b]
            if 0 <= p < ctx:
                place[r] = (b, p)
    return place


def _dev(a):
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


CASES = [
    # lanes' row counts, positions, rows behind the last lane, H, hd, ctx
    ([1], [0], 0, 1, 64, 1),
    ([1], [4], 0, 1, 128, 5),
    ([1] * 8, [0, 3, 7, 15, 16, 17, 63, 64], 0, 16, 128, 65),
    ([0, 5, 0, 17, 1], [9, 0, 3, 2, 39], 3, 3, 64, 40),
    ([33, 0, 64], [0, 0, 11], 1, 4, 128, 75),
    ([0, 0], [0, 0], 2, 2, 64, 8),          # nothing but rows behind the last lane
    ([6, 6], [-3, 5], 0, 2, 128, 8),        # rows before and behind the cache
    ([700], [100], 0, 5, 64, 1000),
]


@pytest.mark.parametrize("counts,pos,behind,H,hd,ctx", CASES)
def test_write_and_read_back_bit_exact(counts, pos, behind, H, hd, ctx):
    cu = np.concatenate([[0], np.cumsum(counts)])
    n = int(cu[-1]) + behind
    k, v = _rows(n, H, hd, 1), _rows(n, H, hd, 2)
    cache = _empty(len(counts), H, ctx, hd)
    place = _place(cu, pos, ctx, n)
    want = _expect(cache, k, v, place)
    tk, tv = (torch.from_numpy(a.reshape(n, H * hd)).cuda() for a in (k, v))
    tl.tl_kv_write_int4(tk, tv, *cache, _dev(pos), _dev(cu))
    torch.cuda.synchronize()
    _same(cache, want)
    # read back: rows without a place are left as they were
    ok, ov = (torch.full((n, H * hd), -123.0, dtype=torch.float16, device="cuda") for _ in range(2))
    tl.tl_kv_read_int4(*cache, _dev(pos), ok, ov, _dev(cu))
    torch.cuda.synchronize()
    for got, wi, pi in ((ok, 0, 1), (ov, 2, 3)):
        got = got.cpu().numpy().reshape(n, H, hd)
        for r, at in enumerate(place):
            if at is None:
                assert (got[r] == -123.0).all()
            else:
                exact = values(want[wi][at[0], :, at[1]], want[pi][at[0], :, at[1]]).astype(np.float16)
                assert np.array_equal(got[r], exact), r


@pytest.mark.parametrize("counts,pos,behind,H,hd,ctx", [
    ([1201, 0, 700, 3, 500], [0, 5, 611, 1310, 100], 2, 16, 128, 1311),   # a lane ends at the cache's end
    ([2400, 1400, 1001], [0, 1001, 1400], 0, 16, 64, 2403),
])
def test_many_rows(counts, pos, behind, H, hd, ctx):
    """Batches large enough for two rows a thread; the last CTA's rows are cut off."""
    test_write_and_read_back_bit_exact(counts, pos, behind, H, hd, ctx)


@pytest.mark.parametrize("hd", [64, 128])
def test_equal_shares_and_column_slices(hd):
    """Without cu every lane takes n / lanes rows; k and v are column slices of
    [q | k | v] rows, the read-back goes into slices too."""
    lanes, per, H, ctx = 3, 5, 2, 20
    n, w = lanes * per, H * hd
    qkv = torch.from_numpy(syn.normal((n, 3 * w), 1.0, 3, "int4.qkv").astype(np.float16)).cuda()
    pos = [0, 7, 15]
    cache = _empty(lanes, H, ctx, hd)
    host = qkv.cpu().numpy()
    place = _place(np.arange(lanes + 1) * per, pos, ctx, n)
    want = _expect(cache, host[:, w:2 * w].reshape(n, H, hd), host[:, 2 * w:].reshape(n, H, hd), place)
    tl.tl_kv_write_int4(qkv[:, w:2 * w], qkv[:, 2 * w:], *cache, _dev(pos))
    torch.cuda.synchronize()
    _same(cache, want)
    out = torch.zeros(n, 3 * w, dtype=torch.float16, device="cuda")
    tl.tl_kv_read_int4(*cache, _dev(pos), out[:, w:2 * w], out[:, 2 * w:])
    torch.cuda.synchronize()
    got = out.cpu().numpy()
    assert (got[:, :w] == 0).all()
    for r, (b, p) in enumerate(place):
        assert np.array_equal(got[r, w:2 * w].reshape(H, hd), values(want[0][b, :, p], want[1][b, :, p]).astype(np.float16))


def test_non_finite_groups_are_marked():
    """A group with a NaN or an infinity holds NaN; its neighbours are untouched."""
    x = syn.normal((4, 1, 128), 1.0, 4, "int4.nan").astype(np.float16)
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 64:96], x[3, 0, 127] = np.nan, np.inf, np.inf, -np.inf
    t = torch.from_numpy(x.reshape(4, 128)).cuda()
    cache = _empty(1, 1, 4, 128)
    want = _expect(cache, x, x, [(0, p) for p in range(4)])
    tl.tl_kv_write_int4(t, t, *cache, _dev([0]))
    k, v = torch.zeros_like(t), torch.zeros_like(t)
    tl.tl_kv_read_int4(*cache, _dev([0]), k, v)
    torch.cuda.synchronize()
    for got, ref in zip(cache[::2], want[::2]):
        assert np.array_equal(got.cpu().numpy(), ref)
    for got, ref in zip(cache[1::2], want[1::2]):
        assert np.array_equal(got.cpu().numpy(), ref, equal_nan=True)
    bad = np.isnan(k.cpu().numpy()).reshape(4, 4, 32)
    assert np.array_equal(bad.all(-1), bad.any(-1))
    assert np.array_equal(bad.all(-1), ~np.isfinite(x).reshape(4, 4, 32).all(-1))


def test_values_stay_within_their_group():
    """The scale is rounded towards zero, so a group over the whole fp16 range
    reads back finite and inside [lo, hi], half a step off at most (plus the
    scale's own rounding, 15 * 2^-10 of a step, and the fp16 rounding)."""
    n = 300
    x = syn.normal((n, 2, 64), 1.0, 5, "int4.range")
    x *= np.exp2(np.linspace(-20, 15.5, n))[:, None, None]
    x = np.clip(x, -65504, 65504).astype(np.float16)
    x[:, :, ::31] = np.float16(65504) * np.sign(x[:, :, ::31])
    t = torch.from_numpy(x.reshape(n, 128)).cuda()
    cache = _empty(1, 2, n, 64)
    tl.tl_kv_write_int4(t, t, *cache, _dev([0]))
    k, v = torch.zeros_like(t), torch.zeros_like(t)
    tl.tl_kv_read_int4(*cache, _dev([0]), k, v)
    g, r = x.reshape(-1, 32).astype(np.float64), k.cpu().numpy().reshape(-1, 32).astype(np.float64)
    lo, hi = g.min(1, keepdims=True), g.max(1, keepdims=True)
    assert np.isfinite(r).all() and (r >= lo).all() and (r <= hi).all()
    step = (hi - lo) / 15
    assert (np.abs(r - g) <= step * (0.5 + 15 * 2.0 ** -10) + np.abs(g) * 2.0 ** -11 + 15 * 2.0 ** -24).all()
    assert torch.equal(k, v)


def test_lane_strides_streams_and_graphs():
    """Lanes further apart than their size; the call on another stream; a captured
    call replayed with new rows and positions."""
    lanes, H, hd, ctx, n = 2, 2, 128, 16, 6
    big = [torch.zeros((lanes, H * (ctx + 4)) + s, dtype=d, device="cuda")
           for s, d in (((hd // 8,), torch.int32), ((hd // 32, 2), torch.float16))]
    kc, kp = (b[:, :H * ctx].view((lanes, H, ctx) + b.shape[2:]) for b in big)
    vc, vp = (b.clone()[:, :H * ctx].view((lanes, H, ctx) + b.shape[2:]) for b in big)
    cache = [kc, kp, vc, vp]
    rows = [_rows(n, H, hd, 6 + i) for i in range(2)]
    tk, tv = (torch.from_numpy(r.reshape(n, -1)).cuda() for r in rows)
    pos = _dev([2, 9])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tl.tl_kv_write_int4(tk, tv, *cache, pos)   # first call outside the capture
    s.synchronize()
    for t in cache:
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tl.tl_kv_write_int4(tk, tv, *cache, pos)
    for at in ([2, 9], [0, 13]):
        new = [_rows(n, H, hd, 20 + at[0] + i) for i in range(2)]
        tk.copy_(torch.from_numpy(new[0].reshape(n, -1)))
        tv.copy_(torch.from_numpy(new[1].reshape(n, -1)))
        pos.copy_(_dev(at))
        want = _expect(cache, new[0], new[1], _place([0, 3, 6], at, ctx, n))
        graph.replay()
        torch.cuda.synchronize()
        _same(cache, want)
    for b in big:
        assert (b[:, H * ctx:] == 0).all()


def test_oracle_pack_matches_canonical_words():
    c = np.arange(64, dtype=np.uint8).reshape(2, 32) % 16
    w = pack(c).view(np.uint32)
    assert w[0, 0] == 0x76543210 and w[1, 1] == 0xFEDCBA98 and w.shape == (2, 4)


@pytest.mark.parametrize("hd", [64, 128])
def test_narrow_groups(hd):
    """Groups whose scale is subnormal or zero: read back within the absolute bound of the
    rows that were written (and the read-back's own rounding)."""
    x = narrow_groups().reshape(-1, hd)
    n = len(x)
    t = torch.from_numpy(x).cuda()
    cache = _empty(1, 1, n, hd)
    tl.tl_kv_write_int4(t, t, *cache, _dev([0]))
    k, v = torch.zeros_like(t), torch.zeros_like(t)
    tl.tl_kv_read_int4(*cache, _dev([0]), k, v)
    torch.cuda.synchronize()
    _same(cache, _expect(cache, x[:, None], x[:, None], [(0, p) for p in range(n)]))
    got, rows = k.cpu().numpy().astype(np.float64), x.astype(np.float64)
    assert (np.abs(got - rows) <= held_bound(x) + np.abs(got) * 2.0 ** -11 + 2.0 ** -25).all()
    assert torch.equal(k, v)
