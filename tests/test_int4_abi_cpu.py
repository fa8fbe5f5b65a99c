"""Host-only behaviour of the 4-bit cache and scoring calls: sizes, argument
checks before any launch, the binding's checks, the oracle's quantiser."""
import ctypes

import numpy as np
import pytest
import torch

import weight_shared_looped_b200 as tl
from oracle import tinyloop_oracle as o

P16 = 16      # never dereferenced: every call below is refused or empty
BAD = tl.TL_ERR_INVALID_ARG


def _cache(**kw):
    f = dict(k_codes=P16, v_codes=P16, k_params=P16, v_params=P16, code_stride=2 * 8 * 16, param_stride=2 * 8 * 4,
             n_lanes=2, n_heads=2, head_dim=128, max_ctx=8)
    f.update(kw)
    return tl.KvInt4Desc(*[f[n] for n, _ in tl.KvInt4Desc._fields_])


def _p(v):
    return None if v is None else ctypes.c_void_p(v)


def _rows(fn, cache=None, k=P16, v=P16, stride=256, cu=None, pos=P16, n=2):
    c = _cache() if cache is None else cache
    return fn(ctypes.byref(c), _p(k), _p(v), stride, _p(cu), _p(pos), n, None)


def _attend(cache=None, q=P16, qs=512, n_q=1, heads=4, lens=P16, window=0, out=P16, os=512, ws=None, wb=0):
    c = _cache() if cache is None else cache
    return tl.lib.tl_attention_int4(ctypes.byref(c), _p(q), qs, n_q, heads, _p(lens), window, _p(out), os, _p(ws), wb, None)


BAD_CACHES = [dict(n_lanes=-1), dict(n_lanes=65536), dict(n_heads=0), dict(n_heads=257), dict(max_ctx=0),
              dict(max_ctx=(1 << 24) + 1), dict(code_stride=252), dict(param_stride=60), dict(code_stride=258),
              dict(k_codes=None), dict(v_params=None), dict(v_codes=24), dict(k_params=18)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_cache_descriptions_are_refused(bad):
    for rc in (_rows(tl.lib.tl_kv_write_int4, _cache(**bad)), _rows(tl.lib.tl_kv_read_int4, _cache(**bad)),
               _attend(_cache(**bad))):
        assert rc == BAD and tl.lib.tl_last_error()


@pytest.mark.parametrize("hd", [0, 32, 96, 256])
def test_other_head_sizes_are_unsupported(hd):
    c = _cache(head_dim=hd)
    assert _rows(tl.lib.tl_kv_write_int4, c) == tl.TL_ERR_UNSUPPORTED
    assert _attend(c) == tl.TL_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(pos=None), dict(k=24), dict(v=2), dict(pos=6),
                                 dict(cu=3), dict(stride=255), dict(stride=260), dict(n=-1), dict(n=3),
                                 dict(n=(1 << 27) + 1)])
def test_row_calls_refuse(bad):
    for fn in (tl.lib.tl_kv_write_int4, tl.lib.tl_kv_read_int4):
        assert _rows(fn, **bad) == BAD and tl.lib.tl_last_error()
        assert fn(None, None, None, 256, None, None, 0, None) == BAD


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(lens=None), dict(q=8), dict(out=24), dict(lens=2),
                                 dict(qs=511), dict(os=511), dict(qs=516), dict(n_q=-1), dict(n_q=9), dict(heads=3),
                                 dict(heads=1), dict(heads=0), dict(heads=1026), dict(window=-1)])
def test_attention_refuses(bad):
    assert _attend(**bad) == BAD and tl.lib.tl_last_error()
    assert tl.lib.tl_attention_int4(None, _p(P16), 512, 1, 4, _p(P16), 0, _p(P16), 512, None, 0, None) == BAD


def test_attention_workspace():
    def need(n_q=1, heads=4, **kw):
        b = ctypes.c_size_t(7)
        c = _cache(code_stride=1 << 40, param_stride=1 << 40, **kw)
        assert tl.lib.tl_attention_int4_workspace_bytes(ctypes.byref(c), n_q, heads, ctypes.byref(b)) == tl.TL_OK
        return b.value
    assert need(max_ctx=8191) == 0 and need(max_ctx=8192) > 0       # two lanes of two heads: the split is wide
    assert need(max_ctx=1 << 20, n_q=0) == 0 and need(max_ctx=1 << 20, n_lanes=0) == 0
    assert need(max_ctx=65536, n_lanes=512) == 0                     # enough lanes fill the GPU without it
    big = need(max_ctx=1 << 20)
    c = dict(max_ctx=1 << 20, code_stride=1 << 40, param_stride=1 << 40)
    assert _attend(_cache(**c), ws=None, wb=1 << 30) == BAD
    assert _attend(_cache(**c), ws=P16, wb=big - 1) == BAD
    assert _attend(_cache(**c), ws=P16 + 8, wb=big) == BAD
    assert tl.lib.tl_attention_int4_workspace_bytes(ctypes.byref(_cache()), 1, 4, None) == BAD
    assert tl.lib.tl_attention_int4_workspace_bytes(ctypes.byref(_cache()), 9, 4, ctypes.byref(ctypes.c_size_t())) == BAD


@pytest.mark.parametrize("units,split", [(37, True), (38, True), (64, True), (65, False), (74, False), (75, True),
                                         (80, True), (128, True), (130, False), (148, False), (149, False)])
def test_long_contexts_use_every_sm(units, split):
    """From 38 to 148 lanes and heads one or two CTAs each only where they fill the GPU; else
    long contexts are split further, through the workspace (up to where four CTAs per SM
    leave a cluster's worth a unit or less)."""
    b = ctypes.c_size_t(7)
    c = _cache(code_stride=1 << 40, param_stride=1 << 40, n_lanes=units, n_heads=1, max_ctx=16384)
    assert tl.lib.tl_attention_int4_workspace_bytes(ctypes.byref(c), 1, 1, ctypes.byref(b)) == tl.TL_OK
    assert (b.value > 0) == (split and 592 // units > 8)


def test_empty_calls_do_nothing():
    none = _cache(n_lanes=0, k_codes=None, v_codes=None, k_params=None, v_params=None)
    for fn in (tl.lib.tl_kv_write_int4, tl.lib.tl_kv_read_int4):
        assert _rows(fn, k=None, v=None, pos=None, n=0) == tl.TL_OK
        assert _rows(fn, none, k=None, v=None, pos=None, n=5) == tl.TL_OK
    assert _attend(n_q=0, q=None, out=None, lens=None) == tl.TL_OK
    assert _attend(none, q=None, out=None, lens=None) == tl.TL_OK
    assert _score(n=0, embed=None, y=None, ws=None) == tl.TL_OK


def _score(embed=P16, vocab=100, d=64, y=P16, ys=64, n=3, targets=None, logp=None, entropy=None, k=2, ids=P16,
           top=P16, ws=256, wb=1 << 30):
    return tl.lib.tl_score_head(_p(embed), vocab, d, _p(y), ys, n, _p(targets), _p(logp), _p(entropy), k, _p(ids),
                                _p(top), _p(ws), wb, None)


@pytest.mark.parametrize("bad", [dict(embed=None), dict(y=None), dict(ws=None), dict(embed=8), dict(y=4), dict(ws=128),
                                 dict(wb=16), dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(d=32), dict(d=96),
                                 dict(d=8256), dict(ys=60), dict(ys=66), dict(n=-1), dict(n=65537), dict(k=-1),
                                 dict(k=17), dict(vocab=1, k=2), dict(ids=None), dict(top=None),
                                 dict(targets=P16), dict(logp=P16)])
def test_score_head_refuses(bad):
    assert _score(**bad) == BAD and tl.lib.tl_last_error()


def test_score_head_workspace_sizes():
    with pytest.raises(tl.TLError):
        tl.tl_score_head_workspace_bytes(1, 100, 65, 0)
    with pytest.raises(tl.TLError):
        tl.tl_score_head_workspace_bytes(1, 10, 64, 11)
    assert tl.lib.tl_score_head_workspace_bytes(1, 100, 64, 0, None) == BAD
    sizes = [tl.tl_score_head_workspace_bytes(n, 50257, 2048, 8) for n in (0, 1, 8, 64, 128, 1024)]
    assert all(s >= 0 for s in sizes) and sizes[-1] < 1024 * 50257 * 4 // 8   # far below the logits


def test_layer_bytes_match_the_closed_form():
    assert 10 * tl.tl_kv_layer_bytes(16, 128, 2048, tl.TL_KV_INT4) == o.kv_cache_bytes(10, 2048, 16, 128, "int4")
    fp16 = tl.tl_kv_layer_bytes(16, 128, 2048, tl.TL_KV_FP16)
    assert tl.tl_kv_layer_bytes(16, 128, 2048, tl.TL_KV_INT4) * 16 == fp16 * 5      # 5 bits a value
    # regions start on 256 bytes: 3 heads x 5 positions x 64
    assert tl.tl_kv_layer_bytes(3, 64, 5, tl.TL_KV_INT4) == 2 * 512 + 2 * 256
    with pytest.raises(tl.TLError):
        tl.tl_kv_layer_bytes(2, 48, 8, tl.TL_KV_INT4)
    with pytest.raises(tl.TLError):
        tl.tl_kv_layer_bytes(2, 64, 8, 4)


def test_the_binding_refuses_what_the_library_cannot_see():
    """Types, shapes, layouts and devices of the tensors: refused on the host."""
    lanes, H, ctx, hd, n = 2, 2, 8, 64, 2
    c = lambda: torch.zeros(lanes, H, ctx, hd // 8, dtype=torch.int32)                  # noqa: E731
    p = lambda: torch.zeros(lanes, H, ctx, hd // 32, 2, dtype=torch.float16)            # noqa: E731
    rows = torch.zeros(n, H * hd, dtype=torch.float16)
    i = torch.zeros(lanes, dtype=torch.int32)
    with pytest.raises(tl.TLError, match="CUDA device"):
        tl.tl_kv_write_int4(rows, rows, c(), p(), c(), p(), i)
    with pytest.raises(tl.TLError, match="dtype"):
        tl.tl_kv_write_int4(rows.float(), rows, c(), p(), c(), p(), i)
    with pytest.raises(tl.TLError, match="dtype"):
        tl.tl_kv_read_int4(c(), p(), c(), p(), i.long(), rows, rows)
    with pytest.raises(tl.TLError, match="dimensions"):
        tl.tl_attention_int4(rows[0], c(), p(), c(), p(), i, rows[0])
    with pytest.raises(tl.TLError, match="dtype"):
        tl.tl_score_head(torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(1, 64), None, None, None, None, None,
                         torch.zeros(1, dtype=torch.uint8))
    with pytest.raises(tl.TLError, match="shape"):
        tl._kv_int4("x", c(), p()[:, :, :4], c(), p())
    with pytest.raises(tl.TLError, match="strides"):
        wide = torch.zeros(lanes, H * ctx + 4, hd // 8, dtype=torch.int32)
        far = torch.as_strided(wide, (lanes, H, ctx, hd // 8), (wide.stride(0), ctx * hd // 8, hd // 8, 1))
        tl._kv_int4("x", far, p(), c(), p())
    with pytest.raises(tl.TLError, match="contiguous"):
        tl._kv_int4("x", c().transpose(1, 2).contiguous().transpose(1, 2), p(), c(), p())
    d = tl._kv_int4("x", c(), p(), c(), p())
    assert (d.n_lanes, d.n_heads, d.head_dim, d.max_ctx) == (lanes, H, hd, ctx)
    assert (d.code_stride, d.param_stride) == (H * ctx * hd // 8, H * ctx * hd // 32)


def test_rows_of_no_values_are_refused():
    """A last dimension of 0 is refused like any other bad shape, before head sizes are divided by."""
    c, p = torch.zeros(2, 2, 8, 0, dtype=torch.int32), torch.zeros(2, 2, 8, 0, 2, dtype=torch.float16)
    with pytest.raises(tl.TLError, match="no values"):
        tl._kv_int4("x", c, p, c, p)
    with pytest.raises(tl.TLError):
        tl.tl_attention_int4_workspace_bytes(c, p, c, p, 1, 2)


@pytest.mark.parametrize("bad", [dict(n=(1 << 32) + 1), dict(vocab=(1 << 32) + 100), dict(d=64 - (1 << 32)), dict(k=1 << 32)])
def test_integers_beyond_32_bits_are_refused(bad):
    """They are not cut to the size of another call."""
    with pytest.raises(tl.TLError, match="out of range"):
        tl.tl_score_head_workspace_bytes(**{**dict(n=1, vocab=100, d=64, k=0), **bad})
    c, p = torch.zeros(1, 1, 9000, 8, dtype=torch.int32), torch.zeros(1, 1, 9000, 2, 2, dtype=torch.float16)
    for n_q, heads in ((1 << 32 | 1, 1), (1, 1 << 32 | 1), (-(1 << 32) + 1, 1)):
        with pytest.raises(tl.TLError, match="out of range"):
            tl.tl_attention_int4_workspace_bytes(c, p, c, p, n_q, heads)


@pytest.mark.parametrize("k", [-1, 17, 101])
def test_a_models_scores_refuse_k(k):
    """By the library's error, before any output is made."""
    from types import SimpleNamespace
    from weight_shared_looped_b200.model import DeviceModel
    model = SimpleNamespace(embed=torch.zeros(100, 64, dtype=torch.float16), d=64)
    with pytest.raises(tl.TLError, match="k = "):
        DeviceModel.score(model, torch.zeros(2, 64), k=k)


def test_score_status_and_the_wait_hook_refuse():
    def hook(copies=1, limit=1000, n=3, ws=256):
        return tl.lib.tl_check_score_wait(_p(P16), 100, 64, _p(P16), n, copies, limit, None, 0, None, None, _p(ws), 1 << 30,
                                          None)
    assert hook(limit=0) == hook(limit=2000001) == hook(copies=-1) == hook(n=-1) == hook(ws=128) == BAD
    assert hook(n=0) == tl.TL_OK
    assert tl.lib.tl_score_head_status(None, None) == tl.lib.tl_score_head_status(_p(128), None) == BAD
    with pytest.raises(tl.TLError, match="workspace"):
        tl.tl_score_head_status(torch.zeros(512, dtype=torch.uint8))


# ---------------------------------------------------------------- the oracle's quantiser

def test_oracle_int4_group_by_hand():
    x = np.array([[0.0, 15.0] + [0.5 * i for i in range(30)]], np.float16)
    c, s, z = o.kv_quant_int4(x)
    assert s[0, 0] == 1 and z[0, 0] == 0
    assert c[0, :6].tolist() == [0, 15, 0, 0, 1, 2]      # 0.5 -> 0 and 1.5 -> 2: ties to even
    assert np.array_equal(o.kv_dequant_int4(c, s, z)[0, :2], [0.0, 15.0])


def test_oracle_int4_scale_rounds_towards_zero():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((400, 64)) * np.exp2(rng.uniform(-20, 14, (400, 1)))).astype(np.float16)
    c, s, z = o.kv_quant_int4(x)
    g = x.reshape(400, 2, 32).astype(np.float64)
    step = (g.max(-1) - g.min(-1)) / 15
    assert (s.astype(np.float64) <= step * (1 + 2.0 ** -23)).all()
    up = np.nextafter(s, np.float16(np.inf)).astype(np.float64)
    assert (up > step * (1 - 2.0 ** -23)).all()
    v = o.kv_dequant_int4(c, s, z).astype(np.float16).astype(np.float64).reshape(400, 2, 32)
    assert (v >= g.min(-1, keepdims=True)).all() and (v <= g.max(-1, keepdims=True)).all()


def test_oracle_int4_narrow_groups():
    """Subnormal scales: the absolute bound holds, one relative to the step does not."""
    from int4_util import held_bound, narrow_groups
    x = narrow_groups()
    c, s, z = o.kv_quant_int4(x)
    err = np.abs(o.kv_dequant_int4(c, s, z) - x.astype(np.float64))
    assert (err <= held_bound(x)).all()
    g = x.reshape(-1, 32).astype(np.float64)
    step = (g.max(-1) - g.min(-1)) / 15
    worst = err.reshape(-1, 32).max(-1)
    assert (worst > 5 * step).any() and (s == 0).any()       # the case of range 28.5 * 2^-24, and collapsed groups


def test_a_planted_mistake_is_seen():
    """The bit-exact comparison tells rounding to nearest from towards zero, a
    missing + 8 of the signed codes, and a swapped nibble order."""
    from int4_util import pack, unpack
    x = np.random.default_rng(5).standard_normal((64, 128)).astype(np.float16)
    c, s, z = o.kv_quant_int4(x)
    g = x.reshape(64, 4, 32).astype(np.float32)
    nearest = ((g.max(-1) - g.min(-1)) / np.float32(15)).astype(np.float16)
    assert (nearest != s).any()
    assert np.array_equal(unpack(pack(c)), c)
    assert not np.array_equal(pack(c), pack(c.reshape(64, 64, 2)[..., ::-1].reshape(64, 128)))
