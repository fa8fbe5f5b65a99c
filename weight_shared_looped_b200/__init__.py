"""Python binding of libtinyloop_b200.so (the looped-block library).

Argument marshalling only: every function here has the name of the C entry
point it calls, converts torch tensors to raw pointers and sizes, and raises
``TLError`` on a non-zero status.  All computation happens in the library's
CUDA kernels.  There is no fallback: if the shared library is missing the
import fails.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtinyloop_b200.so")

TL_OK, TL_ERR_INVALID_ARG, TL_ERR_CUDA, TL_ERR_OOM, TL_ERR_TIMEOUT, TL_ERR_UNSUPPORTED, \
    TL_ERR_NUMERIC = range(7)
TL_KV_FP16, TL_KV_INT8, TL_KV_H, TL_KV_INT4 = 0, 1, 2, 3
STATUS_NAMES = {0: "TL_OK", 1: "TL_ERR_INVALID_ARG", 2: "TL_ERR_CUDA", 3: "TL_ERR_OOM",
                4: "TL_ERR_TIMEOUT", 5: "TL_ERR_UNSUPPORTED", 6: "TL_ERR_NUMERIC"}


class TLError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing; build it with weight_shared_looped_b200.build")

lib = ctypes.CDLL(LIB_PATH)

P = ctypes.c_void_p
I = ctypes.c_int
SZ = ctypes.c_size_t
F = ctypes.c_float
LG = ctypes.c_long


class BlockDesc(ctypes.Structure):
    _fields_ = [("d_model", I), ("n_heads", I), ("head_dim", I), ("ffn", I), ("bits", I),
                ("group", I), ("eps", F), ("rope_theta", F),
                ("w_qkv", P), ("s_qkv", P), ("w_o", P), ("s_o", P), ("w_gate", P), ("s_gate", P),
                ("w_up", P), ("s_up", P), ("w_down", P), ("s_down", P),
                ("gamma_attn", P), ("gamma_ffn", P),
                ("sign_qkv", P), ("sign_o", P), ("sign_gate", P), ("sign_up", P), ("sign_down", P)]


class ModelDesc(ctypes.Structure):
    _fields_ = [("pre", P), ("n_pre", I), ("loop", P), ("embed", P), ("vocab", I),
                ("gamma_final", P), ("max_tokens", I), ("max_lanes", I), ("max_ctx", I),
                ("max_L", I)]


class KvInt4Desc(ctypes.Structure):
    _fields_ = [("k_codes", P), ("v_codes", P), ("k_params", P), ("v_params", P),
                ("code_stride", SZ), ("param_stride", SZ),
                ("n_lanes", I), ("n_heads", I), ("head_dim", I), ("max_ctx", I)]


_SIGS = {
    "tl_last_error": ([], ctypes.c_char_p),
    "tl_abi_version": ([], I),
    "tl_packed_words_per_row": ([I, I, ctypes.POINTER(I)], I),
    "tl_packed_bytes": ([I, I, I, I, ctypes.POINTER(SZ), ctypes.POINTER(SZ)], I),
    "tl_pack_weights": ([P, I, I, I, I, P, P, P], I),
    "tl_unpack_codes": ([P, I, I, I, P, P], I),
    "tl_sign_bits_bytes": ([I, I, ctypes.POINTER(SZ)], I),
    "tl_pack_sign_bits": ([P, I, I, I, I, P, P, P], I),
    "tl_kv_quant_int8": ([P, I, I, P, P, P], I),
    "tl_kv_write_int4": ([ctypes.POINTER(KvInt4Desc), P, P, LG, P, P, I, P], I),
    "tl_kv_read_int4": ([ctypes.POINTER(KvInt4Desc), P, P, LG, P, P, I, P], I),
    "tl_attention_int4_workspace_bytes": ([ctypes.POINTER(KvInt4Desc), I, I, ctypes.POINTER(SZ)], I),
    "tl_attention_int4": ([ctypes.POINTER(KvInt4Desc), P, LG, I, I, P, I, P, LG, P, SZ, P], I),
    "tl_score_head_workspace_bytes": ([I, I, I, I, ctypes.POINTER(SZ)], I),
    "tl_score_head": ([P, I, I, P, LG, I, P, P, P, I, P, P, P, SZ, P], I),
    "tl_score_head_status": ([P, P], I),
    "tl_check_score_wait": ([P, I, I, P, I, I, ctypes.c_uint, P, I, P, P, P, SZ, P], I),
    "tl_attention_prefill": ([P, P, P, I, I, I, P, P], I),
    "tl_block_create": ([ctypes.POINTER(BlockDesc), ctypes.POINTER(P)], I),
    "tl_block_destroy": ([P], I),
    "tl_block_device_bytes": ([P, ctypes.POINTER(SZ)], I),
    "tl_model_create": ([ctypes.POINTER(ModelDesc), ctypes.POINTER(P)], I),
    "tl_model_destroy": ([P], I),
    "tl_model_device_bytes": ([P, ctypes.POINTER(SZ)], I),
    "tl_model_set_graphs": ([P, I], I),
    "tl_model_set_decode_chunks": ([P, I], I),
    "tl_model_set_exit_threshold": ([P, F], I),
    "tl_model_set_cross_iter": ([P, I], I),
    "tl_model_set_iteration_blocks": ([P, P, I], I),
    "tl_loops_used": ([P, P, I, P], I),
    "tl_kv_layer_bytes": ([I, I, I, I, ctypes.POINTER(SZ)], I),
    "tl_kv_bytes": ([P, I, I, P, I, ctypes.POINTER(SZ)], I),
    "tl_kv_create": ([P, I, I, P, I, P, SZ, ctypes.POINTER(P)], I),
    "tl_kv_destroy": ([P], I),
    "tl_kv_reset": ([P, I, P], I),
    "tl_kv_position": ([P, I, ctypes.POINTER(I)], I),
    "tl_kv_set_position": ([P, I, I, P], I),
    "tl_kv_layer_ptrs": ([P, I, I, ctypes.POINTER(P), ctypes.POINTER(P), ctypes.POINTER(P),
                          ctypes.POINTER(P)], I),
    "tl_prefill": ([P, P, P, I, I, P, I, P, P, P], I),
    "tl_decode_step": ([P, P, P, P, P, I, P, P, P], I),
    "tl_sync_status": ([P, P], I),
    "tl_extend": ([P, P, I, P, P, I, I, P, P, P], I),
    "tl_greedy_head": ([P, P, I, P, P], I),
    "tl_spec_step": ([P, P, I, ctypes.c_int32, I, I, I, P, ctypes.POINTER(I), P], I),
    "tl_linear_workspace_bytes": ([I, I, I, ctypes.POINTER(SZ)], I),
    "tl_linear": ([P, P, I, I, I, P, I, P, P, P], I),
    "tl_linear_noalloc": ([P, P, I, I, I, P, I, P, P], I),
    "tl_check_bounded_wait": ([P, ctypes.c_uint, P], I),
    "tl_read_probe": ([P, SZ, I, P, P], I),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


def _check(status: int) -> None:
    if status != TL_OK:
        raise TLError(status, lib.tl_last_error().decode(errors="replace"))


def _ptr(t) -> Optional[int]:
    """Raw address of a tensor (host or device), or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        if torch.cuda.is_available():
            return torch.cuda.current_stream().cuda_stream or None
        return None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _allocating_on(stream, device):
    """A context in which tensors are allocated for use on `stream` (None: the current one).
    A block that the allocator hands out may still be in use on the stream it is for, and
    is handed out again in that stream's order."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream) or 0, device=device)
    return torch.cuda.stream(stream)


# --------------------------------------------------------------------- packing

def tl_abi_version() -> int:
    return lib.tl_abi_version()


def tl_packed_words_per_row(K: int, bits: int) -> int:
    w = I()
    _check(lib.tl_packed_words_per_row(K, bits, ctypes.byref(w)))
    return w.value


def tl_packed_bytes(N: int, K: int, bits: int, group: int):
    c, s = SZ(), SZ()
    _check(lib.tl_packed_bytes(N, K, bits, group, ctypes.byref(c), ctypes.byref(s)))
    return c.value, s.value


def tl_pack_weights(w, bits: int, group: int, packed, scales, stream=None) -> None:
    N, K = w.shape
    _check(lib.tl_pack_weights(_ptr(w), N, K, bits, group, _ptr(packed), _ptr(scales),
                               _stream(stream)))


def tl_sign_bits_bytes(N: int, K: int) -> int:
    b = SZ()
    _check(lib.tl_sign_bits_bytes(N, K, ctypes.byref(b)))
    return b.value


def tl_pack_sign_bits(w, bits: int, group: int, scales, sign, stream=None) -> None:
    """Sign-of-frac bits of fp32 w [N, K] with the scales tl_pack_weights wrote."""
    N, K = w.shape
    _check(lib.tl_pack_sign_bits(_ptr(w), N, K, bits, group, _ptr(scales), _ptr(sign),
                                 _stream(stream)))


def tl_unpack_codes(packed, N: int, K: int, bits: int, codes, stream=None) -> None:
    _check(lib.tl_unpack_codes(_ptr(packed), N, K, bits, _ptr(codes), _stream(stream)))


def tl_kv_quant_int8(x, codes, scales, stream=None) -> None:
    rows, hd = (x.shape[0], x.shape[1]) if x.dim() == 2 else (0, x.shape[-1])
    _check(lib.tl_kv_quant_int8(_ptr(x), rows, hd, _ptr(codes), _ptr(scales), _stream(stream)))


def tl_attention_prefill(q, k, v, H: int, hd: int, out, stream=None) -> None:
    """q, k, v, out: fp16 [T, H * hd] (or [T, H, hd]) device tensors."""
    T = q.shape[0]
    _check(lib.tl_attention_prefill(_ptr(q), _ptr(k), _ptr(v), T, H, hd, _ptr(out),
                                    _stream(stream)))


# --------------------------------------------------------------------- 4-bit KV cache
# These calls take tensors of free shapes and are made once a layer or a step, so
# what the C side cannot see (types, shapes, layouts, devices) is checked here in a
# few attribute reads; only when a check fails is it worked out which.

def _fail(message: str) -> None:
    raise TLError(TL_ERR_INVALID_ARG, message)


def _ints(what: str, **named) -> None:
    """Refuses integers that ctypes would cut to 32 bits without a word."""
    for name, v in named.items():
        if not -(1 << 31) <= v < 1 << 31:
            _fail(f"{what}: {name} = {v} is out of range")


_TORCH: dict = {}


def _torch_names() -> dict:
    if not _TORCH:
        import torch
        f16 = {torch.float16: True, torch.int16: True}   # fp16 values, also as raw bits
        _TORCH.update(f16=f16, i32=torch.int32, f32=torch.float32, u8=torch.uint8,
                      stream=getattr(torch._C, "_cuda_getCurrentRawStream", None),
                      device=getattr(torch._C, "_cuda_getDevice", None), torch=torch)
    return _TORCH


def _explain(what: str, **named) -> None:
    """Raises for the first tensor that is not of its types and dimensions, not on a CUDA
    device, or on another device than the first.  named: name -> (tensor, dtypes, dims)."""
    named = {name: v for name, v in named.items() if v[0] is not None}
    for name, (t, dtypes, dims) in named.items():
        if t.dtype not in dtypes:
            _fail(f"{what}: {name} has dtype {t.dtype}, not {' or '.join(str(d) for d in dtypes)}")
        if t.dim() != dims:
            _fail(f"{what}: {name} has {t.dim()} dimensions, not {dims}")
    device = None
    for name, (t, _, _) in named.items():
        if not t.is_cuda:
            _fail(f"{what}: {name} is not on a CUDA device")
        device = t.device if device is None else device
        if t.device != device:
            _fail(f"{what}: {name} is on {t.device}, not {device}")


def _launch(n, device: int, stream, call, *args) -> None:
    """The C call on `stream` (default: `device`'s current one) with `device` current."""
    raw, current = n["stream"], n["device"]
    if stream is not None:
        s = _stream(stream)
    elif raw is not None:
        s = raw(device)
    else:
        s = n["torch"].cuda.current_stream(device).cuda_stream
    if (current() if current is not None else n["torch"].cuda.current_device()) == device:
        status = call(*args, s)
    else:
        with n["torch"].cuda.device(device):
            status = call(*args, s)
    if status:
        _check(status)


def _kv_int4(what: str, k_codes, k_params, v_codes, v_params) -> KvInt4Desc:
    """The cache description of codes int32 [lanes, heads, ctx, hd / 8] and parameters fp16
    [lanes, heads, ctx, hd / 32, 2]; only the lane stride is free.  ValueError: k_codes does
    not have four dimensions."""
    shape = k_codes.shape
    lanes, heads, ctx, words = shape
    if not words:
        _fail(f"{what}: codes {tuple(shape)} hold rows of no values")
    pshape = (lanes, heads, ctx, words // 4, 2)
    if v_codes.shape != shape or k_params.shape != pshape or v_params.shape != pshape:
        _fail(f"{what}: codes {tuple(shape)} and {tuple(v_codes.shape)}, parameters {tuple(k_params.shape)} and "
              f"{tuple(v_params.shape)} do not have the shapes [lanes, heads, ctx, hd / 8] and "
              "[lanes, heads, ctx, hd / 32, 2]")
    if (k_codes.is_contiguous() and k_params.is_contiguous() and v_codes.is_contiguous()
            and v_params.is_contiguous()):
        cs, ps = heads * ctx * words, heads * ctx * (words // 4)
    else:
        for name, t in (("k_codes", k_codes), ("k_params", k_params), ("v_codes", v_codes),
                        ("v_params", v_params)):
            if lanes == 0 or not t[0].is_contiguous():
                _fail(f"{what}: {name} is not contiguous within a lane")
        cs, ps = k_codes.stride(0), k_params.stride(0)
        if lanes > 1 and (v_codes.stride(0) != cs or v_params.stride(0) != ps or ps % 2):
            _fail(f"{what}: K and V have different lane strides")
        ps //= 2
    return KvInt4Desc(k_codes.data_ptr(), v_codes.data_ptr(), k_params.data_ptr(),
                      v_params.data_ptr(), cs, ps, lanes, heads, words * 8, ctx)


def _kv_int4_rows(what, fn, k, v, k_codes, k_params, v_codes, v_params, pos, cu, stream):
    n = _TORCH or _torch_names()
    f16, i32 = n["f16"], n["i32"]
    dev = k.get_device()
    ok = (dev >= 0 and k.dtype in f16 and v.dtype in f16 and k_codes.dtype is i32
          and v_codes.dtype is i32 and k_params.dtype in f16 and v_params.dtype in f16
          and pos.dtype is i32 and (cu is None or (cu.dtype is i32 and cu.get_device() == dev))
          and v.get_device() == dev == k_codes.get_device() == v_codes.get_device()
          and k_params.get_device() == dev == v_params.get_device() == pos.get_device())
    if ok:
        try:   # what the cache description does not compare: the dimensions it unpacks
            rows, width = shape = k.shape
            d = _kv_int4(what, k_codes, k_params, v_codes, v_params)
        except ValueError:
            ok = False
    if not ok:
        i = (i32,)
        _explain(what, k=(k, f16, 2), v=(v, f16, 2), k_codes=(k_codes, i, 4), k_params=(k_params, f16, 5),
                 v_codes=(v_codes, i, 4), v_params=(v_params, f16, 5), pos=(pos, i, 1), cu=(cu, i, 1))
    lanes = d.n_lanes
    if v.shape != shape or width != d.n_heads * d.head_dim:
        _fail(f"{what}: k {tuple(k.shape)} and v {tuple(v.shape)} are not rows of "
              f"{d.n_heads} x {d.head_dim} values")
    stride, unit = strides = k.stride()
    if rows and (unit != 1 or v.stride() != strides) and (rows > 1 or unit != 1 or v.stride(1) != 1):
        _fail(f"{what}: k and v need unit column stride and the same row stride")
    if pos.shape != (lanes,) or not pos.is_contiguous():
        _fail(f"{what}: pos is not a contiguous [{lanes}]")
    if cu is not None and (cu.shape != (lanes + 1,) or not cu.is_contiguous()):
        _fail(f"{what}: cu is not a contiguous [{lanes + 1}]")
    _launch(n, dev, stream, fn, d, k.data_ptr(), v.data_ptr(), stride if rows > 1 else width,
            None if cu is None else cu.data_ptr(), pos.data_ptr(), rows)


def tl_kv_write_int4(k, v, k_codes, k_params, v_codes, v_params, pos, cu=None, stream=None) -> None:
    """Quantise packed fp16 rows k, v [n, heads * hd] (column slices allowed) into the 4-bit
    caches codes int32 [lanes, heads, ctx, hd / 8] and params fp16 [lanes, heads, ctx, hd / 32,
    2]: lane b takes rows cu[b] .. cu[b + 1] - 1 (or an equal share) at positions pos[b], ..."""
    _kv_int4_rows("tl_kv_write_int4", lib.tl_kv_write_int4, k, v, k_codes, k_params, v_codes,
                  v_params, pos, cu, stream)


def tl_kv_read_int4(k_codes, k_params, v_codes, v_params, pos, k, v, cu=None, stream=None) -> None:
    """Read those positions back into fp16 rows k, v [n, heads * hd]."""
    _kv_int4_rows("tl_kv_read_int4", lib.tl_kv_read_int4, k, v, k_codes, k_params, v_codes,
                  v_params, pos, cu, stream)


_INT4_SPLIT_CTX = 8192   # caches below this many positions need no workspace


def tl_attention_int4_workspace_bytes(k_codes, k_params, v_codes, v_params, n_q: int,
                                      q_heads: int) -> int:
    _ints("tl_attention_int4_workspace_bytes", n_q=n_q, q_heads=q_heads)
    b = SZ()
    _check(lib.tl_attention_int4_workspace_bytes(
        _kv_int4("tl_attention_int4", k_codes, k_params, v_codes, v_params), n_q, q_heads, b))
    return b.value


def tl_attention_int4(q, k_codes, k_params, v_codes, v_params, lens, out, n_q: int = 1,
                      window: int = 0, workspace=None, stream=None) -> None:
    """q, out: fp16 [lanes * n_q, q_heads * hd]; lens int32 [lanes], the queries' own
    positions included; workspace: uint8 of tl_attention_int4_workspace_bytes, allocated here
    if it is needed and not given."""
    n = _TORCH or _torch_names()
    f16, i32 = n["f16"], n["i32"]
    what = "tl_attention_int4"
    dev = q.get_device()
    ok = (dev >= 0 and q.dtype in f16 and out.dtype in f16 and k_codes.dtype is i32
          and v_codes.dtype is i32 and k_params.dtype in f16 and v_params.dtype in f16
          and lens.dtype is i32 and out.get_device() == dev == k_codes.get_device()
          and v_codes.get_device() == dev == k_params.get_device()
          and v_params.get_device() == dev == lens.get_device())
    if ok:
        try:   # what the cache description does not compare: the dimensions it unpacks
            rows, width = shape = q.shape
            d = _kv_int4(what, k_codes, k_params, v_codes, v_params)
        except ValueError:
            ok = False
    if not ok:
        i = (i32,)
        _explain(what, q=(q, f16, 2), k_codes=(k_codes, i, 4), k_params=(k_params, f16, 5),
                 v_codes=(v_codes, i, 4), v_params=(v_params, f16, 5), lens=(lens, i, 1), out=(out, f16, 2))
    lanes, head_dim = d.n_lanes, d.head_dim
    if rows != lanes * n_q or width % head_dim or out.shape != shape:
        _fail(f"{what}: q {tuple(q.shape)} and out {tuple(out.shape)} are not {lanes} x {n_q} "
              f"rows of heads of {head_dim}")
    qs, qu = q.stride()
    os_, ou = out.stride()
    if rows and (qu != 1 or ou != 1):
        _fail(f"{what}: q and out need unit column stride")
    if lens.shape != (lanes,) or not lens.is_contiguous():
        _fail(f"{what}: lens is not a contiguous [{lanes}]")
    if rows <= 1:
        qs = os_ = width
    if not -(1 << 31) <= window < 1 << 31:
        _ints(what, window=window)
    ws, ws_bytes = None, 0
    if d.max_ctx >= _INT4_SPLIT_CTX and rows:
        if workspace is None:
            b = SZ()
            _check(lib.tl_attention_int4_workspace_bytes(d, n_q, width // head_dim, b))
            if b.value:
                with _allocating_on(stream, q.device):
                    workspace = n["torch"].empty(b.value, dtype=n["u8"], device=q.device)
        elif workspace.dtype is not n["u8"] or workspace.get_device() != dev or not workspace.is_contiguous():
            _fail(f"{what}: workspace is not a contiguous uint8 tensor on {q.device}")
        if workspace is not None:
            ws, ws_bytes = workspace.data_ptr(), workspace.numel()
    _launch(n, dev, stream, lib.tl_attention_int4, d, q.data_ptr(), qs, n_q, width // head_dim,
            lens.data_ptr(), window, out.data_ptr(), os_, ws, ws_bytes)


# --------------------------------------------------------------------- scoring head

def tl_score_head_workspace_bytes(n: int, vocab: int, d: int, k: int) -> int:
    _ints("tl_score_head_workspace_bytes", n=n, vocab=vocab, d=d, k=k)
    b = SZ()
    _check(lib.tl_score_head_workspace_bytes(n, vocab, d, k, b))
    return b.value


def tl_score_head(embed, y, targets, logp, entropy, top_ids, top_logp, workspace,
                  stream=None) -> None:
    """Log probabilities of `targets` int32 [n] under logits y . embed^T (y fp32 [n, d], embed
    fp16 [vocab, d]) into logp fp32 [n]; entropy fp32 [n]; the k most probable tokens into
    top_ids int32 [n, k] and top_logp fp32 [n, k].  targets with logp, entropy, and top_ids
    with top_logp may be None."""
    n_ = _TORCH or _torch_names()
    f16, i32, f32 = n_["f16"], n_["i32"], n_["f32"]
    what = "tl_score_head"
    dev = y.get_device()
    ok = (dev >= 0 and embed.dtype in f16 and y.dtype is f32 and workspace.dtype is n_["u8"]
          and embed.dim() == 2 == y.dim() and workspace.dim() == 1
          and embed.get_device() == dev == workspace.get_device())
    for t, dtype, dims in ((targets, i32, 1), (logp, f32, 1), (entropy, f32, 1), (top_ids, i32, 2),
                           (top_logp, f32, 2)):
        ok = ok and (t is None or (t.dtype is dtype and t.dim() == dims and t.get_device() == dev
                                   and t.is_contiguous()))
    if not ok:
        i, f = (i32,), (f32,)
        _explain(what, embed=(embed, f16, 2), y=(y, f, 2), targets=(targets, i, 1), logp=(logp, f, 1),
                 entropy=(entropy, f, 1), top_ids=(top_ids, i, 2), top_logp=(top_logp, f, 2),
                 workspace=(workspace, (n_["u8"],), 1))
        _fail(f"{what}: an output or the targets are not contiguous")
    n, d = y.shape
    vocab, ed = embed.shape
    if ed != d or not embed.is_contiguous():
        _fail(f"{what}: embed {tuple(embed.shape)} is not a contiguous [vocab, {d}]")
    ys, unit = y.stride()
    if n and unit != 1:
        _fail(f"{what}: y needs unit column stride")
    if (top_ids is None) != (top_logp is None):
        _fail(f"{what}: top_ids and top_logp go together")
    k = 0 if top_ids is None else top_ids.shape[1]
    for name, t, want in (("targets", targets, (n,)), ("logp", logp, (n,)),
                          ("entropy", entropy, (n,)), ("top_ids", top_ids, (n, k)),
                          ("top_logp", top_logp, (n, k))):
        if t is not None and t.shape != want:
            _fail(f"{what}: {name} has shape {tuple(t.shape)}, not {want}")
    _launch(n_, dev, stream, lib.tl_score_head, embed.data_ptr(), vocab, d, y.data_ptr(),
            ys if n > 1 else d, n, _ptr(targets), _ptr(logp), _ptr(entropy), k,
            _ptr(top_ids) if k else None, _ptr(top_logp) if k else None, workspace.data_ptr(),
            workspace.numel())


def tl_score_head_status(workspace, stream=None) -> int:
    """TL_OK or TL_ERR_TIMEOUT of the last tl_score_head call with this workspace, after the
    stream's work (default: the current stream of the workspace's device)."""
    n = _TORCH or _torch_names()
    if workspace.dtype is not n["u8"] or not workspace.is_cuda or workspace.numel() < 256:
        _fail("tl_score_head_status: workspace is not a uint8 tensor of a scoring call on a CUDA device")
    with n["torch"].cuda.device(workspace.device):
        s = n["torch"].cuda.current_stream().cuda_stream if stream is None else _stream(stream)
        return lib.tl_score_head_status(workspace.data_ptr(), s)


# --------------------------------------------------------------------- blocks / model

def tl_block_create(cfg: dict, packed: dict) -> int:
    """cfg: d_model, n_heads, head_dim, ffn, bits, group, eps, rope_theta;
    packed: device tensors w_qkv, s_qkv, ..., gamma_attn, gamma_ffn, and optionally
    sign_qkv, ..., sign_down (the sign-of-frac bits of cross-iteration rounding)."""
    d = BlockDesc(cfg["d_model"], cfg["n_heads"], cfg["head_dim"], cfg["ffn"], cfg["bits"],
                  cfg["group"], cfg["eps"], cfg["rope_theta"],
                  *[_ptr(packed[k]) for k in ("w_qkv", "s_qkv", "w_o", "s_o", "w_gate", "s_gate",
                                              "w_up", "s_up", "w_down", "s_down", "gamma_attn",
                                              "gamma_ffn")],
                  *[_ptr(packed.get(k)) for k in ("sign_qkv", "sign_o", "sign_gate", "sign_up",
                                                  "sign_down")])
    out = P()
    _check(lib.tl_block_create(ctypes.byref(d), ctypes.byref(out)))
    return out.value


def tl_block_destroy(block: int) -> None:
    _check(lib.tl_block_destroy(block))


def tl_block_device_bytes(block: int) -> int:
    b = SZ()
    _check(lib.tl_block_device_bytes(block, ctypes.byref(b)))
    return b.value


def tl_model_create(pre: Sequence[int], loop: int, embed, vocab: int, gamma_final,
                    max_tokens: int, max_lanes: int, max_ctx: int, max_L: int) -> int:
    arr = (P * max(1, len(pre)))(*pre)
    d = ModelDesc(ctypes.cast(arr, P) if pre else None, len(pre), loop, _ptr(embed), vocab,
                  _ptr(gamma_final), max_tokens, max_lanes, max_ctx, max_L)
    out = P()
    _check(lib.tl_model_create(ctypes.byref(d), ctypes.byref(out)))
    return out.value


def tl_model_destroy(model: int) -> None:
    _check(lib.tl_model_destroy(model))


def tl_model_device_bytes(model: int) -> int:
    b = SZ()
    _check(lib.tl_model_device_bytes(model, ctypes.byref(b)))
    return b.value


def tl_model_set_graphs(model: int, enable: bool) -> None:
    _check(lib.tl_model_set_graphs(model, 1 if enable else 0))


def tl_model_set_decode_chunks(model: int, chunks_per_cta: int) -> None:
    _check(lib.tl_model_set_decode_chunks(model, chunks_per_cta))


def tl_model_set_exit_threshold(model: int, tau: float) -> None:
    _check(lib.tl_model_set_exit_threshold(model, tau))


def tl_model_set_cross_iter(model: int, on: bool) -> None:
    _check(lib.tl_model_set_cross_iter(model, 1 if on else 0))


def tl_model_set_iteration_blocks(model: int, blocks: Sequence[Optional[int]]) -> None:
    """Loop iteration i < len(blocks) runs blocks[i] (None: the loop block)."""
    arr = (P * max(1, len(blocks)))(*[b or None for b in blocks])
    _check(lib.tl_model_set_iteration_blocks(model, ctypes.cast(arr, P) if blocks else None,
                                             len(blocks)))


def tl_loops_used(model: int, n: int, stream=None):
    arr = (I * n)()
    _check(lib.tl_loops_used(model, ctypes.cast(arr, P), n, _stream(stream)))
    return list(arr)


# --------------------------------------------------------------------- KV cache

def _int_array(vals: Sequence[int]):
    return (I * len(vals))(*vals)


def tl_kv_layer_bytes(n_heads: int, head_dim: int, max_ctx: int, dtype: int) -> int:
    b = SZ()
    _check(lib.tl_kv_layer_bytes(n_heads, head_dim, max_ctx, dtype, ctypes.byref(b)))
    return b.value


def tl_kv_bytes(model: int, max_ctx: int, L_per_lane: Sequence[int], dtype: int) -> int:
    b = SZ()
    arr = _int_array(L_per_lane)
    _check(lib.tl_kv_bytes(model, len(L_per_lane), max_ctx, ctypes.cast(arr, P), dtype,
                           ctypes.byref(b)))
    return b.value


def tl_kv_create(model: int, max_ctx: int, L_per_lane: Sequence[int], dtype: int, buffer) -> int:
    arr = _int_array(L_per_lane)
    out = P()
    nbytes = buffer.numel() * buffer.element_size()
    _check(lib.tl_kv_create(model, len(L_per_lane), max_ctx, ctypes.cast(arr, P), dtype,
                            _ptr(buffer), nbytes, ctypes.byref(out)))
    return out.value


def tl_kv_destroy(kv: int) -> None:
    _check(lib.tl_kv_destroy(kv))


def tl_kv_reset(kv: int, lane: int = -1, stream=None) -> None:
    _check(lib.tl_kv_reset(kv, lane, _stream(stream)))


def tl_kv_position(kv: int, lane: int) -> int:
    p = I()
    _check(lib.tl_kv_position(kv, lane, ctypes.byref(p)))
    return p.value


def tl_kv_set_position(kv: int, lane: int, pos: int, stream=None) -> None:
    _check(lib.tl_kv_set_position(kv, lane, pos, _stream(stream)))


def tl_kv_layer_ptrs(kv: int, lane: int, layer: int):
    k, v, ks, vs = P(), P(), P(), P()
    _check(lib.tl_kv_layer_ptrs(kv, lane, layer, ctypes.byref(k), ctypes.byref(v),
                                ctypes.byref(ks), ctypes.byref(vs)))
    return k.value, v.value, ks.value, vs.value


# --------------------------------------------------------------------- forward

def tl_prefill(model: int, ids=None, h_in=None, *, L: int, y_out, kv: Optional[int] = None,
               lane: int = 0, h_trace=None, stream=None) -> None:
    seq = (ids if ids is not None else h_in).shape[0]
    _check(lib.tl_prefill(model, _ptr(ids), _ptr(h_in), seq, L, kv, lane, _ptr(y_out),
                          _ptr(h_trace), _stream(stream)))


def tl_decode_step(model: int, kv: int, ids=None, h_in=None, *, L_per_lane: Sequence[int],
                   y_out, h_trace=None, stream=None) -> None:
    arr = _int_array(L_per_lane)
    _check(lib.tl_decode_step(model, kv, _ptr(ids), _ptr(h_in), ctypes.cast(arr, P),
                              len(L_per_lane), _ptr(y_out), _ptr(h_trace), _stream(stream)))


def tl_extend(model: int, kv: int, lane: int, ids=None, h_in=None, *, L: int, y_out,
              h_trace=None, stream=None) -> None:
    n = (ids if ids is not None else h_in).shape[0]
    _check(lib.tl_extend(model, kv, lane, _ptr(ids), _ptr(h_in), n, L, _ptr(y_out),
                         _ptr(h_trace), _stream(stream)))


def tl_greedy_head(model: int, y, ids, stream=None) -> None:
    _check(lib.tl_greedy_head(model, _ptr(y), y.shape[0], _ptr(ids), _stream(stream)))


def tl_spec_step(model: int, kv: int, lane: int, token: int, K: int, L_draft: int,
                 L_verify: int, stream=None):
    """Returns the emitted tokens (a list of 1 .. K + 1 ids)."""
    out = (ctypes.c_int32 * (K + 1))()
    n = I()
    _check(lib.tl_spec_step(model, kv, lane, token, K, L_draft, L_verify,
                            ctypes.cast(out, P), ctypes.byref(n), _stream(stream)))
    return list(out[:n.value])


def tl_linear_workspace_bytes(N: int, K: int, T: int) -> int:
    b = SZ()
    _check(lib.tl_linear_workspace_bytes(N, K, T, ctypes.byref(b)))
    return b.value


def tl_linear(packed, scales, N: int, K: int, group: int, x, y, workspace=None,
              stream=None) -> None:
    T = x.shape[0]
    _check(lib.tl_linear(_ptr(packed), _ptr(scales), N, K, group, _ptr(x), T, _ptr(y),
                         _ptr(workspace), _stream(stream)))


def tl_linear_noalloc(packed, scales, N: int, K: int, group: int, x, y, stream=None) -> None:
    T = x.shape[0]
    _check(lib.tl_linear_noalloc(_ptr(packed), _ptr(scales), N, K, group, _ptr(x), T, _ptr(y),
                                 _stream(stream)))


def tl_read_probe(buf, passes: int, sink, stream=None) -> None:
    """Read `buf` (a 16-byte aligned device tensor) `passes` times."""
    nbytes = buf.numel() * buf.element_size()
    _check(lib.tl_read_probe(_ptr(buf), nbytes, passes, _ptr(sink), _stream(stream)))


def tl_check_bounded_wait(model: int, limit_us: int, stream=None) -> None:
    _check(lib.tl_check_bounded_wait(model, limit_us, _stream(stream)))


def tl_sync_status(model: int, stream=None) -> int:
    """Returns the status code (does not raise) so callers can test for it."""
    return lib.tl_sync_status(model, _stream(stream))
