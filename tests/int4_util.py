"""Helpers of the 4-bit KV cache tests: caches built by the oracle's quantiser,
read and attended in fp64."""
from __future__ import annotations

import numpy as np
import torch

from oracle import tinyloop_oracle as o


def pack(codes: np.ndarray) -> np.ndarray:
    """codes [..., hd] -> int32 words [..., hd / 8], element 8j + i in bits 4i of word j."""
    c = codes.reshape(codes.shape[:-1] + (codes.shape[-1] // 8, 8)).astype(np.uint32)
    return (c << (4 * np.arange(8, dtype=np.uint32))).sum(-1, dtype=np.uint32).view(np.int32)


def unpack(words: np.ndarray) -> np.ndarray:
    c = (words.view(np.uint32)[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15
    return c.reshape(words.shape[:-1] + (words.shape[-1] * 8,)).astype(np.uint8)


def quantise(rows: np.ndarray):
    """rows fp16 [..., hd] -> (words int32 [..., hd / 8], params fp16 [..., hd / 32, 2])."""
    c, s, z = o.kv_quant_int4(rows)
    return pack(c), np.stack([s, z], -1)


def values(words: np.ndarray, params: np.ndarray) -> np.ndarray:
    """The values held, in fp64 [..., hd]."""
    return o.kv_dequant_int4(unpack(words), params[..., 0], params[..., 1])


class Cache:
    """K and V caches of [lanes, heads, ctx] rows quantised on the host, and their device copies.
    rows: fp16 [lanes, heads, ctx, hd] for K and for V."""

    def __init__(self, k: np.ndarray, v: np.ndarray, lane_pad: int = 0):
        self.kw, self.kp = quantise(k)
        self.vw, self.vp = quantise(v)
        self.upload(lane_pad)

    def upload(self, lane_pad: int = 0):
        """lane_pad: extra positions between lanes (a lane stride above the lane's size)."""
        def dev(a):
            t = torch.from_numpy(a).cuda()
            if not lane_pad:
                return t
            big = torch.zeros((t.shape[0], t.shape[1] * (t.shape[2] + lane_pad)) + t.shape[3:],
                              dtype=t.dtype, device="cuda")
            view = big[:, :t.shape[1] * t.shape[2]].view(t.shape)
            view.copy_(t)
            return view
        self.t = [dev(a) for a in (self.kw, self.kp, self.vw, self.vp)]

    def K(self, lane):
        return values(self.kw[lane], self.kp[lane])

    def V(self, lane):
        return values(self.vw[lane], self.vp[lane])


def attend(q, K, V, length, n_q, window):
    """fp64 attention of one lane: q [n_q, q_heads, hd], K, V [heads, ctx, hd].  Returns the
    outputs [n_q, q_heads, hd] and a bound of the kernel's error, element by element.

    Roundings of the kernel, in half steps u = 2^-11 of fp16: each value of K and V to fp16 (u of
    the value), each softmax weight to fp16 (u, or 2^-25 where it is subnormal; the largest weight
    is at least 1), the output (u).  A score thus moves by at most u * sum |q_i k_i| / sqrt(hd) =
    e, and a normalised weight by a factor within exp(2 e).  fp32 sums add at most
    (keys + hd) 2^-23 relative to the sum of magnitudes."""
    heads, ctx, hd = K.shape
    group = q.shape[1] // heads
    out = np.zeros((n_q, q.shape[1], hd))
    tol = np.zeros_like(out)
    u = 2.0 ** -11
    for i in range(n_q):
        p = min(length, ctx) - n_q + i
        if p < 0:
            continue
        lo = max(0, p - window + 1) if window > 0 else 0
        for h in range(q.shape[1]):
            k, v = K[h // group, lo:p + 1], V[h // group, lo:p + 1]
            s = k @ q[i, h] / np.sqrt(hd)
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ v
            mag = np.abs(k) @ np.abs(q[i, h]) / np.sqrt(hd)
            f32 = (len(s) + hd) * 2.0 ** -23
            e = (u + f32) * mag.max()
            rel = np.expm1(2 * e) + 2 * u + f32
            tol[i, h] = (w @ np.abs(v)) * rel + 2.0 ** -25 * np.abs(v).sum(0)
            tol[i, h] += np.abs(out[i, h]) * u + 2.0 ** -25
    return out, tol


def narrow_groups():
    """Groups whose ranges pass through the subnormal scales, from 2^-24 to 2^-9, at zero points
    of several sizes; fp16 [n, 64]."""
    rng = np.random.default_rng(9)
    span = np.exp2(np.linspace(-24, -9, 240))[:, None] * rng.random((240, 64))
    span[:, ::32], span[:, 1::32] = 0, np.exp2(np.linspace(-24, -9, 240))[:, None]
    span[0, 1::32] = 28.5 * 2.0 ** -24                      # scale 2^-24, nearly two steps a unit
    lo = np.array([0.0, -2.0 ** -14, 2.0 ** -12, -1.0])[np.arange(240) % 4, None]
    return (lo + span).astype(np.float16)


def held_bound(x):
    """How far a value may be from the one held, element by element: half a scale, or at the
    upper end what rounding the scale towards zero takes (kv_int4.cuh); fp32 steps 2^-22."""
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32)).astype(np.float64)
    width = g.max(-1, keepdims=True) - g.min(-1, keepdims=True)
    most = np.maximum(np.maximum(width / 30, width * 2.0 ** -10), np.minimum(width, 15 * 2.0 ** -24))
    return np.broadcast_to(most * (1 + 2.0 ** -22) + width * 2.0 ** -22, g.shape).reshape(x.shape)
