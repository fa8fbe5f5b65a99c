"""Models with a 4-bit KV cache: the hot path's codes, decode against the
oracle, per-lane independence, extend and speculative steps, and a run of the
cache with the scoring head."""
import numpy as np
import pytest
import torch

import synthetic as syn
import weight_shared_looped_b200 as tl
from oracle import tinyloop_oracle as o

from gpu_util import cosine, device_blocks, device_model, oracle_model, rel_l2, to_dev
from int4_util import pack

pytestmark = pytest.mark.gpu

W = syn.WORKLOADS["tiny"]


def _raw(kv, ptr, shape, dtype):
    off = ptr - kv.buffer.data_ptr()
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    return kv.buffer[off:off + n].view(dtype).view(*shape)


def _fill(m, dtype, Ls, prompts, steps, max_ctx, use_ids, extend=()):
    kv = m.new_kv(Ls, max_ctx=max_ctx, dtype=dtype)
    dev = (lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()) if use_ids else (lambda a: to_dev(a, torch.float16))
    key = "ids" if use_ids else "h_in"
    for b, p in enumerate(prompts):
        m.prefill(**{key: dev(p)}, L=Ls[b], kv=kv, lane=b)
    for s in steps:
        m.decode(kv, **{key: dev(s)}, L_per_lane=Ls)
    for b, e in enumerate(extend):
        m.extend(kv, **{key: dev(e)}, lane=b, L=Ls[b])
    assert m.sync_status() == tl.TL_OK
    return kv


def _check_codes(kv16, kv4, lane, H, hd, n):
    """Layer 0 depends on no cached entry: the FP16 cache holds the rows the 4-bit
    cache quantised."""
    p16, p4 = kv16.layer_ptrs(lane, 0), kv4.layer_ptrs(lane, 0)
    for i, name in ((0, "K"), (1, "V")):
        rows = _raw(kv16, p16[i], (H, kv16.max_ctx, hd), torch.int16)[:, :n].cpu().numpy().view(np.float16)
        words = _raw(kv4, p4[i], (H, kv4.max_ctx, hd // 8), torch.int32)[:, :n].cpu().numpy()
        prm = _raw(kv4, p4[2 + i], (H, kv4.max_ctx, hd // 32, 2), torch.int16)[:, :n].cpu().numpy().view(np.float16)
        c, s, z = o.kv_quant_int4(rows)
        assert np.array_equal(words, pack(c)), name
        assert np.array_equal(prm[..., 0].view(np.uint16), s.view(np.uint16)), name
        assert np.array_equal(prm[..., 1].view(np.uint16), z.view(np.uint16)), name


@pytest.mark.parametrize("graphs", [True, False])
def test_hot_path_codes_bit_exact(graphs):
    m = device_model("tiny", max_tokens=64, max_lanes=2, max_ctx=64)
    m.set_graphs(graphs)
    P, S, E, Ls = 37, 3, 5, [2, 1]
    prompts = [syn.hidden_input(W, P, name=f"int4.prompt{b}") for b in range(2)]
    steps = [np.stack([syn.hidden_input(W, 1, name=f"int4.step{s}.{b}")[0] for b in range(2)]) for s in range(S)]
    ext = [syn.hidden_input(W, E, name=f"int4.ext{b}") for b in range(2)]
    kv16, kv4 = (_fill(m, d, Ls, prompts, steps, 64, False, ext) for d in ("fp16", "int4"))
    for lane in range(2):
        _check_codes(kv16, kv4, lane, W.shape.n_heads, W.shape.head_dim, P + S + E)
    kv16.close()
    kv4.close()
    m.close()


def test_407m_hot_path_codes_bit_exact():
    w = syn.WORKLOADS["prefill407m"]
    m = device_model("prefill407m", max_tokens=128, max_lanes=2, max_ctx=160)
    prompts = [syn.token_ids(128, w.seed, f"int4.prompt{b}") for b in range(2)]
    steps = [syn.token_ids(2, w.seed, f"int4.step{s}") for s in range(2)]
    kv16, kv4 = (_fill(m, d, [2, 1], prompts, steps, 160, True) for d in ("fp16", "int4"))
    for lane in range(2):
        _check_codes(kv16, kv4, lane, w.shape.n_heads, w.shape.head_dim, 130)
    kv16.close()
    kv4.close()
    m.close()


def test_decode_matches_the_oracle():
    """Teacher-forced decode after a prompt against the oracle's 4-bit cache.  The
    two sides' rows differ by the float path (the block bound 5e-3 of the other
    cache types); where such a difference crosses a rounding boundary a code moves
    by one step, of which there are 15 to a group's range, so a row's stored value
    is off by a step of about 0.27 of its deviation in a small share of places: the
    bound is that of the long-prompt decode tests, 1e-2, and the cosine bound."""
    P, S, L = 20, 6, 2
    m = device_model("tiny", max_tokens=64, max_ctx=64)
    om = oracle_model("tiny")
    kv, okv = m.new_kv([L], max_ctx=64, dtype="int4"), om.new_kv(L, "int4")
    prompt = syn.hidden_input(W, P, name="int4.o.prompt")
    y = m.prefill(h_in=to_dev(prompt, torch.float16), L=L, kv=kv)
    ry = om.prefill(prompt.astype(np.float64), L, kv=okv)
    assert rel_l2(y.cpu().numpy(), ry) <= 5e-3
    for s in range(S):
        x = syn.hidden_input(W, 1, name=f"int4.o.step{s}")
        y = m.decode(kv, h_in=to_dev(x, torch.float16), L_per_lane=[L]).cpu().numpy()[0]
        ry = om.decode_step(x[0].astype(np.float64), L, okv)
        assert rel_l2(y, ry) <= 1e-2 and cosine(y, ry) >= 0.999, s
    kv.close()
    m.close()


def test_lanes_are_independent():
    """Each lane of a batch equals its own run bit for bit, at every loop count."""
    Ls, P = [1, 3, 2], [9, 40, 0]
    m = device_model("tiny", max_tokens=64, max_lanes=3, max_ctx=96)
    prompts = [syn.hidden_input(W, p, name=f"int4.l.prompt{b}") if p else None for b, p in enumerate(P)]
    steps = [[syn.hidden_input(W, 1, name=f"int4.l.step{s}.{b}") for b in range(3)] for s in range(4)]
    kv = m.new_kv(Ls, max_ctx=96, dtype="int4")
    for b, p in enumerate(prompts):
        if p is not None:
            m.prefill(h_in=to_dev(p, torch.float16), L=Ls[b], kv=kv, lane=b)
    batch = [m.decode(kv, h_in=to_dev(np.concatenate(s), torch.float16), L_per_lane=Ls).cpu().numpy() for s in steps]
    kv.close()
    for b in range(3):
        one = m.new_kv([Ls[b]], max_ctx=96, dtype="int4")
        if prompts[b] is not None:
            m.prefill(h_in=to_dev(prompts[b], torch.float16), L=Ls[b], kv=one, lane=0)
        for s, x in enumerate(steps):
            y = m.decode(one, h_in=to_dev(x[b], torch.float16), L_per_lane=[Ls[b]]).cpu().numpy()[0]
            assert np.array_equal(y, batch[s][b]), (b, s)
        one.close()
    m.close()


@pytest.mark.parametrize("ctx", [1000, 8200])
def test_any_number_of_lanes_of_sixteen_heads(ctx):
    """The work is spread differently for 1, 3 and 8 lanes (8200 positions: through a
    workspace), and over one query and several: the same bits."""
    w, L, steps = syn.WORKLOADS["prefill407m"], 2, 2
    H, hd = w.shape.n_heads, w.shape.head_dim
    m = device_model("prefill407m", max_tokens=16, max_lanes=8, max_ctx=ctx)
    pos = [ctx - 9, 7, ctx // 2, 129, 0, ctx - steps, 64, 31]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (2, H, ctx, hd // 8), dtype=torch.int32, device="cuda", generator=gen)
    scale = 0.2 * torch.rand(2, H, ctx, hd // 32, device="cuda", generator=gen)
    params = torch.stack((scale, torch.randn(scale.shape, device="cuda", generator=gen) - 7.5 * scale), -1).half()
    ids = torch.from_numpy(syn.token_ids(8 * steps, 71, "int4.lanes").reshape(steps, 8)).cuda()

    def new(lanes):
        kv = m.new_kv([L] * len(lanes), max_ctx=ctx, dtype="int4")
        for at, b in enumerate(lanes):
            for layer in range(w.n_pre + L):
                p = kv.layer_ptrs(at, layer)
                for i in range(2):                     # lanes and layers differ by a rotation of the positions
                    turn = 13 * b + 5 * layer
                    _raw(kv, p[i], (H, ctx, hd // 8), torch.int32).copy_(codes[i].roll(turn, 1))
                    _raw(kv, p[2 + i], (H, ctx, hd // 32, 2), torch.float16).copy_(params[i].roll(turn, 1))
            kv.set_position(at, pos[b])
        return kv

    def run(lanes):
        kv = new(lanes)
        ys = [m.decode(kv, ids[s][lanes].contiguous(), L_per_lane=[L] * len(lanes)).cpu().numpy() for s in range(steps)]
        kv.close()
        return np.stack(ys, 1)
    batch = run(list(range(8)))
    assert np.isfinite(batch).all()
    for lanes in ([0], [2], [5], [4], [0, 5, 2]):
        assert np.array_equal(run(lanes), batch[lanes]), lanes
    a, b = new([0]), new([0])
    x = ids.flatten()[:8].contiguous()
    together = m.extend(a, x, lane=0, L=L).cpu().numpy()
    alone = np.concatenate([m.extend(b, x[i:i + 1], lane=0, L=L).cpu().numpy() for i in range(8)])
    assert np.array_equal(together, alone)
    c = new([0])
    steps_ = np.concatenate([m.decode(c, x[i:i + 1], L_per_lane=[L]).cpu().numpy() for i in range(8)])
    assert np.array_equal(together, steps_)
    for layer in range(w.n_pre + L):                   # and the same entries
        for pa, pc, words in zip(a.layer_ptrs(0, layer), c.layer_ptrs(0, layer), (hd // 8, hd // 8, hd // 32, hd // 32)):
            assert torch.equal(_raw(a, pa, (H, ctx, words), torch.int32), _raw(c, pc, (H, ctx, words), torch.int32))
    for kv in (a, b, c):
        kv.close()
    m.close()


@pytest.mark.parametrize("start", [0, 1, 13, 16, 60])
def test_extend_equals_decode_steps(start):
    n, L = 8, 2
    m = device_model("tiny", max_tokens=64, max_lanes=2, max_ctx=80)
    x = syn.hidden_input(W, n, name="int4.e.x")
    ys = []
    for mode in range(2):
        kv = m.new_kv([1, L], max_ctx=80, dtype="int4")
        if start:
            m.prefill(h_in=to_dev(syn.hidden_input(W, start, name="int4.e.p"), torch.float16), L=L, kv=kv, lane=1)
        if mode == 0:
            ys.append(m.extend(kv, h_in=to_dev(x, torch.float16), lane=1, L=L).cpu().numpy())
        else:
            ys.append(np.stack([m.extend(kv, h_in=to_dev(x[i:i + 1], torch.float16), lane=1, L=L).cpu().numpy()[0]
                                for i in range(n)]))
        assert kv.position(1) == start + n
        kv.close()
    assert np.array_equal(ys[0], ys[1])
    m.close()


def test_speculative_steps_emit_greedy_tokens():
    E = (syn.normal((1000, 256), 0.02, 0, "spec.embed")).astype(np.float16)
    blocks = device_blocks("tiny")
    from weight_shared_looped_b200.model import DeviceModel
    m = DeviceModel([], blocks["loop"], syn.final_gain(W.shape, W.seed), E, max_tokens=16, max_ctx=64)
    prompt = torch.from_numpy(syn.token_ids(8, 0, "int4.spec", 1000)).cuda()
    kv = m.new_kv([4], max_ctx=64, dtype="int4")
    m.prefill(prompt, L=4, kv=kv)
    tok, want = 5, []
    for _ in range(16):
        y = m.decode(kv, torch.tensor([tok], dtype=torch.int32, device="cuda"), L_per_lane=[4])
        tok = int(m.greedy_head(y)[0])
        want.append(tok)
    kv.reset()
    m.prefill(prompt, L=4, kv=kv)
    got = [5]
    while len(got) < 17:
        got += m.spec_step(kv, got[-1], K=3, L_draft=2, L_verify=4)
    assert got[1:17] == want
    kv.close()
    m.close()


def test_graph_replay_equals_direct_launches_and_rebuilt_caches():
    Ls = [2, 2]
    m = device_model("tiny", max_tokens=64, max_lanes=2, max_ctx=64)
    x = [syn.hidden_input(W, 2, name=f"int4.g{s}") for s in range(3)]
    outs = []
    for graphs in (True, False, True):
        m.set_graphs(graphs)
        kv = m.new_kv(Ls, max_ctx=64, dtype="int4")
        kv.buffer[4096:] = 0xFF      # entries nobody wrote hold NaN
        outs.append([m.decode(kv, h_in=to_dev(s, torch.float16), L_per_lane=Ls).cpu().numpy() for s in x])
        kv.close()
    for a in outs[1:]:
        for p, q in zip(outs[0], a):
            assert np.isfinite(p).all() and np.array_equal(p, q)
    m.close()


def test_a_run_of_them_together():
    """A 407M-shaped model decodes with a 4-bit cache; the caller reads the cached
    rows of a layer back, attends over them itself, and scores the tokens."""
    w = syn.WORKLOADS["decode407m"]
    H, hd, P, S = w.shape.n_heads, w.shape.head_dim, 100, 3
    m = device_model("decode407m", max_tokens=128, max_ctx=128)
    ids = syn.token_ids(P + S + 1, 0, "int4.run")
    ys = {}
    for dtype in ("fp16", "int4"):
        kv = m.new_kv([4], max_ctx=128, dtype=dtype)
        m.prefill(torch.from_numpy(ids[:P]).cuda(), L=4, kv=kv)
        ys[dtype] = torch.cat([m.decode(kv, torch.from_numpy(ids[P + s:P + s + 1]).cuda(), L_per_lane=[4]).clone()
                               for s in range(S)])
        if dtype == "fp16":
            k16 = _raw(kv, kv.layer_ptrs(0, 0)[0], (H, 128, hd), torch.int16).clone()
            kv.close()
    kc, vc, kp, vp = kv.layer_ptrs(0, 0)
    t = [_raw(kv, kc, (1, H, 128, hd // 8), torch.int32), _raw(kv, kp, (1, H, 128, hd // 32, 2), torch.float16),
         _raw(kv, vc, (1, H, 128, hd // 8), torch.int32), _raw(kv, vp, (1, H, 128, hd // 32, 2), torch.float16)]
    n = P + S
    k, v = (torch.zeros(n, H * hd, dtype=torch.float16, device="cuda") for _ in range(2))
    tl.tl_kv_read_int4(*t, torch.zeros(1, dtype=torch.int32, device="cuda"), k, v)
    rows = k16.cpu().numpy().view(np.float16)[:, :n]
    c, s, z = o.kv_quant_int4(rows)
    want = o.kv_dequant_int4(c, s, z).astype(np.float16).transpose(1, 0, 2).reshape(n, -1)
    assert np.array_equal(k.cpu().numpy(), want)
    # the last position's attention over the cache equals attention over the rows read back
    q = torch.from_numpy(syn.normal((1, H * hd), 1.0, 0, "int4.run.q").astype(np.float16)).cuda()
    out = torch.empty_like(q)
    tl.tl_attention_int4(q, *t, torch.tensor([n], dtype=torch.int32, device="cuda"), out)
    kk, vv = (a.double().view(n, H, hd) for a in (k, v))
    p = torch.softmax(torch.einsum("hd,jhd->hj", q.double().view(H, hd), kk) / hd ** 0.5, -1)
    ref = torch.einsum("hj,jhd->hd", p, vv).reshape(1, -1)
    assert rel_l2(out.double().cpu(), ref.cpu()) <= 2e-3
    nxt = torch.from_numpy(ids[P + 1:P + S + 1]).cuda()
    a, b = m.score(ys["fp16"], nxt, k=4), m.score(ys["int4"], nxt, k=4)
    for got in (a, b):
        assert (got["logp"] <= 0).all() and (got["top"][:, 0] >= got["logp"]).all()
        assert ((got["entropy"] > 0) & (got["entropy"] <= np.log(50257) + 1e-4)).all()
    assert torch.equal(a["ids"][:, 0], m.greedy_head(ys["fp16"]))
    kv.close()
    m.close()


def test_the_chunk_knob_leaves_a_4bit_cache_alone():
    """tl_model_set_decode_chunks sets how other caches are streamed; no value of it changes a
    4-bit cache's results."""
    m = device_model("tiny", max_tokens=64, max_lanes=1, max_ctx=128)
    x = to_dev(syn.hidden_input(syn.WORKLOADS["tiny"], 41, name="int4.knob"), torch.float16)
    outs = []
    for chunks in (0, 1, 3, 8):
        m.set_decode_chunks(chunks)
        kv = m.new_kv([2], max_ctx=100, dtype="int4")
        m.prefill(h_in=x[:40], L=2, kv=kv, lane=0)
        outs.append(m.decode(kv, h_in=x[40:], L_per_lane=[2]).cpu())
        assert m.sync_status() == tl.TL_OK
        kv.close()
    for y in outs[1:]:
        assert torch.equal(y, outs[0])
    m.close()
