"""Softmax attention with its row statistics and its backward pass: argument checks on the CPU,
and results on the GPU against the formulas in 64 bits.

Error bounds, with e = finfo(type).eps / 2 (the most a rounding to the type changes a value,
relative to it) and, for the sums of the tensor cores and the exponentials, 2^-13 relative to
the sum of the absolute values (exponents up to 2^6 in log2 units, computed in fp32 with
relative error 2^-24 of up to 2^7, an exponential of 2 ulp, fp32 accumulation of at most 2^13
terms whose errors partly cancel):
    o     P is rounded once, o once:                 (e + 2^-13) sum_j P |v| + e |o|
    dv    P is rounded once, dv once:                (e + 2^-13) sum_i P |do| + e |dv|
    dq    dS is rounded once, dq once; delta is made of the rounded o, off by at most
          e sum_c |do o|:  (e + 2^-13) A + e |dq|,  A = scale sum_j P (|dP| + 2 sum_c |do o|) |k|
    dk    the same with the sum over the rows.
fp16 cannot hold values below 2^-14 to e relative: a rounding adds at most 2^-25 per term there.
"""
import ctypes
import importlib.util
import os
import re

import numpy as np
import pytest
import torch

from softmax_attention_ar_b200 import arl2

BF, HF = torch.bfloat16, torch.float16
SUM = 2.0 ** -13


def visible(B, Tq, Tk, q_len, k_len, frame_len, q_start):
    """[B, Tq, Tk] mask in plain loops over nothing but comparisons."""
    i, j = torch.arange(Tq)[None, :, None], torch.arange(Tk)[None, None, :]
    m = torch.ones(B, Tq, Tk, dtype=torch.bool)
    if q_len is not None:
        m &= i < torch.tensor(q_len)[:, None, None]
    if k_len is not None:
        m &= j < torch.tensor(k_len)[:, None, None]
    if frame_len:
        m &= j < (torch.div(i + q_start, frame_len, rounding_mode="floor") + 1) * frame_len
    return m


def reference(q, k, v, do, m, scale):
    """fp64 results and the sums of absolute values that bound the errors; heads first."""
    group = q.shape[2] // k.shape[2]
    q, do = (t.double().permute(0, 2, 1, 3) for t in (q, do))
    k, v = (t.double().permute(0, 2, 1, 3).repeat_interleave(group, 1) for t in (k, v))
    m = m.to(q.device)[:, None]
    s = torch.where(m, scale * (q @ k.transpose(2, 3)), -float("inf"))
    lse = torch.logsumexp(s, 3)
    p = torch.where(m, torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None]), 0.0)
    o = p @ v
    dp = do @ v.transpose(2, 3)
    delta = (do * o).sum(3, keepdim=True)
    ds = p * (dp - delta)
    fold = lambda t: t.unflatten(1, (-1, group)).sum(2)
    big = p * (dp.abs() + 2 * (do * o).abs().sum(3, keepdim=True))
    r = dict(o=o, lse=lse, dq=scale * ds @ k, dk=fold(scale * ds.transpose(2, 3) @ q), dv=fold(p.transpose(2, 3) @ do))
    a = dict(o=p @ v.abs(), dq=scale * big @ k.abs(), dk=fold(scale * big.transpose(2, 3) @ q.abs()),
             dv=fold(p.transpose(2, 3) @ do.abs()))
    # Terms summed, times the other factor: what fp16's smallest steps can add up to.
    one = m.double().expand_as(p)
    t = dict(o=one @ v.abs(), dq=scale * one @ k.abs(), dk=fold(scale * one.transpose(2, 3) @ q.abs()),
             dv=fold(one.transpose(2, 3) @ do.abs()))
    return r, a, t


def make(B, Tq, Tk, H, Hkv, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)
    return r(B, Tq, H, d), r(B, Tk, Hkv, d), r(B, Tk, Hkv, d), r(B, Tq, H, d)


def close(got, r, a, t, name, dtype):
    got = got.double().permute(0, 2, 1, 3)
    e = torch.finfo(dtype).eps / 2
    bound = (e + SUM) * a[name] + e * r[name].abs()
    if dtype == HF:
        bound = bound + 2.0 ** -25 * (t[name] + 1)
    assert torch.isfinite(got).all(), name
    worst = ((got - r[name]).abs() - bound - 1e-30).max().item()
    assert worst <= 0, f"{name}: off by {worst:.3e} more than its bound"


def check(B, Tq, Tk, H, Hkv, d, dtype, q_len=None, k_len=None, frame_len=0, q_start=0, scale=None, seed=0, op=None,
          inputs=None, garbage=True):
    q, k, v, do = inputs or make(B, Tq, Tk, H, Hkv, d, dtype, seed)
    m = visible(B, Tq, Tk, q_len, k_len, frame_len, q_start)
    clean = [t.clone() for t in (q, k, v, do)]
    if garbage:   # what stands behind a length must not matter
        for b in range(B):
            for t, n in ((q, q_len), (do, q_len), (k, k_len), (v, k_len)):
                if n is not None:
                    t[b, max(0, n[b]):] = float("nan")
    for b in range(B):
        for t, n in zip(clean, (q_len, k_len, k_len, q_len)):
            if n is not None:
                t[b, max(0, n[b]):] = 0
    dev = lambda n: None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda")
    kw = dict(q_len=dev(q_len), k_len=dev(k_len), frame_len=frame_len, q_start=q_start, scale=scale)
    op = op or arl2.SoftmaxAttention(H, Tq, Tk, d, B=B, H_kv=Hkv, dtype=dtype)
    o, lse = op.forward(q, k, v, **kw)
    assert op.status() == arl2.ARL2_OK
    r, a, t = reference(*clean[:3], clean[3], m, scale or d ** -0.5)
    close(o, r, a, t, "o", dtype)
    seen = torch.isfinite(r["lse"])
    assert torch.equal(torch.isneginf(lse), ~seen)
    # lse: the exponent's error, 2^-24 of the largest |score|, and that of the sum's logarithm.
    assert ((lse.double() - r["lse"])[seen].abs() <= 2.0 ** -13 + 2.0 ** -22 * r["lse"][seen].abs()).all()
    grads = op.backward(do, q, k, v, o, lse, **kw)
    assert op.status() == arl2.ARL2_OK
    for name, got in zip(("dq", "dk", "dv"), grads):
        close(got, r, a, t, name, dtype)
    for b in range(B):
        if q_len is not None:
            assert (o[b, max(0, q_len[b]):] == 0).all() and (grads[0][b, max(0, q_len[b]):] == 0).all()
        if k_len is not None:
            assert (grads[1][b, max(0, k_len[b]):] == 0).all() and (grads[2][b, max(0, k_len[b]):] == 0).all()
    return op, (q, k, v, do, o, lse, grads, kw)


def on_gpu(f):
    return pytest.mark.gpu(pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")(f))


@on_gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("Tq,Tk", [(1, 1), (1, 200), (127, 128), (128, 129), (129, 127), (257, 300), (300, 1)])
def test_small_shapes(Tq, Tk, d, dtype):
    check(2, Tq, Tk, 2, 2, d, dtype, seed=Tq + Tk)


@on_gpu
@pytest.mark.parametrize("H,Hkv", [(4, 1), (6, 2), (3, 3)])
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, HF)])
def test_shared_key_heads(H, Hkv, d, dtype):
    check(2, 200, 333, H, Hkv, d, dtype, seed=H)


@on_gpu
@pytest.mark.parametrize("Tq,Tk,frame_len,q_start", [
    (300, 300, 1, 0),        # causal
    (260, 400, 1, 140),      # causal, the queries at the end
    (512, 512, 128, 0),      # frames of a tile
    (500, 500, 61, 0),       # frames across tiles
    (300, 300, 7, -50),      # rows before the first key see nothing
    (130, 200, 1000, 5),     # one frame holds all
    (40, 500, 100, 100),
])
@pytest.mark.parametrize("d,dtype", [(128, BF), (32, HF)])
def test_frames(Tq, Tk, frame_len, q_start, d, dtype):
    check(2, Tq, Tk, 2, 1, d, dtype, frame_len=frame_len, q_start=q_start, seed=Tq)


@on_gpu
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, HF)])
@pytest.mark.parametrize("frame_len", [0, 1, 50])
def test_lengths(d, dtype, frame_len):
    # Full, ending in a tile, on a tile's edge, one, empty on either side.
    check(6, 300, 280, 2, 1, d, dtype, q_len=[300, 130, 256, 1, 0, 77], k_len=[280, 131, 128, 1, 90, 0],
          frame_len=frame_len, seed=1)


@on_gpu
@pytest.mark.parametrize("B,T,H,frame_len", [(70, 150, 2, 0), (33, 300, 1, 16), (1, 2500, 2, 200), (2, 2600, 1, 1)])
def test_padded_batches(B, T, H, frame_len):
    # Batches by lanes of the warp that cuts the work, several rounds of them, or one after another.
    g = np.random.default_rng(B)
    q_len, k_len = (g.integers(0, T + 1, B).tolist() for _ in range(2))
    q_len[0], k_len[0] = T - 3, T - 70
    check(B, T, T, H, 1, 64, BF, q_len=q_len, k_len=k_len, frame_len=frame_len, seed=B)


@on_gpu
def test_every_row_empty():
    check(2, 70, 90, 2, 2, 64, BF, k_len=[0, 0])
    check(1, 70, 90, 2, 2, 64, BF, frame_len=10, q_start=-200)


@on_gpu
@pytest.mark.parametrize("B,T,H,Hkv,d,dtype", [
    (1, 1560, 12, 12, 128, BF), (1, 1560, 4, 2, 64, HF), (2, 2048, 3, 1, 32, BF)])
def test_frame_sizes(B, T, H, Hkv, d, dtype):
    check(B, T, T, H, Hkv, d, dtype)


@on_gpu
def test_one_query_over_a_long_cache():
    check(3, 1, 9000, 4, 2, 128, BF, k_len=[9000, 4500, 17])


@on_gpu
def test_long_keys_few_heads_split_a_tile_many_ways():
    check(1, 100, 20000, 1, 1, 64, BF)
    check(1, 5000, 100, 2, 1, 128, BF)


@on_gpu
def test_views_of_a_packed_projection():
    B, T, H, Hkv, d = 2, 333, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn(B, T, H + 2 * Hkv, d, generator=g, device="cuda").to(BF)
    heads_first = lambda t: t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    do = heads_first(torch.randn(B, T, H, d, generator=g, device="cuda").to(BF))
    op, (_, _, _, _, o, lse, grads, kw) = check(B, T, T, H, Hkv, d, BF, inputs=(q, k, v, do), garbage=False)
    # Outputs into views, beside data that stays.
    buf = torch.full((B, T, H + 2 * Hkv + 1, d), 7.0, device="cuda", dtype=BF)
    out = heads_first(torch.empty(B, T, H, d, device="cuda", dtype=BF))
    o2, lse2 = op.forward(q, k, v, out=out)
    op.backward(do, q, k, v, o, lse, dq=buf[:, :, :H], dk=buf[:, :, H:H + Hkv], dv=buf[:, :, H + Hkv:-1])
    torch.cuda.synchronize()
    assert o2 is out and torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(buf[:, :, :H], grads[0]) and torch.equal(buf[:, :, H:H + Hkv], grads[1])
    assert torch.equal(buf[:, :, H + Hkv:-1], grads[2]) and (buf[:, :, -1] == 7).all()


@on_gpu
def test_offsets_beyond_32_bits():
    # Every tensor a view whose last token lies 6 GiB behind its first.
    T, d, step = 4, 32, 1 << 30
    big = torch.empty((T - 1) * step + 4096, dtype=BF, device="cuda")
    views = [torch.as_strided(big, (1, T, 1, d), (big.numel(), step, d, 1), 64 * i) for i in range(8)]
    q, k, v, do = make(1, T, T, 1, 1, d, BF, seed=9)
    for dst, src in zip(views, (q, k, v, do)):
        dst.copy_(src)
    op = arl2.SoftmaxAttention(1, T, T, d)
    o, lse = op.forward(q, k, v, frame_len=1)
    want = (o,) + op.backward(do, q, k, v, o, lse, frame_len=1)
    o2, lse2 = op.forward(*views[:3], out=views[4], frame_len=1)
    got = (o2,) + op.backward(views[3], *views[:3], o2, lse2, dq=views[5], dk=views[6], dv=views[7], frame_len=1)
    assert torch.equal(lse, lse2) and all(torch.equal(x, y) for x, y in zip(want, got))
    assert op.status() == arl2.ARL2_OK


@on_gpu
def test_nan_and_infinity_in_seen_places_stay_in_their_rows():
    # A NaN key makes the rows that see it NaN and no others; an infinite score as well.
    for bad in (float("nan"), float("inf")):
        q, k, v, do = make(1, 300, 300, 2, 2, 64, BF, seed=10)
        k[0, 200, 0, 0] = bad
        q[0, :, 0, 0] = q[0, :, 0, 0].abs() + 0.1
        op = arl2.SoftmaxAttention(2, 300, 300, 64)
        o, lse = op.forward(q, k, v, frame_len=100)
        assert op.status() == arl2.ARL2_OK
        assert torch.isnan(lse[0, 0, 200:]).all() and torch.isnan(o[0, 200:, 0]).all()
        assert torch.isfinite(lse[0, 0, :200]).all() and torch.isfinite(o[0, :200, 0]).all()
        assert torch.isfinite(lse[0, 1]).all() and torch.isfinite(o[0, :, 1]).all()


@on_gpu
@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_nan_query_shows_in_all_its_gradients(dtype):
    # Whichever column it is in: dv of every key that it sees, dk as well, and its own dq.
    T, H, d, F = 150, 2, 64, 50
    op = arl2.SoftmaxAttention(H, T, T, d, dtype=dtype)
    for i in range(60, 76):
        q, k, v, do = make(1, T, T, H, H, d, dtype, seed=11)
        q[0, i, 0, 3] = float("nan")
        o, lse = op.forward(q, k, v, frame_len=F)
        dq, dk, dv = op.backward(do, q, k, v, o, lse, frame_len=F)
        assert op.status() == arl2.ARL2_OK
        assert torch.isnan(o[0, i, 0]).all() and torch.isnan(dq[0, i, 0]).all()
        assert not torch.isfinite(dv[0, :100, 0]).any() and not torch.isfinite(dk[0, :100, 0, 3]).any()
        assert torch.isfinite(dv[0, 100:, 0]).all()
        assert all(torch.isfinite(t[0, :, 1]).all() for t in (o, dq, dk, dv))


@on_gpu
def test_smaller_calls_on_one_context_and_repeats():
    op = arl2.SoftmaxAttention(4, 700, 900, 128, B=2, H_kv=2)
    for Tq, Tk, F in ((700, 900, 0), (1, 900, 0), (257, 100, 1), (700, 700, 64)):
        _, (q, k, v, do, o, lse, grads, kw) = check(2, Tq, Tk, 4, 2, 128, BF, frame_len=F, op=op)
        for _ in range(3):
            o2, lse2 = op.forward(q, k, v, **kw)
            again = op.backward(do, q, k, v, o, lse, **kw)
            torch.cuda.synchronize()
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
            assert all(torch.equal(x, y) for x, y in zip(grads, again))


@on_gpu
def test_large_scores_and_scale():
    # Scores of a few hundred: one key takes all; the running maximum moves from tile to tile.
    q, k, v, do = make(1, 200, 1000, 2, 2, 64, BF, seed=4)
    q *= 8
    k *= torch.linspace(0.1, 4, 1000, device="cuda")[None, :, None, None].to(BF)
    op = arl2.SoftmaxAttention(2, 200, 1000, 64, B=1)
    o, lse = op.forward(q, k, v, scale=0.5)
    r, a, t = reference(q, k, v, do, visible(1, 200, 1000, None, None, 0, 0), 0.5)
    # Scores of up to 2^10: the exponent is off by up to 2^-24 * 2^11, P by as much.
    e = torch.finfo(BF).eps / 2
    assert ((o.double().permute(0, 2, 1, 3) - r["o"]).abs() <= (e + 2.0 ** -11) * a["o"] + e * r["o"].abs()).all()
    assert ((lse.double() - r["lse"]).abs() <= 2.0 ** -12 * r["lse"].abs()).all()


@on_gpu
def test_gradients_against_differences():
    # d/dt of <o(x + t w), do> from the fp64 formula at both ends, against the kernel's gradients.
    B, T, H, Hkv, d = 1, 150, 2, 1, 32
    q, k, v, do = make(B, T, T, H, Hkv, d, HF, seed=5)
    m = visible(B, T, T, None, None, 30, 0)
    op = arl2.SoftmaxAttention(H, T, T, d, B=B, H_kv=Hkv, dtype=HF)
    o, lse = op.forward(q, k, v, frame_len=30)
    grads = op.backward(do, q, k, v, o, lse, frame_len=30)
    r, a, t = reference(q, k, v, do, m, d ** -0.5)
    loss = lambda *x: (reference(*x, do, m, d ** -0.5)[0]["o"] * do.double().permute(0, 2, 1, 3)).sum().item()
    for i, name in enumerate(("dq", "dk", "dv")):
        x = [q.double(), k.double(), v.double()]
        w = torch.randn_like(x[i])
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + 1e-4 * w, x[i] - 1e-4 * w
        diff = (loss(*up) - loss(*down)) / 2e-4
        got = (grads[i].double() * w).sum().item()
        e = torch.finfo(HF).eps / 2
        bound = ((e + SUM) * a[name] + e * r[name].abs() + 2.0 ** -25 * (t[name] + 1)).permute(0, 2, 1, 3)
        assert abs(got - diff) <= (bound * w.abs()).sum().item() + 1e-5 * abs(diff)


@on_gpu
def test_streams_and_graphs():
    op = arl2.SoftmaxAttention(3, 400, 500, 64, B=2, H_kv=1)
    q, k, v, do = make(2, 400, 500, 3, 1, 64, BF, seed=6)
    n = torch.tensor([500, 313], dtype=torch.int32, device="cuda")

    def both(**kw):
        o, lse = op.forward(q, k, v, k_len=n, **kw)
        return (o, lse) + op.backward(do, q, k, v, o, lse, k_len=n, **kw)

    want = both()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        got = both(stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    q.copy_(torch.randn_like(q))
    n.copy_(torch.tensor([1, 480], dtype=torch.int32, device="cuda"))
    for _ in range(3):
        graph.replay()
    want = both()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert op.status() == arl2.ARL2_OK


@on_gpu
def test_two_objects_on_two_streams():
    ops = [arl2.SoftmaxAttention(4, 1000, 1000, 128) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    data = [make(1, 1000, 1000, 4, 4, 128, BF, seed=s) for s in range(2)]
    want = []
    for op, x in zip(ops, data):
        o, lse = op.forward(*x[:3])
        want.append((o, lse) + op.backward(x[3], *x[:3], o, lse))
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for op, x, s in zip(ops, data, streams):
            o, lse = op.forward(*x[:3], stream=s)
            got.append((o, lse) + op.backward(x[3], *x[:3], o, lse, stream=s))
        torch.cuda.synchronize()
        for w, x in zip(want, got):
            assert all(torch.equal(i, j) for i, j in zip(w, x))


@on_gpu
def test_one_frame_equals_the_layers_intra_branch():
    # With a zero state the layer's query is its intra-frame attention.
    B, T, H, d = 1, 390, 4, 128
    q, k, v, _ = make(B, T, T, H, H, d, BF, seed=7)
    layer = arl2.ARL2Layer(H, T, d, B)
    w = torch.zeros(H, d, d, dtype=BF, device="cuda")
    layer.set_feature_maps(w, w, w)
    o, _ = arl2.SoftmaxAttention(H, T, T, d, B=B).forward(q, k, v)
    ref = layer.query(q, k, v)
    torch.cuda.synchronize()
    # Each side's P and o are off by at most 2 e of values whose weighted mean |v| is below 4.
    assert (o.double() - ref.double()).abs().max().item() <= 4 * torch.finfo(BF).eps / 2 * 4


@on_gpu
def test_local_and_recurrent_branches_train_together():
    # One block as a user trains it: attention inside the frames of a clip, a gated recurrence over
    # its tokens, their sum projected to a loss; every gradient against autograd in 64 bits.
    B, frames, F, H, d = 2, 3, 50, 2, 64
    T, C = frames * F, 2 * 64
    g = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    q, k, v, x, w = (r(B, T, H, d).to(BF) for _ in range(5))
    alpha = torch.sigmoid(2 + r(B, H, T))
    op = arl2.SoftmaxAttention(H, T, T, d, B=B)
    o, lse = op.forward(q, k, v, frame_len=F)
    h, final = arl2.scan_forward(x.view(B, T, C), alpha)
    dy = w                                             # loss = <o + h, w>
    dq, dk, dv = op.backward(dy, q, k, v, o, lse, frame_len=F)
    dx, dalpha, _ = arl2.scan_backward(dy.view(B, T, C), alpha, h)
    ref = [t.double().requires_grad_() for t in (q, k, v, x, alpha)]
    s = torch.einsum("bihd,bjhd->bhij", ref[0], ref[1]) * d ** -0.5
    m = visible(B, T, T, None, None, F, 0).cuda()[:, None]
    p = torch.softmax(s.masked_fill(~m, -float("inf")), 3)
    ro = torch.einsum("bhij,bjhd->bihd", p, ref[2])
    state, hs = torch.zeros(B, H, d, dtype=torch.float64, device="cuda"), []
    for t in range(T):
        state = ref[4][:, :, t, None] * state + ref[3][:, t]
        hs.append(state)
    loss = ((ro + torch.stack(hs, 1)) * w.double()).sum()
    want = torch.autograd.grad(loss, ref)
    for name, got, ex in zip(("dq", "dk", "dv", "dx", "dalpha"), (dq, dk, dv, dx.view(B, T, H, d), dalpha), want):
        # Independent roundings of the bf16 values in a gradient's terms: 3 of half a step each.
        assert (got.double() - ex).norm() <= 3 * torch.finfo(BF).eps / 2 * ex.norm(), name
    assert op.status() == arl2.ARL2_OK


# ------------------------------------------------------- the exponential on the FMA pipe
def test_exp2_poly4():
    """Its constants are the fitted ones, and it is within 2.7e-6 over the range that is used."""
    csrc = os.path.join(os.path.dirname(os.path.abspath(arl2.__file__)), "csrc")
    spec = importlib.util.spec_from_file_location("fit_exp2_poly", os.path.join(csrc, "fit_exp2_poly.py"))
    fit = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fit)
    src = open(os.path.join(csrc, "arl2_attn.cuh")).read()
    body = src[src.index("float2 exp2_poly4(float2 x)"):]
    pairs = re.findall(r"make_float2\((-?\d+\.\d+)f, (-?\d+\.\d+)f\)", body[: body.index("}")])
    c = np.array([float(a) for a, b in pairs if a == b and abs(float(a)) < 2][::-1][:5], dtype=np.float32)
    np.testing.assert_allclose(c, fit.remez(4).astype(np.float32), rtol=2e-7)
    x = np.linspace(-125, 64, 400_001, dtype=np.float32)
    assert np.abs(fit.eval_f32(c, x).astype(np.float64) / np.exp2(x.astype(np.float64)) - 1).max() < 2.7e-6


# ------------------------------------------------------------------------------- refusals
@on_gpu
def test_binding_refuses():
    op = arl2.SoftmaxAttention(4, 64, 64, 64, B=2, H_kv=2)
    q, k, v, do = make(2, 64, 64, 4, 2, 64, BF)
    o, lse = op.forward(q, k, v)
    for bad in (q.cpu(), q.half(), q[:, :, :3], q[:1], q.transpose(2, 3), q[..., :32]):
        with pytest.raises(ValueError):
            op.forward(bad, k, v)
    with pytest.raises(TypeError):
        op.forward(None, k, v)
    with pytest.raises(ValueError):
        op.forward(q, k, v[:, :10])
    with pytest.raises(ValueError):
        op.forward(q, k, v, k_len=torch.ones(2, device="cuda"))
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ValueError):
            op.forward(q, k, v, scale=scale)
    with pytest.raises(ValueError):
        op.forward(q, k, v, frame_len=1 << 40)
    with pytest.raises(ValueError):
        op.backward(do, q, k, v, o, lse[:, :, :10])
    long = torch.zeros(2, 65, 4, 64, dtype=BF, device="cuda")
    for args in ((long, k, v), (q[:, :0], k, v)):   # longer than the context, empty
        with pytest.raises(arl2.Arl2Error) as e:
            op.forward(*args)
        assert e.value.status == arl2.ARL2_ERR_INVALID_ARG
    odd = torch.zeros(2, 64, 4, 68, dtype=BF, device="cuda")[..., :64]   # rows not 16-byte aligned
    shared = torch.zeros(2, 1, 4, 64, dtype=BF, device="cuda").expand(2, 64, 4, 64)
    for kw in (dict(q=odd), dict(q=shared), dict(out=shared), dict(frame_len=-1)):
        with pytest.raises(arl2.Arl2Error) as e:
            op.forward(kw.pop("q", q), k, v, **kw)
        assert e.value.status == arl2.ARL2_ERR_INVALID_ARG
    for args in ((4, 64, 64, 96), (4, 64, 64, 64, 20000)):
        with pytest.raises(arl2.Arl2Error) as e:
            arl2.SoftmaxAttention(*args)
        assert e.value.status == arl2.ARL2_ERR_UNSUPPORTED
    with pytest.raises(arl2.Arl2Error):
        arl2.SoftmaxAttention(4, 64, 64, 64, H_kv=3)
    with pytest.raises(ValueError):
        arl2.SoftmaxAttention(4, 64, 64, 64, dtype=torch.float64)
    op.close()
    with pytest.raises(arl2.Arl2Error):
        op.forward(q, k, v)


def test_c_entry_refuses_without_a_gpu():
    from softmax_attention_ar_b200 import build
    build.build()
    lib = arl2.load_library()
    out = ctypes.c_void_p()
    bad, unsup = arl2.ARL2_ERR_INVALID_ARG, arl2.ARL2_ERR_UNSUPPORTED
    create = lambda *a: lib.arl2_attn_create(*a, ctypes.byref(out))
    assert lib.arl2_attn_create(1, 1, 1, 1, 1, 64, 0, None) == bad
    assert create(0, 1, 1, 1, 1, 64, 0) == bad and create(1, 4, 3, 1, 1, 64, 0) == bad
    assert create(1, 1, 1, 0, 1, 64, 0) == bad and create(1, 1, 1, 1, 0, 64, 0) == bad
    assert create(1, 1, 1, 1, 1, 80, 0) == unsup and create(1, 1, 1, 1, 1, 64, 2) == unsup
    assert create(1, 1, 1, 1 << 29, 1, 64, 0) == unsup and create(70000, 1, 1, 1, 1, 64, 0) == unsup
    assert not out.value
    assert lib.arl2_attn_forward(None, None, None) == bad and lib.arl2_attn_backward(None, None, None) == bad
    f = arl2._ATTN_FWD.pack(*[0] * 6, 0.0, *[0] * 17)
    assert lib.arl2_attn_forward(None, f, None) == bad
    assert lib.arl2_attn_get_status(None) == bad and lib.arl2_attn_memory_bytes(None) == 0
    lib.arl2_attn_destroy(None)


@on_gpu
def test_captured_padded_batch_equals_eager():
    # Lengths that change between replays: the captured launches cut the work anew each time.
    B, T, H, d = 40, 150, 2, 64
    q, k, v, do = make(B, T, T, H, H, d, BF, seed=5)
    op = arl2.SoftmaxAttention(H, T, T, d, B=B)
    n = torch.full((B,), T, dtype=torch.int32, device="cuda")
    run = lambda: (lambda o, lse: (o, lse) + op.backward(do, q, k, v, o, lse, q_len=n, k_len=n))(
        *op.forward(q, k, v, q_len=n, k_len=n))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for seed in (1, 2):
        n.copy_(torch.from_numpy(np.random.default_rng(seed).integers(0, T + 1, B).astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        assert all(torch.equal(x, y) for x, y in zip(kept, run()))
    assert op.status() == arl2.ARL2_OK


# ------------------------------------------------------------------------- special values
@on_gpu
@pytest.mark.parametrize("Tq,Tk", [(300, 300), (70, 300), (1, 5), (200, 20000)])
def test_rows_that_see_only_scores_of_minus_infinity(Tq, Tk):
    # Whole tiles, narrow ones and tiles cut between CTAs: exp(-inf) is exactly 0, whichever pipe
    # computes it, so such a row is one that sees nothing.
    H, d = 2, 64
    q, k, v, do = make(1, Tq, Tk, H, H, d, BF, seed=12)
    k[0, :, 0, 0] = -float("inf")
    q[0, :, 0, 0] = q[0, :, 0, 0].abs() + 0.1
    op = arl2.SoftmaxAttention(H, Tq, Tk, d)
    o, lse = op.forward(q, k, v)
    assert op.status() == arl2.ARL2_OK
    assert torch.isneginf(lse[0, 0]).all() and (o[0, :, 0] == 0).all()
    assert torch.isfinite(lse[0, 1]).all() and torch.isfinite(o[0, :, 1]).all()


@on_gpu
@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_nan_query_makes_dv_nan(dtype):
    # A NaN, not an infinity, whichever column the row is in.
    T, H, d, F = 150, 1, 64, 50
    op = arl2.SoftmaxAttention(H, T, T, d, dtype=dtype)
    for i in range(60, 76):
        q, k, v, do = make(1, T, T, H, H, d, dtype, seed=13)
        q[0, i, 0, 3] = float("nan")
        o, lse = op.forward(q, k, v, frame_len=F)
        dq, dk, dv = op.backward(do, q, k, v, o, lse, frame_len=F)
        assert op.status() == arl2.ARL2_OK
        assert torch.isnan(dv[0, :100, 0]).all() and torch.isnan(dk[0, :100, 0]).all()


@on_gpu
@pytest.mark.parametrize("Tq,q_len", [(256, None), (300, None), (300, 200), (1, None), (2000, None)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_rows_behind_the_last_query_reach_no_gradient(Tq, q_len, dtype):
    # Keys of -inf: the rows that fill up the last query tile must not meet them as 0 * inf. Every
    # score is -inf, every probability 0.
    H, Tk, d = 2, 300, 64
    q, k, v, do = make(1, Tq, Tk, H, H, d, dtype, seed=12)
    k[0, :, 0, 0] = -float("inf")
    q[0, :, 0, 0] = q[0, :, 0, 0].abs() + 0.1
    n = None if q_len is None else torch.tensor([q_len], dtype=torch.int32, device="cuda")
    op = arl2.SoftmaxAttention(H, Tq, Tk, d, dtype=dtype)
    o, lse = op.forward(q, k, v, q_len=n)
    dq, dk, dv = op.backward(do, q, k, v, o, lse, q_len=n)
    assert op.status() == arl2.ARL2_OK
    assert (dv[0, :, 0] == 0).all() and (dk[0, :, 0] == 0).all()
    assert all(torch.isfinite(t[0, :, 1]).all() for t in (o, dq, dk, dv))


# ------------------------------------------------------------------- the range of fp16
def norms_close(got, want, name):
    """By norms, dtype fp16. On its way to a gradient a term is rounded to fp16 as P or dS, through o in
    delta and with the stored sum: at most 2^-11 relative each. The terms have independent signs, and so
    have their roundings: in norm 3 * 2^-11 of the gradient's. What fp16 cannot hold of the exact gradient
    (values among its subnormals) comes on top; a value next to a rounding border may go to either side,
    so twice."""
    got, want = got.double(), want.double()
    assert torch.isfinite(got).all(), name
    off, held = (got - want).norm().item(), (want.to(HF).double() - want).norm().item()
    assert off <= 3 * 2.0 ** -11 * want.norm().item() + 2 * held, f"{name}: {off:.3e} of {want.norm().item():.3e}"


def half_gradients(q, k, v, do, op=None, **kw):
    """The kernel's gradients of fp16 inputs and the fp64 ones, heads first."""
    B, Tq, H, d = q.shape
    op = op or arl2.SoftmaxAttention(H, Tq, k.shape[1], d, B=B, H_kv=k.shape[2], dtype=HF)
    o, lse = op.forward(q, k, v, **kw)
    got = op.backward(do, q, k, v, o, lse, **kw)
    assert op.status() == arl2.ARL2_OK
    m = visible(B, Tq, k.shape[1], None, None, kw.get("frame_len", 0), kw.get("q_start", 0))
    r, _, _ = reference(q, k, v, do, m, d ** -0.5)
    return [t.double().permute(0, 2, 1, 3) for t in got], [r[n] for n in ("dq", "dk", "dv")]


@on_gpu
@pytest.mark.parametrize("size", [1e-5, 1e-4, 1e-3, 1.0, 1e3])
@pytest.mark.parametrize("Tq,Tk,H,Hkv,d", [(500, 12480, 2, 1, 128), (2100, 2100, 2, 2, 64)])
def test_fp16_gradients_of_any_size(Tq, Tk, H, Hkv, d, size):
    # Over long keys P and dS lie far below fp16's normal range, whatever do is.
    q, k, v, do = make(1, Tq, Tk, H, Hkv, d, torch.float32, seed=14)
    q, k, v, do = q.to(HF), k.to(HF), v.to(HF), (do * size).to(HF)
    for name, got, want in zip(("dq", "dk", "dv"), *half_gradients(q, k, v, do)):
        norms_close(got, want, name)


@on_gpu
@pytest.mark.parametrize("d", [32, 128])
def test_fp16_scores_gradient_above_the_types_range(d):
    # Two keys with opposite values, a large loss scale: dS is about 128000, the gradients are not.
    g = torch.Generator().manual_seed(15)
    r = lambda *s: torch.randn(*s, generator=g)
    q, k = (0.1 * r(1, 8, 1, d)).to(HF).cuda(), (0.1 * r(1, 2, 1, d)).to(HF).cuda()
    v = torch.ones(1, 2, 1, d, dtype=HF, device="cuda")
    v[:, 1] = -1
    do = (2000 * 128 / d * (1 + 0.1 * r(1, 8, 1, d))).to(HF).cuda()
    for name, x, y in zip(("dq", "dk", "dv"), *half_gradients(q, k, v, do)):
        norms_close(x, y, name)


@on_gpu
def test_fp16_rows_batches_heads_and_frames_of_different_size():
    # Each keeps its own precision: rows for dq; sequences, key heads and the frames that see a key for dk.
    B, T, H, Hkv, d, F = 2, 1024, 4, 2, 64, 256
    q, k, v, do = make(B, T, T, H, Hkv, d, torch.float32, seed=16)
    do[:, 1::2] *= 2.0 ** -12
    do[1] *= 2.0 ** -4
    do[:, :, 2:] *= 2.0 ** -3
    q, k, v, do = q.to(HF), k.to(HF), v.to(HF), (do * 4096).to(HF)
    (dq, dk, dv), (rq, rk, rv) = half_gradients(q, k, v, do, frame_len=F)
    for b in range(B):
        for h in range(H):
            for odd in range(2):
                norms_close(dq[b, h, odd::2], rq[b, h, odd::2], f"dq {b} {h} {odd}")
        for h in range(Hkv):
            norms_close(dk[b, h], rk[b, h], f"dk {b} {h}")
            norms_close(dv[b, h], rv[b, h], f"dv {b} {h}")
    # The last frame's gradients far smaller than the earlier ones': its keys are seen by it alone.
    do[:, 768:] *= 2.0 ** -14
    (dq, dk, dv), (rq, rk, rv) = half_gradients(q, k, v, do, frame_len=F)
    for f in range(4):
        s = slice(f * F, (f + 1) * F)
        for name, x, y in (("dq", dq, rq), ("dk", dk, rk), ("dv", dv, rv)):
            for b in range(B):
                norms_close(x[b, :, s], y[b, :, s], f"{name} {b} frame {f}")


@on_gpu
def test_fp16_range_is_taken_anew_in_every_call():
    # A call with large gradients before one with small ones, eager and replayed, with lengths that
    # leave rows out: equal to a context that saw nothing before.
    B, T, H, d = 2, 700, 2, 64
    n = torch.tensor([700, 300], dtype=torch.int32, device="cuda")
    q, k, v, base = make(B, T, T, H, H, d, HF, seed=17)
    sizes = [2.0 ** e for e in (13, -10, 0, -14)]

    def fresh(size):
        op = arl2.SoftmaxAttention(H, T, T, d, B=B, dtype=HF)
        o, lse = op.forward(q, k, v, q_len=n, k_len=n)
        return op.backward(base * size, q, k, v, o, lse, q_len=n, k_len=n)

    want = [fresh(s) for s in sizes]
    op = arl2.SoftmaxAttention(H, T, T, d, B=B, dtype=HF)
    o, lse = op.forward(q, k, v, q_len=n, k_len=n)
    for s, w in zip(sizes, want):
        got = op.backward(base * s, q, k, v, o, lse, q_len=n, k_len=n)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, w))
    do = base.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = op.backward(do, q, k, v, o, lse, q_len=n, k_len=n)
    for s, w in zip(sizes, want):
        do.copy_(base * s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, w))
    assert op.status() == arl2.ARL2_OK


@on_gpu
@pytest.mark.parametrize("dtype", [BF, HF])
def test_zero_and_infinite_gradients(dtype):
    # All of do 0: gradients of exactly 0. An infinity in one head: the other head's stay as they are.
    T, H, d = 300, 2, 64
    q, k, v, do = make(1, T, T, H, H, d, dtype, seed=18)
    op = arl2.SoftmaxAttention(H, T, T, d, dtype=dtype)
    o, lse = op.forward(q, k, v)
    assert all((t == 0).all() for t in op.backward(torch.zeros_like(do), q, k, v, o, lse))
    want = op.backward(do, q, k, v, o, lse)
    do[0, 77, 0, 5] = float("inf")
    got = op.backward(do, q, k, v, o, lse)
    assert op.status() == arl2.ARL2_OK
    assert all(torch.equal(x[:, :, 1], y[:, :, 1]) for x, y in zip(got, want))
    assert not torch.isfinite(got[2][0, :, 0, 5]).any()
    rows = torch.arange(T, device="cuda") != 77
    assert torch.isfinite(got[0][0, rows]).all()
