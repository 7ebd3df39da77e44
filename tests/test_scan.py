"""The gated linear recurrence and its backward pass: argument checks on the CPU, and results on
the GPU against a token-by-token loop in 64 bits.

Error bounds. The kernels work in fp32: every product and sum on the way from an input to an
output rounds by at most u = 2^-24 relative. A token's gate enters one product of its slice
and one step of the second scan, and slices (of 8 tokens or more) and chunks are composed once
each, so an input passes through fewer than 2 T + 80 roundings; the error of h_t is below
(2 T + 80) u times the same recurrence over absolute values, and a stored value is off by half
a step of its type on top (eps / 2 relative, and half the smallest subnormal of fp16).
"""
import numpy as np
import pytest
import torch

from softmax_attention_ar_b200 import arl2

U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ plain implementation
def loop_forward(x, a, h0, lens):
    """x, a fp64 [B, T, C] (a expanded to channels); returns h, final."""
    B, T, C = x.shape
    h, state = np.zeros((B, T, C)), h0.copy()
    for b in range(B):
        for t in range(lens[b]):
            state[b] = a[b, t] * state[b] + x[b, t]
            h[b, t] = state[b]
    return h, state


def loop_backward(dh, a, h, h0, dfinal, lens):
    B, T, C = dh.shape
    dx, da, lam = np.zeros((B, T, C)), np.zeros((B, T, C)), dfinal.copy()
    for b in range(B):
        for t in range(lens[b] - 1, -1, -1):
            lam[b] = lam[b] + dh[b, t]
            dx[b, t] = lam[b]
            da[b, t] = lam[b] * (h[b, t - 1] if t else h0[b])
            lam[b] = a[b, t] * lam[b]
    return dx, da, lam


def channels(a, heads, C):
    """Gates as [B, T, C]."""
    a = a.double().cpu().numpy()
    return np.repeat(a.transpose(0, 2, 1), C // heads, axis=2) if heads else a


def close(got, ref, spread, depth, dtype):
    """|got - ref| within depth u spread plus half a step of the type."""
    got = got.double().cpu().numpy()
    half = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    err = depth * U * spread
    bound = err + half * (np.abs(ref) + err) + tiny
    assert np.isfinite(got).all()
    worst = (np.abs(got - ref) - bound).max()
    assert worst <= 0, f"off by {worst:.3e} more than the bound"


def make(B, T, C, heads, dtype, gate, seed, lens=None, state=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, dh = r(B, T, C).to(DT[dtype]), r(B, T, C).to(DT[dtype])
    a = torch.sigmoid(2 + r(B, heads, T) if heads else 2 + r(B, T, C)).to(DT[gate])
    h0, dfinal = (r(B, C), r(B, C)) if state else (None, None)
    n = [T] * B if lens is None else lens
    dev = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    return x, dh, a, h0, dfinal, n, dev


def check(B, T, C, heads, dtype, gate, seed=0, lens=None, state=True, view=lambda t: t):
    x, dh, a, h0, dfinal, n, dev = make(B, T, C, heads, dtype, gate, seed, lens, state)
    if lens is not None:   # what stands behind a length is not used, whatever it is
        for b in range(B):
            for t in (x, dh) + (() if heads else (a,)):
                t[b, n[b]:] = float("nan")
            if heads:
                a[b, :, n[b]:] = float("nan")
    h, final = arl2.scan_forward(view(x), a if heads else view(a), h0=h0, lens=dev)
    clean = [max(0, v) for v in n]
    z = lambda t: np.zeros((B, C)) if t is None else t.double().cpu().numpy()
    X, A, D = (np.nan_to_num(v) for v in (x.double().cpu().numpy(), channels(a, heads, C), dh.double().cpu().numpy()))
    rh, rf = loop_forward(X, A, z(h0), clean)
    sh, sf = loop_forward(np.abs(X), np.abs(A), np.abs(z(h0)), clean)
    depth = 2 * T + 80
    close(h, rh, sh, depth, DT[dtype])
    close(final, rf, sf, depth, torch.float32)
    for b in range(B):
        assert (h[b, n[b]:] == 0).all()
    stored = h.clone()
    if lens is not None:
        for b in range(B):
            stored[b, n[b]:] = float("nan")
    dx, da, dh0 = arl2.scan_backward(view(dh), a if heads else view(a), view(stored), h0=h0, dfinal=dfinal, lens=dev)
    H = np.nan_to_num(stored.double().cpu().numpy())
    rdx, rda, rdh0 = loop_backward(D, A, H, z(h0), z(dfinal), clean)
    sdx, sda, sdh0 = loop_backward(np.abs(D), np.abs(A), np.abs(H), np.abs(z(h0)), np.abs(z(dfinal)), clean)
    close(dx, rdx, sdx, depth, DT[dtype])
    close(dh0, rdh0, sdh0, depth + 1, torch.float32)
    if heads:
        fold = lambda v: v.reshape(B, T, heads, C // heads).sum(axis=3).transpose(0, 2, 1)
        close(da, fold(rda), fold(sda), depth + 1 + C // heads, torch.float32)
    else:
        close(da, rda, sda, depth + 1, DT[gate])
    for b in range(B):
        assert (dx[b, n[b]:] == 0).all()
        assert ((da[b, :, n[b]:] if heads else da[b, n[b]:]) == 0).all()


gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def on_gpu(f):
    for m in gpu:
        f = m(f)
    return f


@on_gpu
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 128, 129, 1000, 2049, 4100])
@pytest.mark.parametrize("B,C,dtype,gate", [(1, 128, "bf16", "bf16"), (2, 36, "fp32", "fp32"), (2, 37, "fp16", "fp32"),
                                            (1, 1, "bf16", "fp32"), (3, 132, "fp16", "fp16")])
def test_gates_per_channel(B, T, C, dtype, gate):
    check(B, T, C, 0, dtype, gate, seed=T)


@on_gpu
@pytest.mark.parametrize("T", [1, 3, 16, 130, 1560, 4100])
@pytest.mark.parametrize("B,heads,d,dtype", [(1, 12, 128, "bf16"), (2, 3, 64, "fp16"), (2, 5, 32, "fp32")])
def test_gates_per_head(B, T, heads, d, dtype):
    check(B, T, heads * d, heads, dtype, "fp32", seed=T)


@on_gpu
@pytest.mark.parametrize("heads,C", [(0, 96), (0, 61), (2, 64)])
def test_lengths(heads, C):
    # Full, empty, one token, one short of full, inside a slice; NaN behind each.
    check(5, 300, C, heads, "bf16", "fp32", lens=[300, 0, 1, 299, 129])
    check(3, 2, C, heads, "fp32", "fp32", lens=[0, 2, 1], state=False)


@on_gpu
def test_many_channel_groups():
    # Enough (batch, channel group) pairs that slices are long.
    check(96, 300, 520, 0, "bf16", "fp32", lens=[300 - 3 * b for b in range(96)])


@on_gpu
def test_strided_and_misaligned_inputs():
    def padded(t):   # rows of a wider buffer, starting one element in: no wide accesses
        big = torch.zeros(*t.shape[:2], t.shape[2] + 7, dtype=t.dtype, device=t.device)
        big[..., 1:1 + t.shape[2]] = t
        return big[..., 1:1 + t.shape[2]]

    def time_major(t):
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    for view in (padded, time_major):
        check(2, 150, 40, 0, "bf16", "bf16", view=view)
    check(2, 150, 64, 2, "fp16", "fp32", view=time_major)


@on_gpu
def test_broadcast_input_and_given_outputs():
    B, T, C = 3, 70, 32
    x, dh, a, h0, dfinal, n, _ = make(B, T, C, 0, "fp32", "fp32", 1)
    one = a[:1, :1].expand(B, T, C)
    out = torch.full((B, T, 2 * C), 7.0, device="cuda")
    h, final = arl2.scan_forward(x, one, h0=h0, out=out[..., :C])
    rh, rf = loop_forward(x.double().cpu().numpy(), one.double().cpu().numpy(), h0.double().cpu().numpy(), n)
    sh, _ = loop_forward(x.double().abs().cpu().numpy(), one.double().cpu().numpy(), h0.double().abs().cpu().numpy(), n)
    close(h, rh, sh, 2 * T + 80, torch.float32)
    assert (out[..., C:] == 7).all()


@on_gpu
def test_in_place_equals_out_of_place():
    x, dh, a, h0, dfinal, _, _ = make(2, 2500, 128, 0, "bf16", "fp32", 2)
    h, final = arl2.scan_forward(x, a, h0=h0)
    xi, hi = x.clone(), h0.clone()
    h2, f2 = arl2.scan_forward(xi, a, h0=hi, out=xi, final=hi)
    assert h2 is xi and f2 is hi and torch.equal(h, h2) and torch.equal(final, f2)
    dx, da, dh0 = arl2.scan_backward(dh, a, h, h0=h0, dfinal=dfinal)
    di = dh.clone()
    dx2, da2, dh02 = arl2.scan_backward(di, a, h, h0=h0, dfinal=dfinal, dx=di)
    assert torch.equal(dx, dx2) and torch.equal(da, da2) and torch.equal(dh0, dh02)


@on_gpu
def test_reset_and_keep_gates():
    # a = 0 forgets (h = x), a = 1 keeps (h = running sum): exact in fp32 for small integers.
    x = torch.randint(-4, 5, (2, 500, 33), device="cuda").float()
    h, final = arl2.scan_forward(x, torch.zeros_like(x))
    assert torch.equal(h, x) and torch.equal(final, x[:, -1])
    h, final = arl2.scan_forward(x, torch.ones_like(x))
    assert torch.equal(h, x.cumsum(1)) and torch.equal(final, x.sum(1))


@on_gpu
def test_steps_equal_the_sequence():
    # Serving: one token at a time, carrying the state in place, as one call over all tokens.
    x, _, a, h0, _, _, _ = make(3, 40, 256, 2, "bf16", "fp32", 3)
    h, final = arl2.scan_forward(x, a, h0=h0)
    state = h0.clone()
    steps = [arl2.scan_forward(x[:, t:t + 1], a[:, :, t:t + 1], h0=state, final=state)[0] for t in range(40)]
    X, A, S = x.double().cpu().numpy(), channels(a, 2, 256), h0.double().cpu().numpy()
    spread = loop_forward(np.abs(X), A, np.abs(S), [40] * 3)
    ref = loop_forward(X, A, S, [40] * 3)
    close(torch.cat(steps, 1), ref[0], spread[0], 160, torch.bfloat16)
    close(state, ref[1], spread[1], 160, torch.float32)


@on_gpu
def test_gradients_against_differences():
    # The loss <h, g> + <final, gf> is linear in x and h0 and in each single gate, so
    # differences are exact but for the fp32 roundings of the two losses.
    B, T, C = 2, 300, 64
    x, g, a, h0, gf, _, _ = make(B, T, C, 2, "fp32", "fp32", 4)
    loss = lambda x, a, h0: sum((u.double() * w.double()).sum().item()
                                for u, w in zip(arl2.scan_forward(x, a, h0=h0), (g, gf)))
    h, _ = arl2.scan_forward(x, a, h0=h0)
    dx, da, dh0 = arl2.scan_backward(g, a, h, h0=h0, dfinal=gf)
    size = (arl2.scan_forward(x.abs(), a, h0=h0.abs())[0].double() * g.double().abs()).sum().item()
    size += (arl2.scan_forward(x.abs(), a, h0=h0.abs())[1].double() * gf.double().abs()).sum().item()
    tol = lambda step: 4 * (2 * T + 80) * U * size / step
    base = loss(x, a, h0)
    v = torch.randn_like(x)
    assert abs(loss(x + v, a, h0) - base - (dx.double() * v.double()).sum().item()) <= tol(1) * 3
    w = torch.randn_like(h0)
    assert abs(loss(x, a, h0 + w) - base - (dh0.double() * w.double()).sum().item()) <= tol(1) * 3
    for b, hd, t in ((0, 0, 0), (1, 1, 150), (0, 1, 299)):
        a2 = a.clone()
        a2[b, hd, t] += 0.5
        step = (a2 - a)[b, hd, t].item()
        assert abs((loss(x, a2, h0) - base) / step - da[b, hd, t].item()) <= tol(step) * 3


@on_gpu
def test_streams_and_graphs():
    x, dh, a, h0, dfinal, _, _ = make(2, 1000, 256, 0, "bf16", "bf16", 5)
    ref = arl2.scan_forward(x, a, h0=h0) + arl2.scan_backward(dh, a, x, h0=h0, dfinal=dfinal)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    one = arl2.scan_forward(x, a, h0=h0, stream=s1)
    two = arl2.scan_backward(dh, a, x, h0=h0, dfinal=dfinal, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(one + two, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = arl2.scan_forward(x, a, h0=h0) + arl2.scan_backward(dh, a, x, h0=h0, dfinal=dfinal)
    x.copy_(torch.randn_like(x))
    graph.replay()
    want = arl2.scan_forward(x, a, h0=h0) + arl2.scan_backward(dh, a, x, h0=h0, dfinal=dfinal)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))


@on_gpu
def test_gates_of_the_layer_drive_the_recurrence():
    # The layer's produced gates (alpha [B, H, T]) go straight in as per-head gates.
    B, T, H, d = 2, 200, 4, 32
    g = torch.Generator(device="cuda").manual_seed(6)
    layer = arl2.ARL2Layer(H, T, d, B)
    w = (torch.randn(2, H, H * d, generator=g, device="cuda") / (H * d) ** 0.5).bfloat16()
    bias = torch.full((H,), 2.0, device="cuda")
    layer.set_gate_weights(w[0], w[1], bias, bias)
    x = torch.randn(B, T, H * d, generator=g, device="cuda").bfloat16()
    alpha, beta = layer.gates(x)
    h, final = arl2.scan_forward(x, alpha)
    zero, n = np.zeros((B, H * d)), [T] * B
    X, A = x.double().cpu().numpy(), channels(alpha, H, H * d)
    ref, spread = loop_forward(X, A, zero, n), loop_forward(np.abs(X), A, zero, n)
    close(h, ref[0], spread[0], 2 * T + 80, torch.bfloat16)
    close(final, ref[1], spread[1], 2 * T + 80, torch.float32)
    assert layer.status() == arl2.ARL2_OK
    layer.close()


@on_gpu
def test_offsets_beyond_32_bits():
    # One sequence whose last rows lie past 2^31 elements of a strided view.
    T, C, stride = 4, 64, (1 << 30) // 1
    big = torch.empty(3 * stride + C, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(big, (1, T, C), (big.numel(), stride, 1))
    vals = torch.randn(1, T, C, device="cuda").bfloat16()
    x.copy_(vals)
    a = torch.full((1, T, C), 0.5, device="cuda").bfloat16()
    assert torch.equal(arl2.scan_forward(x, a)[0], arl2.scan_forward(vals, a)[0])


# ------------------------------------------------------------------------------- refusals
@on_gpu
def test_binding_refuses():
    x = torch.zeros(2, 8, 64, device="cuda")
    a = torch.zeros_like(x)
    with pytest.raises(ValueError):
        arl2.scan_forward(x.cpu(), a)
    with pytest.raises(ValueError):
        arl2.scan_forward(x, a.cpu())
    with pytest.raises(ValueError):
        arl2.scan_forward(x, a.bfloat16())
    with pytest.raises(ValueError):
        arl2.scan_forward(x.double(), a.double())
    with pytest.raises(ValueError):
        arl2.scan_forward(x, torch.zeros(2, 3, 8, device="cuda"))   # 3 heads do not divide 64
    with pytest.raises(ValueError):
        arl2.scan_forward(x.transpose(1, 2), a.transpose(1, 2))     # channels not adjacent
    with pytest.raises(ValueError):
        arl2.scan_forward(x, a, h0=torch.zeros(2, 63, device="cuda"))
    with pytest.raises(ValueError):
        arl2.scan_forward(x, a, lens=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(arl2.Arl2Error) as e:
        arl2.scan_forward(x, torch.zeros(2, 4, 8, device="cuda"))   # heads of 16 channels
    assert e.value.status == arl2.ARL2_ERR_UNSUPPORTED
    with pytest.raises(arl2.Arl2Error) as e:   # an output whose rows share memory
        arl2.scan_forward(x, a, out=torch.zeros(2, 1, 64, device="cuda").expand(2, 8, 64))
    assert e.value.status == arl2.ARL2_ERR_INVALID_ARG
    with pytest.raises(arl2.Arl2Error) as e:
        arl2.scan_forward(x[:, :0], a[:, :0])
    assert e.value.status == arl2.ARL2_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        arl2.scan_backward(x, a, None)


def test_c_entry_refuses_without_a_gpu():
    from softmax_attention_ar_b200 import build
    build.build()
    lib = arl2.load_library()
    p = 1 << 20   # an aligned address; never dereferenced by the argument checks

    def fwd(B=2, T=8, C=64, heads=0, dtype=2, gate=2, x=p, a=p, h=p, h0=0, xs=(512, 64), as_=(512, 64, 0),
            hs=(512, 64), ws=0):
        f = arl2._SCAN_FWD.pack(B, T, C, heads, dtype, gate, 0, x, a, h0, h, 0, ws, *xs, *as_, *hs)
        return lib.arl2_scan_forward(f, None)

    bad, unsup = arl2.ARL2_ERR_INVALID_ARG, arl2.ARL2_ERR_UNSUPPORTED
    assert lib.arl2_scan_forward(None, None) == bad and lib.arl2_scan_backward(None, None) == bad
    assert fwd(B=0) == bad and fwd(T=0) == bad and fwd(C=0) == bad and fwd(heads=-1) == bad
    assert fwd(x=0) == bad and fwd(a=0) == bad and fwd(h=0) == bad
    assert fwd(x=p + 2) == bad and fwd(h0=p + 2) == bad
    assert fwd(dtype=3) == bad and fwd(gate=7) == bad
    assert fwd(gate=0) == unsup                       # fp32 values with bf16 gates
    assert fwd(heads=5) == bad and fwd(heads=4) == unsup
    assert fwd(heads=2, gate=0, dtype=0) == unsup     # per-head gates are fp32
    assert fwd(heads=2, xs=(512, 66)) == bad          # rows not aligned to 4 elements
    assert fwd(xs=(-512, 64)) == bad
    assert fwd(hs=(0, 64)) == bad and fwd(hs=(512, 32)) == bad and fwd(hs=(256, 64)) == bad
    assert lib.arl2_scan_workspace_bytes(None) == 0
    assert fwd(B=1, T=5000, xs=(0, 64), as_=(0, 64, 0), hs=(0, 64)) == bad   # needs a workspace
    sh = (2, 8, 64, 0, 2, 2, 0)
    s2, s3 = (512, 64), (512, 64, 0)
    for hole in range(5):
        q = [p] * 5
        q[hole] = 0
        dh, a, h, dx, da = q
        f = arl2._SCAN_BWD.pack(*sh, dh, a, h, 0, 0, dx, da, 0, 0, *s2, *s3, *s2, *s2)
        assert lib.arl2_scan_backward(f, None) == bad
    f = arl2._SCAN_BWD.pack(*sh, p, p, p, 0, 0, p, p, 0, 0, *s2, *s3, *s2, 512, 0)
    assert lib.arl2_scan_backward(f, None) == bad


# ------------------------------------------------------------------------- gates above 1
def against_loop(x, dh, a, h0, dfinal, heads, dtype, gate, lens=None):
    """Both directions on given inputs, compared as check() does."""
    B, T, C = x.shape
    n = [T] * B if lens is None else lens
    dev = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    z = lambda t: np.zeros((B, C)) if t is None else t.double().cpu().numpy()
    X, A, D = x.double().cpu().numpy(), channels(a, heads, C), dh.double().cpu().numpy()
    depth = 2 * T + 80
    h, final = arl2.scan_forward(x, a, h0=h0, lens=dev)
    rh, rf = loop_forward(X, A, z(h0), n)
    sh, sf = loop_forward(np.abs(X), np.abs(A), np.abs(z(h0)), n)
    close(h, rh, sh, depth, DT[dtype])
    close(final, rf, sf, depth, torch.float32)
    dx, da, dh0 = arl2.scan_backward(dh, a, h, h0=h0, dfinal=dfinal, lens=dev)
    H = h.double().cpu().numpy()
    rdx, rda, rdh0 = loop_backward(D, A, H, z(h0), z(dfinal), n)
    sdx, sda, sdh0 = loop_backward(np.abs(D), np.abs(A), np.abs(H), np.abs(z(h0)), np.abs(z(dfinal)), n)
    close(dx, rdx, sdx, depth, DT[dtype])
    close(dh0, rdh0, sdh0, depth + 1, torch.float32)
    if heads:
        fold = lambda v: v.reshape(B, T, heads, C // heads).sum(axis=3).transpose(0, 2, 1)
        close(da, fold(rda), fold(sda), depth + 1 + C // heads, torch.float32)
    else:
        close(da, rda, sda, depth + 1, DT[gate])


@on_gpu
@pytest.mark.parametrize("T", [40, 400, 1000, 2500, 4100])
@pytest.mark.parametrize("C,heads,dtype,gate", [(128, 0, "bf16", "bf16"), (37, 0, "fp32", "fp32"),
                                                (64, 2, "fp32", "fp32")])
def test_a_state_of_zero_stays_zero_under_gates_above_one(T, C, heads, dtype, gate):
    # The gates' product over the part without input passes fp32's range many times; the states do
    # not: 0 there, then values under gates below 1. Before them one gate of 0, which forgets.
    B, n = 2, 30
    r = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=r, device="cuda")
    for part in ("forward", "backward"):
        x, dh = rand(B, T, C).to(DT[dtype]), rand(B, T, C).to(DT[dtype])
        a = torch.sigmoid(rand(B, heads, T) if heads else rand(B, T, C))
        at = (lambda s: a[:, :, s]) if heads else (lambda s: a[:, s])
        if part == "forward":     # no gradient reaches the tokens under large gates
            x[:, :T - n] = 0
            at(slice(0, T - n))[:] = -16.0
            at(T - n - 1)[:] = 0.0
            dh[:, :T - n] = 0
        else:                     # dh = 0 behind the first n tokens, x = 0 as well, and the state forgotten
            dh[:, n:] = 0
            x[:, n:] = 0
            at(slice(n, T))[:] = 16.0
            at(n)[:] = 0.0
        against_loop(x, dh, a.to(DT[gate]), None, None, heads, dtype, gate)


@on_gpu
def test_negative_gates_and_growth_within_range():
    # Gates of either sign, products of up to 2^100 over a sequence.
    B, T, C = 2, 1500, 36
    g = torch.Generator(device="cuda").manual_seed(9)
    x, dh = (torch.randn(B, T, C, generator=g, device="cuda") * 2.0 ** -60 for _ in range(2))
    a = torch.where(torch.rand(B, T, C, generator=g, device="cuda") < 0.5, -1.0, 1.0) * 2.0 ** (100 / T)
    h0, dfinal = (torch.randn(B, C, generator=g, device="cuda") * 2.0 ** -60 for _ in range(2))
    against_loop(x, dh, a, h0, dfinal, 0, "fp32", "fp32")


# ------------------------------------------------------------ lengths over several chunks
@on_gpu
@pytest.mark.parametrize("T", [2100, 4100])
@pytest.mark.parametrize("C,heads,dtype,gate", [(256, 2, "bf16", "fp32"), (128, 0, "bf16", "bf16"),
                                                (61, 0, "fp32", "fp32"), (72, 0, "fp16", "fp32")])
@pytest.mark.parametrize("state", [True, False])
def test_lengths_over_chunks(T, C, heads, dtype, gate, state):
    # Empty, one token, on and next to the edges of slices and chunks (multiples of 8), one short of
    # full; NaN behind each.
    check(8, T, C, heads, dtype, gate, seed=T, lens=[T, 0, 1, 512, 513, 1024, 1031, T - 1], state=state)


@on_gpu
@pytest.mark.parametrize("C,heads,dtype", [(520, 0, "bf16"), (384, 3, "bf16")])
def test_long_slices_of_one_chunk(C, heads, dtype):
    # More (sequence, channel group) pairs than the GPU takes at once: one chunk, slices of over 64 tokens.
    B, T = 150, 1100
    check(B, T, C, heads, dtype, "fp32", lens=[T - 7 * b for b in range(B)])


@on_gpu
def test_gates_above_one_with_lengths():
    # As above, with sequences of different length, one of them empty.
    B, T, C, n = 5, 2600, 72, 30
    lens = [T, 0, 700, 1033, T - 1]
    g = torch.Generator(device="cuda").manual_seed(19)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, dh, a = rand(B, T, C).bfloat16(), rand(B, T, C).bfloat16(), torch.full((B, T, C), -16.0, device="cuda")
    for b, m in enumerate(lens):
        m = max(m, n + 1)
        x[b, :m - n] = 0
        dh[b, :m - n] = 0
        a[b, m - n - 1] = 0
        a[b, m - n:m] = torch.sigmoid(rand(n, C))
    against_loop(x, dh, a.bfloat16(), None, None, 0, "bf16", "bf16", lens=lens)
