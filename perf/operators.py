"""Training operators of the two branches, as they are measured: softmax attention with its
row statistics and its backward pass, and the gated linear recurrence with its backward pass.

    forward    o = softmax(scale q k^T + mask) v,   lse = the log of each row's sum of exponentials
    backward   dq, dk, dv from do, with the probabilities recomputed from lse
    recurrence h_t = a_t h_{t-1} + x_t             (h_0's predecessor is the given state, or 0)
    backward   lam_t = dh_t + a_{t+1} lam_{t+1},  dx_t = lam_t,  da_t = lam_t h_{t-1}

Key j is visible to query i of batch b if i < q_len[b], j < k_len[b] and, with frame_len > 0,
j < (floor((i + q_start) / frame_len) + 1) frame_len: a query sees its own frame and the frames
before it. A row that sees nothing has o = 0 and lse = -inf. Rows and tokens behind a length
give 0.

Layouts: q, o [B, Tq, H, d], k, v [B, Tk, Hkv, d] with H a multiple of Hkv; x, h [B, T, C];
gates [B, T, C], or one gate per head and token, fp32 [B, H, T].
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------- the cases
def _attn(name, op, B, H, Hkv, Tq, Tk, d, dtype, lens="full", frame_len=0, empty=False, packed=False):
    return {"name": name, "op": op, "B": B, "H": H, "Hkv": Hkv, "Tq": Tq, "Tk": Tk, "d": d, "dtype": dtype,
            "lens": lens, "frame_len": frame_len, "empty": empty, "packed": packed}


def _scan_case(name, op, B, T, C, heads, dtype, gate, lens="full", state=False):
    return {"name": name, "op": op, "B": B, "T": T, "C": C, "heads": heads, "dtype": dtype, "gate": gate,
            "lens": lens, "state": state}


def listed():
    return [
        # The smallest frame the layer is checked on: a call's latency.
        _attn("attn_fwd_tiny", "attn_fwd", 1, 2, 2, 64, 64, 32, "fp16"),
        # One 480p frame attending to itself: the intra-frame branch of a training step.
        _attn("attn_fwd_480p", "attn_fwd", 1, 12, 12, 1560, 1560, 128, "bf16"),
        # Eight 480p frames, each token seeing its own frame and the earlier ones (teacher forcing).
        _attn("attn_fwd_8_frames", "attn_fwd", 1, 12, 12, 12480, 12480, 128, "bf16", frame_len=1560),
        # One new token of each of four streams of different lengths over its cached keys.
        _attn("attn_fwd_one_query", "attn_fwd", 4, 12, 12, 1, 16384, 128, "bf16", lens="ragged"),
        # The backward pass of the 480p frame.
        _attn("attn_bwd_480p", "attn_bwd", 1, 12, 12, 1560, 1560, 128, "bf16"),
        # A padded batch of clips with heads that share keys, one clip empty, q, k, v in one buffer.
        _attn("attn_bwd_ragged", "attn_bwd", 3, 8, 2, 999, 999, 64, "fp16", lens="ragged", empty=True, packed=True),
        # The backward pass over eight frames.
        _attn("attn_bwd_8_frames", "attn_bwd", 1, 12, 12, 12480, 12480, 128, "bf16", frame_len=1560),
        # One new token of 64 streams: the serving step.
        _scan_case("scan_fwd_step", "scan_fwd", 64, 1, 1536, 0, "bf16", "fp32", state=True),
        # 21 frames of 480p in token order, one gate per head and token.
        _scan_case("scan_fwd_21_frames", "scan_fwd", 1, 32760, 1536, 12, "bf16", "fp32"),
        # A padded batch at 720p-like lengths with a gate of its own for every channel.
        _scan_case("scan_fwd_channels", "scan_fwd", 4, 3600, 1536, 0, "bf16", "bf16", lens="ragged", state=True),
        # The backward pass of the 21 frames; the gates' gradients are sums over a head's channels.
        _scan_case("scan_bwd_21_frames", "scan_bwd", 1, 32760, 1536, 12, "bf16", "fp32", state=True),
        # An odd width in full precision.
        _scan_case("scan_bwd_odd", "scan_bwd", 3, 1561, 517, 0, "fp32", "fp32", lens="ragged", state=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_bwd", "scan_fwd", "scan_bwd"])
    if op.startswith("attn"):
        B, Hkv, group = _log_int(rng, 1, 8), rng.choice([1, 2, 3, 4, 6, 12]), rng.choice([1, 1, 2, 4])
        d, dtype = rng.choice([32, 64, 128, 128]), rng.choice(["bf16", "bf16", "fp16"])
        kind = rng.choice(["full", "full", "ragged", "frames"])
        H = Hkv * group
        Tk = _log_int(rng, 1 if op == "attn_fwd" else 2, 12480)   # over a single key dq and dk are 0
        Tq = Tk if rng.random() < 0.6 else _log_int(rng, 1, 12480)
        if kind == "frames":
            Tq = min(Tq, Tk)
        most = 12 * 12480 * 12480 * 9 // 16   # visible pairs of the largest listed case
        while B * H * Tq * Tk > most:
            B, Tq, Tk = max(1, B // 2), (Tq + 1) // 2, (Tk + 1) // 2
        frame_len = _log_int(rng, 1, Tk) if kind == "frames" else 0
        return _attn("", op, B, H, Hkv, Tq, Tk, d, dtype, "ragged" if kind == "ragged" else "full", frame_len,
                     kind == "ragged" and rng.random() < 0.5, Tq == Tk and rng.random() < 0.4) | {"name": "drawn"}
    B, T = _log_int(rng, 1, 64), _log_int(rng, 1, 32760)
    heads = rng.choice([0, 0, 2, 4, 12])
    C = heads * rng.choice([32, 64, 128]) if heads else _log_int(rng, 8, 2048)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    gate = "fp32" if heads else rng.choice([dtype, "fp32"])
    while B * T * C > 32760 * 1536:
        B, T = max(1, B // 2), (T + 1) // 2
    return _scan_case("drawn", op, B, T, C, heads, dtype, gate, rng.choice(["full", "ragged"]), rng.random() < 0.5)


def _lens(B, T, empty=False):
    """Lengths of a padded batch: the first full, the others shorter, the last 0 if asked."""
    n = [T - (b * T) // (B + 1) for b in range(B)]
    if empty:
        n[-1] = 0
    return n


def _lengths(case):
    if case["op"].startswith("attn"):
        if case["lens"] == "full":
            return [case["Tq"]] * case["B"], [case["Tk"]] * case["B"]
        q = _lens(case["B"], case["Tq"], case["empty"] and case["Tq"] == case["Tk"])
        return q, _lens(case["B"], case["Tk"], case["empty"])
    n = [case["T"]] * case["B"] if case["lens"] == "full" else _lens(case["B"], case["T"])
    return n, n


def work(case):
    e = 2 if case["dtype"] != "fp32" else 4
    ql, kl = _lengths(case)
    if case["op"].startswith("attn"):
        B, H, Hkv, d, F = case["B"], case["H"], case["Hkv"], case["d"], case["frame_len"]
        start = case["Tk"] - case["Tq"] if F else 0
        pairs = 0
        for nq, nk in zip(ql, kl):
            pairs += sum(min(nk, ((i + start) // F + 1) * F) for i in range(nq)) if F else nq * nk
        q_bytes, k_bytes = sum(ql) * H * d * e, sum(kl) * Hkv * d * e
        stats = sum(ql) * H * 4
        if case["op"] == "attn_fwd":   # reads q, k, v; writes o and lse
            return {"bytes": 2 * q_bytes + 2 * k_bytes + stats, "flops": 4 * d * H * pairs}
        # reads q, k, v, o, do, lse; writes dq, dk, dv
        return {"bytes": 4 * q_bytes + 4 * k_bytes + stats, "flops": 10 * d * H * pairs}
    tokens, C, H = sum(ql), case["C"], case["heads"]
    g = tokens * H * 4 if H else tokens * C * (4 if case["gate"] == "fp32" else 2)
    states = case["B"] * C * 4 * (2 if case["state"] else 1)
    if case["op"] == "scan_fwd":
        return {"bytes": 2 * tokens * C * e + g + states, "flops": 2 * tokens * C}
    return {"bytes": 3 * tokens * C * e + 2 * g + 2 * states, "flops": 4 * tokens * C}


# ------------------------------------------------------------------------------- the inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    dt = DTYPES[case["dtype"]]
    ql, kl = _lengths(case)
    ragged = case["lens"] == "ragged"
    s = {"case": case}
    if case["op"].startswith("attn"):
        B, H, Hkv, Tq, Tk, d = (case[n] for n in ("B", "H", "Hkv", "Tq", "Tk", "d"))
        if case["packed"]:   # q, k, v as one projection writes them, side by side for each token
            qkv = _randn(gen, B, Tq, H + 2 * Hkv, d).to(dt)
            s["q"], s["k"], s["v"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
        else:
            s["q"], s["k"], s["v"] = (_randn(gen, B, T, n, d).to(dt) for T, n in ((Tq, H), (Tk, Hkv), (Tk, Hkv)))
        s["q_len"] = torch.tensor(ql, dtype=torch.int32, device="cuda") if ragged else None
        s["k_len"] = torch.tensor(kl, dtype=torch.int32, device="cuda") if ragged else None
        s["frame_len"], s["q_start"] = case["frame_len"], Tk - Tq if case["frame_len"] else 0
        if case["op"] == "attn_bwd":
            s["do"] = _randn(gen, B, Tq, H, d).to(dt)
            s["o"], s["lse"] = _attention(s)
        if own:
            from softmax_attention_ar_b200 import arl2
            s["op"] = arl2.SoftmaxAttention(H, Tq, Tk, d, B=B, H_kv=Hkv, dtype=dt)
        return s
    B, T, C, H = case["B"], case["T"], case["C"], case["heads"]
    s["x"] = _randn(gen, B, T, C).to(dt)
    s["a"] = torch.sigmoid(2 + 0.5 * (_randn(gen, B, H, T) if H else _randn(gen, B, T, C))).to(DTYPES[case["gate"]])
    s["h0"] = _randn(gen, B, C) if case["state"] else None
    s["lens"] = torch.tensor(ql, dtype=torch.int32, device="cuda") if ragged else None
    if case["op"] == "scan_bwd":
        s["dh"] = _randn(gen, B, T, C).to(dt)
        s["dfinal"] = _randn(gen, B, C) if case["state"] else None
        s["h"] = _recurrence(s)[0]
    return s


# ------------------------------------------------------------------------- the plain forms
def _scores(s):
    """fp32 scores [B, H, Tq, Tk] with -inf where a key is not seen, and k, v per query head."""
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    group = q.shape[2] // k.shape[2]
    k, v = k.repeat_interleave(group, dim=2), v.repeat_interleave(group, dim=2)
    scores = torch.matmul(q.permute(0, 2, 1, 3), k.permute(0, 2, 3, 1)) / math.sqrt(q.shape[3])
    i = torch.arange(q.shape[1], device=q.device)
    j = torch.arange(k.shape[1], device=q.device)
    if s["frame_len"]:
        limit = (torch.div(i + s["q_start"], s["frame_len"], rounding_mode="floor") + 1) * s["frame_len"]
        scores.masked_fill_(j[None, :] >= limit[:, None], -math.inf)
    if s["k_len"] is not None:
        scores.masked_fill_((j[None, :] >= s["k_len"][:, None])[:, None, None, :], -math.inf)
    if s["q_len"] is not None:
        scores.masked_fill_((i[None, :] >= s["q_len"][:, None])[:, None, :, None], -math.inf)
    return scores, q, k, v


def _attention(s):
    scores, q, _, v = _scores(s)
    top = scores.amax(dim=3, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(scores.sub_(top))
    total = p.sum(dim=3, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).squeeze(3)
    return o.permute(0, 2, 1, 3).to(s["q"].dtype).contiguous(), lse


def _attention_backward(s):
    scores, q, k, v = _scores(s)
    lse = s["lse"].unsqueeze(3)
    p = torch.exp(scores.sub_(torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)))
    do = s["do"].float()
    dot = do.permute(0, 2, 1, 3)
    dv = torch.matmul(p.transpose(2, 3), dot)
    ds = torch.matmul(dot, v.permute(0, 2, 3, 1))
    delta = (s["o"].float() * do).sum(dim=3).permute(0, 2, 1).unsqueeze(3)
    ds = ds.sub_(delta).mul_(p)
    scale = 1.0 / math.sqrt(q.shape[3])
    dq = torch.matmul(ds, k.permute(0, 2, 1, 3)) * scale
    dk = torch.matmul(ds.transpose(2, 3), q.permute(0, 2, 1, 3)) * scale
    B, Tk, Hkv, d = s["k"].shape
    dt = s["q"].dtype
    dk, dv = (x.view(B, Hkv, -1, Tk, d).sum(dim=2).permute(0, 2, 1, 3).to(dt).contiguous() for x in (dk, dv))
    return dq.permute(0, 2, 1, 3).to(dt).contiguous(), dk, dv


def _doubling_scan(a, x):
    """h_t = a_t h_{t-1} + x_t along dim 1 from 0, in log2(T) steps."""
    n = 1
    while n < x.shape[1]:
        x = torch.cat([x[:, :n], x[:, n:] + a[:, n:] * x[:, :-n]], dim=1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], dim=1)
        n *= 2
    return x


def _per_token(s, x):
    """x [B, T, C] as fp32 [B, T, H, C / H] and the gates to match ([B, T, H, 1], or per channel with H = 1)."""
    a = s["a"].float()
    if s["case"]["heads"]:
        a = a.permute(0, 2, 1).unsqueeze(3)
        return a, x.float().view(x.shape[0], x.shape[1], a.shape[2], -1)
    return a.unsqueeze(2), x.float().unsqueeze(2)


def _valid(s, T):
    """[B, T, 1, 1]: tokens inside their sequence."""
    return (torch.arange(T, device="cuda")[None, :] < s["lens"][:, None])[:, :, None, None]


def _recurrence(s):
    a, x = _per_token(s, s["x"])
    B, T, H, d = x.shape
    if s["lens"] is not None:   # behind a length the state stays
        valid = _valid(s, T)
        a, x = torch.where(valid, a, torch.ones_like(a)), torch.where(valid, x, torch.zeros_like(x))
    if s["h0"] is not None:
        x = torch.cat([x[:, :1] + a[:, :1] * s["h0"].view(B, 1, H, d), x[:, 1:]], dim=1)
    h = _doubling_scan(a, x)
    final = h[:, -1].reshape(B, H * d).contiguous()
    if s["lens"] is not None:
        h = torch.where(valid, h, torch.zeros_like(h))
    return h.reshape(B, T, H * d).to(s["x"].dtype), final


def _recurrence_backward(s):
    a, dh = _per_token(s, s["dh"])
    B, T, H, d = dh.shape
    h = s["h"].float().view(B, T, H, d)
    h0 = s["h0"].view(B, 1, H, d) if s["h0"] is not None else torch.zeros_like(h[:, :1])
    if s["lens"] is not None:
        valid = _valid(s, T)
        a, dh = torch.where(valid, a, torch.ones_like(a)), torch.where(valid, dh, torch.zeros_like(dh))
    if s["dfinal"] is not None:
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dfinal"].view(B, 1, H, d)], dim=1)
    later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], dim=1)
    dx = _doubling_scan(later.flip(1), dh.flip(1)).flip(1)
    dh0 = (a[:, :1] * dx[:, :1]).reshape(B, H * d)
    da = dx * torch.cat([h0, h[:, :-1]], dim=1)
    if s["lens"] is not None:
        dx, da = torch.where(valid, dx, torch.zeros_like(dx)), torch.where(valid, da, torch.zeros_like(da))
    if s["case"]["heads"]:
        da = da.sum(dim=3).permute(0, 2, 1)
    else:
        da = da.reshape(B, T, H * d)
    return dx.reshape(B, T, H * d).to(s["dh"].dtype), da.to(s["a"].dtype).contiguous(), dh0


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from softmax_attention_ar_b200 import arl2
        mask = {"q_len": s["q_len"], "k_len": s["k_len"], "frame_len": s["frame_len"], "q_start": s["q_start"]} \
            if op.startswith("attn") else None
        if op == "attn_fwd":
            return s["op"].forward(s["q"], s["k"], s["v"], **mask)
        if op == "attn_bwd":
            return s["op"].backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], **mask)
        if op == "scan_fwd":
            return arl2.scan_forward(s["x"], s["a"], h0=s["h0"], lens=s["lens"])
        return arl2.scan_backward(s["dh"], s["a"], s["h"], h0=s["h0"], dfinal=s["dfinal"], lens=s["lens"])
    return {"attn_fwd": _attention, "attn_bwd": _attention_backward, "scan_fwd": _recurrence,
            "scan_bwd": _recurrence_backward}[op](s)


# ----------------------------------------------------------------- the definitions, in fp64
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("attn"):
        return _exact_attention(s, case)
    return _exact_scan(s, case)


def _exact_attention(s, case):
    B, H, Hkv, Tq, Tk, d = (case[n] for n in ("B", "H", "Hkv", "Tq", "Tk", "d"))
    ql, kl = _lengths(case)
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    o, lse = torch.zeros_like(q), torch.full((B, H, Tq), -math.inf, dtype=torch.float64, device="cuda")
    grads = [torch.zeros_like(t) for t in (q, k, v)]
    for b in range(B):
        nq, nk = ql[b], kl[b]
        if not nq or not nk:
            continue
        limit = [min(nk, ((i + Tk - Tq) // case["frame_len"] + 1) * case["frame_len"]) if case["frame_len"] else nk
                 for i in range(nq)]
        seen = torch.arange(nk, device="cuda")[None, :] < torch.tensor(limit, device="cuda")[:, None]
        for h in range(H):
            kv = h // (H // Hkv)
            qh, kh, vh = q[b, :nq, h], k[b, :nk, kv], v[b, :nk, kv]
            z = torch.where(seen, qh @ kh.T * d ** -0.5, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
            total = torch.logsumexp(z, dim=1)
            p = torch.where(seen, torch.exp(z - total[:, None]), torch.zeros_like(z))
            o[b, :nq, h], lse[b, h, :nq] = p @ vh, total
            if case["op"] == "attn_bwd":
                g = s["do"][b, :nq, h].double()
                dp = g @ vh.T
                ds = p * (dp - (p * dp).sum(dim=1, keepdim=True)) * d ** -0.5
                grads[0][b, :nq, h] = ds @ kh
                grads[1][b, :nk, kv] += ds.T @ qh
                grads[2][b, :nk, kv] += p.T @ g
    return tuple(grads) if case["op"] == "attn_bwd" else (o, lse)


def _exact_scan(s, case):
    B, T, C, H = case["B"], case["T"], case["C"], case["heads"]
    n, _ = _lengths(case)
    lens = torch.tensor(n, device="cuda")
    a = s["a"].double()
    gate = (lambda t: a[:, :, t].repeat_interleave(C // H, dim=1)) if H else (lambda t: a[:, t])
    state = s["h0"].double() if s["h0"] is not None else torch.zeros(B, C, dtype=torch.float64, device="cuda")
    if case["op"] == "scan_fwd":
        h = torch.zeros(B, T, C, dtype=torch.float64, device="cuda")
        for t in range(T):
            inside = (t < lens)[:, None]
            new = gate(t) * state + s["x"][:, t].double()
            h[:, t] = torch.where(inside, new, h[:, t])
            state = torch.where(inside, new, state)
        return h, state
    lam = s["dfinal"].double() if s["dfinal"] is not None else torch.zeros_like(state)
    dx = torch.zeros(B, T, C, dtype=torch.float64, device="cuda")
    da = torch.zeros_like(s["a"], dtype=torch.float64)
    for t in range(T - 1, -1, -1):   # lam: the gradient that reaches h_t from later tokens
        inside = (t < lens)[:, None]
        total = torch.where(inside, lam + s["dh"][:, t].double(), lam)
        before = s["h"][:, t - 1].double() if t else state
        dx[:, t] = torch.where(inside, total, dx[:, t])
        if H:
            da[:, :, t] = torch.where(inside, (total * before).view(B, H, -1).sum(dim=2), da[:, :, t])
        else:
            da[:, t] = torch.where(inside, total * before, da[:, t])
        lam = torch.where(inside, gate(t) * total, lam)
    return dx, da, lam
