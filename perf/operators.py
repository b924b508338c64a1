"""What the operators around the memory layer are measured on.

Three operators of a model that holds the memory layer:

* ``glr``   the gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t (prefill, training, one token per request);
* ``qk``    the norm of every query and key head with the position rotation in the same pass (serving, training);
* ``lp``    log probabilities of given tokens with entropy and top alternatives (answers, scoring, training).

``run`` computes them in plain torch operations in 32 bits, or (``own``) through the framework's entry points.
"""

import functools
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SZ = {"bf16": 2, "f32": 4}


# ---- cases -----------------------------------------------------------------------------------------
def listed():
    return [
        # one token for each of 64 requests, whose states lie in a table of 256 (small batch serving)
        dict(name="glr_step_64", op="glr", kind="step", B=64, slots=256, D=2048, gw=1, xt="bf16", gt="bf16"),
        # ragged prompts, packed, one gate per head of 120 channels, states in and out (serving prefill)
        dict(name="glr_prefill", op="glr", kind="fwd", P=24, rows=30011, D=1920, gw=120, xt="bf16", gt="f32",
             ragged=True),
        # a training step of a wide layer: 8 streams of 8192 tokens, a gate per channel
        dict(name="glr_train", op="glr", kind="train", P=8, rows=65536, D=2048, gw=1, xt="bf16", gt="bf16",
             ragged=False),
        # one long f32 stream of a narrow layer, a gate per head of 128 channels
        dict(name="glr_long", op="glr", kind="train", P=1, rows=65537, D=512, gw=128, xt="f32", gt="f32",
             ragged=False),
        # one token for each of 32 requests (serving)
        dict(name="qk_step_32", op="qk", kind="fwd", T=32, Hq=32, Hk=8, hd=128, rd=128, layout="half", xt="bf16",
             max_pos=32768, spread=True),
        # a prompt chunk of an f32 model, the rotation on half of the head, interleaved
        dict(name="qk_prefill", op="qk", kind="fwd", T=4099, Hq=16, Hk=16, hd=64, rd=32, layout="interleaved",
             xt="f32", max_pos=8192, spread=False),
        # a training step's tokens
        dict(name="qk_train", op="qk", kind="train", T=32768, Hq=32, Hk=8, hd=128, rd=128, layout="half", xt="bf16",
             max_pos=8192, spread=False),
        # heads of 120 columns, 64 of them rotated
        dict(name="qk_train_120", op="qk", kind="train", T=5003, Hq=12, Hk=2, hd=120, rd=64, layout="half",
             xt="bf16", max_pos=16384, spread=False),
        # the sampled tokens' log probabilities with 20 alternatives for 8 requests (serving)
        dict(name="lp_step_8", op="lp", kind="fwd", N=8, V=131072, K=20, xt="bf16", scale=1.0, masked=False),
        # scoring a batch of tokens with 5 alternatives, an odd vocabulary, f32 logits at a temperature
        dict(name="lp_score", op="lp", kind="fwd", N=1000, V=50001, K=5, xt="f32", scale=0.8, masked=True),
        # the loss of a training step and its gradient
        dict(name="lp_train", op="lp", kind="train", N=4096, V=65536, K=0, xt="bf16", scale=1.0, masked=False),
        # the same with an odd vocabulary, masked logits and f32
        dict(name="lp_train_odd", op="lp", kind="train", N=777, V=32003, K=0, xt="f32", scale=1.0, masked=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("glr", "qk", "lp"))
    xt = rng.choice(("bf16", "bf16", "f32"))
    if op == "glr":
        kind = rng.choice(("step", "fwd", "train"))
        gw = rng.choice((1, 1, 32, 64, 96, 120, 128, 256))
        D = gw * max(1, _log_int(rng, 64, 4096) // gw) if gw > 1 else 4 * _log_int(rng, 16, 1024)
        D = D - gw if D == 3072 and gw > 1 else D + 4 if D == 3072 else D
        c = dict(op=op, kind=kind, D=D, gw=gw, xt=xt, gt=rng.choice(("bf16", "f32")))
        if kind == "step":
            B = _log_int(rng, 1, 2000)
            return dict(c, B=B, slots=B + rng.randrange(0, 100))
        P = _log_int(rng, 1, 64)
        most = (120_000_000 if xt == "bf16" else 60_000_000) // D
        rows = P * max(1, _log_int(rng, 1, 65536) if P == 1 else _log_int(rng, 1, 8192))
        rows = min(rows, most // P * P)
        return dict(c, P=P, rows=max(P, rows), ragged=bool(rng.randrange(2)))
    if op == "qk":
        hd = rng.choice((64, 96, 120, 128, 128, 256))
        Hk = rng.choice((1, 2, 4, 8, 16))
        Hq = Hk * rng.choice((1, 2, 4))
        T = _log_int(rng, 1, 32768)
        T = max(1, min(T, 80_000_000 // ((Hq + Hk) * hd * (2 if xt == "f32" else 1))))
        return dict(op=op, kind=rng.choice(("fwd", "train")), T=T, Hq=Hq, Hk=Hk, hd=hd, rd=8 * rng.randrange(2, hd // 8 + 1),
                    layout=rng.choice(("half", "interleaved")), xt=xt, max_pos=rng.choice((32768, 40000)),
                    spread=bool(rng.randrange(2)))
    kind = rng.choice(("fwd", "train"))
    V = _log_int(rng, 1000, 131072)
    N = _log_int(rng, 1, 4096)
    N = max(1, min(N, (120_000_000 if xt == "bf16" else 60_000_000) // V))
    return dict(op=op, kind=kind, N=N, V=V, K=0 if kind == "train" else rng.choice((0, 1, 5, 10, 20, 32)), xt=xt,
                scale=rng.choice((1.0, 0.7)), masked=bool(rng.randrange(2)))


# ---- inputs ----------------------------------------------------------------------------------------
def _offsets(case, seed):
    """Row offsets [P + 1] of the sequences: equal lengths, or ragged ones (an empty one among them)."""
    P, rows = case["P"], case["rows"]
    if not case["ragged"] or P == 1:
        return np.arange(P + 1, dtype=np.int64) * (rows // P)
    r = np.random.default_rng(seed)
    share = r.lognormal(0.0, 1.0, P)
    share[r.integers(P)] = 0.0
    off = np.round(np.concatenate([[0.0], np.cumsum(share / share.sum())]) * rows).astype(np.int64)
    off[-1] = rows
    return off


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 17)
    t = DT[case["xt"]]

    def randn(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return (torch.randn(shape, device=dev, generator=gen) * scale + shift).to(dtype)

    s = {"case": dict(case)}
    if case["op"] == "glr":
        D, gw, H = case["D"], case["gw"], case["D"] // case["gw"]
        rows = case["B"] if case["kind"] == "step" else case["rows"]
        s["x"] = randn(rows, D, dtype=t)
        s["g"] = torch.nn.functional.logsigmoid(randn(rows, H, scale=1.0, shift=3.0)).to(DT[case["gt"]])
        s["y"] = torch.empty(rows, D, device=dev, dtype=t)
        if case["kind"] == "step":
            s["state"] = randn(case["slots"], D, scale=2.0)
            perm = torch.randperm(case["slots"], device=dev, generator=gen)
            s["slots"] = perm[:rows].to(torch.int32)
            return s
        P = case["P"]
        off = _offsets(case, seed)
        s["offsets"] = torch.from_numpy(off).to(dev) if case["ragged"] else None
        s["cuts"] = torch.from_numpy(off).to(dev)
        s["h0"] = randn(P, D)
        s["hT"] = torch.empty(P, D, device=dev)
        if case["kind"] == "train":
            s["dy"] = randn(rows, D, dtype=t)
            s["dhT"] = randn(P, D)
            s["dx"] = torch.empty(rows, D, device=dev, dtype=t)
            s["dg"] = torch.empty(rows, H, device=dev, dtype=DT[case["gt"]])
            s["dh0"] = torch.empty(P, D, device=dev)
        return s
    if case["op"] == "qk":
        T, Hq, Hk, hd, rd = (case[k] for k in ("T", "Hq", "Hk", "hd", "rd"))
        # the queries and keys are slices of one projection's rows [T, (Hq + 2 Hk) hd]
        qkv = randn(T, (Hq + 2 * Hk) * hd, dtype=t, scale=1.5)
        s["q"] = qkv[:, :Hq * hd].view(T, Hq, hd)
        s["k"] = qkv[:, Hq * hd:(Hq + Hk) * hd].view(T, Hk, hd)
        s["wq"], s["wk"] = randn(hd, scale=0.1, shift=1.0), randn(hd, scale=0.1, shift=1.0)
        if case["spread"]:
            s["pos"] = torch.randint(case["max_pos"], (T,), device=dev, generator=gen, dtype=torch.int32)
        else:
            s["pos"] = (torch.arange(T, device=dev) % case["max_pos"]).to(torch.int32)
        f = 10000.0 ** (-torch.arange(rd // 2, device=dev, dtype=torch.float64) * 2.0 / rd)
        angle = torch.arange(case["max_pos"], device=dev, dtype=torch.float64)[:, None] * f
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["q_out"] = torch.empty(T, Hq, hd, device=dev, dtype=t)
        s["k_out"] = torch.empty(T, Hk, hd, device=dev, dtype=t)
        if case["kind"] == "train":
            s["dq_out"], s["dk_out"] = randn(T, Hq, hd, dtype=t), randn(T, Hk, hd, dtype=t)
            s["dq"], s["dk"] = torch.empty_like(s["q_out"]), torch.empty_like(s["k_out"])
            s["dwq"], s["dwk"] = torch.empty(hd, device=dev), torch.empty(hd, device=dev)
        return s
    N, V, K = case["N"], case["V"], case["K"]
    x = randn(N, V, scale=2.0)
    if case["masked"]:
        # a quarter of the vocabulary is masked: half of it with -inf, half with the type's lowest value
        u = torch.rand(V, device=dev, generator=gen)
        x.masked_fill_((u < 0.125)[None, :], -math.inf)
        x.masked_fill_(((u >= 0.125) & (u < 0.25))[None, :], torch.finfo(t).min)
    s["logits"] = x.to(t)
    s["targets"] = torch.randint(V, (N,), device=dev, generator=gen, dtype=torch.int32)
    # targets are tokens that a model could give: moved to the next unmasked one; every 16th is ignored
    ok = torch.isfinite(x[0]) & (x[0] > -1e30) if case["masked"] else torch.ones(V, dtype=torch.bool, device=dev)
    free = torch.nonzero(ok).reshape(-1)
    s["targets"] = free[s["targets"].long() % free.numel()].to(torch.int32)
    s["targets"][15::16] = -100
    for name in ("logp", "entropy", "lse"):
        s[name] = torch.empty(N, device=dev)
    if K:
        s["top_vals"] = torch.empty(N, K, device=dev)
        s["top_idx"] = torch.empty(N, K, device=dev, dtype=torch.int32)
    if case["kind"] == "train":
        s["d_logp"] = -torch.rand(N, device=dev, generator=gen) / N
        s["d_entropy"] = randn(N, scale=0.01 / N)
        s["dlogits"] = torch.empty(N, V, device=dev, dtype=t)
    return s


# ---- the framework's calls -------------------------------------------------------------------------
@functools.lru_cache(maxsize=256)
def _glr_spec(P, rows, D, gw, xt, gt):
    import sparse_slot_memory_gb300 as sdm

    return sdm.GlrSpec(P=P, rows=rows, D=D, gate_width=gw, x_dtype=xt, g_dtype=gt)


@functools.lru_cache(maxsize=256)
def _rope_spec(T, Hq, Hk, hd, rd, max_pos, layout, xt):
    import sparse_slot_memory_gb300 as sdm

    return sdm.RopeSpec(tokens=T, q_heads=Hq, k_heads=Hk, hd=hd, rot_dim=rd, max_pos=max_pos, layout=layout, dtype=xt)


@functools.lru_cache(maxsize=256)
def _lp_spec(N, V, K, xt, scale):
    import sparse_slot_memory_gb300 as sdm

    return sdm.LogprobSpec(rows=N, V=V, K=K, dtype=xt, scale=scale)


def _own_glr(s, c):
    import sparse_slot_memory_gb300 as sdm

    if c["kind"] == "step":
        spec = _glr_spec(1, c["B"], c["D"], c["gw"], c["xt"], c["gt"])
        sdm.glr_step(spec, s["x"], s["g"], s["state"], s["y"], slots=s["slots"])
        return {"y": s["y"], "state": s["state"]}
    spec = _glr_spec(c["P"], c["rows"], c["D"], c["gw"], c["xt"], c["gt"])
    if c["kind"] == "fwd":
        sdm.glr_forward(spec, s["x"], s["g"], s["y"], offsets=s["offsets"], h0=s["h0"], hT=s["hT"])
        return {"y": s["y"], "hT": s["hT"]}
    states = sdm.alloc_glr_states(spec)
    sdm.glr_forward(spec, s["x"], s["g"], s["y"], offsets=s["offsets"], h0=s["h0"], hT=s["hT"], states=states)
    sdm.glr_backward(spec, s["x"], s["g"], s["dy"], states, s["dx"], s["dg"], sdm.alloc_glr_workspace(spec),
                     offsets=s["offsets"], dhT=s["dhT"], dh0=s["dh0"])
    return {k: s[k] for k in ("y", "hT", "dx", "dg", "dh0")}


def _own_qk(s, c):
    import sparse_slot_memory_gb300 as sdm

    spec = _rope_spec(c["T"], c["Hq"], c["Hk"], c["hd"], c["rd"], c["max_pos"], c["layout"], c["xt"])
    sdm.qk_norm_rope(spec, s["q"], s["k"], s["pos"], s["table"], s["wq"], s["wk"], s["q_out"], s["k_out"])
    if c["kind"] == "fwd":
        return {"q": s["q_out"], "k": s["k_out"]}
    sdm.qk_norm_rope_backward(spec, s["dq_out"], s["dk_out"], s["q"], s["k"], s["pos"], s["table"], s["wq"], s["wk"],
                              s["dq"], s["dk"], s["dwq"], s["dwk"], sdm.alloc_rope_workspace(spec))
    return {"q": s["q_out"], "k": s["k_out"], "dq": s["dq"], "dk": s["dk"], "dwq": s["dwq"], "dwk": s["dwk"]}


def _own_lp(s, c):
    import sparse_slot_memory_gb300 as sdm

    spec = _lp_spec(c["N"], c["V"], c["K"], c["xt"], c["scale"])
    sdm.token_logprobs(spec, s["logits"], s["targets"], s["logp"], entropy=s["entropy"], lse=s["lse"],
                       top_vals=s.get("top_vals"), top_idx=s.get("top_idx"))
    out = {k: s[k] for k in ("logp", "entropy", "lse", "top_vals", "top_idx") if k in s}
    if c["kind"] == "train":
        sdm.token_logprobs_backward(spec, s["logits"], s["targets"], s["lse"], s["entropy"], s["d_logp"], s["dlogits"],
                                    d_entropy=s["d_entropy"])
        out["dlogits"] = s["dlogits"]
    return out


# ---- the plain forms -------------------------------------------------------------------------------
def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t over dimension 0 from zero, by doubling: pairs (a, b) of spans of n rows are joined
    into spans of 2n."""
    n = 1
    while n < b.shape[0]:
        b = torch.cat([b[:n], a[n:] * b[:-n] + b[n:]])
        a = torch.cat([a[:n], a[n:] * a[:-n]])
        n *= 2
    return b


def _plain_glr(s, c):
    H, gw = c["D"] // c["gw"], c["gw"]
    a = s["g"].float().exp()[:, :, None]
    x = s["x"].float().view(-1, H, gw)
    if c["kind"] == "step":
        i = s["slots"].long()
        h = a * s["state"][i].view(-1, H, gw) + x
        s["state"][i] = h.view(-1, c["D"])
        return {"y": h.view(-1, c["D"]).to(s["y"].dtype), "state": s["state"]}
    cuts, h0 = s["cuts"], s["h0"].view(-1, H, gw)
    full = cuts[1:] > cuts[:-1]
    first, last = cuts[:-1][full], cuts[1:][full] - 1
    before = torch.zeros_like(x)                    # the state before a sequence's first row, elsewhere 0
    before[first] = h0[full]
    inner = a.clone()                               # the gate, 0 where a sequence starts
    inner[first] = 0.0
    h = _scan(inner, x + a * before)
    hT = h0.clone()
    hT[full] = h[last]
    out = {"y": h.reshape(-1, c["D"]).to(s["y"].dtype), "hT": hT.view(-1, c["D"])}
    if c["kind"] == "fwd":
        return out
    dhT = s["dhT"].view(-1, H, gw)
    dy = s["dy"].float().view(-1, H, gw).clone()
    dy[last] += dhT[full]
    follow = torch.cat([inner[1:], torch.zeros_like(inner[:1])])
    lam = _scan(follow.flip(0), dy.flip(0)).flip(0)
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    prev[first] = h0[full]
    dg = (lam * a * prev).sum(2)
    dh0 = dhT.clone()
    dh0[full] = a[first] * lam[first]
    return dict(out, dx=lam.reshape(-1, c["D"]).to(s["dx"].dtype), dg=dg.to(s["dg"].dtype), dh0=dh0.view(-1, c["D"]))


def _turn(n, cos, sin, rd, layout, sign):
    """The rotation of the first rd columns of n [T, H, hd] (sign -1: its inverse)."""
    a = n[..., 0:rd:2] if layout == "interleaved" else n[..., :rd // 2]
    b = n[..., 1:rd:2] if layout == "interleaved" else n[..., rd // 2:rd]
    u, v = a * cos - sign * b * sin, b * cos + sign * a * sin
    r = torch.stack([u, v], -1).flatten(-2) if layout == "interleaved" else torch.cat([u, v], -1)
    return torch.cat([r, n[..., rd:]], -1)


def _plain_head(x, w, dout, cos, sin, c):
    t, x = x.dtype, x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    out = _turn(x * r * w, cos, sin, c["rd"], c["layout"], 1.0).to(t)
    if dout is None:
        return out, None, None
    e = _turn(dout.float(), cos, sin, c["rd"], c["layout"], -1.0)
    n = x * r
    dw = (e * n).sum((0, 1))
    e = e * w
    return out, (r * (e - n * (e * n).mean(-1, keepdim=True))).to(t), dw


def _plain_qk(s, c):
    cs = s["table"][s["pos"].long()][:, None, :]
    cos, sin = cs[..., :c["rd"] // 2], cs[..., c["rd"] // 2:]
    q, dq, dwq = _plain_head(s["q"], s["wq"], s.get("dq_out"), cos, sin, c)
    k, dk, dwk = _plain_head(s["k"], s["wk"], s.get("dk_out"), cos, sin, c)
    if c["kind"] == "fwd":
        return {"q": q, "k": k}
    return {"q": q, "k": k, "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _plain_lp(s, c):
    x = s["logits"].float()
    z = x * c["scale"]
    m = z.amax(1, keepdim=True)
    empty = m == -math.inf
    lse = m + (z - m).exp().sum(1, keepdim=True).log()
    lse = torch.where(empty, m, lse)
    logs = torch.where(empty, -math.inf, z - lse)
    p = logs.exp()
    H = -torch.where(p > 0, p * logs, 0.0).sum(1)
    tgt = s["targets"].long()
    given = tgt >= 0
    logp = torch.where(given, logs.gather(1, tgt.clamp(min=0)[:, None])[:, 0], 0.0)
    out = {"logp": logp, "entropy": H, "lse": lse[:, 0]}
    if c["K"]:
        # one whole number for each logit: its order among the values above, the lower id first among equals
        bits = (x + 0.0).view(torch.int32)
        order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32
        order = order + torch.arange(c["V"] - 1, -1, -1, device=x.device)
        top = (c["V"] - 1 - (order.topk(c["K"], 1).values & 0xFFFFFFFF))
        out["top_vals"], out["top_idx"] = logs.gather(1, top), top.to(torch.int32)
    if c["kind"] == "train":
        dlp = torch.where(given, s["d_logp"], 0.0)[:, None]
        dz = -dlp * p - s["d_entropy"][:, None] * torch.where(p > 0, p * (logs + H[:, None]), 0.0)
        dz.scatter_add_(1, tgt.clamp(min=0)[:, None], dlp)
        out["dlogits"] = (c["scale"] * dz).to(s["logits"].dtype)
    return out


def run(state):
    c = state["case"]
    if own:
        return {"glr": _own_glr, "qk": _own_qk, "lp": _own_lp}[c["op"]](state, c)
    return {"glr": _plain_glr, "qk": _plain_qk, "lp": _plain_lp}[c["op"]](state, c)


# ---- the definition in 64 bits -----------------------------------------------------------------------
def _exact_glr(s, c):
    H, gw, D = c["D"] // c["gw"], c["gw"], c["D"]
    a = torch.exp(s["g"].double())
    a = a if gw == 1 else a.repeat_interleave(gw, 1)
    x = s["x"].double()
    if c["kind"] == "step":
        state = s["state"].double()
        h = torch.addcmul(x, a, state[s["slots"].long()])
        state[s["slots"].long()] = h
        return {"y": h, "state": state}
    off = s["cuts"].tolist()
    h, h0 = torch.empty_like(x), s["h0"].double()
    hT = h0.clone()
    for p in range(c["P"]):
        cur = h0[p]
        for t in range(off[p], off[p + 1]):
            cur = torch.addcmul(x[t], a[t], cur, out=h[t])
        hT[p] = cur
    if c["kind"] == "fwd":
        return {"y": h, "hT": hT}
    dy, dx, dh0 = s["dy"].double(), torch.empty_like(x), s["dhT"].double()
    dg = torch.empty_like(x)
    for p in range(c["P"]):
        cur = dh0[p].clone()
        for t in range(off[p + 1] - 1, off[p] - 1, -1):
            cur = torch.add(dy[t], cur, out=dx[t])
            cur = cur * a[t]
            torch.mul(cur, h[t - 1] if t > off[p] else h0[p], out=dg[t])
        dh0[p] = cur
    return {"y": h, "hT": hT, "dx": dx, "dg": dg.view(-1, H, gw).sum(2), "dh0": dh0}


def _exact_head(x, w, dout, ang, c):
    """A head's row times its weights as complex numbers turned by the angle; the gradient by the formula of the norm."""
    x, w, rd = x.double(), w.double(), c["rd"]
    i = torch.arange(rd // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if c["layout"] == "interleaved" else (i, i + rd // 2)

    def turned(v, z):
        o = v.clone()
        u = torch.complex(v[..., ia], v[..., ib]) * z[:, None, :]
        o[..., ia], o[..., ib] = u.real, u.imag
        return o

    ms = x.square().mean(-1, keepdim=True) + 1e-6
    out = turned(x / ms.sqrt() * w, ang)
    if dout is None:
        return out, None, None
    e = turned(dout.double(), ang.conj())
    dw = (e * x / ms.sqrt()).sum((0, 1))
    ew = e * w
    dx = ew / ms.sqrt() - x * (ew * x).sum(-1, keepdim=True) / (c["hd"] * ms * ms.sqrt())
    return out, dx, dw


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "glr":
        return _exact_glr(s, c)
    if c["op"] == "qk":
        tab = s["table"].double()[s["pos"].long()]
        ang = torch.complex(tab[:, :c["rd"] // 2].contiguous(), tab[:, c["rd"] // 2:].contiguous())
        q, dq, dwq = _exact_head(s["q"], s["wq"], s.get("dq_out"), ang, c)
        k, dk, dwk = _exact_head(s["k"], s["wk"], s.get("dk_out"), ang, c)
        if c["kind"] == "fwd":
            return {"q": q, "k": k}
        return {"q": q, "k": k, "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    parts = []
    for i in range(0, c["N"], 256):
        r = slice(i, min(i + 256, c["N"]))
        x = s["logits"][r].double()
        logs = torch.log_softmax(x * c["scale"], 1)
        p = logs.exp()
        plogp = torch.where(p > 0, p * logs, 0.0)
        tgt = s["targets"][r].long()
        one = torch.zeros_like(p)
        one[torch.arange(len(tgt), device=x.device)[tgt >= 0], tgt[tgt >= 0]] = 1.0
        d = {"logp": torch.where(one > 0, logs, 0.0).sum(1), "entropy": -plogp.sum(1),
             "lse": torch.logsumexp(x * c["scale"], 1)}
        if c["K"]:
            d["top_vals"] = torch.sort(logs, 1, descending=True).values[:, :c["K"]]
        if c["kind"] == "train":
            H = d["entropy"][:, None]
            dl = torch.where(tgt >= 0, s["d_logp"][r].double(), 0.0)[:, None]
            d["dlogits"] = c["scale"] * (dl * (one - p) - s["d_entropy"][r].double()[:, None] * (plogp + p * H))
        parts.append(d)
    out = {k: torch.cat([d[k] for d in parts]) for k in parts[0]}
    if c["K"]:
        out["top_idx"] = None
    return out


# ---- work -------------------------------------------------------------------------------------------
def work(case):
    """Each input read once, each output written once."""
    e = SZ[case["xt"]]
    if case["op"] == "glr":
        D, H, ge = case["D"], case["D"] // case["gw"], SZ[case["gt"]]
        if case["kind"] == "step":
            return {"bytes": case["B"] * (D * (2 * e + 8) + H * ge + 4), "flops": case["B"] * (2 * D + 8 * H)}
        n = case["rows"]
        b, f = n * (2 * D * e + H * ge) + 8 * case["P"] * D, n * (2 * D + 8 * H)
        if case["kind"] == "train":   # dy in; dx, dg out; the states' gradients
            b, f = b + n * (2 * D * e + H * ge) + 8 * case["P"] * D, f + n * 4 * D
        return {"bytes": b, "flops": f}
    if case["op"] == "qk":
        T, n = case["T"], case["T"] * (case["Hq"] + case["Hk"]) * case["hd"]
        b, f = 2 * n * e + T * 4 + min(T, case["max_pos"]) * 4 * case["rd"] + 8 * case["hd"], 7 * n
        if case["kind"] == "train":   # the outputs' gradients in, the inputs' and the weights' out
            b, f = b + 2 * n * e + 8 * case["hd"], f + 12 * n
        return {"bytes": b, "flops": f}
    N, V, K = case["N"], case["V"], case["K"]
    b, f = N * V * e + N * (16 + 8 * K), 12 * N * V
    if case["kind"] == "train":
        b, f = b + N * V * e + 8 * N, f + 14 * N * V
    return {"bytes": b, "flops": f}
