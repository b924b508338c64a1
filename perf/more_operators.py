"""What the operators of a model's trunk around the memory layer are measured on.

* ``gdr``    the gated delta rule S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T, y_t = scale S_t^T q_t: the
             dense counterpart of the memory's decay, read and write (prefill, training, one token per request);
* ``norm``   the norms behind and before a block fused with its gate, the residual's scale and its sum;
* ``embed``  the rows of an embedding table for tokens, scaled, and the table's gradient by sorted tokens.

``run`` computes them in plain torch operations in 32 bits, or (``own``) through the framework's entry points.
"""

import functools
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SZ = {"bf16": 2, "f32": 4}
C = 64   # rows that the plain form takes together


# ---- cases -----------------------------------------------------------------------------------------
def listed():
    return [
        # one token for each of 32 requests, whose states lie in a table of 48 (small batch serving)
        dict(name="gdr_step_32", op="gdr", kind="step", B=32, slots=48, Hk=8, Hv=16, dk=128, dv=128, xt="bf16", gt="f32"),
        # ragged prompts, packed, two value heads to a key head, states in and out (serving prefill)
        dict(name="gdr_prefill", op="gdr", kind="fwd", P=12, rows=20011, Hk=8, Hv=16, dk=128, dv=128, xt="bf16",
             gt="f32", ragged=True),
        # a training step: 8 streams of 4096 tokens
        dict(name="gdr_train", op="gdr", kind="train", P=8, rows=32768, Hk=16, Hv=16, dk=128, dv=128, xt="bf16",
             gt="f32", ragged=False),
        # a training step of a small f32 model with odd heads and ragged sequences
        dict(name="gdr_train_odd", op="gdr", kind="train", P=5, rows=3001, Hk=2, Hv=6, dk=72, dv=56, xt="f32", gt="f32",
             ragged=True),
        # one long document through a narrow layer (prefill of a long context)
        dict(name="gdr_long", op="gdr", kind="fwd", P=1, rows=32769, Hk=4, Hv=8, dk=64, dv=128, xt="bf16", gt="bf16",
             ragged=False),
        # one token for each of 32 requests: the residual's sum and the next block's norm
        dict(name="norm_step_32", op="norm", kind="fwd", rows=32, D=2048, group=2048, post=False, gate="none", res=True,
             cs=False, pre=True, xt="bf16"),
        # a training step's tokens: norms on both sides of the block, its gate and a scale per channel
        dict(name="norm_train", op="norm", kind="train", rows=16384, D=4096, group=4096, post=True, gate="sigmoid",
             res=True, cs=True, pre=True, xt="bf16"),
        # the gated norm of every head before the output projection
        dict(name="norm_heads", op="norm", kind="train", rows=16001, D=1920, group=120, post=True, gate="silu", res=False,
             cs=False, pre=False, xt="bf16"),
        # a prompt of an f32 model of odd width: the residual's sum and the next block's norm
        dict(name="norm_prompt", op="norm", kind="fwd", rows=4099, D=1500, group=1500, post=True, gate="none", res=True,
             cs=False, pre=True, xt="f32"),
        # one token for each of 64 requests (serving)
        dict(name="embed_step_64", op="embed", kind="fwd", T=64, V=131072, D=2048, tt="bf16", xt="bf16", zipf=True),
        # a training step: the tokens of 8 streams of 4096, words by their frequency, float32 gradients
        dict(name="embed_train", op="embed", kind="train", T=32768, V=131072, D=2048, tt="f32", xt="bf16", zipf=True),
        # a small odd vocabulary and width, padding among the tokens
        dict(name="embed_train_odd", op="embed", kind="train", T=5003, V=32003, D=1000, tt="f32", xt="f32", zipf=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gdr", "gdr", "norm", "embed"))
    xt = rng.choice(("bf16", "bf16", "f32"))
    if op == "gdr":
        kind = rng.choice(("step", "fwd", "train"))
        dk, dv = rng.choice((32, 64, 72, 96, 120, 128, 128)), rng.choice((32, 56, 64, 96, 128, 128))
        Hk = rng.choice((1, 2, 4, 8, 16))
        Hv = Hk * rng.choice((1, 1, 2, 3))
        c = dict(op=op, kind=kind, Hk=Hk, Hv=Hv, dk=dk, dv=dv, xt=xt, gt=rng.choice(("bf16", "f32")))
        if kind == "step":
            B = max(1, min(_log_int(rng, 1, 512), 512 * 16 // Hv))
            return dict(c, B=B, slots=B + rng.randrange(0, 50))
        P = _log_int(rng, 1, 32)
        # no more than half of the largest case's work, and no row by row check of 64 bits over many steps
        most = 32768 * 16 * 128 * 128 // (Hv * dk * dv) // (4 if xt == "f32" else 2)
        rows = max(1, min(_log_int(rng, 1, 8192), most // P))
        return dict(c, P=P, rows=P * rows, ragged=bool(rng.randrange(2)))
    if op == "norm":
        group = 4 * _log_int(rng, 8, 2048)
        D = group * max(1, min(rng.choice((1, 1, 1, 4, 7, 16)), 8192 // group))
        rows = max(1, min(_log_int(rng, 1, 16384), 60_000_000 // D // (2 if xt == "f32" else 1)))
        post, res = rng.choice((True, False)), rng.choice((True, True, False))
        return dict(op=op, kind=rng.choice(("fwd", "train")), rows=rows, D=D, group=group, post=post,
                    gate=rng.choice(("none", "sigmoid", "silu")), res=res, cs=rng.choice((True, False)),
                    pre=rng.choice((True, True, False)), xt=xt)
    V = _log_int(rng, 200, 131072)
    D = 4 * _log_int(rng, 16, 1024)
    T = max(1, min(_log_int(rng, 1, 32768), 60_000_000 // D))
    return dict(op=op, kind=rng.choice(("fwd", "train")), T=T, V=min(V, 260_000_000 // D), D=D, tt=rng.choice(("bf16", "f32")),
                xt=xt, zipf=bool(rng.randrange(2)))


# ---- inputs ----------------------------------------------------------------------------------------
def _offsets(case, seed):
    """Row offsets [P + 1] of the sequences: equal lengths, or ragged ones (an empty one among them)."""
    P, rows = case["P"], case["rows"]
    if not case["ragged"] or P == 1:
        return np.arange(P + 1, dtype=np.int64) * (rows // P)
    r = np.random.default_rng(seed)
    share = r.lognormal(0.0, 0.7, P)
    share[r.integers(P)] = 0.0
    off = np.round(np.concatenate([[0.0], np.cumsum(share / share.sum())]) * rows).astype(np.int64)
    off[-1] = rows
    return off


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 29)
    t = DT[case["xt"]]

    def randn(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return (torch.randn(shape, device=dev, generator=gen) * scale + shift).to(dtype)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, device=dev, dtype=dtype)

    s = {"case": dict(case)}
    if case["op"] == "gdr":
        Hk, Hv, dk, dv, gt = case["Hk"], case["Hv"], case["dk"], case["dv"], DT[case["gt"]]
        rows = case["B"] if case["kind"] == "step" else case["rows"]
        # queries and keys of length 1, keys with something in common; slices of one projection's rows
        fused = torch.empty(rows, 2 * Hk * dk + Hv * dv, device=dev, dtype=t)
        q, k = randn(rows, Hk, dk), randn(rows, Hk, dk) + 0.3 * randn(1, Hk, dk)
        s["q"] = fused[:, :Hk * dk].view(rows, Hk, dk)
        s["k"] = fused[:, Hk * dk:2 * Hk * dk].view(rows, Hk, dk)
        s["v"] = fused[:, 2 * Hk * dk:].view(rows, Hv, dv)
        s["q"].copy_(q / q.norm(dim=2, keepdim=True))
        s["k"].copy_(k / k.norm(dim=2, keepdim=True))
        s["v"].copy_(randn(rows, Hv, dv))
        # decays from a few tokens to a thousand, by head; write strengths in (0, 1)
        rate = torch.exp(torch.linspace(math.log(0.02), math.log(4.0), Hv, device=dev))
        s["g"] = (-rate * torch.nn.functional.softplus(randn(rows, Hv, shift=-2.0))).to(gt)
        s["beta"] = torch.sigmoid(randn(rows, Hv)).to(gt)
        s["y"] = empty(rows, Hv, dv, dtype=t)
        if case["kind"] == "step":
            s["state"] = randn(case["slots"], Hv, dk, dv, scale=0.5)
            s["slots"] = torch.randperm(case["slots"], device=dev, generator=gen)[:rows].to(torch.int32)
            return s
        P = case["P"]
        off = _offsets(case, seed)
        s["cuts"] = off.tolist()
        s["offsets"] = torch.from_numpy(off).to(dev) if case["ragged"] else None
        s["h0"], s["hT"] = randn(P, Hv, dk, dv, scale=0.5), empty(P, Hv, dk, dv)
        if case["kind"] == "train":
            s["dy"] = randn(rows, Hv, dv, dtype=t)
            s["dhT"], s["dh0"] = randn(P, Hv, dk, dv, scale=0.1), empty(P, Hv, dk, dv)
            s["dq"], s["dk"] = empty(rows, Hk, dk, dtype=t), empty(rows, Hk, dk, dtype=t)
            s["dv"] = empty(rows, Hv, dv, dtype=t)
            s["dg"], s["dbeta"] = empty(rows, Hv, dtype=gt), empty(rows, Hv, dtype=gt)
        return s
    if case["op"] == "norm":
        n, D = case["rows"], case["D"]
        s["o"] = randn(n, D, dtype=t, scale=0.7)
        s["z"] = randn(n, D, dtype=t) if case["gate"] != "none" else None
        s["x"] = randn(n, D, dtype=t, scale=2.0) if case["res"] else None
        s["w_post"] = randn(case["group"], scale=0.1, shift=1.0) if case["post"] else None
        s["w_pre"] = randn(D, scale=0.1, shift=1.0) if case["pre"] else None
        s["cs"] = randn(D, scale=0.1, shift=0.5) if case["cs"] else None
        s["r"] = empty(n, D, dtype=t)
        s["y"] = empty(n, D, dtype=t) if case["pre"] else None
        if case["kind"] == "train":
            s["dr"] = randn(n, D, dtype=t)
            s["dy"] = randn(n, D, dtype=t) if case["pre"] else None
            s["do"] = empty(n, D, dtype=t)
            s["dz"] = empty(n, D, dtype=t) if s["z"] is not None else None
            s["dx"] = empty(n, D, dtype=t) if case["res"] else None
            s["dw_post"] = empty(case["group"]) if case["post"] else None
            s["dw_pre"] = empty(D) if case["pre"] else None
            s["dcs"] = empty(D) if case["cs"] else None
        return s
    T, V, D = case["T"], case["V"], case["D"]
    u = torch.rand(T, device=dev, generator=gen, dtype=torch.float64)
    # words by their frequency (rank r about as often as 1 / r), or all alike; one in 50 is padding
    r = torch.exp(u * math.log(V)).long() - 1 if case["zipf"] else (u * V).long()
    r = r.clamp(0, V - 1)
    s["ids"] = torch.where(torch.rand(T, device=dev, generator=gen) < 0.02, -1, (r * 48271 + 11) % V).to(torch.int32)
    s["y"] = empty(T, D, dtype=t)
    s["table"] = randn(V, D, dtype=DT[case["tt"]])
    if case["kind"] == "train":
        s["dy"] = randn(T, D, dtype=t)
        s["dtable"] = empty(V, D, dtype=DT[case["tt"]])
    return s


# ---- the framework's calls -------------------------------------------------------------------------
@functools.lru_cache(maxsize=256)
def _gdr_spec(P, rows, Hk, Hv, dk, dv, xt, gt):
    import sparse_slot_memory_gb300 as sdm

    return sdm.GdrSpec(P=P, rows=rows, k_heads=Hk, v_heads=Hv, dk=dk, dv=dv, x_dtype=xt, g_dtype=gt, scale=dk ** -0.5)


@functools.lru_cache(maxsize=256)
def _norm_spec(rows, D, group, post, gate, res, pre, xt):
    import sparse_slot_memory_gb300 as sdm

    return sdm.BlockNormSpec(rows=rows, D=D, group=group, post=post, gate=gate, residual=res, pre=pre, scale=0.8, dtype=xt)


@functools.lru_cache(maxsize=256)
def _embed_spec(T, V, D, tt, xt):
    import sparse_slot_memory_gb300 as sdm

    return sdm.EmbedSpec(tokens=T, V=V, D=D, table_dtype=tt, dtype=xt, scale=D ** 0.5)


def _own_gdr(s, c):
    import sparse_slot_memory_gb300 as sdm

    shape = (c["Hk"], c["Hv"], c["dk"], c["dv"], c["xt"], c["gt"])
    x = [s[k] for k in ("q", "k", "v", "g", "beta")]
    if c["kind"] == "step":
        sdm.gdr_step(_gdr_spec(1, c["B"], *shape), *x, s["state"], s["y"], slots=s["slots"])
        return {"y": s["y"], "state": s["state"]}
    spec = _gdr_spec(c["P"], c["rows"], *shape)
    ws = sdm.alloc_gdr_workspace(spec)
    if c["kind"] == "fwd":
        sdm.gdr_forward(spec, *x, s["y"], ws, offsets=s["offsets"], h0=s["h0"], hT=s["hT"])
        return {"y": s["y"], "hT": s["hT"]}
    states = sdm.alloc_gdr_states(spec)
    sdm.gdr_forward(spec, *x, s["y"], ws, offsets=s["offsets"], h0=s["h0"], hT=s["hT"], states=states)
    sdm.gdr_backward(spec, *x, s["dy"], states, s["dq"], s["dk"], s["dv"], s["dg"], s["dbeta"], ws, offsets=s["offsets"],
                     dhT=s["dhT"], dh0=s["dh0"])
    return {k: s[k] for k in ("y", "hT", "dq", "dk", "dv", "dg", "dbeta", "dh0")}


def _own_norm(s, c):
    import sparse_slot_memory_gb300 as sdm

    spec = _norm_spec(*(c[k] for k in ("rows", "D", "group", "post", "gate", "res", "pre", "xt")))
    sdm.block_norm(spec, s["o"], s["r"], x=s["x"], z=s["z"], y=s["y"], w_post=s["w_post"], w_pre=s["w_pre"],
                   channel_scale=s["cs"])
    names = ("r", "y")
    if c["kind"] == "train":
        sdm.block_norm_backward(spec, s["o"], s["r"], s["dr"], s["do"], sdm.alloc_block_norm_workspace(spec), z=s["z"],
                                dy=s["dy"], w_post=s["w_post"], w_pre=s["w_pre"], channel_scale=s["cs"], dx=s["dx"],
                                dz=s["dz"], dw_post=s["dw_post"], dw_pre=s["dw_pre"], d_channel_scale=s["dcs"])
        names += ("do", "dz", "dx", "dw_post", "dw_pre", "dcs")
    return {k: s[k] for k in names if s[k] is not None}


def _own_embed(s, c):
    import sparse_slot_memory_gb300 as sdm

    spec = _embed_spec(c["T"], c["V"], c["D"], c["tt"], c["xt"])
    sdm.embed(spec, s["ids"], s["table"], s["y"])
    if c["kind"] == "fwd":
        return {"y": s["y"]}
    sdm.embed_backward(spec, s["ids"], s["dy"], s["dtable"], sdm.alloc_embed_workspace(spec))
    return {"y": s["y"], "dtable": s["dtable"]}


# ---- the plain forms -------------------------------------------------------------------------------
def _inverse(n):
    """(I + n)^-1 of strictly lower triangular n [.., C, C]: the product of I + (-n)^(2^i)."""
    eye = torch.eye(C, device=n.device)
    p, inv = -n, eye - n
    for _ in range(5):
        p = p @ p
        inv = inv + p @ inv
    return inv


def _plain_gdr(s, c):
    Hk, Hv, dk, dv, t = c["Hk"], c["Hv"], c["dk"], c["dv"], s["y"].dtype
    scale = dk ** -0.5
    if c["kind"] == "step":
        i = s["slots"].long()
        q, k = (s[n].float().repeat_interleave(Hv // Hk, 1) for n in ("q", "k"))
        S = s["state"][i] * s["g"].float().exp()[:, :, None, None]
        u = s["beta"].float()[:, :, None] * (s["v"].float() - (S * k[..., None]).sum(2))
        S = S + k[..., None] * u[:, :, None, :]
        s["state"][i] = S
        return {"y": ((S * q[..., None]).sum(2) * scale).to(t), "state": s["state"]}
    P, cuts = c["P"], s["cuts"]
    n = max(1, max(-(-(cuts[p + 1] - cuts[p]) // C) for p in range(P)))
    # the rows of every sequence in blocks of C, behind its end a row of zeros
    at = torch.arange(n * C, device="cuda")[None, :] + torch.tensor(cuts[:-1], device="cuda")[:, None]
    inside = at < torch.tensor(cuts[1:], device="cuda")[:, None]
    at = torch.where(inside, at, c["rows"])
    x = [s[k].detach().float().requires_grad_(c["kind"] == "train") for k in ("q", "k", "v", "g", "beta", "h0")]
    with torch.set_grad_enabled(c["kind"] == "train"):
        def blocks(a):   # [P, n, heads, C, ..]
            a = torch.cat([a, torch.zeros_like(a[:1])])[at.view(-1)]
            a = a.view(P, n, C, *a.shape[1:]).transpose(2, 3)
            return a.repeat_interleave(Hv // Hk, 2) if a.shape[2] == Hk != Hv else a

        q, k, v, g, beta = (blocks(a) for a in x[:5])
        gam = g.double().cumsum(3)
        low = torch.ones(C, C, device="cuda", dtype=torch.bool).tril()
        D = (gam[..., :, None] - gam[..., None, :]).masked_fill(~low, -math.inf).float().exp()
        G = (k @ k.transpose(3, 4)) * D
        inv = _inverse(G.tril(-1) * beta[..., None, :])
        A = (q @ k.transpose(3, 4)) * D
        b, e = gam.float().exp()[..., None], (gam[..., -1:] - gam).float().exp()[..., None]
        S, ys = x[5], []
        for i in range(n):
            u = beta[:, i, ..., None] * (inv[:, i] @ (v[:, i] - b[:, i] * (k[:, i] @ S)))
            ys.append(scale * (b[:, i] * (q[:, i] @ S) + A[:, i] @ u))
            S = b[:, i, :, -1:] * S + k[:, i].transpose(2, 3) @ (e[:, i] * u)
        y = torch.stack(ys, 1).transpose(2, 3).reshape(P, n * C, Hv, dv)[inside]
        out = {"y": y.detach().to(t), "hT": S.detach()}
        if c["kind"] == "fwd":
            return out
        d = torch.autograd.grad([y, S], x, [s["dy"].float(), s["dhT"]])
    names = ("dq", "dk", "dv", "dg", "dbeta", "dh0")
    return dict(out, **{k: a.to(s[k].dtype) for k, a in zip(names, d)})


def _plain_norm(s, c):
    n, D, G, t = c["rows"], c["D"], c["group"], s["o"].dtype
    o = s["o"].float().view(n, D // G, G)
    rp = torch.rsqrt((o * o).mean(2, keepdim=True) + 1e-6) if c["post"] else None
    m = (o * rp * s["w_post"] if c["post"] else o).view(n, D)
    z = s["z"].float() if c["gate"] != "none" else None
    sg = torch.sigmoid(z) if z is not None else None
    act = 1.0 if z is None else sg if c["gate"] == "sigmoid" else z * sg
    cs = 0.8 * s["cs"] if c["cs"] else 0.8
    nn = m * act
    r = (nn * cs + (s["x"].float() if c["res"] else 0.0)).to(t)
    out = {"r": r}
    rf = r.float()
    if c["pre"]:
        ri = torch.rsqrt((rf * rf).mean(1, keepdim=True) + 1e-6)
        out["y"] = (rf * ri * s["w_pre"]).to(t)
    if c["kind"] == "fwd":
        return out
    dr = s["dr"].float()
    if c["pre"]:
        dy = s["dy"].float()
        h = rf * ri
        out["dw_pre"] = (dy * h).sum(0)
        u = dy * s["w_pre"]
        dr = dr + ri * (u - h * (u * h).mean(1, keepdim=True))
    if c["res"]:
        out["dx"] = dr.to(t)
    if c["cs"]:
        out["dcs"] = 0.8 * (dr * nn).sum(0)
    dn = dr * cs
    if z is not None:
        slope = sg * (1 - sg) if c["gate"] == "sigmoid" else sg * (1 + z * (1 - sg))
        out["dz"] = (dn * m * slope).to(t)
    dm = (dn * act).view(n, D // G, G)
    if c["post"]:
        h = o * rp
        out["dw_post"] = (dm * h).sum((0, 1))
        u = dm * s["w_post"]
        dm = rp * (u - h * (u * h).mean(2, keepdim=True))
    out["do"] = dm.reshape(n, D).to(t)
    return {k: out[k] for k in ("r", "y", "do", "dz", "dx", "dw_post", "dw_pre", "dcs") if k in out}


def _plain_embed(s, c):
    ids, scale = s["ids"].long(), c["D"] ** 0.5
    real = (ids >= 0)[:, None]
    y = torch.where(real, s["table"][ids.clamp(min=0)].float() * scale, 0.0).to(s["y"].dtype)
    if c["kind"] == "fwd":
        return {"y": y}
    dy = torch.where(real, s["dy"].float() * scale, 0.0)
    d = torch.zeros(c["V"], c["D"], device="cuda").index_add_(0, ids.clamp(min=0), dy)
    return {"y": y, "dtable": d.to(s["dtable"].dtype)}


def run(state):
    c = state["case"]
    if own:
        return {"gdr": _own_gdr, "norm": _own_norm, "embed": _own_embed}[c["op"]](state, c)
    return {"gdr": _plain_gdr, "norm": _plain_norm, "embed": _plain_embed}[c["op"]](state, c)


# ---- the definition in 64 bits -----------------------------------------------------------------------
def _exact_gdr(s, c):
    """The recurrence a row at a time, and its gradients a row at a time backwards."""
    Hk, Hv, dk, dv = c["Hk"], c["Hv"], c["dk"], c["dv"]
    R, scale = Hv // Hk, dk ** -0.5
    q, k = (s[n].double().repeat_interleave(R, 1) for n in ("q", "k"))
    v, a, beta = s["v"].double(), s["g"].double().exp(), s["beta"].double()
    if c["kind"] == "step":
        state, i = s["state"].double(), s["slots"].long()
        S = a[..., None, None] * state[i]
        u = beta[..., None] * (v - torch.einsum("bhij,bhi->bhj", S, k))
        S = S + torch.einsum("bhi,bhj->bhij", k, u)
        state[i] = S
        return {"y": scale * torch.einsum("bhij,bhi->bhj", S, q), "state": state}
    P, cuts, rows = c["P"], s["cuts"], c["rows"]
    n = max(cuts[p + 1] - cuts[p] for p in range(P))
    train = c["kind"] == "train"
    if n > 40000 or (train and (n + 1) * P * Hv * dk * dv * 8 > 90e9):
        return None
    at = torch.arange(n, device="cuda")[None, :] + torch.tensor(cuts[:-1], device="cuda")[:, None]
    inside = at < torch.tensor(cuts[1:], device="cuda")[:, None]
    at = torch.where(inside, at, rows)

    def steps(x, fill=0.0):   # [n, P, heads, ..]
        return torch.cat([x, torch.full_like(x[:1], fill)])[at.t().contiguous()]

    q, k, v, beta, a = steps(q), steps(k), steps(v), steps(beta), steps(a, 1.0)
    S = s["h0"].double()
    y = torch.empty_like(v)
    E = torch.empty_like(v)
    if train:
        kept = torch.empty(n + 1, *S.shape, dtype=torch.float64, device="cuda")
        kept[0] = S
    for t in range(n):
        S = a[t][..., None, None] * S
        E[t] = v[t] - (k[t][..., None, :] @ S)[..., 0, :]
        S = torch.baddbmm(S.view(-1, dk, dv), k[t].reshape(-1, dk, 1), (beta[t][..., None] * E[t]).view(-1, 1, dv)).view(S.shape)
        y[t] = scale * (q[t][..., None, :] @ S)[..., 0, :]
        if train:
            kept[t + 1] = S

    def rows_of(x):
        return x.transpose(0, 1)[inside]

    out = {"y": rows_of(y), "hT": S}
    if not train:
        return out
    dy = steps(s["dy"].double())
    dS = s["dhT"].double()
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, dbeta = torch.empty_like(a), torch.empty_like(a)
    for t in range(n - 1, -1, -1):
        dS = torch.baddbmm(dS.view(-1, dk, dv), scale * q[t].reshape(-1, dk, 1), dy[t].reshape(-1, 1, dv)).view(dS.shape)
        dq[t] = scale * (kept[t + 1] @ dy[t][..., None])[..., 0]
        du = (k[t][..., None, :] @ dS)[..., 0, :]
        dbeta[t] = (du * E[t]).sum(-1)
        dv_[t] = beta[t][..., None] * du
        before = a[t][..., None, None] * kept[t]
        dk_[t] = (dS @ (beta[t][..., None] * E[t])[..., None] - before @ dv_[t][..., None])[..., 0]
        dS = torch.baddbmm(dS.view(-1, dk, dv), -k[t].reshape(-1, dk, 1), dv_[t].reshape(-1, 1, dv)).view(dS.shape)
        dg[t] = (dS * before).sum((-1, -2))
        dS = a[t][..., None, None] * dS
    shared = [rows_of(x).view(rows, Hk, R, dk).sum(2) for x in (dq, dk_)]
    return dict(out, dq=shared[0], dk=shared[1], dv=rows_of(dv_), dg=rows_of(dg), dbeta=rows_of(dbeta), dh0=dS)


def _exact_norm(s, c):
    """By the chain rule of torch's own differentiation over the definition, in 64 bits."""
    n, D, G = c["rows"], c["D"], c["group"]
    leaf = {k: s[k].double().requires_grad_() for k in ("o", "z", "x", "w_post", "w_pre", "cs") if s[k] is not None}
    with torch.enable_grad():
        m = leaf["o"]
        if c["post"]:
            h = m.view(n, D // G, G)
            m = (h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt() * leaf["w_post"]).view(n, D)
        if c["gate"] != "none":
            act = 1.0 / (1.0 + torch.exp(-leaf["z"]))
            m = m * (act if c["gate"] == "sigmoid" else act * leaf["z"])
        m = 0.8 * m * leaf.get("cs", 1.0)
        r = m + leaf["x"] if c["res"] else m
        out = {"r": r.detach()}
        # the norm is of r as it is stored, a value of the rows' type: its rounding passes gradients on as they are
        stored = r + (r.detach().to(s["r"].dtype).double() - r.detach())
        total = 0.0
        if c["pre"]:
            y = stored / (stored.square().mean(-1, keepdim=True) + 1e-6).sqrt() * leaf["w_pre"]
            out["y"] = y.detach()
        if c["kind"] == "fwd":
            return out
        total = (r * s["dr"].double()).sum()
        if c["pre"]:
            total = total + (y * s["dy"].double()).sum()
        d = dict(zip(leaf, torch.autograd.grad(total, list(leaf.values()))))
    for k, name in (("o", "do"), ("z", "dz"), ("x", "dx"), ("w_post", "dw_post"), ("w_pre", "dw_pre"), ("cs", "dcs")):
        if k in d:
            out[name] = d[k]
    return out


def _exact_embed(s, c):
    ids, scale = s["ids"].long(), c["D"] ** 0.5
    y = torch.zeros(c["T"], c["D"], device="cuda", dtype=torch.float64)
    y[ids >= 0] = s["table"][ids[ids >= 0]].double() * scale
    if c["kind"] == "fwd":
        return {"y": y}
    d = torch.zeros(c["V"], c["D"], device="cuda", dtype=torch.float64)
    order = torch.sort(ids, stable=True).indices
    order = order[ids[order] >= 0]
    d.index_put_((ids[order],), s["dy"][order].double() * scale, accumulate=True)
    return {"y": y, "dtable": d}


def exact(case, seed):
    s = prepare(case, seed)
    return {"gdr": _exact_gdr, "norm": _exact_norm, "embed": _exact_embed}[case["op"]](s, s["case"])


# ---- work -------------------------------------------------------------------------------------------
def work(case):
    """Each input read once, each output written once."""
    e = SZ[case["xt"]]
    if case["op"] == "gdr":
        Hk, Hv, dk, dv, ge = case["Hk"], case["Hv"], case["dk"], case["dv"], SZ[case["gt"]]
        row = 2 * Hk * dk * e + 2 * Hv * dv * e + 2 * Hv * ge   # q, k, v, y, g, beta
        state = 4 * Hv * dk * dv
        if case["kind"] == "step":
            return {"bytes": case["B"] * (row + 2 * state + 4), "flops": case["B"] * Hv * 8 * dk * dv}
        n, f = case["rows"], 6 * Hv * dk * dv   # what a row reads of the state, the write, the answer
        b = n * row + 2 * case["P"] * state
        if case["kind"] == "train":   # dy in; dq, dk, dv, dg, dbeta out; the states' gradients
            b += n * (2 * Hk * dk * e + 2 * Hv * dv * e + 2 * Hv * ge) + 2 * case["P"] * state
            f += 14 * Hv * dk * dv
        return {"bytes": b, "flops": n * f}
    if case["op"] == "norm":
        n, D = case["rows"], case["D"]
        arrays = 2 + case["pre"] + case["res"] + (case["gate"] != "none")          # o, r, y, x, z
        small = 4 * (case["group"] * case["post"] + D * case["pre"] + D * case["cs"])
        f = 12 * n * D
        if case["kind"] == "train":   # dr, dy in; do, dz, dx out
            arrays += 2 + case["pre"] + case["res"] + (case["gate"] != "none")
            small, f = 2 * small, 36 * n * D
        return {"bytes": arrays * n * D * e + small, "flops": f}
    T, V, D, te = case["T"], case["V"], case["D"], SZ[case["tt"]]
    b, f = T * 4 + min(T, V) * D * te + T * D * e, T * D
    if case["kind"] == "train":
        b, f = b + T * D * e + V * D * te, f + T * D
    return {"bytes": b, "flops": f}
