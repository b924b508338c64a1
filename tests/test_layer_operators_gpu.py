"""The delta rule, the block's norms and the embedding as a program runs them: in captured graphs that share their workspaces, on
streams of their own, refused where their tensors lie on another GPU, and together as the layers of a model, whose loss and
gradients are compared with the same model in 64 bits."""

import pytest
import torch
import torch.nn.functional as F

import sparse_slot_memory_gb300 as sdm
from sparse_slot_memory_gb300 import operators

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def randn(gen, *shape, dtype=BF16):
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


def zeros(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def delta(P, T, Hk, Hv, d, xt):
    n, dt = P * T, BF16 if xt == "bf16" else F32
    spec = sdm.GdrSpec(P=P, rows=n, k_heads=Hk, v_heads=Hv, dk=d, dv=d, x_dtype=xt, scale=d ** -0.5)
    states, ws = sdm.alloc_gdr_states(spec), sdm.alloc_gdr_workspace(spec)

    def make(gen):
        unit = lambda H: F.normalize(randn(gen, n, H, d, dtype=F32), dim=2).to(dt)
        return {"q": unit(Hk), "k": unit(Hk), "v": randn(gen, n, Hv, d, dtype=dt), "dy": randn(gen, n, Hv, d, dtype=dt),
                "g": -torch.rand(n, Hv, generator=gen).cuda(), "beta": torch.rand(n, Hv, generator=gen).cuda(),
                "dhT": randn(gen, P, Hv, d, d, dtype=F32)}

    def call(i, o, stream=None):
        x = [i[m] for m in ("q", "k", "v", "g", "beta")]
        sdm.gdr_forward(spec, *x, o["y"], ws, hT=o["hT"], states=states, stream=stream)
        sdm.gdr_backward(spec, *x, i["dy"], states, *[o[m] for m in ("dq", "dk", "dv", "dg", "dbeta")], ws, dhT=i["dhT"], dh0=o["dh0"],
                         stream=stream)

    def out():
        return {"y": zeros(n, Hv, d, dtype=dt), "hT": zeros(P, Hv, d, d), "dq": zeros(n, Hk, d, dtype=dt), "dk": zeros(n, Hk, d, dtype=dt),
                "dv": zeros(n, Hv, d, dtype=dt), "dg": zeros(n, Hv), "dbeta": zeros(n, Hv), "dh0": zeros(P, Hv, d, d)}

    return make, call, out


def norms(n, D, group):
    spec = sdm.BlockNormSpec(rows=n, D=D, group=group, gate="silu", scale=0.5)
    ws = sdm.alloc_block_norm_workspace(spec)
    rows, cols = ("o", "x", "z", "dr", "dy"), {"w_post": group or D, "w_pre": D, "channel_scale": D}

    def make(gen):
        return {m: randn(gen, n, D) for m in rows} | {m: randn(gen, c, dtype=F32) for m, c in cols.items()}

    def call(i, o, stream=None):
        w = {m: i[m] for m in cols}
        sdm.block_norm(spec, i["o"], o["r"], x=i["x"], z=i["z"], y=o["y"], **w, stream=stream)
        sdm.block_norm_backward(spec, i["o"], o["r"], i["dr"], o["d_o"], ws, z=i["z"], dy=i["dy"], **w, dx=o["dx"], dz=o["dz"],
                                dw_post=o["dw_post"], dw_pre=o["dw_pre"], d_channel_scale=o["d_channel_scale"], stream=stream)

    def out():
        return {m: zeros(n, D, dtype=BF16) for m in ("r", "y", "d_o", "dx", "dz")} | {"d" + ("_" if m[0] == "c" else "") + m: zeros(c)
                                                                                         for m, c in cols.items()}

    return make, call, out


def words(T, V, D):
    spec = sdm.EmbedSpec(tokens=T, V=V, D=D)
    ws = sdm.alloc_embed_workspace(spec)

    def make(gen):
        return {"ids": (torch.rand(T, generator=gen) ** 3 * V).to(I32).cuda() - 1, "table": randn(gen, V, D, dtype=F32), "dy": randn(gen, T, D)}

    def call(i, o, stream=None):
        sdm.embed(spec, i["ids"], i["table"], o["y"], stream=stream)
        sdm.embed_backward(spec, i["ids"], i["dy"], o["dtable"], ws, stream=stream)

    return make, call, lambda: {"y": zeros(T, D, dtype=BF16), "dtable": zeros(V, D)}


def token_step():
    B, Hv, d = 24, 4, 64
    D = Hv * d
    rule = sdm.GdrSpec(P=1, rows=B, k_heads=Hv, v_heads=Hv, dk=d, dv=d)
    word, norm = sdm.EmbedSpec(tokens=B, V=300, D=D), sdm.BlockNormSpec(rows=B, D=D)

    def make(gen):
        return {"ids": torch.randint(-1, 300, (B,), generator=gen).to(I32).cuda(), "table": randn(gen, 300, D, dtype=F32),
                "q": F.normalize(randn(gen, B, Hv, d, dtype=F32), dim=2).to(BF16), "k": F.normalize(randn(gen, B, Hv, d, dtype=F32), dim=2).to(BF16),
                "g": -torch.rand(B, Hv, generator=gen).cuda(), "beta": torch.rand(B, Hv, generator=gen).cuda(),
                "state": randn(gen, 2 * B, Hv, d, d, dtype=F32), "slots": torch.randperm(2 * B, generator=gen)[:B].to(I32).cuda()}

    def call(i, o, stream=None):
        o["state"].copy_(i["state"])
        sdm.embed(word, i["ids"], i["table"], o["x"], stream=stream)
        sdm.gdr_step(rule, i["q"], i["k"], o["x"].view(B, Hv, d), i["g"], i["beta"], o["state"], o["h"], slots=i["slots"], stream=stream)
        sdm.block_norm(norm, o["h"].view(B, D), o["r"], x=o["x"], y=o["y"], stream=stream)

    def out():
        return {m: zeros(B, D, dtype=BF16) for m in ("x", "r", "y")} | {"h": zeros(B, Hv, d, dtype=BF16), "state": zeros(2 * B, Hv, d, d)}

    return make, call, out


FORMS = {"delta": lambda: delta(3, 200, 2, 4, 64, "bf16"), "delta_f32": lambda: delta(2, 100, 2, 2, 40, "f32"),
         "delta_wide": lambda: delta(20, 130, 8, 8, 128, "bf16"), "norms": lambda: norms(300, 512, 64), "norms_wide": lambda: norms(33, 4096, 0),
         "words": lambda: words(5000, 700, 256), "token_step": token_step}


def captured(call, held, o):
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call(held, o)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call(held, o)
    return graph


@pytest.mark.parametrize("form", list(FORMS))
def test_replays_of_two_graphs_that_share_workspaces(form):
    make, call, out = FORMS[form]()
    gen = torch.Generator().manual_seed(2)
    held, outs = [make(gen), make(gen)], [out(), out()]
    graphs = [captured(call, h, o) for h, o in zip(held, outs)]
    for i in (0, 1, 1, 0):
        new, want = make(gen), out()
        call(new, want)
        for k in new:
            held[i][k].copy_(new[k])
        graphs[i].replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(outs[i][k], want[k]), (form, k)


@pytest.mark.parametrize("form", list(FORMS))
def test_streams(form):
    """Inputs that another stream is still writing, and calls on that stream, given by it or by being the current one."""
    make, call, out = FORMS[form]()
    gen = torch.Generator().manual_seed(3)
    x, want = make(gen), out()
    call(x, want)
    torch.cuda.synchronize()
    if form == "token_step":   # its copy of the states is torch's, on the current stream
        ways = ("current",)
    else:
        ways = ("current", "given")
    for way in ways:
        stream, held, got = torch.cuda.Stream(), {k: torch.zeros_like(v) for k, v in x.items()}, out()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            big = torch.randn(4096, 4096, device="cuda")
            for _ in range(3):
                big = big @ big * 1e-3
            for k in x:
                held[k].copy_(x[k])
            if way == "current":
                call(held, got)
        if way == "given":
            call(held, got, stream=stream)
        stream.synchronize()
        for k in want:
            assert torch.equal(got[k], want[k]), (way, k)


def small_calls():
    spec = sdm.GdrSpec(P=1, rows=8, k_heads=1, v_heads=1, dk=8, dv=8, x_dtype="f32")
    x, g, h = lambda: zeros(8, 1, 8), lambda: zeros(8, 1), zeros(8, 1, 8, 8)
    states, ws = sdm.alloc_gdr_states(spec), sdm.alloc_gdr_workspace(spec)
    sdm.gdr_forward(spec, x(), x(), x(), g(), g(), x(), ws, states=states)   # the states that a backward needs
    norm, word = sdm.BlockNormSpec(rows=8, D=8, dtype="f32"), sdm.EmbedSpec(tokens=8, V=8, D=8, dtype="f32")
    r, ids = lambda: zeros(8, 8), zeros(8, dtype=I32)
    return {
        "gdr_forward": lambda: sdm.gdr_forward(spec, x(), x(), x(), g(), g(), x(), ws),
        "gdr_backward": lambda: sdm.gdr_backward(spec, x(), x(), x(), g(), g(), x(), states, x(), x(), x(), g(), g(), ws),
        "gdr_step": lambda: sdm.gdr_step(spec, x(), x(), x(), g(), g(), h, x()),
        "block_norm": lambda: sdm.block_norm(norm, r(), r(), x=r(), y=r()),
        "block_norm_backward": lambda: sdm.block_norm_backward(norm, r(), r(), r(), r(), dy=r()),
        "embed": lambda: sdm.embed(word, ids, r(), r()),
        "embed_backward": lambda: sdm.embed_backward(word, ids, r(), r(), sdm.alloc_embed_workspace(word)),
    }


@pytest.mark.parametrize("name", ["gdr_forward", "gdr_backward", "gdr_step", "block_norm", "block_norm_backward", "embed", "embed_backward"])
def test_tensors_of_another_gpu_are_refused(name, monkeypatch):
    call = small_calls()[name]
    call()
    torch.cuda.synchronize()
    other = torch.cuda.current_device() + 1
    monkeypatch.setattr(operators, "_alone", False, raising=False)
    monkeypatch.setattr(operators, "_here", lambda: other, raising=False)
    with pytest.raises(ValueError, match=f"lies on GPU {other - 1}, the current one is GPU {other}"):
        call()


# ---- a model of these layers -------------------------------------------------------------------------------------
class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table):
        ctx.spec = sdm.EmbedSpec(tokens=len(ids), V=table.shape[0], D=table.shape[1], dtype="f32")
        ctx.save_for_backward(ids)
        y = torch.empty(len(ids), table.shape[1], device="cuda")
        sdm.embed(ctx.spec, ids, table, y)
        return y

    @staticmethod
    def backward(ctx, dy):
        d = torch.empty(ctx.spec.V, ctx.spec.D, device="cuda")
        sdm.embed_backward(ctx.spec, *ctx.saved_tensors, dy.contiguous(), d, sdm.alloc_embed_workspace(ctx.spec))
        return None, d


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, spec, o, x, z, w_post, w_pre, cs):
        r, y = torch.empty_like(o), torch.empty_like(o) if spec.pre else None
        sdm.block_norm(spec, o, r, x=x, z=z, y=y, w_post=w_post, w_pre=w_pre, channel_scale=cs)
        ctx.spec = spec
        ctx.save_for_backward(o, r, z, w_post, w_pre, cs)
        return (r, y) if spec.pre else r

    @staticmethod
    def backward(ctx, dr, dy=None):
        spec, (o, r, z, w_post, w_pre, cs) = ctx.spec, ctx.saved_tensors
        new = lambda t: None if t is None else torch.empty_like(t)
        d_o, dx, dz, dwo, dwp, dcs = new(o), new(o) if spec.residual else None, new(z), new(w_post), new(w_pre), new(cs)
        sdm.block_norm_backward(spec, o, r, dr.contiguous(), d_o, sdm.alloc_block_norm_workspace(spec), z=z,
                                dy=None if dy is None else dy.contiguous(), w_post=w_post, w_pre=w_pre, channel_scale=cs, dx=dx, dz=dz,
                                dw_post=dwo, dw_pre=dwp, d_channel_scale=dcs)
        return None, d_o, dx, dz, dwo, dwp, dcs


class Delta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, spec, offsets, q, k, v, g, beta, h0):
        y, hT = torch.empty_like(v), torch.empty_like(h0)
        states, ws = sdm.alloc_gdr_states(spec), sdm.alloc_gdr_workspace(spec, backward=False)
        sdm.gdr_forward(spec, q, k, v, g, beta, y, ws, offsets=offsets, h0=h0, hT=hT, states=states)
        ctx.spec, ctx.offsets, ctx.states = spec, offsets, states
        ctx.save_for_backward(q, k, v, g, beta)
        return y, hT

    @staticmethod
    def backward(ctx, dy, dhT):
        q, k, v, g, beta = ctx.saved_tensors
        d = [torch.empty_like(t) for t in (q, k, v, g, beta)]
        dh0 = torch.empty_like(dhT)
        sdm.gdr_backward(ctx.spec, q, k, v, g, beta, dy.contiguous(), ctx.states, *d, sdm.alloc_gdr_workspace(ctx.spec), offsets=ctx.offsets,
                         dhT=dhT.contiguous(), dh0=dh0)
        return None, None, *d, dh0


V, D, HK, HV, DK = 60, 64, 2, 4, 16
LENS = [70, 1, 133]


def weights(dtype):
    gen = torch.Generator().manual_seed(7)
    w = lambda *s: (torch.randn(*s, generator=gen, dtype=torch.float64) * s[0] ** -0.5)
    p = {"emb": w(V, D) * V ** 0.5, "qkv": w(D, (2 * HK + HV) * DK), "gb": w(D, 2 * HV), "z": w(D, HV * DK), "out": w(HV * DK, D), "head": w(D, V),
         "n0": 1 + 0.1 * w(D), "n1": 1 + 0.1 * w(DK), "n2": 1 + 0.1 * w(D), "n3": 1 + 0.1 * w(D), "cs": 0.7 + 0.1 * w(D),
         "h0": 0.3 * w(len(LENS), HV, DK, DK)}
    return {k: v.to(dtype).cuda().requires_grad_() for k, v in p.items()}


def loss_of(p, ids, targets, ours):
    """A delta-rule layer between norms, and the mean loss of the tokens after; with the library or in plain torch."""
    n, cuts = len(ids), [0, *torch.tensor(LENS).cumsum(0).tolist()]
    rms = lambda t: t * (t.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()
    if ours:
        e = Embed.apply(ids, p["emb"])
        r0, y0 = Norm.apply(sdm.BlockNormSpec(rows=n, D=D, post=False, residual=False, dtype="f32"), e, None, None, None, p["n0"], None)
    else:
        r0 = e = p["emb"][ids.long()]
        y0 = rms(e) * p["n0"]
    q, k, v = (y0 @ p["qkv"]).view(n, -1, DK).split((HK, HK, HV), 1)
    q, k = F.normalize(q, dim=2), F.normalize(k, dim=2)
    g, beta = (y0 @ p["gb"]).split((HV, HV), 1)
    g, beta, z = -F.softplus(g - 2.0), beta.sigmoid(), y0 @ p["z"]
    if ours:
        spec = sdm.GdrSpec(P=len(LENS), rows=n, k_heads=HK, v_heads=HV, dk=DK, dv=DK, x_dtype="f32", scale=DK ** -0.5)
        o, hT = Delta.apply(spec, torch.tensor(cuts, device="cuda"), q, k, v, g, beta, p["h0"])
        head = sdm.BlockNormSpec(rows=n, D=HV * DK, group=DK, gate="silu", residual=False, pre=False, dtype="f32")
        a = Norm.apply(head, o.reshape(n, HV * DK), None, z, p["n1"], None, None)
        _, y1 = Norm.apply(sdm.BlockNormSpec(rows=n, D=D, dtype="f32"), a @ p["out"], r0, None, p["n2"], p["n3"], p["cs"])
    else:
        rows, ends = [], []
        for i in range(len(LENS)):
            S = p["h0"][i]
            for t in range(cuts[i], cuts[i + 1]):
                kk, qq = (x[t].repeat_interleave(HV // HK, 0) for x in (k, q))
                S = S * g[t].exp()[:, None, None]
                u = beta[t][:, None] * (v[t] - torch.einsum("hdv,hd->hv", S, kk))
                S = S + kk[:, :, None] * u[:, None, :]
                rows.append(DK ** -0.5 * torch.einsum("hdv,hd->hv", S, qq))
            ends.append(S)
        o, hT = torch.stack(rows), torch.stack(ends)
        a = F.silu(z) * (rms(o) * p["n1"]).reshape(n, HV * DK)
        r1 = r0 + p["cs"] * (rms(a @ p["out"]) * p["n2"])
        y1 = rms(r1) * p["n3"]
    return F.cross_entropy(y1 @ p["head"], targets.long()) + 0.01 * hT.pow(2).mean()


def test_a_models_loss_and_gradients():
    """In float32 throughout. Every operator, ours and torch's, is within a few units of 2^-24 of its results' norm for each of at most
    266 terms that it adds up (2^-16 with all of one sign); a gradient passes 14 of them forth and back, with factors of norms and
    normalizations between 1/4 and 4 that both sides share: 28 2^-16 = 4e-4 of a gradient's norm."""
    n = sum(LENS)
    gen = torch.Generator().manual_seed(8)
    ids, targets = (torch.randint(0, V, (n,), generator=gen).to(I32).cuda() for _ in range(2))
    p, exact = weights(F32), weights(torch.float64)
    loss, want = loss_of(p, ids, targets, True), loss_of(exact, ids, targets, False)
    assert abs(loss.item() - want.item()) < 28 * 2.0 ** -16 * want.item()
    loss.backward()
    want.backward()
    for k in p:
        error, size = float((p[k].grad.double() - exact[k].grad).norm()), float(exact[k].grad.norm())
        assert size > 0 and error < 28 * 2.0 ** -16 * size, (k, error / size)


def test_answers_token_by_token_follow_a_prompt():
    """The prompt at once and then a token of every stream at a time, beside all at once: the same operators' forms for single
    tokens, within the roundings of bfloat16 rows (2^-8 for each of the value, the answer and the norm's two)."""
    B, T, more, Hv, d = 3, 100, 30, 4, 64
    D = Hv * d
    gen = torch.Generator().manual_seed(9)
    ids, table = torch.randint(0, 50, (B, T + more), generator=gen).to(I32).cuda(), randn(gen, 50, D, dtype=F32)
    wq, wk, wg = (randn(gen, D, n, dtype=F32) * D ** -0.5 for n in (D, D, 2 * Hv))

    def rows(n, ids):
        x = torch.empty(n, D, dtype=BF16, device="cuda")
        sdm.embed(sdm.EmbedSpec(tokens=n, V=50, D=D), ids, table, x)
        r, y = torch.empty_like(x), torch.empty_like(x)
        sdm.block_norm(sdm.BlockNormSpec(rows=n, D=D, post=False, residual=False), x, r, y=y)
        h = lambda w: F.normalize((y.float() @ w).view(n, Hv, d), dim=2).to(BF16)
        g, beta = (y.float() @ wg).split((Hv, Hv), 1)
        return x, h(wq), h(wk), y.view(n, Hv, d), (-F.softplus(g)).contiguous(), beta.sigmoid().contiguous()

    def close(n, x, o):
        r, y = torch.empty(n, D, dtype=BF16, device="cuda"), torch.empty(n, D, dtype=BF16, device="cuda")
        sdm.block_norm(sdm.BlockNormSpec(rows=n, D=D), o.view(n, D), r, x=x, y=y)
        return y

    def whole(ids):
        P, n = ids.shape[0], ids.numel()
        spec = sdm.GdrSpec(P=P, rows=n, k_heads=Hv, v_heads=Hv, dk=d, dv=d, scale=d ** -0.5)
        x, *a = rows(n, ids.reshape(-1).contiguous())
        o, hT = torch.empty(n, Hv, d, dtype=BF16, device="cuda"), torch.empty(P, Hv, d, d, device="cuda")
        sdm.gdr_forward(spec, *a, o, sdm.alloc_gdr_workspace(spec, backward=False), hT=hT)
        return close(n, x, o).view(P, -1, D), hT

    want, end = whole(ids)
    _, state = whole(ids[:, :T])
    step = sdm.GdrSpec(P=1, rows=B, k_heads=Hv, v_heads=Hv, dk=d, dv=d, scale=d ** -0.5)
    for t in range(T, T + more):
        x, *a = rows(B, ids[:, t].contiguous())
        o = torch.empty(B, Hv, d, dtype=BF16, device="cuda")
        sdm.gdr_step(step, *a, state, o)
        got = close(B, x, o)
        error = (got.double() - want[:, t].double()).norm(dim=1) / want[:, t].double().norm(dim=1)
        assert float(error.max()) < 4 * 2.0 ** -8, (t, error)
    assert float((state - end).norm() / end.norm()) < 2.0 ** -8
