"""A small language model around the memory layer, trained and asked: every operator of the library in its place.

One chunk of every stream at a time (the memory and the recurrent state go from chunk to chunk, gradients stay in the
chunk). A token's embedding (``embed``) gives a query and a key head, which are normed and rotated (``qk_norm_rope``) and
name their slots among a fixed codebook; the memory is read (``phase1``, ``read``) and later written (``dw``); what was
read joins the embedding as the input of a gated linear recurrence (``glr_forward``), whose states are normed, added to
the embedding and normed again (``block_norm``). A layer of the gated delta rule (``gdr_forward``) follows, its answers
normed and added in the same way; the last norm gives the logits, and ``token_logprobs`` the loss. Back go
``token_logprobs_backward``, ``block_norm_backward``, ``gdr_backward``, ``glr_backward``, the memory's read side
(``gds``), ``qk_norm_rope_backward`` and ``embed_backward``. Answers take one token of each stream at a time: the same
embedding, norms and rotation for single tokens, ``read``, ``glr_step``, ``gdr_step``, and ``token_logprobs`` with the
likeliest alternatives. Matrix products and the optimizer are torch's.

    python examples/small_decoder.py            # trains on streams that repeat a phrase and prints the losses
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_slot_memory_gb300 as sdm  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class SmallDecoder:
    def __init__(self, P=4, C=64, S=512, W=4, R=4, hd=64, D=256, V=256, max_pos=4096, seed=0):
        self.P, self.C, self.W, self.R, self.hd, self.D, self.V = P, C, W, R, hd, D, V
        self.H = D // hd   # heads of the delta rule
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def rand(*shape, scale):
            return torch.randn(shape, device="cuda", generator=gen) * scale

        self.w = {"emb": rand(V, D, scale=1.0), "qk": rand(D, 2 * hd, scale=D ** -0.5), "dv": rand(D, hd, scale=D ** -0.5),
                  "x": rand(D, D, scale=D ** -0.5), "g": rand(D, D, scale=D ** -0.5), "m": rand(hd, D, scale=hd ** -0.5),
                  "out": rand(D, V, scale=D ** -0.5), "nq": torch.ones(hd, device="cuda"), "nk": torch.ones(hd, device="cuda"),
                  "qkv": rand(D, 3 * D, scale=D ** -0.5), "gb": rand(D, 2 * self.H, scale=D ** -0.5)}
        # the norms behind and before the recurrence and the delta rule
        self.w |= {n: torch.ones(D, device="cuda") for n in ("n1", "n2", "n3", "n4")}
        self.codebook = rand(S, hd, scale=1.0).to(BF16)
        # one chunk a call: its shape for the memory, the recurrence, the heads and the loss
        self.shape = sdm.ShapeSpec(P=P, C=C, W=W, R=R, hd=hd, steps=1, S=S, valid_last=C)
        self.one = sdm.ShapeSpec(P=P, C=1, W=W, R=R, hd=hd, steps=1, S=S, valid_last=1)
        self.glr = sdm.GlrSpec(P=P, rows=P * C, D=D, x_dtype="bf16", g_dtype="f32")
        self.step = sdm.GlrSpec(P=P, rows=P, D=D, x_dtype="bf16", g_dtype="f32")
        delta = dict(k_heads=self.H, v_heads=self.H, dk=hd, dv=hd, scale=hd ** -0.5)
        self.gdr, self.gdr_one = sdm.GdrSpec(P=P, rows=P * C, **delta), sdm.GdrSpec(P=P, rows=P, **delta)
        heads = dict(q_heads=1, k_heads=1, hd=hd, rot_dim=hd // 2, max_pos=max_pos)
        self.rope, self.rope_one = sdm.RopeSpec(tokens=P * C, **heads), sdm.RopeSpec(tokens=P, **heads)
        self.table = torch.empty(max_pos, hd // 2, device="cuda")
        sdm.rope_table(self.rope, sdm.rope_frequencies(hd // 2), self.table)
        self.ws, self.out = sdm.alloc_workspace(self.shape), sdm.alloc_outputs(self.shape)
        self.states, self.glr_ws = sdm.alloc_glr_states(self.glr), sdm.alloc_glr_workspace(self.glr)
        self.rope_ws = sdm.alloc_rope_workspace(self.rope)
        self.gdr_states, self.gdr_ws = sdm.alloc_gdr_states(self.gdr), sdm.alloc_gdr_workspace(self.gdr)
        self.norm_ws = sdm.alloc_block_norm_workspace(sdm.BlockNormSpec(rows=P * C, D=D))
        self.embed_ws = sdm.alloc_embed_workspace(sdm.EmbedSpec(tokens=P * C, V=V, D=D))
        self.begin()

    def begin(self):
        """Empty memory and states, position 0."""
        self.bank = torch.zeros(self.P * self.shape.S, self.hd, dtype=BF16, device="cuda")
        self.h = torch.zeros(self.P, self.D, device="cuda")
        self.s = torch.zeros(self.P, self.H, self.hd, self.hd, device="cuda")
        self.pos = 0

    def slots(self, head, n):
        """The n slots of every token's head [tokens, 1, hd] and the weights of their scores."""
        top = (head[:, 0] @ self.codebook.T).float().mul_(self.hd ** -0.5).topk(n, 1)
        return top.indices.to(I32), top.values.softmax(1)

    def heads(self, e, spec):
        qk = (e @ self.w["qk"].to(BF16)).view(spec.tokens, 2, self.hd)
        q, k = qk[:, :1], qk[:, 1:]   # slices of one projection's rows
        n = spec.tokens // self.P
        pos = (self.pos + torch.arange(n, device="cuda", dtype=I32)).repeat(self.P)
        qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
        sdm.qk_norm_rope(spec, q, k, pos, self.table, self.w["nq"], self.w["nk"], qo, ko)
        return q, k, pos, qo, ko

    def embed(self, ids):
        e = torch.empty(len(ids), self.D, dtype=BF16, device="cuda")
        sdm.embed(sdm.EmbedSpec(tokens=len(ids), V=self.V, D=self.D), ids, self.w["emb"], e)
        return e

    def add_norm(self, o, x, post, pre):
        """The stream x with a block's normed output o added, and its norm for the next block."""
        r, y = torch.empty_like(x), torch.empty_like(x)
        sdm.block_norm(sdm.BlockNormSpec(rows=len(x), D=self.D), o, r, x=x, y=y, w_post=self.w[post], w_pre=self.w[pre])
        return r, y

    def add_norm_backward(self, o, r, dr, dy, post, pre, d):
        """The gradients of o and of the stream before; the weights' go into d."""
        do, dx = torch.empty_like(o), torch.empty_like(o)
        d[post], d[pre] = torch.empty_like(self.w[post]), torch.empty_like(self.w[pre])
        sdm.block_norm_backward(sdm.BlockNormSpec(rows=len(o), D=self.D), o, r, dr, do, self.norm_ws, dy=dy, w_post=self.w[post],
                                w_pre=self.w[pre], dx=dx, dw_post=d[post], dw_pre=d[pre])
        return do, dx

    def delta_inputs(self, y):
        """Queries and keys of length 1, values, log decays and write strengths of the rows y, and the lengths' inverses."""
        q, k, v = (y @ self.w["qkv"].to(BF16)).view(len(y), 3, self.H, self.hd).unbind(1)
        iq, ik = (t.float().pow(2).sum(2, keepdim=True).add_(1e-6).rsqrt() for t in (q, k))
        g, b = (y @ self.w["gb"].to(BF16)).float().split((self.H, self.H), 1)
        return (q * iq).to(BF16), (k * ik).to(BF16), v, torch.nn.functional.logsigmoid(g + 3.0), b.sigmoid(), iq, ik

    def train_chunk(self, tokens, targets):
        """One chunk [P, C] of tokens and what follows them: the mean loss and the gradients."""
        P, C, n, w = self.P, self.C, self.P * self.C, self.w
        ids = tokens.reshape(-1).to(I32)
        e = self.embed(ids)
        q, k, pos, qo, ko = self.heads(e, self.rope)
        q_idx, q_val = self.slots(qo, self.R)
        k_idx, k_val = self.slots(ko, self.W)
        g = torch.nn.functional.logsigmoid((e @ w["g"].to(BF16)).float() + 2.0)
        o = self.out
        sdm.phase1(self.shape, k_idx, q_idx, k_val.to(BF16), q_val.to(BF16), g.mean(1).mul_(0.1), o, self.ws)
        y = torch.empty(P, C, self.hd, device="cuda")
        sdm.read(self.shape, q_idx, o["q_w"], self.bank, y)
        yb = y.view(n, self.hd).to(BF16)
        x = e @ w["x"].to(BF16) + yb @ w["m"].to(BF16)
        h, hT = torch.empty_like(x), torch.empty_like(self.h)
        sdm.glr_forward(self.glr, x, g, h, h0=self.h, hT=hT, states=self.states)
        r1, y1 = self.add_norm(h, e, "n1", "n2")
        *a, iq, ik = self.delta_inputs(y1)
        a = [t.contiguous() for t in a]
        u, sT = torch.empty_like(a[2]), torch.empty_like(self.s)
        sdm.gdr_forward(self.gdr, *a, u, self.gdr_ws, h0=self.s, hT=sT, states=self.gdr_states)
        r2, y2 = self.add_norm(u.view(n, self.D), r1, "n3", "n4")
        logits = y2 @ w["out"].to(BF16)
        lp = sdm.LogprobSpec(rows=n, V=self.V)
        tgt = targets.reshape(-1).to(I32)
        logp, ent, lse = (torch.empty(n, device="cuda") for _ in range(3))
        sdm.token_logprobs(lp, logits, tgt, logp, entropy=ent, lse=lse)

        # backward
        d_logits = torch.empty_like(logits)
        sdm.token_logprobs_backward(lp, logits, tgt, lse, ent, torch.full((n,), -1.0 / n, device="cuda"), d_logits)
        d = {"out": y2.T.float() @ d_logits.float()}
        du, dr1 = self.add_norm_backward(u.view(n, self.D), r2, None, d_logits @ w["out"].T.to(BF16), "n3", "n4", d)
        da = [torch.empty_like(t) for t in a]
        sdm.gdr_backward(self.gdr, *a, du.view_as(u), self.gdr_states, *da, self.gdr_ws)
        for i, inv in ((0, iq), (1, ik)):   # through the lengths
            t, dt = a[i].float(), da[i].float()
            da[i] = ((dt - t * (dt * t).sum(2, keepdim=True)) * inv).to(BF16)
        dqkv = torch.stack(da[:3], 1).view(n, 3 * self.D)
        dgb = torch.cat([da[3] * (1 - a[3].exp()), da[4] * a[4] * (1 - a[4])], 1)
        d["qkv"], d["gb"] = y1.T.float() @ dqkv.float(), y1.T.float() @ dgb
        dy1 = (dqkv.float() @ w["qkv"].T + dgb @ w["gb"].T).to(BF16)
        dh, de1 = self.add_norm_backward(h, r1, dr1, dy1, "n1", "n2", d)
        dx, dg = torch.empty_like(x), torch.empty_like(g)
        sdm.glr_backward(self.glr, x, g, dh, self.states, dx, dg, self.glr_ws)
        dz = dg * (1 - g.exp())   # of the gates' sigmoid
        d["x"], d["g"], d["m"] = e.T.float() @ dx.float(), e.T.float() @ dz, yb.T.float() @ dx.float()
        de = de1.float() + dx.float() @ w["x"].T + dz @ w["g"].T
        # the read weights' gradient, and through the scores' softmax the query's
        gr = (dx @ w["m"].T.to(BF16)).float()
        d_qw = torch.empty(n, self.R, device="cuda")
        sdm.gds(self.shape, o["sorted_q"], q_idx, q_val.to(BF16), o["log_q"], gr, self.bank,
                torch.zeros(self.bank.shape, device="cuda"), d_qw)
        dv = d_qw * o["log_q"].view(n, self.R).exp()
        ds = q_val * (dv - (dv * q_val).sum(1, keepdim=True)) * self.hd ** -0.5
        dq_out = torch.einsum("nr,nrd->nd", ds, self.codebook[q_idx.long()].float()).to(BF16).view(n, 1, self.hd)
        dq, dk = torch.empty_like(qo), torch.empty_like(ko)
        d["nq"], dnk = torch.empty(self.hd, device="cuda"), torch.empty(self.hd, device="cuda")
        sdm.qk_norm_rope_backward(self.rope, dq_out, torch.zeros_like(ko), q, k, pos, self.table, w["nq"], w["nk"], dq, dk,
                                  d["nq"], dnk, self.rope_ws)
        dqk = torch.cat([dq, dk], 1).view(n, 2 * self.hd)
        d["qk"] = e.T.float() @ dqk.float()
        de += dqk.float() @ w["qk"].T
        d["emb"] = torch.empty_like(w["emb"])
        sdm.embed_backward(sdm.EmbedSpec(tokens=n, V=self.V, D=self.D, dtype="f32"), ids, de, d["emb"], self.embed_ws)

        # the chunk is written, its state goes on
        sdm.dw(self.shape, e @ w["dv"].to(BF16), self.bank, self.ws)
        self.h, self.s = hT, sT
        self.pos += C
        return -logp.mean(), d

    def train(self, stream, steps, lr=0.0015):
        """``steps`` passes over the chunks of ``stream`` [P, n C + 1] with Adam; the mean loss of each."""
        m = {k: torch.zeros_like(v) for k, v in self.w.items()}
        v2 = {k: torch.zeros_like(v) for k, v in self.w.items()}
        losses, t = [], 0
        for _ in range(steps):
            self.begin()
            total = []
            for c in range((stream.shape[1] - 1) // self.C):
                s = stream[:, c * self.C:(c + 1) * self.C + 1]
                loss, d = self.train_chunk(s[:, :-1], s[:, 1:])
                total.append(loss)
                t += 1
                for k, grad in d.items():
                    m[k].mul_(0.9).add_(grad, alpha=0.1)
                    v2[k].mul_(0.99).addcmul_(grad, grad, value=0.01)
                    self.w[k].addcdiv_(m[k] / (1 - 0.9 ** t), (v2[k] / (1 - 0.99 ** t)).sqrt_().add_(1e-8), value=-lr)
            losses.append(float(torch.stack(total).mean()))
        return losses

    def answer(self, tokens, n, K=5):
        """``n`` tokens after ``tokens`` [P], the likeliest each time, with their log probabilities and those of K
        alternatives: one token of every stream a step."""
        lp = sdm.LogprobSpec(rows=self.P, V=self.V, K=K)
        y = torch.empty(self.P, 1, self.hd, device="cuda")
        h = torch.empty(self.P, self.D, dtype=BF16, device="cuda")
        logp = torch.empty(self.P, device="cuda")
        vals, idx = torch.empty(self.P, K, device="cuda"), torch.empty(self.P, K, dtype=I32, device="cuda")
        none = torch.full((self.P,), -1, dtype=I32, device="cuda")
        out = []
        for _ in range(n):
            e = self.embed(tokens.to(I32))
            _, _, _, qo, _ = self.heads(e, self.rope_one)
            q_idx, q_val = self.slots(qo, self.R)
            sdm.read(self.one, q_idx, q_val.to(BF16), self.bank, y)
            g = torch.nn.functional.logsigmoid((e @ self.w["g"].to(BF16)).float() + 2.0)
            x = e @ self.w["x"].to(BF16) + y.view(self.P, self.hd).to(BF16) @ self.w["m"].to(BF16)
            sdm.glr_step(self.step, x, g, self.h, h)
            r, z = self.add_norm(h, e, "n1", "n2")
            *a, _, _ = self.delta_inputs(z)
            u = torch.empty(self.P, self.H, self.hd, dtype=BF16, device="cuda")
            sdm.gdr_step(self.gdr_one, *(t.contiguous() for t in a), self.s, u)
            _, z = self.add_norm(u.view(self.P, self.D), r, "n3", "n4")
            sdm.token_logprobs(lp, z @ self.w["out"].to(BF16), none, logp, top_vals=vals, top_idx=idx)
            tokens = idx[:, 0].long()
            self.pos += 1
            out.append((tokens.clone(), vals.clone(), idx.clone()))
        return out


def phrases(P, V, n, length=24, seed=1):
    """Streams that repeat a phrase of their own."""
    gen = torch.Generator().manual_seed(seed)
    p = torch.randint(V, (P, length), generator=gen)
    return p.repeat(1, -(-n // length))[:, :n].cuda()


def main():
    model = SmallDecoder()
    stream = phrases(model.P, model.V, 4 * model.C + 1)
    for i, loss in enumerate(model.train(stream, 20)):
        print(f"pass {i}: loss {loss:.3f}")
    right = sum(int((t == s).sum()) for (t, _, _), s in zip(model.answer(stream[:, -1], 24), phrases(
        model.P, model.V, 4 * model.C + 25)[:, -24:].T))
    print(f"answers: {right} of {24 * model.P} tokens follow the phrases")


if __name__ == "__main__":
    main()
