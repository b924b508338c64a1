"""The operators inside a captured CUDA graph, as a server replays a token's step: every launch form (single blocks,
clusters, segments, several kernels to a call) gives on replay, with new inputs in the same buffers, what a plain call
gives."""

import pytest
import torch

import sparse_slot_memory_gb300 as sdm

pytestmark = pytest.mark.gpu


def randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


def recurrence(P, T, D, gw):
    def make(gen):
        return {"x": randn(gen, P * T, D), "dy": randn(gen, P * T, D),
                "g": torch.nn.functional.logsigmoid(randn(gen, P * T, D // gw, dtype=torch.float32) + 3)}

    spec = sdm.GlrSpec(P=P, rows=P * T, D=D, gate_width=gw)
    states, ws = sdm.alloc_glr_states(spec), sdm.alloc_glr_workspace(spec)

    def call(i, o):
        sdm.glr_forward(spec, i["x"], i["g"], o["y"], hT=o["hT"], states=states)
        sdm.glr_backward(spec, i["x"], i["g"], i["dy"], states, o["dx"], o["dg"], ws)

    out = lambda: {"y": torch.zeros(P * T, D, dtype=torch.bfloat16, device="cuda"), "hT": torch.zeros(P, D, device="cuda"),
                   "dx": torch.zeros(P * T, D, dtype=torch.bfloat16, device="cuda"),
                   "dg": torch.zeros(P * T, D // gw, device="cuda")}
    return make, call, out


def token_step():
    B, D, V = 24, 256, 20000
    step = sdm.GlrSpec(P=1, rows=B, D=D)
    heads = sdm.RopeSpec(tokens=B, q_heads=4, k_heads=2, hd=64, rot_dim=64, max_pos=512)
    lp = sdm.LogprobSpec(rows=B, V=V, K=5)
    table = torch.empty(512, 64, device="cuda")
    sdm.rope_table(heads, sdm.rope_frequencies(64), table)

    def make(gen):
        return {"x": randn(gen, B, D), "g": -torch.rand(B, D, generator=gen).cuda(), "state": randn(gen, B, D, dtype=torch.float32),
                "q": randn(gen, B, 4, 64), "k": randn(gen, B, 2, 64),
                "pos": torch.randint(0, 512, (B,), generator=gen).to(torch.int32).cuda(),
                "logits": randn(gen, B, V), "targets": torch.randint(0, V, (B,), generator=gen).to(torch.int32).cuda()}

    def call(i, o):
        o["state"].copy_(i["state"])
        sdm.glr_step(step, i["x"], i["g"], o["state"], o["y"])
        sdm.qk_norm_rope(heads, i["q"], i["k"], i["pos"], table, None, None, o["q"], o["k"])
        sdm.token_logprobs(lp, i["logits"], i["targets"], o["logp"], top_vals=o["vals"], top_idx=o["idx"])

    def out():
        z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")
        return {"state": z(B, D), "y": z(B, D, dtype=torch.bfloat16), "q": z(B, 4, 64, dtype=torch.bfloat16),
                "k": z(B, 2, 64, dtype=torch.bfloat16), "logp": z(B), "vals": z(B, 5), "idx": z(B, 5, dtype=torch.int32)}

    return make, call, out


@pytest.mark.parametrize("form", ["blocks", "clusters", "segments", "wide_heads", "token_step"])
def test_replays_equal_plain_calls(form):
    make, call, out = {"blocks": lambda: recurrence(60, 70, 512, 1), "clusters": lambda: recurrence(2, 1000, 256, 1),
                       "segments": lambda: recurrence(1, 6000, 128, 64), "wide_heads": lambda: recurrence(2, 300, 512, 256),
                       "token_step": token_step}[form]()
    gen = torch.Generator().manual_seed(2)
    held, o = make(gen), out()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call(held, o)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call(held, o)
    for _ in range(3):
        new, want = make(gen), out()
        call(new, want)
        for k in held:
            held[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(o[k], want[k]), (form, k)
