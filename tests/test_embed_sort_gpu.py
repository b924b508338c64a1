"""The sort behind the embedding's gradient at its own borders: 10 bits a pass, so one pass up to 1023 ids, two up to 2^20 - 1, three
beyond; 256 warps that keep 128 tokens each in registers, so more than 32768 tokens are read twice."""

import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from test_embed_gpu import case, compare

pytestmark = pytest.mark.gpu


def ids_of(T, V, skew, seed=0):
    """Ids of the whole range, more often low ones with `skew`, with both ends, the digits' borders and padding among them."""
    gen = torch.Generator().manual_seed(seed)
    ids = (torch.rand(T, generator=gen, dtype=torch.float64) ** (1 + skew) * V).long().clamp(0, V - 1)
    ends = torch.tensor([v for v in (0, 1, 1022, 1023, 1024, 1025, 2 ** 20 - 1, 2 ** 20, 2 ** 20 + 1, V - 2, V - 1) if 0 <= v < V])
    at = torch.randperm(T, generator=gen)
    k = min(4 * len(ends), T)
    ids[at[:k]] = ends.repeat(4)[:k]
    ids[at[k:k + T // 40]] = -1
    return ids


def repeats(s, c, times=2):
    out = []
    for _ in range(times):
        d, ws = torch.empty(s.V, s.D, dtype=c["table"].dtype, device="cuda"), sdm.alloc_embed_workspace(s)
        ws.fill_(255)
        sdm.embed_backward(s, c["ids"], c["dy"], d, ws)
        out.append(d)
    return all(torch.equal(out[0], d) for d in out[1:])


@pytest.mark.parametrize("skew", [0.0, 6.0])
@pytest.mark.parametrize("V", [1023, 1024, 2 ** 20 - 1, 2 ** 20, 2 ** 20 + 77])
def test_passes(V, skew):
    s, c = case(5000, V, 8, ids=ids_of(5000, V, skew))
    assert compare(s, c)[0] == 0 and repeats(s, c)


@pytest.mark.parametrize("V", [700, 3000, 2 ** 20 + 5])
@pytest.mark.parametrize("T", [32767, 32768, 32769, 33025, 100003])
def test_tokens_that_leave_the_registers(T, V):
    s, c = case(T, V, 4, ids=ids_of(T, V, 3.0, seed=T))
    assert compare(s, c)[0] == 0 and repeats(s, c)


@pytest.mark.parametrize("xt, tt", [("f32", "bf16"), ("bf16", "f32")])
def test_long_batches_in_wide_rows(xt, tt):
    """Added to what the table's gradient holds, and to nothing; all tokens of one word, and of two that take turns."""
    T, V = 40009, 1500
    s, c = case(T, V, 36, xt=xt, tt=tt, ids=ids_of(T, V, 9.0))
    assert compare(s, c, accumulate=True)[0] == 0 and compare(s, c)[0] == 0
    for ids in (torch.full((T,), V - 1), torch.arange(T) % 2 * 1024):
        s, c = case(T, V, 4, xt=xt, tt=tt, ids=ids)
        assert compare(s, c)[0] == 0 and repeats(s, c)


def test_the_order_of_the_tokens_is_kept_over_reloads():
    """Rows of up to 16 tokens that lie 5000 apart are added in the tokens' order, which float32's roundings show."""
    T, V = 70001, 5000
    ids = torch.arange(T) % V   # 14 or 15 tokens an id, 5000 apart
    s, c = case(T, V, 4, xt="f32", ids=ids)
    d = torch.empty(V, 4, device="cuda")
    sdm.embed_backward(s, c["ids"], c["dy"], d, sdm.alloc_embed_workspace(s))
    want = torch.zeros(V, 4, device="cuda")
    for b in range(0, T, V):
        n = min(V, T - b)
        want[:n] += c["dy"][b:b + n]
    assert torch.equal(d, want * s.scale)


def test_the_largest_table():
    V, T = 1 << 28, 40000
    ids = ids_of(T, V, 0.0)
    s = sdm.EmbedSpec(tokens=T, V=V, D=4, table_dtype="bf16", dtype="bf16")
    dy = torch.randn(T, 4, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    d = torch.full((V, 4), float("nan"), dtype=torch.bfloat16, device="cuda")
    sdm.embed_backward(s, ids.to(torch.int32).cuda(), dy, d, sdm.alloc_embed_workspace(s))
    real = ids >= 0
    rows, inverse, counts = ids[real].unique(return_inverse=True, return_counts=True)
    sums = torch.zeros(len(rows), 4, dtype=torch.float64).index_add_(0, inverse, dy[real.cuda()].double().cpu())
    mags = torch.zeros(len(rows), 4, dtype=torch.float64).index_add_(0, inverse, dy[real.cuda()].double().cpu().abs())
    got = d[rows.cuda()].double().cpu()
    assert bool(((got - sums).abs() <= 2.0 ** -8 * sums.abs() + (counts[:, None] + 2) * 2.0 ** -23 * mags).all())
    d[rows.cuda()] = 0
    assert bool((d.view(torch.int16) == 0).all())
