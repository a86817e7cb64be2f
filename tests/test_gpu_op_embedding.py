"""Embedding lookup and its gradient on the GPU against sums in 64 bits (-m gpu)."""
import pytest
import torch

import op_util as ou
import zero_gradient_sync_gb300 as dp

pytestmark = pytest.mark.gpu


def make_ids(kind, tokens, vocab, dtype, gen):
    if kind == "uniform":
        ids = torch.randint(0, vocab, (tokens,), generator=gen)
    elif kind == "same":
        ids = torch.full((tokens,), vocab - 1)
    elif kind == "two":
        ids = torch.where(torch.rand(tokens, generator=gen) < 0.5, 0, vocab // 2)
    elif kind == "dropped":
        ids = torch.full((tokens,), -1)
    elif kind == "mixed":      # some outside on both sides, many equal
        ids = torch.randint(-2, vocab + 2, (tokens,), generator=gen)
        ids[tokens // 3:tokens // 2] = min(3, vocab - 1)
    return ids.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,vocab,dim,off", [(0, 5, 8, 0), (1, 1, 1, 0), (3, 7, 8, 0), (33, 50, 77, 0), (257, 1000, 768, 0),
                                                  (100, 64, 264, 3), (5, 9, 2048, 8)])
def test_lookup(dev, dtype, tokens, vocab, dim, off):
    gen = torch.Generator().manual_seed(tokens * 7 + dim)
    table, _ = ou.flat_view(vocab * dim, (vocab, dim), dtype, off)
    table.copy_(torch.randn(vocab, dim, generator=gen))
    for id_type in (torch.int32, torch.int64):
        ids = make_ids("mixed" if tokens > 3 else "uniform", tokens, vocab, id_type, gen)
        out, check = ou.flat_view(tokens * dim, (tokens, dim), dtype, off)
        dp.dp_embedding(out, table, ids, scale=1.7)
        torch.cuda.synchronize()
        live = (ids >= 0) & (ids < vocab)
        want = table.double()[ids.long().clamp(0, vocab - 1)] * float(torch.tensor(1.7, dtype=torch.float32)) * live[:, None]
        ou.close(out, want, ou.EPS * want.abs(), "lookup")
        check()


@pytest.mark.parametrize("kind", ["uniform", "same", "two", "dropped", "mixed"])
@pytest.mark.parametrize("tokens,vocab,dim,off,dtype,id_type", [
    (1, 1, 1, 0, torch.bfloat16, torch.int64), (1, 300, 768, 0, torch.bfloat16, torch.int32),
    (31, 3, 8, 0, torch.float32, torch.int64), (257, 70000, 16, 0, torch.bfloat16, torch.int64),
    (1000, 40, 77, 1, torch.bfloat16, torch.int32), (5000, 50257, 264, 0, torch.bfloat16, torch.int64),
    (5000, 130, 768, 8, torch.float32, torch.int32), (20011, 1000, 256, 0, torch.bfloat16, torch.int64),
    (200003, 70000, 8, 0, torch.float32, torch.int32), (140001, 40, 33, 1, torch.bfloat16, torch.int64)])
def test_gradient(dev, kind, tokens, vocab, dim, off, dtype, id_type):
    gen = torch.Generator().manual_seed(tokens + vocab)
    ids = make_ids(kind, tokens, vocab, id_type, gen)
    dout = torch.randn(tokens, dim, generator=gen).to(dtype).cuda()
    pad = 3
    ws = torch.empty(dp.dp_embedding_workspace_size(tokens, vocab, dim), dtype=torch.uint8, device="cuda")
    scale = float(torch.tensor(0.3, dtype=torch.float32))
    live = (ids >= 0) & (ids < vocab) & (ids != pad)
    at, rows = ids.long()[live], dout.double()[live]
    total = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, at, rows) * scale
    size = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, at, rows.abs()) * scale
    count = torch.bincount(at, minlength=vocab)[:, None].double()
    old = torch.randn(vocab, dim, generator=gen).to(dtype).cuda()
    for accumulate in (False, True):
        dtable, check = ou.flat_view(vocab * dim, (vocab, dim), dtype, off)
        got = []
        for _ in range(2):
            dtable.copy_(old)
            ws.fill_(0xA5)
            dp.dp_embedding_grad(dtable, dout, ids, scale=scale, pad_id=pad, accumulate=accumulate, ws=ws)
            got.append(dtable.clone())
        assert torch.equal(got[0], got[1]), "not the same run to run"
        want = total + old.double() if accumulate else total
        # count - 1 additions, the scale and (added) one more addition
        ou.close(got[0], want, ou.EPS * ((count + 1) * size + want.abs()), "gradient, accumulate=%s" % accumulate)
        untouched = count[:, 0] == 0
        assert torch.equal(got[0][untouched], old[untouched] if accumulate else torch.zeros_like(old[untouched]))
        check()


def test_no_tokens(dev):
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    dout = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda")
    table = torch.ones(11, 24, dtype=torch.bfloat16, device="cuda")
    dp.dp_embedding_grad(table, dout, ids, accumulate=True)
    assert bool((table == 1).all())
    dp.dp_embedding_grad(table, dout, ids)
    assert bool((table == 0).all())


def test_gradient_on_another_stream(dev):
    gen = torch.Generator().manual_seed(4)
    ids = make_ids("uniform", 4000, 500, torch.int64, gen)
    dout = torch.randn(4000, 64, generator=gen).bfloat16().cuda()
    ws = torch.empty(dp.dp_embedding_workspace_size(4000, 500, 64), dtype=torch.uint8, device="cuda")
    a, b = torch.empty(500, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(500, 64, dtype=torch.bfloat16, device="cuda")
    dp.dp_embedding_grad(a, dout, ids, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dp.dp_embedding_grad(b, dout, ids, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(a, b)


def test_non_finite_rows_stay_theirs(dev):
    """An infinity or a NaN in one token's gradient reaches its own row only."""
    ids = torch.tensor([4, 2, 4, 7, 2, 2], dtype=torch.int32, device="cuda")
    dout = torch.ones(6, 40, device="cuda")
    dout[2, 5], dout[3, 6] = float("inf"), float("nan")
    out = torch.empty(9, 40, device="cuda")
    ws = torch.empty(dp.dp_embedding_workspace_size(6, 9, 40), dtype=torch.uint8, device="cuda")
    dp.dp_embedding_grad(out, dout, ids, ws=ws)
    want = torch.zeros(9, 40, device="cuda").index_add_(0, ids.long(), dout)
    assert torch.equal(torch.nan_to_num(out, nan=-5.0), torch.nan_to_num(want, nan=-5.0))
