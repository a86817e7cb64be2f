"""Tensors of more than 2^31 elements: the last rows of a long call equal, bit for bit, those of a short call on them (-m gpu)."""
import pytest
import torch

import zero_gradient_sync_gb300 as dp

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def big(rows, dim, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(rows, dim, dtype=BF, device="cuda")
    part = torch.randn(4096, dim, generator=gen, device="cuda", dtype=BF)
    for r in range(0, rows, 4096):
        x[r:r + 4096] = part[:min(4096, rows - r)]
        part = part.roll(1, 0)
    return x


@pytest.mark.parametrize("dim", [16384, 16383])
def test_norm_rows_beyond_32_bits(dev, dim):
    rows, last = (1 << 31) // dim + 300, 5
    y, x = big(rows, dim, 1), big(rows, dim, 2)
    w = torch.linspace(0.5, 1.5, dim, device="cuda").to(BF)
    r, z = torch.empty_like(x), torch.empty_like(x)
    ps, qs = torch.empty(rows, 2, device="cuda"), torch.empty(rows, 2, device="cuda")
    dp.dp_block_norm(r, z, x, y, w_post=w, w_pre=w, post_stats=ps, pre_stats=qs)
    tail = [t[-last:].clone() for t in (x, y)]
    r2, z2 = torch.empty_like(tail[0]), torch.empty_like(tail[0])
    dp.dp_block_norm(r2, z2, *tail, w_post=w, w_pre=w)
    assert torch.equal(r[-last:], r2) and torch.equal(z[-last:], z2)
    ws = torch.empty(dp.dp_block_norm_workspace_size(rows, dim), dtype=torch.uint8, device="cuda")
    dx, dy = torch.empty_like(x), z
    args = dict(w_post=w, w_pre=w)
    dp.dp_block_norm_grad(dx, dy, None, x, r, y, post_stats=ps, pre_stats=qs, ws=ws, **args)
    dx2, dy2 = torch.empty_like(r2), torch.empty_like(r2)
    dp.dp_block_norm_grad(dx2, dy2, None, tail[0], r2, tail[1], post_stats=ps[-last:].clone(), pre_stats=qs[-last:].clone(), ws=ws, **args)
    assert torch.equal(dx[-last:], dx2) and torch.equal(dy[-last:], dy2)


@pytest.mark.parametrize("dim", [8192, 8191])
def test_checkpoints_beyond_32_bits(dev, dim):
    rows, last = (1 << 31) // dim + 300, 7
    g = big(rows, dim, 3)
    g8, h, dg = dp.new_ckpt8(rows, dim), torch.empty_like(g), torch.empty_like(g)
    dp.dp_act_ckpt8(h, g, act=dp.DP_ACT_GELU, g8=g8)
    tail = g[-last:].clone()
    t8, h2, dg2, back = dp.new_ckpt8(last, dim), torch.empty_like(tail), torch.empty_like(tail), torch.empty_like(tail)
    dp.dp_act_ckpt8(h2, tail, act=dp.DP_ACT_GELU, g8=t8)
    assert torch.equal(h[-last:], h2) and torch.equal(g8[0][-last:], t8[0]) and torch.equal(g8[1][-last:], t8[1])
    dp.dp_act_ckpt8_grad(dg, None, g, act=dp.DP_ACT_GELU, g8=g8)
    dp.dp_act_ckpt8_grad(dg2, None, tail, act=dp.DP_ACT_GELU, g8=t8)
    assert torch.equal(dg[-last:], dg2)
    dp.dp_ckpt8_decode(h, *g8)
    dp.dp_ckpt8_decode(back, *t8)
    assert torch.equal(h[-last:], back)


def test_embedding_beyond_32_bits(dev):
    """A table of more than 2^31 elements, looked up and added to at its end."""
    dim = 4096
    vocab = (1 << 31) // dim + 100
    table = big(vocab, dim, 4)
    ids = torch.tensor([vocab - 1, 0, vocab - 3, vocab - 1, vocab - 1], device="cuda")
    out = torch.empty(5, dim, dtype=BF, device="cuda")
    dp.dp_embedding(out, table, ids)
    assert torch.equal(out, table[ids])
    ws = torch.empty(dp.dp_embedding_workspace_size(5, vocab, dim), dtype=torch.uint8, device="cuda")
    want = table[-4:].float()
    want[3] += out.float()[[0, 3, 4]].sum(0)
    want[1] += out.float()[2]
    dp.dp_embedding_grad(table, out, ids, accumulate=True, ws=ws)
    assert torch.allclose(table[-4:].float(), want, rtol=2.0 ** -8, atol=0)     # one rounding to bf16
    dp.dp_embedding_grad(table, out, ids, ws=ws)
    assert bool((table[-4] == 0).all()) and bool((table[1000:1010] == 0).all())
    assert torch.equal(table[-3], out[2])


def test_weight_gradient_beyond_32_bits(dev):
    """dy of more than 2^31 elements whose first rows are zeros: the rest gives the gradient."""
    n, k, last = 2048, 64, 256
    rows = (1 << 31) // n + 1024
    dy = torch.zeros(rows, n, dtype=BF, device="cuda")
    dy[-last:] = big(last, n, 5)
    x = big(rows, k, 6)
    c = dp.new_ckpt8(rows, k)
    dp.dp_ckpt8_encode(*c, x)
    dw, dw2 = torch.empty(n, k, device="cuda"), torch.empty(n, k, device="cuda")
    ws = torch.empty(max(dp.dp_wgrad8_workspace_size(rows, n, k), dp.dp_wgrad8_workspace_size(last, n, k)), dtype=torch.uint8, device="cuda")
    dp.dp_wgrad8(dw, dy, *c, ws=ws)
    dp.dp_wgrad8(dw2, dy[-last:].clone(), c[0][-last:].clone(), c[1][-last:].clone(), ws=ws)
    # the same 256 products a value, added in other groups: at most 256 roundings of their magnitudes' sum
    size = dy[-last:].double().abs().t() @ x[-last:].double().abs()
    assert bool(((dw - dw2).double().abs() <= 2 * 264 * 2.0 ** -23 * size).all())
