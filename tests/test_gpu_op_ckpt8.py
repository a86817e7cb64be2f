"""8-bit activation checkpoints, the gated activation and the weight gradient on the GPU against 64 bits (-m gpu)."""
import pytest
import torch

import op_util as ou
import zero_gradient_sync_gb300 as dp

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def encode64(x):
    """Codes and bytes from the format's definition: the least step that does, found by trying them from below."""
    rows, dim = x.shape
    pitch = dp.dp_ckpt8_pitch(dim)
    g = torch.zeros(rows, pitch, dtype=torch.float64, device=x.device)
    g[:, :dim] = x.double()
    g = g.view(rows, pitch // 32, 32)
    bad = ~torch.isfinite(g).all(2)
    g = torch.where(bad[:, :, None], torch.zeros_like(g), g)
    top = g.abs().amax(2)
    k = torch.full_like(top, -126)
    for _ in range(260):
        k = torch.where(top > 127 * torch.exp2(k), k + 1, k)
    codes = torch.round(g / torch.exp2(k)[:, :, None]).to(torch.int8)
    return codes.view(rows, pitch), torch.where(bad, 255, (k + 127).long()).to(torch.uint8)


def fresh(rows, dim):
    c, s = dp.new_ckpt8(rows, dim)
    return c.fill_(99), s.fill_(99)


def values(rows, dim, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, dim, generator=gen) * torch.exp(3 * torch.randn(rows, 1, generator=gen))
    x[:, ::17] *= 30
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,dim,ld,off", [(0, 8, 8, 0), (1, 1, 1, 0), (3, 31, 31, 0), (2, 32, 32, 0), (5, 33, 33, 0), (7, 1111, 1111, 0),
                                             (64, 768, 768, 0), (3, 40, 48, 8), (3, 40, 41, 3), (1, 11008, 11008, 0), (300, 72, 72, 0)])
def test_round_trip(dev, dtype, rows, dim, ld, off):
    full, _ = ou.flat_view(rows * ld, (rows, ld), dtype, off)
    full.copy_(values(rows, ld, dtype, rows + dim))
    x = full[:, :dim]
    codes, scales = fresh(rows, dim)
    dp.dp_ckpt8_encode(codes, scales, x)
    c64, s64 = encode64(x)
    assert torch.equal(codes, c64) and torch.equal(scales, s64)
    back_full, check = ou.flat_view(rows * ld, (rows, ld), dtype, off)
    kept = back_full.clone()
    dp.dp_ckpt8_decode(back_full[:, :dim], codes, scales)
    assert torch.equal(back_full[:, :dim].double(), ou.decode64(codes, scales, dim))   # exact in both types
    assert torch.equal(back_full[:, dim:], kept[:, dim:])
    check()


def test_extreme_groups(dev):
    x = torch.zeros(1, 32 * 12, device="cuda")
    x[0, 32:64] = 1e-40                       # subnormal
    x[0, 64] = float("inf")
    x[0, 97] = float("nan")
    x[0, 128:160] = 3.3e38
    x[0, 160:192] = torch.linspace(-1, 1, 32)
    x[0, 192] = 127.0                         # a code of 127 with step 1
    x[0, 224] = 127.0000076                   # the next fp32: step 2
    x[0, 256:258] = torch.tensor([127.0, 2.5])   # ties to even
    x[0, 288] = -float("inf")
    x[0, 320] = 2.0 ** -126
    codes, scales = fresh(1, x.shape[1])
    dp.dp_ckpt8_encode(codes, scales, x)
    c64, s64 = encode64(x)
    assert torch.equal(codes, c64) and torch.equal(scales, s64)
    assert scales[0, 6] == 127 and scales[0, 7] == 128 and int(codes[0, 257]) == 2
    assert [int(scales[0, g]) for g in (2, 3, 9)] == [255, 255, 255]
    back = torch.empty_like(x)
    dp.dp_ckpt8_decode(back, codes, scales)
    nan = torch.isnan(back[0]).view(12, 32)
    assert nan[[2, 3, 9]].all() and not nan[[0, 1, 4, 5, 6, 7, 8, 10, 11]].any()
    b16 = torch.empty(1, x.shape[1], dtype=BF, device="cuda")
    dp.dp_ckpt8_decode(b16, codes, scales)
    assert torch.equal(torch.nan_to_num(b16.float(), nan=5.0), torch.nan_to_num(back, nan=5.0))


def act_err(g, kind):
    """Bound of the fp32 error of f and f', relative to |f| + s (1 + |g|): 2 + 1.2 |v| ulp of the fast exponential at
    argument v (and v's own rounding, |v| 2^-23), 2 of the quotient, and a few products."""
    v = g.abs() if kind == "silu" else 2 * 0.8 * g.abs() * (1 + 0.0448 * g * g)
    return 2.0 ** -23 * (12 + 4 * v.clamp(max=100.0))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("rows,dim,halves", [(0, 8, False), (1, 1, False), (3, 33, False), (65, 264, True), (5, 1111, True), (17, 2048, True)])
def test_activation(dev, kind, gated, rows, dim, halves):
    act = dp.DP_ACT_SILU if kind == "silu" else dp.DP_ACT_GELU
    gen = torch.Generator().manual_seed(rows + dim)
    both = (torch.randn(rows, 2 * dim, generator=gen) * 3).bfloat16().cuda()
    if rows:
        both[0, 0], both[rows - 1, dim - 1] = -60.0, 45.0
    g = both[:, :dim] if halves else both[:, :dim].contiguous()
    u = (both[:, dim:] if halves else both[:, dim:].contiguous()) if gated else None
    h = torch.empty(rows, dim, dtype=BF, device="cuda")
    g8 = fresh(rows, dim)
    u8 = fresh(rows, dim) if gated else None
    dp.dp_act_ckpt8(h, g, u, act=act, g8=g8, u8=u8)
    for t, c in ((g, g8), (u, u8)):
        if t is not None:
            c64, s64 = encode64(t)
            assert torch.equal(c[0], c64) and torch.equal(c[1], s64)
    g64 = g.double()
    f = ou.act64(g64, kind)
    mul = u.double() if gated else torch.ones_like(f)
    ou.close(h, f * mul, act_err(g64, kind) * f.abs() * mul.abs() + 1e-37, "h")
    # the gradient, from what the checkpoints stand for
    dh = torch.randn(rows, dim, generator=gen).bfloat16().cuda()
    wide = torch.full((rows, 2 * dim), 7.0, dtype=BF, device="cuda")
    dg = wide[:, :dim] if halves else torch.empty(rows, dim, dtype=BF, device="cuda")
    du = (wide[:, dim:] if halves else torch.empty(rows, dim, dtype=BF, device="cuda")) if gated else None
    again = torch.empty(rows, dim, dtype=BF, device="cuda")
    dp.dp_act_ckpt8_grad(dg, du, dh, act=act, g8=g8, u8=u8, h=again)
    gv = ou.decode64(*g8, dim).requires_grad_()
    uv = ou.decode64(*u8, dim).requires_grad_() if gated else None
    f = ou.act64(gv, kind)
    hv = f * uv if gated else f
    want = torch.autograd.grad(hv, [gv] + ([uv] if gated else []), dh.double())
    gd, d = gv.detach(), dh.double().abs()
    m = uv.detach().abs() if gated else torch.ones_like(d)
    err = act_err(gd, kind)
    s = torch.sigmoid(gd if kind == "silu" else 1.6 * gd * (1 + 0.0447 * gd * gd))
    slope = 1 + gd.abs() if kind == "silu" else 1 + gd.abs() * (1 + 0.14 * gd * gd)
    ou.close(dg, want[0], err * d * m * s * slope + 1e-37, "dg")
    if gated:
        ou.close(du, want[1], err * d * f.detach().abs() + 1e-37, "du")
    ou.close(again, hv.detach(), err * hv.detach().abs() + 1e-37, "h again")
    # without h, and with h over dh
    dg2 = torch.empty(rows, dim, dtype=BF, device="cuda")
    du2 = torch.empty_like(dg2) if gated else None
    dp.dp_act_ckpt8_grad(dg2, du2, dh, act=act, g8=g8, u8=u8, h=dh)
    assert torch.equal(dg2, dg) and torch.equal(dh, again)
    if halves and not gated:
        assert bool((wide[:, dim:] == 7).all())


def test_overflow_reaches_the_gradients(dev):
    g = torch.randn(4, 64, device="cuda").bfloat16()
    g[2, 40] = float("inf")
    h, g8 = torch.empty_like(g), dp.new_ckpt8(4, 64)
    dp.dp_act_ckpt8(h, g, act=dp.DP_ACT_SILU, g8=g8)
    dg = torch.empty_like(g)
    dp.dp_act_ckpt8_grad(dg, None, torch.ones_like(g), act=dp.DP_ACT_SILU, g8=g8)
    nan = torch.isnan(dg)
    assert nan[2, 32:].all() and int(nan.sum()) == 32
    dy = torch.randn(4, 16, device="cuda").bfloat16()
    dw = torch.empty(16, 64, device="cuda")
    dp.dp_wgrad8(dw, dy, *g8, ws=torch.empty(dp.dp_wgrad8_workspace_size(4, 16, 64), dtype=torch.uint8, device="cuda"))
    assert torch.isnan(dw[:, 32:]).all() and torch.isfinite(dw[:, :32]).all()


@pytest.mark.parametrize("rows,n,k,ldx,off", [(1, 1, 1, 0, 0), (1, 64, 64, 0, 0), (3, 8, 40, 0, 0), (64, 256, 256, 0, 0), (65, 264, 300, 0, 0),
                                              (200, 130, 31, 0, 0), (513, 77, 500, 0, 1), (1000, 520, 264, 8, 0), (700, 256, 512, 3, 0),
                                              (5000, 128, 96, 0, 0), (1537, 2304, 768, 0, 0), (96, 4000, 2600, 0, 0)])
@pytest.mark.parametrize("dtype,accumulate", [(F32, False), (BF, True)])
def test_weight_gradient(dev, rows, n, k, ldx, off, dtype, accumulate):
    gen = torch.Generator().manual_seed(rows + n + k)
    x = values(rows, k, BF, rows)
    codes, scales = fresh(rows, k)
    dp.dp_ckpt8_encode(codes, scales, x)
    full = torch.randn(rows, n + ldx, generator=gen).bfloat16().cuda()
    dy = full[:, :n]
    old = torch.randn(n, k, generator=gen).to(dtype).cuda()
    dw, check = ou.flat_view(n * k, (n, k), dtype, off)
    need = dp.dp_wgrad8_workspace_size(rows, n, k, dy_aligned=ldx % 8 == 0)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(2):
        dw.copy_(old)
        dp.dp_wgrad8(dw, dy, codes, scales, alpha=0.5, accumulate=accumulate, ws=ws)
        got.append(dw.clone())
    assert torch.equal(got[0], got[1])
    x64 = ou.decode64(codes, scales, k)
    want = 0.5 * dy.double().t() @ x64
    size = 0.5 * dy.double().abs().t() @ x64.abs()
    if accumulate:
        want += old.double()
        size += old.double().abs()
    # rows additions and the alpha, truncated rather than rounded where the tensor cores add: 2 EPS each
    ou.close(got[0], want, (rows + 8) * 2 * ou.EPS * size, "dw")
    check()


def test_weight_gradient_of_no_rows(dev):
    dw = torch.ones(40, 64, device="cuda")
    dy = torch.empty(0, 40, dtype=BF, device="cuda")
    dp.dp_wgrad8(dw, dy, *dp.new_ckpt8(0, 64), accumulate=True)
    assert bool((dw == 1).all())
    dp.dp_wgrad8(dw, dy, *dp.new_ckpt8(0, 64))
    assert bool((dw == 0).all())
