"""The norms around a block and their gradient on the GPU against 64 bits (-m gpu)."""
import pytest
import torch

import op_util as ou
import zero_gradient_sync_gb300 as dp

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
K = 64   # fp32 roundings on the way to one value: a thread's <= 32 sequential terms, the tree over the row, a few products


def build(rows, dim, layer, gate, ts, tb, tp, off, seed=0, mean=0.3):
    gen = torch.Generator().manual_seed(rows * 31 + dim + seed)
    checks = []

    def mk(shape, dtype, std=1.0, add=0.0):
        n = 1
        for s in shape:
            n *= s
        t, check = ou.flat_view(n, shape, dtype, off)
        t.copy_(torch.randn(shape, generator=gen) * std + add)
        checks.append(check)
        return t
    s = {"x": mk((rows, dim), ts), "y": mk((rows, dim), tb, 2.0, mean), "r": mk((rows, dim), ts, 1.5, mean),
         "dr": mk((rows, dim), ts), "dz": mk((rows, dim), tb), "w_post": mk((dim,), tp, 0.2, 1.0),
         "w_pre": mk((dim,), tp, 0.2, 1.0), "b_post": mk((dim,), tp, 0.3) if layer else None,
         "b_pre": mk((dim,), tp, 0.3) if layer else None,
         "gate": None if gate == "none" else mk((dim,) if gate == "channel" else (rows,), tp, 0.5, 0.5)}
    return s, mk, checks


def d64(t):
    return None if t is None else t.double()


SHAPES = [(1, 1, 0), (5, 8, 0), (3, 77, 0), (7, 768, 0), (130, 264, 8), (9, 2048, 1), (33, 4096, 0), (3, 5000, 0), (2, 11008, 0),
          (2, 16384, 0), (2, 16383, 0), (37, 60, 1), (21, 128, 0), (50, 100, 3), (19, 24, 0)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("rows,dim,off", SHAPES)
def test_forward(dev, kind, gate, rows, dim, off):
    layer = kind == "layer"
    for ts, tb, tp in ((BF, BF, BF), (F32, BF, F32), (F32, F32, BF)):
        s, mk, checks = build(rows, dim, layer, gate, ts, tb, tp, off)
        r, z = mk((rows, dim), ts), mk((rows, dim), tb)
        post, pre = torch.empty(rows, 2, device="cuda"), torch.empty(rows, 2, device="cuda")
        a, b = 0.75, 1.25   # exact in fp32
        dp.dp_block_norm(r, z, s["x"], s["y"], w_post=s["w_post"], b_post=s["b_post"], gate=s["gate"],
                         gate_per_token=gate == "token", w_pre=s["w_pre"], b_pre=s["b_pre"],
                         kind=dp.DP_NORM_LAYER if layer else dp.DP_NORM_RMS, eps=2.0 ** -16, res_scale=a, branch_scale=b,
                         post_stats=post, pre_stats=pre)
        y, x = s["y"].double(), s["x"].double()
        ps = ou.stats64(y, layer, 2.0 ** -16)
        h, n = ou.norm64(y, d64(s["w_post"]), d64(s["b_post"]), ps)
        want = a * x + b * ou.gate64(s, gate) * n
        # errors of the mean (against the row's mean magnitude) and of rstd (relative) reach every element
        spread = y.abs().mean(1, keepdim=True) * ps[:, 1:] + h.abs()
        en = K * ou.EPS * (spread * s["w_post"].double().abs() + n.abs())
        er = en * b * torch.as_tensor(ou.gate64(s, gate)).abs() + 4 * ou.EPS * (a * x.abs() + want.abs())
        ou.close(r, want, er, "r")
        sx = K * ou.EPS * (y.abs().mean(1) + 1e-30)
        ou.close(post[:, 0].contiguous(), ps[:, 0], sx, "post mean")
        # 1-column layer rows have no variance: rstd is 1 / sqrt(eps) up to the mean's own error squared
        ou.close(post[:, 1].contiguous(), ps[:, 1], ps[:, 1] * (K * ou.EPS + (sx * ps[:, 1]) ** 2 + 2 * sx * sx * ps[:, 1] ** 2), "post rstd")
        qs = ou.stats64(want, layer, 2.0 ** -16)
        hz, nz = ou.norm64(want, d64(s["w_pre"]), d64(s["b_pre"]), qs)
        # z sees r's error directly, through the mean and through rstd
        e1 = (er + er.mean(1, keepdim=True)) * qs[:, 1:] + hz.abs() * (er * hz.abs()).mean(1, keepdim=True) * qs[:, 1:]
        sp = want.abs().mean(1, keepdim=True) * qs[:, 1:] + hz.abs()
        ez = (2 * e1 + K * ou.EPS * sp) * s["w_pre"].double().abs() + K * ou.EPS * nz.abs()
        ou.close(z, nz, ez, "z")
        for c in checks:
            c()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("rows,dim,off", SHAPES + [(1300, 64, 0)])
def test_gradient(dev, kind, gate, rows, dim, off):
    layer = kind == "layer"
    a, b = 0.75, 1.25
    for (ts, tb, tp), accumulate in (((BF, BF, BF), False), ((F32, BF, F32), True), ((F32, F32, BF), False)):
        s, mk, checks = build(rows, dim, layer, gate, ts, tb, tp, off)
        ps32 = ou.stats64(s["y"].double(), layer, 1e-5).float()
        qs32 = ou.stats64(s["r"].double(), layer, 1e-5).float()
        dx, dy = mk((rows, dim), ts), mk((rows, dim), tb)
        names = ["dw_post", "dw_pre"] + (["db_post", "db_pre"] if layer else []) + (["dgate"] if gate != "none" else [])
        grads = {k: mk((rows,) if k == "dgate" and gate == "token" else (dim,), tp) for k in names}
        old = {k: v.clone() for k, v in grads.items()}
        ws = torch.empty(dp.dp_block_norm_workspace_size(rows, dim), dtype=torch.uint8, device="cuda").fill_(0xFF)
        dp.dp_block_norm_grad(dx, dy, s["dr"], s["dz"], s["r"], s["y"], w_post=s["w_post"], b_post=s["b_post"], gate=s["gate"],
                              gate_per_token=gate == "token", w_pre=s["w_pre"],
                              kind=dp.DP_NORM_LAYER if layer else dp.DP_NORM_RMS, res_scale=a, branch_scale=b,
                              post_stats=ps32, pre_stats=qs32, accumulate=accumulate, ws=ws, **grads)
        want, mag = ou.norm_grad64(s, gate, layer, a, b, ps32.double(), qs32.double())
        ou.close(dx, want["dx"], K * ou.EPS * mag["dx"], "dx")
        ou.close(dy, want["dy"], K * ou.EPS * mag["dy"], "dy")
        for k in names:
            w = want[k] + old[k].double() if accumulate else want[k]
            # summed over rows (or over a row's dim values): at most that many roundings more
            n = (dim if k == "dgate" and gate == "token" else rows) + K
            ou.close(grads[k], w, n * ou.EPS * (mag[k] + w.abs()), k)
        for c in checks:
            c()


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_parts_left_out(dev, kind):
    """No post norm; no norm before the next block; no block yet; no gradient from the stream; in-place outputs."""
    layer, rows, dim = kind == "layer", 19, 520
    code = dp.DP_NORM_LAYER if layer else dp.DP_NORM_RMS
    s, mk, _ = build(rows, dim, layer, "channel", BF, BF, BF, 0)
    s["dx_shape"] = (rows, dim)
    qs = ou.stats64(s["r"].double(), layer, 1e-5).float()
    ws = torch.empty(dp.dp_block_norm_workspace_size(rows, dim), dtype=torch.uint8, device="cuda")
    # y straight into the stream through the gate; no z
    r = mk((rows, dim), BF)
    dp.dp_block_norm(r, None, s["x"], s["y"], gate=s["gate"], post=False, pre=False, kind=code)
    ou.close(r, s["x"].double() + s["gate"].double() * s["y"].double(), 4 * ou.EPS * (s["x"].double().abs() + (s["gate"].double() * s["y"].double()).abs()), "r")
    dx, dy, dgate = mk((rows, dim), BF), mk((rows, dim), BF), mk((dim,), BF)
    dp.dp_block_norm_grad(dx, dy, s["dr"], None, s["r"], s["y"], gate=s["gate"], post=False, pre=False, kind=code, dgate=dgate, ws=ws)
    want, mag = ou.norm_grad64(s, "channel", layer, 1.0, 1.0, None, None, post=False, pre=False)
    for k, t in (("dx", dx), ("dy", dy), ("dgate", dgate)):
        ou.close(t, want[k], (rows + K) * ou.EPS * mag[k], k)
    # only the norm before the first block: z = N(x); r is x
    z, stats = mk((rows, dim), BF), torch.empty(rows, 2, device="cuda")
    dp.dp_block_norm(None, z, s["x"], w_pre=s["w_pre"], b_pre=s["b_pre"], kind=code, pre_stats=stats)
    xs = ou.stats64(s["x"].double(), layer, 1e-5)
    h, n = ou.norm64(s["x"].double(), d64(s["w_pre"]), d64(s["b_pre"]), xs)
    ou.close(z, n, K * ou.EPS * (1 + h.abs()) * 2 * s["w_pre"].double().abs() + K * ou.EPS * n.abs(), "z")
    q = dict(s, y=None, dr=None)
    want, mag = ou.norm_grad64(q, "none", layer, 1.0, 1.0, None, qs.double())
    dw = mk((dim,), BF)
    dp.dp_block_norm_grad(dx, None, None, s["dz"], s["r"], w_pre=s["w_pre"], kind=code, pre_stats=qs, dw_pre=dw, ws=ws)
    ou.close(dx, want["dx"], K * ou.EPS * mag["dx"], "dx")
    ou.close(dw, want["dw_pre"], (rows + K) * ou.EPS * mag["dw_pre"], "dw_pre")
    # in place: dx over dr, dy over dz; the forward's r over x
    dr, dz = s["dr"].clone(), s["dz"].clone()
    args = dict(w_post=s["w_post"], b_post=s["b_post"], gate=s["gate"], w_pre=s["w_pre"], kind=code,
                post_stats=ou.stats64(s["y"].double(), layer, 1e-5).float(), pre_stats=qs, ws=ws)
    dp.dp_block_norm_grad(dx, dy, s["dr"], s["dz"], s["r"], s["y"], **args)
    dp.dp_block_norm_grad(dr, dz, dr, dz, s["r"], s["y"], **args)
    assert torch.equal(dr, dx) and torch.equal(dz, dy)
    x = s["x"].clone()
    fw = dict(w_post=s["w_post"], b_post=s["b_post"], w_pre=s["w_pre"], b_pre=s["b_pre"], kind=code)
    z2 = torch.empty_like(z)
    dp.dp_block_norm(r, z, s["x"], s["y"], **fw)
    dp.dp_block_norm(x, z2, x, s["y"], **fw)
    assert torch.equal(x, r) and torch.equal(z, z2)


def test_no_rows_and_weightless(dev):
    e = torch.empty(0, 24, dtype=BF, device="cuda")
    w = torch.ones(24, dtype=BF, device="cuda")
    st = torch.empty(0, 2, device="cuda")
    dp.dp_block_norm(e, e.clone(), e.clone(), e.clone(), w_post=w, w_pre=w, post_stats=st, pre_stats=st)
    dw, dv = torch.full_like(w, 3.0), torch.full_like(w, 3.0)
    dp.dp_block_norm_grad(e, e.clone(), None, e.clone(), e.clone(), e.clone(), w_post=w, w_pre=w, post_stats=st, pre_stats=st, dw_post=dw, accumulate=True)
    assert bool((dw == 3).all())
    dp.dp_block_norm_grad(e, e.clone(), None, e.clone(), e.clone(), e.clone(), w_post=w, w_pre=w, post_stats=st, pre_stats=st, dw_post=dw, dw_pre=dv)
    assert bool((dw == 0).all()) and bool((dv == 0).all())
    # weights left out are ones
    x, y = torch.randn(6, 40, device="cuda"), torch.randn(6, 40, device="cuda")
    got = [[torch.empty_like(x), torch.empty_like(x)] for _ in range(2)]
    one = torch.ones(40, device="cuda")
    dp.dp_block_norm(*got[0], x, y)
    dp.dp_block_norm(*got[1], x, y, w_post=one, b_post=0 * one, w_pre=one, b_pre=0 * one)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_zero_and_non_finite_rows(dev):
    """A row of zeros has a finite norm; a NaN or an infinity stays in its row."""
    x = torch.randn(5, 96, device="cuda")
    x[1] = 0.0
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    z = torch.empty_like(x)
    dp.dp_block_norm(None, z, x)
    assert bool((z[1] == 0).all()) and bool(torch.isfinite(z[[0, 4]]).all())
    assert bool(torch.isnan(z[2]).all()) and not bool(torch.isfinite(z[3]).all())
