"""Helpers of the operators' tests: 64-bit references and error bounds.

Every bound is (rounding of the output) + (fp32 arithmetic): an output of type T may be off by one rounding to T, half
an ulp, and by the fp32 error of its sums, which is bounded by counting the roundings: a sum of m terms in any order
errs by at most m * EPS * (sum of the terms' magnitudes), EPS = 2^-24.
"""
import torch

EPS = 2.0 ** -24
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -23}   # half an ulp relative to the value, at worst (twice
#                                                                     the nominal 2^-9, 2^-24: values just above a power of two)


def close(got, want, err32, what=""):
    """got (fp32 or bf16) within half an ulp of want +- err32, elementwise; NaN and infinities in the same places."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    g, w = got.double(), want.double()
    err = torch.as_tensor(err32, dtype=torch.float64, device=w.device).expand_as(w)
    fine = torch.isfinite(w)
    assert torch.equal(torch.isfinite(g), fine), what + ": non-finite values differ"
    assert torch.equal(torch.isnan(g), torch.isnan(w)), what + ": NaNs differ"
    off = (g - w).abs()[fine]
    may = ((w.abs() + err) * HALF_ULP[got.dtype] + err)[fine] + 1e-45
    bad = off > may
    assert not bad.any(), "%s: %d of %d beyond the bound, worst %.3g times" % (
        what, int(bad.sum()), off.numel(), float((off / may).max()))


def flat_view(numel, shape, dtype, offset, device="cuda"):
    """A tensor that begins `offset` elements into a larger buffer filled with a mark; returns (view, check)."""
    mark = 7.0
    buf = torch.full((offset + numel + 64,), mark, dtype=dtype, device=device)
    view = buf[offset:offset + numel].view(shape)

    def check():
        assert bool((buf[:offset] == mark).all()) and bool((buf[offset + numel:] == mark).all()), "written outside"
    return view, check


def decode64(codes, scales, dim):
    """What an 8-bit checkpoint stands for."""
    e = scales.double().repeat_interleave(32, 1)
    v = codes.double() * torch.exp2(e - 127)
    return torch.where(e == 255, torch.full_like(v, float("nan")), v)[:, :dim]


def act64(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    c = (2.0 / torch.pi) ** 0.5
    return g * torch.sigmoid(2 * c * (g + 0.044715 * g ** 3))   # (1 + tanh y) / 2 = s(2 y), without its cancellation


def norm64(v, w, b, stats):
    """The norm with given (mean, rstd)."""
    h = (v - stats[:, :1]) * stats[:, 1:]
    n = h if w is None else h * w
    return h, (n if b is None else n + b)


def stats64(v, layer, eps):
    mean = v.mean(1, keepdim=True) if layer else torch.zeros(v.shape[0], 1, dtype=v.dtype, device=v.device)
    return torch.cat([mean, ((v - mean) ** 2).mean(1, keepdim=True).add(eps).rsqrt()], 1)


def gate64(s, gate):
    if s["gate"] is None:
        return 1.0
    return s["gate"].double() if gate == "channel" else s["gate"].double()[:, None]


def norm_grad64(s, gate, layer, a, b, ps, qs, post=True, pre=True):
    """The gradient's formulas in 64 bits, with the magnitudes that its sums run over."""
    dim = s["r"].shape[1] if s.get("r") is not None else s["y"].shape[1]
    out, mag = {}, {}
    D = torch.zeros(s["dx_shape"], dtype=torch.float64, device=s["w_pre"].device) if s["dr"] is None else s["dr"].double()
    eD = D.abs() * 2
    if pre:
        rh = (s["r"].double() - qs[:, :1]) * qs[:, 1:]
        rm = (s["r"].double().abs() + qs[:, :1].abs()) * qs[:, 1:]
        dz = s["dz"].double()
        v = dz * s["w_pre"].double()
        c1 = (v * rh).mean(1, keepdim=True)
        c0 = v.mean(1, keepdim=True) if layer else 0.0
        D = D + qs[:, 1:] * (v - rh * c1 - c0)
        m1 = (v.abs() * rm).mean(1, keepdim=True)
        m0 = v.abs().mean(1, keepdim=True)
        eD = eD + qs[:, 1:] * (v.abs() + rm * m1 * 2 + m0)
        out["dw_pre"], out["db_pre"] = (dz * rh).sum(0), dz.sum(0)
        mag["dw_pre"], mag["db_pre"] = (dz.abs() * rm).sum(0), dz.abs().sum(0)
    out["dx"], mag["dx"] = a * D, eD * a
    if s["y"] is not None:
        y = s["y"].double()
        yh = (y - ps[:, :1]) * ps[:, 1:] if post else y
        ym = (y.abs() + ps[:, :1].abs()) * ps[:, 1:] if post else y.abs()
        w = s["w_post"].double() if post else torch.ones(dim, dtype=torch.float64, device=s["w_pre"].device)
        c = s["b_post"].double() if post and s["b_post"] is not None else torch.zeros_like(w)
        g = gate64(s, gate)
        ga = torch.as_tensor(g).abs()
        v = b * g * w * D
        ev = b * ga * w.abs() * eD
        if post:
            out["dy"] = ps[:, 1:] * (v - yh * (v * yh).mean(1, keepdim=True) - (v.mean(1, keepdim=True) if layer else 0.0))
            mag["dy"] = ps[:, 1:] * (ev + 2 * ym * (ev * ym).mean(1, keepdim=True) + ev.mean(1, keepdim=True))
        else:
            out["dy"], mag["dy"] = v, ev
        out["dw_post"], mag["dw_post"] = (b * g * D * yh).sum(0), (b * ga * eD * ym).sum(0)
        out["db_post"], mag["db_post"] = (b * g * D).sum(0) * torch.ones_like(w), (b * ga * eD).sum(0) * torch.ones_like(w)
        axis = 0 if gate == "channel" else 1
        out["dgate"], mag["dgate"] = (b * D * (yh * w + c)).sum(axis), (b * eD * (ym * w.abs() + c.abs())).sum(axis)
    return out, mag
