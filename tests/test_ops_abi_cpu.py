"""The operators' C ABI on the CPU: the library exports what dpops.h declares, the size queries answer, and every bad argument
is refused before anything is launched (no GPU is touched)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dpops.h")
FAKE = 1 << 20        # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def dp():
    import importlib.util
    spec = importlib.util.spec_from_file_location(
        "_dpstep_build", os.path.join(ROOT, "zero_gradient_sync_gb300", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    b.build()
    import zero_gradient_sync_gb300 as z
    return z


def declared():
    text = re.sub(r"/\*.*?\*/", " ", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(dp_[a-z0-9_]+)\s*\(", text)))


def test_exports_and_binding(dp):
    names = declared()
    assert len(names) == 13
    lib = ctypes.CDLL(dp.LIB_PATH)
    assert not [n for n in names if not hasattr(lib, n)]
    assert not [n for n in names if not hasattr(dp, n)]
    assert ctypes.sizeof(dp.dp_block_norm_t) == 56


def test_sizes(dp):
    assert [dp.dp_ckpt8_pitch(d) for d in (1, 31, 32, 33, 4096)] == [32, 32, 32, 64, 4096]
    assert dp.LIB.dp_ckpt8_pitch(0) == -1
    with pytest.raises(ValueError):
        dp.dp_ckpt8_pitch(0)
    assert dp.dp_embedding_workspace_size(1, 10, 8) > 0
    # sorted pairs and partial rows: a fraction of what the tokens' gradients take
    assert dp.dp_embedding_workspace_size(65536, 50257, 2048) < 65536 * 2048
    assert dp.dp_block_norm_workspace_size(10 ** 6, 4096) == dp.dp_block_norm_workspace_size(10 ** 7, 4096)
    # the decoded x, and a copy of dy only where its rows cannot be 16-byte aligned
    x = 1000 * 96 * 2
    assert dp.dp_wgrad8_workspace_size(1000, 64, 96) >= x
    assert dp.dp_wgrad8_workspace_size(1000, 63, 96) >= dp.dp_wgrad8_workspace_size(1000, 64, 96) + 1000 * 64 * 2
    assert dp.dp_wgrad8_workspace_size(1000, 64, 96, dy_aligned=False) == dp.dp_wgrad8_workspace_size(1000, 63, 96)
    for bad in ((-1, 10, 8), (1 << 31, 10, 8), (5, 0, 8), (5, 10, 0)):
        with pytest.raises(dp.DPError):
            dp.dp_embedding_workspace_size(*bad)
    for bad in ((-1, 8), (1, 0), (1, dp.DP_MAX_NORM_DIM + 1)):
        with pytest.raises(dp.DPError):
            dp.dp_block_norm_workspace_size(*bad)
    assert dp.LIB.dp_wgrad8_workspace_size(1, 0, 5, 1) == 0


def refused(dp, code, call, *args):
    before = dp.dp_kernel_launches()
    rc = call(*args)
    assert rc == code, (rc, dp.LIB.dp_last_error())
    assert dp.LIB.dp_last_error()
    assert dp.dp_kernel_launches() == before


def test_embedding_refusals(dp):
    ok = [FAKE, FAKE, FAKE, 4, 10, 8, 1.0, dp.DP_BF16, 32, None]
    for k, v in ((0, None), (1, None), (2, None), (3, -1), (3, 1 << 31), (4, 0), (5, 0), (7, 2), (8, 16)):
        refused(dp, dp.DP_ERR_INVALID_ARG, dp.LIB.dp_embedding, *(ok[:k] + [v] + ok[k + 1:]))
    for k, v in ((0, FAKE + 1), (1, FAKE + 1), (2, FAKE + 2)):
        refused(dp, dp.DP_ERR_ALIGNMENT, dp.LIB.dp_embedding, *(ok[:k] + [v] + ok[k + 1:]))
    ok = [FAKE, FAKE, FAKE, 4, 10, 8, 1.0, -1, 0, dp.DP_F32, 64, FAKE, None]
    for k, v in ((0, None), (1, None), (2, None), (3, -1), (4, 0), (5, 0), (8, 2), (9, -1), (10, 33), (11, None)):
        refused(dp, dp.DP_ERR_INVALID_ARG, dp.LIB.dp_embedding_grad, *(ok[:k] + [v] + ok[k + 1:]))
    for k, v in ((0, FAKE + 2), (1, FAKE + 2), (2, FAKE + 4), (11, FAKE + 16)):
        refused(dp, dp.DP_ERR_ALIGNMENT, dp.LIB.dp_embedding_grad, *(ok[:k] + [v] + ok[k + 1:]))


def test_block_norm_refusals(dp):
    T = dp.dp_block_norm_t
    base = dict(rows=4, dim=64, kind=0, norms=3, gate_mode=0, stream_dtype=0, block_dtype=0, param_dtype=0, accumulate=0, eps=1e-5,
                res_scale=1.0, branch_scale=1.0)

    def forward(code, ptr=None, **change):
        p = T(**{**base, **change})
        args = dict(r=FAKE, z=FAKE, x=FAKE, y=FAKE, w_post=None, b_post=None, gate=None, w_pre=None, b_pre=None, ps=None, qs=None)
        args.update(ptr or {})
        refused(dp, code, dp.LIB.dp_block_norm, ctypes.byref(p), *args.values(), None)
    bad, align = dp.DP_ERR_INVALID_ARG, dp.DP_ERR_ALIGNMENT
    for change in (dict(rows=-1), dict(dim=0), dict(dim=dp.DP_MAX_NORM_DIM + 1), dict(kind=2), dict(norms=4), dict(gate_mode=3),
                   dict(stream_dtype=2), dict(block_dtype=1), dict(param_dtype=-1), dict(accumulate=2), dict(eps=0.0),
                   dict(eps=float("nan")), dict(res_scale=float("inf")), dict(branch_scale=float("nan")), dict(gate_mode=1)):
        forward(bad, **change)
    for ptr in (dict(x=None), dict(r=None), dict(z=None), dict(y=None), dict(gate=FAKE)):
        forward(bad, ptr)
    forward(bad, dict(y=None, r=None), norms=2, res_scale=0.5)      # no block: nothing to scale
    forward(bad, dict(y=None), norms=2)                             # no block: r is x itself
    forward(bad, dict(z=None), norms=1, dim=0)
    forward(bad, norms=1)                                           # z without a norm for it
    for ptr in (dict(x=FAKE + 1), dict(w_pre=FAKE + 1), dict(ps=FAKE + 4)):
        forward(align, ptr)
    refused(dp, bad, dp.LIB.dp_block_norm, None, *[FAKE] * 11, None)

    def grad(code, ptr=None, **change):
        p = T(**{**base, **change})
        args = dict(dx=FAKE, dy=FAKE, dr=FAKE, dz=FAKE, r=FAKE, y=FAKE, w_post=None, b_post=None, gate=None, w_pre=None, ps=FAKE,
                    qs=FAKE, dw_post=None, db_post=None, dgate=None, dw_pre=None, db_pre=None, ws=FAKE)
        args.update(ptr or {})
        refused(dp, code, dp.LIB.dp_block_norm_grad, ctypes.byref(p), *args.values(), None)
    for ptr in (dict(dx=None), dict(dy=None), dict(dz=None), dict(r=None), dict(ps=None), dict(qs=None), dict(ws=None), dict(dgate=FAKE),
                dict(gate=FAKE)):
        grad(bad, ptr)
    grad(bad, dict(dw_post=FAKE), norms=2)
    grad(bad, dict(db_pre=FAKE), norms=1)
    for ptr in (dict(dr=FAKE + 1), dict(ws=FAKE + 128), dict(dw_pre=FAKE + 1)):
        grad(align, ptr)


def test_ckpt8_refusals(dp):
    bad, align = dp.DP_ERR_INVALID_ARG, dp.DP_ERR_ALIGNMENT
    ok = [FAKE, FAKE, FAKE, 4, 64, 64, dp.DP_BF16, None]
    for f in (dp.LIB.dp_ckpt8_encode, dp.LIB.dp_ckpt8_decode):
        for k, v in ((0, None), (1, None), (2, None), (3, -1), (4, 0), (5, 63), (6, 5)):
            refused(dp, bad, f, *(ok[:k] + [v] + ok[k + 1:]))
    refused(dp, align, dp.LIB.dp_ckpt8_encode, *([FAKE + 16] + ok[1:]))
    refused(dp, align, dp.LIB.dp_ckpt8_decode, *([FAKE + 1] + ok[1:]))
    refused(dp, align, dp.LIB.dp_ckpt8_decode, *([FAKE, FAKE + 16] + ok[2:]))
    ok = [FAKE] * 7 + [4, 64, 64, 64, 0, None]
    for k, v in ((0, None), (1, None), (3, None), (4, None), (5, None), (6, None), (2, None), (7, -1), (8, 0), (9, 63), (10, 63), (11, 2)):
        refused(dp, bad, dp.LIB.dp_act_ckpt8, *(ok[:k] + [v] + ok[k + 1:]))    # (k = 2: a checkpoint of u without u)
    ok = [FAKE] * 8 + [4, 64, 64, 64, 1, None]
    for k, v in ((0, None), (1, None), (3, None), (4, None), (5, None), (6, None), (7, None), (8, -1), (9, 0), (10, 63), (11, 63), (12, -1)):
        refused(dp, bad, dp.LIB.dp_act_ckpt8_grad, *(ok[:k] + [v] + ok[k + 1:]))


def test_wgrad8_refusals(dp):
    bad, align = dp.DP_ERR_INVALID_ARG, dp.DP_ERR_ALIGNMENT
    ok = [FAKE, FAKE, FAKE, FAKE, 4, 64, 64, 64, 1.0, 0, dp.DP_F32, FAKE, None]
    for k, v in ((0, None), (1, None), (2, None), (3, None), (4, -1), (5, 0), (6, 0), (7, 63), (8, float("nan")), (9, 2), (10, 2), (11, None)):
        refused(dp, bad, dp.LIB.dp_wgrad8, *(ok[:k] + [v] + ok[k + 1:]))
    for k, v in ((0, FAKE + 2), (1, FAKE + 1), (2, FAKE + 16), (11, FAKE + 16)):
        refused(dp, align, dp.LIB.dp_wgrad8, *(ok[:k] + [v] + ok[k + 1:]))


def test_binding_refuses_host_tensors(dp):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    codes, scales = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: dp.dp_embedding(x, x, ids), lambda: dp.dp_embedding_grad(x, x, ids), lambda: dp.dp_block_norm(x, x, x, x),
                 lambda: dp.dp_block_norm_grad(x, x, x, x, x, x), lambda: dp.dp_ckpt8_encode(codes, scales, x),
                 lambda: dp.dp_ckpt8_decode(x, codes, scales), lambda: dp.dp_act_ckpt8(x, x, g8=(codes, scales)),
                 lambda: dp.dp_act_ckpt8_grad(x, None, x, g8=(codes, scales)), lambda: dp.dp_wgrad8(x, x, codes, scales),
                 lambda: dp.dp_block_norm(None, x, x, w_pre=w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def _formulas(x, y, w_post, b_post, gate, w_pre, b_pre, layer, a, b, eps):
    import op_util as ou
    n = ou.norm64(y, w_post, b_post, ou.stats64(y, layer, eps))[1]
    r = a * x + b * gate * n
    return r, ou.norm64(r, w_pre, b_pre, ou.stats64(r, layer, eps))[1]


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("token", [False, True])
def test_gradient_formulas_against_differences(layer, token):
    """The formulas the kernels compute (and the GPU tests compare with) against central differences of the forward, in 64 bits."""
    import torch
    import op_util as ou
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    rows, dim, a, b, eps = 3, 7, 0.75, 1.25, 1e-3
    t = dict(x=rnd(rows, dim), y=rnd(rows, dim), w_post=rnd(dim), b_post=rnd(dim), gate=rnd(rows, 1) if token else rnd(dim), w_pre=rnd(dim),
             b_pre=rnd(dim))
    dr, dz = rnd(rows, dim), rnd(rows, dim)
    r, _ = _formulas(**t, layer=layer, a=a, b=b, eps=eps)
    got = ou.norm_grad64(dict(t, r=r, dr=dr, dz=dz, gate=t["gate"].reshape(-1)), "token" if token else "channel", layer, a, b,
                         ou.stats64(t["y"], layer, eps), ou.stats64(r, layer, eps))[0]
    names = {"x": "dx", "y": "dy", "w_post": "dw_post", "b_post": "db_post", "gate": "dgate", "w_pre": "dw_pre", "b_pre": "db_pre"}
    h = 1e-6
    for name, grad in names.items():
        for i in range(t[name].numel()):
            vals = []
            for sign in (1, -1):
                moved = {k: v.clone() for k, v in t.items()}
                moved[name].view(-1)[i] += sign * h
                r2, z2 = _formulas(**moved, layer=layer, a=a, b=b, eps=eps)
                vals.append(float((dr * r2).sum() + (dz * z2).sum()))
            # central differences: h^2 of the third derivative and 2^-52 / h of the function's value
            assert abs((vals[0] - vals[1]) / (2 * h) - float(got[grad].reshape(-1)[i])) < 1e-6 * (1 + abs(vals[0]) + abs(float(got[grad].reshape(-1)[i])))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activation_derivative_against_differences(kind):
    import torch
    import op_util as ou
    g = torch.linspace(-8, 8, 401, dtype=torch.float64, requires_grad=True)
    d, = torch.autograd.grad(ou.act64(g, kind).sum(), g)
    h = 1e-5
    diff = (ou.act64(g.detach() + h, kind) - ou.act64(g.detach() - h, kind)) / (2 * h)
    assert float((d - diff).abs().max()) < 1e-8
