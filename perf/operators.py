"""The training-pass operators that feed the data-parallel step, as cases to be timed: embedding lookup and its gradient,
the norms around a block with gate and residual scale and their gradient, 8-bit activation checkpoints (round trip, through
the gated activation, and in the weight gradient).

Sizes are those of the package's workloads (GPT-2-small: vocabulary 50257, width 768; the 1.3B list: 2048 and 8192; the
Llama-shaped layers: 4096 and 11008) or generic.  `run` computes an operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end) unless `own` is set, when it calls the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32                      # elements of a row that share one step in an 8-bit checkpoint
C_GELU = math.sqrt(2.0 / math.pi)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one sequence's lookup at the start of a forward pass: latency counts
        {"name": "embedding 1k x 768", "op": "embedding", "tokens": 1024, "vocab": 50257, "dim": 768, "ids": "i64",
         "dtype": "bf16", "scale": 1.0},
        # a micro-batch of GPT-2-small: the gradient is written over the whole table's slice of a rank buffer
        {"name": "embedding grad 8k x 768", "op": "embedding_grad", "tokens": 8192, "vocab": 50257, "dim": 768,
         "ids": "i64", "dtype": "bf16", "scale": 1.0, "accumulate": False, "pad": 0.0},
        # tied embedding of the 1.3B list: the output layer's gradient is there already and the lookup's is added; padded
        {"name": "embedding grad 64k x 2048 add", "op": "embedding_grad", "tokens": 65536, "vocab": 50257, "dim": 2048,
         "ids": "i32", "dtype": "bf16", "scale": 45.25, "accumulate": True, "pad": 0.03},
        # a short sequence through a layer-norm block boundary with a per-channel gate: latency counts
        {"name": "block norm ln 333 x 768", "op": "block_norm", "rows": 333, "dim": 768, "kind": "layer",
         "gate": "channel", "stream": "bf16", "res": 1.0, "branch": 1.0},
        # a long micro-batch of the Llama-shaped layers, norms on both sides of the block, scaled branch
        {"name": "block norm grad rms 16k x 4096", "op": "block_norm_grad", "rows": 16384, "dim": 4096, "kind": "rms",
         "gate": "channel", "stream": "bf16", "res": 1.0, "branch": 0.25},
        # the 1.3B width with the residual stream kept in 32 bits, a gate per token, an odd row count
        {"name": "block norm grad ln 8191 x 2048", "op": "block_norm_grad", "rows": 8191, "dim": 2048, "kind": "layer",
         "gate": "token", "stream": "f32", "res": 0.5, "branch": 1.0},
        # SwiGLU of a Llama-shaped layer, forward with its 8-bit checkpoint and the gradient from it
        {"name": "swiglu step 8k x 11008", "op": "act_step", "rows": 8192, "dim": 11008, "act": "silu", "gated": True},
        # the gradient of a GELU block of the 1.3B list alone, a short ragged micro-batch
        {"name": "gelu grad 1001 x 8192", "op": "act_grad", "rows": 1001, "dim": 8192, "act": "gelu", "gated": False},
        # a small odd-shaped activation put away in 8 bits and taken back
        {"name": "checkpoint 129 x 1111", "op": "ckpt8", "rows": 129, "dim": 1111, "dtype": "bf16"},
        # the input of a Llama-shaped layer's blocks
        {"name": "checkpoint 16k x 4096", "op": "ckpt8", "rows": 16384, "dim": 4096, "dtype": "bf16"},
        # GPT-2-small's fused query/key/value weight, one odd-length sequence, written in bf16
        {"name": "wgrad 1023 x 2304 x 768", "op": "wgrad", "rows": 1023, "n": 2304, "k": 768, "out": "bf16",
         "accumulate": False},
        # the gate projection of a Llama-shaped layer, added in 32 bits
        {"name": "wgrad 8k x 11008 x 4096", "op": "wgrad", "rows": 8192, "n": 11008, "k": 4096, "out": "f32",
         "accumulate": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embedding", "embedding_grad", "block_norm", "block_norm_grad", "act_step", "act_grad", "ckpt8", "wgrad"])
    dim = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024), 768, 2048, 4096])
    rows = max(1, min(_log(rng, 1, 65536), (1 << 27) // dim))
    if op == "embedding":
        return {"op": op, "tokens": rows, "vocab": _log(rng, 100, 100000), "dim": min(dim, 4096),
                "ids": rng.choice(["i32", "i64"]), "dtype": rng.choice(["bf16", "f32"]), "scale": rng.choice([1.0, 27.7])}
    if op == "embedding_grad":
        return {"op": op, "tokens": rows, "vocab": _log(rng, 100, 100000), "dim": min(dim, 2048),
                "ids": rng.choice(["i32", "i64"]), "dtype": rng.choice(["bf16", "f32"]), "scale": rng.choice([1.0, 27.7]),
                "accumulate": rng.random() < 0.5, "pad": rng.choice([0.0, 0.1])}
    if op in ("block_norm", "block_norm_grad"):
        rows = min(rows, (1 << 26) // dim)
        return {"op": op, "rows": rows, "dim": dim, "kind": rng.choice(["rms", "layer"]),
                "gate": rng.choice(["none", "channel", "token"]), "stream": rng.choice(["bf16", "f32"]),
                "res": rng.choice([1.0, 0.8]), "branch": rng.choice([1.0, 0.3])}
    if op in ("act_step", "act_grad"):
        return {"op": op, "rows": min(rows, (1 << 26) // dim), "dim": dim, "act": rng.choice(["silu", "gelu"]),
                "gated": rng.random() < 0.6}
    if op == "ckpt8":
        return {"op": op, "rows": rows, "dim": dim, "dtype": rng.choice(["bf16", "f32"])}
    return {"op": op, "rows": _log(rng, 1, 16384), "n": rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024)]),
            "k": rng.choice([_log(rng, 64, 4096), 768, 2048]), "out": rng.choice(["bf16", "f32"]),
            "accumulate": rng.random() < 0.5}


# ----------------------------------------------------------------------------------------------------------- inputs

def _randn(gen, *shape, dtype=torch.bfloat16, std=1.0, mean=0.0):
    return torch.randn(*shape, generator=gen, device=DEV).mul_(std).add_(mean).to(dtype)


def _activation(gen, rows, dim, dtype=torch.bfloat16):
    """Activations with a few channels far larger than the rest, as in trained models."""
    x = torch.randn(rows, dim, generator=gen, device=DEV)
    ch = torch.rand(dim, generator=gen, device=DEV)
    return x.mul_(torch.where(ch > 0.995, 20.0, 1.0)).to(dtype)


def _token_ids(gen, tokens, vocab, kind):
    """Token numbers whose frequencies fall off like 1/rank, scattered over the vocabulary."""
    u = torch.rand(tokens, generator=gen, device=DEV, dtype=torch.float64)
    rank = torch.exp(u * math.log(vocab)).floor_().long().sub_(1).clamp_(0, vocab - 1)
    perm = torch.randperm(vocab, generator=gen, device=DEV)
    return perm[rank].to(torch.int64 if kind == "i64" else torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 17)
    c, op = dict(case), case["op"]
    s = {"case": c}
    if op in ("embedding", "embedding_grad"):
        T, V, d, dt = c["tokens"], c["vocab"], c["dim"], DT[c["dtype"]]
        s["ids"] = _token_ids(gen, T, V, c["ids"])
        if op == "embedding":
            s["table"] = _randn(gen, V, d, dtype=dt, std=0.02)
            s["out"] = torch.empty(T, d, dtype=dt, device=DEV)
        else:
            s["pad_id"] = 0
            s["ids"][T - int(T * c["pad"]):] = 0
            s["dout"] = _randn(gen, T, d, dtype=dt, std=1e-3)
            s["dtable"] = _randn(gen, V, d, dtype=dt, std=1e-3) if c["accumulate"] else torch.empty(V, d, dtype=dt, device=DEV)
    elif op in ("block_norm", "block_norm_grad"):
        T, d, st = c["rows"], c["dim"], DT[c["stream"]]
        ln = c["kind"] == "layer"
        s["y"] = _activation(gen, T, d)
        s["w_post"], s["w_pre"] = (_randn(gen, d, std=0.1, mean=1.0) for _ in range(2))
        s["b_post"], s["b_pre"] = (_randn(gen, d, std=0.1) for _ in range(2)) if ln else (None, None)
        s["gate"] = None if c["gate"] == "none" else _randn(gen, d if c["gate"] == "channel" else T, std=0.2, mean=0.7)
        if op == "block_norm":
            s["x"] = _activation(gen, T, d, st)
            s["r"], s["z"] = torch.empty_like(s["x"]), torch.empty_like(s["y"])
            s["post_stats"], s["pre_stats"] = (torch.empty(T, 2, device=DEV) for _ in range(2))
        else:
            s["r"] = _activation(gen, T, d, st)
            s["dr"], s["dz"] = _randn(gen, T, d, dtype=st, std=1e-3), _randn(gen, T, d, std=1e-3)
            s["post_stats"], s["pre_stats"] = _stats(s["y"], ln), _stats(s["r"], ln)
            s["dx"], s["dy"] = torch.empty_like(s["r"]), torch.empty_like(s["y"])
            for k in ("w_post", "b_post", "w_pre", "b_pre", "gate"):
                s["d" + k] = None if s[k] is None else torch.empty_like(s[k])
    elif op in ("act_step", "act_grad"):
        T, F = c["rows"], c["dim"]
        s["g"] = _activation(gen, T, F)
        s["u"] = _randn(gen, T, F) if c["gated"] else None
        s["dh"] = _randn(gen, T, F, std=1e-3)
        s["g8"] = _encode(s["g"].float())
        s["u8"] = _encode(s["u"].float()) if c["gated"] else None
        for k in ("h", "h_again", "dg") + (("du",) if c["gated"] else ()):
            s[k] = torch.empty(T, F, dtype=torch.bfloat16, device=DEV)
        if op == "act_step":      # the checkpoint is the pass's own
            s["g8"], s["u8"] = [tuple(torch.empty_like(t) for t in p) if p else None for p in (s["g8"], s["u8"])]
        else:
            s["g"] = s["u"] = None
    elif op == "ckpt8":
        s["x"] = _activation(gen, c["rows"], c["dim"], DT[c["dtype"]])
        s["codes"], s["scales"] = (torch.empty_like(t) for t in _encode(s["x"].float()))
        s["back"] = torch.empty_like(s["x"])
    else:
        T, n, k = c["rows"], c["n"], c["k"]
        s["dy"] = _randn(gen, T, n, std=1e-3)
        s["codes"], s["scales"] = _encode(_activation(gen, T, k).float())
        s["dw"] = _randn(gen, n, k, dtype=DT[c["out"]], std=1e-3) if c["accumulate"] else \
            torch.empty(n, k, dtype=DT[c["out"]], device=DEV)
    return s


def _stats(x, ln):
    x = x.float()
    mean = x.mean(1) if ln else torch.zeros(x.shape[0], device=x.device)
    return torch.stack([mean, torch.rsqrt((x - mean[:, None]).square().mean(1) + 1e-5)], 1)


# ------------------------------------------------------------------------------------------------------ plain forms

def _encode(x):
    """Codes and step bytes of a float32 matrix: the step of a group of 32 is the least power of two with all codes in +-127."""
    rows, d = x.shape
    wide = -(-d // GROUP) * GROUP
    if wide != d:
        x = torch.cat([x, x.new_zeros(rows, wide - d)], 1)
    g = x.view(rows, wide // GROUP, GROUP)
    f, e = torch.frexp(g.abs().amax(2))
    k = torch.where(f > 127.0 / 128.0, e - 6, e - 7).clamp(min=-126)
    k = torch.where(f == 0, -126, k)
    codes = torch.round(torch.ldexp(g, -k[:, :, None])).to(torch.int8)
    return codes.view(rows, wide), (k + 127).to(torch.uint8)


def _decode(codes, scales, d):
    rows, wide = codes.shape
    v = codes.view(rows, wide // GROUP, GROUP).float()
    return torch.ldexp(v, scales.int()[:, :, None] - 127).view(rows, wide)[:, :d]


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    th = torch.tanh(C_GELU * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * C_GELU * (1.0 + 3 * 0.044715 * g * g)


def _act_back(dh, g, u, kind):
    f, df = _act(g, kind)
    if u is None:
        return [(dh * df).bfloat16(), f.bfloat16()]
    return [(dh * u * df).bfloat16(), (dh * f).bfloat16(), (f * u).bfloat16()]


def _hat(x, stats):
    return (x.float() - stats[:, :1]) * stats[:, 1:]


def _norm_back(v, hat, stats, ln):
    v2 = v - hat * (v * hat).mean(1, keepdim=True)
    if ln:
        v2 = v2 - v.mean(1, keepdim=True)
    return v2 * stats[:, 1:]


def _gate_of(s):
    gate = s["gate"]
    if gate is None:
        return 1.0
    return gate.float()[None, :] if s["case"]["gate"] == "channel" else gate.float()[:, None]


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "embedding":
        return (s["table"][s["ids"].long()].float() * c["scale"]).to(s["out"].dtype)
    if op == "embedding_grad":
        keep = s["ids"] != s["pad_id"]
        g = torch.zeros(c["vocab"], c["dim"], device=DEV)
        g.index_add_(0, s["ids"].long(), s["dout"].float() * keep[:, None])
        g *= c["scale"]
        if c["accumulate"]:
            g += s["dtable"].float()
        return s["dtable"].copy_(g)
    if op == "block_norm":
        ln = c["kind"] == "layer"
        ps = _stats(s["y"], ln)
        n = _hat(s["y"], ps) * s["w_post"].float()
        n = n + s["b_post"].float() if ln else n
        r = c["res"] * s["x"].float() + c["branch"] * _gate_of(s) * n
        qs = _stats(r, ln)
        z = _hat(r, qs) * s["w_pre"].float()
        z = z + s["b_pre"].float() if ln else z
        return [r.to(s["r"].dtype), z.bfloat16(), ps, qs]
    if op == "block_norm_grad":
        ln = c["kind"] == "layer"
        rh, yh, dz = _hat(s["r"], s["pre_stats"]), _hat(s["y"], s["post_stats"]), s["dz"].float()
        gate = _gate_of(s)
        dr = s["dr"].float() + _norm_back(dz * s["w_pre"].float(), rh, s["pre_stats"], ln)
        n = yh * s["w_post"].float()
        n = n + s["b_post"].float() if ln else n
        dn = c["branch"] * gate * dr
        out = {"dx": (c["res"] * dr).to(s["dx"].dtype),
               "dy": _norm_back(dn * s["w_post"].float(), yh, s["post_stats"], ln).bfloat16(),
               "dw_post": (dn * yh).sum(0).bfloat16(), "dw_pre": (dz * rh).sum(0).bfloat16()}
        if ln:
            out["db_post"], out["db_pre"] = dn.sum(0).bfloat16(), dz.sum(0).bfloat16()
        if s["gate"] is not None:
            out["dgate"] = (c["branch"] * dr * n).sum(0 if c["gate"] == "channel" else 1).bfloat16()
        return out
    if op in ("act_step", "act_grad"):
        out = []
        if op == "act_step":
            f = _act(s["g"].float(), c["act"])[0]
            out = [(f * s["u"].float() if c["gated"] else f).bfloat16()]
            g8 = _encode(s["g"].float())
            u8 = _encode(s["u"].float()) if c["gated"] else None
        else:
            g8, u8 = s["g8"], s["u8"]
        return out + _act_back(s["dh"].float(), _decode(*g8, c["dim"]), _decode(*u8, c["dim"]) if u8 else None, c["act"])
    if op == "ckpt8":
        return _decode(*_encode(s["x"].float()), c["dim"]).to(s["x"].dtype)
    g = torch.matmul(s["dy"].float().t(), _decode(s["codes"], s["scales"], c["k"]))
    if c["accumulate"]:
        g += s["dw"].float()
    return s["dw"].copy_(g)


# ----------------------------------------------------------------------------------------------- the package's calls

def _ws(s, size):
    """The workspace that a program keeps for a call: made at the state's first pass."""
    if "ws" not in s:
        s["ws"] = torch.empty(size(), dtype=torch.uint8, device=DEV)
    return s["ws"]


def _own(s):
    import zero_gradient_sync_gb300 as dp
    c, op = s["case"], s["case"]["op"]
    if op == "embedding":
        dp.dp_embedding(s["out"], s["table"], s["ids"], scale=c["scale"])
        return s["out"]
    if op == "embedding_grad":
        ws = _ws(s, lambda: dp.dp_embedding_workspace_size(c["tokens"], c["vocab"], c["dim"]))
        dp.dp_embedding_grad(s["dtable"], s["dout"], s["ids"], scale=c["scale"], pad_id=s["pad_id"],
                             accumulate=c["accumulate"], ws=ws)
        return s["dtable"]
    if op in ("block_norm", "block_norm_grad"):
        kind = dp.DP_NORM_LAYER if c["kind"] == "layer" else dp.DP_NORM_RMS
        if op == "block_norm":
            dp.dp_block_norm(s["r"], s["z"], s["x"], s["y"], w_post=s["w_post"], b_post=s["b_post"], gate=s["gate"],
                             gate_per_token=c["gate"] == "token", w_pre=s["w_pre"], b_pre=s["b_pre"], kind=kind, eps=1e-5,
                             res_scale=c["res"], branch_scale=c["branch"], post_stats=s["post_stats"],
                             pre_stats=s["pre_stats"])
            return [s["r"], s["z"], s["post_stats"], s["pre_stats"]]
        ws = _ws(s, lambda: dp.dp_block_norm_workspace_size(c["rows"], c["dim"]))
        dp.dp_block_norm_grad(s["dx"], s["dy"], s["dr"], s["dz"], s["r"], s["y"], w_post=s["w_post"], b_post=s["b_post"],
                              gate=s["gate"], gate_per_token=c["gate"] == "token", w_pre=s["w_pre"], kind=kind,
                              res_scale=c["res"], branch_scale=c["branch"], post_stats=s["post_stats"],
                              pre_stats=s["pre_stats"], dw_post=s["dw_post"], db_post=s["db_post"], dgate=s["dgate"],
                              dw_pre=s["dw_pre"], db_pre=s["db_pre"], ws=ws)
        return {k: s[k] for k in ("dx", "dy", "dw_post", "dw_pre", "db_post", "db_pre", "dgate") if s[k] is not None}
    if op in ("act_step", "act_grad"):
        act = dp.DP_ACT_SILU if c["act"] == "silu" else dp.DP_ACT_GELU
        out = []
        if op == "act_step":
            dp.dp_act_ckpt8(s["h"], s["g"], s["u"], act=act, g8=s["g8"], u8=s["u8"])
            out = [s["h"]]
        du = s["du"] if c["gated"] else None
        dp.dp_act_ckpt8_grad(s["dg"], du, s["dh"], act=act, g8=s["g8"], u8=s["u8"], h=s["h_again"])
        return out + [s["dg"]] + ([du] if c["gated"] else []) + [s["h_again"]]
    if op == "ckpt8":
        dp.dp_ckpt8_encode(s["codes"], s["scales"], s["x"])
        dp.dp_ckpt8_decode(s["back"], s["codes"], s["scales"])
        return s["back"]
    ws = _ws(s, lambda: dp.dp_wgrad8_workspace_size(c["rows"], c["n"], c["k"]))
    dp.dp_wgrad8(s["dw"], s["dy"], s["codes"], s["scales"], accumulate=c["accumulate"], ws=ws)
    return s["dw"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------------------- work

def _distinct(tokens, vocab):
    """Expected number of different tokens among `tokens` draws of _token_ids."""
    k = torch.arange(1, vocab + 1, dtype=torch.float64)
    p = torch.log((k + 1) / k) / math.log(vocab)
    return float((1 - (1 - p.clamp(max=1.0)).pow(tokens)).sum())


def work(case):
    c, op = case, case["op"]
    if op == "embedding":
        e = SIZE[c["dtype"]]
        rows = min(_distinct(c["tokens"], c["vocab"]), c["tokens"])
        return {"bytes": c["dim"] * e * (rows + c["tokens"]) + c["tokens"] * (8 if c["ids"] == "i64" else 4),
                "flops": c["tokens"] * c["dim"]}
    if op == "embedding_grad":
        e = SIZE[c["dtype"]]
        table = 2 * _distinct(c["tokens"], c["vocab"]) if c["accumulate"] else c["vocab"]
        live = c["tokens"] - int(c["tokens"] * c["pad"])
        return {"bytes": c["dim"] * e * (live + table) + c["tokens"] * (8 if c["ids"] == "i64" else 4),
                "flops": live * c["dim"]}
    if op in ("block_norm", "block_norm_grad"):
        st, each = SIZE[c["stream"]], c["rows"] * c["dim"]
        if op == "block_norm":
            return {"bytes": each * (2 * st + 4) + 16 * c["rows"] + 12 * c["dim"], "flops": 16 * each}
        return {"bytes": each * (3 * st + 6) + 16 * c["rows"] + 20 * c["dim"], "flops": 30 * each}
    q = 1 + 1 / GROUP
    if op in ("act_step", "act_grad"):
        each, m = c["rows"] * c["dim"], 2 if c["gated"] else 1
        grad = each * (2 + m * q + 2 * m + 2)
        return {"bytes": grad + (each * (2 * m + 2 + m * q) if op == "act_step" else 0), "flops": 20 * each}
    if op == "ckpt8":
        return {"bytes": c["rows"] * c["dim"] * 2 * (SIZE[c["dtype"]] + q), "flops": 4 * c["rows"] * c["dim"]}
    return {"bytes": c["rows"] * (2 * c["n"] + q * c["k"]) + c["n"] * c["k"] * SIZE[c["out"]] * (2 if c["accumulate"] else 1),
            "flops": 2 * c["rows"] * c["n"] * c["k"]}


# --------------------------------------------------------------------------------------- the definitions, in 64 bits

def _norm64(x, w, b, ln):
    """A norm from its definition, and its (mean, 1/deviation)."""
    mu = x.sum(1, keepdim=True) / x.shape[1] if ln else torch.zeros(x.shape[0], 1, dtype=x.dtype, device=x.device)
    inv = ((x - mu).pow(2).sum(1, keepdim=True) / x.shape[1] + 1e-5).pow(-0.5)
    n = (x - mu) * inv * w
    return (n if b is None else n + b), torch.cat([mu, inv], 1)


def _ckpt64(x):
    """What an 8-bit checkpoint of x stands for, by counting the step up from the smallest that could do."""
    rows, d = x.shape
    out = torch.empty(rows, d, dtype=torch.float64, device=x.device)
    full = d // GROUP * GROUP
    parts = ([x[:, :full].double().reshape(-1, GROUP)] if full else []) + ([x[:, full:].double()] if full < d else [])
    done = []
    for p in parts:
        top = p.abs().max(1, keepdim=True).values
        k = torch.floor(torch.log2(top.clamp(min=2.0 ** -126) / 127.0)) - 1
        for _ in range(3):
            k = torch.where(top > 127.0 * torch.exp2(k), k + 1, k)
        step = torch.exp2(k.clamp(min=-126))
        done.append(torch.round(p / step) * step)
    if full:
        out[:, :full] = done[0].reshape(rows, full)
    if full < d:
        out[:, full:] = done[-1]
    return out


def _act64(g, kind):
    return g * torch.sigmoid(g) if kind == "silu" else 0.5 * g * (1 + torch.tanh(C_GELU * (g + 0.044715 * g ** 3)))


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    d64 = lambda k: None if s[k] is None else s[k].double()  # noqa: E731
    if op == "embedding":
        return torch.index_select(s["table"].double(), 0, s["ids"].long()) * c["scale"]
    if op == "embedding_grad":
        ids = s["ids"].long()
        live = torch.nonzero(ids != s["pad_id"])[:, 0]
        out = s["dtable"].double() if c["accumulate"] else torch.zeros(c["vocab"], c["dim"], dtype=torch.float64, device=DEV)
        return out.index_put_((ids[live],), s["dout"][live].double() * c["scale"], accumulate=True)
    if op in ("block_norm", "block_norm_grad"):
        ln = c["kind"] == "layer"
        gate = d64("gate")
        if op == "block_norm":
            n, ps = _norm64(d64("y"), d64("w_post"), d64("b_post"), ln)
            gated = n if gate is None else n * (gate if c["gate"] == "channel" else gate[:, None])
            r = c["res"] * d64("x") + c["branch"] * gated
            z, qs = _norm64(r, d64("w_pre"), d64("b_pre"), ln)
            return [r, z, ps, qs]
        leaf = {k: d64(k).requires_grad_() for k in ("y", "r", "w_post", "b_post", "w_pre", "b_pre", "gate") if s[k] is not None}
        n, _ = _norm64(leaf["y"], leaf["w_post"], leaf.get("b_post"), ln)
        if gate is not None:
            n = n * (leaf["gate"] if c["gate"] == "channel" else leaf["gate"][:, None])
        z, _ = _norm64(leaf["r"], leaf["w_pre"], leaf.get("b_pre"), ln)
        # the stream's gradient: what comes down it, and what comes through the norm before the next block
        pre = [k for k in ("r", "w_pre", "b_pre") if k in leaf]
        got = dict(zip(pre, torch.autograd.grad(z, [leaf[k] for k in pre], d64("dz"))))
        dr = d64("dr") + got.pop("r")
        post = [k for k in ("y", "w_post", "b_post", "gate") if k in leaf]
        got.update(zip(post, torch.autograd.grad(n, [leaf[k] for k in post], c["branch"] * dr)))
        return {"dx": c["res"] * dr, **{"d" + k: v for k, v in got.items()}}
    if op in ("act_step", "act_grad"):
        if op == "act_step":
            f = _act64(d64("g"), c["act"])
            out = [f * d64("u") if c["gated"] else f]
            g, u = _ckpt64(s["g"]), _ckpt64(s["u"]) if c["gated"] else None
        else:
            val = lambda p: p[0].double().mul_(torch.exp2(p[1].double() - 127).repeat_interleave(GROUP, 1))[:, :c["dim"]].contiguous()  # noqa: E731
            out, g, u = [], val(s["g8"]), val(s["u8"]) if c["gated"] else None
        leaf = [g.requires_grad_()] + ([u.requires_grad_()] if c["gated"] else [])
        h = _act64(g, c["act"])
        h = h * u if c["gated"] else h
        return out + list(torch.autograd.grad(h, leaf, d64("dh"))) + [h.detach()]
    if op == "ckpt8":
        return _ckpt64(s["x"])
    x = s["codes"].double() * torch.exp2(s["scales"].double() - 127).repeat_interleave(GROUP, 1)
    out = s["dy"].double().t() @ x[:, :c["k"]]
    return out + s["dw"].double() if c["accumulate"] else out
