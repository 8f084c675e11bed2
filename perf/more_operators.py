"""The measured cases of what stands around a block's layers: norms with gate
and residual, the gated feed-forward, and activation checkpoints in 8 bits.

Operators, by a case's "op":

  norm            the residual stream after a block, skip x + scale phi(z) v
                  with v = norm(f) w_after, and the next block's normed rows;
                  without f the normed rows of x alone, and x's checkpoint
  norm_backward   its gradients, from rows or from their checkpoints
  gated           h = act(x Wg^T) * (x Wu^T)
  gated_backward  its gradients, from the two projections kept in 8 bits, or
                  with both formed again from x
  checkpoint      rows to 8 bits with an exponent for each 32, and back

`run` computes a case in its plain form, or, where `own` is set, by the calls
of this package.
"""
import math

import numpy as np
import torch

own = False

_T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-6


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one token's residual added and normed between two blocks of a decoding model; latency
        dict(name="norm_decode_1", op="norm", M=1, d=4096, xt="f32", ft="f32", nt="bf16", f=True, norm_f=False,
             gate="none", span=1, keep=False),
        # prompts of a model that norms a block's result and gates it row by row, f32 stream
        dict(name="norm_prefill_8192", op="norm", M=8192, d=4096, xt="f32", ft="f32", nt="bf16", f=True, norm_f=True,
             gate="sigmoid", span=1, keep=False),
        # the ragged training batch in bf16: a block's first norm, its rows kept in 8 bits
        dict(name="norm_keep_30000", op="norm", M=30000, d=5120, xt="bf16", ft="bf16", nt="bf16", f=False,
             norm_f=False, gate="none", span=1, keep=True),
        # gradients of a short odd batch in f16, one gate for each sequence
        dict(name="norm_backward_333", op="norm_backward", M=333, d=2048, xt="f16", ft="f16", nt="f16", f=True,
             norm_f=True, gate="linear", span=100, keep=False),
        # gradients of 8 x 1024 tokens, f32 stream, both rows from their checkpoints
        dict(name="norm_backward_8192", op="norm_backward", M=8192, d=4096, xt="f32", ft="f32", nt="bf16", f=True,
             norm_f=True, gate="none", span=1, keep=True),
        # one request that decodes alone; the weights' bytes
        dict(name="gated_decode_1", op="gated", M=1, d=4096, ff=12288, act="bf16", ht="bf16", kind="silu"),
        # 64 requests that decode together, f16, h in f32 for a layer of f32 rows
        dict(name="gated_decode_64", op="gated", M=64, d=2048, ff=5504, act="f16", ht="f32", kind="gelu"),
        # the ragged batch through the largest layer
        dict(name="gated_prefill_30000", op="gated", M=30000, d=5120, ff=17408, act="bf16", ht="bf16", kind="silu"),
        # a short odd batch trained in f16, the projections formed again
        dict(name="gated_train_300", op="gated_backward", M=300, d=2048, ff=5504, act="f16", ht="f16", kind="gelu",
             tape=False, gscale=64.0),
        # 8 x 1024 tokens through the MLP shape, trained in bf16 from the projections in 8 bits
        dict(name="gated_train_8192", op="gated_backward", M=8192, d=4096, ff=12288, act="bf16", ht="bf16",
             kind="silu", tape=True, gscale=1.0),
        # a decoding batch's rows to 8 bits and back; latency
        dict(name="checkpoint_64", op="checkpoint", M=64, d=2048, t="f32"),
        # the MLP's inner rows of a training batch
        dict(name="checkpoint_8192", op="checkpoint", M=8192, d=12288, t="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "norm_backward", "gated", "gated", "gated_backward",
                     "gated_backward", "checkpoint"])
    if op == "checkpoint":
        return dict(op=op, M=_log(rng, 1, 16384), d=32 * _log(rng, 4, 256), t=rng.choice(["f32", "f16", "bf16"]))
    if op.startswith("norm"):
        xt, ft, nt = rng.choice([("f32", "f32", "f32"), ("f32", "f32", "bf16"), ("f32", "f32", "f16"),
                                 ("f32", "bf16", "bf16"), ("f32", "f16", "f16"), ("bf16", "bf16", "bf16"),
                                 ("f16", "f16", "f16")])
        f = rng.random() < 0.8
        keep = rng.random() < 0.4 and (op == "norm_backward" or not f)
        gate = rng.choice(["none", "linear", "sigmoid", "silu"]) if f else "none"
        M = _log(rng, 1, 16384)
        return dict(op=op, M=M, d=32 * _log(rng, 4, 192) if keep else 8 * _log(rng, 16, 768), xt=xt, ft=ft, nt=nt,
                    f=f, norm_f=f and rng.random() < 0.6, gate=gate,
                    span=rng.choice([1, 1, _log(rng, 2, 2048), M]) if gate != "none" else 1, keep=keep)
    act = rng.choice(["f16", "bf16"])
    c = dict(op=op, M=_log(rng, 1, 8192), d=128 * _log(rng, 2, 40), ff=128 * _log(rng, 2, 96), act=act,
             ht=rng.choice([act, act, "f32"]), kind=rng.choice(["silu", "gelu"]))
    if op == "gated_backward":
        c.update(tape=rng.random() < 0.5, gscale=64.0 if act == "f16" else 1.0)
    return c


# ----------------------------------------------------------------- inputs --
def _two_to(e):
    """2^e in 64 bits, from the bits of its exponent."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _pack(x):
    """(q int8, b uint8): 32 values a block of x's last axis share the step 2^(b - 133), the least power of two with
    round(x / step) within 127; b = 255 where a value is not finite."""
    v = x.double().reshape(*x.shape[:-1], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    fine = torch.isfinite(top)
    step = torch.clamp(torch.frexp(torch.where(fine, top, 1.0)).exponent - 7, min=-133)
    step = step + (torch.round(torch.where(fine, top, 1.0) * _two_to(-step)) > 127).int()
    # past the type's largest exponent there is no wider step to take: the block's largest values are cut off there
    step = torch.clamp(step, max=9 if x.dtype == torch.float16 else 121)
    q = torch.where(fine, torch.round(torch.where(fine, v, 0.0) * _two_to(-step)).clamp(-127, 127), 0.0)
    return q.reshape(x.shape).to(torch.int8), torch.where(fine, step + 133, 255).squeeze(-1).to(torch.uint8)


def _unpack(q, b):
    """The values that a checkpoint stands for, in f32."""
    v = (q.double().reshape(*q.shape[:-1], -1, 32) * _two_to(b.int()[..., None] - 133)).float()
    return torch.where(b[..., None] == 255, math.nan, v).reshape(q.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, sigma, t):
        return torch.randn(shape, generator=g, device="cuda").mul_(sigma).to(_T[t])

    def weights(n):  # of a norm: near one
        return 1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")

    s, M, d = dict(case), case["M"], case["d"]
    if case["op"] == "checkpoint":
        # activations: rows of different size, a few columns that stand out
        s["x"] = normal((M, 1), 1.0, "f32").exp() * normal((M, d), 1.0, "f32")
        s["x"] = (s["x"] * torch.where(torch.rand(d, generator=g, device="cuda") < 0.01, 20.0, 1.0)).to(_T[case["t"]])
        return s
    if case["op"].startswith("norm"):
        s["x"] = normal((M, d), 2.0, case["xt"])
        s["w"] = weights(d)
        s["skip"], s["scale"] = (1.0, 0.5) if case["f"] else (1.0, 1.0)
        s["fr"] = s["w_after"] = s["z"] = None
        if case["f"]:
            s["fr"] = normal((M, d), 0.7, case["ft"])
            s["w_after"] = weights(d) if case["norm_f"] else None
            if case["gate"] != "none":
                s["z"] = normal((-(-M // case["span"]), d), 1.0, case["ft"])
        if case["op"] == "norm_backward":
            s["dn"], s["dout"] = normal((M, d), 1e-2, case["nt"]), normal((M, d), 1e-2, case["xt"])
            # what the forward leaves: its result and the statistics, as rows or as checkpoints
            fwd = _norm(s)
            s["out"], s["stats"] = fwd["out"], fwd["stats"]
            if case["keep"]:
                s["out_kept"] = _pack(s["out"])
                s["fr_kept"] = _pack(s["fr"]) if case["f"] else None
                s["out"] = s["fr"] = None
            del s["x"]
        return s
    ff, act = case["ff"], case["act"]
    s["x"] = normal((M, d), 1.0, act)
    s["w_gate"], s["w_up"] = normal((ff, d), d ** -0.5, act), normal((ff, d), d ** -0.5, act)
    if case["op"] == "gated_backward":
        s["dh"] = normal((M, ff), 1e-2, case["ht"])
        if case["tape"]:
            x = s["x"].float()
            kept = [_pack(x @ w.float().T) for w in (s["w_gate"], s["w_up"])]
            s["tape"] = tuple(torch.stack(t) for t in zip(*kept))
        else:
            s["tape"] = None
    return s


# ----------------------------------------------------------------- passes --
def _phi(kind, z):
    """(phi(z), its derivative)."""
    if kind == "linear":
        return z, torch.ones_like(z)
    p = torch.sigmoid(z)
    if kind == "sigmoid":
        return p, p * (1 - p)
    return z * p, p * (1 + z * (1 - p))


def _act(kind, g):
    """(act(g), its derivative)."""
    if kind == "silu":
        return _phi("silu", g)
    a, b = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(a * (g + b * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * a * (1 + 3 * b * g * g)


def _rstd(v):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + _EPS)


def _gate(s, M):
    if s["z"] is None:
        return 1.0, 0.0
    phi, slope = _phi(s["gate"], s["z"].float())
    row = torch.arange(M, device=phi.device) // s["span"]
    return phi[row], slope[row]


def _norm(s):
    x, M = s["x"].float(), s["M"]
    stats = torch.zeros((2, M), device=x.device)
    if s["fr"] is not None:
        v = s["fr"].float()
        if s["norm_f"]:
            r = _rstd(v)
            stats[1] = r[:, 0]
            v = v * r * s["w_after"]
        out = (s["skip"] * x + s["scale"] * _gate(s, M)[0] * v).to(_T[s["xt"]])
        x = out.float()
    r = _rstd(x)
    stats[0] = r[:, 0]
    n = (x * r * s["w"]).to(_T[s["nt"]])
    if s["fr"] is not None:
        return {"out": out, "n": n, "stats": stats}
    got = {"out": s["x"], "n": n, "stats": stats}
    if s["op"] == "norm":
        del got["out"]
        if s["keep"]:
            got["kept"] = _unpack(*_pack(s["x"])).to(_T[s["xt"]])
    return got


def _norm_backward(s):
    M = s["M"]

    def through(v, row, r):  # the gradient of row * r by way of the norm
        hat = row * r
        return r * (v - hat * (v * hat).mean(1, keepdim=True))

    out = s["out"].float() if s["out"] is not None else _unpack(*s["out_kept"])
    r = s["stats"][0][:, None]
    dn = s["dn"].float()
    dO = s["dout"].float() + through(s["w"] * dn, out, r)
    got = {"dx": (s["skip"] * dO).to(_T[s["xt"]]), "dw": (dn * out * r).sum(0)}
    if not s["f"]:
        return got
    f = s["fr"].float() if s["fr"] is not None else _unpack(*s["fr_kept"])
    phi, slope = _gate(s, M)
    p = s["scale"] * phi * dO
    if s["norm_f"]:
        rf = s["stats"][1][:, None]
        got["df"] = through(s["w_after"] * p, f, rf).to(_T[s["ft"]])
        got["dw_after"] = (p * f * rf).sum(0)
        f = f * rf * s["w_after"]
    else:
        got["df"] = p.to(_T[s["ft"]])
    if s["z"] is not None:
        dz = s["scale"] * slope * f * dO
        if s["span"] == 1:
            got["dz"] = dz.to(_T[s["ft"]])
        else:
            G = s["z"].shape[0]
            dz = torch.cat([dz, dz.new_zeros((G * s["span"] - M, dz.shape[1]))])
            got["dz"] = dz.view(G, s["span"], -1).sum(1)
    return got


def _gated(s):
    x = s["x"].float()
    return {"h": (_act(s["kind"], x @ s["w_gate"].float().T)[0] * (x @ s["w_up"].float().T)).to(_T[s["ht"]])}


def _gated_backward(s):
    x, wg, wu, dh = s["x"].float(), s["w_gate"].float(), s["w_up"].float(), s["dh"].float()
    if s["tape"] is None:
        g, u = x @ wg.T, x @ wu.T
    else:
        g, u = _unpack(*s["tape"])
    a, slope = _act(s["kind"], g)
    dg, du = dh * u * slope, dh * a
    t = _T[s["act"]]
    return {"dx": (dg @ wg + du @ wu).to(t), "dw_gate": (dg.T @ x).to(t), "dw_up": (du.T @ x).to(t)}


def _plain(s):
    if s["op"] == "checkpoint":
        return {"x": _unpack(*_pack(s["x"])).to(s["x"].dtype)}
    return {"norm": _norm, "norm_backward": _norm_backward, "gated": _gated, "gated_backward": _gated_backward}[
        s["op"]](s)


def _own(s):
    import binary_rank_linear_amd as blr

    op = s["op"]
    if op == "checkpoint":
        q, b = blr.blr_checkpoint_save(s["x"])
        return {"x": blr.blr_checkpoint_load(q, b, s["x"].dtype)}
    if op.startswith("norm"):
        how = dict(w_after=s["w_after"], gate=s["z"], span=s["span"], norm_f=s["norm_f"], skip=s["skip"],
                   scale=s["scale"])
        if s["gate"] != "none":
            how["gate_kind"] = {"linear": blr.GATE_LINEAR, "sigmoid": blr.GATE_SIGMOID, "silu": blr.GATE_SILU}[
                s["gate"]]
        if op == "norm":
            out, n, stats, kept = blr.blr_norm_forward(s["x"], s["fr"], s["w"], eps=_EPS, n_dtype=_T[s["nt"]],
                                                       keep=s["keep"], **how)
            got = {"out": out, "n": n, "stats": stats}
            if s["fr"] is None:
                del got["out"]
                if s["keep"]:
                    got["kept"] = blr.blr_checkpoint_load(*kept, s["x"].dtype)
            return got
        if "ws" not in s:  # the buffer that a program keeps over its steps
            s["ws"] = blr.workspace_norm(s["M"], s["d"], s["span"])
        out = s["out_kept"] if s["keep"] else s["out"]
        f = s["fr_kept"] if s["keep"] else s["fr"]
        dx, df, dz, dw, dw_after = blr.blr_norm_backward(s["dn"], s["dout"], out, f, s["w"], s["stats"],
                                                         f_dtype=_T[s["ft"]], ws=s["ws"], **how)
        got = {"dx": dx, "dw": dw}
        if s["f"]:
            got["df"] = df
            if s["norm_f"]:
                got["dw_after"] = dw_after
            if s["z"] is not None:
                got["dz"] = dz
        return got
    kind = {"silu": blr.ACT_SILU, "gelu": blr.ACT_GELU}[s["kind"]]
    if op == "gated":
        h, _ = blr.blr_gated_forward(s["x"], s["w_gate"], s["w_up"], kind=kind, h_dtype=_T[s["ht"]])
        return {"h": h}
    if "ws" not in s:
        s["ws"] = blr.workspace_gated(s["M"], s["d"], s["ff"])
    dx, dwg, dwu = blr.blr_gated_backward(s["x"], s["dh"], s["w_gate"], s["w_up"], s["tape"], kind=kind,
                                          gscale=s["gscale"], ws=s["ws"])
    return {"dx": dx, "dw_gate": dwg, "dw_up": dwu}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- what a pass needs --
def work(case):
    c, M, d = case, case["M"], case["d"]
    if c["op"] == "checkpoint":  # rows in, 8 bits out; and back
        return {"bytes": M * d * 2 * (_SIZE[c["t"]] + 1 + 1 / 32), "flops": 4 * M * d}
    if c["op"].startswith("norm"):
        x, f, n, z = (_SIZE[c[k]] for k in ("xt", "ft", "nt", "ft"))
        z = 0 if c["gate"] == "none" else z * (-(-M // c["span"]) / M)
        if c["op"] == "norm":
            rows = x + n + (f + z + x if c["f"] else 0) + (2 * (1 + 1 / 32) + x if c["keep"] else 0)
            return {"bytes": M * d * rows + 8 * M + 4 * d, "flops": 8 * M * d}
        kept = 1 + 1 / 32
        rows = 2 * x + n + (kept if c["keep"] else x) + ((kept if c["keep"] else f) + f + 2 * z if c["f"] else 0)
        return {"bytes": M * d * rows + 8 * M + 8 * d, "flops": 20 * M * d}
    ff, a, h = c["ff"], _SIZE[c["act"]], _SIZE[c["ht"]]
    weights = 2 * ff * d * a
    if c["op"] == "gated":
        return {"bytes": M * d * a + weights + M * ff * h, "flops": 4 * M * d * ff}
    tape = 2 * M * ff * (1 + 1 / 32) if c["tape"] else 0
    return {"bytes": 2 * M * d * a + 2 * weights + M * ff * h + tape, "flops": (8 if c["tape"] else 12) * M * d * ff}


# ---------------------------------------------------------------- 64 bits --
def _exact_rows(q, b):
    """A checkpoint's values by its definition, in 64 bits."""
    e = b.cpu().numpy().astype(np.int64)
    v = np.ldexp(q.cpu().numpy().astype(np.float64), np.repeat(e, 32, axis=-1) - 133)
    return torch.from_numpy(np.where(np.repeat(e == 255, 32, axis=-1), np.nan, v)).cuda()


def _exact_checkpoint(x):
    """x by way of its checkpoint: each 32 values to the nearest multiple of the least step that 127 of reach."""
    half = x.dtype == torch.float16
    v = x.double().view(x.shape[0], -1, 32)
    top = v.abs().amax(2)
    step = torch.full_like(top, 2.0 ** -133)
    for e in range(-132, 10 if half else 122):
        step = torch.where(top >= 127.5 * step, 2.0 ** e, step)
    k = torch.clamp(torch.round(v / step[:, :, None]), -127, 127)
    return (k * step[:, :, None]).view(x.shape)


def exact(case, seed):
    s, M, d = prepare(case, seed), case["M"], case["d"]
    if case["op"] == "checkpoint":
        return {"x": _exact_checkpoint(s["x"])}
    if case["op"].startswith("norm"):
        gates = None
        if s["z"] is not None:
            z = s["z"].double()
            sig = 1 / (1 + torch.exp(-z))
            one = torch.ones_like(z)
            gates = {"linear": (z, one), "sigmoid": (sig, sig - sig ** 2), "silu": (z * sig, sig + z * (sig - sig ** 2))}
            gates = [t.repeat_interleave(s["span"], 0)[:M] for t in gates[s["gate"]]]
        if case["op"] == "norm":
            x, stats = s["x"].double(), torch.zeros((2, M), dtype=torch.float64, device="cuda")
            got = {}
            if case["f"]:
                v = s["fr"].double()
                if case["norm_f"]:
                    stats[1] = 1 / torch.sqrt((v ** 2).sum(1) / d + _EPS)
                    v = v * stats[1][:, None] * s["w_after"].double()
                if gates:
                    v = v * gates[0]
                got["out"] = x = s["skip"] * x + s["scale"] * v
                x = x.to(_T[case["xt"]]).double()  # the norm is of the stream as it is stored
            stats[0] = 1 / torch.sqrt((x ** 2).sum(1) / d + _EPS)
            got["n"], got["stats"] = x * stats[0][:, None] * s["w"].double(), stats
            if case["keep"] and not case["f"]:
                got["kept"] = _exact_checkpoint(s["x"])
            return got
        out = s["out"].double() if s["out"] is not None else _exact_rows(*s["out_kept"])
        r, dn, w = s["stats"][0].double()[:, None], s["dn"].double(), s["w"].double()
        inner = (w * dn * out).sum(1, keepdim=True) / d
        dO = s["dout"].double() + r * w * dn - r ** 3 * inner * out
        got = {"dx": s["skip"] * dO, "dw": (dn * out * r).sum(0)}
        if case["f"]:
            f = s["fr"].double() if s["fr"] is not None else _exact_rows(*s["fr_kept"])
            p = s["scale"] * dO if gates is None else s["scale"] * dO * gates[0]
            if case["norm_f"]:
                rf, wa = s["stats"][1].double()[:, None], s["w_after"].double()
                inner = (wa * p * f).sum(1, keepdim=True) / d
                got["df"], got["dw_after"] = rf * wa * p - rf ** 3 * inner * f, (p * f * rf).sum(0)
                f = f * rf * wa
            else:
                got["df"] = p
            if gates:
                dz = s["scale"] * gates[1] * f * dO
                if case["span"] == 1:
                    got["dz"] = dz
                else:
                    got["dz"] = torch.stack([t.sum(0) for t in dz.split(case["span"])])
        return got
    x, wg, wu = s["x"].double(), s["w_gate"].double(), s["w_up"].double()
    if case["op"] == "gated" or s["tape"] is None:
        g, u = x @ wg.T, x @ wu.T
    else:
        g, u = (_exact_rows(s["tape"][0][i], s["tape"][1][i]) for i in (0, 1))
    if case["kind"] == "silu":
        sig = 1 / (1 + torch.exp(-g))
        a, slope = g * sig, sig + g * (sig - sig ** 2)
    else:  # 0.5 g (1 + tanh y) = g sigmoid(2 y)
        y = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        sig = 1 / (1 + torch.exp(-2 * y))
        a, slope = g * sig, sig + 2 * g * (sig - sig ** 2) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    if case["op"] == "gated":
        return {"h": a * u}
    dh = s["dh"].double()
    dg, du = dh * u * slope, dh * a
    return {"dx": dg @ wg + du @ wu, "dw_gate": dg.T @ x, "dw_up": du.T @ x}
