"""The measured cases of the low-rank adapters and of the token routing.

Operators, by a case's "op":

  adapters            y += scale_e (x A_e^T) B_e^T, rows of many requests, each
                      with its own adapter e (or none), beside a projection
                      whose result y already holds
  adapters_backward   the gradients of the rows, and of every adapter
  dispatch            tokens sorted by expert and their rows laid out in that
                      order
  combine             the experts' rows weighted and summed back into tokens
  combine_backward    the gradients of the experts' rows and of the weights

`run` computes a case in its plain form, or, where `own` is set, by the calls
of this package.
"""
import math

import numpy as np
import torch

own = False

_T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one request that decodes alone: one row, a short adapter; latency
        dict(name="adapters_decode_1", op="adapters", M=1, d_in=2048, d_out=2048, r=8, E=4, act="f32", wt="f32",
             rows="tokens", none=0.0),
        # a serving step: 64 requests decode together, 32 adapters kept in f16
        dict(name="adapters_decode_64", op="adapters", M=64, d_in=4096, d_out=4096, r=16, E=32, act="f32", wt="f16",
             rows="tokens", none=0.1),
        # prompts of several requests through an MLP up-projection
        dict(name="adapters_prefill_8192", op="adapters", M=8192, d_in=4096, d_out=12288, r=64, E=8, act="f32",
             wt="f32", rows="runs", none=0.1),
        # a short ragged batch of a fine-tuning step in f16, five adapters trained at once
        dict(name="adapters_train_300", op="adapters_backward", M=300, d_in=2048, d_out=2048, r=24, E=5, act="f16",
             wt="f16", rows="runs", none=0.0),
        # the attention-projection shape, 8 x 1024 tokens, trained in f32
        dict(name="adapters_train_8192", op="adapters_backward", M=8192, d_in=4096, d_out=4096, r=16, E=8, act="f32",
             wt="f32", rows="runs", none=0.0),
        # the largest layer, ragged tokens, bf16
        dict(name="adapters_train_30000", op="adapters_backward", M=30000, d_in=5120, d_out=17408, r=64, E=16,
             act="bf16", wt="bf16", rows="runs", none=0.05),
        # a decoding step's tokens to two of eight experts; latency
        dict(name="dispatch_64", op="dispatch", T=64, k=2, E=8, d=2048, act="f32", none=0.0),
        # a batch of prompts to eight of 128 experts
        dict(name="dispatch_8192", op="dispatch", T=8192, k=8, E=128, d=4096, act="bf16", none=0.0),
        # 2048 tokens back from two of 16 experts, some pairs dropped at an expert's capacity
        dict(name="combine_2048", op="combine", T=2048, k=2, E=16, d=2048, act="f32", none=0.05),
        # the largest batch back from four of 64 experts
        dict(name="combine_30000", op="combine", T=30000, k=4, E=64, d=5120, act="bf16", none=0.0),
        # gradients of an odd, short batch in f16
        dict(name="combine_backward_333", op="combine_backward", T=333, k=3, E=16, d=2048, act="f16", none=0.1),
        # gradients of a training batch, eight of 128 experts
        dict(name="combine_backward_8192", op="combine_backward", T=8192, k=8, E=128, d=4096, act="f32", none=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "adapters_backward", "adapters_backward", "dispatch", "combine",
                     "combine_backward"])
    none = rng.choice([0.0, 0.0, 0.05, 0.3])
    if op.startswith("adapters"):
        act, wt = rng.choice([("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
        rows = rng.choice(["tokens", "runs"])
        return dict(op=op, M=_log(rng, 1, 8192), d_in=128 * _log(rng, 2, 64), d_out=128 * _log(rng, 2, 64),
                    r=8 * _log(rng, 1, 8), E=_log(rng, 1, 32), act=act, wt=wt, rows=rows, none=none)
    k = rng.choice([1, 2, 3, 4, 6, 8])
    return dict(op=op, T=_log(rng, 1, 8192), k=k, E=max(k, _log(rng, 2, 256)), d=8 * _log(rng, 16, 512),
                act=rng.choice(["f32", "f16", "bf16"]), none=none)


# ----------------------------------------------------------------- inputs --
def _adapter_ids(c, rng):
    """The adapter of each row, -1 for none. "tokens": every row a request of
    its own, the first adapters asked for most; "runs": requests of several
    rows one after another."""
    M, E = c["M"], c["E"]
    p = 1.0 / (1.0 + np.arange(E))
    p /= p.sum()
    if c["rows"] == "tokens":
        ids = rng.choice(E, size=M, p=p)
        return np.where(rng.random(M) < c["none"], -1, ids).astype(np.int32)
    n = max(1, min(M, 2 * E))
    cuts = np.sort(rng.integers(0, M + 1, size=n - 1))
    of = rng.permutation(n) % E
    of = np.where(rng.random(n) < c["none"], -1, of)
    return np.repeat(of, np.diff(np.concatenate([[0], cuts, [M]]))).astype(np.int32)


def _plan(ids, E):
    """offsets [E+1], order and its inverse (in the ids' shape): stable by id, rows without one last."""
    key = torch.where((ids < 0) | (ids >= E), E, ids).reshape(-1).long()
    order = torch.sort(key, stable=True).indices
    slot = torch.empty_like(order)
    slot[order] = torch.arange(order.numel(), device=ids.device)
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=ids.device))
    return offsets.int(), order.int(), slot.int().view(ids.shape)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, sigma, t):
        return torch.randn(shape, generator=g, device="cuda").mul_(sigma).to(_T[t])

    s = dict(case)
    if case["op"].startswith("adapters"):
        M, d_in, d_out, r, E, act = (case[k] for k in ("M", "d_in", "d_out", "r", "E", "act"))
        s["ids"] = torch.from_numpy(_adapter_ids(case, rng)).cuda()
        s["offsets"], s["order"], _ = _plan(s["ids"], E)
        s["x"] = normal((M, d_in), 1.0, act)
        s["down"] = normal((E, r, d_in), d_in ** -0.5, case["wt"])
        s["up"] = normal((E, d_out, r), r ** -0.5, case["wt"])
        s["scale"] = torch.from_numpy(rng.uniform(0.25, 2.0, E).astype(np.float32)).cuda()
        if case["op"] == "adapters":
            s["y"] = normal((M, d_out), 1.0, act)  # the shared projection's result
        else:
            s["dy"] = normal((M, d_out), 1e-2, act)
            s["tape"] = _pick(s["x"].float() @ s["down"].float().flatten(0, 1).T, s["ids"], E).sum(1)  # the forward's
        return s
    T, k, E, d, act = (case[q] for q in ("T", "k", "E", "d", "act"))
    # top k of skewed random scores, softmax of their values as weights
    scores = torch.randn((T, E), generator=g, device="cuda") - 0.5 * torch.log(1.0 + torch.arange(E, device="cuda"))
    top = torch.topk(scores, k, dim=1)
    s["weights"] = torch.softmax(top.values, 1)
    drop = torch.rand((T, k), generator=g, device="cuda") < case["none"]
    s["ids"] = torch.where(drop, -1, top.indices).int()
    if case["op"] == "dispatch":
        s["x"] = normal((T, d), 1.0, act)
        return s
    s["offsets"], _, s["slot"] = _plan(s["ids"], E)
    s["z"] = normal((T * k, d), 1.0, act)
    if case["op"] == "combine_backward":
        s["dy"] = normal((T, d), 1e-2, act)
    return s


# ----------------------------------------------------------------- passes --
def _pick(s, ids, E):
    """[M][E r] -> [M][E][r] with every adapter's columns but the row's own at zero."""
    s = s.view(s.shape[0], E, -1)
    return torch.where(torch.arange(E, device=s.device)[None, :, None] == ids[:, None, None], s, 0.0)


def _plain(s):
    if s["op"].startswith("adapters"):
        ids, E, r = s["ids"], s["E"], s["r"]
        x, A = s["x"].float(), s["down"].float().flatten(0, 1)            # [E r][d_in]
        B = s["up"].float().permute(1, 0, 2).flatten(1)                    # [d_out][E r]
        if s["op"] == "adapters":
            h = _pick(x @ A.T, ids, E)
            s["y"].copy_(s["y"].float() + (h * s["scale"][:, None]).flatten(1) @ B.T)
            return {"y": s["y"], "tape": h.sum(1)}
        dy = s["dy"].float()
        ds = _pick(dy @ B, ids, E) * s["scale"][:, None]
        h = _pick(s["tape"].repeat(1, E), ids, E) * s["scale"][:, None]
        ds, h = ds.flatten(1), h.flatten(1)
        return {"dx": (ds @ A).to(s["x"].dtype), "grad_down": (ds.T @ x).view(E, r, -1),
                "grad_up": (dy.T @ h).view(-1, E, r).permute(1, 0, 2).contiguous()}
    if s["op"] == "dispatch":
        offsets, order, slot = _plan(s["ids"], s["E"])
        placed = torch.arange(order.numel(), device=order.device) < offsets[-1]
        rows = s["x"][(order // s["k"]).long()]
        return {"offsets": offsets, "order": order, "slot": slot, "rows": torch.where(placed[:, None], rows, 0)}
    slot = s["slot"].long()                                                # [T][k]
    placed = slot < s["offsets"][-1]
    w = torch.where(placed, s["weights"], 0.0)
    z = s["z"][slot].float()                                               # [T][k][d]
    if s["op"] == "combine":
        return {"y": (z * w[:, :, None]).sum(1).to(s["z"].dtype)}
    dy = s["dy"].float()[:, None, :]
    dz = torch.empty_like(s["z"])
    dz[slot.view(-1)] = (dy * w[:, :, None]).flatten(0, 1).to(dz.dtype)
    return {"dz": dz, "dw": torch.where(placed, (z * dy).sum(2), 0.0)}


def _own(s):
    import binary_rank_linear_amd as blr

    if "kept" not in s:  # the buffers that a program keeps over its steps
        s["kept"] = {}
        if s["op"].startswith("adapters"):
            s["kept"]["ws"] = blr.workspace_adapters(s["M"], s["d_in"], s["d_out"], s["r"], s["E"])
    kept = s["kept"]
    if s["op"] == "adapters":
        y, tape = blr.blr_adapters_forward(s["x"], s["down"], s["up"], s["offsets"], s["order"], s["scale"], y=s["y"],
                                           accumulate_y=True, keep_tape=True, **kept)
        return {"y": y, "tape": tape}
    if s["op"] == "adapters_backward":
        gd, gu, dx = blr.blr_adapters_backward(s["x"], s["dy"], s["down"], s["up"], s["offsets"], s["order"],
                                               s["scale"], s["tape"], **kept)
        return {"dx": dx, "grad_down": gd, "grad_up": gu}
    if s["op"] == "dispatch":
        offsets, order, slot = blr.blr_route_sort(s["ids"], s["E"])
        return {"offsets": offsets, "order": order, "slot": slot,
                "rows": blr.blr_route_gather(s["x"], offsets, slot)}
    if s["op"] == "combine":
        return {"y": blr.blr_route_combine(s["z"], s["offsets"], s["slot"], s["weights"])}
    dz, dw = blr.blr_route_combine_backward(s["dy"], s["z"], s["offsets"], s["slot"], s["weights"])
    return {"dz": dz, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- what a pass needs --
def work(case):
    c, a = case, _SIZE[case["act"]]
    if c["op"].startswith("adapters"):
        M, r, width = c["M"] * (1.0 - c["none"]), c["r"], c["d_in"] + c["d_out"]
        used = min(c["E"], c["M"])
        weights = used * r * width * _SIZE[c["wt"]]
        if c["op"] == "adapters":  # x, y read and written, the tape
            return {"bytes": M * (c["d_in"] + 2 * c["d_out"]) * a + weights + 4 * M * r, "flops": 2 * M * r * width}
        return {"bytes": M * (2 * c["d_in"] + c["d_out"]) * a + weights + 4 * M * r + 4 * c["E"] * r * width,
                "flops": 4 * M * r * width}
    P, d = c["T"] * c["k"], c["d"]
    if c["op"] == "dispatch":  # ids, order and slot; x, and a row for each pair
        return {"bytes": 12 * P + (c["T"] + P) * d * a, "flops": 0}
    if c["op"] == "combine":
        return {"bytes": 8 * P + (c["T"] + P) * d * a, "flops": 2 * P * d}
    return {"bytes": 12 * P + (c["T"] + 2 * P) * d * a, "flops": 3 * P * d}


# ---------------------------------------------------------------- 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("adapters"):
        x, ids = s["x"].double(), s["ids"]
        first = s["y"] if case["op"] == "adapters" else s["dy"]
        first = first.double()
        tape = torch.zeros((case["M"], case["r"]), dtype=torch.float64, device="cuda")
        dx = torch.zeros_like(x)
        gd, gu = torch.zeros_like(s["down"], dtype=torch.float64), torch.zeros_like(s["up"], dtype=torch.float64)
        for e in range(case["E"]):
            rows = torch.nonzero(ids == e).flatten()
            if rows.numel() == 0:
                continue
            c, A, B, xe = float(s["scale"][e]), s["down"][e].double(), s["up"][e].double(), x[rows]
            if case["op"] == "adapters":
                tape[rows] = xe @ A.T
                first[rows] += c * (tape[rows] @ B.T)
            else:
                ds = c * (first[rows] @ B)
                dx[rows] = ds @ A
                gd[e] = ds.T @ xe
                gu[e] = c * (first[rows].T @ s["tape"][rows].double())
        if case["op"] == "adapters":
            return {"y": first, "tape": tape}
        return {"dx": dx, "grad_down": gd, "grad_up": gu}
    T, k, E, d = (case[q] for q in ("T", "k", "E", "d"))
    ids = s["ids"].cpu().numpy().reshape(-1)
    key = np.where(ids < 0, E, ids)
    order = np.lexsort((np.arange(T * k), key))
    slot = np.argsort(order)
    n = int((key < E).sum())
    if case["op"] == "dispatch":
        rows = torch.zeros((T * k, d), dtype=torch.float64, device="cuda")
        rows[:n] = s["x"].double()[torch.from_numpy(order[:n] // k).cuda()]
        count = np.bincount(key, minlength=E + 1)
        return {"offsets": torch.from_numpy(np.concatenate([[0], np.cumsum(count[:E])]).astype(np.int32)),
                "order": torch.from_numpy(order.astype(np.int32)),
                "slot": torch.from_numpy(slot.reshape(T, k).astype(np.int32)),
                "rows": rows}
    y = torch.zeros((T, d), dtype=torch.float64, device="cuda")
    dz = torch.zeros((T * k, d), dtype=torch.float64, device="cuda")
    dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        at = slot.reshape(T, k)[:, j]
        t = torch.from_numpy(np.nonzero(at < n)[0]).cuda()
        at = torch.from_numpy(at).cuda()[t]
        w = s["weights"][t, j].double()[:, None]
        if case["op"] == "combine":
            y[t] += w * s["z"][at].double()
        else:
            dy = s["dy"][t].double()
            dz[at] = w * dy
            dw[t, j] = (dy * s["z"][at].double()).sum(1)
    return {"y": y} if case["op"] == "combine" else {"dz": dz, "dw": dw}
