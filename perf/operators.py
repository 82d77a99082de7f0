"""The operators that stand around the sparse MoE layer in a decoder block, as measured cases.

  norm          h_out = res_scale h + block_scale g * N(y),  x = N(h_out): the residual step after a
                block fused with its gate and scales, the optional norm of the block's output before
                it and the norm that feeds the next block behind it; y absent: the norm before a
                block alone. N(v) = v / sqrt(mean v^2 + eps) * (w_offset + w).
  norm_grad     its gradients: h, y, gate and both weights.
  balance       per-expert counts, mean probabilities, balance loss and z loss of a router's rows.
  balance_grad  the gradient of both losses with respect to the logits.
  gemv          y = x W^T for 1..32 rows of x and a W in the int4 group-32 format.

`run` computes a case in plain torch operations, or with the library's kernels where `own` is true.
`exact` computes it in 64 bits.
"""

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-6


# ---------------------------------------------------------------------------- cases
def _norm(name, op, T, H, h="bf16", y="f32", x="bf16", w="bf16", post=False, gate="none", act="linear", gdt="bf16",
          offset=0.0, res=1.0, block=1.0, branch=True):
    # branch False: the norm before a block alone (no block output, gate or residual step)
    return dict(name=name, op=op, T=T, H=H, h=h, y=y, x=x, w=w, post=post and branch, gate=gate if branch else "none",
                act=act, gdt=gdt, offset=offset, res=res, block=block, branch=branch)


def listed():
    return [
        # one decode token between two MoE layers of the Qwen3-Next width: add the layer's output
        # to the residual stream and normalise for the next block (the smallest call: latency)
        _norm("norm_decode_t1", "norm", 1, 2048),
        # a 2048-token prompt chunk, the block's output normalised and scaled per channel
        _norm("norm_chunk_t2048", "norm", 2048, 2048, post=True, gate="channel", offset=1.0),
        # a long batch of a wider model, fp32 residual stream, element gate behind a sigmoid
        _norm("norm_wide_gated", "norm", 8191, 5120, h="f32", y="bf16", post=True, gate="element", act="sigmoid",
              res=0.9, block=0.5),
        # gradients of a small odd layer in fp32, token gate
        _norm("norm_grad_small", "norm_grad", 37, 264, h="f32", y="f32", x="f32", w="f32", post=True, gate="token",
              act="sigmoid", gdt="f32", block=0.25),
        # a training batch in bf16 with a norm on both sides and a per-channel gate
        _norm("norm_grad_batch", "norm_grad", 8192, 2048, y="bf16", post=True, gate="channel"),
        # router statistics of one 2048-token chunk
        dict(name="balance_chunk", op="balance", T=2048, E=512, k=10, dtype="f32", masked=0.0),
        # a large training batch, part of it padding
        dict(name="balance_batch", op="balance", T=65521, E=512, k=10, dtype="f32", masked=0.2),
        # a few tokens through a small router of odd width
        dict(name="balance_grad_small", op="balance_grad", T=33, E=61, k=4, dtype="f32", masked=0.1),
        # the training batch's gradient from bf16 logits
        dict(name="balance_grad_batch", op="balance_grad", T=32768, E=512, k=10, dtype="bf16", masked=0.2),
        # one token through a projection of the expert's size
        dict(name="gemv_small_t1", op="gemv", T=1, N=512, K=2048, out="f32"),
        # one token through the vocabulary head (weights larger than L2)
        dict(name="gemv_head_t1", op="gemv", T=1, N=151936, K=2048, out="f32"),
        # a small decode batch through a wide projection, ragged rows and bf16 results
        dict(name="gemv_rows_t13", op="gemv", T=13, N=24571, K=4096, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "balance", "balance_grad", "gemv"])
    if op in ("norm", "norm_grad"):
        H = 8 * _log(rng, 16, 1024)
        top = (40 << 20) if op == "norm" else (16 << 20)
        c = _norm("", op, _log(rng, 1, min(16384, top // H)), H, h=rng.choice(["f32", "bf16"]),
                  y=rng.choice(["f32", "bf16"]), x=rng.choice(["f32", "bf16"]), w=rng.choice(["f32", "bf16"]),
                  post=rng.random() < 0.5, gate=rng.choice(["none", "token", "channel", "element"]),
                  act=rng.choice(["linear", "sigmoid"]), gdt=rng.choice(["f32", "bf16"]),
                  offset=rng.choice([0.0, 1.0]), res=rng.choice([1.0, 0.9]), block=rng.choice([1.0, 0.25]),
                  branch=rng.random() < 0.85)
        del c["name"]
        return c
    if op in ("balance", "balance_grad"):
        E = _log(rng, 2, 1024)
        top = (33 << 20) if op == "balance" else (16 << 20)
        return dict(op=op, T=_log(rng, 1, min(65536, top // E)), E=E, k=rng.randint(1, min(E, 16)),
                    dtype=rng.choice(["f32", "bf16"]), masked=rng.choice([0.0, 0.1, 0.5]))
    N, K, T = _log(rng, 16, 65536), 32 * _log(rng, 2, 256), rng.choice([1, 1, 2, 3, 4, 7, 8, 13, 16, 21, 32])
    return dict(op="gemv", T=T, N=min(N, (256 << 20) // K), K=K, out=rng.choice(["f32", "bf16"]))


# ---------------------------------------------------------------------------- inputs
def _randn(g, *shape, dtype="f32"):
    return torch.randn(*shape, generator=g, device="cuda").to(DT[dtype])


def _prepare_norm(c, g):
    T, H = c["T"], c["H"]
    s = {"h": _randn(g, T, H, dtype=c["h"])}
    s["y"] = (0.5 * _randn(g, T, H)).to(DT[c["y"]]) if c["branch"] else None
    # weights near the value a trained norm has: 1 in all (w_offset included)
    s["pre_w"] = (1.0 - c["offset"] + 0.1 * _randn(g, H)).to(DT[c["w"]])
    s["post_w"] = (1.0 - c["offset"] + 0.1 * _randn(g, H)).to(DT[c["w"]]) if c["post"] else None
    gshape = {"none": None, "token": (T,), "channel": (H,), "element": (T, H)}[c["gate"]]
    s["gate"] = None if gshape is None else _randn(g, *gshape, dtype=c["gdt"])
    if c["op"] == "norm":
        s["h_out"] = torch.empty_like(s["h"]) if c["branch"] else None
        s["x"] = torch.empty(T, H, device="cuda", dtype=DT[c["x"]])
    else:  # the residual stream that the forward pass left, and the gradients that arrive
        s["h_out"] = s.pop("h")
        s["dh_out"] = _randn(g, T, H, dtype=c["h"])
        s["dx"] = _randn(g, T, H, dtype=c["x"])
        s["dh"] = torch.empty_like(s["dh_out"])
        s["dy"] = torch.empty_like(s["y"]) if c["branch"] else None
        s["dpre_w"] = torch.empty(H, device="cuda")
        s["dpost_w"] = torch.empty(H, device="cuda") if c["post"] else None
        s["dgate"] = None
        if gshape is not None:
            s["dgate"] = torch.empty(gshape, device="cuda", dtype=DT[c["gdt"]] if c["gate"] == "element" else DT["f32"])
    if own:
        import sparse_moe_gemv_b200 as smg
        s["norm"] = smg.Norm(H, h_dtype=c["h"], y_dtype=c["y"], x_dtype=c["x"], pre_w=s["pre_w"], post_w=s["post_w"],
                             post_norm=c["post"], gate=c["gate"], gate_act=c["act"], gate_dtype=c["gdt"], eps=EPS,
                             w_offset=c["offset"], res_scale=c["res"], block_scale=c["block"])
        s["workspace"] = smg.new_norm_workspace(s["norm"], T) if c["op"] == "norm_grad" else None
    return s


def _prepare_balance(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    # router logits with a power-law preference for some experts
    pref = -1.1 * torch.log(1.0 + torch.randperm(E, generator=g, device="cuda").float())
    logits = (_randn(g, T, E) + pref - pref.mean()).to(DT[c["dtype"]])
    ids = logits.float().topk(k, dim=1).indices.to(torch.int32)
    mask = None
    if c["masked"]:
        mask = (torch.rand(T, generator=g, device="cuda") >= c["masked"]).to(torch.uint8)
        # what padding rows hold is anything: no number, infinities, no expert
        pad = torch.nonzero(mask == 0)[:, 0]
        logits[pad] = float("nan")
        logits[pad[::3]] = float("inf")
        ids[pad] = -1
    s = {"logits": logits, "mask": mask, "k": k}
    if c["op"] == "balance":
        s["ids"] = ids
        s["loss"] = torch.empty(2, device="cuda")
        s["counts"] = torch.empty(E, device="cuda", dtype=torch.int32)
        s["prob"] = torch.empty(E, device="cuda")
        s["n_rows"] = torch.empty(1, device="cuda", dtype=torch.int32)
        if own:
            import sparse_moe_gemv_b200 as smg
            s["workspace"] = smg.new_balance_workspace(T, E)
    else:
        live = ids.long().clamp(min=0)
        s["counts"] = torch.zeros(E, device="cuda", dtype=torch.int32).index_add_(
            0, live.reshape(-1), (ids >= 0).reshape(-1).to(torch.int32))
        s["n_rows"] = (ids[:, :1] >= 0).sum(0, dtype=torch.int32)
        s["grad_loss"] = torch.tensor([0.01, 0.001], device="cuda") * (0.5 + torch.rand(2, generator=g, device="cuda"))
        s["dlogits"] = torch.empty_like(logits)
    return s


def _prepare_gemv(c, g):
    N, K = c["N"], c["K"]
    w = torch.empty(N, K // 2, device="cuda", dtype=torch.uint8)
    sc = torch.empty(N, K // 32, device="cuda", dtype=torch.bfloat16)
    for a in range(0, N, 32768):  # weights drawn and quantised in slices: bounded temporaries
        b = min(N, a + 32768)
        v = (0.02 * _randn(g, b - a, K)).reshape(b - a, K // 32, 32)
        sc[a:b] = (v.abs().amax(-1) / 7.0).to(torch.bfloat16)
        f = sc[a:b].float().unsqueeze(-1)
        q = (torch.round(v / torch.where(f == 0, torch.ones_like(f), f)).clamp(-7, 7) + 8).to(torch.uint8).reshape(b - a, K)
        w[a:b] = q[:, 0::2] | (q[:, 1::2] << 4)
    s = {"w": w, "s": sc, "x": _randn(g, c["T"], K, dtype="bf16"),
         "y": torch.empty(c["T"], N, device="cuda", dtype=DT[c["out"]])}
    if own:
        import sparse_moe_gemv_b200 as smg
        s["matrix"] = smg.Matrix(w, sc, rows=N, cols=K, dtype="int4g32")
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = (_prepare_norm if op.startswith("norm") else _prepare_balance if op.startswith("balance") else _prepare_gemv)(case, g)
    s["case"] = dict(case)
    return s


# ---------------------------------------------------------------------------- plain forms
def _gate_of(s, c, T, H):
    """The gate's value, shaped to broadcast over [T, H], and its derivative; fp32."""
    if c["gate"] == "none":
        return None, None
    a = s["gate"].float()
    a = a.reshape(T, 1) if c["gate"] == "token" else a
    if c["act"] == "linear":
        return a, torch.ones_like(a)
    v = 1.0 / (1.0 + torch.exp(-a))
    return v, v * (1.0 - v)


def _plain_norm(s, c):
    t, out = s["h"].float(), {}
    if c["branch"]:
        t = _plain_residual(s, c, t)
        out["h_out"] = t.to(DT[c["h"]])
    x = t * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS) * (c["offset"] + s["pre_w"].float())
    out["x"] = x.to(DT[c["x"]])
    return out


def _plain_residual(s, c, h):
    u = s["y"].float()
    if c["post"]:
        u = u * torch.rsqrt((u * u).mean(1, keepdim=True) + EPS) * (c["offset"] + s["post_w"].float())
    v, _ = _gate_of(s, c, c["T"], c["H"])
    if v is not None:
        u = v * u
    return c["res"] * h + c["block"] * u


def _plain_norm_grad(s, c):
    t, dx = s["h_out"].float(), s["dx"].float()
    r2 = torch.rsqrt((t * t).mean(1, keepdim=True) + EPS)
    a = dx * (c["offset"] + s["pre_w"].float())
    G = s["dh_out"].float() + r2 * (a - t * (r2 * r2 * (a * t).mean(1, keepdim=True)))
    out = {"dpre_w": (dx * t * r2).sum(0)}
    if not c["branch"]:
        out["dh"] = G.to(DT[c["h"]])
        return out
    out["dh"] = (c["res"] * G).to(DT[c["h"]])
    u = y = s["y"].float()
    if c["post"]:
        r1 = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        w1 = c["offset"] + s["post_w"].float()
        u = y * r1 * w1
    v, dv = _gate_of(s, c, c["T"], c["H"])
    du = c["block"] * G
    if v is not None:
        dg = du * u * dv
        out["dgate"] = (dg.sum(1) if c["gate"] == "token" else dg.sum(0) if c["gate"] == "channel" else dg.to(DT[c["gdt"]]))
        du = du * v
    if c["post"]:
        out["dpost_w"] = (du * y * r1).sum(0)
        a = du * w1
        du = r1 * (a - y * (r1 * r1 * (a * y).mean(1, keepdim=True)))
    out["dy"] = du.to(DT[c["y"]])
    return out


def _plain_probs(s):
    """Probabilities and log-sum-exp of the rows that count (others: zero), and that choice of rows."""
    l = s["logits"].float()
    top = l.amax(1, keepdim=True)
    live = top != -math.inf  # a row that allows no expert does not count
    if s["mask"] is not None:
        live = live & (s["mask"] != 0).unsqueeze(1)
    l = torch.where(live, l, torch.zeros_like(l))
    top = torch.where(live, top, torch.zeros_like(top))
    e = torch.exp(l - top)
    z = e.sum(1, keepdim=True)
    zero = torch.zeros_like(z)
    return torch.where(live, e / z, zero), torch.where(live, top + torch.log(z), zero), live


def _plain_balance(s, c):
    p, lse, live = _plain_probs(s)
    E, k = c["E"], c["k"]
    ids = torch.where(live, s["ids"].long(), torch.full_like(s["ids"], -1, dtype=torch.int64))
    ok = (ids >= 0) & (ids < E)
    counts = torch.zeros(E, device=ids.device, dtype=torch.int32).index_add_(
        0, torch.where(ok, ids, torch.zeros_like(ids)).reshape(-1), ok.reshape(-1).to(torch.int32))
    n = live.sum(dtype=torch.int32)
    nf = n.clamp(min=1).float()
    prob = p.sum(0) / nf
    balance = E * (counts.float() / (nf * k) * prob).sum()
    return {"loss": torch.stack([balance, (lse * lse).sum() / nf]), "counts": counts, "prob": prob, "n_rows": n.reshape(1)}


def _plain_balance_grad(s, c):
    p, lse, live = _plain_probs(s)
    nf = s["n_rows"].clamp(min=1).float()
    f = s["counts"].float()
    gb, gz = s["grad_loss"][0], s["grad_loss"][1]
    d = p * (f - (p * f).sum(1, keepdim=True)) * (gb * c["E"] / (nf * nf * c["k"])) + p * lse * (2.0 * gz / nf)
    return {"dlogits": d.to(DT[c["dtype"]])}


def _plain_gemv(s, c):
    w = s["w"]
    q = torch.stack((w & 15, w >> 4), dim=-1).reshape(c["N"], c["K"] // 32, 32).float() - 8.0
    q = (q * s["s"].float().unsqueeze(-1)).reshape(c["N"], c["K"])
    return {"y": (s["x"].float() @ q.t()).to(DT[c["out"]])}


PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "balance": _plain_balance,
         "balance_grad": _plain_balance_grad, "gemv": _plain_gemv}


# ---------------------------------------------------------------------------- one pass
def _own(s, c):
    import sparse_moe_gemv_b200 as smg
    op = c["op"]
    if op == "norm":
        smg.redmoe_norm_forward(s["norm"], s["h"], h_out=s["h_out"], x=s["x"], y=s["y"], gate=s["gate"])
        return {n: s[n] for n in ("h_out", "x") if s[n] is not None}
    if op == "norm_grad":
        smg.redmoe_norm_backward(s["norm"], s["h_out"], s["dh"], s["workspace"], dh_out=s["dh_out"], dx=s["dx"],
                                 y=s["y"], gate=s["gate"], dy=s["dy"], dgate=s["dgate"], dpost_w=s["dpost_w"],
                                 dpre_w=s["dpre_w"])
        return {n: s[n] for n in ("dh", "dy", "dgate", "dpost_w", "dpre_w") if s[n] is not None}
    if op == "balance":
        smg.redmoe_balance_forward(s["logits"], s["ids"], s["loss"], s["counts"], s["prob"], s["n_rows"],
                                   s["workspace"], mask=s["mask"])
        return {n: s[n] for n in ("loss", "counts", "prob", "n_rows")}
    if op == "balance_grad":
        smg.redmoe_balance_backward(s["logits"], s["counts"], s["n_rows"], s["grad_loss"], s["dlogits"], s["k"],
                                    mask=s["mask"])
        return {"dlogits": s["dlogits"]}
    smg.redmoe_gemv(s["matrix"], s["x"], s["y"])
    return {"y": s["y"]}


def run(state):
    c = state["case"]
    return _own(state, c) if own else PLAIN[c["op"]](state, c)


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c, op = case, case["op"]
    if op == "norm" or op == "norm_grad":
        n, H = c["T"] * c["H"], c["H"]
        gn = {"none": 0, "token": c["T"], "channel": H, "element": n}[c["gate"]]
        weights = H * SIZE[c["w"]] * (2 if c["post"] else 1)
        if not c["branch"]:
            grad = op == "norm_grad"
            return {"bytes": n * (SIZE[c["h"]] * (3 if grad else 1) + SIZE[c["x"]]) + weights + (4 * H if grad else 0),
                    "flops": n * (12.0 if grad else 4.0)}
        if op == "norm":
            return {"bytes": n * (2 * SIZE[c["h"]] + SIZE[c["y"]] + SIZE[c["x"]]) + gn * SIZE[c["gdt"]] + weights,
                    "flops": n * 12.0}
        gout = gn * (SIZE[c["gdt"]] if c["gate"] == "element" else 4)
        return {"bytes": n * (3 * SIZE[c["h"]] + 2 * SIZE[c["y"]] + SIZE[c["x"]]) + gn * SIZE[c["gdt"]] + gout + weights
                + 4 * H * (2 if c["post"] else 1), "flops": n * 30.0}
    if op == "balance" or op == "balance_grad":
        live = c["T"] * (1.0 - c["masked"])  # padding rows need not be read
        n = live * c["E"]
        rows = c["T"] if c["masked"] else 0
        if op == "balance":
            return {"bytes": n * SIZE[c["dtype"]] + 4.0 * live * c["k"] + rows + 8.0 * c["E"] + 12, "flops": n * 6.0}
        return {"bytes": (n + c["T"] * c["E"]) * SIZE[c["dtype"]] + rows + 4.0 * c["E"] + 12, "flops": n * 10.0}
    N, K, T = c["N"], c["K"], c["T"]
    return {"bytes": N * K * 0.5 + N * (K // 32) * 2.0 + 2.0 * T * K + SIZE[c["out"]] * T * N, "flops": 2.0 * N * K * T}


# ---------------------------------------------------------------------------- the definition in 64 bits
def _exact_scale(v):
    """1 / sqrt(mean v^2 + eps) of each row."""
    return 1.0 / torch.sqrt(torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / v.shape[1] + EPS)


def _exact_gate(s, c):
    if s["gate"] is None:
        return torch.ones(1, 1, device="cuda", dtype=torch.float64), None
    a = s["gate"].double()
    a = a[:, None] if c["gate"] == "token" else a[None, :] if c["gate"] == "channel" else a
    if c["act"] == "sigmoid":
        return torch.sigmoid(a), torch.sigmoid(a) * torch.sigmoid(-a)
    return a, torch.ones_like(a)


def _exact_norm(s, c):
    w = lambda n: s[n].double()[None, :] + c["offset"]  # noqa: E731
    if not c["branch"]:
        t = s["h"].double()
        return {"x": t * _exact_scale(t) * w("pre_w")}
    y = s["y"].double()
    if c["post"]:
        y = y * _exact_scale(y) * w("post_w")
    g, _ = _exact_gate(s, c)
    t = s["h"].double() * c["res"] + y * g * c["block"]
    return {"h_out": t, "x": t * _exact_scale(t) * w("pre_w")}


def _exact_norm_grad(s, c):
    # d(v r w)/dv = r (I - n n^T / H) w with n = v r, applied to the gradient that arrives
    def through(v, d, wt):
        r = _exact_scale(v)
        n = v * r
        dn = d * wt
        return r * (dn - n * torch.linalg.vecdot(n, dn, dim=1)[:, None] / v.shape[1]), torch.einsum("th,th->h", d, n)

    t = s["h_out"].double()
    back, dpre = through(t, s["dx"].double(), s["pre_w"].double()[None, :] + c["offset"])
    total = s["dh_out"].double() + back
    if not c["branch"]:
        return {"dh": total, "dpre_w": dpre}
    y = s["y"].double()
    res = {"dh": total * c["res"], "dpre_w": dpre}
    g, dg = _exact_gate(s, c)
    w1 = s["post_w"].double()[None, :] + c["offset"] if c["post"] else None
    u = y * _exact_scale(y) * w1 if c["post"] else y
    branch = total * c["block"]
    if dg is not None:
        if c["gate"] == "token":
            res["dgate"] = torch.einsum("th,th->t", branch, u) * dg[:, 0]
        elif c["gate"] == "channel":
            res["dgate"] = torch.einsum("th,th->h", branch, u) * dg[0]
        else:
            res["dgate"] = branch * u * dg
    arriving = branch * g
    if c["post"]:
        res["dy"], res["dpost_w"] = through(y, arriving, w1)
    else:
        res["dy"] = arriving.expand(y.shape)
    return res


def _exact_rows(s):
    keep = torch.arange(s["logits"].shape[0], device="cuda")
    if s["mask"] is not None:
        keep = keep[s["mask"].bool()]
    keep = keep[(s["logits"][keep] > -math.inf).any(1) | s["logits"][keep].isnan().any(1)]
    l = s["logits"][keep].double()
    return keep, torch.softmax(l, 1), torch.logsumexp(l, 1)


def _exact_balance(s, c):
    keep, p, lse = _exact_rows(s)
    n, E = keep.numel(), c["E"]
    chosen = s["ids"][keep].long().reshape(-1)
    counts = torch.bincount(chosen, minlength=E)
    prob = p.mean(0) if n else torch.zeros(E, device="cuda", dtype=torch.float64)
    loss = torch.stack([E * torch.dot(counts.double() / max(1, n * c["k"]), prob), (lse ** 2).mean() if n else prob.sum()])
    return {"loss": loss, "counts": counts.to(torch.int32), "prob": prob,
            "n_rows": torch.tensor([n], device="cuda", dtype=torch.int32)}


def _exact_balance_grad(s, c):
    keep, p, lse = _exact_rows(s)
    n = max(1, keep.numel())
    f = s["counts"].double() / (n * c["k"])
    gb, gz = s["grad_loss"].double().tolist()
    d = torch.zeros(c["T"], c["E"], device="cuda", dtype=torch.float64)
    d[keep] = gb * c["E"] / n * p * (f[None, :] - torch.mv(p, f)[:, None]) + gz * 2.0 / n * lse[:, None] * p
    return {"dlogits": d}


def _exact_gemv(s, c):
    x = s["x"].double()
    y = torch.empty(c["T"], c["N"], device="cuda", dtype=torch.float64)
    for a in range(0, c["N"], 8192):
        b = s["w"][a:a + 8192].to(torch.int16)
        q = torch.empty(b.shape[0], c["K"], device="cuda", dtype=torch.float64)
        q[:, 0::2] = (b % 16 - 8).double()
        q[:, 1::2] = (torch.div(b, 16, rounding_mode="floor") - 8).double()
        y[:, a:a + 8192] = x @ (q * s["s"][a:a + 8192].double().repeat_interleave(32, dim=1)).T
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "balance": _exact_balance,
            "balance_grad": _exact_balance_grad, "gemv": _exact_gemv}[op](s, case)
