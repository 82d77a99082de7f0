"""Plain 64-bit forms of the operators around the layer (test helper): values straight from
their definitions and, beside each, the magnitude its rounding errors scale with (the same
expression with every term made positive), from which the tests derive tolerances.

U is the unit roundoff of fp32. A result made of n fp32 operations is off by at most about
n U times its magnitude.
"""

from __future__ import annotations

import torch

U = 2.0 ** -24


def store_tol(value: torch.Tensor, err: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """Bound on a stored result: its computation's error plus half a step of rounding."""
    half = torch.finfo(dtype).eps / 2
    return err * (1 + half) + half * value.abs()


def d(t):
    return None if t is None else t.detach().to("cpu").double()


class NormCase:
    """The step between blocks on fp64 copies of the given tensors."""

    def __init__(self, h=None, y=None, gate=None, pre_w=None, post_w=None, post=False, kind="none", act="linear",
                 eps=1e-6, offset=0.0, res=1.0, block=1.0):
        self.h, self.y, self.gate, self.pre_w, self.post_w = d(h), d(y), d(gate), d(pre_w), d(post_w)
        self.post, self.kind, self.act = post, kind, act
        self.eps, self.offset, self.res, self.block = eps, offset, res, block

    def r(self, v):
        return (v.pow(2).mean(1, keepdim=True) + self.eps).rsqrt()

    def w(self, w):
        return torch.ones(1, dtype=torch.float64) if w is None else self.offset + w

    def act_gate(self):
        if self.kind == "none":
            return torch.ones(1, 1, dtype=torch.float64), torch.zeros(1, 1, dtype=torch.float64)
        a = self.gate[:, None] if self.kind == "token" else self.gate
        if self.act == "linear":
            return a, torch.ones_like(a)
        s = torch.sigmoid(a)
        return s, s * (1 - s)

    def u(self):
        return self.y * self.r(self.y) * self.w(self.post_w) if self.post else self.y

    def forward(self):
        """h_out, x and their magnitudes."""
        if self.y is None:
            t, m = self.h, self.h.abs()
        else:
            b = self.block * self.act_gate()[0] * self.u()
            t = self.res * self.h + b
            m = (self.res * self.h).abs() + b.abs()
        r, w = self.r(t), self.w(self.pre_w)
        x = t * r * w
        # an error of m in h_out moves its scale too: at most by rms(m) / rms(h_out)
        spread = 1 + m.pow(2).mean(1, keepdim=True).sqrt() * r
        return t, x, m, m * r * w.abs() + x.abs() * spread

    def backward(self, dh_out=None, dx=None):
        """{name: (value, magnitude)} at the point h (the stored h_out)."""
        t = self.h
        z = torch.zeros_like(t)
        dho = z if dh_out is None else d(dh_out)
        r2, w2 = self.r(t), self.w(self.pre_w)
        G, mG = dho, dho.abs()
        out = {}
        if dx is not None:
            a = d(dx) * w2
            G = dho + r2 * (a - t * r2 ** 2 * (a * t).mean(1, keepdim=True))
            mG = dho.abs() + r2 * (a.abs() + t.abs() * r2 ** 2 * (a * t).abs().mean(1, keepdim=True))
            out["dpre_w"] = ((d(dx) * t * r2).sum(0), (d(dx) * t * r2).abs().sum(0))
        if self.y is None:
            out["dh"] = (G, mG)
            return out
        out["dh"] = (self.res * G, abs(self.res) * mG)
        g, dg = self.act_gate()
        u = self.u()
        e, me = self.block * G * u * dg, abs(self.block) * mG * u.abs() * dg.abs()
        if self.kind == "token":
            out["dgate"] = (e.sum(1), me.sum(1))
        elif self.kind == "channel":
            out["dgate"] = (e.sum(0), me.sum(0))
        elif self.kind == "element":
            out["dgate"] = (e, me)
        dd, md = self.block * G * g, abs(self.block) * mG * g.abs()
        if not self.post:
            out["dy"] = (dd.expand(t.shape), md.expand(t.shape))
            return out
        y, r1, w1 = self.y, self.r(self.y), self.w(self.post_w)
        out["dpost_w"] = ((dd * y * r1).sum(0), (md * y.abs() * r1).sum(0))
        c, mc = dd * w1, md * w1.abs()
        out["dy"] = (r1 * (c - y * r1 ** 2 * (c * y).mean(1, keepdim=True)),
                     r1 * (mc + y.abs() * r1 ** 2 * (mc * y.abs()).mean(1, keepdim=True)))
        return out


def balance_live(logits, mask=None):
    l = d(logits)
    live = ~(l == -float("inf")).all(1)
    return live if mask is None else live & (mask.cpu() != 0)


def balance_forward(logits, ids, mask=None):
    """loss, counts, prob, n and the magnitudes of both losses (prob's is itself)."""
    l, T, E, k = d(logits), logits.shape[0], logits.shape[1], ids.shape[1]
    live = balance_live(logits, mask)
    n = int(live.sum())
    chosen = ids.cpu()[live].long().reshape(-1)
    chosen = chosen[(chosen >= 0) & (chosen < E)]
    counts = torch.bincount(chosen, minlength=E).to(torch.int32)
    if n == 0:
        z = torch.zeros(2, dtype=torch.float64)
        return z, counts, torch.zeros(E, dtype=torch.float64), 0, z
    l = l[live]
    prob = torch.softmax(l, 1).mean(0)
    top = l.amax(1)
    lse = torch.logsumexp(l, 1)
    loss = torch.stack([E * (counts.double() / (n * k) * prob).sum(), lse.pow(2).mean()])
    # lse = max + log(sum): both enter, and log's argument is off by some U
    mag = torch.stack([loss[0], (2 * lse.abs() * (top.abs() + (lse - top).abs() + 1)).mean()])
    return loss, counts, prob, n, mag


def balance_backward(logits, counts, n, k, grad, mask=None):
    """dlogits and its magnitude."""
    l, E = d(logits), logits.shape[1]
    live = balance_live(logits, mask)
    n = max(n, 1)
    gb, gz = (float(v) for v in grad)
    f = counts.cpu().double()
    out, mag = torch.zeros_like(l), torch.zeros_like(l)
    ll = l[live]
    p, lse, top = torch.softmax(ll, 1), torch.logsumexp(ll, 1, keepdim=True), ll.amax(1, keepdim=True)
    cb, cz = gb * E / (n * n * k), 2 * gz / n
    out[live] = p * (cb * (f - (p * f).sum(1, keepdim=True)) + cz * lse)
    fc = (f - n * k // E).abs()  # the kernel's centred counts
    mag[live] = p * (abs(cb) * (fc + (p * fc).sum(1, keepdim=True)) + abs(cz) * (top.abs() + (lse - top).abs() + 1))
    return out, mag


def gemv_rows(w, s, x, rows=None):
    """x W^T, sum |x W| and sum |x| scale for the int4 group-32 matrix (rows: only those of W)."""
    w, s, x = w.cpu(), s.cpu(), d(x)
    if rows is not None:
        w, s = w[rows], s[rows]
    q = torch.stack(((w & 15).double(), (w >> 4).double()), dim=-1).reshape(w.shape[0], -1) - 8
    S = s.double().repeat_interleave(32, dim=1)
    return x @ (q * S).T, x.abs() @ (q * S).abs().T, x.abs() @ S.abs().T


def gemv_err(m, ms, K):
    """Bound on the kernel's error from sum |x W| and sum |x| scale, in exact arithmetic's place:

    A group's sum starts at -8 X, X the fp32 sum of its 32 x: 8 additions of a lane and two of its
    quad, 10 U sum |x|, so 80 U. Eight tensor-core accumulations follow over nibbles of 0 .. 15; each
    may round or truncate (2 U) a partial sum of at most (8 + 15) sum |x|: 368 U. Then one U for the
    product with the scale and one for each of the K / 32 additions and up to 16 + 3 more (warps,
    lanes), of partial sums of |x W|."""
    return U * (448 * ms + (K / 32 + 20) * (m + 448 * U * ms))
