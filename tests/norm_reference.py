"""The norms around a block in 64 bits, with a bound of what binary32 may be off by.

``Near`` is a value and such a bound, carried along by the rules of a running error
analysis: with u = 2^-24, an operation adds u times its result to what its operands
bring.  Contracted or reordered operations round less often or as often.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24


class Near:
    def __init__(self, v, e=None):
        self.v = v
        self.e = torch.zeros_like(v) if e is None else e

    def _done(self, v, e):
        # (1 + 2^-10: terms of second order in u, over the few operations here)
        return Near(v, (e + U * v.abs()) * (1 + 2.0 ** -10))

    def __add__(self, o):
        return self._done(self.v + o.v, self.e + o.e)

    def __sub__(self, o):
        return self._done(self.v - o.v, self.e + o.e)

    def __mul__(self, o):
        if not isinstance(o, Near):
            return self._done(self.v * o, self.e * abs(o))
        return self._done(self.v * o.v,
                          self.e * o.v.abs() + o.e * self.v.abs() + self.e * o.e)

    def sum(self, dim, steps):
        """A sum in any order in which no term takes part in more than `steps` additions."""
        v = self.v.sum(dim, keepdim=True)
        s = (self.v.abs() + self.e).sum(dim, keepdim=True)
        return self._done(v, self.e.sum(dim, keepdim=True) + steps * U * s)

    def mean(self, steps):
        D = self.v.shape[1]
        t = self.sum(1, steps)
        # times 1 / D, itself rounded
        return self._done(t.v / D, t.e / D + U * (t.v / D).abs())

    def square(self):
        return self * self

    def inverse_root(self, eps):
        """1 / sqrt(self + eps): a sum, a root and a division, each rounded once."""
        v = 1 / (self.v + eps).sqrt()
        low = (self.v - self.e).clamp(min=0) + eps
        return self._done(v, (1 / low.sqrt() - v) + 3 * U * v)

    def rounded(self, dtype):
        """The bound of a store: half a step more (binary16: or half its smallest)."""
        size = self.v.abs() + self.e
        half = torch.finfo(dtype).eps / 2 * size if dtype != torch.float32 else U * size
        return self.e + half + (2.0 ** -25 if dtype == torch.float16 else 0.0) + 2.0 ** -149


def steps_of(D):
    """Additions that a term of a row's sum goes through: 8 elements a lane, or D / 1024 of a
    wide row, 6 steps in a wave and 16 waves."""
    return 32 + D // 1024


def rows(v, M):
    v = v.double()
    if v.dim() == 1:
        return Near(v[None].expand(M, -1))
    return Near(v.repeat_interleave(M // v.shape[0], 0))


def normed(v, kind, eps):
    """(normalized, 1 / deviation)"""
    steps = steps_of(v.v.shape[1])
    if kind == "layer":
        v = v - v.mean(steps)
    inverse = v.square().mean(steps).inverse_root(eps)
    return v * inverse, inverse


def normed_gradient(g, n, inverse, kind):
    steps = steps_of(g.v.shape[1])
    back = g - n * (g * n).mean(steps)
    if kind == "layer":
        back = back - g.mean(steps)
    return back * inverse


def vector_sum(t, like):
    M, D = t.v.shape
    G = like.shape[0] if like.dim() == 2 else 1
    parts = [Near(t.v[i * (M // G):(i + 1) * (M // G)], t.e[i * (M // G):(i + 1) * (M // G)])
             .sum(0, M // G) for i in range(G)]
    s = Near(torch.cat([p.v for p in parts]), torch.cat([p.e for p in parts]))
    return Near(s.v.view(like.shape), s.e.view(like.shape))


def reference(t, kind="rms", post="none", scale=1.0, eps=1e-6, dr=None, dy=None):
    """Outputs and, given dr or dy, gradients of add_norm (norm: no "h" in t) as Near
    values; t has x, h, gate, weight, bias, post_weight, post_bias, or some of them."""
    get = t.get
    M = t["x"].shape[0]
    out = {}
    r = Near(t["x"].double())
    h = get("h")
    if h is not None:
        n = behind = Near(h.double())
        if post != "none":
            n, inv_h = normed(n, post, eps)
            behind = n
            if get("post_weight") is not None:
                behind = behind * rows(t["post_weight"], M)
            if get("post_bias") is not None:
                behind = behind + rows(t["post_bias"], M)
        gate = rows(t["gate"], M) if get("gate") is not None else None
        r = r * scale + (behind if gate is None else behind * gate)
        out["r"] = r
    g = Near(torch.zeros_like(r.v))
    if kind != "none":
        nr, inv_r = normed(r, kind, eps)
        y = nr
        if get("weight") is not None:
            y = y * rows(t["weight"], M)
        if get("bias") is not None:
            y = y + rows(t["bias"], M)
        out["y"] = y
        if dy is not None:
            d = Near(dy.double())
            if get("weight") is not None:
                out["dweight"] = vector_sum(d * nr, t["weight"])
            if get("bias") is not None:
                out["dbias"] = vector_sum(d, t["bias"])
            if get("weight") is not None:
                d = d * rows(t["weight"], M)
            g = normed_gradient(d, nr, inv_r, kind)
    if dr is None and dy is None:
        return out
    if dr is not None:
        g = g + Near(dr.double())
    if h is None:
        out["dx"] = g
        return out
    out["dx"] = g * scale
    if gate is not None:
        out["dgate"] = vector_sum(g * behind, t["gate"])
        g = g * gate
    if post != "none":
        if get("post_weight") is not None:
            out["dpost_weight"] = vector_sum(g * n, t["post_weight"])
        if get("post_bias") is not None:
            out["dpost_bias"] = vector_sum(g, t["post_bias"])
        if get("post_weight") is not None:
            g = g * rows(t["post_weight"], M)
        g = normed_gradient(g, n, inv_h, post)
    out["dh"] = g
    return out
