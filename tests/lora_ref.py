"""Low-rank adapters on routed rows in 64 bits, one adapter at a time, on the
CPU, from the definitions in include/ep_lora.h."""
from __future__ import annotations

import torch


def rows_of(idx: torch.Tensor, E: int, mode: int = 0, max_tokens: int = 0):
    """[(row, adapter, token)] of every routed pair, in the layout's order."""
    T, K = idx.shape
    seen, start, out = [0] * E, 0, []
    by = [[] for _ in range(E)]
    for t in range(T):
        for k in range(K):
            e = int(idx[t, k])
            if 0 <= e < E:
                by[e].append(t)
    for e in range(E):
        for i, t in enumerate(by[e]):
            if mode == 1:
                if i < max_tokens:
                    out.append((e * max_tokens + i, e, t))
            else:
                out.append((start + i, e, t))
        start += len(by[e])
    return out


class Ref:
    """tokens: x, base, out are in token order; else in row order."""

    def __init__(self, idx, a, b, scales, num_rows, tokens, mode=0, max_tokens=0):
        self.E = a.shape[0]
        self.a, self.b = a.double(), b.double()
        self.s = torch.ones(self.E, dtype=torch.float64) if scales is None else scales.double()
        self.num_rows = num_rows
        rows = [(r, e, t) for r, e, t in rows_of(idx, self.E, mode, max_tokens) if r < num_rows]
        self.groups = []  # (adapter, row indices, data indices)
        for e in range(self.E):
            mine = [(r, t) for r, ee, t in rows if ee == e]
            r = torch.tensor([m[0] for m in mine], dtype=torch.int64)
            at = torch.tensor([m[1] for m in mine], dtype=torch.int64) if tokens else r
            self.groups.append((e, r, at))
        self.tokens = tokens
        routed = torch.zeros(idx.shape[0], dtype=torch.bool)
        routed[(idx >= 0).any(dim=1) & (idx < self.E).any(dim=1)] = True
        self.unrouted = ~routed

    def forward(self, x, base, out_before):
        """(out, h, and the sums of the products' sizes that bound the rounding)."""
        r = self.a.shape[1]
        out, size = out_before.double().clone(), torch.zeros(out_before.shape, dtype=torch.float64)
        h, hsize = torch.zeros((self.num_rows, r), dtype=torch.float64), torch.zeros((self.num_rows, r),
                                                                                     dtype=torch.float64)
        if self.tokens:
            out[self.unrouted] = 0.0 if base is None else base.double()[self.unrouted]
        for e, rows, at in self.groups:
            if rows.numel() == 0:
                continue
            h[rows] = self.s[e] * (x[at].double() @ self.a[e].T)
            hsize[rows] = self.s[e].abs() * (x[at].double().abs() @ self.a[e].abs().T)
            out[at] = (0.0 if base is None else base[at].double()) + h[rows] @ self.b[e].T
            size[at] = hsize[rows] @ self.b[e].abs().T + (0.0 if base is None else base[at].double().abs())
        return out, h, size, hsize

    def backward(self, dy, x, h, dx_base, dx_before):
        E, r, hin = self.a.shape
        hout = self.b.shape[1]
        z = lambda *s: torch.zeros(s, dtype=torch.float64)  # noqa: E731
        dx, dxs = dx_before.double().clone(), z(*dx_before.shape)
        da, das, db, dbs = z(E, r, hin), z(E, r, hin), z(E, hout, r), z(E, hout, r)
        if self.tokens:
            dx[self.unrouted] = 0.0 if dx_base is None else dx_base.double()[self.unrouted]
        for e, rows, at in self.groups:
            if rows.numel() == 0:
                continue
            g = dy[at].double()
            dh = self.s[e] * (g @ self.b[e])
            dhs = self.s[e].abs() * (g.abs() @ self.b[e].abs())
            dx[at] = (0.0 if dx_base is None else dx_base[at].double()) + dh @ self.a[e]
            dxs[at] = dhs @ self.a[e].abs() + (0.0 if dx_base is None else dx_base[at].double().abs())
            da[e], das[e] = dh.T @ x[at].double(), dhs.T @ x[at].double().abs()
            db[e], dbs[e] = g.T @ h[rows].double(), g.abs().T @ h[rows].double().abs()
        return (dx, da, db), (dxs, das, dbs)
