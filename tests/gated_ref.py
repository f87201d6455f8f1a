"""64-bit reference of the gated recurrence, its gradients and the 8-bit checkpoints, with running
error bounds for kernels that compute in fp32.

Inputs are numpy float64 arrays [l, d] (one batch row) holding the values of the kernel's inputs.

Bounds.  One fp32 rounding is r = 2^-24 of its result (half a step).  With hb_t = a_t hb_{t-1} +
|w_t x_t| (which dominates |h_t| and every partial sum of it), the error of a computed state obeys

    E_t = a_t E_{t-1} + da_t hb_{t-1} + dw_t |x_t| + 8 r hb_t

where da and dw bound the errors of the computed decay and input weight, and 8 roundings a token
cover the step itself (2), the input product (1) and, in a scan that joins parts, the products of
decays and the joins (a few per part of at least 16 tokens).  The gradient that runs backward obeys
the same recursion.  A result rounded to its type adds half a step of it.

    decay      16-bit: the approximate exponential and reciprocal, relative error below 2^-21
               fp32: two floats; expf / expm1f of 2 ulp leave 2^-22 min(a, 1 - a), doubled
    weight     16-bit: 2^-16 (the series below 1/16 and the difference above it are below 2^-18),
               logit 2^-20;  fp32: 2^-21

A relative bound ends at fp32's smallest normal number: below it numbers are 2^-149 apart (exp(-100)
is 27 of them, so the nearest one is already 2^-6 off), and the fast instructions may give 0.
Decays and weights are therefore allowed 2^-126 besides.
"""
import math

import numpy as np
import torch

R = 2.0 ** -24
SPAN, BLOCK = 64, 16
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def decay(g, gate):
    """a and 1 - a."""
    with np.errstate(over="ignore"):
        if gate == "log":
            return np.exp(g), -np.expm1(g)
        return 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))


def decay_errors(a, u, gate, dtype):
    """Bounds of the computed a (absolute) and of the computed 1 - a (absolute)."""
    tiny = 2.0 ** -126
    if dtype == "f32":
        return 2.0 ** -21 * np.minimum(a, np.abs(u)) + tiny, 2.0 ** -21 * np.abs(u) + tiny
    return (2.0 ** -21 * a + tiny,
            (2.0 ** -16 if gate == "log" else 2.0 ** -20) * np.abs(u) + tiny)


def rounded(v, dtype):
    """Half a step of each value in the output type (with its smallest step near zero)."""
    f = torch.finfo(TYPES[dtype])
    return np.abs(v) * f.eps / 2 + f.smallest_normal * f.eps / 2


def held_gate(g, gate):
    return np.maximum(g, -16.0) if gate == "log" else np.clip(g, -16.0, 16.0)


def coded(v, valid=None):
    """(codes, exponents, values) of the checkpoint of v [l, d]; rows outside `valid` count as 0."""
    l, d = v.shape
    ok = np.ones(l, bool) if valid is None else valid
    q, val = np.zeros((l, d)), np.zeros((l, d))
    e = np.zeros((-(-l // BLOCK), d))
    for i in range(e.shape[0]):
        rows = slice(i * BLOCK, min(l, (i + 1) * BLOCK))
        blk = np.where(ok[rows, None], v[rows], 0.0)
        for c in range(d):
            top = np.abs(blk[:, c]).max()
            if not np.isfinite(top):
                e[i, c], q[rows, c], val[rows, c] = 255, 0, np.nan
                continue
            k = -126
            if top > 0:
                k = max(k, math.floor(math.log2(top)) - 6)
            q[rows, c] = np.clip(np.rint(np.ldexp(blk[:, c], -k)), -127, 127)
            val[rows, c] = np.ldexp(q[rows, c], k)
            e[i, c] = k + 127
    return q, e, val


class Case:
    """One batch row of l tokens, cut into `offsets` (sequence s: tokens offsets[s] to
    offsets[s + 1]; tokens outside are ignored)."""

    def __init__(self, x, g, gate, inp, offsets=None, init=None, dtype="f32"):
        self.x, self.g, self.gate, self.plain, self.dtype = x, g, gate, inp == "plain", dtype
        self.l, self.d = x.shape
        self.packed = offsets is not None
        self.off = list(offsets) if self.packed else [0, self.l]
        n = len(self.off) - 1
        self.init = np.zeros((n, self.d)) if init is None else init
        self.seqs = [(s, self.off[s], self.off[s + 1]) for s in range(n)]
        self.valid = np.zeros(self.l, bool)
        for _, i, j in self.seqs:
            self.valid[i:j] = True

    def _terms(self, x, g):
        a, u = decay(g, self.gate)
        da, du = decay_errors(a, u, self.gate, self.dtype)
        one = np.ones_like(a)
        return (a, u, da, du) + ((one, 0 * one) if self.plain else (u, du))

    def forward(self):
        """Fills y, its bound ey, and per sequence the final state and its bound."""
        a, u, da, du, w, dw = self._terms(self.x, self.g)
        self.y, self.hb, self.eh = (np.full((self.l, self.d), np.nan) for _ in range(3))
        self.before, self.bb, self.eb = (np.full((self.l, self.d), np.nan) for _ in range(3))
        self.final, self.efinal = self.init.copy(), np.zeros_like(self.init)
        for s, i, j in self.seqs:
            h, hb, e = self.init[s], np.abs(self.init[s]), np.zeros(self.d)
            for t in range(i, j):
                self.before[t], self.bb[t], self.eb[t] = h, hb, e
                e = a[t] * e + da[t] * hb + dw[t] * np.abs(self.x[t])
                h = a[t] * h + w[t] * self.x[t]
                hb = a[t] * hb + np.abs(w[t] * self.x[t])
                e = e + 8 * R * hb
                self.y[t], self.hb[t], self.eh[t] = h, hb, e
            self.final[s], self.efinal[s] = h, e
        self.ey = self.eh + rounded(self.y, self.dtype)
        return self

    def span_states(self):
        """The state before tokens 0, 64, .. and its bound (packed: 0 where a sequence begins there
        or none holds the token)."""
        at = range(0, self.l, SPAN)
        out, err = np.zeros((len(at), self.d)), np.zeros((len(at), self.d))
        for k, t in enumerate(at):
            if not self.packed or any(i < t < j for _, i, j in self.seqs):
                out[k], err[k] = self.before[t], self.eb[t]
        return out, err

    def rebuilt(self):
        """The case as the backward pass from checkpoints sees it: x and gate decoded, `before`
        rebuilt in each span from the exact state before it."""
        q = Case(coded(self.x, self.valid)[2], coded(held_gate(self.g, self.gate), self.valid)[2],
                 self.gate,
                 "plain" if self.plain else "complement",
                 self.off if self.packed else None, self.init, self.dtype)
        a, u, da, du, w, dw = q._terms(q.x, q.g)
        q.before, q.bb, q.eb = (np.full((self.l, self.d), np.nan) for _ in range(3))
        for s, i, j in self.seqs:
            for t in range(i, j):
                if t == i or t % SPAN == 0:
                    h, hb, e = self.before[t], self.bb[t], self.eb[t]
                q.before[t], q.bb[t], q.eb[t] = h, hb, e
                e = a[t] * e + da[t] * hb + dw[t] * np.abs(q.x[t])
                h = a[t] * h + w[t] * q.x[t]
                hb = a[t] * hb + np.abs(w[t] * q.x[t])
                e = e + 8 * R * hb
        return q

    def backward(self, dy, dfinal=None):
        """Fills dx, dgate, dinit and their bounds edx, edgate, edinit."""
        a, u, da, du, w, dw = self._terms(self.x, self.g)
        self.dx, self.edx = (np.full((self.l, self.d), np.nan) for _ in range(2))
        self.dgate, self.edgate = (np.full((self.l, self.d), np.nan) for _ in range(2))
        self.dinit = np.zeros_like(self.init) if dfinal is None else dfinal.copy()
        self.edinit = np.zeros_like(self.init)
        for s, i, j in self.seqs:
            back = self.dinit[s].copy()
            bb, e = np.abs(back), np.zeros(self.d)
            for t in range(j - 1, i - 1, -1):
                dh, db = dy[t] + back, np.abs(dy[t]) + bb
                ed = e + 2 * R * db
                back, bb = a[t] * dh, a[t] * db
                e = a[t] * ed + da[t] * db + 8 * R * bb
                self.dx[t] = w[t] * dh
                self.edx[t] = w[t] * ed + dw[t] * db + 2 * R * np.abs(w[t]) * db
                m = self.before[t] if self.plain else self.before[t] - self.x[t]
                mb = self.bb[t] if self.plain else self.bb[t] + np.abs(self.x[t])
                f = np.ones(self.d) if self.gate == "log" else u[t]
                df = 0 * f if self.gate == "log" else du[t]
                self.dgate[t] = back * m * f
                self.edgate[t] = (e * mb * f + bb * (self.eb[t] + 2 * R * mb) * f
                                  + bb * mb * df + 4 * R * bb * mb * f)
            self.dinit[s], self.edinit[s] = back, e
        self.edx += rounded(self.dx, self.dtype)
        self.edgate += rounded(self.dgate, self.dtype)
        return self
