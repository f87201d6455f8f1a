"""The gated recurrence on the GPU: forward, backward, packed rows, strides, checkpoints, the decode
step and their run together, against the 64-bit reference within its running error bounds."""
import zlib

import numpy as np
import pytest
import torch

import gated_ref as ref
from quantized_mamba_ssd_b200 import build as qbuild
from quantized_mamba_ssd_b200 import ssd_i8

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
FORMS = [(g, i) for g in ("log", "logit") for i in ("plain", "complement")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qbuild.build()
    ssd_i8.library()


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, err, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - want) <= err)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside the bound, first at "
                           f"{np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]} +- {err[bad][0]}")


def draw(rng, shape, gate, dtype):
    """x and gate as tensors of `dtype` on the GPU."""
    x = rng.laplace(size=shape) * rng.uniform(0.2, 8, shape[-1])
    g = (-np.logaddexp(0, rng.normal(-2, 0.5, shape)) * np.exp(rng.uniform(0, np.log(16), shape[-1]))
         if gate == "log" else rng.normal(2, 2, shape))
    dt = ref.TYPES[dtype]
    return torch.from_numpy(x).to(dt).to(DEV), torch.from_numpy(g).to(dt).to(DEV)


def tensor(a, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a)).to(ref.TYPES[dtype]).to(DEV)


def dense_cases(x, g, gate, inp, dtype, init):
    return [ref.Case(f64(x[b]), f64(g[b]), gate, inp, None,
                     None if init is None else f64(init[b:b + 1]), dtype).forward()
            for b in range(x.shape[0])]


def check_dense(x, g, gate, inp, dtype, *, state=True, ckpt=False, seed=0):
    b, l, d = x.shape
    rng = np.random.default_rng(seed + 1)
    form = dict(gate_form=gate, input_form=inp)
    init = tensor(rng.normal(size=(b, d))) if state else None
    dfin = tensor(rng.normal(size=(b, d))) if state else None
    dy = tensor(rng.normal(size=(b, l, d)), dtype)
    nan = lambda *s: torch.full(s, float("nan"), device=DEV)
    final, dinit, spans = nan(b, d), nan(b, d), nan(b, -(-l // 64), d)
    ck = ssd_i8.ssd_i8_gated_ckpt_empty(x) if ckpt else None
    y = ssd_i8.ssd_i8_gated_scan(x, g, init_state=init, final_state=final, span_states=spans,
                                 ckpt=ck, **form)
    states = dict(init_state=init, dfinal_state=dfin, dinit_state=dinit, **form)
    if ckpt:
        dx, dg = ssd_i8.ssd_i8_gated_scan_bwd_ckpt(dy, ck, spans, **states)
    else:
        dx, dg = ssd_i8.ssd_i8_gated_scan_bwd(dy, x, g, spans, **states)
    assert y.dtype == dx.dtype == dg.dtype == x.dtype and y.shape == dx.shape == dg.shape == x.shape
    for i, c in enumerate(dense_cases(x, g, gate, inp, dtype, init)):
        within(y[i], c.y, c.ey, "y")
        within(final[i:i + 1], c.final, c.efinal, "final_state")
        within(spans[i], *c.span_states(), "span_states")
        if ckpt:
            for got_q, got_e, v in ((ck.x_q, ck.x_e, c.x), (ck.gate_q, ck.gate_e, ref.held_gate(c.g, gate))):
                q, e, _ = ref.coded(v)
                assert np.array_equal(f64(got_q[i]), q) and np.array_equal(f64(got_e[i]), e)
            c = c.rebuilt()
        c.backward(f64(dy[i]), None if dfin is None else f64(dfin[i:i + 1]))
        within(dx[i], c.dx, c.edx, "dx")
        within(dg[i], c.dgate, c.edgate, "dgate")
        within(dinit[i:i + 1], c.dinit, c.edinit, "dinit_state")


SIZES = [(1, 1, 1), (3, 2, 33), (2, 15, 7), (1, 16, 64), (1, 17, 65), (2, 63, 2), (1, 64, 32),
         (2, 65, 31), (1, 127, 128), (2, 300, 66), (1, 1030, 40), (5, 129, 130), (1, 2500, 9)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("gate,inp", FORMS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_dense(dtype, gate, inp, size):
    rng = np.random.default_rng(zlib.crc32(repr((size, gate, inp)).encode()))
    x, g = draw(rng, size, gate, dtype)
    check_dense(x, g, gate, inp, dtype, state=sum(size) % 2 == 0)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("gate,inp", FORMS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_dense_on_checkpoints(dtype, gate, inp, size):
    rng = np.random.default_rng(zlib.crc32(repr((size, gate, inp)).encode()) + 1)
    x, g = draw(rng, size, gate, dtype)
    check_dense(x, g, gate, inp, dtype, state=sum(size) % 2 == 1, ckpt=True)


def test_long_sequences_over_many_parts():
    # strips cut into chunks of tokens, several steps in each, a ragged end
    for l, d, dtype in ((5000, 33, "f32"), (9001, 64, "bf16")):
        x, g = draw(np.random.default_rng(l), (1, l, d), "log", dtype)
        check_dense(x, g, "log", "complement", dtype)


@pytest.mark.parametrize("gate,inp", FORMS)
def test_long_memory_in_fp32(gate, inp):
    # a steady gate with a memory of 1e5 tokens: an fp32 decay rounded once would be off by
    # 2^-25 / 1e-5 = 3e-3 of 1 - a, far outside the bound, whose decay term is 2^-21 (1 - a)
    l, d = 4000, 34
    rng = np.random.default_rng(5)
    g = np.full((1, l, d), -1e-5 if gate == "log" else 11.5) * rng.uniform(0.9, 1.1, d)
    check_dense(tensor(np.abs(rng.normal(size=(1, l, d))) + 0.5), tensor(g), gate, inp, "f32")


def packed_offsets(kind):
    if kind == "ragged":  # empty ones, single tokens, one that fills a span, ends inside tiles
        lens = [0, 1, 70, 0, 0, 64, 58, 1, 1, 200, 15, 16, 17, 0]
        return np.concatenate([[0], np.cumsum(lens)])
    if kind == "gap":     # tokens before the first and behind the last sequence
        return np.array([37, 37, 100, 230, 230, 301])
    if kind == "single":
        return np.array([0, 333])
    return np.arange(0, 261, 2)  # many short ones


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("kind", ["ragged", "gap", "single", "short"])
@pytest.mark.parametrize("gate,inp,dtype", [("log", "plain", "bf16"), ("logit", "complement", "f32"),
                                            ("log", "complement", "f16"), ("logit", "plain", "bf16")])
def test_packed(gate, inp, dtype, kind, state, ckpt):
    off = packed_offsets(kind)
    T, n, d = int(off[-1]) + 45, len(off) - 1, 70
    rng = np.random.default_rng(len(off))
    x, g = draw(rng, (T, d), gate, dtype)
    outside = torch.ones(T, dtype=torch.bool, device=DEV)
    outside[int(off[0]):int(off[-1])] = False
    for t in (x, g):  # rows of no sequence may hold anything
        t[outside] = float("nan")
        t[int(off[-1])] = float("inf")
    cu = torch.tensor(off, dtype=torch.int32, device=DEV)
    form = dict(gate_form=gate, input_form=inp)
    init = tensor(rng.normal(size=(n, d))) if state else None
    dfin = tensor(rng.normal(size=(n, d))) if state else None
    dy = tensor(rng.normal(size=(T, d)), dtype)
    dy[outside] = float("nan")
    final, dinit = (torch.full((n, d), float("nan"), device=DEV) for _ in range(2))
    spans = torch.full((-(-T // 64), d), float("nan"), device=DEV)
    y, dx, dg = (torch.full_like(x, 7.0) for _ in range(3))
    ck = None
    if ckpt:
        ck = ssd_i8.ssd_i8_gated_ckpt_empty(x)
        for t in ck:
            t.fill_(9)
    ssd_i8.ssd_i8_gated_scan(x, g, cu, init_state=init, final_state=final, y=y, span_states=spans,
                             ckpt=ck, **form)
    states = dict(init_state=init, dfinal_state=dfin, dinit_state=dinit, dx=dx, dgate=dg, **form)
    if ckpt:
        ssd_i8.ssd_i8_gated_scan_bwd_ckpt(dy, ck, spans, cu, **states)
    else:
        ssd_i8.ssd_i8_gated_scan_bwd(dy, x, g, spans, cu, **states)
    c = ref.Case(f64(x), f64(g), gate, inp, off, None if init is None else f64(init), dtype).forward()
    v = c.valid
    assert np.array_equal(v, ~outside.cpu().numpy())
    within(f64(y)[v], c.y[v], c.ey[v], "y")
    within(final, c.final, c.efinal, "final_state")
    within(spans, *c.span_states(), "span_states")
    if ckpt:
        for got_q, got_e, val in ((ck.x_q, ck.x_e, c.x), (ck.gate_q, ck.gate_e, ref.held_gate(c.g, gate))):
            q, e, _ = ref.coded(val, v)
            assert np.array_equal(f64(got_q)[v], q[v]) and np.array_equal(f64(got_e), e)
            assert (got_q[outside] == 9).all()
        c = c.rebuilt()
    c.backward(f64(dy), None if dfin is None else f64(dfin))
    within(f64(dx)[v], c.dx[v], c.edx[v], "dx")
    within(f64(dg)[v], c.dgate[v], c.edgate[v], "dgate")
    within(dinit, c.dinit, c.edinit, "dinit_state")
    for t in (y, dx, dg):  # rows of no sequence are left as they were
        assert (t[outside] == 7.0).all()


def long_packed_offsets(kind):
    """Rows long enough for several chunks of tokens per strip (with 1 to 3 strips)."""
    if kind == "one":        # one sequence over every chunk
        return np.array([0, 9000])
    if kind == "edges":      # beginnings and ends on every multiple of a tile of the kernels
        return np.arange(0, 9001, 128)
    if kind == "ragged":
        return np.concatenate([[0], np.cumsum(np.random.default_rng(3).integers(0, 900, 22))])
    return np.array([3100, 3100, 3105, 8000])  # whole chunks before and behind the sequences


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("kind", ["one", "edges", "ragged", "gap"])
@pytest.mark.parametrize("gate,inp,dtype,d", [("log", "plain", "bf16", 136), ("logit", "complement", "f32", 40),
                                              ("log", "complement", "f16", 33)])
def test_packed_in_chunks(gate, inp, dtype, d, kind, ckpt):
    off = long_packed_offsets(kind)
    T, n = int(off[-1]) + 700, len(off) - 1
    assert ssd_i8.ssd_i8_gated_scan_workspace_size(1, T, d, dtype) > 0
    rng = np.random.default_rng(len(off))
    x, g = draw(rng, (T, d), gate, dtype)
    outside = torch.ones(T, dtype=torch.bool, device=DEV)
    outside[int(off[0]):int(off[-1])] = False
    x[outside], g[outside] = float("nan"), float("inf")
    dy = tensor(rng.normal(size=(T, d)), dtype)
    dy[outside] = float("nan")
    cu = torch.tensor(off, dtype=torch.int32, device=DEV)
    form = dict(gate_form=gate, input_form=inp)
    init, dfin = tensor(rng.normal(size=(n, d))), tensor(rng.normal(size=(n, d)))
    final, dinit = (torch.full((n, d), float("nan"), device=DEV) for _ in range(2))
    spans = torch.empty((-(-T // 64), d), device=DEV)
    ck = ssd_i8.ssd_i8_gated_ckpt_empty(x) if ckpt else None
    y, dx, dg = (torch.full_like(x, 7.0) for _ in range(3))
    ssd_i8.ssd_i8_gated_scan(x, g, cu, init_state=init, final_state=final, y=y, span_states=spans,
                             ckpt=ck, **form)
    states = dict(init_state=init, dfinal_state=dfin, dinit_state=dinit, dx=dx, dgate=dg, **form)
    if ckpt:
        ssd_i8.ssd_i8_gated_scan_bwd_ckpt(dy, ck, spans, cu, **states)
    else:
        ssd_i8.ssd_i8_gated_scan_bwd(dy, x, g, spans, cu, **states)
    # (the reference goes token by token: a few channels of either end are enough)
    pick = [0, 1, d // 2, d - 1]
    c = ref.Case(f64(x[:, pick]), f64(g[:, pick]), gate, inp, off, f64(init[:, pick]), dtype).forward()
    v = c.valid
    within(f64(y[:, pick])[v], c.y[v], c.ey[v], "y")
    within(final[:, pick], c.final, c.efinal, "final_state")
    within(spans[:, pick], *c.span_states(), "span_states")
    if ckpt:
        c = c.rebuilt()
    c.backward(f64(dy[:, pick]), f64(dfin[:, pick]))
    within(f64(dx[:, pick])[v], c.dx[v], c.edx[v], "dx")
    within(f64(dg[:, pick])[v], c.dgate[v], c.edgate[v], "dgate")
    within(dinit[:, pick], c.dinit, c.edinit, "dinit_state")
    for t in (y, dx, dg):
        assert (t[outside] == 7.0).all()


@pytest.mark.parametrize("d", [72, 2000])
def test_many_short_and_empty_sequences(d):
    # thousands of sequences of 0 to 9 tokens, in chunks of strips too
    rng = np.random.default_rng(d)
    lens = rng.integers(0, 10, 3001) * (rng.random(3001) < 0.6)
    lens[-40:] = 0
    off = np.concatenate([[0], np.cumsum(lens)])
    n, T = len(lens), int(off[-1])
    x, g = draw(rng, (T, d), "log", "f32")
    init, dfin, dy = (tensor(rng.normal(size=s)) for s in ((n, d), (n, d), (T, d)))
    cu = torch.tensor(off, dtype=torch.int32, device=DEV)
    nan = lambda *s: torch.full(s, float("nan"), device=DEV)
    final, dinit, spans = nan(n, d), nan(n, d), nan(-(-T // 64), d)
    y = ssd_i8.ssd_i8_gated_scan(x, g, cu, init_state=init, final_state=final, span_states=spans)
    dx, dg = ssd_i8.ssd_i8_gated_scan_bwd(dy, x, g, spans, cu, init_state=init, dfinal_state=dfin,
                                          dinit_state=dinit)
    pick = [0, 33, d - 1]
    c = ref.Case(f64(x[:, pick]), f64(g[:, pick]), "log", "plain", off, f64(init[:, pick]), "f32").forward()
    within(y[:, pick], c.y, c.ey, "y")
    within(final[:, pick], c.final, c.efinal, "final_state")
    within(spans[:, pick], *c.span_states(), "span_states")
    c.backward(f64(dy[:, pick]), f64(dfin[:, pick]))
    within(dx[:, pick], c.dx, c.edx, "dx")
    within(dg[:, pick], c.dgate, c.edgate, "dgate")
    within(dinit[:, pick], c.dinit, c.edinit, "dinit_state")
    empty = torch.from_numpy(lens == 0).to(DEV)
    assert torch.equal(final[empty], init[empty]) and torch.equal(dinit[empty], dfin[empty])


def test_infinite_states_do_not_cross_into_another_sequence():
    # the first sequence's state and gradient overflow; whole chunks follow them
    T, d = 9000, 64
    x, g = draw(np.random.default_rng(21), (T, d), "log", "bf16")
    x[:4000] = torch.finfo(torch.bfloat16).max
    g[:4000] = 0.0
    dy = torch.ones_like(x)
    dy[5000:] = torch.finfo(torch.bfloat16).max
    cu = torch.tensor([0, 4500, 5000, T], dtype=torch.int32, device=DEV)
    spans = torch.empty(-(-T // 64), d, device=DEV)
    y = ssd_i8.ssd_i8_gated_scan(x, g, cu, span_states=spans)
    assert not torch.isfinite(y[3999]).any() and torch.isfinite(y[4500:]).all()
    dx, dg = ssd_i8.ssd_i8_gated_scan_bwd(dy, x, g, spans, cu)
    assert torch.isfinite(dx[:5000]).all() and torch.isfinite(dg[4500:5000]).all()
    alone = torch.empty(-(-500 // 64), d, device=DEV)
    one = torch.tensor([0, 500], dtype=torch.int32, device=DEV)
    y1 = ssd_i8.ssd_i8_gated_scan(x[4500:5000], g[4500:5000], one, span_states=alone)
    assert (y1.float() - y[4500:5000].float()).abs().max() <= 2 ** -7 * y1.float().abs().max()


def test_packed_matches_separate_calls_and_empty_rows():
    # no token at all: the states pass through
    x = torch.empty((0, 40), device=DEV, dtype=torch.bfloat16)
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    init, final = torch.randn(3, 40, device=DEV), torch.empty(3, 40, device=DEV)
    y = ssd_i8.ssd_i8_gated_scan(x, x, cu, init_state=init, final_state=final)
    assert y.shape == x.shape and torch.equal(final, init)
    ssd_i8.ssd_i8_gated_scan(x, x, cu, final_state=final)
    assert not final.any()
    dinit = torch.empty_like(init)
    ssd_i8.ssd_i8_gated_scan_bwd(x, x, x, torch.empty((0, 40), device=DEV), cu, dfinal_state=init,
                                 dinit_state=dinit)
    assert torch.equal(dinit, init)
    z = torch.empty((2, 0, 40), device=DEV)
    final = torch.empty(2, 40, device=DEV)
    ssd_i8.ssd_i8_gated_scan(z, z, init_state=init[:2].contiguous(), final_state=final)
    assert torch.equal(final, init[:2])
    none = torch.empty((0, 5, 40), device=DEV)
    assert ssd_i8.ssd_i8_gated_scan(none, none).shape == none.shape


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["slices", "odd slices", "time major", "row pitch"])
def test_strides(layout, dtype):
    # the same values through contiguous tensors and through views give the same bits
    b, l, d = 3, 140, 66
    rng = np.random.default_rng(3)
    x, g = draw(rng, (b, l, d), "log", dtype)
    dy = tensor(rng.normal(size=(b, l, d)), dtype)
    spans = torch.empty(b, 3, d, device=DEV)

    def views(n):
        """n [b,l,d] views in the layout, and a buffer whose other elements stay 5"""
        if layout == "time major":
            buf = torch.full((n, l, b, d), 5.0, device=DEV, dtype=x.dtype)
            return [t.transpose(0, 1) for t in buf], buf
        first = 3 if layout == "odd slices" else 2
        gap = 1 if layout == "odd slices" else 4
        buf = torch.full((b, l, first + n * (d + gap)), 5.0, device=DEV, dtype=x.dtype)
        if layout == "row pitch":
            buf = torch.full((b, l + 3, first + n * (d + gap)), 5.0, device=DEV, dtype=x.dtype)[:, 1:-2]
        return [buf[:, :, first + i * (d + gap):][:, :, :d] for i in range(n)], buf

    (vx, vg, vdy), _ = views(3)
    for v, t in ((vx, x), (vg, g), (vdy, dy)):
        v.copy_(t)
    (vy,), by = views(1)
    (vdx, vdg), bd = views(2)
    want_y = ssd_i8.ssd_i8_gated_scan(x, g, span_states=spans)
    want = ssd_i8.ssd_i8_gated_scan_bwd(dy, x, g, spans)
    spans2 = torch.empty_like(spans)
    before = by.clone(), bd.clone()
    ssd_i8.ssd_i8_gated_scan(vx, vg, y=vy, span_states=spans2)
    ssd_i8.ssd_i8_gated_scan_bwd(vdy, vx, vg, spans2, dx=vdx, dgate=vdg)
    assert torch.equal(vy, want_y) and torch.equal(spans, spans2)
    assert torch.equal(vdx, want[0]) and torch.equal(vdg, want[1])
    # nothing but the rows was written
    vy.fill_(5.0), vdx.fill_(5.0), vdg.fill_(5.0)
    assert torch.equal(by, before[0]) and torch.equal(bd, before[1])
    q, e = ssd_i8.ssd_i8_ckpt_pack(vx)
    q2, e2 = ssd_i8.ssd_i8_ckpt_pack(x)
    assert torch.equal(q, q2) and torch.equal(e, e2)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [1, 66, 71, 129])
def test_rows_at_every_place(d, dtype, packed):
    # every tensor with a first element and a row pitch of its own modulo 16 bytes, codes at odd
    # addresses: the same bits as through contiguous tensors
    l, form = 150, dict(gate_form="logit", input_form="complement")
    rng = np.random.default_rng(d)
    x, g = draw(rng, (l, d), "logit", dtype)
    dy = tensor(rng.normal(size=(l, d)), dtype)
    cu = torch.tensor([3, 3, 40, 41, 130, 149], dtype=torch.int32, device=DEV) if packed else None
    lead = (lambda t: t) if packed else (lambda t: t[None])
    zeros = lambda: lead(torch.zeros_like(x))

    def run(x, g, dy, ck, y, dxs):
        spans = lead(torch.zeros(-(-l // 64), d, device=DEV))
        for t in ck:
            t.zero_()
        ssd_i8.ssd_i8_gated_scan(lead(x), lead(g), cu, y=y, span_states=spans, ckpt=ck, **form)
        ssd_i8.ssd_i8_gated_scan_bwd(lead(dy), lead(x), lead(g), spans, cu, dx=dxs[0], dgate=dxs[1], **form)
        ssd_i8.ssd_i8_gated_scan_bwd_ckpt(lead(dy), ck, spans, cu, dx=dxs[2], dgate=dxs[3], **form)
        return [y, spans, *ck, *dxs]

    want = run(x, g, dy, ssd_i8.ssd_i8_gated_ckpt_empty(lead(x)), zeros(), [zeros() for _ in range(4)])
    for k in range(8):
        def place(n, t=None):  # a view of zeros, or of t's values, at place k + n
            first, pitch = (3 * k + 5 * n) % 16, d + (k + 3 * n) % 16
            flat = torch.zeros(first + l * pitch + 16, dtype=x.dtype, device=DEV)
            v = flat[first:first + l * pitch].view(l, pitch)[:, :d]
            return v if t is None else v.copy_(t)

        def codes(t, n):
            first = (k + n) % 5
            return torch.zeros(first + t.numel(), dtype=t.dtype, device=DEV)[first:].view(t.shape)

        ck = ssd_i8.GatedCkpt(*(codes(t, n) for n, t in enumerate(ssd_i8.ssd_i8_gated_ckpt_empty(lead(x)))))
        got = run(place(0, x), place(1, g), place(2, dy), ck, lead(place(3)),
                  [lead(place(n)) for n in (4, 5, 6, 7)])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_broadcast_gradient():
    # the gradient of y.sum() is one element with stride 0; channels must be contiguous, so rows
    # of ones are given once for all tokens
    x, g = draw(np.random.default_rng(4), (2, 100, 32), "log", "f32")
    spans = torch.empty(2, 2, 32, device=DEV)
    ssd_i8.ssd_i8_gated_scan(x, g, span_states=spans)
    ones = torch.ones(32, device=DEV).expand(2, 100, 32)
    a = ssd_i8.ssd_i8_gated_scan_bwd(ones, x, g, spans)
    b = ssd_i8.ssd_i8_gated_scan_bwd(ones.contiguous(), x, g, spans)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError, match="contiguous"):
        ssd_i8.ssd_i8_gated_scan_bwd(torch.ones(1, device=DEV).expand(2, 100, 32), x, g, spans)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gate,inp", FORMS)
def test_extreme_gates(gate, inp, dtype):
    # decays of exactly 0 and 1, masks of the type's lowest value, infinite gates
    x, g = draw(np.random.default_rng(6), (1, 90, 34), gate, dtype)
    low = torch.finfo(x.dtype).min
    g[0, 5], g[0, 20], g[0, 40:43], g[0, 60] = low, float("-inf"), 0.0, -100.0
    if gate == "logit":
        g[0, 50], g[0, 51] = -low, float("inf")
    init = torch.randn(1, 34, device=DEV)
    form = dict(gate_form=gate, input_form=inp)
    spans, dinit = torch.empty(1, 2, 34, device=DEV), torch.empty(1, 34, device=DEV)
    ck = ssd_i8.ssd_i8_gated_ckpt_empty(x)
    y = ssd_i8.ssd_i8_gated_scan(x, g, init_state=init, span_states=spans, ckpt=ck, **form)
    c = dense_cases(x, g, gate, inp, dtype, init)[0]
    within(y[0], c.y, c.ey, "y")
    dy = tensor(np.random.default_rng(7).normal(size=(1, 90, 34)), dtype)
    dx, dg = ssd_i8.ssd_i8_gated_scan_bwd(dy, x, g, spans, init_state=init, dinit_state=dinit, **form)
    c.backward(f64(dy[0]))
    within(dx[0], c.dx, c.edx, "dx")
    within(dg[0], c.dgate, c.edgate, "dgate")
    within(dinit, c.dinit, c.edinit, "dinit_state")
    # the checkpoint holds the gate limited, so the lowest value does not swamp its block
    c = c.rebuilt().backward(f64(dy[0]))
    dx, dg = ssd_i8.ssd_i8_gated_scan_bwd_ckpt(dy, ck, spans, init_state=init, dinit_state=dinit, **form)
    assert np.isfinite(c.dgate).all()
    within(dx[0], c.dx, c.edx, "dx on checkpoints")
    within(dg[0], c.dgate, c.edgate, "dgate on checkpoints")


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("d", [33, 64])
@pytest.mark.parametrize("dtype,size", [("f32", 1e36), ("bf16", 1e35), ("f16", 6e3), ("bf16", 1e-36), ("f16", 1e-6)])
def test_largest_and_smallest_values(dtype, size, d, ckpt):
    # x near the ends of its type, gradients that keep the products inside it
    l, form = 70, dict(gate_form="log", input_form="complement")
    rng = np.random.default_rng(int(d))
    x = tensor(rng.normal(size=(1, l, d)) * size, dtype)
    _, g = draw(rng, (1, l, d), "log", dtype)
    dy = tensor(rng.normal(size=(1, l, d)) * min(1e3 / size, 1e30 if dtype != "f16" else 1e3), dtype)
    spans, dinit = torch.empty(1, 2, d, device=DEV), torch.empty(1, d, device=DEV)
    ck = ssd_i8.ssd_i8_gated_ckpt_empty(x) if ckpt else None
    y = ssd_i8.ssd_i8_gated_scan(x, g, span_states=spans, ckpt=ck, **form)
    c = ref.Case(f64(x[0]), f64(g[0]), "log", "complement", None, None, dtype).forward()
    within(y[0], c.y, c.ey, "y")
    if ckpt:
        dx, dg = ssd_i8.ssd_i8_gated_scan_bwd_ckpt(dy, ck, spans, dinit_state=dinit, **form)
        c = c.rebuilt()
    else:
        dx, dg = ssd_i8.ssd_i8_gated_scan_bwd(dy, x, g, spans, dinit_state=dinit, **form)
    c.backward(f64(dy[0]), None)
    within(dx[0], c.dx, c.edx, "dx")
    within(dg[0], c.dgate, c.edgate, "dgate")
    within(dinit, c.dinit, c.edinit, "dinit_state")


def test_nan_stays_in_its_channel_and_sequence():
    x, g = draw(np.random.default_rng(8), (200, 40), "log", "bf16")
    x[30, 3], g[150, 7] = float("nan"), float("nan")
    cu = torch.tensor([0, 100, 200], dtype=torch.int32, device=DEV)
    spans = torch.empty(4, 40, device=DEV)
    y = ssd_i8.ssd_i8_gated_scan(x, g, cu, span_states=spans)
    bad = torch.zeros(200, 40, dtype=torch.bool, device=DEV)
    bad[30:100, 3] = bad[150:, 7] = True
    assert torch.equal(torch.isnan(y), bad)
    dx, dg = ssd_i8.ssd_i8_gated_scan_bwd(torch.ones_like(x), x, g, spans, cu)
    bad[:] = False
    bad[100:150, 7] = True  # the gradient runs backward through a NaN decay
    assert torch.equal(torch.isnan(dx), bad)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [(1, 1), (1, 4096), (3, 37), (128, 514), (7, 1001)])
@pytest.mark.parametrize("gate,inp", FORMS)
def test_step(gate, inp, size, dtype):
    x, g = draw(np.random.default_rng(9), size, gate, dtype)
    st = torch.randn(size, device=DEV)
    c = [ref.Case(f64(x[i:i + 1]), f64(g[i:i + 1]), gate, inp, None, f64(st[i:i + 1]), dtype).forward()
         for i in range(size[0])]
    y = ssd_i8.ssd_i8_gated_step(st, x, g, gate_form=gate, input_form=inp)
    cat = lambda k: np.concatenate([getattr(v, k) for v in c])
    within(st, cat("final"), cat("efinal"), "state")
    within(y, cat("y"), cat("ey"), "y")


def test_step_on_unaligned_views():
    # contiguous tensors that start at odd elements of their buffers
    buf = torch.randn(4 * 999, device=DEV)
    h = torch.randn(4 * 999, device=DEV).to(torch.bfloat16)
    st, x, g = buf[3:3 + 900].view(9, 100), h[1:901].view(9, 100), -h[1001:1901].view(9, 100).abs()
    st2 = st.clone()
    y = torch.full((2000,), 5.0, device=DEV, dtype=torch.bfloat16)
    ssd_i8.ssd_i8_gated_step(st, x, g, y=y[7:907].view(9, 100))
    y2 = ssd_i8.ssd_i8_gated_step(st2, x.clone(), g.clone())
    assert torch.equal(st, st2) and torch.equal(y[7:907].view(9, 100), y2)
    assert (y[:7] == 5).all() and (y[907:] == 5).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 16, 33), (1, 100, 64), (3, 47, 130), (1000, 7),
                                   (0, 5), (2, 0, 8)])
def test_checkpoint(shape, dtype):
    rng = np.random.default_rng(10)
    v = rng.laplace(size=shape) * np.exp2(rng.integers(-20, 12, shape[-1]))
    if len(shape) == 2 and shape[0] > 64:
        v[:16, 0] = 0
        v[20, 1], v[40, 2], v[3, 3] = np.nan, np.inf, torch.finfo(ref.TYPES[dtype]).max
    x = tensor(v, dtype)
    q, e = ssd_i8.ssd_i8_ckpt_pack(x)
    back = ssd_i8.ssd_i8_ckpt_unpack(q, e, dtype=dtype)
    assert back.dtype == x.dtype and back.shape == x.shape
    wide = ssd_i8.ssd_i8_ckpt_unpack(q, e, dtype="f32")
    for i in range(shape[0] if len(shape) == 3 else 1):
        pick = (lambda t: t[i]) if len(shape) == 3 else (lambda t: t)
        if pick(x).numel() == 0:
            continue
        wq, we, wv = ref.coded(f64(pick(x)))
        assert np.array_equal(f64(pick(q)), wq) and np.array_equal(f64(pick(e)), we)
        np.testing.assert_array_equal(f64(pick(wide)), wv)
        np.testing.assert_array_equal(f64(pick(back)), wv)


def test_prefill_then_decode_then_more_prefill():
    # the state is the hand-over: a scan of 200 tokens equals a scan of 120, 30 steps, a scan of 50
    x, g = draw(np.random.default_rng(11), (4, 200, 96), "logit", "f32")
    form = dict(gate_form="logit", input_form="complement")
    whole_state, st = torch.empty(4, 96, device=DEV), torch.empty(4, 96, device=DEV)
    ssd_i8.ssd_i8_gated_scan(x, g, final_state=whole_state, **form)
    parts = [ssd_i8.ssd_i8_gated_scan(x[:, :120], g[:, :120], final_state=st, **form)]
    for t in range(120, 150):
        parts.append(ssd_i8.ssd_i8_gated_step(st, x[:, t].contiguous(), g[:, t].contiguous(), **form)[:, None])
    last = torch.empty_like(st)
    parts.append(ssd_i8.ssd_i8_gated_scan(x[:, 150:], g[:, 150:], init_state=st, final_state=last, **form))
    got = torch.cat(parts, 1)
    for b, c in enumerate(dense_cases(x, g, "logit", "complement", "f32", None)):
        within(got[b], c.y, c.ey, "y in parts")
        within(last[b:b + 1], c.final, c.efinal, "state in parts")
        within(whole_state[b:b + 1], c.final, c.efinal, "state")


class Recurrence(torch.autograd.Function):
    """How a training program wraps the calls."""

    @staticmethod
    def forward(ctx, x, gate, keep8):
        spans = torch.empty(x.shape[0], -(-x.shape[1] // ssd_i8.GATED_SPAN), x.shape[2],
                            device=x.device)
        ck = ssd_i8.ssd_i8_gated_ckpt_empty(x) if keep8 else None
        y = ssd_i8.ssd_i8_gated_scan(x, gate, input_form="complement", span_states=spans, ckpt=ck)
        ctx.save_for_backward(spans, *(ck if keep8 else (x, gate)))
        ctx.keep8 = keep8
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        spans, *kept = ctx.saved_tensors
        form = dict(input_form="complement")
        if ctx.keep8:
            dx, dg = ssd_i8.ssd_i8_gated_scan_bwd_ckpt(dy.contiguous(), kept, spans, **form)
        else:
            dx, dg = ssd_i8.ssd_i8_gated_scan_bwd(dy.contiguous(), *kept, spans, **form)
        return dx, dg, None


@pytest.mark.parametrize("keep8", [False, True])
def test_training_step_of_a_small_layer(keep8):
    # projection, recurrence, output: the weights' gradients against fp64 autograd of the same
    # layer.  On checkpoints x and gate are off by half a scale step, 2^-7 of the largest of 16,
    # and all sums here are of some hundred terms of either sign: the mean error stays below 2 %.
    torch.manual_seed(0)
    b, l, i, d = 2, 70, 24, 48
    inp = torch.randn(b, l, i, device=DEV)
    w = (torch.randn(i, 2 * d, device=DEV) / i ** 0.5).requires_grad_()

    proj = inp @ w
    y = Recurrence.apply(proj[..., :d], -torch.nn.functional.softplus(proj[..., d:]), keep8)
    y.square().sum().backward()

    w64 = w.detach().double().requires_grad_()
    p = inp.double() @ w64
    x64, g64 = p[..., :d], -torch.nn.functional.softplus(p[..., d:])
    h, ys = torch.zeros(b, d, device=DEV, dtype=torch.float64), []
    for t in range(l):
        h = g64[:, t].exp() * h - torch.expm1(g64[:, t]) * x64[:, t]
        ys.append(h)
    torch.stack(ys, 1).square().sum().backward()
    off = (w.grad.double() - w64.grad).norm() / w64.grad.norm()
    assert off < (2e-2 if keep8 else 1e-5), off


def test_streams_graphs_and_repeats():
    x, g = draw(np.random.default_rng(12), (2, 700, 100), "log", "bf16")
    cu = torch.tensor([0, 300, 300, 700], dtype=torch.int32, device=DEV)
    dy = torch.randn_like(x)
    spans, s1 = torch.empty(2, 11, 100, device=DEV), torch.empty(11, 100, device=DEV)

    def all_of_it(**kw):
        y = ssd_i8.ssd_i8_gated_scan(x, g, span_states=spans, **kw)
        ck = ssd_i8.ssd_i8_gated_ckpt_empty(x[0])
        y1 = ssd_i8.ssd_i8_gated_scan(x[0], g[0], cu, span_states=s1, ckpt=ck, **kw)
        q, e = ssd_i8.ssd_i8_ckpt_pack(x, **kw)
        return [y, y1, *ck, *ssd_i8.ssd_i8_gated_scan_bwd(dy, x, g, spans, **kw),
                *ssd_i8.ssd_i8_gated_scan_bwd_ckpt(dy[0], ck, s1, cu, **kw), q, e,
                ssd_i8.ssd_i8_ckpt_unpack(q, e, **kw),
                ssd_i8.ssd_i8_gated_step(spans[0].contiguous(), x[0, :11].contiguous(),
                                         g[0, :11].contiguous(), **kw)]

    want = [t.clone() for t in all_of_it()]
    for got, w in zip(all_of_it(), want):  # no result depends on the run
        assert torch.equal(got, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got = all_of_it(stream=stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_of_it()
    for t in out:
        t.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    # new contents of the captured offsets are followed
    cu.copy_(torch.tensor([0, 10, 650, 700], dtype=torch.int32))
    graph.replay()
    assert torch.equal(out[1], ssd_i8.ssd_i8_gated_scan(x[0], g[0], cu))


def test_two_calls_at_once_and_two_graphs():
    # calls on two streams with a workspace each, and two graphs replayed in turn
    sets = [draw(np.random.default_rng(30 + i), (1, 6000, 96), "log", "bf16") for i in range(2)]
    need = ssd_i8.ssd_i8_gated_scan_workspace_size(1, 6000, 96, "bf16")
    assert need > 0
    want = [ssd_i8.ssd_i8_gated_scan(x, g) for x, g in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in range(2)]
    out = [torch.empty_like(x) for x, _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (x, g) in enumerate(sets):
            ssd_i8.ssd_i8_gated_scan(x, g, y=out[i], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graphs, outs = [], []
    for x, g in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(ssd_i8.ssd_i8_gated_scan(x, g))
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_larger_workspace_and_output_slices():
    # a workspace larger than needed; gradients into the two halves of one projection's gradient
    x, g = draw(np.random.default_rng(40), (2, 3000, 130), "logit", "f16")
    need = ssd_i8.ssd_i8_gated_scan_workspace_size(2, 3000, 130, "f16")
    ws = torch.empty(need + 1000, dtype=torch.uint8, device=DEV)
    spans = torch.empty(2, -(-3000 // 64), 130, device=DEV)
    form = dict(gate_form="logit", input_form="complement")
    y = ssd_i8.ssd_i8_gated_scan(x, g, span_states=spans, workspace=ws, **form)
    dproj = torch.empty(2, 3000, 260, device=DEV, dtype=torch.float16)
    ssd_i8.ssd_i8_gated_scan_bwd(y, x, g, spans, dx=dproj[..., :130], dgate=dproj[..., 130:],
                                 workspace=ws, **form)
    dx, dg = ssd_i8.ssd_i8_gated_scan_bwd(y, x, g, spans, **form)
    assert torch.equal(dproj, torch.cat([dx, dg], -1))
    for bad, err in ((ws[:need - 1], ssd_i8.SSDError), (ws[1:], ssd_i8.SSDError), (ws.cpu(), ValueError),
                     (ws.view(torch.int8), TypeError)):
        with pytest.raises(err):
            ssd_i8.ssd_i8_gated_scan(x, g, workspace=bad, **form)


def test_wrong_offsets_stay_inside_the_tensors():
    # contents that break the rules give wrong values in the rows, nothing outside the tensors
    T, d, n = 200, 40, 4
    buf = torch.full((3, T + 2, d), 5.0, device=DEV)
    x, g = draw(np.random.default_rng(13), (T, d), "log", "f32")
    for off in ([500, -7, 90, 20, 300], [-100, -50, 250, 260, 270], [200, 150, 100, 50, 0]):
        cu = torch.tensor(off, dtype=torch.int32, device=DEV)
        guard = torch.full((n + 2, d), 5.0, device=DEV)
        spans = torch.zeros(4, d, device=DEV)
        ssd_i8.ssd_i8_gated_scan(x, g, cu, y=buf[0, 1:-1], final_state=guard[1:-1],
                                 span_states=spans)
        ssd_i8.ssd_i8_gated_scan_bwd(x, x, g, spans, cu, dx=buf[1, 1:-1], dgate=buf[2, 1:-1])
        torch.cuda.synchronize()
        assert (buf[:, 0] == 5).all() and (buf[:, -1] == 5).all()
        assert (guard[0] == 5).all() and (guard[-1] == 5).all()


def test_python_refusals():
    x = torch.zeros(2, 8, 4, device=DEV)
    f, s = torch.zeros(2, 4, device=DEV), torch.zeros(2, 1, 4, device=DEV)
    scan, bwd = ssd_i8.ssd_i8_gated_scan, ssd_i8.ssd_i8_gated_scan_bwd
    cu = torch.zeros(2, dtype=torch.int32, device=DEV)
    for err, call in (
            (ValueError, lambda: scan(x, x[:, :7])), (TypeError, lambda: scan(x, x.half())),
            (TypeError, lambda: scan(x.double(), x.double())),
            (ValueError, lambda: scan(x.transpose(1, 2), x.transpose(1, 2))),
            (ValueError, lambda: scan(x[0], x[0])), (ValueError, lambda: scan(x, x, cu)),
            (ValueError, lambda: scan(x, x.cpu())), (ValueError, lambda: scan(x[0], x[0], cu.cpu())),
            (TypeError, lambda: scan(x[0], x[0], cu.long())), (ValueError, lambda: scan(x[0], x[0], cu[:0])),
            (ValueError, lambda: scan(x[0], x[0], [0, 8])),
            (ValueError, lambda: scan(x, x, gate_form="exp")),
            (ValueError, lambda: scan(x, x, input_form="")),
            (ValueError, lambda: scan(x, x, init_state=f[:1])),
            (TypeError, lambda: scan(x, x, final_state=f.half())),
            (ValueError, lambda: scan(x, x, span_states=f)),
            (ValueError, lambda: scan(x, x, y=torch.zeros(2, 8, 8, device=DEV)[:, :, ::2])),
            (ssd_i8.SSDError, lambda: scan(x, x, y=x)),
            (ssd_i8.SSDError, lambda: scan(x, x, init_state=f, final_state=f)),
            (ssd_i8.SSDError, lambda: scan(x, x, y=torch.zeros(4, device=DEV).expand(2, 8, 4))),
            (ValueError, lambda: scan(x, x, ckpt=(f, f))),
            (ValueError, lambda: scan(x, x, ckpt=ssd_i8.ssd_i8_gated_ckpt_empty(x[0]))),
            (TypeError, lambda: bwd(x, x, x, None)), (ValueError, lambda: bwd(x, x, x, f)),
            (ssd_i8.SSDError, lambda: bwd(x, x, x, s, dx=x)),
            (ssd_i8.SSDError, lambda: bwd(x, x, x, s, dinit_state=f, dfinal_state=f)),
            (ValueError, lambda: ssd_i8.ssd_i8_gated_step(f, f[:1], f)),
            (ValueError, lambda: ssd_i8.ssd_i8_gated_step(f.t(), f.t(), f.t())),
            (ssd_i8.SSDError, lambda: ssd_i8.ssd_i8_gated_step(f, f, f)),
            (ValueError, lambda: ssd_i8.ssd_i8_ckpt_pack(f[0])),
            (ValueError, lambda: ssd_i8.ssd_i8_ckpt_unpack(x.to(torch.int8), x.to(torch.uint8))),
            (ValueError, lambda: ssd_i8.ssd_i8_ckpt_unpack(x.to(torch.int8), s.to(torch.uint8), dtype="i8"))):
        with pytest.raises(err):
            call()


def test_offsets_past_32_bits():
    # 2.4e9 elements: the last rows lie behind 2^31 elements of every tensor
    l, d = 74000, 32768
    x = torch.empty((1, l, d), dtype=torch.bfloat16, device=DEV)
    g = torch.empty_like(x)
    for t in range(0, l, 2000):
        x[:, t:t + 2000].normal_()
        g[:, t:t + 2000].uniform_(-2, -0.01)
    cols = [0, 1, 31, 20000, d - 1]
    spans = torch.empty(1, -(-l // 64), d, device=DEV)
    y = ssd_i8.ssd_i8_gated_scan(x, g, span_states=spans)
    c = ref.Case(f64(x[0][:, cols]), f64(g[0][:, cols]), "log", "plain", dtype="bf16").forward()
    within(y[0][:, cols], c.y, c.ey, "y")
    dx, dg = ssd_i8.ssd_i8_gated_scan_bwd(y, x, g, spans)
    c.backward(f64(y[0][:, cols]))
    within(dx[0][:, cols], c.dx, c.edx, "dx")
    within(dg[0][:, cols], c.dgate, c.edgate, "dgate")
    q, e = ssd_i8.ssd_i8_ckpt_pack(x)
    wq, we, wv = ref.coded(c.x)
    assert np.array_equal(f64(q[0][:, cols]), wq) and np.array_equal(f64(e[0][:, cols]), we)
    del y, dx, dg
    x.zero_()
    ssd_i8.ssd_i8_ckpt_unpack(q, e, x=x)
    assert np.array_equal(f64(x[0][:, cols]), wv)
