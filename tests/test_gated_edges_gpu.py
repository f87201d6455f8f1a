"""The gated recurrence on the GPU at its edges: sequences that share checkpoint blocks, rows without a
sequence, parts of one buffer, and how exact the decays and weights of 16-bit gates are."""
import numpy as np
import pytest
import torch

import gated_ref as ref
from quantized_mamba_ssd_b200 import build as qbuild
from quantized_mamba_ssd_b200 import ssd_i8
from test_gated_gpu import DEV, FORMS, draw, f64, tensor, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qbuild.build()
    ssd_i8.library()


# offsets, rows behind them, channels, and (tensor, token, value) of what is not finite
NAN, INF = float("nan"), float("inf")
SHARED = [
    # borders inside blocks (20, 40, 43, 100, 150) and on a block's edge (96)
    ([0, 20, 40, 43, 96, 100, 150], 20, 70,
     [("x", 18, INF), ("x", 41, NAN), ("x", 97, -INF), ("x", 99, NAN), ("x", 149, NAN), ("x", 10, NAN),
      ("gate", 20, NAN), ("gate", 19, NAN), ("gate", 42, NAN), ("gate", 100, NAN), ("gate", 120, NAN)]),
    # a gap and empty sequences before the border
    ([5, 9, 9, 60, 60, 61, 64, 90], 7, 33,
     [("x", 8, NAN), ("x", 60, INF), ("x", 61, NAN), ("x", 64, NAN), ("gate", 9, NAN), ("gate", 8, NAN),
      ("gate", 60, NAN)]),
    # strips in chunks
    ([0, 4005, 6011, 9000], 100, 40,
     [("x", 4004, NAN), ("x", 6011, INF), ("gate", 4005, NAN), ("gate", 6010, NAN), ("gate", 3000, NAN)]),
]


@pytest.mark.parametrize("case", range(len(SHARED)))
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gate,inp", FORMS)
def test_not_finite_values_stay_in_their_sequence_on_checkpoints(gate, inp, dtype, case):
    # Sequences that share a block with a value that is not finite get the bits that they get when a
    # zero stands there: the value has no part in the block's scale.
    off, behind, d, bad = SHARED[case]
    T, n = off[-1] + behind, len(off) - 1
    rng = np.random.default_rng(case)
    x, g = draw(rng, (T, d), gate, dtype)
    init, dfin, dy = tensor(rng.normal(size=(n, d))), tensor(rng.normal(size=(n, d))), tensor(
        rng.normal(size=(T, d)), dtype)
    cu = torch.tensor(off, dtype=torch.int32, device=DEV)
    form = dict(gate_form=gate, input_form=inp)

    def run(x, g):
        spans = torch.zeros(-(-T // 64), d, device=DEV)
        final, dinit = (torch.zeros(n, d, device=DEV) for _ in range(2))
        y, dx, dg = (torch.zeros_like(x) for _ in range(3))
        ck = ssd_i8.ssd_i8_gated_ckpt_empty(x)
        for t in ck:
            t.zero_()
        ssd_i8.ssd_i8_gated_scan(x, g, cu, init_state=init, final_state=final, y=y, span_states=spans,
                                 ckpt=ck, **form)
        ssd_i8.ssd_i8_gated_scan_bwd_ckpt(dy, ck, spans, cu, init_state=init, dfinal_state=dfin,
                                          dinit_state=dinit, dx=dx, dgate=dg, **form)
        return ck, (y, dx, dg), (final, dinit)

    for part in range(2):  # every second value: two of one block are then also tried apart
        put = [(which, t, v, (5 * i + 3) % d) for i, (which, t, v) in enumerate(bad)][part::2]
        bx, bg, cx, cg = x.clone(), g.clone(), x.clone(), g.clone()
        row_hit = torch.zeros(T, d, dtype=torch.bool, device=DEV)
        seq_hit = torch.zeros(n, d, dtype=torch.bool, device=DEV)
        for which, t, v, c in put:
            (bx if which == "x" else bg)[t, c] = v
            (cx if which == "x" else cg)[t, c] = 0.0
            s = next(s for s in range(n) if off[s] <= t < off[s + 1])
            row_hit[off[s]:off[s + 1], c] = seq_hit[s, c] = True
        ck, rows, states = run(bx, bg)
        clean_ck, clean_rows, clean_states = run(cx, cg)
        for a, b in zip(rows, clean_rows):
            assert torch.equal(a[~row_hit], b[~row_hit])
        for a, b in zip(states, clean_states):
            assert torch.equal(a[~seq_hit], b[~seq_hit])
        for which, t, _, c in put:
            s = next(s for s in range(n) if off[s] <= t < off[s + 1])
            if which == "x":  # the state behind it, and with it the later tokens' gate gradients
                assert not torch.isfinite(rows[2][t + 1:off[s + 1], c]).any()
            else:             # the gradients of all tokens before it
                assert not torch.isfinite(rows[1][off[s]:t, c]).any()
            # a block of several sequences marks the token, one of a single sequence the block
            at = 0 if which == "x" else 2
            blk = t // 16
            mixed = sum(min(off[i + 1], 16 * blk + 16) > max(off[i], 16 * blk) for i in range(n)) > 1
            values = ssd_i8.ssd_i8_ckpt_unpack(ck[at], ck[at + 1], dtype=dtype)
            want = ssd_i8.ssd_i8_ckpt_unpack(clean_ck[at], clean_ck[at + 1], dtype=dtype)
            inside = slice(16 * blk, min(16 * blk + 16, T))
            others = [u for u in range(*inside.indices(T)) if u not in [p[1] for p in put
                                                                        if p[0] == which and p[3] == c]]
            assert torch.isnan(values[t, c])
            if mixed:
                assert ck[at][t, c] == -128 and ck[at + 1][blk, c] == clean_ck[at + 1][blk, c]
                assert torch.equal(values[others, c], want[others, c])
            else:
                assert ck[at + 1][blk, c] == 255 and (ck[at][inside, c] == 0).all()
                assert torch.isnan(values[inside, c]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [1, 2, 6, 8, 33])
def test_unpack_reads_the_code_of_no_value(d, dtype):
    # every code at every place: -128 is NaN, the others times the scale (a power of two: exact)
    codes = torch.arange(-128, 128, device=DEV, dtype=torch.int16).to(torch.int8)
    q = torch.stack([codes.roll(7 * c) for c in range(d)], 1).contiguous()
    e = torch.full((16, d), 127 - 7, dtype=torch.uint8, device=DEV)
    got = ssd_i8.ssd_i8_ckpt_unpack(q, e, dtype=dtype).float()
    want = q.float() / 128
    want[q == -128] = NAN
    assert torch.equal(torch.isnan(got), q == -128)
    assert torch.equal(got[q != -128], want[q != -128])


@pytest.mark.parametrize("T", [5, 16, 200, 9000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_without_a_sequence(dtype, T):
    # offsets of no sequence: the span states and the scales of blocks without a token are written, no
    # row is
    d = 33
    x = torch.full((T, d), NAN, device=DEV, dtype=torch.float32 if dtype == "f32" else torch.bfloat16)
    cu = torch.zeros(1, dtype=torch.int32, device=DEV)
    spans = torch.full((-(-T // 64), d), 7.0, device=DEV)
    y = torch.full_like(x, 7.0)
    ck = ssd_i8.ssd_i8_gated_ckpt_empty(x)
    for t in ck:
        t.fill_(9)
    ssd_i8.ssd_i8_gated_scan(x, x, cu, y=y, span_states=spans, ckpt=ck)
    assert (y == 7).all() and not spans.any()
    assert (ck.x_q == 9).all() and (ck.gate_q == 9).all()
    assert (ck.x_e == 1).all() and (ck.gate_e == 1).all()
    empty = torch.empty(0, d, device=DEV)
    for call in (lambda **k: ssd_i8.ssd_i8_gated_scan_bwd(x, x, x, spans, cu, **k),
                 lambda **k: ssd_i8.ssd_i8_gated_scan_bwd_ckpt(x, ck, spans, cu, **k)):
        dx, dg = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
        call(dx=dx, dgate=dg, init_state=empty, dfinal_state=empty)
        assert (dx == 7).all() and (dg == 7).all()


@pytest.mark.parametrize("layout", ["stack", "token halves", "time-major stack", "columns at a pitch of their own"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_halves_of_one_buffer(dtype, layout):
    # x and gate, y and a copy of it, dx and dgate as the two halves of one buffer: the same bits as from
    # tensors of their own, and a half moved onto the other one is refused
    b, l, d = 2, 100, 64
    x, g = draw(np.random.default_rng(17), (b, l, d), "log", dtype)
    dy = torch.randn_like(x)

    def halves(n=2):
        t = dict(device=DEV, dtype=x.dtype)
        if layout == "stack":
            buf = torch.zeros(b, n, l, d, **t)
            return [buf[:, i] for i in range(n)]
        if layout == "token halves":
            buf = torch.zeros(b, n * l, d, **t)
            return [buf[:, i * l:(i + 1) * l] for i in range(n)]
        if layout == "time-major stack":
            buf = torch.zeros(l, n, b, d, **t)
            return [buf[:, i].transpose(0, 1) for i in range(n)]
        buf = torch.zeros(b, l * n * d + 24, **t)[:, :l * n * d].unflatten(1, (l, n * d))
        return [buf[..., i * d:(i + 1) * d] for i in range(n)]

    spans = torch.empty(b, 2, d, device=DEV)
    want = ssd_i8.ssd_i8_gated_scan(x, g, span_states=spans)
    want_bwd = ssd_i8.ssd_i8_gated_scan_bwd(dy, x, g, spans)
    vx, vy, vg = halves(3)
    vx.copy_(x), vg.copy_(g)
    ssd_i8.ssd_i8_gated_scan(vx, vg, y=vy)
    assert torch.equal(vy, want)
    assert torch.equal(vx, x) and torch.equal(vg, g)
    dx, dg = halves()
    ssd_i8.ssd_i8_gated_scan_bwd(dy, vx, vg, spans, dx=dx, dgate=dg)
    assert torch.equal(dx, want_bwd[0]) and torch.equal(dg, want_bwd[1])
    for off in (1, d // 2):  # one element, half a row
        st, at = dx.stride(), dg.storage_offset()
        near = torch.as_strided(dg, dg.shape, st, at - off)
        with pytest.raises(ssd_i8.SSDError):
            ssd_i8.ssd_i8_gated_scan_bwd(dy, vx, vg, spans, dx=dx, dgate=near)
    with pytest.raises(ssd_i8.SSDError):
        ssd_i8.ssd_i8_gated_scan(vx, vg, y=vx)


def every_gate(dtype, gate):
    """All finite gates of a 16-bit type (log: up to 0), [n], and their values in 64 bits."""
    g = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(ref.TYPES[dtype])
    g = g[torch.isfinite(g)]
    if gate == "log":
        g = g[g <= 0]
    return g.to(DEV), g.double().numpy()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_weights_of_every_log_gate(dtype):
    # One step from 0 with x = 1 leaves 1 - a as the fp32 state.  Below 1/16 the series: the term it
    # leaves out, g^4 / 120 < 2^-22.9, and six roundings of at most 2^-24, of which those of the inner
    # terms shrink with g.  Above, a's error over 1 - a: the exponential's instruction 2^-22, its
    # argument's rounding and that of log2(e) 1.5 |g| 2^-24.  Below 2^-126 the product may be 0.
    g, v = every_gate(dtype, "log")
    st = torch.zeros(1, g.numel(), device=DEV)
    ssd_i8.ssd_i8_gated_step(st, torch.ones_like(g)[None], g[None], input_form="complement")
    a, u = np.exp(v), -np.expm1(v)
    far = a * (2.0 ** -22 + 1.5 * np.abs(v) * 2.0 ** -24) + 2.0 ** -24 * u
    within(st[0], u, np.where(np.abs(v) < 0.0625, 2.0 ** -21 * u, far) + 2.0 ** -126, "1 - a")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gate", ["log", "logit"])
def test_decays_of_every_gate(gate, dtype):
    # One step from 1 with x = 0 leaves the decay as the fp32 state.  From 1/2 on it is as exact as the
    # header says: an error of 1.9 x 2^-24, relative to 1 (the decay of a long memory).  Below, the instructions' errors: 2^-22 of the exponential with 1.5
    # |gate| 2^-24 of its argument, for logits also 2^-23 of the reciprocal and 2^-24 of its sum.  Below
    # 2^-126 it may be 0.
    g, v = every_gate(dtype, gate)
    st = torch.ones(1, g.numel(), device=DEV)
    ssd_i8.ssd_i8_gated_step(st, torch.zeros_like(g)[None], g[None], gate_form=gate)
    a = ref.decay(v, gate)[0]
    small = 2.0 ** -22 + 1.5 * np.abs(v) * 2.0 ** -24 + (2.0 ** -23 + 2.0 ** -24 if gate == "logit" else 0)
    small = np.minimum(small, 1.0)
    within(st[0], a, np.where(a >= 0.5, 1.9 * 2.0 ** -24, small * a) + 2.0 ** -126, "decay")


@pytest.mark.parametrize("parts", ["chunks", "whole"])
@pytest.mark.parametrize("dtype,memory", [("f16", 4400), ("bf16", 34000)])
def test_long_memory_in_16_bits(dtype, memory, parts):
    # Steady gates with the memories, in tokens, at which the decay's error reaches half a step of y.  Per
    # token and 2^-24 of the state: 1.9 of the decay, 0.5 of the step and 0.5 of the decays' product, and
    # for the joins of 16 tokens' maps less than 0.3.  Positive x: the state bounds every partial sum.
    l = 2 * memory
    d = 24 if parts == "chunks" else 64 * 200  # strips for every SM are not cut
    some = [0, 1, d // 2, d - 1]
    rng = np.random.default_rng(memory)
    gen = torch.Generator(device=DEV).manual_seed(memory)
    x = torch.rand(1, l, d, device=DEV, generator=gen).add_(0.5).div_(memory).to(ref.TYPES[dtype])
    g = torch.from_numpy(-rng.uniform(0.9, 1.1, d) / memory).to(ref.TYPES[dtype]).to(DEV).expand(1, l, d)
    assert (ssd_i8.ssd_i8_gated_scan_workspace_size(1, l, d, dtype) > 0) == (parts == "chunks")
    final = torch.empty(1, d, device=DEV)
    y = ssd_i8.ssd_i8_gated_scan(x, g, final_state=final)
    a = np.exp(f64(g[0, 0, some]))
    h = e = np.zeros(len(some))
    want, err = np.empty((2, l, len(some)))
    for t, row in enumerate(f64(x[0][:, some])):
        h = a * h + row
        e = a * e + 3.2 * 2.0 ** -24 * h
        want[t], err[t] = h, e
    within(y[0][:, some], want, err + ref.rounded(want, dtype), "y")
    within(final[0, some], h, e, "final_state")


def test_tensors_that_require_gradients(monkeypatch):
    # the values are those of any other call, nothing is recorded, and each call says so once
    import warnings
    x, g = draw(np.random.default_rng(3), (2, 70, 33), "log", "f32")
    dy = torch.randn_like(x)
    st = torch.randn(2, 33, device=DEV)
    spans = torch.empty(2, 2, 33, device=DEV)
    calls = {
        "ssd_i8_gated_scan": lambda x, g, dy: ssd_i8.ssd_i8_gated_scan(x, g, span_states=spans),
        "ssd_i8_gated_scan_bwd": lambda x, g, dy: ssd_i8.ssd_i8_gated_scan_bwd(dy, x, g, spans)[0],
        "ssd_i8_gated_step": lambda x, g, dy: ssd_i8.ssd_i8_gated_step(
            st.clone(), x[:, 0].contiguous(), g[:, 0].contiguous()),
        "ssd_i8_ckpt_pack": lambda x, g, dy: ssd_i8.ssd_i8_ckpt_pack(x)[0],
    }
    monkeypatch.setattr(ssd_i8, "_said", set())
    leaves = [t.clone().requires_grad_() for t in (x, g, dy)]
    for name, call in calls.items():
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            want = call(x, g, dy)
            with torch.no_grad():
                assert torch.equal(call(*leaves), want)
        with pytest.warns(UserWarning, match=name + " records no gradients"):
            got = call(*leaves)
        assert torch.equal(got, want) and not got.requires_grad
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            call(*leaves)
    # one leaf is enough
    monkeypatch.setattr(ssd_i8, "_said", set())
    with pytest.warns(UserWarning):
        ssd_i8.ssd_i8_gated_scan(x, leaves[1])
    monkeypatch.setattr(ssd_i8, "_said", set())
    with pytest.warns(UserWarning):
        ssd_i8.ssd_i8_gated_scan(x, g, init_state=st.clone().requires_grad_())


@pytest.mark.parametrize("tokens", [2 ** 31, 2 ** 32 + 8])
def test_sizes_past_32_bits_are_refused(tokens):
    # the second one's low 32 bits are a small scan, which must not be what runs; no memory behind them
    wide = lambda *s, **k: torch.zeros((1,) * len(s), device=DEV, **k).expand(*s)
    row, packed = wide(1, tokens, 1), wide(tokens, 1)
    cu = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    spans = torch.zeros(1, 1, 1, device=DEV)
    codes, exps = wide(1, tokens, 1, dtype=torch.int8), wide(1, -(-tokens // 16), 1, dtype=torch.uint8)
    many = torch.zeros(8, 1, device=DEV)
    for call in (lambda: ssd_i8.ssd_i8_gated_scan(row, row), lambda: ssd_i8.ssd_i8_gated_scan(packed, packed, cu),
                 lambda: ssd_i8.ssd_i8_gated_scan(wide(tokens, 8, 1), wide(tokens, 8, 1)),
                 lambda: ssd_i8.ssd_i8_gated_scan(many, many, wide(tokens + 1, dtype=torch.int32)),
                 lambda: ssd_i8.ssd_i8_gated_scan_bwd(row, row, row, spans),
                 lambda: ssd_i8.ssd_i8_gated_scan_bwd_ckpt(row, (codes, exps, codes, exps), spans),
                 lambda: ssd_i8.ssd_i8_gated_step(packed, packed, packed),
                 lambda: ssd_i8.ssd_i8_ckpt_pack(row), lambda: ssd_i8.ssd_i8_ckpt_unpack(codes, exps)):
        with pytest.raises(ssd_i8.SSDError) as err:
            call()
        assert err.value.status == 2
