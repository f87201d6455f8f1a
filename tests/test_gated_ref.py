"""CPU pins of the gated recurrence's 64-bit reference: its gradients against differences of the
forward pass, a packed row against separate sequences, and the checkpoint's rule."""
import numpy as np
import pytest

import gated_ref as ref


def case(gate, inp, l=9, d=4, seed=0, offsets=None, init=True):
    rng = np.random.default_rng(seed)
    g = -rng.exponential(0.5, (l, d)) if gate == "log" else rng.normal(1, 2, (l, d))
    n = 1 if offsets is None else len(offsets) - 1
    return ref.Case(rng.normal(size=(l, d)), g, gate, inp, offsets,
                    rng.normal(size=(n, d)) if init else None)


@pytest.mark.parametrize("offsets", [None, [0, 3, 3, 8]])
@pytest.mark.parametrize("inp", ["plain", "complement"])
@pytest.mark.parametrize("gate", ["log", "logit"])
def test_gradients_match_differences(gate, inp, offsets):
    c = case(gate, inp, offsets=offsets).forward()
    rng = np.random.default_rng(1)
    dy, dfin = rng.normal(size=c.x.shape), rng.normal(size=c.init.shape)
    c.backward(dy, dfin)

    def loss(**over):
        a = dict(x=c.x, g=c.g, init=c.init)
        a.update(over)
        k = ref.Case(a["x"], a["g"], gate, inp, offsets, a["init"]).forward()
        return np.sum(dy[c.valid] * k.y[c.valid]) + np.sum(dfin * k.final)

    # central differences: the truncation is step^2 times a third derivative of order 1 (these
    # gates and values), the rounding 2^-52 / step
    step = 1e-5
    for name, grad in (("x", c.dx), ("g", c.dgate), ("init", c.dinit)):
        base = {"x": c.x, "g": c.g, "init": c.init}[name]
        for i in np.ndindex(base.shape):
            if name != "init" and not c.valid[i[0]]:
                continue
            up, down = base.copy(), base.copy()
            up[i] += step
            down[i] -= step
            num = (loss(**{name: up}) - loss(**{name: down})) / (2 * step)
            assert abs(num - grad[i]) < 1e-8 * max(1.0, abs(grad[i])) * 10, (name, i)


def test_packed_row_is_its_sequences():
    off = [0, 0, 4, 5, 9]
    c = case("log", "complement", offsets=off).forward()
    for s, i, j in c.seqs:
        if i == j:
            assert np.array_equal(c.final[s], c.init[s])
            continue
        one = ref.Case(c.x[i:j], c.g[i:j], "log", "complement", None, c.init[s:s + 1]).forward()
        assert np.array_equal(one.y, c.y[i:j]) and np.array_equal(one.final[0], c.final[s])


def test_checkpoint_rule():
    v = np.zeros((16 * 5 + 3, 1))
    v[0], v[16], v[32], v[48] = 1.0, 1.9921875, 2.0, 3e-41
    v[64] = np.inf
    v[80:, 0] = [0.3, -5.0, 0.02]
    q, e, val = ref.coded(v)
    # 1 = 64 * 2^-6; 127.5 scales stay at 127; 2 begins the next exponent; scales stop at 2^-126; a
    # block that is not finite is NaN
    assert list(e[:, 0]) == [121, 121, 122, 1, 255, 123]
    assert q[0] == 64 and q[16] == 127 and q[32] == 64 and np.isnan(val[64:80]).all()
    assert np.abs(val[80:] - v[80:]).max() <= 2.0 ** (123 - 127) / 2
