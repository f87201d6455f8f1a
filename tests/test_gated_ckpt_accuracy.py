"""How far gradients from 8-bit checkpoints are from the exact ones: the figures that the header gives, from
the 64-bit reference alone (the kernels are compared with its decoded values elsewhere).

The figures are properties of the format, with no bound to derive: codes round a block's values to half
a scale, a 64th to a 128th of its largest one.  They are asked for to the digit given, half of its last
place added."""
import numpy as np
import pytest
import torch

import gated_ref as ref


def off(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def gradients(gate, inp, resets, offsets=None, seed=0, l=800, d=64, spike=None):
    """(from checkpoints, exact) cases of bf16 values like those of the kernels' tests."""
    rng = np.random.default_rng(seed)
    bf16 = lambda v: torch.from_numpy(v).bfloat16().double().numpy()
    x = bf16(rng.laplace(size=(l, d)) * rng.uniform(0.2, 8, d))
    g = bf16(-np.logaddexp(0, rng.normal(-2, 0.5, (l, d))) * np.exp(rng.uniform(0, np.log(16), d))
             if gate == "log" else rng.normal(2, 2, (l, d)))
    if resets:
        g[50::100] = -1e4
    if spike is not None:
        g[spike[0]] = spike[1]
    dy = rng.normal(size=(l, d))
    exact = ref.Case(x, g, gate, inp, offsets).forward()
    coded = exact.rebuilt().backward(dy)
    return coded, exact.backward(dy)


@pytest.mark.parametrize("gate,inp,dx,dgate", [("log", "plain", 0.0035, 0.0105), ("log", "complement", 0.0065, 0.0105),
                                               ("logit", "plain", 0.0055, 0.0145),
                                               ("logit", "complement", 0.0095, 0.0145)])
def test_without_resets(gate, inp, dx, dgate):
    coded, exact = gradients(gate, inp, False)
    assert off(coded.dx, exact.dx) < dx and off(coded.dgate, exact.dgate) < dgate


@pytest.mark.parametrize("gate,inp,dx,dgate", [("log", "plain", 0.085, 0.175), ("log", "complement", 0.125, 0.175),
                                               ("logit", "plain", 0.035, 0.045),
                                               ("logit", "complement", 0.035, 0.045)])
def test_blocks_with_a_reset(gate, inp, dx, dgate):
    # a reset every 100 tokens, of the decay's lowest values: its block's scale is 2^-2
    coded, exact = gradients(gate, inp, True)
    rows = np.zeros(len(exact.dx), bool)
    for t in range(50, len(rows), 100):
        rows[t // 16 * 16:t // 16 * 16 + 16] = True
    e = ref.coded(ref.held_gate(exact.g, gate))[1]
    assert (e[50 // 16] == 127 - 2).all()
    got = ref.coded(ref.held_gate(exact.g, gate))[2]
    small = rows[:, None] & (np.abs(exact.g) < 0.125)
    assert small.any() and (got[small] == 0).all()
    assert off(coded.dx[rows], exact.dx[rows]) < dx and off(coded.dgate[rows], exact.dgate[rows]) < dgate


def test_sequences_that_meet_in_a_block_share_its_scale():
    # tokens 20 to 31, of the second sequence, share the block of the first one's token 18
    alone, exact = gradients("log", "complement", False, [0, 20, 40], l=40)
    beside, exact2 = gradients("log", "complement", False, [0, 20, 40], l=40, spike=(18, -8.0))
    rows = slice(20, 32)
    assert np.array_equal(exact.dx[rows], exact2.dx[rows])
    assert off(alone.dx[rows], exact.dx[rows]) < 0.01 < off(beside.dx[rows], exact.dx[rows]) < 0.35
    after = slice(32, 40)  # blocks of their own
    assert np.array_equal(alone.dx[after], beside.dx[after])
