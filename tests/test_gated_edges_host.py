"""Host-side edges of the gated recurrence (no GPU, nothing launched)."""
import os
import subprocess

import pytest
import torch

from quantized_mamba_ssd_b200 import build as qbuild
from quantized_mamba_ssd_b200 import ssd_i8
from test_gated_host import GB, bwd, scan

# placeholder pointers: only where no GPU could be reached by them
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-only argument checks run where no GPU is present")

OK, REFUSED, ACCEPTED = 0, 1, 4  # an accepted call fails at its launch (SSD_ERR_CUDA) without a GPU


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return ssd_i8.library()


def test_rows_without_a_sequence_are_not_skipped_where_something_is_written(lib):
    none = dict(batch=1, cu=11 * GB, nseq=0)
    q = [6 * GB, 7 * GB, 8 * GB, 9 * GB]
    assert scan(lib, **none) == OK
    assert scan(lib, **none, spans=10 * GB) == ACCEPTED
    assert scan(lib, **none, q=q) == ACCEPTED
    assert scan(lib, **none, spans=10 * GB, l=0) == OK  # neither a span nor a block
    assert scan(lib, **none, spans=3 * GB) == REFUSED   # on y
    assert bwd(lib, **none) == OK
    assert bwd(lib, True, **none) == OK


def spans_of(at, bs, ts, batch, tokens, width):
    return [(at + i * bs + j * ts, at + i * bs + j * ts + width) for i in range(batch) for j in range(tokens)]


def share(a, b):
    return any(lo < hi2 and lo2 < hi for lo, hi in a for lo2, hi2 in b)


def test_overlap_of_two_halves_of_one_buffer(lib):
    # disjoint output rows that the header allows, and each moved by one row or element onto the other
    b, l, d, e = 2, 100, 64, 4
    layouts = {  # (batch stride, token stride, distance of the second rows), in elements
        "stack [b,2,l,d]": (2 * l * d, d, l * d),
        "halves of the tokens of [b,2l,d]": (2 * l * d, d, l * d),
        "time-major stack [l,2,b,d]": (d, 2 * b * d, b * d),
        "columns of [b,l,2d], a batch pitch off the token pitch": (2 * l * d + 20, 2 * d, d),
        "columns of [b,l,2d]": (2 * l * d, 2 * d, d),
        "rows between rows": (l * d * 2, 2 * d, d),
    }
    for name, (bs, ts, off) in layouts.items():
        def call(off, which):
            first, second = [GB, bs, ts], [GB + off * e, bs, ts]
            far = dict(batch=b, l=l, d=d)
            if which == "dx dgate":
                return bwd(lib, **far, dy=[2 * GB, l * d, d], x=[3 * GB, l * d, d], gate=[4 * GB, l * d, d],
                           dx=first, dgate=second)
            return scan(lib, **far, x=first, gate=[2 * GB, l * d, d], y=second)
        for which in ("dx dgate", "x y"):
            assert call(off, which) == ACCEPTED, (name, which)
            for wrong in (0, off - 1, off + bs if bs < ts else off + 1, off + ts):
                a, c = spans_of(0, bs, ts, b, l, d), spans_of(wrong, bs, ts, b, l, d)
                assert call(wrong, which) == (REFUSED if share(a, c) else ACCEPTED), (name, which, wrong)
            assert call(off - 1, which) == REFUSED


def test_overlap_against_every_byte(lib):
    # x and y rows of random layouts in one small buffer: those of equal strides (or without one) are
    # told apart byte by byte, others may be refused though they only interleave
    import random
    rng = random.Random(7)
    seen = {OK: 0, REFUSED: 0, ACCEPTED: 0}
    e, told = 4, 0
    for _ in range(6000):
        b, l, d = rng.randint(1, 4), rng.randint(1, 5), rng.randint(1, 4)
        if rng.random() < 0.5:
            ts = rng.randint(d, 3 * d)
            bs = rng.randint((l - 1) * ts + d, (l + 1) * ts + 2 * d)
        else:
            bs = rng.randint(d, 3 * d)
            ts = rng.randint((b - 1) * bs + d, (b + 1) * bs + 2 * d)
        xs = [bs, ts] if rng.random() < 0.7 else [rng.choice([0, bs, rng.randint(0, 40)]), rng.choice([0, ts])]
        off = rng.randint(-60, 60)
        x = spans_of(4000 + off * e, xs[0] * e, xs[1] * e, b, l, d * e)
        y = spans_of(4000, bs * e, ts * e, b, l, d * e)
        got = scan(lib, batch=b, l=l, d=d, x=[GB + 4000 + off * e, *xs], y=[GB + 4000, bs, ts],
                   gate=[2 * GB, l * d, d])
        seen[got] += 1
        if share(x, y):
            assert got == REFUSED, (b, l, d, bs, ts, xs, off)
        elif (b == 1 or xs[0] in (0, bs)) and (l == 1 or xs[1] in (0, ts)):
            told += 1
            assert got == ACCEPTED, (b, l, d, bs, ts, xs, off)
    assert seen[OK] == 0 and told > 1500 and seen[REFUSED] > 1000
    # contiguous states in the gaps of y's rows
    for _ in range(2000):
        b, l, d = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 3)
        ts = rng.randint(d, 4 * d)
        bs = (l - 1) * ts + d + rng.randint(0, 12)
        off = rng.randint(-10, 60)
        y = spans_of(4000, bs * e, ts * e, b, l, d * e)
        f = [(4000 + off * e, 4000 + (off + b * d) * e)]
        got = scan(lib, batch=b, l=l, d=d, x=[3 * GB, l * d, d], gate=[2 * GB, l * d, d],
                   y=[GB + 4000, bs, ts], final=GB + 4000 + off * e)
        assert got == (REFUSED if share(y, f) else ACCEPTED), (b, l, d, bs, ts, off)


def test_overlap_of_far_rows(lib):
    # the second rows lie 2^62 bytes behind the first
    far = dict(batch=2, l=1, d=4, x=[GB, 1 << 60, 4], gate=[GB + 32, 1 << 60, 4], ws=None)
    assert scan(lib, **far, y=[GB, 1 << 60, 4]) == REFUSED
    assert scan(lib, **far, y=[GB + 12, 1 << 60, 4]) == REFUSED
    assert scan(lib, **far, y=[GB + 16, 1 << 60, 4]) == ACCEPTED
    assert scan(lib, **far, y=[GB, 4, 4]) == REFUSED


def test_workspace_of_sizes_past_32_bits(lib):
    f = ssd_i8.ssd_i8_gated_scan_workspace_size
    assert f(1, 20000, 4, "f32") > 0
    for sizes in ((1, 2 ** 32 + 20000, 4), (2 ** 32 + 1, 20000, 4), (1, 20000, 2 ** 32 + 4),
                  (1, 20000 - 2 ** 32, 4), (1, 2 ** 31, 4)):
        assert f(*sizes, "f32") == 0


DEVICES = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"
int main() {
    static ssd::PerDevice sms;
    int asked = 0, answers[3] = {0, 132, 148};
    auto get = [&](int dev) { return sms.get(dev, 99, [&](int d) { ++asked; return answers[d % 3]; }); };
    // the first device cannot be asked yet: the fallback, which is not kept
    if (get(0) != 99 || get(0) != 99 || asked != 2) return 1;
    if (get(1) != 132 || get(2) != 148 || asked != 4) return 2;
    answers[0] = 160;
    if (get(0) != 160 || asked != 5) return 3;
    // each device keeps its own
    answers[0] = answers[1] = answers[2] = 1;
    if (get(0) != 160 || get(1) != 132 || get(2) != 148 || asked != 5) return 4;
    if (get(-1) != 99 || asked != 5) return 5;                            // no current device
    if (get(64) != 1 || get(64) != 1 || get(1000) != 1 || asked != 8) return 6;  // asked every time
    static ssd::PerDevice other;
    std::vector<std::thread> threads;
    int bad[8] = {};
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([&bad, t] {
            for (int i = 0; i < 6400; ++i) bad[t] += other.get(i % 64, 0, [](int d) { return d + 1; }) != i % 64 + 1;
        });
    for (auto& t : threads) t.join();
    for (int b : bad) if (b) return 7;
    return 0;
}
"""


def test_a_device_keeps_its_own_number(tmp_path):
    # what the scans ask of a device, compiled alone: no machine here has two kinds of GPU
    src, exe = tmp_path / "devices.cpp", tmp_path / "devices"
    src.write_text(DEVICES)
    csrc = os.path.join(os.path.dirname(qbuild.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I", csrc, "-o", str(exe), str(src)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
