"""Host-side refusals of the gated recurrence and the checkpoints (no GPU, nothing launched)."""
import ctypes

import pytest
import torch

from quantized_mamba_ssd_b200 import build as qbuild
from quantized_mamba_ssd_b200 import ssd_i8

# placeholder pointers: only where no GPU could be reached by them
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-only argument checks run where no GPU is present")

GB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return ssd_i8.library()


def rows(at, l=8, d=4):
    return [at, l * d, d]


def scan(lib, **over):
    a = dict(x=rows(GB), gate=rows(2 * GB), y=rows(3 * GB), batch=2, l=8, d=4, cu=None, nseq=0,
             form=0, io=0, init=None, final=None, spans=None, q=[None] * 4, ws=20 * GB, wsb=1 << 24)
    a.update(over)
    return lib.ssd_i8_gated_scan(*a["x"], *a["gate"], *a["y"], a["batch"], a["l"], a["d"],
                                 a["cu"], a["nseq"], a["form"], a["io"], a["init"], a["final"],
                                 a["spans"], *a["q"], a["ws"], a["wsb"], None)


def bwd(lib, ckpt=False, **over):
    a = dict(dy=rows(GB), x=rows(2 * GB), gate=rows(3 * GB), dx=rows(4 * GB), dgate=rows(5 * GB),
             q=[6 * GB, 7 * GB, 8 * GB, 9 * GB], batch=2, l=8, d=4, cu=None, nseq=0, form=0, io=0,
             init=None, spans=10 * GB, dfinal=None, dinit=None, ws=20 * GB, wsb=1 << 24)
    a.update(over)
    ins = a["q"] if ckpt else a["x"] + a["gate"]
    f = lib.ssd_i8_gated_scan_bwd_ckpt if ckpt else lib.ssd_i8_gated_scan_bwd
    return f(*a["dy"], *ins, *a["dx"], *a["dgate"], a["batch"], a["l"], a["d"], a["cu"],
             a["nseq"], a["form"], a["io"], a["init"], a["spans"], a["dfinal"], a["dinit"], a["ws"],
             a["wsb"], None)


SHAPES = [
    (dict(batch=-1), 1), (dict(l=-1), 1), (dict(d=0), 1), (dict(nseq=-1), 1),
    (dict(nseq=1), 1),                       # nseq without cu_seqlens
    (dict(cu=11 * GB, nseq=3), 1),           # cu_seqlens with batch 2
    (dict(cu=11 * GB + 2, nseq=3, batch=1), 1),  # misaligned offsets
    (dict(form=2), 1), (dict(form=32), 1), (dict(io=2), 1), (dict(io=4), 1),
    (dict(l=0x7fffffff), 2),                 # token indices past 32 bits with the last tile
    (dict(batch=1 << 25, d=4), 2),           # 2^31 CTAs with 64 chunks a strip
]


@pytest.mark.parametrize("over,status", SHAPES + [
    (dict(x=[None, 32, 4]), 1), (dict(gate=[None, 32, 4]), 1), (dict(y=[None, 32, 4]), 1),
    (dict(x=[GB + 2, 32, 4]), 1),            # not aligned to its element
    (dict(x=[GB, -32, 4]), 1), (dict(gate=[2 * GB, 32, -4]), 1),
    (dict(y=[3 * GB, 32, 0]), 1),            # output rows that overlap one another
    (dict(y=[3 * GB, 31, 4]), 1), (dict(y=[3 * GB, 0, 4]), 1), (dict(y=[3 * GB, 32, 3]), 1),
    (dict(y=[3 * GB, 4, 7]), 1),             # time-major rows too close for 2 batches
    (dict(y=rows(GB)), 1), (dict(y=rows(2 * GB + 4)), 1),  # y on x, y inside gate
    (dict(y=[GB + 8, 96, 12], x=[GB, 96, 12]), 1),         # column slices that overlap
    (dict(init=12 * GB, final=12 * GB), 1), (dict(final=3 * GB), 1),
    (dict(init=12 * GB + 2), 1),
    (dict(spans=3 * GB), 1),
    (dict(q=[6 * GB, 7 * GB, 8 * GB, None]), 1),           # some of the checkpoint's tensors
    (dict(q=[6 * GB, 7 * GB, 6 * GB, 9 * GB]), 1),         # both codes in one place
])
def test_scan_refuses(lib, over, status):
    assert scan(lib, **over) == status


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("over,status", SHAPES + [
    (dict(dy=[None, 32, 4]), 1), (dict(dx=[None, 32, 4]), 1), (dict(dgate=[None, 32, 4]), 1),
    (dict(spans=None), 1), (dict(spans=10 * GB + 1), 1),
    (dict(dx=rows(GB)), 1), (dict(dgate=rows(4 * GB)), 1), (dict(dgate=rows(10 * GB)), 1),
    (dict(dx=[4 * GB, 0, 4]), 1),
    (dict(dfinal=12 * GB, dinit=12 * GB), 1), (dict(dinit=10 * GB), 1), (dict(dinit=13 * GB + 3), 1),
])
def test_backward_refuses(lib, ckpt, over, status):
    assert bwd(lib, ckpt, **over) == status


def test_backward_refuses_its_inputs(lib):
    assert bwd(lib, x=[None, 32, 4]) == 1
    assert bwd(lib, gate=[3 * GB, 32, -1]) == 1
    assert bwd(lib, dx=rows(2 * GB)) == 1
    for k in range(4):
        q = [6 * GB, 7 * GB, 8 * GB, 9 * GB]
        q[k] = None
        assert bwd(lib, True, q=q) == 1
    assert bwd(lib, True, dgate=rows(8 * GB)) == 1


LONG = dict(batch=1, l=20000, d=4, x=rows(GB, 20000), gate=rows(2 * GB, 20000))


@pytest.mark.parametrize("over,status", [
    (dict(ws=None), 3), (dict(wsb=16), 3), (dict(ws=20 * GB + 128), 3),  # missing, small, misaligned
])
def test_workspace_is_checked(lib, over, status):
    need = lib.ssd_i8_gated_scan_workspace_size(1, 20000, 4, 0)
    assert need > 512 and need % 512 == 0 and need <= 64 * 512
    assert scan(lib, **LONG, y=rows(3 * GB, 20000), **over) == status
    assert scan(lib, **LONG, y=[20 * GB - 256, 80000, 4]) == 1  # y runs into the workspace
    for ckpt in (False, True):
        assert bwd(lib, ckpt, **LONG, dy=rows(15 * GB, 20000), dx=rows(4 * GB, 20000),
                   dgate=rows(5 * GB, 20000), **over) == status
    f = lib.ssd_i8_gated_scan_workspace_size
    assert f(0, 20000, 4, 0) == f(1, -1, 4, 0) == f(1, 20000, 0, 0) == f(1, 20000, 4, 2) == 0
    assert f(64, 4096, 8192, 3) == 0  # enough strips for every SM


def test_nothing_to_do_is_ok(lib):
    for k in (scan, bwd):
        assert k(lib, batch=0) == 0
        assert k(lib, batch=1, cu=11 * GB, nseq=0) == 0
        assert k(lib, l=0) == 0


def test_step_and_checkpoint_refuse(lib):
    st = lib.ssd_i8_gated_step
    ok = [GB, 2 * GB, 3 * GB, 4 * GB, 2, 4, 0, 0, None]
    for at, v, status in ((0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (4, -1, 1),
                          (5, 0, 1), (6, 2, 1), (7, 2, 1), (0, GB + 2, 1), (3, GB, 1),
                          (3, 2 * GB, 1), (1, GB + 16, 1)):
        a = list(ok)
        a[at] = v
        assert st(*a) == status, (at, v)
    assert st(*ok[:4], 0, 4, 0, 0, None) == 0
    pk = lib.ssd_i8_ckpt_pack
    ok = [GB, 32, 4, 2, 8, 4, 0, 2 * GB, 3 * GB, None]
    for at, v, status in ((0, None, 1), (0, GB + 1, 1), (1, -1, 1), (2, -1, 1), (3, -1, 1),
                          (4, -1, 1), (5, 0, 1), (6, 2, 1), (7, None, 1), (8, None, 1),
                          (7, GB, 1), (8, 2 * GB, 1), (4, 0x7fffffff, 2)):
        a = list(ok)
        a[at] = v
        assert pk(*a) == status, (at, v)
    assert pk(*ok[:4], 0, *ok[5:]) == 0
    un = lib.ssd_i8_ckpt_unpack
    ok = [GB, 2 * GB, 2, 8, 4, 0, 3 * GB, None]
    for at, v, status in ((0, None, 1), (1, None, 1), (2, -1, 1), (3, -1, 1), (4, 0, 1),
                          (5, 7, 1), (6, None, 1), (6, 3 * GB + 2, 1), (6, GB, 1), (6, 2 * GB, 1)):
        a = list(ok)
        a[at] = v
        assert un(*a) == status, (at, v)
    assert un(*ok[:2], 0, *ok[3:]) == 0


def test_binding_refuses_cpu_tensors(lib):
    x = torch.zeros(1, 8, 4)
    for call in (lambda: ssd_i8.ssd_i8_gated_scan(x, x), lambda: ssd_i8.ssd_i8_ckpt_pack(x),
                 lambda: ssd_i8.ssd_i8_gated_step(x[0], x[0], x[0]),
                 lambda: ssd_i8.ssd_i8_gated_scan_bwd(x, x, x, x),
                 lambda: ssd_i8.ssd_i8_gated_scan("x", x)):
        with pytest.raises(ValueError):
            call()
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_workspace_size_of_the_binding(lib):
    assert ssd_i8.ssd_i8_gated_scan_workspace_size(1, 20000, 4, "f32") > 0
    assert ssd_i8.ssd_i8_gated_scan_workspace_size(64, 20000, 4096, "bf16") == 0  # strips enough
    with pytest.raises(ValueError):
        ssd_i8.ssd_i8_gated_scan_workspace_size(1, 20000, 4, "i8")
