"""Host-side edges of the gated recurrence (no GPU, nothing launched)."""
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
