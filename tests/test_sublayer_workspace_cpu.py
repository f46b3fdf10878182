"""The workspace of the layer norm's gradient: one that is large enough for a call does for a
call of fewer rows of the same width and type."""
import pytest

from hyper_connection_mix_gb300 import build as hbuild
from hyper_connection_mix_gb300 import sublayer

# bytes a row: every width at which the kernels change, and some between
ROW_BYTES = [4, 32, 1024, 4096, 4100, 8192, 10240, 10244, 20480, 20484, 40960, 40964, 163840]
ROWS = sorted({*range(0, 6000, 7), *range(290, 720), 2432, 4863, 4864, 4865, 100000, (1 << 31) - 1})


@pytest.fixture(scope="module")
def workspace_bytes():
    hbuild.build()
    return sublayer.lib().hc_mix_layer_norm_workspace_bytes


@pytest.mark.parametrize("dtype", sublayer.TYPES)
@pytest.mark.parametrize("row", ROW_BYTES)
def test_never_falls_as_rows_are_added(workspace_bytes, row, dtype):
    need = [workspace_bytes(sublayer.TYPES[dtype], M, row // dtype.itemsize) for M in ROWS]
    assert need[0] == 0 and need == sorted(need)


def test_a_batch_and_its_last_part(workspace_bytes):
    """512 values of 16 bits: 304 rows once needed more than 700."""
    assert workspace_bytes(0, 304, 512) <= workspace_bytes(0, 700, 512)
