"""The layer harness's buffers, sized without a GPU (the queries then take a default SM count)."""
import pytest

import linear_attention_mixer_gb300 as K
from linear_attention_mixer_gb300 import layer as L


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_mixer_gb300 import build
    build.build()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shapes", [[(2048, 256), (256, 1024)], [(1152, 320), (320, 768)], [(7168, 2048)]])
@pytest.mark.parametrize("rows", [1, 40, 256, 700])
def test_the_workspace_serves_every_number_of_rows(fp8, shapes, rows):
    """The k split, and with it the need, does not grow with the rows: 60 rows may split where 256 do not."""
    need = K.kda_linear_fp8_workspace_bytes if fp8 else K.kda_linear_workspace_bytes
    ws = L.Products(shapes, rows, "cpu", fp8).ws
    for m in range(1, rows + 1):
        for N, Kw in shapes:
            assert ws.numel() >= need(m, N, Kw), (m, N, Kw)
