"""Host-side sizes of the operators' workspaces: one made for the largest batch serves every
smaller one, so the size must not fall as the batch grows."""
import pytest

import sparse_mixture_experts_argmax_b200 as swl
from sparse_mixture_experts_argmax_b200 import build as swl_build


@pytest.fixture(scope="module", autouse=True)
def _library():
    swl_build.build()


@pytest.mark.parametrize("dtype", [swl.SWL_F32, swl.SWL_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,O", [(1, 8), (3, 136), (17, 1032), (128, 4096), (2048, 512)])
def test_grouped_workspace_never_falls_with_more_rows(N, O, dtype):
    edge = 40 * N                        # the tiles change here
    near = range(max(0, edge - 130), edge + 400)
    far = [edge * k // 7 for k in range(1, 40)]
    rows = sorted({0, 1, 63, 64, 65, 255, 256, 257, *near, *far, 1 << 20})
    sizes = [swl.switch_layer_grouped_workspace_size(R, 64, O, N, dtype) for R in rows]
    for R, small, R2, large in zip(rows, sizes, rows[1:], sizes[1:]):
        assert small <= large, (R, R2)
