"""The verify-step operators on the GPU where their rules meet: pages given back before a window, rows and cells without
weight, far apart scores, and the edges of the tcgen05 attention kernel (more than 32 rows per kv head)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dflash_block_drafter_gb300 as D  # noqa: E402
import verify_ref as V  # noqa: E402
from test_gpu_verify import R, TYPES, attn_case, check_attn, ints, status  # noqa: E402,F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- windows
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,G", [(2, 4), (1, 5)])  # 32 and 40 rows per kv head: the warp-level and the tcgen05 kernel
@pytest.mark.parametrize("page,window", [(16, 1), (16, 33), (16, 100), (32, 70), (128, 20)])
@pytest.mark.parametrize("causal", [True, False])
def test_window_with_pages_given_back(R, d, heads, G, page, window, causal):
    """Pages that lie wholly before the window are gone from the table: no report, and the right outputs."""
    case = attn_case(d + window, d, heads, G, [300, 31, 4, 650], [8, 1, 4, 2], page, "bf16")
    cache, q, table, lens, offsets = case
    for s, n in enumerate(lens):
        first = max(int(n) - (int(offsets[s + 1] - offsets[s]) - 1 if causal else 0) - window, 0)  # that any row sees
        table[s, : first // page] = -1
    assert (table[0, 0] == -1) and (table[3, 0] == -1)
    check_attn(R, case, causal, window)
