"""Workspace of the attention's forward and backward by the batch's counts (no GPU)."""
import ctypes
import os
from ctypes import byref

import pytest
import torch

from equivariant_gnn_tensor_receiver_amd import tpconv as tp

pytestmark = pytest.mark.skipif(not os.path.exists(tp.LIB_PATH), reason="libtpconv.so not built")
if os.path.exists(tp.LIB_PATH):
    from equivariant_gnn_tensor_receiver_amd import attention as at

FAKE = ctypes.c_void_p(64).value


def sizes(n, graphs, y, heads=8, features=64):
    h = at.Attention(f"{features}x0e", f"{features}x0e", heads, x_dtype=y, y_dtype=y)
    b = at.Batch(n, torch.zeros(graphs + 1, dtype=torch.int32))
    return h.workspace_size(b, at.OP_FORWARD), h.workspace_size(b, at.OP_BACKWARD)


def test_a_forward_without_fp32_results_needs_room_for_the_sums_of_runs():
    """Only where a graph may be longer than a run of 4096 rows, and one copy of the output in fp32."""
    assert sizes(4096, 128, at.TPCONV_BF16)[0] == 0 and sizes(8192, 128, at.TPCONV_F32)[0] == 0
    assert sizes(8192, 128, at.TPCONV_BF16)[0] == 8192 * 64 * 4
    h = at.Attention("64x0e", "64x0e", 8, x_dtype=at.TPCONV_BF16, y_dtype=at.TPCONV_BF16)
    batch = at.AttentionBatch(128, 8192, FAKE, None, 0, None, None)
    inputs = at.AttentionInputs(FAKE, FAKE, FAKE, 0, 0, 0, None)
    L = at._lib()
    for ws, size in ((None, 0), (FAKE, 8192 * 64 * 4 - 1), (FAKE + 8, 1 << 40)):
        assert L.tpconv_attention_forward(h.handle, byref(batch), byref(inputs), FAKE, None, ws, size, None) == 4


def test_parts_of_long_graphs_are_at_most_eight_copies():
    n, f = 32768, 1024
    forward, backward = sizes(n, 1, at.TPCONV_F32, 16, f)
    copies = n * f * 4
    assert forward <= 8 * (copies + 16 * n * 8) and 3 * copies <= backward <= 3 * 8 * copies + 16 * n * 4
