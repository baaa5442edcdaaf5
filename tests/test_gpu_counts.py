"""Counts at the ends of int32 (a buffer that was never filled): refused like any others that do not fit, by the
tree masks and the compaction, and the other requests of the call are served.
"""
import numpy as np
import pytest
import torch

import oracle
import tensor_linear_layers_gb300 as tl
from test_gpu_kv_pages import bits, built, compact_case, dev, handle, run_compact, status  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("length", [LOW, LOW + 3, -1, HIGH])
def test_compaction_of_lengths_at_the_ends(length):
    h, bs, ctx, kept = handle(8, 2, 2), 16, [5, 20, 7], [[0, 2], [], [1, 3]]
    c = compact_case(h, ctx, [6, 6, 6], [[0, 2], [1, 5], [1, 3]], bs, 2, 9, True)
    c["lens"][1] = length
    before = [bits(x) for x in c["ck"] + c["cv"]]
    new, ws = run_compact(h, c)
    assert status(ws) == tl.TP_ERR_SHAPE and new.tolist() == [7, length, 9]
    for a, b in zip(before, c["ck"] + c["cv"]):
        np.testing.assert_array_equal(bits(b), oracle.compact(a, ctx, kept, c["src"], c["dst"], bs))


@pytest.mark.parametrize("qsl", [[0, HIGH, LOW], [0, LOW, 6], [0, 6, LOW], [LOW, 6, 12]])
def test_compaction_of_offsets_at_the_ends(qsl):
    h, bs = handle(8, 2, 2), 16
    c = compact_case(h, [5, 20], [6, 6], [[], []], bs, 1, 9, True, m=2)
    c["qsl"] = np.array(qsl)
    before = [bits(x) for x in c["ck"] + c["cv"]]
    _, ws = run_compact(h, c)
    assert status(ws) == tl.TP_ERR_SHAPE
    for a, b in zip(before, c["ck"] + c["cv"]):
        np.testing.assert_array_equal(bits(b), a)


def test_masks_of_counts_at_the_ends():
    parents = dev([-1, 0, -1, 0, 1])
    for qsl, lens in (([0, 2, 5], [LOW, 9]), ([0, 2, 5], [LOW + 1, 9]), ([0, HIGH, LOW], [9, 9]), ([LOW, 2, 5], [9, 9]),
                      ([HIGH, LOW, 5], [9, 9])):
        mask, pos = (torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((5, 1), (5,)))
        _, _, ws = tl.tree_mask(parents, dev(qsl), dev(lens), 4, out=(mask, pos))
        assert status(ws) == tl.TP_ERR_SHAPE
        good = qsl[1] == 2 and lens[1] == 9                  # the second request is whole
        assert (mask[:2] == 77).all() and (pos[:2] == 77).all()
        assert mask[2:, 0].tolist() == ([1, 3, 7] if good else [77] * 3)
        assert pos[2:].tolist() == ([6, 7, 8] if good else [77] * 3)
