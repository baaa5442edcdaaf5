"""Elements from rotary_dim on are not rotated: whatever they hold (infinities, NaN, -0) stays theirs alone, in both
layouts, with and without a norm.

Without a norm they are copies: equal bits (a NaN stays a NaN). With one, a head that holds an infinity has an infinite
mean square: its finite elements become 0 with their sign, the infinite ones NaN; a head with a NaN is NaN throughout.
"""
import numpy as np
import pytest
import torch

import workloads
import tensor_linear_layers_gb300 as tl
from test_gpu_rope import built, gamma, handle, width  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu

NQ, NKV, T = 4, 2, 9
SPECIAL = (float("inf"), -float("inf"), float("nan"), -0.0)


def same(a, b):
    """Equal bits, any NaN for a NaN."""
    a, b = a.cpu(), b.cpu()
    return bool(((a.view(torch.int16) == b.view(torch.int16)) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("layout", [tl.TP_ROPE_HALF, tl.TP_ROPE_INTERLEAVED])
@pytest.mark.parametrize("hd,rd", [(128, 64), (128, 96), (128, 20), (128, 2), (128, 126), (64, 16), (72, 36), (256, 130)])
def test_unrotated_elements_stay_as_they_are(layout, hd, rd):
    h = handle(NQ, NKV, hd, 1)
    r = tl.Rope(4096, rd, layout=layout)
    qkv = workloads.draw((1, T, width(NQ, NKV, hd, 1)), hd + rd, 0)
    pos = torch.from_numpy(np.random.default_rng(rd).integers(1, 4096, T).astype(np.int32)).cuda()
    clean, _ = h.qk_norm_rope(qkv.cuda(), pos, r)
    heads = qkv.view(T, NQ + 2 * NKV, hd)
    for i in range(rd, hd):                                   # one in two pairs' partners, each kind in turn
        if (i // 2 + i) % 2:
            heads[:, :, i] = SPECIAL[(i // 2) % 4]
    out, ws = h.qk_norm_rope(qkv.cuda(), pos, r)
    got = out.view(T, -1, hd)
    assert int(ws[:4].view(torch.int32)) == 0
    assert same(got[..., rd:], heads[..., rd:])
    assert same(got[..., :rd], clean.view(T, -1, hd)[..., :rd])


@pytest.mark.parametrize("layout", [tl.TP_ROPE_HALF, tl.TP_ROPE_INTERLEAVED])
@pytest.mark.parametrize("rd", [64, 20])
def test_unrotated_elements_under_the_norm(layout, rd):
    hd = 128
    h = handle(NQ, NKV, hd, 1)
    r = tl.Rope(4096, rd, layout=layout, q_gamma=gamma(hd, 0).cuda())           # k heads are not normed
    qkv = workloads.draw((1, T, width(NQ, NKV, hd, 1)), rd, 0)
    heads = qkv.view(T, NQ + 2 * NKV, hd)
    heads[:, :, 100] = float("inf")
    heads[:, :, 103] = -0.0
    heads[5:, :, 110] = float("nan")
    out, _ = h.qk_norm_rope(qkv.cuda(), torch.arange(1, T + 1, dtype=torch.int32, device="cuda"), r)
    got = out.view(T, -1, hd)
    q = heads[:5, :NQ, rd:]
    assert same(got[:5, :NQ, rd:], torch.where(q.isinf(), float("nan"), q * 0.0))
    assert (got[:5, :NQ, :rd] == 0).all() and got[5:, :NQ].isnan().all()
    assert same(got[:, NQ:, rd:], heads[:, NQ:, rd:])
    assert torch.isfinite(got[:, NQ:NQ + NKV, :rd].float()).all()
