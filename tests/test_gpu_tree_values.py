"""Tree attention where many drafted tokens' values are not finite, so that every lane of the warp that looks
over them changes its tile before the product reads it. Bits equal to the same call on finite values.
"""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_tree import build, built, check, handle, run, status  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nq,nkv,t,ctx,n", [
    (8, 2, 2, [120, 5], [30, 9]),          # one tile of rows
    (8, 2, 1, [300, 0], [200, 256]),       # groups of 256 rows, drafts over several chunks
])
def test_every_other_draft_not_finite_and_unseen(nq, nkv, t, ctx, n):
    bs = 16
    c = build(nq, nkv, t, ctx, n, bs, seed=140)
    rng = np.random.default_rng(7)
    # random masks over the even drafts only
    sees = [(rng.random((k, k)) < 0.5) & (np.arange(k) % 2 == 0) for k in n]
    words = -(-max(n) // 32)
    mask = torch.cat([torch.from_numpy(oracle.mask_words(s, words)) for s in sees]).cuda()
    h = handle(nq, nkv, t)
    clean, _ = run(h, c, mask=mask)
    check(clean, c, nq, nkv, t, sees)
    ck, cv = c["ck"].clone(), c["cv"].clone()
    for b, k in enumerate(n):
        for j in range(1, k, 2):
            s = oracle.slot_of(c["tables"], b, ctx[b] + j, bs)
            ck[:, s // bs, s % bs] = float("nan")
            cv[:, s // bs, s % bs] = (float("nan"), float("inf"), -float("inf"))[j % 3]
    d = dict(c, ck=ck, cv=cv)
    for _ in range(20):
        got, ws = run(h, d, mask=mask)
        assert status(ws) == 0 and torch.equal(got, clean)
