"""Trees of about 100 drafted tokens, several requests one after another on every SM: while the values of one
item's drafted tokens are looked over, the next item's keys come, and none of them may be read early."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_tree import build, built, handle, run, status  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,ctx", [(100, 2028), (120, 2056), (128, 2048)])
def test_weights_of_the_key_chunks(n, ctx):
    # v of cached position j is 1 in dimension j / 128: the output is every chunk's share of the softmax
    reqs, heads = 40, 8
    c = build(heads, heads, 1, [ctx], [n], 16, seed=60)
    chunks, slots = ctx // 128, [oracle.slot_of(c["tables"], 0, j, 16) for j in range(ctx + n)]
    v = torch.zeros_like(c["cv"])
    for j, s in enumerate(slots[:chunks * 128]):
        v[0, s // 16, s % 16, :, j // 128] = 1
    many = dict(c, cv=v, tables=np.repeat(c["tables"], reqs, 0), lens=[ctx + n] * reqs, qsl=np.arange(reqs + 1) * n, n=[n] * reqs,
                T=reqs * n, qkv=c["qkv"].repeat(1, reqs, 1), parents=c["parents"] * reqs)
    out, ws = run(handle(heads, heads, 1), many)
    assert status(ws) == 0
    k = c["ck"].double()[0].reshape(-1, heads, 128)[torch.tensor(slots)]
    q = c["qkv"][0, :, :heads * 128].double().view(n, heads, 128)
    s = torch.einsum("nhd,lhd->nhl", q, k) / 128 ** 0.5
    sees = torch.ones(n, ctx + n, dtype=torch.bool)
    sees[:, ctx:] = torch.from_numpy(oracle.tree_sees(c["parents"][0]))
    p = s.masked_fill(~sees[:, None], -float("inf")).softmax(-1)
    want = p[..., :chunks * 128].view(n, heads, chunks, 128).sum(-1)
    got = out.double().cpu()[0].view(reqs, n, heads, 128)[..., :chunks]
    # P and the output are rounded to bf16, 2^-8 of each; scores in fp32 add some 2^-12
    assert float(((got - want) / want).abs().max()) <= 2.1 * 2.0 ** -8
