"""Attention of chunks of new tokens where a kv head has up to eight query rows (tp_chunk_attention's kernel of
warp-level products): one token's values and another's output."""
import pytest
import torch

import oracle
from test_gpu_chunk import build, check, run
from test_gpu_kv_quant import built, handle, status  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu


def scaled_k(c, power):
    """A copy of a call's arrays with the keys of every request's last token times 2^power."""
    name = "ck" if c["sk"] is None else "sk"
    x = c[name].clone()
    for b, L in enumerate(c["lens"]):
        s = oracle.slot_of(c["tables"], b, L - 1, c["bs"])
        at = x[:, s // c["bs"], s % c["bs"]]
        at.copy_(at.float() * 2.0 ** power if name == "ck" else at + power)
    return dict(c, **{name: x})


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("nq,nkv,n", [(8, 2, 2), (4, 4, 8), (6, 2, 2)])
@pytest.mark.parametrize("ctx", [[300], [5000], [700] * 40])
def test_a_later_token_leaves_an_earlier_ones_bits(nq, nkv, n, ctx, q8):
    # the last token's k is seen by itself alone, its q by no other: however large its scores are and wherever they
    # grow, the other rows of its group keep their references, and so every bit
    c = build(nq, nkv, 1, ctx, [n] * len(ctx), 16, seed=ctx[0] + n, q8=q8)
    h = handle(nq, nkv, 1)
    want = run(h, c)[0].clone()
    check(want, c)
    last = c["qsl"][1:] - 1
    others = [i for i in range(c["T"]) if i not in set(last.tolist())]
    for power in (3, 6, 9):
        d = scaled_k(c, power)
        d["qkv"] = c["qkv"].clone()
        d["qkv"][:, last, :nq * 128] *= 2.0 ** power
        out, ws = run(h, d)
        assert status(ws) == 0
        assert torch.equal(out[:, others], want[:, others]), power
