"""As test_streams.py, for the calls of the 8-bit cache and the attention of chunks: what a call makes for itself
belongs to the stream that it was given."""
import pytest
import torch

import tensor_linear_layers_gb300 as tl
from test_streams import CACHE, CALLER, FakeStream, bf16, handle, i32, made  # noqa: F401 (made: the fixture)


def quant():
    codes = [torch.zeros(CACHE, dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2)]
    return (*codes, *(torch.zeros(CACHE[:-1], dtype=torch.uint8) for _ in range(2)))


CALLS = {  # call, tensors made
    "kv_quant_cache": (lambda h, q, s: h.kv_quant_cache(4, 16, stream=s), 4),
    "kv_quant_write": (lambda h, q, s: h.kv_quant_write(bf16(1, 3, 512), i32(3), *q, stream=s), 1),
    "kv_quant_read": (lambda h, q, s: h.kv_quant_read(i32(5), *q, stream=s), 3),
    "chunk_attention": (lambda h, q, s: h.chunk_attention(bf16(1, 3, 512), i32(2), i32(1), i32(1, 4), bf16(*CACHE),
                                                          bf16(*CACHE), 3, 64, 16, 1, stream=s), 2),
    "chunk_attention_q8": (lambda h, q, s: h.chunk_attention(bf16(1, 3, 512), i32(2), i32(1), i32(1, 4), q[0], q[1], 3, 64,
                                                             scales_k=q[2], scales_v=q[3], stream=s), 2),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("given", [True, False])
def test_made_on_the_calls_stream(made, name, given):
    call, n = CALLS[name]
    h, q, st = handle(made), quant(), FakeStream() if given else None
    made.clear()
    keep = call(h, q, st)
    assert keep is not None
    assert [on for on, _, _ in made] == [st if given else CALLER] * n
    assert all(recorded == ([CALLER] if given else []) for _, recorded, _ in made)


def test_null_handles_are_refused():
    import ctypes
    from tensor_linear_layers_gb300 import _build
    _build.build()
    L, p, b = tl.lib(), ctypes.c_void_p(0x10000), ctypes.c_int64()
    assert L.tp_kv_quant_write(None, 4, p, p, p, p, p, p, 8, 16, p, 16, None) == tl.TP_ERR_ARG
    assert L.tp_kv_quant_read(None, 4, p, p, p, p, p, 8, 16, p, p, p, 16, None) == tl.TP_ERR_ARG
    assert L.tp_chunk_attention_workspace_size(None, 1, 1, 1, ctypes.byref(b)) == tl.TP_ERR_ARG
    assert L.tp_chunk_attention(None, 4, p, p, p, 1, 1, 64, p, 4, 0, 0, p, p, None, None, 8, 16, p, p, 1 << 20,
                                None) == tl.TP_ERR_ARG
