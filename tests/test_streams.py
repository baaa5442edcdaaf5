"""The tensors that a call makes for itself (outputs, workspaces, tables) belong to the stream that it was given.

On the CPU, with the library and torch's streams replaced: each is allocated, and where need be zeroed, with the
call's stream current, so that neither the fill nor other work in the same memory can meet the kernels; and each is
marked as used by the stream the caller is on.
"""
import contextlib

import pytest
import torch

import tensor_linear_layers_gb300 as tl

CALLER = "the caller's stream"


class FakeStream:
    cuda_stream = 0x1234


class FakeLib:
    def __getattr__(self, name):
        def call(*args):
            if name.endswith(("workspace_size", "packed_weight_bytes")):
                for a in args:
                    if hasattr(a, "_obj"):
                        a._obj.value = 64
            return 0
        return call


@pytest.fixture
def made(monkeypatch):
    """[(stream current at the allocation, streams recorded on the tensor)] of what the calls make."""
    log, current, recorded = [], [CALLER], {}

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    def wrap(real):
        def make(*a, device=None, **kw):
            x = real(*a, **kw)
            log.append((current[0], recorded.setdefault(id(x), []), x))
            return x
        return make
    for name in ("zeros", "empty", "empty_like"):
        monkeypatch.setattr(torch, name, wrap(getattr(torch, name)))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[0])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: recorded.setdefault(id(self), []).append(s))
    monkeypatch.setattr(tl, "lib", lambda: FakeLib())
    monkeypatch.setattr(tl, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(tl, "_stream", lambda stream=None: 0)
    return log


def bf16(*shape):
    return torch.ones(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.ones(shape, dtype=torch.int32)


def handle(log):
    h = tl.TPLinear(tl.make_config(tl.TP_BLOCK_ATTN_PROJ, 1, 64, n_q_heads=2, n_kv_heads=1, head_dim=128),
                    [bf16(256, 64), bf16(128, 64), bf16(128, 64), bf16(64, 256)])
    h._dev, h._index = torch.device("cpu"), 0
    log.clear()
    return h


CACHE = (1, 4, 16, 1, 128)
CALLS = {
    "qk_norm_rope": lambda h, s: h.qk_norm_rope(bf16(1, 3, 512), i32(3), ROPE, stream=s),
    "kv_cache_copy_blocks": lambda h, s: h.kv_cache_copy_blocks(i32(1, 2), [bf16(*CACHE)], [bf16(*CACHE)], stream=s),
    "kv_cache_compact": lambda h, s: h.kv_cache_compact(i32(2), i32(1), i32(1, 3), i32(1, 4), i32(1, 4), [bf16(*CACHE)],
                                                        [bf16(*CACHE)], stream=s),
    "tree_attention": lambda h, s: h.tree_attention(bf16(1, 3, 512), i32(2), i32(1), i32(1, 4), i32(3, 1), bf16(*CACHE),
                                                    bf16(*CACHE), 3, 64, stream=s),
    "tree_mask": lambda h, s: tl.tree_mask(i32(3), i32(2), i32(1), 3, stream=s),
    "Rope": lambda h, s: tl.Rope(16, 128, stream=s),
}
MADE = {"qk_norm_rope": 2, "kv_cache_copy_blocks": 1, "kv_cache_compact": 2, "tree_attention": 2, "tree_mask": 3, "Rope": 1}


class ROPE:
    args = None

    @staticmethod
    def check(index, head_dim):
        pass


@pytest.mark.parametrize("name", CALLS)
def test_made_on_the_calls_stream(made, name):
    h, st = handle(made), FakeStream()
    keep = CALLS[name](h, st)
    assert keep is not None
    assert [on is st for on, _, _ in made] == [True] * MADE[name]
    assert all(recorded == [CALLER] for _, recorded, _ in made)


@pytest.mark.parametrize("name", CALLS)
def test_made_on_the_current_stream_without_one(made, name):
    CALLS[name](handle(made), None)
    assert [(on, recorded) for on, recorded, _ in made] == [(CALLER, [])] * MADE[name]


# ------------------------------------------------------------------ the blocks, the layer, the cache and the captures
def block(kind, flags=0, n_experts=0):
    w = {tl.TP_BLOCK_MLP: [bf16(128, 64), bf16(128, 64), bf16(64, 128)],
         tl.TP_BLOCK_ATTN_PROJ: [bf16(256, 64), bf16(128, 64), bf16(128, 64), bf16(64, 256)],
         tl.TP_BLOCK_MOE: [bf16(2, 128, 64), bf16(2, 128, 64), bf16(2, 64, 128)]}[kind]
    cfg = tl.make_config(kind, 1, 64, 128, 2, 1, 128, flags=flags, n_experts=n_experts)
    return tl.TPLinear(cfg, w, bf16(64) if flags else None)


def mlp():
    return block(tl.TP_BLOCK_MLP, tl.TP_FLAG_HAS_NORM)


def attn():
    return block(tl.TP_BLOCK_ATTN_PROJ, tl.TP_FLAG_HAS_NORM)


BLOCK_CALLS = {  # handle, call, tensors made
    "weights": (lambda: None, lambda h, s: tl.TPLinear(tl.make_config(tl.TP_BLOCK_MLP, 1, 64, 128),
                                                       [bf16(128, 64), bf16(128, 64), bf16(64, 128)], stream=s), 2),
    "mlp_forward": (mlp, lambda h, s: h.mlp_forward(bf16(3, 64), bf16(3, 64), stream=s), 4),
    "mlp_forward_no_alloc": (mlp, lambda h, s: h.mlp_forward_no_alloc(bf16(3, 64), bf16(3, 64), stream=s), 3),
    "gate_up": (mlp, lambda h, s: h.gate_up(bf16(3, 64), stream=s), 2),
    "down": (mlp, lambda h, s: h.down(bf16(1, 3, 128), bf16(3, 64), stream=s), 3),
    "moe_forward": (lambda: block(tl.TP_BLOCK_MOE, n_experts=2),
                    lambda h, s: h.moe_forward(bf16(3, 64), i32(3, 2), torch.ones(3, 2), stream=s), 2),
    "attn_proj_forward": (attn, lambda h, s: h.attn_proj_forward(bf16(3, 64), bf16(1, 3, 256), stream=s), 3),
    "attention_forward": (attn, lambda h, s: h.attention_forward(bf16(1, 3, 512), i32(2), 3, stream=s), 2),
    "kv_cache_write": (attn, lambda h, s: h.kv_cache_write(bf16(1, 3, 512), i32(3), bf16(*CACHE), bf16(*CACHE), stream=s), 1),
    "paged_attention": (attn, lambda h, s: h.paged_attention(bf16(1, 3, 512), i32(2), i32(1), i32(1, 4), bf16(*CACHE),
                                                             bf16(*CACHE), 3, 64, stream=s), 2),
    "layer": (lambda: tl.TPLayer(attn(), mlp(), 8), lambda h, s: h.forward(bf16(3, 64), None, i32(2), 3, stream=s), 6),
    "add_rms_norm": (lambda: None, lambda h, s: tl.add_rms_norm(bf16(3, 64), None, bf16(64), 1e-5, stream=s), 2),
    "capture_rows": (lambda: None, lambda h, s: tl.capture_rows(i32(3), i32(3), torch.ones(2, dtype=torch.int64),
                                                                [bf16(3, 64)], [0], 0, 4, stream=s), 4),
}


@pytest.mark.parametrize("name", BLOCK_CALLS)
@pytest.mark.parametrize("given", [True, False])
def test_the_blocks_calls(made, name, given):
    make, call, n = BLOCK_CALLS[name]
    h, st = make(), FakeStream() if given else None
    made.clear()
    keep = call(h, st)
    assert keep is not None
    assert [on for on, _, _ in made] == [st if given else CALLER] * n
    assert all(recorded == ([CALLER] if given else []) for _, recorded, _ in made)


def test_a_cached_workspace_outlives_the_calls_of_other_streams(made):
    h, a, b = mlp(), FakeStream(), FakeStream()
    ws = h.workspace(8, a)
    h.mlp_forward(bf16(3, 64), stream=b)
    (recorded,) = [r for _, r, x in made if x is ws]
    assert h.workspace(8) is ws and recorded == [CALLER, b]


@pytest.mark.parametrize("given", [True, False])
def test_routing_arrays_of_other_strides_last_until_the_launch(made, monkeypatch, given):
    # copies made of ids and gates that are not contiguous: both alive, and whole, when the library reads them
    import ctypes
    seen = {}

    class Reads(FakeLib):
        @staticmethod
        def tp_moe_forward(h, T, k, x, ids, gates, *rest):
            seen["ids"] = list((ctypes.c_int32 * (T * k)).from_address(ids.value))
            seen["gates"] = list((ctypes.c_float * (T * k)).from_address(gates.value))
            return 0
    monkeypatch.setattr(tl, "lib", lambda: Reads())
    copies, real, st = [], torch.Tensor.contiguous, FakeStream() if given else None
    monkeypatch.setattr(torch.Tensor, "contiguous", lambda self: copies.append(torch.cuda.current_stream()) or real(self))
    h, T = block(tl.TP_BLOCK_MOE, n_experts=2), 37
    ids, gates = torch.arange(2 * T, dtype=torch.int32).view(2, T).t(), torch.arange(2 * T).float().view(2, T).t() + 0.5
    for _ in range(20):
        h.moe_forward(bf16(T, 64), ids, gates, stream=st)
        assert seen == {"ids": ids.flatten().tolist(), "gates": gates.flatten().tolist()}
    assert set(copies) == {st if given else CALLER}
