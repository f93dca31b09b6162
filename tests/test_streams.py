"""Where the convenience calls of the binding take their memory when they run on a given stream
(CPU: torch's streams and allocation are replaced by records)."""
import contextlib

import pytest
import torch

from speculative_decoding_tree_mask_gb300 import binding as G


class Stream:
    cuda_stream = 7


class Raw:
    cuda_stream = 7


class Tensor:
    def __init__(self, pool, shape):
        self.pool, self.shape, self.users = pool, tuple(shape), []

    def record_stream(self, s):
        self.users.append(s)


class Input:
    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype, self.device = shape, dtype, "cuda:0"


class Handle:
    ptr, device, torch_device, attention_sizes, attention_bytes = None, 0, "cuda:0", None, 0


class Cache:
    H, D = 2, 64


x, rows = Input(2, 3, 4, 64), Input(2, 3, 64)
CALLS = {
    "verify_greedy": ("spec_verify_greedy",
                      lambda s: G.verify_greedy(Handle(), rows, x, x, stream=s)),
    "verify_sample": ("spec_verify_sample",
                      lambda s: G.verify_sample(Handle(), rows, x, x, 1.0, x, stream=s)),
    "verify_greedy_lazy": ("spec_verify_greedy_lazy",
                           lambda s: G.verify_greedy_lazy(Handle(), rows, x, x, stream=s)),
    "verify_sample_lazy": ("spec_verify_sample_lazy",
                           lambda s: G.verify_sample_lazy(Handle(), rows, x, x, 1.0, x, stream=s)),
    "build_tree_mask": ("spec_build_tree_mask",
                        lambda s: G.build_tree_mask(Handle(), Input(2, 3), stream=s)),
    "qk_norm_rope": ("spec_qk_norm_rope",
                     lambda s: G.qk_norm_rope(Handle(), x, x, None, x, stream=s)),
    "kv_load_fp4": ("spec_kv_load_fp4",
                    lambda s: G.kv_load_fp4(Handle(), Cache(), Input(2, 4), x, x, 5, stream=s)),
    "tree_attention_fp4": ("spec_tree_attention_fp4",
                           lambda s: G.tree_attention_fp4(Handle(), x, x, x, Cache(), x, x, x, 1.0,
                                                          stream=s)),
}


@pytest.mark.parametrize("stream", [None, Stream(), Raw()], ids=["none", "stream", "raw"])
@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_belongs_to_its_stream(monkeypatch, name, stream):
    """All memory that a call takes for itself comes from the stream it runs on, so that no
    earlier work of another stream is still to run on it; what it returns is noted as used by
    the current stream, where the caller may free it. Without a stream: the current one."""
    here = Stream()
    current, taken, given = [here], [], []

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()

    def empty(shape, dtype, device):
        taken.append(Tensor(current[-1], shape if isinstance(shape, tuple) else (shape,)))
        return taken[-1]

    def external(ptr, device=None):
        assert ptr == stream.cuda_stream
        return stream

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: here)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(G, "spec_tree_attention_workspace", lambda *a: 512)
    entry, call = CALLS[name]
    monkeypatch.setattr(G, entry, lambda *a, **kw: given.extend(list(a) + list(kw.values())))
    out = call(stream)
    out = list(out.values()) if isinstance(out, dict) else list(out)
    assert taken and all(any(t is g for g in given) for t in taken)
    assert all(t.pool is (here if stream is None else stream) for t in taken)
    if stream is not None:
        assert all(t.users == ([here] if any(t is o for o in out) else []) for t in taken)
        assert any(g is stream for g in given)


@pytest.mark.parametrize("name", ["kv_load_fp4", "tree_attention_fp4"])
def test_status_reaches_the_library(monkeypatch, name):
    """The convenience calls hand a status tensor on."""
    given, status = [], Tensor(None, (2,))
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: Tensor(None, (1,)))
    monkeypatch.setattr(G, "spec_tree_attention_workspace", lambda *a: 512)
    monkeypatch.setattr(G, "spec_" + name, lambda *a, **kw: given.extend([*a, *kw.values()]))
    if name == "kv_load_fp4":
        G.kv_load_fp4(Handle(), Cache(), Input(2, 4), x, x, 5, status=status)
    else:
        G.tree_attention_fp4(Handle(), x, x, x, Cache(), x, x, x, 1.0, status=status)
    assert any(g is status for g in given)
