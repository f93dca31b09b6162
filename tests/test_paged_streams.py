"""The convenience calls of the paged step take their memory from the stream they run on and hand a
status on (CPU: torch's streams and allocation are replaced by records)."""
import pytest

import test_streams as T
from speculative_decoding_tree_mask_gb300 import binding as G


class Handle(T.Handle):
    paged_sizes, paged_bytes = None, 0


x = T.Input(6, 4, 64)
CALLS = {
    "kv_append": ("spec_kv_append", lambda s: [G.kv_append(Handle(), x, x, x, None, x, x, stream=s)]),
    "paged_attention": ("spec_paged_attention",
                        lambda s: G.paged_attention(Handle(), x, T.Cache(), x, x, 1.0, stream=s)),
    "token_logprobs": ("spec_token_logprobs",
                       lambda s: G.token_logprobs(Handle(), T.Input(2, 3, 9), T.Input(2, 3), top=2,
                                                  stream=s)),
}


@pytest.mark.parametrize("stream", [None, T.Stream(), T.Raw()], ids=["none", "stream", "raw"])
@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_belongs_to_its_stream(monkeypatch, name, stream):
    monkeypatch.setitem(T.CALLS, name, CALLS[name])
    monkeypatch.setattr(G, "spec_paged_attention_workspace", lambda *a: 512)
    T.test_memory_of_a_call_belongs_to_its_stream(monkeypatch, name, stream)


@pytest.mark.parametrize("name", ["kv_append", "paged_attention"])
def test_status_reaches_the_library(monkeypatch, name):
    given, status = [], object()
    monkeypatch.setattr(G, "_new", lambda dev, stream, *specs, returned=True: [object() for _ in specs])
    monkeypatch.setattr(G, "spec_paged_attention_workspace", lambda *a: 512)
    monkeypatch.setattr(G, "spec_" + name, lambda *a, **kw: given.extend([*a, *kw.values()]))
    if name == "kv_append":
        G.kv_append(Handle(), x, x, x, None, x, x, status=status)
    else:
        G.paged_attention(Handle(), x, T.Cache(), x, x, 1.0, status=status)
    assert any(g is status for g in given)
