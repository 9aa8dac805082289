"""Memory that a call on a stream allocates comes from that stream's pool (no
GPU needed: the library's entry points are replaced, on CPU tensors)."""
import contextlib
import types

import pytest
import torch

from block_sparse_masked_blockmask_gb300 import _build, flexattn as fa

STREAM = 7


@pytest.fixture
def calls(monkeypatch):
    """Allocations as (shape, type, stream), and the conversions made outside of the stream's context."""
    _build.build()
    real = fa.load_library()
    seen = types.SimpleNamespace(taken=[], elsewhere=[], inside=[])
    empty = torch.empty

    class Library:
        def __getattr__(self, name):
            return getattr(real, name) if name.startswith("flex_block_mask_sizes") else lambda *a: fa.FLEX_OK

    def taken(shape, dtype, device, stream):
        seen.taken.append((tuple(shape), dtype, stream))
        return empty(shape, dtype=dtype, device=device)

    def elsewhere(*a, **k):
        seen.elsewhere.append(a)
        return empty(*a, **k)

    @contextlib.contextmanager
    def on_stream(stream, device):
        seen.inside.append(stream)
        yield

    monkeypatch.setattr(fa, "load_library", lambda: Library())
    monkeypatch.setattr(fa, "_empty", taken)
    monkeypatch.setattr(fa, "_on_stream", on_stream, raising=False)
    monkeypatch.setattr(fa, "_call", lambda device, f, *a: f(*a))
    monkeypatch.setattr(fa, "_device_guard", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(fa, "_stream_handle", lambda stream, device: stream)
    monkeypatch.setattr(torch, "empty", elsewhere)
    return seen


B, H, S, D = 2, 3, 200, 64


def mask(**more):
    return fa.flex_block_mask_create(fa.FLEX_MASK_CAUSAL, B, H, S, S, device="cpu", stream=STREAM, **more)


def check(seen, count):
    assert not seen.elsewhere
    assert len(seen.taken) == count and all(s == STREAM for _, _, s in seen.taken), seen.taken


def test_block_mask_and_its_transpose(calls):
    bm = mask()
    check(calls, 4)
    fa.flex_block_mask_transpose(bm, stream=STREAM)
    check(calls, 8)


def test_document_ids_are_converted_on_the_stream(calls):
    ids = torch.zeros((B, S), dtype=torch.int64)
    bm = fa.flex_block_mask_create(fa.FLEX_MASK_DOCUMENT, B, H, S, S, doc_ids=ids, stream=STREAM)
    assert bm.doc_ids.dtype == torch.int32
    assert calls.inside == [STREAM]


def test_forward(calls):
    q = torch.zeros((B, H, S, D))
    bm = mask()
    fa.flex_attention_fwd(q, q, q, bm, stream=STREAM)
    check(calls, 6)
    fa.flex_attention_fwd_opts(q, q, q, bm, output_max=True, stream=STREAM)
    check(calls, 9)


def test_backward(calls):
    q = torch.zeros((B, H, S, D))
    bm = mask()
    bq = fa.flex_block_mask_transpose(bm, stream=STREAM)
    fa.flex_attention_bwd(q, q, q, q, torch.zeros((B, H, S)), q, bm, bq, stream=STREAM)
    check(calls, 12)
    assert ((B, H, S), torch.float32, STREAM) in calls.taken  # delta, which nobody holds after the call
