"""Forward and backward on a stream of their own, while torch's current stream
allocates and writes: equal bits to a run on one stream."""
import pytest
import torch

from block_sparse_masked_blockmask_gb300 import flexattn as fa

pytestmark = pytest.mark.gpu


def pool_of(x):
    """The stream whose pool a tensor's memory belongs to."""
    at = x.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= at < s["address"] + s["total_size"])


def inputs(B, H, S, D, dtype):
    gen = torch.Generator().manual_seed(S + D)
    return [torch.randn((B, H, S, D), generator=gen).to(dtype).cuda() for _ in range(4)]


def step(x, kind, stream, **more):
    q, k, v, g = x
    B, H, S, _ = q.shape
    bm = fa.flex_block_mask_create(kind, B, H, S, S, stream=stream, **more)
    bq = fa.flex_block_mask_transpose(bm, stream=stream)
    out, lse, top = fa.flex_attention_fwd_opts(q, k, v, bm, output_max=True, stream=stream)
    again, _ = fa.flex_attention_fwd(q, k, v, bm, stream=stream)
    grads = fa.flex_attention_bwd(q, k, v, out, lse, g, bm, bq, stream=stream)
    return (out, lse, top, again) + tuple(grads), bm, bq


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("kind,more", [(fa.FLEX_MASK_CAUSAL, {}), (fa.FLEX_MASK_WINDOW_SINKS, dict(window=128, sinks=4))],
                         ids=["causal", "window_sinks"])
def test_beside_work_of_the_current_stream(kind, more, dtype):
    x = inputs(1, 4, 4100, 64, dtype)
    want, _, _ = step(x, kind, None, **more)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        for _ in range(3):
            # blocks that the current stream is still writing go back to its pool ...
            for t in want:
                torch.empty_like(t).fill_(float("nan"))
            got, bm, bq = step(x, kind, handle, **more)
            # ... and what it takes next is written while the call may still run
            held = [torch.empty_like(t).fill_(float("nan")) for t in want]
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            del held
        assert {pool_of(t) for t in got} == {s.cuda_stream}
        assert {pool_of(t) for t in (bm.kv_num_blocks, bm.kv_indices, bq.q_indices)} == {s.cuda_stream}
        torch.cuda.synchronize()
    assert fa.flex_device_status() == fa.FLEX_OK


def test_document_ids_of_another_type():
    S = 512
    x = inputs(2, 2, S, 64, torch.bfloat16)
    ids = torch.arange(S, device="cuda").div(100, rounding_mode="floor").expand(2, S)  # int64, not contiguous
    want, _, _ = step(x, fa.FLEX_MASK_DOCUMENT, None, doc_ids=ids)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, bm, _ = step(x, fa.FLEX_MASK_DOCUMENT, s, doc_ids=ids)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert pool_of(bm.doc_ids) == s.cuda_stream
