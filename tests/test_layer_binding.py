"""What the binding of the layer operators refuses, and what it hands the library, without a GPU."""
import pytest
import torch

import precision_quantized_gemm_b200 as qg


def _call(T=3, B=1, Hq=2, **kw):
    """attend on CPU tensors: refused for the device unless something else is refused before."""
    cache = qg.Cache(qg.QG_FP8_DYNAMIC, 2, 16, 1, 64, device="cpu")
    ints = lambda *shape: torch.zeros(*shape, dtype=torch.int32)  # noqa: E731
    return qg.attend(cache, torch.zeros(T, Hq, 64, dtype=torch.bfloat16), ints(B + 1), ints(B), ints(B, 2), **kw)


def test_tokens_past_the_default_max_q():
    """Without max_q any sequence may have every token: more than the library takes are not cut silently."""
    with pytest.raises(ValueError, match="max_q"):
        _call(T=qg.QGEMM_ATTEND_MAX_Q + 1)
    with pytest.raises(ValueError, match="CUDA"):
        _call(T=qg.QGEMM_ATTEND_MAX_Q)
    with pytest.raises(ValueError, match="CUDA"):
        _call(T=qg.QGEMM_ATTEND_MAX_Q + 1, max_q=1)


def test_scratch_is_apart_from_the_zeroed_workspace():
    """What attend leaves in its scratch buffer never reaches a product's counters, in either order and growing."""
    ws = qg.Workspace("cpu")
    for nbytes in (64, 256, 128, 1024):
        p, n = ws.scratch(nbytes)
        assert n >= nbytes and ws.buf.data_ptr() == p
        ws.buf.fill_(0xff)
        z, m = ws.get(nbytes)
        assert m >= nbytes and z != p and ws.buf.data_ptr() == z and not ws.buf.any()
    assert ws.get(0) == (None, 0)


def test_an_outgrown_scratch_buffer_stays():
    """A captured graph holds its address."""
    ws = qg.Workspace("cpu")
    ws.scratch(64)
    first = ws.buf
    ws.scratch(128)
    assert ws.buf is not first and any(t is first for t in ws._outgrown)
    ws.scratch(64)
    assert len(ws._outgrown) == 1


def test_a_mask_without_words_is_refused():
    """Its address is null, which the library reads as no mask: causal, where the caller means nothing drafted."""
    with pytest.raises(ValueError, match="tree_mask"):
        _call(tree_mask=torch.zeros(3, 0, dtype=torch.int64))
    with pytest.raises(ValueError, match="tree_mask"):
        _call(tree_mask=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        _call(tree_mask=torch.zeros(3, 1, dtype=torch.int64))


def test_strides_past_32_bits_are_refused():
    """A row stride of 2^32 + 256 elements is not one of 256."""
    from precision_quantized_gemm_b200 import layer
    with pytest.raises(ValueError, match="CUDA"):
        _call()  # (the module's torch is there from the first call on)
    far = torch.empty(1, dtype=torch.bfloat16, device="meta").as_strided((2, 256), ((1 << 32) + 256, 1))
    with pytest.raises(ValueError, match="stride"):
        layer._rows("x", far, 2, 256, far.device)
    with pytest.raises(ValueError, match="stride"):
        layer._heads("k", far.view(2, 4, 64), 2, 4, 64, far.device)
    near = torch.empty(1, dtype=torch.bfloat16, device="meta").as_strided((2, 256), ((1 << 31) - 8, 1))
    assert layer._rows("x", near, 2, 256, near.device) == (1 << 31) - 8
    assert layer._rows("x", far[:1], 1, 256, far.device) == 256


def _sizes(batch, tokens, max_q, positions, q_heads=64, kv_heads=8, dim=128):
    p = 0x100000  # stands in for every address
    c = qg.qg_cache(format=0, pages=64, page_size=64, kv_heads=kv_heads, head_dim=dim, k=p, v=p, k_scale=p, v_scale=p)
    a = qg.qg_attend(q=p, out=p, q_offsets=p, kv_len=p, page_table=p, ldq=q_heads * dim, ldo=q_heads * dim,
                     q_heads=q_heads, batch=batch, tokens=tokens, max_q=max_q, max_pages=positions // 64, scale=0.125)
    return qg.qgemm_attend(c, a, p, 1 << 30, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on stand-in pointers")
def test_what_fits_is_not_refused():
    """Units of work are counted as the kernel cuts them: 16 row tiles of 128, not 256 of 8, and no more tokens than
    there are."""
    assert _sizes(1024, 1024 * 256, 256, 131072) != qg.QG_ERR_UNSUPPORTED   # 134 million units
    assert _sizes(1024, 1024, 256, 131072) != qg.QG_ERR_UNSUPPORTED
    assert _sizes(1024, 1024 * 256, 256, 1 << 25) == qg.QG_ERR_UNSUPPORTED  # 34 billion
    assert _sizes(1024, 1024, 256, 1 << 25) == qg.QG_ERR_UNSUPPORTED
