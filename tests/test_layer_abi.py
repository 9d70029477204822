"""Boundary tests of the layer operators that need no GPU: sizes, host-side
refusals before any launch (aligned stand-ins for device pointers, never
dereferenced), and the binding's checks."""
import ctypes

import pytest
import torch

import precision_quantized_gemm_b200 as qg

P = 0x100000  # an aligned, never-dereferenced stand-in for a device pointer
INVALID, UNSUPPORTED = qg.QG_ERR_INVALID_ARG, qg.QG_ERR_UNSUPPORTED


def _accepted(status):
    """Past every argument check: without a device the launch is what fails."""
    return status in (qg.QG_OK, qg.QG_ERR_NO_DEVICE, qg.QG_ERR_CUDA, UNSUPPORTED)


needs_no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on stand-in pointers")


# ---------------------------------------------------------------------- norm --
def _norm(**kw):
    n = qg.qg_norm(residual=P, x=P, pre_weight=P, h=P, y=P, ldr=256, ldx=256, ldh=256, ldy=256, pre_norm=qg.QG_NORM_RMS,
                   residual_scale=1.0, block_scale=1.0, eps=1e-6)
    for k, v in kw.items():
        setattr(n, k, v)
    return n


def _call_norm(n, M=4, N=256, fmt=0, out=None, amax=None):
    return qg.qgemm_norm(n, M, N, fmt, out, amax, None)


@pytest.mark.parametrize("change", [
    dict(residual=None, x=None), dict(residual=P + 8), dict(ldr=255), dict(ldr=248), dict(ldx=260), dict(ldh=128),
    dict(y=P + 2), dict(h=None, y=None), dict(pre_norm=3), dict(post_norm=-1), dict(pre_weight=None),
    dict(pre_norm=0), dict(post_norm=1), dict(post_weight=P), dict(post_bias=P), dict(gate=P, x=None, ldg=0),
    dict(gate=P, ldg=64), dict(gate=P + 4, ldg=0), dict(eps=-1.0), dict(eps=float("nan")), dict(pre_bias=P + 8),
    dict(post_norm=1, post_weight=P, x=None)])
def test_norm_refuses(change):
    assert _call_norm(_norm(**change)) == INVALID


@pytest.mark.parametrize("M,N", [(0, 256), (4, 0), (-1, 256), (4, 252)])
def test_norm_refuses_sizes(M, N):
    assert _call_norm(_norm(), M, N) == INVALID


def test_norm_refuses_wide_rows():
    n = _norm(ldr=65536, ldx=65536, ldh=65536, ldy=65536)
    assert _call_norm(n, 1, 32768 + 8) == UNSUPPORTED


def test_norm_refuses_operands():
    out = qg.qg_operand(P, P, P, 4, 256)
    assert _call_norm(_norm(), N=200, out=qg.qg_operand(P, P, None, 4, 200)) == INVALID        # K multiple of 16
    assert _call_norm(_norm(), fmt=9, out=out) == INVALID
    assert _call_norm(_norm(), out=qg.qg_operand(P, P, None, 3, 256)) == INVALID               # rows
    assert _call_norm(_norm(), out=qg.qg_operand(P + 1, P, None, 4, 256)) == INVALID
    assert _call_norm(_norm(pre_norm=0, pre_weight=None, y=None), out=out) == INVALID          # nothing to quantise
    assert _call_norm(_norm(), fmt=qg.QG_NVFP4, out=out) == UNSUPPORTED                        # needs static_amax


@needs_no_device
def test_norm_accepts():
    assert _accepted(_call_norm(_norm()))
    assert _accepted(_call_norm(_norm(h=None, gate=P), out=qg.qg_operand(P, P, None, 4, 256)))
    assert _accepted(_call_norm(_norm(x=None, h=None)))


# --------------------------------------------------------------------- cache --
@pytest.mark.parametrize("args,want", [
    ((0, 3, 16, 2, 64), (3 * 16 * 2 * 64, 3 * 16 * 2 * 4)), ((1, 1, 1024, 1, 128), (1024 * 128, 4096)),
    ((0, 1 << 20, 128, 8, 128), (1 << 37, 1 << 32))])
def test_cache_bytes(args, want):
    assert qg.qgemm_cache_bytes(*args) == want


@pytest.mark.parametrize("args,status", [
    ((0, 0, 16, 2, 64), INVALID), ((0, 3, 16, 0, 64), INVALID), ((7, 3, 16, 2, 64), INVALID),
    ((2, 3, 16, 2, 64), UNSUPPORTED), ((3, 3, 16, 2, 64), UNSUPPORTED), ((0, 3, 8, 2, 64), UNSUPPORTED),
    ((0, 3, 48, 2, 64), UNSUPPORTED), ((0, 3, 2048, 2, 64), UNSUPPORTED), ((0, 3, 16, 2, 96), UNSUPPORTED),
    ((0, 1 << 21, 128, 8, 128), UNSUPPORTED)])
def test_cache_bytes_refuses(args, status):
    with pytest.raises(qg.QGemmError) as e:
        qg.qgemm_cache_bytes(*args)
    assert e.value.status == status


def _cache(**kw):
    c = qg.qg_cache(format=0, pages=4, page_size=16, kv_heads=2, head_dim=64, k=P, v=P, k_scale=P, v_scale=P)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _write(**kw):
    w = qg.qg_cache_write(q=P, k=P, v=P, q_out=P, ldq=256, ldk=128, ldv=128, ldqo=256, q_heads=4, slots=P, positions=P,
                          frequency=P, rope_dim=64, interleaved=0, magnitude=1.0)
    for k, v in kw.items():
        setattr(w, k, v)
    return w


@pytest.mark.parametrize("change", [dict(k=None), dict(v=P + 8), dict(k_scale=None), dict(v_scale=P + 4), dict(pages=0)])
def test_cache_is_checked(change):
    c = _cache(**change)
    assert qg.qgemm_cache_write(c, _write(), 3, None) == INVALID
    assert qg.qgemm_cache_read(c, P, 3, P, 128, P, 128, None) == INVALID
    assert qg.qgemm_attend(c, _attend(), P, 1 << 30, None) == INVALID


def test_rows_per_key_head_past_32_bits():
    """max_q * q_heads / kv_heads is counted in 32 bits."""
    c, a = _cache(kv_heads=1), _attend(q_heads=1 << 24, max_q=256, batch=1, max_pages=1, ldq=1 << 30, ldo=1 << 30)
    assert qg.qgemm_attend_workspace_size(c, a) == 0
    assert qg.qgemm_attend(c, a, P, 1 << 30, None) == UNSUPPORTED


def test_a_token_of_too_many_channels():
    """kv_heads * head_dim past 32 bits: no stride could hold it."""
    c = _cache(pages=1, kv_heads=1 << 25, head_dim=128)
    assert qg.qgemm_cache_write(c, _write(), 3, None) == UNSUPPORTED
    assert qg.qgemm_cache_read(c, P, 3, P, 128, P, 128, None) == UNSUPPORTED
    assert qg.qgemm_attend(c, _attend(q_heads=1 << 25), P, 1 << 30, None) == UNSUPPORTED


@pytest.mark.parametrize("change", [
    dict(slots=None), dict(slots=P + 2), dict(k=None), dict(ldk=120), dict(ldv=124), dict(q=None), dict(q_out=None),
    dict(q_heads=0), dict(q_heads=-1), dict(ldq=248), dict(ldqo=128), dict(rope_dim=72), dict(rope_dim=8),
    dict(rope_dim=80), dict(rope_dim=-16), dict(positions=None), dict(frequency=None), dict(frequency=P + 4)])
def test_cache_write_refuses(change):
    assert qg.qgemm_cache_write(_cache(), _write(**change), 3, None) == INVALID
    assert qg.qgemm_cache_write(_cache(), _write(), 0, None) == INVALID


@pytest.mark.parametrize("args", [(None, 3, P, 128, P, 128), (P, 0, P, 128, P, 128), (P, 3, None, 128, P, 128),
                                  (P, 3, P, 64, P, 128), (P, 3, P, 128, P, 132), (P + 1, 3, P, 128, P, 128)])
def test_cache_read_refuses(args):
    assert qg.qgemm_cache_read(_cache(), *args, None) == INVALID


# ------------------------------------------------------------------ attention --
def _attend(**kw):
    a = qg.qg_attend(q=P, out=P, q_offsets=P, kv_len=P, page_table=P, ldq=256, ldo=256, q_heads=4, batch=2, tokens=8,
                     max_q=4, max_pages=4, scale=0.125)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), INVALID), (dict(tokens=0), INVALID), (dict(max_q=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(q_heads=3), INVALID), (dict(q=None), INVALID), (dict(ldq=128), INVALID), (dict(ldo=260), INVALID),
    (dict(out=P + 2), INVALID), (dict(q_offsets=None), INVALID), (dict(kv_len=P + 1), INVALID),
    (dict(page_table=None), INVALID), (dict(tree_mask=P), INVALID), (dict(tree_mask=P + 4, mask_words=1), INVALID),
    (dict(lse=P + 2), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(batch=1025), UNSUPPORTED), (dict(max_q=257), UNSUPPORTED), (dict(max_pages=1 << 27), UNSUPPORTED)])
def test_attend_refuses(change, status):
    assert qg.qgemm_attend(_cache(), _attend(**change), P, 1 << 30, None) == status


@needs_no_device
def test_workspace_is_checked():
    c, a = _cache(), _attend()
    need = qg.qgemm_attend_workspace_size(c, a)
    assert need > 0
    assert _accepted(qg.qgemm_attend(c, a, P, need, None))


def test_workspace_size_of_nothing():
    assert qg.qgemm_attend_workspace_size(_cache(), _attend(q_heads=0)) == 0


# -------------------------------------------------------------------- binding --
def test_binding_wants_cuda_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qg.norm(x, x[0])
    with pytest.raises(ValueError):
        qg.norm(None, x[0])
    with pytest.raises(ValueError):
        qg.norm(x, None, fmt=qg.QG_FP8_DYNAMIC)
    with pytest.raises(ValueError):
        qg.norm(x, x[0], kind="batch")


def test_binding_checks_the_cache():
    c = qg.Cache(qg.QG_FP8_DYNAMIC, 2, 16, 1, 64, device="cpu")
    assert (c.pages, c.page_size, c.kv_heads, c.head_dim) == (2, 16, 1, 64)
    with pytest.raises(ValueError):
        qg.Cache(qg.QG_FP8_DYNAMIC, 2, 16, 1)
    with pytest.raises(ValueError):
        qg.Cache(qg.QG_FP8_DYNAMIC, k=c.k, v=c.v, k_scale=c.k_scale, v_scale=c.v_scale.double())
    with pytest.raises(qg.QGemmError):
        qg.Cache(qg.QG_BLOCK_FP8, 2, 16, 1, 64, device="cpu")
    with pytest.raises(ValueError):
        qg.Rope(torch.ones(4))


def test_structures_match_the_header():
    """The binding's structures have the C layout's sizes (pointers 8, ints and floats 4 bytes)."""
    assert ctypes.sizeof(qg.qg_norm) == 9 * 8 + 7 * 4 + 4 * 4 + 4
    assert ctypes.sizeof(qg.qg_cache) == 5 * 4 + 4 + 4 * 8
    assert ctypes.sizeof(qg.qg_cache_write) == 4 * 8 + 5 * 4 + 4 + 3 * 8 + 3 * 4 + 4
    assert ctypes.sizeof(qg.qg_attend) == 7 * 8 + 9 * 4 + 4


@pytest.mark.parametrize("scaling", [None, "linear", "base", "bands", "ramp"])
def test_rope_frequencies(scaling):
    plain, one = qg.rope_frequencies(64, 10000.0, device="cpu")
    assert one == 1.0 and plain.dtype == torch.float64 and plain[0] == 1.0
    assert torch.allclose(plain[1:] / plain[:-1], torch.full((31,), 10000.0 ** (-2 / 64), dtype=torch.float64))
    f, mag = qg.rope_frequencies(64, 10000.0, scaling=scaling, factor=4.0, original=4096, device="cpu")
    assert (f <= plain * (1 + 1e-12)).all() and (f >= plain / 4 * (1 - 1e-12)).all()
    assert f[-1] == pytest.approx(plain[-1] / (1.0 if scaling is None else 4.0))
    if scaling != "linear":
        assert f[0] == pytest.approx(1.0)
    assert mag == (pytest.approx(1.1386294361119891) if scaling == "ramp" else 1.0)
    with pytest.raises(ValueError):
        qg.rope_frequencies(63, device="cpu")
    with pytest.raises(ValueError):
        qg.rope_frequencies(64, scaling="other", device="cpu")
