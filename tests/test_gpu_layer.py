"""GPU parity of the operators between the quantised products against the
float64 oracle: norms, rotary cache write, cache read, attention over the
cache, and a decoder step that runs them with the quantised products.

Tolerances count roundings: half a step of bf16 is 2^-8 of the value, of f16
2^-11, of fp32 2^-24, of e4m3 2^-4 (2^-10 of the scale below its normal
range), of int8 half the scale."""
import itertools

import numpy as np
import pytest
import torch

import precision_quantized_gemm_b200 as qg
from oracle import layer as OL

pytestmark = pytest.mark.gpu

BF16, F16, F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24
# fp32 error of a row's norm in units of its terms: a sum over at most 64
# elements in a chain and 15 levels of a tree (80 roundings), then under 20 more
ROW = 100 * F32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    qg.lib()
    yield
    assert qg.qgemm_device_error() == qg.QG_OK


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(g, *shape, scale=1.0, offset=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale + offset).to(torch.bfloat16)


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _close(got, want, tol, what):
    got = _np(got) if torch.is_tensor(got) else got
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of tolerance, first at {i}: got {got[i]}, "
                             f"want {want[i]} within {np.broadcast_to(tol, bad.shape)[i]}")


# ---------------------------------------------------------------------- norm --
def _norm_inputs(M, N, seed, kind="rms", post=False, gate="none", bias=None):
    g = _gen(seed)
    bias = kind == "layer" if bias is None else bias
    kw = dict(kind=kind, eps=1e-5, block_scale=0.7, residual_scale=1.3)
    r, x, w = _rand(g, M, N, scale=2.0), _rand(g, M, N), _rand(g, N, scale=0.2, offset=1.0)
    kw["bias"] = _rand(g, N, scale=0.3) if bias else None
    if post:
        kw["post_weight"] = _rand(g, N, scale=0.2, offset=1.0)
        kw["post_bias"] = _rand(g, N, scale=0.3) if bias else None
    if gate != "none":
        kw["gate"] = _rand(g, *((N,) if gate == "row" else (M, N)))
    return r, x, w, kw


def _norm_oracle(r, x, w, kw):
    kw = {k: (_np(v) if torch.is_tensor(v) else v) for k, v in kw.items()}
    h, y = OL.block_norm(_np(r), _np(x), weight=_np(w), **kw)
    # the largest magnitude among a row's terms bounds each term's own error
    terms = np.abs(h)
    for t in (r, x):
        if t is not None:
            terms = np.maximum(terms, 1.3 * np.abs(_np(t)))
    if kw.get("post_weight") is not None:
        b = OL.norm_rows(_np(x), kw["post_weight"], kw.get("post_bias"), kw["kind"], kw["eps"])
        terms = np.maximum(terms, 0.7 * np.abs(b if kw.get("gate") is None else b * kw["gate"]) + 1.0)
    elif kw.get("gate") is not None:
        terms = np.maximum(terms, 0.7 * np.abs(_np(x) * kw["gate"]))
    dh = ROW * terms.max(axis=1, keepdims=True)
    if w is None:
        return h, None, dh, None
    # y is h, less its mean, over its root mean square, times the weight:
    # h's error and the norm's own, on the scale of the row
    c = h - h.mean(axis=1, keepdims=True) if kw["kind"] == "layer" else h
    rms = np.sqrt((c * c).mean(axis=1, keepdims=True) + kw["eps"])
    gain = np.abs(_np(w)) + kw.get("weight_offset", 0.0)
    dy = (2 * dh + ROW * np.abs(h).max(axis=1, keepdims=True)) / rms * gain + ROW * np.abs(y)
    return h, y, dh, dy


def _operand_values(op, fmt, M, N):
    """(values, scale of each element, scales) of an 8-bit activation operand."""
    s = op.scale.view(torch.float32).double().cpu().numpy()
    q = op.q.view(torch.int8 if fmt == qg.QG_W8A8_INT8 else torch.float8_e4m3fn).view(M, N).double().cpu().numpy()
    s = s.reshape(M, -1)
    wide = np.repeat(s, N // s.shape[1], axis=1)
    return q * wide, wide, s


def _check_codes(op, fmt, y, dy):
    M, N = y.shape
    got, wide, s = _operand_values(op, fmt, M, N)
    group = N // s.shape[1]
    top = 127.0 if fmt == qg.QG_W8A8_INT8 else 448.0
    want_s = OL.row_scales(y.reshape(M, -1, group), top)
    d_s = dy.reshape(M, -1, group).max(axis=2) / top + 2 * F32 * want_s
    _close(s, want_s, d_s, "scale")
    half = 0.5 * wide if fmt == qg.QG_W8A8_INT8 else np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * wide)
    # the largest code stands for top * scale, which may be d_s * top short of y
    _close(got, y, half * (1 + 2.0 ** -10) + 2 * dy + np.repeat(d_s, group, axis=1) * top, "codes")


NORMS = [(1, 8, "rms", False, "none"), (3, 64, "layer", True, "full"), (5, 256, "rms", True, "row"),
         (2, 5120, "rms", False, "none"), (300, 1032, "layer", False, "row"), (297, 2064, "rms", True, "full"),
         (2, 8192, "layer", True, "none"), (1, 8200, "rms", True, "row"), (2, 32768, "rms", True, "full"),
         (1, 32760, "layer", False, "none"), (300, 16384, "rms", False, "row")]


@pytest.mark.parametrize("M,N,kind,post,gate", NORMS)
def test_norm_bf16(M, N, kind, post, gate):
    r, x, w, kw = _norm_inputs(M, N, M * 7 + N, kind, post, gate)
    out = qg.norm(r, w, x, **kw)
    h, y, dh, dy = _norm_oracle(r, x, w, kw)
    assert out.operand is None
    _close(out.h, h, BF16 * np.abs(h) + dh, "h")
    _close(out.y, y, BF16 * np.abs(y) + dy, "y")


@pytest.mark.parametrize("fmt", [qg.QG_FP8_DYNAMIC, qg.QG_W8A8_INT8, qg.QG_BLOCK_FP8])
@pytest.mark.parametrize("M,N,kind,post,gate", [(1, 128, "rms", False, "none"), (7, 5120, "layer", True, "row"),
                                                (299, 1152, "rms", True, "full"), (3, 24576, "rms", False, "none")])
def test_norm_operand(fmt, M, N, kind, post, gate):
    r, x, w, kw = _norm_inputs(M, N, M + N, kind, post, gate)
    y_buf = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    out = qg.norm(r, w, x, fmt=fmt, y=y_buf, **kw)
    h, y, dh, dy = _norm_oracle(r, x, w, kw)
    _close(out.h, h, BF16 * np.abs(h) + dh, "h")
    _close(y_buf, y, BF16 * np.abs(y) + dy, "y")
    _check_codes(out.operand, fmt, y, dy)


@pytest.mark.parametrize("M,N", [(1, 32), (5, 288), (130, 512)])
def test_norm_nvfp4(M, N):
    """Codes and block scales against the recipe in float64: g = amax / 2688,
    scale e4m3(amax_b / 6 / g), code e2m1(y / (scale g)).  Away from a border
    they are the oracle's; the padding of the scales is zero."""
    from oracle import formats as OF
    from gpu_util import sf_padding_is_zero, unpack_nvfp4_codes, unpack_sf_128x4
    r, x, w, kw = _norm_inputs(M, N, M + N, "rms", True, "row")
    h, y, dh, dy = _norm_oracle(r, x, w, kw)
    amax = torch.tensor([float(np.abs(y).max())], device="cuda")
    op = qg.Operand(qg.QG_NVFP4, False, M, N, "cuda")
    op.scale.fill_(0x55)  # the padding has to be written
    qg.norm(r, w, x, out=op, static_amax=amax, **kw)
    torch.cuda.synchronize()
    sf = op.scale.cpu().numpy()
    assert sf_padding_is_zero(sf, M, N)
    g = np.float32(op.global_scale.cpu().numpy()[0])
    assert g == np.float32(amax.item()) / np.float32(2688)
    codes = unpack_nvfp4_codes(op.q.cpu().numpy(), M, N)
    scales = OF.E4M3_VALUES[unpack_sf_128x4(sf, M, N)].astype(np.float64) if hasattr(OF, "E4M3_VALUES") else \
        torch.from_numpy(unpack_sf_128x4(sf, M, N).copy()).view(torch.float8_e4m3fn).double().numpy()
    want = np.abs(y).reshape(M, -1, 16).max(axis=2) / 6 / g
    # half a step of e4m3, and the error of y
    _close(scales, want, np.maximum(2.0 ** -4 * want, 2.0 ** -10) * (1 + 1e-6) + dy.reshape(M, -1, 16).max(axis=2) / 6 / g,
           "block scales")
    values = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
    d = np.repeat(scales, 16, axis=1) * g
    got = values[codes] * d
    # half a step is 1/4 up to 2, 1/2 up to 4, 1 up to 6, of the block's unit d; the largest saturates
    t = np.abs(y) / np.where(d > 0, d, 1)
    half = np.where(t < 2, 0.25, np.where(t < 4, 0.5, np.maximum(1.0, t - 6)))
    _close(got, y, np.where(d > 0, half * d * (1 + 1e-5), np.abs(y) * (1 + 1e-5)) + dy, "codes")


def test_norm_parts():
    """Without x, without a residual, without the norm, in place, weight offset, strided rows."""
    M, N = 9, 512
    r, x, w, _ = _norm_inputs(M, N, 3)
    for args, kw in (((r, w), {}), ((None, w, x), {}), ((r, None, x), dict(block_scale=0.5)),
                     ((r, w, x), dict(weight_offset=1.0, residual_scale=0.9))):
        kw = dict(kind="rms", eps=1e-5, **kw)
        out = qg.norm(*args, **kw)
        a = args + (None,) * (3 - len(args))
        h, y, dh, dy = _norm_oracle(a[0], a[2], a[1], kw)
        assert (out.h is None) == (a[2] is None)
        if out.h is not None:
            _close(out.h, h, BF16 * np.abs(h) + dh, "h")
        assert (out.y is None) == (a[1] is None)
        if out.y is not None:
            _close(out.y, y, BF16 * np.abs(y) + dy, "y")
    ref = qg.norm(r, w, x)
    wide = torch.full((M, 2 * N), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :N] = r
    out = qg.norm(wide[:, :N], w, x, h=wide[:, :N], y=wide[:, N:])
    assert torch.equal(wide[:, :N], ref.h) and torch.equal(wide[:, N:], ref.y) and out.h.data_ptr() == wide.data_ptr()
    guard = torch.full((M, N + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    qg.norm(r, w, x, y=guard[:, :N])
    assert torch.equal(guard[:, :N], ref.y) and (guard[:, N:] == 7).all()


def test_norm_edge_rows():
    """A zero row, and rows with a NaN or an infinity: scale NaN, codes 0."""
    N = 256
    r = _rand(_gen(1), 4, N)
    r[1], r[2, 5], r[3, 7] = 0, float("nan"), float("inf")
    w = torch.ones(N, dtype=torch.bfloat16, device="cuda")
    for fmt in (qg.QG_FP8_DYNAMIC, qg.QG_W8A8_INT8, qg.QG_BLOCK_FP8):
        op = qg.norm(r, w, fmt=fmt).operand
        s = op.scale.view(torch.float32).view(4, -1)
        q = op.q.view(4, N)
        assert (s[1] == 1).all() and not q[1].any()
        assert s[2].isnan().all() and not q[2].any()
        # the infinite row's root mean square is infinite: y is NaN at the
        # infinity and +-0 elsewhere, so another group of the row is a zero group
        assert s[3, 0].isnan() and (s[3, 1:] == 1).all() and not (q[3] & 0x7f).any()
        assert s[0].isfinite().all() and q[0].any()


# --------------------------------------------------------------------- cache --
FMTS = [qg.QG_FP8_DYNAMIC, qg.QG_W8A8_INT8]


def _top(fmt):
    return 127.0 if fmt == qg.QG_W8A8_INT8 else 448.0


def _cache_values(cache, slots):
    """(codes, scales) of slots as float64 [T, H, D], [T, H]: key, then value."""
    s = slots.long()
    page, place = s // cache.page_size, s % cache.page_size
    t = torch.int8 if cache.fmt == qg.QG_W8A8_INT8 else torch.float8_e4m3fn
    return [(c[page, :, place].view(t).double().cpu().numpy(), sc[page, :, place].double().cpu().numpy())
            for c, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]


def _check_rows(codes, scale, want, slack, fmt, what):
    ws = OL.row_scales(want, _top(fmt))
    ds = slack.max(axis=-1) / _top(fmt) + 2 * F32 * ws
    _close(scale, ws, ds, what + " scale")
    wide = scale[..., None]
    half = 0.5 * wide if fmt == qg.QG_W8A8_INT8 else np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * wide)
    _close(codes * wide, want, half * (1 + 2.0 ** -10) + 2 * slack + ds[..., None] * _top(fmt), what)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,Hq,Hkv,D,rope,pairs,page", [
    (1, 1, 1, 64, 64, False, 16), (1, 40, 8, 128, 128, False, 64), (5, 6, 2, 128, 16, True, 32),
    (33, 7, 1, 64, 32, False, 16), (300, 4, 4, 64, 48, True, 128), (299, 15, 5, 128, 96, False, 1024),
    (17, 3, 3, 128, 0, False, 16)])
def test_cache_write(fmt, T, Hq, Hkv, D, rope, pairs, page):
    g = _gen(T + D + rope)
    qkv = _rand(g, T, Hq + 2 * Hkv, D)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    pages = -(-T // page) + 2
    cache = qg.Cache(fmt, pages, page, Hkv, D)
    for t in (cache.k, cache.v):
        t.fill_(0x5a)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].int()
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda").int()
    r = None
    if rope:
        freq, _ = qg.rope_frequencies(rope, 500000.0)
        r = qg.Rope(freq, interleaved=pairs, magnitude=1.2)
    out = qg.cache_write(cache, k, v, slots, q=q, rope=r, positions=pos)
    freq = _np(r.frequency) if r else []
    mag = 1.2 if r else 1.0
    want_q, want_k = (OL.rotate(_np(t), _np(pos), freq, pairs, mag) for t in (q, k))
    # the turn's cosine and sine: half a turn of angle error 2^-24, one and a
    # half ulp of the function, and the products' and sum's roundings, all
    # relative to the pair's larger channel
    sq, sk = (16 * F32 * mag * np.abs(_np(t)).max(axis=-1, keepdims=True) * np.ones(D) for t in (q, k))
    _close(out, want_q, BF16 * np.abs(want_q) + sq, "q")
    (kc, ks), (vc, vs) = _cache_values(cache, slots)
    _check_rows(kc, ks, want_k, sk, fmt, "k")
    _check_rows(vc, vs, _np(v), np.zeros((T, Hkv, D)), fmt, "v")
    # every other place as it was
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    rest = rest.view(pages, 1, page).expand(-1, Hkv, -1)
    assert (cache.k[rest] == 0x5a).all() and (cache.v[rest] == 0x5a).all()
    assert not cache.k_scale[rest].any() and not cache.v_scale[rest].any()
    # in place, with a padded token: its query turns, nothing is stored
    before = cache.k.clone(), cache.v.clone(), cache.k_scale.clone()
    slots[0] = -1
    got = qg.cache_write(cache, k, v, slots, q=q, rope=r, positions=pos, q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(q, out)
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_scale)))
    slots[0] = pages * page
    qg.cache_write(cache, k, v, slots, rope=r, positions=pos)
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_scale)))


def test_cache_write_of_very_many_heads():
    """More passes of rows than a grid has places for: the first, the last and those in between."""
    Hq, D = 8 * 65535 + 1000, 128
    g = _gen(0)
    q, k = _rand(g, 1, Hq, D), _rand(g, 1, 1, D)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    rope = qg.Rope(qg.rope_frequencies(D)[0])
    cache = qg.Cache(qg.QG_FP8_DYNAMIC, 1, 16, 1, D)
    out = qg.cache_write(cache, k, k, one, q=q, rope=rope, positions=one + 7)
    first = cache.k.clone(), cache.v.clone()
    cut = Hq // 2
    for part, want in ((q[:, :cut], out[:, :cut]), (q[:, cut:], out[:, cut:])):
        got = qg.cache_write(cache, k, k, one, q=part, rope=rope, positions=one + 7)
        assert torch.equal(got, want)
    assert torch.equal(first[0], cache.k) and torch.equal(first[1], cache.v)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_unrotated_rows_bit_for_bit(fmt, D):
    """Values, and keys without a rotation: the scale is the fp32 product amax * (1 / top), the codes are those of
    the correctly rounded quotient (formed in 64 bits: 53 >= 2 * 24 + 2 bits round once more like the division).
    Rows of bf16 values with exact ties, ordinary rows, rows over the whole range of fp32 scales."""
    g = _gen(D)
    x = _rand(g, 4096, D)
    x[:1024] = (torch.randint(-254, 255, (1024, D), generator=g, device="cuda") / 2).to(torch.bfloat16)  # k / 2
    x[:1024, 0] = 127.0
    x[512:1024, 0] = 224.0
    x[1024:2048] = (x[1024:2048].float() * 2.0 ** torch.randint(-130, 120, (1024, 1), generator=g, device="cuda")).to(
        torch.bfloat16)
    one = torch.ones((), device="cuda")
    amax = x.float().abs().amax(-1)
    want_scale = torch.where(amax > 0, amax * (one / _top(fmt)), one)
    quotient = (x.double() / want_scale.double()[:, None]).float()
    want = quotient.round().to(torch.int8) if fmt == qg.QG_W8A8_INT8 else quotient.to(torch.float8_e4m3fn)
    cache = qg.Cache(fmt, 4096 // 64, 64, 1, D)
    qg.cache_write(cache, x.view(-1, 1, D), x.view(-1, 1, D), torch.arange(4096, dtype=torch.int32, device="cuda"))
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        assert torch.equal(scale.view(-1), want_scale)
        same = codes.view(-1, D) == want.view(torch.uint8)
        assert same.all(), (int((~same).sum()), (~same).nonzero()[:4].tolist())


@pytest.mark.parametrize("fmt", [qg.QG_FP8_DYNAMIC, qg.QG_W8A8_INT8])
def test_norm_codes_are_the_quantisers(fmt):
    """y in bf16 values (weights and rows chosen so that y is exact in bf16): the operand is quantize_act's, bit for bit."""
    g = _gen(3)
    N = 512
    x = (torch.randint(0, 2, (300, N), generator=g, device="cuda") * 2 - 1).to(torch.bfloat16)  # mean square 1
    w = (torch.randint(-254, 255, (N,), generator=g, device="cuda") / 2).to(torch.bfloat16)
    w[0] = 127.0
    r = qg.norm(x, w, fmt=fmt, eps=0.0)
    op = qg.quantize_act(fmt, x * w)
    assert torch.equal(r.operand.q.view(-1), op.q.view(-1)) and torch.equal(
        r.operand.scale.view(torch.float32), op.scale.view(torch.float32))


@pytest.mark.parametrize("fmt", FMTS)
def test_cache_write_edge_rows(fmt):
    """Zero rows (scale 1), rows with a NaN or an infinity (scale NaN, codes 0, NaN when read)."""
    cache = qg.Cache(fmt, 2, 16, 1, 64)
    k = _rand(_gen(0), 4, 1, 64)
    k[1], k[2, 0, 3], k[3, 0, 63] = 0, float("inf"), float("nan")
    slots = torch.tensor([3, 17, 0, 31], dtype=torch.int32, device="cuda")
    qg.cache_write(cache, k, k.flip(0).contiguous(), slots)
    (kc, ks), (vc, vs) = _cache_values(cache, slots)
    assert np.isfinite(ks[:2]).all() and ks[1, 0] == 1 and np.isnan(ks[2:]).all() and not kc[1:].any()
    assert np.isnan(vs[:2]).all() and vs[2, 0] == 1 and not vc[:3].any()
    rk, rv = qg.cache_read(cache, slots)
    assert rk[2:].isnan().all() and rv[:2].isnan().all() and not rk[1].any() and rk[0].isfinite().all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 64, 16), (77, 3, 128, 32), (1000, 8, 64, 64)])
def test_cache_read(fmt, T, H, D, page):
    """bf16(code * scale) exactly, for every code, for repeated and unknown slots, into strided rows."""
    g = _gen(T)
    pages = 9
    cache = qg.Cache(fmt, pages, page, H, D)
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c.copy_(torch.randint(0, 256, c.shape, generator=g, device="cuda"))
        s.copy_(torch.rand(s.shape, generator=g, device="cuda") * 0.1)
    slots = torch.randint(-2, pages * page + 2, (T,), generator=g, device="cuda").int()
    wide = torch.zeros(T, 2, H, D, dtype=torch.bfloat16, device="cuda")
    k, v = qg.cache_read(cache, slots, k=wide[:, 0], v=wide[:, 1])
    inside = (slots >= 0) & (slots < pages * page)
    for got, c, s in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        at = slots.clamp(0, pages * page - 1).long()
        code = c[at // page, :, at % page].view(torch.int8 if fmt == qg.QG_W8A8_INT8 else torch.float8_e4m3fn).float()
        want = (code * s[at // page, :, at % page][..., None]).to(torch.bfloat16)
        want[~inside] = 0
        assert torch.equal(got.view(torch.int16)[~want.isnan()], want.view(torch.int16)[~want.isnan()])
        assert torch.equal(got.isnan(), want.isnan())
    k2, v2 = qg.cache_read(cache, slots)
    assert torch.equal(k2.view(torch.int16), k.contiguous().view(torch.int16))


# ------------------------------------------------------------------ attention --
class Batch:
    """Sequences with cached positions and drafted tokens, on the device and as float64."""

    def __init__(self, fmt, lens, ns, Hq, Hkv, D, page, seed, tree=True, words=None, junk=True, spread=1.0):
        g = _gen(seed)
        self.lens, self.ns, self.fmt, self.D, self.Hq, self.Hkv = lens, ns, fmt, D, Hq, Hkv
        B, T = len(lens), sum(ns)
        each = [-(-a // page) for a in lens]
        pages = sum(each) + 2
        self.cache = qg.Cache(fmt, pages, page, Hkv, D)
        c = self.cache
        if junk:  # places that no position uses hold anything: e4m3 NaN codes, NaN and infinite scales
            c.k.fill_(0x7f), c.v.fill_(0xff)
            c.k_scale.fill_(float("nan")), c.v_scale.fill_(float("inf"))
        self.table = torch.full((B, max(each + [1]) + 1), 1 << 30 if junk else 0, dtype=torch.int32, device="cuda")
        order, at, slots = torch.randperm(pages, generator=g, device="cuda").int(), 0, []
        for b, e in enumerate(each):
            self.table[b, :e] = order[at:at + e]
            p = torch.arange(lens[b], device="cuda")
            slots.append(order[at:at + e].long()[p // page] * page + p % page)
            at += e
        slots = torch.cat(slots)
        n = slots.numel()
        if n:
            k = _rand(g, n, Hkv, D) * (torch.rand(n, 1, 1, generator=g, device="cuda") * spread + 0.1).to(torch.bfloat16)
            v = _rand(g, n, Hkv, D) * (4.0 ** torch.randn(n, Hkv, 1, generator=g, device="cuda")).to(torch.bfloat16)
            qg.cache_write(c, k, v, slots.int())
        self.slots = slots
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.offs = torch.tensor(list(itertools.accumulate(ns, initial=0)), dtype=torch.int32, device="cuda")
        self.T = T
        self.q = _rand(g, T + 3, Hq, D, scale=1.5)  # three rows behind the last sequence
        self.see = self.mask = None
        if tree:
            most = max(ns + [1])
            words = words or -(-most // 64)
            self.see = torch.rand(T + 3, words * 64, generator=g, device="cuda") < 0.5
            self.see[:: 5] = False  # rows that see no drafted token at all
            weight = torch.ones((), dtype=torch.int64, device="cuda") << torch.arange(64, device="cuda")
            self.mask = (self.see.view(T + 3, words, 64).long() * weight).sum(-1)
            self.see = self.see.cpu().numpy()

    def values(self):
        (kc, ks), (vc, vs) = _cache_values(self.cache, self.slots)
        return kc * ks[..., None], vc * vs[..., None]

    def run(self, **kw):
        out = torch.full((self.T + 3, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.T + 3, self.Hq), 7.0, device="cuda")
        kw.setdefault("max_q", max(self.ns + [1]))
        qg.attend(self.cache, self.q, self.offs, self.lens_t, self.table, tree_mask=self.mask, out=out, lse=lse, **kw)
        return out, lse

    def check(self, out, lse, scale=None, rows=None):
        """Every row, or a sample of `rows` rows, against the oracle."""
        scale = self.D ** -0.5 if scale is None else scale
        k, v = self.values()
        q = _np(self.q)
        out, lse = _np(out), _np(lse)
        G = self.Hq // self.Hkv
        pick = np.random.default_rng(0)
        at = row = 0
        for length, n in zip(self.lens, self.ns):
            ids = range(n) if rows is None or n <= rows else sorted(pick.choice(n, rows, replace=False))
            for i in ids:
                see = OL.visible(n, length, i, None if self.see is None else self.see[row + i])
                for h in range(self.Hq) if rows is None else pick.choice(self.Hq, min(self.Hq, 4), replace=False):
                    kk, vv = k[at:at + length, h // G], v[at:at + length, h // G]
                    qq = q[row + i, h]
                    o, l, mag = OL.attend_one(qq, kk, vv, scale, see)
                    if l == -np.inf:
                        assert not out[row + i, h].any() and lse[row + i, h] == -np.inf
                        continue
                    if np.isnan(l) or np.isnan(o).any():  # a NaN row, key or value: out and lse
                        assert np.isnan(out[row + i, h]).all() and np.isnan(lse[row + i, h])
                        continue
                    # a score: D products summed in fp32 (the unit may
                    # truncate: a whole step each), and three more roundings
                    ds = abs(scale) * (self.D + 8) * 2 * F32 * (np.abs(kk[see]) @ np.abs(qq)).max() + 2 * F32 * abs(l)
                    # a weight: f16, the exponential's 2^-22 and the sums' chain
                    rel = F16 + 2.0 ** -22 + 4 * F32 + see.sum() * 2 * F32 + 2 * ds
                    # weights below 2^-24 of the largest weight x value scale are lost: 2^-24 each of the largest term
                    lost = see.sum() * 2.0 ** -25 * np.abs(vv[see]).max() * np.exp((scale * (kk[see] @ qq) - l).max())
                    _close(out[row + i, h], o, BF16 * np.abs(o) + rel * mag + lost, f"out {row + i} {h}")
                    _close(lse[row + i, h:h + 1], np.array([l]), ds + see.sum() * 2 * F32 + 2.0 ** -21 + 4 * F32 * abs(l),
                           "lse")
            at += length
            row += n
        assert (out[self.T:] == 7).all() and (lse[self.T:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,ns,Hq,Hkv,D,page", [
    ([1], [1], 1, 1, 64, 16), ([1], [1], 8, 8, 128, 64), ([63], [1], 5, 1, 128, 16), ([64], [1], 16, 1, 64, 16),
    ([65, 31, 33], [1, 1, 1], 12, 4, 128, 32), ([1000, 1, 257, 512], [1, 1, 1, 1], 8, 2, 128, 64),
    ([5000], [1], 7, 7, 64, 1024), ([300] * 40, [1] * 40, 8, 8, 128, 128)])
def test_single_tokens(fmt, lens, ns, Hq, Hkv, D, page):
    b = Batch(fmt, lens, ns, Hq, Hkv, D, page, seed=len(lens) + Hq, tree=False)
    b.check(*b.run(), rows=None if sum(lens) < 3000 else 2)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("lens,ns,Hq,Hkv,D,page", [
    ([3], [3], 1, 1, 64, 16), ([2, 40], [2, 9], 4, 2, 128, 16), ([130, 127, 400], [5, 1, 16], 10, 2, 64, 32),
    ([70], [70], 2, 1, 128, 64), ([700, 129], [64, 65], 8, 8, 64, 64), ([256, 300], [33, 128], 16, 2, 128, 128),
    ([600], [256], 3, 1, 128, 16), ([1500, 1300], [17, 30], 5, 1, 128, 64)])
def test_trees(fmt, tree, lens, ns, Hq, Hkv, D, page):
    b = Batch(fmt, lens, ns, Hq, Hkv, D, page, seed=sum(ns) + Hq, tree=tree)
    b.check(*b.run(), rows=6)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,ns,Hq,Hkv,D,page", [  # rows of a key head: 20, 24, 24, 28, 32, 32
    ([500, 40, 1000], [1, 1, 1], 20, 1, 128, 64), ([900, 77], [3, 2], 16, 2, 128, 16), ([130, 700], [2, 3], 8, 1, 64, 32),
    ([700, 90], [7, 5], 8, 2, 64, 128), ([1200, 100], [4, 8], 8, 2, 64, 16), ([1200, 100], [4, 8], 8, 2, 128, 16)])
def test_row_counts_between(fmt, lens, ns, Hq, Hkv, D, page):
    """The most rows that the warp-level kernel takes, and the first that go to the tiles."""
    b = Batch(fmt, lens, ns, Hq, Hkv, D, page, seed=sum(lens) + D, tree=ns[0] > 1)
    b.check(*b.run(), rows=6)


@pytest.mark.parametrize("B,Hq,most", [(1024, 4, 1), (700, 3, 3), (300, 64, 5)])
def test_many_sequences(B, Hq, most):
    """More sequences than threads plan, a third of them without tokens, some without positions."""
    r = np.random.default_rng(B)
    ns = [int(n) if i % 3 else 0 for i, n in enumerate(r.integers(1, most + 1, B))]
    lens = [0 if i % 7 == 1 else int(a) for i, a in enumerate(r.integers(most, 150, B))]
    b = Batch(qg.QG_FP8_DYNAMIC, lens, ns, Hq, 1, 64, 16, seed=B, tree=most > 1)
    b.check(*b.run(), rows=1)


@pytest.mark.parametrize("scale", [0.0, -0.3])
@pytest.mark.parametrize("Hq,n", [(8, 2), (64, 9)])
def test_any_scale(Hq, n, scale):
    b = Batch(qg.QG_W8A8_INT8, [300, 90], [n, 1], Hq, 2, 128, 32, seed=5)
    b.check(*b.run(scale=scale), scale=scale, rows=3)


def test_offsets_that_start_late():
    """Rows before the first sequence belong to none, and offsets past the tokens are cut."""
    b = Batch(qg.QG_FP8_DYNAMIC, [200, 77], [2, 3], 8, 2, 128, 16, seed=5, tree=False)
    want, want_lse = b.run()
    q = b.q.clone()
    b.q[4:] = q[:4]
    b.offs += 4  # 4, 6, 9 of 8 rows
    out, lse = torch.full_like(b.q, 7.0), torch.full((8, 8), 7.0, device="cuda")
    qg.attend(b.cache, b.q, b.offs, b.lens_t, b.table, out=out, lse=lse, max_q=3)
    assert (out[:4] == 7).all() and (lse[:4] == 7).all()
    assert torch.equal(out[4:6], want[:2]) and torch.equal(lse[4:6], want_lse[:2])
    assert (out[6:] != 7).any() and out[6:].isfinite().all()


@pytest.mark.parametrize("Hq,n", [(20, 1), (64, 9)])
def test_one_workspace_in_two_graphs(Hq, n):
    """Two captured calls of different sizes share a workspace and are replayed in turn on one stream."""
    b = Batch(qg.QG_FP8_DYNAMIC, [900, 1200], [n, n], Hq, 4, 128, 16, seed=2)
    c = Batch(qg.QG_W8A8_INT8, [3000], [1], 8, 2, 64, 64, seed=3, tree=False)
    want = [x.run() for x in (b, c)]
    ws, graphs, got = qg.Workspace("cuda"), [], []
    for x in (b, c):
        x.run(workspace=ws)  # the workspace is as large as the larger needs
    torch.cuda.synchronize()
    for x in (b, c):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(x.run(workspace=ws))
        graphs.append(graph)
    for turn in (0, 1, 1, 0, 1):
        for t in got[turn]:
            t.fill_(7)
        graphs[turn].replay()
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (40, 2)])
def test_empty_sequences(fmt, Hq, Hkv):
    """Padded sequences: no tokens, no positions, tokens without positions, more tokens than positions."""
    b = Batch(fmt, [50, 0, 0, 33, 2, 100], [2, 0, 3, 0, 4, 7], Hq, Hkv, 128, 16, seed=3)
    b.check(*b.run())
    b = Batch(fmt, [0, 0], [1, 2], Hq, Hkv, 64, 16, seed=4, tree=False)
    b.check(*b.run())


@pytest.mark.parametrize("Hq,n", [(4, 3), (24, 30)])
def test_rows_whose_mask_leaves_nothing(Hq, n):
    """Without a prefix, a mask row of zeros sees nothing: zeros, and a log-sum of -inf."""
    b = Batch(qg.QG_FP8_DYNAMIC, [n, 200 + n], [n, n], Hq, 4, 128, 16, seed=9)
    out, lse = b.run()
    b.check(out, lse)
    empty = [i for i in range(n) if not b.see[i, :n].any()]
    assert empty and (lse[empty] == -float("inf")).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hq,n", [(2, 4), (32, 40)])
def test_hidden_rows_may_hold_anything(fmt, Hq, n):
    """A drafted token with NaN keys and values reaches those that see it, and no one else."""
    b = Batch(fmt, [90 + n], [n], Hq, 2, 128, 16, seed=12)
    k = _rand(_gen(5), 1, 2, 128)
    k[0, :, 3] = float("nan")
    bad = 2
    qg.cache_write(b.cache, k, k, b.slots[90 + bad:91 + bad].int())
    out, lse = b.run()
    sees = b.see[:n, bad]
    assert sees.any() and not sees.all()
    got = out[:n].isnan().flatten(1)
    assert (got.all(1).cpu().numpy() == sees).all() and (got.any(1).cpu().numpy() == sees).all()
    b.check(out, lse)
    # a NaN value under a finite key does the same (to the log-sum as well)
    qg.cache_write(b.cache, _rand(_gen(6), 1, 2, 128), k, b.slots[90 + bad:91 + bad].int())
    out, lse = b.run()
    assert (out[:n].isnan().flatten(1).all(1).cpu().numpy() == sees).all()
    b.check(out, lse)


@pytest.mark.parametrize("Hq,n", [(2, 1), (32, 5)])
def test_values_of_very_different_scale(Hq, n):
    """Value scales 60 powers of two apart: the largest product of weight and scale sets the f16 range."""
    b = Batch(qg.QG_FP8_DYNAMIC, [200], [n], Hq, 2, 64, 16, seed=1, tree=False)
    for mul in (2.0 ** -30, 2.0 ** 30):
        b.cache.v_scale.view(-1)[::3] *= mul
        b.check(*b.run())
    b.q[:, :, :] *= 2.0 ** 40          # queries outside the f16 range
    b.check(*b.run(scale=2.0 ** -44), scale=2.0 ** -44)
    b.q[:, :, :] *= 2.0 ** -90
    b.check(*b.run(scale=2.0 ** 46), scale=2.0 ** 46)


def test_mask_words_and_max_q():
    """Drafted tokens past the mask's words are hidden; tokens past max_q get no output."""
    b = Batch(qg.QG_FP8_DYNAMIC, [300], [100], 2, 2, 64, 16, seed=2, words=1)
    b.check(*b.run())
    b = Batch(qg.QG_FP8_DYNAMIC, [100, 60], [20, 3], 24, 2, 64, 16, seed=2, tree=False)
    whole, _ = b.run()
    part, lse = b.run(max_q=7)
    done = list(range(7)) + list(range(20, 23))
    # the same rows, split over the CTAs otherwise: the sums' order differs
    assert torch.allclose(part[done].float(), whole[done].float(), rtol=2 * BF16, atol=1e-3)
    assert (part[7:20] == 7).all() and (lse[7:20] == 7).all()


@pytest.mark.parametrize("Hq,n", [(8, 1), (32, 12)])
def test_repeatable(Hq, n):
    """The same call twice gives the same bits, in a workspace that holds anything."""
    b = Batch(qg.QG_W8A8_INT8, [3000, 500, 77], [n] * 3, Hq, 4, 128, 64, seed=8)
    ws = qg.Workspace("cuda")
    first = b.run(workspace=ws)
    ws.buf.fill_(0xff)
    second = b.run(workspace=ws)
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])


@pytest.mark.parametrize("Hq,n", [(8, 1), (64, 9)])
def test_strides_streams_and_graphs(Hq, n):
    """Queries and outputs inside wider rows, another stream, and a graph whose lengths change between replays."""
    b = Batch(qg.QG_FP8_DYNAMIC, [900, 1200], [n, n], Hq, 4, 128, 16, seed=6, tree=n > 1)
    ref, ref_lse = b.run()
    wide = torch.zeros(b.T + 3, Hq + 8, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 4:Hq + 4] = b.q
    out = torch.full_like(wide, 7.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qg.attend(b.cache, wide[:, 4:Hq + 4], b.offs, b.lens_t, b.table, tree_mask=b.mask, max_q=n, out=out[:, 8:],
              stream=side)
    side.synchronize()
    assert torch.equal(out[:b.T, 8:], ref[:b.T]) and (out[:, :8] == 7).all() and (out[b.T:] == 7).all()
    ws, got = qg.Workspace("cuda"), torch.empty_like(b.q)
    qg.attend(b.cache, b.q, b.offs, b.lens_t, b.table, tree_mask=b.mask, max_q=n, out=got, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg.attend(b.cache, b.q, b.offs, b.lens_t, b.table, tree_mask=b.mask, max_q=n, out=got, workspace=ws)
    for lens in ([900, 1200], [40, 1200], [900, n]):
        b.lens_t.copy_(torch.tensor(lens, dtype=torch.int32))
        got.zero_()
        graph.replay()
        eager, _ = b.run()
        assert torch.equal(got[:b.T], eager[:b.T])


def test_two_streams_at_once():
    """Two calls that overlap, each with its own workspace."""
    b = Batch(qg.QG_FP8_DYNAMIC, [6000] * 4, [1] * 4, 32, 4, 128, 64, seed=6, tree=False)
    c = Batch(qg.QG_W8A8_INT8, [2000] * 4, [8] * 4, 32, 4, 128, 64, seed=7)
    want = b.run()[0], c.run()[0]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(5):
        for x, st, o in zip((b, c), streams, outs):
            with torch.cuda.stream(st):
                o.append(x.run()[0])
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, y) for y in o)


def test_far_pages():
    """Rows whose byte offset passes 32 bits."""
    D, page, H = 128, 1024, 8
    pages = (1 << 32) // (page * H * D) + 4
    cache = qg.Cache(qg.QG_FP8_DYNAMIC, pages, page, H, D)
    g = _gen(0)
    T = 40
    k, v, q = _rand(g, T, H, D), _rand(g, T, H, D), _rand(g, 1, H, D)
    near = qg.Cache(qg.QG_FP8_DYNAMIC, 1, page, H, D)
    place = torch.arange(T, dtype=torch.int32, device="cuda")
    qg.cache_write(near, k, v, place)
    qg.cache_write(cache, k, v, place + (pages - 1) * page)
    for a, b in zip(qg.cache_read(cache, place + (pages - 1) * page), qg.cache_read(near, place)):
        assert torch.equal(a, b)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    a = qg.attend(cache, q, ints(0, 1), ints(T), ints(pages - 1).view(1, 1))
    b = qg.attend(near, q, ints(0, 1), ints(T), ints(0).view(1, 1))
    assert torch.equal(a, b) and a.isfinite().all()


# ------------------------------------------------------------------- together --
@pytest.mark.parametrize("fmt", [qg.QG_FP8_DYNAMIC, qg.QG_W8A8_INT8, qg.QG_BLOCK_FP8])
def test_decoder_step(fmt):
    """norm -> product -> rotary cache write -> attention -> product -> norm, eager against the float64
    oracle stage by stage (each stage on the previous one's own output), and captured into a graph."""
    T, hidden, Hq, Hkv, D, page = 6, 512, 8, 2, 128, 16
    kv_fmt = qg.QG_W8A8_INT8 if fmt == qg.QG_W8A8_INT8 else qg.QG_FP8_DYNAMIC
    lens, ns = [40, 3, 75], [1, 3, 2]
    b = Batch(kv_fmt, lens, ns, Hq, Hkv, D, page, seed=4)
    g = _gen(11)
    w1, w2 = _rand(g, hidden, scale=0.1, offset=1.0), _rand(g, hidden, scale=0.1, offset=1.0)
    Wqkv = qg.quantize_weight(fmt, _rand(g, (Hq + 2 * Hkv) * D, hidden, scale=0.05))
    Wo = qg.quantize_weight(fmt, _rand(g, hidden, Hq * D, scale=0.05))
    resid = _rand(g, T, hidden)
    freq, _ = qg.rope_frequencies(64, 10000.0)
    rope = qg.Rope(freq)
    at = list(itertools.accumulate(lens, initial=0))
    slots = torch.cat([b.slots[at[i + 1] - n:at[i + 1]] for i, n in enumerate(ns)]).int()
    pos = torch.cat([torch.arange(a - n, a) for a, n in zip(lens, ns)]).int().cuda()
    mask = b.mask[:T].contiguous()

    def step():
        n1 = qg.norm(resid, w1, fmt=fmt)
        qkv = qg.run(fmt, n1.operand, Wqkv).view(T, Hq + 2 * Hkv, D)
        q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
        qr = qg.cache_write(b.cache, k, v, slots, q=q, rope=rope, positions=pos)
        o = qg.attend(b.cache, qr, b.offs, b.lens_t, b.table, tree_mask=mask, max_q=3)
        a = qg.quantize_act(fmt, o.view(T, Hq * D))
        proj = qg.run(fmt, a, Wo)
        return n1, qkv, qr, o, proj, qg.norm(resid, w2, proj, fmt=fmt)

    n1, qkv, qr, o, proj, n2 = step()
    kw = dict(kind="rms", eps=1e-6)
    h, y, dh, dy = _norm_oracle(resid, None, w1, kw)
    _check_codes(n1.operand, fmt, y, dy)
    want_k = OL.rotate(_np(qkv[:, Hq:Hq + Hkv]), _np(pos), _np(freq), False)
    (kc, ks), _ = _cache_values(b.cache, slots)
    _check_rows(kc, ks, want_k, 16 * F32 * np.abs(_np(qkv[:, Hq:Hq + Hkv])).max(axis=-1, keepdims=True) * np.ones(D),
                kv_fmt, "k")
    b.q[:T] = qr
    out7 = torch.full((T + 3, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out7[:T] = o
    _, lse = b.run()
    b.check(out7, lse)
    h, y, dh, dy = _norm_oracle(resid, proj, w2, dict(kw, block_scale=1.0, residual_scale=1.0))
    _close(n2.h, h, BF16 * np.abs(h) + dh, "h")
    _check_codes(n2.operand, fmt, y, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap[3], o) and torch.equal(cap[5].h, n2.h) and torch.equal(cap[5].operand.q, n2.operand.q)


@pytest.mark.parametrize("Hq,n", [(8, 1), (64, 9)])
def test_rewritten_slots_are_read_afresh(Hq, n):
    """Writes and reads of the same slots in turn, eager and captured: each call sees what the one before it wrote."""
    D, Hkv, T, turns = 128, 4, 40, 12
    g = _gen(8)
    cache = qg.Cache(qg.QG_FP8_DYNAMIC, 4, 16, Hkv, D)
    kv = _rand(g, turns, 2, T, Hkv, D)
    q = _rand(g, n, Hq, D)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    place = torch.arange(T, device="cuda")
    slots = (table[0, place // 16] * 16 + place % 16).int()
    offs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    ws = qg.Workspace("cuda")

    def turn(i, sync):
        qg.cache_write(cache, kv[i, 0], kv[i, 1], slots)
        if sync:
            torch.cuda.synchronize()
        o = qg.attend(cache, q, offs, lens, table, max_q=n, workspace=ws)
        if sync:
            torch.cuda.synchronize()
        return [o, *qg.cache_read(cache, slots)]

    want = [turn(i, True) for i in range(turns)]
    got = [turn(i, False) for i in range(turns)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = [turn(i, False) for i in range(turns)]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for w, a, b in zip(want, got, cap):
            assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(w, a, b))


def test_binding_refuses():
    c = qg.Cache(qg.QG_FP8_DYNAMIC, 4, 16, 2, 64)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    rope = qg.Rope(qg.rope_frequencies(64)[0])
    for bad in (lambda: qg.cache_write(c, k, k, slots.long()), lambda: qg.cache_write(c, k.float(), k, slots),
                lambda: qg.cache_write(c, k, k[:2], slots), lambda: qg.cache_write(c, k, k, slots, rope=rope),
                lambda: qg.cache_write(c, k, k, slots, q_out=k), lambda: qg.cache_read(c, slots, k=k.transpose(1, 2)),
                lambda: qg.cache_write(c, k, k, slots, rope=qg.Rope(rope.frequency.cpu()), positions=slots),
                lambda: qg.norm(k.view(3, 128), k.view(3, 128)[0, :64].contiguous()),
                lambda: qg.norm(k.view(3, 128).t(), k.view(3, 128)[0]),
                lambda: qg.attend(c, k, slots, slots, slots.view(3, 1)),
                lambda: qg.attend(c, k, slots[:2], slots[:1], slots[:1].view(1, 1), tree_mask=slots.view(3, 1)),
                lambda: qg.attend(c, k, slots[:2], slots[:1], slots[:1].view(1, 1), lse=k)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(qg.QGemmError):
        qg.attend(c, k, slots[:2], slots[:1], slots[:1].view(1, 1), max_q=0)
    with pytest.raises(qg.QGemmError):
        qg.attend(c, k[:, :1].contiguous(), slots[:2], slots[:1], slots[:1].view(1, 1))
