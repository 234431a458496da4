"""Writing the quantised KV cache (fa_kv_quantize_*, fa_kv_append_*_paged) and reading it back
(fa_kv_dequantize_*, fa_kv_gather_*_paged).  The definition fixes every rounding (scale and quotient
are 32-bit numbers, codes round half to even, values are one fp32 product rounded to bf16), so codes,
scales and values are compared bit for bit with a 64-bit evaluation of it."""
import numpy as np
import pytest

import tiled_attention_26_b200 as fa

ST = fa.STATUS
FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails before any CUDA call


# ------------------------------------------------------------------------------ the definition
def bf16_to_f64(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bf16_bits(x):
    """fp32 values (held in 64 bits) to bf16, ties to even; NaN to a NaN."""
    u = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7fff + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7fc0), r)


def quantize_f64(bits, m):
    """bf16 bit patterns [..., D] -> (whole codes [..., D] int64, fp32 scales [...])."""
    x = bf16_to_f64(bits)
    finite = np.isfinite(x).all(-1)
    a = np.where(finite, np.abs(np.where(np.isfinite(x), x, 0)).max(-1), 0)
    scale = (a / m).astype(np.float32)
    div = np.where(scale > 0, scale, 1).astype(np.float64)[..., None]
    with np.errstate(over="ignore", invalid="ignore"):
        q = (np.where(finite[..., None], x, 0) / div).astype(np.float32).astype(np.float64)
    codes = np.clip(np.rint(q), -m, m).astype(np.int64)
    codes[a == 0] = 0
    return codes, np.where(finite, scale, np.float32(np.nan)).astype(np.float32)


def pack(codes, bits):
    if bits == 8:
        return codes.astype(np.int8)
    n = (codes & 15).astype(np.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def values_bits(codes, scale):
    """bf16 bit patterns of code * scale (one fp32 product)."""
    with np.errstate(over="ignore"):
        prod = (codes.astype(np.float64) * scale[..., None].astype(np.float64)).astype(np.float32)
    return f64_to_bf16_bits(prod.astype(np.float64))


def make_rows(seed, shape, kind):
    """bf16 bit patterns of the named kind of row."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape).astype(np.float32)
    if kind == "ties":  # max|x| = 254 * 2^e: the quotient of every odd multiple of 2^e is k + 1/2
        x = rng.integers(-254, 255, shape).astype(np.float32) * np.float32(2.0) ** -6
        x[..., 0] = np.float32(254 * 2.0 ** -6)
    elif kind == "ties4":  # the same for m = 7
        x = rng.integers(-14, 15, shape).astype(np.float32) * np.float32(0.25)
        x[..., -1] = np.float32(-3.5)
    elif kind == "huge":
        x *= np.float32(6e37)
    elif kind == "tiny":  # scales below the normal range of fp32, where quotients pass m
        x *= np.float32(2.0) ** rng.integers(-132, -120, shape[:-1] + (1,)).astype(np.float32)
    elif kind == "zeros":
        x[...] = 0
        x[..., 1::2, :] *= -1
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)  # truncated: any bf16 will do
    if kind == "nonfinite":
        bits[..., 0, 3] = 0x7f80
        bits[..., 1 % shape[-2], 5] = 0xff80
        bits[0, ..., 7] = 0x7fc1
    return bits


# --------------------------------------------------------------------------- refusals (no GPU)
def quantize(name="fa_kv_quantize_int8", k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, B=2,
             S=100, Hkv=2, D=128):
    return getattr(fa.lib(), name)(k, v, kc, vc, ks, vs, B, S, Hkv, D, None)


@pytest.fixture(scope="module")
def built():
    from tiled_attention_26_b200 import build
    build.build()


@pytest.mark.parametrize("name", ["fa_kv_quantize_int8", "fa_kv_quantize_int4",
                                  "fa_kv_dequantize_int8", "fa_kv_dequantize_int4"])
@pytest.mark.parametrize("kw,code", [
    (dict(k=None), "FA_ERR_INVALID_ARG"), (dict(vs=None), "FA_ERR_INVALID_ARG"),
    (dict(B=0), "FA_ERR_INVALID_ARG"), (dict(S=0), "FA_ERR_INVALID_ARG"),
    (dict(Hkv=-1), "FA_ERR_INVALID_ARG"), (dict(B=1 << 16, S=1 << 15), "FA_ERR_INVALID_ARG"),
    (dict(D=96), "FA_ERR_UNSUPPORTED"), (dict(v=FAKE + 8), "FA_ERR_ALIGNMENT"),
    (dict(kc=FAKE + 4), "FA_ERR_ALIGNMENT"), (dict(ks=FAKE + 4), "FA_ERR_ALIGNMENT"),
])
def test_contiguous_rejects(built, name, kw, code):
    assert quantize(name, **kw) == ST[code]


def paged(name, k=FAKE, v=FAKE, kst=256, vst=256, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, bt=FAKE,
          pos=FAKE, cu=FAKE, N=10, B=2, Hkv=2, P=64, max_pages=8, num_pages=16, D=128):
    L = fa.lib()
    if "append" in name:
        return getattr(L, name)(k, v, kst, vst, kp, vp, ks, vs, bt, pos, cu, N, B, Hkv, P,
                                max_pages, num_pages, D, None)
    return getattr(L, name)(kp, vp, ks, vs, bt, pos, cu, k, v, N, B, Hkv, P, max_pages, num_pages,
                            D, None)


@pytest.mark.parametrize("name", ["fa_kv_append_int8_paged", "fa_kv_append_int4_paged",
                                  "fa_kv_gather_int8_paged", "fa_kv_gather_int4_paged"])
@pytest.mark.parametrize("kw,code", [
    (dict(k=None), "FA_ERR_INVALID_ARG"), (dict(vp=None), "FA_ERR_INVALID_ARG"),
    (dict(bt=None), "FA_ERR_INVALID_ARG"), (dict(N=-1), "FA_ERR_INVALID_ARG"),
    (dict(B=0), "FA_ERR_INVALID_ARG"), (dict(P=48), "FA_ERR_INVALID_ARG"),
    (dict(P=8), "FA_ERR_INVALID_ARG"), (dict(max_pages=1 << 25), "FA_ERR_INVALID_ARG"),
    (dict(num_pages=0), "FA_ERR_INVALID_ARG"),
    (dict(cu=None, N=11), "FA_ERR_INVALID_ARG"),  # not the same number of tokens of each sequence
    (dict(D=32), "FA_ERR_UNSUPPORTED"), (dict(kp=FAKE + 8), "FA_ERR_ALIGNMENT"),
    (dict(v=FAKE + 2), "FA_ERR_ALIGNMENT"), (dict(pos=FAKE + 2), "FA_ERR_ALIGNMENT"),
    (dict(cu=FAKE + 1), "FA_ERR_ALIGNMENT"), (dict(bt=FAKE + 3), "FA_ERR_ALIGNMENT"),
    (dict(N=0, k=None, v=None), "FA_OK"),
])
def test_paged_rejects(built, name, kw, code):
    assert paged(name, **kw) == ST[code]


@pytest.mark.parametrize("kw,code", [(dict(kst=255), "FA_ERR_INVALID_ARG"),
                                     (dict(vst=-256), "FA_ERR_INVALID_ARG"),
                                     (dict(vst=260), "FA_ERR_ALIGNMENT")])
def test_append_rejects_strides(built, kw, code):
    assert paged("fa_kv_append_int8_paged", **kw) == ST[code]


def test_binding_rejects():
    import torch
    bf = dict(dtype=torch.bfloat16)
    k = torch.zeros(2, 4, 2, 64, **bf)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_kv_quantize_int8(k, k)
    with pytest.raises(TypeError):
        fa.fa_kv_quantize_int8(k.float(), k)
    with pytest.raises(ValueError, match="shape"):
        fa.fa_kv_quantize_int4(k, k[:, :3].contiguous())
    pool = [torch.zeros(5, 16, 2, 64, dtype=torch.int8)] * 2 + [torch.zeros(5, 2, 16)] * 2
    bt = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="evenly spaced"):
        fa.fa_kv_append_int8_paged(torch.zeros(2, 6, 2, 64, **bf)[:, :4], k, *pool, bt)
    with pytest.raises(ValueError, match="contiguous"):
        fa.fa_kv_append_int8_paged(k.transpose(2, 3).contiguous().transpose(2, 3), k, *pool, bt)
    with pytest.raises(ValueError, match="sequences"):
        fa.fa_kv_append_int8_paged(k[:1], k[:1], *pool, bt)
    with pytest.raises(TypeError):
        fa.fa_kv_append_int8_paged(k, k, *pool, bt.long())
    with pytest.raises(ValueError, match="positions"):
        fa.fa_kv_append_int8_paged(k, k, *pool, bt, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="negative"):
        fa.fa_kv_gather_int8_paged(*pool, bt, -1)


# --------------------------------------------------------------------------------- on the GPU
gpu = pytest.mark.gpu


def _bf16(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def _bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def same_values(got_bits, want_bits):
    """Equal bit patterns, any NaN for a NaN."""
    g, w = bf16_to_f64(got_bits), bf16_to_f64(want_bits)
    return np.array_equal(got_bits[~np.isnan(w)], want_bits[~np.isnan(w)]) and np.isnan(g[np.isnan(w)]).all()


def _call(op, bits, paged=False):
    return getattr(fa, f"fa_kv_{op}_int{bits}" + ("_paged" if paged else ""))


CONTIGUOUS = [  # B, S, Hkv, D, kind
    (1, 1, 1, 128, "normal"), (1, 1, 1, 64, "normal"), (2, 33, 3, 128, "normal"),
    (3, 31, 5, 64, "ties"), (2, 70, 2, 128, "ties"), (2, 65, 2, 128, "ties4"),
    (1, 40, 2, 64, "huge"), (2, 64, 3, 128, "tiny"), (1, 32, 2, 64, "zeros"),
    (2, 35, 4, 128, "nonfinite"), (1, 4097, 8, 128, "normal"),
    # enough rows for 32 tokens a warp (37888)
    (2, 3001, 8, 128, "normal"), (3, 2543, 5, 64, "ties"), (1, 12701, 3, 64, "tiny"), (2, 9501, 2, 128, "nonfinite"),
]


@gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("B,S,Hkv,D,kind", CONTIGUOUS)
def test_contiguous_matches_definition(built, bits, B, S, Hkv, D, kind):
    m = 127 if bits == 8 else 7
    kb, vb = (make_rows(s, (B, S, Hkv, D), kind) for s in (1, 2))
    got = _call("quantize", bits)(_bf16(kb), _bf16(vb))
    back = _call("dequantize", bits)(*got)
    for x, codes, scale, val in ((kb, got[0], got[2], back[0]), (vb, got[1], got[3], back[1])):
        c, s = quantize_f64(x, m)
        assert np.array_equal(codes.cpu().numpy(), pack(c, bits))
        assert np.array_equal(scale.cpu().numpy(), s.transpose(0, 2, 1), equal_nan=True)
        assert same_values(_bits(val), values_bits(c, s))


@gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_every_quotient_of_mantissas(built, bits):
    """Rows whose largest value has each of the 128 mantissas, against every bf16 of a smaller or equal size
    that can round to a code other than 0: quotients on and next to a half among them.  A power of two in
    front changes nothing: small, large, and where 1 / scale would leave the normal range."""
    m = 127 if bits == 8 else 7
    x = np.arange(0x3f80 - 10 * 128, 0x4000, dtype=np.uint16)  # 2^-10 .. 2
    x = np.concatenate([x, x | 0x8000])
    rows = []
    for top in range(0x3f80, 0x4000):
        fit = x[(x & 0x7fff) <= top]
        fit = np.concatenate([fit, np.zeros(-len(fit) % 127, np.uint16)]).reshape(-1, 127)
        rows.append(np.concatenate([fit, np.full((len(fit), 1), top, np.uint16)], 1))
    rows = np.concatenate(rows)
    rows = np.concatenate([rows, np.zeros((-len(rows) % 3, 128), np.uint16)])
    for e in (0, 126, -30, -100, -116):
        b = rows if e == 0 else (bf16_to_f64(rows) * 2.0 ** e).astype(np.float32).view(np.uint32) >> 16
        b = b.astype(np.uint16).reshape(1, -1, 3, 128)
        codes, scale = quantize_f64(b, m)
        got = _call("quantize", bits)(_bf16(b), _bf16(b[:, ::-1].copy()))
        assert np.array_equal(got[0].cpu().numpy(), pack(codes, bits))
        assert np.array_equal(got[1].cpu().numpy(), pack(codes, bits)[:, ::-1])
        assert np.array_equal(got[2].cpu().numpy(), scale.transpose(0, 2, 1))


PAGED = [  # bits, Hkv, D, P, history, new tokens, padding rows
    (8, 8, 128, 64, [0], [1], 0),
    (8, 2, 128, 16, [0, 15, 16, 31], [1, 1, 1, 1], 0),
    (8, 3, 64, 32, [5, 0, 100, 7], [40, 0, 33, 1], 3),
    (4, 2, 128, 16, [9, 3, 0], [0, 129, 0], 2),
    (4, 5, 64, 64, [63, 1], [2, 300], 0),
    (8, 1, 128, 256, [0, 0, 0, 0, 255], [0, 0, 257, 0, 1], 31),
    # enough rows for 32 tokens a warp (37888)
    (8, 8, 128, 64, [5, 0, 100, 7, 63], [1700, 0, 33, 2900, 401], 3),
    (4, 5, 64, 16, [9 * b for b in range(37)], [(613 * b) % 420 for b in range(37)], 40),
]


def _paged_case(bits, Hkv, D, P, hist, new, pad, seed=3):
    import torch
    rng = np.random.default_rng(seed)
    B, n = len(hist), sum(new) + pad
    need = [-(-(h + t) // P) for h, t in zip(hist, new)]
    width, pages = max(max(need), 1), sum(need) + 2
    order = rng.permutation(pages)
    bt = np.full((B, width), -7, np.int32)
    at = 0
    for b, c in enumerate(need):
        bt[b, :c] = order[at:at + c]
        at += c
    code = np.int8 if bits == 8 else np.uint8
    row = D if bits == 8 else D // 2
    pool = [rng.integers(-128 if bits == 8 else 0, 127, (pages, P, Hkv, row)).astype(code) for _ in range(2)]
    pool += [rng.random((pages, Hkv, P)).astype(np.float32) for _ in range(2)]
    x = [make_rows(seed + i, (n, Hkv, D), "normal") for i in range(2)]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    dev = dict(pool=[torch.from_numpy(p.copy()).cuda() for p in pool], bt=torch.from_numpy(bt).cuda(),
               pos=torch.tensor(hist, dtype=torch.int32).cuda(), cu=torch.from_numpy(cu).cuda(),
               x=[_bf16(t) for t in x])
    return B, n, bt, pool, x, cu, dev


def _written(bits, P, hist, bt, pool, x, cu):
    """The pool after the append, by the definition, and each token's (page, row)."""
    m = 127 if bits == 8 else 7
    pool = [p.copy() for p in pool]
    place = [(bt[b, (hist[b] + i) // P], (hist[b] + i) % P)
             for b in range(len(hist)) for i in range(cu[b + 1] - cu[b])]
    for w in range(2):
        c, s = quantize_f64(x[w], m)
        for i, (pg, r) in enumerate(place):
            pool[w][pg, r] = pack(c[i], bits)
            pool[2 + w][pg, :, r] = s[i]
    return pool, place


@gpu
@pytest.mark.parametrize("bits,Hkv,D,P,hist,new,pad", PAGED)
def test_append_and_gather(built, bits, Hkv, D, P, hist, new, pad):
    import torch
    B, n, bt, pool, x, cu, dev = _paged_case(bits, Hkv, D, P, hist, new, pad)
    _call("append", bits, True)(*dev["x"], *dev["pool"], dev["bt"], dev["pos"], dev["cu"])
    want, place = _written(bits, P, hist, bt, pool, x, cu)
    for got, w in zip(dev["pool"], want):  # the new rows, and nothing else
        assert np.array_equal(got.cpu().numpy(), w)
    m = 127 if bits == 8 else 7
    out = [torch.full((n, Hkv, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    _call("gather", bits, True)(*dev["pool"], dev["bt"], n, dev["pos"], dev["cu"], *out)
    for w in range(2):
        v = values_bits(*quantize_f64(x[w], m))
        v[len(place):] = _bits(out[w].new_full((1,), 9.0))[0]  # behind the last sequence: untouched
        assert same_values(_bits(out[w]), v)
    assert fa.fa_device_status() == 0


@gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_append_uniform_strided(built, bits):
    """K and V as slices of one projection's output, the same number of tokens of each sequence."""
    import torch
    Hkv, D, P, T = 2, 128, 16, 3
    hist, new = [4, 14, 30], [T] * 3
    B, n, bt, pool, x, cu, dev = _paged_case(bits, Hkv, D, P, hist, new, 0)
    qkv = torch.zeros(B, T, 6 * D + 2 * Hkv * D + 8, dtype=torch.bfloat16, device="cuda")
    ks = qkv[..., 6 * D:6 * D + Hkv * D].view(B, T, Hkv, D)
    vs = qkv[..., 6 * D + Hkv * D:6 * D + 2 * Hkv * D].view(B, T, Hkv, D)
    ks.copy_(dev["x"][0].view(B, T, Hkv, D))
    vs.copy_(dev["x"][1].view(B, T, Hkv, D))
    _call("append", bits, True)(ks, vs, *dev["pool"], dev["bt"], dev["pos"])
    want, _ = _written(bits, P, hist, bt, pool, x, cu)
    for got, w in zip(dev["pool"], want):
        assert np.array_equal(got.cpu().numpy(), w)


@gpu
@pytest.mark.parametrize("what", ["page", "negative page", "position", "negative position", "cu order",
                                  "cu start", "cu end"])
def test_bad_indices_are_reported_and_skipped(built, what):
    hist, new, P = [5, 20], [30, 12], 16
    B, n, bt, pool, x, cu, dev = _paged_case(8, 2, 64, P, hist, new, 0)
    pages = pool[0].shape[0]
    untouched = None
    if what == "page":
        dev["bt"][1, 1] = pages
    elif what == "negative page":
        dev["bt"][1, 1] = -1
    elif what == "position":
        dev["pos"][1] = 2 ** 31 - 3
    elif what == "negative position":
        dev["pos"][1] = -2 ** 31
    elif what == "cu order":
        dev["cu"][1] = n + 5
    elif what == "cu start":
        dev["cu"][0] = 1
    else:
        dev["cu"][2] = n + 100
    _call("append", 8, True)(*dev["x"], *dev["pool"], dev["bt"], dev["pos"], dev["cu"])
    assert fa.fa_device_status() == ST["FA_ERR_DEVICE_INDEX"]
    if "page" in what or "position" in what:  # sequence 0 is written, the rows concerned are not
        want, place = _written(8, P, hist, bt, pool, x, cu)
        for (pg, r) in place[new[0]:]:
            for w in range(2):
                want[w][pg, r], want[2 + w][pg, :, r] = pool[w][pg, r], pool[2 + w][pg, :, r]
        for got, w in zip(dev["pool"], want):
            assert np.array_equal(got.cpu().numpy(), w)
    _call("gather", 8, True)(*dev["pool"], dev["bt"], n, dev["pos"], dev["cu"])
    assert fa.fa_device_status() == ST["FA_ERR_DEVICE_INDEX"]
    assert fa.fa_device_status() == 0


@gpu
def test_deterministic_mode_fills_new_buffers(built):
    """Rows behind the last sequence of a buffer that the call allocates: NaN in deterministic mode."""
    import torch
    B, n, bt, pool, x, cu, dev = _paged_case(8, 2, 64, 16, [3, 0], [2, 1], 4)
    args = (*dev["pool"], dev["bt"], n, dev["pos"], dev["cu"])
    want = fa.fa_kv_gather_int8_paged(*args)
    torch.use_deterministic_algorithms(True)
    try:
        got = fa.fa_kv_gather_int8_paged(*args)
    finally:
        torch.use_deterministic_algorithms(False)
    for g, w in zip(got, want):
        assert torch.equal(g[:3], w[:3]) and bool(g[3:].isnan().all())


@gpu
def test_zero_tokens(built):
    import torch
    B, n, bt, pool, x, cu, dev = _paged_case(8, 2, 64, 16, [3], [1], 0)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    fa.fa_kv_append_int8_paged(e, e, *dev["pool"], dev["bt"], dev["pos"])
    k, v = fa.fa_kv_gather_int8_paged(*dev["pool"], dev["bt"], 0)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)
    for got, w in zip(dev["pool"], pool):
        assert np.array_equal(got.cpu().numpy(), w)


@gpu
def test_offsets_past_32_bits(built):
    """A pool of more than 2^32 bytes of codes: the last page's rows are the ones written and read."""
    import torch
    Hkv, D, P = 8, 128, 64
    pages = 2 ** 32 // (P * Hkv * D) + 5
    pool = [torch.empty(pages, P, Hkv, D, dtype=torch.int8, device="cuda") for _ in range(2)]
    pool += [torch.empty(pages, Hkv, P, device="cuda") for _ in range(2)]
    x = [make_rows(s, (P, Hkv, D), "normal") for s in (5, 6)]
    bt = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    for p in pool:
        p[5 - 1].zero_()  # where a page id times the page's bytes, cut to 32 bits, would land
    fa.fa_kv_append_int8_paged(*(_bf16(t) for t in x), *pool, bt)
    out = fa.fa_kv_gather_int8_paged(*pool, bt, P)
    for w in range(2):
        c, s = quantize_f64(x[w], 127)
        assert np.array_equal(pool[w][-1].cpu().numpy(), c.astype(np.int8))
        assert np.array_equal(pool[2 + w][-1].cpu().numpy(), s.T)
        assert not pool[w][4].any() and not pool[2 + w][4].any()
        assert same_values(_bits(out[w]), values_bits(c, s))


@gpu
def test_graph_and_side_stream(built):
    """A captured append + gather replayed with positions and inputs rewritten in place; eager calls on a
    stream of their own."""
    import torch
    hist, new, P = [3, 17], [1, 1], 16
    B, n, bt, pool, x, cu, dev = _paged_case(8, 2, 128, P, hist, new, 0)
    out = [torch.empty(n, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def step(stream=None):
        fa.fa_kv_append_int8_paged(*dev["x"], *dev["pool"], dev["bt"], dev["pos"], stream=stream)
        fa.fa_kv_gather_int8_paged(*dev["pool"], dev["bt"], n, dev["pos"], None, *out, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    for w in range(2):
        assert same_values(_bits(out[w]), values_bits(*quantize_f64(x[w], 127)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(2):
        dev["pos"].add_(1)
        x = [make_rows(50 + 2 * k + w, (n, 2, 128), "normal") for w in range(2)]
        for t, b in zip(dev["x"], x):
            t.copy_(_bf16(b))
        g.replay()
        torch.cuda.synchronize()
        for w in range(2):
            assert same_values(_bits(out[w]), values_bits(*quantize_f64(x[w], 127)))
    want = [p.copy() for p in pool]
    assert fa.fa_device_status() == 0 and want[0].shape == tuple(dev["pool"][0].shape)


@gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("S,splits", [(5, 1), (300, 2), (300, 16)])
def test_decode_of_a_row_written_from_nan_is_nan(built, bits, S, splits):
    """K (then V) of one token of KV head 1 holds a NaN: the heads that read it are NaN, the others are not."""
    import torch
    B, Hq, Hkv, D = 2, 12, 3, 64
    k, v, q = (_bf16(make_rows(s, (B, n, h, D), "normal")) for s, n, h in ((1, S, Hkv), (2, S, Hkv), (3, 1, Hq)))
    for x in (k, v):
        kept = x[1, 2, 1].clone()
        x[1, 2, 1, 9] = float("nan")
        cache = _call("quantize", bits)(k, v)
        o, lse = getattr(fa, f"fa_decode_int{bits}")(q, *cache, num_splits=splits)
        assert torch.isnan(o[1, 0, 4:8]).all() and torch.isnan(lse[1, 4:8]).all() == (x is k)
        o[1, 0, 4:8], lse[1, 4:8] = 0, 0
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
        x[1, 2, 1] = kept


@gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_with_a_stream_as_without(built, bits):
    """The calls made directly (no stream argument) and those that go through the Python checks agree."""
    import torch
    here = torch.cuda.current_stream()
    k, v = (_bf16(make_rows(s, (2, 70, 3, 64), "normal")) for s in (1, 2))
    a, b = _call("quantize", bits)(k, v), _call("quantize", bits)(k, v, stream=here)
    a += _call("dequantize", bits)(*a)
    b += _call("dequantize", bits)(*b, stream=here)
    B, n, bt, pool, x, cu, dev = _paged_case(bits, 3, 64, 16, [3, 0, 40], [20, 1, 9], 2)
    twin = [t.clone() for t in dev["pool"]]
    _call("append", bits, True)(*dev["x"], *dev["pool"], dev["bt"], dev["pos"], dev["cu"])
    _call("append", bits, True)(*dev["x"], *twin, dev["bt"], dev["pos"], dev["cu"], stream=here)
    a += tuple(dev["pool"]) + _call("gather", bits, True)(*dev["pool"], dev["bt"], 30, dev["pos"], dev["cu"])
    b += tuple(twin) + _call("gather", bits, True)(*twin, dev["bt"], 30, dev["pos"], dev["cu"], stream=here)
    for s, t in zip(a, b):
        assert s.dtype == t.dtype and s.shape == t.shape and torch.equal(s, t)


@gpu
def test_refusals_on_the_gpu(built):
    """What the direct calls leave to the Python checks is refused there, and nothing is launched."""
    import torch
    B, n, bt, pool, x, cu, dev = _paged_case(8, 2, 64, 16, [3], [20], 0)
    args = [*dev["x"], *dev["pool"], dev["bt"], dev["pos"], dev["cu"]]
    for i, bad, err in ((0, dev["x"][0].float(), TypeError), (1, dev["x"][1][:, :1], ValueError),
                        (2, dev["pool"][0].view(torch.uint8), TypeError), (4, dev["pool"][2].transpose(1, 2), ValueError),
                        (6, dev["bt"].cpu(), ValueError), (7, dev["pos"].long(), TypeError),
                        (8, dev["cu"][:1], ValueError)):
        with pytest.raises(err):
            fa.fa_kv_append_int8_paged(*args[:i], bad, *args[i + 1:])
    with pytest.raises(fa.FaError):  # rows of 96 dims
        fa.fa_kv_quantize_int8(*[torch.zeros(1, 4, 2, 96, dtype=torch.bfloat16, device="cuda")] * 2)
    with pytest.raises(fa.FaError):  # 16-byte alignment
        odd = torch.zeros(4 * 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(1, 4, 2, 64)
        fa.fa_kv_quantize_int8(odd, odd)
    for got, w in zip(dev["pool"], pool):
        assert np.array_equal(got.cpu().numpy(), w)


@gpu
@pytest.mark.parametrize("bits,Hkv,D,P", [(8, 2, 128, 16), (4, 3, 64, 16)])
@pytest.mark.parametrize("ragged", [False, True])
def test_replayed_append_writes_the_right_rows(built, bits, Hkv, D, P, ragged):
    """A captured append replayed while positions, inputs and token counts change in place: every code and scale of the
    pool is what the appends in turn leave, the rows that no replay concerns included.  Ragged: num_tokens is
    an upper bound, most of whose rows belong to no sequence."""
    import torch
    hist, most = [3, 10, 20], [5, 3, 9]
    B, n, bt, pool, x, cu, dev = _paged_case(bits, Hkv, D, P, hist, most, 4)
    steps = [[5, 0, 9], [1, 2, 0], [0, 0, 0], [2, 1, 3]] if ragged else [[2, 2, 2], [1, 1, 1]]
    n = n if ragged else 6
    src = [torch.zeros(n, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    starts = torch.tensor([0] * B, dtype=torch.int32, device="cuda")
    call = lambda k: _call("append", bits, True)(  # noqa: E731
        *(t[:k] for t in src), *dev["pool"], dev["bt"], starts, dev["cu"] if ragged else None)
    graphs = {}
    for i, new in enumerate(steps):
        k = n if ragged else sum(new)
        if k not in graphs:
            graphs[k] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[k]):
                call(k)
        x = [make_rows(80 + 2 * i + w, (k, Hkv, D), "normal") for w in range(2)]
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        for t, b in zip(src, x):
            t[:k].copy_(_bf16(b))
        dev["cu"].copy_(torch.from_numpy(cu))
        starts.copy_(torch.tensor(hist, dtype=torch.int32))
        graphs[k].replay()
        pool, _ = _written(bits, P, hist, bt, pool, x, cu)
        for got, w in zip(dev["pool"], pool):
            assert np.array_equal(got.cpu().numpy(), w), i
        hist = [h + t for h, t in zip(hist, new)]
    assert fa.fa_device_status() == 0
