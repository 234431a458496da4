"""Decode over a prefix that the batch shares (fa_decode_int8_shared, fa_decode_int4_shared) against
its definition in 64 bits.

Bound of the differences, per output element, from the roundings the kernels make: the output to bf16
(half a step, 2^-8 of the value); the probabilities, the value scales and their products with the codes
to fp16 (2^-11 each, of sum p |v|); fp16 values below its normal range (2^-30 of the largest |v| a
key).  Scores are fp32 sums of exact products: 128 additions, each off by at most 2^-23 of
X = max_j scale sum_d |q_d k_jd|, so 2^-16 X, doubled for the scaling by k_scale and the exponent's
argument; a weight is off by twice that (its own score and the sum's) and 2^-20 for exp and the merges."""
import numpy as np
import pytest

import tiled_attention_26_b200 as fa
from test_kv_cache import _bf16, _bits, bf16_to_f64, built, make_rows, pack, quantize_f64  # noqa: F401

ST = fa.STATUS
FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails before any CUDA call
gpu = pytest.mark.gpu


# --------------------------------------------------------------------------- refusals (no GPU)
def raw_call(name, q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pt=FAKE, pl=FAKE, bt=FAKE, sl=FAKE, o=FAKE,
             lse=FAKE, B=2, Hq=8, Hkv=2, P=64, mpp=8, mp=8, pages=16, D=128, scale=0.1, splits=0, ws=FAKE,
             nb=1 << 40):
    return getattr(fa.lib(), name)(q, k, v, ks, vs, pt, pl, bt, sl, o, lse, B, Hq, Hkv, P, mpp, mp, pages, D,
                                   scale, splits, ws, nb, None)


@pytest.mark.parametrize("name", ["fa_decode_int8_shared", "fa_decode_int4_shared"])
@pytest.mark.parametrize("kw,code", [
    (dict(q=None), "FA_ERR_INVALID_ARG"), (dict(pt=None), "FA_ERR_INVALID_ARG"),
    (dict(pl=None), "FA_ERR_INVALID_ARG"), (dict(sl=None), "FA_ERR_INVALID_ARG"),
    (dict(o=None), "FA_ERR_INVALID_ARG"), (dict(B=0), "FA_ERR_INVALID_ARG"),
    (dict(Hq=7), "FA_ERR_INVALID_ARG"), (dict(P=48), "FA_ERR_INVALID_ARG"),
    (dict(P=8), "FA_ERR_INVALID_ARG"), (dict(mpp=0), "FA_ERR_INVALID_ARG"),
    (dict(mp=0), "FA_ERR_INVALID_ARG"), (dict(mpp=1 << 25), "FA_ERR_INVALID_ARG"),
    (dict(pages=0), "FA_ERR_INVALID_ARG"), (dict(splits=-1), "FA_ERR_INVALID_ARG"),
    (dict(splits=65536), "FA_ERR_INVALID_ARG"), (dict(B=65536), "FA_ERR_INVALID_ARG"),
    (dict(scale=0.0), "FA_ERR_INVALID_ARG"), (dict(scale=float("inf")), "FA_ERR_INVALID_ARG"),
    (dict(D=96), "FA_ERR_UNSUPPORTED"), (dict(k=FAKE + 8), "FA_ERR_ALIGNMENT"),
    (dict(pt=FAKE + 2), "FA_ERR_ALIGNMENT"), (dict(pl=FAKE + 1), "FA_ERR_ALIGNMENT"),
    (dict(lse=FAKE + 2), "FA_ERR_ALIGNMENT"), (dict(ws=None), "FA_ERR_WORKSPACE"),
    (dict(nb=1000), "FA_ERR_WORKSPACE"),
])
def test_rejects(built, name, kw, code):
    assert raw_call(name, **kw) == ST[code]


def test_workspace_bytes(built):
    f = fa.fa_decode_shared_workspace_bytes
    need = f(2, 8, 2, 128, 512, 512)
    assert need > 0 and raw_call("fa_decode_int8_shared", nb=need - 1) == ST["FA_ERR_WORKSPACE"]
    assert f(0, 8, 2, 128, 512, 512) == 0 and f(2, 7, 2, 128, 512, 512) == 0
    assert f(2, 8, 2, 128, 0, 512) == 0 and f(2, 8, 2, 128, 512, 512, -1) == 0
    assert f(2, 8, 2, 128, 512, 512, 40) > f(2, 8, 2, 128, 512, 512, 1)


def test_binding_rejects():
    import torch
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    pool = [torch.zeros(5, 16, 2, 64, dtype=torch.int8)] * 2 + [torch.zeros(5, 2, 16)] * 2
    i32 = dict(dtype=torch.int32)
    args = [torch.zeros(3, **i32), torch.zeros(1, **i32), torch.zeros(2, 3, **i32), torch.zeros(2, **i32)]

    def call(**kw):
        a = list(args)
        for i, x in kw.get("at", {}).items():
            a[i] = x
        return fa.fa_decode_int8_shared(kw.get("q", q), *pool, *a)

    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(ValueError, match="one query"):
        call(q=q.expand(2, 2, 4, 64).contiguous())
    with pytest.raises(ValueError, match="prefix_table"):
        call(at={0: args[2]})
    with pytest.raises(ValueError, match="prefix_len"):
        call(at={1: torch.zeros(2, **i32)})
    with pytest.raises(TypeError):
        call(at={0: args[0].long()})
    with pytest.raises(ValueError, match="seqlens"):
        call(at={3: torch.zeros(3, **i32)})
    with pytest.raises(ValueError, match="block_table"):
        call(at={2: torch.zeros(3, 3, **i32)})


# --------------------------------------------------------------------------------- on the GPU
class Case:
    """Inputs of one call on the host, the device tensors, and the definition's result."""

    def __init__(self, bits, B, Hq, Hkv, D, P, prefix, lens, seed=1, spare=2, kind="normal", scale=None):
        import torch
        rng = np.random.default_rng(seed)
        self.bits, self.B, self.Hq, self.Hkv, self.D, self.P = bits, B, Hq, Hkv, D, P
        self.prefix, self.lens = prefix, list(lens)
        up = lambda n: -(-n // P)  # noqa: E731
        npre, counts = up(prefix), [up(n) for n in lens]
        pages = npre + sum(counts) + 2
        order = rng.permutation(pages).astype(np.int32)
        m = 127 if bits == 8 else 7
        self.pool, self.codes, self.scales = [], [], []
        for w in range(2):
            c, s = quantize_f64(make_rows(seed + 10 + w, (pages, P, Hkv, D), "normal"), m)
            s = s.copy()
            if kind == "scales":  # scales of all sizes, rising over the prefix, zeros among them
                for i, pg in enumerate(order[:npre]):
                    s[pg] *= np.float32(2.0) ** (3 * i - 40 if w else 0)
                s[rng.random(s.shape) < 0.1] = 0
            self.codes.append(c)
            self.scales.append(s)
            self.pool.append(pack(c, bits))
        # entries behind the last page hold ids that must not be read
        self.pt = np.full(npre + spare, -9, np.int32)
        self.pt[:npre] = order[:npre]
        self.bt = np.full((B, max(counts + [1])), 1 << 30, np.int32)
        at = npre
        for b, n in enumerate(counts):
            self.bt[b, :n] = order[at:at + n]
            at += n
        self.qb = make_rows(seed + 5, (B, 1, Hq, D), "normal")
        if kind == "peaked":  # scores whose maximum keeps growing along the keys
            q = bf16_to_f64(self.qb) * 12
            self.qb = (q.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
        if kind == "rows":  # rows of very different sizes, and a row of zeros
            q = bf16_to_f64(self.qb) * (2.0 ** rng.integers(-130, 3, (B, 1, Hq, 1)))
            q[0, 0, 0] = 0
            self.qb = (q.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
        self.scale = D ** -0.5 if scale is None else scale
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.dev = dict(q=_bf16(self.qb), kp=t(self.pool[0]), vp=t(self.pool[1]),
                        ks=t(self.scales[0].transpose(0, 2, 1)), vs=t(self.scales[1].transpose(0, 2, 1)),
                        pt=t(self.pt), pl=t(np.array([prefix], np.int32)), bt=t(self.bt),
                        sl=t(np.array(lens, np.int32)))

    def call(self, splits=0, **kw):
        d = self.dev
        return getattr(fa, f"fa_decode_int{self.bits}_shared")(
            d["q"], d["kp"], d["vp"], d["ks"], d["vs"], d["pt"], d["pl"], d["bt"], d["sl"], num_splits=splits,
            scale=self.scale, **kw)

    def keys(self, w, b):
        """[Hkv, n, D]: the prefix's rows, then the sequence's own."""
        if not hasattr(self, "_prefix"):
            self._prefix = {}
        if (w, self.prefix) not in self._prefix:
            j = np.arange(self.prefix)
            self._prefix[w, self.prefix] = self._rows(w, self.pt[j // self.P], j % self.P)
        i = np.arange(self.lens[b])
        own = self._rows(w, self.bt[b, i // self.P], i % self.P)
        return np.concatenate([self._prefix[w, self.prefix], own], 1)

    def _rows(self, w, pg, r):
        return (self.codes[w][pg, r] * self.scales[w][pg, r].astype(np.float64)[..., None]).transpose(1, 0, 2)

    def check(self, o, lse):
        o, lse = bf16_to_f64(_bits(o)), lse.cpu().numpy().astype(np.float64)
        Hkv, G = self.Hkv, self.Hq // self.Hkv
        q = bf16_to_f64(self.qb)
        for b in range(self.B):
            k, v = self.keys(0, b), self.keys(1, b)
            n = k.shape[1]
            if n == 0:
                assert (o[b] == 0).all() and np.isneginf(lse[b]).all()
                continue
            qb = q[b, 0].reshape(Hkv, G, self.D)
            x = self.scale * (qb @ k.transpose(0, 2, 1))  # [Hkv, G, n]
            X = self.scale * (np.abs(qb) @ np.abs(k).transpose(0, 2, 1)).max(-1)
            top = x.max(-1, keepdims=True)
            p = np.exp(x - top)
            total = p.sum(-1)
            want, size = p @ v / total[..., None], p @ np.abs(v) / total[..., None]
            L = top[..., 0] + np.log(total)
            weight = (2 * 2.0 ** -15 * X + 2.0 ** -20)[..., None]
            tol = (2.0 ** -8 * np.abs(want) + (3 * 2.0 ** -11 + weight) * size +
                   (n + 1) * 2.0 ** -30 * np.abs(v).max((1, 2))[:, None, None] + 1e-38)
            err = np.abs(o[b, 0].reshape(Hkv, G, self.D) - want)
            assert (err <= tol).all(), (b, np.argwhere(~(err <= tol))[0], err.max())
            err = np.abs(lse[b].reshape(Hkv, G) - L)
            assert (err <= 2.0 ** -15 * X + 2.0 ** -20 + 2.0 ** -21 * np.abs(L)).all(), (b, err.max())


CASES = [  # bits, B, Hq, Hkv, D, P, prefix, own lengths, num_splits
    # one block of rows: 1, 2, 3 and more tiles of the prefix in two streams
    (8, 1, 1, 1, 128, 16, 1, [1], 0),
    (8, 2, 8, 2, 128, 64, 128, [5, 60], 0),
    (8, 2, 8, 2, 128, 64, 129, [64, 65], 1),
    (8, 3, 6, 2, 64, 16, 257, [0, 1, 17], 0),
    (4, 3, 21, 3, 128, 32, 500, [130, 2, 31], 3),
    (4, 16, 8, 1, 64, 256, 4000, list(range(16)), 0),   # R = 128
    (8, 13, 16, 2, 128, 128, 3001, [300 - 20 * b for b in range(13)], 0),
    (8, 1, 4, 4, 128, 64, 30001, [100], 0),  # every SM a few tiles
    # two blocks of rows and more: a part block, a full one, several CTAs of 256 rows
    (8, 43, 6, 2, 128, 64, 127, [3] * 43, 0),           # R = 129
    (4, 16, 32, 2, 128, 16, 700, [9 * b for b in range(16)], 0),  # R = 256
    (8, 3, 232, 1, 64, 64, 1000, [40, 0, 129], 0),      # R = 696: three blocks
    (4, 5, 116, 1, 64, 64, 300, [1, 2, 3, 4, 5], 2),    # R = 580
    (8, 10, 64, 2, 128, 128, 2600, [100] * 10, 4),      # R = 320: a block of 64 rows
    # no prefix, no keys of their own, neither
    (8, 3, 8, 2, 128, 64, 0, [7, 0, 300], 0),
    (8, 40, 8, 2, 64, 64, 0, [b % 3 for b in range(40)], 0),
    (4, 2, 8, 2, 128, 64, 300, [0, 0], 0),
    (8, 130, 4, 2, 64, 16, 50, [b % 20 for b in range(130)], 0),
    # more pages in one split than the kernel stages (256); 16 rows a CTA
    (8, 2, 4, 1, 64, 16, 40, [5000, 3], 1),
    (4, 1, 16, 1, 128, 16, 20, [4700], 1),
    (8, 2, 29, 1, 128, 32, 4500, [0, 700], 2),
]


@gpu
@pytest.mark.parametrize("bits,B,Hq,Hkv,D,P,prefix,lens,splits", CASES)
def test_matches_definition(built, bits, B, Hq, Hkv, D, P, prefix, lens, splits):
    c = Case(bits, B, Hq, Hkv, D, P, prefix, lens)
    c.check(*c.call(splits))
    assert fa.fa_device_status() == 0


# The same where the rows and the tiles per SM are many enough for the tcgen05 kernel: 128 rows a CTA as two
# streams of tiles (1, 2 and 3 tiles), blocks of 256 rows (whole, part, several), padding rows, every page size.
WIDE = [
    (8, 16, 736, 92, 64, 64, 1, [b % 3 for b in range(16)], 0),         # R = 128, one key
    (4, 16, 736, 92, 128, 16, 127, list(range(16)), 0),                 # one tile
    (8, 32, 384, 96, 128, 64, 129, [5 * b for b in range(32)], 1),      # two tiles, the second of one key
    (8, 13, 280, 40, 64, 32, 1000, [300 - 20 * b for b in range(13)], 0),  # R = 91, splits of 2 and 3 tiles
    (4, 13, 28, 4, 128, 16, 9003, [60 * b for b in range(13)], 3),
    (8, 13, 16, 2, 128, 256, 9500, [300 - 20 * b for b in range(13)], 0),
    (8, 43, 150, 50, 128, 64, 200, [3] * 43, 0),                        # R = 129
    (4, 16, 480, 30, 128, 16, 515, [9 * b for b in range(16)], 0),      # R = 256
    (8, 12, 232, 1, 64, 64, 641, [40, 0, 129] * 4, 0),                  # R = 2784: 11 blocks
    (4, 5, 116, 1, 64, 64, 3500, [1, 2, 3, 4, 5], 2),                   # R = 580
    (8, 10, 64, 2, 128, 128, 3001, [100] * 10, 4),                      # R = 320: a block of 64 rows
]


@gpu
@pytest.mark.parametrize("bits,B,Hq,Hkv,D,P,prefix,lens,splits", WIDE)
def test_wide_matches_definition(built, bits, B, Hq, Hkv, D, P, prefix, lens, splits):
    c = Case(bits, B, Hq, Hkv, D, P, prefix, lens)
    c.check(*c.call(splits))
    assert fa.fa_device_status() == 0


@gpu
@pytest.mark.parametrize("prefix", [0, 1, 130])
def test_prefix_shorter_than_its_table(built, prefix):
    """The launch follows the table's size, the work the length on the device."""
    c = Case(8, 16, 480, 30, 128, 16, 700, [0, 1, 30, 200] * 4)
    c.prefix = prefix
    c.dev["pl"].fill_(prefix)
    c.check(*c.call())
    assert fa.fa_device_status() == 0


@gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kind", ["scales", "peaked", "rows"])
@pytest.mark.parametrize("B,Hq,Hkv,D,prefix", [(16, 192, 24, 128, 700), (20, 192, 24, 64, 700)])
def test_wide_ranges(built, bits, kind, B, Hq, Hkv, D, prefix):
    c = Case(bits, B, Hq, Hkv, D, 64, prefix, [(37 * b) % 100 for b in range(B)], kind=kind)
    c.check(*c.call())


@gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kind", ["scales", "peaked", "rows"])
@pytest.mark.parametrize("B,Hq,Hkv,D,prefix", [(2, 8, 2, 128, 900), (20, 16, 2, 64, 700)])
def test_ranges(built, bits, kind, B, Hq, Hkv, D, prefix):
    c = Case(bits, B, Hq, Hkv, D, 64, prefix, [(37 * b) % 100 for b in range(B)], kind=kind)
    c.check(*c.call())


@gpu
def test_single_split_of_a_long_prefix_rescales(built):
    """Many tiles of one CTA (a batch of many KV heads leaves one split): maximum and value scales rise."""
    for kind in ("scales", "peaked"):
        c = Case(8, 33, 296, 74, 64, 64, 1500, [1] * 33, kind=kind)
        c.check(*c.call())


@gpu
def test_equals_paged_decode_over_joined_tables(built):
    """The same batch through fa_decode_int8_paged, its tables beginning with the prefix's pages."""
    import torch
    c = Case(8, 9, 32, 4, 128, 64, 1024, [1 + 50 * b for b in range(9)])
    o, lse = c.call()
    d = c.dev
    joined = torch.cat([d["pt"][:16].expand(9, 16), d["bt"]], 1).contiguous()
    o2, lse2 = fa.fa_decode_int8_paged(d["q"], d["kp"], d["vp"], d["ks"], d["vs"], joined,
                                       d["sl"] + 1024, num_splits=4, scale=c.scale)
    c.check(o2, lse2)
    assert (lse - lse2).abs().max() < 1e-4 and (o.float() - o2.float()).abs().max() < 2 ** -7


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("what", ["prefix page", "negative page", "prefix_len", "negative prefix_len", "page", "len"])
def test_bad_indices_are_reported(built, what, wide):
    c = Case(8, 43, 240, 80, 64, 16, 200, [20, 30, 0] + [1] * 40) if wide else Case(8, 3, 8, 2, 64, 16, 200, [20, 30, 0])
    d = c.dev
    if what == "prefix page":
        d["pt"][3] = c.pool[0].shape[0]
    elif what == "negative page":
        d["pt"][12] = -1
    elif what == "prefix_len":
        d["pl"][0] = 10 ** 9
        d["pt"].fill_(0)
    elif what == "negative prefix_len":
        d["pl"][0] = -1
    elif what == "page":
        d["bt"][1, 1] = 1 << 20
    else:
        d["sl"][1] = 49  # more than the table holds
    c.call()
    assert fa.fa_device_status() == ST["FA_ERR_DEVICE_INDEX"]
    assert fa.fa_device_status() == 0


@gpu
@pytest.mark.parametrize("B,Hkv", [(2, 2), (40, 2), (32, 64), (40, 64)])  # (64: the tcgen05 kernel)
def test_nan_rows(built, B, Hkv):
    """A row written from NaN (scale NaN): who reads it is NaN, the others are as they were; NaN in rows that
    nobody reads (the rest of the last pages) changes nothing."""
    import torch
    c = Case(8, B, 4 * Hkv, Hkv, 64, 64, 200, [30 + b for b in range(B)])
    d = c.dev
    for s in (d["ks"], d["vs"]):
        s[int(c.pt[3]), :, 200 % 64:] = float("nan")
        for b in range(B):
            if c.lens[b] % 64:
                s[int(c.bt[b, c.lens[b] // 64]), :, c.lens[b] % 64:] = float("nan")
    c.check(*c.call())
    for which in ("ks", "vs"):
        s = d[which]
        pg = int(c.pt[1])
        s[pg, 1, 7] = float("nan")
        o, lse = c.call()
        assert torch.isnan(o[:, 0, 4:8]).all() and torch.isnan(lse[:, 4:8]).all() == (which == "ks")
        o[:, 0, 4:8], lse[:, 4:8] = 0, 0
        assert not torch.isnan(o).any() and not torch.isnan(lse).any()
        s[pg, 1, 7] = 1.0
        own = int(c.bt[1, 0])
        s[own, 0, 3] = float("nan")
        o, lse = c.call()
        assert torch.isnan(o[1, 0, :4]).all() and torch.isnan(lse[1, :4]).all() == (which == "ks")
        o[1, 0, :4] = 0
        assert not torch.isnan(o).any()
        s[own, 0, 3] = 1.0


@gpu
@pytest.mark.parametrize("B,G,prefix", [(4, 1, 150), (16, 8, 1500)])
def test_offsets_past_32_bits(built, B, G, prefix):
    """A prefix in the last pages of a pool of more than 2^32 bytes of codes."""
    import torch
    c = Case(8, B, 8 * G, 8, 128, 64, prefix, [3, 70, 1, 0] * (B // 4))
    d, n = c.dev, c.pool[0].shape[0]
    pages = 2 ** 32 // (64 * 8 * 128) + n
    for key in ("kp", "vp", "ks", "vs"):
        big = torch.empty((pages, *d[key].shape[1:]), dtype=d[key].dtype, device="cuda")
        big[pages - n:] = d[key]
        big[:n].zero_()
        d[key] = big
    d["pt"] += pages - n
    d["bt"] += pages - n
    c.check(*c.call())


@gpu
@pytest.mark.parametrize("Hkv,G", [(2, 4), (46, 33)])  # (33 x 4 rows: the tcgen05 kernel)
def test_step_captured_and_replayed(built, Hkv, G):
    """A serving step (append the step's token, then decode) captured once and replayed while lengths, prefix and
    inputs change in place; a second graph with its own workspace; outputs of a replay do not change between runs."""
    import torch
    lens = [40, 63, 64, 10]
    Hq = Hkv * G
    c = Case(8, 4, Hq, Hkv, 128, 64, 333, [n + 3 for n in lens], spare=4)
    d = c.dev
    d["sl"].copy_(torch.tensor(lens, dtype=torch.int32))
    o, lse = torch.empty_like(d["q"]), torch.empty(4, Hq, device="cuda")
    ws = torch.empty(fa.fa_decode_shared_workspace_bytes(4, Hq, Hkv, 128, len(c.pt) * 64, c.bt.shape[1] * 64),
                     dtype=torch.uint8, device="cuda")
    k, v = (torch.empty(4, 1, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k.zero_()
    v.zero_()

    def step():
        fa.fa_kv_append_int8_paged(k, v, d["kp"], d["vp"], d["ks"], d["vs"], d["bt"], d["sl"])
        d["sl"].add_(1)
        c.call(o=o, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.call(o=o, lse=lse, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    c.lens = list(lens)
    c.check(o, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        kb, vb = (make_rows(70 + 2 * i + w, (4, 1, Hkv, 128), "normal") for w in range(2))
        k.copy_(_bf16(kb))
        v.copy_(_bf16(vb))
        if i == 2:
            c.prefix = 100
            d["pl"].fill_(100)
        ws.fill_(255)
        g.replay()
        for w, b in enumerate((kb, vb)):
            codes, scales = quantize_f64(b, 127)
            for s in range(4):
                pg, r = c.bt[s, c.lens[s] // 64], c.lens[s] % 64
                c.codes[w][pg, r], c.scales[w][pg, r] = codes[s, 0], scales[s, 0]
        c.lens = [n + 1 for n in c.lens]
        c.check(o, lse)
        o1, lse1 = c.call()
        assert torch.equal(o1, o) and torch.equal(lse1, lse)
    assert fa.fa_device_status() == 0


@gpu
def test_two_streams_at_once(built):
    import torch
    c = Case(8, 8, 32, 8, 128, 64, 3000, [100] * 8)
    e = Case(4, 20, 28, 4, 128, 16, 5000, [64] * 20, seed=7)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        outs += [x.call(stream=s) for x, s in zip((c, e), streams)]
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(outs):
        (c if i % 2 == 0 else e).check(o, lse) if i < 2 else None
        assert torch.equal(o, outs[i % 2][0]) and torch.equal(lse, outs[i % 2][1])
    assert fa.fa_device_status() == 0


@gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_given_buffers_and_a_stream_change_nothing(built, bits):
    import torch
    c = Case(bits, 3, 12, 2, 64, 16, 100, [20, 0, 33])
    o, lse = c.call()
    o2, none = c.call(return_lse=False)
    assert none is None and torch.equal(o, o2)
    out = dict(o=torch.empty_like(o), lse=torch.empty_like(lse),
               workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    o3, lse3 = c.call(**out)
    assert o3.data_ptr() == out["o"].data_ptr() and torch.equal(o, o3) and torch.equal(lse, lse3)
    o4, lse4 = c.call(stream=torch.cuda.current_stream())
    assert torch.equal(o, o4) and torch.equal(lse, lse4)
    with pytest.raises(fa.FaError):
        c.call(workspace=out["workspace"][:1000])
    with pytest.raises(fa.FaError):
        c.call(workspace=out["workspace"][8:])
    with pytest.raises(ValueError, match="workspace"):
        c.call(workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="lse"):
        c.call(lse=lse.flatten())


@gpu
@pytest.mark.parametrize("wide", [False, True])
def test_one_workspace_for_different_calls_in_a_row(built, wide):
    """Calls of different inputs that follow each other on one stream, in one workspace: none sees the partials
    of another."""
    import torch
    shape = (8, 16, 480, 30, 128, 64, 600) if wide else (8, 16, 16, 2, 128, 64, 3000)
    cases = [Case(*shape, [(37 * b + 50 * i) % 300 for b in range(16)], seed=40 + i) for i in range(3)]
    ref = [c.call() for c in cases]
    cases[0].check(*ref[0])
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    outs = [cases[i % 3].call(workspace=ws) for i in range(60)]
    for i, (o, lse) in enumerate(outs):
        assert torch.equal(o, ref[i % 3][0]) and torch.equal(lse, ref[i % 3][1]), i
