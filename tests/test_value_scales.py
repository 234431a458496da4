"""Decode over caches whose value scales span a wide range: blocks of zero rows (which the write stores with
scale 0), negative scales (a value is code * scale, whatever the sign), and values and queries near the ends of
bf16's range.  Against the definition in 64 bits.

Bound of the differences, per output element: the output to bf16 (half a step, 2^-8 of the value); the
probabilities, the value scales and their products with the codes to fp16 (2^-11 each, of sum p |v|); fp16
values below its normal range: the kernels scale the products so that the largest so far lies in
2^6 .. 2^8 times the probability, a step there is 2^-24, half of it at most 2^-30 of the largest |v|
a key.  Scores are fp32 sums of exact products, 128 additions off by at most 2^-23 of
X = max_j scale sum_d |q_d k_jd| each, 2^-16 X, doubled for the scaling and the exponent's argument; a weight is
off by twice that and 2^-20 for exp and the merges."""
import numpy as np
import pytest

import tiled_attention_26_b200 as fa
from test_kv_cache import _bf16, _bits, bf16_to_f64, built, make_rows, pack, quantize_f64  # noqa: F401
from test_shared_decode import Case

gpu = pytest.mark.gpu


class Cache:
    """A cache of B sequences of S tokens with changed value scales, contiguous or in pages of 64."""

    def __init__(self, bits, B, S, Hkv, D, change, seed=21):
        m = 127 if bits == 8 else 7
        self.bits, self.B, self.S, self.Hkv, self.D = bits, B, S, Hkv, D
        self.codes, self.scales = [], []
        for w in range(2):
            c, s = quantize_f64(make_rows(seed + w, (B, S, Hkv, D), "normal"), m)
            self.codes.append(c)
            self.scales.append(s.copy())
        self.qb = make_rows(seed + 2, (B, 1, 4 * Hkv, D), "normal")
        change(self)

    def contiguous(self):
        import torch
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return (*(t(pack(c, self.bits)) for c in self.codes), *(t(s.transpose(0, 2, 1)) for s in self.scales))

    def paged(self, P=64):
        import torch
        n = -(-self.S // P)
        order = np.random.default_rng(3).permutation(self.B * n).reshape(self.B, n)
        pool = []
        for x in [pack(c, self.bits) for c in self.codes] + self.scales:
            full = np.zeros((self.B, n * P, *x.shape[2:]), x.dtype)
            full[:, :self.S] = x
            pages = np.empty((self.B * n, P, *x.shape[2:]), x.dtype)
            pages[order.reshape(-1)] = full.reshape(self.B * n, P, *x.shape[2:])
            pool.append(pages if x.ndim == 4 else pages.transpose(0, 2, 1))
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return [t(x) for x in pool], t(order.astype(np.int32)), t(np.full(self.B, self.S, np.int32))

    def check(self, o, lse):
        o, lse = bf16_to_f64(_bits(o)), lse.cpu().numpy().astype(np.float64)
        q = bf16_to_f64(self.qb)
        for b in range(self.B):
            k, v = ((c[b] * s[b].astype(np.float64)[..., None]).transpose(1, 0, 2)
                    for c, s in zip(self.codes, self.scales))
            agree(o[b, 0], lse[b], q[b, 0], k, v, self.D ** -0.5)


def agree(o, lse, q, k, v, scale):
    """One sequence: o, q [Hq, D], lse [Hq], k, v [Hkv, n, D]."""
    Hkv, n, D = k.shape
    q = q.reshape(Hkv, -1, D)
    x = scale * (q @ k.transpose(0, 2, 1))
    X = scale * (np.abs(q) @ np.abs(k).transpose(0, 2, 1)).max(-1)
    top = x.max(-1, keepdims=True)
    p = np.exp(x - top)
    total = p.sum(-1)
    want, size = p @ v / total[..., None], p @ np.abs(v) / total[..., None]
    weight = (2 * 2.0 ** -15 * X + 2.0 ** -20)[..., None]
    tol = (2.0 ** -8 * np.abs(want) + (3 * 2.0 ** -11 + weight) * size +
           (n + 1) * 2.0 ** -30 * np.abs(v).max((1, 2))[:, None, None] + 1e-38)
    err = np.abs(o.reshape(want.shape) - want)
    assert (err <= tol).all(), (np.argwhere(~(err <= tol))[0], err.max(), size.max())
    L = top[..., 0] + np.log(total)
    err = np.abs(lse.reshape(L.shape) - L)
    assert (err <= 2.0 ** -15 * X + 2.0 ** -20 + 2.0 ** -21 * np.abs(L)).all(), err.max()


def zero_rows(n, size):
    """The first n rows hold zeros, the others values of magnitude ``size``."""
    def change(c):
        c.scales[1] *= np.float32(size)
        c.scales[1][:, :n] = 0
        c.codes[1][:, :n] = 0
    return change


def negative(c):
    """Small scales first, larger ones of the other sign behind them; keys' signs at random."""
    rng = np.random.default_rng(5)
    n = c.S // 2
    c.scales[1][:, :n] *= np.float32(2.0 ** -9)
    c.scales[1][:, n:] *= -1
    c.scales[0] *= rng.choice(np.float32([-1, 1]), c.scales[0].shape)


def all_negative(c):
    c.scales[1] *= -1


def huge_values(c):
    c.scales[1] *= np.float32(2.0 ** 122)


def tiny_values(c):
    c.scales[1] *= np.float32(2.0 ** -100)


def huge_queries(c):
    """Queries of 2^118 over keys of 2^-118: ordinary scores."""
    c.scales[0] *= np.float32(2.0 ** -118)
    c.qb = ((bf16_to_f64(c.qb) * 2.0 ** 118).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


CHANGES = [zero_rows(128, 1e-4), zero_rows(32, 2.0 ** -14), zero_rows(128, 1e3), negative, all_negative,
           huge_values, tiny_values, huge_queries]


@gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,S,splits", [(128, 4096, 1), (64, 1001, 2)])
@pytest.mark.parametrize("change", range(len(CHANGES)))
def test_decode(built, bits, D, S, splits, change):
    c = Cache(bits, 2, S, 2, D, CHANGES[change])
    q, name = _bf16(c.qb), f"fa_decode_int{bits}"
    c.check(*getattr(fa, name)(q, *c.contiguous(), num_splits=splits))
    pool, table, lens = c.paged()
    c.check(*getattr(fa, name + "_paged")(q, *pool, table, lens, num_splits=splits))
    assert fa.fa_device_status() == 0


def shared_zero(c):
    """Zeros on the prefix's first 128 keys and on each sequence's first 64; small values elsewhere."""
    c.scales[1] *= np.float32(1e-4)
    for pg in [*c.pt[:128 // c.P], *c.bt[:, 0][[n > 0 for n in c.lens]]]:
        c.scales[1][pg] = 0
        c.codes[1][pg] = 0


def shared_negative(c):
    n = c.prefix // c.P // 2
    c.scales[1][c.pt[:n]] *= np.float32(2.0 ** -9)
    c.scales[1][c.pt[n:-(-c.prefix // c.P)]] *= -1
    for b, k in enumerate(c.lens):
        if k > c.P:
            c.scales[1][c.bt[b, 1:-(-k // c.P)]] *= np.float32(-100)


SHARED = [(2, 8, 2, 128, 900), (20, 16, 2, 64, 700),                 # through the split kernel
          (16, 192, 24, 128, 700), (20, 192, 24, 64, 700)]           # through the tcgen05 kernel


def shared_case(bits, B, Hq, Hkv, D, prefix, change):
    import torch
    c = Case(bits, B, Hq, Hkv, D, 64, prefix, [(97 * b) % 300 for b in range(B)])
    change(c)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    c.dev.update(q=_bf16(c.qb), vp=t(pack(c.codes[1], bits)), ks=t(c.scales[0].transpose(0, 2, 1)),
                 vs=t(c.scales[1].transpose(0, 2, 1)))
    return c


@gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("B,Hq,Hkv,D,prefix", SHARED)
@pytest.mark.parametrize("change", [shared_zero, shared_negative, huge_values, tiny_values, huge_queries])
def test_shared_decode(built, bits, B, Hq, Hkv, D, prefix, change):
    c = shared_case(bits, B, Hq, Hkv, D, prefix, change)
    c.check(*c.call())
    assert fa.fa_device_status() == 0
