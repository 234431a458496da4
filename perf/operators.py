"""Cases that time the quantised KV cache: writing it, reading it back, and decoding over it for a batch
that shares a prefix.

``run`` computes each case in its plain form (elementary torch operations in 32 bits) or, where ``own``
is true, through the package's entry points.  A cache row is one token of one KV head: ``D`` codes and one
fp32 scale, ``value = code * scale``, ``scale = max|x| / m`` with m = 127 (INT8) or 7 (INT4).
"""
import math
import random

import torch

own = False

# --------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------


def listed():
    return [
        # One sequence, one new token: the write of a single-user decode step (latency).
        dict(name="append_token_b1", kind="append", bits=8, B=1, Hkv=8, D=128, page=64, tokens=1, ragged=False),
        # A batch of ragged prompts written into its pages after the prefill.
        dict(name="append_prompts_int8", kind="append", bits=8, B=16, Hkv=8, D=128, page=64, tokens=4096, ragged=True),
        # The same into an INT4 cache of a 64-dim model with odd sizes and small pages.
        dict(name="append_prompts_int4_d64", kind="append", bits=4, B=37, Hkv=5, D=64, page=16, tokens=2999, ragged=True),
        # A whole contiguous cache quantised at once (a quarter of the INT8 decode workload's cache).
        dict(name="quantize_cache_int8", kind="quantize", bits=8, B=4, Hkv=8, D=128, tokens=32768),
        # A context read back for the next chunk of a long prompt.
        dict(name="gather_context_int8", kind="gather", bits=8, B=1, Hkv=8, D=128, page=64, tokens=131072, ragged=False),
        # Ragged INT4 contexts of a batch.
        dict(name="gather_contexts_int4", kind="gather", bits=4, B=16, Hkv=8, D=128, page=64, tokens=2048, ragged=True),
        # Two answers sampled from one short prompt: the smallest shared decode (latency).
        dict(name="shared_b2_prefix512", kind="shared", bits=8, B=2, Hq=32, Hkv=8, D=128, page=64, prefix=512, suffix=48),
        # A serving step: a system prompt of 4096 tokens, 32 users with up to 1024 tokens of their own;
        # the step's token is appended first.
        dict(name="step_b32_prefix4096", kind="step", bits=8, B=32, Hq=32, Hkv=8, D=128, page=64, prefix=4096, suffix=1024),
        # A long document shared by 64 questions.
        dict(name="shared_b64_prefix32768", kind="shared", bits=8, B=64, Hq=32, Hkv=8, D=128, page=64, prefix=32768, suffix=512),
        # Few sequences over a very long document (bound by reading it).
        dict(name="shared_b4_prefix131072", kind="shared", bits=8, B=4, Hq=32, Hkv=8, D=128, page=128, prefix=131072, suffix=200),
        # MQA with 232 heads of 64 dims: 2784 query rows over one KV head.
        dict(name="shared_mqa_d64_b12", kind="shared", bits=8, B=12, Hq=232, Hkv=1, D=64, page=64, prefix=8192, suffix=256),
        # INT4, odd group of 7 heads, odd batch, a prefix that ends inside a 16-token page.
        dict(name="shared_int4_b13_prefix5003", kind="shared", bits=4, B=13, Hq=28, Hkv=4, D=128, page=16, prefix=5003, suffix=777),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "quantize", "gather", "shared", "shared", "step"])
    c = dict(kind=kind, bits=rng.choice([8, 4]), D=rng.choice([128, 64]))
    if kind == "quantize":
        c.update(B=_log(rng, 1, 8), Hkv=rng.choice([1, 2, 4, 5, 8]))
        c["tokens"] = _log(rng, 1, 2 ** 17 // c["B"])
        return c
    c["page"] = rng.choice([16, 32, 64, 128, 256])
    if kind in ("append", "gather"):
        c.update(B=_log(rng, 1, 64), Hkv=rng.choice([1, 2, 4, 5, 8]), ragged=rng.random() < 0.75)
        c["tokens"] = _log(rng, 1, 2 ** 17 // c["B"])
        return c
    c["Hkv"] = rng.choice([1, 2, 4, 8])
    c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 7, 8, 16])
    c["B"] = _log(rng, 1, 64)
    c["suffix"] = _log(rng, 1, 1024)
    c["prefix"] = _log(rng, 64, min(131072, 2 ** 26 // (c["B"] * c["Hq"])))
    return c


def _lengths(c, most, ragged=True):
    """The batch's lengths, 1 .. most, from the case alone: spread evenly and out of order."""
    if not ragged:
        return [most] * c["B"]
    return [max(1, math.ceil(most * ((b + 1) * 0.6180339887 % 1.0))) for b in range(c["B"])]


def work(c):
    row = c["Hkv"] * (c["D"] * c["bits"] // 8 + 4)  # bytes of one token's K (or V) codes and scales
    if c["kind"] == "quantize":
        n = c["B"] * c["tokens"]
    elif c["kind"] in ("append", "gather"):
        n = sum(_lengths(c, c["tokens"], c["ragged"]))
    else:
        lens = _lengths(c, c["suffix"])
        pairs = c["B"] * c["prefix"] + sum(lens)
        io = c["B"] * c["Hq"] * (4 * c["D"] + 4)
        if c["kind"] == "step":
            io += 2 * c["B"] * (2 * c["Hkv"] * c["D"] + row)
        return {"bytes": 2 * row * (c["prefix"] + sum(lens)) + io, "flops": 4 * c["D"] * c["Hq"] * pairs}
    # write and read back what was written: bf16 in, cache out, cache in, bf16 out
    passes = 1 if c["kind"] == "gather" else 2
    n_bytes = passes * 2 * n * (2 * c["Hkv"] * c["D"] + row)
    return {"bytes": n_bytes, "flops": 2 * passes * n * c["Hkv"] * c["D"]}


# --------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------


def _levels(bits):
    return 127.0 if bits == 8 else 7.0


def _quantize(x, bits):
    """bf16 [..., D] -> whole codes and scales [...], both fp32."""
    m = _levels(bits)
    x = x.float()
    # rounded once: a last-bit error of the scale moves the values that lie halfway between two codes
    scale = (x.abs().amax(-1).double() / m).float()
    codes = torch.round(x / scale.clamp_min(1e-38).unsqueeze(-1)).clamp(-m, m)
    return codes, scale


def _pack(codes, bits):
    """Whole codes as they are stored: int8, or two 4-bit two's-complement codes per byte (even dim low)."""
    if bits == 8:
        return codes.to(torch.int8)
    c = codes.to(torch.int32) & 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def _unpack(stored, bits):
    if bits == 8:
        return stored.float()
    c = stored.to(torch.int32)
    c = torch.stack((c & 15, c >> 4), -1).flatten(-2)
    return (c - 16 * (c > 7)).float()


def _kv(gen, shape):
    """Keys or values of a trained model's spread: each token and each channel has a size of its own."""
    x = torch.randn(shape, generator=gen, device="cuda")
    token = torch.exp(0.3 * torch.randn(shape[:-1], generator=gen, device="cuda"))
    channel = torch.exp(0.3 * torch.randn(shape[-2:], generator=gen, device="cuda"))
    return (x.mul_(token.unsqueeze(-1)).mul_(channel)).bfloat16()


def _pool(gen, c, pages):
    """A pool of pages that already hold a cache: codes [pages, P, Hkv, row], scales [pages, Hkv, P]."""
    pool = []
    for _ in range(2):
        codes, scale = _quantize(_kv(gen, (pages, c["page"], c["Hkv"], c["D"])), c["bits"])
        pool.append((_pack(codes, c["bits"]), scale.transpose(1, 2).contiguous()))
    (kp, ks), (vp, vs) = pool
    return dict(kp=kp, vp=vp, ks=ks, vs=vs)


def _table(order, first, counts, width):
    """Rows of page ids: row b takes the next counts[b] pages of ``order`` from place ``first`` on."""
    t = torch.zeros((len(counts), width), dtype=torch.int32)
    for b, n in enumerate(counts):
        t[b, :n] = order[first:first + n]
        first += n
    return t.cuda()


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    order_gen = torch.Generator().manual_seed(int(seed))
    s = dict(c)
    if c["kind"] == "quantize":
        shape = (c["B"], c["tokens"], c["Hkv"], c["D"])
        s.update(k=_kv(gen, shape), v=_kv(gen, shape))
        return s
    up = lambda n: -(-n // c["page"])  # noqa: E731
    if c["kind"] in ("append", "gather"):
        lens = _lengths(c, c["tokens"], c["ragged"])
        # appended tokens follow a history of their own; a context is read from its start
        starts = [(37 * b) % 200 if c["kind"] == "append" else 0 for b in range(c["B"])]
        counts = [up(a + n) for a, n in zip(starts, lens)]
        order = torch.randperm(sum(counts) + 3, generator=order_gen, dtype=torch.int32)
        s.update(_pool(gen, c, sum(counts) + 3))
        s["table"] = _table(order, 0, counts, max(counts))
        s["starts"] = torch.tensor(starts, dtype=torch.int32).cuda()
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["n"] = cu[-1]
        s["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
        if c["kind"] == "append":
            s.update(k=_kv(gen, (s["n"], c["Hkv"], c["D"])), v=_kv(gen, (s["n"], c["Hkv"], c["D"])))
        return s
    lens = _lengths(c, c["suffix"])
    shared, counts = up(c["prefix"]), [up(n) for n in lens]
    pages = shared + sum(counts) + 3
    order = torch.randperm(pages, generator=order_gen, dtype=torch.int32)
    s.update(_pool(gen, c, pages))
    s["prefix_table"] = order[:shared].cuda()
    s["prefix_len"] = torch.tensor([c["prefix"]], dtype=torch.int32).cuda()
    s["table"] = _table(order, shared, counts, max(counts))
    s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    s["longest"] = max(lens)
    s["q"] = torch.randn((c["B"], 1, c["Hq"], c["D"]), generator=gen, device="cuda").bfloat16()
    if c["kind"] == "step":  # the step's token is the last of each sequence
        s["starts"] = s["lens"] - 1
        s.update(k=_kv(gen, (c["B"], 1, c["Hkv"], c["D"])), v=_kv(gen, (c["B"], 1, c["Hkv"], c["D"])))
    return s


# --------------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------------


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import tiled_attention_26_b200 as fa
    name = "int%d" % s["bits"]
    if s["kind"] == "quantize":
        cache = getattr(fa, "fa_kv_quantize_" + name)(s["k"], s["v"])
        return *getattr(fa, "fa_kv_dequantize_" + name)(*cache), *cache[2:]
    pool = s["kp"], s["vp"], s["ks"], s["vs"]
    if s["kind"] in ("append", "step"):
        cu = s.get("cu")
        getattr(fa, "fa_kv_append_%s_paged" % name)(s["k"], s["v"], *pool, s["table"], s["starts"], cu)
    if s["kind"] in ("append", "gather"):
        out = getattr(fa, "fa_kv_gather_%s_paged" % name)(*pool, s["table"], s["n"], s["starts"], s["cu"])
        return (*out, s["ks"], s["vs"]) if s["kind"] == "append" else out
    return getattr(fa, "fa_decode_%s_shared" % name)(s["q"], *pool, s["prefix_table"], s["prefix_len"], s["table"],
                                                     s["lens"])


def _run_plain(s):
    bits = s["bits"]
    if s["kind"] == "quantize":
        cache = []
        for x in (s["k"], s["v"]):
            codes, scale = _quantize(x, bits)
            cache.append((_pack(codes, bits), scale.transpose(1, 2).contiguous()))
        return (*((_unpack(codes, bits) * scale.transpose(1, 2).unsqueeze(-1)).bfloat16() for codes, scale in cache),
                *(scale for _, scale in cache))
    if s["kind"] == "step":
        _write(s, s["k"].flatten(0, 1), s["v"].flatten(0, 1), *_places(s, torch.arange(s["B"], device="cuda"), s["starts"]))
    if s["kind"] in ("append", "gather"):
        token = torch.arange(s["n"], device="cuda")
        seq = torch.searchsorted(s["cu"], token, right=True) - 1
        page, row = _places(s, seq, s["starts"][seq] + token - s["cu"][seq])
        if s["kind"] == "append":
            _write(s, s["k"], s["v"], page, row)
        out = tuple((_unpack(codes[page, row], bits) * scale[page, :, row].unsqueeze(-1)).bfloat16()
                    for codes, scale in ((s["kp"], s["ks"]), (s["vp"], s["vs"])))
        return (*out, s["ks"], s["vs"]) if s["kind"] == "append" else out
    return _decode_plain(s)


def _places(s, seq, position):
    """Page and row of position ``position`` of sequence ``seq``."""
    position = position.long()
    return s["table"][seq, position // s["page"]].long(), position % s["page"]


def _write(s, k, v, page, row):
    for x, codes, scale in ((k, s["kp"], s["ks"]), (v, s["vp"], s["vs"])):
        c, a = _quantize(x, s["bits"])
        codes[page, row] = _pack(c, s["bits"])
        scale[page, :, row] = a


def _decode_plain(s):
    B, Hq, Hkv, D, bits = s["B"], s["Hq"], s["Hkv"], s["D"], s["bits"]
    G = Hq // Hkv
    # [B, Hkv, G, D]: query head h reads KV head h // G
    q = s["q"].float().view(B, Hkv, G, D) / math.sqrt(D)

    def rows(codes, scale, page, row):  # [..., Hkv, D]
        return _unpack(codes[page, row], bits) * scale[page, :, row].unsqueeze(-1)

    j = torch.arange(s["prefix"], device="cuda")
    page, row = s["prefix_table"][j // s["page"]].long(), j % s["page"]
    kp, vp = rows(s["kp"], s["ks"], page, row), rows(s["vp"], s["vs"], page, row)  # [Lp, Hkv, D]
    shared_rows = q.transpose(0, 1).reshape(Hkv, B * G, D)
    xp = shared_rows @ kp.permute(1, 2, 0)  # [Hkv, B * G, Lp]

    seq = torch.arange(B, device="cuda").unsqueeze(1)
    j = torch.arange(s["longest"], device="cuda").unsqueeze(0)
    page, row = _places(s, seq, j)
    ko, vo = rows(s["kp"], s["ks"], page, row), rows(s["vp"], s["vs"], page, row)  # [B, Ls, Hkv, D]
    xo = q @ ko.permute(0, 2, 3, 1)  # [B, Hkv, G, Ls]
    xo = xo.masked_fill((j >= s["lens"].unsqueeze(1))[:, None, None, :], -math.inf)

    top_p = xp.amax(-1, keepdim=True)
    top_o = xo.amax(-1, keepdim=True)
    top = torch.maximum(top_p.view(Hkv, B, G, 1).transpose(0, 1), top_o)  # [B, Hkv, G, 1]
    pp = torch.exp(xp - top.transpose(0, 1).reshape(Hkv, B * G, 1))
    po = torch.exp(xo - top)
    total = pp.sum(-1).view(Hkv, B, G).transpose(0, 1) + po.sum(-1)  # [B, Hkv, G]
    o = (pp @ vp.transpose(0, 1)).view(Hkv, B, G, D).transpose(0, 1) + po @ vo.transpose(1, 2)
    o = (o / total.unsqueeze(-1)).reshape(B, 1, Hq, D).bfloat16()
    return o, (top.squeeze(-1) + total.log()).reshape(B, Hq)


# --------------------------------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------------------------------


def exact(c, seed):
    s = prepare(c, seed)
    m = 127 if c["bits"] == 8 else 7
    f64 = torch.float64

    def scale_of(x):
        return (x.to(f64).abs().max(-1, keepdim=True).values / m).to(torch.float32).to(f64)

    def stored(x):
        """The value each element of x is stored as: its scale and its quotient are 32-bit numbers."""
        a = scale_of(x)
        n = (x.to(f64) / torch.where(a > 0, a, 1.0)).to(torch.float32).to(f64)
        return n.round().clamp(-m, m) * a

    def cached(which, page, row):
        """Cache rows as values: [..., Hkv, D]."""
        codes, scale = s[which + "p"][page, row], s[which + "s"][page, :, row]
        if c["bits"] == 4:
            low, high = codes.to(torch.int64) % 16, codes.to(torch.int64) // 16
            codes = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.int64, device="cuda")
            codes[..., 0::2], codes[..., 1::2] = low, high
            codes[codes >= 8] -= 16
        return codes.to(f64) * scale.to(f64).unsqueeze(-1)

    if c["kind"] == "quantize":
        return (stored(s["k"]), stored(s["v"]), scale_of(s["k"])[..., 0].transpose(1, 2),
                scale_of(s["v"])[..., 0].transpose(1, 2))
    if c["kind"] == "append":
        scales = [s["ks"].to(f64), s["vs"].to(f64)]
        for b, n in enumerate(_lengths(c, c["tokens"], c["ragged"])):
            at = torch.arange(n, device="cuda") + int(s["starts"][b])
            page, row, first = s["table"][b][at // c["page"]].long(), at % c["page"], int(s["cu"][b])
            for kept, x in zip(scales, (s["k"], s["v"])):
                kept[page, :, row] = scale_of(x[first:first + n])[..., 0]
        return stored(s["k"]), stored(s["v"]), *scales
    if c["kind"] == "gather":
        out = ([], [])
        for b, n in enumerate(_lengths(c, c["tokens"], c["ragged"])):
            at = torch.arange(n, device="cuda") + int(s["starts"][b])
            page, row = s["table"][b][at // c["page"]].long(), at % c["page"]
            out[0].append(cached("k", page, row))
            out[1].append(cached("v", page, row))
        return torch.cat(out[0]), torch.cat(out[1])
    G, lens = c["Hq"] // c["Hkv"], _lengths(c, c["suffix"])
    new = (stored(s["k"]), stored(s["v"])) if c["kind"] == "step" else None
    at = torch.arange(c["prefix"], device="cuda")
    page, row = s["prefix_table"][at // c["page"]].long(), at % c["page"]
    prefix = [cached(w, page, row) for w in "kv"]  # [Lp, Hkv, D]
    o = torch.empty((c["B"], 1, c["Hq"], c["D"]), dtype=f64, device="cuda")
    lse = torch.empty((c["B"], c["Hq"]), dtype=f64, device="cuda")
    for b, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        page, row = s["table"][b][at // c["page"]].long(), at % c["page"]
        tail = [cached(w, page, row) for w in "kv"]
        if new:
            for t, x in zip(tail, new):
                t[n - 1] = x[b, 0]
        q = s["q"][b, 0].to(f64).view(c["Hkv"], G, c["D"])
        x = torch.cat([torch.einsum("hgd,jhd->hgj", q, t) for t in (prefix[0], tail[0])], -1) / math.sqrt(c["D"])
        total = torch.logsumexp(x, -1)
        p = torch.exp(x - total.unsqueeze(-1))
        o[b, 0] = sum(torch.einsum("hgj,jhd->hgd", w, t) for w, t in
                      zip(p.split([c["prefix"], n], -1), (prefix[1], tail[1]))).reshape(c["Hq"], c["D"])
        lse[b] = total.reshape(-1)
    return o, lse
