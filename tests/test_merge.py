"""The merge of split partials: few rows of many splits (several in flight, the last ones empty or not a whole
batch), and so many rows that they fill the GPU more than once.  Against the definition in 64 bits, bounds as in
test_value_scales.py."""
import pytest

import tiled_attention_26_b200 as fa
from test_kv_cache import _bf16, built  # noqa: F401
from test_value_scales import Cache

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("bits,B,S,Hkv,D,splits", [
    (8, 1, 9000, 2, 128, 71),   # every split holds keys: 2 batches of 32, one of 7
    (8, 2, 9000, 1, 64, 70),    # 36 of 70 hold keys
    (4, 1, 300, 1, 128, 300),   # 3 of 300
    (8, 1, 1000, 3, 128, 8),    # one whole batch
    (4, 1, 1100, 3, 64, 9),     # one and a single split
    (8, 300, 40, 4, 128, 3),    # 4800 rows: more than fit at once, 1 of 3
    (4, 160, 300, 8, 64, 3),    # 5120 rows, 3 of 3
])
def test_merge(built, bits, B, S, Hkv, D, splits):
    c = Cache(bits, B, S, Hkv, D, lambda c: None)
    q, name = _bf16(c.qb), f"fa_decode_int{bits}"
    c.check(*getattr(fa, name)(q, *c.contiguous(), num_splits=splits))
    pool, table, lens = c.paged()
    c.check(*getattr(fa, name + "_paged")(q, *pool, table, lens, num_splits=splits))
    assert fa.fa_device_status() == 0
