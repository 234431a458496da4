"""Which token rows the cache write may read: rows from cu_tokens[B] on belong to no sequence and need not exist,
so a buffer may end there although num_tokens (an upper bound in a captured step, say) is larger.  The
bound of the kernel's loads is compiled for the host and compared with its definition for every warp of a call."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from tiled_attention_26_b200 import build

PROGRAM = r"""
#include "kvcache.cuh"
extern "C" int rows_to_read(const int32_t* cu, int B, int N, long long tok0, int tokens) {
  fa::KvMap m{};
  m.cu_tokens = cu;
  m.B = B;
  m.N = N;
  return fa::kv_rows_to_read(m, tok0, tokens);
}
"""


@pytest.fixture(scope="module")
def rows_to_read(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    src, out = str(d / "rows.cu"), str(d / "rows.so")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run([build.nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-shared",
                    "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-I", build.CSRC, src, "-o", out], check=True)
    f = ctypes.CDLL(out).rows_to_read
    f.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_longlong, ctypes.c_int]
    return f


@pytest.mark.parametrize("tokens", [4, 8, 32])  # rows of one warp
@pytest.mark.parametrize("N", [1, 31, 32, 33, 100, 1000])
@pytest.mark.parametrize("end", [None, 0, 1, 30, 32, 99, 1000, 1 << 30, -1, -2 ** 31])
def test_rows_up_to_the_last_sequence(rows_to_read, tokens, N, end):
    cu = None if end is None else np.array([0, min(max(end, 0), 7), end], np.int32)
    have = N if end is None else max(0, min(N, end))
    read = []
    for tok0 in range(0, N, tokens):
        n = rows_to_read(cu.ctypes.data if cu is not None else None, 2, N, tok0, tokens)
        assert 0 <= n <= tokens
        read += range(tok0, tok0 + n)
    assert read == list(range(have))


def test_offsets_past_32_bits(rows_to_read):
    top = 2 ** 31 - 1
    cu = np.array([0, top], np.int32)
    assert rows_to_read(cu.ctypes.data, 1, top, top - 5, 32) == 5
    assert rows_to_read(None, 1, top, 2 ** 31 - 1 + 31, 32) == 0
    assert rows_to_read(None, 1, top, 2 ** 32, 32) == 0


def test_the_kernel_is_bound_by_it():
    """Every load of token rows in the write kernel is guarded by that bound."""
    with open(os.path.join(build.CSRC, "kvcache.cuh")) as f:
        kernel = f.read().split("fa_kv_write_kernel(")[1].split("\n}\n")[0]
    assert "const int left = kv_rows_to_read(map, tok0, kTokens);" in kernel
    assert kernel.count("reinterpret_cast<const uint4*>(x") == 1
    assert "if (r < left) {\n        const uint4* src = reinterpret_cast<const uint4*>(x + r * stride);" in kernel
