"""The direct calls for torch tensors (csrc/torch_calls.cpp): other Python threads run while one is inside the
library, and only a file built for the running torch and Python is loaded."""
import ctypes
import subprocess
import threading
import time

import pytest

import tiled_attention_26_b200 as fa
from tiled_attention_26_b200 import build
from test_kv_cache import built  # noqa: F401

gpu = pytest.mark.gpu

SECONDS = 0.2
PROGRAM = """
#include <unistd.h>
static int calls;
long slow(void) { ++calls; usleep(%d); return 0; }
int count(void) { return calls; }
long zero(void) { return 0; }
""" % int(SECONDS * 1e6)


@pytest.fixture
def slow_library(built, tmp_path):
    """The direct calls over functions that launch nothing and take their time on the host."""
    src, out = str(tmp_path / "slow.c"), str(tmp_path / "slow.so")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", src, "-o", out], check=True)
    L = ctypes.CDLL(out)
    calls = fa._direct()
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    try:  # (the last one is the size of a workspace)
        calls.init(*[address(L.slow)] * (len(fa._CALLS) - 1), address(L.zero))
        yield L
    finally:
        fa._direct_calls = None
        fa._direct()


def arguments():
    import torch
    bf = dict(dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.zeros(2, 4, 2, 64, **bf)
    codes = [torch.zeros(2, 4, 2, 64, dtype=torch.int8, device="cuda")] * 2 + [torch.zeros(2, 2, 4, device="cuda")] * 2
    pool = [torch.zeros(5, 16, 2, 64, dtype=torch.int8, device="cuda")] * 2 + [torch.zeros(5, 2, 16, device="cuda")] * 2
    bt = torch.zeros(2, 3, **i32)
    return dict(
        fa_kv_quantize_int8=(k, k), fa_kv_dequantize_int8=(*codes,), fa_kv_append_int8_paged=(k, k, *pool, bt),
        fa_kv_gather_int8_paged=(*pool, bt, 8),
        fa_decode_int8_shared=(torch.zeros(2, 1, 4, 64, **bf), *pool, bt[0], torch.zeros(1, **i32), bt,
                               torch.zeros(2, **i32)))


@gpu
@pytest.mark.parametrize("name", ["fa_kv_quantize_int8", "fa_kv_dequantize_int8", "fa_kv_append_int8_paged",
                                  "fa_kv_gather_int8_paged", "fa_decode_int8_shared"])
def test_other_threads_run_meanwhile(slow_library, name):
    args = arguments()[name]
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.001)

    t = threading.Thread(target=tick)
    t.start()
    try:
        while not ticks:
            time.sleep(0.001)
        start, before = time.monotonic(), slow_library.count()
        getattr(fa, name)(*args)
        end = time.monotonic()
    finally:
        stop.set()
        t.join()
    assert slow_library.count() == before + 1 and end - start >= SECONDS
    # a thread that waits a millisecond at a time: about 200 turns, none while the lock is held
    assert sum(start < x < end for x in ticks) >= 10


class Compiles(Exception):
    pass


@pytest.mark.parametrize("what", ["torch", "python"])
def test_another_torch_or_python_is_another_file(built, monkeypatch, what):
    """After a change of version the old file is neither loaded nor taken for up to date."""
    import torch
    fa._direct()
    here = build.calls_path()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "999.0.0")
    else:
        monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: ".cpython-999-x86_64-linux-gnu.so")
    there = build.calls_path()
    assert there != here and not build.os.path.exists(there)
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        raise Compiles

    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(Compiles):
        build.build_calls()
    assert commands[0][commands[0].index("-o") + 1] == there + ".tmp"
    monkeypatch.setattr(fa, "_direct_calls", None)
    with pytest.raises(RuntimeError, match="build.py"):
        fa._direct()
    monkeypatch.undo()
    assert build.build_calls() == here
    monkeypatch.setattr(fa, "_direct_calls", None)
    assert fa._direct().kv_append is not None
