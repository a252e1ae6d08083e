"""The compiled binding lets other Python threads run while the library works on a call (no GPU: the entry point that it
is bound to is a C function that sleeps)."""
import ctypes
import importlib.util
import shutil
import subprocess
import threading
import time

import pytest
import torch  # noqa: F401  (the extension's symbols)

from ragged_grouped_gemm_device_gb300 import _lib, build

STUB = r"""
#include <unistd.h>
int slow() { usleep(600000); return 0; }
"""


class Stream:
    cuda_stream = 0


def test_other_threads_run_during_a_call(tmp_path):
    path = build.build_binding()
    if path is None:
        pytest.skip("no compiler or headers for the extension")
    (tmp_path / "stub.c").write_text(STUB)
    subprocess.run([shutil.which("gcc") or "cc", "-shared", "-fPIC", str(tmp_path / "stub.c"), "-o",
                    str(tmp_path / "stub.so")], check=True)
    stub = ctypes.CDLL(str(tmp_path / "stub.so"))
    # a copy of its own: the package's extension stays bound to the library
    shutil.copy(path, tmp_path / "_binding.so")
    spec = importlib.util.spec_from_file_location("_binding", tmp_path / "_binding.so")
    binding = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(binding)
    slow = ctypes.cast(stub.slow, ctypes.c_void_p).value
    binding.bind({n: slow for n in _lib.COMPILED + ("moe_workspace_bytes",)}, _lib._check)
    call = threading.Thread(target=lambda: binding.moe_route_offsets(*[None] * 1, 0, 1, 1, *[None] * 5, stream=Stream()))
    call.start()
    beats, start = 0, time.monotonic()
    while call.is_alive() and time.monotonic() - start < 20:
        time.sleep(0.01)
        beats += 1
    call.join()
    assert time.monotonic() - start >= 0.5  # the call did take its time
    assert beats >= 10  # with the lock held: one or two
