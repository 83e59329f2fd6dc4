"""Reading the device error word waits for the given stream alone where nothing could have raised a flag."""

import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def test_read_does_not_wait_for_other_streams():
    """A process without a workspace and without FP8 calls: the read returns while the default stream is busy."""
    code = textwrap.dedent("""
        import time
        import torch
        from bit_quantized_moe_quantize_gb300 import _lib, build
        build.build()
        L = _lib.load()
        import ctypes
        flags = ctypes.c_uint32(7)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        _lib._check(L.ft_moe_read_device_error(side.cuda_stream, ctypes.byref(flags)))     # first-call costs
        done = torch.cuda.Event()
        torch.cuda._sleep(1_000_000_000)          # about half a second of the default stream
        done.record()
        st = L.ft_moe_read_device_error(side.cuda_stream, ctypes.byref(flags))
        busy = not done.query()
        torch.cuda.synchronize()
        print("busy" if busy and st == 0 and flags.value == 0 else f"waited {st} {flags.value}")
    """)
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "busy", (r.stdout, r.stderr[-2000:])
