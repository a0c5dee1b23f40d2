"""The Python binding without its C++ marshalling, and the streams that it takes (no GPU)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys, warnings
sys.path.insert(0, {root!r})
import torch
import fp8_block_scaled_bsgemm_b200 as bsg
from fp8_block_scaled_bsgemm_b200 import build

def no_compiler(force=False):
    raise RuntimeError("g++ failed")

if {build_fails}:
    build.build_binding = no_compiler
else:
    sys.modules[bsg.__name__ + "._bsgemm_torch"] = None      # its import fails, as another torch's module does
with warnings.catch_warnings(record=True) as caught:
    warnings.simplefilter("always")
    assert bsg.make_plan(128, 256, 512, 128)["grid"] > 0
    assert bsg.status_string(0)
    assert bsg.lib().bsgemm_version() > 0
    for call in (lambda: bsg.quantize(torch.zeros(16, 16)), lambda: bsg.activation_quantize(torch.zeros(16, 16), "gelu"),
                 lambda: bsg.rms_norm_quantize(torch.zeros(16, 16), torch.ones(16))):
        try:
            call()
        except ValueError:
            continue
        raise AssertionError("a host tensor was taken")
assert bsg._fast is None and bsg._marshal() is None
told = [w for w in caught if "marshalled in Python" in str(w.message)]
assert len(told) == 1, caught
print("ok")
"""


@pytest.mark.parametrize("build_fails", [True, False])
def test_the_python_code_serves_without_the_module(build_fails):
    code = WITHOUT.format(root=ROOT, build_fails=build_fails)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


def test_a_missing_library_is_built_without_the_module(monkeypatch):
    """Building the library asks for nothing of the binding's; the complete build makes both."""
    from fp8_block_scaled_bsgemm_b200 import build
    calls = []
    monkeypatch.setattr(build, "build_binding", lambda force=False: calls.append(force) or "")
    build.build_library()
    assert calls == []
    build.build()
    assert calls == [False]


class Streams:
    """Stand-ins for torch's streams on a machine without a GPU; records what is made current."""

    class Stream:
        def __init__(self, handle, device=None):
            self.cuda_stream, self.device = handle, device

    def __init__(self, monkeypatch, torch):
        self.current = []
        monkeypatch.setattr(torch.cuda, "Stream", self.Stream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", self.Stream)
        monkeypatch.setattr(torch.cuda, "stream", lambda s: self.current.append(s) or s)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


class OnlyAHandle:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_streams_are_taken_by_object_and_by_handle(monkeypatch):
    import torch

    import fp8_block_scaled_bsgemm_b200 as bsg
    streams = Streams(monkeypatch, torch)
    dev = torch.device("cuda", 0)
    own = streams.Stream(0x10, dev)
    bsg._on(dev, own)
    assert streams.current.pop() is own
    for given, handle in ((OnlyAHandle(0x20), 0x20), (0x30, 0x30), (OnlyAHandle(0), 0), (0, 0), (1, 0), (2, 2)):
        bsg._on(dev, given)
        made = streams.current.pop()
        assert (made.cuda_stream, made.device) == (handle, dev)
    assert bsg._on(dev, None) is bsg._HERE_AND_NOW


def test_a_stream_of_another_device_is_refused(monkeypatch):
    import torch

    import fp8_block_scaled_bsgemm_b200 as bsg
    streams = Streams(monkeypatch, torch)
    other = streams.Stream(0x10, torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        bsg._on(torch.device("cuda", 0), other)
    assert streams.current == []
