"""What is kept per device (csrc/moe_device.cuh), against a CUDA runtime of several devices that only remembers its calls,
and the device that the layer's scored entry point runs on."""
import ctypes as C
import os
import subprocess

import pytest
import torch

import nvfp4_expert_gemms_gb300 as M
from nvfp4_expert_gemms_gb300 import block

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def device(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("device") / "device.so")
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wall", "-o", lib, os.path.join(HERE, "device_host.cpp")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return C.CDLL(lib)


def test_opt_in_on_each_device(device):
    calls, has = C.c_int(), C.c_int()
    opt = lambda dev, de=0, se=0: (device.opt_in(dev, de, se, 200000, C.byref(calls), C.byref(has)), calls.value, has.value)  # noqa: E731
    assert opt(0, se=1) == (1, 1, 0)  # refused: told, and not taken for done
    assert opt(0) == (0, 2, 200000)
    assert opt(0) == (0, 2, 200000)  # once
    assert opt(1) == (0, 3, 200000)  # another device needs its own
    assert opt(0) == opt(1) == (0, 3, 200000)
    assert opt(2, de=100) == (100, 3, 0)  # no current device
    assert opt(70) == (0, 4, 200000) and opt(70) == (0, 5, 200000)  # more devices than are remembered


def test_numbers_of_each_device(device):
    assert [device.number(0, 2), device.number(1, 5), device.number(0, 1), device.number(1, 0), device.number(64, 1)] == [3 - 1, 5, 3, 5, -1]


def test_no_kernel_keeps_its_opt_in_for_the_process():
    """Every opt-in of the sources goes through SmemOptIn, or is made at every launch."""
    import glob
    import re

    sources = [p for p in glob.glob(os.path.join(os.path.dirname(HERE), "nvfp4_expert_gemms_gb300", "csrc", "*.cu*"))
               if not p.endswith("moe_device.cuh")]
    assert sources
    for p in sources:
        text = open(p).read()
        assert "cudaFuncSetAttribute" not in text and not re.search(r"static (std::atomic<)?bool>? (attr|set)\b", text), p


class OnDevice:
    """Stands for a CUDA tensor of device 1 where this process has none."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, torch.device("cuda", 1), True

    def is_contiguous(self):
        return True

    def stride(self, i):
        return 1 if i == len(self.shape) - 1 else self.shape[1]

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 1


def test_scored_layer_runs_on_its_tensors_device(monkeypatch):
    on, now = [], [0]

    class Device:
        def __init__(self, d):
            self.d = d.index

        def __enter__(self):
            self.was, now[0] = now[0], self.d

        def __exit__(self, *e):
            now[0] = self.was

    class Stream:
        cuda_stream = 7

    class Fake:
        def moe_layer_forward_scored(self, *a):
            on.append(now[0])
            return 0

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream)
    monkeypatch.setattr(block, "_f", Fake)
    bf = torch.bfloat16
    M.moe_layer_forward_scored(OnDevice((4, 128), bf), OnDevice((4, 8), bf), M.Router(), M.moe_packed_size("bf16", 8, 128, 128), OnDevice((9,), torch.uint8),
                               2, OnDevice((4, 128), bf), OnDevice((9,), torch.uint8))
    assert on == [1] and now == [0]
