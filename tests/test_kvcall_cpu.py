"""kv.py's native calls with stand-ins for the tensors and for the library's entry points: what
they check and that they let other threads run (no GPU needed)."""

import ctypes
import importlib.machinery
import importlib.util
import os
import shutil
import threading
import time

import pytest

from ternary_weight_linear_block_gb300 import build as BUILD

I32, I64, F32, B16 = "int32", "int64", "float32", "bfloat16"


class Tensor:
    """What the calls read of a tensor."""

    def __init__(self, dtype, *shape, ptr=1 << 20):
        self.dtype, self.shape, self.ptr = dtype, tuple(shape), ptr
        self.is_cuda, self.device = True, 0

    def get_device(self):
        return self.device

    def stride(self):
        out, step = [], 1
        for n in reversed(self.shape):
            out.append(step)
            step *= n
        return tuple(reversed(out))

    def data_ptr(self):
        return self.ptr


@pytest.fixture
def calls(tmp_path):
    """A copy of the module of its own, with every entry point replaced by ``bind_to``."""
    BUILD.ensure_built()
    path = str(tmp_path / "_kvcall.so")
    shutil.copy(BUILD.EXT, path)
    spec = importlib.util.spec_from_file_location(
        "_kvcall", path, loader=importlib.machinery.ExtensionFileLoader("_kvcall", path))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)

    def bind_to(name):
        module.bind(*[ctypes.cast(getattr(ctypes.CDLL(None), name), ctypes.c_void_p).value] * 4, I32, I64, F32,
                    lambda: 0)
        return module
    return bind_to


def plan_args(ptr=1 << 20):
    """Two requests; ``ptr`` is the first argument that the entry point gets."""
    return [Tensor(I32, 2, ptr=ptr), Tensor(I32, 2), Tensor(I32, 2, 4), Tensor(I32, 5), None, 16, 3,
            Tensor(I32, 3), Tensor(I64, 3), Tensor(I32, 3), Tensor(I32, 3), Tensor(I32, 4), None, None, 0]


def write_args(ptr=1 << 20):
    return [ptr, B16, 2, 64, 0, Tensor(B16, 3, 2, 64), Tensor(B16, 3, 2, 64), Tensor(I64, 3), 0]


def commit_args():
    return [bytes(80), 1, 0, Tensor(I32, 2, 4), Tensor(I32, 2), Tensor(I32, 2, 3), Tensor(I32, 2), Tensor(I32, 2), 0]


def attention_args(ptr=1 << 20):
    return [1 << 20, B16, 2, 64, 0, Tensor(B16, 3, 4, 64, ptr=ptr), Tensor(I32, 2, 4), Tensor(I32, 2), Tensor(I32, 3), 2,
            Tensor(I64, 3, 1), 0.125, Tensor(B16, 3, 4, 64), Tensor(F32, 3, 4), 1 << 20, 1 << 20, 0]


@pytest.mark.parametrize("name,args", [("plan", plan_args), ("write", write_args), ("attention", attention_args)])
def test_other_threads_run_during_a_call(calls, name, args):
    """A launch waits where the queue is full, e.g. behind a host callback that needs the interpreter."""
    module, ticks, stop = calls("usleep"), [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.005)
    thread = threading.Thread(target=tick)
    thread.start()
    try:
        first = time.monotonic()
        assert getattr(module, name)(*args(ptr=300000)) == 0       # usleep(300000), whatever else it is given
        last = time.monotonic()
    finally:
        stop.set()
        thread.join()
    assert last - first >= 0.3 and sum(first + 0.02 < t < last - 0.02 for t in ticks) >= 5


@pytest.mark.parametrize("name,args", [("plan", plan_args), ("write", write_args), ("attention", attention_args),
                                       ("commit", commit_args)])
def test_what_is_on_another_device_is_refused(calls, name, args):
    """Every tensor and the cache; the entry point (abs, which does nothing) is reached without one."""
    call = getattr(calls("abs"), name)

    def given():
        a = args()
        if name == "plan":
            a[4], a[12], a[13] = Tensor(I32, 1), Tensor(I32, 2), Tensor(I32, 2)
        return a
    call(*given())
    at = [i for i, x in enumerate(given()) if isinstance(x, Tensor)]
    assert len(at) == {"plan": 12, "write": 3, "attention": 7, "commit": 5}[name]
    for i in at:
        a = given()
        a[i].device = 1
        with pytest.raises(ValueError, match="current device"):
            call(*a)
    if name != "plan":
        a = given()
        a[2 if name == "commit" else 4] = 1
        with pytest.raises(ValueError, match="current device"):
            call(*a)
