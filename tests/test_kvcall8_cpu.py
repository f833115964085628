"""The native calls of the 8-bit cache, the rotation and the sampling with stand-ins for tensors
and for the library's entry points: what they check (no GPU needed)."""

import ctypes
import importlib.machinery
import importlib.util
import shutil
import threading
import time

import pytest

from ternary_weight_linear_block_gb300 import build as BUILD
from tests.test_kvcall_cpu import B16, F32, I32, I64, Tensor

ADDRESS = 1 << 20


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
        at = ctypes.cast(getattr(ctypes.CDLL(None), name), ctypes.c_void_p).value
        module.bind(*[at] * 4, I32, I64, F32, lambda: 0)
        module.bind8(*[at] * 4)
        module.bind_tokens(*[at] * 2)
        return module
    return bind_to


def rows(heads, ptr=ADDRESS):
    return Tensor(B16, 3, heads, 64, ptr=ptr)


def rotate_args(ptr=ADDRESS):
    return [0, ptr, B16, 0, 2, 64, 0, rows(4), rows(2), rows(2), Tensor(I64, 3), Tensor(I32, 3, 3), True,
            Tensor(I64, 32), Tensor(I32, 32), False, Tensor(F32, 64), Tensor(F32, 64), F32, 1e-6, rows(4), 0]


def read_args(ptr=ADDRESS):
    return [ptr, 2, 64, 0, Tensor(I64, 3), B16, 0, rows(2), rows(2), 0]


def attention8_args(ptr=ADDRESS):
    return [ADDRESS, B16, 2, 64, 0, rows(4, ptr), Tensor(I32, 2, 4), Tensor(I32, 2), Tensor(I32, 3), 2, Tensor(I64, 3, 1),
            0.125, rows(4), Tensor(F32, 3, 4), ADDRESS, 1 << 20, 0, 0]


def commit8_args(ptr=ADDRESS):
    return [bytes(112), 1, 0, Tensor(I32, 2, 4), Tensor(I32, 2), Tensor(I32, 2, 3), Tensor(I32, 2), Tensor(I32, 2), 0]


def sample_args(ptr=ADDRESS):
    return [Tensor(B16, 3, 50, ptr=ptr), B16, 0, Tensor(F32, 3), Tensor(F32, 3), Tensor(I32, 3), Tensor(F32, 3),
            Tensor(F32, 3), Tensor(I32, 3), 0]


def accept_args(ptr=ADDRESS):
    return [Tensor(I32, 9, ptr=ptr), Tensor(I32, 9), Tensor(I32, 9), Tensor(I32, 3), Tensor(I32, 2, 4), Tensor(I32, 2),
            Tensor(I32, 2), 0]


ALL = [("rotate", rotate_args, 10), ("read", read_args, 3), ("attention8", attention8_args, 7),
       ("commit8", commit8_args, 5), ("sample", sample_args, 7), ("accept", accept_args, 7)]


@pytest.mark.parametrize("name,args,tensors", ALL)
def test_what_is_on_another_device_is_refused(calls, name, args, tensors):
    call = getattr(calls("abs"), name)
    call(*args())
    at = [i for i, x in enumerate(args()) if isinstance(x, Tensor)]
    assert len(at) == tensors
    for i in at:
        a = args()
        a[i].device = 1
        with pytest.raises(ValueError, match="current device"):
            call(*a)


@pytest.mark.parametrize("name,args,tensors", ALL)
def test_types_axes_and_counts_are_checked(calls, name, args, tensors):
    call = getattr(calls("abs"), name)
    at = [i for i, x in enumerate(args()) if isinstance(x, Tensor)]
    for i in at:
        for change in ("dtype", "ndim", "host"):
            a = args()
            if change == "dtype":
                a[i].dtype = "complex64"
            elif change == "ndim":
                a[i].shape += (1, 1)
            else:
                a[i].is_cuda = False
            with pytest.raises(ValueError):
                call(*a)
    with pytest.raises(TypeError):
        call(*args()[:-1])


@pytest.mark.parametrize("name,args,at,shape", [
    ("rotate", rotate_args, 7, (4, 4, 64)), ("rotate", rotate_args, 9, (2, 2, 64)), ("rotate", rotate_args, 10, (2,)),
    ("rotate", rotate_args, 11, (3, 4)), ("rotate", rotate_args, 14, (31,)), ("rotate", rotate_args, 16, (63,)),
    ("rotate", rotate_args, 20, (3, 2, 64)), ("read", read_args, 4, (2,)), ("read", read_args, 8, (4, 2, 64)),
    ("attention8", attention8_args, 5, (3, 3, 64)), ("attention8", attention8_args, 8, (2,)),
    ("commit8", commit8_args, 5, (3, 3)), ("sample", sample_args, 3, (2,)), ("sample", sample_args, 5, (4,)),
    ("sample", sample_args, 8, (4,)), ("accept", accept_args, 1, (8,)), ("accept", accept_args, 4, (3, 4)),
    ("accept", accept_args, 6, (3,))])
def test_shapes_that_do_not_belong_together(calls, name, args, at, shape):
    a = args()
    a[at].shape = shape
    with pytest.raises(ValueError):
        getattr(calls("abs"), name)(*a)


def test_strides(calls):
    module = calls("abs")

    def strided(t, *stride):
        t.stride = lambda: stride
        return t
    a = rotate_args()
    a[8] = strided(rows(2), 400, 64, 2)                 # not dense along a head
    with pytest.raises(ValueError, match="k: expected"):
        module.rotate(*a)
    a = rotate_args()
    a[11] = strided(Tensor(I32, 3, 3), 3, 2)
    with pytest.raises(ValueError, match="positions"):
        module.rotate(*a)
    a = sample_args()
    a[0] = strided(Tensor(B16, 3, 50), 1, 3)
    with pytest.raises(ValueError, match="logits"):
        module.sample(*a)
    a = sample_args()
    a[0] = strided(Tensor(B16, 3, 50), 64, 1)           # rows apart
    module.sample(*a)


@pytest.mark.parametrize("name,args", [("attention8", attention8_args), ("sample", sample_args), ("accept", accept_args)])
def test_other_threads_run_during_a_call(calls, name, args):
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
