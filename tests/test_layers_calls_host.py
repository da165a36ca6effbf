"""What the layer calls do around their launches, with stand-ins for CUDA
tensors and for the library (CPU only): through the extension and through the
interpreter."""
import ctypes
import gc
import subprocess
import threading

import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg
from dense_fp32_tiled_gb300 import build as sg_build
from tests import _stand_ins as S

WITH_SCRATCH = ["linear_forward", "linear_backward", "expert_linear_forward", "expert_linear_backward", "expert_sort"]


@pytest.fixture(scope="module")
def real():
    sg_build.build()
    return sg.load_library()


@pytest.fixture(params=["extension", "interpreter"])
def lib(request, real, monkeypatch, tmp_path):
    return S.install(monkeypatch, real, request.param, str(tmp_path))


def _call(name):
    """A call of each operator that takes scratch; x is not 16-byte aligned, so every product asks for some."""
    x, w, dy = S.Tensor((20, 8), address=(1 << 50) + 2), S.Tensor((8, 16)), S.Tensor((20, 16))
    we, off = S.Tensor((3, 8, 16)), S.Tensor((4,), torch.int32)
    return {"linear_forward": lambda: sg.linear(x, w), "linear_backward": lambda: sg.linear_backward(dy, x, w),
            "expert_linear_forward": lambda: sg.expert_linear(x, we, off),
            "expert_linear_backward": lambda: sg.expert_linear_backward(dy, x, we, off),
            "expert_sort": lambda: sg.expert_sort(S.Tensor((9000, 2), torch.int32), 4)}[name]


@pytest.mark.parametrize("name", WITH_SCRATCH)
def test_scratch_is_its_calls_own(lib, name):
    """A call that begins while another one is still enqueueing (another thread's, on the same
    stream) has other scratch; a call's scratch lives until it has enqueued its kernels, and
    nothing holds it any longer (a captured graph's then belongs to that graph alone)."""
    seen, alive, call = [], [], _call(name)

    def addresses():
        gc.collect()
        return {t().data_ptr() for t in lib.made if t() is not None and t().dtype is torch.uint8}

    def enqueue(*args):  # ..., workspace, its bytes, stream
        seen.append(args[-3])
        if len(seen) == 1:
            call()
        alive.append(args[-3] in addresses())
        return 0

    lib.does[name + "_workspace_size"] = lambda *a: 4096
    lib.does[name] = enqueue
    call()
    assert len(seen) == 2 and seen[0] and seen[1] and seen[0] != seen[1]
    assert alive == [True, True] and not addresses()


WAITS = r"""
#include <unistd.h>
int flag;
int wait_for_flag() {
    for (int i = 0; i < 3000 && !*(volatile int *)&flag; ++i) usleep(1000);
    return flag ? 0 : -6;
}
"""


@pytest.mark.parametrize("name", WITH_SCRATCH + ["expert_gather", "expert_combine", "expert_combine_backward"])
def test_other_threads_run_while_a_launch_waits(real, monkeypatch, tmp_path, name):
    """The library's functions may wait for room in a stream's queue, and what runs there may
    need the interpreter: here another thread sets the flag that the function waits for."""
    (tmp_path / "waits.c").write_text(WAITS)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(tmp_path / "waits.so"), str(tmp_path / "waits.c")], check=True)
    waits = ctypes.CDLL(str(tmp_path / "waits.so"))
    S.install(monkeypatch, real, "extension", str(tmp_path),
              {name: ctypes.cast(waits.wait_for_flag, ctypes.c_void_p).value})
    calls = {"expert_gather": lambda: sg.expert_gather(S.Tensor((5, 8)), S.Tensor((5, 2), torch.int32), S.Tensor((3,), torch.int32)),
             "expert_combine": lambda: sg.expert_combine(S.Tensor((10, 8)), S.Tensor((5, 2), torch.int32)),
             "expert_combine_backward": lambda: sg.expert_combine_backward(
                 S.Tensor((5, 8)), S.Tensor((10, 8)), S.Tensor((5, 2), torch.int32), None, S.Tensor((3,), torch.int32))}
    flag = ctypes.c_int.in_dll(waits, "flag")
    setter = threading.Timer(0.05, lambda: setattr(flag, "value", 1))
    setter.start()
    (calls.get(name) or _call(name))()  # raises SgemmError if the wait ran out
    setter.join()


def _given(stream):
    """Every operator's call with a stream."""
    x, w, dy = S.Tensor((20, 8)), S.Tensor((8, 16)), S.Tensor((20, 16))
    we, off, rows = S.Tensor((3, 8, 16)), S.Tensor((4,), torch.int32), S.Tensor((10, 2), torch.int32)
    return {"linear": lambda: sg.linear(x, w, stream=stream), "linear_backward": lambda: sg.linear_backward(dy, x, w, stream=stream),
            "expert_linear": lambda: sg.expert_linear(x, we, off, stream=stream),
            "expert_linear_backward": lambda: sg.expert_linear_backward(dy, x, we, off, stream=stream),
            "expert_sort": lambda: sg.expert_sort(rows, 3, stream=stream),
            "expert_gather": lambda: sg.expert_gather(S.Tensor((10, 8)), rows, off, stream=stream),
            "expert_combine": lambda: sg.expert_combine(x, rows, stream=stream),
            "expert_gather_backward": lambda: sg.expert_gather_backward(x, rows, stream=stream),
            "expert_combine_backward": lambda: sg.expert_combine_backward(S.Tensor((10, 8)), x, rows, None, off, stream=stream)}


@pytest.mark.parametrize("name", _given(None))
def test_stream_of_another_device_is_refused(lib, name):
    with pytest.raises(ValueError, match="stream"):
        _given(S.Stream(1))[name]()
    assert not lib.entered and lib.calls == 0
    own = S.Stream(0)
    _given(own)[name]()
    assert lib.entered == [own] and lib.calls == 1


BIG = 2 ** 32 + 16  # 16 in 32 bits


@pytest.mark.parametrize("name,call", [
    ("rows of x", lambda: sg.linear(S.Tensor((BIG, 8)), S.Tensor((8, 16)))),
    ("inputs", lambda: sg.linear(S.Tensor((4, BIG)), S.Tensor((BIG, 16)))),
    ("outputs", lambda: sg.linear(S.Tensor((4, 8)), S.Tensor((8, BIG)))),
    ("rows of experts", lambda: sg.expert_linear(S.Tensor((BIG, 8)), S.Tensor((2, 8, 16)), S.Tensor((3,), torch.int32))),
    ("rows of dy", lambda: sg.linear_backward(S.Tensor((BIG, 16)), S.Tensor((BIG, 8)), S.Tensor((8, 16)))),
    ("tokens sorted", lambda: sg.expert_sort(S.Tensor((BIG, 2), torch.int32), 4)),
    ("experts", lambda: sg.expert_sort(S.Tensor((4, 2), torch.int32), BIG)),
    ("less than no experts", lambda: sg.expert_sort(S.Tensor((4, 2), torch.int32), 16 - 2 ** 32)),
    ("choices", lambda: sg.expert_sort(S.Tensor((4, BIG), torch.int32), 4)),
    ("gathered", lambda: sg.expert_gather(S.Tensor((BIG, 8)), S.Tensor((BIG, 2), torch.int32), S.Tensor((4,), torch.int32))),
    ("width", lambda: sg.expert_gather(S.Tensor((4, BIG)), S.Tensor((4, 2), torch.int32), S.Tensor((4,), torch.int32))),
    ("combined", lambda: sg.expert_combine(S.Tensor((BIG, 8)), S.Tensor((BIG, 1), torch.int32))),
    ("spread", lambda: sg.expert_combine_backward(S.Tensor((BIG, 8)), S.Tensor((BIG, 8)), S.Tensor((BIG, 1), torch.int32), None,
                                                  S.Tensor((4,), torch.int32))),
])
def test_sizes_past_32_bits_are_refused(lib, name, call):
    with pytest.raises(ValueError):
        call()
    assert lib.calls == 0


def test_experts_without_offsets_are_refused(lib):
    x, w, dy, rows = S.Tensor((20, 8)), S.Tensor((8, 16)), S.Tensor((20, 16)), S.Tensor((10, 2), torch.int32)
    for call in (lambda: sg.expert_linear(x, w, None), lambda: sg.expert_linear_backward(dy, x, w, None),
                 lambda: sg.expert_linear(x, w, None, stream=S.Stream()), lambda: sg.expert_linear_backward(dy, x, w, None, stream=S.Stream())):
        with pytest.raises(ValueError, match="offsets"):
            call()
    assert lib.calls == 0
