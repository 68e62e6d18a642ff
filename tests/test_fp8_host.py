"""What the norm and e4m3 calls of the binding do on the host, watched without a device."""
import contextlib
import threading

import pytest

from trellis_coded_gemv_amd import binding as tg


@pytest.mark.parametrize("stream", [7, None])
def test_experts_are_allocated_on_the_stream_that_fills_them(stream, monkeypatch):
    """Memory that another stream's allocator hands out may still be in that stream's use: from_dense enters the caller's stream before it
    allocates, and quantises on it."""
    torch = pytest.importorskip("torch")
    entered, allocated, filled = [], [], []

    class Weight:                                                   # of the current device, as far as from_dense looks
        shape, device, dtype = (3, 130, 144), torch.device("cpu"), torch.float32

        def dim(self):
            return 3

        def get_device(self):
            return 0

        def __getitem__(self, e):
            return e

    @contextlib.contextmanager
    def enter(at, s):
        entered.append((at, s))
        yield
        entered.pop()

    real = torch.empty

    def empty(*a, **kw):
        allocated.append(list(entered))
        return real(*a, **kw)

    def quantize(x, q, scales, block_rows=1, stream=None):
        filled.append(list(entered) + ([stream] if stream is not None else []))
        assert block_rows == 128 and q.shape == (130, 144) and scales.shape == (2, 2)
    monkeypatch.setattr(tg, "_Entered", enter)
    monkeypatch.setattr(tg, "_common_device", lambda *a: 0)
    monkeypatch.setattr(tg, "fp8_quantize", quantize)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    experts = tg.Fp8Experts.from_dense(Weight(), stream=stream)
    where = [] if stream is None else [(0, stream)]
    assert allocated == [where] * 2 and filled == [where] * 3
    assert experts.q.shape == (3, 130, 144) and experts.scales.shape == (3, 2, 2)


def test_a_second_thread_finds_the_output_types_whole(monkeypatch):
    """rms_norm's table of output types is made by its first call: a call of another thread meanwhile finds none of it or all."""
    torch = pytest.importorskip("torch")
    failures = []

    def call(out_dtype):
        try:
            tg.rms_norm(torch.zeros(2, 8), torch.zeros(8), out_dtype=out_dtype)
        except ValueError as e:                                     # on a host tensor: the device is refused, behind the type
            if "on a GPU" not in str(e):
                failures.append(str(e))

    class Watched(dict):
        def update(self, *a):
            super().update(*a)
            if threading.current_thread() is threading.main_thread():
                for out_dtype in (torch.float32, torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn):
                    t = threading.Thread(target=call, args=(out_dtype,))
                    t.start()
                    t.join()
    monkeypatch.setattr(tg, "_OUT_TYPES", Watched())
    call(torch.float32)
    assert not failures and len(tg._OUT_TYPES) == 5
