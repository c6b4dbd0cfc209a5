"""The paged-cache binding's streams and devices (on the CPU, with stand-ins for what needs a GPU)."""
import importlib.util
import types

import pytest

import dequant_gemv_q4g32_amd as qg

torch = pytest.importorskip("torch")


def test_stream_of_another_device_is_refused():
    """A torch stream belongs to a device; on any other than the pool's a call must not run elsewhere."""
    pool = types.SimpleNamespace(device=torch.device("cuda", 0), _index=0)
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=64)
    x = None
    for call in (lambda: qg.kv_append(pool, x, x, x, x, stream=other), lambda: qg.kv_gather(pool, x, x, stream=other),
                 lambda: qg.paged_attention(pool, x, x, x, stream=other), lambda: qg.kv_copy_pages(pool, x, x, stream=other),
                 lambda: qg.kv_fork(pool, x, x, x, x, x, x, stream=other), lambda: qg.kv_free(pool, x, x, x, x, stream=other),
                 lambda: qg.kv_compact(pool, x, x, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()


def _second_copy():
    """The package's module once more, under another name."""
    spec = importlib.util.spec_from_file_location("qg_second_copy", qg.__file__)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_torch_without_the_short_accessors(monkeypatch):
    """The binding uses torch's private accessors of the current device and stream where they are, and
    the public ones where a torch does not have them."""
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    mod = _second_copy()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: types.SimpleNamespace(cuda_stream=1000 + index))
    assert mod._device_now() == 3 and mod._stream_now(2) == 1002


@pytest.mark.gpu
def test_short_and_public_accessors_agree():
    torch.zeros(1, device="cuda")
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            assert qg._device_now() == torch.cuda.current_device()
            assert qg._stream_now(0) == torch.cuda.current_stream(0).cuda_stream == stream.cuda_stream
