"""The C interface's mirrors in _lib run on the current device: tensors of another one are
refused there before a launch.  (The calls of api place themselves on their tensors' device.)
Stand-ins for tensors, no GPU."""
import pytest
import torch

FAKE = 0x10000   # never dereferenced


class OnDevice:
    """What the checks ask of a contiguous tensor of another device."""

    def __init__(self, device, shape, dtype):
        self.device_index, self.shape, self.dtype = device, shape, dtype
        self.is_cuda = True

    def get_device(self):
        return self.device_index

    def stride(self):
        out, n = [], 1
        for s in reversed(self.shape):
            out.insert(0, n)
            n *= s
        return tuple(out)

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def element_size(self):
        return 4

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


def test_tensors_of_another_device_than_the_current(monkeypatch):
    from fp8_gemms_b200 import _lib

    launched = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: launched.append(name) or 0
    monkeypatch.setattr(_lib, "lib", Library())
    monkeypatch.setattr(_lib, "_stream", lambda s: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    f32, i64 = torch.float32, torch.int64

    def calls(device):
        def t(*shape, dtype=f32):
            return OnDevice(device, shape, dtype)
        x, w, m, rng, q = t(4, 64), t(64), t(4), t(2, dtype=i64), t(1, 2, 3, 64)
        ws, f = t(4096), t(32, dtype=torch.float64)
        return [lambda: _lib.lm_layernorm_fwd(x, w, w, x, m, m),
                lambda: _lib.lm_layernorm_bwd(x, x, w, m, m, x, w, w, ws),
                lambda: _lib.lm_dropout_add_fwd(x, None, x, 0.1, rng),
                lambda: _lib.lm_dropout_add_bwd(x, x, 0.1, rng),
                lambda: _lib.lm_dropout_add_layernorm_fwd(x, x, w, w, x, x, 0.1, rng),
                lambda: _lib.lm_dropout_add_layernorm_bwd(x, x, x, w, m, m, 0.1, rng, x, x, w, w, ws),
                lambda: _lib.lm_rope([q], [q], f)]
    for call in calls(0):
        call()
    assert len(launched) == 7
    for call in calls(1):
        with pytest.raises(_lib.LmError) as e:
            call()
        assert e.value.status == 1
    assert len(launched) == 7
