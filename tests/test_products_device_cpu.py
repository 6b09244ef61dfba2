"""The 4-bit products' tensors have to be on their handle's device: a kernel that reads another's memory faults.

No GPU here, so the tensors only say where they are, and the library is a stub that must not be reached."""
import types

import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P

BF16, U8 = torch.bfloat16, torch.uint8


class Placed:
    """A CPU tensor that says it is on cuda:`device`."""

    def __init__(self, t, device):
        self._t, self._device = t, device

    def __getattr__(self, name):
        return getattr(self._t, name)

    @property
    def is_cuda(self):
        return self._device >= 0

    @property
    def device(self):
        return torch.device("cuda", self._device) if self._device >= 0 else torch.device("cpu")

    def get_device(self):
        return self._device


def _handle(cls, reached, **fields):
    h = object.__new__(cls)
    for k, v in fields.items():
        setattr(h, k, v)

    def call(*a):
        reached.append(a)
        return 0

    names = ("nvfp4_grouped_pack", "nvfp4_grouped_forward", "nvfp4_grouped_backward", "nvfp4_int4_pack",
             "nvfp4_int4_forward", "nvfp4_moe_destroy")
    h.lib, h.h, h.device, h._act, h._out = types.SimpleNamespace(**{n: call for n in names}), None, 1, BF16, BF16
    h._current_stream = lambda device: 0
    return h


STREAM = types.SimpleNamespace(cuda_stream=0)


def _calls(h, places):
    """(name, a call whose tensors are in these places) of a handle on cuda:1."""
    z = lambda i, shape, dt: Placed(torch.zeros(shape, dtype=dt), places[i])
    if isinstance(h, P.Grouped):
        yield lambda: h.nvfp4_grouped_pack(z(0, (2, 16, 64), U8), z(1, (2, 16, 8), U8), z(2, (2,), torch.float32), STREAM)
        yield lambda: h.nvfp4_grouped_forward(z(0, (4, 128), BF16), z(1, (3,), torch.int32), z(2, (4, 16), BF16))
        yield lambda: h.nvfp4_grouped_backward(z(0, (4, 16), BF16), z(1, (3,), torch.int32), z(2, (4, 128), BF16))
    else:
        yield lambda: h.nvfp4_int4_pack(z(0, (16, 64), U8), z(1, (16, 2), BF16), z(2, (16, 2), U8), STREAM)
        yield lambda: h.nvfp4_int4_forward(z(0, (4, 128), BF16), z(1, (4, 16), BF16))


@pytest.mark.parametrize("cls,fields", [(P.Grouped, dict(E=2, N=16, K=128, _int32=torch.int32)),
                                        (P.Int4Linear, dict(N=16, K=128, group=64))])
def test_tensors_on_another_device_are_refused(cls, fields):
    reached = []
    h = _handle(cls, reached, **fields)
    for call in _calls(h, (1, 1, 1)):          # all where they belong: the library is called
        call()
    assert len(reached) == len(list(_calls(h, (1, 1, 1))))
    del reached[:]
    for other in (0, -1):                      # another GPU, the CPU
        for i in range(3):
            places = [1, 1, 1]
            places[i] = other
            for n, call in enumerate(_calls(h, places)):
                if cls is P.Int4Linear and n == 1 and i == 2:
                    continue                   # a forward of two tensors
                with pytest.raises(ValueError, match="cuda:1"):
                    call()
    assert not reached
