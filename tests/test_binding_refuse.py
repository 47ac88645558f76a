"""What the quick check of a call's tensors refuses is never passed on, also where the closer look finds
nothing (no GPU: tensors that only say what they are)."""
import pytest
import torch

import mla_latent_kv_42_b200 as M
from mla_latent_kv_42_b200 import synth


class Fake:
    def __init__(self, shape, dtype, device=0, stride=None):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, f"cuda:{device}"
        self._device, self._stride = device, stride

    def get_device(self):
        return self._device

    def data_ptr(self):
        return 1 << 20

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self._stride is None

    def stride(self, i):
        return self._stride[i] if self._stride else int(torch.empty(self.shape, device="meta").stride(i))


def test_always_raises():
    t = Fake((3, 8), torch.bfloat16)
    assert M._ok(t, torch.bfloat16, (3, 8), 0)
    with pytest.raises(ValueError, match="x"):
        M._refuse(0, (t, "x", torch.bfloat16, (3, 8)))
    with pytest.raises(ValueError):
        M._refuse(0, (Fake((3, 8), torch.bfloat16, stride=(16, 1)), "x", torch.bfloat16, (3, 8)), strided="x")


def test_a_list_that_is_short_of_the_condition_still_refuses(monkeypatch):
    """A condition that fails for a tensor the list does not name ends in an error, not in the library."""
    d = synth.RUNNING
    i32 = lambda *s: Fake(s, torch.int32)
    called = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(M, "_ok", lambda *a: False)
    monkeypatch.setattr(M, "_rows_ok", lambda *a: False)
    monkeypatch.setattr(M, "_raw_stream", lambda *a: 0)

    class Lib:
        def __getattr__(self, name):
            return lambda *a: called.append(name) or 0

    monkeypatch.setattr(M, "_lib", lambda: Lib())
    pool, x, table = Fake((4, 64, d.D), torch.bfloat16), Fake((3, d.D), torch.bfloat16), i32(3, 2)
    with pytest.raises(ValueError):
        M.norm_append_kv(d, x, i32(3), i32(3), table, pool)
    with pytest.raises(ValueError):
        M.read_kv(d, pool, i32(3), i32(3), table, out=x)
    q = Fake((3, d.n_heads, d.D), torch.bfloat16)
    with pytest.raises(ValueError):
        M.shared_prefix_attention(d, q, pool, table, i32(3), 128, i32(1), o_lat=Fake((3, 8, d.d_c), torch.bfloat16),
                                  lse=Fake((3, 8), torch.float32))
    assert not called
