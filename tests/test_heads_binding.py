"""The heads' calls of the binding hand the native marshalling only descriptions
that are what they should be: it follows their addresses."""
import types

import pytest
import torch

from w4a4_quantized_linear_cube_amd import dq


class _Recorder:
    """Stands in for the native calls; takes every call as done."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


def _of(cls):
    o = cls.__new__(cls)
    o.address, o.device = 1 << 32, 0
    o.heads, o.head_dim, o.seqs = 1, 64, 1
    return o


# what has an address and a device and is no rotation: another description, an object of the caller's
@pytest.mark.parametrize("rope", [_of(dq.KV), _of(dq.Seqs), types.SimpleNamespace(address=1 << 32, device=0), 5])
@pytest.mark.parametrize("which", ["norm_rope", "kv_write"])
def test_a_rotation_that_is_none_is_not_followed(monkeypatch, rope, which):
    native = _Recorder()
    monkeypatch.setattr(dq, "_CALL", native)
    x = torch.zeros(2, 64)
    with pytest.raises(dq.DQError) as e:
        if which == "norm_rope":
            dq.dq_norm_rope(x, 1, x, rope=rope)
        else:
            dq.dq_kv_write(_of(dq.KV), _of(dq.Seqs), x, x, rope=rope)
    assert e.value.status == 1 and not native.calls


@pytest.mark.parametrize("rope", [None, _of(dq.Rope)])
def test_a_rotation_and_none_are(monkeypatch, rope):
    native = _Recorder()
    monkeypatch.setattr(dq, "_CALL", native)
    x = torch.zeros(2, 64)
    dq.dq_norm_rope(x, 1, x, rope=rope)
    dq.dq_kv_write(_of(dq.KV), _of(dq.Seqs), x, x, rope=rope)
    assert native.calls == ["norm_rope", "kv_write"]


@pytest.mark.gpu
def test_the_refusal_names_the_rotation(lib):
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda:0")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda:0")
    z = lambda w: torch.zeros(1, 1, 16, w, dtype=torch.uint8, device="cuda:0")
    kv, seqs = dq.KV(z(64), z(2), z(64), z(2)), dq.Seqs(i32(0, 2), i32(2), i32(0)[None])
    for rope in (kv, seqs, types.SimpleNamespace(address=1 << 32, device=0)):
        for call in (lambda: dq.dq_norm_rope(x, 1, x, rope=rope), lambda: dq.dq_kv_write(kv, seqs, x, x, rope=rope)):
            with pytest.raises(dq.DQError, match="rope must be a Rope"):
                call()
