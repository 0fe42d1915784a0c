"""Heads, cache and attention without a GPU: every refusal of the C entry points
and of the binding, and the oracle they are compared with."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import heads, mx, rows
from w4a4_quantized_linear_cube_amd import dq

A = 1 << 32              # addresses that are never followed: every call below is refused first


def _at(i):
    return A + i * (1 << 28)


def _rope(**kw):
    a = dict(axes=1, interleaved=1, pairs=(32, 0, 0), positions=(100, 0, 0), table=(_at(20), 0, 0))
    a.update(kw)
    r = dq._Rope(a["axes"], a["interleaved"])
    for i in range(3):
        r.pairs[i], r.positions[i], r.table[i] = a["pairs"][i], a["positions"][i], a["table"][i] or None
    return r


def _ops(norm=1, gain_dt=0, eps=1e-6, rope=None, pos=None):
    o = dq._HeadOps(norm, gain_dt, eps, ctypes.addressof(rope) if rope else None, pos)
    o.keep = rope
    return o


def _norm_rope(lib, **kw):
    a = dict(x=_at(0), ldx=256, dt=1, N=4, heads=4, dim=64, gain=_at(1), ops=_ops(), y=_at(2), ldy=256, ydt=1, device=0)
    a.update(kw)
    return lib.dq_norm_rope(a["x"], a["ldx"], a["dt"], a["N"], a["heads"], a["dim"], a["gain"],
                            ctypes.byref(a["ops"]) if a["ops"] else None, a["y"], a["ldy"], a["ydt"], a["device"], None)


@pytest.mark.parametrize("status,kw", [
    (1, dict(dt=2)), (1, dict(ydt=7)), (1, dict(x=None)), (1, dict(y=None)), (1, dict(ops=None)), (2, dict(N=-1)), (2, dict(N=2 ** 31)),
    (2, dict(heads=0)), (2, dict(dim=48)), (2, dict(dim=16)), (2, dict(dim=512)), (2, dict(heads=513)), (2, dict(ldx=255)), (2, dict(ldx=260)),
    (2, dict(ldy=128)), (2, dict(ldy=2 ** 50)), (1, dict(x=_at(0) + 8)), (1, dict(y=_at(2) + 2)), (1, dict(gain=_at(1) + 4)),
    (1, dict(ops=_ops(norm=3))), (1, dict(ops=_ops(norm=-1))), (1, dict(ops=_ops(gain_dt=2))), (1, dict(ops=_ops(eps=0.0))),
    (1, dict(ops=_ops(eps=math.nan))), (1, dict(ops=_ops(eps=math.inf))), (1, dict(ops=_ops(eps=1e-61))), (1, dict(ops=_ops(eps=-1.0))),
    (1, dict(ops=_ops(rope=_rope(axes=0)))), (1, dict(ops=_ops(rope=_rope(axes=4)))), (1, dict(ops=_ops(rope=_rope(interleaved=2)))),
    (2, dict(ops=_ops(rope=_rope(pairs=(0, 0, 0))))), (2, dict(ops=_ops(rope=_rope(pairs=(33, 0, 0))))),
    (2, dict(ops=_ops(rope=_rope(pairs=(200, 0, 0))))), (2, dict(ops=_ops(rope=_rope(pairs=(12, 0, 0), interleaved=0)))),
    (2, dict(ops=_ops(rope=_rope(positions=(0, 0, 0))))), (2, dict(ops=_ops(rope=_rope(positions=(2 ** 31, 0, 0))))),
    (1, dict(ops=_ops(rope=_rope(table=(0, 0, 0))))), (1, dict(ops=_ops(rope=_rope(table=(_at(20) + 4, 0, 0))))),
    (1, dict(ops=_ops(rope=_rope(axes=2, pairs=(16, 16, 0), positions=(9, 9, 0), table=(_at(20), _at(21), 0))))),   # no positions
    (1, dict(ops=_ops(rope=_rope(axes=2, pairs=(16, 16, 0), positions=(9, 9, 0), table=(_at(20), 0, 0)), pos=_at(22)))),
    (2, dict(ops=_ops(rope=_rope(axes=2, pairs=(16, 17, 0), positions=(9, 9, 0), table=(_at(20), _at(21), 0)), pos=_at(22)))),
    (1, dict(ops=_ops(rope=_rope(), pos=_at(22) + 2))),
    (1, dict(y=_at(0) + 512)), (1, dict(y=_at(0), ydt=0)), (1, dict(y=_at(0), ldy=512)), (1, dict(y=_at(1) - 1024)),
    (1, dict(y=_at(20), ops=_ops(rope=_rope()))), (1, dict(y=_at(22) - 16, ops=_ops(rope=_rope(), pos=_at(22)))),
])
def test_norm_rope_refusals(lib, status, kw):
    assert _norm_rope(lib, **kw) == status, lib.dq_last_error().decode()
    assert lib.dq_last_error().decode()


def test_table_refusals(lib):
    f = np.ones(4)
    p = ctypes.c_void_p(f.ctypes.data)
    call = lambda freq=p, pairs=4, n=10, t=A, d=0: lib.dq_rope_table(freq, pairs, n, t, d, None)
    assert call(freq=None) == 1 and call(t=None) == 1 and call(t=A + 4) == 1
    assert call(pairs=0) == 2 and call(pairs=129) == 2 and call(n=0) == 2 and call(n=2 ** 31) == 2
    for bad in (math.nan, math.inf):
        f[2] = bad
        assert call() == 1 and "finite" in lib.dq_last_error().decode()


def _kv(**kw):
    a = dict(kc=_at(3), ks=_at(4), vc=_at(5), vs=_at(6), pages=10, tokens=16, heads=2, dim=64, bits=8)
    a.update(kw)
    return dq._KV(a["kc"], a["ks"], a["vc"], a["vs"], a["pages"], a["tokens"], a["heads"], a["dim"], a["bits"])


def _seqs(**kw):
    a = dict(seqs=3, first=_at(7), length=_at(8), pages=_at(9), ld=5)
    a.update(kw)
    return dq._Seqs(a["seqs"], a["first"], a["length"], a["pages"], a["ld"])


BAD_KV = [(1, dict(bits=6)), (1, dict(kc=None)), (1, dict(vs=None)), (1, dict(kc=_at(3) + 8)), (1, dict(ks=_at(4) + 2)), (2, dict(dim=96)),
          (2, dict(heads=0)), (2, dict(heads=513)), (2, dict(tokens=8)), (2, dict(tokens=48)), (2, dict(tokens=131072)), (2, dict(pages=0)),
          (2, dict(pages=2 ** 31)), (2, dict(pages=2 ** 31 - 1, tokens=65536))]
BAD_SEQS = [(2, dict(seqs=0)), (2, dict(seqs=2 ** 20 + 1)), (2, dict(ld=0)), (2, dict(ld=2 ** 31)), (1, dict(first=None)), (1, dict(length=None)),
            (1, dict(pages=None)), (1, dict(length=_at(8) + 2))]


def _write(lib, kv=None, seqs=None, **kw):
    a = dict(N=4, dt=1, k=_at(0), ldk=128, v=_at(1), ldv=128, gk=_at(2), q=_at(10), ldq=512, qh=8, gq=_at(11), y=_at(12), ldy=512, ydt=1,
             ops=_ops(), device=0)
    a.update(kw)
    kv, seqs = kv or _kv(), seqs or _seqs()
    return lib.dq_kv_write(ctypes.byref(kv), ctypes.byref(seqs), a["N"], a["dt"], a["k"], a["ldk"], a["v"], a["ldv"], a["gk"], a["q"],
                           a["ldq"], a["qh"], a["gq"], a["y"], a["ldy"], a["ydt"], ctypes.byref(a["ops"]) if a["ops"] else None, a["device"], None)


def _read(lib, kv=None, seqs=None, **kw):
    a = dict(N=4, k=_at(0), ldk=128, v=_at(1), ldv=128, dt=1, device=0)
    a.update(kw)
    kv, seqs = kv or _kv(), seqs or _seqs()
    return lib.dq_kv_read(ctypes.byref(kv), ctypes.byref(seqs), a["N"], a["k"], a["ldk"], a["v"], a["ldv"], a["dt"], a["device"], None)


_FAKE = ctypes.create_string_buffer(64)          # a workspace of device 0, never used


def _attn(lib, kv=None, seqs=None, ops=(0.125, 0.0, 1, 0, None), **kw):
    a = dict(N=4, q=_at(0), ldq=256, dt=1, qh=4, a=ctypes.addressof(_FAKE), y=_at(1), ldy=256, device=0)
    a.update(kw)
    kv, seqs = kv or _kv(), seqs or _seqs()
    o = dq._AttnOps(*ops) if ops else None
    return lib.dq_attn_rows(ctypes.byref(kv), ctypes.byref(seqs), a["N"], a["q"], a["ldq"], a["dt"], a["qh"], ctypes.byref(o) if o else None,
                            a["a"], a["y"], a["ldy"], a["device"], None)


@pytest.mark.parametrize("call", [_write, _read, _attn])
def test_caches_and_batches_that_are_refused(lib, call):
    for status, kw in BAD_KV:
        assert call(lib, kv=_kv(**kw)) == status, (kw, lib.dq_last_error().decode())
    for status, kw in BAD_SEQS:
        assert call(lib, seqs=_seqs(**kw)) == status, (kw, lib.dq_last_error().decode())


def test_null_descriptions(lib):
    kv, seqs = _kv(), _seqs()
    assert lib.dq_kv_read(None, ctypes.byref(seqs), 1, A, 128, None, 0, 1, 0, None) == 1
    assert lib.dq_kv_read(ctypes.byref(kv), None, 1, A, 128, None, 0, 1, 0, None) == 1


@pytest.mark.parametrize("status,kw", [
    (2, dict(N=-1)), (2, dict(N=2 ** 31)), (1, dict(dt=5)), (1, dict(ydt=5)), (1, dict(k=None)), (1, dict(v=None)), (1, dict(ops=None)),
    (1, dict(q=None)), (1, dict(y=None)), (2, dict(qh=0)), (2, dict(qh=513)), (2, dict(ldk=64)), (2, dict(ldv=132)), (2, dict(ldq=256)),
    (2, dict(ldy=256)), (1, dict(k=_at(0) + 4)), (1, dict(q=_at(10) + 8)), (1, dict(gk=_at(2) + 8)), (1, dict(gq=_at(11) + 8)),
    (1, dict(ops=_ops(norm=9))), (1, dict(k=_at(3))), (1, dict(v=_at(4) - 128)), (1, dict(y=_at(5))), (1, dict(y=_at(0))), (1, dict(gk=_at(6))),
    (1, dict(y=_at(10), ydt=0)), (1, dict(y=_at(10) + 512)), (1, dict(y=_at(7) - 16)),
])
def test_write_refusals(lib, status, kw):
    assert _write(lib, **kw) == status, lib.dq_last_error().decode()
    assert lib.dq_last_error().decode()


@pytest.mark.parametrize("kw", [dict(vc=_at(3)), dict(ks=_at(3) + 16), dict(vs=_at(4)), dict(vc=_at(3) + 10 * 2 * 16 * 64 - 16)])
def test_a_cache_whose_arrays_meet_is_not_written(lib, kw):
    assert _write(lib, kv=_kv(**kw)) == 1 and "overlaps" in lib.dq_last_error().decode()


@pytest.mark.parametrize("status,kw", [
    (2, dict(N=-1)), (1, dict(dt=2)), (1, dict(k=None, v=None)), (2, dict(ldk=120)), (2, dict(ldv=129)), (1, dict(v=_at(1) + 2)),
    (1, dict(k=_at(1) + 256)), (1, dict(k=_at(3))), (1, dict(v=_at(6))), (1, dict(v=_at(9) - 16)),
])
def test_read_refusals(lib, status, kw):
    assert _read(lib, **kw) == status, lib.dq_last_error().decode()


@pytest.mark.parametrize("status,kw", [
    (2, dict(N=-1)), (2, dict(N=2 ** 24 + 1)), (1, dict(dt=3)), (2, dict(qh=0)), (2, dict(qh=3)), (2, dict(qh=1024)), (1, dict(ops=None)),
    (1, dict(a=None)), (1, dict(q=None)), (1, dict(y=None)), (1, dict(q=_at(0) + 8)), (1, dict(y=_at(1) + 4)), (2, dict(ldq=128)),
    (2, dict(ldy=260)), (1, dict(ops=(0.0, 0.0, 1, 0, None))), (1, dict(ops=(-1.0, 0.0, 1, 0, None))), (1, dict(ops=(math.nan, 0.0, 1, 0, None))),
    (1, dict(ops=(math.inf, 0.0, 1, 0, None))), (1, dict(ops=(0.1, -1.0, 1, 0, None))), (1, dict(ops=(0.1, math.nan, 1, 0, None))),
    (1, dict(ops=(0.1, 1e-30, 1, 0, None))), (2, dict(ops=(0.1, 0.0, -1, 0, None))), (2, dict(ops=(0.1, 0.0, 2 ** 31, 0, None))),
    (2, dict(ops=(0.1, 0.0, 1, -1, None))), (2, dict(ops=(0.1, 0.0, 1, 2 ** 31, None))), (1, dict(ops=(0.1, 0.0, 0, 5, None))),
    (1, dict(ops=(0.1, 0.0, 1, 0, A + 2))), (1, dict(y=_at(0))), (1, dict(y=_at(3))), (1, dict(y=_at(8) - 16)), (1, dict(device=1)),
    (1, dict(ops=(0.1, 0.0, 1, 0, _at(1) + 4))),
])
def test_attention_refusals(lib, status, kw):
    assert _attn(lib, **kw) == status, lib.dq_last_error().decode()


def test_attention_head_dims_and_sizes(lib):
    assert _attn(lib, kv=_kv(dim=32)) == 2 and _attn(lib, kv=_kv(dim=256, heads=1)) == 2
    assert _attn(lib, kv=_kv(heads=1), N=2 ** 24, qh=16, ldq=1024, ldy=1024) == 2 and "2^27" in lib.dq_last_error().decode()


def test_no_rows_is_no_work(lib):
    assert _norm_rope(lib, N=0, x=None, y=None) == 0
    assert _write(lib, N=0, k=None, v=None) == 0
    assert _read(lib, N=0, k=None, v=None) == 0
    assert _attn(lib, N=0, q=None, y=None) == 0


def test_workspace_without_a_place_for_it(lib):
    assert lib.dq_attn_create(0, None) == 1
    lib.dq_attn_destroy(None)


# ----------------------------------------------------------------- the binding ----
def test_descriptions_take_gpu_tensors_only():
    z = lambda *s, **k: torch.zeros(*s, **k)
    for make in (lambda: dq.Rope([z(4, 8, 2)]), lambda: dq.Rope([]), lambda: dq.Rope([z(4, 8, 2)] * 4), lambda: dq.Rope([None]),
                 lambda: dq.KV(*(z(2, 1, 16, n, dtype=torch.uint8) for n in (64, 2, 64, 2))),
                 lambda: dq.Seqs(z(2, dtype=torch.int32), z(1, dtype=torch.int32), z(1, 1, dtype=torch.int32))):
        with pytest.raises(dq.DQError) as e:
            make()
        assert e.value.status == 1


def test_binding_refuses_what_is_no_description():
    for call in (lambda: dq.dq_kv_write(None, None, None, None), lambda: dq.dq_kv_read(None, None, k=torch.zeros(1)),
                 lambda: dq.dq_attn_rows(None, None, None, None, None), lambda: dq.dq_norm_rope(torch.zeros(2, 64), 1, torch.zeros(2, 64)),
                 lambda: dq.dq_norm_rope(None, 1, None), lambda: dq.dq_rope_table([1.0], 4, torch.zeros(4, 1, 2))):
        with pytest.raises(dq.DQError) as e:
            call()
        assert e.value.status == 1


# ------------------------------------------------------------------ the oracle ----
@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_is_a_product_of_complex_numbers(interleaved):
    g = np.random.default_rng(1)
    v, P = g.standard_normal((7, 3, 64)).astype(np.float32), 24
    freqs = [10.0 ** -np.arange(8), 3.0 ** -np.arange(16)]
    pos = np.stack([g.integers(0, 50, 7), g.integers(0, 40, 7)], 1)
    got = heads.rotate(v, [heads.table(f, n) for f, n in zip(freqs, (50, 40))], pos, interleaved)
    angle = np.concatenate([pos[:, i:i + 1] * f for i, f in enumerate(freqs)], 1)[:, None]
    a, b = (v[..., 0:2 * P:2], v[..., 1:2 * P:2]) if interleaved else (v[..., :P], v[..., P:2 * P])
    z = (a + 1j * b.astype(np.float64)) * np.exp(1j * angle)
    ga, gb = (got[..., 0:2 * P:2], got[..., 1:2 * P:2]) if interleaved else (got[..., :P], got[..., P:2 * P])
    # two products, each of a coefficient and a value rounded, and their sum: 2^-24 of each, 4 times
    assert np.abs(ga + 1j * gb - z).max() <= 8 * 2.0 ** -24 * np.abs(v).max() * 2
    assert np.array_equal(got[..., 2 * P:], v[..., 2 * P:])


def test_rotation_keeps_lengths_and_turns_back():
    g = np.random.default_rng(2)
    v = g.standard_normal((5, 2, 32)).astype(np.float32)
    t = heads.table(np.linspace(0.1, 1, 16), 100)
    pos = g.integers(0, 100, (5, 1))
    r = heads.rotate(v, [t], pos, True)
    assert np.allclose((r.astype(np.float64) ** 2).sum(-1), (v.astype(np.float64) ** 2).sum(-1), rtol=1e-6)
    back = heads.rotate(r, [t * np.float32([1, -1])], pos, True)
    assert np.abs(back - v).max() <= 1e-6 * np.abs(v).max()


def test_norms_are_those_of_the_rows():
    g = np.random.default_rng(3)
    x, gain = g.standard_normal((4, 192)).astype(np.float32), g.standard_normal(192).astype(np.float32)
    assert np.array_equal(heads.norm_rope(x, 3, "row", gain).reshape(4, -1), rows.rms_norm(x, None, gain, 1e-6, "f32")[1])
    one = heads.norm_rope(x, 3, "head", gain[:64])
    for h in range(3):
        assert np.array_equal(one[:, h], rows.rms_norm(x[:, 64 * h:64 * h + 64], None, gain[:64], 1e-6, "f32")[1])


@pytest.mark.parametrize("nbits", [8, 4])
def test_codes_hold_what_they_stand_for(nbits):
    v = np.random.default_rng(4).standard_normal((9, 64)).astype(np.float32)
    c, s = heads.encode(v, nbits)
    again = heads.encode(heads.decode(c, s, nbits).astype(np.float32), nbits)
    assert np.array_equal(heads.decode(c, s, nbits), heads.decode(*again, nbits))
    fmt = "fp8" if nbits == 8 else "fp4"
    codes, scales = mx.mx_quantize(v, fmt)
    assert np.array_equal(s, scales) and np.array_equal(c, codes if nbits == 8 else mx.pack_fp4(codes))
    v[2, 3], v[5, 40] = np.inf, np.nan
    c, s = heads.encode(v, nbits)
    d = heads.decode(c, s, nbits)
    where = np.zeros(v.shape, bool)
    if nbits == 8:
        where[2, 3] = where[5, 40] = True
    else:
        where[2, :32] = where[5, 32:] = True
    assert np.array_equal(np.isnan(d), where)


def test_visible_against_a_list():
    for t in range(-2, 12):
        for block in (1, 3, 5):
            for window in (0, 1, 4):
                for prefix in (0, 2, 20):
                    mine = (t - t % block) + block - 1              # the last token of the row's own block
                    want = [tok < prefix or (tok <= mine and (window == 0 or tok > mine - window)) for tok in range(10)]
                    assert heads.visible(t, 10, block, window, prefix).tolist() == want
    assert heads.visible(3, 5, 0, 0, 0).all()


def test_attention_against_a_scalar_sum():
    g = np.random.default_rng(6)
    q, k, v = g.standard_normal((2, 8)), g.standard_normal((5, 8)), g.standard_normal((5, 8))
    on = np.array([True, False, True, True, False])
    y = heads.attend(q, k, v, on, 0.3, 2.0)[0]
    for i in range(2):
        w = [math.exp(2.0 * math.tanh(0.3 * float(q[i] @ k[t]) / 2.0)) if on[t] else 0.0 for t in range(5)]
        want = sum(w[t] * v[t] for t in range(5)) / sum(w)
        assert np.allclose(y[i], want, rtol=1e-13)
    assert not heads.attend(q, k, v, np.zeros(5, bool), 1.0)[0].any()


def test_places_and_pages():
    b, t = heads.places([1, 3, 3, 4], [10, 7, 2], 6)
    assert b.tolist() == [-1, 0, 0, 2, -1, -1] and t[[1, 2, 3]].tolist() == [8, 9, 1]
    pages = np.array([[4, -1, 9]])
    assert [heads.page_of(pages, 8, 16, 0, t) for t in (-1, 0, 15, 16, 32, 48)] == [-1, 4, 4, -1, -1, -1]
