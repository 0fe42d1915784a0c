"""Calls of the heads' entry points that a program may make and that are easily
got wrong: the binding without its native part, arrays of a batch that break its
rules, buffers beside those that are written, no queries or no rows, another
dtype of the output, shared pages."""
import numpy as np
import pytest
import torch

from heads_util import Batch, TYPES, attend_all, bits, device_cache, f32, host_cache, near, same_bits, stream_rows
from oracle import heads
from parity_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dqm(lib):
    from w4a4_quantized_linear_cube_amd import dq
    return dq


def _rope(dqm, pairs, positions, interleaved=True):
    table = torch.empty(positions, pairs, 2, device=DEV)
    dqm.dq_rope_table(10000.0 ** (-np.arange(pairs) / pairs), positions, table)
    return dqm.Rope([table], interleaved)


def _all_calls(dqm, seed):
    """Outputs of one call of each kind, with every option given."""
    batch = Batch([2, 3], [40, 9], 16, DEV, seed=seed)
    kv, seqs = device_cache(dqm, host_cache(batch, 2, 64, 8, seed), DEV), batch.seqs(dqm)
    x = stream_rows(5, 8 * 64, "bf16", seed + 1).to(DEV)
    q, k, v = x[:, :256], x[:, 256:384], x[:, 384:]
    rope, pos = _rope(dqm, 32, 50), torch.arange(5, dtype=torch.int32, device=DEV)[:, None].contiguous()
    g = (1 + 0.1 * torch.randn(64, generator=torch.Generator().manual_seed(seed))).to(DEV)
    y, z, out = (torch.empty(5, 256, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    back = [torch.empty(5, 128, device=DEV) for _ in range(2)]
    dqm.dq_norm_rope(q, 4, y, norm="head", gain=g, eps=1e-5, rope=rope, pos=pos)
    dqm.dq_kv_write(kv, seqs, k, v, q=q, y=z, norm="head", gain=g, gain_q=g, eps=1e-5, rope=rope)
    dqm.dq_kv_read(kv, seqs, *back)
    dqm.dq_attn_rows(kv, seqs, z, dqm.dq_attn_create(0), out, scale=0.2, block=2, window=30,
                     prefix=torch.tensor([3, 1], dtype=torch.int32, device=DEV), cap=5.0)
    return [y, z, out, *back, *kv.tensors]


def test_without_the_native_marshalling(dqm, monkeypatch):
    want = _all_calls(dqm, 3)
    monkeypatch.setattr(dqm, "_CALL", None)
    monkeypatch.setattr(dqm, "_native", lambda: None)
    for a, b in zip(_all_calls(dqm, 3), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("native", [True, False])
def test_refusals_of_the_binding(dqm, monkeypatch, native):
    if not native:
        monkeypatch.setattr(dqm, "_CALL", None)
        monkeypatch.setattr(dqm, "_native", lambda: None)
    batch = Batch([2], [20], 16, DEV)
    cache = host_cache(batch, 2, 64, 8, 1)
    kv, seqs, work = device_cache(dqm, cache, DEV), batch.seqs(dqm), dqm.dq_attn_create(0)
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device=DEV)
    i32 = lambda *s: z(*s, d=torch.int32)
    rope = _rope(dqm, 32, 50)
    two = dqm.Rope([z(5, 16, 2, d=torch.float32)] * 2)
    for call in [
        lambda: dqm.dq_norm_rope(z(2, 128), 3, z(2, 128)), lambda: dqm.dq_norm_rope(z(2, 128), 2, z(2, 127)),
        lambda: dqm.dq_norm_rope(z(2, 128), 2, z(3, 128)), lambda: dqm.dq_norm_rope(z(2, 128, d=torch.float16), 2, z(2, 128)),
        lambda: dqm.dq_norm_rope(z(2, 128), 2, z(2, 128), norm="heads"), lambda: dqm.dq_norm_rope(z(2, 128), 2, z(2, 128), gain=z(64)),
        lambda: dqm.dq_norm_rope(z(2, 128), 2, z(2, 128), norm="head", gain=z(128)),
        lambda: dqm.dq_norm_rope(z(2, 128), 2, z(2, 128), norm="row", gain=z(64)),
        lambda: dqm.dq_norm_rope(z(2, 128), 2, z(2, 128), pos=i32(2, 1)),
        lambda: dqm.dq_norm_rope(z(2, 128), 2, z(2, 128), rope=rope, pos=i32(2, 2)),
        lambda: dqm.dq_norm_rope(z(2, 128), 2, z(2, 128), rope=rope, pos=z(2, 1, d=torch.int64)),
        lambda: dqm.dq_norm_rope(z(2, 128), 2, z(2, 128), rope=two),
        lambda: dqm.dq_norm_rope(z(2, 128).cpu(), 2, z(2, 128)), lambda: dqm.dq_norm_rope(z(2, 256)[:, ::2], 2, z(2, 128)),
        lambda: dqm.dq_norm_rope(z(2, 130)[:, 1:129], 2, z(2, 128)), lambda: dqm.dq_norm_rope(z(2, 128), 2, z(2, 128), eps=0.0, norm="row"),
        lambda: dqm.dq_kv_write(kv, seqs, z(2, 128), z(2, 64)), lambda: dqm.dq_kv_write(kv, seqs, z(2, 128), z(2, 128, d=torch.float32)),
        lambda: dqm.dq_kv_write(kv, seqs, z(2, 128), z(2, 128), q=z(2, 128)),
        lambda: dqm.dq_kv_write(kv, seqs, z(2, 128), z(2, 128), q=z(2, 96), y=z(2, 96)),
        lambda: dqm.dq_kv_write(kv, seqs, z(2, 128), z(2, 128), norm="head", gain_q=z(64)),
        lambda: dqm.dq_kv_write(kv, seqs, z(2, 128), z(2, 128), q=z(2, 128), y=z(2, 128), norm="head", gain=z(64), gain_q=z(64, d=torch.float32)),
        lambda: dqm.dq_kv_read(kv, seqs), lambda: dqm.dq_kv_read(kv, seqs, z(2, 64)),
        lambda: dqm.dq_kv_read(kv, seqs, z(2, 128), z(2, 128, d=torch.float32)),
        lambda: dqm.dq_attn_rows(kv, seqs, z(2, 128), work, z(2, 256)), lambda: dqm.dq_attn_rows(kv, seqs, z(2, 192), work, z(2, 192)),
        lambda: dqm.dq_attn_rows(kv, seqs, z(2, 128), work, z(2, 128, d=torch.float32)),
        lambda: dqm.dq_attn_rows(kv, seqs, z(2, 128), None, z(2, 128)),
        lambda: dqm.dq_attn_rows(kv, seqs, z(2, 128), work, z(2, 128), scale=-1.0),
        lambda: dqm.dq_attn_rows(kv, seqs, z(2, 128), work, z(2, 128), block=-1),
        lambda: dqm.dq_attn_rows(kv, seqs, z(2, 128), work, z(2, 128), block=0, window=3),
        lambda: dqm.dq_attn_rows(kv, seqs, z(2, 128), work, z(2, 128), block=2 ** 40),
        lambda: dqm.dq_attn_rows(kv, seqs, z(2, 128), work, z(2, 128), prefix=i32(2)),
        lambda: dqm.dq_attn_rows(kv, seqs, z(2, 128), work, z(2, 128), cap=-3.0),
        lambda: dqm.KV(*kv.tensors, bits=4), lambda: dqm.KV(kv.tensors[0][:, :, ::2], *kv.tensors[1:]),
        lambda: dqm.KV(kv.tensors[0].float(), *kv.tensors[1:]),
        lambda: dqm.KV(kv.tensors[0], kv.tensors[1][1:], *kv.tensors[2:]), lambda: dqm.Seqs(i32(3), i32(3), i32(3, 2)),
        lambda: dqm.Seqs(i32(4), i32(3), i32(3, 2)[:, :1]), lambda: dqm.Seqs(z(4, d=torch.int64), i32(3), i32(3, 2)),
        lambda: dqm.Rope([z(4, 8, 2)]), lambda: dqm.Rope([z(4, 8, 3, d=torch.float32)]), lambda: dqm.Rope([z(0, 8, 2, d=torch.float32)]),
    ]:
        with pytest.raises(dqm.DQError):
            call()
    torch.cuda.synchronize()
    for t, a in zip(kv.tensors, cache):
        assert np.array_equal(bits(t), a)


@pytest.mark.parametrize("device", [-1, 63, 64, 1 << 30])
def test_a_device_that_is_not_there(dqm, lib, device):
    import ctypes
    h = ctypes.c_void_p()
    f = np.ones(2)
    kv, seqs = dqm._KV(1 << 32, 2 << 32, 3 << 32, 4 << 32, 1, 16, 1, 64, 8), dqm._Seqs(1, 5 << 32, 6 << 32, 7 << 32, 1)
    ops = dqm._HeadOps(0, 0, 0.0, None, None)
    r = ctypes.byref
    for status in (lib.dq_attn_create(device, r(h)), lib.dq_rope_table(ctypes.c_void_p(f.ctypes.data), 2, 4, 8 << 32, device, None),
                   lib.dq_norm_rope(9 << 32, 64, 1, 1, 1, 64, None, r(ops), 10 << 32, 64, 1, device, None),
                   lib.dq_kv_write(r(kv), r(seqs), 1, 1, 11 << 32, 64, 12 << 32, 64, None, None, 0, 0, None, None, 0, 1, r(ops), device, None),
                   lib.dq_kv_read(r(kv), r(seqs), 1, 13 << 32, 64, None, 0, 1, device, None)):
        assert status == 1 and "device index out of range" in lib.dq_last_error().decode()


def test_no_rows(dqm):
    batch = Batch([0], [20], 16, DEV)
    kv, seqs = device_cache(dqm, host_cache(batch, 1, 64, 8, 1), DEV), batch.seqs(dqm)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    before = [t.clone() for t in kv.tensors]
    dqm.dq_norm_rope(e, 1, e)
    dqm.dq_kv_write(kv, seqs, e, e, q=e, y=e)
    dqm.dq_kv_read(kv, seqs, k=e)
    dqm.dq_attn_rows(kv, seqs, e, dqm.dq_attn_create(0), e)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kv.tensors, before))


def test_queries_change_their_type_and_place(dqm):
    """q in fp32 and y in bf16, the other way round, and y over q inside the stacked projection."""
    batch = Batch([3], [30], 16, DEV)
    n, c = 3, 64
    tables = [heads.table(10000.0 ** (-np.arange(32) / 32), 40)]
    pos = np.arange(27, 30)[:, None]
    for dt, ydt in (("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")):
        cache = host_cache(batch, 1, 64, 8, 5)
        kv, seqs = device_cache(dqm, cache, DEV), batch.seqs(dqm)
        x = stream_rows(n, 4 * c, dt, 7).to(DEV)
        keep = x.clone()
        y = torch.empty(n, 2 * c, dtype=TYPES[ydt], device=DEV) if dt != ydt else x[:, :2 * c]
        dqm.dq_kv_write(kv, seqs, x[:, 2 * c:3 * c], x[:, 3 * c:], q=x[:, :2 * c], y=y, norm="head", rope=_rope(dqm, 32, 40))
        want = heads.norm_rope(f32(keep[:, :2 * c]), 2, "head", None, 1e-6, tables, pos, True).reshape(n, -1)
        same_bits(y, want, ydt)
        assert torch.equal(x[:, 2 * c:], keep[:, 2 * c:])


def test_more_than_a_tables_sequences(dqm):
    """64 sequences and more, empty ones among them, for rows of several to a wave and of several waves."""
    for kv_heads, dim in ((1, 32), (1, 64), (8, 128)):
        for B in (63, 64, 65, 200, 5000):
            g = np.random.default_rng(B)
            rows = g.integers(0, 3, B)
            length = rows + g.integers(0, 30, B)
            batch = Batch(rows.tolist(), length.tolist(), 16, DEV, seed=B, tail=1)
            n, c = batch.n, kv_heads * dim
            z = lambda w: torch.zeros(batch.count, kv_heads, 16, w, dtype=torch.uint8, device=DEV)
            kv, seqs = dqm.KV(z(dim), z(dim // 32), z(dim), z(dim // 32)), batch.seqs(dqm)
            x = stream_rows(n, 2 * c, "f32", B)
            xd = x.to(DEV)
            dqm.dq_kv_write(kv, seqs, xd[:, :c], xd[:, c:])
            got = [torch.full((n, c), 9.0, device=DEV) for _ in range(2)]
            dqm.dq_kv_read(kv, seqs, *got)
            for i in range(2):
                want = heads.decode(*heads.encode(x[:, i * c:(i + 1) * c].numpy().reshape(-1, 32), 8), 8).reshape(n, c).astype(np.float32)
                want[-1] = 9.0
                same_bits(got[i], want, "f32")


def test_a_batch_that_breaks_its_rules(dqm):
    """Starts that fall, lie outside of the rows or are negative, negative and huge
    lengths: no more is promised than that nothing outside of the outputs and the
    cache is touched.  (Every index is held to its array: rows by [0, N), places by
    the table's width, pages by their number, tiles by the most that there can be.)"""
    work = dqm.dq_attn_create(0)
    for kv_heads, n in ((1, 40), (2, 200)):
        c = kv_heads * 64
        for first, length in (([0, n, 0, n, 0, n, 0, n], [500] * 7), ([5, 3, -7, 2 ** 31 - 1], [100, -5, 2 ** 31 - 1]), ([-2 ** 31, n + 900], [2 ** 31 - 1]),
                              ([n, n, 0], [7, 0]), ([0] + [n] * 64, [300] * 64), ([0, n] * 50 + [0], [90] * 100)):
            batch = Batch([1] * (len(first) - 1), [1000] * (len(first) - 1), 16, DEV)
            batch.first, batch.length = np.array(first, np.int64).astype(np.int32), np.array(length, np.int64).astype(np.int32)
            wide = [torch.full((a.size + 512,), 0x5A, dtype=torch.uint8, device=DEV) for a in host_cache(batch, kv_heads, 64, 8, 1)]
            shapes = [(batch.count, kv_heads, 16, w) for w in (64, 2, 64, 2)]
            kv = dqm.KV(*(w[256:-256].view(s) for w, s in zip(wide, shapes)))
            for t in kv.tensors:
                t.zero_()
            seqs = batch.seqs(dqm)
            frame = torch.full((n + 2, 3 * c), 3.0, dtype=torch.bfloat16, device=DEV)
            x = torch.randn(n, 2 * c, device=DEV).bfloat16()
            dqm.dq_kv_write(kv, seqs, x[:, :c], x[:, c:], q=x[:, :c], y=frame[1:-1, c:2 * c])
            dqm.dq_kv_read(kv, seqs, frame[1:-1, c:2 * c], torch.empty(n, c, dtype=torch.bfloat16, device=DEV))
            for how in (dict(), dict(block=0), dict(block=3, window=20)):
                dqm.dq_attn_rows(kv, seqs, x[:, :c], work, frame[1:-1, c:2 * c], **how)
            torch.cuda.synchronize()
            assert (frame[0] == 3).all() and (frame[-1] == 3).all() and (frame[:, :c] == 3).all() and (frame[:, 2 * c:] == 3).all()
            assert all((w[:256] == 0x5A).all() and (w[-256:] == 0x5A).all() for w in wide)
    # and the workspace still serves
    batch = Batch([1, 2], [900, 70], 16, DEV)
    cache = host_cache(batch, 1, 64, 8, 3)
    kv, seqs = device_cache(dqm, cache, DEV), batch.seqs(dqm)
    q = torch.randn(3, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    y = torch.empty(3, 64, dtype=torch.bfloat16, device=DEV)
    dqm.dq_attn_rows(kv, seqs, q.to(DEV), work, y)
    near(y, *attend_all(q, batch, cache, 8, 1, 64, "bf16"))


def test_pages_that_sequences_share(dqm):
    """A prefix in common: the same pages in several rows of the table, read by all."""
    batch = Batch([1, 1, 2], [100, 70, 64], 32, DEV)
    batch.pages[1, :2] = batch.pages[0, :2]
    batch.pages[2, :2] = batch.pages[0, :2]
    cache = host_cache(batch, 2, 64, 8, 9)
    kv, seqs = device_cache(dqm, cache, DEV), batch.seqs(dqm)
    q = torch.randn(4, 512, generator=torch.Generator().manual_seed(11)).bfloat16()
    y = torch.empty(4, 512, dtype=torch.bfloat16, device=DEV)
    dqm.dq_attn_rows(kv, seqs, q.to(DEV), dqm.dq_attn_create(0), y)
    near(y, *attend_all(q, batch, cache, 8, 2, 64, "bf16"))


def test_two_threads_call_at_once(dqm):
    """Each with its own stream, cache and workspace."""
    import threading
    out, errors = {}, []

    def serve(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    out[i] = _all_calls(dqm, 20 + i)
            s.synchronize()
        except Exception as e:      # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=serve, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(out[i], _all_calls(dqm, 20 + i)):
            assert torch.equal(a, b)
