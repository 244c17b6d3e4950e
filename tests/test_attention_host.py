"""Attention operators on the host: what the C calls and the bindings refuse before
anything is enqueued, and the frequencies (no GPU; fake pointers are never read)."""
import ctypes
import math
from decimal import Decimal, getcontext

import pytest
import torch

import attention_reference as ref
import fake_quant_numerics_gb300 as fq
from fake_quant_numerics_gb300 import _lib as L

A = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)
INV, UNS, MIS, DIM = L.QAT_ERR_INVALID_ARGUMENT, L.QAT_ERR_UNSUPPORTED, L.QAT_ERR_MISALIGNED, L.QAT_ERR_DIMENSION_MISMATCH


@pytest.fixture(scope="module")
def lib():
    from fake_quant_numerics_gb300 import build

    build.build()
    return L.load(build_if_missing=False)


def rope(lib, back=False, dt=L.BF16, tokens=2, hq=4, hk=2, d=64, rot=32, layout=0, amp=1.0, norm=1, eps=1e-6, ws=A,
         wsb=1 << 30, strides=(256, 64, 128, 64), **kw):
    a = dict(q=A, k=A, positions=A, turns=A, wq=A, wk=A, yq=A, yk=A, gq=A, gk=A, dwq=A, dwk=A)
    a.update(kw)
    mid = (dt, tokens, hq, hk, d) + strides + (a["positions"], a["turns"], rot, layout, amp, norm, a["wq"], a["wk"], eps,
                                               a["yq"], a["yk"])
    if back:
        return lib.qat_head_norm_rope_backward(a["gq"], a["gk"], a["q"], a["k"], *mid, a["dwq"], a["dwk"], ws, wsb, None)
    return lib.qat_head_norm_rope(a["q"], a["k"], *mid, None)


@pytest.mark.parametrize("back", [False, True])
def test_rope_refusals(lib, back):
    def call(**kw):
        return rope(lib, back, **kw)

    assert call(dt=5) == UNS and call(layout=2) == UNS
    assert call(d=0) == INV and call(d=513, rot=0) == INV
    assert call(rot=31) == INV and call(rot=66) == INV and call(rot=-2) == INV
    assert call(tokens=-1) == INV and call(hq=-1) == INV and call(hk=-1) == INV and call(hq=1 << 31) == INV
    assert call(tokens=1 << 48) == INV and call(strides=(1 << 60, 64, 64, 64)) == INV
    for bad in (-1e-6, float("nan"), float("inf")):
        assert call(eps=bad) == INV
    for bad in (float("nan"), float("inf")):
        assert call(amp=bad) == INV
    assert call(norm=0) == INV  # with weights
    assert all(call(**{n: None}) == INV for n in ("q", "k", "positions", "turns"))
    assert all(call(**{n: ODD}) == MIS for n in ("q", "k", "wq", "wk", "yq", "yk", "positions", "turns"))
    if back:
        assert all(call(**{n: None}) == INV for n in ("gq", "gk"))
        assert all(call(**{n: ODD}) == MIS for n in ("gq", "gk", "dwq", "dwk"))
        assert call(norm=0, wq=None, wk=None) == INV  # weight gradients
        need = lib.qat_head_norm_rope_backward_workspace_bytes(64)
        assert need > 0 and call(wsb=need - 1) == L.QAT_ERR_WORKSPACE and call(ws=None) == L.QAT_ERR_WORKSPACE
        assert call(ws=ODD) == MIS
        assert call(tokens=0, dwq=None, dwk=None, q=None, k=None) == L.QAT_OK
        assert call(yq=None, yk=None, dwq=None, dwk=None, q=None, gq=None) == L.QAT_OK  # nothing wanted
        assert lib.qat_head_norm_rope_backward_workspace_bytes(513) == 0
    else:
        assert call(yq=None) == INV and call(yk=None) == INV
        assert call(tokens=0, q=None, k=None, yq=None, yk=None, positions=None) == L.QAT_OK
        assert call(hq=0, hk=0, q=None, k=None) == L.QAT_OK


def cache(**kw):
    a = dict(k=0x10000, v=0x10000, ks=0x10000, vs=0x10000, kz=None, vz=None, pages=4, heads=2, page_size=16,
             head_dim=64, format=L.CACHE_INT8)
    a.update(kw)
    return L.KvCacheStruct(*a.values())


BAD_CACHES = [
    (dict(format=5), UNS), (dict(format=-1), UNS), (dict(head_dim=60), UNS), (dict(head_dim=0), UNS),
    (dict(head_dim=264), UNS), (dict(page_size=8), INV), (dict(page_size=24), INV), (dict(page_size=0), INV),
    (dict(pages=-1), INV), (dict(pages=1 << 27), INV), (dict(heads=0), INV), (dict(heads=32768), INV),
    (dict(kz=0x10000), INV), (dict(kz=0x10000, vz=0x10000, format=L.CACHE_E4M3), INV), (dict(k=None), INV),
    (dict(vs=None), INV), (dict(v=0x10008), MIS), (dict(ks=0x10008), MIS), (dict(kz=0x10004, vz=0x10000), MIS),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_refusals(lib, kw, status):
    c = cache(**kw)
    at = ctypes.addressof(c)
    assert lib.qat_kv_write(at, A, A, L.BF16, 2, 128, 64, 128, 64, A, None) == status
    assert lib.qat_kv_read(at, A, 2, A, A, L.BF16, None) == status
    assert attend(lib, at) == status
    assert lib.qat_kv_attention_workspace_bytes(at, 4) == 0


def attend(lib, at, dt=L.BF16, batch=2, heads=4, qs=(256, 64), cols=3, stride=3, scale=0.125, ws=A, wsb=1 << 40, **kw):
    a = dict(q=A, table=A, lengths=A, y=A, lse=A)
    a.update(kw)
    return lib.qat_kv_attention(a["q"], dt, batch, heads, *qs, at, a["table"], cols, stride, a["lengths"], scale, a["y"],
                                a["lse"], ws, wsb, None)


def test_kv_call_refusals(lib):
    c = cache()
    at = ctypes.addressof(c)

    def write(k=A, v=A, dt=L.F32, tokens=2, strides=(128, 64, 128, 64), slots=A, where=at):
        return lib.qat_kv_write(where, k, v, dt, tokens, *strides, slots, None)

    assert write(dt=7) == UNS and write(where=None) == INV
    assert write(tokens=-1) == INV and write(tokens=1 << 50) == INV and write(strides=(1 << 60, 64, 64, 64)) == INV
    assert write(k=None) == INV and write(v=None) == INV and write(slots=None) == INV
    assert write(k=ODD) == MIS and write(v=ODD) == MIS and write(slots=ctypes.c_void_p(0x10004)) == MIS
    assert write(tokens=0, k=None, v=None, slots=None) == L.QAT_OK
    read = lib.qat_kv_read
    assert read(at, A, 2, A, A, 7, None) == UNS and read(None, A, 2, A, A, L.F32, None) == INV
    assert read(at, None, 2, A, A, L.F32, None) == INV and read(at, A, 2, None, A, L.F32, None) == INV
    assert read(at, A, -1, A, A, L.F32, None) == INV
    assert read(at, A, 2, ctypes.c_void_p(0x10008), A, L.F32, None) == MIS
    assert read(at, None, 0, None, None, L.F32, None) == L.QAT_OK
    assert [lib.qat_kv_row_bytes(f, 72) for f in range(-1, 6)] == [0, 144, 80, 48, 80, 80, 0]


def test_kv_attention_refusals(lib):
    c = cache()
    at = ctypes.addressof(c)
    assert attend(lib, at, dt=4) == UNS and attend(lib, None) == INV
    assert attend(lib, at, heads=3) == DIM
    assert attend(lib, at, batch=-1) == INV and attend(lib, at, batch=65536) == INV and attend(lib, at, heads=-2) == INV
    assert attend(lib, at, cols=-1) == INV and attend(lib, at, cols=1 << 31) == INV
    assert attend(lib, at, batch=60000, heads=1 << 16) == INV
    assert attend(lib, at, qs=(1 << 60, 64)) == INV and attend(lib, at, stride=1 << 60) == INV
    for bad in (float("nan"), float("inf")):
        assert attend(lib, at, scale=bad) == INV
    assert all(attend(lib, at, **{n: None}) == INV for n in ("q", "y", "lengths", "table"))
    assert all(attend(lib, at, **{n: ODD}) == MIS for n in ("q", "y", "lengths", "table", "lse"))
    need = lib.qat_kv_attention_workspace_bytes(at, 4)
    assert need > 0
    assert attend(lib, at, wsb=need - 1) == L.QAT_ERR_WORKSPACE and attend(lib, at, ws=None) == L.QAT_ERR_WORKSPACE
    assert attend(lib, at, ws=ODD) == MIS
    assert attend(lib, at, batch=0, q=None) == L.QAT_OK and attend(lib, at, heads=0, q=None) == L.QAT_OK
    assert lib.qat_kv_attention_workspace_bytes(at, 5) == 0


def meta(t):
    return t.to("meta")


def status(call):
    with pytest.raises(fq.QatError) as e:
        call()
    return e.value.status


def test_rope_binding_refusals():
    q, k, turns = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64), fq.rope_turns(fq.rope_frequencies(32))
    p, w = torch.arange(3), torch.ones(64)
    for back in (False, True):
        def call(q=q, k=k, p=p, t=turns, wq=None, wk=None, g=None, **kw):
            if back:
                return fq.head_norm_rope_backward(q if g is None else g, k, q, k, p, t, wq, wk, **kw)
            return fq.head_norm_rope(q, k, p, t, wq, wk, **kw)

        assert status(lambda: call(p=p[:2])) == DIM
        assert status(lambda: call(q=torch.zeros(64), k=None, p=p[:1])) == DIM
        assert status(lambda: call(k=k[:2])) == DIM and status(lambda: call(k=k[..., :32])) == DIM
        assert status(lambda: call(wq=w[:63])) == DIM and status(lambda: call(t=turns.view(2, -1))) == DIM
        for bad in (dict(p=p.int()), dict(t=turns.double()), dict(k=k.bfloat16()), dict(wq=w.bfloat16()),
                    dict(q=q.half(), k=None), dict(k=meta(k)), dict(p=meta(p)), dict(wk=meta(w)),
                    dict(wq=w, norm=False), dict(k=None, wk=w), dict(layout="other")):
            with pytest.raises((TypeError, ValueError)):
                call(**bad)
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()
    assert status(lambda: fq.head_norm_rope_backward(q[:2], k, q, k, p, turns)) == DIM
    assert status(lambda: fq.head_norm_rope_backward(q, None, q, k, p, turns)) == DIM


def test_cache_binding_refusals():
    c = fq.kv_cache(3, 2, 16, 64, "int4", "affine", device="cpu")
    parts = dict(k=c.k, v=c.v, format="int4", head_dim=64, k_scale=c.k_scale, v_scale=c.v_scale,
                 k_zero_point=c.k_zero_point, v_zero_point=c.v_zero_point)
    assert fq.KVCache(**parts).pages == 3

    def make(**kw):
        return fq.KVCache(**{**parts, **kw})

    assert status(lambda: make(k=c.k[:2])) == DIM and status(lambda: make(head_dim=128)) == DIM
    assert status(lambda: make(k_scale=c.k_scale[:2])) == DIM
    for bad in (dict(format="int3"), dict(head_dim=60), dict(head_dim=264), dict(k=c.k.char(), v=c.v.char()),
                dict(k_scale=c.k_scale.double()), dict(k_zero_point=c.k_zero_point.int()), dict(v_scale=None),
                dict(k_zero_point=None), dict(v=meta(c.v)), dict(v_scale=meta(c.v_scale)),
                dict(k_scale=c.k_scale.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(k=torch.zeros(3 * 2 * 16 * 32 + 1, dtype=torch.uint8)[1:].view(3, 2, 16, 32))):
        with pytest.raises((TypeError, ValueError)):
            make(**bad)
    for bad in (lambda: fq.kv_cache(1, 1, 8, 64, device="cpu"), lambda: fq.kv_cache(1, 1, 24, 64, device="cpu"),
                lambda: fq.kv_cache(1, 0, 16, 64, device="cpu"), lambda: fq.kv_cache(1, 1, 16, 64, "e4m3", "affine"),
                lambda: fq.kv_cache(1, 1, 16, 64, "fp8"), lambda: fq.kv_cache(1, 1, 16, 20, device="cpu")):
        with pytest.raises(ValueError):
            bad()
    x, slots = torch.zeros(5, 2, 64), torch.arange(5)
    assert status(lambda: fq.kv_write(c, x[:, :1], x[:, :1], slots)) == DIM
    assert status(lambda: fq.kv_write(c, x, x[:4], slots)) == DIM
    assert status(lambda: fq.kv_write(c, x, x, slots[:4])) == DIM
    for bad in (lambda: fq.kv_write(c, x, x.bfloat16(), slots), lambda: fq.kv_write(c, x, x, slots.int()),
                lambda: fq.kv_write(c, x.half(), x.half(), slots), lambda: fq.kv_write(c, meta(x), meta(x), slots),
                lambda: fq.kv_read(c, slots.int()), lambda: fq.kv_read(c, slots, torch.float16),
                lambda: fq.kv_read(c, meta(slots))):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for call in (lambda: fq.kv_write(c, x, x, slots), lambda: fq.kv_read(c, slots)):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()


def test_kv_attention_binding_refusals():
    c = fq.kv_cache(3, 2, 16, 64, "int8", device="cpu")
    q, table, n = torch.zeros(5, 4, 64), torch.zeros(5, 2, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    for bad in (lambda: fq.kv_attention(q[..., :32], c, table, n), lambda: fq.kv_attention(q[:, :3], c, table, n),
                lambda: fq.kv_attention(q[0], c, table, n), lambda: fq.kv_attention(q, c, table[:4], n),
                lambda: fq.kv_attention(q, c, table[0], n), lambda: fq.kv_attention(q, c, table, n[:4])):
        assert status(bad) == DIM
    for bad in (lambda: fq.kv_attention(q, c, table.long(), n), lambda: fq.kv_attention(q, c, table, n.long()),
                lambda: fq.kv_attention(q.half(), c, table, n), lambda: fq.kv_attention(meta(q), c, table, n),
                lambda: fq.kv_attention(q, c, meta(table), n)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(ValueError, match="CUDA tensors only"):
        fq.kv_attention(q, c, table, n)


def test_rope_frequencies():
    f = fq.rope_frequencies(64, base=500000.0)
    assert f.dtype == torch.float64 and f.shape == (32,) and f[0] == 1.0
    assert abs(float(f[31]) - 500000.0 ** (-62 / 64)) < 1e-18
    assert torch.equal(fq.rope_frequencies(64, factor=4.0), fq.rope_frequencies(64) / 4)
    assert fq.rope_frequencies(0).numel() == 0
    g, f = fq.rope_frequencies(64, factor=8.0, original_length=4096), fq.rope_frequencies(64)
    turns = f * 4096 / math.tau
    assert torch.equal(g[turns >= 32], f[turns >= 32])
    assert torch.allclose(g[turns <= 1], f[turns <= 1] / 8, rtol=1e-15, atol=0)
    between = (turns > 1) & (turns < 32)
    assert between.any() and (g[between] < f[between]).all() and (g[between] > f[between] / 8).all()
    for bad in (lambda: fq.rope_frequencies(3), lambda: fq.rope_frequencies(-2), lambda: fq.rope_frequencies(4, base=0.0),
                lambda: fq.rope_frequencies(4, factor=-1.0),
                lambda: fq.rope_frequencies(4, factor=2.0, original_length=8, slow=4.0, fast=4.0),
                lambda: fq.rope_turns(torch.tensor([float("nan")]))):
        with pytest.raises(ValueError):
            bad()
    assert status(lambda: fq.rope_turns(torch.zeros(2, 2))) == DIM


def test_rope_turns_are_exact():
    """f / (2 pi) of a turn to 53 bits: a position of 2^24 is then at most 2^-27 of a
    turn off for f = 1."""
    getcontext().prec = 60
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194988918")
    f = [1.0, 0.1, 1e-4, 2.5, -0.3, 7.0, 0.0, 1e-12]
    for x, t in zip(f, fq.rope_turns(torch.tensor(f, dtype=torch.float64)).tolist()):
        exact = Decimal(x) / two_pi * (1 << 64)
        off = (Decimal(t) - exact) % (1 << 64)
        off = min(off, (1 << 64) - off)
        assert off <= 1 + 4 * abs(exact) * Decimal(2) ** -53 + (1 << 12 if abs(x) > math.tau else 0), x
    c, s = ref.angles([3, -3], [1 << 62], 1.0)
    assert abs(c[0, 0]) < 1e-15 and abs(s[0, 0] + 1) < 1e-15 and abs(s[1, 0] - 1) < 1e-15


@pytest.mark.parametrize("current,guarded", [(None, False), (1, True)])
def test_calls_launch_on_the_tensors_device(monkeypatch, current, guarded):
    """A launch goes to the current device, so tensors of another one make theirs
    current for the call (host tensors, whose device has no index, stand for them)."""
    from fake_quant_numerics_gb300 import attention, layers

    entered, seen = [], []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)

        def __exit__(self, *args):
            entered.pop()

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 64
            return lambda *a: seen.append((name, bool(entered))) or 0

    monkeypatch.setattr(layers._lib, "lib", lambda: Lib())
    monkeypatch.setattr(attention, "_ptr", lambda t: t.data_ptr())
    monkeypatch.setattr(layers, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(layers, "_current_device", lambda: current, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    q, w, p = torch.zeros(3, 4, 64), torch.ones(64), torch.arange(3)
    turns, c = fq.rope_turns(fq.rope_frequencies(64)), fq.kv_cache(3, 2, 16, 64, device="cpu")
    fq.head_norm_rope(q, q, p, turns, w, w)
    fq.head_norm_rope_backward(q, q, q, q, p, turns, w, w)
    fq.kv_write(c, q[:, :2], q[:, 2:], p)
    fq.kv_read(c, p)
    fq.kv_attention(q, c, torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32))
    assert not entered
    names = ["head_norm_rope", "head_norm_rope_backward", "kv_write", "kv_read", "kv_attention"]
    assert seen == [("qat_" + name, guarded) for name in names]
