"""A cache of few bits, drafted tokens and distillation without a GPU: what the host
checks and the binding refuse before any HIP call, and the references by hand."""
import ctypes as C
import re

import numpy as np
import pytest
import torch

import lm_draft_reference as ref
from byte_level_bpe_pretokenize_amd import _lib, lm
from test_lm_checks import P, header, z

I32, I64, I8, U8, F8 = torch.int32, torch.int64, torch.int8, torch.uint8, torch.float8_e4m3fn
EINVAL = _lib.BPE_EINVAL


def test_header_constants():
    for name, value in (("STATUS_BAD_SLOT", f"{_lib.STATUS_BAD_SLOT}u"),
                        ("STATUS_NOT_FINITE", f"{_lib.STATUS_NOT_FINITE}u"),
                        ("STATUS_NO_TOKEN", f"{_lib.STATUS_NO_TOKEN}u"), ("E4M3", _lib.E4M3),
                        ("INT8", _lib.INT8), ("UINT4", _lib.UINT4), ("MAX_HEADS", _lib.MAX_HEADS),
                        ("MAX_DIM", _lib.MAX_DIM), ("MAX_TOP", _lib.MAX_TOP)):
        assert re.search(rf"#define BPE_{name} {value}\s", header()), name


def test_cache_struct():
    text = re.sub(r"/\*.*?\*/", "", header(), flags=re.S)
    fields = re.findall(r"typedef struct \{([^{}]*)\} bpe_cache;", text)[0]
    names = [n.split()[-1].strip("*") for line in fields.split(";") for n in line.split(",") if n.strip()]
    assert names == [n for n, _ in _lib.Cache._fields_]


# ---- the C ABI ----------------------------------------------------------------------
def cache(**kw):
    a = dict(codes=P, scales=P, n_slots=100, codes_stride=2048, scales_stride=16, heads=16, dim=128,
             group=128, format=0)
    a.update(kw)
    return C.byref(_lib.Cache(**a))


def write_rc(c=None, x=P, xt=1, n=5, ts=2048, hs=128, slots=P, status=P, **kw):
    return _lib.load().bpe_cache_write(cache(**kw) if c is None else None, x, xt, n, ts, hs, slots, status, None)


def read_rc(c=None, table=P, R=3, W=4, stride=4, bs=16, off=P, start=None, n=5, out=P, ot=1, ts=2048, hs=128,
            status=P, **kw):
    return _lib.load().bpe_cache_read(cache(**kw) if c is None else None, table, R, W, stride, bs, off, start,
                                      n, out, ot, ts, hs, status, None)


BAD_CACHE = [dict(codes=None), dict(scales=None), dict(n_slots=-1), dict(codes_stride=2047),
             dict(scales_stride=15), dict(heads=0), dict(dim=0), dict(dim=1025), dict(heads=1025), dict(group=8),
             dict(group=48), dict(group=1024), dict(format=3), dict(codes_stride=(1 << 22) + 1),
             dict(format=2, scales_stride=31), dict(n_slots=(1 << 40) + 1)]


@pytest.mark.parametrize("bad", BAD_CACHE + [
    dict(c=0), dict(x=None), dict(slots=None), dict(status=None), dict(xt=3), dict(n=-1), dict(ts=2047), dict(hs=127),
    dict(n=1 << 28), dict(ts=(1 << 32) + 1)])
def test_cache_write_refuses(bad):
    assert write_rc(**bad) == EINVAL


@pytest.mark.parametrize("bad", BAD_CACHE + [
    dict(c=0), dict(table=None), dict(off=None), dict(out=None), dict(status=None), dict(R=-1), dict(W=-1),
    dict(W=1 << 31, stride=1 << 31), dict(stride=3), dict(bs=0), dict(n=-1), dict(ot=-1), dict(ts=2047),
    dict(n=1 << 28), dict(R=(1 << 30) + 1)])
def test_cache_read_refuses(bad):
    assert read_rc(**bad) == EINVAL


def test_cache_of_nothing():
    assert write_rc(n=0, x=None, slots=None) == _lib.BPE_OK
    assert read_rc(n=0, out=None) == _lib.BPE_OK
    assert read_rc(R=0, table=None, off=None) == _lib.BPE_OK


def verify_rc(target=P, pt=0, N=9, V=100, ps=100, draft=P, qs=100, ids=P, off=P, R=3, accept=P, sample=P,
              tokens=P, counts=P, ws=None, ws_bytes=0, status=P):
    return _lib.load().bpe_verify_drafts(target, pt, N, V, ps, draft, qs, ids, off, R, accept, sample, tokens,
                                         counts, ws, ws_bytes, status, None)


@pytest.mark.parametrize("bad", [
    dict(target=None), dict(ids=None), dict(off=None), dict(accept=None), dict(sample=None), dict(tokens=None),
    dict(counts=None), dict(status=None), dict(pt=3), dict(N=-1), dict(V=0), dict(V=_lib.MAX_ROWS + 1, ps=1 << 28),
    dict(ps=99), dict(qs=99), dict(R=-1), dict(R=1 << 20), dict(N=(1 << 30) + 1)])
def test_verify_refuses(bad):
    assert verify_rc(**bad) == EINVAL


def test_verify_workspace():
    assert lm.verify_drafts_workspace_bytes(1000, 768) == 0
    assert lm.verify_drafts_workspace_bytes(0, 50000) == 0
    assert lm.verify_drafts_workspace_bytes(256, 65536) == 0
    big = dict(V=70000, ps=70000, qs=70000)
    need = lm.verify_drafts_workspace_bytes(3, 70000)
    assert 0 < need <= 3 * (8 * 70000 / 512 + 40)
    assert verify_rc(**big, ws=P, ws_bytes=need - 1) == _lib.BPE_EWORKSPACE
    assert verify_rc(**big, ws=None, ws_bytes=need) == EINVAL
    assert verify_rc(**big, ws=P + 4, ws_bytes=need) == EINVAL
    # the limit of the launch
    R, V = 1 << 16, 1 << 21
    assert verify_rc(V=V, ps=V, qs=V, R=R, ws=P, ws_bytes=1 << 50) == EINVAL
    assert verify_rc(V=V, ps=V, qs=V, R=R - 1, ws=P, ws_bytes=0) == _lib.BPE_EWORKSPACE
    assert verify_rc(V=_lib.MAX_ROWS, ps=_lib.MAX_ROWS, qs=_lib.MAX_ROWS, R=R, ws=P, ws_bytes=1 << 50) == EINVAL


def test_verify_of_nothing():
    assert verify_rc(N=0, R=0, target=None, ids=None, off=None, accept=None, sample=None, tokens=None,
                     counts=None) == _lib.BPE_OK


def distill_rc(student=P, st=1, N=9, V=100, ss=100, ids=P, is_=5, teacher=P, tt=0, ts=5, K=5, T=1.0, losses=P,
               stats=P, status=P):
    return _lib.load().bpe_distill(student, st, N, V, ss, ids, is_, teacher, tt, ts, K, T, losses, stats, status, None)


def grad_rc(student=P, st=1, N=9, V=100, ss=100, ids=P, is_=5, teacher=P, tt=0, ts=5, K=5, stats=P, dloss=P,
            T=1.0, grad=2 * P, gt=1, gs=100, status=P):
    return _lib.load().bpe_distill_grad(student, st, N, V, ss, ids, is_, teacher, tt, ts, K, stats, dloss, T, grad,
                                        gt, gs, status, None)


BAD_ROWS = [dict(student=None), dict(ids=None), dict(teacher=None), dict(status=None), dict(st=3), dict(tt=-1),
            dict(N=-1), dict(N=1 << 24), dict(V=0), dict(V=_lib.MAX_ROWS + 1, ss=1 << 28), dict(ss=99),
            dict(is_=4), dict(ts=4), dict(K=1025, is_=2000, ts=2000), dict(K=-1), dict(T=0.0), dict(T=-1.0),
            dict(T=float("nan")), dict(T=float("inf")), dict(T=2.0 ** -21), dict(T=2.0 ** 21), dict(stats=None)]


@pytest.mark.parametrize("bad", BAD_ROWS + [dict(losses=None)])
def test_distill_refuses(bad):
    assert distill_rc(**bad) == EINVAL


@pytest.mark.parametrize("bad", BAD_ROWS + [
    dict(dloss=None), dict(grad=None), dict(gt=7), dict(gs=99), dict(grad=P, gt=0), dict(grad=P, gs=101),
    dict(N=1 << 21, V=1 << 20, ss=1 << 20, gs=1 << 20)])
def test_distill_grad_refuses(bad):
    assert grad_rc(**bad) == EINVAL


def test_distill_of_nothing():
    assert distill_rc(N=0, student=None, ids=None, teacher=None, losses=None, stats=None) == _lib.BPE_OK
    assert grad_rc(N=0, student=None, ids=None, teacher=None, stats=None, dloss=None, grad=None) == _lib.BPE_OK


# ---- the binding ---------------------------------------------------------------------
def c8(S=6, H=2, D=32, dtype=F8):
    return z(S, H, D, dtype=U8).view(dtype)


def read(codes=None, scales=None, group=32, table=None, bs=4, off=None, n=3, **kw):
    return lm.cache_read(c8() if codes is None else codes, z(6, 2, 1) if scales is None else scales, group,
                         z(1, 2, dtype=I32) if table is None else table, bs,
                         z(2, dtype=I64) if off is None else off, n, **kw)


def verify(target=None, ids=None, off=None, accept=None, sample=None, **kw):
    return lm.verify_drafts(z(4, 50) if target is None else target, z(4, dtype=I32) if ids is None else ids,
                            z(3, dtype=I64) if off is None else off, z(4) if accept is None else accept,
                            z(2) if sample is None else sample, **kw)


@pytest.mark.parametrize("error,call", [
    (TypeError, lambda: lm.empty_cache(4, 2, 32, torch.float32, device="cpu")),
    (TypeError, lambda: lm.cache_write(z(3, 2, 32, dtype=I32), z(3, dtype=I64), c8(), z(6, 2, 1), 32)),
    (ValueError, lambda: lm.cache_write(z(3, 64), z(3, dtype=I64), c8(), z(6, 2, 1), 32)),
    (TypeError, lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I32), c8(), z(6, 2, 1), 32)),
    (ValueError, lambda: lm.cache_write(z(3, 2, 32), z(4, dtype=I64), c8(), z(6, 2, 1), 32)),
    (TypeError, lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), z(6, 2, 32), z(6, 2, 1), 32)),
    (TypeError, lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), c8(), z(6, 2, 1, dtype=torch.float16), 32)),
    (ValueError, lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), c8(D=31), z(6, 2, 1), 32)),
    (ValueError, lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), c8(H=3), z(6, 3, 1), 32)),
    (ValueError, lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), c8(), z(6, 2, 1), 16)),
    (ValueError, lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), c8(), z(5, 2, 1), 32)),
    (ValueError, lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), c8(), z(6, 2, 1), 0)),
    (ValueError, lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), c8(dtype=U8), z(6, 2, 1, 2), 32)),
    (ValueError, lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), c8(D=16, dtype=U8), z(6, 2, 1), 32)),
    (ValueError, lambda: lm.cache_write(z(3, 32, 2).transpose(1, 2), z(3, dtype=I64), c8(), z(6, 2, 1), 32)),
    (ValueError, lambda: lm.cache_write(z(1, 2, 32).expand(3, 2, 32), z(3, dtype=I64), c8(), z(6, 2, 1), 32)),
    (ValueError, lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), c8(S=1).expand(6, 2, 32), z(6, 2, 1), 32)),
    (ValueError, lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), c8(D=64)[..., ::2], z(6, 2, 1), 32)),
    (ValueError, lambda: read(codes=z(6, 64, dtype=U8).view(F8))),
    (TypeError, lambda: read(table=z(1, 2, dtype=I64))),
    (ValueError, lambda: read(table=z(2, dtype=I32))),
    (ValueError, lambda: read(off=z(3, dtype=I64))),
    (TypeError, lambda: read(off=z(2, dtype=I32))),
    (TypeError, lambda: read(start=z(1, dtype=I64))),
    (ValueError, lambda: read(start=z(2, dtype=I32))),
    (ValueError, lambda: read(bs=0)),
    (ValueError, lambda: read(n=-1)),
    (ValueError, lambda: read(out=z(3, 2, 31))),
    (ValueError, lambda: read(out=z(3, 2, 32), out_dtype=torch.float16)),
    (ValueError, lambda: read(out=z(1, 2, 32).expand(3, 2, 32))),
    (TypeError, lambda: read(out_dtype=torch.float64)),
    (ValueError, lambda: read(dim=30)),
    (TypeError, lambda: verify(target=z(4, 50, dtype=torch.float64))),
    (ValueError, lambda: verify(target=z(200))),
    (TypeError, lambda: verify(ids=z(4, dtype=I64))),
    (ValueError, lambda: verify(ids=z(3, dtype=I32))),
    (TypeError, lambda: verify(off=z(3, dtype=I32))),
    (ValueError, lambda: verify(off=z(0, dtype=I64))),
    (ValueError, lambda: verify(accept=z(3))),
    (ValueError, lambda: verify(sample=z(3))),
    (TypeError, lambda: verify(draft=z(4, 50, dtype=torch.float16))),
    (ValueError, lambda: verify(draft=z(4, 51))),
    (ValueError, lambda: verify(tokens=z(3, dtype=I32))),
    (TypeError, lambda: verify(counts=z(2, dtype=I64))),
    (ValueError, lambda: verify(workspace=z(4, 4).t())),
    (TypeError, lambda: lm.distill(z(3, 40, dtype=I32), z(3, 5, dtype=I32), z(3, 5))),
    (TypeError, lambda: lm.distill(z(3, 40), z(3, 5, dtype=I64), z(3, 5))),
    (ValueError, lambda: lm.distill(z(3, 40), z(3, 5, dtype=I32), z(3, 4))),
    (ValueError, lambda: lm.distill(z(3, 40), z(2, 5, dtype=I32), z(2, 5))),
    (ValueError, lambda: lm.distill(z(3, 40), z(3, 5, dtype=I32), z(3, 5), losses=z(2))),
    (ValueError, lambda: lm.distill(z(3, 40), z(3, 5, dtype=I32), z(3, 5), stats=z(3))),
    (ValueError, lambda: lm.distill(z(40, 3).t(), z(3, 5, dtype=I32), z(3, 5))),
    (ValueError, lambda: lm.distill_grad(z(3, 40), z(3, 5, dtype=I32), z(3, 5), z(3, 3), z(3))),
    (ValueError, lambda: lm.distill_grad(z(3, 40), z(3, 5, dtype=I32), z(3, 5), z(3, 4), z(1).expand(3))),
    (TypeError, lambda: lm.distill_grad(z(3, 40), z(3, 5, dtype=I32), z(3, 5), z(3, 4), z(3, dtype=torch.float16))),
    (ValueError, lambda: lm.distill_grad(z(3, 40), z(3, 5, dtype=I32), z(3, 5), z(3, 4), z(3), out=z(3, 41))),
])
def test_binding_refuses(error, call):
    with pytest.raises(error):
        call()


def leaf(*shape):
    return torch.zeros(*shape, requires_grad=True)


@pytest.mark.parametrize("call", [
    lambda: lm.cache_write(leaf(3, 2, 32), z(3, dtype=I64), c8(), z(6, 2, 1), 32),
    lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), c8(), leaf(6, 2, 1) * 1, 32),
    lambda: read(scales=leaf(6, 2, 1)),
    lambda: read(out=leaf(3, 2, 32) * 1),
    lambda: verify(target=leaf(4, 50)),
    lambda: verify(draft=leaf(4, 50)),
    lambda: verify(accept=leaf(4)),
    lambda: lm.distill(leaf(3, 40), z(3, 5, dtype=I32), z(3, 5)),
    lambda: lm.distill(z(3, 40), z(3, 5, dtype=I32), leaf(3, 5)),
    lambda: lm.distillation(leaf(3, 40), z(3, 5, dtype=I32), leaf(3, 5)),
    lambda: lm.distill_grad(leaf(3, 40), z(3, 5, dtype=I32), z(3, 5), z(3, 4), z(3)),
    lambda: lm.distill_grad(z(3, 40), z(3, 5, dtype=I32), z(3, 5), z(3, 4), leaf(3)),
])
def test_calls_without_a_gradient_refuse(call):
    with pytest.raises(RuntimeError, match="gives no gradient"):
        call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
@pytest.mark.parametrize("call", [
    read, verify, lambda: lm.distillation(leaf(3, 40), z(3, 5, dtype=I32), z(3, 5)),
    lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), c8(), z(6, 2, 1), 32),
    lambda: lm.cache_write(z(2, 3, 32).transpose(0, 1), z(3, dtype=I64), c8(), z(6, 2, 1), 32),
    lambda: lm.cache_write(z(3, 2, 33), z(3, dtype=I64), c8(D=17, dtype=U8), z(6, 2, 2, 2), 32)])
def test_binding_needs_a_gpu(call):
    with pytest.raises(RuntimeError, match="HIP device"):
        call()


@pytest.mark.parametrize("D,dtype,group,shape,scales", [
    (128, F8, 128, (5, 2, 128), (5, 2, 1)), (80, I8, 128, (5, 2, 80), (5, 2, 1)), (1, F8, 16, (5, 2, 1), (5, 2, 1)),
    (77, U8, 128, (5, 2, 39), (5, 2, 1, 2)), (1000, I8, 512, (5, 2, 1000), (5, 2, 2))])
def test_empty_cache(D, dtype, group, shape, scales):
    c, s, g = lm.empty_cache(5, 2, D, dtype, device="cpu")
    assert tuple(c.shape) == shape and tuple(s.shape) == scales and g == group and c.dtype == dtype


# ---- the references against the definitions, by hand --------------------------------
def test_reference_e4m3():
    y = np.array([0.0, 1.0, 1.0625, 1.1875, -448.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 0.9, 17.0, 433.0])
    want = torch.tensor(y).to(F8).double().numpy()
    assert np.array_equal(ref.e4m3(y), want)
    x = np.random.default_rng(0).uniform(-448, 448, 100000) * 2.0 ** np.random.default_rng(1).integers(-18, 1, 100000)
    x = x.astype(np.float32)
    assert np.array_equal(ref.e4m3(x), torch.tensor(x).to(F8).double().numpy())


def test_reference_quantise():
    x = np.array([[[1.1, -2.0, 0.5, np.nan, np.inf, 4.0, -np.inf, 0.0]]], np.float32)
    c, s, _ = ref.quantise(x, 16, "int8")
    assert c.tolist() == [[[35, -64, 16, 0, 127, 127, -127, 0]]] and abs(s[0, 0, 0] - 4 / 127) < 1e-8
    c, s, lo = ref.quantise(x, 16, "u4")
    assert c.tolist() == [[[8, 0, 6, 0, 15, 15, 0, 5]]] and lo.item() == -2 and abs(s.item() - 0.4) < 1e-7
    rng = np.random.default_rng(2)
    x = (rng.normal(size=(50, 3, 100)) * 2.0 ** rng.integers(-30, 30, (50, 3, 1))).astype(np.float32)
    for kind in ref.TOP:
        for group in (16, 32, 128):
            c, s, lo = ref.quantise(x, group, kind)
            s4 = np.stack((s, lo), -1) if kind == "u4" else s
            v, _ = ref.values(c, s4, group, kind == "u4")
            assert np.all(np.abs(v - x) <= ref.quantise_error(x, group, kind)), (kind, group)


def test_reference_verify():
    p = np.array([[0.5, 0.25, 0.25], [0.125, 0.375, 0.5], [0.25, 0.25, 0.5]])
    q = np.array([[0.25, 0.5, 0.25], [0.5, 0.25, 0.25], [9.0, 9.0, 9.0]])
    run = lambda ids, acc, u: [x.tolist() for x in ref.verify(p, ids, [0, 3], acc, [u], q)]  # noqa: E731
    assert run([0, 2, 7], [0.99, 0.99, 0], 0.5) == [[0, 2, 2], [3]]     # 0.5 of 1: past 0.25 + 0.25
    assert run([0, 2, 7], [0.99, 0.99, 0], 0.49) == [[0, 2, 1], [3]]
    assert run([0, 0, 7], [0.99, 0.25, 0], 0.3) == [[0, 1, -1], [2]]    # 0.25 * 0.5 is not below 0.125
    assert run([0, 0, 7], [0.99, 0.2499, 0], 0.1) == [[0, 0, 0], [3]]
    assert run([1, 0, 7], [0.5, 0.0, 0], 0.9) == [[0, -1, -1], [1]]
    t, c = ref.verify(p[:1], [5], [0, 1], [0], [0.6])
    assert t.tolist() == [1] and c.tolist() == [1]
    t, c = ref.verify(p[:2], [1, 0], [0, 2], [0.25, 0], [0.6])          # certain: 1 is taken out
    assert t.tolist() == [0, -1] and c.tolist() == [1]


def test_reference_distill_gradient():
    """The gradient's formula against differences of the loss."""
    rng = np.random.default_rng(3)
    z, t = rng.normal(size=(6, 30)) * 2, rng.normal(size=(6, 5)) * 2
    ids = np.stack([rng.choice(30, 5, replace=False) for _ in range(6)])
    ids[1, 2] = -1
    ids[2] = -1
    ids[3, 1] = ids[3, 4]  # one token twice
    d, dl = rng.normal(size=(6, 30)), rng.normal(size=6)
    for T in (1.0, 2.5, 0.4):
        _, _, g, _ = ref.distill(z, ids, t, T, dl)
        e = 1e-6
        up, down = (ref.distill(z + s * e * d, ids, t, T)[0] for s in (1, -1))
        assert abs(((up - down) / (2 * e) * dl).sum() - (g * d).sum()) < 1e-6 * max(1, np.abs(g).sum())
        assert np.all(g[2] == 0) and ref.distill(z, ids, t, T)[0][2] == 0
        # against torch, and no loss where the student agrees
        lp = torch.log_softmax(torch.tensor(z[0] / T), 0)[torch.tensor(ids[0])]
        P = torch.softmax(torch.tensor(t[0] / T), 0)
        want = T * T * float((P * (P.log() - lp)).sum())
        assert abs(ref.distill(z, ids, t, T)[0][0] - want) < 1e-12 * max(1, abs(want))
    full = np.arange(30)[None].repeat(6, 0)
    assert np.all(np.abs(ref.distill(z, full, z, 1.7)[0]) < 1e-14)
