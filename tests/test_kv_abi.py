"""The tpla_kv_* entry points refuse bad calls before touching a GPU, with the
documented status; the Python calls raise the module's exceptions.  CPU only:
descriptors with made-up addresses that are never read."""
import ctypes

import pytest
import torch

import mla_latent_kv_dim_b200 as tp
from mla_latent_kv_dim_b200 import _native as N

BF, F32, I32, F16 = 1, 2, 3, 4


def _t(shape, dtype=BF, ptr=0x10000, stride=None):
    d = N.TplaTensor()
    d.data, d.dtype, d.ndim = ptr, dtype, len(shape)
    st = 1
    for i in reversed(range(len(shape))):
        d.shape[i] = shape[i]
        d.stride[i] = stride[i] if stride else st
        st *= shape[i]
    return d


def _p(d):
    return None if d is None else ctypes.byref(d)


def _append(**ch):
    a = dict(k=_t((3, 2, 64)), v=_t((3, 2, 64)), pos=_t((3,), I32), req=_t((3,), I32),
             pt=_t((4, 5), I32), kc=_t((9, 64, 2, 64)), vc=_t((9, 64, 2, 64)),
             cs=_t((300, 64), F32), off=0, inter=0, q=_t((3, 4, 64)), qo=_t((3, 4, 64), ptr=0x90000),
             qoff=0)
    a.update(ch)
    return tp.lib().tpla_kv_append(_p(a["k"]), _p(a["v"]), _p(a["pos"]), _p(a["req"]), _p(a["pt"]),
                                   _p(a["kc"]), _p(a["vc"]), _p(a["cs"]), a["off"], a["inter"],
                                   _p(a["q"]), _p(a["qo"]), a["qoff"], None)


INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -4


@pytest.mark.parametrize("want,ch", [
    (INVALID, dict(k=None)), (INVALID, dict(kc=None)), (INVALID, dict(pos=None)),
    (INVALID, dict(k=_t((3, 2, 64), F16))),                 # not the cache's type
    (INVALID, dict(k=_t((3, 2, 32)))), (INVALID, dict(k=_t((3, 1, 64)))),
    (INVALID, dict(v=None)), (INVALID, dict(vc=None)),      # one without the other
    (INVALID, dict(v=_t((2, 2, 64)))), (INVALID, dict(v=_t((3, 2, 64), F32))),
    (INVALID, dict(pos=_t((4,), I32))), (INVALID, dict(pos=_t((3,), I32, stride=(2,)))),
    (INVALID, dict(req=_t((2,), I32))),
    (INVALID, dict(req=None)),                              # three tokens, four requests
    (INVALID, dict(k=_t((3, 2, 64), ptr=0x10004))),
    (INVALID, dict(k=_t((3, 2, 64), stride=(130, 65, 1)))),
    (INVALID, dict(kc=_t((9, 64, 2, 64), stride=(0, 128, 64, 1)))),  # pages on one another
    (INVALID, dict(kc=_t((9, 64, 2, 64), F32))),
    (INVALID, dict(cs=_t((300, 72), F32))), (INVALID, dict(cs=_t((300, 64)))),
    (INVALID, dict(cs=_t((300, 128), F32))),                # more columns than the key has
    (INVALID, dict(off=4)), (INVALID, dict(off=8)), (INVALID, dict(off=-8)),
    (INVALID, dict(inter=2)), (INVALID, dict(qoff=8)), (INVALID, dict(qo=None)),
    (INVALID, dict(q=None)), (INVALID, dict(cs=None)),      # queries without a table
    (INVALID, dict(qo=_t((3, 4, 64), F32, ptr=0x90000))), (INVALID, dict(qo=_t((3, 2, 64)))),
    (INVALID, dict(q=_t((3, 4, 64), F32), qo=_t((3, 4, 64)))),      # in place, other type
    (INVALID, dict(qo=_t((3, 4, 64), ptr=0x10000, stride=(512, 64, 1)))),  # in place, other rows
    (UNSUPPORTED, dict(kc=_t((9, 32, 2, 64)), vc=_t((9, 32, 2, 64)))),
    (UNSUPPORTED, dict(pt=_t((4, 1 << 25), I32))),
])
def test_append_refusals(want, ch):
    assert _append(**ch) == want
    assert tp.launch_count() == 0


def _decode(sizes=False, **ch):
    a = dict(q=_t((4, 8, 128)), k=_t((9, 64, 2, 128)), v=_t((9, 64, 2, 128)), seq=_t((4,), I32),
             pt=_t((4, 5), I32), scale=0.1, out=_t((4, 8, 128), F32), lse=_t((4, 8, 1), F32),
             ws=None, bytes=0)
    a.update(ch)
    return tp.lib().tpla_kv_decode(_p(a["q"]), _p(a["k"]), _p(a["v"]), _p(a["seq"]), _p(a["pt"]),
                                   a["scale"], _p(a["out"]), _p(a["lse"]), a["ws"], a["bytes"],
                                   None)


@pytest.mark.parametrize("want,ch", [
    (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(v=None)),
    (INVALID, dict(seq=None)), (INVALID, dict(out=None)),
    (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=float("inf"))),
    (INVALID, dict(q=_t((4, 7, 128)))), (INVALID, dict(q=_t((3, 8, 128)))),
    (INVALID, dict(q=_t((4, 8, 128), F16))), (INVALID, dict(q=_t((4, 8, 64)))),
    (INVALID, dict(v=_t((9, 64, 2, 128), F16))), (INVALID, dict(v=_t((8, 64, 2, 128)))),
    (INVALID, dict(v=_t((9, 64, 1, 128)))),
    (INVALID, dict(seq=_t((5,), I32))), (INVALID, dict(seq=_t((4,), F32))),
    (INVALID, dict(pt=_t((3, 5), I32))), (INVALID, dict(pt=None)),
    (INVALID, dict(out=_t((4, 8, 64), F32))), (INVALID, dict(out=_t((4, 8, 128), F16))),
    (INVALID, dict(out=_t((4, 8, 128), ptr=0x10008))), (INVALID, dict(lse=_t((4, 8), F32))),
    (INVALID, dict(out=_t((4, 8, 128), F32, stride=(1024, 0, 1)))),
    (INVALID, dict(k=_t((9, 64, 2, 128), stride=(16384, 256, 0, 1)))),
    (INVALID, dict(k=_t((9, 64, 2, 128), stride=(16384, 257, 128, 1)))),
    (UNSUPPORTED, dict(k=_t((9, 32, 2, 128)), v=_t((9, 32, 2, 128)))),
    (UNSUPPORTED, dict(q=_t((4, 8, 96)), k=_t((9, 64, 2, 96)), v=_t((9, 64, 2, 96)),
                       out=_t((4, 8, 96), F32))),
    (UNSUPPORTED, dict(v=_t((9, 64, 2, 64)), out=_t((4, 8, 64), F32))),
    (UNSUPPORTED, dict(k=_t((9, 64, 2, 128), stride=(1 << 39, 256, 128, 1)))),
    (UNSUPPORTED, {}),  # a good call on a machine without a GPU
])
def test_decode_refusals(want, ch):
    if ch == {} and torch.cuda.is_available():
        pytest.skip("the call would run")
    assert _decode(**ch) == want
    assert tp.launch_count() == 0


def _prefill(**ch):
    a = dict(q=_t((30, 8, 128)), k=_t((30, 2, 128)), v=_t((30, 2, 128)), cq=_t((4,), I32), ck=None,
             seq=None, pt=None, causal=1, scale=0.1, out=_t((30, 8, 128), F32),
             lse=_t((30, 8, 1), F32), ws=None, bytes=0)
    a.update(ch)
    return tp.lib().tpla_kv_prefill(_p(a["q"]), _p(a["k"]), _p(a["v"]), _p(a["cq"]), _p(a["ck"]),
                                    _p(a["seq"]), _p(a["pt"]), a["causal"], a["scale"],
                                    _p(a["out"]), _p(a["lse"]), a["ws"], a["bytes"], None)


PAGED = dict(k=_t((9, 64, 2, 128)), v=_t((9, 64, 2, 128)), seq=_t((3,), I32), pt=_t((3, 5), I32))


@pytest.mark.parametrize("want,ch", [
    (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(cq=None)),
    (INVALID, dict(cq=_t((0,), I32))), (INVALID, dict(cq=_t((4,), I32, stride=(2,)))),
    (INVALID, dict(causal=2)), (INVALID, dict(scale=float("nan"))),
    (INVALID, dict(ck=_t((3,), I32))), (INVALID, dict(seq=_t((3,), I32))),
    (INVALID, dict(k=_t((31, 2, 128)))), (INVALID, dict(k=_t((30, 3, 128)), v=_t((30, 3, 128)))),
    (INVALID, dict(k=_t((30, 2, 128), F16))), (INVALID, dict(q=_t((30, 8, 64)))),
    (INVALID, dict(out=_t((29, 8, 128), F32))), (INVALID, dict(lse=_t((30, 8, 2), F32))),
    (INVALID, dict(q=_t((30, 8, 128), stride=(1024, 0, 1)))),
    (INVALID, dict(PAGED, seq=None)), (INVALID, dict(PAGED, seq=_t((4,), I32))),
    (INVALID, dict(PAGED, pt=_t((2, 5), I32))), (INVALID, dict(PAGED, ck=_t((4,), I32))),
    (UNSUPPORTED, dict(q=_t((30, 8, 80)), k=_t((30, 2, 80)), v=_t((30, 2, 80)),
                       out=_t((30, 8, 80), F32))),
    (UNSUPPORTED, dict(PAGED, k=_t((9, 16, 2, 128)), v=_t((9, 16, 2, 128)))),
    (UNSUPPORTED, {}),
])
def test_prefill_refusals(want, ch):
    if ch == {} and torch.cuda.is_available():
        pytest.skip("the call would run")
    assert _prefill(**ch) == want
    assert tp.launch_count() == 0


def test_workspace_sizes():
    L, n = tp.lib(), ctypes.c_size_t(0)
    q, k, pt = _t((4, 8, 128)), _t((9, 64, 2, 128)), _t((4, 5), I32)
    assert L.tpla_kv_decode_workspace_size(_p(q), _p(k), _p(k), _p(pt), ctypes.byref(n)) == 0
    # 4 requests x 2 heads x (5 pages + 3) units, two slots each of 4 rows
    assert n.value >= 2 * 64 * 4 * 129 * 4
    assert L.tpla_kv_decode_workspace_size(_p(q), _p(k), None, _p(pt), ctypes.byref(n)) == INVALID
    cu = _t((2,), I32)
    size = L.tpla_kv_prefill_workspace_size
    short = _t((77, 2, 128))
    assert size(_p(_t((77, 8, 128))), _p(short), _p(short), _p(cu), None, ctypes.byref(n)) == 0
    assert n.value == 0  # one short prompt needs none
    assert size(_p(q), _p(k), _p(k), _p(cu), _p(_t((1, 500), I32)), ctypes.byref(n)) == 0
    assert n.value > 0   # few tokens against many keys: pieces
    assert size(_p(q), _p(k), _p(k), _p(cu), None, ctypes.byref(n)) == INVALID
    assert size(None, _p(k), _p(k), _p(cu), None, ctypes.byref(n)) == INVALID


def test_python_checks():
    b = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((1, 64, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros((1,), dtype=torch.int32)
    t = torch.zeros((1, 1), dtype=torch.int32)
    for call in (lambda: tp.kv_append(b, b, i, t, c, c), lambda: tp.kv_decode(b, c, c, i, t, 0.1),
                 lambda: tp.kv_prefill(b, b, b, i, scale=0.1)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()
    with pytest.raises(ValueError, match="scale"):
        tp.kv_decode(b, c, c, i, t)
    with pytest.raises(ValueError, match="scale"):
        tp.kv_prefill(b, b, b, i)
    with pytest.raises(TypeError):
        tp.kv_decode([1.0], c, c, i, t, scale=0.1)
    assert tp.launch_count() == 0
