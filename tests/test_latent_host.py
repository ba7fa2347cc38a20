"""Latent attention on the host: what the C ABI and the binding refuse, before any CUDA call."""
import ctypes

import pytest
import torch

import linear_attention_06_gb300 as kda
from linear_attention_06_gb300 import _lib
from linear_attention_06_gb300 import build as kbuild

FAKE, MIS = 0x10000, 0x10008            # never dereferenced; MIS is not 16-byte aligned
OK, ARG, UNS = _lib.KDA_OK, _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return _lib.lib()


def shape(n=2, T=2, H=4, latent=512, rope=64, page=64, pages=8, per=4, dtype=_lib.KDA_BF16):
    return ctypes.byref(_lib.KdaLatentShape(n, T, H, latent, rope, page, pages, per, dtype))


def append(L, sh=None, lat=FAKE, lat_s=512, kr=FAKE, kr_s=64, freq=FAKE, inter=0, q=FAKE, q_s=64, qo=FAKE, qo_s=64,
           cu=None, lens=FAKE, table=FAKE, cache=FAKE):
    return L.kda_latent_append(shape() if sh is None else sh, lat, lat_s, kr, kr_s, freq, inter, q, q_s, qo, qo_s, cu,
                               lens, table, cache, None)


def gather(L, sh=None, cache=FAKE, table=FAKE, cu=FAKE, starts=None, lat=FAKE, kr=FAKE):
    return L.kda_latent_gather(shape() if sh is None else sh, cache, table, cu, starts, lat, kr, None)


def decode(L, sh=None, q=FAKE, qr=FAKE, cache=FAKE, table=FAKE, lens=FAKE, scale=1.0, out=FAKE, lse=None, ws=FAKE,
           size=1 << 40):
    return L.kda_latent_decode(shape() if sh is None else sh, q, qr, cache, table, lens, scale, out, lse, ws, size, None)


def prefill(L, n=2, T=4, H=3, dk=192, dv=128, dt=_lib.KDA_BF16, S=4, q=FAKE, k=FAKE, v=FAKE, step=128, kr=FAKE,
            scale=1.0, cu=None, ck=None, out=FAKE, lse=None, null=False):
    sh = None if null else ctypes.byref(_lib.KdaShape(n, T, H, dk, dv, dt))
    return L.kda_latent_prefill(sh, S, q, k, v, step, kr, scale, cu, ck, out, lse, None)


BAD_SHAPES = [(dict(n=-1), ARG), (dict(T=-1), ARG), (dict(H=0), ARG), (dict(latent=0), ARG), (dict(rope=-1), ARG),
              (dict(page=0), ARG), (dict(pages=-1), ARG), (dict(per=-1), ARG), (dict(latent=256), UNS),
              (dict(rope=32), UNS), (dict(page=8), UNS), (dict(page=48), UNS), (dict(page=2048), UNS),
              (dict(H=1025), UNS), (dict(dtype=_lib.KDA_F32), UNS), (dict(dtype=9), UNS),
              (dict(pages=2 ** 31 - 1), UNS), (dict(per=2 ** 30), UNS)]


@pytest.mark.parametrize("kw,code", BAD_SHAPES)
def test_shapes_refused_by_every_call(L, kw, code):
    assert append(L, shape(**kw)) == code
    assert gather(L, shape(**kw)) == code
    assert decode(L, shape(**kw)) == code
    size = ctypes.c_size_t(5)
    assert L.kda_latent_decode_workspace_size(shape(**kw), ctypes.byref(size)) == code and size.value == 0


def test_null_shape(L):
    for f in (append, gather, decode):
        assert f(L, ctypes.POINTER(_lib.KdaLatentShape)()) == ARG
    assert prefill(L, null=True) == ARG
    assert L.kda_latent_decode_workspace_size(shape(), None) == ARG


def test_append_refusals(L):
    for kw in (dict(lat=None), dict(kr=None), dict(lens=None), dict(table=None), dict(cache=None), dict(qo=None),
               dict(lat_s=511), dict(kr_s=63), dict(q_s=0), dict(qo_s=8), dict(inter=2), dict(sh=shape(n=3, T=4)),
               dict(sh=shape(n=0, T=4)), dict(sh=shape(rope=0))):
        assert append(L, **kw) == ARG, kw
    for kw in (dict(lat=MIS), dict(kr=MIS), dict(q=MIS), dict(qo=MIS), dict(cache=MIS), dict(table=FAKE + 2),
               dict(lens=FAKE + 1), dict(freq=FAKE + 2), dict(cu=FAKE + 2), dict(lat_s=513), dict(kr_s=65),
               dict(q_s=68), dict(qo_s=67), dict(sh=shape(T=2 ** 31))):
        assert append(L, **kw) == UNS, kw
    assert append(L, shape(n=0, T=0), lat=None, lens=None, cache=None, table=None) == OK
    assert append(L, shape(T=0), lat=None) == OK


def test_gather_refusals(L):
    for kw in (dict(lat=None), dict(kr=None), dict(table=None), dict(cache=None), dict(sh=shape(n=0)),
               dict(sh=shape(T=3), cu=None)):
        assert gather(L, **kw) == ARG, kw
    for kw in (dict(lat=MIS), dict(kr=MIS), dict(cache=MIS), dict(table=FAKE + 1), dict(cu=FAKE + 2), dict(starts=FAKE + 2)):
        assert gather(L, **kw) == UNS, kw
    assert gather(L, shape(T=0), lat=None, kr=None, cache=None) == OK


def test_decode_refusals(L):
    for kw in (dict(q=None), dict(qr=None), dict(cache=None), dict(table=None), dict(lens=None), dict(out=None),
               dict(ws=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(sh=shape(n=4, T=6)), dict(sh=shape(T=0)), dict(sh=shape(n=0, T=2)), dict(size=0)):
        assert decode(L, **kw) == ARG, kw
    for kw in (dict(q=MIS), dict(qr=MIS), dict(cache=MIS), dict(out=MIS), dict(lse=FAKE + 2), dict(table=FAKE + 3),
               dict(lens=FAKE + 2), dict(ws=FAKE + 128), dict(sh=shape(n=2, T=34)), dict(sh=shape(n=2 ** 22, T=2 ** 22, H=512))):
        assert decode(L, **kw) == UNS, kw
    assert decode(L, shape(n=0, T=0), q=None, qr=None, cache=None, ws=None) == OK


def test_decode_workspace(L):
    for T, H in ((1, 1), (1, 32), (16, 32), (1, 128), (16, 1024)):
        size = kda.kda_latent_decode_workspace_size(3, 3 * T, H)
        assert 0 < size <= 48 << 20
        sh = shape(n=3, T=3 * T, H=H)
        assert decode(L, sh, size=size - 1) == ARG
        assert size == kda.kda_latent_decode_workspace_size(1000, 1000 * T, H, rope_dim=0)
    assert kda.kda_latent_decode_workspace_size(0, 0, 4) == 0


def test_prefill_refusals(L):
    for kw in (dict(n=-1), dict(T=-1), dict(H=0), dict(S=-1), dict(n=0), dict(n=3), dict(n=3, cu=FAKE), dict(S=5),
               dict(q=None), dict(k=None), dict(v=None), dict(kr=None), dict(out=None), dict(step=120),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert prefill(L, **kw) == ARG, kw
    for kw in (dict(dk=64), dict(dk=160), dict(dv=64), dict(dt=_lib.KDA_F32), dict(H=1025), dict(q=MIS), dict(k=MIS),
               dict(v=MIS), dict(kr=MIS), dict(out=MIS), dict(lse=FAKE + 2), dict(cu=FAKE + 1), dict(ck=FAKE + 2),
               dict(step=132), dict(T=2 ** 31), dict(S=2 ** 31), dict(T=2 ** 31 - 2, H=1024)):
        assert prefill(L, **kw) == UNS, kw
    assert prefill(L, T=0, q=None, out=None) == OK
    assert prefill(L, n=0, T=0, S=0, q=None, k=None, v=None, kr=None, out=None) == OK


def test_valid_calls_without_a_gpu_report_a_cuda_error(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for f in (append, gather, decode, prefill):
        assert f(L) == _lib.KDA_ERR_CUDA


def test_binding_refuses_cpu_tensors(L):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    t = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_latent_append(z(1, 512), z(1, 64), z(1, 16, 576), t, t[0])
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_latent_decode(z(1, 1, 512), z(1, 1, 64), z(1, 16, 576), t, t[0], 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_latent_prefill(z(1, 1, 192), z(1, 1, 128), z(1, 1, 128), z(1, 64), 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_latent_gather(z(1, 16, 576), t, [0, 1], 1)


@pytest.mark.parametrize("t,step", [
    (torch.zeros(4, 3, 64), 64), (torch.zeros(4, 3, 192)[..., 128:], 192), (torch.zeros(1, 1, 64), 64),
    (torch.zeros(5, 576)[:, 512:], 576), (torch.zeros(4, 6, 64)[:, 2:3], 384), (torch.zeros(1, 3, 192)[..., :64], 192)])
def test_row_strides_read_from_a_tensor(L, t, step):
    assert _lib._latent().row_stride("t", t) == step


@pytest.mark.parametrize("t", [torch.zeros(4, 6, 64)[:, ::2][:, :2], torch.zeros(3, 4, 64).transpose(0, 1),
                               torch.zeros(4, 3, 128)[..., ::2], torch.zeros(1, 64).expand(4, 64)])
def test_rows_that_are_not_evenly_spaced_are_refused(L, t):
    with pytest.raises(ValueError):
        _lib._latent().row_stride("t", t)


def test_a_stream_of_another_device_is_refused():
    class Stream:
        cuda_stream, device = FAKE, torch.device("cuda", 1)
    t = torch.zeros(2, 16, 576, dtype=torch.bfloat16)
    i = torch.zeros(1, 2, dtype=torch.int32)
    for call in (lambda: kda.kda_latent_append(t[0, :1, :512], t[0, :1, 512:], t, i, i[0, :1], stream=Stream()),
                 lambda: kda.kda_latent_gather(t, i, [0, 1], 1, stream=Stream()),
                 lambda: kda.kda_latent_decode(t[:1, :4, :512], t[:1, :4, 512:], t, i, i[0, :1], 1.0, stream=Stream()),
                 lambda: kda.kda_latent_prefill(t[:, :, :192], t[:, :, :128], t[:, :, :128], t[0, :2, :64], 1.0,
                                                stream=Stream())):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()
