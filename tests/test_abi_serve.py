"""Refusals of append, prefill, beam selection and page reordering, on the host
before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd

PTR = 0x100000
ARG, UNSUPPORTED, ALIGN, WORKSPACE = fd.FD_ERR_ARG, fd.FD_ERR_UNSUPPORTED, fd.FD_ERR_ALIGN, fd.FD_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def L():
    fdbuild.build()
    return fd.lib()


def fake(shape, dtype=fd.FD_BF16, strides=None, ptr=PTR):
    t = fd.FdTensor()
    t.data, t.dtype, t.ndim = ptr, dtype, len(shape)
    if strides is None:
        strides, acc = [], 1
        for s in reversed(shape):
            strides.insert(0, acc)
            acc *= s
    for i, (s, st) in enumerate(zip(shape, strides)):
        t.shape[i], t.stride[i] = s, st
    return t


def ref(x):
    return ctypes.byref(x) if isinstance(x, ctypes.Structure) else x


def opts(**kw):
    o = fd.FdOpts()
    for k, v in kw.items():
        setattr(o, k, v)
    return o


def cache(int8=False, **kw):
    t = fd.FD_I8 if int8 else fd.FD_BF16
    a = dict(k=fake((2, 2, 64, 128), t), v=fake((2, 2, 64, 128), t), ks=fake((2, 2, 64), fd.FD_F32) if int8 else None,
             vs=fake((2, 2, 64), fd.FD_F32) if int8 else None, table=None, max_pages=0)
    a.update(kw)
    return a


def append(int8=False, **kw):
    c = cache(int8)
    a = dict(kn=fake((2, 3, 2, 128)), vn=fake((2, 3, 2, 128)), new=None, q=fake((2, 3, 8, 128)),
             q_out=fake((2, 3, 8, 128), ptr=0x900000), rope=fake((64, 128), fd.FD_F32), inter=0, **c, lens=PTR, after=None, o=opts())
    assert set(kw) <= set(a)
    a.update(kw)
    return fd.lib().fd_append(*(ref(x) for x in a.values()))


def prefill(int8=False, **kw):
    a = dict(q=fake((2, 9, 8, 128)), **cache(int8), lens=PTR, new=None, causal=1, scale=0.1, out=fake((2, 9, 8, 128)), o=opts())
    assert set(kw) <= set(a)
    a.update(kw)
    return fd.lib().fd_prefill(*(ref(x) for x in a.values()))


def select(**kw):
    a = dict(logits=fake((2, 4, 1000), fd.FD_F32), scores=PTR, fin=None, end=-1, n=8, so=PTR, bo=PTR, to=PTR, o=opts())
    assert set(kw) <= set(a)
    a.update(kw)
    return fd.lib().fd_beam_select(*(ref(x) for x in a.values()))


def reorder(**kw):
    a = dict(table=PTR, B=4, mp=8, lens=PTR, page=16, refs=PTR, pages=40, src=PTR, o=opts())
    a.update(kw)
    return fd.lib().fd_pages_reorder(*(ref(x) for x in a.values()))


@pytest.mark.parametrize("call", [append, prefill, lambda: append(True), lambda: prefill(True), select, reorder])
def test_good_arguments_want_only_a_workspace(call):
    assert call() == WORKSPACE


CACHES = [
    (dict(k=None), ARG), (dict(v=fake((2, 2, 64, 128), fd.FD_I8)), ARG), (dict(k=fake((2, 2, 64, 128), fd.FD_F32)), ARG),
    (dict(v=fake((2, 2, 65, 128))), ARG), (dict(ks=fake((2, 2, 64), fd.FD_F32)), ARG),
    (dict(k=fake((2, 2, 64, 128), strides=(16384, 8192, 128, 2))), ARG),
    (dict(k=fake((2, 2, 64, 128), ptr=PTR + 8)), ALIGN), (dict(v=fake((2, 2, 64, 128), strides=(16384, 8196, 128, 1))), ALIGN),
    (dict(k=fake((2, 2, 64, 96)), v=fake((2, 2, 64, 96))), UNSUPPORTED), (dict(table=PTR), ARG), (dict(max_pages=3), ARG),
    (dict(k=fake((3, 2, 64, 128)), v=fake((3, 2, 64, 128))), ARG), (dict(k=fake((2, 0, 64, 128)), v=fake((2, 0, 64, 128))), ARG),
    (dict(table=PTR, max_pages=1 << 26), UNSUPPORTED), (dict(lens=None), ARG),
]


@pytest.mark.parametrize("call", [append, prefill])
@pytest.mark.parametrize("i", range(len(CACHES)))
def test_caches(call, i):
    kw, code = CACHES[i]
    assert call(**kw) == code


@pytest.mark.parametrize("call", [append, prefill])
def test_int8_caches(call):
    assert call(True, ks=None) == ARG and call(True, vs=fake((2, 2, 63), fd.FD_F32)) == ARG
    assert call(True, vs=fake((2, 2, 64), fd.FD_BF16)) == ARG and call(True, ks=fake((2, 2, 64), fd.FD_F32, ptr=PTR + 2)) == ALIGN
    assert call(True, k=fake((2, 2, 64, 128), fd.FD_I8, strides=(16384, 8192, 120, 1))) == ALIGN
    pools = {x: fake((40, 2, 64, 128), fd.FD_I8) for x in "kv"}
    scales = {x: fake((40, 2, 64), fd.FD_F32) for x in ("ks", "vs")}
    assert call(True, table=PTR, max_pages=3, **pools, **scales) == WORKSPACE


OPTIONS = [dict(num_ctas=-1), dict(kernel=9), dict(wait_limit_us=-1), dict(wait_limit_us=3000000)]


@pytest.mark.parametrize("call", [append, prefill, select, reorder])
def test_options(call):
    assert call(o=None) == ARG
    for kw in OPTIONS:
        assert call(o=opts(**kw)) == ARG
    bad = opts()
    bad.reserved[1] = 1
    assert call(o=bad) == ARG
    for kernel in (fd.FD_KERNEL_SIMT, fd.FD_KERNEL_TC):
        assert call(o=opts(kernel=kernel)) == (WORKSPACE if call is prefill else ARG)


def test_append():
    for name in ("kn", "vn"):
        assert append(**{name: None}) == ARG and append(**{name: fake((2, 3, 2, 128), fd.FD_F32)}) == ARG
        assert append(**{name: fake((2, 3, 2, 128), ptr=PTR + 2)}) == ALIGN
        assert append(**{name: fake((2, 3, 2, 128), strides=(772, 256, 128, 1))}) == ALIGN
        assert append(**{name: fake((2, 3, 4, 128))}) == ARG and append(**{name: fake((2, 3, 2, 256))}) == ARG
        assert append(**{name: fake((2, 3, 256))}) == ARG
    assert append(kn=fake((2, 0, 2, 128)), vn=fake((2, 0, 2, 128))) == ARG
    assert append(q=None) == ARG and append(q_out=None) == ARG and append(q=None, q_out=None) == WORKSPACE
    assert append(q=fake((2, 3, 8, 64))) == ARG and append(q_out=fake((2, 3, 9, 128))) == ARG
    assert append(q=fake((2, 3, 8, 128), ptr=PTR + 8)) == ALIGN and append(q_out=fake((2, 3, 8, 128), ptr=PTR + 8)) == ALIGN
    assert append(q_out=fake((2, 3, 8, 128))) == WORKSPACE                       # q itself
    assert append(q_out=fake((2, 3, 8, 128), strides=(1024, 2048, 128, 1))) == ARG
    assert append(rope=None) == WORKSPACE and append(inter=2) == ARG
    assert append(rope=fake((64, 128))) == ARG and append(rope=fake((64, 144), fd.FD_F32)) == ARG
    assert append(rope=fake((64, 40), fd.FD_F32)) == UNSUPPORTED and append(rope=fake((0, 64), fd.FD_F32)) == ARG
    assert append(rope=fake((64, 64), fd.FD_F32, ptr=PTR + 4)) == ALIGN
    assert append(rope=fake((64, 64), fd.FD_F32, strides=(66, 1))) == ALIGN
    assert append(rope=fake((64, 64), fd.FD_F32, strides=(128, 2))) == ARG
    assert append(after=PTR) == WORKSPACE and append(after=PTR + 4) == ARG and append(after=PTR + 8) == WORKSPACE
    assert append(new=PTR + 64, after=PTR + 60) == ARG


def test_prefill():
    for name in ("q", "out"):
        assert prefill(**{name: None}) == ARG and prefill(**{name: fake((2, 9, 8, 128), fd.FD_F32)}) == ARG
        assert prefill(**{name: fake((2, 9, 8, 128), ptr=PTR + 4)}) == ALIGN
        assert prefill(**{name: fake((2, 9, 8, 128), strides=(9216, 1028, 128, 1))}) == ALIGN
        assert prefill(**{name: fake((2, 9, 8, 128), strides=(9216, 1024, 128, 2))}) == ARG
    assert prefill(out=fake((2, 9, 4, 128))) == ARG and prefill(q=fake((2, 9, 7, 128)), out=fake((2, 9, 7, 128))) == ARG
    assert prefill(q=fake((2, 0, 8, 128)), out=fake((2, 0, 8, 128))) == ARG
    assert prefill(q=fake((2, 9, 258, 128)), out=fake((2, 9, 258, 128))) == UNSUPPORTED
    assert prefill(causal=2) == ARG and prefill(scale=float("nan")) == ARG and prefill(scale=float("inf")) == ARG


def test_select():
    assert select(logits=None) == ARG and select(logits=fake((2, 4, 1000), fd.FD_I32)) == ARG
    assert select(logits=fake((8, 1000), fd.FD_F32)) == ARG and select(logits=fake((2, 4, 1000), fd.FD_F32, strides=(8000, 2000, 2))) == ARG
    assert select(logits=fake((2, 4, 1000), fd.FD_F32, ptr=PTR + 2)) == ALIGN
    assert select(logits=fake((2, 4, 1000), fd.FD_BF16, ptr=PTR + 2)) == WORKSPACE
    for name in ("scores", "so", "bo", "to"):
        assert select(**{name: None}) == ARG
    assert select(n=0) == ARG and select(n=65) == UNSUPPORTED
    assert select(logits=fake((2, 129, 1000), fd.FD_F32)) == UNSUPPORTED and select(logits=fake((1, 1, 1 << 24), fd.FD_F32)) == UNSUPPORTED
    assert select(logits=fake((2, 4, 0), fd.FD_F32)) == ARG
    assert select(fin=PTR) == ARG and select(fin=PTR, end=1000) == ARG and select(fin=PTR, end=999) == WORKSPACE
    for bad in ((0, 4, 10, 1), (1, 129, 10, 1), (1, 4, 1 << 24, 1), (1, 4, 10, 65)):
        assert fd.lib().fd_beam_scratch_bytes(*bad) == 0
    assert fd.lib().fd_beam_scratch_bytes(2, 4, 1000, 8) > 0


def test_reorder():
    for name in ("table", "lens", "refs", "src"):
        assert reorder(**{name: None}) == ARG
    for name in ("B", "mp", "page", "pages"):
        assert reorder(**{name: 0}) == ARG
    assert reorder(B=49153) == UNSUPPORTED and reorder(mp=1 << 30, page=4) == UNSUPPORTED


def test_the_binding_refuses_what_is_on_no_gpu():
    x = torch.zeros(1, 3, 2, 128, dtype=torch.bfloat16)
    lens = torch.zeros(1, dtype=torch.int32)
    c = torch.zeros(1, 2, 8, 128, dtype=torch.bfloat16)
    for call in (lambda: fd.append(x, x, c, c, lens), lambda: fd.prefill(x, c, c, lens),
                 lambda: fd.beam_select(torch.zeros(1, 2, 9), torch.zeros(1, 2), 3),
                 lambda: fd.pages_reorder(torch.zeros(1, 1, dtype=torch.int32), lens, lens, 16, lens)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fd.append(None, x, c, c, lens), lambda: fd.prefill(3, c, c, lens), lambda: fd.beam_select(None, None, 3)):
        with pytest.raises(TypeError):
            call()


def test_prefill_scratch():
    need = fd.lib().fd_prefill_scratch_bytes
    for bad in ((-1, 128), (65536, 128), (1, 64), (1, 0)):
        assert need(*bad) == 0
    # two slots of 256 rows (128 at d 256) and their two numbers a block
    assert need(3, 128) == 3 * 2 * 256 * 130 * 4 and need(3, 256) == 3 * 2 * 128 * 258 * 4
