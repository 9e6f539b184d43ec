"""Refusals of the 4-bit cache and page calls, on the host before any CUDA
call (no GPU needed): bad types, shapes, strides, alignment, factors, options
and missing workspaces, through the C ABI and through the binding."""
import ctypes

import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd

PTR = 0x100000


@pytest.fixture(scope="module", autouse=True)
def L():
    fdbuild.build()
    return fd.lib()


def fake(shape, dtype, strides=None, ptr=PTR):
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


def decode_args(**kw):
    a = dict(q=fake((2, 1, 8, 128), fd.FD_BF16), k=fake((2, 2, 64, 64), fd.FD_U8), v=fake((2, 2, 64, 64), fd.FD_U8),
             ks=fake((2, 2, 64, 8), fd.FD_E4M3), vs=fake((2, 2, 64, 8), fd.FD_E4M3), kg=1.0, vg=1.0, table=None,
             max_pages=0, lens=PTR, n_q=1, causal=0, scale=0.1, out=fake((2, 1, 8, 128), fd.FD_BF16), o=opts())
    a.update(kw)
    return [ref(x) for x in a.values()]


def append_args(**kw):
    a = dict(kn=fake((2, 3, 2, 128), fd.FD_BF16), vn=fake((2, 3, 2, 128), fd.FD_BF16), new=None,
             k=fake((2, 2, 64, 64), fd.FD_U8), v=fake((2, 2, 64, 64), fd.FD_U8),
             ks=fake((2, 2, 64, 8), fd.FD_E4M3), vs=fake((2, 2, 64, 8), fd.FD_E4M3), kg=1.0, vg=1.0, table=None,
             max_pages=0, lens=PTR, after=None, o=opts())
    a.update(kw)
    return [ref(x) for x in a.values()]


def read_args(**kw):
    a = dict(k=fake((2, 2, 64, 64), fd.FD_U8), v=fake((2, 2, 64, 64), fd.FD_U8),
             ks=fake((2, 2, 64, 8), fd.FD_E4M3), vs=fake((2, 2, 64, 8), fd.FD_E4M3), kg=1.0, vg=1.0, table=None,
             max_pages=0, start=None, lens=PTR, ko=fake((2, 5, 2, 128), fd.FD_BF16),
             vo=fake((2, 5, 2, 128), fd.FD_BF16), o=opts())
    a.update(kw)
    return [ref(x) for x in a.values()]


# with everything else in order the missing workspace is what is left to refuse
def test_only_the_workspace_is_missing(L):
    assert L.fd_decode_fp4(*decode_args()) == fd.FD_ERR_WORKSPACE
    assert L.fd_append_fp4(*append_args()) == fd.FD_ERR_WORKSPACE
    assert L.fd_read_fp4(*read_args()) == fd.FD_ERR_WORKSPACE


CACHE_FAULTS = [
    (dict(k=fake((2, 2, 64, 64), fd.FD_I8)), fd.FD_ERR_ARG),
    (dict(ks=fake((2, 2, 64, 8), fd.FD_U8)), fd.FD_ERR_ARG),
    (dict(v=fake((2, 2, 63, 64), fd.FD_U8)), fd.FD_ERR_ARG),
    (dict(vs=fake((2, 2, 64, 16), fd.FD_E4M3)), fd.FD_ERR_ARG),
    (dict(ks=fake((2, 2, 63, 8), fd.FD_E4M3)), fd.FD_ERR_ARG),
    (dict(k=fake((2, 2, 64, 64), fd.FD_U8, (16384, 8192, 128, 2))), fd.FD_ERR_ARG),
    (dict(k=fake((2, 2, 64, 64), fd.FD_U8, ptr=PTR + 8)), fd.FD_ERR_ALIGN),
    (dict(v=fake((2, 2, 64, 64), fd.FD_U8, (8192, 4096, 72, 1))), fd.FD_ERR_ALIGN),
    (dict(ks=fake((2, 2, 64, 8), fd.FD_E4M3, ptr=PTR + 4)), fd.FD_ERR_ALIGN),
    (dict(vs=fake((2, 2, 64, 8), fd.FD_E4M3, (1024, 512, 9, 1))), fd.FD_ERR_ALIGN),
    (dict(kg=0.0), fd.FD_ERR_ARG),
    (dict(kg=-1.0), fd.FD_ERR_ARG),
    (dict(vg=float("nan")), fd.FD_ERR_ARG),
    (dict(vg=float("inf")), fd.FD_ERR_ARG),
    (dict(kg=1e-30), fd.FD_ERR_ARG),
    (dict(max_pages=3), fd.FD_ERR_ARG),
    (dict(table=PTR, max_pages=0), fd.FD_ERR_ARG),
    (dict(table=PTR, max_pages=2 ** 26), fd.FD_ERR_UNSUPPORTED),
    (dict(lens=None), fd.FD_ERR_ARG),
    (dict(o=opts(kernel=fd.FD_KERNEL_TC)), fd.FD_ERR_ARG),
    (dict(o=opts(num_ctas=-1)), fd.FD_ERR_ARG),
    (dict(o=None), fd.FD_ERR_ARG),
    (dict(k=None), fd.FD_ERR_ARG),
]


@pytest.mark.parametrize("at", range(len(CACHE_FAULTS)))
def test_cache_faults_are_refused_by_every_call(L, at):
    change, want = CACHE_FAULTS[at]
    assert L.fd_decode_fp4(*decode_args(**change)) == want
    assert L.fd_append_fp4(*append_args(**change)) == want
    assert L.fd_read_fp4(*read_args(**change)) == want


def test_decode_refusals(L):
    def rc(**kw):
        return L.fd_decode_fp4(*decode_args(**kw))
    assert rc(q=fake((2, 1, 8, 128), fd.FD_F32)) == fd.FD_ERR_ARG
    assert rc(q=fake((3, 1, 8, 128), fd.FD_BF16), out=fake((3, 1, 8, 128), fd.FD_BF16)) == fd.FD_ERR_ARG
    assert rc(q=fake((2, 1, 7, 128), fd.FD_BF16), out=fake((2, 1, 7, 128), fd.FD_BF16)) == fd.FD_ERR_ARG
    assert rc(q=fake((2, 1, 8, 256), fd.FD_BF16), out=fake((2, 1, 8, 256), fd.FD_BF16)) == fd.FD_ERR_ARG
    assert rc(out=fake((2, 1, 8, 128), fd.FD_I32)) == fd.FD_ERR_ARG
    assert rc(out=fake((2, 1, 4, 128), fd.FD_BF16)) == fd.FD_ERR_ARG
    assert rc(n_q=2) == fd.FD_ERR_ARG
    assert rc(causal=2) == fd.FD_ERR_ARG
    assert rc(scale=float("nan")) == fd.FD_ERR_ARG
    seven = fake((2, 7, 8, 128), fd.FD_BF16)
    assert rc(q=seven, out=seven, n_q=7) == fd.FD_ERR_UNSUPPORTED
    many = fake((2, 6, 22, 128), fd.FD_BF16)       # 11 heads a kv head, 66 rows
    assert rc(q=many, out=many, n_q=6) == fd.FD_ERR_UNSUPPORTED
    odd = dict(k=fake((2, 2, 64, 32), fd.FD_U8), v=fake((2, 2, 64, 32), fd.FD_U8))
    assert rc(**odd) == fd.FD_ERR_UNSUPPORTED


def test_append_and_read_refusals(L):
    def rc(**kw):
        return L.fd_append_fp4(*append_args(**kw))
    assert rc(kn=fake((2, 3, 2, 128), fd.FD_F32)) == fd.FD_ERR_ARG
    assert rc(vn=fake((2, 4, 2, 128), fd.FD_BF16)) == fd.FD_ERR_ARG
    assert rc(kn=fake((2, 3, 1, 128), fd.FD_BF16)) == fd.FD_ERR_ARG
    assert rc(kn=fake((3, 3, 2, 128), fd.FD_BF16), vn=fake((3, 3, 2, 128), fd.FD_BF16)) == fd.FD_ERR_ARG
    assert rc(kn=fake((2, 3, 2, 128), fd.FD_BF16, ptr=PTR + 2)) == fd.FD_ERR_ALIGN
    assert rc(vn=fake((2, 3, 2, 128), fd.FD_BF16, (768, 260, 128, 1))) == fd.FD_ERR_ALIGN
    assert rc(after=PTR) == fd.FD_ERR_WORKSPACE            # in place is fine
    assert rc(after=PTR + 4) == fd.FD_ERR_ARG              # overlapping is not
    assert rc(new=PTR + 64, after=PTR + 64) == fd.FD_ERR_ARG
    def rd(**kw):
        return L.fd_read_fp4(*read_args(**kw))
    assert rd(ko=fake((2, 5, 2, 128), fd.FD_F32)) == fd.FD_ERR_ARG          # mixed types
    assert rd(ko=fake((2, 5, 2, 128), fd.FD_I32), vo=fake((2, 5, 2, 128), fd.FD_I32)) == fd.FD_ERR_ARG
    assert rd(vo=fake((2, 6, 2, 128), fd.FD_BF16)) == fd.FD_ERR_ARG
    assert rd(ko=fake((2, 5, 2, 128), fd.FD_BF16, ptr=PTR + 8)) == fd.FD_ERR_ALIGN


def test_page_refusals(L):
    o = ctypes.byref(opts())
    assert L.fd_pages_reserve(PTR, 2, 4, PTR, None, 1, 16, PTR, 10, PTR, PTR, o) == fd.FD_ERR_WORKSPACE
    assert L.fd_pages_reserve(PTR, 2, 4, PTR, None, 1, 16, PTR, 10, PTR, PTR, None) == fd.FD_ERR_ARG
    assert L.fd_pages_reserve(None, 2, 4, PTR, None, 1, 16, PTR, 10, PTR, PTR, o) == fd.FD_ERR_ARG
    assert L.fd_pages_reserve(PTR, 0, 4, PTR, None, 1, 16, PTR, 10, PTR, PTR, o) == fd.FD_ERR_ARG
    assert L.fd_pages_reserve(PTR, 2, 0, PTR, None, 1, 16, PTR, 10, PTR, PTR, o) == fd.FD_ERR_ARG
    assert L.fd_pages_reserve(PTR, 2, 4, PTR, None, 1, 0, PTR, 10, PTR, PTR, o) == fd.FD_ERR_ARG
    assert L.fd_pages_reserve(PTR, 2, 4, PTR, None, 1, 16, PTR, 0, PTR, PTR, o) == fd.FD_ERR_ARG
    assert L.fd_pages_reserve(PTR, 2 ** 16, 2 ** 15, PTR, None, 1, 16, PTR, 10, PTR, PTR, o) == fd.FD_ERR_UNSUPPORTED
    assert L.fd_pages_reserve(PTR, 2, 2 ** 20, PTR, None, 1, 2 ** 11, PTR, 10, PTR, PTR, o) == fd.FD_ERR_UNSUPPORTED
    assert L.fd_pages_fork(PTR, 2, 4, PTR, 16, PTR, 10, None, PTR, None, 1, o) == fd.FD_ERR_WORKSPACE
    assert L.fd_pages_free(PTR, 2, 4, None, 16, PTR, 10, PTR, None, 1, o) == fd.FD_ERR_ARG
    assert L.fd_pages_compact(PTR, 2, 4, None, 10, PTR, PTR, o) == fd.FD_ERR_ARG
    assert L.fd_pages_scratch_bytes(1000) >= 12000 and L.fd_pages_scratch_bytes(0) == 0


def test_copy_refusals(L):
    o = ctypes.byref(opts())
    def rc(pools, n=None, pairs=PTR, count=PTR, most=4):
        arr = (fd.FdTensor * max(len(pools), 1))(*pools)
        return L.fd_pages_copy(arr, len(pools) if n is None else n, pairs, count, most, o)
    good = fake((10, 2, 16, 64), fd.FD_U8)
    assert rc([good, fake((10, 8), fd.FD_F32)]) == fd.FD_ERR_WORKSPACE
    assert rc([fake((10, 2, 16, 64), fd.FD_U8, (2048, 64, 128, 1))]) == fd.FD_ERR_WORKSPACE   # token-major pages
    assert rc([]) == fd.FD_ERR_ARG
    assert rc([good] * 2, n=257) == fd.FD_ERR_ARG
    assert rc([good], pairs=None) == fd.FD_ERR_ARG
    assert rc([good], most=0) == fd.FD_ERR_ARG
    assert rc([good, fake((9, 8), fd.FD_F32)]) == fd.FD_ERR_ARG                               # other page counts
    assert rc([fake((10, 2, 16, 64), fd.FD_U8, (4096, 2048, 128, 1))]) == fd.FD_ERR_ARG       # gaps within a page
    assert rc([fake((10, 2, 16, 64), fd.FD_U8, (1024, 1024, 64, 1))]) == fd.FD_ERR_ARG        # pages overlap
    assert rc([fake((10, 2, 16, 64), 77)]) == fd.FD_ERR_ARG


def test_the_binding_refuses_host_tensors_and_wrong_lists():
    z = torch.zeros
    k, s = z(1, 1, 8, 64, dtype=torch.uint8), z(1, 1, 8, 8).to(torch.float8_e4m3fn)
    i = z(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fd.decode_fp4(z(1, 1, 2, 128, dtype=torch.bfloat16), k, k, s, s, i)
    with pytest.raises(ValueError):
        fd.append_fp4(z(1, 1, 1, 128, dtype=torch.bfloat16), z(1, 1, 1, 128, dtype=torch.bfloat16), k, k, s, s, i)
    with pytest.raises(ValueError):
        fd.read_fp4(k, k, s, s, i, 4)
    with pytest.raises(ValueError):
        fd.pages_reserve(z(1, 4, dtype=torch.int32), i, i, 16, 1)
    with pytest.raises(ValueError):
        fd.PagePools([k])
    with pytest.raises(ValueError):
        fd.PagePools([])
    assert len(fd._pack(k)) == ctypes.sizeof(fd.FdTensor) and fd._OPTS.size == ctypes.sizeof(fd.FdOpts)
    t = fd.FdTensor.from_buffer_copy(fd._pack(k[0, 0]))
    assert list(t.shape) == [8, 64, 0, 0] and list(t.stride)[:2] == [64, 1] and t.ndim == 2 and t.dtype == fd.FD_U8


def test_the_binding_refuses_what_is_no_tensor():
    k, s = torch.zeros(1, 1, 8, 64, dtype=torch.uint8), torch.zeros(1, 1, 8, 8).to(torch.float8_e4m3fn)
    with pytest.raises(TypeError):
        fd.decode_fp4(None, k, k, s, s, [8])
    with pytest.raises(TypeError):
        fd.pages_free([[0]], [1], [1], 16)
    with pytest.raises(TypeError):
        fd.pages_compact(None, None)
