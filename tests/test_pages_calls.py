"""What the page calls take: lists with nothing in them, pages of any order
of dimensions, a workspace sized by the header."""
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


def with_room():
    """opts whose workspace is host memory: for calls that return before the
    first launch."""
    room = ctypes.create_string_buffer(1024)
    o = fd.FdOpts()
    o.ws = ctypes.addressof(room)
    return room, ctypes.byref(o)


def test_a_list_of_nothing_is_no_error(L):
    room, o = with_room()
    assert L.fd_pages_free(PTR, 2, 4, PTR, 16, PTR, 10, PTR, None, 0, o) == fd.FD_OK
    assert L.fd_pages_free(PTR, 2, 4, PTR, 16, PTR, 10, None, None, 0, o) == fd.FD_OK
    assert L.fd_pages_fork(PTR, 2, 4, PTR, 16, PTR, 10, PTR, PTR, PTR, 0, o) == fd.FD_OK
    assert L.fd_pages_fork(PTR, 2, 4, PTR, 16, PTR, 10, None, None, None, 0, o) == fd.FD_OK
    # with everything else as it has to be
    assert L.fd_pages_free(PTR, 2, 4, PTR, 16, None, 10, PTR, None, 0, o) == fd.FD_ERR_ARG
    assert L.fd_pages_fork(PTR, 2, 4, PTR, 0, PTR, 10, PTR, PTR, None, 0, o) == fd.FD_ERR_ARG
    assert L.fd_pages_free(PTR, 2, 4, PTR, 16, PTR, 10, PTR, None, -1, o) == fd.FD_ERR_ARG
    assert L.fd_pages_free(PTR, 2, 4, PTR, 16, PTR, 10, None, None, 1, o) == fd.FD_ERR_ARG
    assert L.fd_pages_fork(PTR, 2, 4, PTR, 16, PTR, 10, None, PTR, None, 1, o) == fd.FD_ERR_ARG
    assert L.fd_pages_fork(PTR, 2, 4, PTR, 16, PTR, 10, PTR, PTR, None, -1, o) == fd.FD_ERR_ARG
    assert not any(room.raw)


@pytest.mark.parametrize("shape,strides,dense", [
    ((10, 2, 3), (6, 3, 1), True), ((10, 2, 3), (6, 1, 2), True), ((10, 2, 3), (7, 3, 1), True),
    ((10,), (1,), True), ((10,), (3,), True), ((10, 1, 4), (4, 99, 1), True), ((10, 1, 1), (1, 5, 7), True),
    ((10, 3, 2), (6, 1, 3), True),
    ((10, 4, 2, 3), (24, 2, 1, 8), True), ((1, 2, 3), (0, 3, 1), True),
    # as many elements as the memory they span, but some of them the same and
    # memory of others between
    ((10, 2, 3), (6, 5, 0), False), ((10, 2, 2, 2), (8, 3, 3, 1), False),
    ((10, 2, 3), (8, 4, 1), False), ((10, 3), (3, 0), False), ((10, 2, 3), (5, 3, 1), False),
])
def test_pages_that_do_not_fill_their_memory_are_refused(L, shape, strides, dense):
    t = fd.FdTensor()
    t.data, t.dtype, t.ndim = PTR, fd.FD_U8, len(shape)
    t.shape[:len(shape)], t.stride[:len(shape)] = shape, strides
    o = fd.FdOpts()     # (no workspace: what is left to refuse)
    rc = L.fd_pages_copy(ctypes.byref(t), 1, PTR, PTR, 4, ctypes.byref(o))
    assert rc == (fd.FD_ERR_WORKSPACE if dense else fd.FD_ERR_ARG)


@pytest.mark.parametrize("segments,rows,head_dim,ctas", [(1, 1, 1, 1), (1, 1, 128, 1), (64, 16, 256, 1024), (1, 64, 256, 65535),
                                                         (1000001, 1, 128, 7), (3, 5, 100, 100003)])
def test_the_room_of_a_workspace_is_what_the_header_says(L, segments, rows, head_dim, ctas):
    room = (segments + ctas) * fd.slot_floats(rows, head_dim) * 4     # of the split partials
    said = L.fd_workspace_bytes(segments, rows, head_dim, ctas) - (8 * segments + 4 * ctas + 1024)
    assert room - 1024 <= said <= room


@pytest.mark.gpu
def test_a_step_in_which_nobody_leaves_or_forks():
    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    table, lengths, refs, none = ints([[0, 1], [2, -1]]), ints([7, 3]), ints([1, 1, 1, 0]), ints([])
    fd.pages_free(table, lengths, refs, 4, seqs=none)
    fd.pages_free(table, lengths, refs, 4, seqs=none, lengths=none)
    fd.pages_fork(table, lengths, refs, 4, none, none)
    fd.pages_fork(table, lengths, refs, 4, none, none, none)
    assert table.tolist() == [[0, 1], [2, -1]] and lengths.tolist() == [7, 3] and refs.tolist() == [1, 1, 1, 0]
    with pytest.raises(ValueError):
        fd.pages_fork(table, lengths, refs, 4, none, ints([1]))


def test_a_dtype_is_packed_by_its_size():
    def kind(dtype):
        return fd.FdTensor.from_buffer_copy(fd._pack(torch.zeros(3, 2, dtype=dtype))).dtype

    assert [kind(t) for t in (torch.bfloat16, torch.float32, torch.int8, torch.int32, torch.uint8, torch.float8_e4m3fn)] == \
        [fd.FD_BF16, fd.FD_F32, fd.FD_I8, fd.FD_I32, fd.FD_U8, fd.FD_E4M3]
    assert kind(torch.float16) == kind(torch.int16) == fd.FD_BF16
    assert kind(torch.bool) == kind(torch.float8_e5m2) == fd.FD_U8
    for dtype in (torch.int64, torch.float64, torch.complex64):
        with pytest.raises(TypeError):
            kind(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.int16, torch.bool, torch.float8_e5m2, torch.int32])
def test_pools_of_any_dtype_are_copied(dtype):
    raw = torch.randint(0, 2 if dtype == torch.bool else 120, (9, 3, 8, 16), dtype=torch.uint8, device="cuda")
    pool = raw.view(dtype)
    want = raw.clone()
    want[0], want[5] = raw[7], raw[8]
    pairs = torch.tensor([[7, 0], [8, 5]], dtype=torch.int32, device="cuda")
    fd.pages_copy([pool], pairs, torch.tensor([2], dtype=torch.int32, device="cuda"))
    assert torch.equal(raw, want)
