"""Calls of the 4-bit cache: tables without columns, strides past 32 bits, two
threads."""
import threading

import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from fp4_util import bf16, cache, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def test_a_block_table_without_columns_is_refused():
    # two sequences and two pages: without its table the pool would pass for a
    # flat cache
    rng = np.random.default_rng(111)
    (kd, ksd), (vd, vsd) = (to_dev(*cache(rng, 2, 2, 16, 128)) for _ in range(2))
    lens = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    new = bf16(rng, (2, 1, 2, 128)).cuda()
    before = kd.clone()
    for call in (lambda: fd.decode_fp4(bf16(rng, (2, 1, 4, 128)).cuda(), kd, vd, ksd, vsd, lens, block_table=table),
                 lambda: fd.append_fp4(new, new, kd, vd, ksd, vsd, lens, block_table=table),
                 lambda: fd.read_fp4(kd, vd, ksd, vsd, lens, 3, block_table=table)):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert torch.equal(before, kd)


def far(t):
    """The same memory, with a stride past 32 bits in its dimension of size 1."""
    assert t.shape[0] == 1
    return t.as_strided(t.shape, (1 << 33, *t.stride()[1:]), t.storage_offset())


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,aligned", [(37, True), (37, False), (500, True)])
def test_append_and_read_with_strides_past_32_bits(d, out_dtype, n, aligned):
    # (1 << 33 and more take address products of 64 bits)
    rng = np.random.default_rng(112)
    Hkv, cap = 3, 520
    at = 0 if aligned else 8
    wide = [bf16(rng, (1, n, Hkv, d + 16)).cuda() for _ in range(2)]
    kn, vn = (x[..., at:at + d] for x in wide)
    lens = torch.tensor([11], dtype=torch.int32, device="cuda")
    results = []
    for stretch in (lambda t: t, far):
        rng = np.random.default_rng(113)
        (kd, ksd), (vd, vsd) = (to_dev(*cache(rng, 1, Hkv, cap, d)) for _ in range(2))
        after = torch.zeros_like(lens)
        where = [stretch(t) for t in (kd, vd, ksd, vsd)]
        assert where[0].stride(0) == (kd.stride(0) if stretch is not far else 1 << 33)
        fd.append_fp4(stretch(kn), stretch(vn), *where, lens, lengths_out=after, k_global=0.5)
        outs = [torch.full((1, n + 9, Hkv, d + 16), 7.0, dtype=out_dtype, device="cuda") for _ in range(2)]
        fd.read_fp4(*where, after, n + 9, start=torch.tensor([4], dtype=torch.int32, device="cuda"), k_global=0.5,
                    out=tuple(stretch(o[..., at:at + d]) for o in outs))
        results.append([x.view(torch.uint8).clone() for x in (kd, vd, ksd, vsd, *outs)] + [after])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert results[1][-1].item() == 11 + n
    got = results[1][4].view(out_dtype)
    assert got[0, :n + 7, :, at:at + d].any() and not got[0, n + 7:, :, at:at + d].any()
    assert (got[..., :at] == 7).all() and (got[..., at + d:] == 7).all()


def test_two_threads_on_two_streams_finish_all_their_calls():
    rng = np.random.default_rng(114)
    jobs, times = [], 50
    for i in range(2):
        (kd, ksd), (vd, vsd) = (to_dev(*cache(rng, 2, 2, 3000, 128)) for _ in range(2))
        lens = torch.tensor([3000, 1234 + i], dtype=torch.int32, device="cuda")
        args = (bf16(rng, (2, 1 + 2 * i, 8, 128)).cuda(), kd, vd, ksd, vsd, lens)
        jobs.append((i, args, fd.decode_fp4(*args)))
    torch.cuda.synchronize()
    right, errors = [0, 0], []

    def work(i, args, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got = [fd.decode_fp4(*args) for _ in range(times)]
                torch.cuda.current_stream().synchronize()
                right[i] = sum(bool((g == want).all()) for g in got)
        except Exception as e:   # (a thread's own exception ends nothing)
            errors.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not any(t.is_alive() for t in threads) and not errors and right == [times, times]
