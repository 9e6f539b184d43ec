"""GPU parity of the 4-bit cache (fd_decode_fp4, fd_append_fp4, fd_read_fp4)
against the 64-bit oracle: both head dims, every row count class, lengths from
0 and 1 up, split counts, causal windows that leave rows empty, layouts, pages
of any size, poisoned memory past the lengths, streams and graphs."""
import sys
import threading

import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from fp4_util import bf16, cache, check, decode_bound, scale_of, to_dev
from oracle import fp4

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def scattered(rng, B, max_pages, spare=3):
    return rng.permutation(B * max_pages + spare)[:B * max_pages].reshape(B, max_pages).astype(np.int32)


def decode_case(seed, B, n_q, Hq, Hkv, d, cap, lengths, causal, page=0, token_major=False, kg=1.0, vg=1.0,
                out_dtype=BF, num_ctas=0, poison=True, q_spread=1.0, table_edit=None, spread=1.0):
    rng = np.random.default_rng(seed)
    table = None
    lead, rows = B, cap
    if page:
        mp = -(-cap // page)
        table = scattered(rng, B, mp)
        lead, rows = B * mp + 3, page
    (k, ks), (v, vs) = (cache(rng, lead, Hkv, rows, d, g, spread) for g in (kg, vg))
    if poison:   # every row that holds no position below its length reads as NaN
        live = np.zeros((lead, rows), dtype=bool)
        for b, L in enumerate(lengths):
            pos = np.arange(max(0, min(L, cap)))
            live[(table[b, pos // page], pos % page) if page else (b, pos)] = True
        ks[~np.broadcast_to(live[:, None], ks.shape[:3])] = 0x7F
        vs[~np.broadcast_to(live[:, None], vs.shape[:3])] = 0x7F
    if table_edit:
        table_edit(table, lead)
    q = bf16(rng, (B, n_q, Hq, d), q_spread)
    scale = scale_of(d)
    want, weight, size = fp4.decode(q.double().numpy(), k, v, ks, vs, lengths, causal, scale, kg, vg, table)
    kd, ksd = to_dev(k, ks, token_major)
    vd, vsd = to_dev(v, vs, token_major)
    ws = fd.Workspace(B * Hkv * 4, 64, 256, 2048)
    got = fd.decode_fp4(q.cuda(), kd, vd, ksd, vsd, ints(lengths), causal=causal, scale=scale, k_global=kg, v_global=vg,
                        block_table=None if table is None else torch.from_numpy(table).cuda(), out_dtype=out_dtype,
                        num_ctas=num_ctas, workspace=ws)
    torch.cuda.synchronize()
    top = np.nan_to_num(np.abs(fp4.values(v, vs, vg))).max()
    check(got, want, decode_bound(want, weight, size, max(max(lengths), 1), top, out_dtype), "decode")
    return got, want, ws


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("length", [0, 1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 255, 257, 700])
def test_lengths(d, length):
    got, want, _ = decode_case(1, 1, 1, 4, 1, d, 701, [length], False)
    if length == 0:
        assert not got.any()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n_q,g", [(1, 1), (1, 5), (1, 8), (2, 5), (3, 4), (4, 4), (6, 4), (5, 5), (4, 8), (6, 8), (6, 10), (1, 64)])
def test_row_counts(d, n_q, g):
    decode_case(2, 2, n_q, 2 * g, 2, d, 300, [300, 77], n_q > 1, out_dtype=F32)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("ctas", [1, 2, 7, 40, 152, 999])
def test_splits(d, ctas):
    decode_case(3, 3, 3, 8, 2, d, 2000, [1999, 5, 640], True, num_ctas=ctas, out_dtype=F32)


@pytest.mark.parametrize("d", [128, 256])
def test_causal_rows_that_see_nothing(d):
    got, want, _ = decode_case(4, 4, 6, 8, 2, d, 50, [1, 3, 0, 6], True)
    assert not got[0, :5].any() and got[0, 5].any() and not got[1, :3].any() and got[1, 3].any() and not got[2].any()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("page", [1, 7, 16, 48, 64, 256])
@pytest.mark.parametrize("token_major", [False, True])
def test_pages(d, page, token_major):
    decode_case(5, 3, 2, 8, 2, d, 400 // page * page + page, [400, 1, 133], True, page=page, token_major=token_major)


@pytest.mark.parametrize("d", [128, 256])
def test_token_major_and_factors(d):
    decode_case(6, 2, 1, 8, 4, d, 300, [299, 64], False, token_major=True, kg=0.25, vg=3.0, out_dtype=F32)
    decode_case(7, 2, 1, 8, 4, d, 300, [299, 64], False, kg=1e-6, vg=1e5, out_dtype=F32, spread=1e-3)


def test_missing_pages_are_skipped_and_flagged():
    def edit(table, lead):
        table[0, 2], table[1, 0], table[1, 9] = -1, lead, -7
    _, _, ws = decode_case(8, 2, 2, 8, 2, 128, 320, [300, 140], True, page=32, table_edit=edit, poison=False)
    assert ws.device_status() & fd.FD_DEV_BAD_INDEX
    _, want, ws = decode_case(9, 1, 1, 4, 1, 256, 64, [60], False, page=64, poison=False,
                              table_edit=lambda t, lead: t.fill(-1))
    assert (want == 0).all()


def test_lengths_out_of_range_are_clamped_and_flagged():
    _, _, ws = decode_case(10, 3, 1, 4, 1, 128, 90, [95, -4, 20], False, poison=False)
    assert ws.device_status() & fd.FD_DEV_BAD_LENGTH


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("spread", [1e-30, 1e-3, 40.0, 3e4])
def test_query_magnitudes(d, spread):
    # tiny queries give the mean, large ones pick single positions
    decode_case(11, 1, 2, 8, 1, d, 500, [500], True, q_spread=spread, out_dtype=F32)


def test_a_rising_maximum_rescales():
    # keys aligned with the query and growing along the prefix: every step
    # raises the running reference
    rng = np.random.default_rng(12)
    d, L = 128, 2048
    q = bf16(rng, (1, 1, 4, d))
    direction = q[0, 0, 0].double().numpy() / np.linalg.norm(q[0, 0, 0].double().numpy())
    rows = np.linspace(0.1, 60, L)[:, None] * direction * 2
    k, ks = fp4.quantise(rows[None, None])
    v, vs = cache(rng, 1, 1, L, d)
    want, weight, size = fp4.decode(q.double().numpy(), k, v, ks, vs, [L], False, scale_of(d))
    kd, ksd = to_dev(k, ks)
    vd, vsd = to_dev(v, vs)
    for ctas in (0, 1, 3):
        got = fd.decode_fp4(q.cuda(), kd, vd, ksd, vsd, ints([L]), out_dtype=F32, num_ctas=ctas)
        check(got, want, decode_bound(want, weight, size, L, np.abs(fp4.values(v, vs)).max(), F32), "rising")


def test_one_outlier_over_a_long_flat_prefix():
    # one position some 2^13 above 20000 equal ones: their small weights must
    # still add up
    d, L = 128, 20000
    rng = np.random.default_rng(13)
    q = torch.zeros(1, 1, 8, d, dtype=BF)
    q[..., 0] = 1.0
    x = np.zeros((1, 1, L, d))
    x[0, 0, 777, 0] = 96.0                 # score 96 / sqrt(128) = 8.5, 2^12.2
    k, ks = fp4.quantise(x)
    v, vs = cache(rng, 1, 1, L, d)
    want, weight, size = fp4.decode(q.double().numpy(), k, v, ks, vs, [L], False, scale_of(d))
    kd, ksd = to_dev(k, ks)
    vd, vsd = to_dev(v, vs)
    got = fd.decode_fp4(q.cuda(), kd, vd, ksd, vsd, ints([L]), out_dtype=F32)
    check(got, want, decode_bound(want, weight, size, L, np.abs(fp4.values(v, vs)).max(), F32), "outlier")


@pytest.mark.parametrize("d", [128, 256])
def test_strided_query_and_output(d):
    rng = np.random.default_rng(14)
    k, ks = cache(rng, 2, 2, 200, d)
    v, vs = cache(rng, 2, 2, 200, d)
    q = bf16(rng, (2, 3, 9, d + 8))
    out = torch.full((2, 3, 9, d + 3), 7.0, dtype=BF, device="cuda")
    qd = q.cuda()[:, :, 1:9, 3:d + 3]      # odd offset: not 16-byte aligned
    (kd, ksd), (vd, vsd) = to_dev(k, ks), to_dev(v, vs)
    got = fd.decode_fp4(qd, kd, vd, ksd, vsd, ints([200, 33]), causal=True, out=out[:, :, :8, 1:d + 1])
    want, weight, size = fp4.decode(q[:, :, 1:9, 3:d + 3].double().numpy(), k, v, ks, vs, [200, 33], True, scale_of(d))
    check(got, want, decode_bound(want, weight, size, 200, np.abs(fp4.values(v, vs)).max(), BF), "strided")
    assert (out[:, :, 8] == 7).all() and (out[..., 0] == 7).all() and (out[..., d + 1:] == 7).all()


def test_nan_row_reaches_what_sees_it():
    rng = np.random.default_rng(15)
    k, ks = cache(rng, 1, 1, 64, 128)
    v, vs = cache(rng, 1, 1, 64, 128)
    vs[0, 0, 5, 3] = 0x7F
    (kd, ksd), (vd, vsd) = to_dev(k, ks), to_dev(v, vs)
    got = fd.decode_fp4(bf16(rng, (1, 1, 2, 128)).cuda(), kd, vd, ksd, vsd, ints([64]))
    assert torch.isnan(got[0, 0, :, 48:64]).all() and torch.isfinite(got[0, 0, :, :48]).all()
    ks[0, 0, 9, 0] = 0x7F
    _, ksd = to_dev(k, ks)
    got = fd.decode_fp4(bf16(rng, (1, 1, 2, 128)).cuda(), kd, vd, ksd, vsd, ints([64]))
    assert torch.isnan(got).all()
    got = fd.decode_fp4(bf16(rng, (1, 1, 2, 128)).cuda(), kd, vd, ksd, vsd, ints([5]))
    assert torch.isfinite(got).all()


def test_positions_past_32_bit_offsets():
    # a token-major cache whose rows lie 1 MiB + 16 bytes apart: position 2100
    # starts past 2^31 bytes
    d, cap, L = 128, 2200, 2190
    rng = np.random.default_rng(16)
    k, ks = cache(rng, 1, 1, cap, d)
    v, vs = cache(rng, 1, 1, cap, d)
    step = (1 << 20) + 16
    room = torch.zeros(cap * step, dtype=torch.uint8, device="cuda")
    kd = room.as_strided((1, 1, cap, 64), (cap * step, 64, step, 1), 0)
    vd = room.as_strided((1, 1, cap, 64), (cap * step, 64, step, 1), 1 << 12)
    ksd = room.as_strided((1, 1, cap, 8), (cap * step, 8, step, 1), 1 << 13).view(torch.float8_e4m3fn)
    vsd = room.as_strided((1, 1, cap, 8), (cap * step, 8, step, 1), 1 << 14).view(torch.float8_e4m3fn)
    q = bf16(rng, (1, 1, 4, d))
    new_k, new_v = bf16(rng, (1, L, 1, d)), bf16(rng, (1, L, 1, d))
    lens = ints([0])
    fd.append_fp4(new_k.cuda(), new_v.cuda(), kd, vd, ksd, vsd, lens, lengths_out=lens)
    (k, ks), (v, vs) = (fp4.quantise(x.double().numpy().transpose(0, 2, 1, 3)) for x in (new_k, new_v))
    assert (kd[:, :, :L].cpu().numpy() == k).all() and (vsd[:, :, :L].view(torch.uint8).cpu().numpy() == vs).all()
    got = fd.decode_fp4(q.cuda(), kd, vd, ksd, vsd, lens)
    want, weight, size = fp4.decode(q.double().numpy(), k, v, ks, vs, [L], False, scale_of(d))
    check(got, want, decode_bound(want, weight, size, L, np.abs(fp4.values(v, vs)).max(), BF), "far rows")
    rk, _ = fd.read_fp4(kd, vd, ksd, vsd, lens, 20, start=ints([L - 10]), out_dtype=F32)
    assert (rk[0, :10, 0].double().cpu().numpy() == fp4.values(k, ks)[0, 0, L - 10:]).all() and not rk[0, 10:].any()


# ------------------------------------------------------------ append and read
def bits(t):
    return t.view(torch.uint8).cpu().numpy()


def append_case(seed, B, n, Hkv, d, cap, lengths, new, page=0, token_major=False, kg=1.0, vg=1.0, rows=None,
                dtype=np.float64, inplace=False):
    rng = np.random.default_rng(seed)
    table = None
    lead, r = B, cap
    if page:
        table = scattered(rng, B, cap // page)
        lead, r = B * (cap // page) + 3, page
    (k, ks), (v, vs) = (cache(rng, lead, Hkv, r, d) for _ in range(2))
    kn, vn = (bf16(rng, (B, n, Hkv, d)) if rows is None else rows(rng, (B, n, Hkv, d)) for _ in range(2))
    (kd, ksd), (vd, vsd) = to_dev(k, ks, token_major), to_dev(v, vs, token_major)
    tab = None if table is None else torch.from_numpy(table).cuda()
    lens, ws = ints(lengths), fd.Workspace(1, 1, 128, 1)
    after = lens if inplace else torch.full_like(lens, -9)
    fd.append_fp4(kn.cuda(), vn.cuda(), kd, vd, ksd, vsd, lens, new_lengths=None if new is None else ints(new),
                  lengths_out=after, k_global=kg, v_global=vg, block_table=tab, workspace=ws)
    for x, codes, scales, g, cd, sd in ((kn, k, ks, kg, kd, ksd), (vn, v, vs, vg, vd, vsd)):
        wc, wsc, wl = fp4.append(x.double().numpy(), codes, scales, lengths, new, g, table, dtype)
        assert (bits(sd) == wsc).all()
        assert (bits(cd) == wc).all()
        assert after.tolist() == wl.tolist()
    return ws, (kd, vd, ksd, vsd), tab


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("page,token_major", [(0, False), (0, True), (16, True), (7, False)])
def test_append_ragged_rows(d, page, token_major, inplace):
    ws, _, _ = append_case(20, 4, 9, 3, d, 70, [0, 61, 13, 5], [9, 9, 0, 1], page, token_major, inplace=inplace)
    # four 16-position pages end at 64: the second sequence's 70 are past them
    assert ws.device_status() == (fd.FD_DEV_BAD_LENGTH if page == 16 else 0)


def test_append_past_the_capacity_and_bad_arguments_are_flagged():
    ws, _, _ = append_case(21, 4, 6, 2, 128, 20, [18, 25, -3, 2], [6, 2, 8, -1], inplace=True)
    assert ws.device_status() == fd.FD_DEV_BAD_LENGTH


def awkward(rng, shape):
    """Ties between codes, tiny and huge groups, zeros of both signs, and
    groups that are not finite."""
    x = rng.standard_normal(shape)
    flat = x.reshape(-1, 16)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    n = len(flat)
    for i in range(0, n, 2):
        s = 2.0 ** rng.integers(-8, 9) * rng.choice([1, 1.125, 1.25, 1.5, 1.75])
        flat[i] = rng.choice(ties, 16) * rng.choice([-1, 1], 16) * s
        flat[i, 0] = 6 * s
    flat[1::16] *= 1e-6
    flat[3::16] *= 1e30
    flat[5::32] = 0.0
    flat[7::32] = -0.0
    flat[9::32, 3] = np.nan
    flat[11::32, 5] = np.inf
    flat[13::32, 6] = -np.inf
    flat[15::32] = 2.0 ** rng.integers(-133, -120, 16)[None]
    return torch.from_numpy(x).to(torch.bfloat16)


@pytest.mark.parametrize("g", [1.0, 0.125, 2.0 ** 40])
def test_append_awkward_values_exactly(g):
    append_case(22, 2, 33, 2, 128, 40, [0, 3], None, kg=g, vg=1.0, rows=awkward)


def test_append_with_a_factor_that_is_no_power_of_two():
    # the steps round to fp32: followed in fp32
    append_case(23, 2, 33, 2, 256, 40, [0, 3], None, kg=0.3, vg=7e-5, dtype=np.float32)


def test_append_every_bf16_value_against_a_scale():
    # one group per bf16 magnitude below 8, its largest entry 6 (scale 1)
    mags = torch.arange(0, 0x4100, dtype=torch.int16).view(torch.bfloat16)
    rows = torch.zeros(len(mags), 16, dtype=torch.bfloat16)
    rows[:, 0] = torch.clamp(mags, min=6)
    rows[:, 1], rows[:, 2] = mags, -mags
    x = rows.reshape(1, -1, 1, 128)
    n = x.shape[1]
    c = [torch.zeros(1, 1, n, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.zeros(1, 1, n, 8, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    fd.append_fp4(x.cuda(), x.cuda(), *c, *s, ints([0]))
    wc, wsc = fp4.quantise(x.double().numpy()[:, :, 0])
    assert (bits(s[0])[0, 0] == wsc[0]).all() and (bits(c[0])[0, 0] == wc[0]).all() and (bits(c[1]) == bits(c[0])).all()


def test_append_strided_rows_leave_padding_unread():
    rng = np.random.default_rng(24)
    wide = bf16(rng, (2, 5, 2, 3 * 128)).cuda()
    wide[0, 2:] = float("nan")                       # padding of sequence 0
    c = [torch.zeros(2, 2, 8, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.zeros(2, 2, 8, 8, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    fd.append_fp4(wide[..., 128:256], wide[..., 256:], *c, *s, ints([1, 2]), new_lengths=ints([2, 5]))
    for x, cc, ss in ((wide[..., 128:256], c[0], s[0]), (wide[..., 256:], c[1], s[1])):
        wc, wsc, _ = fp4.append(x.double().cpu().numpy(), np.zeros((2, 2, 8, 64), np.uint8),
                                np.zeros((2, 2, 8, 8), np.uint8), [1, 2], [2, 5])
        assert (bits(cc) == wc).all() and (bits(ss) == wsc).all()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("page,token_major", [(0, False), (16, True), (5, False)])
def test_read(d, out_dtype, page, token_major):
    rng = np.random.default_rng(25)
    B, Hkv, cap, n, kg, vg = 3, 2, 60, 23, 0.5, 0.3
    table = scattered(rng, B, cap // page) if page else None
    lead, rows = (B * (cap // page) + 3, page) if page else (B, cap)
    (k, ks), (v, vs) = (cache(rng, lead, Hkv, rows, d) for _ in range(2))
    (kd, ksd), (vd, vsd) = to_dev(k, ks, token_major), to_dev(v, vs, token_major)
    lengths, start = [60, 30, 0], [0, 20, 5]
    got = fd.read_fp4(kd, vd, ksd, vsd, ints(lengths), n, start=ints(start), k_global=kg, v_global=vg,
                      block_table=None if table is None else torch.from_numpy(table).cuda(), out_dtype=out_dtype)
    most = cap // page * page if page else cap       # what the pages hold: 60, or 48 of 16-position ones
    for x, c, s, g in ((got[0], k, ks, kg), (got[1], v, vs, vg)):
        for b in range(B):
            L = min(lengths[b], most)
            for h in range(Hkv):
                rows_b = fp4.values(fp4.rows_of(c, b, h, L, table)[0], fp4.rows_of(s, b, h, L, table)[0])
                want = np.zeros((n, d))
                part = rows_b[start[b]:start[b] + n]
                # code * scale is exact, the factor is applied in fp32 and
                # the product rounded to the output's type
                want[:len(part)] = part.astype(np.float32) * np.float32(g)
                assert (x[b, :, h].cpu() == torch.from_numpy(want).float().to(out_dtype)).all()


def test_read_negative_start_and_missing_page():
    rng = np.random.default_rng(26)
    k, ks = cache(rng, 4, 1, 8, 128)
    (kd, ksd) = to_dev(k, ks)
    ws = fd.Workspace(1, 1, 128, 1)
    out = tuple(torch.full((1, 12, 1, 128), 9.0, device="cuda") for _ in range(2))
    fd.read_fp4(kd, kd, ksd, ksd, ints([16]), 12, start=ints([-2]), block_table=ints([[2, -1]]), out=out, workspace=ws)
    assert not out[0][0, :2].any() and not out[0][0, 10:].any()
    assert (out[0][0, 2:10, 0].double().cpu().numpy() == fp4.values(k, ks)[2, 0]).all()
    assert ws.device_status() == fd.FD_DEV_BAD_LENGTH | fd.FD_DEV_BAD_INDEX


# ------------------------------------------------------------ streams, graphs
def test_side_stream_and_graph_replay():
    rng = np.random.default_rng(30)
    B, Hkv, d, cap = 2, 2, 128, 300
    (k, ks), (v, vs) = (cache(rng, B, Hkv, cap, d) for _ in range(2))
    (kd, ksd), (vd, vsd) = to_dev(k, ks), to_dev(v, vs)
    q, lens = bf16(rng, (B, 2, 8, d)), ints([100, 7])
    kn, vn = bf16(rng, (B, 2, Hkv, d)), bf16(rng, (B, 2, Hkv, d))
    qd, knd, vnd = q.cuda(), kn.cuda(), vn.cuda()
    out = torch.empty_like(qd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = fd.Workspace(64, 32, 256, 1024, stream=side)
    fd.decode_fp4(qd, kd, vd, ksd, vsd, lens, out=out, stream=side, workspace=ws)   # warm
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        fd.append_fp4(knd, vnd, kd, vd, ksd, vsd, lens, lengths_out=lens, stream=side, workspace=ws)
        fd.decode_fp4(qd, kd, vd, ksd, vsd, lens, causal=True, out=out, stream=side, workspace=ws)
    now = [100, 7]
    for step in range(3):
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        k, ks, after = fp4.append(kn.double().numpy(), k, ks, now, None)
        v, vs, _ = fp4.append(vn.double().numpy(), v, vs, now, None)
        now = after.tolist()
        assert lens.tolist() == now
        want, weight, size = fp4.decode(q.double().numpy(), k, v, ks, vs, now, True, scale_of(d))
        check(out, want, decode_bound(want, weight, size, 110, np.abs(fp4.values(v, vs)).max(), BF), "replay %d" % step)
    assert ws.device_status() == 0


def test_two_graphs_share_a_workspace_in_turn():
    rng = np.random.default_rng(31)
    d = 256
    (k, ks), (v, vs) = (cache(rng, 1, 1, 2000, d) for _ in range(2))
    (kd, ksd), (vd, vsd) = to_dev(k, ks), to_dev(v, vs)
    ws = fd.Workspace(8, 32, 256, 1024)
    calls = []
    for n_q, L in ((1, 2000), (4, 1111)):
        q, lens = bf16(rng, (1, n_q, 4, d)), ints([L])
        qd = q.cuda()
        out = torch.empty_like(qd)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fd.decode_fp4(qd, kd, vd, ksd, vsd, lens, causal=True, out=out, workspace=ws)
        calls.append((g, q, qd, out, L, lens))
    for _ in range(3):
        for g, *_ in calls:
            g.replay()
    torch.cuda.synchronize()
    for _, q, _, out, L, _ in calls:
        want, weight, size = fp4.decode(q.double().numpy(), k, v, ks, vs, [L], True, scale_of(d))
        check(out, want, decode_bound(want, weight, size, L, np.abs(fp4.values(v, vs)).max(), BF), "graph")


def test_equal_calls_give_equal_bits():
    a, _, _ = decode_case(32, 3, 4, 16, 2, 128, 3000, [3000, 17, 1500], True, out_dtype=F32)
    b, _, _ = decode_case(32, 3, 4, 16, 2, 128, 3000, [3000, 17, 1500], True, out_dtype=F32)
    assert torch.equal(a, b)


def test_workspace_too_small_is_refused():
    rng = np.random.default_rng(33)
    (k, ks) = cache(rng, 1, 1, 64, 128)
    kd, ksd = to_dev(k, ks)
    ws = fd.Workspace(1, 16, 128, 4)
    q = bf16(rng, (1, 6, 8, 128)).cuda()            # 48 rows: two parts, two segments
    with pytest.raises(fd.FdError) as e:
        fd.decode_fp4(q, kd, kd, ksd, ksd, ints([64]), workspace=ws)
    assert e.value.code == fd.FD_ERR_WORKSPACE


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-20])
def test_other_scales(scale):
    # 0 weighs every visible position alike; a negative one turns the order
    rng = np.random.default_rng(34)
    for d in (128, 256):
        (k, ks), (v, vs) = (cache(rng, 2, 1, 150, d) for _ in range(2))
        (kd, ksd), (vd, vsd) = to_dev(k, ks), to_dev(v, vs)
        q = bf16(rng, (2, 3, 4, d))
        got = fd.decode_fp4(q.cuda(), kd, vd, ksd, vsd, ints([150, 2]), causal=True, scale=scale, out_dtype=F32)
        want, weight, size = fp4.decode(q.double().numpy(), k, v, ks, vs, [150, 2], True, scale)
        check(got, want, decode_bound(want, weight, size, 150, np.abs(fp4.values(v, vs)).max(), F32), "scale")


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n_q,g", [(6, 4), (4, 8), (6, 10)])
@pytest.mark.parametrize("ctas", [0, 1, 5, 60])
def test_many_rows_split(d, n_q, g, ctas):
    # 24, 32 and 60 rows (two parts) over several pieces
    decode_case(40, 2, n_q, 2 * g, 2, d, 1500, [1500, 333], True, num_ctas=ctas, out_dtype=F32)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("page", [8, 24, 11])
@pytest.mark.parametrize("n_q,g", [(1, 4), (3, 4), (6, 4), (5, 8)])
def test_rows_and_pages(d, page, n_q, g):
    # runs of eight rows on a page, and pages that end inside one
    decode_case(41, 2, n_q, 2 * g, 2, d, 700 // page * page + page, [700, 95], n_q > 1, page=page, kg=0.5)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("ctas", [0, 1, 9, 200])
def test_a_large_batch_with_empty_sequences(d, ctas):
    # more sequences than a warp has lanes, some of them empty (the first and
    # the last too), many of less than a tile
    rng = np.random.default_rng(42)
    lengths = [int(x) for x in rng.integers(0, 400, 70)]
    for b in (0, 5, 31, 32, 33, 64, 69):
        lengths[b] = 0
    got, _, _ = decode_case(43, 70, 2, 2, 1, d, 400, lengths, True, num_ctas=ctas)
    for b in (0, 5, 31, 32, 33, 64, 69):
        assert not got[b].any()


def test_all_sequences_empty():
    got, _, _ = decode_case(44, 40, 1, 4, 2, 128, 64, [0] * 40, False)
    assert not got.any()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("rows", [1, 16, 24])
def test_many_pieces_of_one_segment(d, rows):
    # one kv head over every block: joined in two levels
    decode_case(45, 1, 1, rows, 1, d, 30000, [29999], False, out_dtype=F32, num_ctas=150)
    decode_case(45, 1, 1, rows, 1, d, 6000, [5999], False, out_dtype=F32, num_ctas=13)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("page", [0, 16, 11])
@pytest.mark.parametrize("n_q,g", [(6, 1), (3, 4), (4, 6), (6, 5), (5, 8)])
@pytest.mark.parametrize("hole", ["k", "v"])
def test_nan_hidden_by_the_window(d, page, n_q, g, hole):
    rng = np.random.default_rng(61)
    lengths, cap = [301, 96, 4], 304
    mp = -(-cap // page) if page else 0
    table = scattered(rng, 3, mp) if page else None
    lead, rows = (3 * mp + 3, page) if page else (3, cap)
    (k, ks), (v, vs) = (cache(rng, lead, 2, rows, d) for _ in range(2))
    bad = ks if hole == "k" else vs
    for b, L in enumerate(lengths):
        for back, group, value in ((1, 0, 0x7F), (2, 3, 0xFF), (2, d // 16 - 1, 0x7F)):   # the last two positions
            at = (table[b, (L - back) // page], 0, (L - back) % page) if page else (b, 0, L - back)
            bad[at + (group,)] = value
    q = bf16(rng, (3, n_q, 2 * g, d))
    want, weight, size = fp4.decode(q.double().numpy(), k, v, ks, vs, lengths, True, scale_of(d), block_table=table)
    (kd, ksd), (vd, vsd) = to_dev(k, ks), to_dev(v, vs)
    got = fd.decode_fp4(q.cuda(), kd, vd, ksd, vsd, ints(lengths), causal=True, out_dtype=F32,
                        block_table=None if table is None else torch.from_numpy(table).cuda()).cpu()
    nan = np.isnan(want)
    assert nan[:, -2:, :g].any() and not nan[:, :-2].any() and not nan[:, :, g:].any()
    assert (torch.isnan(got).numpy() == nan).all()
    top = np.nan_to_num(np.abs(fp4.values(v, vs))).max()
    clean = [np.where(np.isnan(x), 0, x) for x in (want, weight)] + [np.nan_to_num(size)]
    check(torch.nan_to_num(got), clean[0], decode_bound(clean[0], clean[1], clean[2], 301, top, F32), "hidden")


def test_the_binding_refuses_and_keeps_no_references():
    rng = np.random.default_rng(71)
    (kd, ksd), (vd, vsd) = to_dev(*cache(rng, 2, 2, 32, 128)), to_dev(*cache(rng, 2, 2, 32, 128))
    q, lens = bf16(rng, (2, 1, 4, 128)).cuda(), ints([32, 7])
    new = bf16(rng, (2, 3, 2, 128)).cuda()
    good = fd.decode_fp4(q, kd, vd, ksd, vsd, lens)
    out = torch.zeros_like(good)
    bad = [
        (ValueError, lambda: fd.decode_fp4(q, kd, vd, ksd, vsd, lens.long())),
        (ValueError, lambda: fd.decode_fp4(q, kd, vd, ksd, vsd, ints([1, 2, 3]))),
        (ValueError, lambda: fd.decode_fp4(q, kd, vd, ksd, vsd, ints([1, 2, 3, 4])[::2])),
        (ValueError, lambda: fd.decode_fp4(q, kd, vd, ksd, vsd, lens.cpu())),
        (ValueError, lambda: fd.decode_fp4(q, kd, vd.cpu(), ksd, vsd, lens)),
        (ValueError, lambda: fd.decode_fp4(q[0], kd, vd, ksd, vsd, lens)),
        (ValueError, lambda: fd.decode_fp4(q, kd, vd, ksd, vsd, lens, block_table=ints([0, 1]))),
        (ValueError, lambda: fd.decode_fp4(q, kd, vd, ksd, vsd, lens, n_q=1 << 40)),
        (TypeError, lambda: fd.decode_fp4(q.half(), kd, vd, ksd, vsd, lens)),
        (TypeError, lambda: fd.decode_fp4(q, kd, vd, ksd, vsd, lens, scale="x")),
        (TypeError, lambda: fd.decode_fp4(q, kd, vd, ksd, vsd, lens, out_dtype="bf16")),
        (fd.FdError, lambda: fd.decode_fp4(q.float(), kd, vd, ksd, vsd, lens)),
        (fd.FdError, lambda: fd.decode_fp4(q, kd, vd, ksd, vsd, lens, out=out[:, :, :2])),
        (fd.FdError, lambda: fd.decode_fp4(q, kd, vd, ksd, vsd, lens, n_q=2)),
        (ValueError, lambda: fd.append_fp4(new, new, kd, vd, ksd, vsd, lens, new_lengths=ints([1]))),
        (fd.FdError, lambda: fd.append_fp4(new, new[:, :2], kd, vd, ksd, vsd, lens)),
        (ValueError, lambda: fd.read_fp4(kd, vd, ksd, vsd, lens, 3, out=(new,))),
        (ValueError, lambda: fd.read_fp4(kd, vd, ksd, vsd, lens, 4, out=(new, new))),
        (ValueError, lambda: fd.read_fp4(kd, vd, ksd, vsd, lens, -1)),
        (fd.FdError, lambda: fd.read_fp4(kd, vd, ksd, vsd, lens, 0)),
        (ValueError, lambda: fd.read_fp4(kd[0, 0, 0], vd, ksd, vsd, lens, 3)),
    ]
    kept = (q, kd, vd, ksd, vsd, lens, new, out)
    counts = [sys.getrefcount(t) for t in kept]
    for _ in range(3):
        for i, (kind, call) in enumerate(bad):
            with pytest.raises(kind):
                call()
                pytest.fail("call %d was accepted" % i)
        assert fd.decode_fp4(q, kd, vd, ksd, vsd, lens, out=out) is out
        k, v = fd.read_fp4(kd, vd, ksd, vsd, lens, 3, out=(new, new.clone()))
        del k, v
    assert [sys.getrefcount(t) for t in kept] == counts
    assert (out == good).all()


def test_a_given_stream_owns_what_the_call_makes():
    rng = np.random.default_rng(72)
    (kd, ksd), (vd, vsd) = to_dev(*cache(rng, 2, 2, 32, 128)), to_dev(*cache(rng, 2, 2, 32, 128))
    q, lens = bf16(rng, (2, 1, 4, 128)).cuda(), ints([32, 7])
    want = fd.decode_fp4(q, kd, vd, ksd, vsd, lens, out_dtype=F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fd.decode_fp4(q, kd, vd, ksd, vsd, lens, out_dtype=F32, stream=side)
    k, v = fd.read_fp4(kd, vd, ksd, vsd, lens, 5, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert (got == want).all() and got.shape == want.shape
    for a, b in zip(fd.read_fp4(kd, vd, ksd, vsd, lens, 5), (k, v)):
        assert (a == b).all()
    torch.cuda.synchronize()
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def test_more_sequences_than_a_grid_is_high():
    B, d = 66001, 128
    rng = np.random.default_rng(81)
    new = bf16(rng, (B, 1, 1, d))
    lens = torch.arange(B, dtype=torch.int32) % 3          # 2 is the capacity: nothing is written there
    codes, scales = np.zeros((B, 1, 2, d // 2), np.uint8), np.zeros((B, 1, 2, d // 16), np.uint8)
    want_c, want_s = fp4.quantise(new[:, 0].float().numpy(), 1.0, np.float32)
    for at in range(2):
        rows = np.arange(B) % 3 == at
        codes[rows, :, at], scales[rows, :, at] = want_c[rows], want_s[rows]
    (kd, ksd), (vd, vsd) = (to_dev(np.zeros_like(codes), np.zeros_like(scales)) for _ in range(2))
    after = lens.cuda()
    ws = fd.Workspace(64, 16, 256, 64)
    fd.append_fp4(new.cuda(), new.cuda(), kd, vd, ksd, vsd, after, lengths_out=after, workspace=ws)
    assert (after.cpu() == torch.clamp(lens + 1, max=2)).all()
    assert ws.device_status() == fd.FD_DEV_BAD_LENGTH
    for c, s in ((kd, ksd), (vd, vsd)):
        assert (c.cpu().numpy() == codes).all() and (s.view(torch.uint8).cpu().numpy() == scales).all()
    k, v = fd.read_fp4(kd, vd, ksd, vsd, after, 2, out_dtype=F32)
    want = fp4.values(codes, scales).transpose(0, 2, 1, 3)
    assert (k.cpu().numpy() == want).all() and (v.cpu().numpy() == want).all()


def test_a_query_that_is_one_row_for_all():
    rng = np.random.default_rng(82)
    k, ks = cache(rng, 3, 2, 90, 256)
    v, vs = cache(rng, 3, 2, 90, 256)
    (kd, ksd), (vd, vsd) = to_dev(k, ks), to_dev(v, vs)
    q = bf16(rng, (1, 1, 1, 256)).cuda().expand(3, 2, 8, 256)
    lens = ints([90, 41, 2])
    got = fd.decode_fp4(q, kd, vd, ksd, vsd, lens, causal=True)
    assert (got == fd.decode_fp4(q.contiguous(), kd, vd, ksd, vsd, lens, causal=True)).all()
    want, weight, size = fp4.decode(q.cpu().double().numpy(), k, v, ks, vs, [90, 41, 2], True, scale_of(256))
    check(got, want, decode_bound(want, weight, size, 90, np.abs(fp4.values(v, vs)).max(), BF), "expanded")


def test_two_threads_on_two_streams():
    rng = np.random.default_rng(83)
    jobs = []
    for i in range(2):
        (kd, ksd), (vd, vsd) = to_dev(*cache(rng, 2, 2, 3000, 128)), to_dev(*cache(rng, 2, 2, 3000, 128))
        q, lens = bf16(rng, (2, 1 + 2 * i, 8, 128)).cuda(), ints([3000, 1234 + i])
        jobs.append((q, kd, vd, ksd, vsd, lens, fd.decode_fp4(q, kd, vd, ksd, vsd, lens)))
    torch.cuda.synchronize()
    wrong = []

    def work(q, kd, vd, ksd, vsd, lens, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got = [fd.decode_fp4(q, kd, vd, ksd, vsd, lens) for _ in range(50)]
                torch.cuda.current_stream().synchronize()
                wrong.extend(i for i, g in enumerate(got) if not (g == want).all())
        except Exception as e:   # (a thread's own exception ends nothing)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not wrong
