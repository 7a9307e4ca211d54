"""The 4-bit cache on the GPU: append and read back against the record's
definition, attention against the fp64 oracle on the values the records stand
for, and the three as a run."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import q4_util as u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gqa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import grouped_query_attention_fwd_b200 as m
    return m


def _ok(gqa):
    st = gqa.device_status()
    assert st == gqa.GQA_OK, gqa.status_string(st)


# ------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [8, 24, 32, 40, 64, 80, 96, 128])
@pytest.mark.parametrize("n", [1, 5])
def test_append_records(gqa, dtype, D, n):
    rng = np.random.default_rng(1000 * D + n)
    B, H, cap = 3, 2, 37
    lens = np.array([0, 11, cap - n], np.int32)
    old = rng.integers(0, 256, (2, B, H, cap, u.record_bytes(D)), dtype=np.uint8)
    kb, vb = u.random_rows(rng, (B, H, n, D), dtype, True), u.random_rows(rng, (B, H, n, D), dtype)
    ck, cv = (torch.from_numpy(x.copy()).cuda() for x in old)
    dl = torch.from_numpy(lens).cuda()
    gqa.kv_append_q4(ck, cv, u.dev16(kb, dtype), u.dev16(vb, dtype), dl)
    _ok(gqa)
    assert np.array_equal(dl.cpu().numpy(), lens + n)
    for got, want, bits in ((ck, old[0].copy(), kb), (cv, old[1].copy(), vb)):
        rec = u.quantise(bits, dtype)
        for b in range(B):
            want[b, :, lens[b]:lens[b] + n] = rec[b]
        assert np.array_equal(got.cpu().numpy(), want)  # every other record as it was


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_corner_values(gqa, dtype):
    big = 3.0e38 if dtype == "bf16" else 6.0e4
    tiny = 1.0e-39 if dtype == "bf16" else 6.0e-8
    rows = np.zeros((12, 64), np.float32)
    rng = np.random.default_rng(5)
    rows[0] = 2.5
    rows[1, 3] = np.nan
    rows[2, 40] = np.inf
    rows[3, 40], rows[3, 41] = np.inf, -np.inf
    rows[4, :32], rows[4, 0] = big, -big
    rows[5, 0:32:2], rows[5, 1:32:2] = tiny, -tiny
    rows[6, 7] = 10 * tiny
    rows[7] = 100 + 0.01 * rng.standard_normal(64)
    # Values on the borders between codes: scale 1, minimum 0, halves in between.
    rows[8, :32] = np.concatenate([np.arange(16), np.arange(16) - 0.5 + 1])
    rows[8, 31] = 15
    rows[9] = -0.0
    rows[10, :32] = np.linspace(-1, 1, 32)
    rows[11] = rng.standard_normal(64) * 1e-3
    bits = u.bits_of(rows, dtype)[None, None]
    ck = torch.zeros(1, 1, 12, u.record_bytes(64), dtype=torch.uint8, device="cuda")
    cv = torch.zeros_like(ck)
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = u.dev16(bits, dtype)
    gqa.kv_append_q4(ck, cv, x, x, lens)
    _ok(gqa)
    want = u.quantise(bits, dtype)
    got = ck.cpu().numpy()
    # A zero minimum may be stored as either zero.
    a, b = u.parts(got, 64, dtype), u.parts(want, 64, dtype)
    for g, w in zip(a, b):
        assert np.array_equal(g, w, equal_nan=True)
    assert torch.equal(ck, cv)
    k, _ = gqa.kv_read_q4(ck, cv, 64, u.TORCH[dtype])
    y = u.to64(k)[0, 0]
    for r, g in ((1, 0), (2, 1), (3, 1)):
        assert np.all(np.isnan(y[r, 32 * g:32 * g + 32])) and not np.any(
            np.isnan(y[r, 32 * (1 - g):32 * (1 - g) + 32]))


@pytest.mark.parametrize("page", [64, 128])
def test_append_paged_padded_batch(gqa, page):
    """New rows of a padded batch that cross pages; the padding writes nothing."""
    dtype, D, B, H, n = "bf16", 128, 4, 3, 150
    rng = np.random.default_rng(page)
    lens = np.array([0, 60, 63, 200], np.int32)
    counts = np.array([150, 1, 0, 77], np.int32)
    cap = 6 * 64
    _, table = u.paged(np.zeros((B, H, cap, 80), np.uint8), page, rng)
    pool0 = rng.integers(0, 256, (table.size + 2, H, page, 80), dtype=np.uint8)
    kb, vb = u.random_rows(rng, (B, H, n, D), dtype), u.random_rows(rng, (B, H, n, D), dtype)
    ck, cv = torch.from_numpy(pool0.copy()).cuda(), torch.from_numpy(pool0.copy()).cuda()
    dl, dc, dt = (torch.from_numpy(x).cuda() for x in (lens, counts, table))
    for advance in (False, True):  # the same rows again: the same records
        gqa.kv_append_q4(ck, cv, u.dev16(kb, dtype), u.dev16(vb, dtype), dl, new_lens=dc,
                         advance=advance, block_table=dt)
        _ok(gqa)
        assert np.array_equal(dl.cpu().numpy(), lens + (counts if advance else 0))
    for got, bits in ((ck, kb), (cv, vb)):
        want, rec = pool0.copy(), u.quantise(bits, dtype)
        for b in range(B):
            for t in range(counts[b]):
                j = lens[b] + t
                want[table[b, j // page], :, j % page] = rec[b, :, t]
        assert np.array_equal(got.cpu().numpy(), want)


def test_append_strided_and_unaligned_rows(gqa):
    dtype, D, B, H, n, cap = "fp16", 64, 2, 3, 7, 20
    rng = np.random.default_rng(8)
    bits = u.random_rows(rng, (B, H, n, D), dtype)
    want = u.quantise(bits, dtype)
    # [B, n, H, D] buffers viewed as [B, H, n, D]; one of them two bytes off the 16-byte grid.
    flat = torch.zeros(B * n * H * D + 1, dtype=torch.float16, device="cuda")
    odd = flat[1:].view(B, n, H, D).transpose(1, 2)
    even = torch.zeros(B, n, H, D, dtype=torch.float16, device="cuda").transpose(1, 2)
    odd.copy_(u.dev16(bits, dtype))
    even.copy_(u.dev16(bits, dtype))
    # Caches laid out [B, capacity, H, record].
    caches = [torch.zeros(B, cap, H, 48, dtype=torch.uint8, device="cuda").transpose(1, 2)
              for _ in range(2)]
    lens = torch.tensor([3, 13], dtype=torch.int32, device="cuda")
    gqa.kv_append_q4(*caches, odd, even, lens)
    _ok(gqa)
    for c in caches:
        for b, l0 in enumerate((3, 13)):
            assert np.array_equal(c[b, :, l0:l0 + n].cpu().numpy(), want[b])


def test_append_that_does_not_fit(gqa):
    dtype, D, B, H, n, cap = "bf16", 32, 4, 1, 4, 10
    rng = np.random.default_rng(9)
    x = u.dev16(u.random_rows(rng, (B, H, n, D), dtype), dtype)
    ck = torch.full((B, H, cap, 32), 7, dtype=torch.uint8, device="cuda")
    cv = ck.clone()
    lens = torch.tensor([6, 7, -1, 2], dtype=torch.int32, device="cuda")
    counts = torch.tensor([4, 4, 1, 5], dtype=torch.int32, device="cuda")
    gqa.kv_append_q4(ck, cv, x, x, lens, new_lens=counts)
    assert gqa.device_status() == gqa.GQA_ERR_KV_LENGTH
    assert gqa.device_status() == gqa.GQA_OK
    assert lens.tolist() == [10, 7, -1, 2]
    assert torch.all(ck[1:] == 7) and torch.all(cv[1:] == 7) and torch.all(ck[0, :, :6] == 7)


def test_append_bad_page(gqa):
    dtype, D = "bf16", 32
    rng = np.random.default_rng(10)
    x = u.dev16(u.random_rows(rng, (2, 1, 4, D), dtype), dtype)
    ck = torch.full((3, 1, 64, 32), 7, dtype=torch.uint8, device="cuda")
    cv = ck.clone()
    table = torch.tensor([[0, 5], [1, 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([62, 62], dtype=torch.int32, device="cuda")
    gqa.kv_append_q4(ck, cv, x, x, lens, block_table=table)
    assert gqa.device_status() == gqa.GQA_ERR_PAGE
    assert lens.tolist() == [62, 66]
    assert torch.all(ck[0, :, :62] == 7) and torch.all(ck[2, :, 2:] == 7)


# ------------------------------------------------------------ read back

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [8, 40, 64, 96, 128])
def test_read_values(gqa, dtype, D):
    rng = np.random.default_rng(D)
    B, H, cap, n = 3, 2, 70, 33
    rec = [u.quantise(u.random_rows(rng, (B, H, cap, D), dtype, i == 0), dtype) for i in (0, 1)]
    lens = np.array([0, 20, 70], np.int32)
    starts = np.array([0, 5, 60], np.int32)
    ck, cv = (torch.from_numpy(r).cuda() for r in rec)
    outs = gqa.kv_read_q4(ck, cv, D, u.TORCH[dtype], kv_lens=torch.from_numpy(lens).cuda(),
                          start=torch.from_numpy(starts).cuda(), n=n)
    _ok(gqa)
    for out, r in zip(outs, rec):
        got, ref = u.to64(out), u.dequantise(r, D, dtype)
        for b in range(B):
            live = max(0, min(n, lens[b] - starts[b]))
            want = ref[b, :, starts[b]:starts[b] + live]
            # One rounding to fp32 (scale * code + minimum), one to 16 bits;
            # 2^-25 covers fp16's subnormal step.
            bound = (u.UNIT[dtype] + 2.0 ** -23) * np.abs(want) + 2.0 ** -25
            assert np.all(np.abs(got[b, :, :live] - want) <= bound)
            assert np.all(got[b, :, live:] == 0)


def test_read_paged_strided_and_whole(gqa):
    dtype, D, B, H, S, page = "bf16", 128, 2, 3, 130, 64
    rng = np.random.default_rng(2)
    rec = u.quantise(u.random_rows(rng, (B, H, S, D), dtype), dtype)
    pool, table = u.paged(rec, page, rng)
    c, dt = torch.from_numpy(pool).cuda(), torch.from_numpy(table).cuda()
    lens = torch.tensor([130, 64], dtype=torch.int32, device="cuda")
    flat = torch.full((B * 192 * H * D + 1,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = flat[1:].view(B, 192, H, D).transpose(1, 2)  # rows off the 16-byte grid
    k, v = gqa.kv_read_q4(c, c, D, torch.bfloat16, kv_lens=lens, out_k=out, block_table=dt)
    _ok(gqa)
    assert k.data_ptr() == out.data_ptr() and v.shape == (B, H, 192, D) and torch.equal(k, v)
    ref = u.dequantise(rec, D, dtype)
    for b, l in enumerate((130, 64)):
        got = u.to64(v)[b]
        assert np.all(np.abs(got[:, :l] - ref[b, :, :l]) <=
                      (2.0 ** -8 + 2.0 ** -23) * np.abs(ref[b, :, :l]))
        assert np.all(got[:, l:] == 0)
    assert flat[0] == 9.0


def test_read_errors(gqa):
    c = torch.zeros(2, 1, 64, 32, dtype=torch.uint8, device="cuda")
    lens = torch.tensor([65, 3], dtype=torch.int32, device="cuda")
    k, _ = gqa.kv_read_q4(c, c, 32, torch.float16, kv_lens=lens)
    assert gqa.device_status() == gqa.GQA_ERR_KV_LENGTH
    starts = torch.tensor([-1, 3], dtype=torch.int32, device="cuda")
    k, _ = gqa.kv_read_q4(c, c, 32, torch.float16, start=starts, n=2)
    assert gqa.device_status() == gqa.GQA_ERR_KV_LENGTH and torch.all(k == 0)
    table = torch.tensor([[0, 2]], dtype=torch.int32, device="cuda")
    k, _ = gqa.kv_read_q4(c, c, 32, torch.float16, block_table=table)
    assert gqa.device_status() == gqa.GQA_ERR_PAGE and torch.all(k[:, :, 64:] == 0)


# ------------------------------------------------------------ attention

def _bound(probs, vrec, D, g, dtype):
    """Elementwise error bound of the output from the roundings that the
    formulas take: the weight of each (key, group) is rounded to 16 bits before
    it multiplies codes counted from the middle of the group's range (at most
    8 scales away), and the output is rounded once.  fp32 sums and exponents
    add at most 2^-14 of the largest term here (up to 2^10 terms of 2^-24)."""
    spans = u.half_spans(vrec, D, dtype)  # [B, Hkv, S, D]
    top = np.abs(u.dequantise(vrec, D, dtype)) + spans
    B, Hq, Sq, S = probs.shape
    p = probs.reshape(B, Hq // g, g * Sq, S)
    w = np.einsum("bhrs,bhsd->bhrd", p, np.nan_to_num(spans)) * u.UNIT[dtype]
    t = np.einsum("bhrs,bhsd->bhrd", p, np.nan_to_num(top)) * 2.0 ** -14
    return (w + t).reshape(B, Hq, Sq, D)


def _check(out, ref, probs, vrec, D, g, dtype):
    got = u.to64(out)
    empty = np.isnan(ref).all(-1)
    assert np.array_equal(np.isnan(got).all(-1), empty)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    bound = _bound(np.nan_to_num(probs), vrec, D, g, dtype) + \
        u.UNIT[dtype] * np.abs(ref) * 1.01 + 2.0 ** -24
    err = np.abs(got - ref)
    assert np.all((err <= bound) | np.isnan(ref)), float(np.nanmax(err / bound))
    if not empty.all():
        d, r = (got - ref)[~empty], ref[~empty]
        assert np.linalg.norm(d) <= 1e-2 * np.linalg.norm(r)


def _case(gqa, dtype, B, Hq, Hkv, Sq, Sk, D, seed, mask=None, causal=False, offset=None, window=0,
          lens=None, page=0, layout="bhsd"):
    rng = np.random.default_rng(seed)
    qb = u.random_rows(rng, (B, Hq, Sq, D), dtype)
    krec = u.quantise(u.random_rows(rng, (B, Hkv, Sk, D), dtype, True), dtype)
    vrec = u.quantise(u.random_rows(rng, (B, Hkv, Sk, D), dtype), dtype)
    k64, v64 = u.dequantise(krec, D, dtype), u.dequantise(vrec, D, dtype)
    kd, vd = krec.copy(), vrec.copy()
    if lens is not None:  # NaN scales past each length must not reach the result
        for b in range(B):
            kd[b, :, lens[b]:] = vd[b, :, lens[b]:] = 0xFF
    kw = dict(causal=causal, window=window)
    if causal:
        kw["causal_offset"] = offset
    okw = dict(kw)
    if lens is not None:
        kw["kv_lens"] = torch.from_numpy(np.asarray(lens, np.int32)).cuda()
        okw["kv_lens"] = lens
    if page:
        assert Sk % page == 0
        pk, table = u.paged(kd, page, np.random.default_rng(seed + 1))
        pv, _ = u.paged(vd, page, np.random.default_rng(seed + 1))
        ck, cv = torch.from_numpy(pk).cuda(), torch.from_numpy(pv).cuda()
        kw["block_table"] = torch.from_numpy(table).cuda()
    else:
        ck, cv = torch.from_numpy(kd).cuda(), torch.from_numpy(vd).cuda()
    q = u.dev16(qb, dtype)
    if layout == "bshd":
        ck, cv, q = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (ck, cv, q))
    dm = None if mask is None else torch.from_numpy(mask).cuda()
    out = gqa.forward_q4(q, ck, cv, mask=dm, **kw)
    _ok(gqa)
    om = None if mask is None else mask.astype(np.uint8)
    q64 = u.values_of(qb, dtype)
    ref = oracle.forward(q64, k64, v64, mask=om, **okw)
    probs = _probs(q64, k64, om, Hq // Hkv, **okw)
    _check(out, ref, probs, vrec, D, Hq // Hkv, dtype)
    return out


def _probs(q, k, mask, g, causal=False, causal_offset=0, window=0, kv_lens=None):
    B, Hq, Sq, D = q.shape
    Sk = k.shape[2]
    s = np.einsum("bhid,bhjd->bhij", q, np.repeat(k, g, 1)) / np.sqrt(D)
    lens = np.full(B, Sk) if kv_lens is None else np.asarray(kv_lens)
    j, i = np.arange(Sk)[None, None, :], np.arange(Sq)[None, :, None]
    see = np.broadcast_to(j < lens[:, None, None], (B, Sq, Sk)).copy()
    if causal:
        top = i + (0 if causal_offset is None else causal_offset) + (lens - Sk)[:, None, None]
        see &= j <= top
        if window:
            see &= j > top - window
    if mask is not None:
        see &= mask != 0
    s = np.where(see[:, None], s, -np.inf)
    with np.errstate(all="ignore"):
        e = np.exp(s - s.max(-1, keepdims=True))
        return e / e.sum(-1, keepdims=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("g", [1, 3, 4, 8, 12, 20])
@pytest.mark.parametrize("Sk,D", [(1, 128), (2, 64), (15, 128), (16, 64), (17, 32), (63, 128),
                                  (128, 128), (129, 64), (333, 128), (1000, 96)])
def test_decode(gqa, dtype, g, Sk, D):
    _case(gqa, dtype, 2, 2 * g, 2, 1, Sk, D, seed=100 * g + Sk)


@pytest.mark.parametrize("D", [8, 16, 24, 40, 56, 72, 80, 112, 120])
def test_decode_head_dims(gqa, D):
    _case(gqa, "bf16", 2, 8, 2, 1, 190, D, seed=D)
    _case(gqa, "fp16", 1, 4, 1, 3, 77, D, seed=D)


@pytest.mark.parametrize("Sq,g", [(2, 1), (2, 4), (4, 4), (5, 3), (16, 1), (3, 8), (9, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_short_query_blocks(gqa, Sq, g, D):
    _case(gqa, "bf16", 2, 2 * g, 2, Sq, 140, D, seed=Sq + g, causal=True, offset=140 - Sq)
    _case(gqa, "fp16", 1, g, 1, Sq, 260, D, seed=Sq + g)


@pytest.mark.parametrize("Sq", [17, 64, 129, 200])
@pytest.mark.parametrize("dtype,D,g", [("bf16", 128, 4), ("fp16", 64, 6), ("bf16", 40, 1)])
def test_query_chunks(gqa, Sq, dtype, D, g):
    _case(gqa, dtype, 2, 2 * g, 2, Sq, 300, D, seed=Sq, causal=True, offset=300 - Sq)


@pytest.mark.parametrize("page", [0, 64, 192])
@pytest.mark.parametrize("Sq", [1, 3, 40])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_lengths(gqa, page, Sq, dtype):
    Sk = 576
    lens = [0, 1, 63, 64, 65, 200, 575, 576]
    _case(gqa, dtype, len(lens), 8, 2, Sq, Sk, 128, seed=page + Sq, lens=lens, page=page,
          causal=Sq > 1, offset=Sk - Sq)


@pytest.mark.parametrize("Sq", [1, 4, 50])
@pytest.mark.parametrize("window", [1, 16, 100])
def test_windows(gqa, Sq, window):
    _case(gqa, "bf16", 3, 8, 2, Sq, 256, 64, seed=window, causal=True, offset=256 - Sq,
          window=window, lens=[50, 180, 256])


@pytest.mark.parametrize("Sq", [1, 4, 33])
def test_masks_that_leave_rows_empty(gqa, Sq):
    rng = np.random.default_rng(Sq)
    B, Sk = 3, 200
    mask = rng.random((B, Sq, Sk)) < 0.3
    mask[0, 0] = False             # an empty row
    mask[1, :, :150] = False       # whole tiles hidden
    mask[2] = False                # an entry without a visible key
    for D, dtype in ((128, "bf16"), (64, "fp16")):
        _case(gqa, dtype, B, 8, 2, Sq, Sk, D, seed=Sq, mask=mask)


def test_layouts(gqa):
    _case(gqa, "bf16", 2, 8, 2, 1, 300, 128, seed=1, layout="bshd")
    _case(gqa, "bf16", 2, 8, 2, 40, 300, 128, seed=2, layout="bshd", causal=True, offset=260)


def test_split_over_many_ctas(gqa):
    """Few rows and long keys: every key range is split and merged."""
    _case(gqa, "bf16", 1, 8, 1, 1, 20011, 128, seed=3)
    _case(gqa, "fp16", 3, 4, 1, 2, 7000, 64, seed=4, causal=True, offset=6998,
          lens=[1, 7000, 5003])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("vscale", [1e-4, 1.0, 1e3])
def test_value_ranges(gqa, dtype, vscale):
    """Weights are rounded to 16 bits after the value scale is folded in: small
    and large values keep their relative precision."""
    rng = np.random.default_rng(11)
    B, H, g, Sk, D = 1, 2, 4, 150, 64
    qb = u.random_rows(rng, (B, H * g, 1, D), dtype)
    krec = u.quantise(u.random_rows(rng, (B, H, Sk, D), dtype), dtype)
    x = rng.standard_normal((B, H, Sk, D)).astype(np.float32) * vscale
    vrec = u.quantise(u.bits_of(x, dtype), dtype)
    out = u.to64(gqa.forward_q4(u.dev16(qb, dtype), torch.from_numpy(krec).cuda(),
                                torch.from_numpy(vrec).cuda()))
    _ok(gqa)
    ref = oracle.forward(u.values_of(qb, dtype), u.dequantise(krec, D, dtype),
                         u.dequantise(vrec, D, dtype))
    # fp16 outputs of 1e-5 are subnormal: their step of 2^-24 counts too.
    slack = 2.0 ** -25 * np.sqrt(ref.size) if dtype == "fp16" else 0.0
    assert np.linalg.norm(out - ref) <= 4 * u.UNIT[dtype] * np.linalg.norm(ref) + slack


def test_no_keys_and_no_queries(gqa):
    c = torch.zeros(2, 2, 0, 80, dtype=torch.uint8, device="cuda")
    q = torch.ones(2, 4, 1, 128, dtype=torch.bfloat16, device="cuda")
    assert torch.all(gqa.forward_q4(q, c, c) == 0)
    c = torch.zeros(2, 2, 9, 80, dtype=torch.uint8, device="cuda")
    assert gqa.forward_q4(q[:, :, :0], c, c).shape == (2, 4, 0, 128)
    assert torch.all(torch.isnan(gqa.forward_q4(q, c, c, causal=True, causal_offset=-3)))
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert torch.all(torch.isnan(gqa.forward_q4(q, c, c, kv_lens=lens)))
    _ok(gqa)


def test_reported_lengths_and_pages(gqa):
    rng = np.random.default_rng(12)
    q = u.dev16(u.random_rows(rng, (2, 4, 1, 128), "bf16"), "bf16")
    c = torch.from_numpy(u.quantise(u.random_rows(rng, (4, 1, 64, 128), "bf16"), "bf16")).cuda()
    lens = torch.tensor([70, 5], dtype=torch.int32, device="cuda")
    gqa.forward_q4(q, c[:2], c[:2], kv_lens=lens)
    assert gqa.device_status() == gqa.GQA_ERR_KV_LENGTH
    table = torch.tensor([[0, 4], [1, 2]], dtype=torch.int32, device="cuda")
    gqa.forward_q4(q, c, c, block_table=table)
    assert gqa.device_status() == gqa.GQA_ERR_PAGE
    # A bad entry past the length is never looked at.
    lens = torch.tensor([64, 100], dtype=torch.int32, device="cuda")
    gqa.forward_q4(q, c, c, block_table=table, kv_lens=lens)
    _ok(gqa)


def test_hidden_keys_never_reach_a_token(gqa):
    """NaN records that the mask hides from the one query of each head."""
    rng = np.random.default_rng(13)
    B, Hq, Hkv, Sk, D = 2, 8, 2, 300, 128
    qb = u.random_rows(rng, (B, Hq, 1, D), "bf16")
    rec = [u.quantise(u.random_rows(rng, (B, Hkv, Sk, D), "bf16"), "bf16") for _ in range(2)]
    mask = rng.random((B, 1, Sk)) < 0.5
    clean = [torch.from_numpy(r).cuda() for r in rec]
    dirty = [torch.from_numpy(np.where(mask[:, 0][:, None, :, None], r, 0xFF).astype(np.uint8))
             .cuda() for r in rec]
    q, dm = u.dev16(qb, "bf16"), torch.from_numpy(mask).cuda()
    a, b = gqa.forward_q4(q, *clean, mask=dm), gqa.forward_q4(q, *dirty, mask=dm)
    _ok(gqa)
    assert torch.all(torch.isfinite(a)) and torch.equal(a, b)


def test_nan_key_reaches_its_heads_only(gqa):
    rng = np.random.default_rng(14)
    rec = u.quantise(u.random_rows(rng, (1, 2, 64, 64), "bf16"), "bf16")
    krec = rec.copy()
    krec[0, 1, 40, :4] = 0xFF
    q = u.dev16(u.random_rows(rng, (1, 4, 1, 64), "bf16"), "bf16")
    out = gqa.forward_q4(q, torch.from_numpy(krec).cuda(), torch.from_numpy(rec).cuda())
    _ok(gqa)
    assert torch.all(torch.isfinite(out[:, :2])) and torch.all(torch.isnan(out[:, 2:]))


def test_same_inputs_same_bits(gqa):
    rng = np.random.default_rng(15)
    q = u.dev16(u.random_rows(rng, (2, 16, 1, 128), "bf16"), "bf16")
    c = torch.from_numpy(u.quantise(u.random_rows(rng, (2, 2, 5000, 128), "bf16"), "bf16")).cuda()
    a = gqa.forward_q4(q, c, c)
    for _ in range(20):
        assert torch.equal(a, gqa.forward_q4(q, c, c))
    _ok(gqa)


# ------------------------------------------------------------ the operators as a run

@pytest.mark.parametrize("page", [0, 64])
def test_generation_run(gqa, page):
    """A padded prompt batch stored, a prompt chunk attended, then tokens
    appended and attended one at a time; every step against the oracle."""
    dtype, D, B, Hq, Hkv, cap, n = "bf16", 64, 3, 6, 2, 192, 70
    rng = np.random.default_rng(16 + page)
    R = u.record_bytes(D)
    table = None
    if page:
        shape = (B * 3 + 1, Hkv, page, R)
        table = torch.from_numpy(rng.permutation(B * 3 + 1)[:B * 3].reshape(B, 3)
                                 .astype(np.int32)).cuda()
    else:
        shape = (B, Hkv, cap, R)
    ck = torch.full(shape, 0xFF, dtype=torch.uint8, device="cuda")
    cv = ck.clone()
    ref = [np.zeros((B, Hkv, cap, R), np.uint8) for _ in range(2)]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    held = np.zeros(B, np.int32)

    def append(n, counts=None):
        bits = [u.random_rows(rng, (B, Hkv, n, D), dtype, i == 0) for i in range(2)]
        dc = None if counts is None else torch.from_numpy(counts).cuda()
        gqa.kv_append_q4(ck, cv, *(u.dev16(x, dtype) for x in bits), lens, new_lens=dc,
                         block_table=table)
        for r, x in zip(ref, bits):
            rec = u.quantise(x, dtype)
            for b in range(B):
                c = n if counts is None else counts[b]
                r[b, :, held[b]:held[b] + c] = rec[b, :, :c]
        held[:] += n if counts is None else counts

    def attend(Sq):
        qb = u.random_rows(rng, (B, Hq, Sq, D), dtype)
        out = gqa.forward_q4(u.dev16(qb, dtype), ck, cv, causal=True,
                             causal_offset="bottom_right", kv_lens=lens, block_table=table)
        q64 = u.values_of(qb, dtype)
        k64, v64 = (u.dequantise(r, D, dtype) for r in ref)
        kw = dict(causal=True, causal_offset=cap - Sq, kv_lens=held.tolist())
        _check(out, oracle.forward(q64, k64, v64, **kw), _probs(q64, k64, None, 3, **kw),
               ref[1], D, 3, dtype)

    append(n, np.array([70, 33, 1], np.int32))
    attend(33)
    for _ in range(4):
        append(1)
        attend(1)
    _ok(gqa)
    assert np.array_equal(lens.cpu().numpy(), held)
    k, _ = gqa.kv_read_q4(ck, cv, D, torch.bfloat16, kv_lens=lens, block_table=table)
    want = u.dequantise(ref[0], D, dtype)
    for b in range(B):
        assert np.all(np.abs(u.to64(k)[b, :, :held[b]] - want[b, :, :held[b]]) <=
                      (2.0 ** -8 + 2.0 ** -23) * np.abs(want[b, :, :held[b]]))


def test_two_streams(gqa):
    rng = np.random.default_rng(17)
    q = u.dev16(u.random_rows(rng, (1, 8, 1, 128), "bf16"), "bf16")
    cs = [torch.from_numpy(u.quantise(u.random_rows(rng, (1, 1, 9000, 128), "bf16"), "bf16"))
          .cuda() for _ in range(2)]
    want = [gqa.forward_q4(q, c, c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for s, c, o in zip(streams, cs, got):
            o.append(gqa.forward_q4(q, c, c, stream=s.cuda_stream))
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert all(torch.equal(w, x) for x in o)


@pytest.mark.parametrize("Sq", [1, 40])
def test_graphs_side_by_side(gqa, Sq):
    """Two captured steps (append, attend), replayed at the same time on two
    streams, give what eager calls give: neither shares a workspace."""
    rng = np.random.default_rng(18)
    B, Hq, Hkv, D, cap = 1, 8, 2, 128, 6000
    new = [u.dev16(u.random_rows(rng, (B, Hkv, Sq, D), "bf16"), "bf16") for _ in range(4)]
    q = u.dev16(u.random_rows(rng, (B, Hq, Sq, D), "bf16"), "bf16")
    rec = torch.from_numpy(u.quantise(u.random_rows(rng, (B, Hkv, cap, D), "bf16"), "bf16")).cuda()
    lens = torch.full((B,), cap - Sq, dtype=torch.int32, device="cuda")
    after = lens + Sq

    def step(c, k, v):
        gqa.kv_append_q4(c[0], c[1], k, v, lens, advance=False)
        return gqa.forward_q4(q, c[0], c[1], causal=True, causal_offset="bottom_right",
                              kv_lens=after)

    caches = [(rec.clone(), rec.clone()) for _ in range(4)]
    want = [step(caches[2 + i], new[2 * i], new[2 * i + 1]) for i in range(2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(caches[i], new[2 * i], new[2 * i + 1]))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w, o)


def test_binding_refuses_on_the_gpu(gqa):
    c = torch.zeros(1, 2, 64, 80, dtype=torch.uint8, device="cuda")
    q = torch.zeros(1, 4, 1, 128, dtype=torch.bfloat16, device="cuda")
    bad = [
        dict(q=q.float()), dict(cache_k=c.view(torch.int8)), dict(cache_v=c[:, :, :32]),
        dict(cache_k=c[:, :1], cache_v=c[:, :1].repeat(1, 3, 1, 1)),
        dict(mask=torch.ones(1, 1, 63, dtype=torch.bool, device="cuda")),
        dict(mask=torch.ones(1, 1, 64, device="cuda")),
        dict(mask=torch.ones(1, 1, 64, dtype=torch.bool)),
        dict(kv_lens=torch.ones(1, dtype=torch.int64, device="cuda")),
        dict(kv_lens=torch.ones(2, dtype=torch.int32, device="cuda")),
        dict(window=3), dict(scale=float("nan")), dict(causal=True, window=-1),
        dict(out=torch.empty(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")),
        dict(out=torch.empty(1, 4, 1, 128, dtype=torch.float16, device="cuda")),
        dict(workspace=torch.zeros(128, dtype=torch.uint8, device="cuda")),
    ]
    for kw in bad:
        args = dict(q=q, cache_k=c, cache_v=c)
        args.update(kw)
        with pytest.raises((ValueError, TypeError, gqa.GQAError)):
            gqa.forward_q4(**args)
    with pytest.raises(gqa.GQAError):  # rows off the 16-byte grid
        flat = torch.zeros(2 * 64 * 88, dtype=torch.uint8, device="cuda")
        odd = flat.as_strided((1, 2, 64, 80), (2 * 64 * 88, 64 * 88, 88, 1))
        gqa.forward_q4(q, odd, odd)
    p = gqa.q4_problem_for(q, c, c)
    assert gqa._lib.gqa_forward_q4(ctypes.byref(p), q.data_ptr(), c.data_ptr(), None, None,
                                   q.data_ptr(), None, 0, None) == gqa.GQA_ERR_NULL
    _ok(gqa)


@pytest.mark.parametrize("dtype,g,Sk,D,lens", [
    ("bf16", 32, 600, 128, None), ("fp16", 64, 300, 64, [300, 1]), ("bf16", 129, 77, 128, None),
    ("fp16", 129, 1000, 128, [1000, 130]), ("bf16", 256, 400, 64, [3, 400]),
    ("fp16", 200, 1, 40, None),
])
def test_one_token_of_many_heads_per_kv_head(gqa, dtype, g, Sk, D, lens):
    _case(gqa, dtype, 2, 2 * g, 2, 1, Sk, D, seed=g + Sk, lens=lens)


def _group_factors(pattern, ratio, S, G, t):
    """Powers of two on the values of each (key, group of 32 dims), [S, G]."""
    f = np.ones((S, G))
    r = 2.0 ** round(np.log2(ratio) / 2)
    if pattern == "apart":           # one group far above, one far below the others
        f[:, 0], f[:, 1] = r, 1.0 / r
    elif pattern == "outlier":       # the keys that matter least hold large values in one group
        f[np.argsort(t)[:S // 8], 0] = ratio
    elif pattern == "turns":         # keys in turn, and late keys of other sizes
        f[0::2, 0], f[1::2, 1] = r, 1.0 / r
        f[S // 2:] /= r
    return f


@pytest.mark.parametrize("Sq", [1, 2])
@pytest.mark.parametrize("pattern", ["apart", "outlier", "turns"])
@pytest.mark.parametrize("dtype,ratio,D", [
    ("bf16", 2.0 ** 10, 128), ("bf16", 2.0 ** 20, 128), ("bf16", 2.0 ** 30, 64),
    ("bf16", 2.0 ** 60, 128), ("fp16", 2.0 ** 10, 128), ("fp16", 2.0 ** 16, 64),
    ("fp16", 2.0 ** 20, 128),
])
def test_groups_of_different_sizes(gqa, dtype, ratio, D, pattern, Sq):
    """Each group of 32 dims keeps its own relative precision, whatever its
    neighbours' values are, and whichever keys hold the large ones."""
    rng = np.random.default_rng(int(np.log2(ratio)) + D)
    B, H, g, S, G = 1, 2, 3, 3000, -(-D // 32)
    q = rng.standard_normal((B, H * g, Sq, D)).astype(np.float32) * 3
    k = rng.standard_normal((B, H, S, D)).astype(np.float32)
    qb, kb = u.bits_of(q, dtype), u.bits_of(k, dtype)
    krec = u.quantise(kb, dtype)
    q64, k64 = u.values_of(qb, dtype), u.dequantise(krec, D, dtype)
    t = (q64[0, 0, 0] @ k64[0, 0].T)
    f = np.repeat(_group_factors(pattern, ratio, S, G, t), 32, -1)[:, :D]
    if dtype == "fp16" and pattern == "outlier":  # (within its range)
        f = f * 2.0 ** -8
    v = rng.standard_normal((B, H, S, D)) * f
    vrec = u.quantise(u.bits_of(v, dtype), dtype)
    v64 = u.dequantise(vrec, D, dtype)
    assert np.all(np.isfinite(v64))
    out = u.to64(gqa.forward_q4(u.dev16(qb, dtype), torch.from_numpy(krec).cuda(),
                                torch.from_numpy(vrec).cuda()))
    _ok(gqa)
    ref = oracle.forward(q64, k64, v64)
    p = _probs(q64, k64, None, g).reshape(B, H, g * Sq, S)
    # Roundings: each weight once to fp16, half a step of 2^-11 of it, times
    # codes of at most 15 scales (fp16 caches: 8, from the middle) and at least
    # 2^-32 of the row's largest weight of the group; fp32 sums and exponents,
    # 2^-14 of the terms; the result once (fp16's subnormal step: 2^-25).
    s = np.repeat(u.parts(vrec, D, dtype)[0], u.GROUP, -1)[..., :D]
    far = 15 if dtype == "bf16" else 8
    ps = np.einsum("bhrs,bhsd->bhrsd", p, s)
    lost = S * 2.0 ** -32 * ps.max(3)
    bound = far * (2.0 ** -11 * ps.sum(3) + lost) + \
        2.0 ** -14 * np.einsum("bhrs,bhsd->bhrd", p, np.abs(v64) + far * s)
    bound = bound.reshape(B, H * g, Sq, D) + 1.01 * u.UNIT[dtype] * np.abs(ref) + 2.0 ** -25
    err = np.abs(out - ref)
    assert np.all(err <= bound), float((err / bound).max())


def test_a_group_up_to_the_largest_number(gqa):
    """Spread over fp16's whole range: the scale is rounded up, and the code of
    the largest number stands for one past it.  Attention does not round it."""
    x = np.zeros((1, 1, 2, 32), np.float32)
    x[0, 0, :, 3], x[0, 0, :, 4] = 65504, 30000
    bits = u.bits_of(x, "fp16")
    rec = u.quantise(bits, "fp16")
    want = u.dequantise(rec, 32, "fp16")
    assert want[0, 0, 0, 3] == 65520.0
    c = torch.from_numpy(rec).cuda()
    k, _ = gqa.kv_read_q4(c, c, 32, torch.float16)
    got = u.to64(k)
    assert np.all(np.isposinf(got[..., 3])) and np.all(np.isfinite(got[..., :3]))
    q = torch.zeros(1, 1, 1, 32, dtype=torch.float16, device="cuda")
    zero = torch.from_numpy(u.quantise(np.zeros_like(bits), "fp16")).cuda()
    both = torch.cat([c[:, :, :1], zero[:, :, :1]], 2)
    out = u.to64(gqa.forward_q4(q, both, both))  # the mean of the two keys
    _ok(gqa)
    assert abs(out[0, 0, 0, 3] - 32760.0) <= 2.0 ** -11 * 32760 * 2
