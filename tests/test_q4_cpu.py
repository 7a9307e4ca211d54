"""The 4-bit cache without a GPU: records' sizes, refusals and plans, and the
record definition itself."""
import ctypes

import numpy as np
import pytest

import q4_util as u


@pytest.fixture(scope="module")
def gqa():
    import grouped_query_attention_fwd_b200 as m
    return m


def test_record_bytes(gqa):
    for D in range(0, 200):
        want = u.record_bytes(D) if D % 8 == 0 and 8 <= D <= 128 else 0
        assert gqa._lib.gqa_q4_record_bytes(D) == want
    assert gqa._lib.gqa_q4_record_bytes(-8) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [8, 24, 32, 80, 128])
def test_definition_is_within_half_a_step(dtype, D):
    rng = np.random.default_rng(D)
    bits = u.random_rows(rng, (2, 3, 17, D), dtype, keys=True)
    x = u.values_of(bits, dtype)
    rec = u.quantise(bits, dtype)
    s = np.repeat(u.parts(rec, D, dtype)[0], u.GROUP, -1)[..., :D]
    # The scale is short of (max - min) / 15 by at most half a step of its
    # type, so the top value may be off by 15 * UNIT steps more.
    assert np.all(np.abs(u.dequantise(rec, D, dtype) - x) <= s * (0.5 + 15 * u.UNIT[dtype]))
    # The minimum is kept exactly.
    for g in range(-(-D // 32)):
        xs = x[..., 32 * g:32 * g + 32]
        assert np.array_equal(u.dequantise(rec, D, dtype)[..., 32 * g:32 * g + 32].min(-1),
                              xs.min(-1))


def test_definition_corner_groups():
    x = np.zeros((1, 1, 6, 32), np.float32)
    x[0, 0, 0] = 2.5                       # constant: scale 0
    x[0, 0, 1, 3] = np.nan
    x[0, 0, 2, 4] = np.inf
    x[0, 0, 3, 5], x[0, 0, 3, 6] = 3e38, -3e38  # spread overflows fp32
    x[0, 0, 4, :16] = -1.0
    rec = u.quantise(u.bits_of(x, "bf16"), "bf16")
    y = u.dequantise(rec, 32, "bf16")
    assert np.array_equal(y[0, 0, 0], np.full(32, 2.5))
    assert np.all(np.isnan(y[0, 0, 1:4]))
    assert y[0, 0, 4, 0] == -1.0 and abs(y[0, 0, 4, 31]) <= 15 * 2.0 ** -8 / 15
    assert np.array_equal(y[0, 0, 5], np.zeros(32))


def _problem(gqa, B=2, Hq=8, Hkv=2, Sq=1, Sk=100, D=128, dtype=0, mask=False, **over):
    R = gqa._lib.gqa_q4_record_bytes(D) or 16
    q, o = (Hq * Sq * D, Sq * D, D, 1), (Hq * Sq * D, Sq * D, D, 1)
    k = over.pop("k_stride", (Hkv * Sk * R, Sk * R, R, 1))
    p = gqa.make_problem(dtype, B, Hq, Hkv, Sq, Sk, D, over.pop("q_stride", q), k,
                         over.pop("v_stride", k), o, (Sq * Sk, Sk, 1) if mask else None,
                         causal=over.pop("causal", False), scale=over.pop("scale", None))
    for name, v in over.items():
        setattr(p, name, v)
    return p


def _rc(gqa, p):
    plan = gqa.Plan()
    return gqa._lib.gqa_query_q4(ctypes.byref(p), 148, ctypes.byref(plan)), plan


@pytest.mark.parametrize("kw,code", [
    (dict(), 0),
    (dict(dtype=2), 0),
    (dict(D=24), 0),
    (dict(D=8), 0),
    (dict(dtype=1), 4),                       # fp32
    (dict(dtype=7), 8),
    (dict(D=12), 4),
    (dict(D=136), 4),
    (dict(D=256), 4),
    (dict(Hq=9), 2),
    (dict(batch=-1), 2),
    (dict(k_stride=(16000, 8000, 80, 2)), 3),  # record bytes not contiguous
    (dict(k_stride=(16000, 8000, 72, 1)), 3),  # rows off the 16-byte grid
    (dict(v_stride=(16000, 8008, 80, 1)), 3),
    (dict(k_stride=(-16000, 8000, 80, 1)), 3),
    (dict(window=5), 8),                       # window without causal
    (dict(scale=float("inf")), 8),
])
def test_forward_validation(gqa, kw, code):
    rc, _ = _rc(gqa, _problem(gqa, **kw))
    assert rc == code, gqa.status_string(rc)


def test_paged_validation(gqa):
    table = ctypes.c_int32(0)
    base = dict(block_table=ctypes.addressof(table), block_table_stride=2, page_size=64,
                num_pages=4)
    assert _rc(gqa, _problem(gqa, **base))[0] == 0
    for over in (dict(page_size=48), dict(page_size=0), dict(num_pages=0),
                 dict(block_table_stride=1)):
        assert _rc(gqa, _problem(gqa, **{**base, **over}))[0] == 2


def test_forward_nulls(gqa):
    assert gqa._lib.gqa_query_q4(None, 148, ctypes.byref(gqa.Plan())) == 1
    assert gqa._lib.gqa_query_q4(ctypes.byref(_problem(gqa)), 148, None) == 1
    # Without a device a call is an error, never a fallback.
    import torch
    if not torch.cuda.is_available():
        p = _problem(gqa)
        assert gqa._lib.gqa_forward_q4(ctypes.byref(p), None, None, None, None, None, None, 0,
                                       None) == 9


def test_plans(gqa):
    rc, plan = _rc(gqa, _problem(gqa, B=16, Hq=32, Hkv=8, Sk=4096))
    assert rc == 0 and plan.algorithmic_bytes == 2 * 16 * 32 * 128 * 2 + 2 * 16 * 8 * 4096 * 80
    assert plan.workspace_bytes >= 256 and plan.workspace_bytes % 256 == 0
    assert _rc(gqa, _problem(gqa, B=0))[1].kernel == 0
    assert _rc(gqa, _problem(gqa, Sk=0))[1].kernel == 4
    p = _problem(gqa, causal=True)
    p.causal_offset = -5
    assert _rc(gqa, p)[1].kernel == 5


def _desc(gqa, B=2, Hkv=2, cap=100, D=64, n=3, **over):
    R = u.record_bytes(D) if D % 8 == 0 else 32
    d = gqa.Q4RowsDesc()
    d.dtype, d.batch, d.heads_kv, d.capacity, d.head_dim, d.n = 0, B, Hkv, cap, D, n
    for i, s in enumerate((Hkv * cap * R, cap * R, R, 1)):
        d.cache_k_stride[i] = d.cache_v_stride[i] = s
    for i, s in enumerate((Hkv * n * D, n * D, D, 1)):
        d.k_stride[i] = d.v_stride[i] = s
    for name, v in over.items():
        if isinstance(v, tuple):
            for i, s in enumerate(v):
                getattr(d, name)[i] = s
        else:
            setattr(d, name, v)
    return d


@pytest.mark.parametrize("over,append,read", [
    (dict(), 1, 1),  # null pointers: everything before them was accepted
    (dict(dtype=1), 4, 4),
    (dict(dtype=5), 8, 8),
    (dict(D=20), 4, 4),
    (dict(batch=-1), 2, 2),
    (dict(heads_kv=0), 2, 2),
    (dict(n=-1), 2, 2),
    (dict(n=101), 2, 1),                        # longer than the cache: nothing can be appended
    (dict(start=4), 8, 1),
    (dict(start=-1), 8, 8),
    (dict(advance=1), 1, 8),
    (dict(counts=64), 1, 8),
    (dict(starts=64), 8, 1),
    (dict(cache_k_stride=(9600, 4800, 40, 1)), 3, 3),
    (dict(cache_v_stride=(9600, 4800, 48, 2)), 3, 3),
    (dict(k_stride=(384, 192, 64, 2)), 3, 3),
    (dict(v_stride=(384, -192, 64, 1)), 3, 3),
    (dict(block_table=64, block_table_stride=1, page_size=64, num_pages=9), 2, 2),
    (dict(block_table=64, block_table_stride=2, page_size=64, num_pages=0), 2, 2),
    (dict(batch=1 << 20, heads_kv=1 << 12), 4, 4),  # more heads than 32 bits count
    (dict(batch=0), 0, 0),
    (dict(n=0), 0, 0),
])
def test_rows_validation(gqa, over, append, read):
    d = _desc(gqa, **over)
    assert gqa._lib.gqa_kv_append_q4(ctypes.byref(d), None, None, None, None, None, None, 0,
                                     None) == append
    assert gqa._lib.gqa_kv_read_q4(ctypes.byref(d), None, None, None, None, None, None, 0,
                                   None) == read


def test_rows_pointers(gqa):
    # Addresses are checked, never read, before a launch: made-up ones do.
    d = _desc(gqa)
    lib = gqa._lib

    def append(ck=256, k=512, lens=1024, ws=4096, nbytes=256):
        return lib.gqa_kv_append_q4(ctypes.byref(d), ck, 256, k, 512, lens, ws, nbytes, None)

    assert append(ck=None) == 1 and append(k=None) == 1 and append(lens=None) == 1
    assert append(ws=None) == 5 and append(ws=4100) == 5 and append(nbytes=255) == 5
    assert append(ck=264) == 3 and append(k=513) == 3 and append(lens=1026) == 3
    assert lib.gqa_kv_append_q4(None, 256, 256, 512, 512, 1024, 4096, 256, None) == 1


def test_binding_refuses(gqa):
    import torch
    c = torch.zeros(1, 2, 64, 80, dtype=torch.uint8)
    x = torch.zeros(1, 2, 1, 128, dtype=torch.bfloat16)
    lens = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        gqa.forward_q4(x, c, c)
    with pytest.raises(ValueError):
        gqa.kv_append_q4(c, c, x, x, lens)
    with pytest.raises(ValueError):
        gqa.kv_read_q4(c, c, 128, torch.bfloat16)
    with pytest.raises(ValueError):
        gqa.q4_record_bytes(130)
    with pytest.raises(TypeError):
        gqa.query_q4(x.float(), c, c, sm_count=148)
    with pytest.raises(ValueError):
        gqa.query_q4(x, c[..., :64], c[..., :64], sm_count=148)
    assert gqa.query_q4(x, c, c, sm_count=148)["kernel_name"] == "q4"


@pytest.mark.parametrize("B,Hkv,g,Sq,Sk,D,entries,heads", [
    # Widths of the slices (entries x heads); the prefill sorts its items by
    # cost, which takes scratch, in the narrow ones only.
    (1, 8, 8, 40000, 40000, 64, [1], [6, 2]),
    (1, 8, 16, 43000, 43000, 128, [1], [3, 3, 2]),
    (1, 4, 16, 40960, 40960, 128, [1], [3, 1]),
    (1, 8, 16, 28672, 28672, 80, [1], [7, 1]),
    (5, 1, 128, 2050, 65536, 64, [4, 1], [1]),
    # And in all of them, or in none.
    (2, 24, 4, 1024, 8192, 128, [1, 1], [16, 8]),
    (1, 8, 16, 60000, 60000, 128, [1], [2, 2, 2, 2]),
])
def test_slices_of_every_width_keep_clear_of_the_keys(gqa, B, Hkv, g, Sq, Sk, D, entries, heads):
    rc, plan = _rc(gqa, _problem(gqa, B, Hkv * g, Hkv, Sq, Sk, D, mask=True))
    assert rc == 0 and gqa.KERNEL_NAMES[plan.kernel] == "q4_prefill"
    head = -(-Sk * D * 2 // 256) * 256
    keys_at = plan.workspace_bytes - 2 * entries[0] * heads[0] * head
    launches = work = 0
    for nb in entries:
        for nh in heads:
            part = gqa.query_problem(gqa.make_problem(
                0, nb, nh * g, nh, Sq, Sk, D, *[(nh * g * Sq * D, Sq * D, D, 1)] * 4,
                (Sq * Sk, Sk, 1)), 148)
            assert part.workspace_bytes <= keys_at, (nb, nh)
            launches += 1 + part.launches
            work += part.work_units
    assert plan.launches == launches and plan.work_units == work


@pytest.mark.parametrize("g", [128, 129, 200, 256, 1000])
@pytest.mark.parametrize("D", [64, 128])
def test_one_token_of_many_heads_per_kv_head(gqa, g, D):
    """More query heads per kv head than a 128-row tile holds: planned as the
    16-bit library plans it, for one token; refused for more."""
    rc, plan = _rc(gqa, _problem(gqa, 2, 3 * g, 3, 1, 500, D))
    assert rc == 0 and gqa.KERNEL_NAMES[plan.kernel] == "q4"
    assert plan.work_units == 2 * 3 * -(-g // 8) * 4
    rc, _ = _rc(gqa, _problem(gqa, 2, 3 * g, 3, 2, 500, D))
    assert rc == (0 if g <= 128 else 4)


def test_no_non_coherent_loads():
    """The kernels over records start while earlier kernels of the stream still
    write what they read (masks, block tables, lengths, partials): none of it
    may go through the read-only path, which promises that nothing writes."""
    import glob
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "grouped_query_attention_fwd_b200", "csrc")
    sources = glob.glob(os.path.join(csrc, "*q4*"))
    assert len(sources) >= 5
    for path in sources:
        text = open(path).read()
        assert not re.search(r"__ldg\s*\(|\.nc\.|__restrict__", text), path


@pytest.mark.parametrize("B,Hkv,g,Sq,Sk,D,way,times", [
    # Measured with each way, us: decode, 128-row tiles, slices.  Many short
    # groups: their changes cost a decode more than their units.
    (16, 8, 8, 8, 1024, 128, "q4_chunk", (96, 38, 45)),
    (16, 8, 8, 6, 1024, 64, "q4_chunk", (49, 29, 31)),
    (2, 8, 8, 24, 1024, 128, "q4_chunk", (46, 26, 29)),
    # Few groups, long keys: the tiles' partials cost more than unpacking again.
    (1, 2, 8, 16, 16384, 64, "q4", (23, 45, 215)),
    (1, 2, 4, 32, 16384, 128, "q4", (30, 49, 256)),
    (2, 8, 8, 128, 1024, 64, "q4_prefill", (110, 36, 26)),
])
def test_the_way_follows_measured_times(gqa, B, Hkv, g, Sq, Sk, D, way, times):
    p = _problem(gqa, B, Hkv * g, Hkv, Sq, Sk, D, causal=True)
    p.causal_offset = Sk - Sq
    assert gqa.KERNEL_NAMES[_rc(gqa, p)[1].kernel] == way


def test_workspace_head(gqa):
    """What a captured call clears is what the header says has to be zero."""
    import os
    import re
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                          "gqa.h")
    said = re.search(r"#define GQA_WORKSPACE_HEAD_BYTES (\d+)", open(header).read())
    assert gqa.WORKSPACE_HEAD_BYTES == int(said.group(1))
