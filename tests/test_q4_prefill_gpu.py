"""Long query blocks over the 4-bit cache: 128-row tiles that unpack the records
once, or records read back into scratch, a slice of the heads at a time, and
attended to there.  Checked against attention
in 64 bits (torch, on the device) over the values the records stand for."""
import math

import numpy as np
import pytest
import torch

import q4_util as u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gqa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import grouped_query_attention_fwd_b200 as m
    return m


def _records(gqa, B, Hkv, S, D, dtype, seed, keys):
    """Records written by kv_append_q4 (tested on its own), and their values in
    float64, decoded from the bytes here."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, Hkv, S, D, generator=g, device="cuda")
    if keys:
        x += torch.randn(1, Hkv, 1, D, generator=g, device="cuda")
    x = x.to(u.TORCH[dtype])
    c = torch.zeros(B, Hkv, S, u.record_bytes(D), dtype=torch.uint8, device="cuda")
    gqa.kv_append_q4(c, c.clone(), x, x, torch.zeros(B, dtype=torch.int32, device="cuda"))
    G = -(-D // 32)
    par = c[..., :4 * G].contiguous().view(u.TORCH[dtype]).double().unflatten(-1, (G, 2))
    body = c[..., 16:].long()
    code = torch.stack([body % 16, body // 16], -1).double().flatten(-2).unflatten(-1, (G, 32))
    return c, (code * par[..., :1] + par[..., 1:]).flatten(-2)[..., :D]


CASES = [
    # B, Hq, Hkv, Sq, Sk, D, dtype, lens, page, window, mask, kernel
    (4, 8, 2, 512, 2048, 128, "bf16", None, 0, 0, False, "q4_chunk"),
    (4, 8, 2, 512, 2048, 128, "fp16", [2048, 1, 513, 700], 64, 0, False, "q4_chunk"),
    (3, 12, 2, 700, 1536, 64, "bf16", [1536, 900, 701], 128, 300, False, "q4_prefill"),
    (2, 8, 1, 33, 20000, 96, "fp16", None, 0, 0, False, "q4_chunk"),
    (3, 8, 2, 30, 20032, 128, "bf16", [20000, 30, 9000], 64, 0, False, "q4_chunk"),
    (2, 4, 1, 31, 60000, 64, "fp16", None, 0, 50000, False, "q4_chunk"),
    (2, 16, 1, 9, 30000, 128, "bf16", [30000, 0], 0, 0, False, "q4_chunk"),
    (1, 5, 1, 300, 12345, 40, "bf16", None, 0, 9000, False, "q4_chunk"),
    (5, 3, 3, 500, 1000, 120, "fp16", [1000, 300, 299, 129, 128], 0, 0, False, "q4_chunk"),
    (12, 8, 2, 1024, 8192, 128, "bf16", None, 0, 0, False, "q4_chunk"),
    (4, 8, 4, 640, 1111, 80, "bf16", None, 0, 0, True, "q4_prefill"),
    (1, 32, 8, 2048, 2048, 128, "bf16", None, 0, 0, False, "q4_prefill"),
    (2, 32, 8, 1500, 1536, 64, "fp16", [1536, 1501], 64, 200, False, "q4_prefill"),
    (2, 96, 24, 1024, 8192, 128, "bf16", [8192, 5000], 64, 0, True, "q4_prefill"),
]


@pytest.mark.parametrize("case", CASES)
def test_long_query_blocks(gqa, case):
    B, Hq, Hkv, Sq, Sk, D, dtype, lens, page, window, masked, kernel = case
    ck, k64 = _records(gqa, B, Hkv, Sk, D, dtype, 1, True)
    cv, v64 = _records(gqa, B, Hkv, Sk, D, dtype, 2, False)
    gen = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(B, Hq, Sq, D, generator=gen, device="cuda").to(u.TORCH[dtype])
    kw = dict(causal=True, causal_offset="bottom_right", window=window)
    held = lens or [Sk] * B
    if lens:
        kw["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b in range(B):  # NaN scales past each length
            ck[b, :, lens[b]:] = cv[b, :, lens[b]:] = 0xFF
    mask = None
    if masked:
        mask = torch.rand(B, Sq, Sk, generator=gen, device="cuda") < 0.7
        mask[:, 5] = False  # an empty row
        kw["mask"] = mask
    if page:
        rng = np.random.default_rng(0)
        per = Sk // page
        order = torch.from_numpy(rng.permutation(B * per + 2)[:B * per].reshape(B, per)).cuda()
        pools = []
        for c in (ck, cv):
            pool = torch.full((B * per + 2, Hkv, page, c.shape[-1]), 0xFF, dtype=torch.uint8,
                              device="cuda")
            pool[order] = c.unflatten(2, (per, page)).transpose(1, 2)
            pools.append(pool)
        kw["block_table"] = order.int()
    else:
        pools = [ck, cv]
    plan = gqa.query_q4(q, *pools, **kw)
    assert plan["kernel_name"] == kernel
    if kernel == "q4_prefill" and Hkv == 24:  # several slices, one of them narrower
        assert plan["launches"] > 4
    # Rows behind the result are left alone: the output is a part of a larger buffer.
    buf = torch.full((B, Hq, Sq + 1, D), 7.0, dtype=q.dtype, device="cuda")
    out = gqa.forward_q4(q, *pools, out=buf[:, :, :Sq], **kw)
    assert gqa.device_status() == gqa.GQA_OK
    assert torch.all(buf[:, :, Sq] == 7.0)

    g, unit, scale = Hq // Hkv, u.UNIT[dtype], 1.0 / math.sqrt(D)
    worst, off, norm = 0.0, 0.0, 0.0
    for b in range(B):
        n = held[b]
        if n == 0:  # no key at all: NaN
            assert torch.all(torch.isnan(out[b]))
            continue
        i = torch.arange(Sq, device="cuda")[:, None] + n - Sq
        j = torch.arange(n, device="cuda")[None, :]
        see = j <= i
        if window:
            see &= j > i - window
        if masked:
            see &= mask[b, :, :n]
        for h in range(Hq):
            k, v = k64[b, h // g, :n], v64[b, h // g, :n]
            qh = q[b, h].double()
            s = (qh @ k.T * scale).masked_fill(~see, -math.inf)
            p = torch.softmax(s, -1)
            ref = p @ v
            # Roundings, each at most `unit` relative: keys (a score moves by
            # at most scale * unit * sum |q k|, a weight by twice that), values,
            # weights, the output; 2^-14 for fp32 sums and exponentials.
            move = 2.1 * scale * unit * (qh.abs() @ k.abs().T).amax(-1, keepdim=True)
            bound = (p @ v.abs()) * (2.02 * unit + move + 2.0 ** -14) + 1.01 * unit * ref.abs() + \
                2.0 ** -24
            got = out[b, h].double()
            empty = ~see.any(-1)
            assert torch.equal(torch.isnan(got).all(-1), empty)
            assert torch.equal(torch.isnan(got), torch.isnan(ref))
            err = (got - ref)[~empty].abs()
            worst = max(worst, float((err / bound[~empty]).max()) if err.numel() else 0.0)
            off += float(err.square().sum())
            norm += float(ref[~empty].square().sum())
    assert worst <= 1.0, worst
    assert math.sqrt(off) <= 1e-2 * math.sqrt(norm)


def test_chunk_equals_short_blocks(gqa):
    """The two ways of attending agree: a long block's last rows against a
    short block of the same queries."""
    ck, _ = _records(gqa, 4, 2, 2048, 128, "bf16", 5, True)
    cv, _ = _records(gqa, 4, 2, 2048, 128, "bf16", 6, False)
    gen = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randn(4, 8, 512, 128, generator=gen, device="cuda").bfloat16()
    kw = dict(causal=True, causal_offset="bottom_right")
    assert gqa.query_q4(q, ck, cv, **kw)["kernel_name"] == "q4_chunk"
    tail = q[:, :, -4:]
    assert gqa.query_q4(tail, ck, cv, **kw)["kernel_name"] == "q4"
    a = gqa.forward_q4(q, ck, cv, **kw)[:, :, -4:].double()
    b = gqa.forward_q4(tail, ck, cv, **kw).double()
    assert gqa.device_status() == gqa.GQA_OK
    assert float((a - b).norm() / b.norm()) <= 1e-2


@pytest.mark.parametrize("Sq,masked", [(700, True), (100, False)])
def test_long_block_in_a_graph(gqa, Sq, masked):
    ck, _ = _records(gqa, 4, 2, 2048, 64, "fp16", 8, True)
    cv, _ = _records(gqa, 4, 2, 2048, 64, "fp16", 9, False)
    gen = torch.Generator(device="cuda").manual_seed(10)
    q = torch.randn(4, 8, Sq, 64, generator=gen, device="cuda").half()
    lens = torch.tensor([2048, 700, 1500, 2000], dtype=torch.int32, device="cuda")
    kw = dict(causal=True, causal_offset="bottom_right", kv_lens=lens)
    if masked:
        kw["mask"] = torch.rand(4, Sq, 2048, generator=gen, device="cuda") < 0.9
    assert gqa.query_q4(q, ck, cv, **kw)["kernel_name"] == ("q4_prefill" if masked else "q4_chunk")
    want = gqa.forward_q4(q, ck, cv, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = gqa.forward_q4(q, ck, cv, **kw)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_narrow_last_slice_keeps_its_keys(gqa):
    """Five entries in slices of four and one, of which only the narrow one sorts
    its items: its first keys, where a wrong place for the order would fall, are
    all that every other query sees."""
    B, g, Sq, Sk, D = 5, 128, 2050, 65536, 64
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    ck, k64 = _records(gqa, B, 1, Sk, D, "bf16", 11, True)
    cv, v64 = _records(gqa, B, 1, Sk, D, "bf16", 12, False)
    gen = torch.Generator(device="cuda").manual_seed(13)
    q = torch.randn(B, g, Sq, D, generator=gen, device="cuda").bfloat16()
    mask = torch.zeros(B, Sq, Sk, dtype=torch.bool, device="cuda")
    mask[:, ::2, :40] = True
    mask[:, 1::2, 5::3] = True
    plan = gqa.query_q4(q, ck, cv, mask=mask)
    assert plan["kernel_name"] == "q4_prefill" and plan["launches"] == 7
    out = gqa.forward_q4(q, ck, cv, mask=mask)
    assert gqa.device_status() == gqa.GQA_OK
    unit, scale = u.UNIT["bf16"], 1.0 / math.sqrt(D)
    rows = [0, 1, 2, 255, 256, 1024, 1025, 2048, 2049]
    for b in range(B):
        k, v = k64[b, 0], v64[b, 0]
        for i in rows:
            qi = q[b, :, i].double()
            s = (qi @ k.T * scale).masked_fill(~mask[b, i], -math.inf)
            p = torch.softmax(s, -1)
            ref = p @ v
            # The roundings of test_long_query_blocks.
            move = 2.1 * scale * unit * (qi.abs() @ k.abs().T).amax(-1, keepdim=True)
            bound = (p @ v.abs()) * (2.02 * unit + move + 2.0 ** -14) + 1.01 * unit * ref.abs() + \
                2.0 ** -24
            err = (out[b, :, i].double() - ref).abs()
            assert torch.all(err <= bound), (b, i, float((err / bound).max()))
            assert float(err.norm() / ref.norm()) <= 1e-2, (b, i)


@pytest.mark.parametrize("Sq,window,page,masked,kernel", [
    (1, 0, 0, False, "q4"), (3, 100, 64, False, "q4"),
    (100, 0, 0, False, "q4_chunk"), (300, 0, 64, False, "q4_chunk"),
    (300, 700, 0, False, "q4_chunk"), (220, 700, 128, False, "q4_chunk"),
    (700, 0, 0, True, "q4_prefill"), (700, 0, 64, True, "q4_prefill"),
    (701, 444, 0, True, "q4_prefill"),
])
def test_keys_that_no_query_sees_hold_anything(gqa, Sq, window, page, masked, kernel):
    """A cache written up to a position, without lengths: NaN records past the
    last query's diagonal, and below the first one's window, change nothing."""
    B, Hq, Hkv, Sk, D, at = 3, 8, 2, 2944, 128, 1701
    ck, _ = _records(gqa, B, Hkv, Sk, D, "bf16", 21, True)
    cv, _ = _records(gqa, B, Hkv, Sk, D, "bf16", 22, False)
    gen = torch.Generator(device="cuda").manual_seed(23)
    q = torch.randn(B, Hq, Sq, D, generator=gen, device="cuda").bfloat16()
    kw = dict(causal=True, causal_offset=at - Sq, window=window)
    if masked:
        kw["mask"] = torch.rand(B, Sq, Sk, generator=gen, device="cuda") < 0.8
    if page:
        per = Sk // page
        order = torch.randperm(B * per, generator=gen, device="cuda").view(B, per)
        kw["block_table"] = order.int()

    def call(k, v):
        if page:
            pools = []
            for c in (k, v):
                pool = torch.empty(B * per, Hkv, page, c.shape[-1], dtype=torch.uint8,
                                   device="cuda")
                pool[order] = c.unflatten(2, (per, page)).transpose(1, 2)
                pools.append(pool)
            k, v = pools
        assert gqa.query_q4(q, k, v, **kw)["kernel_name"] == kernel
        return gqa.forward_q4(q, k, v, **kw)

    clean = call(ck, cv)
    for c in (ck, cv):
        c[:, :, at:] = 0xFF
        if window:
            c[:, :, :at - Sq + 1 - window] = 0xFF
    dirty = call(ck, cv)
    assert gqa.device_status() == gqa.GQA_OK
    assert torch.all(torch.isfinite(clean)) and torch.equal(clean, dirty)


@pytest.mark.parametrize("scale", [0.02, 0.3, 0.0, -0.11, -1.0])
@pytest.mark.parametrize("Sq,masked,causal,dtype,kernel", [
    (1, False, False, "bf16", "q4"), (3, True, True, "fp16", "q4"), (2, False, True, "bf16", "q4"),
    (40, False, False, "bf16", "q4_chunk"), (300, False, False, "fp16", "q4_chunk"),
    (300, False, True, "bf16", "q4_chunk"), (700, True, False, "bf16", "q4_prefill"),
])
def test_scales_and_blocks_without_a_diagonal(gqa, Sq, masked, causal, dtype, kernel, scale):
    """Scales other than 1 / sqrt(D), zero and negative ones among them, and
    long blocks whose queries see every key of their sequence."""
    B, Hq, Hkv, Sk, D = 2, 16, 2, 3700, 128
    ck, k64 = _records(gqa, B, Hkv, Sk, D, dtype, 31, True)
    cv, v64 = _records(gqa, B, Hkv, Sk, D, dtype, 32, False)
    gen = torch.Generator(device="cuda").manual_seed(33)
    q = torch.randn(B, Hq, Sq, D, generator=gen, device="cuda").to(u.TORCH[dtype])
    lens = torch.tensor([Sk, 2900], dtype=torch.int32, device="cuda")
    kw = dict(scale=scale, kv_lens=lens)
    if causal:
        kw.update(causal=True, causal_offset="bottom_right")
    if masked:
        kw["mask"] = torch.rand(B, Sq, Sk, generator=gen, device="cuda") < 0.7
    assert gqa.query_q4(q, ck, cv, **kw)["kernel_name"] == kernel
    out = gqa.forward_q4(q, ck, cv, **kw)
    assert gqa.device_status() == gqa.GQA_OK
    g, unit = Hq // Hkv, u.UNIT[dtype]
    for b, n in enumerate(lens.tolist()):
        see = torch.ones(Sq, n, dtype=torch.bool, device="cuda")
        if causal:
            top = torch.arange(Sq, device="cuda")[:, None] + n - Sq
            see = torch.arange(n, device="cuda") <= top
        if masked:
            see = see & kw["mask"][b, :, :n]
        for h in range(Hq):
            k, v, qh = k64[b, h // g, :n], v64[b, h // g, :n], q[b, h].double()
            p = torch.softmax((qh @ k.T * scale).masked_fill(~see, -math.inf), -1)
            ref = p @ v
            # The roundings of test_long_query_blocks; fewer in the short blocks.
            move = 2.1 * abs(scale) * unit * (qh.abs() @ k.abs().T).amax(-1, keepdim=True)
            bound = (p @ v.abs()) * (2.02 * unit + move + 2.0 ** -14) + \
                1.01 * unit * ref.abs() + 2.0 ** -24
            err = (out[b, h].double() - ref).abs()
            assert torch.all(err <= bound), float((err / bound).max())


def _chunk_case(gqa, D, Sq, Sk, kf, vf, qf, seed, dtype="bf16", groups=None):
    """A block whose K, V and Q are kf, vf and qf times normal numbers (groups:
    factors of V's groups of 32 dims); attention in 64 bits over the records,
    and each element's bound with keys, values and weights rounded to `unit`."""
    B, Hq, Hkv = 2, 8, 2
    gen = torch.Generator(device="cuda").manual_seed(seed)
    caches, values = [], []
    for f, parts in ((kf, None), (vf, groups)):
        x = torch.randn(B, Hkv, Sk, D, generator=gen, device="cuda") * f
        if parts:
            for i, y in enumerate(parts):
                x[..., 32 * i:32 * i + 32] *= y
        x = x.to(u.TORCH[dtype])
        c = torch.zeros(B, Hkv, Sk, u.record_bytes(D), dtype=torch.uint8, device="cuda")
        gqa.kv_append_q4(c, c.clone(), x, x, torch.zeros(B, dtype=torch.int32, device="cuda"))
        G = -(-D // 32)
        par = c[..., :4 * G].contiguous().view(u.TORCH[dtype]).double().unflatten(-1, (G, 2))
        code = torch.stack([c[..., 16:] % 16, c[..., 16:] // 16], -1).double().flatten(-2)
        caches.append(c)
        x = code.unflatten(-1, (G, 32)) * par[..., :1] + par[..., 1:]
        values.append(x.flatten(-2)[..., :D])
    q = (torch.randn(B, Hq, Sq, D, generator=gen, device="cuda") * qf).to(u.TORCH[dtype])
    kw = dict(causal=True, causal_offset="bottom_right", scale=1.0 / (kf * qf * math.sqrt(D)))
    assert gqa.query_q4(q, *caches, **kw)["kernel_name"] == "q4_chunk"
    see = torch.arange(Sk, device="cuda") <= torch.arange(Sq, device="cuda")[:, None] + Sk - Sq
    ref, move, size = [], [], []
    for b in range(B):
        for h in range(Hq):
            k, v, qh = values[0][b, h // 4], values[1][b, h // 4], q[b, h].double()
            p = torch.softmax((qh @ k.T * kw["scale"]).masked_fill(~see, -math.inf), -1)
            ref.append(p @ v)
            size.append(p @ v.abs())
            move.append(kw["scale"] * (qh.abs() @ k.abs().T).amax(-1, keepdim=True))
    ref, size = (torch.stack(x).view(B, Hq, Sq, D) for x in (ref, size))
    move = torch.stack(move).view(B, Hq, Sq, 1)

    def bound(unit, out):
        return size * (2.02 * unit + 2.1 * unit * move + 2.0 ** -14) + 1.01 * out * ref.abs()

    return q, caches, kw, ref, bound


@pytest.mark.parametrize("D,Sq,Sk", [(128, 512, 2048), (128, 20, 20000), (64, 300, 4000),
                                     (96, 777, 3333)])
def test_bf16_chunks_keep_more_bits_than_bf16(gqa, D, Sq, Sk):
    """bf16 caches are multiplied in fp16 operands: what is off is the result's
    own rounding, in norm within a quarter."""
    q, caches, kw, ref, bound = _chunk_case(gqa, D, Sq, Sk, 1.0, 1.0, 1.0, 41)
    out = gqa.forward_q4(q, *caches, **kw)
    assert gqa.device_status() == gqa.GQA_OK
    err = (out.double() - ref).abs()
    # fp16 roundings of keys, values and weights, bf16's of the result.
    assert torch.all(err <= bound(2.0 ** -11, 2.0 ** -8))
    own = (ref.bfloat16().double() - ref).norm()
    assert float(err.norm() / own) <= 1.25


@pytest.mark.parametrize("D,Sq,Sk", [(128, 512, 2048), (64, 32, 16384)])
@pytest.mark.parametrize("kf,vf,qf,groups", [
    (1.0, 1e-6, 1.0, None), (1.0, 3e4, 1.0, None), (1.0, 1e30, 1.0, None),
    (1e-7, 1.0, 1e7, None), (1e9, 1.0, 1e-9, None), (300.0, 40.0, 1e-20, None),
    (1.0, 1.0, 1e20, None), (1.0, 1.0, 1.0, [1.0, 2.0 ** -18]), (1.0, 1.0, 1.0, [2.0 ** 12, 1.0]),
])
def test_bf16_chunks_of_any_size(gqa, kf, vf, qf, groups, D, Sq, Sk):
    """Keys, values or queries that fp16 would not hold come out as bf16
    operands give them, and the next call is as before."""
    q, caches, kw, ref, bound = _chunk_case(gqa, D, Sq, Sk, kf, vf, qf, 42, groups=groups)
    plan = gqa.query_q4(q, *caches, **kw)
    nq, nc, nkw, nref, nbound = _chunk_case(gqa, D, Sq, Sk, 1.0, 1.0, 1.0, 43)
    ws = torch.zeros(plan["workspace_bytes"], dtype=torch.uint8, device="cuda")
    for _ in range(2):
        out = gqa.forward_q4(q, *caches, workspace=ws, **kw).double()
        off = (out - ref).abs() / bound(2.0 ** -8, 2.0 ** -8)
        assert torch.all(off <= 1.0), float(off.max())
        assert not ws[:256].any()
        out = gqa.forward_q4(nq, *nc, workspace=ws, **nkw).double()
        assert torch.all((out - nref).abs() <= nbound(2.0 ** -11, 2.0 ** -8))
    assert gqa.device_status(ws) == gqa.GQA_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("share", [2.0 ** -6, 2.0 ** -14])
def test_weight_on_a_key_of_zeros(gqa, dtype, share):
    """Nearly all weight on one key whose values are zeros, as heads that have
    nothing to add put it: what the other keys add, `share` of the weight over
    2000 keys, keeps its bits."""
    B, Hq, Hkv, Sq, Sk, D = 1, 8, 2, 512, 2048, 128
    gen = torch.Generator(device="cuda").manual_seed(51)
    t = u.TORCH[dtype]
    k, v = (torch.randn(B, Hkv, Sk, D, generator=gen, device="cuda") for _ in range(2))
    q = torch.randn(B, Hq, Sq, D, generator=gen, device="cuda") * 0.1
    k[:, :, 0], q[..., 0] = 0, 1.0
    k[..., 0] = 0
    # Score of key 0 above the others', whose weights are about equal.
    k[:, :, 0, 0] = math.sqrt(D) * (math.log(Sk) - math.log(share))
    v[:, :, 0] = 0
    k, v, q = k.to(t), v.to(t), q.to(t)
    ck = torch.zeros(B, Hkv, Sk, u.record_bytes(D), dtype=torch.uint8, device="cuda")
    cv = torch.zeros_like(ck)
    gqa.kv_append_q4(ck, cv, k, v, torch.zeros(B, dtype=torch.int32, device="cuda"))
    k64, v64 = [], []
    for c, out in ((ck, k64), (cv, v64)):
        par = c[..., :16].contiguous().view(t).double().unflatten(-1, (4, 2))
        code = torch.stack([c[..., 16:] % 16, c[..., 16:] // 16], -1).double().flatten(-2)
        out.append((code.unflatten(-1, (4, 32)) * par[..., :1] + par[..., 1:]).flatten(-2))
    k64, v64 = k64[0], v64[0]
    kw = dict(causal=True, causal_offset="bottom_right")
    assert gqa.query_q4(q, ck, cv, **kw)["kernel_name"] == "q4_chunk"
    out = gqa.forward_q4(q, ck, cv, **kw).double()
    assert gqa.device_status() == gqa.GQA_OK
    see = torch.arange(Sk, device="cuda") <= torch.arange(Sq, device="cuda")[:, None] + Sk - Sq
    for h in range(Hq):
        kk, vv, qh = k64[0, h // 4], v64[0, h // 4], q[0, h].double()
        p = torch.softmax((qh @ kk.T / math.sqrt(D)).masked_fill(~see, -math.inf), -1)
        assert float(p[:, 0].min()) > 0.5 and not vv[0].any()
        ref = p @ vv
        # The one key's score, off by half a step of fp16, moves all other weights
        # alike: `fit`.  Beside that, keys and values rounded to fp16's 2^-11,
        # weights to that or 2^-32 of the largest, the result to its type (fp16's
        # subnormal step: 2^-25).
        moves = qh.abs() @ kk.abs().T / math.sqrt(D)
        fit = (out[0, h] * ref).sum(-1, keepdim=True) / (ref * ref).sum(-1, keepdim=True)
        assert torch.all((fit - 1).abs() <= 2.1 * 2.0 ** -11 * moves[:, :1] + 2.0 ** -6)
        move = moves[:, 1:].amax(-1, keepdim=True)
        bound = (p @ vv.abs()) * (2.02 * 2.0 ** -11 + 2.1 * 2.0 ** -11 * move + 2.0 ** -14) + \
            2.0 ** -32 * vv.abs().sum(0) + 1.01 * u.UNIT[dtype] * ref.abs() + 2.0 ** -25
        err = (out[0, h] - fit * ref).abs()
        assert torch.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("Sq,Sk", [(512, 2048), (20, 20000)])
def test_one_record_past_fp16(gqa, Sq, Sk):
    """A single value row that fp16 does not hold: the CTAs that meet it go over
    to bf16, and their partials meet those of the others."""
    q, (ck, cv), kw, _, _ = _chunk_case(gqa, 128, Sq, Sk, 1.0, 1.0, 1.0, 44)
    B, Hq, D, at = 2, 8, 128, Sk // 3
    row = torch.zeros(1, 2, 1, D, device="cuda")
    row[:, 1] = torch.linspace(-3e5, 3e5, D, device="cuda")
    lens = torch.tensor([at], dtype=torch.int32, device="cuda")
    keep = cv[0, 0, at].clone()
    gqa.kv_append_q4(cv[:1].clone(), cv[:1], row.bfloat16(), row.bfloat16(), lens)
    cv[0, 0, at] = keep  # (head 0 stays as it was)
    vals = []
    for c in (ck, cv):
        par = c[..., :16].contiguous().view(torch.bfloat16).double().unflatten(-1, (4, 2))
        code = torch.stack([c[..., 16:] % 16, c[..., 16:] // 16], -1).double().flatten(-2)
        vals.append((code.unflatten(-1, (4, 32)) * par[..., :1] + par[..., 1:]).flatten(-2))
    out = gqa.forward_q4(q, ck, cv, **kw).double()
    assert gqa.device_status() == gqa.GQA_OK
    see = torch.arange(Sk, device="cuda") <= torch.arange(Sq, device="cuda")[:, None] + Sk - Sq
    for b in range(B):
        for h in range(Hq):
            k, v, qh = vals[0][b, h // 4], vals[1][b, h // 4], q[b, h].double()
            p = torch.softmax((qh @ k.T * kw["scale"]).masked_fill(~see, -math.inf), -1)
            ref = p @ v
            # bf16's roundings of keys, values and weights where the row is.
            unit = 2.0 ** -8 if b == 0 else 2.0 ** -11
            move = kw["scale"] * (qh.abs() @ k.abs().T).amax(-1, keepdim=True)
            bound = (p @ v.abs()) * (2.02 * unit + 2.1 * unit * move + 2.0 ** -14) + \
                1.01 * 2.0 ** -8 * ref.abs()
            err = (out[b, h] - ref).abs()
            assert torch.all(err <= bound), (b, h, float((err / bound).max()))
