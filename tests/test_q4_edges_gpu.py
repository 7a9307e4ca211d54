"""The 4-bit cache where calls meet: threads, streams, captured steps, a shared
workspace, offsets past 32 bits, and a wait that runs out.  Values are checked
against eager calls on fresh workspaces, which other tests check against the
oracle; equal launches give equal bits."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gqa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import grouped_query_attention_fwd_b200 as m
    return m


def _cache(gqa, B, Hkv, S, D, dtype=torch.bfloat16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ck = torch.zeros(B, Hkv, S, gqa.q4_record_bytes(D), dtype=torch.uint8, device="cuda")
    cv = torch.zeros_like(ck)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(B, Hkv, S, D, generator=gen, device="cuda").to(dtype) for _ in range(2))
    gqa.kv_append_q4(ck, cv, k, v, lens)
    return ck, cv


def _q(B, Hq, Sq, D, dtype=torch.bfloat16, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(B, Hq, Sq, D, generator=gen, device="cuda").to(dtype)


# One call of each way of attending, over the same cache: (Sq, mask, kernel).
WAYS = [(1, False, "q4"), (1, True, "q4"), (512, False, "q4_chunk"), (700, True, "q4_prefill")]


def _ways(gqa, ck, cv):
    B, Hkv, S, _ = ck.shape
    calls = []
    for i, (Sq, masked, kernel) in enumerate(WAYS):
        q = _q(B, 4 * Hkv, Sq, 128, seed=10 + i)
        kw = dict(causal=True, causal_offset="bottom_right")
        if masked:
            gen = torch.Generator(device="cuda").manual_seed(20 + i)
            kw["mask"] = torch.rand(B, Sq, S, generator=gen, device="cuda") < 0.8
        assert gqa.query_q4(q, ck, cv, **kw)["kernel_name"] == kernel
        calls.append((q, kw))
    return calls


def _fresh(gqa, q, ck, cv, kw):
    n = gqa.query_q4(q, ck, cv, **kw)["workspace_bytes"]
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out = gqa.forward_q4(q, ck, cv, workspace=ws, **kw)
    assert gqa.device_status(ws) == gqa.GQA_OK
    return out


def test_ways_share_a_workspace(gqa):
    ck, cv = _cache(gqa, 4, 2, 2048, 128)
    calls = _ways(gqa, ck, cv)
    want = [_fresh(gqa, q, ck, cv, kw) for q, kw in calls]
    most = max(gqa.query_q4(q, ck, cv, **kw)["workspace_bytes"] for q, kw in calls)
    ws = torch.zeros(most, dtype=torch.uint8, device="cuda")
    for order in ([0, 2, 1, 3], [3, 0, 1, 2], [2, 3, 1, 0]):
        got = [(i, gqa.forward_q4(calls[i][0], ck, cv, workspace=ws, **calls[i][1]))
               for i in order]
        assert gqa.device_status(ws) == gqa.GQA_OK
        assert all(torch.equal(o, want[i]) for i, o in got)


def test_threads_on_one_stream(gqa):
    """Calls of several launches from two threads keep their scratch apart."""
    ck, cv = _cache(gqa, 4, 2, 2048, 128)
    calls = _ways(gqa, ck, cv)
    want = [_fresh(gqa, q, ck, cv, kw) for q, kw in calls]
    torch.cuda.synchronize()
    got = [[], []]

    def work(t):
        for _ in range(25):
            for i in ([2, 3, 1, 0], [3, 1, 2, 0])[t]:
                q, kw = calls[i]
                got[t].append((i, gqa.forward_q4(q, ck, cv, **kw)))

    threads = [threading.Thread(target=work, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert gqa.device_status() == gqa.GQA_OK
    assert len(got[0]) == len(got[1]) == 100
    assert all(torch.equal(o, want[i]) for t in range(2) for i, o in got[t])


@pytest.mark.parametrize("B,Hq,Hkv,Sq,S,D,dtype,kernel", [
    (4, 8, 2, 512, 2048, 128, torch.bfloat16, "q4_chunk"),
    (4, 8, 2, 512, 2048, 128, torch.float16, "q4_chunk"),
    (4, 8, 2, 512, 2048, 64, torch.bfloat16, "q4_chunk"),
    (8, 32, 8, 32, 8192, 128, torch.bfloat16, "q4_chunk"),
    (8, 32, 8, 1, 8192, 128, torch.bfloat16, "q4"),
    (8, 32, 8, 5, 4000, 64, torch.float16, "q4"),
])
def test_same_bits_call_after_call(gqa, B, Hq, Hkv, Sq, S, D, dtype, kernel):
    """A tile refilled before its last reader is done would change some calls."""
    ck, cv = _cache(gqa, B, Hkv, S, D, dtype)
    q = _q(B, Hq, Sq, D, dtype)
    kw = dict(causal=True, causal_offset="bottom_right")
    assert gqa.query_q4(q, ck, cv, **kw)["kernel_name"] == kernel
    outs = [gqa.forward_q4(q, ck, cv, **kw) for _ in range(60)]
    assert gqa.device_status() == gqa.GQA_OK
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_stream_argument(gqa):
    ck, cv = _cache(gqa, 2, 2, 900, 96, torch.float16)
    q = _q(2, 8, 3, 96, torch.float16)
    kw = dict(causal=True, causal_offset="bottom_right")
    want = gqa.forward_q4(q, ck, cv, **kw)
    wk, wv = gqa.kv_read_q4(ck, cv, 96, torch.float16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = gqa.forward_q4(q, ck, cv, stream=s.cuda_stream, **kw)
    k, v = gqa.kv_read_q4(ck, cv, 96, torch.float16, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(k, wk) and torch.equal(v, wv)
    # An append on the other stream, read on it too: the same records again.
    c2 = [torch.zeros_like(ck), torch.zeros_like(cv)]
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    gqa.kv_append_q4(c2[0], c2[1], wk, wv, lens, stream=s.cuda_stream)
    s.synchronize()
    assert lens.tolist() == [900, 900]


def test_captured_generation(gqa):
    """A captured step that advances its lengths, replayed token after token."""
    B, Hkv, D, cap, steps = 3, 2, 64, 300, 5
    new = [torch.empty(B, Hkv, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q = torch.empty(B, 8, 1, D, dtype=torch.bfloat16, device="cuda")
    rows = [_q(B, Hkv, steps, D, seed=30 + i) for i in range(2)]
    qs = _q(B, 8, steps, D, seed=40)
    ck, cv = _cache(gqa, B, Hkv, cap, D)
    start = torch.tensor([0, 64, cap - steps], dtype=torch.int32, device="cuda")
    kw = dict(causal=True, causal_offset="bottom_right")

    def step(c, lens, k, v, x):
        gqa.kv_append_q4(c[0], c[1], k, v, lens)
        return gqa.forward_q4(x, c[0], c[1], kv_lens=lens, **kw)

    c1, l1 = (ck.clone(), cv.clone()), start.clone()
    want = [step(c1, l1, rows[0][:, :, t:t + 1].contiguous(), rows[1][:, :, t:t + 1].contiguous(),
                 qs[:, :, t:t + 1].contiguous()) for t in range(steps)]
    torch.cuda.synchronize()
    c2, l2 = (ck.clone(), cv.clone()), start.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(c2, l2, new[0], new[1], q)
    for t in range(steps):
        for dst, src in ((new[0], rows[0]), (new[1], rows[1]), (q, qs)):
            dst.copy_(src[:, :, t:t + 1])
        g.replay()
        assert torch.equal(out, want[t])
    assert torch.equal(l1, l2) and torch.equal(c1[0], c2[0]) and torch.equal(c1[1], c2[1])


def test_offsets_past_32_bits(gqa):
    """The last rows of a cache of 4.5 GB (x 2) are those of a small one."""
    cap, n, D, tail = 56_000_000, 320, 128, 7
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GB")
    R = gqa.q4_record_bytes(D)
    assert (cap - n) * R > 1 << 32
    big = [torch.empty(1, 1, cap, R, dtype=torch.uint8, device="cuda") for _ in range(2)]
    small = [torch.zeros(1, 1, n, R, dtype=torch.uint8, device="cuda") for _ in range(2)]
    k, v = _q(1, 1, n, D, seed=50), _q(1, 1, n, D, seed=51)
    at, zero = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (cap - n - tail, 0))
    for c in big:
        c[:, :, -n - tail - 200:] = 0
    gqa.kv_append_q4(big[0], big[1], k, v, at)
    gqa.kv_append_q4(small[0], small[1], k, v, zero)
    assert at.item() == cap - tail
    for b, s in zip(big, small):
        assert torch.equal(b[:, :, cap - n - tail:cap - tail], s)
    got = gqa.kv_read_q4(big[0], big[1], D, torch.bfloat16, kv_lens=at, start=cap - n - tail, n=n)
    want = gqa.kv_read_q4(small[0], small[1], D, torch.bfloat16)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for Sq in (1, 5, 40):
        q = _q(1, 4, Sq, D, seed=52 + Sq)
        kw = dict(causal=True, causal_offset="bottom_right", window=n - Sq)
        a = gqa.forward_q4(q, big[0], big[1], kv_lens=at, **kw).double()
        b = gqa.forward_q4(q, small[0], small[1], **kw).double()
        # Two results of the same sums in other tiles: P's and the result's
        # roundings differ, each at most half a step of 2^-8 and 2^-11.
        assert float((a - b).norm() / b.norm()) <= 2 * (2.0 ** -8 + 2.0 ** -8)
    assert gqa.device_status() == gqa.GQA_OK


@pytest.mark.parametrize("unit", [0, 100, 383])
def test_wait_runs_out_and_is_reported(gqa, unit):
    """A launch whose producer withholds one tile's copies gives up its bounded
    wait and says so; the next call with the same workspace is right."""
    ck, cv = _cache(gqa, 4, 4, 3000, 128)
    q = _q(4, 16, 1, 128)
    plan = gqa.query_q4(q, ck, cv)
    assert plan["kernel_name"] == "q4" and plan["work_units"] == 384
    want = _fresh(gqa, q, ck, cv, {})
    ws = torch.zeros(plan["workspace_bytes"], dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    gqa.debug_decode_withhold(unit, 200_000)  # 200 us limit, this launch only
    gqa.forward_q4(q, ck, cv, workspace=ws)
    assert gqa.device_status(ws) == gqa.GQA_ERR_TIMEOUT
    out = gqa.forward_q4(q, ck, cv, workspace=ws)
    assert gqa.device_status(ws) == gqa.GQA_OK
    assert torch.equal(out, want)


def test_scalars_written_again(gqa):
    """Scalars given as 0-d tensors count by their value at each call."""
    ck, cv = _cache(gqa, 2, 2, 200, 64)
    q = _q(2, 4, 3, 64)
    scale, window, offset = torch.tensor(0.125), torch.tensor(50), torch.tensor(197)
    n, D = torch.tensor(5), torch.tensor(64)
    for s, w, o, t in ((0.125, 50, 197, 5), (0.5, 50, 197, 6), (0.5, 7, 197, 6), (0.5, 7, 100, 4)):
        scale.fill_(s), window.fill_(w), offset.fill_(o), n.fill_(t)
        got = gqa.forward_q4(q, ck, cv, causal=True, scale=scale, window=window,
                             causal_offset=offset)
        want = gqa.forward_q4(q, ck, cv, causal=True, scale=s, window=w, causal_offset=o)
        assert torch.equal(got, want)
        k, _ = gqa.kv_read_q4(ck, cv, D, torch.bfloat16, start=3, n=n)
        assert torch.equal(k, gqa.kv_read_q4(ck, cv, 64, torch.bfloat16, start=3, n=t)[0])
    lens, on = torch.tensor([10, 20], dtype=torch.int32, device="cuda"), torch.tensor(True)
    new = _q(2, 2, 1, 64, seed=9)
    gqa.kv_append_q4(ck, cv, new, new, lens, advance=on)
    on.fill_(False)
    gqa.kv_append_q4(ck, cv, new, new, lens, advance=on)
    assert lens.tolist() == [11, 21]
    assert gqa.device_status() == gqa.GQA_OK


@pytest.mark.parametrize("B,Hq,Hkv,S,D,lens", [
    (16, 32, 8, 4096, 128, None),
    (5, 40, 8, 6000, 64, None),
    (9, 32, 8, 4000, 128, [4000, 100, 2500, 3999, 1, 3000, 777, 1500, 2048]),
])
def test_same_bits_whoever_merges(gqa, B, Hq, Hkv, S, D, lens):
    """Which CTA merges a split group's partials, and in which of two ways, is
    a matter of timing, which other work on the machine changes; the sums are
    taken in one order."""
    ck, cv = _cache(gqa, B, Hkv, S, D, torch.float16)
    q = _q(B, Hq, 1, D, torch.float16)
    kw = {} if lens is None else dict(kv_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    want = gqa.forward_q4(q, ck, cv, **kw)
    side, x = torch.cuda.Stream(), torch.zeros(1 << 24, device="cuda")
    torch.cuda.synchronize()
    outs = []
    for i in range(300):
        if i % 3 == 0:
            with torch.cuda.stream(side):
                x[: 1 << (10 + i % 15)].add_(1.0)
        outs.append(gqa.forward_q4(q, ck, cv, **kw))
    assert gqa.device_status() == gqa.GQA_OK
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("B,Hkv,Sq,S,D,unit", [
    (4, 2, 512, 2048, 128, 0),      # two query tiles per group: 64 groups of 16 key tiles
    (4, 2, 512, 2048, 128, 249),
    (2, 8, 32, 8192, 64, 700),      # one query tile, split over CTAs
])
def test_chunk_wait_runs_out_and_is_reported(gqa, B, Hkv, Sq, S, D, unit):
    """The chunk kernel without the copies of one key tile gives up its bounded
    wait (1 s) and says so; the next call with the same workspace is right."""
    ck, cv = _cache(gqa, B, Hkv, S, D)
    q = _q(B, 4 * Hkv, Sq, D)
    plan = gqa.query_q4(q, ck, cv)
    assert plan["kernel_name"] == "q4_chunk" and unit < plan["work_units"]
    want = _fresh(gqa, q, ck, cv, {})
    ws = torch.zeros(plan["workspace_bytes"], dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    gqa.debug_decode_withhold(unit, 1_000_000)
    gqa.forward_q4(q, ck, cv, workspace=ws)
    assert gqa.device_status(ws) == gqa.GQA_ERR_TIMEOUT
    out = gqa.forward_q4(q, ck, cv, workspace=ws)
    assert gqa.device_status(ws) == gqa.GQA_OK
    assert torch.equal(out, want)


@pytest.mark.parametrize("layout", ["heads", "pages"])
@pytest.mark.parametrize("Sq,masked,kernel,dtype", [
    (1, False, "q4", "bf16"), (5, True, "q4", "fp16"), (200, False, "q4_chunk", "bf16"),
    (200, False, "q4_chunk", "fp16"), (600, True, "q4_prefill", "bf16"),
])
def test_attention_past_32_bits(gqa, Sq, masked, kernel, dtype, layout):
    """Records past 4 GB of a cache's base, by the strides of its heads or by
    their pages, each way, against 64 bits with the roundings of that way."""
    n, D, H, g, page = 2048, 128, 2, 8, 64
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GB")
    t, unit = (torch.bfloat16, 2.0 ** -8) if dtype == "bf16" else (torch.float16, 2.0 ** -11)
    R, far, table = gqa.q4_record_bytes(D), (1 << 32) + (1 << 20), None
    big = [torch.empty(far + n * 80 * 2 + (1 << 20), dtype=torch.uint8, device="cuda")
           for _ in range(2)]
    if layout == "heads":  # the second head starts past 4 GB
        far = far // 16 * 16
        caches = [c.as_strided((1, H, n, R), (far * H, far, R, 1)) for c in big]
    else:
        pages = big[0].numel() // (H * page * R)
        caches = [c[:pages * H * page * R].view(pages, H, page, R) for c in big]
        table = (pages - 1 - 2 * torch.arange(n // page, device="cuda")).int()[None]
        assert (pages - 1 - n // page * 2) * H * page * R > (1 << 32) - (1 << 20)
        assert (pages - 1) * H * page * R > 1 << 32
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = _q(1, H, n, D, t, seed=60), _q(1, H, n, D, t, seed=61)
    gqa.kv_append_q4(caches[0], caches[1], k, v, lens, block_table=table)
    q = _q(1, g * H, Sq, D, t, seed=62)
    kw = dict(causal=True, causal_offset="bottom_right", block_table=table)
    i = torch.arange(Sq, device="cuda")[:, None] + n - Sq
    see = torch.arange(n, device="cuda")[None, :] <= i
    if masked:
        kw["mask"] = (torch.rand(1, Sq, n, device="cuda",
                                 generator=torch.Generator(device="cuda").manual_seed(63)) < 0.7)
        see &= kw["mask"][0]
    assert gqa.query_q4(q, *caches, **kw)["kernel_name"] == kernel
    out = gqa.forward_q4(q, *caches, **kw).double()[0]
    assert gqa.device_status() == gqa.GQA_OK
    for h in range(H):
        # The records' values, in 64 bits.
        vals = []
        for c in caches:
            rec = c[0, h] if table is None else c[table[0].long()][:, h].reshape(n, R)
            par = rec[:, :16].contiguous().view(t).double().view(n, 4, 2)
            code = torch.stack([rec[:, 16:] % 16, rec[:, 16:] // 16], -1).double().view(n, 4, 32)
            vals.append((code * par[..., :1] + par[..., 1:]).flatten(-2))
        kk, vv = vals
        scale_v = par[..., 0].repeat_interleave(32, -1)
        for x in range(g):
            qh = q[0, h * g + x].double()
            p = torch.softmax((qh @ kk.T / D ** 0.5).masked_fill(~see, -torch.inf), -1)
            ref = p @ vv
            bound = 1.01 * unit * ref.abs() + 2.0 ** -14 * (p @ vv.abs()) + 2.0 ** -24
            if kernel == "q4":  # the weights, once to fp16, times codes of at most 15 scales
                bound += 2.0 ** -11 * 15 * (p @ scale_v)
            else:               # keys, values and weights, once to the type
                move = 2.1 * unit / D ** 0.5 * (qh.abs() @ kk.abs().T).amax(-1, keepdim=True)
                bound += (p @ vv.abs()) * (2.02 * unit + move)
            err = (out[h * g + x] - ref).abs()
            assert torch.all(err <= bound), float((err / bound).max())
            # Most roundings fall on both sides of half of their bound: in norm,
            # the result's alone stays within it, with three more within twice.
            assert float(err.norm() / ref.norm()) <= unit * (1 if kernel == "q4" else 2)
