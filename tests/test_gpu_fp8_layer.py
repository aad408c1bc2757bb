"""The 8-bit layer's operators where a launch is larger or calls are closer than the
formula's tests make them: workgroups that take several rows, results in place of
their inputs, byte offsets over 2^32, calls on two streams at once, one buffer as
two operands, and graphs that are replayed beside eager calls.

A row's norm and a product's element are sums of their own in a fixed order, so
results are compared bit by bit with those of calls on small parts.
"""
import pytest
import torch

import sharded_state_amd as ss

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def _rand(shape, dtype=torch.float32, seed=0, sigma=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * sigma).to(dtype)


def _equal(a, b):
    """Bit by bit, NaN too."""
    ints = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(a.contiguous().view(ints), b.contiguous().view(ints))


# ------------------------------------------------------- several rows a workgroup
@pytest.mark.parametrize("m,d", [(7000, 40), (6200, 77), (1700, 5000), (1500, 5003), (900, 9001), (800, 12_000), (500, 20_001)])
@pytest.mark.parametrize("xt,ht", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32)])
def test_norm_of_many_rows_is_that_of_its_parts(m, d, xt, ht):
    print("case", m, d, xt, ht, flush=True)
    x, res, w = _rand((m, d), xt, 1), _rand((m, d), ht, 2), 1 + _rand((d,), seed=3, sigma=0.1)
    o = ss.fsdp_rms_norm_fp8(x, w, res, y=True)
    for i in list(range(0, m, max(m // 5, 1))) + [m - 3]:
        p = ss.fsdp_rms_norm_fp8(x[i:i + 3], w, res[i:i + 3], y=True)
        n = p.h.shape[0]
        for name, a, b in (("codes", o.q.codes, p.q.codes), ("scales", o.q.scales, p.q.scales), ("h", o.h, p.h),
                           ("rstd", o.rstd, p.rstd), ("y", o.y, p.y)):
            assert _equal(a[i:i + n], b), (name, i)
    own = res.clone()
    again = ss.fsdp_rms_norm_fp8(x, w, own, h=own)
    assert again.h is own and _equal(own, o.h) and _equal(again.q.codes, o.q.codes) and _equal(again.rstd, o.rstd)


@pytest.mark.parametrize("m,d", [(5000, 40), (3000, 77), (2500, 2001), (900, 5003), (700, 9001), (600, 12_000), (300, 20_001)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gradients_in_place_of_many_rows(m, d, dtype):
    print("case", m, d, dtype, flush=True)
    h, dy, dh = (_rand((m, d), dtype, i) for i in range(3))
    w = 1 + _rand((d,), seed=4, sigma=0.1)
    rstd = ss.fsdp_rms_norm_fp8(h, w).rstd
    dx, dw = ss.fsdp_rms_norm_grads(dy, h, w, rstd, dh=dh)
    for i in (0, m // 2, m - 2):
        part, _ = ss.fsdp_rms_norm_grads(dy[i:i + 2], h[i:i + 2], w, rstd[i:i + 2], dh=dh[i:i + 2], dw=False)
        assert _equal(dx[i:i + 2], part), i
    for own in ("dh", "dy"):
        t = dict(dh=dh.clone(), dy=dy.clone())
        got, gw = ss.fsdp_rms_norm_grads(t["dy"], h, w, rstd, dh=t["dh"], dx=t[own])
        assert got is t[own] and _equal(got, dx) and _equal(gw, dw), own
    # one buffer as two operands
    same, sw = ss.fsdp_rms_norm_grads(h, h, w, rstd, dh=h)
    twin, tw = ss.fsdp_rms_norm_grads(h.clone(), h, w, rstd, dh=h.clone())
    assert _equal(same, twin) and _equal(sw, tw)


# ------------------------------------------------------------ offsets over 2^32
def test_rows_behind_4_gib():
    m, d = 1_100_000, 2056                                       # 4.5 GB in 16 bits, ragged blocks
    x = torch.empty((m, d), dtype=torch.bfloat16, device="cuda")
    for i in range(0, m, 100_000):
        x[i:i + 100_000] = _rand((min(100_000, m - i), d), torch.bfloat16, i)
    w = torch.ones(d, device="cuda")
    tail = slice(m - 257, m)
    q = ss.fsdp_fp8_quantize(x)
    p = ss.fsdp_fp8_quantize(x[tail])
    assert q.codes.numel() > 2 ** 31 and _equal(q.codes[tail], p.codes) and _equal(q.scales[tail], p.scales)
    o, n = ss.fsdp_rms_norm_fp8(x, w), ss.fsdp_rms_norm_fp8(x[tail], w)
    assert _equal(o.q.codes[tail], n.q.codes) and _equal(o.rstd[tail], n.rstd)
    dx, _ = ss.fsdp_rms_norm_grads(x, x, w, o.rstd, dw=False)
    part, _ = ss.fsdp_rms_norm_grads(x[tail], x[tail], w, n.rstd, dw=False)
    assert _equal(dx[tail], part)
    del dx, o
    # more rows than a product's launch counts; whole numbers, so that the order of a sum does not show
    whole = ss.fsdp_fp8_quantize(x.clamp_(-3, 3).round_())
    b = ss.fsdp_fp8_quantize(_rand((40, d), seed=7).clamp(-3, 3).round())
    got = ss.fsdp_fp8_matmul(whole, b, dtype=torch.float32)
    want = x[tail].double().cpu() @ _rand((40, d), seed=7).clamp(-3, 3).round().double().cpu().t()
    assert torch.equal(got[tail].double().cpu(), want)
    back = ss.fsdp_fp8_matmul(b, whole, dtype=torch.float32)
    assert torch.equal(back[:, tail].double().cpu(), want.t())


def test_columns_and_gather_behind_4_gib():
    rows, cols = 2_200_000, 1024                                 # 4.5 GB
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 200_000):
        x[i:i + 200_000] = _rand((200_000, cols), torch.bfloat16, i)
    last = rows - 64                                             # a multiple of 128 behind which 64 rows are left
    assert last % 128 == 0
    for tile in (False, True):
        t = ss.fsdp_fp8_quantize(x, form="columns", tile=tile)
        p = ss.fsdp_fp8_quantize(x[last:], form="columns", tile=tile)
        assert _equal(t.codes[:, -128:], p.codes) and _equal(t.scales[:, -1:], p.scales)
        del t
    flat = ss.fsdp_fp8_quantize(x.view(-1))
    full = ss.fsdp_fp8_gather([flat, flat], dtype=torch.bfloat16)
    end = ss.Fp8(flat.codes[:, -1024:], flat.scales[:, -8:], 1024)
    want = ss.fsdp_fp8_gather([end], dtype=torch.bfloat16)
    assert full.numel() == 2 * rows * cols and _equal(full[-1024:], want)
    assert _equal(full[rows * cols - 1024:rows * cols], want)


# --------------------------------------------------- calls at once, and one buffer twice
def test_a_buffer_as_both_operands():
    a = ss.fsdp_fp8_quantize(_rand((300, 1000), torch.bfloat16, 1))
    twin = ss.Fp8(a.codes.clone(), a.scales.clone(), a.cols)
    assert _equal(ss.fsdp_fp8_matmul(a, a), ss.fsdp_fp8_matmul(a, twin))
    x, w = _rand((50, 700), torch.bfloat16, 2), torch.ones(700, device="cuda")
    o, p = ss.fsdp_rms_norm_fp8(x, w, x), ss.fsdp_rms_norm_fp8(x, w, x.clone())
    assert _equal(o.h, x + x) and _equal(o.q.codes, p.q.codes)
    s = ss.fsdp_fp8_quantize(_rand((1, 500), seed=3))
    assert _equal(*ss.fsdp_fp8_gather([s, s], dtype=torch.float32).view(2, 500))


@pytest.mark.parametrize("m,n,k", [(24, 1600, 6400), (200, 300, 1500), (700, 1600, 6400), (5, 2000, 9000)])
def test_two_streams_at_once(m, n, k):
    """Sums split over workgroups keep their parts in a workspace: each call has its own."""
    sets = []
    for i in range(2):
        w, wt = ss.fsdp_fp8_quantize(_rand((n, k), torch.bfloat16, 10 + i), form="both", tile=True)
        x, dy = _rand((m, k), torch.bfloat16, 20 + i), _rand((m, n), torch.bfloat16, 30 + i)
        g = 1 + _rand((k,), seed=40 + i, sigma=0.1)
        sets.append((w, wt, x, dy, g))

    def work(s, stream=None):
        w, wt, x, dy, g = s
        o = ss.fsdp_rms_norm_fp8(x, g, stream=stream)
        y, z = ss.fsdp_fp8_linear(o.q, w, stream=stream), ss.fsdp_fp8_linear(x, w, stream=stream)
        dn, dw = ss.fsdp_fp8_linear_grads(dy, x, wt, stream=stream)
        return (y, z, dn, dw, *ss.fsdp_rms_norm_grads(dn, x, g, o.rstd, stream=stream))

    want = [work(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [None, None]
        for i in (0, 1):
            got[i] = work(sets[i], streams[i])
        torch.cuda.synchronize()
        for i in (0, 1):
            assert all(_equal(a, b) for a, b in zip(got[i], want[i])), i
    graphs = []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = work(s)
        graphs.append((graph, out))
    for replay in range(3):
        for stream, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(_equal(a, b) for i in (0, 1) for a, b in zip(graphs[i][1], want[i])), replay


def test_norm_of_the_widest_features_and_of_one():
    for d in (1, 32_767, 32_768):
        x, w = _rand((3, d), torch.bfloat16, d), torch.ones(d, device="cuda")
        o = ss.fsdp_rms_norm_fp8(x, w, y=True)
        r = 1 / (x.double().square().mean(dim=1) + 1e-6).sqrt()
        assert ((o.rstd.double() - r).abs() <= r * 2.0 ** -24 * (1 + 2.0 ** -20)).all()
        dx, dw = ss.fsdp_rms_norm_grads(x, x, w, o.rstd)
        assert torch.isfinite(dx.float()).all() and torch.isfinite(dw).all()
    with pytest.raises(ss.FsdpError):
        ss.fsdp_rms_norm_fp8(_rand((2, 32_769)), torch.ones(32_769, device="cuda"))
