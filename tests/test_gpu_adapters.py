"""Per-row adapters beside the quantized product, on the GPU, against float64.

Bound of an output element, with e = 2^-24: the product adds K + 3 R terms (T
enters in up to three bf16 parts) in float32, each sum rounded: at most
(K + 3 R + 24) e times the sum of the terms' magnitudes (24: the partial sums
of K splits).  T itself adds K terms and is scaled: (K + 10) e of its own
magnitudes, times |U|; its bf16 parts leave 2^-16 (bf16 Y) or 2^-24 (float32
Y) of T.  A bf16 Y is rounded once more, by at most 2^-8 of its value."""
import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def _case(msg):
    print(f"\n[case] {msg}", flush=True)


def _pool(api, gen, a, n, k, r):
    down = (torch.randn(a, r, k, generator=gen, device="cuda") / k ** 0.5).bfloat16()
    up = (torch.randn(a, n, r, generator=gen, device="cuda") * 0.2).bfloat16()
    return api.AdapterPool(down, up, torch.rand(a, generator=gen, device="cuda") * 2 - 0.5)


def _setup(api, seed, m, n, k, bits, a, r):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(n, k, generator=gen, device="cuda") * 0.02
    qw = api.quantize_pack(w, bits)
    x = torch.randn(m, k, generator=gen, device="cuda").bfloat16()
    return x, qw, _pool(api, gen, a, n, k, r)


def _reference(api, x, qw, pool, rows):
    """(float64 Y, magnitudes of the product, of T |U|, of |T| |U| from T's own terms)."""
    w = api.dequantize(qw).double()                 # bit-exact, checked against the oracle elsewhere
    xd = x.double()
    y, mag = xd @ w.t(), xd.abs() @ w.abs().t()
    tu, own = torch.zeros_like(y), torch.zeros_like(y)
    for a in range(pool.down.shape[0]):
        ids = (rows == a).nonzero().view(-1)
        if ids.numel() == 0:
            continue
        s, d, u = float(pool.scales[a]), pool.down[a].double(), pool.up[a].double()
        t = s * (xd[ids] @ d.t())
        y[ids] += t @ u.t()
        tu[ids] += t.abs() @ u.abs().t()
        own[ids] += abs(s) * (xd[ids].abs() @ d.abs().t()) @ u.abs().t()
    return y, mag, tu, own


def _check(y, ref, k, r, what):
    want, mag, tu, own = ref
    tol = (k + 3 * r + 24) * E * (mag + tu) + (k + 10) * E * own + (2.0 ** -16 if y.dtype == BF else E) * tu
    if y.dtype == BF:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    err = (y.double() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), float((err / tol).max()))
    # far inside the worst case: rounding errors add up like random signs
    rel = float((y.double() - want).norm() / want.norm())
    assert rel <= (2.0 ** -8 if y.dtype == BF else 64 * E * (1 + k ** 0.5 / 8)), (what, rel)


def _rows(kind, m, a, seed):
    rng = np.random.default_rng(seed)
    if kind == "one":
        r = np.full(m, a - 1)
    elif kind == "each":
        r = np.arange(m) % a
        rng.shuffle(r)
    elif kind == "runs":
        cuts = np.sort(rng.integers(0, m + 1, 2 * a))
        r = rng.integers(-1, a, 2 * a + 1)[np.searchsorted(cuts, np.arange(m), side="right")]
    elif kind == "none":
        r = np.full(m, -1)
    elif kind == "wild":                              # numbers outside the pool: no adapter
        r = rng.choice([-2 ** 31, -7, -1, 0, a - 1, a, a + 1, 2 ** 31 - 1], m)
    else:
        raise ValueError(kind)
    return torch.from_numpy(r.astype(np.int32)).cuda()


SHAPES = [(1, 48, 256, 4), (1, 5120, 1280, 3), (3, 640, 1152, 5), (16, 16, 8192, 6), (16, 12816, 640, 5), (13, 2064, 8320, 4),
          (17, 272, 896, 7), (32, 4112, 1024, 3), (37, 528, 512, 6), (64, 1040, 384, 4), (65, 272, 384, 4),
          (300, 512, 2560, 5), (257, 784, 128, 7), (1001, 1296, 640, 4), (600, 5136, 256, 3), (4100, 3088, 256, 6)]


@pytest.mark.parametrize("kind", ["one", "each", "runs", "none", "wild"])
@pytest.mark.parametrize("m,n,k,bits", SHAPES)
def test_shapes_and_mixes(gpu_lib, m, n, k, bits, kind):
    for a, r, dt in [(5, 16, BF), (1, 8, F32), (40, 40, F32), (3, 128, BF)]:
        _case(f"adapter_gemm {m}x{n}x{k} b{bits} {kind} adapters={a} rank={r} {dt}")
        x, qw, pool = _setup(gpu_lib, m + n + r, m, n, k, bits, a, r)
        rows = _rows(kind, m, a, m + a)
        y = gpu_lib.adapter_gemm(x, qw, pool, rows, out_dtype=dt)
        _check(y, _reference(gpu_lib, x, qw, pool, rows), k, r, (kind, a, r))


@pytest.mark.parametrize("m,n,k", [(64, 272, 384), (65, 272, 384), (256, 1040, 640), (300, 528, 1536), (511, 5136, 256),
                                   (4100, 3088, 256)])
def test_every_row_its_own_adapter(gpu_lib, m, n, k):
    """As many adapters as rows, in any order and with a few rows of none: 256
    of them in a tile, 16 in a row block of the pre-pass."""
    for r, dt in [(16, BF), (8, F32), (40, F32)]:
        _case(f"every row its own adapter {m}x{n}x{k} rank={r} {dt}")
        a = min(m, 700)
        x, qw, pool = _setup(gpu_lib, m + r, m, n, k, 4, a, r)
        rows = _rows("each", m, a, m)
        rows[::37] = -1
        y = gpu_lib.adapter_gemm(x, qw, pool, rows, out_dtype=dt)
        _check(y, _reference(gpu_lib, x, qw, pool, rows), k, r, (m, r))
        assert torch.equal(y, gpu_lib.adapter_gemm(x, qw, pool, rows, out_dtype=dt))


@pytest.mark.parametrize("r", [8, 16, 24, 32, 48, 56, 64, 72, 80, 96, 104, 112, 120, 128])
@pytest.mark.parametrize("m", [5, 70, 2100])
def test_ranks(gpu_lib, m, r):
    """Every rank tile of the pre-pass, and its row blocks per workgroup."""
    _case(f"adapter_gemm ranks m={m} r={r}")
    x, qw, pool = _setup(gpu_lib, 3 * m + r, m, 272, 384, 4, 4, r)
    rows = _rows("runs", m, 4, r)
    _check(gpu_lib.adapter_gemm(x, qw, pool, rows, out_dtype=F32), _reference(gpu_lib, x, qw, pool, rows), 384, r, r)


@pytest.mark.parametrize("m", [20000, 33000])
def test_many_rows(gpu_lib, m):
    """Two and four row blocks per workgroup of the pre-pass, mixed inside them."""
    for kind, r in [("each", 16), ("runs", 32), ("runs", 64)]:
        _case(f"adapter_gemm many rows m={m} {kind} r={r}")
        x, qw, pool = _setup(gpu_lib, m + r, m, 272, 256, 4, 7, r)
        rows = _rows(kind, m, 7, r)
        _check(gpu_lib.adapter_gemm(x, qw, pool, rows), _reference(gpu_lib, x, qw, pool, rows), 256, r, (kind, r))


@pytest.mark.parametrize("m,n", [(3, 272), (16, 12816), (50, 272), (300, 512), (700, 784)])
def test_branch_bits(gpu_lib, m, n):
    """The branch alone: a zero weight, one nonzero input per row (T is then
    one product, exact in float32) and rank 8, so that the bound is 27 e of
    |T| |U| and a lost bf16 part of T would show."""
    _case(f"branch alone m={m} n={n}")
    k, a, r = 256, 3, 8
    gen = torch.Generator(device="cuda").manual_seed(m)
    qw = gpu_lib.quantize_pack(torch.zeros(n, k, device="cuda"), 4)
    x = torch.zeros(m, k, device="cuda")
    x[torch.arange(m), torch.arange(m) % k] = torch.randn(m, generator=gen, device="cuda")
    x = x.bfloat16()
    pool = _pool(gpu_lib, gen, a, n, k, r)
    pool.scales.fill_(1.0)
    rows = _rows("each", m, a, m)
    y = gpu_lib.adapter_gemm(x, qw, pool, rows, out_dtype=F32).double()
    t = torch.stack([x[i].double() @ pool.down[int(rows[i])].double().t() for i in range(m)])
    u = pool.up.double()[rows.long()]
    want = (u @ t[:, :, None])[:, :, 0]
    mag = (u.abs() @ t.abs()[:, :, None])[:, :, 0]
    assert bool(((y - want).abs() <= 27 * E * mag).all()), float(((y - want).abs() / mag.clamp_min(1e-30)).max() / E)


def test_rows_without_an_adapter_equal_the_product(gpu_lib):
    for m, n, k, bits in SHAPES:
        _case(f"no adapter {m}x{n}x{k} b{bits}")
        x, qw, pool = _setup(gpu_lib, m, m, n, k, bits, 2, 16)
        want = gpu_lib.dequant_gemm(x, qw)
        assert torch.equal(gpu_lib.adapter_gemm(x, qw, pool, _rows("none", m, 2, 0)), want)
        some = _rows("runs", m, 2, 5)
        got = gpu_lib.adapter_gemm(x, qw, pool, some)
        assert torch.equal(got[some < 0], want[some < 0])


@pytest.mark.parametrize("m,n", [(16, 272), (16, 12816), (60, 272), (300, 512), (300, 3088), (700, 784)])
def test_a_broken_adapter_stays_with_its_rows(gpu_lib, m, n):
    """Infinities and NaNs in one adapter's factors, and in one row of X,
    reach the rows that name it (that row) and no other, which keep their bits."""
    _case(f"broken adapter m={m} n={n}")
    x, qw, pool = _setup(gpu_lib, m + n, m, n, 384, 5, 4, 24)
    rows = _rows("each", m, 4, 1)
    want = gpu_lib.adapter_gemm(x, qw, pool, rows)
    for where, val in [("up", float("inf")), ("up", float("nan")), ("down", float("nan")), ("down", float("inf"))]:
        keep = getattr(pool, where)[2].clone()
        getattr(pool, where)[2] = val
        got = gpu_lib.adapter_gemm(x, qw, pool, rows)
        getattr(pool, where)[2] = keep
        assert torch.equal(got[rows != 2], want[rows != 2]), (where, val)
        assert not bool(torch.isfinite(got[rows == 2]).any()), (where, val)
    pool.scales[1] = float("nan")
    got = gpu_lib.adapter_gemm(x, qw, pool, rows)
    pool.scales[1] = 1.0
    assert torch.equal(got[rows != 1], want[rows != 1]) and bool(torch.isnan(got[rows == 1]).all())
    base = gpu_lib.adapter_gemm(x, qw, pool, rows)
    x[1, 7] = float("nan")
    got = gpu_lib.adapter_gemm(x, qw, pool, rows)
    others = torch.arange(m, device="cuda") != 1
    assert torch.equal(got[others], base[others]) and bool(torch.isnan(got[1]).all())


@pytest.mark.parametrize("m,n,k,a", [(300, 512, 2560, 1), (300, 512, 2560, 3), (300, 784, 256, 1), (700, 784, 384, 4)])
def test_a_broken_high_rank_stays_with_its_rows(gpu_lib, m, n, k, a):
    """One infinite entry of U past the first 64 ranks, in a tile of one
    adapter (with rows of none) and in tiles that mix them, whole and split."""
    _case(f"broken high rank {m}x{n}x{k} adapters={a}")
    x, qw, pool = _setup(gpu_lib, m + n + a, m, n, k, 4, a, 128)
    rows = _rows("each", m, a, 1)
    rows[::5] = -1
    for dt in (BF, F32):
        want = gpu_lib.adapter_gemm(x, qw, pool, rows, out_dtype=dt)
        keep = pool.up[0, 17, 100].clone()
        pool.up[0, 17, 100] = float("inf")
        got = gpu_lib.adapter_gemm(x, qw, pool, rows, out_dtype=dt)
        pool.up[0, 17, 100] = keep
        assert torch.equal(got[rows != 0], want[rows != 0])
        hit = got[rows == 0]
        assert not bool(torch.isfinite(hit[:, 17]).any())
        hit[:, 17] = want[rows == 0][:, 17]
        assert torch.equal(hit, want[rows == 0])


def test_repeats_and_workspace(gpu_lib):
    """The same bits on every call, with a workspace of exactly the required
    bytes between guards, NaN inside; the output fully written."""
    for m, n, k, bits in SHAPES:
        _case(f"workspace {m}x{n}x{k} b{bits}")
        x, qw, pool = _setup(gpu_lib, m, m, n, k, bits, 3, 32)
        rows = _rows("runs", m, 3, 2)
        first = gpu_lib.adapter_gemm(x, qw, pool, rows, out_dtype=F32)
        assert torch.equal(first, gpu_lib.adapter_gemm(x, qw, pool, rows, out_dtype=F32))
        for split in (False, True):
            need = gpu_lib.adapter_workspace_bytes(m, n, k, 32, split)
            buf = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
            outs = []
            for _ in range(2):
                out = torch.full((m + 2, n), float("nan"), device="cuda")
                gpu_lib.adapter_gemm(x, qw, pool, rows, out=out[1:m + 1], workspace=buf[256:256 + need])
                outs.append(out)
            torch.cuda.synchronize()
            assert bool((buf[:256] == 0xFF).all()) and bool((buf[256 + need:] == 0xFF).all())
            assert bool(torch.isnan(outs[0][0]).all()) and bool(torch.isnan(outs[0][m + 1]).all())
            assert torch.equal(outs[0][1:m + 1], outs[1][1:m + 1])
            if split:
                assert torch.equal(outs[0][1:m + 1], first)
            else:
                _check(outs[0][1:m + 1], _reference(gpu_lib, x, qw, pool, rows), k, 32, "no split")
            if need:
                with pytest.raises(gpu_lib.DDGError):
                    gpu_lib.adapter_gemm(x, qw, pool, rows, workspace=buf[:gpu_lib.adapter_workspace_bytes(
                        m, n, k, 32, False) - 256])


def test_padded_inputs_and_stack(gpu_lib):
    """An input dimension that the record pads, adapters of several ranks."""
    _case("stacked adapters, padded inputs")
    gen = torch.Generator(device="cuda").manual_seed(4)
    n, orig, m = 272, 300, 40
    qw = gpu_lib.quantize_pack(torch.randn(n, orig, generator=gen, device="cuda") * 0.02, 5)
    x = torch.randn(m, orig, generator=gen, device="cuda").bfloat16()
    parts = [((torch.randn(r, orig, generator=gen, device="cuda") / 17).bfloat16(),
              (torch.randn(n, r, generator=gen, device="cuda") * 0.2).bfloat16(), 0.5 + r / 16) for r in (4, 16, 1, 20)]
    pool = gpu_lib.AdapterPool.stack(parts, qw)
    assert pool.down.shape == (4, 24, 384) and pool.up.shape == (4, n, 24)
    rows = _rows("each", m, 4, 3)
    y = gpu_lib.adapter_gemm(x, qw, pool, rows, out_dtype=F32)
    xp = torch.nn.functional.pad(x, (0, 84))
    _check(y, _reference(gpu_lib, xp, qw, pool, rows), 384, 24, "stack")
    want = x.double() @ gpu_lib.dequantize(qw).double()[:, :orig].t()
    for i in range(m):
        d, u, s = parts[int(rows[i])]
        want[i] += s * (x[i].double() @ d.double().t()) @ u.double().t()
    assert float((y.double() - want).norm() / want.norm()) < 1e-5


def test_a_pool_keeps_its_tensors(gpu_lib):
    """Tensors that were checked together cannot be exchanged one by one; their
    values may change between calls."""
    _case("pool tensors")
    x, qw, pool = _setup(gpu_lib, 2, 8, 64, 256, 4, 2, 16)
    for name in ("down", "up", "scales"):
        with pytest.raises(AttributeError):
            setattr(pool, name, getattr(pool, name)[:1])
    rows = _rows("each", 8, 2, 0)
    first = gpu_lib.adapter_gemm(x, qw, pool, rows, out_dtype=F32)
    pool.scales.mul_(2.0)
    again = gpu_lib.adapter_gemm(x, qw, pool, rows, out_dtype=F32)
    assert not torch.equal(first, again)
    _check(again, _reference(gpu_lib, x, qw, pool, rows), 256, 16, "changed scales")


def test_refused_calls(gpu_lib):
    _case("refusals")
    x, qw, pool = _setup(gpu_lib, 1, 8, 64, 256, 4, 2, 16)
    rows = torch.zeros(8, dtype=torch.int32, device="cuda")
    P = gpu_lib.AdapterPool
    for args in [(pool.down[0], pool.up, pool.scales), (pool.down.float(), pool.up, pool.scales),
                 (pool.down, pool.up, pool.scales.double()), (pool.down, pool.up, pool.scales[:1]),
                 (pool.down, pool.up[:1], pool.scales), (pool.down, pool.up[..., :8].contiguous(), pool.scales),
                 (pool.down.transpose(1, 2), pool.up, pool.scales), (pool.down.cpu(), pool.up, pool.scales)]:
        with pytest.raises(ValueError):
            P(*args)
    odd = P(pool.down[:, :12].contiguous(), pool.up[..., :12].contiguous(), pool.scales)
    with pytest.raises(gpu_lib.DDGError):
        gpu_lib.adapter_gemm(x, qw, odd, rows)
    for kw in [dict(rows=rows.long()), dict(rows=rows[:7]), dict(rows=rows.cpu()), dict(x=x.float()),
               dict(x=x[:, :128].contiguous()), dict(out=torch.empty(8, 48, device="cuda")),
               dict(out=torch.empty(8, 64, device="cuda").half()),
               dict(pool=P(pool.down[..., :128].contiguous(), pool.up, pool.scales)),
               dict(pool=P(pool.down, pool.up[:, :48].contiguous(), pool.scales))]:
        with pytest.raises(ValueError):
            gpu_lib.adapter_gemm(**{**dict(x=x, qw=qw, pool=pool, rows=rows), **kw})
    assert gpu_lib.adapter_gemm(x[:0], qw, pool, rows[:0]).shape == (0, 64)


def test_pool_past_4_gib(gpu_lib):
    """Factors whose byte offsets pass 32 bits: the last adapters of pools of 4.5 GB each."""
    _case("pool past 4 GiB")
    n, k, r = 512, 384, 128
    a = (1 << 31) // (k * r) + 3000
    gen = torch.Generator(device="cuda").manual_seed(8)
    qw = gpu_lib.quantize_pack(torch.randn(n, k, generator=gen, device="cuda") * 0.02, 4)
    small = _pool(gpu_lib, gen, 2, n, k, r)
    down = torch.empty(a, r, k, dtype=BF, device="cuda")
    up = torch.empty(a, n, r, dtype=BF, device="cuda")
    assert down.numel() * 2 > 2 ** 32 and up.numel() * 2 > 2 ** 32
    scales = torch.ones(a, device="cuda")
    at = [a - 1, a - 2500]
    for i, p in enumerate(at):
        down[p], up[p], scales[p] = small.down[i], small.up[i], small.scales[i]
    pool = gpu_lib.AdapterPool(down, up, scales)
    for m in (2, 40, 300):
        x = torch.randn(m, k, generator=gen, device="cuda").bfloat16()
        rows = _rows("each", m, 2, m)
        want = gpu_lib.adapter_gemm(x, qw, small, rows)
        far = torch.tensor(at, dtype=torch.int32, device="cuda")[rows.long()]
        assert torch.equal(gpu_lib.adapter_gemm(x, qw, pool, far), want)
    del down, up, pool
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m,n,k,bits", [(16, 1040, 8192, 4), (16, 12816, 640, 5), (50, 272, 384, 4), (700, 2320, 1536, 5)])
def test_graph_replays(gpu_lib, m, n, k, bits):
    """Two graphs captured on one stream and replayed on two streams at once
    with new inputs and rows, eager calls in between: each replay's bits are
    those of an eager call given a workspace without room for split K."""
    _case(f"graph {m}x{n}x{k}")
    x, qw, pool = _setup(gpu_lib, m, m, n, k, bits, 4, 16)
    ws = torch.empty(gpu_lib.adapter_workspace_bytes(m, n, k, 16, False), dtype=torch.uint8, device="cuda")
    xs, rs = [x.clone(), x.clone()], [_rows("each", m, 4, 0), _rows("runs", m, 4, 0)]
    gpu_lib.adapter_gemm(x, qw, pool, rs[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gpu_lib.adapter_gemm(xs[i], qw, pool, rs[i]))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        wants = []
        for i in range(2):
            xs[i].copy_(torch.randn(m, k, device="cuda").bfloat16())
            rs[i].copy_(_rows(["each", "runs", "one", "none"][rep], m, 4, rep + i))
            wants.append(gpu_lib.adapter_gemm(xs[i], qw, pool, rs[i], workspace=ws))
        gpu_lib.adapter_gemm(x, qw, pool, rs[0])                   # eager, split K
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, wants):
            assert torch.equal(o, w), rep


def test_two_streams_at_once(gpu_lib):
    _case("two streams")
    setups = [(_setup(gpu_lib, i, 16 + 300 * i, 1040, 8192, 4, 4, 16), _rows("each", 16 + 300 * i, 4, i))
              for i in range(2)]
    wants = [gpu_lib.adapter_gemm(*s, r) for s, r in setups]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(5):
        for i, (s, r) in enumerate(setups):
            with torch.cuda.stream(streams[i]):
                outs[i].append(gpu_lib.adapter_gemm(*s, r))
    torch.cuda.synchronize()
    for o, w in zip(outs, wants):
        assert all(torch.equal(t, w) for t in o)


def test_projection_norms_and_rotation_together(gpu_lib):
    """A block's way from its tokens to attention: the fused q, k, v
    projection with each request's adapter, then the norms and the rotation
    in place inside its output; and the output projection with adapters."""
    _case("qkv with adapters, norms and rotation in place, output projection")
    m, h, d, bits, r, a = 85, 8, 64, 5, 16, 3
    k = 3 * h * d
    x, qw, pool = _setup(gpu_lib, 77, m, k, 640, bits, a, r)
    rows = _rows("runs", m, a, 9)
    pos = torch.from_numpy(np.stack([np.arange(m) // 20, np.arange(m) // 5 % 4, np.arange(m) % 5], -1).astype(np.int32)).cuda()
    sections = (12, 10, 10)
    f = torch.cat([gpu_lib.rope_frequencies(2 * s)[0] for s in sections])
    wq, wk = (1 + 0.1 * torch.randn(d, device="cuda") for _ in range(2))
    qkv = gpu_lib.adapter_gemm(x, qw, pool, rows)
    got = qkv.clone().view(m, 3, h, d)
    gpu_lib.qk_norm_rope(got[:, 0], got[:, 1], pos, f, q_weight=wq, k_weight=wk, sections=sections,
                         out_q=got[:, 0], out_k=got[:, 1])
    src = qkv.double().view(m, 3, h, d)
    assert torch.equal(got[:, 2], qkv.view(m, 3, h, d)[:, 2])
    axis = torch.tensor([0] * 12 + [1] * 10 + [2] * 10, device="cuda")
    ang = pos.double()[:, axis] * f
    z = torch.polar(torch.ones_like(ang), ang)[:, None]
    for i, w in enumerate((wq, wk)):
        nrm = src[:, i] / torch.sqrt(src[:, i].square().mean(-1, keepdim=True) + 1e-6) * w.double()
        turned = torch.view_as_real(torch.view_as_complex(nrm.reshape(m, h, d // 2, 2)) * z).reshape(m, h, d)
        mag = nrm.abs().view(m, h, d // 2, 2).sum(-1, keepdim=True).expand(m, h, d // 2, 2).reshape(m, h, d)
        tol = 60 * E * mag
        assert bool(((got[:, i].double() - turned).abs() <= tol + 2.0 ** -8 * (turned.abs() + tol)).all())
    _check(qkv, _reference(gpu_lib, x, qw, pool, rows), 640, r, "qkv")
    o, qo, po = _setup(gpu_lib, 78, m, 640, h * d, bits, a, r)
    attended = got[:, 0].reshape(m, h * d).contiguous()
    _check(gpu_lib.adapter_gemm(attended, qo, po, rows, out_dtype=F32), _reference(gpu_lib, attended, qo, po, rows),
           h * d, r, "out")
