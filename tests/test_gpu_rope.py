"""Rotary positions and the norms of queries and keys on the GPU, against the
formulas in float64.

Bounds, with e = 2^-24 and a the magnitude |n_u| + |n_v| of the pair's normed
values times the amplitude: a cosine or sine carries at most 5 e (its
argument's rounding, at most pi/4 e; the Taylor sum's last steps 2 e and
truncation 0.04 e; the amplitude's own rounding and its product 2 e); the sum
of squares adds positive float32 terms, at most N - 1 additions deep, so its
relative error is below N e and the reciprocal root's below N e / 2 + 3 e;
the two products of the norm and the rotation's two steps add 4 e.  The
deepest sum here is 64 (head) or 96 (token) additions: 12 e + N e / 2 <= 60 e
in all, times a.  float64 angles: |angle| 2^-51 besides.  A bf16 output is
rounded once more, by at most 2^-8 of its value."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def _case(msg):
    print(f"\n[case] {msg}", flush=True)


def _axis_angles(positions, freqs, sections):
    axis = np.repeat(np.arange(len(sections)), sections)
    return positions.astype(np.float64)[..., axis] * freqs          # (..., tokens, pairs)


def _reference(x, positions, freqs, sections, layout, amplitude=1.0, inverse=False, weight=None, norm=None, eps=1e-6):
    """(float64 result, magnitude for the bound) of x (batch, tokens, heads, dim) float64."""
    n = x
    if norm is not None:
        axes = (-1,) if norm == "head" else (-1, -2)
        n = x / np.sqrt(np.mean(x * x, axis=axes, keepdims=True) + eps)
        if weight is not None:
            n = n * (weight if norm == "head" else weight.reshape(x.shape[-2], x.shape[-1]))
    out, mag = n.copy(), np.abs(n)
    pairs = len(freqs)
    if pairs:
        ang = _axis_angles(positions, freqs, sections)
        ang = ang[None] if ang.ndim == 2 else ang
        c, s = np.cos(ang)[:, :, None] * amplitude, np.sin(ang)[:, :, None] * amplitude * (-1 if inverse else 1)
        u, v = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if layout == "interleaved" else \
            (slice(0, pairs), slice(pairs, 2 * pairs))
        a, b = n[..., u], n[..., v]
        out[..., u], out[..., v] = a * c - b * s, b * c + a * s
        m = (np.abs(a) + np.abs(b)) * abs(amplitude)
        extra = np.abs(ang)[:, :, None] * 2.0 ** -51 / E / 60
        mag[..., u] = mag[..., v] = m * (1 + extra)
    return out, mag


def _check(got, ref, mag, what):
    bf = got.dtype == torch.bfloat16
    g = got.detach().cpu().to(torch.float64).numpy()
    tol = 60 * E * mag
    if bf:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           float(np.max(np.abs(g - ref) / np.maximum(tol, 1e-300))))


def _freqs(pairs, seed=0):
    f = 10000.0 ** (-np.arange(pairs) / max(pairs, 1))
    return np.asarray(f, dtype=np.float64)


def _heads(rng, shape, dtype, how):
    """A heads tensor laid out as `how`, its float64 values, and its buffer."""
    b, s, h, d = shape
    vals = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)
    if how == "dense":
        buf = torch.empty(shape, dtype=dtype, device="cuda")
        t = buf
    elif how == "fused":                         # the middle slice of a fused row
        buf = torch.full((b, s, 3 * h * d + 16), float("nan"), dtype=dtype, device="cuda")
        t = buf[..., h * d:2 * h * d].view(b, s, h, d)
    elif how == "head_major":
        buf = torch.full((b, h, s, d), float("nan"), dtype=dtype, device="cuda")
        t = buf.transpose(1, 2)
    elif how == "odd":                           # rows at odd element offsets: no wide access
        buf = torch.full((b, s, h * (d + 1) + 3), float("nan"), dtype=dtype, device="cuda")
        t = buf[..., 1:1 + h * (d + 1)].view(b, s, h, d + 1)[..., :d]
    else:
        raise ValueError(how)
    t.copy_(vals.cuda())
    return t, vals.double().numpy(), buf


DIMS = [(128, 128), (128, 64), (64, 64), (72, 72), (80, 40), (96, 64), (256, 256), (512, 512), (2, 2), (6, 4),
        (72, 36), (40, 6), (16, 16), (160, 160)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dim,rot", DIMS)
def test_rope_dims(gpu_lib, dtype, layout, dim, rot):
    rng = np.random.default_rng(dim * 7 + rot)
    for i, (b, s, h, how) in enumerate([(1, 1, 1, "dense"), (2, 5, 3, "fused"), (1, 67, 9, "head_major"),
                                        (2, 3, 5, "odd")]):
        inverse = i % 2 == 1
        _case(f"rope {dtype} {layout} dim={dim} rot={rot} {b}x{s}x{h} {how} inverse={inverse}")
        x, xv, _ = _heads(rng, (b, s, h, dim), dtype, how)
        pos = rng.integers(-50, 4000, (s, 1)).astype(np.int32)
        f = _freqs(rot // 2)
        y = gpu_lib.rope(x, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(), layout=layout, amplitude=1.25,
                         inverse=inverse)
        assert y.is_contiguous() and y.shape == x.shape
        ref, mag = _reference(xv, pos, f, (rot // 2,), layout, 1.25, inverse)
        _check(y, ref, mag, (dim, rot, how))
        # what is not rotated passes through bit for bit
        assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", ["head", "token"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dim,rot", DIMS)
def test_qk_norm_rope_dims(gpu_lib, dtype, norm, layout, dim, rot):
    rng = np.random.default_rng(dim * 11 + rot)
    for b, s, hq, hk, how, wdt in [(1, 1, 1, 1, "dense", torch.float32), (2, 5, 6, 2, "fused", dtype),
                                   (1, 35, 10, 5, "head_major", torch.float32), (2, 3, 7, 7, "odd", dtype)]:
        _case(f"qk_norm_rope {norm} {dtype} {layout} dim={dim} rot={rot} {b}x{s}x{hq},{hk} {how}")
        q, qv, _ = _heads(rng, (b, s, hq, dim), dtype, how)
        k, kv, _ = _heads(rng, (b, s, hk, dim), dtype, how)
        wq, wk = (torch.from_numpy((1 + 0.3 * rng.standard_normal(dim * (h if norm == "token" else 1))).astype(
            np.float32)).to(wdt) for h in (hq, hk))
        pos = rng.integers(0, 100000, (b, s, 2)).astype(np.int32)
        sections = (rot // 2 - rot // 6, rot // 6)
        f = np.concatenate([_freqs(sections[0]), _freqs(sections[1])])
        oq, ok = gpu_lib.qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(),
                                      q_weight=wq.cuda(), k_weight=wk.cuda(), eps=1e-5, norm=norm, layout=layout,
                                      sections=sections)
        for got, v, w in ((oq, qv, wq), (ok, kv, wk)):
            ref, mag = _reference(v, pos, f, sections, layout, weight=w.double().numpy(), norm=norm, eps=1e-5)
            _check(got, ref, mag, (dim, rot, how, norm))


@pytest.mark.parametrize("norm", ["head", "token"])
@pytest.mark.parametrize("hq,hk,dim", [(40, 40, 128), (5, 5, 64), (70, 1, 256), (129, 3, 72), (96, 32, 512)])
def test_many_heads(gpu_lib, norm, hq, hk, dim):
    """More heads than a pass of lanes holds, bf16, three position axes."""
    _case(f"qk_norm_rope {norm} heads {hq},{hk} dim {dim}")
    rng = np.random.default_rng(hq)
    b, s = 1, 19
    q, qv, _ = _heads(rng, (b, s, hq, dim), torch.bfloat16, "fused")
    k, kv, _ = _heads(rng, (b, s, hk, dim), torch.bfloat16, "fused")
    part = dim // 2 // 3
    sections = (dim // 2 - 2 * part, part, part)
    f = np.concatenate([_freqs(n) for n in sections])
    pos = rng.integers(0, 300, (s, 3)).astype(np.int32)
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(dim * (hq if norm == "token" else 1))).astype(np.float32))
    oq, ok = gpu_lib.qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(), q_weight=w.cuda(),
                                  norm=norm, sections=sections, layout="half", amplitude=0.75)
    for got, v, wt in ((oq, qv, w.double().numpy()), (ok, kv, None)):
        # a token's sum of 96 x 512 squares runs up to 2 x 96 + 14 additions deep
        ref, mag = _reference(v, pos, f, sections, "half", 0.75, weight=wt, norm=norm)
        _check(got, ref, mag * (2 if hq * dim > 16384 else 1), (hq, dim, norm))


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hk,dim,rot", [(1, 1, 128, 128), (3, 1, 64, 32), (2, 2, 72, 72), (4, 2, 128, 64), (1, 1, 16, 0),
                                           (1, 2, 40, 40), (5, 3, 96, 48), (2, 1, 256, 256), (2, 1, 72, 36), (4, 4, 76, 20)])
def test_few_heads_of_many_tokens(gpu_lib, dtype, layout, hq, hk, dim, rot):
    """Waves that take several tokens: the formulas, the bits of a call over
    few tokens, a position row per batch entry, in place, and the rows behind."""
    b, s = 3, 3461 if hq > 2 else 12289
    _case(f"few heads {dtype} {layout} {hq}+{hk} heads of {dim}, {rot} rotated, {b}x{s}")
    rng = np.random.default_rng(dim + rot + hq)
    pos = rng.integers(0, 5000, (b, s, 1)).astype(np.int32)
    f = _freqs(rot // 2)
    post, ft = torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda()
    buf = torch.full((b * s + 9, (hq + hk) * dim + 8), float("nan"), dtype=dtype, device="cuda")
    vals = torch.from_numpy(rng.standard_normal((b * s, (hq + hk) * dim)).astype(np.float32)).to(dtype)
    buf[:b * s, :(hq + hk) * dim] = vals.cuda()
    rows = buf[:b * s].view(b, s, -1)
    q = rows[..., :hq * dim].view(b, s, hq, dim)
    k = rows[..., hq * dim:(hq + hk) * dim].view(b, s, hk, dim)
    vals = vals.double().numpy().reshape(b, s, -1)
    wq, wk = (torch.from_numpy(rng.uniform(0.5, 1.5, dim).astype(np.float32)).to(dtype).cuda() for _ in range(2))
    yq, yk = gpu_lib.qk_norm_rope(q, k, post, ft, q_weight=wq, k_weight=wk, norm="head", layout=layout)
    for y, v, w, what in ((yq, vals[..., :hq * dim].reshape(b, s, hq, dim), wq, "q"),
                          (yk, vals[..., hq * dim:].reshape(b, s, hk, dim), wk, "k")):
        ref, mag = _reference(v, pos, f, (rot // 2,), layout, weight=w.double().cpu().numpy(), norm="head")
        _check(y, ref, mag, what)
    lo = s - 29                                           # a call over few tokens: the same bits
    fq, fk = gpu_lib.qk_norm_rope(q[:, lo:], k[:, lo:], post[:, lo:].contiguous(), ft, q_weight=wq, k_weight=wk,
                                  norm="head", layout=layout)
    assert torch.equal(fq, yq[:, lo:]) and torch.equal(fk, yk[:, lo:])
    if rot:
        turned = gpu_lib.rope(q, post, ft, layout=layout)
        assert torch.equal(turned[:, lo:], gpu_lib.rope(q[:, lo:], post[:, lo:].contiguous(), ft,
                                                            layout=layout))
    gpu_lib.qk_norm_rope(q, k, post, ft, q_weight=wq, k_weight=wk, norm="head", layout=layout, out_q=q,
                         out_k=k)
    assert torch.equal(q, yq) and torch.equal(k, yk)
    assert bool(torch.isnan(buf[b * s:]).all()) and bool(torch.isnan(buf[:, (hq + hk) * dim:]).all())


def test_far_positions(gpu_lib):
    """The angle stays exact where float32 has lost it, up to the largest int32."""
    _case("far positions")
    rng = np.random.default_rng(3)
    pos = np.array([[2 ** 31 - 1], [-2 ** 31], [2 ** 30 + 1], [12345678], [-1], [0], [1]], dtype=np.int32)
    x, xv, _ = _heads(rng, (1, len(pos), 2, 64), torch.float32, "dense")
    f = _freqs(32)
    y = gpu_lib.rope(x, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda())
    ref, mag = _reference(xv, pos, f, (32,), "interleaved")
    _check(y, ref, mag, "far")
    assert torch.equal(y[:, 5], x[:, 5])                     # position 0 turns nothing


@pytest.mark.parametrize("norm", [None, "head", "token"])
def test_in_place_and_neighbours(gpu_lib, norm):
    """q and k turned in place inside the fused row: the same bits as into
    new tensors, and nothing else in the buffer changes."""
    _case(f"in place, norm={norm}")
    rng = np.random.default_rng(17)
    b, s, hq, hk, d = 2, 37, 12, 4, 128
    row = (hq + 2 * hk) * d
    vals = torch.from_numpy(rng.standard_normal((b, s, row)).astype(np.float32)).bfloat16().cuda()
    buf = torch.full((b * s * row + 64,), 7.5, dtype=torch.bfloat16, device="cuda")
    body = buf[32:32 + b * s * row].view(b, s, row)
    body.copy_(vals)
    q, k = body[..., :hq * d].view(b, s, hq, d), body[..., hq * d:(hq + hk) * d].view(b, s, hk, d)
    pos = torch.arange(s, dtype=torch.int32, device="cuda")
    f = torch.from_numpy(_freqs(d // 2)).cuda()
    if norm is None:
        want_q = gpu_lib.rope(q, pos, f, layout="half")
        want_k = gpu_lib.rope(k, pos, f, layout="half")
        assert gpu_lib.rope(q, pos, f, layout="half", out=q) is q
        gpu_lib.rope(k, pos, f, layout="half", out=k)
    else:
        want_q, want_k = gpu_lib.qk_norm_rope(q, k, pos, f, norm=norm, layout="half")
        oq, ok = gpu_lib.qk_norm_rope(q, k, pos, f, norm=norm, layout="half", out_q=q, out_k=k)
        assert oq is q and ok is k
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(body[..., (hq + hk) * d:], vals[..., (hq + hk) * d:])
    assert (buf[:32] == 7.5).all() and (buf[32 + b * s * row:] == 7.5).all()


def test_inverse_is_the_gradient(gpu_lib):
    """<rope(x), g> = <x, rope(g, inverse)>, and each directional derivative
    of the rotation (linear: any step) against the inverse's."""
    _case("inverse against differences")
    rng = np.random.default_rng(23)
    b, s, h, d, rot = 1, 9, 3, 96, 64
    x, xv, _ = _heads(rng, (b, s, h, d), torch.float32, "dense")
    g, gv, _ = _heads(rng, (b, s, h, d), torch.float32, "dense")
    dx, dxv, _ = _heads(rng, (b, s, h, d), torch.float32, "dense")
    pos = torch.from_numpy(rng.integers(0, 999, s).astype(np.int32)).cuda()
    f = torch.from_numpy(_freqs(rot // 2)).cuda()
    for layout in ("interleaved", "half"):
        run = lambda t, inv=False: gpu_lib.rope(t, pos, f, layout=layout, amplitude=1.5, inverse=inv)
        grad = run(g, True).double().cpu().numpy()
        step = (run(x + dx).double() - run(x).double()).cpu().numpy()
        lhs, rhs = float((step * gv).sum()), float((dxv * grad).sum())
        # each side sums 2592 products of values within 60 e of theirs; x + dx
        # is rounded once more
        size = float((np.abs(gv) * (np.abs(xv) + np.abs(dxv)) * 3).sum())
        assert abs(lhs - rhs) <= 3 * 64 * E * size, (lhs, rhs)
        back = run(run(x), True).double().cpu().numpy()
        scale = np.ones(d)
        scale[:rot] = 1.5 ** 2
        assert np.max(np.abs(back - xv * scale)) <= 4 * 64 * E * 2.25 * 2 * np.max(np.abs(xv))


def test_norm_alone_and_zero_rows(gpu_lib):
    _case("norm without rotation; zero, tiny and non-finite rows")
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(6, 4, 64, device="cuda").to(dtype)
        x[0] = 0
        x[1] = 1e-20
        x[2, 1, 5] = float("inf")
        x[3, 0, 0] = float("nan")
        for norm in ("head", "token"):
            y, none = gpu_lib.qk_norm_rope(x, None, None, None, norm=norm)
            assert none is None
            xv = x.double().cpu().numpy()
            with np.errstate(invalid="ignore"):
                ref, mag = _reference(xv, None, [], (), "half", norm=norm)
            got = y.double().cpu().numpy()
            assert not got[0].any() and np.isfinite(got[1]).all()
            # a row with an infinity or a NaN touches no other row
            clean = np.ones(got.shape[:2], bool)
            clean[2, slice(None) if norm == "token" else 1] = False
            clean[3, slice(None) if norm == "token" else 0] = False
            _check(y[torch.from_numpy(clean).cuda()], ref[clean], mag[clean], norm)
            assert np.isnan(got[3, 0]).all()
            assert np.isnan(got[2, 1, 5]) and (np.delete(got[2, 1], 5) == 0).all()


def test_empty_and_refused_calls(gpu_lib):
    _case("refusals")
    f = torch.from_numpy(_freqs(32)).cuda()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    x = torch.randn(4, 2, 64, device="cuda")
    assert gpu_lib.rope(x[:0], pos[:0], f).shape == (0, 2, 64)
    bad = [(dict(x=x.half()), "bf16 or float32"), (dict(x=x.transpose(-1, -2)), "dense"), (dict(x=x[0]), "tokens, heads"),
           (dict(positions=pos.long()), "int32"), (dict(positions=pos[:3]), "positions must"),
           (dict(positions=pos.cpu()), "GPU"), (dict(freqs=f.float()), "float64"), (dict(freqs=f.cpu()), "GPU"),
           (dict(freqs=f.view(1, -1)), "1-D"), (dict(layout="other"), "layout"), (dict(sections=(16, 15)), "sections"),
           (dict(sections=(8,) * 5), "sections"), (dict(out=torch.empty(4, 2, 64, device="cuda").bfloat16()), "out"),
           (dict(out=torch.empty(4, 3, 64, device="cuda")), "out"), (dict(positions=None), "positions"),
           (dict(freqs=None), "freqs")]
    for kw, match in bad:
        with pytest.raises(ValueError, match=match):
            gpu_lib.rope(**{**dict(x=x, positions=pos, freqs=f), **kw})
    for kw in (dict(freqs=torch.cat([f, f])), dict(freqs=f[:0]), dict(amplitude=float("nan")),
               dict(out=x[:1].expand(4, 2, 64))):
        with pytest.raises((gpu_lib.DDGError, ValueError)):
            gpu_lib.rope(**{**dict(x=x, positions=pos, freqs=f), **kw})
    big = torch.randn(5, 2, 64, device="cuda")
    with pytest.raises(gpu_lib.DDGError):
        gpu_lib.rope(big[:4], pos, f, out=big[1:])                # shifted by a token
    for kw, match in [(dict(k=x.bfloat16()), "agree"), (dict(k=x[:3]), "agree"), (dict(norm="row"), "norm"),
                      (dict(q_weight=torch.ones(63, device="cuda")), "q_weight"),
                      (dict(q_weight=torch.ones(64, device="cuda"), k_weight=torch.ones(64, device="cuda").bfloat16()),
                       "one dtype"), (dict(k=None, k_weight=torch.ones(64, device="cuda")), "need k"),
                      (dict(positions=None), "positions"), (dict(freqs=None), "freqs")]:
        with pytest.raises(ValueError, match=match):
            gpu_lib.qk_norm_rope(**{**dict(q=x, k=x.clone(), positions=pos, freqs=f), **kw})
    with pytest.raises(gpu_lib.DDGError):
        gpu_lib.qk_norm_rope(x, x, pos, f, out_q=torch.empty_like(x), out_k=x)      # k's output is q's input


def test_past_4_gib(gpu_lib):
    """Rows whose byte offsets pass 32 bits: a fused buffer of 5 GB, read and
    written in place at its far end."""
    _case("offsets past 4 GiB")
    s, hq, d, row = 3, 4, 64, 900_000_000 // 8 * 8
    buf = torch.empty(s * row, dtype=torch.bfloat16, device="cuda")
    assert buf.numel() * 2 > 2 ** 32
    x = torch.as_strided(buf, (s, hq, d), (row, 800_000_000 // 4 // 8 * 8, 1))
    vals = torch.randn(s, hq, d, device="cuda").bfloat16()
    x.copy_(vals)
    pos = torch.tensor([5, 600, 70000], dtype=torch.int32, device="cuda")
    f = torch.from_numpy(_freqs(32)).cuda()
    want = gpu_lib.rope(vals, pos, f)
    assert torch.equal(gpu_lib.rope(x, pos, f), want)
    gpu_lib.rope(x, pos, f, out=x)
    assert torch.equal(x, want)
    wq = gpu_lib.qk_norm_rope(vals, None, pos, f, norm="token")[0]
    x.copy_(vals)
    assert torch.equal(gpu_lib.qk_norm_rope(x, None, pos, f, norm="token", out_q=x)[0], wq)
    del buf, x
    torch.cuda.empty_cache()


def test_streams_and_graph_replay(gpu_lib):
    """On a side stream, and captured into a graph that is replayed with new
    inputs between eager calls: the same bits as an eager call."""
    _case("side stream and graph replay")
    s, h, d = 33, 8, 128
    pos = torch.arange(s, dtype=torch.int32, device="cuda")
    f = torch.from_numpy(_freqs(d // 2)).cuda()
    q, k = (torch.randn(s, h, d, device="cuda").bfloat16() for _ in range(2))
    want = gpu_lib.qk_norm_rope(q, k, pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = gpu_lib.qk_norm_rope(q, k, pos, f)
        tok = gpu_lib.qk_norm_rope(q, k, pos, f, norm="token")
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    qs, ks = q.clone(), k.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        head = gpu_lib.qk_norm_rope(qs, ks, pos, f)
        token = gpu_lib.qk_norm_rope(qs, ks, pos, f, norm="token")
        turned = gpu_lib.rope(qs, pos, f, inverse=True)
    for i in range(4):
        a, b = (torch.randn(s, h, d, device="cuda").bfloat16() for _ in range(2))
        if i == 3:
            a, b = q, k
        qs.copy_(a)
        ks.copy_(b)
        e1, e2 = gpu_lib.qk_norm_rope(a, b, pos, f), gpu_lib.qk_norm_rope(a, b, pos, f, norm="token")
        e3 = gpu_lib.rope(a, pos, f, inverse=True)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for x, y in ((head, e1), (token, e2)):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1]), i
        assert torch.equal(turned, e3)
    assert torch.equal(token[0], tok[0])


def test_scaled_frequencies_end_to_end(gpu_lib):
    _case("yarn frequencies through rope")
    rng = np.random.default_rng(9)
    f, amp = gpu_lib.rope_frequencies(64, scaling="yarn", factor=4.0, original_length=8192)
    assert f.is_cuda and math.isclose(amp, 0.1 * math.log(4.0) + 1.0)
    x, xv, _ = _heads(rng, (2, 11, 3, 96), torch.bfloat16, "head_major")
    pos = (np.arange(11, dtype=np.int32) + 30000)[:, None]
    y = gpu_lib.rope(x, torch.from_numpy(pos[:, 0].copy()).cuda(), f, layout="half", amplitude=amp)
    ref, mag = _reference(xv, pos, f.cpu().numpy(), (32,), "half", amp)
    _check(y, ref, mag, "yarn")
