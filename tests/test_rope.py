"""Rotary positions on the host (CPU only): the frequency table against the
formulas in extended precision, and the calls' refusals, which all return
before anything is launched (the fake addresses below never reach a kernel)."""
import ctypes
import math
import os
import random
from decimal import Decimal, getcontext

import pytest
import torch

from dit_dequant_gemm_amd import api

OK, E_ARG, E_SHAPE, E_ALIGN = 0, -1, -2, -3
FAKE = 0x10000000
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(api.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return api.load_library()


def _freqs(lib, rot, base=10000.0, scaling=0, factor=1.0, length=0.0, fast=32.0, slow=1.0):
    out = (ctypes.c_double * max(rot // 2, 1))()
    amp = ctypes.c_double()
    st = lib.ddg_rope_frequencies(rot, base, scaling, factor, length, fast, slow, out, ctypes.byref(amp))
    return st, list(out), amp.value


@pytest.mark.parametrize("rot", [2, 4, 44, 64, 72, 128, 512])
@pytest.mark.parametrize("base,scaling,factor,length", [
    (10000.0, "none", 1.0, 0.0), (500000.0, "none", 1.0, 0.0), (10000.0, "linear", 8.0, 0.0),
    (10000.0, "ntk", 4.0, 0.0), (10000.0, "yarn", 4.0, 8192.0), (1000000.0, "yarn", 32.0, 4096.0),
    (10000.0, "yarn", 1.0, 100.0)])
def test_frequencies_follow_the_formulas(lib, rot, base, scaling, factor, length):
    code = api.ROPE_SCALINGS[scaling]
    if scaling == "ntk" and rot < 4:
        assert _freqs(lib, rot, base, code, factor, length)[0] == E_SHAPE
        return
    st, got, amp = _freqs(lib, rot, base, code, factor, length)
    assert st == OK
    getcontext().prec = 40
    b = Decimal(base)
    if scaling == "ntk":
        b = b * Decimal(factor) ** (Decimal(rot) / Decimal(rot - 2))

    def pair_of(turns):
        return rot * math.log(length / (2.0 * math.pi * turns)) / (2.0 * math.log(base))

    for i, g in enumerate(got):
        f = b ** (Decimal(-2 * i) / Decimal(rot))
        if scaling == "linear":
            f = f / Decimal(factor)
        elif scaling == "yarn":
            lo, hi = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), rot - 1)
            r = Decimal(min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0))
            f = f * (1 - r) + f / Decimal(factor) * r
        # pow within an ulp, at most four more roundings; the exponent's own
        # rounding (2^-53 of at most ln(base) plus ln(factor)) counts 20 times
        assert abs(Decimal(g) - f) <= f * Decimal(32 * 2.0 ** -53), (i, g, f)
    want = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
    assert abs(amp - want) <= 4 * 2.0 ** -52


def test_frequencies_refusals(lib):
    nan, inf = float("nan"), float("inf")
    assert _freqs(lib, 3)[0] == E_SHAPE and _freqs(lib, 0)[0] == E_SHAPE and _freqs(lib, 514)[0] == E_SHAPE
    for base in (1.0, 0.0, -2.0, nan, inf):
        assert _freqs(lib, 64, base=base)[0] == E_ARG
    assert _freqs(lib, 64, scaling=4)[0] == E_ARG and _freqs(lib, 64, scaling=-1)[0] == E_ARG
    for factor in (0.5, nan, inf):
        assert _freqs(lib, 64, scaling=1, factor=factor)[0] == E_ARG
    for kw in (dict(length=0.0), dict(length=nan), dict(length=100.0, slow=0.0), dict(length=100.0, fast=0.5),
               dict(length=100.0, fast=inf)):
        assert _freqs(lib, 64, scaling=3, factor=2.0, **kw)[0] == E_ARG
    amp = ctypes.c_double()
    assert lib.ddg_rope_frequencies(64, 10000.0, 0, 1.0, 0.0, 32.0, 1.0, None, ctypes.byref(amp)) == E_ARG


def _tensor(x=FAKE, y=2 * FAKE, heads=4, xs=(4096, 512, 128), ys=(4096, 512, 128), weight=None):
    return api.RopeTensor(x, y, weight, heads, *xs, *ys)


def _desc(**kw):
    d = api.RopeDesc(positions=3 * FAKE, positions_batch=0, freqs=4 * FAKE, axes=1, rot_dim=128, layout=0, inverse=0,
                     amplitude=1.0)
    d.sections[0] = 64
    for k, v in kw.items():
        if k == "sections":
            for i, s in enumerate(v):
                d.sections[i] = s
        else:
            setattr(d, k, v)
    return d


def _rope(lib, t=None, d=None, dtype=BF16, batch=2, tokens=8, dim=128):
    t, d = t or _tensor(), d or _desc()
    return lib.ddg_rope(ctypes.byref(t), dtype, batch, tokens, dim, ctypes.byref(d), None)


def _norm(lib, q=None, k=None, d=None, dtype=BF16, wdtype=BF16, batch=2, tokens=8, dim=128, norm=1, eps=1e-6):
    q, d = q or _tensor(), d or _desc()
    return lib.ddg_qk_norm_rope(ctypes.byref(q), None if k is None else ctypes.byref(k), dtype, wdtype, batch, tokens,
                                dim, norm, eps, ctypes.byref(d), None)


def test_empty_calls_are_no_ops(lib):
    assert _rope(lib, tokens=0) == OK and _rope(lib, batch=0) == OK
    assert _rope(lib, t=_tensor(x=None, y=None), tokens=0) == OK
    assert _norm(lib, tokens=0) == OK and _norm(lib, batch=0, norm=2) == OK


def test_argument_refusals(lib):
    nan, inf = float("nan"), float("inf")
    for call in (_rope, _norm):
        assert call(lib, dtype=2) == E_ARG
        assert call(lib, d=_desc(layout=2)) == E_ARG
        assert call(lib, d=_desc(inverse=2)) == E_ARG
        for amp in (nan, inf, -inf):
            assert call(lib, d=_desc(amplitude=amp)) == E_ARG
        assert call(lib, d=_desc(positions=None)) == E_ARG
        assert call(lib, d=_desc(freqs=None)) == E_ARG
        assert call(lib, batch=-1) == E_SHAPE and call(lib, tokens=-1) == E_SHAPE
        assert call(lib, batch=1 << 16, tokens=1 << 15) == E_SHAPE
        for dim in (0, 127, 514):
            assert call(lib, dim=dim) == E_SHAPE
        assert call(lib, d=_desc(rot_dim=130, sections=(65,))) == E_SHAPE
        assert call(lib, d=_desc(rot_dim=63)) == E_SHAPE
        assert call(lib, d=_desc(rot_dim=-2, sections=(-1,))) == E_SHAPE
        assert call(lib, d=_desc(axes=0)) == E_SHAPE and call(lib, d=_desc(axes=5)) == E_SHAPE
        assert call(lib, d=_desc(sections=(63,))) == E_SHAPE
        assert call(lib, d=_desc(axes=2, sections=(65, -1))) == E_SHAPE
        assert call(lib, d=_desc(positions_batch=-1)) == E_SHAPE
        assert call(lib, d=_desc(positions=3 * FAKE + 2)) == E_ALIGN
        assert call(lib, d=_desc(freqs=4 * FAKE + 4)) == E_ALIGN
    assert _rope(lib, d=_desc(rot_dim=0, sections=(0,))) == E_SHAPE
    for eps in (-1e-6, nan, inf):
        assert _norm(lib, eps=eps) == E_ARG
    for norm in (0, 3, -1):
        assert _norm(lib, norm=norm) == E_ARG
    assert _norm(lib, wdtype=2) == E_ARG
    assert lib.ddg_rope(None, BF16, 1, 1, 128, ctypes.byref(_desc()), None) == E_ARG
    assert lib.ddg_rope(ctypes.byref(_tensor()), BF16, 1, 1, 128, None, None) == E_ARG
    for which in ("q", "k"):
        def bad(**kw):
            t = _tensor(**{"x": 8 * FAKE, "y": 9 * FAKE, **kw})
            return _norm(lib, q=t) if which == "q" else _norm(lib, k=t)
        assert bad(x=None) == E_ARG and bad(y=None) == E_ARG
        assert bad(heads=0) == E_SHAPE and bad(heads=65536) == E_SHAPE
        assert bad(xs=(4096, -512, 128)) == E_SHAPE
        assert bad(ys=(1 << 60, 512, 128)) == E_SHAPE
        assert bad(x=8 * FAKE + 1) == E_ALIGN and bad(y=9 * FAKE + 1) == E_ALIGN
        assert bad(weight=FAKE + 1) == E_ALIGN


def test_overlap_refusals(lib):
    row = (3 * 512) * 8, 3 * 512, 128                # batch, token, head strides of a fused q, k, v row
    two = 2                                          # bytes of a bf16

    # an output that names an element twice
    assert _rope(lib, t=_tensor(ys=(4096, 512, 64))) == E_ARG
    assert _rope(lib, t=_tensor(ys=(0, 512, 128))) == E_ARG
    assert _rope(lib, t=_tensor(ys=(4096, 256, 128))) == E_ARG
    # in place under other strides, or shifted by a value, a head, a token
    assert _rope(lib, t=_tensor(y=FAKE, ys=(8192, 1024, 128))) == E_ARG
    assert _rope(lib, t=_tensor(y=FAKE + 8 * two)) == E_ARG
    for shift in (128, 512, 4096):
        assert _rope(lib, t=_tensor(y=FAKE + shift * two)) == E_ARG
        assert _rope(lib, t=_tensor(x=FAKE + shift * two, y=FAKE)) == E_ARG
    # the next slice of the fused row, too far by half a head
    assert _rope(lib, t=_tensor(y=FAKE + (512 - 64) * two, xs=row, ys=row)) == E_ARG
    # q and k: each output against the other input and output
    q, k = _tensor(), _tensor(x=8 * FAKE, y=2 * FAKE + 512 * two)
    assert _norm(lib, q=q, k=k) == E_ARG
    assert _norm(lib, q=_tensor(), k=_tensor(x=2 * FAKE, y=9 * FAKE)) == E_ARG
    assert _norm(lib, q=_tensor(), k=_tensor(x=9 * FAKE, y=FAKE)) == E_ARG


def _cells(batch, tokens, heads, dim, strides, start):
    return {start + b * strides[0] + t * strides[1] + h * strides[2] + e
            for b in range(batch) for t in range(tokens) for h in range(heads) for e in range(dim)}


def test_overlap_rule_against_enumeration(lib):
    """Random small views of one buffer: a call that the rule lets through
    (here: up to the missing GPU) shares no element between input and output
    unless they are the same view, and writes none twice; slices of a fused
    row and of head-major copies are let through."""
    if torch.cuda.is_available():
        pytest.skip("accepted calls would launch: runs where there is no GPU")
    rng = random.Random(5)
    past = None
    for _ in range(3000):
        batch, tokens, heads, dim = rng.randint(1, 3), rng.randint(1, 3), rng.randint(1, 3), 4

        def strides():
            unit = [4, heads * 4, heads * 8, 12, 24, 36, tokens * heads * 4, tokens * heads * 8, 3 * tokens * heads * 4]
            return tuple(rng.choice(unit) for _ in range(3))
        xs = strides()
        ys = xs if rng.random() < 0.7 else strides()
        xo, yo = 64, 64 + rng.choice([0, 4, -4, 8, heads * 4, -heads * 4, 12, 24, tokens * heads * 4, 2, 100, 400])
        t = _tensor(x=FAKE + 4 * xo, y=FAKE + 4 * yo, heads=heads, xs=xs, ys=ys)
        d = _desc(rot_dim=4, sections=(2,), positions=64 * FAKE, freqs=65 * FAKE)
        st = _rope(lib, t=t, d=d, dtype=F32, batch=batch, tokens=tokens, dim=dim)
        y = _cells(batch, tokens, heads, dim, ys, yo)
        x = _cells(batch, tokens, heads, dim, xs, xo)
        same = xo == yo and all(n == 1 or a == b for n, a, b in zip((batch, tokens, heads), xs, ys))
        twice = len(y) < batch * tokens * heads * dim
        if st != E_ARG:
            past = st if past is None else past
            assert st == past and not twice and (same or not (x & y)), (batch, tokens, heads, xs, ys, xo, yo)
        elif same:
            assert twice or not _nested(y, (batch, tokens, heads), ys, dim), (batch, tokens, heads, xs)
    assert past is not None


def _nested(cells, sizes, strides, dim):
    reach = dim
    for st, n in sorted((st, n) for n, st in zip(sizes, strides) if n > 1):
        if st < reach:
            return False
        reach += (n - 1) * st
    return True


def test_binding_refusals_on_the_host():
    with pytest.raises(ValueError, match="scaling"):
        api.rope_frequencies(64, scaling="other", device="cpu")
    with pytest.raises(ValueError, match="dim"):
        api.rope_frequencies(63, device="cpu")
    f, amp = api.rope_frequencies(64, scaling="yarn", factor=4.0, original_length=8192, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and amp > 1.0
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        api.rope(x, torch.zeros(4, dtype=torch.int32), f)
    with pytest.raises(ValueError, match="norm"):
        api.qk_norm_rope(x, x, None, None, norm="layer")
