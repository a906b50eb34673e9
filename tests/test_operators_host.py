"""CPU-only checks of the rotary, paged-cache and token log-probability entry points: every refusal is
decided on the host before a device is touched, and bi_rope_freqs agrees with its formulas."""
import ctypes
import math

import pytest
import torch

from invariant_bi_matmul_02_b200 import binding
from invariant_bi_matmul_02_b200.csrc import build as libbuild

I, U, A = binding.BI_ERR_INVALID_ARG, binding.BI_ERR_UNSUPPORTED, binding.BI_ERR_ALIGNMENT
OK = binding.BI_OK
FAKE = 0x10000
NULL = None


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    libbuild.build_marshal()
    return binding.load()


def test_rope_refusals(lib):
    def rope(x=FAKE, xt=512, xh=128, y=2 * FAKE, yt=512, yh=128, dt=0, pos=FAKE, f=FAKE, T=4, H=4, D=128, R=128,
             layout=0):
        return lib.bi_rope(x, xt, xh, y, yt, yh, dt, pos, f, T, H, D, R, layout, 1.0, 0, NULL)

    for bad in (dict(T=-1), dict(H=-1), dict(D=0), dict(R=-2), dict(R=3), dict(R=130), dict(dt=7), dict(layout=2),
                dict(x=NULL), dict(y=NULL), dict(pos=NULL), dict(f=NULL), dict(xt=-1), dict(yh=127), dict(yt=64),
                dict(y=FAKE, yt=1024)):
        assert rope(**bad) == I, bad
    for bad in (dict(T=1 << 31), dict(H=65536, yt=1 << 30), dict(D=1026, R=2)):
        assert rope(**bad) == U, bad
    for bad in (dict(x=FAKE + 1), dict(y=2 * FAKE + 1), dict(dt=1, x=FAKE + 2), dict(pos=FAKE + 2), dict(f=FAKE + 4)):
        assert rope(**bad) == A, bad
    assert rope(T=0, x=NULL, y=NULL) == OK
    assert rope(H=0, x=NULL, y=NULL) == OK


def cache(**kw):
    d = dict(k=FAKE, v=2 * FAKE, pages=8, page_size=16, heads=2, head_dim=128, page_stride=4096, token_stride=256,
             head_stride=128)
    d.update(kw)
    return binding.PagedCache(*[d[n] for n, _ in binding.PagedCache._fields_])


BAD_CACHES = [(dict(k=NULL), I), (dict(v=NULL), I), (dict(pages=0), I), (dict(page_size=-1), I), (dict(heads=0), I),
              (dict(head_dim=0), I), (dict(token_stride=-256), I), (dict(head_stride=64), I), (dict(page_stride=8), I),
              (dict(pages=1 << 31), U), (dict(heads=65536), U), (dict(head_dim=2048), U), (dict(page_stride=1 << 40), U),
              (dict(k=FAKE + 8), A), (dict(page_stride=4100), A), (dict(token_stride=260), A), (dict(head_stride=132), A)]


def test_append_refusals(lib):
    def append(c=None, k=FAKE, kt=256, kh=128, v=FAKE, vt=256, vh=128, q=FAKE, qt=512, qh=128, qo=2 * FAKE, qot=512,
               qoh=128, Hq=4, table=FAKE, ts=8, mp=8, lens=FAKE, cu=NULL, pos=NULL, f=FAKE, R=128, layout=0, T=4, B=4):
        c = cache() if c is None else c
        return lib.bi_paged_append(k, kt, kh, v, vt, vh, q, qt, qh, qo, qot, qoh, Hq, ctypes.byref(c), table, ts, mp,
                                   lens, cu, pos, f, R, layout, 1.0, T, B, NULL)

    for kw, status in BAD_CACHES:
        assert append(c=cache(**kw)) == status, kw
    for bad in (dict(T=-1), dict(B=-1), dict(mp=-1), dict(R=1), dict(R=256), dict(layout=9), dict(qo=NULL),
                dict(q=NULL), dict(Hq=0), dict(T=5), dict(k=NULL), dict(v=NULL), dict(lens=NULL), dict(table=NULL),
                dict(f=NULL), dict(ts=4), dict(kt=-1), dict(qot=64), dict(qo=FAKE, qot=1024)):
        assert append(**bad) == I, bad
    for bad in (dict(T=1 << 31), dict(Hq=65536), dict(mp=1 << 31, ts=1 << 31)):
        assert append(**bad) == U, bad
    for bad in (dict(k=FAKE + 1), dict(table=FAKE + 2), dict(lens=FAKE + 1), dict(cu=FAKE + 2), dict(pos=FAKE + 2),
                dict(f=FAKE + 4)):
        assert append(**bad) == A, bad
    assert append(T=0, B=0, k=NULL) == OK
    assert lib.bi_paged_append(FAKE, 0, 0, FAKE, 0, 0, NULL, 0, 0, NULL, 0, 0, 0, NULL, FAKE, 1, 1, FAKE, NULL, NULL,
                               NULL, 0, 0, 1.0, 1, 1, NULL) == I  # no cache


def test_paged_attention_refusals(lib):
    def attend(c=None, q=FAKE, qs=1024, table=FAKE, ts=8, mp=8, lens=FAKE, out=FAKE, B=4, Hq=8, max_len=100,
               scratch=FAKE, nbytes=1 << 30):
        c = cache() if c is None else c
        return lib.bi_paged_decode_attention(q, qs, ctypes.byref(c), table, ts, mp, lens, out, B, Hq, max_len, 1.0,
                                             scratch, nbytes, NULL)

    for kw, status in BAD_CACHES:
        assert attend(c=cache(**kw)) == status, kw
    for bad in (dict(B=-1), dict(Hq=0), dict(Hq=7), dict(max_len=0), dict(mp=0), dict(max_len=129), dict(q=NULL),
                dict(table=NULL), dict(lens=NULL), dict(out=NULL), dict(qs=512), dict(ts=7),
                dict(mp=100, ts=100, max_len=600, scratch=NULL), dict(mp=100, ts=100, max_len=600, nbytes=1000)):
        assert attend(**bad) == I, bad
    for bad in (dict(c=cache(head_dim=96, head_stride=96)), dict(Hq=34), dict(B=65536), dict(Hq=65536),
                dict(mp=1 << 31, ts=1 << 31), dict(mp=1 << 30, ts=1 << 30, max_len=(1 << 31) - 2)):
        assert attend(**bad) == U, bad
    for bad in (dict(q=FAKE + 2), dict(out=FAKE + 8), dict(lens=FAKE + 2), dict(table=FAKE + 1), dict(qs=1028),
                dict(mp=100, ts=100, max_len=600, scratch=FAKE + 4)):
        assert attend(**bad) == A, bad
    assert attend(B=0, q=NULL) == OK and attend(B=0, mp=0, max_len=0) == OK
    need = lib.bi_paged_decode_attention_scratch_bytes
    assert need(4, 8, 128, 512) == 0 and need(0, 8, 128, 999) == 0
    assert need(4, 8, 128, 513) == 4 * 8 * 3 * (128 * 4 + 8)
    assert need(5000, 8, 128, 513) == need(2048, 8, 128, 513)  # sequences are taken 2048 at a time


def test_token_logprobs_refusals(lib):
    def lp(x=FAKE, ld=1000, dt=0, tok=FAKE, scale=1.0, k=5, out=FAKE, ent=FAKE, lse=FAKE, tl=FAKE, tt=FAKE, M=2, V=1000):
        return lib.bi_token_logprobs(x, ld, dt, tok, scale, k, out, ent, lse, tl, tt, M, V, NULL)

    for bad in (dict(M=-1), dict(V=-1), dict(k=-1), dict(dt=3), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=math.nan), dict(scale=math.inf), dict(scale=3e38), dict(V=0), dict(x=NULL), dict(ld=999),
                dict(V=4, k=5), dict(tok=NULL), dict(tl=NULL), dict(tt=NULL)):
        assert lp(**bad) == I, bad
    for bad in (dict(V=262145, ld=262145), dict(k=33), dict(M=1 << 30)):
        assert lp(**bad) == U, bad
    for bad in (dict(x=FAKE + 1), dict(dt=1, x=FAKE + 2), dict(tok=FAKE + 2), dict(out=FAKE + 1), dict(ent=FAKE + 2),
                dict(lse=FAKE + 2), dict(tl=FAKE + 2), dict(tt=FAKE + 3)):
        assert lp(**bad) == A, bad
    assert lp(M=0, x=NULL) == OK


def freqs(R, theta, kind="plain", **kw):
    f, s = binding.bi_rope_freqs(R, theta, kind, device="cpu", **kw)
    assert f.dtype == torch.float64 and f.shape == (R // 2,)
    return f.tolist(), s


def test_rope_freqs_formulas(lib):
    R, theta = 128, 1.0e6
    base = [theta ** (-2.0 * i / R) for i in range(R // 2)]
    got, scale = freqs(R, theta)
    assert scale == 1.0 and got == pytest.approx(base, rel=1e-14)
    got, scale = freqs(R, theta, "linear", factor=4.0)
    assert scale == 1.0 and got == pytest.approx([f / 4 for f in base], rel=1e-14)
    got, scale = freqs(R, theta, "ntk", factor=4.0)
    t = theta * 4.0 ** (R / (R - 2))
    assert scale == 1.0 and got == pytest.approx([t ** (-2.0 * i / R) for i in range(R // 2)], rel=1e-13)
    # yarn: pairs below the lower bound keep their frequency, above the upper one it is divided
    L, fast, slow = 32768.0, 32.0, 1.0
    lo = max(math.floor(R * math.log(L / (fast * 2 * math.pi)) / (2 * math.log(theta))), 0)
    hi = min(math.ceil(R * math.log(L / (slow * 2 * math.pi)) / (2 * math.log(theta))), R - 1)
    ramp = [min(max((i - lo) / (hi - lo), 0.0), 1.0) for i in range(R // 2)]
    got, scale = freqs(R, theta, "yarn", factor=4.0, original_length=L)
    assert scale == pytest.approx(0.1 * math.log(4.0) + 1.0, rel=1e-15)
    assert got == pytest.approx([f / 4 * r + f * (1 - r) for f, r in zip(base, ramp)], rel=1e-13)
    assert got[0] == base[0] and got[-1] == pytest.approx(base[-1] / 4, rel=1e-14)
    # banded: short wavelengths kept, long ones divided, a linear blend between
    got, scale = freqs(R, theta, "banded", factor=8.0, original_length=8192.0, low=1.0, high=4.0)
    for f, g in zip(base, got):
        wave = 2 * math.pi / f
        if wave < 8192 / 4:
            want = f
        elif wave > 8192:
            want = f / 8
        else:
            s = (8192 / wave - 1.0) / 3.0
            want = (1 - s) * f / 8 + s * f
        assert g == pytest.approx(want, rel=1e-13)
    assert scale == 1.0
    assert freqs(0, theta)[0] == []


@pytest.mark.parametrize("R", [2, 64, 128])
@pytest.mark.parametrize("theta", [1.0e4, 1.0e6])
def test_yarn_keeps_fast_pairs_and_divides_slow_ones_whatever_the_length(lib, R, theta):
    """Also where both bounds lie before the first pair or behind the last."""
    fast, slow, factor = 32.0, 1.0, 4.0
    base = [theta ** (-2.0 * i / R) for i in range(R // 2)]
    at = lambda turns, L: R * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    kept = divided = 0
    for e in range(-40, 40):
        L = 10.0 ** (e / 2)
        got, _ = freqs(R, theta, "yarn", factor=factor, original_length=L)
        for i, (f, g) in enumerate(zip(base, got)):
            assert f / factor * (1 - 1e-14) <= g <= f * (1 + 1e-14)
            if i <= at(fast, L) - 1:  # a whole pair clear of the bound, which is rounded to one
                assert g == pytest.approx(f, rel=1e-14), (L, i)
                kept += 1
            if i >= at(slow, L) + 1:
                assert g == pytest.approx(f / factor, rel=1e-14), (L, i)
                divided += 1
    assert kept and divided


def test_rope_freqs_refusals(lib):
    for args, kw in [((3, 1e4), {}), ((-2, 1e4), {}), ((2048, 1e4), {}), ((64, 1.0), {}), ((64, math.inf), {}),
                     ((64, 1e4, "linear"), dict(factor=0.5)), ((64, 1e4, "linear"), dict(factor=math.nan)),
                     ((2, 1e4, "ntk"), dict(factor=2.0)),
                     ((64, 1e4, "yarn"), dict(factor=2.0, original_length=100.0, beta_fast=1.0, beta_slow=1.0)),
                     ((64, 1e4, "banded"), dict(factor=2.0, original_length=100.0, low=4.0, high=1.0)),
                     ((64, 1e4, "banded"), dict(factor=2.0, original_length=-1.0, low=1.0, high=4.0))]:
        with pytest.raises(binding.BiError):
            binding.bi_rope_freqs(*args, device="cpu", **kw)
    with pytest.raises(ValueError):
        binding.bi_rope_freqs(64, 1e4, "spiral", device="cpu")
    with pytest.raises(ValueError):
        binding.bi_rope_freqs(64, 1e4, "linear", device="cpu")


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 3, 8, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(4, 16, 3, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.bi_rope(x, n, torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.bi_paged_append(x, x, c, c, n.view(2, 1), n)
    with pytest.raises(ValueError):
        binding.bi_paged_decode_attention(x, c, c, n.view(2, 1), n)
    with pytest.raises(ValueError):
        binding.bi_token_logprobs(torch.zeros(2, 8))


def test_missing_extension_module_fails_loudly(monkeypatch):
    import sys
    monkeypatch.setattr(binding, "_marshal", None)
    monkeypatch.setitem(sys.modules, "invariant_bi_matmul_02_b200._marshal", None)
    monkeypatch.delattr(sys.modules["invariant_bi_matmul_02_b200"], "_marshal", raising=False)
    with pytest.raises(RuntimeError, match="_marshal.so"):
        binding.load_marshal()


def test_extension_module_of_another_torch(lib, monkeypatch):
    """An extension module built for another torch is rebuilt, and refused where it is loaded."""
    assert libbuild.marshal_current()
    runs = []
    monkeypatch.setattr(libbuild.subprocess, "run", lambda cmd, **kw: runs.append(cmd))
    libbuild.build_marshal()
    assert not runs
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    libbuild.build_marshal()
    assert len(runs) == 1
    monkeypatch.setattr(binding, "_marshal", None)
    with pytest.raises(RuntimeError, match="0.0.1"):
        binding.load_marshal()
