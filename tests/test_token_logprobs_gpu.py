"""bi_token_logprobs against log_softmax in fp64, ties, masks and the bits across launch shapes.

Tolerances, with u = 2^-24, d_j = scale (x_j - max x), p the probabilities, E1 = sum p |d|, E2 = sum p d^2:
* S = sum exp(d): each exponential is off by u (4 + 3 |d|) of itself (ex2.approx 2^-22; the difference, the
  constant and the product round once each); a term passes at most 16 + 1 + 5 additions and 21 merges of 3 roundings
  and two exp2f (2 units each): 22 + 21 * 7 < 180.  So log S is off by at most s_err = u (190 + 3 E1) + 2 u log S.
* logprob = d_t - log S: s_err + u (3 |d_t| + |logprob|).   logsumexp = scale max + log S: s_err + u (2 |scale max| + |value|).
* T = sum e d: each d is off by 3 u |d| on top of e's error, same chain: T / S by u (190 E1 + 6 E2) + s_err E1;
  entropy = log S - T / S: that plus s_err + 2 u (E1 + |entropy|).
"""
import ctypes
import io
import math

import pytest
import torch

from bi_testutil import same_bits
from invariant_bi_matmul_02_b200 import binding as bi

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def definition(x, tokens, scale, k):
    z = x.double() * scale
    m = z.amax(1, keepdim=True)
    d = z - m
    log_s = torch.logsumexp(d, 1)
    lp = d - log_s[:, None]
    p = lp.exp()
    dz = torch.where(p > 0, d, torch.zeros_like(d))
    e1, e2 = (p * dz.abs()).sum(1), (p * dz * dz).sum(1)
    h = log_s + e1
    s_err = U * (190 + 3 * e1) + 2 * U * log_s
    t = tokens.long().clamp(min=0)[:, None]
    want = torch.where(tokens < 0, 0.0, lp.gather(1, t)[:, 0])
    dt = d.gather(1, t)[:, 0].abs()
    order = torch.sort(x.double(), dim=1, descending=True, stable=True)[1][:, :k]
    tl, td = lp.gather(1, order), d.gather(1, order).abs()
    return dict(logprobs=(want, s_err + U * (3 * dt + want.abs())),
                logsumexp=(m[:, 0] + log_s, s_err + U * (2 * m[:, 0].abs() + (m[:, 0] + log_s).abs())),
                entropy=(h, U * (190 * e1 + 6 * e2) + s_err * (1 + e1) + 2 * U * (e1 + h)),
                top_logprobs=(tl, s_err[:, None] + U * (3 * td + tl.abs()))), order


def check(x, tokens, scale=1.0, k=0):
    got = bi.bi_token_logprobs(x, tokens, k, scale)
    want, order = definition(x, tokens, scale, k)
    assert torch.equal(got.top_tokens.long(), order)
    for name, (ref, bound) in want.items():
        g = getattr(got, name).double()
        inf = ref.float() == -math.inf  # a value below -FLT_MAX rounds to -inf in the output's type
        assert torch.equal(g == -math.inf, inf), name
        err = torch.where(inf, 0.0, (g - ref).abs())
        assert bool((err <= torch.where(inf, 0.0, bound)).all()), (name, float((err - bound).max()))
    return got


def rows(seed, M, V, dtype, std=1.3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (std * torch.randn(M, V, generator=g, device=DEV)).to(dtype)
    return x, torch.randint(0, V, (M,), generator=g, device=DEV).to(torch.int32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V,k", [
    (1, 1, 1), (3, 2, 2), (5, 31, 5), (2, 33, 32), (7, 1000, 20), (4, 8192, 32), (4, 8193, 1), (3, 16384, 7),
    (3, 16385, 20), (1, 151936, 20), (9, 151936, 32), (33, 50257, 8), (20, 32001, 0), (2, 262144, 32), (300, 4096, 4),
    (310, 40000, 20), (1, 262143, 5),
])
def test_parity(M, V, k, dtype):
    x, t = rows(M + V, M, V, dtype)
    check(x, t, 1.0, k)
    check(x, t, 1.0 / 0.7, k)
    assert bi.bi_get_device_status() == bi.BI_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_go_to_the_lowest_token(dtype):
    V = 40000
    g = torch.Generator(device=DEV).manual_seed(1)
    t = torch.zeros(1, dtype=torch.int32, device=DEV)
    for x in (torch.zeros(1, V), torch.full((1, V), -3.5), torch.randint(0, 3, (1, V)).float(),
              torch.randint(0, 40, (1, V)).float(), torch.arange(V).float()[None] // 7, -torch.arange(V).float()[None],
              torch.tensor([0.0, -0.0] * (V // 2))[None]):
        x = x.to(DEV).to(dtype)
        check(x, t, 1.0, 32)
        check(x, t, 1.0, 1)
        check(x[:, torch.randperm(V, generator=g, device=DEV)].contiguous(), t, 2.0, 20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("low", [-math.inf, None])
def test_masked_rows(dtype, low):
    """Masks of -inf or of the type's lowest value; rows with fewer live entries than top_k, and with one."""
    M, V = 6, 50257
    x, t = rows(5, M, V, dtype)
    fill = torch.finfo(dtype).min if low is None else low
    keep = torch.rand(M, V, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV) < 0.001
    keep[1] = False
    keep[1, 40000] = True
    keep[2] = False
    keep[2, :3] = True
    keep[3, :16384] = False
    x = torch.where(keep, x, torch.full_like(x, fill))
    t = torch.tensor([int(torch.nonzero(r)[0]) for r in keep], dtype=torch.int32, device=DEV)
    check(x, t, 1.0, 20)
    if low is None:
        same = torch.full((2, V), fill, dtype=dtype, device=DEV)  # everything masked by the lowest value: uniform
        got = bi.bi_token_logprobs(same, t[:2], 3)
        assert torch.allclose(got.logprobs.double(), torch.tensor(-math.log(V), dtype=torch.float64, device=DEV), atol=1e-5)
        assert torch.allclose(got.entropy.double(), torch.tensor(math.log(V), dtype=torch.float64, device=DEV), atol=1e-5)
        assert got.top_tokens.tolist() == [[0, 1, 2]] * 2


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_without_a_distribution(dtype):
    V = 20000
    x, t = rows(6, 5, V, dtype)
    x[0] = -math.inf
    x[1, 7] = math.nan
    x[2, 19999] = math.inf
    x[3] = math.nan
    got = bi.bi_token_logprobs(x, t, 3)
    for r in range(4):
        assert math.isnan(float(got.logprobs[r])) and math.isnan(float(got.entropy[r])), r
        assert bool(got.top_logprobs[r].isnan().all()), r
    assert float(got.logsumexp[0]) == -math.inf
    assert bool(got.logsumexp[1:4].isnan().all())
    assert got.top_tokens[0].tolist() == [0, 1, 2] and got.top_tokens[3].tolist() == [0, 1, 2]
    ranked = torch.sort(torch.where(x[1].isnan(), -math.inf, x[1].double()), descending=True, stable=True)[1][:3]
    assert got.top_tokens[1].tolist() == ranked.tolist()
    assert int(got.top_tokens[2, 0]) == 19999
    want, _ = definition(x[4:], t[4:], 1.0, 3)
    assert abs(float(got.logprobs[4]) - float(want["logprobs"][0][0])) <= float(want["logprobs"][1][0])
    # Fewer numbers than top_k: NaN entries fill up, lowest token first.
    y = torch.full((1, 6), math.nan, dtype=dtype, device=DEV)
    y[0, 3] = 1.0
    y[0, 5] = -math.inf
    assert bi.bi_token_logprobs(y, None, 5).top_tokens.tolist() == [[3, 5, 0, 1, 2]]


def test_far_values():
    x, t = rows(7, 4, 5000, torch.float32)
    check(x + 1.0e4, t, 1.0, 5)
    check(x * 1.0e4, t, 1.0, 5)
    check(x * 1.0e30, t, 1.0, 5)
    check(x, t, 1.0e-6, 5)
    big = torch.zeros(1, 300, device=DEV)
    big[0, 0], big[0, 1] = 3.0e38, -3.0e38
    check(big, t[:1] % 2, 1.0, 3)


def test_tokens_outside_the_vocabulary():
    x, t = rows(8, 4, 1000, torch.float32)
    want = bi.bi_token_logprobs(x, t)
    t2 = t.clone()
    t2[1], t2[2] = -1, -100
    got = bi.bi_token_logprobs(x, t2)
    assert got.logprobs[1:3].tolist() == [0.0, 0.0] and same_bits(got.logprobs[3:], want.logprobs[3:])
    assert bi.bi_get_device_status() == bi.BI_OK
    t2[0] = 1000
    got = bi.bi_token_logprobs(x, t2)
    assert math.isnan(float(got.logprobs[0])) and same_bits(got.entropy, want.entropy)
    assert bi.bi_get_device_status() == bi.BI_ERR_INVALID_ARG
    assert bi.bi_token_logprobs(x).logprobs is None


def equal(a, b):
    return all((x is None and y is None) or same_bits(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [50257, 151936, 9000])
def test_rows_do_not_depend_on_the_batch(V, dtype):
    """A row alone (shared by 8 blocks) and in batches of every sharing has the same bits, aligned or not."""
    M = 330
    x, t = rows(9, M, V, dtype)
    want = bi.bi_token_logprobs(x, t, 20, 1.25)
    for m in (1, 30, 60, 100, 200):
        for r0 in (0, M - m):
            got = bi.bi_token_logprobs(x[r0:r0 + m], t[r0:r0 + m], 20, 1.25)
            assert equal(got, [w[r0:r0 + m].contiguous() for w in want]), (m, r0)
    wide = torch.full((40, V + 13), 99.0, dtype=dtype, device=DEV)
    wide[:, 5:V + 5] = x[:40]
    got = bi.bi_token_logprobs(wide[:, 5:V + 5], t[:40], 20, 1.25)
    assert equal(got, [w[:40].contiguous() for w in want])
    for _ in range(20):
        assert equal(bi.bi_token_logprobs(x, t, 20, 1.25), want)


def test_empty_streams_graphs_and_refusals():
    x, t = rows(10, 5, 30000, torch.bfloat16)
    empty = bi.bi_token_logprobs(x[:0], t[:0], 3)
    assert empty.logprobs.shape == (0,) and empty.top_tokens.shape == (0, 3)
    want = bi.bi_token_logprobs(x, t, 3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = bi.bi_token_logprobs(x, t, 3, stream=side)
    side.synchronize()
    assert equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bi.bi_token_logprobs(x, t, 3)
    x2, t2 = rows(11, 5, 30000, torch.bfloat16)
    want = bi.bi_token_logprobs(x2, t2, 3)
    x.copy_(x2)
    t.copy_(t2)
    graph.replay()
    torch.cuda.synchronize()
    assert equal(got, want)
    for bad in (lambda: bi.bi_token_logprobs(x[0]), lambda: bi.bi_token_logprobs(x, t[:2]),
                lambda: bi.bi_token_logprobs(x, t, -1), lambda: bi.bi_token_logprobs(x[:, :3], t, 4),
                lambda: bi.bi_token_logprobs(x.t()), lambda: bi.bi_token_logprobs(x, t.view(5, 1))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        bi.bi_token_logprobs(x, t.long())
    for bad in (lambda: bi.bi_token_logprobs(x, t, 33), lambda: bi.bi_token_logprobs(x, t, 0, 0.0),
                lambda: bi.bi_token_logprobs(torch.zeros(1, 262145, device=DEV))):
        with pytest.raises(bi.BiError):
            bad()


def test_log_softmax_agrees():
    """The library's own log_softmax over the same rows, at its tolerance."""
    x, t = rows(12, 8, 151936, torch.bfloat16)
    y = bi.bi_log_softmax(x)
    got = bi.bi_token_logprobs(x, t, 4)
    assert float((y.gather(1, t.long()[:, None])[:, 0] - got.logprobs).abs().max()) <= 1e-4
    assert float((y.gather(1, got.top_tokens.long()) - got.top_logprobs).abs().max()) <= 1e-4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("low", [-math.inf, -1e30, -1e4, 0.0])
@pytest.mark.parametrize("M,V,kept", [(1, 50257, 40), (5, 50257, 3), (3, 9000, 700), (90, 50257, 100), (170, 40000, 8),
                                      (330, 20000, 15)])
def test_few_tokens_clear_of_a_mask(M, V, kept, low, dtype):
    """Blocks of a row in which fewer than k threads have a token that the mask left, at every cluster size."""
    x, _ = rows(V + kept, M, V, dtype)
    g = torch.Generator(device=DEV).manual_seed(kept)
    at = torch.rand(M, V, generator=g, device=DEV).topk(kept, dim=1)[1]
    y = torch.full_like(x, low)
    y.scatter_(1, at, x.gather(1, at).abs() + 1)
    check(y, at[:, 0].to(torch.int32), 0.9, 8)
    check(y, at[:, 0].to(torch.int32), 0.9, 32)


def nan_last(row, k):
    """The k best tokens of a row: numbers in descending order, then NaN, equals by ascending token."""
    by = torch.sort(torch.where(row.isnan(), -math.inf, row.double()), descending=True, stable=True)[1]
    return by[torch.sort(row.isnan()[by].int(), stable=True)[1]][:k]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [2, 40, 1000, 1024, 9000, 50257])
@pytest.mark.parametrize("M", [9, 711])
def test_every_place_of_the_best_is_written_in_rows_of_nan(M, V, dtype):
    """Rows with fewer numbers than top_k, and their last group of elements cut by the row's end, at one block a row and
    at more: every place holds a token, numbers first."""
    nan, inf = math.nan, math.inf
    kinds = torch.full((9, V), nan, dtype=dtype)
    kinds[1, 0] = 1.0
    kinds[2, V - 1] = 1.0
    kinds[3, V // 2] = -inf
    kinds[4, :V - 1] = -inf
    kinds[5, :V // 2] = -2.0
    kinds[6, :V - 1] = 3.0
    kinds[7, ::7] = 0.5
    kinds[8, 0], kinds[8, V - 1] = -inf, -inf if V > 2 else nan
    x = kinds.to(DEV).repeat(-(-M // 9), 1)[:M].contiguous()
    for k in (1, 2, 5, 32):
        if k > V:
            continue
        tl = torch.full((M, k), 77.0, device=DEV)
        tt = torch.full((M, k), -12345, dtype=torch.int32, device=DEV)
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert bi.load().bi_token_logprobs(x.data_ptr(), V, bi._DT[dtype], None, 1.0, k, None, None, None, tl.data_ptr(),
                                           tt.data_ptr(), M, V, stream) == bi.BI_OK
        want = torch.stack([nan_last(r, k) for r in x[:9]])
        assert torch.equal(tt.long(), want.repeat(-(-M // 9), 1)[:M]), k
        assert bool(tl.isnan().all()), k


@pytest.mark.parametrize("k", [0, 4])
def test_results_can_be_saved_and_kept_apart(k):
    x, t = rows(13, 3, 500, torch.bfloat16)
    r = bi.bi_token_logprobs(x, t, k)
    at = io.BytesIO()
    torch.save(tuple(r), at)
    at.seek(0)
    assert all(same_bits(a, b) for a, b in zip(torch.load(at), r))
    assert all(v.untyped_storage().nbytes() == v.numel() * v.element_size() for v in r)
    assert bi.bi_token_logprobs(x, None, k).logprobs is None
