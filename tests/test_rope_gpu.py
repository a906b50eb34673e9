"""bi_rope against the definition in fp64 (complex multiplication), and its bits across launch shapes.

Tolerance: with pair (a, b) and scale s, the kernel's fp32 value is off by at most
  s (|a| + |b|) * 2^-21:  the fraction of a turn is rounded once (2^-26 turns = 2^-23.3 radians), sincospif is within
  2 units of its last place (2^-23), and the scale, the product and the fused sum round once each (2^-24 of |a| + |b|);
then one rounding to the output's type (eps / 2 of the value).
"""
import pytest
import torch

from bi_testutil import same_bits
from invariant_bi_matmul_02_b200 import binding as bi

pytestmark = pytest.mark.gpu
DEV = "cuda"


def definition(x, pos, inv_freq, layout, scale, inverse):
    T, H, D = x.shape
    R = 2 * inv_freq.shape[0]
    w = torch.exp(1j * (pos.double()[:, None] * inv_freq).to(torch.complex128))
    w = (w.conj() if inverse else w)[:, None, :]
    y, mag = x.double(), torch.zeros(T, H, D, dtype=torch.float64, device=x.device)
    if layout == "half":
        a, b = slice(0, R // 2), slice(R // 2, R)
    else:
        a, b = slice(0, R, 2), slice(1, R, 2)
    z = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * w * scale
    both = (x.double()[..., a].abs() + x.double()[..., b].abs()) * scale
    y[..., a], y[..., b] = z.real, z.imag
    mag[..., a] = mag[..., b] = both
    return y, mag


def check(got, x, pos, inv_freq, layout, scale, inverse):
    want, mag = definition(x, pos, inv_freq, layout, scale, inverse)
    bound = mag * 2.0 ** -21 + torch.finfo(got.dtype).eps / 2 * want.abs() * (1 + 2.0 ** -20)
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), float((err - bound).max())


def make(seed, T, H, D, R, dtype, theta=1e6, start=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, D, generator=g, device=DEV).to(dtype)
    pos = (start + torch.arange(T, device=DEV)).to(torch.int32)
    return x, pos, bi.bi_rope_freqs(R, theta)[0]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D,R", [
    (1, 40, 128, 128),    # one token
    (3, 13, 96, 64),      # part of the head
    (7, 5, 80, 74),       # no 16-byte pieces
    (5, 3, 9, 6),         # odd head size
    (2, 1, 2, 2),
    (4, 2, 64, 0),        # nothing turned: a copy
    (2, 7, 1024, 1024),   # the largest head
    (2501, 6, 64, 64),    # several tokens per block, the last block not full
    (2401, 3, 10, 4),
])
def test_rope_against_definition(T, H, D, R, dtype, layout):
    x, pos, f = make(T + D, T, H, D, R, dtype, start=900000)
    for inverse in (False, True):
        check(bi.bi_rope(x, pos, f, layout, 1.25, inverse), x, pos, f, layout, 1.25, inverse)


def test_rope_extreme_positions():
    x, _, f = make(3, 8, 4, 128, 128, torch.float32)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 16777217, -1048577, 131071], dtype=torch.int32, device=DEV)
    y = bi.bi_rope(x, pos, f)
    # At 2^31 positions the fp64 product itself is off by 2^31 * 2^-53 turns of its own rounding (2^-22 radians or
    # less), in the definition and in the kernel: twice that on top of the bound.
    want, mag = definition(x, pos, f, "half", 1.0, False)
    bound = mag * (2.0 ** -21 + 2.0 ** -19) + 2.0 ** -24 * want.abs()
    assert bool(((y.double() - want).abs() <= bound).all())
    assert same_bits(y[:1], x[:1])  # position 0 turns nothing


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_strides_in_place_and_alignment_give_the_same_bits(dtype, layout):
    T, H, D, R = 600, 5, 64, 48
    x, pos, f = make(11, T, H, D, R, dtype)
    want = bi.bi_rope(x, pos, f, layout)
    wide = torch.zeros(T, 3 * H * D, dtype=dtype, device=DEV)
    view = wide[:, H * D:2 * H * D].view(T, H, D)
    view.copy_(x)
    guard = wide.clone()
    assert bi.bi_rope(view, pos, f, layout, out=view) is view
    assert same_bits(view.contiguous(), want)
    guard[:, H * D:2 * H * D] = wide[:, H * D:2 * H * D]
    assert same_bits(wide, guard)  # nothing outside the view was written
    off = torch.zeros(T * H * D + 1, dtype=dtype, device=DEV)[1:].view(T, H, D)  # no 16-byte alignment
    off.copy_(x)
    assert same_bits(bi.bi_rope(off, pos, f, layout), want)
    swapped = x.transpose(0, 1).contiguous().transpose(0, 1)  # head first
    assert same_bits(bi.bi_rope(swapped, pos, f, layout, out=torch.empty_like(swapped)).contiguous(), want)
    same = x[:, :1].expand(T, H, D)  # one head for all: stride 0
    assert same_bits(bi.bi_rope(same, pos, f, layout)[:, 3].contiguous(), want[:, 0].contiguous())


def test_rope_rows_do_not_depend_on_the_batch():
    x, pos, f = make(17, 3000, 8, 128, 128, torch.bfloat16)
    y = bi.bi_rope(x, pos, f)
    for i in (0, 1, 1234, 2999):
        assert same_bits(bi.bi_rope(x[i:i + 1], pos[i:i + 1], f), y[i:i + 1])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_inverse_is_the_gradient(layout):
    """<g, f(x + u) - f(x)> = <f^T(g), u>: the map is linear, so the difference quotient is its derivative."""
    T, H, D, R = 9, 3, 40, 32
    x, pos, f = make(23, T, H, D, R, torch.float32, start=77)
    u, _, _ = make(24, T, H, D, R, torch.float32)
    g, _, _ = make(25, T, H, D, R, torch.float32)
    dx = bi.bi_rope(g, pos, f, layout, 0.8, True)
    left = (g.double() * (bi.bi_rope(x + u, pos, f, layout, 0.8).double() - bi.bi_rope(x, pos, f, layout, 0.8).double())).sum()
    right = (dx.double() * u.double()).sum()
    # Each side sums T H D products of values up to about 4, each off by 2^-20 of them.
    assert abs(float(left - right)) <= T * H * D * 16 * 2.0 ** -20


def test_rope_empty_calls_streams_and_graphs():
    x, pos, f = make(29, 6, 2, 64, 64, torch.bfloat16)
    assert bi.bi_rope(x[:0], pos[:0], f).shape == (0, 2, 64)
    want = bi.bi_rope(x, pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(x)
    bi.bi_rope(x, pos, f, out=out, stream=side)
    side.synchronize()
    assert same_bits(out, want)
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(graph):
        bi.bi_rope(x, pos, f, out=out)
    x2 = torch.randn_like(x)
    want2 = bi.bi_rope(x2, pos, f)
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert same_bits(out, want2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D", [(1, 1, 1), (5, 3, 64), (7, 2, 10), (2400, 7, 80), (2401, 3, 9)])
def test_rope_nothing_turned_needs_no_positions(T, H, D, dtype):
    """R = 0 through the C entry with positions and inv_freq NULL: a copy, streamed or not."""
    x, _, _ = make(37, T, H, D, 0, dtype)
    y = torch.full_like(x, 7.0)
    s = torch.cuda.current_stream().cuda_stream
    for out in (y, x):  # in place nothing moves
        assert bi.load().bi_rope(x.data_ptr(), H * D, D, out.data_ptr(), H * D, D, bi._DT[dtype], None, None, T, H, D, 0, 0,
                                 1.0, 0, s) == bi.BI_OK
        assert same_bits(y, x)


def test_rope_binding_refusals():
    x, pos, f = make(31, 4, 2, 8, 8, torch.bfloat16)
    for bad in (lambda: bi.bi_rope(x.half(), pos, f), lambda: bi.bi_rope(x, pos.long(), f),
                lambda: bi.bi_rope(x, pos, f.float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: bi.bi_rope(x.view(4, 16), pos, f), lambda: bi.bi_rope(x, pos[:3], f),
                lambda: bi.bi_rope(x, pos, f, "spiral"), lambda: bi.bi_rope(x.transpose(1, 2), pos, f),
                lambda: bi.bi_rope(x, pos, f, out=torch.empty(4, 2, 4, dtype=x.dtype, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(bi.BiError):
        bi.bi_rope(x[..., :4], pos, f)  # R = 8 > D = 4


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D,R", [
    (2369, 75, 64, 64),     # more steps a warp than it has on its way at once, the last not full
    (1300, 61, 128, 96),    # two warps a token, some units turned and some copied
    (2400, 9, 200, 176),    # an odd number of copied pieces
    (2400, 5, 100, 96),     # the same in fp32
    (2400, 3, 1024, 1024),  # heads of more than 32 units
    (1200, 3, 1024, 16),
    (2400, 7, 80, 0),       # nothing turned
])
def test_rope_streamed_walks(T, H, D, R, dtype, layout):
    x, pos, f = make(T + H, T, H, D, R, dtype, start=5000)
    y = bi.bi_rope(x, pos, f, layout, 0.75)
    check(y, x, pos, f, layout, 0.75, False)
    some = torch.tensor([0, 1, T // 2, T - 1], device=DEV)
    assert same_bits(bi.bi_rope(x[some], pos[some], f, layout, 0.75), y[some])  # few tokens: other walks, the same bits
    z = x.clone()
    assert same_bits(bi.bi_rope(z, pos, f, layout, 0.75, out=z), y)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D,R", [(1, 32, 80, 20), (2400, 29, 80, 20), (2400, 13, 192, 74), (1203, 5, 512, 510),
                                     (77, 1, 24, 22), (2, 48, 256, 2), (9, 3, 1024, 1022)])
def test_rope_pairs_that_fill_no_pieces(T, H, D, R, dtype, layout):
    x, pos, f = make(T + D + R, T, H, D, R, dtype, start=70000)
    y = bi.bi_rope(x, pos, f, layout, 1.1, True)
    check(y, x, pos, f, layout, 1.1, True)
    off = torch.empty(T * H * D + 1, dtype=dtype, device=DEV)[1:].view(T, H, D)  # no 16-byte alignment
    off.copy_(x)
    assert same_bits(bi.bi_rope(off, pos, f, layout, 1.1, True), y)
    wide = torch.full((T, H, D + 16), 3.0, dtype=dtype, device=DEV)
    wide[..., :D] = x
    bi.bi_rope(wide[..., :D], pos, f, layout, 1.1, True, out=wide[..., :D])
    assert same_bits(wide[..., :D].contiguous(), y) and bool((wide[..., D:] == 3.0).all())


def test_rope_inverse_without_a_truth_value():
    """`inverse` that has no truth value raises its own error and turns nothing."""
    x, pos, f = make(41, 4, 2, 8, 8, torch.bfloat16)
    out = torch.full_like(x, 7.0)
    with pytest.raises(RuntimeError, match="ambiguous"):
        bi.bi_rope(x, pos, f, inverse=torch.ones(2, dtype=torch.bool), out=out)
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
    assert same_bits(bi.bi_rope(x, pos, f, inverse=torch.tensor(True)), bi.bi_rope(x, pos, f, inverse=True))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,D,R", [(32, 80, 20), (9, 192, 74), (3, 96, 36), (5, 64, 6), (4, 256, 250), (2, 192, 132)])
def test_rope_staged_or_walked_gives_the_same_bits(H, D, R, dtype, layout):
    """At every number of tokens where the choice, the warps that share a token or the blocks' spreading change: between two
    tensors, in place, and without 16-byte alignment."""
    for T in (1, 147, 148, 300, 700, 1800, 2048, 2300, 3600, 4300, 5000, 5400):
        x, pos, f = make(T + D + R, T, H, D, R, dtype, start=300)
        y = bi.bi_rope(x, pos, f, layout, 0.9)
        check(y[-3:], x[-3:], pos[-3:], f, layout, 0.9, False)
        off = torch.empty(T * H * D + 1, dtype=dtype, device=DEV)[1:].view(T, H, D)
        off.copy_(x)
        assert same_bits(bi.bi_rope(off, pos, f, layout, 0.9), y), T
        assert bi.bi_rope(x, pos, f, layout, 0.9, out=x) is x
        assert same_bits(x, y), T


@pytest.mark.parametrize("H", [1, 40])
@pytest.mark.parametrize("T", [300, 60000])
def test_rope_sines_and_cosines_to_an_ulp_and_a_half(T, H):
    """Pairs (1, 0) and (0, 1) give the cosines and sines themselves: sincospif is within one unit of the last place (2^-24
    below 1), what the angle's rounding to fp32 leaves out (up to 1.3 units) is put back with one rounding of half a
    unit, and its square is below 2^-46."""
    f = torch.tensor([1.0, 0.7310585786300049, 0.25, 0.0123456789, 1e-5, 3.0e-7, 0.5, 0.9], dtype=torch.float64, device=DEV)
    pos = (torch.arange(T, device=DEV) * 7 - 300000).to(torch.int32)
    angle = pos.double()[:, None] * f
    for first in (True, False):
        x = torch.zeros(T, H, 16, device=DEV)
        x[..., :8 if first else 16] = 1.0
        if not first:
            x[..., :8] = 0.0
        y = bi.bi_rope(x, pos, f).double()
        for got, want in ((y[..., :8], angle.cos() if first else -angle.sin()), (y[..., 8:], angle.sin() if first else angle.cos())):
            assert float((got - want[:, None]).abs().max()) <= 1.5 * 2.0 ** -24 + 2.0 ** -34
