"""bi_paged_append and bi_paged_decode_attention: against their definitions in fp64, batch and page
invariance, and what the documentation allows at the edges (empty places, bad pages, strides, streams, graphs).

Attention tolerance: with p the weights, A = sum_t p_t |v_t| and s_max = max_t scale sum_d |q_d k_d|,
  |out - ref| <= 2^-8 |ref| + A (2 (D + 4) 2^-24 s_max + 2^-16 + (2 n_t) 2^-24):
a score's D fp32 products and its scaling are off by (D + 4) 2^-24 of s_max and enter numerator and denominator; the weights
are two bf16 terms (2^-17 of each, numerator against the denominator's fp32 ones) through ex2 (2^-22); sums run over 32
tokens, up to 16 tiles and the splits (n_t = 64 + splits terms in a chain, in both); then one rounding to bf16.
"""
import pytest
import torch

from bi_testutil import same_bits
from invariant_bi_matmul_02_b200 import binding as bi
from test_rope_gpu import definition as rope_definition

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make_cache(g, pages, page, heads, D, order="nhd"):
    """Caches [pages, page, heads, D] as views of several memory layouts."""
    def one(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)
    if order == "nhd":
        return one(pages, page, heads, D), one(pages, page, heads, D)
    if order == "hnd":
        return one(pages, heads, page, D).transpose(1, 2), one(pages, heads, page, D).transpose(1, 2)
    if order == "kv":  # keys beside values in one buffer
        both = one(pages, 2, page, heads, D)
        return both[:, 0], both[:, 1]
    if order == "head_major":  # every head's pages together
        return one(heads, pages, page, D).permute(1, 2, 0, 3), one(heads, pages, page, D).permute(1, 2, 0, 3)
    raise AssertionError(order)


def make_table(g, lens, page, pages, width=None):
    need = [-(-n // page) for n in lens]
    width = max(max(need), 1) if width is None else width
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).tolist()
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
    return table.to(DEV)


def attend_definition(q, kc, vc, table, lens, scale):
    """(reference, bound) in fp64."""
    B, Hq, D = q.shape
    page, Hkv = kc.shape[1], kc.shape[2]
    ref = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(ref)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        at = table[b, :-(-n // page)].long()
        k = kc[at].reshape(-1, Hkv, D)[:n].double()
        v = vc[at].reshape(-1, Hkv, D)[:n].double()
        qq = q[b].double().view(Hkv, Hq // Hkv, D)
        p = torch.softmax(scale * torch.einsum("hgd,lhd->hgl", qq, k), -1)
        smax = scale * torch.einsum("hgd,lhd->hgl", qq.abs(), k.abs()).amax(-1)
        ref[b] = torch.einsum("hgl,lhd->hgd", p, v).reshape(Hq, D)
        mag = torch.einsum("hgl,lhd->hgd", p, v.abs())
        c = 2 * (D + 4) * 2.0 ** -24 * smax + 2.0 ** -16 + 2 * (64 + -(-n // 256)) * 2.0 ** -24
        bound[b] = (mag * c[..., None]).reshape(Hq, D)
    return ref, bound + 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8)


def run_attend(seed, lens, Hq, Hkv, D, page, order="nhd", width=None, spare=2):
    g = gen(seed)
    pages = sum(-(-n // page) for n in lens) + spare
    kc, vc = make_cache(g, pages, page, Hkv, D, order)
    table = make_table(g, lens, page, pages, width)
    q = torch.randn(len(lens), Hq, D, generator=g, device=DEV).to(torch.bfloat16)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    return q, kc, vc, table, sl


def close(o, ref, bound):
    err = (o.double() - ref).abs()
    assert bool((err <= bound).all()), float((err - bound).max())


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("page", [16, 1, 2, 5, 8, 24, 32, 48, 64, 256])
def test_attention_page_sizes(page, D):
    lens = [1, 31, 32, 33, 255, 256, 257, 0, 700, 511, 512, 513, 768]
    q, kc, vc, table, sl = run_attend(100 + page, lens, 8, 2, D, page)
    o = bi.bi_paged_decode_attention(q, kc, vc, table, sl)
    close(o, *attend_definition(q, kc, vc, table, lens, D ** -0.5))
    assert bool((o[7] == 0).all())
    assert bi.bi_get_device_status() == bi.BI_OK


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (6, 2), (5, 1), (28, 4), (8, 1), (9, 1), (32, 2), (13, 1)])
def test_attention_groups(Hq, Hkv, D):
    lens = [300, 1, 64, 513]
    q, kc, vc, table, sl = run_attend(7 * Hq + Hkv, lens, Hq, Hkv, D, 16)
    close(bi.bi_paged_decode_attention(q, kc, vc, table, sl), *attend_definition(q, kc, vc, table, lens, D ** -0.5))


@pytest.mark.parametrize("order", ["nhd", "hnd", "kv", "head_major"])
@pytest.mark.parametrize("page", [16, 24])
def test_attention_layouts_give_the_same_bits(order, page):
    lens = [513, 40, 0, 1000]
    q, kc, vc, table, sl = run_attend(55, lens, 8, 4, 128, page)
    want = bi.bi_paged_decode_attention(q, kc, vc, table, sl)
    k2, v2 = make_cache(gen(1), kc.shape[0], page, 4, 128, order)
    k2.copy_(kc)
    v2.copy_(vc)
    assert same_bits(bi.bi_paged_decode_attention(q, k2, v2, table, sl), want)
    wide = torch.zeros(4, 24, 128, dtype=torch.bfloat16, device=DEV)
    wide[:, 8:16] = q  # rows of a wider projection
    assert same_bits(bi.bi_paged_decode_attention(wide[:, 8:16], k2, v2, table, sl), want)


def test_attention_does_not_depend_on_batch_pages_or_max_len():
    lens = [5000, 256, 257, 1, 0, 3000, 2048, 130]
    q, kc, vc, table, sl = run_attend(77, lens, 16, 4, 128, 16, width=400)
    want = bi.bi_paged_decode_attention(q, kc, vc, table, sl)
    close(want, *attend_definition(q, kc, vc, table, lens, 128 ** -0.5))
    for i, n in enumerate(lens):
        alone = bi.bi_paged_decode_attention(q[i:i + 1], kc, vc, table[i:i + 1], sl[i:i + 1], max_len=max(n, 1))
        assert same_bits(alone, want[i:i + 1]), f"sequence {i}"
    idx = torch.randperm(8, generator=gen(5), device=DEV)
    assert same_bits(bi.bi_paged_decode_attention(q[idx], kc, vc, table[idx].contiguous(), sl[idx], max_len=5000), want[idx])
    for _ in range(20):
        assert same_bits(bi.bi_paged_decode_attention(q, kc, vc, table, sl, max_len=6400), want)
    # The same tokens in pages of 40, somewhere else.
    pages = sum(-(-n // 40) for n in lens) + 3
    k2, v2 = make_cache(gen(78), pages, 40, 4, 128)
    t2 = make_table(gen(79), lens, 40, pages)
    for b, n in enumerate(lens):
        for p in range(-(-n // 40)):
            rows = torch.arange(40 * p, min(40 * p + 40, n), device=DEV)
            src = table[b].long()[rows // 16]
            k2[t2[b, p].long(), : len(rows)] = kc[src, rows % 16]
            v2[t2[b, p].long(), : len(rows)] = vc[src, rows % 16]
    assert same_bits(bi.bi_paged_decode_attention(q, k2, v2, t2, sl), want)


@pytest.mark.parametrize("D", [128, 64])
def test_attention_long_sequence_and_many_splits(D):
    """More than 32 splits are folded by groups, up to 32 in order, whichever the longest of the call asks for."""
    lens = [70001, 300, 8192, 8193, 0, 600]
    q, kc, vc, table, sl = run_attend(91, lens, 4, 1, D, 64)
    o = bi.bi_paged_decode_attention(q, kc, vc, table, sl)
    close(o, *attend_definition(q, kc, vc, table, lens, D ** -0.5))
    for i in (1, 2, 3, 5):
        assert same_bits(bi.bi_paged_decode_attention(q[i:i + 1], kc, vc, table[i:i + 1], sl[i:i + 1], max_len=lens[i]), o[i:i + 1])


def test_attention_more_sequences_than_one_launch_takes():
    lens = [1 + (i * 37) % 300 for i in range(2098)] + [700, 1300]
    q, kc, vc, table, sl = run_attend(92, lens, 2, 1, 64, 16)
    o = bi.bi_paged_decode_attention(q, kc, vc, table, sl)
    close(o, *attend_definition(q, kc, vc, table, lens, 0.125))
    for i in (0, 2047, 2048, 2099):
        assert same_bits(bi.bi_paged_decode_attention(q[i:i + 1], kc, vc, table[i:i + 1], sl[i:i + 1], max_len=int(sl[i])), o[i:i + 1])


@pytest.mark.parametrize("page,Hkv", [(1, 1), (64, 1), (64, 3), (1, 2), (7, 1)])
def test_one_page_caches(page, Hkv):
    """A cache of one page, and pages or heads of one entry: strides that are never stepped over may be anything."""
    g = gen(page + Hkv)
    kc, vc = make_cache(g, 1, page, Hkv, 64)
    odd = [1 if n == 1 else s for n, s in zip(kc.shape, kc.stride())]
    kc, vc = kc.as_strided(kc.shape, odd), vc.as_strided(vc.shape, odd)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    sl = torch.tensor([page], dtype=torch.int32, device=DEV)
    k, v = (torch.randn(1, Hkv, 64, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(1, 2 * Hkv, 64, generator=g, device=DEV).to(torch.bfloat16)
    bi.bi_paged_append(k, v, kc, vc, table, sl)
    assert same_bits(kc[0, -1], k[0]) and same_bits(vc[0, -1], v[0])
    close(bi.bi_paged_decode_attention(q, kc, vc, table, sl), *attend_definition(q, kc, vc, table, [page], 0.125))
    empty = bi.bi_paged_decode_attention(q[:0], kc, vc, table[:0, :0], sl[:0])
    assert empty.shape == (0, 2 * Hkv, 64)
    assert bi.bi_get_device_status() == bi.BI_OK


def test_attention_offsets_beyond_32_bits():
    """A cache of more than 2^32 elements: pages at its far end are read and written where they are."""
    page, Hkv, D = 64, 8, 128
    pages = 2 ** 32 // (page * Hkv * D) + 8
    kc = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    g = gen(93)
    table = torch.tensor([[pages - 1, 0, pages - 5]], dtype=torch.int32, device=DEV)
    lens = [150]
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    k = torch.randn(150, Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
    v = torch.randn(150, Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
    cu = torch.tensor([0, 150], dtype=torch.int32, device=DEV)
    bi.bi_paged_append(k, v, kc, vc, table, sl, cu_new=cu)
    assert same_bits(kc[pages - 1], k[:64]) and same_bits(vc[pages - 5, :22], v[128:])
    q = torch.randn(1, 8, D, generator=g, device=DEV).to(torch.bfloat16)
    close(bi.bi_paged_decode_attention(q, kc, vc, table, sl), *attend_definition(q, kc, vc, table, lens, D ** -0.5))
    assert bi.bi_get_device_status() == bi.BI_OK


def test_attention_ignores_what_lies_past_a_sequence():
    """Rows past a sequence's end, in its last page, hold NaN: nothing of them reaches the output."""
    lens = [5, 33, 300, 256]
    q, kc, vc, table, sl = run_attend(94, lens, 8, 2, 128, 16)
    want = bi.bi_paged_decode_attention(q, kc, vc, table, sl)
    for b, n in enumerate(lens):
        if n % 16:
            kc[table[b, n // 16].long(), n % 16:] = float("nan")
            vc[table[b, n // 16].long(), n % 16:] = float("inf")
    assert same_bits(bi.bi_paged_decode_attention(q, kc, vc, table, sl), want)


def test_attention_large_scores_and_equal_scores():
    lens = [777, 40]
    q, kc, vc, table, sl = run_attend(95, lens, 4, 2, 128, 16)
    q2 = q * 60  # weights of one or two tokens
    close(bi.bi_paged_decode_attention(q2, kc, vc, table, sl), *attend_definition(q2, kc, vc, table, lens, 128 ** -0.5))
    zero = torch.zeros_like(q)  # all weights equal
    close(bi.bi_paged_decode_attention(zero, kc, vc, table, sl), *attend_definition(zero, kc, vc, table, lens, 128 ** -0.5))


def test_attention_bad_lengths_and_pages_are_recorded():
    lens = [100, 64]
    q, kc, vc, table, sl = run_attend(96, lens, 4, 2, 128, 16)
    want = bi.bi_paged_decode_attention(q, kc, vc, table, sl)
    assert bi.bi_get_device_status() == bi.BI_OK
    o = bi.bi_paged_decode_attention(q, kc, vc, table, torch.tensor([100, -3], dtype=torch.int32, device=DEV))
    assert bi.bi_get_device_status() == bi.BI_ERR_INVALID_ARG
    assert same_bits(o[:1], want[:1]) and bool((o[1] == 0).all())
    o = bi.bi_paged_decode_attention(q, kc, vc, table, torch.tensor([100, 9999], dtype=torch.int32, device=DEV), max_len=100)
    assert bi.bi_get_device_status() == bi.BI_ERR_INVALID_ARG
    assert same_bits(o[:1], want[:1])
    for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 2] = bad
        o = bi.bi_paged_decode_attention(q, kc, vc, t, sl)
        assert bi.bi_get_device_status() == bi.BI_ERR_INVALID_ARG
        assert same_bits(o[1:], want[1:])
        # Its tokens count with keys and values of zero.
        k0, v0 = torch.cat([kc, torch.zeros_like(kc[:1])]), torch.cat([vc, torch.zeros_like(vc[:1])])
        t[0, 2] = kc.shape[0]
        assert same_bits(o[:1], bi.bi_paged_decode_attention(q, k0, v0, t, sl)[:1])
    assert bi.bi_get_device_status() == bi.BI_OK


def test_attention_streams_graphs_and_scratch():
    lens = [600, 300, 1]
    q, kc, vc, table, sl = run_attend(97, lens, 8, 2, 64, 16)
    want = bi.bi_paged_decode_attention(q, kc, vc, table, sl)
    B, Hq, D = q.shape
    max_len = table.shape[1] * 16
    need = bi.bi_paged_decode_attention_scratch_bytes(B, Hq, D, max_len)
    scratch = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full_like(q, float("nan"))
    assert bi.bi_paged_decode_attention(q, kc, vc, table, sl, scratch=scratch[:need], out=out) is out
    assert same_bits(out, want) and bool((scratch[need:] == 0xFF).all())
    with pytest.raises(bi.BiError):
        bi.bi_paged_decode_attention(q, kc, vc, table, sl, scratch=scratch[:need - 16])
    # On another stream without scratch: the allocation made for the call outlives its work there.
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    made = [bi.bi_paged_decode_attention(q, kc, vc, table, sl, stream=side) for _ in range(20)]
    side.synchronize()
    assert all(same_bits(o, want) for o in made)
    # Two calls at once on two streams, each with its own scratch.
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.empty_like(q) for _ in range(8)]
    scr = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in range(2)]
    for i in range(8):
        bi.bi_paged_decode_attention(q, kc, vc, table, sl, scratch=scr[i % 2], out=outs[i], stream=(s1, s2)[i % 2])
    torch.cuda.synchronize()
    assert all(same_bits(o, want) for o in outs)
    # Captured and replayed with another length in place.
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bi.bi_paged_decode_attention(q, kc, vc, table, sl, scratch=scr[0], out=out)
    sl.copy_(torch.tensor([17, 0, 1], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert same_bits(out, bi.bi_paged_decode_attention(q, kc, vc, table, sl))
    assert bool((out[1] == 0).all())


# ------------------------------------------------------------------------------------------- append

def append_definition(k, v, kc, vc, table, lens, cu, f, layout, scale, q, positions, q_out):
    kc, vc = kc.clone(), vc.clone()
    page = kc.shape[1]
    where, place = [], []
    for b, n in enumerate(lens):
        for t in range(cu[b], cu[b + 1]):
            if n:
                where.append((b, t))
                place.append(n - (cu[b + 1] - t))
    if not where:
        return kc, vc, q_out, None, None
    b = torch.tensor([w[0] for w in where], device=DEV)
    t = torch.tensor([w[1] for w in where], device=DEV)
    p = torch.tensor(place, device=DEV)
    pos = p if positions is None else positions[t].long()
    rk, mk = (k[t].double(), None) if f is None else rope_definition(k[t], pos, f, layout, scale, False)
    at = table.long()[b, p // page]
    return (kc, vc, at, p % page, t, rk, mk, pos)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("order", ["nhd", "hnd", "kv", "head_major"])
@pytest.mark.parametrize("Hq,Hkv,D,R,page", [(32, 8, 128, 128, 16), (6, 3, 64, 32, 5), (3, 1, 96, 90, 24), (2, 2, 24, 0, 1),
                                             (4, 2, 256, 256, 64)])
@pytest.mark.parametrize("decode", [True, False])
def test_append_against_definition(Hq, Hkv, D, R, page, order, layout, decode):
    g = gen(D + R + page)
    lens = [70, 1, 0, 33, 129] if decode else [70, 5, 300, 64, 0, 9]
    new = [1] * 5 if decode else [70, 2, 41, 1, 0, 9]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    pages = sum(-(-n // page) for n in lens) + 2
    kc, vc = make_cache(g, pages, page, Hkv, D, order)
    table = make_table(g, lens, page, pages, width=-(-400 // page))
    behind = 0 if decode else 4  # tokens behind the last sequence
    T = cu[-1] + behind
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = (qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),
               qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D))
    f = bi.bi_rope_freqs(R, 1e4)[0] if R else None
    scale = 1.1 if R else 1.0
    before_k, before_v = kc.clone(), vc.clone()
    q_out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got_q = bi.bi_paged_append(k, v, kc, vc, table, sl, None if decode else torch.tensor(cu, dtype=torch.int32, device=DEV),
                               f, layout, scale, q, q_out)
    assert got_q is q_out
    wk, wv, at, row, t, rk, mk, pos = append_definition(k, v, before_k, before_v, table, lens, cu, f, layout, scale, q, None, None)
    wv[at, row] = v[t]
    assert same_bits(vc.contiguous(), wv.contiguous())
    got_k = kc[at, row]
    if R == 0:
        wk[at, row] = k[t]
        assert same_bits(kc.contiguous(), wk.contiguous())
        assert same_bits(q_out[t], q[t])
    else:
        close(got_k, rk, mk * 2.0 ** -21 + 2.0 ** -8 * rk.abs() * (1 + 2.0 ** -20))
        wk[at, row] = got_k  # elsewhere the cache is as it was
        assert same_bits(kc.contiguous(), wk.contiguous())
        rq, mq = rope_definition(q[t], pos, f, layout, scale, False)
        close(q_out[t], rq, mq * 2.0 ** -21 + 2.0 ** -8 * rq.abs() * (1 + 2.0 ** -20))
        # The same bits as bi_rope's.
        assert same_bits(got_k, bi.bi_rope(k[t], pos.to(torch.int32), f, layout, scale))
    live = torch.zeros(T, dtype=torch.bool, device=DEV)
    live[t] = True
    assert bool((q_out[~live] == 7.0).all())  # skipped tokens' rows are as they were
    assert bi.bi_get_device_status() == bi.BI_OK


def test_append_many_tokens_positions_in_place_and_unaligned_give_the_same_bits():
    g = gen(3)
    Hq, Hkv, D, page = 4, 2, 64, 16
    lens = [3000, 500]
    cu = torch.tensor([0, 2700, 3100], dtype=torch.int32, device=DEV)
    T, pages = 3100, 230
    kc, vc = make_cache(g, pages, page, Hkv, D)
    table = make_table(g, lens, page, pages)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    k, v = (torch.randn(T, Hkv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(T, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
    f = bi.bi_rope_freqs(D, 1e6)[0]
    want_q = bi.bi_paged_append(k, v, kc, vc, table, sl, cu, f, q=q)
    place = torch.cat([torch.arange(300, 3000), torch.arange(100, 500)]).to(DEV)
    seq = torch.cat([torch.zeros(2700), torch.ones(400)]).to(DEV).long()
    at = table.long()[seq, place // page]
    assert same_bits(kc[at, place % page], bi.bi_rope(k, place.to(torch.int32), f))
    assert same_bits(vc[at, place % page], v)
    assert same_bits(want_q, bi.bi_rope(q, place.to(torch.int32), f))
    k2, v2 = make_cache(gen(4), pages, page, Hkv, D)
    pos = (place * 3 - 1000).to(torch.int32)
    q2 = q.clone()
    assert bi.bi_paged_append(k, v, k2, v2, table, sl, cu, f, q=q2, q_out=q2, positions=pos) is q2
    assert same_bits(q2, bi.bi_rope(q, pos, f))
    assert same_bits(k2[at, place % page], bi.bi_rope(k, pos, f))
    off = torch.zeros(T * Hkv * D + 1, dtype=torch.bfloat16, device=DEV)[1:].view(T, Hkv, D)  # no 16-byte pieces
    off.copy_(k)
    k3, v3 = make_cache(gen(4), pages, page, Hkv, D)
    assert bi.bi_paged_append(off, v, k3, v3, table, sl, cu, f) is None
    assert same_bits(k3[at, place % page], kc[at, place % page])


def test_append_refuses_bad_places_on_the_device():
    g = gen(5)
    kc, vc = make_cache(g, 4, 16, 2, 64)
    k, v = (torch.randn(4, 2, 64, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    good = torch.tensor([[0], [1], [2], [3]], dtype=torch.int32, device=DEV)
    ones = torch.full((4,), 5, dtype=torch.int32, device=DEV)
    for lens, table, cu in [
        ([5, 5, 17, 5], None, None),                       # past the table
        ([5, -5, 5, 5], None, None),                       # a negative length
        ([5, 5, 5, 5], [[0], [1], [4], [3]], None),        # a page past the cache
        ([5, 5, 5, 5], [[0], [-1], [2], [3]], None),       # no page
        ([5, 5, 5, 2 ** 31 - 1], None, None),
        ([5, 1, 5, 5], None, [0, 1, 3, 4, 4]),             # two new tokens of a sequence of one
    ]:
        k1, v1 = kc.clone(), vc.clone()
        t = good if table is None else torch.tensor(table, dtype=torch.int32, device=DEV)
        c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
        bi.bi_paged_append(k, v, k1, v1, t, torch.tensor(lens, dtype=torch.int32, device=DEV), c)
        assert bi.bi_get_device_status() == bi.BI_ERR_INVALID_ARG, (lens, table)
        assert same_bits(k1[0, 4:5], k[0:1])  # the good tokens are in place
        keep = torch.ones(4, 16, dtype=torch.bool, device=DEV)
        keep[:, 0] = keep[:, 4] = False
        assert same_bits(k1[keep], kc[keep]) and same_bits(v1[keep], vc[keep])
    for cu in ([0, 0, 0, 0, 0], [4, 4, 4, 4, 4], [3, 1, 2, 0, 4], [-5, -4, -3, -2, -1]):
        # Whatever the boundaries say, nothing is written outside the sequences' own places.
        k1, v1 = kc.clone(), vc.clone()
        bi.bi_paged_append(k, v, k1, v1, good, ones, torch.tensor(cu, dtype=torch.int32, device=DEV))
        bi.bi_get_device_status()
        assert same_bits(k1[:, 5:], kc[:, 5:])
    bi.bi_paged_append(k, v, kc, vc, good, torch.zeros(4, dtype=torch.int32, device=DEV))
    assert bi.bi_get_device_status() == bi.BI_OK


def test_binding_refusals():
    g = gen(6)
    kc, vc = make_cache(g, 4, 16, 2, 64)
    k = torch.randn(3, 2, 64, generator=g, device=DEV).to(torch.bfloat16)
    t = torch.zeros(3, 1, dtype=torch.int32, device=DEV)
    n = torch.ones(3, dtype=torch.int32, device=DEV)
    for bad in (lambda: bi.bi_paged_append(k, k[:2], kc, vc, t, n), lambda: bi.bi_paged_append(k, k, kc, vc[:, :8], t, n),
                lambda: bi.bi_paged_append(k, k, kc, vc, t[:2], n), lambda: bi.bi_paged_append(k[:2], k[:2], kc, vc, t, n),
                lambda: bi.bi_paged_append(k, k, kc, vc, t, n, q_out=k), lambda: bi.bi_paged_append(k, k, kc, vc, t, n, n),
                lambda: bi.bi_paged_decode_attention(k[:, :, :32], kc, vc, t, n),
                lambda: bi.bi_paged_decode_attention(k, kc, vc, t, n[:2]),
                lambda: bi.bi_paged_decode_attention(k, kc, vc, t, n, out=torch.empty_like(k[:2])),
                lambda: bi.bi_paged_decode_attention(k.transpose(0, 1).contiguous().transpose(0, 1), kc, vc, t, n)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        bi.bi_paged_decode_attention(k, kc, vc, t.long(), n)
    with pytest.raises(bi.BiError):
        bi.bi_paged_decode_attention(k, kc, vc, t, n, max_len=17)


def test_a_prefill_and_decode_steps_together():
    """The operators as they are used: prompts enter the cache in one call, then each step turns and appends one token
    and attends over what is there; each step's output equals a dense computation over the tokens so far, and a
    sequence generated alone gives the same bits as in the batch."""
    g = gen(8)
    Hq, Hkv, D, page, steps = 8, 2, 64, 16, 5
    prompts = [40, 1, 17, 255]
    B, width = len(prompts), 17
    f, scale = bi.bi_rope_freqs(D, 1e6, "yarn", factor=4.0, original_length=64.0)
    total = [n + steps for n in prompts]
    data = {b: [torch.randn(total[b], h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)] for b in range(B)}

    def generate(seqs, seed):
        kc, vc = make_cache(gen(seed), 80, page, Hkv, D)
        table = make_table(gen(seed + 1), [total[b] for b in seqs], page, 80, width)
        cu = torch.tensor([0] + [prompts[b] for b in seqs], device=DEV).cumsum(0).to(torch.int32)
        sl = torch.tensor([prompts[b] for b in seqs], dtype=torch.int32, device=DEV)
        cat = lambda i: torch.cat([data[b][i][:prompts[b]] for b in seqs])  # noqa: E731
        bi.bi_paged_append(cat(1), cat(2), kc, vc, table, sl, cu, f, scale=scale)
        outs = []
        for s in range(steps):
            at = [prompts[b] + s for b in seqs]
            q, k, v = (torch.stack([data[b][i][n] for b, n in zip(seqs, at)]) for i in range(3))
            sl += 1
            q = bi.bi_paged_append(k, v, kc, vc, table, sl, inv_freq=f, scale=scale, q=q)
            outs.append(bi.bi_paged_decode_attention(q, kc, vc, table, sl))
        return torch.stack(outs, 1), q, kc, vc, table, sl

    outs, q, kc, vc, table, sl = generate(list(range(B)), 200)
    close(outs[:, -1], *attend_definition(q, kc, vc, table, sl.tolist(), D ** -0.5))
    for b in range(B):
        dense = bi.bi_rope(data[b][1], torch.arange(total[b], dtype=torch.int32, device=DEV), f, scale=scale)
        rows = torch.arange(total[b], device=DEV)
        assert same_bits(kc[table[b].long()[rows // page], rows % page], dense)
        assert same_bits(generate([b], 300 + b)[0], outs[b:b + 1])
    assert bi.bi_get_device_status() == bi.BI_OK


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("Hq,Hkv,D,R", [(24, 7, 128, 128), (20, 5, 64, 32), (0, 9, 128, 96), (9, 3, 72, 48), (5, 2, 96, 0),
                                        (3, 1, 1024, 1024)])
def test_append_long_prompts_take_one_warp_per_token(Hq, Hkv, D, R, layout):
    """A warp walks a whole token's queries, keys and values: more steps than it has on its way at once."""
    g = gen(Hq + D)
    lens, cu, page = [2000, 600, 0, 40], [0, 1990, 2590, 2590, 2600], 16
    T, pages = 2603, 200
    kc, vc = make_cache(g, pages, page, Hkv, D)
    table = make_table(g, lens, page, pages)
    sl, c = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (lens, cu))
    k, v = (torch.randn(T, Hkv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(T, Hq, D, generator=g, device=DEV).to(torch.bfloat16) if Hq else None
    f = bi.bi_rope_freqs(R, 1e5)[0] if R else None
    scale = 1.1 if R else 1.0
    before_k, before_v = kc.clone(), vc.clone()
    q_out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV) if Hq else None
    bi.bi_paged_append(k, v, kc, vc, table, sl, c, f, layout, scale, q, q_out)
    wk, wv, at, row, t, _, _, pos = append_definition(k, v, before_k, before_v, table, lens, cu, f, layout, scale, q, None, None)
    turned = lambda x: bi.bi_rope(x[t], pos.to(torch.int32), f, layout, scale) if R else x[t]
    wk[at, row], wv[at, row] = turned(k), v[t]
    assert same_bits(kc.contiguous(), wk.contiguous()) and same_bits(vc.contiguous(), wv.contiguous())
    if Hq:
        assert same_bits(q_out[t], turned(q)) and bool((q_out[2600:] == 7.0).all())
    assert bi.bi_get_device_status() == bi.BI_OK


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("Hq,Hkv,D,R", [(32, 32, 80, 20), (0, 5, 192, 74), (4, 2, 512, 510), (7, 1, 24, 22)])
def test_append_pairs_that_fill_no_pieces(Hq, Hkv, D, R, layout):
    test_append_long_prompts_take_one_warp_per_token(Hq, Hkv, D, R, layout)
    g = gen(D)  # a few tokens, values and then keys without 16-byte alignment: other walks, the same bits
    lens, page, T = [5, 0, 33, 128], 16, 4
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    k, v = (torch.randn(T, Hkv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    f = bi.bi_rope_freqs(R, 1e4)[0]
    kc, vc = make_cache(g, 14, page, Hkv, D)
    table = make_table(g, lens, page, 14)
    odd = []
    for x in (k, v):
        odd.append(torch.empty(T * Hkv * D + 1, dtype=torch.bfloat16, device=DEV)[1:].view(T, Hkv, D))
        odd[-1].copy_(x)
    want = None
    for a, b in ((k, v), (k, odd[1]), (odd[0], v)):
        k2, v2 = kc.clone(), vc.clone()
        bi.bi_paged_append(a, b, k2, v2, table, sl, None, f, layout)
        want = want or (k2, v2)
        assert same_bits(k2, want[0]) and same_bits(v2, want[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [8, 16])
def test_attention_weights_keep_their_24_bits(G, D):
    """Three tokens of weights 1, 1 and p in (1/2, 1), whose values -hi, -mid and 1 (hi = bf16(p), mid = bf16(p - hi)) leave
    p's last bits.  In units of 2^-24: p is off by at most 4 (score's scaling and rounding 1.4, ex2 2), the sums of a dozen
    terms below 1 by 24; over the sum of the weights, 2 + p, and with one rounding of a value below 2^-17."""
    B = 64
    s = (0.69 * torch.rand(B, G, generator=gen(17), device=DEV)).to(torch.bfloat16)
    p = torch.exp(-s.double())
    hi = p.float().to(torch.bfloat16)
    mid = (p - hi.double()).float().to(torch.bfloat16)
    kc, vc = (torch.zeros(B, 4, 1, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kc[:, 2, 0, 0] = -1.0
    vc[:, 0, 0, :G], vc[:, 1, 0, :G], vc[:, 2, 0, :G] = -hi, -mid, 1.0  # entry h for head h
    q = torch.zeros(B, G, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = s
    table = torch.arange(B, dtype=torch.int32, device=DEV).view(B, 1)
    o = bi.bi_paged_decode_attention(q, kc, vc, table, torch.full((B,), 3, dtype=torch.int32, device=DEV), scale=1.0)
    got = torch.diagonal(o[..., :G].double(), dim1=1, dim2=2)
    want = (p - hi.double() - mid.double()) / (2 + p)
    close(got, want, 28 * 2.0 ** -24 / (2 + p) + 2.0 ** -8 * want.abs())
