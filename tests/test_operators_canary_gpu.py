"""Out-of-bounds stores of the decode-step operators: every output lies in the middle of a sentinel-filled buffer, at
ragged sizes, and every sentinel byte must survive.  (The append's caches are compared whole in test_paged_gpu.py.)"""
import ctypes

import pytest
import torch

from bi_testutil import same_bits
from invariant_bi_matmul_02_b200 import binding as bi

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAD = 64  # elements on either side


class Guarded:
    """A tensor inside a sentinel-filled buffer; `rows` of `cols` with `ld` elements between rows."""

    def __init__(self, shape, dtype, ld=None):
        n = 1
        for s in shape:
            n *= s
        self.ld = ld
        size = n if ld is None else shape[0] * ld
        self.raw = torch.full((size + 2 * PAD,), 77, dtype=dtype, device=DEV)
        body = self.raw[PAD:PAD + size]
        self.t = body.view(shape) if ld is None else body.view(shape[0], ld)[:, :n // shape[0]].view(*shape)

    def check(self):
        assert bool((self.raw[:PAD] == 77).all()) and bool((self.raw[-PAD:] == 77).all())
        if self.ld is not None:
            rows = self.raw[PAD:-PAD].view(self.t.shape[0], self.ld)
            assert bool((rows[:, self.t[0].numel():] == 77).all())


@pytest.mark.parametrize("T,H,D,R", [(1, 40, 128, 128), (7, 3, 24, 20), (13, 5, 9, 6), (3001, 2, 64, 64), (5, 1, 10, 0)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_stores(T, H, D, R, layout, dtype):
    x = torch.randn(T, H, D, device=DEV).to(dtype)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    f = bi.bi_rope_freqs(R, 1e4)[0]
    for ld in (None, H * D + 24, H * D + 1):
        out = Guarded((T, H, D), dtype, ld)
        bi.bi_rope(x, pos, f, layout, out=out.t)
        out.check()
        assert same_bits(out.t.contiguous(), bi.bi_rope(x, pos, f, layout))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(3, 1), (16, 1), (6, 2)])
def test_attention_stores(Hq, Hkv, D):
    lens = [0, 1, 300, 513, 700]
    page, pages = 24, 70
    g = torch.Generator(device=DEV).manual_seed(1)
    kc, vc = (torch.randn(pages, page, Hkv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(5, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
    table = torch.randint(0, pages, (5, 30), generator=g, device=DEV).to(torch.int32)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    need = bi.bi_paged_decode_attention_scratch_bytes(5, Hq, D, 720)
    out, scratch = Guarded((5, Hq, D), torch.bfloat16), Guarded((need,), torch.uint8)
    bi.bi_paged_decode_attention(q, kc, vc, table, sl, out=out.t, scratch=scratch.t)
    out.check()
    scratch.check()
    assert same_bits(out.t, bi.bi_paged_decode_attention(q, kc, vc, table, sl))


@pytest.mark.parametrize("M,V,k", [(1, 40, 32), (3, 50257, 20), (600, 1000, 1), (2, 8193, 7)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_token_logprobs_stores_and_optional_outputs(M, V, k, dtype):
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(M, V, generator=g, device=DEV).to(dtype)
    tok = torch.randint(0, V, (M,), generator=g, device=DEV).to(torch.int32)
    want = bi.bi_token_logprobs(x, tok, k)
    f32 = [Guarded((M,), torch.float32) for _ in range(3)]
    tl, tt = Guarded((M, k), torch.float32), Guarded((M, k), torch.int32)
    lib, p = bi.load(), ctypes.c_void_p
    stream = p(torch.cuda.current_stream().cuda_stream)

    def call(lp, h, lse, top):
        return lib.bi_token_logprobs(p(x.data_ptr()), V, bi._DT[dtype], p(tok.data_ptr()) if lp else None, 1.0, k if top else 0,
                                     lp, h, lse, p(tl.t.data_ptr()) if top else None,
                                     p(tt.t.data_ptr()) if top else None, M, V, stream)

    ptrs = [p(t.t.data_ptr()) for t in f32]
    assert call(*ptrs, True) == bi.BI_OK
    for t in f32 + [tl, tt]:
        t.check()
    assert all(same_bits(a.t, b) for a, b in zip(f32 + [tl, tt], want))
    for keep in range(3):  # each output alone
        for t in f32:
            t.t.fill_(77)
        assert call(*[ptrs[i] if i == keep else None for i in range(3)], False) == bi.BI_OK
        for i, t in enumerate(f32):
            t.check()
            assert same_bits(t.t, want[i]) if i == keep else bool((t.t == 77).all())
