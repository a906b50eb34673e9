"""Memory that the library's operators make for a call on a given stream belongs to that stream, as under
torch.cuda.stream: it is neither memory that another stream's work still uses, nor reused before the call's own work."""
import pytest
import torch

from bi_testutil import same_bits
from invariant_bi_matmul_02_b200 import binding as bi

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, HQ, HKV, D, PAGE, LONGEST = 3, 8, 2, 64, 16, 960


def calls():
    """Each operator's call as a function of its stream, with outputs made by the call."""
    g = torch.Generator(device=DEV).manual_seed(4)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)

    pages = B * LONGEST // PAGE
    kc, vc, q, k, x = rand(pages, PAGE, HKV, D), rand(pages, PAGE, HKV, D), rand(B, HQ, D), rand(B, HKV, D), rand(B, 500)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(B, -1)
    lens = torch.tensor([300, 940, 17], dtype=torch.int32, device=DEV)
    pos = torch.arange(B, dtype=torch.int32, device=DEV)
    f = bi.bi_rope_freqs(D, 1e4)[0]
    return {
        "rope": lambda s: (bi.bi_rope(q, pos, f, stream=s),),
        "append": lambda s: (bi.bi_paged_append(k, k, kc, vc, table, lens, None, f, q=q, stream=s),),
        "attend": lambda s: (bi.bi_paged_decode_attention(q, kc, vc, table, lens, stream=s),),
        "logprobs": lambda s: bi.bi_token_logprobs(x, pos, 3, stream=s),
    }


def other_calls():
    """The same for the library's other operators."""
    g = torch.Generator(device=DEV).manual_seed(5)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)

    a, w, x, gain, q, kc, long = (rand(5, 64), rand(128, 64), rand(5, 128), rand(128), rand(2, 8, 64), rand(2, 600, 2, 64),
                                  rand(2, 40000))
    xf = x.float()
    lens = torch.tensor([600, 33], dtype=torch.int32, device=DEV)
    return {
        "matmul": lambda s: (bi.bi_matmul(a, w, stream=s),),
        "addmm": lambda s: (bi.bi_addmm(x, a, w, stream=s),),
        "matmul_silu_mul": lambda s: (bi.bi_matmul_silu_mul(a, w, stream=s),),
        "silu_mul": lambda s: (bi.bi_silu_mul(x, stream=s),),
        "rmsnorm": lambda s: (bi.bi_rmsnorm(x, gain, stream=s),),
        "mean": lambda s: (bi.bi_mean(xf, stream=s),),
        "log_softmax": lambda s: (bi.bi_log_softmax(x, stream=s),),
        "log_softmax_cluster": lambda s: (bi.bi_log_softmax_cluster(long, stream=s),),
        "log_softmax_split": lambda s: (bi.bi_log_softmax_split(long, stream=s),),
        "decode_attention": lambda s: (bi.bi_decode_attention(q, kc, kc, lens, stream=s),),
    }


def pool_stream(t):
    """The stream whose pool the tensor's memory is from."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


def check_outputs(call):
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = call(None)
    default = torch.cuda.default_stream()
    for s, of in ((side, side), (side.cuda_stream, side), (None, default), (0, default), (1, default)):
        got = call(s)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert same_bits(a, b)
            assert pool_stream(a) == of.cuda_stream
    with torch.cuda.stream(side):  # the current stream is another than the call's
        assert all(pool_stream(a) == default.cuda_stream for a in call(default))
        assert torch.cuda.current_stream() == side
    torch.cuda.synchronize()
    assert torch.cuda.current_stream() == default


@pytest.mark.parametrize("op", ["rope", "append", "attend", "logprobs"])
def test_outputs_are_of_the_calls_stream(op):
    check_outputs(calls()[op])


@pytest.mark.parametrize("op", ["matmul", "addmm", "matmul_silu_mul", "silu_mul", "rmsnorm", "mean", "log_softmax",
                                "log_softmax_cluster", "log_softmax_split", "decode_attention"])
def test_outputs_of_the_other_operators_are_of_the_calls_stream(op):
    check_outputs(other_calls()[op])


def test_scratch_is_of_the_calls_stream():
    """A block freed on the current stream is not the scratch of a call on another one: it is handed out again here."""
    call, side = calls()["attend"], torch.cuda.Stream()
    need = bi.bi_paged_decode_attention_scratch_bytes(B, HQ, D, LONGEST)
    assert need > 0
    torch.cuda.synchronize()
    block = torch.empty(need, dtype=torch.uint8, device=DEV)
    at = block.data_ptr()
    del block
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    o = call(side)
    assert torch.empty(need, dtype=torch.uint8, device=DEV).data_ptr() == at
    torch.cuda.synchronize()
    assert same_bits(o[0], call(None)[0])


@pytest.mark.parametrize("op", ["rope", "append", "attend", "logprobs"])
def test_results_dropped_before_the_work_is_done(op):
    """Results of a waiting stream dropped and their memory asked for on the current one: what is written there stays."""
    call, side = calls()[op], torch.cuda.Stream()
    sizes = [t.untyped_storage().nbytes() for t in call(None)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    for _ in range(4):
        call(side)
    kept = [torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert all(bool((t == 0x5A).all()) for t in kept)


def test_a_refused_call_restores_the_current_stream():
    side = torch.cuda.Stream()
    x = torch.zeros(2, 8, device=DEV)
    with pytest.raises(bi.BiError):
        bi.bi_token_logprobs(x, None, 0, 0.0, stream=side)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


@pytest.mark.parametrize("op,need", [("decode_attention", lambda: bi.bi_decode_attention_scratch_bytes(2, 8, 64, 600)),
                                     ("log_softmax_split", lambda: bi.bi_log_softmax_split_scratch_bytes(2, 40000))])
def test_scratch_of_the_other_operators_is_of_the_calls_stream(op, need):
    call, side, n = other_calls()[op], torch.cuda.Stream(), need()
    assert n > 0
    torch.cuda.synchronize()
    block = torch.empty(n, dtype=torch.uint8, device=DEV)
    at = block.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    del block
    o = call(side)
    other = torch.empty(n, dtype=torch.uint8, device=DEV)
    assert other.data_ptr() == at
    other.fill_(0x5A)
    torch.cuda.synchronize()
    assert bool((other == 0x5A).all()) and same_bits(o[0], call(None)[0])
