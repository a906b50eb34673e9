"""The failure path of the bounded device-side waits, without a GPU fault.

A kernel waits on a barrier that nothing completes, through the same bounded wait
the GEMM's pipeline uses; the wait gives up after its limit, records BI_ERR_TIMEOUT
in the device status word and returns, and the context stays usable.
"""
import time

import pytest
import torch

from invariant_bi_matmul_02_b200 import binding as bi

pytestmark = pytest.mark.gpu


def test_wait_that_runs_out_reports_timeout_and_context_survives():
    assert bi.bi_get_device_status() == bi.BI_OK
    t0 = time.perf_counter()
    bi.bi_selftest_wait_timeout(2_000_000)  # 2 ms
    assert bi.bi_get_device_status() == bi.BI_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 5.0
    assert bi.bi_get_device_status() == bi.BI_OK  # reading clears the word
    a = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, 64, dtype=torch.bfloat16, device="cuda")
    c = bi.bi_matmul(a, w, "nk")
    assert torch.all(c == 64)
    assert bi.bi_get_device_status() == bi.BI_OK


def test_selftest_limit_is_validated():
    with pytest.raises(bi.BiError):
        bi.bi_selftest_wait_timeout(10)


def bad_calls():
    """Calls that each record BI_ERR_INVALID_ARG: a token, a length, a page and a place out of range."""
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    n = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q, cache, table = z(1, 1, 64), z(2, 16, 1, 64), n(9).view(1, 1)
    return {
        "token": lambda: bi.bi_token_logprobs(z(1, 8), n(8)),
        "length": lambda: bi.bi_decode_attention(q, z(1, 16, 1, 64), z(1, 16, 1, 64), n(17)),
        "paged length": lambda: bi.bi_paged_decode_attention(q, cache, cache, n(0).view(1, 1), n(-1)),
        "page": lambda: bi.bi_paged_decode_attention(q, cache, cache, table, n(5)),
        "place": lambda: bi.bi_paged_append(q, q, cache, cache, table, n(5)),
    }


@pytest.mark.parametrize("kind", ["token", "length", "paged length", "page", "place"])
def test_the_first_error_is_kept(kind):
    bad = bad_calls()[kind]
    assert bi.bi_get_device_status() == bi.BI_OK
    bad()
    assert bi.bi_get_device_status() == bi.BI_ERR_INVALID_ARG
    bi.bi_selftest_wait_timeout(1_000_000)
    bad()
    assert bi.bi_get_device_status() == bi.BI_ERR_TIMEOUT
    bad()
    bi.bi_selftest_wait_timeout(1_000_000)
    assert bi.bi_get_device_status() == bi.BI_ERR_INVALID_ARG
    assert bi.bi_get_device_status() == bi.BI_OK
