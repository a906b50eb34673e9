"""The decode-step operators with the library's others, as a server runs them: a one-layer decoder over a paged cache
(RMSNorm, fused q/k/v GEMM, rotation and append, attention over the pages, output GEMM with residual, gated MLP, LM
head, log-probabilities of the greedy token).  Every prompt's tokens, log-probabilities and entropies are the same bits alone
and in a batch of others, in eager calls and replayed from a graph, and the scores equal a dense fp64 computation from
the logits."""
import pytest
import torch

from bi_testutil import same_bits
from invariant_bi_matmul_02_b200 import binding as bi
from invariant_bi_matmul_02_b200 import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
HID, HQ, HKV, D, FFN, VOCAB, PAGE, STEPS = 256, 8, 2, 64, 512, 5003, 16, 6


class Decoder:
    def __init__(self):
        w = lambda seed, shape: inputs.weight_normal(seed, shape).to(DEV)  # noqa: E731
        self.embed = inputs.rows_normal(40, 0, VOCAB, HID).to(DEV)
        self.g1, self.g2, self.g3 = (inputs.gain(41 + i, HID).to(DEV) for i in range(3))
        self.qkv, self.o = w(44, ((HQ + 2 * HKV) * D, HID)), w(45, (HID, HQ * D))
        self.gu, self.down, self.head = w(46, (2 * FFN, HID)), w(47, (HID, FFN)), w(48, (VOCAB, HID))
        self.freq, self.scale = bi.bi_rope_freqs(D, 1.0e6)

    def cache(self, lens, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        width = -(-(max(lens) + STEPS) // PAGE)
        pages = len(lens) * width + 5
        k, v = (torch.randn(pages, PAGE, HKV, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
        return k, v, torch.randperm(pages, generator=g, device=DEV)[:len(lens) * width].to(torch.int32).view(len(lens), width)

    def layer(self, tokens, cache, lens, cu):
        """One pass over new tokens; with cu None one per sequence.  Returns hidden states and the turned queries."""
        k_cache, v_cache, table = cache
        x = self.embed[tokens.long()]
        T = x.shape[0]
        h = bi.bi_matmul(bi.bi_rmsnorm(x, self.g1), self.qkv)
        q, k, v = (h[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
        bi.bi_paged_append(k, v, k_cache, v_cache, table, lens, cu, self.freq, scale=self.scale, q=q, q_out=q)
        return x, q

    def step(self, tokens, cache, lens):
        x, q = self.layer(tokens, cache, lens, None)
        B = x.shape[0]
        a = bi.bi_paged_decode_attention(q, *cache, lens)
        x = bi.bi_addmm(x, a.view(B, HQ * D), self.o)
        m = bi.bi_matmul_silu_mul(bi.bi_rmsnorm(x, self.g2), self.gu)
        x = bi.bi_addmm(x, m, self.down)
        # A row of 5003 logits is padded to the GEMM's alignment: the log-probabilities take the strided view.
        wide = torch.empty(B, VOCAB + 5, dtype=torch.bfloat16, device=DEV)
        logits = bi.bi_matmul(bi.bi_rmsnorm(x, self.g3), self.head, out=wide[:, :VOCAB])
        best = bi.bi_token_logprobs(logits, None, 4)
        return logits, best.top_tokens[:, 0].contiguous(), best

    def generate(self, prompts, seed):
        lens = [len(p) for p in prompts]
        cache = self.cache(lens, seed)
        sl = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device=DEV)
        cu = torch.tensor([0] + [n - 1 for n in lens], device=DEV).cumsum(0).to(torch.int32)
        # All but each prompt's last token enter the cache in one call (a prompt of one token: nothing of it).
        body = torch.cat([p[:-1] for p in prompts])
        if len(body):
            self.layer(body, cache, sl, cu)
        tokens = torch.stack([p[-1] for p in prompts])
        out = []
        for _ in range(STEPS):
            sl += 1
            logits, tokens, best = self.step(tokens, cache, sl)
            scored = bi.bi_token_logprobs(logits, tokens)
            assert same_bits(scored.logprobs, best.top_logprobs[:, 0].contiguous()) and same_bits(scored.entropy, best.entropy)
            lp = torch.log_softmax(logits.double(), 1)
            assert float((scored.logprobs - lp.gather(1, tokens.long()[:, None])[:, 0]).abs().max()) <= 1e-4
            out.append((tokens, scored.logprobs, scored.entropy, best.top_tokens, best.top_logprobs))
        return [torch.stack([o[i] for o in out], 1) for i in range(5)], cache, sl, tokens


def test_a_decoder_over_pages_is_batch_invariant_and_replays_from_a_graph():
    net = Decoder()
    g = torch.Generator(device=DEV).manual_seed(9)
    prompts = [torch.randint(0, VOCAB, (n,), generator=g, device=DEV).to(torch.int32) for n in (37, 1, 530, 16, 90, 257)]
    together, cache, sl, tokens = net.generate(prompts, 1)
    for i, p in enumerate(prompts):
        alone = net.generate([p], 10 + i)[0]
        assert all(same_bits(a, t[i:i + 1].contiguous()) for a, t in zip(alone, together)), f"prompt {i}"
    shuffled = [4, 2, 0, 5]
    again = net.generate([prompts[i] for i in shuffled], 2)[0]
    assert all(same_bits(a, t[shuffled].contiguous()) for a, t in zip(again, together))
    # The same step captured: replayed over the cache's next place, with a place of the batch emptied.
    keep = [t.clone() for t in cache]
    sl += 1
    sl[3] = 0
    want = net.step(tokens, cache, sl)
    for t, k in zip(cache, keep):
        t.copy_(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = net.step(tokens, cache, sl)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    live = [0, 1, 2, 4, 5]  # the emptied place's query is not turned: nothing reads its row
    assert same_bits(got[0][live].contiguous(), want[0][live].contiguous())
    assert all(same_bits(a[live].contiguous(), b[live].contiguous()) for a, b in zip(got[2][1:], want[2][1:]))
    assert bi.bi_get_device_status() == bi.BI_OK
