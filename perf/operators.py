"""The operators around a decode step's kernels, as measurable cases: rotary positions, appending keys
and values to a paged cache, attention over that cache, and log-probabilities of chosen tokens.

``run`` computes each operator either in plain torch arithmetic (``own`` false: fp32, fp64 for the
angles, rounded once at the end) or through this package's entry points (``own`` true).  ``exact`` is the
definition in fp64.  Sizes follow the package's workloads (32 query heads and 8 key/value heads of 128,
a vocabulary of 151936, 64 sequences of 4096 tokens) and spread around them.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One new token of one sequence: the rotation of its 32 query and 8 key heads, in the fused
        # projection's output.  Latency only.
        {"name": "rope_one_token", "op": "rope", "tokens": 1, "heads": 40, "dim": 128, "rotary": 128,
         "layout": "half", "dtype": "bf16", "inverse": False, "strided": True, "far": False, "stretch": 1.0},
        # A batch of prompts in prefill, with frequencies stretched for a long context.
        {"name": "rope_prompt_8192", "op": "rope", "tokens": 8192, "heads": 40, "dim": 128, "rotary": 128,
         "layout": "half", "dtype": "bf16", "inverse": False, "strided": True, "far": True, "stretch": 8.0},
        # The transposed rotation (the gradient of the forward one) of fp32 values, adjacent pairs, on
        # part of an odd number of heads.
        {"name": "rope_inverse_part_fp32", "op": "rope", "tokens": 3001, "heads": 13, "dim": 96, "rotary": 64,
         "layout": "interleaved", "dtype": "f32", "inverse": True, "strided": False, "far": True, "stretch": 1.0},
        # A decode step of 64 sequences: each one's new key and value into its last page, its query
        # and key rotated on the way.
        {"name": "append_step_b64", "op": "append", "seqs": 64, "new": "one", "length": 1024, "page": 16,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128, "layout": "half", "heads_first": False,
         "query": True},
        # Prompts of mixed lengths entering the cache in one call (a prefill step), pages laid out head first.
        {"name": "append_prompts", "op": "append", "seqs": 9, "new": "prompt", "length": 2048, "page": 64,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128, "layout": "half", "heads_first": True,
         "query": True},
        # One short conversation: attention of a single token over 300 cached ones.
        {"name": "attend_one_short", "op": "attend", "seqs": 1, "length": 300, "ragged": False, "page": 16,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "heads_first": False},
        # The serving batch: 64 sequences of 4096 tokens in pages of 16.
        {"name": "attend_b64_4096", "op": "attend", "seqs": 64, "length": 4096, "ragged": False, "page": 16,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "heads_first": False},
        # One very long context.
        {"name": "attend_one_131072", "op": "attend", "seqs": 1, "length": 131072, "ragged": False, "page": 64,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "heads_first": False},
        # A mixed batch of lengths from none to 5000, head size 64, seven query heads per key head, pages of 24
        # tokens (no divisor of a power of two) laid out head first.
        {"name": "attend_ragged_d64", "op": "attend", "seqs": 37, "length": 5000, "ragged": True, "page": 24,
         "q_heads": 28, "kv_heads": 4, "dim": 64, "heads_first": True},
        # Sampling one token: its log-probability, the entropy and the 20 best alternatives.
        {"name": "logprobs_one_row", "op": "logprobs", "rows": 1, "vocab": 151936, "dtype": "bf16", "top": 20,
         "masked": False, "scale": 1.0},
        # Scoring 1024 positions of bf16 logits, with the five best alternatives of each.
        {"name": "logprobs_1024_rows", "op": "logprobs", "rows": 1024, "vocab": 151936, "dtype": "bf16", "top": 5,
         "masked": False, "scale": 1.0},
        # fp32 logits of an odd vocabulary under a mask that forbids most tokens, sampled at temperature 0.7.
        {"name": "logprobs_masked_fp32", "op": "logprobs", "rows": 77, "vocab": 50257, "dtype": "f32", "top": 8,
         "masked": True, "scale": 1.0 / 0.7},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "logprobs"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        heads = rng.randint(1, 48)
        tokens = _log_int(rng, 1, max(1, min(16384, 8192 * 40 * 128 // (heads * dim))))
        dtype = rng.choice(["bf16", "f32"])
        if dtype == "f32":
            tokens = max(1, tokens // 2)
        return {"op": "rope", "tokens": tokens, "heads": heads, "dim": dim,
                "rotary": rng.choice([dim, dim // 2, 2 * rng.randint(1, dim // 2)]),
                "layout": rng.choice(["half", "interleaved"]), "dtype": dtype, "inverse": rng.random() < 0.4,
                "strided": rng.random() < 0.5, "far": rng.random() < 0.5, "stretch": rng.choice([1.0, 4.0, 8.0])}
    if op == "append":
        dim = rng.choice([64, 96, 128, 256])
        kv = rng.randint(1, 8)
        one = rng.random() < 0.5
        return {"op": "append", "seqs": _log_int(rng, 1, 128) if one else rng.randint(1, 9),
                "new": "one" if one else "prompt", "length": _log_int(rng, 1, 128 * 1024 // dim),
                "page": rng.choice([1, 8, 16, 24, 32, 64, 128]), "q_heads": kv * rng.randint(1, 4), "kv_heads": kv,
                "dim": dim, "rotary": rng.choice([0, dim, dim, dim // 2]),
                "layout": rng.choice(["half", "interleaved"]), "heads_first": rng.random() < 0.5,
                "query": rng.random() < 0.7}
    if op == "attend":
        dim = rng.choice([64, 128])
        kv = rng.randint(1, 8)
        seqs = _log_int(rng, 1, 200)
        room = 64 * 4096 * 8 * 128 // (seqs * kv * dim)
        return {"op": "attend", "seqs": seqs, "length": _log_int(rng, 1, min(100000, room)),
                "ragged": rng.random() < 0.6, "page": rng.choice([4, 8, 16, 24, 32, 48, 64, 128, 256]),
                "q_heads": kv * rng.randint(1, 16), "kv_heads": kv, "dim": dim, "heads_first": rng.random() < 0.5}
    vocab = _log_int(rng, 1000, 200000)
    if rng.random() < 0.4:
        vocab = vocab // 64 * 64 + 64
    dtype = rng.choice(["bf16", "f32"])
    room = 1024 * 151936 // vocab // (2 if dtype == "f32" else 1)
    return {"op": "logprobs", "rows": _log_int(rng, 1, min(2048, room)), "vocab": vocab, "dtype": dtype,
            "top": rng.choice([0, 1, 5, 20, 32]), "masked": rng.random() < 0.3,
            "scale": rng.choice([1.0, 1.0, 1.0 / 0.7, 0.5])}


# ---------------------------------------------------------------------------------------- inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * (seed + 1))
    return g


def _inv_freq(rotary, stretch=1.0):
    """theta^(-2i/R), divided by `stretch` where the wavelength exceeds a context of 8192 tokens."""
    i = torch.arange(rotary // 2, dtype=torch.float64)
    f = torch.exp(i * (-2.0 / max(rotary, 1) * math.log(1.0e6)))
    return torch.where(2.0 * math.pi / f > 8192.0, f / stretch, f).to(DEV)


def _lengths(case):
    """Cached tokens of each sequence, settled by the case alone: all `length`, or spread over
    0 .. length with the first one full and (from three sequences on) one empty."""
    n, top = case["seqs"], case["length"]
    if not case.get("ragged", False):
        return [top] * n
    lens = [top - (i * 2654435761 % 4294967296) * top // 4294967296 for i in range(n)]
    if n >= 3:
        lens[2] = 0
    return lens


def _new_counts(case):
    """New tokens of each sequence: one, or prompts of mixed lengths (some of them the rest of a longer one)."""
    if case["new"] == "one":
        return [1] * case["seqs"]
    return [max(1, case["length"] - (i * 2654435761 % 4294967296) * case["length"] // 4294967296)
            for i in range(case["seqs"])]


def _paged(case, lens, g):
    """A cache whose pages are handed out in random order: k, v [pages, page, heads, dim] views, the
    block table with -1 past each sequence's pages."""
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    need = [-(-n // page) for n in lens]
    width = max(max(need), 1)
    pages = sum(need) + 3
    shape = (pages, heads, page, dim) if case["heads_first"] else (pages, page, heads, dim)
    k = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    if case["heads_first"]:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)[None]
    n = torch.tensor(need, device=DEV)[:, None]
    first = torch.cumsum(n, 0) - n
    at = torch.where(col < n, first + col, 0)
    table = torch.where(col < n, order[at], torch.full_like(order[at], -1)).contiguous()
    return k, v, table


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case}
    if op == "rope":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        row = H * D + (16 * D if case["strided"] else 0)  # a projection's row holds the values too
        wide = torch.randn((T, row), generator=g, device=DEV).to(_dtype(case))
        s["x"] = wide[:, :H * D].view(T, H, D)
        start = 1000000 if case["far"] else 4096
        s["positions"] = (torch.randint(0, start, (1,), generator=g, device=DEV)
                          + torch.arange(T, device=DEV)).to(torch.int32)
        s["inv_freq"] = _inv_freq(case["rotary"], case["stretch"])
        s["scale"] = 0.1 * math.log(case["stretch"]) + 1.0
        s["out"] = torch.empty((T, H, D), dtype=s["x"].dtype, device=DEV)
    elif op == "append":
        new = _new_counts(case)
        lens = [case["length"]] * case["seqs"]
        lens = [max(a, b) for a, b in zip(lens, new)]
        T, D, Hq, Hkv = sum(new), case["dim"], case["q_heads"], case["kv_heads"]
        s["k_cache"], s["v_cache"], s["table"] = _paged(case, lens, g)
        qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=DEV).to(torch.bfloat16)
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D) if case["query"] else None
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        s["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV) if case["query"] else None
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        cu = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
        s["cu_new"] = None if case["new"] == "one" else cu
        s["inv_freq"] = _inv_freq(case["rotary"]) if case["rotary"] else None
    elif op == "attend":
        lens = _lengths(case)
        s["k_cache"], s["v_cache"], s["table"] = _paged(case, lens, g)
        s["q"] = torch.randn((case["seqs"], case["q_heads"], case["dim"]), generator=g, device=DEV).to(torch.bfloat16)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["max_len"] = max(max(lens), 1)
        s["out"] = torch.empty_like(s["q"])
        s["scratch"] = torch.empty(  # the workspace a server keeps between steps
            case["seqs"] * case["q_heads"] * (-(-s["max_len"] // 128) + 1) * (case["dim"] + 4), device=DEV)
    else:
        M, V = case["rows"], case["vocab"]
        x = 1.3 * torch.randn((M, V), generator=g, device=DEV)
        if case["masked"]:
            keep = torch.rand((M, V), generator=g, device=DEV) < 0.002
            keep[:, 7] = True
            x = torch.where(keep, x, torch.full_like(x, -math.inf))
            tokens = torch.argmax(torch.where(keep, torch.rand((M, V), generator=g, device=DEV), 0.0), 1)
        else:
            tokens = torch.randint(0, V, (M,), generator=g, device=DEV)
        s["logits"] = x.to(_dtype(case))
        s["tokens"] = tokens.to(torch.int32)
        s["scale"] = case["scale"]
    return s


# ---------------------------------------------------------------------------------------- one pass

def _rotate(x, cos, sin, rotary, layout):
    """x [T, H, D] rotated by [T, R/2] cosines and sines over its first R entries; x's type throughout."""
    h = rotary // 2
    c, s = cos[:, None, :].to(x.dtype), sin[:, None, :].to(x.dtype)
    out = x.clone()
    if layout == "half":
        a, b = x[..., :h], x[..., h:rotary]
        out[..., :h] = a * c - b * s
        out[..., h:rotary] = b * c + a * s
    else:
        a, b = x[..., 0:rotary:2], x[..., 1:rotary:2]
        out[..., 0:rotary:2] = a * c - b * s
        out[..., 1:rotary:2] = b * c + a * s
    return out


def _places(s):
    """Each new token's sequence, place in it, and (page, row) in the cache."""
    T = s["k"].shape[0]
    lens = s["seq_lens"].long()
    t = torch.arange(T, device=DEV)
    if s["cu_new"] is None:
        seq, pos = t, lens - 1
    else:
        cu = s["cu_new"].long()
        seq = torch.searchsorted(cu, t, right=True) - 1
        pos = lens[seq] - (cu[seq + 1] - t)
    page = s["k_cache"].shape[1]
    return pos, s["table"].long()[seq, pos // page], pos % page


def _plain_append(s):
    case = s["case"]
    pos, pages, rows = _places(s)
    k, v, q = s["k"].float(), s["v"], s["q"]
    if s["inv_freq"] is not None:
        angle = pos.double()[:, None] * s["inv_freq"]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        k = _rotate(k, cos, sin, case["rotary"], case["layout"])
        if q is not None:
            s["q_out"].copy_(_rotate(q.float(), cos, sin, case["rotary"], case["layout"]))
    elif q is not None:
        s["q_out"].copy_(q)
    s["k_cache"][pages, rows] = k.to(torch.bfloat16)
    s["v_cache"][pages, rows] = v
    out = {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if q is not None:
        out["q"] = s["q_out"]
    return out


def _attend(q, k_cache, v_cache, table, seq_lens, max_len, kind):
    """softmax(q . k / sqrt(D)) v over each sequence's pages, in `kind`; an empty sequence gives zeros."""
    B, Hq, D = q.shape
    page, Hkv = k_cache.shape[1], k_cache.shape[2]
    n = -(-max_len // page)
    at = table[:, :n].long().clamp(min=0)
    L = n * page
    k = k_cache[at].reshape(B, L, Hkv, D).permute(0, 2, 3, 1).to(kind)
    scores = torch.matmul(q.to(kind).view(B, Hkv, Hq // Hkv, D), k) * (D ** -0.5)
    del k
    live = torch.arange(L, device=DEV)[None] < seq_lens[:, None]
    scores = torch.where(live[:, None, None], scores, torch.full_like(scores, -math.inf))
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    v = v_cache[at].reshape(B, L, Hkv, D).permute(0, 2, 1, 3).to(kind)
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    return o.reshape(B, Hq, D)


def _logprobs(x, tokens, scale, top, kind):
    """Log-probability of each row's token, entropy, log of the sum of exponentials, and the `top` largest
    log-probabilities with their tokens (ties to the lower token), of the logits times `scale`."""
    z = x.to(kind) * scale
    m = z.amax(1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    picked = torch.gather(d, 1, tokens.long()[:, None]) - log_total
    entropy = log_total - (e * torch.where(e > 0, d, torch.zeros_like(d))).sum(1, keepdim=True) / total
    out = {"logprobs": picked[:, 0], "entropy": entropy[:, 0], "logsumexp": (m + log_total)[:, 0]}
    if top:
        order = torch.sort(x.float(), dim=1, descending=True, stable=True)[1][:, :top]
        out["top_logprobs"] = torch.gather(d, 1, order) - log_total
        out["top_tokens"] = order.to(torch.int32)
    return out


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import invariant_bi_matmul_02_b200 as bi
        if op == "rope":
            return bi.bi_rope(s["x"], s["positions"], s["inv_freq"], layout=case["layout"], scale=s["scale"],
                              inverse=case["inverse"], out=s["out"])
        if op == "append":
            q = bi.bi_paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"],
                                   cu_new=s["cu_new"], inv_freq=s["inv_freq"], layout=case["layout"], q=s["q"],
                                   q_out=s["q_out"])
            out = {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
            if s["q"] is not None:
                out["q"] = q
            return out
        if op == "attend":
            return bi.bi_paged_decode_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"],
                                                max_len=s["max_len"], scratch=s["scratch"], out=s["out"])
        r = bi.bi_token_logprobs(s["logits"], s["tokens"], top_k=case["top"], scale=s["scale"])
        out = {"logprobs": r.logprobs, "entropy": r.entropy, "logsumexp": r.logsumexp}
        if case["top"]:
            out["top_logprobs"], out["top_tokens"] = r.top_logprobs, r.top_tokens
        return out
    if op == "rope":
        angle = s["positions"].double()[:, None] * s["inv_freq"]
        sign = -1.0 if case["inverse"] else 1.0
        y = _rotate(s["x"].float(), torch.cos(angle).float() * s["scale"], torch.sin(angle).float() * (sign * s["scale"]),
                    case["rotary"], case["layout"])
        return y.to(s["x"].dtype)
    if op == "append":
        return _plain_append(s)
    if op == "attend":
        return _attend(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"], s["max_len"],
                       torch.float32).to(torch.bfloat16)
    return _logprobs(s["logits"], s["tokens"], s["scale"], case["top"], torch.float32)


# ---------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * size + 4 * case["tokens"] + 4 * case["rotary"],
                "flops": 3 * case["tokens"] * case["heads"] * case["rotary"]}
    if op == "append":
        T = sum(_new_counts(case))
        heads = (case["q_heads"] if case["query"] else 0) + 2 * case["kv_heads"]
        turned = (case["q_heads"] if case["query"] else 0) + case["kv_heads"]
        return {"bytes": 2 * 2 * T * heads * case["dim"] + 8 * case["seqs"] + 4 * T,
                "flops": 3 * T * turned * case["rotary"]}
    if op == "attend":
        lens = _lengths(case)
        total = sum(lens)
        return {"bytes": 4 * total * case["kv_heads"] * case["dim"] + 4 * case["seqs"] * case["q_heads"] * case["dim"]
                + 4 * sum(-(-n // case["page"]) for n in lens) + 4 * case["seqs"],
                "flops": 4 * total * case["q_heads"] * case["dim"]}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + case["rows"] * (16 + 8 * case["top"]),
            "flops": 6 * n}


# ---------------------------------------------------------------------------------------- fp64 definition

def _turned(x, positions, inv_freq, rotary, layout, inverse=False):
    """x [T, H, D] in fp64 with each pair (a, b) taken to (a + ib) e^{i p w}."""
    T, H, D = x.shape
    w = torch.exp(1j * (positions.double()[:, None] * inv_freq).to(torch.complex128))
    if inverse:
        w = w.conj()
    pairs = x[..., :rotary].double()
    if layout == "half":
        z = torch.complex(pairs[..., :rotary // 2].contiguous(), pairs[..., rotary // 2:].contiguous())
    else:
        z = torch.view_as_complex(pairs.reshape(T, H, rotary // 2, 2).contiguous())
    z = z * w[:, None, :]
    turned = torch.cat([z.real, z.imag], -1) if layout == "half" else torch.view_as_real(z).reshape(T, H, rotary)
    return turned


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        out = s["x"].double()
        out[..., :case["rotary"]] = s["scale"] * _turned(s["x"], s["positions"], s["inv_freq"], case["rotary"],
                                                         case["layout"], case["inverse"])
        return out
    if op == "append":
        new, lens = _new_counts(case), s["seq_lens"].tolist()
        page, R = case["page"], case["rotary"]
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        place = torch.cat([torch.arange(n - c, n) for n, c in zip(lens, new)]).to(DEV)
        seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).to(DEV)
        k, q = s["k"].double(), None if s["q"] is None else s["q"].double()
        if R:
            k[..., :R] = _turned(s["k"], place, s["inv_freq"], R, case["layout"])
            if q is not None:
                q[..., :R] = _turned(s["q"], place, s["inv_freq"], R, case["layout"])
        at = s["table"][seq, torch.div(place, page, rounding_mode="floor")].long()
        k_cache[at, place % page] = k
        v_cache[at, place % page] = s["v"].double()
        out = {"k_cache": k_cache, "v_cache": v_cache}
        if q is not None:
            out["q"] = q
        return out
    if op == "attend":
        B, Hq, D = s["q"].shape
        page, Hkv = case["page"], case["kv_heads"]
        out = torch.zeros((B, Hq, D), dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["seq_lens"].tolist()):
            if n == 0:
                continue
            at = s["table"][b, :-(-n // page)].long()
            k = s["k_cache"][at].reshape(-1, Hkv, D)[:n].double()
            v = s["v_cache"][at].reshape(-1, Hkv, D)[:n].double()
            q = s["q"][b].double().view(Hkv, Hq // Hkv, D)
            p = torch.softmax(torch.einsum("hgd,lhd->hgl", q, k) / math.sqrt(D), -1)
            out[b] = torch.einsum("hgl,lhd->hgd", p, v).reshape(Hq, D)
        return out
    parts = []
    for r in range(0, case["rows"], 128):
        x = s["logits"][r:r + 128]
        z = x.double() * s["scale"]
        lse = torch.logsumexp(z, 1)
        lp = z - lse[:, None]
        part = {"logprobs": lp.gather(1, s["tokens"][r:r + 128].long()[:, None])[:, 0],
                "entropy": -torch.xlogy(lp.exp(), lp.exp()).sum(1), "logsumexp": lse}
        if case["top"]:
            # The k-th largest value bounds the candidates; among equals the lower token comes first.
            kth = x.double().topk(case["top"], 1)[0][:, -1:]
            tokens = torch.arange(x.shape[1], device=DEV).expand_as(x)
            above, level = x.double() > kth, x.double() == kth
            room = case["top"] - above.sum(1, keepdim=True)
            chosen = above | (level & (level.cumsum(1) <= room))
            ids = tokens[chosen].view(x.shape[0], case["top"])
            vals = x.double().gather(1, ids)
            by = torch.sort(vals, dim=1, descending=True, stable=True)[1]  # ids ascend, so equals keep their order
            ids = ids.gather(1, by)
            part["top_logprobs"] = lp.gather(1, ids)
            part["top_tokens"] = ids.to(torch.int32)
        parts.append(part)
    return {n: torch.cat([p[n] for p in parts]) for n in parts[0]}
