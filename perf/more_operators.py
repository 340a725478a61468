"""What is measured of the operators of a prompt.

Three operators that take many tokens at once, each in a plain form (elementary
torch operations in fp32) and as a user calls it from this package:

  prompt  causal attention of packed sequences of query tokens over a paged
          cache: a shared prefix, then a sequence's own positions up to the
          token's own; query heads share key-value heads
  linear  y[T][N] = x[T][K] W^T with W in the int4 group format of pack_int4
          (value = scale q + bias), for more tokens than a decoding step has:
          the projections either side of the attention, and an output head
  scores  of an output head's scores [T][V]: the log probabilities of given
          tokens, the entropy, and the most probable alternatives
"""
import math

import torch

own = False

GROUPS = (32, 64, 128)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one short question, nothing before it; latency
        dict(name="prompt 77", op="prompt", S=1, lo=77, hi=77, hist=0, prefix=0, Hq=16, Hkv=2, D=128, page=64,
             heads_first=True),
        # seven requests of odd lengths packed together, other heads (three to
        # a key-value head, D = 64), small pages laid out position by position
        dict(name="prompt ragged 7", op="prompt", S=7, lo=3, hi=1531, hist=0, prefix=0, Hq=24, Hkv=8, D=64, page=16,
             heads_first=False),
        # the next piece of a long prompt that is worked through in pieces
        dict(name="prompt piece 509 of 32K", op="prompt", S=1, lo=509, hi=509, hist=32259, prefix=0, Hq=16, Hkv=2,
             D=128, page=64, heads_first=True),
        # eight requests behind a system prompt that they share
        dict(name="prompt 8 prefix 8191", op="prompt", S=8, lo=130, hi=700, hist=0, prefix=8191, Hq=16, Hkv=2, D=128,
             page=64, heads_first=True),
        # the largest: a whole prompt of 16384 tokens
        dict(name="prompt 16384", op="prompt", S=1, lo=16384, hi=16384, hist=0, prefix=0, Hq=16, Hkv=2, D=128,
             page=64, heads_first=True),
        # one token more than a decoding step takes: (16 + 2 * 2) heads of 128
        # from a hidden size of 2048
        dict(name="linear qkv 65", op="linear", T=65, K=2048, N=2560, group=64, fp32=False),
        # the same projection for a prompt of 4096 tokens
        dict(name="linear qkv 4096", op="linear", T=4096, K=2048, N=2560, group=64, fp32=False),
        # odd sizes: rows, columns and tokens off every tile, fp32 results
        dict(name="linear odd 1021", op="linear", T=1021, K=2080, N=5003, group=32, fp32=True),
        # an output head over a piece of a prompt, fp32 scores for what follows
        dict(name="linear head 512", op="linear", T=512, K=2048, N=131072, group=64, fp32=True),
        # the scores of one new token with twenty alternatives; latency
        dict(name="scores 1", op="scores", T=1, V=131072, n_top=20, fp32=True),
        # a short prompt, odd vocabulary, bf16 scores (many of them equal)
        dict(name="scores odd 257", op="scores", T=257, V=50021, n_top=5, fp32=False),
        # scoring a whole prompt; bandwidth
        dict(name="scores 4096", op="scores", T=4096, V=131072, n_top=8, fp32=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prompt", "linear", "scores"))
    if op == "linear":
        # at most the listed head's products and results
        while True:
            group = rng.choice(GROUPS)
            K = group * max(1, _log_int(rng, 128, 4096) // group)
            T, N = _log_int(rng, 65, 16384), _log_int(rng, 16, 131072)
            if T * N <= 512 * 131072 and T * N * K <= 512 * 131072 * 2048:
                return dict(op=op, T=T, K=K, N=N, group=group, fp32=rng.random() < 0.4)
    if op == "scores":
        while True:
            T, V = _log_int(rng, 1, 4096), _log_int(rng, 100, 200000)
            if T * V <= 4096 * 131072:
                return dict(op=op, T=T, V=V, n_top=rng.choice((0, 1, rng.randint(2, 32))), fp32=rng.random() < 0.6)
    D = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    Hq = Hkv * rng.randint(1, 8)
    # at most the largest listed case's products and, padded, its scores
    while True:
        S = _log_int(rng, 1, 32)
        hi = _log_int(rng, 1, 16384)
        hist = 0 if rng.random() < 0.5 else _log_int(rng, 1, 65536)
        prefix = 0 if rng.random() < 0.6 else _log_int(rng, 1, 65536)
        case = dict(op=op, S=S, lo=rng.randint(1, hi), hi=hi, hist=hist, prefix=prefix, Hq=Hq, Hkv=Hkv, D=D,
                    page=rng.choice((16, 32, 64, 128, 256)), heads_first=rng.random() < 0.5)
        n = prefix + max(_seq_lens(case))
        if S * Hq * hi * n <= 16 * 16384 ** 2 and S * n * Hkv * D <= 1 << 28 and S * hi <= 32768:
            return case


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(g, *shape, std=1.0):
    return torch.empty(*shape, device="cuda", dtype=torch.float32).normal_(0.0, std, generator=g).to(torch.bfloat16)


def _q_lens(case):
    """The sequences' numbers of query tokens: spread evenly over [lo, hi] in a mixed order."""
    n, lo, hi = case["S"], case["lo"], case["hi"]
    return [lo + (hi - lo) * ((7 * i + n - 1) % n) // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _seq_lens(case):
    """Their lengths with what is in the cache already."""
    return [q + (case["hist"] + 3 * i if case["hist"] else 0) for i, q in enumerate(_q_lens(case))]


def _pool(g, case, n_pages):
    """One page pool [n_pages][Hkv][page][D] (a view of position-major memory
    unless heads_first)."""
    a, b = (case["Hkv"], case["page"]) if case["heads_first"] else (case["page"], case["Hkv"])
    p = _bf16(g, n_pages, a, b, case["D"])
    return p if case["heads_first"] else p.transpose(1, 2)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "linear":
        T, K, N, G = case["T"], case["K"], case["N"], case["group"]
        pitch = (K // G + 7) // 8 * 8
        q = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g, device="cuda", dtype=torch.int32)
        # weights ~ N(0, 0.02): a group's range is about 4.5 sigma over 15 steps
        s = (torch.rand(N, K // G, generator=g, device="cuda") * 0.004 + 0.004).to(torch.bfloat16)
        b = (-7.5 * s.float() + 0.004 * (torch.rand(N, K // G, generator=g, device="cuda") - 0.5)).to(torch.bfloat16)
        sp = torch.zeros(N, pitch, device="cuda", dtype=torch.bfloat16)
        bp = torch.zeros(N, pitch, device="cuda", dtype=torch.bfloat16)
        sp[:, :K // G] = s
        bp[:, :K // G] = b
        st = dict(case=case, q=q, s=sp.view(torch.int16), b=bp.view(torch.int16), x=_bf16(g, T, K))
        st["y"] = torch.empty(T, N, device="cuda", dtype=torch.float32 if case["fp32"] else torch.bfloat16)
        if own:
            from int4_grouped_gemm_gb300 import moe
            st["w"] = moe.QMatrix(st["q"], st["s"], st["b"], N, K, G)
            st["ws"] = moe.linear_prompt_workspace(st["w"], T)
        return st
    if case["op"] == "scores":
        T, V = case["T"], case["V"]
        x = torch.empty(T, V, device="cuda", dtype=torch.float32).normal_(0.0, 2.5, generator=g)
        targets = torch.randint(0, V, (T,), generator=g, device="cuda")
        # most given tokens are among the more probable ones
        x[torch.arange(T, device="cuda"), targets] += 8 * torch.rand(T, generator=g, device="cuda")
        st = dict(case=case, x=x if case["fp32"] else x.to(torch.bfloat16), targets=targets.to(torch.int32))
        if own:
            from int4_grouped_gemm_gb300 import scores
            st["ws"] = scores.workspace(T, V, case["n_top"])
        return st
    S, Hq, Hkv, D, page = (case[n] for n in ("S", "Hq", "Hkv", "D", "page"))
    cpu = torch.Generator().manual_seed(seed)
    q_lens, lens = _q_lens(case), _seq_lens(case)
    T = sum(q_lens)
    n_prefix = -(-case["prefix"] // page)
    n_own = [-(-n // page) for n in lens]
    total = n_prefix + sum(n_own) + 1
    perm = torch.randperm(total, generator=cpu).to(torch.int32)
    table = torch.zeros(S, max(n_own), dtype=torch.int32)
    at = n_prefix
    for b in range(S):
        table[b, :n_own[b]] = perm[at:at + n_own[b]]
        at += n_own[b]
    starts = [sum(q_lens[:b]) for b in range(S + 1)]
    st = dict(case=case, kp=_pool(g, case, total), vp=_pool(g, case, total), table=table.cuda(),
              prefix_pages=perm[:n_prefix].cuda() if n_prefix else None,
              q_start=torch.tensor(starts, dtype=torch.int32).cuda(),
              lens=torch.tensor(lens, dtype=torch.int32).cuda(), q=_bf16(g, T, Hq, D), scale=1.0 / math.sqrt(D))
    st["out"] = torch.empty(T, Hq, D, device="cuda", dtype=torch.bfloat16)
    if own:
        from int4_grouped_gemm_gb300 import attention
        st["cache"] = attention.PagedCache(st["kp"], st["vp"])
        st["ws"] = st["cache"].prompt_workspace(T, S, Hq)
    return st


# ------------------------------------------------------------ one pass through

def run(st):
    case = st["case"]
    if own:
        if case["op"] == "linear":
            from int4_grouped_gemm_gb300 import moe
            return moe.linear_prompt(st["w"], st["x"], st["y"], ws=st["ws"])
        if case["op"] == "scores":
            from int4_grouped_gemm_gb300 import scores
            r = scores.token_logprobs(st["x"], st["targets"], case["n_top"], ws=st["ws"])
            return dict(logprob=r.logprob, entropy=r.entropy, ids=r.top_ids, top=r.top_logprobs)
        return st["cache"].attend_prompt(st["q"], st["q_start"], st["table"], st["lens"], st["prefix_pages"],
                                         case["prefix"], scale=st["scale"], out=st["out"], ws=st["ws"])
    return {"linear": _linear, "scores": _scores, "prompt": _prompt}[case["op"]](st)


def _bf16_bits(t):
    return (t.to(torch.int32) << 16).view(torch.float32)


def _linear(st):
    case = st["case"]
    N, K, G = case["N"], case["K"], case["group"]
    # element k of a word is nibble (k % 8) / 2 + 4 ((k % 8) % 2)
    shifts = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device="cuda", dtype=torch.int32)
    codes = (st["q"].view(N, K // 8, 1) >> shifts) & 15
    s = _bf16_bits(st["s"])[:, :K // G].unsqueeze(2)
    b = _bf16_bits(st["b"])[:, :K // G].unsqueeze(2)
    w = (codes.view(N, K // G, G).float() * s + b).view(N, K)
    st["y"].copy_(st["x"].float() @ w.t())
    return st["y"]


def _scores(st):
    case = st["case"]
    x = st["x"].float()
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    lse = m + total.log()
    entropy = total.log() - (e * (x - m)).sum(-1, keepdim=True) / total
    # equal scores in the order of their ids
    top, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    n = case["n_top"]
    given = x.gather(1, st["targets"].long().unsqueeze(1))
    return dict(logprob=(given - lse)[:, 0], entropy=entropy[:, 0], ids=ids[:, :n].to(torch.int32),
                top=top[:, :n] - lse)


def _prompt(st):
    case = st["case"]
    S, Hq, Hkv, D, page = (case[n] for n in ("S", "Hq", "Hkv", "D", "page"))
    P, G, nq, n, T = case["prefix"], Hq // Hkv, case["hi"], max(_seq_lens(case)), st["q"].shape[0]
    # the sequences' queries, padded to the most: [S][Hkv][G][nq][D]
    starts, lens = st["q_start"].long(), st["lens"].long()
    q_lens = starts[1:] - starts[:-1]
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), q_lens, output_size=T)
    i = torch.arange(T, device="cuda") - starts[seq]
    q = torch.zeros(S, nq, Hkv, G, D, device="cuda")
    q[seq, i] = st["q"].float().view(T, Hkv, G, D) * st["scale"]
    q = q.permute(0, 2, 3, 1, 4).reshape(S, Hkv, G * nq, D)
    # their keys and values, the prefix first, padded to the longest: [S][Hkv][P + n][D]
    at = torch.arange(n, device="cuda")
    pages, off = st["table"].long()[:, at // page], (at % page).expand(S, n)
    k, v = (p[pages, :, off].float().permute(0, 2, 1, 3) for p in (st["kp"], st["vp"]))
    if P:
        at = torch.arange(P, device="cuda")
        pages, off = st["prefix_pages"].long()[at // page], at % page
        k, v = (torch.cat((p[pages, :, off].float().transpose(0, 1).expand(S, Hkv, P, D), x), 2)
                for p, x in ((st["kp"], k), (st["vp"], v)))
    s = (q @ k.transpose(2, 3)).view(S, Hkv, G, nq, P + n)
    last = P + (lens - q_lens)[:, None] + torch.arange(nq, device="cuda")
    s.masked_fill_((torch.arange(P + n, device="cuda") > last[:, :, None])[:, None, None], -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    o = (s.view(S, Hkv, G * nq, P + n) @ v).view(S, Hkv, G, nq, D) / total
    st["out"].copy_(o.permute(0, 3, 1, 2, 4)[seq, i].reshape(T, Hq, D))
    return st["out"]


# ---------------------------------------------------------- work and 64 bits

def work(case):
    if case["op"] == "linear":
        T, K, N, G = case["T"], case["K"], case["N"], case["group"]
        return dict(bytes=N * K // 2 + 4 * N * (K // G) + 2 * T * K + (4 if case["fp32"] else 2) * T * N,
                    flops=2 * T * N * K)
    if case["op"] == "scores":
        T, V = case["T"], case["V"]
        # a subtraction, an exponential, a product and two sums for each score
        return dict(bytes=(4 if case["fp32"] else 2) * T * V + 12 * T + 8 * T * case["n_top"], flops=5 * T * V)
    Hq, Hkv, D, P = (case[n] for n in ("Hq", "Hkv", "D", "prefix"))
    q_lens, lens = _q_lens(case), _seq_lens(case)
    seen = sum(q * P + q * (n - q) + q * (q + 1) // 2 for q, n in zip(q_lens, lens))
    n = P + sum(lens)
    return dict(bytes=4 * Hkv * D * n + 4 * sum(q_lens) * Hq * D + 4 * (n // case["page"]), flops=4 * Hq * D * seen)


def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    if case["op"] == "linear":
        N, K, G = case["N"], case["K"], case["group"]
        outs = []
        x = st["x"].to(d)
        for r in range(0, N, 8192):
            q = st["q"][r:r + 8192].to(torch.int64) & 0xFFFFFFFF
            w = torch.empty(q.shape[0], K, device="cuda", dtype=d)
            for e in range(8):
                nibble = e // 2 + 4 * (e % 2)
                w[:, e::8] = ((q >> (4 * nibble)) & 15).to(d)
            s = st["s"][r:r + 8192, :K // G].contiguous().view(torch.bfloat16).to(d).repeat_interleave(G, 1)
            b = st["b"][r:r + 8192, :K // G].contiguous().view(torch.bfloat16).to(d).repeat_interleave(G, 1)
            outs.append(x @ (w * s + b).t())
        return torch.cat(outs, 1)
    if case["op"] == "scores":
        rows = []
        for r in range(0, case["T"], 256):
            lp = torch.log_softmax(st["x"][r:r + 256].to(d), dim=-1)
            h = -(lp.exp() * lp).sum(-1)
            given = torch.stack([lp[i, t] for i, t in enumerate(st["targets"][r:r + 256].tolist())])
            rows.append((given, h, lp.topk(case["n_top"], dim=-1).values))
        return dict(logprob=torch.cat([a for a, _, _ in rows]), entropy=torch.cat([h for _, h, _ in rows]), ids=None,
                    top=torch.cat([t for _, _, t in rows]))
    Hq, Hkv, D, page, P = (case[n] for n in ("Hq", "Hkv", "D", "page", "prefix"))
    G = Hq // Hkv
    q_lens, lens = _q_lens(case), _seq_lens(case)
    out = torch.zeros(sum(q_lens), Hq, D, device="cuda", dtype=d)
    for h in range(Hkv):
        k0 = v0 = torch.zeros(0, D, device="cuda", dtype=d)
        if P:
            k0 = st["kp"][st["prefix_pages"].long(), h].reshape(-1, D)[:P].to(d)
            v0 = st["vp"][st["prefix_pages"].long(), h].reshape(-1, D)[:P].to(d)
        row = 0
        for b, (nq, n) in enumerate(zip(q_lens, lens)):
            own_pages = st["table"][b, :-(-n // page)].long()
            k = torch.cat((k0, st["kp"][own_pages, h].reshape(-1, D)[:n].to(d)))
            v = torch.cat((v0, st["vp"][own_pages, h].reshape(-1, D)[:n].to(d)))
            for i0 in range(0, nq, 2048):
                i1 = min(nq, i0 + 2048)
                end = P + n - nq + i1  # what the last of these tokens sees
                hidden = torch.ones(i1 - i0, end, device="cuda", dtype=torch.bool).triu(P + n - nq + i0 + 1)
                for g in range(h * G, (h + 1) * G):
                    s = st["q"][row + i0:row + i1, g].to(d) @ k[:end].t() * st["scale"]
                    out[row + i0:row + i1, g] = torch.softmax(s.masked_fill(hidden, -math.inf), dim=-1) @ v[:end]
            row += nq
    return out
