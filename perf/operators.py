"""What is measured of the attention operators of a decoder layer.

Three operators that together make the attention sub-layer of a decoding
step, each in a plain form (elementary torch operations in fp32) and as a user
calls it from this package:

  linear  y[B][N] = x[B][K] W^T with W in the int4 group format of pack_int4
          (value = scale q + bias), 1 to 64 rows: the projections either side
          of the attention, and an output head
  append  rotate new queries and keys by their positions and write keys and
          values into a paged cache
  attend  one query row per sequence against a prefix that all sequences share
          and the sequence's own pages, query heads sharing key-value heads
"""
import math

import torch

own = False

GROUPS = (32, 64, 128)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token's query/key/value projection: (16 + 2 * 2) heads of 128
        # from a hidden size of 2048; latency
        dict(name="linear qkv 1", op="linear", B=1, K=2048, N=2560, group=64, fp32=False),
        # the output projection of eight tokens (a batch of draft tokens)
        dict(name="linear out 8", op="linear", B=8, K=2048, N=2048, group=64, fp32=False),
        # odd sizes: rows, columns and tokens off every tile
        dict(name="linear odd 37", op="linear", B=37, K=2080, N=5003, group=32, fp32=False),
        # an output head for one token, fp32 scores; bandwidth
        dict(name="linear head 1", op="linear", B=1, K=4096, N=131072, group=128, fp32=True),
        # the same for a batch of 64 sequences
        dict(name="linear head 64", op="linear", B=64, K=2048, N=131072, group=64, fp32=False),
        # a decoding step's eight tokens, far into their sequences; latency
        dict(name="append step 8", op="append", T=8, n_seq=8, Hq=16, Hkv=2, D=128, rot=128, inter=False,
             page=64, heads_first=True, first=32000, offset=0),
        # a prompt of 8192 tokens of three sequences; bandwidth
        dict(name="append prompt 8192", op="append", T=8192, n_seq=3, Hq=16, Hkv=2, D=128, rot=128, inter=False,
             page=64, heads_first=True, first=0, offset=0),
        # odd count, D = 64, half of each head rotated in interleaved pairs,
        # small pages laid out position by position, behind a shared prefix
        dict(name="append odd 1021", op="append", T=1021, n_seq=7, Hq=24, Hkv=8, D=64, rot=32, inter=True,
             page=16, heads_first=False, first=5, offset=131072),
        # one sequence, a thousand positions of its own; latency
        dict(name="attend 1 of 1000", op="attend", B=1, Hq=16, Hkv=2, D=128, page=64, heads_first=True, prefix=0,
             lo=1000, hi=1000),
        # a ragged batch of long sequences that share nothing; bandwidth
        dict(name="attend 8 to 32768", op="attend", B=8, Hq=16, Hkv=2, D=128, page=64, heads_first=True, prefix=0,
             lo=50, hi=32768),
        # 32 sequences behind a shared prefix of 32K, small pages, odd ends
        dict(name="attend 32 prefix 32749", op="attend", B=32, Hq=16, Hkv=2, D=128, page=16, heads_first=False,
             prefix=32749, lo=1, hi=600),
        # the largest: 128 sequences behind 128K shared positions
        dict(name="attend 128 prefix 131072", op="attend", B=128, Hq=16, Hkv=2, D=128, page=64, heads_first=True,
             prefix=131072, lo=1, hi=512),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "append", "attend"))
    if op == "linear":
        group = rng.choice(GROUPS)
        K = group * max(1, _log_int(rng, 128, 4096) // group)
        N = _log_int(rng, 16, 131072)
        return dict(op=op, B=_log_int(rng, 1, 64), K=K, N=N, group=group, fp32=rng.random() < 0.3)
    D = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    Hq = Hkv * rng.randint(1, 8)
    page = rng.choice((16, 32, 64, 128, 256))
    heads_first = rng.random() < 0.5
    if op == "append":
        T = _log_int(rng, 1, 8192)
        return dict(op=op, T=T, n_seq=rng.randint(1, min(T, 16)), Hq=Hq, Hkv=Hkv, D=D,
                    rot=rng.choice((0, D // 4, D // 2, D)), inter=rng.random() < 0.5, page=page,
                    heads_first=heads_first, first=_log_int(rng, 1, 40000) - 1,
                    offset=rng.choice((0, _log_int(rng, 1, 1000000))))
    # at most the largest listed case's products and cache
    while True:
        B = _log_int(rng, 1, 128)
        prefix = 0 if rng.random() < 0.3 else _log_int(rng, 1, 131072)
        hi = _log_int(rng, 1, 32768)
        rows = B * Hq * (prefix + hi) * D
        own_bytes = B * Hkv * hi * D * 4
        if rows <= 128 * 16 * 131072 * 128 and own_bytes + prefix * Hkv * D * 4 <= 1 << 28:
            break
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, heads_first=heads_first, prefix=prefix,
                lo=rng.randint(0 if prefix else 1, hi), hi=hi)


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(g, *shape, std=1.0):
    return torch.empty(*shape, device="cuda", dtype=torch.float32).normal_(0.0, std, generator=g).to(torch.bfloat16)


def _pool(g, case, n_pages, filled):
    """One page pool [n_pages][Hkv][page][D] (a view of position-major memory
    unless heads_first)."""
    a, b = (case["Hkv"], case["page"]) if case["heads_first"] else (case["page"], case["Hkv"])
    p = _bf16(g, n_pages, a, b, case["D"]) if filled else torch.zeros(n_pages, a, b, case["D"], device="cuda",
                                                                      dtype=torch.bfloat16)
    return p if case["heads_first"] else p.transpose(1, 2)


def _lengths(case):
    """The sequences' own lengths: spread evenly over [lo, hi] in a mixed order."""
    n, lo, hi = case["B"], case["lo"], case["hi"]
    return [lo + (hi - lo) * ((7 * i + n - 1) % n) // max(1, n - 1) if n > 1 else hi for i in range(n)]


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "linear":
        B, K, N, G = case["B"], case["K"], case["N"], case["group"]
        pitch = (K // G + 7) // 8 * 8
        q = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g, device="cuda", dtype=torch.int32)
        # weights ~ N(0, 0.02): a group's range is about 4.5 sigma over 15 steps
        s = (torch.rand(N, K // G, generator=g, device="cuda") * 0.004 + 0.004).to(torch.bfloat16)
        b = (-7.5 * s.float() + 0.004 * (torch.rand(N, K // G, generator=g, device="cuda") - 0.5)).to(torch.bfloat16)
        sp = torch.zeros(N, pitch, device="cuda", dtype=torch.bfloat16)
        bp = torch.zeros(N, pitch, device="cuda", dtype=torch.bfloat16)
        sp[:, :K // G] = s
        bp[:, :K // G] = b
        st = dict(case=case, q=q, s=sp.view(torch.int16), b=bp.view(torch.int16), x=_bf16(g, B, K))
        st["y"] = torch.empty(B, N, device="cuda", dtype=torch.float32 if case["fp32"] else torch.bfloat16)
        if own:
            from int4_grouped_gemm_gb300 import moe
            st["w"] = moe.QMatrix(st["q"], st["s"], st["b"], N, K, G)
        return st
    if case["op"] == "append":
        T, S, Hq, Hkv, D, page = (case[n] for n in ("T", "n_seq", "Hq", "Hkv", "D", "page"))
        cpu = torch.Generator().manual_seed(seed)
        # the tokens of sequence s are [s T / S, (s + 1) T / S), from position
        # first + 3 s on
        bounds = [s * T // S for s in range(S + 1)]
        seq = torch.cat([torch.full((bounds[s + 1] - bounds[s],), s, dtype=torch.int32) for s in range(S)])
        index = torch.cat([torch.arange(bounds[s + 1] - bounds[s], dtype=torch.int32) + case["first"] + 3 * s
                           for s in range(S)])
        ld = int(index.max()) // page + 1
        # the pages that the tokens touch, shuffled; a sequence's earlier pages
        # are of no concern here and share one
        touched = sorted({(int(a), int(b) // page) for a, b in zip(seq.tolist(), index.tolist())})
        order = (torch.randperm(len(touched), generator=cpu) + 1).tolist()
        table = torch.zeros(S, ld, dtype=torch.int32)
        for (s, p), n in zip(touched, order):
            table[s, p] = n
        st = dict(case=case, kp=_pool(g, case, len(touched) + 1, False), vp=_pool(g, case, len(touched) + 1, False),
                  seq=seq.cuda(), index=index.cuda(), table=table.cuda())
        # queries, keys and values are columns of one projection's output
        qkv = _bf16(g, T, (Hq + 2 * Hkv) * D)
        st["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        st["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        st["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        st["q_out"] = torch.empty(T, Hq, D, device="cuda", dtype=torch.bfloat16)
        rot = case["rot"]
        st["inv_freq"] = None if rot == 0 else \
            (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
        if own:
            from int4_grouped_gemm_gb300 import attention
            st["cache"] = attention.PagedCache(st["kp"], st["vp"])
        return st
    B, Hq, Hkv, D, page = (case[n] for n in ("B", "Hq", "Hkv", "D", "page"))
    cpu = torch.Generator().manual_seed(seed)
    lens = _lengths(case)
    n_prefix = -(-case["prefix"] // page)
    n_own = [-(-n // page) for n in lens]
    total = n_prefix + sum(n_own) + 1
    perm = torch.randperm(total, generator=cpu).to(torch.int32)
    table = torch.zeros(B, max(1, max(n_own)), dtype=torch.int32)
    at = n_prefix
    for b in range(B):
        table[b, :n_own[b]] = perm[at:at + n_own[b]]
        at += n_own[b]
    st = dict(case=case, kp=_pool(g, case, total, True), vp=_pool(g, case, total, True), table=table.cuda(),
              prefix_pages=perm[:n_prefix].cuda() if n_prefix else None,
              lens=torch.tensor(lens, dtype=torch.int32).cuda(), q=_bf16(g, B, Hq, D), scale=1.0 / math.sqrt(D))
    st["out"] = torch.empty(B, Hq, D, device="cuda", dtype=torch.bfloat16)
    if own:
        from int4_grouped_gemm_gb300 import attention
        st["cache"] = attention.PagedCache(st["kp"], st["vp"])
        st["ws"] = st["cache"].workspace(B, Hq, case["prefix"])
    return st


# ------------------------------------------------------------ one pass through

def run(st):
    case = st["case"]
    if own:
        if case["op"] == "linear":
            from int4_grouped_gemm_gb300 import moe
            return moe.linear(st["w"], st["x"], st["y"])
        if case["op"] == "append":
            st["cache"].append(st["q"], st["k"], st["v"], st["seq"], st["index"], st["table"], st["inv_freq"],
                               pos_offset=case["offset"], interleaved=case["inter"], q_out=st["q_out"])
            return dict(q=st["q_out"], k=st["kp"], v=st["vp"])
        return st["cache"].attend(st["q"], st["table"], st["lens"], st["prefix_pages"], case["prefix"],
                                  scale=st["scale"], out=st["out"], ws=st["ws"])
    return {"linear": _linear, "append": _append, "attend": _attend}[case["op"]](st)


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


def _append(st):
    case = st["case"]
    rot, page = case["rot"], case["page"]

    def turn(x):
        x = x.float()
        if rot == 0:
            return x
        ang = (st["index"].double() + case["offset"])[:, None] * st["inv_freq"].double()
        c, s = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
        if case["inter"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            both = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            both = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
        return torch.cat((both, x[..., rot:]), dim=-1)

    at = st["index"].long()
    pages = st["table"][st["seq"].long(), at // page].long()
    st["q_out"].copy_(turn(st["q"]))
    st["kp"][pages, :, at % page] = turn(st["k"]).to(torch.bfloat16)
    st["vp"][pages, :, at % page] = st["v"]
    return dict(q=st["q_out"], k=st["kp"], v=st["vp"])


def _attend(st):
    case = st["case"]
    B, Hq, Hkv, D, page = (case[n] for n in ("B", "Hq", "Hkv", "D", "page"))
    P, G, n = case["prefix"], Hq // Hkv, case["hi"]
    q = st["q"].float().view(B, Hkv, G, D)

    # own pages, padded to the longest sequence: [B][Hkv][n][D]
    at = torch.arange(n, device="cuda")
    pages = st["table"].long()[:, at // page]
    off = (at % page).expand(B, n)
    k = st["kp"][pages, :, off].float().permute(0, 2, 1, 3)
    v = st["vp"][pages, :, off].float().permute(0, 2, 1, 3)
    s = (q @ k.transpose(2, 3)) * st["scale"]
    s = s.masked_fill(at >= st["lens"].view(B, 1, 1, 1), -math.inf)
    if not P:
        m = s.amax(-1, keepdim=True)
        e = (s - m).exp()
        o = (e @ v) / e.sum(-1, keepdim=True)
    else:
        at = torch.arange(P, device="cuda")
        pages = st["prefix_pages"].long()[at // page]
        pk = st["kp"][pages, :, at % page].float().transpose(0, 1)
        pv = st["vp"][pages, :, at % page].float().transpose(0, 1)
        qp = q.transpose(0, 1).reshape(Hkv, B * G, D)
        sp = (qp @ pk.transpose(1, 2)) * st["scale"]
        sp = sp.view(Hkv, B, G, P).transpose(0, 1)
        m = torch.maximum(sp.amax(-1, keepdim=True), s.amax(-1, keepdim=True))
        e, ep = (s - m).exp(), (sp - m).exp()
        num = (ep.transpose(0, 1).reshape(Hkv, B * G, P) @ pv).view(Hkv, B, G, D).transpose(0, 1) + e @ v
        o = num / (e.sum(-1, keepdim=True) + ep.sum(-1, keepdim=True))
    st["out"].copy_(o.reshape(B, Hq, D))
    return st["out"]


# ---------------------------------------------------------- work and 64 bits

def work(case):
    if case["op"] == "linear":
        B, K, N, G = case["B"], case["K"], case["N"], case["group"]
        return dict(bytes=N * K // 2 + 4 * N * (K // G) + 2 * B * K + (4 if case["fp32"] else 2) * B * N,
                    flops=2 * B * N * K)
    if case["op"] == "append":
        T, Hq, Hkv, D = (case[n] for n in ("T", "Hq", "Hkv", "D"))
        return dict(bytes=T * D * 4 * (Hq + 2 * Hkv) + 12 * T, flops=3 * T * (Hq + Hkv) * case["rot"])
    B, Hq, Hkv, D = (case[n] for n in ("B", "Hq", "Hkv", "D"))
    n = sum(_lengths(case))
    return dict(bytes=4 * Hkv * D * (case["prefix"] + n) + 4 * B * Hq * D + 4 * (n + case["prefix"]) // case["page"],
                flops=4 * Hq * D * (n + B * case["prefix"]))


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
    if case["op"] == "append":
        rot = case["rot"]
        pos = (st["index"].to(torch.int64) + case["offset"]).to(d)

        def spin(x):
            y = x.to(d).clone()
            for i in range(rot // 2):
                f = st["inv_freq"][i].to(d)
                c, s = torch.cos(pos * f)[:, None], torch.sin(pos * f)[:, None]
                i0, i1 = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)
                a, b = x[..., i0].to(d), x[..., i1].to(d)
                y[..., i0] = a * c - b * s
                y[..., i1] = a * s + b * c
            return y

        kp, vp = st["kp"].to(d), st["vp"].to(d)
        page = torch.div(st["index"], case["page"], rounding_mode="floor").long()
        slot = (st["index"] - page * case["page"]).long()
        where = st["table"].long()[st["seq"].long(), page]
        k = spin(st["k"])
        for h in range(case["Hkv"]):
            kp[where, h, slot] = k[:, h]
            vp[where, h, slot] = st["v"][:, h].to(d)
        return dict(q=spin(st["q"]), k=kp, v=vp)
    B, Hq, Hkv, D, page = (case[n] for n in ("B", "Hq", "Hkv", "D", "page"))
    G, P = Hq // Hkv, case["prefix"]
    lens = _lengths(case)
    out = torch.zeros(B, Hq, D, device="cuda", dtype=d)
    for h in range(Hkv):
        k0 = v0 = torch.zeros(0, D, device="cuda", dtype=d)
        if P:
            k0 = st["kp"][st["prefix_pages"].long(), h].reshape(-1, D)[:P].to(d)
            v0 = st["vp"][st["prefix_pages"].long(), h].reshape(-1, D)[:P].to(d)
        for b in range(B):
            own_pages = st["table"][b, :-(-lens[b] // page)].long()
            k = torch.cat((k0, st["kp"][own_pages, h].reshape(-1, D)[:lens[b]].to(d)))
            v = torch.cat((v0, st["vp"][own_pages, h].reshape(-1, D)[:lens[b]].to(d)))
            rows = slice(h * G, (h + 1) * G)
            p = torch.softmax(st["q"][b, rows].to(d) @ k.t() * st["scale"], dim=-1)
            out[b, rows] = p @ v
    return out
