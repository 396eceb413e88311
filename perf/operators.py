"""What is measured of the operators around a projection: residual addition
with root-mean-square norm, low-rank adapters of many requests beside a shared
projection, and log probabilities of given tokens.

``run`` computes an operator in its plain form (elementary torch operations in
float32), or, with ``own`` true, through the library's binding.
"""
import math

import torch

own = False

BF16, F32, E4M3 = "bf16", "f32", "e4m3"
DTYPE = {BF16: torch.bfloat16, F32: torch.float32, E4M3: torch.float8_e4m3fn}
BYTES = {BF16: 2, F32: 4, E4M3: 1}
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
EPS = 1e-6


def listed():
    return [
        # one decoded token of a small model: the shortest call there is
        norm("norm_token", T=1, H=2048, x=BF16, res=BF16, y=BF16),
        # a decode batch whose 8-bit consumer takes a scale for each 128 columns
        norm("norm_decode_e4m3", T=64, H=4096, x=BF16, res=BF16, y=E4M3, group=128),
        # an fp32 projection's output on an fp32 residual stream, an odd width
        norm("norm_odd_f32", T=777, H=1409, x=F32, res=F32, y=BF16, w=F32),
        # a prompt batch with one scale a token
        norm("norm_prompt_e4m3", T=8192, H=4096, x=BF16, res=BF16, y=E4M3),
        # one decoded token of one request with an adapter
        adapters("adapter_token", T=1, cols=4096, rows=4096, n=8, rank=16),
        # a decode batch: a token a request, requests of 32 adapters in any order
        adapters("adapter_decode", T=64, cols=2048, rows=5632, n=32, rank=64, requests=64, mixed=True),
        # short prompts, odd widths and rank, some without an adapter, bf16 output
        adapters("adapter_odd", T=517, cols=1409, rows=1003, n=6, rank=12, requests=9, y=BF16),
        # a prompt batch of eight requests beside the widest projection
        adapters("adapter_prompt", T=4096, cols=4096, rows=14336, n=4, rank=64, requests=8),
        # one sampled token with its five best alternatives
        logprobs("logprob_token", T=1, V=32000, z=F32, top=5),
        # a decode batch of 16-bit logits with 20 alternatives
        logprobs("logprob_decode", T=64, V=128009, z=BF16, top=20),
        # constrained decoding: most of the vocabulary masked, in some rows all of it
        logprobs("logprob_masked", T=333, V=50021, z=F32, top=8, masked=True),
        # scoring a prompt batch's own tokens
        logprobs("logprob_prompt", T=4096, V=128000, z=F32),
    ]


def norm(name, T, H, x, res, y, w=BF16, group=0, pad=0):
    """T rows of H; x, res, w, y: types; group: columns a scale (0: the row);
    pad: unused elements behind each row of x."""
    return dict(name=name, op="norm", T=T, H=H, x=x, res=res, w=w, y=y, group=group, pad=pad)


def adapters(name, T, cols, rows, n, rank, requests=1, mixed=False, y=F32):
    """T tokens of `requests` requests (a request's tokens one after the
    other) beside a rows x cols projection; n adapters of at most `rank`
    (mixed: ranks differ); from four requests on, every fourth has none."""
    return dict(name=name, op="adapters", T=T, cols=cols, rows=rows, n=n, rank=rank, requests=requests, mixed=mixed, y=y)


def logprobs(name, T, V, z, top=0, masked=False, pad=0):
    """T rows of V logits; top: alternatives; masked: one in 50 tokens allowed,
    and one row in 16 with none."""
    return dict(name=name, op="logprobs", T=T, V=V, z=z, top=top, masked=masked, pad=pad)


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))

    def width(lo, hi):                       # a multiple of 128, of 8, or any
        return max(lo, size(lo, hi) // (m := rng.choice((128, 8, 1))) * m)

    op = rng.choice(("norm", "adapters", "logprobs"))
    if op == "norm":
        H = width(64, 14336)
        c = norm(None, T=size(1, min(16384, 8192 * 4096 // H)), H=H, x=rng.choice((BF16, F32)), res=rng.choice((BF16, F32)),
                 w=rng.choice((BF16, F32)), y=rng.choice((BF16, E4M3)), pad=rng.choice((0, 0, 8, 3)))
        c["group"] = rng.choice((0, 128)) if c["y"] == E4M3 else 0
    elif op == "adapters":
        cols, rows = width(64, 14336), width(64, 14336)
        T = size(1, min(4096, 4096 * (4096 + 4 * 14336) // (cols + 4 * rows)))
        decode = T <= 256 and rng.random() < 0.6
        rank = rng.choice((4, 8, 12, 16, 32, 64))
        c = adapters(None, T=T, cols=cols, rows=rows, n=size(1, min(64, 1024 // rank)), rank=rank,
                     requests=T if decode else size(1, min(T, 32)), mixed=rng.random() < 0.5, y=rng.choice((F32, F32, BF16)))
    else:
        V = width(500, 256000)
        top = rng.choice((0, 1, 5, 20))
        c = logprobs(None, T=size(1, min(4096, (64 << 20 if top else 4096 * 128000) // V)), V=V, z=rng.choice((F32, BF16)), top=top,
                     masked=rng.random() < 0.25, pad=rng.choice((0, 0, 8, 3)))
    del c["name"]
    return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _rows(g, T, n, pad, dtype, std=1.0):
    t = torch.empty((T, n + pad), dtype=dtype, device="cuda").normal_(0.0, std, generator=g)
    return t[:, :n] if pad else t


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s["x"] = _rows(g, T, H, case["pad"], DTYPE[case["x"]])
        s["res"] = _rows(g, T, H, 0, DTYPE[case["res"]], 4.0)
        s["w"] = torch.empty(H, dtype=DTYPE[case["w"]], device="cuda").normal_(1.0, 0.2, generator=g)
    elif case["op"] == "adapters":
        T, n, r, q = case["T"], case["n"], case["rank"], case["requests"]
        s["x"] = _rows(g, T, case["cols"], 0, torch.bfloat16)
        s["a"] = _rows(g, n * r, case["cols"], 0, torch.bfloat16, case["cols"] ** -0.5).view(n, r, -1)
        s["b"] = _rows(g, n * case["rows"], r, 0, torch.bfloat16, 0.2).view(n, -1, r)
        s["scale"] = torch.empty(n, device="cuda").uniform_(0.5, 2.0, generator=g)
        s["ranks"] = _ranks(case).cuda()
        s["base"] = _rows(g, T, case["rows"], 0, DTYPE[case["y"]])
        # requests take the adapters in turn, in a shuffled order; a request
        # has at least one token, the rest fall to requests at random
        of_request = torch.arange(q, device="cuda") % n
        if q >= 4:
            of_request[3::4] = -1
        of_request = of_request[torch.randperm(q, generator=g, device="cuda")]
        cuts = torch.randperm(T - 1, generator=g, device="cuda")[: q - 1] + 1 if T > 1 else torch.empty(0, dtype=torch.long, device="cuda")
        starts = torch.zeros(T, dtype=torch.long, device="cuda")
        starts[cuts] = 1
        s["ids"] = of_request[starts.cumsum(0)].to(torch.int32)
    else:
        T, V = case["T"], case["V"]
        z = _rows(g, T, V, case["pad"], DTYPE[case["z"]], 2.5)
        s["tokens"] = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        likely = torch.randint(0, V, (T,), generator=g, device="cuda")
        peak = torch.empty(T, device="cuda").uniform_(0.0, 24.0, generator=g)
        z[torch.arange(T, device="cuda"), likely] = peak.to(z.dtype)
        half = torch.rand(T, generator=g, device="cuda") < 0.5
        s["tokens"] = torch.where(half, likely.to(torch.int32), s["tokens"])
        if case["masked"]:
            for r in range(0, T, 512):
                allowed = torch.rand((min(512, T - r), V), generator=g, device="cuda") < 0.02
                allowed[15::16] = False
                z[r:r + 512].masked_fill_(~allowed, -math.inf)
        s["z"] = z
    return s


def _ranks(case):
    r = [max(1, case["rank"] >> (i % 3)) if case["mixed"] else case["rank"] for i in range(case["n"])]
    return torch.tensor(r, dtype=torch.int32)


def run(s):
    return {"norm": _run_norm, "adapters": _run_adapters, "logprobs": _run_logprobs}[s["case"]["op"]](s)


def _run_norm(s):
    c = s["case"]
    if own:
        from any_precision_weight_pw_b200 import binding
        y, scales, res = binding.add_rms_norm(s["x"], s["w"], EPS, residual=s["res"], y_type=DTYPE[c["y"]], scale_group=c["group"])
        return (y, res) if scales is None else (y, scales, res)
    h = s["x"].float() + s["res"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["w"].float()
    res = h.to(s["res"].dtype)
    if c["y"] == BF16:
        return y.to(torch.bfloat16), res
    T, H = y.shape
    n = -(-H // c["group"]) if c["group"] else 1
    per = c["group"] or H
    groups = torch.nn.functional.pad(y, (0, n * per - H)).view(T, n, per)
    scales = (groups.abs().amax(2) / E4M3_MAX).clamp(min=SCALE_MIN)
    q = (groups / scales[:, :, None]).to(torch.float8_e4m3fn).view(T, n * per)[:, :H]
    return q, scales, res


def _run_adapters(s):
    if own:
        from any_precision_weight_pw_b200 import binding
        return binding.add_adapters(s["x"], s["a"], s["b"], s["ids"], base=s["base"], scale=s["scale"], ranks=s["ranks"])
    n, r, cols = s["a"].shape
    # the products with every adapter, those of a token's own kept
    v = (s["x"].float() @ s["a"].float().view(n * r, cols).t()).view(-1, n, r)
    keep = (s["ids"][:, None] == torch.arange(n, device="cuda"))[:, :, None] & (torch.arange(r, device="cuda") < s["ranks"][:, None])
    v = torch.where(keep, v * s["scale"][:, None], 0.0).view(-1, n * r)
    y = s["base"].float() + v @ s["b"].float().transpose(1, 2).reshape(n * r, -1)
    return y.to(s["base"].dtype)


def _run_logprobs(s):
    c = s["case"]
    if own:
        from any_precision_weight_pw_b200 import binding
        lp, ent, idx, top = binding.token_logprobs(s["z"], s["tokens"], n_top=c["top"])
        return (lp, ent) if idx is None else (lp, ent, idx, top)
    z = s["z"].float()
    m = z.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    d = z - m
    e = torch.exp(d)
    total = e.sum(1)
    norm = m[:, 0] + torch.log(total)
    lp = z.gather(1, s["tokens"].long()[:, None])[:, 0]
    lp = torch.where(lp == -math.inf, lp, lp - norm)
    ent = torch.log(total) - torch.where(e > 0, e * d, 0.0).sum(1) / total
    ent = torch.where(total > 0, ent, 0.0)
    if not c["top"]:
        return lp, ent
    top, idx = torch.sort(z, dim=1, descending=True, stable=True)
    top = top[:, : c["top"]]
    top = torch.where(top == -math.inf, top, top - norm[:, None])
    return lp, ent, idx[:, : c["top"]].to(torch.int32), top


def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        scales = (-(-H // case["group"]) if case["group"] else 1) if case["y"] == E4M3 else 0
        return {"bytes": T * H * (BYTES[case["x"]] + 2 * BYTES[case["res"]] + BYTES[case["y"]]) + 4 * T * scales + H * BYTES[case["w"]],
                "flops": 7 * T * H}
    if case["op"] == "adapters":
        T, q = case["T"], case["requests"]
        with_one = [i % case["n"] for i in range(q) if q < 4 or i % 4 != 3]
        ranks = _ranks(case).tolist()
        used = sum(ranks[i] for i in set(with_one))
        mean = sum(ranks[i] for i in with_one) / q
        return {"bytes": 2 * T * case["cols"] + 2 * T * case["rows"] * BYTES[case["y"]] + 2 * used * (case["cols"] + case["rows"]) + 4 * T,
                "flops": 2 * T * mean * (case["cols"] + case["rows"])}
    T, V = case["T"], case["V"]
    return {"bytes": T * V * BYTES[case["z"]] + T * (12 + 8 * case["top"]), "flops": 6 * T * V}


def exact(case, seed):
    """The definitions in float64, a slice of the rows at a time."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "adapters":
        return _exact_adapters(case, s)
    return _exact_logprobs(case, s)


def _exact_norm(case, s):
    ys, scales, res = [], [], []
    for x, r in zip(s["x"].split(1024), s["res"].split(1024)):
        h = x.double().add(r.double())
        y = h.div((h.square().sum(-1) / case["H"] + EPS).sqrt()[:, None]).mul(s["w"].double())
        res.append(h)
        if case["y"] == E4M3:
            parts = y.split(case["group"] or case["H"], dim=1)
            top = torch.stack([p.abs().max(1).values for p in parts], 1).div(E4M3_MAX).clamp(min=SCALE_MIN)
            y = torch.cat([p / top[:, i:i + 1] for i, p in enumerate(parts)], 1)
            scales.append(top)
        ys.append(y)
    out = [torch.cat(ys)] + ([torch.cat(scales)] if scales else []) + [torch.cat(res)]
    return tuple(out)


def _exact_adapters(case, s):
    y = s["base"].double()
    ids, ranks = s["ids"].tolist(), _ranks(case).tolist()
    for i in sorted(set(ids) - {-1}):
        rows = torch.tensor([t for t, k in enumerate(ids) if k == i], device="cuda")
        r = ranks[i]
        v = torch.einsum("tc,rc->tr", s["x"][rows].double(), s["a"][i, :r].double())
        y[rows] += float(s["scale"][i]) * torch.einsum("tr,or->to", v, s["b"][i, :, :r].double())
    return y


def _exact_logprobs(case, s):
    lps, ents, idxs, tops = [], [], [], []
    for z, t in zip(s["z"].split(256), s["tokens"].split(256)):
        z = z.double()
        lp = torch.log_softmax(z, 1)
        lp = torch.where(z == -math.inf, z, lp)             # a row with nothing allowed: all -inf
        p = lp.exp()
        lps.append(lp[torch.arange(len(z), device="cuda"), t.long()])
        ents.append(-torch.where(p > 0, p * lp, 0.0).sum(1))
        if case["top"]:
            order = torch.argsort(z, dim=1, descending=True, stable=True)[:, : case["top"]]
            idxs.append(order.to(torch.int32))
            tops.append(torch.gather(lp, 1, order))
    out = [torch.cat(lps), torch.cat(ents)]
    return tuple(out + ([torch.cat(idxs), torch.cat(tops)] if case["top"] else []))
