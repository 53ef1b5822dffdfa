"""The per-request operators around the LM head and the expert layer: what they compute, on which inputs, and how they are called.

adapters -- low-rank adapters of many requests beside a shared projection:
    y[t] = base[t] + scale[a] * B_a (A_a x[t])    with a = adapter[t];  y[t] = base[t] where a = -1
logits -- penalties for repeated tokens, biases and grammar masks on logits, and the greedy token of what is left:
    s = seen at all in the row's history,  c = times generated in it
    l1 = l / rep if l > 0 else l * rep   (where s)
    l2 = (l1 - freq * c) - pres          (where c > 0)
    l3 = l2 + bias                       (where the row lists one)
    out = l3 where the row's mask has the token's bit, else -inf
    token = argmax (lowest index on ties, -1 where nothing is left),  lse = log(sum(exp(out)))
"""
import math

import torch

own = False

NEG = float("-inf")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    A, L = "adapters", "logits"
    return [
        # one sequence's decode step: its adapter beside the expert layer (hidden 2048); latency
        dict(name="adapters_decode_t1", op=A, T=1, H=2048, N=2048, r=16, n=8, type="bf16", ids="mixed", pad=0),
        # a decode batch of 64 sequences, each with an adapter of its own choice or none
        dict(name="adapters_decode_t64", op=A, T=64, H=2048, N=2048, r=16, n=64, type="bf16", ids="mixed", pad=0),
        # eight sequences' adapters on the LM head (131072 x 2048), the widest product there is
        dict(name="adapters_head_t8", op=A, T=8, H=2048, N=131072, r=16, n=8, type="fp16", ids="mixed", pad=0),
        # a prompt of 947 tokens batched from the prompts of a few requests
        dict(name="adapters_prompt_t947", op=A, T=947, H=2048, N=2048, r=64, n=4, type="fp16", ids="runs", pad=0),
        # odd sizes: a ragged batch in a wider buffer, an odd number of outputs, 32-bit weights
        dict(name="adapters_odd_t333", op=A, T=333, H=768, N=1001, r=24, n=16, type="fp32", ids="mixed", pad=8),
        # the largest prefill: 16384 tokens of many requests in one pass
        dict(name="adapters_prompt_t16384", op=A, T=16384, H=2048, N=2048, r=64, n=8, type="bf16", ids="runs", pad=0),
        # one sequence after a 947-token prompt: penalties, greedy token and its log-probability; latency
        dict(name="logits_t1", op=L, T=1, V=131072, hist=1000, bias=0, masks=0, want="pick", pad=0),
        # a decode batch with everything on; the processed logits go to a sampler
        dict(name="logits_t64", op=L, T=64, V=131072, hist=2000, bias=64, masks=8, want="both", pad=0),
        # long contexts: the history is as long as a prompt of 16384 tokens
        dict(name="logits_long_t32", op=L, T=32, V=131072, hist=16384, bias=0, masks=0, want="out", pad=0),
        # odd sizes: a vocabulary that is no multiple of 32 in a wider buffer, short histories, many biases
        dict(name="logits_odd_t33", op=L, T=33, V=32003, hist=100, bias=300, masks=3, want="both", pad=5),
        # the largest batch, constrained decoding: masks for most rows
        dict(name="logits_t256", op=L, T=256, V=131072, hist=1000, bias=0, masks=32, want="both", pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        T = _log(rng, 1, 16384)
        H = 256 * rng.randint(1, 10)
        N = _log(rng, 16384, 131072) if T <= 16 and rng.random() < 0.5 else _log(rng, 200, 4000 if T <= 2048 else 2048)
        r = rng.choice([8, 16, 24, 32, 48, 64, 128])
        n = _log(rng, 1, 64)
        if T > 256:  # what the largest listed case costs bounds the products of long batches
            n = min(n, max(1, 512 * 16384 // (r * T)), 512 // r if T > 2048 else 64)
            H = min(H, 2048) if T > 2048 else H
        return dict(op="adapters", T=T, H=H, N=N, r=r, n=max(n, 1), type=rng.choice(["bf16", "fp16", "fp32"]),
                    ids=rng.choice(["mixed", "runs", "one"]), pad=rng.choice([0, 0, 4, 8]))
    T = _log(rng, 1, 256)
    V = _log(rng, 1000, 160000)
    if T * V > 256 * 131072:
        V = 256 * 131072 // T
    hist = rng.choice([0, _log(rng, 1, 16384 if T <= 32 else 2048)])
    return dict(op="logits", T=T, V=V, hist=hist, bias=rng.choice([0, _log(rng, 1, 300)]),
                masks=rng.choice([0, rng.randint(1, 32)]), want=rng.choice(["out", "both"] if T > 4 else ["out", "both", "pick"]), pad=rng.choice([0, 0, 1, 5, 8]))


def work(case):
    T = case["T"]
    if case["op"] == "adapters":
        H, N, r, size = case["H"], case["N"], case["r"], 4 if case["type"] == "fp32" else 2
        n = 1 if case["ids"] == "one" else case["n"]
        share = {"one": 1.0, "mixed": 0.85, "runs": (n + 1) / (n + 2)}[case["ids"]]  # of the tokens have an adapter
        used = 1 if case["ids"] == "one" else n * (1 - (1 - share / n) ** min(T, n + 2 if case["ids"] == "runs" else T))
        return {"bytes": 4 * T * (share * H + 2 * N + 1) + used * r * (H + N) * size, "flops": 2 * share * T * r * (H + N)}
    V = case["V"]
    moved = 4 * T * V * (2 if case["want"] in ("out", "both") else 1)
    moved += 4 * T * case["hist"] + 8 * T * case["bias"] + min(case["masks"], T) * ((V + 31) // 32) * 4
    return {"bytes": moved, "flops": T * V * (6 if case["want"] == "out" else 10)}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    kw = dict(device="cuda", generator=g)
    T, pad = case["T"], case["pad"]
    if case["op"] == "adapters":
        H, N, r, n, kind = case["H"], case["N"], case["r"], case["n"], TYPES[case["type"]]
        x = torch.randn(T, H + pad, **kw)[:, :H]
        base = torch.randn(T, N + pad, **kw)[:, :N]
        a = torch.empty(n, r, H, device="cuda", dtype=kind)
        b = torch.empty(n, N, r, device="cuda", dtype=kind)
        for i in range(n):
            a[i] = (torch.randn(r, H, **kw) / math.sqrt(H)).to(kind)
            b[i] = (torch.randn(N, r, **kw) * 0.05).to(kind)
        scale = torch.rand(n, **kw) * 3 + 0.5
        if case["ids"] == "one":
            ids = torch.randint(0, n, (1,), **kw).expand(T)
        elif case["ids"] == "mixed":  # each token its own choice; about one in seven has no adapter
            ids = torch.randint(0, n, (T,), **kw)
            ids = torch.where(torch.rand(T, **kw) < 0.15, -1, ids)
        else:  # requests' prompts one after another: a few runs of one adapter each, one of them without
            runs = n + 2
            cut = torch.sort(torch.randint(0, T, (runs - 1,), **kw)).values
            which = torch.randint(0, n, (runs,), **kw)
            which[0] = -1
            ids = which[torch.searchsorted(cut, torch.arange(T, device="cuda"), right=True)]
        return dict(op="adapters", x=x, base=base, a=a, b=b, scale=scale, adapter=ids.to(torch.int32).contiguous(),
                    y=torch.empty(T, N + pad, device="cuda")[:, :N])
    V = case["V"]
    logits = (torch.randn(T, V + pad, **kw) * 3)[:, :V]
    s = dict(op="logits", logits=logits, want=case["want"])
    if case["hist"]:
        # prompt and generated tokens, row after row: frequent tokens come again and again; some rows are empty
        lens = torch.randint(0, 2 * case["hist"] + 1, (T,), **kw)
        if T == 1:
            lens[:] = case["hist"]
        s["start"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(lens, 0)])
        total = int(s["start"][-1])
        s["tokens"] = (torch.rand(total, **kw) ** 4 * V).to(torch.int32).clamp_(max=V - 1)
        s["generated"] = s["start"][:-1] + (torch.rand(T, **kw) * lens).to(torch.int64)
        plain = torch.rand(T, **kw) < 0.3  # rows of requests that ask for none
        s["rep"] = torch.where(plain, 1.0, 1.0 + torch.rand(T, **kw) * 0.5)
        s["pres"] = torch.where(plain, 0.0, torch.rand(T, **kw))
        s["freq"] = torch.where(plain, 0.0, torch.rand(T, **kw) * 0.5)
    if case["bias"]:
        k = min(case["bias"], V // 2)
        tok = torch.stack([torch.randperm(V, **kw)[:k] for _ in range(T)])
        keep = torch.rand(T, 1, **kw) < 0.7
        cnt = torch.where(keep[:, 0], k, 0)
        s["bias_start"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(cnt, 0)])
        s["bias_token"] = tok[keep.expand_as(tok)].to(torch.int32)
        val = torch.randn(T, k, **kw) * 5
        val = torch.where(torch.rand(T, k, **kw) < 0.1, NEG, val)  # some tokens are banned outright
        s["bias_value"] = val[keep.expand_as(val)]
    if case["masks"]:
        # what each state of a grammar allows: nearly all, about half, a handful, and the last of several nothing at all
        m, W = case["masks"], (V + 31) // 32
        share = torch.rand(m, 1, **kw) ** 6
        share[0] = 0.9
        if m > 2:
            share[-1] = 0.0
        bits = torch.rand(m, W * 32, **kw) < share
        words = (bits.view(m, W, 32).to(torch.int64) << torch.arange(32, device="cuda")).sum(2)
        s["mask"] = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
        s["mask_row"] = torch.randint(-1, m, (T,), **kw).to(torch.int32)
    if case["want"] != "pick":
        s["out"] = torch.empty(T, V + pad, device="cuda")[:, :V]
    if case["want"] != "out":
        s["token"] = torch.empty(T, dtype=torch.int32, device="cuda")
        s["lse"] = torch.empty(T, device="cuda")
    return s


def run(state):
    if own:
        return _own(state)
    return _plain_adapters(state) if state["op"] == "adapters" else _plain_logits(state)


def _own(s):
    import quantized_moe_q4_b200 as m
    if s["op"] == "adapters":
        if "handle" not in s:  # a server's adapters and workspace outlive the calls
            s["handle"] = m.Adapters(s["a"], s["b"], s["scale"])
            s["ws"] = m.alloc_workspace(m.moe_q4_adapters_workspace_bytes(s["handle"], s["x"].shape[0]))
        return m.moe_q4_adapters_apply(s["handle"], s["x"], s["adapter"], base=s["base"], y=s["y"], workspace=s["ws"])
    # the histories grow and the masks change with each token, so the rules are put together for each step
    rules = m.LogitRules(tokens=s.get("tokens"), row_start=s.get("start"), generated_start=s.get("generated"),
                         repetition=s.get("rep"), presence=s.get("pres"), frequency=s.get("freq"),
                         bias_token=s.get("bias_token"), bias_value=s.get("bias_value"), bias_start=s.get("bias_start"),
                         mask=s.get("mask"), mask_row=s.get("mask_row"))
    m.moe_q4_logits_apply(rules, s["logits"], out=s.get("out"), token=s.get("token"), lse=s.get("lse"))
    return {k: s[k] for k in ("out", "token", "lse") if k in s}


def _plain_adapters(s):
    x, base, ids = s["x"], s["base"], s["adapter"]
    n, r, H = s["a"].shape
    T, N = base.shape
    if T <= n:  # few tokens: each with its own adapter's matrices
        e = ids.clamp(min=0).long()
        u = torch.bmm(s["a"][e].float(), x[:, :, None])
        d = torch.bmm(s["b"][e].float(), u)[:, :, 0] * s["scale"][e, None]
        return base + torch.where(ids[:, None] >= 0, d, 0.0)
    u = (x @ s["a"].float().view(n * r, H).t()).view(T, n, r)  # every adapter's product, then the token's own
    u = torch.where((ids[:, None] == torch.arange(n, device=x.device))[:, :, None], u * s["scale"][:, None], 0.0)
    return base + u.view(T, n * r) @ s["b"].float().permute(0, 2, 1).reshape(n * r, N)


def _plain_logits(s):
    l = s["logits"]
    T, V = l.shape
    row = torch.arange(T, device=l.device)
    if "tokens" in s:
        at = torch.arange(s["tokens"].numel(), device=l.device)
        of = torch.repeat_interleave(row, s["start"][1:] - s["start"][:-1], output_size=at.numel())
        flat = of * V + s["tokens"]
        seen = torch.zeros(T * V, dtype=torch.int32, device=l.device).index_fill_(0, flat, 1).view(T, V) > 0
        made = (at >= s["generated"][of]).int()
        c = torch.zeros(T * V, dtype=torch.int32, device=l.device).scatter_add_(0, flat, made).view(T, V)
        rep = s["rep"][:, None]
        l = torch.where(seen, torch.where(l > 0, l / rep, l * rep), l)
        l = torch.where(c > 0, (l - s["freq"][:, None] * c) - s["pres"][:, None], l)
    if "bias_token" in s:
        of = torch.repeat_interleave(row, s["bias_start"][1:] - s["bias_start"][:-1], output_size=s["bias_token"].numel())
        bias = torch.zeros(T * V, device=l.device).index_copy_(0, of * V + s["bias_token"], s["bias_value"]).view(T, V)
        l = l + bias
    if "mask" in s:
        bits = (s["mask"][:, :, None] >> torch.arange(32, dtype=torch.int32, device=l.device)) & 1
        allowed = bits.view(s["mask"].shape[0], -1)[:, :V] > 0
        m = s["mask_row"]
        l = torch.where(allowed[m.clamp(min=0).long()] | (m < 0)[:, None], l, NEG)
    got = {}
    if s["want"] != "pick":
        got["out"] = l
    if s["want"] != "out":
        top = l.amax(1, keepdim=True)
        first = torch.where(l == top, torch.arange(V, device=l.device), V).amin(1)
        got["token"] = torch.where(top[:, 0] == NEG, -1, first).to(torch.int32)
        shift = torch.where(torch.isinf(top), 0.0, top)
        got["lse"] = torch.log(torch.exp(l - shift).sum(1)) + shift[:, 0]
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adapters":
        y = s["base"].double()
        for e in range(case["n"]):
            at = torch.nonzero(s["adapter"] == e)[:, 0]
            if at.numel():
                u = s["x"][at].double() @ s["a"][e].double().t()
                y[at] += s["scale"][e].double() * (u @ s["b"][e].double().t())
        return y
    outs, lses = [], []
    for t in range(case["T"]):
        l = s["logits"][t].double()
        if case["hist"]:
            lo, mid, hi = int(s["start"][t]), int(s["generated"][t]), int(s["start"][t + 1])
            every = torch.bincount(s["tokens"][lo:hi].long(), minlength=case["V"])
            made = torch.bincount(s["tokens"][mid:hi].long(), minlength=case["V"])
            rep, pres, freq = (float(s[k][t]) for k in ("rep", "pres", "freq"))
            l = torch.where(every == 0, l, torch.where(l > 0, l / rep, l * rep))
            l = l - freq * made - pres * (made > 0)
        if case["bias"]:
            lo, hi = int(s["bias_start"][t]), int(s["bias_start"][t + 1])
            l[s["bias_token"][lo:hi].long()] += s["bias_value"][lo:hi].double()
        if case["masks"] and int(s["mask_row"][t]) >= 0:
            words = s["mask"][int(s["mask_row"][t])].long() & 0xFFFFFFFF
            i = torch.arange(case["V"], device=l.device)
            l[(words[i // 32] >> (i % 32)) % 2 == 0] = NEG
        outs.append(l)
        lses.append(torch.logsumexp(l, 0))
    got = {}
    if case["want"] != "pick":
        got["out"] = torch.stack(outs)
    if case["want"] != "out":
        got["token"] = None
        got["lse"] = torch.stack(lses)
    return got
