"""Cases of the operators around the int4 output head: what is measured and what it has to give.

Five operators, in the order in which a decoding step runs them:

* ``norm``    the final root-mean-square norm with the residual's addition,
              whose output is the head's hidden state;
* ``norm8``   the same norm with an output in 8 bits, one scale per row, the
              activations of an int4 linear layer;
* ``linear``  8-bit activations times packed int4 weights, with scales, bias,
              activation and residual in the epilogue;
* ``apply``   penalties for repeated tokens, biases and grammar masks on the
              head's logits, written out for a sampler of the caller's own;
* ``select``  the same rules with the verification of drafted tokens behind
              them: argmax, top-k, log-sum-exp, draft probabilities and the
              accepted count, straight from the logits.

``run`` computes the plain forms with elementary torch operations, or, where
``own`` is true, calls the library's entry points.
"""
import math

import torch

own = False

# Sizes: H = 5120, V = 151936, 18992 (one of eight shards) and 8192 (the draft
# vocabulary) are the output head's own; T <= 16 positions per request and 64
# requests x T = 4 are its verify blocks and its batch.


def listed():
    return [
        # the final norm of one wide verify block, in front of the head
        dict(name="norm_block16", op="norm", M=16, H=5120, dtype="float16", residual=True),
        # the norm of a long chunk of prompt tokens of a bfloat16 model
        dict(name="norm_prefill", op="norm", M=4096, H=8192, dtype="bfloat16", residual=True),
        # one token's norm into a quantised linear layer: latency counts
        dict(name="norm8_single", op="norm8", M=1, H=5120, dtype="float16", residual=True, channel=True),
        # a ragged chunk of prompt tokens into a quantised linear layer
        dict(name="norm8_ragged", op="norm8", M=1021, H=5120, dtype="bfloat16", residual=True, channel=True),
        # a verify block through a square projection: the weights' stream
        dict(name="linear_block16", op="linear", M=16, N=5120, K=5120, dtype="float16", act="silu", bias=True,
             out_scales=True, residual=False),
        # 64 requests x T = 4 through a layer of a shard's width
        dict(name="linear_batch256", op="linear", M=256, N=18992, K=5120, dtype="float16", act="none", bias=False,
             out_scales=True, residual=False),
        # a chunk of prompt tokens, back onto the residual stream
        dict(name="linear_prefill", op="linear", M=4096, N=5120, K=8192, dtype="bfloat16", act="none", bias=True,
             out_scales=True, residual=True),
        # one request's single token, every rule: the logits go to the caller's sampler
        dict(name="apply_single", op="apply", R=1, T=1, V=151936, history=2048, bias=64, mask=True, penal=True),
        # 64 requests x T = 4, half of the rows under a grammar
        dict(name="apply_batch", op="apply", R=64, T=4, V=151936, history=1024, bias=16, mask=True, penal=True),
        # greedy single decode over the draft vocabulary: latency counts
        dict(name="select_draft_vocab", op="select", R=1, T=1, V=8192, history=512, bias=0, mask=False, penal=True,
             top_k=0, sampled=False, temperature=1.0),
        # a wide verify block of a 25000-token request, top-16 sampling
        dict(name="select_block16", op="select", R=1, T=16, V=151936, history=25000, bias=32, mask=True, penal=True,
             top_k=16, sampled=True, temperature=0.7),
        # 64 requests x T = 4, top-16 sampling
        dict(name="select_batch", op="select", R=64, T=4, V=151936, history=1024, bias=16, mask=True, penal=True,
             top_k=16, sampled=True, temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm8", "linear", "apply", "select"])
    if op in ("norm", "norm8"):
        c = dict(op=op, M=_log_int(rng, 1, 4096), H=_log_int(rng, 32, 8192),
                 dtype=rng.choice(["float16", "bfloat16"]), residual=rng.random() < 0.7)
        if op == "norm8":
            c["channel"] = rng.random() < 0.5
        return c
    if op == "linear":
        return dict(op=op, M=_log_int(rng, 1, 4096), N=_log_int(rng, 16, 5120), K=32 * _log_int(rng, 1, 256),
                    dtype=rng.choice(["float16", "bfloat16", "float32"]),
                    act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.5,
                    out_scales=rng.random() < 0.5, residual=rng.random() < 0.5)
    T = rng.randint(1, 16)
    c = dict(op=op, R=_log_int(rng, 1, 256 // T if T > 4 else 64), T=T, V=_log_int(rng, 1000, 151936),
             history=_log_int(rng, 1, 1024), bias=rng.choice([0, 1, 16, 64]), mask=rng.random() < 0.6,
             penal=rng.random() < 0.8)
    if op == "select":
        c["sampled"] = rng.random() < 0.7
        c["top_k"] = rng.choice([0, 1, 5, 8, 16]) if c["sampled"] else 0
        c["temperature"] = rng.choice([0.6, 0.8, 1.0, 1.3])
    return c


# ---------------------------------------------------------------- inputs

def _dtype(case):
    return getattr(torch, case["dtype"])


def _prepare_norm(case, g, dev):
    M, H, dt = case["M"], case["H"], _dtype(case)
    # a residual stream: a few channels are far larger than the rest
    spread = torch.exp(0.5 * torch.randn(H, generator=g, device=dev))
    s = dict(x=(torch.randn(M, H, generator=g, device=dev) * spread).to(dt),
             weight=(1.0 + 0.2 * torch.randn(H, generator=g, device=dev)).to(dt), eps=1e-6, residual=None,
             channel_scales=None)
    if case["residual"]:
        s["residual"] = (3.0 * torch.randn(M, H, generator=g, device=dev) * spread).to(dt)
    if case.get("channel"):
        # the head's recipe for per-channel scales: lognormal(-4, 0.5)
        s["channel_scales"] = torch.exp(-4.0 + 0.5 * torch.randn(H, generator=g, device=dev)).to(torch.float16)
    return s


def _prepare_linear(case, g, dev):
    M, N, K = case["M"], case["N"], case["K"]
    codes = (42.0 * torch.randn(M, K, generator=g, device=dev)).round().clamp(-127, 127).to(torch.int8)
    q = torch.randint(-7, 8, (N, K), generator=g, device=dev, dtype=torch.int8)
    packed = ((q[:, 0::2] & 15) | ((q[:, 1::2] & 15) << 4)).view(torch.uint8)
    s = dict(codes=codes, row_scales=torch.exp(-7.0 + 0.3 * torch.randn(M, generator=g, device=dev)), packed=packed,
             out_scales=None, bias=None, residual=None, act=case["act"], out_dtype=_dtype(case))
    if case["out_scales"]:
        s["out_scales"] = torch.exp(-1.0 + 0.3 * torch.randn(N, generator=g, device=dev))
    if case["bias"]:
        s["bias"] = (0.5 * torch.randn(N, generator=g, device=dev)).to(_dtype(case))
    if case["residual"]:
        s["residual"] = torch.randn(M, N, generator=g, device=dev).to(_dtype(case))
    return s


def _prepare_logits(case, g, dev):
    R, T, V = case["R"], case["T"], case["V"]
    M = R * T
    s = dict(R=R, T=T, V=V, logits=2.5 * torch.randn(M, V, generator=g, device=dev), history=None, offsets=None,
             n_prompt=None, repetition=None, frequency=None, presence=None, bias_ids=None, bias_values=None,
             bias_offsets=None, mask=None, mask_index=None, drafts=None, draft_probs=None, uniforms=None)
    # a row's likely tokens stand out, as a model's do
    top = torch.randint(0, V, (M, 8), generator=g, device=dev)
    s["logits"].scatter_add_(1, top, 9.0 + 2.0 * torch.randn(M, 8, generator=g, device=dev))
    likely = s["logits"].topk(min(V, 8), dim=1).indices.view(R, T, -1)
    if T > 1:
        # most drafts agree with the row's best token, the others are near it
        pick = (torch.rand(R, T - 1, 1, generator=g, device=dev) ** 4 * likely.shape[2]).long()
        s["drafts"] = likely[:, : T - 1].gather(2, pick)[..., 0].to(torch.int32).contiguous()
        if case.get("sampled"):
            s["draft_probs"] = 0.2 + 0.8 * torch.rand(R, T - 1, generator=g, device=dev)
            s["uniforms"] = torch.rand(R, T - 1, generator=g, device=dev)
    if case["penal"]:
        # ragged histories (a prompt, then generated tokens) of unequal words,
        # some of them the rows' likely tokens
        n = 1 + (torch.rand(R, generator=g, device=dev) * case["history"]).long()
        if R == 1:
            n[:] = case["history"]
        s["offsets"] = torch.zeros(R + 1, dtype=torch.int64, device=dev)
        s["offsets"][1:] = n.cumsum(0)
        total = R * (1 + case["history"])
        words = (V * torch.rand(total, generator=g, device=dev) ** 4).long().clamp(max=V - 1)
        words[::7] = likely.reshape(-1)[torch.randint(0, likely.numel(), (len(words[::7]),), generator=g, device=dev)]
        s["history"] = words.to(torch.int32)
        s["n_prompt"] = (0.7 * n).to(torch.int32)
        s["repetition"] = 1.0 + 0.3 * torch.rand(R, generator=g, device=dev)
        s["frequency"] = 0.5 * torch.rand(R, generator=g, device=dev)
        s["presence"] = 0.5 * torch.rand(R, generator=g, device=dev)
    if case["bias"]:
        nb = case["bias"]
        # distinct ids of each request: one in each of nb stretches of the vocabulary
        at = torch.arange(nb, device=dev) * (V // nb) + torch.randint(0, V // nb, (R, nb), generator=g, device=dev)
        s["bias_ids"] = at.to(torch.int32).reshape(-1)
        s["bias_values"] = 4.0 * torch.randn(R * nb, generator=g, device=dev)
        s["bias_offsets"] = nb * torch.arange(R + 1, device=dev)
    if case["mask"]:
        # a grammar allows some thousands of tokens; every second row is free
        n = max(1, (M + 1) // 2)
        words = (V + 31) // 32
        bits = torch.randint(-2 ** 31, 2 ** 31, (3, n, words), generator=g, device=dev)
        s["mask"] = (bits[0] & bits[1] & bits[2]).to(torch.int32)
        rows = torch.arange(M, device=dev)
        s["mask_index"] = torch.where(rows % 2 == 0, rows // 2, -1).to(torch.int32)
    return s


def prepare(case, seed):
    dev = torch.device("cuda:0" if torch.cuda.is_available() else "cpu")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    kind = {"norm": _prepare_norm, "norm8": _prepare_norm, "linear": _prepare_linear}.get(case["op"], _prepare_logits)
    s = kind(case, g, dev)
    s["op"] = case["op"]
    for k in ("top_k", "sampled", "temperature"):
        if k in case:
            s[k] = case[k]
    return s


# ---------------------------------------------------------------- plain forms

def _norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + s["eps"])
    out = dict(hidden=(h * rstd * s["weight"].float()).to(torch.float16))
    if s["residual"] is not None:
        out["sum"] = h.to(s["x"].dtype)
    return out


def _norm8(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + s["eps"])
    t = h * s["weight"].float()
    if s["channel_scales"] is not None:
        t = t * s["channel_scales"].float()
    peak = t.abs().amax(dim=1, keepdim=True)
    codes = torch.round(t * (127.0 / peak)).to(torch.int8)
    row_scales = peak * rstd / 127.0
    out = dict(values=torch.mul(codes, row_scales.to(s["x"].dtype)), row_scales=row_scales[:, 0])
    if s["residual"] is not None:
        out["sum"] = h.to(s["x"].dtype)
    return out


def _linear(s):
    w = s["packed"].to(torch.int32)
    q = torch.stack((w & 15, w >> 4), dim=2).view(w.shape[0], -1)
    q = torch.where(q > 7, q - 16, q).float()
    # whole numbers: every partial sum is below 2^24, exact in 32 bits
    y = (s["codes"].float() @ q.T) * s["row_scales"][:, None]
    if s["out_scales"] is not None:
        y = y * s["out_scales"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if s["act"] == "relu":
        y = y.clamp(min=0)
    elif s["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif s["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["out_dtype"])


def _ruled(s):
    """The logits [R*T, V] under the rules, in 32 bits."""
    R, T, V = s["R"], s["T"], s["V"]
    x = s["logits"].view(R, T, V)
    if s["history"] is not None:
        dev = x.device
        total = s["history"].shape[0]
        place = torch.arange(total, device=dev)
        request = torch.bucketize(place, s["offsets"][1:], right=True)
        live = request < R
        request = request.clamp(max=R - 1)
        key = request * V + s["history"]
        generated = place >= s["offsets"][request] + s["n_prompt"][request]
        seen = torch.zeros(R * V, device=dev).index_add_(0, key, live.float()).view(R, 1, V)
        count = torch.zeros(R * V, device=dev).index_add_(0, key, (live & generated).float()).view(R, 1, V)
        if T > 1:
            # position t also counts the drafts in front of it
            before = torch.arange(T, device=dev)[:, None] > torch.arange(T - 1, device=dev)
            key = (torch.arange(R * T, device=dev).view(R, T, 1) * V + s["drafts"][:, None, :]).reshape(-1)
            extra = before.expand(R, T, T - 1).reshape(-1).float()
            count = count + torch.zeros(R * T * V, device=dev).index_add_(0, key, extra).view(R, T, V)
        penalty = torch.where((seen > 0) | (count > 0), s["repetition"].view(R, 1, 1), 1.0)
        x = torch.where(x > 0, x / penalty, x * penalty)
        x = x - s["frequency"].view(R, 1, 1) * count
        x = x - torch.where(count > 0, s["presence"].view(R, 1, 1), 0.0)
    if s["bias_ids"] is not None:
        per = s["bias_ids"].shape[0] // R
        request = torch.arange(R, device=x.device).repeat_interleave(per)
        table = torch.zeros(R * V, device=x.device).index_add_(0, request * V + s["bias_ids"], s["bias_values"])
        x = x + table.view(R, 1, V)
    x = x.reshape(R * T, V)
    if s["mask"] is not None:
        tokens = torch.arange(V, device=x.device)
        words = s["mask"][s["mask_index"].clamp(min=0)][:, tokens // 32]
        allowed = (((words >> (tokens % 32)) & 1) > 0) | (s["mask_index"] < 0)[:, None]
        x = torch.where(allowed, x, -math.inf)
    return x


def _select(s):
    R, T, V, k = s["R"], s["T"], s["V"], s["top_k"]
    x = _ruled(s)
    out = dict(logits_max=x.amax(dim=1), argmax_ids=x.argmax(dim=1).to(torch.int32))
    if k:
        order = torch.sort(x, dim=1, descending=True, stable=True)
        out["topk_logits"], out["topk_ids"] = order.values[:, :k].contiguous(), order.indices[:, :k].to(torch.int32)
    if s["sampled"]:
        z = (out["topk_logits"] if k else x).double() / s["temperature"]
        peak = z.amax(dim=1, keepdim=True)
        total = torch.exp(z - peak).sum(dim=1, keepdim=True)
        if not k:
            out["lse"] = (peak + torch.log(total))[:, 0].float()
    n = torch.zeros(R, dtype=torch.int32, device=x.device)
    if T > 1:
        if s["sampled"]:
            d = s["drafts"].long()
            rows = torch.arange(R * T, device=x.device).view(R, T)[:, : T - 1]
            p = torch.exp(x[rows, d].double() / s["temperature"] - peak[rows, 0]) / total[rows, 0]
            if k:
                among = (out["topk_ids"].view(R, T, k)[:, : T - 1] == s["drafts"][..., None]).any(dim=2)
                p = torch.where(among, p, 0.0)
            out["p_draft"] = p.float()
            accepted = s["uniforms"] * s["draft_probs"] < p
        else:
            accepted = out["argmax_ids"].view(R, T)[:, : T - 1] == s["drafts"]
        n = accepted.int().cumprod(dim=1).sum(dim=1).to(torch.int32)
    out["n_accepted"] = n
    return out


def run(s):
    if own:
        return _run_own(s)
    return {"norm": _norm, "norm8": _norm8, "linear": _linear, "apply": _ruled, "select": _select}[s["op"]](s)


# ---------------------------------------------------------------- the library's calls

def _run_own(s):
    from int4_output_head_amd import binding

    if s["op"] == "norm":
        got = binding.rms_norm(s["x"], s["weight"], s["residual"], eps=s["eps"], out_dtype=torch.float16)
        return dict(hidden=got) if s["residual"] is None else dict(hidden=got[0], sum=got[1])
    if s["op"] == "norm8":
        got = binding.rms_norm_int8(s["x"], s["weight"], s["residual"], eps=s["eps"],
                                    channel_scales=s["channel_scales"])
        # what the codes stand for, in the type of the rows that they replace
        out = dict(values=torch.mul(got[0], got[1].to(s["x"].dtype)[:, None]), row_scales=got[1])
        if s["residual"] is not None:
            out["sum"] = got[2]
        return out
    if s["op"] == "linear":
        return binding.linear_int4(s["codes"], s["row_scales"], s["packed"], out_scales=s["out_scales"],
                                   bias=s["bias"], activation=None if s["act"] == "none" else s["act"],
                                   residual=s["residual"], out_dtype=s["out_dtype"])
    rules = binding.LogitRules(history=s["history"], history_offsets=s["offsets"], n_prompt=s["n_prompt"],
                               repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                               bias_ids=s["bias_ids"], bias_values=s["bias_values"], bias_offsets=s["bias_offsets"],
                               mask=s["mask"], mask_index=s["mask_index"])
    if s["op"] == "apply":
        return binding.apply_logit_rules(s["logits"], rules, s["drafts"], R=s["R"])
    lmax, amax, tids, tlog, pdr, nacc, lse = binding.verify_logits(
        s["logits"], rules, s["drafts"], s["draft_probs"], s["uniforms"], R=s["R"], top_k=s["top_k"],
        temperature=s["temperature"], want_lse=s["sampled"] and not s["top_k"])
    out = dict(logits_max=lmax, argmax_ids=amax, n_accepted=nacc)
    if s["top_k"]:
        out["topk_logits"], out["topk_ids"] = tlog, tids
    elif s["sampled"]:
        out["lse"] = lse
    if s["T"] > 1 and s["sampled"]:
        out["p_draft"] = pdr
    return out


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] in ("norm", "norm8"):
        M, H = case["M"], case["H"]
        rows = 4 if case["residual"] else 2            # x and the output, the residual and the sum: 2 bytes each
        per = 2 * rows - (1 if case["op"] == "norm8" else 0)
        return dict(bytes=M * H * per + 2 * H * (2 if case.get("channel") else 1), flops=6 * M * H)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        size = 4 if case["dtype"] == "float32" else 2
        return dict(bytes=N * K // 2 + M * K + M * N * size * (2 if case["residual"] else 1) + 4 * (M + 2 * N),
                    flops=2 * M * N * K)
    M, V = case["R"] * case["T"], case["V"]
    b = 4 * M * V
    if case["penal"]:
        b += case["R"] * case["history"] * (4 if case["R"] == 1 else 2)
    if case["mask"]:
        b += (M + 1) // 2 * ((V + 31) // 32) * 4
    b += 8 * case["R"] * case["bias"]
    if case["op"] == "apply":
        b += 4 * M * V
    else:
        b += M * (16 + 8 * case["top_k"])
    return dict(bytes=b, flops=6 * M * V)


# ---------------------------------------------------------------- 64 bits

def _exact_norm(case, s):
    h = s["x"].double()
    if s["residual"] is not None:
        h = h + s["residual"].double()
    root = torch.linalg.vector_norm(h, dim=1, keepdim=True) / math.sqrt(h.shape[1])
    y = h / torch.hypot(root, torch.full_like(root, math.sqrt(s["eps"]))) * s["weight"].double()
    kept = h if s["residual"] is not None else None
    if case["op"] == "norm":
        return dict(hidden=y, sum=kept)
    if s["channel_scales"] is not None:
        y = y * s["channel_scales"].double()
    step = torch.linalg.vector_norm(y, ord=math.inf, dim=1, keepdim=True) / 127
    return dict(values=torch.round(y / step) * step, row_scales=step[:, 0], sum=kept)


def _exact_linear(case, s):
    u = s["packed"].long()
    low, high = ((u % 16 + 8) % 16 - 8).double(), ((u // 16 + 8) % 16 - 8).double()
    c = s["codes"].double()
    y = c[:, 0::2] @ low.T.contiguous() + c[:, 1::2] @ high.T.contiguous()
    y = y * s["row_scales"].double()[:, None]
    if s["out_scales"] is not None:
        y = y * s["out_scales"].double()
    if s["bias"] is not None:
        y = y + s["bias"].double()
    y = {"none": lambda v: v, "relu": lambda v: torch.where(v > 0, v, 0.0), "silu": lambda v: v * torch.sigmoid(v),
         "gelu": lambda v: v * torch.special.ndtr(v)}[s["act"]](y)
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_rows(s):
    """The logits under the rules in 64 bits, row by row."""
    R, T, V = s["R"], s["T"], s["V"]
    rows = s["logits"].double()
    at = s["offsets"].tolist() if s["offsets"] is not None else None
    for i in range(R):
        for t in range(T):
            x = rows[i * T + t]
            if at is not None:
                words = s["history"][at[i]: at[i + 1]].long()
                made = words[int(s["n_prompt"][i]):]
                if t:
                    made = torch.cat((made, s["drafts"][i, :t].long()))
                count = torch.bincount(made, minlength=V).double()
                known = torch.bincount(torch.cat((words, made)), minlength=V) > 0
                r = s["repetition"][i].double()
                x[known] = torch.where(x[known] > 0, x[known] / r, x[known] * r)
                x -= s["frequency"][i].double() * count + s["presence"][i].double() * (count > 0)
            if s["bias_ids"] is not None:
                span = slice(int(s["bias_offsets"][i]), int(s["bias_offsets"][i + 1]))
                x[s["bias_ids"][span].long()] += s["bias_values"][span].double()
            if s["mask"] is not None and int(s["mask_index"][i * T + t]) >= 0:
                word = s["mask"][int(s["mask_index"][i * T + t])].long() & 0xFFFFFFFF
                bits = (word[:, None] // 2 ** torch.arange(32, device=x.device)) % 2
                x[bits.reshape(-1)[:V] == 0] = -math.inf
    return rows


def _exact_select(case, s):
    R, T, k = s["R"], s["T"], s["top_k"]
    x = _exact_rows(s)
    out = dict(logits_max=x.max(dim=1).values, argmax_ids=None, n_accepted=None)
    if k:
        best = x.topk(k, dim=1)
        out["topk_logits"], out["topk_ids"] = best.values, None
    if s["sampled"]:
        z = x / s["temperature"]
        if not k:
            out["lse"] = torch.logsumexp(z, dim=1)
        if T > 1:
            if k:
                z = torch.full_like(z, -math.inf).scatter_(1, best.indices, best.values / s["temperature"])
            p = torch.softmax(z, dim=1).view(R, T, -1)[:, : T - 1]
            out["p_draft"] = p.gather(2, s["drafts"].long()[..., None])[..., 0]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm8"):
        return {k: v for k, v in _exact_norm(case, s).items() if v is not None}
    if case["op"] == "linear":
        return _exact_linear(case, s)
    if case["op"] == "apply":
        return _exact_rows(s)
    return _exact_select(case, s)
