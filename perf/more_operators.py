"""Cases of a decoding step's operators with 4-bit floating-point layers and a sampler: what is measured and what it
has to give.

* ``block``   the norm behind a block, its gate and scale, the residual's addition and the next block's norm, whose
              output is the next layer's input in 16 bits or, as ``block8``, in 8 bits with one scale per row;
* ``mx``      rows rounded to microscaled 4-bit floating point (one power of two for 32 channels) and read back;
* ``linear``  the product of two matrices in that format, with bias, activation and residual in the epilogue;
* ``sample``  a token of every row drawn by a given uniform number at a temperature, among the top k, the top p and
              those above min p, under the rules of a request; drafted tokens verified with the same distribution.

``run`` computes the plain forms with elementary torch operations, or, where ``own`` is true, calls the library's
entry points.
"""
import math

import torch

own = False

# Sizes: H = 5120 and 8192, V = 151936 and 8192 (the draft vocabulary), up to 16 positions per request and 64 requests
# x 4 are those of the output head's own workloads and of the norm and linear layers in front of it.


def listed():
    return [
        # one token between two blocks: latency counts
        dict(name="block_single", op="block", M=1, H=5120, dtype="float16", post=True, gate="channel", act="none",
             scale=1.0),
        # a long chunk of prompt tokens of a bfloat16 model with a gate of every element
        dict(name="block_prefill", op="block", M=4096, H=8192, dtype="bfloat16", post=True, gate="element",
             act="sigmoid", scale=1.0),
        # a ragged chunk into an 8-bit linear layer
        dict(name="block8_ragged", op="block8", M=1021, H=5120, dtype="bfloat16", post=True, gate="none", act="none",
             scale=0.22, channel=True),
        # the activations of one verify block
        dict(name="mx_block16", op="mx", M=16, H=5120, dtype="float16"),
        # the activations of a long chunk of prompt tokens, or a weight matrix
        dict(name="mx_prefill", op="mx", M=4096, H=8192, dtype="bfloat16"),
        # a verify block through a square projection: the weights' stream
        dict(name="linear_block16", op="linear", M=16, N=5120, K=5120, dtype="float16", act="silu", bias=True,
             residual=False),
        # 64 requests x T = 4 through a layer of a vocabulary shard's width
        dict(name="linear_batch256", op="linear", M=256, N=18992, K=5120, dtype="float16", act="none", bias=False,
             residual=False),
        # a chunk of prompt tokens, back onto the residual stream
        dict(name="linear_prefill", op="linear", M=4096, N=5120, K=8192, dtype="bfloat16", act="none", bias=True,
             residual=True),
        # one draft token over the draft vocabulary at a temperature: latency counts
        dict(name="sample_draft_vocab", op="sample", R=1, T=1, V=8192, dtype="float32", history=0, mask=False,
             mixed=False, temperature=0.8, top_k=0, top_p=1.0, min_p=0.0),
        # one request's token, penalised for repetition, with the usual top-k and top-p
        dict(name="sample_single", op="sample", R=1, T=1, V=151936, dtype="float32", history=2048, mask=False,
             mixed=False, temperature=0.7, top_k=50, top_p=0.95, min_p=0.0),
        # a wide verify block of copied drafts, nucleus sampling
        dict(name="sample_block16", op="sample", R=1, T=16, V=151936, dtype="float32", history=0, mask=False,
             mixed=False, temperature=0.9, top_k=0, top_p=0.9, min_p=0.02),
        # 64 requests x T = 4, each with settings of its own, half of the rows under a grammar
        dict(name="sample_batch", op="sample", R=64, T=4, V=151936, dtype="float32", history=1024, mask=True,
             mixed=True, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["block", "block8", "mx", "linear", "sample"])
    if op in ("block", "block8"):
        c = dict(op=op, M=_log_int(rng, 1, 4096), H=_log_int(rng, 32, 8192),
                 dtype=rng.choice(["float16", "bfloat16"]), post=rng.random() < 0.7,
                 gate=rng.choice(["none", "channel", "element"]), act=rng.choice(["none", "sigmoid"]),
                 scale=rng.choice([1.0, 0.22]))
        if op == "block8":
            c["channel"] = rng.random() < 0.5
        return c
    if op == "mx":
        return dict(op=op, M=_log_int(rng, 1, 4096), H=32 * _log_int(rng, 1, 256),
                    dtype=rng.choice(["float16", "bfloat16"]))
    if op == "linear":
        return dict(op=op, M=_log_int(rng, 1, 4096), N=_log_int(rng, 16, 5120), K=32 * _log_int(rng, 1, 256),
                    dtype=rng.choice(["float16", "bfloat16", "float32"]),
                    act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    T = rng.randint(1, 16)
    return dict(op=op, R=_log_int(rng, 1, 256 // T if T > 4 else 64), T=T, V=_log_int(rng, 1000, 151936),
                dtype=rng.choice(["float32", "bfloat16"]), history=rng.choice([0, _log_int(rng, 1, 1024)]),
                mask=rng.random() < 0.5, mixed=rng.random() < 0.5, temperature=rng.choice([0.0, 0.6, 0.8, 1.0, 1.3]),
                top_k=rng.choice([0, 1, 20, 50]), top_p=rng.choice([0.5, 0.9, 0.95, 1.0]),
                min_p=rng.choice([0.0, 0.05]))


# ---------------------------------------------------------------- inputs

def _dtype(case):
    return getattr(torch, case["dtype"])


def _rows(g, dev, M, H, dt):
    # a residual stream: a few channels are far larger than the rest
    spread = torch.exp(0.5 * torch.randn(H, generator=g, device=dev))
    return (torch.randn(M, H, generator=g, device=dev) * spread).to(dt)


def _prepare_block(case, g, dev):
    M, H, dt = case["M"], case["H"], _dtype(case)
    s = dict(x=_rows(g, dev, M, H, dt), residual=3 * _rows(g, dev, M, H, dt), post=None, gate=None,
             pre=(1.0 + 0.2 * torch.randn(H, generator=g, device=dev)).to(dt), eps=1e-6, channel_scales=None)
    if case["post"]:
        s["post"] = (0.5 + 0.1 * torch.randn(H, generator=g, device=dev)).to(dt)
    if case["gate"] != "none":
        shape = (H,) if case["gate"] == "channel" else (M, H)
        s["gate"] = torch.randn(shape, generator=g, device=dev).to(dt)
    if case.get("channel"):
        # the head's recipe for per-channel scales: lognormal(-4, 0.5)
        s["channel_scales"] = torch.exp(-4.0 + 0.5 * torch.randn(H, generator=g, device=dev)).to(torch.float16)
    return s


def _prepare_linear(case, g, dev):
    M, N, K, dt = case["M"], case["N"], case["K"], _dtype(case)
    s = dict(bias=None, residual=None, out_dtype=dt)
    s["codes"], s["scales"] = _round_mx(_rows(g, dev, M, K, torch.float32))
    s["w"], s["w_scales"] = _round_mx(0.02 * torch.randn(N, K, generator=g, device=dev))
    if case["bias"]:
        s["bias"] = (0.5 * torch.randn(N, generator=g, device=dev)).to(dt)
    if case["residual"]:
        s["residual"] = torch.randn(M, N, generator=g, device=dev).to(dt)
    return s


def _prepare_sample(case, g, dev):
    R, T, V = case["R"], case["T"], case["V"]
    M = R * T
    s = dict(R=R, T=T, V=V, history=None, mask=None, mask_index=None, drafts=None, accept=None)
    # a row's likely tokens follow a power law, as a model's do, and the rest lies far below
    n = min(V, 512)
    x = 2.0 * torch.randn(M, V, generator=g, device=dev)
    # (one in each of n stretches of the vocabulary, their ranks in any order)
    likely = torch.arange(n, device=dev) * (V // n) + torch.randint(0, V // n, (M, n), generator=g, device=dev)
    rank = 1.0 + torch.argsort(torch.rand(M, n, generator=g, device=dev), dim=1)
    x.scatter_(1, likely, 18.0 - 1.3 * torch.log(rank) + 0.5 * torch.randn(M, n, generator=g, device=dev))
    s["logits"] = x.to(_dtype(case))
    s["uniforms"] = torch.rand(M, generator=g, device=dev)
    if T > 1:
        # most drafts agree with one of the row's best tokens
        best = s["logits"].float().topk(min(V, 8), dim=1).indices.view(R, T, -1)
        pick = (torch.rand(R, T - 1, 1, generator=g, device=dev) ** 4 * best.shape[2]).long()
        s["drafts"] = best[:, : T - 1].gather(2, pick)[..., 0].to(torch.int32).contiguous()
        s["accept"] = torch.rand(R, T - 1, generator=g, device=dev)
    if case["history"]:
        # ragged histories, some of their words the rows' likely tokens
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
        s["presence"] = 0.5 * torch.rand(R, generator=g, device=dev)
    if case["mask"]:
        # a grammar allows an eighth of the tokens; every second row is free
        n = max(1, (M + 1) // 2)
        bits = torch.randint(-2 ** 31, 2 ** 31, (3, n, (V + 31) // 32), generator=g, device=dev)
        s["mask"] = (bits[0] & bits[1] & bits[2]).to(torch.int32)
        rows = torch.arange(M, device=dev)
        s["mask_index"] = torch.where(rows % 2 == 0, rows // 2, -1).to(torch.int32)
    if case["mixed"]:
        # every request brings settings of its own
        def choice(*values):
            at = torch.randint(0, len(values), (R,), generator=g, device=dev)
            return torch.tensor(values, device=dev)[at]
        s["temperature"] = choice(0.0, 0.6, 0.8, 1.0, 1.0, 1.3)
        s["top_k"] = choice(0, 0, 1, 20, 50, 64).to(torch.int32)
        s["top_p"] = choice(0.5, 0.9, 0.95, 1.0)
        s["min_p"] = choice(0.0, 0.0, 0.05)
    else:
        for k in ("temperature", "top_k", "top_p", "min_p"):
            s[k] = case[k]
    return s


def prepare(case, seed):
    dev = torch.device("cuda:0" if torch.cuda.is_available() else "cpu")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    if case["op"] == "mx":
        s = dict(x=_rows(g, dev, case["M"], case["H"], _dtype(case)))
    else:
        s = {"linear": _prepare_linear, "sample": _prepare_sample}.get(case["op"], _prepare_block)(case, g, dev)
    s["op"] = case["op"]
    for k in ("act", "scale"):
        if k in case:
            s[k] = case[k]
    return s


# ---------------------------------------------------------------- plain forms

def _block(s):
    u = s["x"].float()
    if s["post"] is not None:
        u = u * (1.0 / torch.sqrt((u * u).mean(dim=1, keepdim=True) + s["eps"])) * s["post"].float()
    if s["gate"] is not None:
        gate = s["gate"].float()
        u = u * (1.0 / (1.0 + torch.exp(-gate)) if s["act"] == "sigmoid" else gate)
    h = s["residual"].float() + u * s["scale"]
    rstd = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + s["eps"])
    if s["op"] == "block":
        return dict(normed=(h * rstd * s["pre"].float()).to(torch.float16), sum=h.to(s["x"].dtype))
    t = h * s["pre"].float()
    if s["channel_scales"] is not None:
        t = t * s["channel_scales"].float()
    peak = t.abs().amax(dim=1, keepdim=True)
    codes = torch.round(t * (127.0 / peak)).to(torch.int8)
    row_scales = peak * rstd / 127.0
    return dict(values=torch.mul(codes, row_scales.to(s["x"].dtype)), row_scales=row_scales[:, 0],
                sum=h.to(s["x"].dtype))


def _round_mx(x):
    """Rows in microscaled 4 bits: two codes a byte (the even channel in the low half), and the exponents + 127."""
    v = x.float().view(x.shape[0], -1, 32)
    peak = v.abs().amax(dim=2, keepdim=True)
    # the exponent of the largest value, less that of the format's (4 = 2^2)
    e = (torch.frexp(peak)[1] - 3).clamp(-127, 127)
    e = torch.where(peak > 0, e, -127)
    t = torch.ldexp(v.double(), -e).float().abs()
    # 0, .5, 1, 1.5, 2, 3, 4, 6: ties go to the even code, beyond 6 stays 6
    code = ((t > 0.25).int() + (t >= 0.75).int() + (t > 1.25).int() + (t >= 1.75).int() + (t > 2.5).int()
            + (t >= 3.5).int() + (t > 5.0).int())
    code = (code + 8 * torch.signbit(v).int()).view(x.shape)
    return ((code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8), (e + 127).to(torch.uint8)[..., 0])


def _values_mx(codes, scales):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat((table, -table))
    v = table[torch.stack((codes & 15, codes >> 4), dim=2).long()]
    v = v.view(codes.shape[0], -1, 32).double()
    return torch.ldexp(v, scales.int()[..., None] - 127).float().view(codes.shape[0], -1)


def _mx(s):
    return _values_mx(*_round_mx(s["x"])).to(s["x"].dtype)


def _linear(s):
    y = _values_mx(s["codes"], s["scales"]) @ _values_mx(s["w"], s["w_scales"]).T
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
    x = s["logits"].float().view(R, T, V)
    if s["history"] is not None:
        dev = x.device
        place = torch.arange(s["history"].shape[0], device=dev)
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
        x = x - torch.where(count > 0, s["presence"].view(R, 1, 1), 0.0)
    x = x.reshape(R * T, V)
    if s["mask"] is not None:
        tokens = torch.arange(V, device=x.device)
        words = s["mask"][s["mask_index"].clamp(min=0)][:, tokens // 32]
        allowed = (((words >> (tokens % 32)) & 1) > 0) | (s["mask_index"] < 0)[:, None]
        x = torch.where(allowed, x, -math.inf)
    return x


def _settings(s, dev):
    """(temperature, top_k, top_p, min_p) of every row, the numbers as 32 bits hold them."""
    out = []
    for name, dt in (("temperature", torch.float32), ("top_k", torch.int64), ("top_p", torch.float32),
                     ("min_p", torch.float32)):
        v = s[name]
        v = v.to(dt) if isinstance(v, torch.Tensor) else torch.full((s["R"],), v, dtype=dt, device=dev)
        out.append(v.repeat_interleave(s["T"])[:, None])
    return out


def _sample(s):
    R, T, V = s["R"], s["T"], s["V"]
    x = _ruled(s)
    temperature, top_k, top_p, min_p = _settings(s, x.device)
    order = torch.sort(x, dim=1, descending=True, stable=True)
    sorted_x = order.values.double()
    # the mass of the tokens from the best to the worst, 1 for the best; without a temperature the best alone
    mass = torch.exp((sorted_x - sorted_x[:, :1]) / torch.where(temperature > 0, temperature, 1.0).double())
    rank = torch.arange(V, device=x.device)
    kept = (rank < torch.where(top_k > 0, top_k, V)) & ((temperature > 0) | (rank < 1))
    mass = torch.where(kept, mass, 0.0)
    before = mass.cumsum(dim=1) - mass
    kept = kept & ((before < top_p.double() * mass.sum(dim=1, keepdim=True)) | (top_p >= 1)) & (mass >= min_p.double())
    mass = torch.where(kept, mass, 0.0)
    mass = torch.zeros_like(mass).scatter_(1, order.indices, mass)     # by token again
    total = mass.sum(dim=1, keepdim=True)
    out = {}
    if T > 1:
        rows = torch.arange(R * T, device=x.device).view(R, T)[:, : T - 1].reshape(-1)
        d = s["drafts"].long().reshape(-1)
        p = (mass[rows, d] / total[rows, 0]).float().view(R, T - 1)
        out["p_draft"] = p
        out["n_accepted"] = (s["accept"] < p).int().cumprod(dim=1).sum(dim=1).to(torch.int32)
        # the token of a refused draft's place is another one
        mass[rows, d] = 0.0
        total = mass.sum(dim=1, keepdim=True)
    reached = mass.cumsum(dim=1) > s["uniforms"].double()[:, None] * total
    token = reached.int().argmax(dim=1)
    some = total[:, 0] > 0
    p = mass.gather(1, token[:, None])[:, 0] / total[:, 0]
    out["tokens"] = torch.where(some, token, -1).to(torch.int32)
    out["probs"] = torch.where(some, p, 0.0).float()
    return out


def run(s):
    if own:
        return _run_own(s)
    return {"block": _block, "block8": _block, "mx": _mx, "linear": _linear, "sample": _sample}[s["op"]](s)


# ---------------------------------------------------------------- the library's calls

def _run_own(s):
    from int4_output_head_amd import binding

    act = None if s.get("act") == "none" else s.get("act")
    if s["op"] in ("block", "block8") and s["gate"] is None:
        act = None                             # without a gate there is none to activate
    if s["op"] == "block":
        normed, total = binding.rms_norm_block(s["x"], s["residual"], s["post"], s["pre"], gate=s["gate"],
                                               gate_activation=act, scale=s["scale"], eps=s["eps"],
                                               out_dtype=torch.float16)
        return dict(normed=normed, sum=total)
    if s["op"] == "block8":
        codes, row_scales, total = binding.rms_norm_block_int8(s["x"], s["residual"], s["post"], s["pre"],
                                                               gate=s["gate"], gate_activation=act, scale=s["scale"],
                                                               channel_scales=s["channel_scales"], eps=s["eps"])
        # what the codes stand for, in the type of the rows that they replace
        return dict(values=torch.mul(codes, row_scales.to(s["x"].dtype)[:, None]), row_scales=row_scales, sum=total)
    if s["op"] == "mx":
        codes, scales = binding.quantize_mxfp4(s["x"])
        return binding.dequantize_mxfp4(codes, scales, out_dtype=s["x"].dtype)
    if s["op"] == "linear":
        return binding.linear_mxfp4(s["codes"], s["scales"], s["w"], s["w_scales"], bias=s["bias"], activation=act,
                                    residual=s["residual"], out_dtype=s["out_dtype"])
    rules = None
    if s["history"] is not None or s["mask"] is not None:
        rules = binding.LogitRules(history=s["history"], history_offsets=s.get("offsets"),
                                   n_prompt=s.get("n_prompt"), repetition=s.get("repetition"),
                                   presence=s.get("presence"), mask=s["mask"], mask_index=s["mask_index"])
    tokens, probs, p_draft, n_accepted = binding.sample_logits(
        s["logits"], s["uniforms"], rules, s["drafts"], R=s["R"], temperature=s["temperature"], top_k=s["top_k"],
        top_p=s["top_p"], min_p=s["min_p"], accept=s["accept"])
    out = dict(tokens=tokens, probs=probs)
    if s["T"] > 1:
        out["p_draft"], out["n_accepted"] = p_draft, n_accepted
    return out


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] in ("block", "block8"):
        M, H = case["M"], case["H"]
        per = 8 if case["op"] == "block" else 7        # x, residual, sum: 2 bytes each; the normed row 2, or 1
        if case["gate"] == "element":
            per += 2
        return dict(bytes=M * H * per + 2 * H * 3, flops=12 * M * H)
    if case["op"] == "mx":
        return dict(bytes=case["M"] * case["H"] * 4, flops=4 * case["M"] * case["H"])
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        size = 4 if case["dtype"] == "float32" else 2
        return dict(bytes=(N + M) * K * 17 // 32 + M * N * size * (2 if case["residual"] else 1) + N * size,
                    flops=2 * M * N * K)
    M, V = case["R"] * case["T"], case["V"]
    b = M * V * (4 if case["dtype"] == "float32" else 2) + 24 * M
    if case["history"]:
        b += case["R"] * case["history"] * (4 if case["R"] == 1 else 2)
    if case["mask"]:
        b += (M + 1) // 2 * ((V + 31) // 32) * 4
    return dict(bytes=b, flops=8 * M * V)


# ---------------------------------------------------------------- 64 bits

def _exact_block(case, s):
    def normed(v, weight):
        root = torch.linalg.vector_norm(v, dim=1, keepdim=True) / math.sqrt(v.shape[1])
        return v / torch.hypot(root, torch.full_like(root, math.sqrt(s["eps"]))) * weight.double()
    h = s["x"].double()
    if s["post"] is not None:
        h = normed(h, s["post"])
    if s["gate"] is not None:
        h = h * (torch.sigmoid(s["gate"].double()) if case["act"] == "sigmoid" else s["gate"].double())
    h = torch.add(s["residual"].double(), h, alpha=case["scale"])
    y = normed(h, s["pre"])
    if case["op"] == "block":
        return dict(normed=y, sum=h)
    if s["channel_scales"] is not None:
        y = y * s["channel_scales"].double()
    step = torch.linalg.vector_norm(y, ord=math.inf, dim=1, keepdim=True) / 127
    return dict(values=torch.round(y / step) * step, row_scales=step[:, 0], sum=h)


def _exact_mx(s):
    v = s["x"].double().unflatten(1, (-1, 32))
    step = torch.exp2((torch.floor(torch.log2(torch.linalg.vector_norm(v, ord=math.inf, dim=2, keepdim=True))) - 2
                       ).nan_to_num(neginf=-127.0).clamp(-127, 127))
    # steps of a half below 2, of 1 below 4 and of 2 above; torch.round goes to even
    t = (v / step).clamp(-6, 6)
    grain = torch.where(t.abs() < 2, 0.5, torch.where(t.abs() < 4, 1.0, 2.0))
    return (torch.round(t / grain) * grain * step).flatten(1)


def _exact_linear(case, s):
    def values(codes, scales):
        halves = torch.stack((codes % 16, codes // 16), dim=-1).flatten(1).double()
        size = halves % 8
        # the exponent's two bits and the mantissa's one
        e, m = torch.div(size, 2, rounding_mode="floor"), size % 2
        v = torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2) * torch.where(halves >= 8, -1.0, 1.0)
        return (v.unflatten(1, (-1, 32)) * torch.exp2(scales.double() - 127)[..., None]).flatten(1)
    y = torch.nn.functional.linear(values(s["codes"], s["scales"]), values(s["w"], s["w_scales"]))
    if s["bias"] is not None:
        y = y + s["bias"].double()
    y = {"none": lambda v: v, "relu": lambda v: torch.where(v > 0, v, 0.0), "silu": lambda v: v * torch.sigmoid(v),
         "gelu": lambda v: v * torch.special.ndtr(v)}[case["act"]](y)
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_rows(s):
    """The logits under the rules, row by row: in 32 bits, as the rules are defined, and then in 64."""
    R, T, V = s["R"], s["T"], s["V"]
    rows = s["logits"].float().clone()
    at = s["offsets"].tolist() if s["history"] is not None else None
    for i in range(R):
        for t in range(T):
            x = rows[i * T + t]
            if at is not None:
                words = s["history"][at[i]: at[i + 1]].long()
                made = words[int(s["n_prompt"][i]):]
                if t:
                    made = torch.cat((made, s["drafts"][i, :t].long()))
                known = torch.bincount(torch.cat((words, made)), minlength=V) > 0
                r = s["repetition"][i]
                x[known] = torch.where(x[known] > 0, x[known] / r, x[known] * r)
                x[torch.unique(made)] -= s["presence"][i]
            if s["mask"] is not None and int(s["mask_index"][i * T + t]) >= 0:
                word = s["mask"][int(s["mask_index"][i * T + t])].long() & 0xFFFFFFFF
                bits = (word[:, None] // 2 ** torch.arange(32, device=x.device)) % 2
                x[bits.reshape(-1)[:V] == 0] = -math.inf
    return rows.double()


def _exact_sample(case, s):
    R, T, V = s["R"], s["T"], s["V"]
    x = _exact_rows(s)
    settings = torch.cat([v.double() for v in _settings(s, x.device)], dim=1).tolist()
    probs = torch.zeros(R * T, dtype=torch.float64)
    p_draft = torch.zeros(R * T, dtype=torch.float64)
    for r, (temperature, k, top_p, min_p) in enumerate(settings):
        row = x[r]
        k = 1 if temperature == 0 else min(int(k) or V, V)
        at = torch.sort(row, descending=True, stable=True).indices[:k]
        if row[at[0]] == -math.inf:
            continue
        p = torch.softmax(row[at] / (temperature or 1.0), dim=0)
        if top_p < 1:
            n = 1 + int(torch.searchsorted(torch.cumsum(p, 0), torch.tensor(top_p, dtype=p.dtype, device=p.device)))
            at, p = at[:n], p[:n]
        good = p >= min_p * p[0]
        at, p = at[good], p[good]
        by_token = torch.argsort(at)
        at, p = at[by_token], p[by_token] / p.sum()
        if r % T < T - 1:
            other = at != s["drafts"][r // T, r % T]
            p_draft[r] = p[~other].sum()
            at, p = at[other], p[other]
        if len(p):
            c = torch.cumsum(p, 0)
            n = int(torch.searchsorted(c, s["uniforms"][r].double() * c[-1], right=True))
            probs[r] = p[min(n, len(p) - 1)] / c[-1]
    out = dict(tokens=None, probs=probs)
    if T > 1:
        out["p_draft"], out["n_accepted"] = p_draft.view(R, T)[:, : T - 1].contiguous(), None
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("block", "block8"):
        return _exact_block(case, s)
    if case["op"] == "mx":
        return _exact_mx(s)
    return _exact_linear(case, s) if case["op"] == "linear" else _exact_sample(case, s)
