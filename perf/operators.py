"""What a preference fine-tuning run over a frozen NF4 base spends its time on beside the layers' products.

Three operators, each in its plain form (elementary torch operations in 32 bits, 64 where 32 lose what matters) and
through this repository's own calls:

  decode   y = x W^T + s (x A^T) B^T for 1 to 16 tokens, W an NF4 weight (16 levels, blocks of 64 with a
           double-quantised absmax), one projection or all of a layer: the forward of a model that answers token by token;
  score    the log-probability of every sequence of a packed batch under its logits: the reference model's pass;
  train    the preference loss of chosen and rejected answers from the policy's logits, with the logits' gradient;
  clip     the norm of all adapter gradients together, and the gradients scaled down to a largest norm.
"""
import math
import random
from statistics import NormalDist

import torch

own = False

VOCAB = 151936          # the token embeddings of the smallest stack
LARGEST = 2048 * VOCAB  # logits of the largest listed batch
WEIGHTS = 8192 * 29568  # weights of the largest listed projection

# (hidden, kv, mlp) of decoder stacks, and their depth
STACKS = {"0.5b": (24, 896, 128, 4864), "3b": (36, 2048, 256, 11008), "8b": (32, 4096, 1024, 14336)}


def _layer(h, kv, m):
    """K, N and the index of the input of the seven projections: q, k and v read one input, gate and up another."""
    return [[h, h, 0], [h, kv, 0], [h, kv, 0], [h, h, 1], [h, m, 2], [h, m, 2], [m, h, 3]]


def _projs(case):
    return _layer(case["h"], case["kv"], case["m"]) if "h" in case else [[case["K"], case["N"], 0]]


def listed():
    _, h, kv, m = STACKS["8b"]
    return [
        # the smallest projection of the tests: launches and latency are all there is
        dict(name="decode 512x512", kind="decode", T=1, r=8, adapter=True, K=512, N=512),
        # one token through the 8B stack's attention projection
        dict(name="decode q 8B", kind="decode", T=1, r=16, adapter=True, K=h, N=h),
        # one token through a whole 8B layer, the step that a decode loop repeats for every layer
        dict(name="decode layer 8B", kind="decode", T=1, r=16, adapter=True, h=h, kv=kv, m=m),
        # eight sequences at once through the largest projection (72B down)
        dict(name="decode down 72B 8 tokens", kind="decode", T=8, r=16, adapter=True, K=29568, N=8192),
        # an odd number of tokens with the adapter off: the reference model's answers, 0.5B shapes
        dict(name="decode layer 0.5B 13 tokens", kind="decode", T=13, r=16, adapter=False, h=896, kv=128, m=4864),
        # a short pair scored by the reference model over the whole vocabulary: few rows, long ones
        dict(name="score 1 pair", kind="score", T=37, P=1, V=VOCAB, pad=0, dtype="bf16", prompt=0.3, tail=0, average=False),
        # the reference pass over a full batch
        dict(name="score 8 pairs", kind="score", T=2048, P=8, V=VOCAB, pad=0, dtype="bf16", prompt=0.25, tail=0, average=False),
        # the policy's pass over the same batch, with the gradient: the largest case
        dict(name="train 8 pairs", kind="train", T=2048, P=8, V=VOCAB, pad=0, dtype="bf16", prompt=0.25, tail=0, average=False,
             loss="sigmoid", beta=0.1, smooth=0.0),
        # 32-bit logits of an odd vocabulary in padded rows, rows behind the last sequence, smoothed labels
        dict(name="train fp32 odd vocabulary", kind="train", T=389, P=3, V=32003, pad=5, dtype="fp32", prompt=0.4, tail=11, average=False,
             loss="sigmoid", beta=0.25, smooth=0.1),
        # many short answers, squared loss on the mean log ratio per token
        dict(name="train 48 short pairs", kind="train", T=1021, P=48, V=32000, pad=0, dtype="bf16", prompt=0.5, tail=0, average=True,
             loss="squared", beta=0.5, smooth=0.0),
        # every adapter gradient of the 8B stack (448 tensors of one buffer), over the largest norm
        dict(name="clip 8B rank 16", kind="clip", sizes="8b", r=16, n=0, dtype="fp32", ratio=0.3),
        # a few hundred odd-sized tensors of both types, under the largest norm
        dict(name="clip 300 odd tensors", kind="clip", sizes="odd", r=0, n=300, dtype="mixed", ratio=4.0),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "decode", "score", "train", "train", "clip"])
    if kind == "decode":
        case = dict(kind=kind, T=rng.randint(1, 16), r=rng.choice([8, 16, 24, 32, 64]), adapter=rng.random() < 0.8)
        if rng.random() < 0.5:
            K = 64 * _spread(rng, 1, 462)
            return dict(case, K=K, N=64 * _spread(rng, 1, min(462, WEIGHTS // K // 64)))
        h = 64 * _spread(rng, 4, 80)
        return dict(case, h=h, kv=64 * rng.randint(1, h // 64), m=64 * _spread(rng, h // 64, 4 * h // 64))
    if kind == "clip":
        if rng.random() < 0.5:
            return dict(kind=kind, sizes=rng.choice(["0.5b", "3b", "8b"]), r=rng.choice([8, 16]), n=0, dtype=rng.choice(["fp32", "bf16"]), ratio=rng.choice([0.1, 0.5, 2.0]) * rng.uniform(0.8, 1.2))
        return dict(kind=kind, sizes="odd", r=0, n=_spread(rng, 1, 1200), dtype=rng.choice(["fp32", "bf16", "mixed"]), ratio=rng.choice([0.1, 0.5, 2.0]) * rng.uniform(0.8, 1.2))
    V = _spread(rng, 1000, 152000)
    T = _spread(rng, 8, min(2048, LARGEST // V))
    case = dict(kind=kind, T=T, P=_spread(rng, 1, max(1, min(64, T // 8))), V=V, pad=rng.choice([0, 0, 1, 3, 8, 64]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                prompt=rng.choice([0.0, 0.25, 0.5]), tail=rng.choice([0, 0, 2, 9]) if T > 40 else 0, average=rng.random() < 0.4)
    if case["dtype"] == "fp32":
        case["T"] = max(8, T // 2)
        case["P"] = min(case["P"], max(1, case["T"] // 8))
    if kind == "train":
        loss = rng.choice(["sigmoid", "sigmoid", "squared", "hinge"])
        case.update(loss=loss, beta=rng.uniform(0.5, 2.0) if case["average"] else rng.uniform(0.05, 0.3), smooth=rng.choice([0.0, 0.1]) if loss == "sigmoid" else 0.0)
    return case


# ---------------------------------------------------------------- inputs ---

def _levels():
    """The 16 NF4 levels: normal quantiles of 7 negative and 8 positive equal steps up to p_max, over the last one."""
    top = 1 - (1 / 32 + 1 / 30) / 2
    q = NormalDist().inv_cdf
    return [-q(0.5 + (top - 0.5) * i / 7) / q(top) for i in range(7, 0, -1)] + [0.0] + [q(0.5 + (top - 0.5) * i / 8) / q(top) for i in range(1, 9)]


def _weight(K, N, g):
    """An NF4 weight of N(0, 0.02) values: packed codes, and the double-quantised absmax of its blocks."""
    levels = torch.tensor(_levels(), device="cuda")
    packed = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    amax = torch.empty(N, K // 64, device="cuda")
    step = max(1, (1 << 26) // K)
    for a in range(0, N, step):
        w = (torch.randn(min(step, N - a), K // 64, 64, generator=g, device="cuda") * 0.02)
        m = w.abs().amax(-1)
        c = torch.bucketize(w / m[..., None], (levels[1:] + levels[:-1]) / 2).view(-1, K // 2, 2)
        packed[a:a + step] = (c[..., 0] * 16 + c[..., 1]).to(torch.uint8)
        amax[a:a + step] = m
    amax = amax.view(-1)
    offset = amax.double().mean().float()
    d = torch.nn.functional.pad(amax - offset, (0, -amax.numel() % 256)).view(-1, 256)
    s2 = d.abs().amax(-1)
    q = (d / s2.clamp_min(1e-30)[:, None] * 127).round().add(127).to(torch.uint8).view(-1)[:amax.numel()]
    return dict(packed=packed.view(-1), q=q.contiguous(), s2=s2.contiguous(), offset=offset.view(1).contiguous())


def _bf16(*shape, g, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _lengths(case):
    """The lengths of the 2 P sequences, chosen and rejected in turn, uneven, and the scored tokens behind their prompts."""
    rng = random.Random(case["T"] * 1000003 + case["P"])
    n, rows = 2 * case["P"], case["T"] - case["tail"]
    cuts = [rng.uniform(0.6, 1.4) for _ in range(n)]
    at = [int(round(rows * sum(cuts[:i]) / sum(cuts))) for i in range(n + 1)]
    return at, [int(case["prompt"] * (at[i + 1] - at[i])) for i in range(n)]


def _batch(case, g):
    T, V, ld = case["T"], case["V"], case["V"] + case["pad"]
    at, prompt = _lengths(case)
    tgt = torch.randint(0, V, (T,), generator=g, device="cuda")
    f = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    logits = torch.empty(T, ld, dtype=f, device="cuda")
    step = max(1, (1 << 27) // ld)
    for a in range(0, T, step):
        logits[a:a + step].normal_(0.0, 2.0, generator=g)
    rows = torch.arange(T, device="cuda")
    # a trained model gives its own answers' tokens far more than a uniform share
    logits[rows, tgt] += (6.0 + 3.0 * torch.randn(T, generator=g, device="cuda")).to(f)
    for i in range(2 * case["P"]):
        tgt[at[i]:at[i] + prompt[i]] = -100
    tgt[at[-1]:] = -100
    start = torch.tensor(at, dtype=torch.int32, device="cuda")
    scored = torch.tensor([at[i + 1] - at[i] - prompt[i] for i in range(2 * case["P"])], dtype=torch.float64, device="cuda")
    # the reference's values lie about the policy's: a token costs log V + 2 less what its own logit brings
    ref = -scored * (math.log(V) + 2.0 - 6.0) + scored.sqrt() * 3.0 * torch.randn(2 * case["P"], generator=g, device="cuda", dtype=torch.float64)
    return dict(logits=logits, targets=tgt.to(torch.int32), start=start, ref=ref / scored.clamp_min(1) if case["average"] else ref)


def _sizes(case):
    if case["sizes"] != "odd":
        L, h, kv, m = STACKS[case["sizes"]]
        return [n * case["r"] for K, N, _ in _layer(h, kv, m) * L for n in (K, N)]
    rng = random.Random(case["n"] * 7919 + 3)
    return [_spread(rng, 1, 300000) for _ in range(case["n"])]


def _groups(case):
    """The tensors by type, as (offset, size) in one buffer a type, each on a 16-byte boundary, and the buffers' sizes."""
    names = {"fp32": ["fp32"], "bf16": ["bf16"], "mixed": ["fp32", "bf16"]}[case["dtype"]]
    at, end = {n: [] for n in names}, dict.fromkeys(names, 0)
    for i, s in enumerate(_sizes(case)):
        n = names[i % len(names)]
        at[n].append((end[n], s))
        end[n] += -(-s // 8) * 8
    return at, end


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    if case["kind"] == "decode":
        T, r = case["T"], case["r"]
        width = {i: K for K, _, i in _projs(case)}
        s["x"] = {i: _bf16(T, K, g=g) for i, K in width.items()}
        s["w"] = [_weight(K, N, g) for K, N, _ in _projs(case)]
        s["A"] = [((torch.rand(r, K, generator=g, device="cuda") * 2 - 1) / K ** 0.5).to(torch.bfloat16) if case["adapter"] else None for K, _, _ in _projs(case)]
        s["B"] = [_bf16(N, r, g=g, std=0.01) if case["adapter"] else None for _, N, _ in _projs(case)]
    elif case["kind"] == "clip":
        at, end = _groups(case)
        s["at"] = at
        s["src"] = {n: torch.zeros(e, dtype=torch.float32 if n == "fp32" else torch.bfloat16, device="cuda") for n, e in end.items()}
        for n, flat in s["src"].items():
            flat.normal_(0.0, 1e-3, generator=g)
            inside = torch.zeros(flat.numel() + 1, dtype=torch.int32, device="cuda")
            inside[torch.tensor([a for a, _ in at[n]], device="cuda")] += 1
            ends = torch.tensor([a + k for a, k in at[n]], device="cuda")
            inside.index_add_(0, ends, torch.full_like(ends, -1, dtype=torch.int32))
            flat *= inside[:-1].cumsum(0)
        s["max_norm"] = case["ratio"] * 1e-3 * math.sqrt(sum(_sizes(case)))
    else:
        s.update(_batch(case, g))
    if own:
        _keep(s)
    return s


def _keep(s):
    """The descriptors, outputs and workspaces that a program makes once."""
    from layer_streamed_nf4_b200 import lsnf4
    case = s["case"]
    if case["kind"] == "decode":
        s["y"] = [torch.empty(case["T"], N, dtype=torch.bfloat16, device="cuda") for _, N, _ in _projs(case)]
        s["base"] = [lsnf4.base_nf4(lsnf4.make_nf4_weight(N, K, w["packed"], w["q"], w["s2"], w["offset"])) for (K, N, _), w in zip(_projs(case), s["w"])]
        s["projs"] = lsnf4.proj_array([lsnf4.lora_proj(b, s["x"][i], A, B, y=y) for b, (_, _, i), A, B, y in zip(s["base"], _projs(case), s["A"], s["B"], s["y"])])
        n = lsnf4.decode_ws_bytes(s["projs"], case["T"], case["r"])
    elif case["kind"] == "clip":
        s["dst"] = {k: torch.zeros_like(v) for k, v in s["src"].items()}
        dt = {"fp32": lsnf4.LSN_DT_F32, "bf16": lsnf4.LSN_DT_BF16}
        s["tensors"] = lsnf4.grad_array([lsnf4.grad_tensor(s["src"][k][a:a + n], n, dt[k], dst=s["dst"][k][a:a + n]) for k, v in s["at"].items() for a, n in v])
        s["norm"] = torch.zeros(1, device="cuda")
        n = lsnf4.grad_ws_bytes(s["tensors"])
    else:
        T, V, P = case["T"], case["V"], case["P"]
        s["in"] = lsnf4.seq_logits(s["logits"], T, V, V + case["pad"], lsnf4.LSN_DT_BF16 if case["dtype"] == "bf16" else lsnf4.LSN_DT_F32, s["targets"], 2 * P, s["start"],
                                   average=case["average"])
        s["lse"] = torch.zeros(T, device="cuda")
        s["logp"] = torch.zeros(2 * P, dtype=torch.float64, device="cuda")
        s["count"] = torch.zeros(2 * P, dtype=torch.int32, device="cuda")
        if case["kind"] == "train":
            s["pref"] = lsnf4.preference({"sigmoid": lsnf4.LSN_PREF_SIGMOID, "squared": lsnf4.LSN_PREF_SQUARED, "hinge": lsnf4.LSN_PREF_HINGE}[case["loss"]],
                                         case["beta"], label_smoothing=case["smooth"])
            s["reward"], s["dlogp"] = torch.zeros(2 * P, device="cuda"), torch.zeros(2 * P, device="cuda")
            s["loss"], s["mean"] = torch.zeros(P, device="cuda"), torch.zeros(1, device="cuda")
            s["dlogits"] = torch.empty(T, V, dtype=s["logits"].dtype, device="cuda")
        n = lsnf4.seq_logp_ws_bytes(s["in"])
    s["ws"], s["ws_bytes"] = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda"), n


# ------------------------------------------------------------ plain forms ---

def _dequant(w, K, N):
    """W in 32 bits: level[code] times its block's absmax, itself offset + table[q] s2."""
    levels = torch.tensor(_levels(), device="cuda")
    codes = torch.stack([w["packed"] >> 4, w["packed"] & 15], 1).view(-1, 64).int()
    table = (torch.arange(256, device="cuda") - 127).float() / 127
    amax = table[w["q"].int()] * w["s2"].repeat_interleave(256)[:w["q"].numel()] + w["offset"]
    return (levels[codes] * amax[:, None]).view(N, K)


def _decode(x, w, A, B, K, N, scale):
    y = x.float() @ _dequant(w, K, N).T
    if A is not None:
        y = y + scale * (x.float() @ A.float().T) @ B.float().T
    return y.to(torch.bfloat16)


def _logp(s):
    """Each row's log sum exp (0 where it is not scored), each sequence's sum or mean of log-probabilities, in 64 bits, and its scored tokens."""
    case, V = s["case"], s["case"]["V"]
    n = 2 * case["P"]
    x = s["logits"][:, :V].float()
    t = torch.arange(case["T"], device="cuda", dtype=torch.int32)
    seq = torch.bucketize(t, s["start"][1:], right=True).clamp_max(n - 1)
    on = (s["targets"] >= 0) & (s["targets"] < V) & (t >= s["start"][0]) & (t < s["start"][-1])
    top = x.amax(1, keepdim=True)
    lse = (top + (x - top).exp().sum(1, keepdim=True).log())[:, 0]
    own_logit = x.gather(1, s["targets"].clamp(0, V - 1).long()[:, None])[:, 0]
    # the difference of two numbers near one another, summed over hundreds of tokens: 64 bits
    one = torch.where(on, own_logit.double() - top[:, 0].double() - (x - top).exp().sum(1, dtype=torch.float64).log(), 0.0)
    logp = torch.zeros(n, dtype=torch.float64, device="cuda").index_add_(0, seq, one)
    count = torch.zeros(n, dtype=torch.float64, device="cuda").index_add_(0, seq, on.double()).clamp_min(1)
    return x, torch.where(on, lse, 0.0), logp / count if case["average"] else logp, count, seq, on


def _train(s):
    case, P = s["case"], s["case"]["P"]
    x, lse, logp, count, seq, on = _logp(s)
    beta, e = case["beta"], case["smooth"]
    ratio = (logp - s["ref"]).view(P, 2)
    h = ratio[:, 0] - ratio[:, 1]
    if case["loss"] == "sigmoid":
        up, down = torch.log1p(torch.exp(-(beta * h).abs())) + (-beta * h).clamp_min(0), torch.log1p(torch.exp(-(beta * h).abs())) + (beta * h).clamp_min(0)
        loss = (1 - e) * up + e * down
        d = -beta * ((1 - e) / (1 + torch.exp(beta * h)) - e / (1 + torch.exp(-beta * h)))
    elif case["loss"] == "hinge":
        loss = (1 - beta * h).clamp_min(0)
        d = torch.where(1 - beta * h > 0, -beta, 0.0)
    else:
        loss = (h - 0.5 / beta).square()
        d = 2 * (h - 0.5 / beta)
    dlogp = torch.stack([d, -d], 1).view(-1) / P
    row = torch.where(on, (dlogp / count if case["average"] else dlogp)[seq], 0.0).float()
    grad = (x - torch.where(on, lse, float("inf"))[:, None]).exp()
    grad *= -row[:, None]
    grad[torch.arange(case["T"], device="cuda"), s["targets"].clamp_min(0).long()] += row
    return dict(loss=loss.float(), mean=loss.mean().float().view(1), reward=(beta * ratio).float().view(-1), dlogits=grad.to(s["logits"].dtype))


def _clip(s):
    norm = sum(f.double().square().sum() for f in s["src"].values()).sqrt()
    factor = (s["max_norm"] / norm).clamp_max(1.0).float()
    return dict(norm=norm.float().view(1), **{k: (f.float() * factor).to(f.dtype) for k, f in s["src"].items()})


def run(s):
    case = s["case"]
    if own:
        from layer_streamed_nf4_b200 import lsnf4
        if case["kind"] == "decode":
            scale = 32.0 / case["r"]
            if len(s["y"]) == 1:
                lsnf4.lora_linear_decode(s["base"][0], s["x"][0], case["T"], s["A"][0], s["B"][0], case["r"], scale, s["y"][0], s["ws"], s["ws_bytes"])
            else:
                lsnf4.lora_layer_decode(s["projs"], case["T"], case["r"], scale, s["ws"], s["ws_bytes"])
            return s["y"]
        if case["kind"] == "score":
            lsnf4.seq_logp_fwd(s["in"], s["lse"], s["logp"], s["count"], s["ws"], s["ws_bytes"])
            return dict(lse=s["lse"], logp=s["logp"].float())
        if case["kind"] == "train":
            lsnf4.preference_loss_fwd_bwd(s["in"], s["ref"], s["pref"], s["lse"], s["logp"], s["count"], s["reward"], s["loss"], s["mean"], s["dlogp"], s["dlogits"], case["V"],
                                          s["ws"], s["ws_bytes"])
            return dict(loss=s["loss"], mean=s["mean"], reward=s["reward"], dlogits=s["dlogits"])
        lsnf4.grad_clip(s["tensors"], s["max_norm"], s["norm"], s["ws"], s["ws_bytes"])
        return dict(norm=s["norm"], **s["dst"])
    if case["kind"] == "decode":
        return [_decode(s["x"][i], w, A, B, K, N, 32.0 / case["r"]) for (K, N, i), w, A, B in zip(_projs(case), s["w"], s["A"], s["B"])]
    if case["kind"] == "score":
        _, lse, logp, _, _, _ = _logp(s)
        return dict(lse=lse, logp=logp.float())
    return _train(s) if case["kind"] == "train" else _clip(s)


# ----------------------------------------------------------------- exact ---

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "decode":
        out = []
        for (K, N, i), w, A, B in zip(_projs(case), s["w"], s["A"], s["B"]):
            x = s["x"][i].double()
            lv = torch.tensor(_levels(), device="cuda").double()  # the format's levels are 32-bit numbers
            nb = K // 64
            y = torch.empty(case["T"], N, dtype=torch.float64, device="cuda")
            for a in range(0, N, 1024):
                b = min(N, a + 1024)
                p = w["packed"][a * K // 2:b * K // 2].long()
                v = torch.empty(b - a, K, dtype=torch.float64, device="cuda")
                v.view(-1)[0::2], v.view(-1)[1::2] = lv[p // 16], lv[p % 16]
                blk = torch.arange(a * nb, b * nb, device="cuda")
                m = (w["q"][blk].double() - 127) / 127 * w["s2"].double()[blk // 256] + w["offset"].double()
                y[:, a:b] = torch.einsum("tbk,nbk,nb->tn", x.view(-1, nb, 64), v.view(b - a, nb, 64), m.view(b - a, nb))
            if A is not None:
                y += 32.0 / case["r"] * torch.einsum("tr,nr->tn", torch.einsum("tk,rk->tr", x, A.double()), B.double())
            out.append(y)
        return out
    if case["kind"] == "clip":
        total = math.sqrt(sum(float(torch.dot(f.double(), f.double())) for f in s["src"].values()))
        return dict(norm=torch.tensor([total], dtype=torch.float64), **{k: f.double() * min(1.0, s["max_norm"] / total) for k, f in s["src"].items()})
    T, V, P = case["T"], case["V"], case["P"]
    at, tgt = s["start"].tolist(), s["targets"].tolist()
    lse, own_logit = torch.zeros(T, dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
    for a in range(0, T, 128):
        x = s["logits"][a:a + 128, :V].double()
        lse[a:a + 128] = torch.logsumexp(x, 1).cpu()
        own_logit[a:a + 128] = x[torch.arange(x.shape[0], device="cuda"), torch.tensor([max(t, 0) for t in tgt[a:a + 128]], device="cuda")].cpu()
    rows = [[t for t in range(at[i], at[i + 1]) if tgt[t] >= 0] for i in range(2 * P)]
    on = torch.zeros(T, dtype=torch.bool)
    on[[t for r in rows for t in r]] = True
    logp = torch.tensor([float((own_logit[r] - lse[r]).sum()) / (max(1, len(r)) if case["average"] else 1) for r in rows], dtype=torch.float64)
    if case["kind"] == "score":
        return dict(lse=torch.where(on, lse, 0.0), logp=logp)
    beta, e = case["beta"], case["smooth"]
    reward = beta * (logp - s["ref"].cpu())
    z = (reward[0::2] - reward[1::2]).tolist()
    soft = lambda v: max(v, 0.0) + math.log1p(math.exp(-abs(v)))  # noqa: E731
    sig = lambda v: 1 / (1 + math.exp(-v)) if v >= 0 else math.exp(v) / (1 + math.exp(v))  # noqa: E731
    if case["loss"] == "sigmoid":
        loss, d = [(1 - e) * soft(-v) + e * soft(v) for v in z], [beta * (e * sig(v) - (1 - e) * sig(-v)) for v in z]
    elif case["loss"] == "hinge":
        loss, d = [max(0.0, 1 - v) for v in z], [-beta if v < 1 else 0.0 for v in z]
    else:
        loss, d = [(v / beta - 0.5 / beta) ** 2 for v in z], [2 * (v / beta - 0.5 / beta) for v in z]
    grad = torch.zeros(T, V, dtype=torch.float64 if T * V < 1 << 29 else torch.float32, device="cuda")
    for i, r in enumerate(rows):
        c = (d[i // 2] if i % 2 == 0 else -d[i // 2]) / P / (max(1, len(r)) if case["average"] else 1)
        for a in range(0, len(r), 128):
            k = torch.tensor(r[a:a + 128], device="cuda")
            p = torch.softmax(s["logits"][k, :V].double(), 1)
            p[torch.arange(len(k), device="cuda"), s["targets"][k].long()] -= 1
            grad[k] = (p * -c).to(grad.dtype)
    loss = torch.tensor(loss, dtype=torch.float64)
    return dict(loss=loss, mean=loss.mean().view(1), reward=reward, dlogits=grad)


def work(case):
    if case["kind"] == "decode":
        T, r = case["T"], case["r"] if case["adapter"] else 0
        x = {i: K for K, _, i in _projs(case)}
        nf4 = sum(K * N / 2 + K * N / 64 + 4 * -(-K * N // 16384) + 4 for K, N, _ in _projs(case))
        return dict(bytes=nf4 + sum(2 * T * K for K in x.values()) + sum(2 * r * (K + N) + 2 * T * N for K, N, _ in _projs(case)),
                    flops=sum(2.0 * T * (K * N + r * (K + N)) for K, N, _ in _projs(case)))
    if case["kind"] == "clip":
        at, _ = _groups(case)
        n = {k: sum(size for _, size in v) for k, v in at.items()}
        return dict(bytes=sum(2 * (4 if k == "fp32" else 2) * v for k, v in n.items()) + 4, flops=3.0 * sum(n.values()))
    at, prompt = _lengths(case)
    scored, size = at[-1] - at[0] - sum(prompt), 2 if case["dtype"] == "bf16" else 4
    few = 8 * case["T"] + 16 * 2 * case["P"]
    if case["kind"] == "score":
        return dict(bytes=scored * case["V"] * size + few, flops=4.0 * scored * case["V"])
    return dict(bytes=(scored + case["T"]) * case["V"] * size + few, flops=8.0 * scored * case["V"])
