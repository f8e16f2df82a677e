"""Cases and plain forms of the operators of a step that serves several requests at once.

Three operators, in the order in which such a step meets them:

  linear_lora  a projection over 8-bit codes and, beside it, each row's own low-rank adapter:
               out[m] = a_scale[m] * (w_scale * (W a[m]) + scale_j * B_j (A_j a[m])), j = adapter[m]
  batch        the whole 4-bit mixture-of-experts layer for a few tokens: selection (with or
               without scores, a bias and groups of experts), the SwiGLU experts and the shared
               expert, optionally weighted per token, and the weighted sum
  logprobs     of rows of logits: the log probability of a given token, the entropy, and the
               most probable tokens with their log probabilities

`own` False computes them with elementary torch operations in 32 bits (64 where a selection
hangs on the last bit), `own` True with the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
# selection by the logits alone, weights by a softmax over the chosen
CHOSEN = dict(score="chosen", n_groups=1, topk_groups=1, group_score="max", renormalise=True, scale=1.0)


def listed():
    return [
        # a projection of one token with its request's adapter
        dict(name="lora, one token", op="linear_lora", M=1, N=4096, K=2048, R=16, n=8, mix="rows"),
        # a decode step of 48 requests, each with an adapter of its own, some with none
        dict(name="lora, 48 requests", op="linear_lora", M=48, N=4096, K=4096, R=16, n=48, mix="rows"),
        # a short ragged batch of a few requests into an odd number of channels
        dict(name="lora, 333 tokens, odd", op="linear_lora", M=333, N=1001, K=2048, R=8, n=5, mix="runs"),
        # prompts of several requests in one long chunk, adapters of a high rank
        dict(name="lora, 8192 tokens", op="linear_lora", M=8192, N=4096, K=4096, R=64, n=6, mix="runs"),
        # two requests' tokens, or one drafted token with its successor
        dict(name="batch, 2 tokens", op="batch", T=2, H=2048, I=512, I_sh=512, E=256, k=8, **CHOSEN,
             gated=False, layout="packed", skew=0.0),
        # a layer of few wide experts, weights as they were loaded, an odd number of tokens
        dict(name="batch, 7 tokens, 60 experts", op="batch", T=7, H=2048, I=1408, I_sh=2816, E=60, k=4,
             **CHOSEN, gated=True, layout="rows", skew=0.0),
        # sixteen requests under sigmoid scores, a balance bias, 4 of 8 groups
        dict(name="batch, 16 tokens, scored", op="batch", T=16, H=2048, I=512, I_sh=512, E=256, k=8,
             score="sigmoid", n_groups=8, topk_groups=4, group_score="top2", renormalise=True, scale=2.5,
             gated=True, layout="packed", skew=0.0),
        # the largest batch, of unequal expert popularity
        dict(name="batch, 64 tokens, skewed", op="batch", T=64, H=2048, I=512, I_sh=512, E=256, k=8,
             **CHOSEN, gated=False, layout="packed", skew=1.1),
        # the token that one request sampled, with five alternatives
        dict(name="logprobs, one token", op="logprobs", T=1, V=131072, dtype="bf16", n_top=5, masked=False),
        # a step of 48 requests, fp32 logits, an odd vocabulary of which a grammar allows a part
        dict(name="logprobs, 48 tokens, odd", op="logprobs", T=48, V=100003, dtype="f32", n_top=20,
             masked=True),
        # 192 positions of a text whose perplexity and best tokens are compared
        dict(name="logprobs, 192 positions", op="logprobs", T=192, V=150001, dtype="bf16", n_top=1,
             masked=False),
        # the positions of a chunk of a prompt, all with twenty alternatives
        dict(name="logprobs, 2048 positions", op="logprobs", T=2048, V=131072, dtype="bf16", n_top=20,
             masked=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear_lora", "batch", "logprobs"])
    if op == "linear_lora":
        K, N = 64 * _log(rng, 4, 112), _log(rng, 16, 8192)
        M = _log(rng, 1, max(2, min(8192, 8192 * 4096 * 4096 // (N * K))))
        n = _log(rng, 1, 64)
        # adapters of all requests together no larger than 1 GB
        R = 8 * rng.randint(1, max(1, min(16, (1 << 29) // (8 * n * (N + K)))))
        return dict(op=op, M=M, N=N, K=K, R=R, n=n, mix=rng.choice(["rows", "runs"]))
    if op == "batch":
        E = rng.choice([16, 60, 64, 128, 160, 256])
        rule = CHOSEN
        if rng.random() < 0.5:
            groups = rng.choice([1, 2, 4]) if E % 8 else rng.choice([1, 2, 4, 8])
            rule = dict(score=rng.choice(["softmax", "sigmoid"]), n_groups=groups,
                        topk_groups=rng.randint(max(1, groups // 2), groups),
                        group_score=rng.choice(["top2", "max"]), renormalise=rng.random() < 0.5,
                        scale=rng.choice([1.0, 2.5]))
        return dict(op=op, T=_log(rng, 1, 64), H=64 * rng.randint(8, 32), I=64 * rng.randint(2, 8),
                    I_sh=64 * rng.randint(0, 8), E=E, k=rng.randint(1, 8), **rule,
                    gated=rng.random() < 0.5, layout=rng.choice(["packed", "packed", "tiles", "rows"]),
                    skew=rng.choice([0.0, 0.0, 1.1]))
    V = _log(rng, 1000, 200000)
    return dict(op=op, T=_log(rng, 1, max(1, min(2048, 2048 * 131072 // (2 * V)))), V=V,
                dtype=rng.choice(["bf16", "f32"]), n_top=rng.randint(0, 20), masked=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 6007 + 29)


def _to_codes(v):
    """Rows of fp32 values as 8-bit codes and one scale a row."""
    top = v.abs().amax(-1)
    q = torch.round(v * (127.0 / top.clamp_min(1e-30))[..., None]).to(torch.int8)
    return q, top / 127.0


def _i8_tiles(q):
    """The codes [N, K] in 16 x 64 tiles, as an engine keeps them after loading."""
    N, K = q.shape
    return q.view(N // 16, 16, K // 64, 4, 16).permute(0, 2, 3, 1, 4).contiguous()


def _q4(g, n_exp, N, K):
    """4-bit codes, eight a word, and bf16 scales and biases of each 64 weights."""
    codes = torch.randint(-2 ** 31, 2 ** 31, (n_exp, N, K // 8), dtype=torch.int64, device=DEV,
                          generator=g).to(torch.int32)
    s = (0.005 + 0.015 * torch.rand((n_exp, N, K // 64), device=DEV, generator=g)).bfloat16()
    b = (-8 * s.float() * (1 + 0.1 * torch.randn((n_exp, N, K // 64), device=DEV, generator=g))).bfloat16()
    return codes, s, b


def _q4_tiles(codes):
    """The code words in tiles of 64 rows x 64 weights, as an engine keeps them after loading."""
    n_exp, N, K8 = codes.shape
    t = codes.view(n_exp, N // 64, 4, 16, K8 // 8, 8).permute(0, 1, 4, 2, 3, 5)
    return t.reshape(codes.shape)


def _q4_packed(s, b):
    """Scale and bias of 64 weights in one word, in the order of the tiles' rows."""
    n_exp, N, G = s.shape
    w = torch.stack([s.view(torch.int16), b.view(torch.int16)], -1).view(torch.int32)[..., 0]
    return w.view(n_exp, N // 64, 64, G).permute(0, 1, 3, 2).reshape(n_exp, N, G)


def _prepare_lora(c, g, s):
    M, N, K, R, n = c["M"], c["N"], c["K"], c["R"], c["n"]
    s["a"], s["a_scale"] = _to_codes(torch.randn((M, K), device=DEV, generator=g))
    w, ws = _to_codes(torch.randn((N, K), device=DEV, generator=g).mul_(K ** -0.5))
    s["w"], s["w_scale"] = w, ws
    s["w_tiles"] = _i8_tiles(w) if N % 16 == 0 else None   # an odd number of channels stays in rows
    s["A"] = (torch.randn((n, R, K), device=DEV, generator=g) * K ** -0.5).bfloat16()
    s["B"] = (0.5 * torch.randn((n, N, R), device=DEV, generator=g) * R ** -0.5).bfloat16()
    s["scale"] = 0.5 + 1.5 * torch.rand(n, device=DEV, generator=g)
    if c["mix"] == "rows":   # a row each, in no order; one in eight without an adapter
        of = torch.randint(0, n, (M,), device=DEV, generator=g)
        if M > 1:
            of = torch.where(torch.rand(M, device=DEV, generator=g) < 0.125, -1, of)
    else:   # n + 1 sequences of unequal lengths after one another, one of them without an adapter
        cut = torch.sort(torch.randint(0, M + 1, (n,), device=DEV, generator=g))[0]
        seq = (torch.arange(M, device=DEV)[:, None] >= cut).sum(1)
        which = torch.randperm(n + 1, device=DEV, generator=g) - 1
        of = which[seq]
    s["adapter"] = of.to(torch.int32)


def _prepare_batch(c, g, s):
    T, H, I, I_sh, E = c["T"], c["H"], c["I"], c["I_sh"], c["E"]
    s["x"] = torch.randn((T, H), device=DEV, generator=g).bfloat16()
    lg = torch.randn((T, E), device=DEV, generator=g)
    if c["skew"]:
        rank = torch.randperm(E, device=DEV, generator=g) + 1
        lg = lg - c["skew"] * torch.log(rank.float())
    s["logits"] = lg
    s["bias"] = 0.1 * torch.randn(E, device=DEV, generator=g) if c["score"] != "chosen" else None
    s["shared_gate"] = torch.sigmoid(torch.randn(T, device=DEV, generator=g)) if c["gated"] and I_sh else None
    mats = {}
    for name, n_exp, N, K in (("gate", E, I, H), ("up", E, I, H), ("down", E, H, I),
                              ("sh_gate", 1, I_sh, H), ("sh_up", 1, I_sh, H), ("sh_down", 1, H, I_sh)):
        if not N or not K:
            mats[name] = None
            continue
        codes, sc, b = _q4(g, n_exp, N, K)
        as_loaded = (codes, sc, b)
        if c["layout"] != "rows":
            codes = _q4_tiles(codes)
        packed = _q4_packed(sc, b) if c["layout"] == "packed" and "down" not in name else None
        mats[name] = dict(rows=as_loaded, codes=codes, packed=packed)
    s["mats"] = mats


def _prepare_logprobs(c, g, s):
    T, V = c["T"], c["V"]
    lg = 2.5 * torch.randn((T, V), device=DEV, generator=g)
    target = torch.randint(0, V, (T,), device=DEV, generator=g)
    rows = torch.arange(T, device=DEV)
    # the text's next token is among the likely ones more often than not
    lg[rows, target] += 14 * torch.rand(T, device=DEV, generator=g)
    if c["masked"]:   # a grammar forbids most tokens, the target not
        off = torch.rand((T, V), device=DEV, generator=g) < 0.6
        off[rows, target] = False
        lg.masked_fill_(off, -math.inf)
    s["logits"] = lg.bfloat16() if c["dtype"] == "bf16" else lg
    s["target"] = target.to(torch.int32)


def prepare(case, seed):
    g, s = _gen(seed), dict(case=case)
    {"linear_lora": _prepare_lora, "batch": _prepare_batch, "logprobs": _prepare_logprobs}[case["op"]](case, g, s)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _lora_plain(s):
    a, n = s["a"].float(), s["A"].shape[0]
    out = torch.matmul(a, s["w"].float().t()) * s["w_scale"]
    of = s["adapter"]
    for j in range(n):
        u = torch.matmul(a, s["A"][j].float().t()) * ((of == j) * s["scale"][j])[:, None]
        out = out + torch.matmul(u, s["B"][j].float().t())
    return (out * s["a_scale"][:, None]).bfloat16()


def _first(v, n):
    """Indices of the n largest of each row, ties to the lowest index."""
    return torch.sort(v, dim=-1, descending=True, stable=True)[1][:, :n]


def _select(s):
    """topk_idx [T, k] and the weights fp32 [T, k]."""
    c, lg = s["case"], s["logits"]
    T, E = lg.shape
    if c["score"] == "chosen":
        idx = _first(lg, c["k"])
        p = torch.gather(lg, 1, idx)
        p = torch.exp(p - p[:, :1])
        return idx, p / p.sum(-1, keepdim=True)
    G = c["n_groups"]
    d = lg.double()
    if c["score"] == "sigmoid":
        score = (1 / (1 + torch.exp(-d))).float()
    else:
        p = torch.exp(d - d.amax(-1, keepdim=True))
        score = (p / p.sum(-1, keepdim=True)).float()
    choice = score + s["bias"]
    if G > 1:
        by = choice.view(T, G, E // G)
        two = torch.sort(by, dim=-1, descending=True)[0][:, :, :2]
        worth = two[:, :, 0] if c["group_score"] == "max" else two[:, :, 0] + two[:, :, 1]
        keep = torch.zeros((T, G), dtype=torch.bool, device=DEV)
        keep.scatter_(1, _first(worth, c["topk_groups"]), True)
        choice = torch.where(keep[:, :, None], by, torch.full_like(by, -math.inf)).view(T, E)
    idx = _first(choice, c["k"])
    w = torch.gather(score, 1, idx)
    if c["renormalise"]:
        w = w / w.sum(-1, keepdim=True).clamp_min(1e-30)
    return idx, w * c["scale"]


def _weights(m, e):
    """The experts' weights in fp32: bf16 of code * scale + bias."""
    codes, sc, b = (t[e] for t in m["rows"])
    q = torch.stack([(codes >> 4 * i) & 15 for i in range(8)], -1).float()
    w = q.view(*sc.shape, 64) * sc.float()[..., None] + b.float()[..., None]
    return w.bfloat16().float().view(*sc.shape[:2], -1)


def _ffn_plain(x, mats, e):
    """x [T, H] through each of the experts e: [n, T, H]."""
    g = torch.matmul(x, _weights(mats[0], e).transpose(-1, -2))
    u = torch.matmul(x, _weights(mats[1], e).transpose(-1, -2))
    return torch.matmul(g / (1 + torch.exp(-g)) * u, _weights(mats[2], e).transpose(-1, -2))


def _batch_plain(s):
    c, m, x = s["case"], s["mats"], s["x"].float()
    T, E, k = c["T"], c["E"], c["k"]
    idx, w = _select(s)
    by_expert = torch.zeros((T, E), device=DEV).scatter_(1, idx, w)
    used = torch.zeros(E, device=DEV).index_fill_(0, idx.reshape(-1), 1.0)
    e = _first(used[None], min(E, T * k))[0]   # the experts that any token chose come first
    y = torch.zeros((T, c["H"]), device=DEV)
    for part in e.split(64):
        out = _ffn_plain(x, (m["gate"], m["up"], m["down"]), part)
        y = y + (out * by_expert[:, part].t()[:, :, None]).sum(0)
    if c["I_sh"]:
        zero = torch.zeros(1, dtype=torch.int64, device=DEV)
        sh = _ffn_plain(x, (m["sh_gate"], m["sh_up"], m["sh_down"]), zero)[0]
        y = y + (sh if s["shared_gate"] is None else sh * s["shared_gate"][:, None])
    return dict(y=y.bfloat16(), topk_idx=idx.to(torch.int32), topk_w=w)


def _logprobs_plain(s):
    z, n = s["logits"].float(), s["case"]["n_top"]
    top = z.amax(-1, keepdim=True)
    d = z - top
    p = torch.exp(d)
    total = p.sum(-1, keepdim=True)
    log_total = torch.log(total)
    out = dict(logprob=(torch.gather(d, 1, s["target"].long()[:, None]) - log_total)[:, 0],
               entropy=(log_total - torch.where(p > 0, d * p, 0.0).sum(-1, keepdim=True) / total)[:, 0])
    if n:
        idx = _first(z, n)
        out.update(top_idx=idx.to(torch.int32), top_logprob=torch.gather(d, 1, idx) - log_total)
    return out


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _lora_own(s):
    import bit_quantized_grouped_amd as bq
    if "handle" not in s:   # what a program keeps: the matrix, the adapters, buffers
        M, N, K, R = (s["case"][n] for n in "MNKR")
        if s["w_tiles"] is None:
            s["mat"] = bq.DeviceI8Mat(s["w"][None], s["w_scale"][None])
        else:
            s["mat"] = bq.DeviceI8Mat(s["w_tiles"].view(1, N, K), s["w_scale"][None], bq.LAYOUT_TILES)
        s["handle"] = bq.DeviceAdapters(s["A"], s["B"], s["scale"])
        s["out"] = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
        s["ws"] = torch.empty(max(256, bq.linear_lora_i8_workspace_bytes(M, N, K, R)), dtype=torch.uint8, device=DEV)
    bq.moe_linear_lora_i8(s["a"], s["a_scale"], s["mat"], s["handle"], s["adapter"], s["out"], s["ws"])
    return s["out"]


def _batch_own(s):
    import bit_quantized_grouped_amd as bq
    c = s["case"]
    if "handle" not in s:
        layout = bq.LAYOUT_ROWS if c["layout"] == "rows" else bq.LAYOUT_TILES
        mats = []
        for m in s["mats"].values():
            if m is None:
                mats.append(None)
            elif m["packed"] is not None:
                mats.append(bq.DeviceQMat(m["codes"], m["packed"], None, bq.LAYOUT_TILES_SB))
            else:
                mats.append(bq.DeviceQMat(m["codes"], m["rows"][1], m["rows"][2], layout))
        s["handle"] = bq.MoeLayer.from_device(mats, c["H"], c["I"], c["I_sh"], c["E"], c["k"], DEV)
        s["rule"] = None
        if c["score"] != "chosen":
            s["rule"] = bq.ScoreRule(score=c["score"], n_groups=c["n_groups"], topk_groups=c["topk_groups"],
                                     group_score=c["group_score"], renormalise=c["renormalise"], scale=c["scale"])
    b = s["handle"].decode_batch(s["x"], s["logits"], rule=s["rule"], score_bias=s["bias"],
                                 shared_gate=s["shared_gate"])
    return dict(y=b["y"], topk_idx=b["topk_idx"], topk_w=b["topk_w"])


def _logprobs_own(s):
    import bit_quantized_grouped_amd as bq
    T, V, n = s["case"]["T"], s["case"]["V"], s["case"]["n_top"]
    if "out" not in s:
        s["out"] = dict(logprob=torch.empty(T, device=DEV), entropy=torch.empty(T, device=DEV))
        if n:
            s["out"]["top_idx"] = torch.empty((T, n), dtype=torch.int32, device=DEV)
            s["out"]["top_logprob"] = torch.empty((T, n), device=DEV)
        s["ws"] = torch.empty(max(256, bq.logprobs_workspace_bytes(T, V, n)), dtype=torch.uint8, device=DEV)
    bq.moe_logprobs(s["logits"], s["target"], ws=s["ws"], **s["out"])
    return s["out"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear_lora": _lora_own, "batch": _batch_own, "logprobs": _logprobs_own}[op](state)
    return {"linear_lora": _lora_plain, "batch": _batch_plain, "logprobs": _logprobs_plain}[op](state)


def work(case):
    c = case
    if c["op"] == "linear_lora":
        M, N, K, R = c["M"], c["N"], c["K"], c["R"]
        # adapters that at least one row has: all of those of the runs, uniform choice otherwise
        n = c["n"] if c["mix"] == "runs" else c["n"] * (1 - (1 - 1 / c["n"]) ** (0.875 * M if M > 1 else 1))
        return {"bytes": M * K + N * K + 4 * (2 * M + N) + 2 * M * N + 2 * n * R * (N + K),
                "flops": 2 * M * N * K + 2 * M * R * (N + K)}
    if c["op"] == "batch":
        T, H, I, I_sh, E, k = c["T"], c["H"], c["I"], c["I_sh"], c["E"], c["k"]
        # experts that at least one token picks, as uniform routing would have them; 4.5 bits a weight
        touched = min(E, E * (1 - (1 - k / E) ** T))
        return {"bytes": 3 * H * (touched * I + I_sh) * 36 // 64 + T * (4 * H + 4 * E + 8 * k),
                "flops": 6 * T * H * (k * I + I_sh)}
    T, V, n = c["T"], c["V"], c["n_top"]
    return {"bytes": T * (V * (2 if c["dtype"] == "bf16" else 4) + 12 + 8 * n), "flops": 5 * T * V}


# ---------------------------------------------------------------------------
# From the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_lora(s):
    a = s["a"].double()
    out = torch.mm(a, (s["w"].double() * s["w_scale"].double()[:, None]).t().contiguous())
    of = s["adapter"].cpu().numpy()
    for j in np.unique(of[of >= 0]):
        rows = torch.from_numpy(np.nonzero(of == j)[0]).to(DEV)
        low = torch.mm(a[rows], s["A"][j].double().t().contiguous())
        out[rows] += s["scale"][j].double() * torch.mm(low, s["B"][j].double().t().contiguous())
    return out * s["a_scale"].double()[:, None]


def _exact_select(s):
    c = s["case"]
    lg = s["logits"].cpu().numpy().astype(np.float64)
    T, E = lg.shape
    rows = np.arange(T)
    if c["score"] == "chosen":
        idx = np.argsort(-lg, axis=1, kind="stable")[:, :c["k"]]
        w = np.exp(np.take_along_axis(lg, idx, 1) - lg.max(1, keepdims=True))
        return idx, w / w.sum(1, keepdims=True)
    G = c["n_groups"]
    if c["score"] == "sigmoid":
        small = np.exp(-np.abs(lg))
        p = np.where(lg >= 0, 1 / (1 + small), small / (1 + small))
    else:
        p = np.exp(lg - lg.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    choice = p.astype(np.float32) + s["bias"].cpu().numpy()
    if G > 1:
        parted = choice.reshape(T, G, E // G)
        ordered = np.sort(parted, axis=2)
        worth = ordered[:, :, -1] if c["group_score"] == "max" else ordered[:, :, -1] + ordered[:, :, -2]
        free = np.zeros((T, G), bool)
        for _ in range(c["topk_groups"]):
            free[rows, np.where(free, -np.inf, worth).argmax(1)] = True
        choice = np.where(np.repeat(free, E // G, axis=1), choice, -np.inf)
    idx = np.argsort(-choice, axis=1, kind="stable")[:, :c["k"]]
    w = np.take_along_axis(p, idx, 1)
    if c["renormalise"]:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-30)
    return idx, w * c["scale"]


def _exact_ffn(x, mats, e):
    def of(m):
        codes, sc, b = (t[e] for t in m["rows"])
        shift = torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)
        q = torch.bitwise_right_shift(codes[..., None], shift) & 15
        q = q.reshape(*sc.shape, 64).double()
        w = (q * sc.double()[..., None] + b.double()[..., None]).float().bfloat16()
        return w.double().reshape(sc.shape[0], -1).t().contiguous()
    g, u = torch.mm(x, of(mats[0])), torch.mm(x, of(mats[1]))
    return torch.mm(g * torch.special.expit(g) * u, of(mats[2]))


def _exact_batch(s):
    c, m = s["case"], s["mats"]
    x = s["x"].double()
    idx, w = _exact_select(s)
    y = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        at = torch.from_numpy(t).to(DEV)
        part = _exact_ffn(x[at], (m["gate"], m["up"], m["down"]), int(e))
        y[at] += part * torch.from_numpy(w[t, j]).to(DEV)[:, None]
    if c["I_sh"]:
        sh = _exact_ffn(x, (m["sh_gate"], m["sh_up"], m["sh_down"]), 0)
        y += sh if s["shared_gate"] is None else sh * s["shared_gate"].double()[:, None]
    return dict(y=y, topk_idx=idx.astype(np.int32), topk_w=w)


def _exact_logprobs(s):
    T, V, n = s["case"]["T"], s["case"]["V"], s["case"]["n_top"]
    parts = []
    for rows in torch.arange(T, device=DEV).split(max(1, (1 << 25) // V)):
        z = s["logits"][rows].double()
        lse = torch.logsumexp(z, 1, keepdim=True)
        lp = z - lse
        one = dict(logprob=torch.gather(lp, 1, s["target"][rows].long()[:, None])[:, 0],
                   entropy=torch.special.entr(torch.exp(lp)).sum(1))
        if n:
            left, at = lp.clone(), torch.arange(V, device=DEV)
            idx = torch.empty((len(rows), n), dtype=torch.int64, device=DEV)
            taken = torch.zeros_like(left, dtype=torch.bool)
            for i in range(n):   # the lowest index of the largest value that is not taken
                left.masked_fill_(taken, -math.inf)
                best = (left == left.amax(1, keepdim=True)) & ~taken
                idx[:, i] = torch.where(best, at, V).amin(1)
                taken.scatter_(1, idx[:, i:i + 1], True)
            one.update(top_idx=idx.to(torch.int32), top_logprob=torch.gather(lp, 1, idx))
        parts.append(one)
    return {name: torch.cat([p[name] for p in parts]) for name in parts[0]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear_lora": _exact_lora, "batch": _exact_batch, "logprobs": _exact_logprobs}[case["op"]](s)
