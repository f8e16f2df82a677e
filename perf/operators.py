"""Cases and plain forms of the 8-bit block's operators.

Four operators, in the order in which a mixture-of-experts block runs them:

  norm    s = x + residual; y = s / sqrt(mean(s^2) + eps) * weight; the row's 8-bit
          codes q = rne(y / scale) with scale = max|y| / 127
  route   scores (softmax or sigmoid of the logits), a selection bias, groups of
          experts, top-k with ties to the lowest index, renormalised weights, and
          the expert histogram, scan, scatter and row-block map
  linear  out[m, n] = a_scale[m] * w_scale[n] * sum_k a[m, k] * w[n, k], 8-bit codes
  layer   route (softmax), the experts' SwiGLU FFNs and the shared expert's over 8-bit
          codes, and their weighted sum

`own` False computes them with elementary torch operations in 32 bits (64 where a
selection hangs on the last bit), `own` True with the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
EPS = 1e-6


def listed():
    return [
        # one token of a decode step before its router and experts
        dict(name="norm, one token", op="norm", T=1, H=2048, residual=True),
        # a prefill chunk of the 256-expert layer
        dict(name="norm, 2048 tokens", op="norm", T=2048, H=2048, residual=True),
        # a long chunk of a wide model, with an odd number of tokens
        dict(name="norm, 8191 tokens, wide", op="norm", T=8191, H=7168, residual=True),
        # one token of a decode step: sigmoid scores, balance bias, 4 of 8 groups
        dict(name="route, one token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True,
             n_groups=8, topk_groups=4, group_score="top2", renormalise=True, scale=2.5, masked=False),
        # a prefill chunk routed by the same rule
        dict(name="route, 2048 tokens", op="route", T=2048, E=256, k=8, score="sigmoid", bias=True,
             n_groups=8, topk_groups=4, group_score="top2", renormalise=True, scale=2.5, masked=False),
        # a whole long prompt: softmax scores, the best expert speaks for its group, some
        # experts switched off and some padded tokens
        dict(name="route, 8192 tokens", op="route", T=8192, E=160, k=6, score="softmax", bias=False,
             n_groups=8, topk_groups=3, group_score="max", renormalise=False, scale=16.0, masked=True),
        # a projection of one token
        dict(name="linear, one token", op="linear", M=1, N=4096, K=2048),
        # a short ragged batch into an odd number of channels
        dict(name="linear, 333 tokens, odd", op="linear", M=333, N=1001, K=2048),
        # a projection of a long chunk
        dict(name="linear, 8192 tokens", op="linear", M=8192, N=4096, K=4096),
        # one token through the 256-expert layer
        dict(name="layer, one token", op="layer", T=1, H=2048, I=512, I_sh=512, E=256, k=8, skew=0.0),
        # a 512-token prompt
        dict(name="layer, 512 tokens", op="layer", T=512, H=2048, I=512, I_sh=512, E=256, k=8, skew=0.0),
        # a 2048-token chunk of a long prompt with unequal expert popularity
        dict(name="layer, 2048 tokens, skewed", op="layer", T=2048, H=2048, I=512, I_sh=512, E=256,
             k=8, skew=1.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "linear", "layer"])
    if op == "norm":
        H = 64 * _log(rng, 4, 112)
        return dict(op=op, T=_log(rng, 1, 8191), H=H, residual=rng.random() < 0.75)
    if op == "route":
        n_groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = n_groups * rng.randint(2, 512 // n_groups)
        topk_groups = rng.randint(max(1, n_groups // 2), n_groups)
        k = rng.randint(1, min(16, topk_groups * (E // n_groups)))
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, n_groups=n_groups, topk_groups=topk_groups,
                    group_score=rng.choice(["top2", "max"]), renormalise=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5, 16.0]), masked=rng.random() < 0.5)
    if op == "linear":
        K = 64 * _log(rng, 4, 112)
        N = _log(rng, 16, 8192)
        return dict(op=op, M=_log(rng, 1, max(2, min(8192, 8192 * 4096 * 4096 // (N * K)))), N=N, K=K)
    E = rng.choice([16, 60, 64, 128, 256])
    return dict(op=op, T=_log(rng, 1, 2048), H=64 * rng.randint(8, 32), I=64 * rng.randint(2, 8),
                I_sh=64 * rng.randint(0, 8), E=E, k=rng.randint(1, 8),
                skew=rng.choice([0.0, 0.0, 1.1]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)


def _to_codes(v):
    """Rows of fp32 values as 8-bit codes and one scale a row."""
    top = v.abs().amax(-1)
    q = torch.round(v * (127.0 / top.clamp_min(1e-30))[..., None]).to(torch.int8)
    return q, top / 127.0


def _weights(g, n_exp, N, K):
    """8-bit codes [n_exp, N, K] of normal weights of variance 1 / K, scales [n_exp, N]."""
    q = torch.empty((n_exp, N, K), dtype=torch.int8, device=DEV)
    s = torch.empty((n_exp, N), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, n_exp, step):
        v = torch.randn((min(step, n_exp - e), N, K), device=DEV, generator=g)
        q[e:e + step], s[e:e + step] = _to_codes(v.mul_(K ** -0.5))
    return q, s


def _tiles(q):
    """The codes in 16 x 64 tiles, as an engine keeps them after loading: in a tile the four
    16-wide pieces of K one after another, each with its 16 rows."""
    n_exp, N, K = q.shape
    return q.view(n_exp, N // 16, 16, K // 64, 4, 16).permute(0, 1, 3, 4, 2, 5).contiguous()


def _logits(g, T, E, skew):
    lg = torch.randn((T, E), device=DEV, generator=g)
    if skew:
        rank = torch.randperm(E, device=DEV, generator=g) + 1
        lg = lg - skew * torch.log(rank.float())
    return lg


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        s["x"] = torch.randn((T, H), device=DEV, generator=g).bfloat16()
        s["residual"] = (3 * torch.randn((T, H), device=DEV, generator=g)).bfloat16() if c["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn(H, device=DEV, generator=g)).bfloat16()
    elif c["op"] == "route":
        T, E = c["T"], c["E"]
        lg = torch.randn((T, E), device=DEV, generator=g)
        if c["masked"]:
            off = torch.rand(E, device=DEV, generator=g) < 0.05
            pad = torch.rand(T, device=DEV, generator=g) < 0.02
            lg = lg.masked_fill(off[None, :] | pad[:, None], -math.inf)
        s["logits"] = lg
        s["bias"] = 0.1 * torch.randn(E, device=DEV, generator=g) if c["bias"] else None
    elif c["op"] == "linear":
        s["a"], s["a_scale"] = _to_codes(torch.randn((c["M"], c["K"]), device=DEV, generator=g))
        w, ws = _weights(g, 1, c["N"], c["K"])
        s["w"], s["w_scale"] = w, ws
        # an odd number of channels stays in rows
        s["w_tiles"] = _tiles(w) if c["N"] % 16 == 0 else None
    else:
        T, H, I, I_sh, E = c["T"], c["H"], c["I"], c["I_sh"], c["E"]
        s["x"], s["x_scale"] = _to_codes(torch.randn((T, H), device=DEV, generator=g))
        s["logits"] = _logits(g, T, E, c["skew"])
        for name, shape in (("gate", (E, I, H)), ("up", (E, I, H)), ("down", (E, H, I)),
                            ("sh_gate", (1, I_sh, H)), ("sh_up", (1, I_sh, H)), ("sh_down", (1, H, I_sh))):
            if shape[1] and shape[2]:
                q, sc = _weights(g, *shape)
                s[name] = (q, sc, _tiles(q))
            else:
                s[name] = None
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _norm_plain(s):
    x, res, w = s["x"], s["residual"], s["weight"]
    v = x.float() if res is None else x.float() + res.float()
    y = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w.float()
    top = y.abs().amax(-1, keepdim=True)
    scale = top / 127.0
    q = torch.round(y * torch.where(top > 0, 127.0 / top, torch.zeros_like(top)))
    return dict(sum=v.bfloat16(), y=y.bfloat16(), values=(q * scale).bfloat16(), scale=scale[:, 0])


def _first(v, n):
    """Indices of the n largest of each row, ties to the lowest index."""
    return torch.sort(v, dim=-1, descending=True, stable=True)[1][:, :n]


def _grouping(idx, E, block_rows):
    """Histogram, exclusive scan, stable scatter and row-block map of idx [T, k]."""
    n = idx.numel()
    flat = idx.reshape(-1)
    counts = (flat[:, None] == torch.arange(E, device=DEV)).sum(0)
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    offsets = torch.cat([zero, counts.cumsum(0)])
    order = torch.sort(flat, stable=True)[1]
    row = torch.empty_like(order)
    row[order] = torch.arange(n, device=DEV)
    blocks = (counts + block_rows - 1) // block_rows
    end = blocks.cumsum(0)
    b = torch.arange(-(-n // block_rows) + min(E, n), device=DEV)
    e = (b[:, None] >= end).sum(1)
    used = e < E
    e_in = e.clamp_max(E - 1)
    first = offsets[e_in] + block_rows * (b - (end - blocks)[e_in])
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    return dict(counts=i32(counts), offsets=i32(offsets), sorted_assign=i32(order), assign_row=i32(row),
                block_expert=i32(torch.where(used, e, -1)), block_row=i32(torch.where(used, first, -1)),
                n_blocks=i32(end[-1:]))


def _route_plain(s):
    c, lg = s["case"], s["logits"]
    T, E = lg.shape
    if c["score"] == "sigmoid":
        score = (1 / (1 + torch.exp(-lg.double()))).float()
    else:
        d = lg.double()
        top = d.amax(-1, keepdim=True)
        p = torch.where(top > -math.inf, torch.exp(d - top), torch.zeros_like(d))
        score = (p / p.sum(-1, keepdim=True).clamp_min(1e-300)).float()
    choice = score if s["bias"] is None else score + s["bias"]
    G = c["n_groups"]
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
    return dict(topk_idx=idx.to(torch.int32), topk_w=w * c["scale"], **_grouping(idx, E, 32))


def _product(a, a_scale, w, w_scale):
    """a [.., M, K] and w [.., N, K] codes as fp32, out [.., M, N]."""
    return torch.matmul(a, w.transpose(-1, -2)) * a_scale[..., None] * w_scale[..., None, :]


def _linear_plain(s):
    w, ws = s["w"][0], s["w_scale"][0]
    return _product(s["a"].float(), s["a_scale"], w.float(), ws).bfloat16()


def _ffn_plain(x, xs, gate, up, down):
    g = _product(x, xs, gate[0].float(), gate[1])
    u = _product(x, xs, up[0].float(), up[1])
    h = g / (1 + torch.exp(-g)) * u
    top = h.abs().amax(-1)
    q = torch.round(h * torch.where(top > 0, 127.0 / top, torch.zeros_like(top))[..., None])
    return _product(q, top / 127.0, down[0].float(), down[1])


def _layer_plain(s):
    c, lg, x, xs = s["case"], s["logits"], s["x"].float(), s["x_scale"]
    T, E, k, H = c["T"], c["E"], c["k"], c["H"]
    idx = _first(lg, k)
    p = torch.gather(lg, 1, idx)
    p = torch.exp(p - p[:, :1])
    p = p / p.sum(-1, keepdim=True)
    # blocks of up to 64 rows of one expert, each with its expert's weights
    to = _grouping(idx, E, 64)
    order, row = to["sorted_assign"].long(), to["assign_row"].long()
    e = to["block_expert"].long()
    at = to["block_row"].long()[:, None] + torch.arange(64, device=DEV)
    e_in = e.clamp_min(0)
    used = (e >= 0)[:, None] & (at < to["offsets"].long()[e_in + 1][:, None])
    token = order[at.clamp(0, T * k - 1)] // k
    mats = [(s[n][0][e_in], s[n][1][e_in]) for n in ("gate", "up", "down")]
    out = _ffn_plain(x[token], xs[token], *mats)
    part = torch.empty((T * k + 1, H), device=DEV)   # the last row takes the blocks' unused rows
    part[torch.where(used, at, T * k)] = out
    y = (part[row].view(T, k, H) * p[:, :, None]).sum(1)
    if c["I_sh"]:
        y = y + _ffn_plain(x[None], xs[None], s["sh_gate"], s["sh_up"], s["sh_down"])[0]
    return y.bfloat16()


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _norm_own(s):
    import bit_quantized_grouped_amd as bq
    x = s["x"]
    T, H = x.shape
    if "out" not in s:   # the buffers that a program keeps
        bf = lambda: torch.empty((T, H), dtype=torch.bfloat16, device=DEV)  # noqa: E731
        s["out"] = dict(sum=bf(), y=bf(), values=bf(), scale=torch.empty(T, device=DEV))
        s["q"] = torch.empty((T, H), dtype=torch.int8, device=DEV)
    o = s["out"]
    bq.moe_norm_i8(x, s["residual"], s["weight"], EPS, o["sum"], o["y"], s["q"], o["scale"])
    bq.moe_dequant_i8_bf16(s["q"], o["scale"], o["values"])
    return o


def _route_own(s):
    import bit_quantized_grouped_amd as bq
    c, lg = s["case"], s["logits"]
    T, E = lg.shape
    if "routing" not in s:
        s["routing"] = bq.DeviceRouting(T, E, c["k"], 32, DEV)
        s["ws"] = torch.empty(max(256, bq.route_workspace_bytes(T, E, c["k"], 32)), dtype=torch.uint8, device=DEV)
        s["rule"] = bq.ScoreRule(score=c["score"], n_groups=c["n_groups"], topk_groups=c["topk_groups"],
                                 group_score=c["group_score"], renormalise=c["renormalise"], scale=c["scale"])
    r = s["routing"]
    bq.moe_route_scored(lg, s["bias"], s["rule"], c["k"], 32, r, s["ws"])
    return dict(topk_idx=r.topk_idx, topk_w=r.topk_w, counts=r.counts, offsets=r.offsets,
                sorted_assign=r.sorted_assign, assign_row=r.assign_row, block_expert=r.block_expert,
                block_row=r.block_row, n_blocks=r.n_blocks)


def _own_mat(bq, q, scale, tiles):
    if tiles is None:
        return bq.DeviceI8Mat(q, scale)
    return bq.DeviceI8Mat(tiles.view(q.shape), scale, bq.LAYOUT_TILES)


def _linear_own(s):
    import bit_quantized_grouped_amd as bq
    if "mat" not in s:
        s["mat"] = _own_mat(bq, s["w"], s["w_scale"], s["w_tiles"])
        M, N, K = s["case"]["M"], s["case"]["N"], s["case"]["K"]
        s["out"] = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
        s["ws"] = torch.empty(max(256, bq.linear_i8_workspace_bytes(M, N, K)), dtype=torch.uint8, device=DEV)
    bq.moe_linear_i8(s["a"], s["a_scale"], s["mat"], s["out"], s["ws"])
    return s["out"]


def _layer_own(s):
    import bit_quantized_grouped_amd as bq
    if "handle" not in s:
        c = s["case"]
        mats = [None if s[n] is None else _own_mat(bq, *s[n])
                for n in ("gate", "up", "down", "sh_gate", "sh_up", "sh_down")]
        s["handle"] = bq.MoeLayerI8(mats, c["H"], c["I"], c["I_sh"], c["E"], c["k"], DEV)
    return s["handle"].forward(s["x"], s["x_scale"], s["logits"])["y"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _norm_own, "route": _route_own, "linear": _linear_own, "layer": _layer_own}[op](state)
    return {"norm": _norm_plain, "route": _route_plain, "linear": _linear_plain, "layer": _layer_plain}[op](state)


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        # x, residual, the sum, y and the codes' values in bf16; the scales
        return {"bytes": n * (10 if c["residual"] else 8) + 2 * c["H"] + 4 * c["T"], "flops": 8 * n}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        blocks = -(-T * k // 32) + min(E, T * k)
        return {"bytes": 4 * (T * E + (E if c["bias"] else 0) + 4 * T * k + 2 * E + 2 + 2 * blocks),
                "flops": 8 * T * E}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K + N * K + 4 * (M + N) + 2 * M * N, "flops": 2 * M * N * K}
    T, H, I, I_sh, E, k = c["T"], c["H"], c["I"], c["I_sh"], c["E"], c["k"]
    # experts that at least one token picks, as uniform routing would have them
    touched = min(E, E * (1 - (1 - k / E) ** T))
    per = lambda n: 3 * n * H + 4 * (2 * n + H) if n else 0  # noqa: E731
    return {"bytes": touched * per(I) + per(I_sh) + T * (H + 4 + 4 * E + 2 * H),
            "flops": 6 * T * H * (k * I + I_sh)}


# ---------------------------------------------------------------------------
# From the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_norm(s):
    f = torch.float64
    total = s["x"].to(f)
    if s["residual"] is not None:
        total = total + s["residual"].to(f)
    mean = torch.linalg.vector_norm(total, dim=1) ** 2 / total.shape[1]
    y = total * s["weight"].to(f) / torch.sqrt(mean + EPS)[:, None]
    step = torch.maximum(y.amax(1), -y.amin(1)) / 127
    values = torch.where(step[:, None] > 0, torch.round(y / step[:, None]) * step[:, None], 0.0)
    return dict(sum=total, y=y, values=values, scale=step)


def _exact_route(s):
    c = s["case"]
    lg = s["logits"].cpu().numpy().astype(np.float64)
    T, E = lg.shape
    with np.errstate(all="ignore"):
        if c["score"] == "sigmoid":
            p = np.where(lg >= 0, 1 / (1 + np.exp(-np.abs(lg))), np.exp(-np.abs(lg)) / (1 + np.exp(-np.abs(lg))))
        else:
            best = lg.max(1, keepdims=True)
            p = np.where(np.isfinite(best), np.exp(lg - np.where(np.isfinite(best), best, 0)), 0)
            p = np.divide(p, p.sum(1, keepdims=True), out=np.zeros_like(p), where=p.sum(1, keepdims=True) > 0)
    choice = p.astype(np.float32)
    if s["bias"] is not None:
        choice = choice + s["bias"].cpu().numpy()
    G, per, rows = c["n_groups"], E // c["n_groups"], np.arange(T)
    free = np.ones((T, E), bool)
    if G > 1:
        parted = choice.reshape(T, G, per)
        worth = parted.max(2)
        if c["group_score"] == "top2":
            rest = parted.copy()
            np.put_along_axis(rest, parted.argmax(2)[:, :, None], -np.inf, 2)
            worth = worth + rest.max(2)
        open_, free = np.ones((T, G), bool), np.zeros((T, G, per), bool)
        for _ in range(c["topk_groups"]):
            key = np.where(open_, worth, -np.inf)
            key = np.where(open_ & (worth == -np.inf), np.float32(-3e38), key)
            pick = key.argmax(1)
            open_[rows, pick] = False
            free[rows, pick] = True
        free = free.reshape(T, E)
    idx = np.zeros((T, c["k"]), np.int64)
    left = np.where(free, np.maximum(choice, np.float32(-3e38)), -np.inf)
    for j in range(c["k"]):
        idx[:, j] = left.argmax(1)
        left[rows, idx[:, j]] = -np.inf
    w = np.take_along_axis(p, idx, 1)
    if c["renormalise"]:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    none = dict.fromkeys(("counts", "offsets", "sorted_assign", "assign_row", "block_expert", "block_row",
                          "n_blocks"))
    return dict(topk_idx=idx.astype(np.int32), topk_w=w * c["scale"], **none)


def _exact_linear(s):
    a = s["a"].double() * s["a_scale"].double()[:, None]
    w = s["w"][0].double() * s["w_scale"][0].double()[:, None]
    return torch.mm(a, w.t().contiguous())


def _exact_ffn(x, gate, up, down, e):
    of = lambda m: (m[0][e].double() * m[1][e].double()[:, None]).t().contiguous()  # noqa: E731
    g, u = torch.mm(x, of(gate)), torch.mm(x, of(up))
    h = g * torch.special.expit(g) * u
    step = h.abs().amax(1, keepdim=True) / 127
    h = torch.where(step > 0, torch.round(h / step) * step, torch.zeros_like(h))
    return torch.mm(h, of(down))


def _exact_layer(s):
    c = s["case"]
    x = s["x"].double() * s["x_scale"].double()[:, None]
    lg = s["logits"].cpu().numpy()
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :c["k"]]
    w = np.exp(np.take_along_axis(lg, idx, 1).astype(np.float64))
    w = w / w.sum(1, keepdims=True)
    y = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        t_dev = torch.from_numpy(t).to(DEV)
        part = _exact_ffn(x[t_dev], s["gate"], s["up"], s["down"], int(e))
        y[t_dev] += part * torch.from_numpy(w[t, j]).to(DEV)[:, None]
    if c["I_sh"]:
        y += _exact_ffn(x, s["sh_gate"], s["sh_up"], s["sh_down"], 0)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "linear": _exact_linear,
            "layer": _exact_layer}[case["op"]](s)
