"""The measured cases of the router, the balance loss and the low-rank adapters.

Four kinds of pass:

  route     router logits -> the experts of every token and their weights
  balance   a training step's balance and z losses, the per-expert counts, and the gradient of the router's logits from
            them and from the gate weights
  lora      a shared projection's output plus the rows' low-rank products
  lora_grad the gradients of the rows, of both factors, from the gradient of the output

``run`` computes them in plain torch operations, or, with ``own`` set, by this framework's entry points.
"""
import math

import torch

own = False

F32_MAX = torch.finfo(torch.float32).max
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step's router: one token for each of 128 requests
        dict(name="route-decode", kind="route", T=128, E=256, K=8, score="softmax", dtype="fp32", bias=False, groups=1,
             topk_groups=1, group_top=1, normalize=True, scale=1.0, mask=0.0, closed=0.0),
        # a prefill's router: sigmoid scores, a balancing bias, experts chosen from the best 4 of 8 groups
        dict(name="route-prefill-groups", kind="route", T=4096, E=256, K=8, score="sigmoid", dtype="fp32", bias=True,
             groups=8, topk_groups=4, group_top=2, normalize=True, scale=2.5, mask=0.0, closed=0.0),
        # a packed batch of odd size with padded tokens and some experts closed, bf16 logits
        dict(name="route-packed-odd", kind="route", T=16381, E=160, K=6, score="softmax", dtype="bf16", bias=False,
             groups=1, topk_groups=1, group_top=1, normalize=False, scale=1.0, mask=0.07, closed=0.02),
        # a small model's training step
        dict(name="balance-small", kind="balance", T=128, E=8, K=2, S=1, score="softmax", dtype="fp32", normalize=True,
             scale=1.0, mask=0.0),
        # one batch-wide balance loss, sigmoid scores
        dict(name="balance-batch", kind="balance", T=4096, E=256, K=8, S=1, score="sigmoid", dtype="fp32",
             normalize=True, scale=2.5, mask=0.0),
        # a loss for each of 13 packed sequences of uneven length, padded tokens among them, bf16 logits
        dict(name="balance-sequences", kind="balance", T=16384, E=256, K=8, S=13, score="softmax", dtype="bf16",
             normalize=False, scale=1.0, mask=0.05),
        # one request being decoded, its adapter one of 32 in memory
        dict(name="lora-one-token", kind="lora", T=1, K=1, E=32, rank=16, h_in=7168, h_out=7168, rows="tokens", none=0.0),
        # a decode step of 128 requests that use 64 adapters
        dict(name="lora-decode", kind="lora", T=128, K=1, E=64, rank=16, h_in=7168, h_out=4096, rows="tokens", none=0.1),
        # a prefill of many requests' prompts
        dict(name="lora-prefill", kind="lora", T=4096, K=1, E=16, rank=32, h_in=7168, h_out=7168, rows="tokens",
             none=0.05),
        # low-rank experts on dispatched rows, about 64 rows each, an odd output width
        dict(name="lora-rows-experts", kind="lora", T=1021, K=8, E=128, rank=64, h_in=4096, h_out=2056, rows="compact",
             none=0.1),
        # fine-tuning on short uneven batches
        dict(name="lora-grad-odd", kind="lora_grad", T=531, K=1, E=5, rank=24, h_in=1032, h_out=4096, rows="tokens",
             none=0.1),
        # fine-tuning a full-width projection
        dict(name="lora-grad-batch", kind="lora_grad", T=4096, K=1, E=8, rank=32, h_in=7168, h_out=7168, rows="tokens",
             none=0.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "balance", "lora", "lora_grad"])
    if kind == "route":
        groups = rng.choice([1, 1, 4, 8])
        per = _log(rng, 2, 40 if groups > 1 else 256)
        E = max(4, groups * per)
        topk_groups = rng.randint(1, groups)
        T = min(_log(rng, 1, 16384), 4194304 // E)
        return dict(kind=kind, T=T, E=E, K=rng.randint(1, min(8, topk_groups * (E // groups))),
                    score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["bf16", "fp32"]),
                    bias=rng.random() < 0.5, groups=groups, topk_groups=topk_groups, group_top=rng.choice([1, 2]),
                    normalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), mask=rng.choice([0.0, 0.1]),
                    closed=rng.choice([0.0, 0.05]))
    if kind == "balance":
        E = _log(rng, 4, 256)
        T = _log(rng, 1, 16384)
        return dict(kind=kind, T=T, E=E, K=rng.randint(1, min(8, E)), S=rng.choice([1, 1, rng.randint(2, 40)]),
                    score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["bf16", "fp32"]),
                    normalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), mask=rng.choice([0.0, 0.1]))
    while True:
        rows = rng.choice(["tokens", "tokens", "compact"])
        K = rng.randint(2, 8) if rows == "compact" else 1
        E = _log(rng, 8 if K > 1 else 1, 128)
        c = dict(kind=kind, T=_log(rng, 1, 8192 // K), K=K, E=E, rank=8 * _log(rng, 1, 16), h_in=8 * _log(rng, 16, 896),
                 h_out=8 * _log(rng, 16, 896), rows=rows, none=rng.choice([0.0, 0.15]))
        # no more data than the largest listed case, and no more products in the plain form
        if work(c)["bytes"] <= 2.4e8 and c["T"] * K * E * c["rank"] * (c["h_in"] + c["h_out"]) <= 3.5e11:
            return c


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _logits(g, T, E, dtype, spread):
    """Logits as a trained router gives them: some experts are liked more than others by every token."""
    return (_randn(g, T, E) + spread * _randn(g, 1, E)).to(DT[dtype])


def _ids(g, c):
    """Expert (or adapter) ids [T, K], distinct within a token, some more popular than others; a share of -1 = none."""
    T, K, E = c["T"], c["K"], c["E"]
    ids = (_randn(g, T, E) + _randn(g, 1, E)).topk(K, dim=1).indices.contiguous()
    ids.view(-1)[torch.randperm(T * K, generator=g, device="cuda")[:int(c["none"] * T * K)]] = -1
    return ids


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(c)
    if c["kind"] in ("route", "balance"):
        T, E = c["T"], c["E"]
        st["logits"] = _logits(g, T, E, c["dtype"], 0.5)
        st["token_mask"] = (_rand(g, T) >= c["mask"]).to(torch.uint8) if c["mask"] else None
    if c["kind"] == "route":
        if c["closed"]:
            st["logits"][_rand(g, T, E) < c["closed"]] = -math.inf
        st["bias"] = 0.2 * _randn(g, E) if c["bias"] else None
        st["topk_idx"] = torch.empty((T, c["K"]), dtype=torch.int64, device="cuda")
        st["topk_weights"] = torch.empty((T, c["K"]), device="cuda")
        if own:
            st["router"] = _router(c)
        return st
    if c["kind"] == "balance":
        K, S = c["K"], c["S"]
        st["topk_idx"] = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True).indices[:, :K].contiguous()
        if st["token_mask"] is not None:
            st["topk_idx"][st["token_mask"] == 0] = -1
        st["d_topk_weights"] = 0.1 * _randn(g, T, K)
        cuts = (_rand(g, S - 1) * (T + 1)).to(torch.int32).clamp(max=T).sort().values
        ends = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        st["seq_offsets"] = torch.cat([ends[:1], cuts, ends[1:]]) if S > 1 else None
        st["d_losses"] = (torch.tensor([[1e-2, 1e-3]], device="cuda") / S).expand(S, 2).contiguous()
        st["d_logits"] = torch.empty_like(st["logits"])
        if own:
            from combine_ep_get_10_b200 import binding as B
            st["router"] = _router(c)
            st["stats"] = B.BalanceStats(st["router"], T, num_seqs=S)
        return st
    E, r = c["E"], c["rank"]
    ids = _ids(g, c)
    flat = ids.reshape(-1)
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices[:int((flat >= 0).sum())]  # row -> pair
    rows = c["T"] if c["rows"] == "tokens" else order.numel()
    st["ids"] = ids
    # the adapter of each row of x: its token's own, or the rows in expert order
    st["row_ids"] = flat if c["rows"] == "tokens" else flat[order]
    st["x"] = _randn(g, rows, c["h_in"]).to(torch.bfloat16)
    st["a"] = (_randn(g, E, r, c["h_in"]) / math.sqrt(c["h_in"])).to(torch.bfloat16)
    st["b"] = (_randn(g, E, c["h_out"], r) / math.sqrt(r)).to(torch.bfloat16)
    st["scales"] = 0.25 + _rand(g, E)
    if c["kind"] == "lora":
        st["base"] = _randn(g, rows, c["h_out"]).to(torch.bfloat16)
        st["out"] = torch.empty_like(st["base"])
        st["h"] = torch.empty((max(1, order.numel()), r), device="cuda")
    else:
        st["dy"] = _randn(g, rows, c["h_out"]).to(torch.bfloat16)
        st["dx_base"] = _randn(g, rows, c["h_in"]).to(torch.bfloat16)
        # what the forward pass kept: the scaled products with the first factor, one row for each routed row
        at = order // c["K"] if c["rows"] == "tokens" else torch.arange(rows, device="cuda")
        st["h_at"] = at
        st["h"] = torch.empty((max(1, order.numel()), r), device="cuda")
        for e in range(E):
            sel = (flat[order] == e).nonzero().squeeze(1)
            st["h"][sel] = st["scales"][e] * (st["x"][at[sel]].float() @ st["a"][e].float().T)
        st["dh"], st["dx"] = torch.empty_like(st["h"]), torch.empty_like(st["x"])
        st["da"], st["db"] = torch.empty_like(st["a"]), torch.empty_like(st["b"])
    if own:
        from combine_ep_get_10_b200 import binding as B
        st["routing"] = B.Routing.topk(ids, E, 1)
        st["layout"] = B.ep_get_layout(st["routing"], B.Layout(st["routing"]))
        st["lora"] = B.Lora(st["a"], st["b"], scales=st["scales"])
        st["row_token"] = None
        if c["rows"] == "tokens":
            st["row_token"] = torch.empty(c["T"], dtype=torch.int32, device="cuda")
            B.ep_row_tokens(st["routing"], st["layout"], st["row_token"])
    return st


def _router(c):
    from combine_ep_get_10_b200 import binding as B
    return B.Router(c["E"], c["K"], score=B.EP_SCORE_SIGMOID if c["score"] == "sigmoid" else B.EP_SCORE_SOFTMAX,
                    num_groups=c.get("groups", 1), topk_groups=c.get("topk_groups", 1),
                    group_top=c.get("group_top", 1), normalize=c["normalize"], scale=c["scale"])


# ----------------------------------------------------------------------------- one pass
def run(st):
    if own:
        return _run_own(st)
    return {"route": _route, "balance": _balance, "lora": _lora, "lora_grad": _lora_grad}[st["kind"]](st)


def _run_own(st):
    from combine_ep_get_10_b200 import binding as B
    kind = st["kind"]
    if kind == "route":
        B.ep_router_topk(st["logits"], st["router"], st["topk_idx"], st["topk_weights"], bias=st["bias"],
                         token_mask=st["token_mask"])
        return {"topk_idx": st["topk_idx"], "topk_weights": st["topk_weights"]}
    if kind == "balance":
        s = st["stats"]
        B.ep_balance_loss(st["logits"], st["router"], st["topk_idx"], s, token_mask=st["token_mask"],
                          seq_offsets=st["seq_offsets"])
        B.ep_router_backward(st["logits"], st["router"], st["topk_idx"], st["d_logits"],
                             d_topk_weights=st["d_topk_weights"], stats=s, d_losses=st["d_losses"],
                             token_mask=st["token_mask"], seq_offsets=st["seq_offsets"])
        return {"losses": s.losses, "counts": s.counts, "mean_scores": s.mean_scores, "d_logits": st["d_logits"]}
    if kind == "lora":
        B.ep_lora(st["x"], st["routing"], st["layout"], st["lora"], st["out"], st["h"], base=st["base"],
                  row_token=st["row_token"])
        return {"out": st["out"]}
    B.ep_lora_backward(st["dy"], st["x"], st["h"], st["routing"], st["layout"], st["lora"], st["dh"], dx=st["dx"],
                       da=st["da"], db=st["db"], dx_base=st["dx_base"], row_token=st["row_token"])
    return {"dx": st["dx"], "da": st["da"], "db": st["db"]}


def _open(l):
    """Which logits take part: -inf and NaN close an expert; a value above the largest finite one counts as that."""
    return l > -math.inf


def _safe(l, fill):
    return torch.where(_open(l), l.clamp(max=F32_MAX), torch.full_like(l, fill))


def _softmax(l):
    """Softmax over the open logits; a row with none gives zeros."""
    l = _safe(l, -math.inf)
    m = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    return e / e.sum(dim=1, keepdim=True).clamp(min=1e-300 if l.dtype == torch.float64 else 1e-30)


def _scores(l, score):
    if score == "softmax":
        return _softmax(l)
    return torch.where(_open(l), torch.sigmoid(_safe(l, 0.0)), torch.zeros_like(l))


def _route(st):
    l = st["logits"]
    T, E = l.shape
    # the choice, in 64 bits: neighbours in the order may be closer than 32 bits tell apart
    wide = l.double()
    if st["bias"] is None and st["groups"] == 1:
        choice = _safe(wide, -math.inf)
    else:
        choice = _scores(wide, st["score"])
        if st["bias"] is not None:
            choice = choice + st["bias"].double()
        choice = torch.where(_open(wide), choice, torch.full_like(choice, -math.inf))
    if st["token_mask"] is not None:
        choice = torch.where((st["token_mask"] != 0)[:, None], choice, torch.full_like(choice, -math.inf))
    if st["groups"] > 1:
        grouped = choice.view(T, st["groups"], -1)
        best = torch.sort(grouped, dim=2, descending=True).values[:, :, :st["group_top"]]
        total = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(dim=2)
        total = torch.where(best[:, :, 0] > -math.inf, total, torch.full_like(total, -math.inf))
        kept = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :st["topk_groups"]]
        stay = torch.zeros_like(total, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(stay[:, :, None], grouped, torch.full_like(grouped, -math.inf)).view(T, E)
    top = torch.sort(choice, dim=1, descending=True, stable=True)
    taken = top.values[:, :st["K"]] > -math.inf
    idx = top.indices[:, :st["K"]]
    # the weights, in 32 bits
    w = torch.where(taken, torch.gather(_scores(l.float(), st["score"]), 1, idx), torch.zeros((), device=l.device))
    if st["normalize"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-30)
    return {"topk_idx": torch.where(taken, idx, torch.full_like(idx, -1)), "topk_weights": st["scale"] * w}


def _sequence_of(st, T, device):
    if st["seq_offsets"] is None:
        return torch.zeros(T, dtype=torch.int64, device=device)
    at = torch.arange(T, dtype=torch.int32, device=device)
    return torch.searchsorted(st["seq_offsets"][1:].contiguous(), at, right=True)


def _balance(st):
    l = st["logits"].float()
    T, E = l.shape
    K, S, dev = st["K"], st["S"], l.device
    idx = st["topk_idx"]
    seq = _sequence_of(st, T, dev)
    live = torch.ones(T, dtype=torch.bool, device=dev) if st["token_mask"] is None else st["token_mask"] != 0
    part = live.float()
    p = _softmax(l)
    s = _scores(l, st["score"])
    q = p if st["score"] == "softmax" else s / s.sum(dim=1, keepdim=True)
    lse = torch.logsumexp(l, dim=1)
    # one row of 0s and 1s for each sequence: sums over its tokens are products with it
    member = torch.zeros((S, T), device=dev).scatter_(0, seq[None, :], part[None, :])
    n = member.sum(dim=1)
    nz = n.clamp(min=1.0)
    hit = torch.zeros((T, E + 1), device=dev).scatter_add_(
        1, torch.where(idx >= 0, idx, torch.full_like(idx, E)), torch.ones(idx.shape, device=dev))[:, :E]
    counts = member @ hit
    mean = (member @ q) / nz[:, None]
    f = counts * (E / (K * nz))[:, None]
    losses = torch.stack([(f * mean).sum(dim=1), (member @ (lse * lse)) / nz], dim=1)
    # the gradient of the logits
    db, dz = st["d_losses"][seq, 0], st["d_losses"][seq, 1]
    gain = (db * part / nz[seq])[:, None] * f[seq]
    flat = gain - (gain * q).sum(dim=1, keepdim=True)
    d = q * flat if st["score"] == "softmax" else q * (1 - s) * flat
    d = d + (dz * part * 2 * lse / nz[seq])[:, None] * p
    taken = (idx >= 0) & live[:, None]
    at = torch.where(taken, idx, torch.zeros_like(idx))
    dw = torch.where(taken, st["scale"] * st["d_topk_weights"], torch.zeros((), device=dev))
    sel = torch.where(taken, torch.gather(s, 1, at), torch.zeros((), device=dev))
    if st["normalize"]:
        total = sel.sum(dim=1, keepdim=True).clamp(min=1e-30)
        dw = (dw - (dw * sel).sum(dim=1, keepdim=True) / total) / total
    ds = torch.zeros((T, E), device=dev).scatter_add_(1, at, torch.where(taken, dw, torch.zeros((), device=dev)))
    if st["score"] == "softmax":
        d = d + p * (ds - (ds * p).sum(dim=1, keepdim=True))
    else:
        d = d + ds * s * (1 - s)
    return {"losses": losses, "counts": counts.to(torch.int32), "mean_scores": mean, "d_logits": d.to(st["logits"].dtype)}


def _pick(st):
    """[rows, E] of 0s and scales: which adapter each row uses."""
    ids, E = st["row_ids"], st["E"]
    rows = torch.zeros((ids.numel(), E + 1), device=ids.device)
    return rows.scatter_(1, torch.where(ids >= 0, ids, torch.full_like(ids, E))[:, None], 1.0)[:, :E]


def _lora(st):
    E, r = st["E"], st["rank"]
    pick = _pick(st) * st["scales"]
    u = (st["x"].float() @ st["a"].float().view(E * r, -1).T).view(-1, E, r) * pick[:, :, None]
    delta = u.view(-1, E * r) @ st["b"].float().transpose(1, 2).reshape(E * r, -1)
    return {"out": (st["base"].float() + delta).to(torch.bfloat16)}


def _lora_grad(st):
    E, r = st["E"], st["rank"]
    pick = _pick(st)
    dy, x = st["dy"].float(), st["x"].float()
    b = st["b"].float().transpose(1, 2).reshape(E * r, -1)
    dh = (dy @ b.T).view(-1, E, r) * (pick * st["scales"])[:, :, None]
    dh = dh.view(-1, E * r)
    dx = st["dx_base"].float() + dh @ st["a"].float().view(E * r, -1)
    da = (dh.T @ x).view(E, r, -1)
    u = torch.zeros((x.shape[0], r), device=x.device)
    u[st["h_at"]] = st["h"][:st["h_at"].numel()]
    u = (u[:, None, :] * pick[:, :, None]).view(-1, E * r)
    db = (u.T @ dy).view(E, r, -1).transpose(1, 2)
    return {"dx": dx.to(torch.bfloat16), "da": da.to(torch.bfloat16), "db": db.to(torch.bfloat16).contiguous()}


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["kind"] == "route":
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": c["T"] * (c["E"] * size + c["K"] * 12), "flops": 8 * c["T"] * c["E"]}
    if c["kind"] == "balance":
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": c["T"] * (2 * c["E"] * size + c["K"] * 12) + c["S"] * c["E"] * 8, "flops": 20 * c["T"] * c["E"]}
    pairs = c["T"] * c["K"] - int(c["none"] * c["T"] * c["K"])
    rows = c["T"] if c["rows"] == "tokens" else pairs
    used = min(c["E"], pairs)
    wide = c["h_in"] + c["h_out"]
    if c["kind"] == "lora":
        return {"bytes": 2 * (pairs * c["h_in"] + 2 * rows * c["h_out"] + used * c["rank"] * wide),
                "flops": 2 * pairs * c["rank"] * wide}
    return {"bytes": 2 * (pairs * wide + 2 * rows * c["h_in"] + used * c["rank"] * wide + c["E"] * c["rank"] * wide)
            + 4 * pairs * c["rank"], "flops": 4 * pairs * c["rank"] * wide}


# ----------------------------------------------------------------------------- 64 bits, from the definitions
def _route_exact(st):
    l = st["logits"].double()
    T, E = l.shape
    neg = torch.tensor(-math.inf, dtype=torch.float64, device=l.device)
    shut = torch.isneginf(l) | torch.isnan(l)
    l = torch.where(shut, neg, l)
    if st["score"] == "softmax":
        s = torch.exp(l - torch.logsumexp(l, dim=1, keepdim=True)).nan_to_num(0.0)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    key = l if st["bias"] is None and st["groups"] == 1 else s + (0.0 if st["bias"] is None else st["bias"].double())
    key = torch.where(shut, neg, key)
    if st["token_mask"] is not None:
        key[st["token_mask"] == 0] = -math.inf
    if st["groups"] > 1:
        per = E // st["groups"]
        sums = []
        for g in range(st["groups"]):
            part = key[:, g * per:(g + 1) * per].sort(dim=1, descending=True).values[:, :st["group_top"]]
            none = torch.isneginf(part[:, 0])
            sums.append(torch.where(none, neg, part.masked_fill(torch.isneginf(part), 0.0).sum(dim=1)))
        sums = torch.stack(sums, dim=1)
        for g in range(st["groups"]):  # a group goes when topk_groups others are before it
            before = (sums > sums[:, g:g + 1]).sum(dim=1) + (sums[:, :g] == sums[:, g:g + 1]).sum(dim=1)
            key[:, g * per:(g + 1) * per][before >= st["topk_groups"]] = -math.inf
    idx, w = [], []
    for _ in range(st["K"]):
        best = key.amax(dim=1, keepdim=True)
        first = (key == best).to(torch.uint8).argmax(dim=1)  # the lowest id among equals
        got = ~torch.isneginf(best[:, 0])
        idx.append(torch.where(got, first, torch.full_like(first, -1)))
        w.append(torch.where(got, s[torch.arange(T, device=l.device), first], torch.zeros_like(best[:, 0])))
        key[torch.arange(T, device=l.device), first] = -math.inf
    w = torch.stack(w, dim=1)
    if st["normalize"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, w)
    return {"topk_idx": torch.stack(idx, dim=1), "topk_weights": w * st["scale"]}


def _balance_exact(st):
    l = st["logits"].double().requires_grad_(True)
    T, E = l.shape
    K, S = st["K"], st["S"]
    live = torch.ones(T, dtype=torch.bool, device=l.device) if st["token_mask"] is None else st["token_mask"].bool()
    cuts = [0, T] if st["seq_offsets"] is None else st["seq_offsets"].tolist()
    s = torch.softmax(l, dim=1) if st["score"] == "softmax" else torch.sigmoid(l)
    q = s / s.sum(dim=1, keepdim=True)
    lse = torch.logsumexp(l, dim=1)
    idx, losses, counts, means = st["topk_idx"], [], [], []
    for i in range(S):
        at = torch.arange(cuts[i], cuts[i + 1], device=l.device)
        at = at[live[at]]
        n = at.numel()
        count = torch.bincount(idx[at][idx[at] >= 0].reshape(-1), minlength=E)
        counts.append(count)
        if n == 0:
            means.append(torch.zeros(E, dtype=torch.float64, device=l.device))
            losses.append(torch.zeros(2, dtype=torch.float64, device=l.device))
            continue
        means.append(q[at].sum(dim=0) / n)
        losses.append(torch.stack([(count.double() * E / (K * n) * means[-1]).sum(), (lse[at] ** 2).sum() / n]))
    losses = torch.stack(losses)
    taken = (idx >= 0) & live[:, None]
    w = torch.where(taken, torch.gather(s, 1, idx.clamp(min=0)), torch.zeros((), dtype=torch.float64, device=l.device))
    if st["normalize"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    whole = (losses * st["d_losses"].double()).sum() + (st["scale"] * w * st["d_topk_weights"].double()).sum()
    grad, = torch.autograd.grad(whole, l)
    return {"losses": losses.detach(), "counts": torch.stack(counts).to(torch.int32),
            "mean_scores": torch.stack(means).detach(), "d_logits": grad}


def _lora_exact(st):
    out = st["base"].double()
    for e in range(st["E"]):
        at = (st["row_ids"] == e).nonzero().squeeze(1)
        h = st["x"][at].double() @ st["a"][e].double().T
        out[at] += st["scales"][e].double() * (h @ st["b"][e].double().T)
    return {"out": out}


def _lora_grad_exact(st):
    dx = st["dx_base"].double()
    da = torch.zeros(st["a"].shape, dtype=torch.float64, device=dx.device)
    db = torch.zeros(st["b"].shape, dtype=torch.float64, device=dx.device)
    h = torch.zeros((dx.shape[0], st["rank"]), dtype=torch.float64, device=dx.device)
    h[st["h_at"]] = st["h"][:st["h_at"].numel()].double()
    for e in range(st["E"]):
        at = (st["row_ids"] == e).nonzero().squeeze(1)
        dy = st["dy"][at].double()
        dh = st["scales"][e].double() * (dy @ st["b"][e].double())
        dx[at] += dh @ st["a"][e].double()
        da[e] = dh.T @ st["x"][at].double()
        db[e] = dy.T @ h[at]
    return {"dx": dx, "da": da, "db": db}


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _route_exact, "balance": _balance_exact, "lora": _lora_exact, "lora_grad": _lora_grad_exact}[st["kind"]](st)
