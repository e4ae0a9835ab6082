"""Measured cases of the grouped router, the multi-adapter projection and the
shared expert: each operator in its plain form (elementary torch products,
exponentials, comparisons and indexing) and as the calls a serving program
makes of aware_expert_routing_amd.

  route       scores (softmax or sigmoid) -> selection values (+ a per-expert
              balance bias) -> the best groups -> the top k inside them ->
              unbiased weights, renormalised and scaled.
  dispatch    the same, followed by the token permutation the expert FFN reads.
  lora        y_i = W x_i + s_a B_a A_a x_i, a the adapter of token i.
  shared      a SwiGLU FFN every token passes, with adapters of many requests
              on its gate, up and down projections.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _route(name, B, N, k, score, G, topk_group, group_score, bias, renorm, scale, dtype, op="route"):
    return {"name": name, "op": op, "B": B, "N": N, "k": k, "score": score, "groups": G, "topk_group": topk_group,
            "group_score": group_score, "bias": bias, "renorm": renorm, "scale": scale, "dtype": dtype}


def _lora(name, B, H, O, R, ranks, runs, x, y):
    return {"name": name, "op": "lora", "B": B, "H": H, "O": O, "adapters": R, "ranks": ranks, "runs": runs,
            "x": x, "y": y}


def _shared(name, B, H, I, R, ranks, runs, x, y):
    return {"name": name, "op": "shared", "B": B, "H": H, "I": I, "adapters": R, "ranks": ranks, "runs": runs,
            "x": x, "y": y}


def listed():
    return [
        # one decoding request: a sigmoid router with a balance bias and groups (latency only)
        _route("route_one", 1, 256, 8, "sigmoid", 8, 4, "top2", True, True, 2.5, "f32"),
        # an uneven batch on a softmax router that keeps raw probabilities, groups ranked by their best expert
        _route("route_softmax_77", 77, 160, 6, "softmax", 8, 3, "max", False, False, 16.0, "bf16"),
        # a long prompt chunk through the sigmoid router
        _route("route_prompt", 16384, 256, 8, "sigmoid", 8, 4, "top2", True, True, 2.5, "f32"),
        # a full decode batch routed and dispatched for the expert FFN
        _route("dispatch_128", 128, 128, 8, "sigmoid", 8, 4, "top2", True, True, 1.0, "f32", op="dispatch"),
        # one request with its adapter on a square projection (latency)
        _lora("lora_one", 1, 2048, 2048, 4, "16", False, "bf16", "bf16"),
        # float activations, an odd batch, ranks that differ and are no multiple of 16
        _lora("lora_f32_13", 13, 2048, 768, 6, "4,8,24", False, "f32", "f32"),
        # a decode batch that mixes many adapters in every group of tokens
        _lora("lora_mixed_64", 64, 4096, 4096, 24, "8,16,32,64", False, "bf16", "bf16"),
        # prompt chunks of a few requests in one batch, tokens of a request side by side
        _lora("lora_prompts", 4096, 4096, 4096, 8, "16,32,64", True, "bf16", "bf16"),
        # the shared expert of one decoding request, added to float outputs
        _shared("shared_one", 1, 2048, 768, 4, "16", False, "bf16", "f32"),
        # an ordinary decode batch
        _shared("shared_32", 32, 2048, 768, 12, "8,16,32", False, "bf16", "f32"),
        # the largest decode batch on the wide shape, many adapters
        _shared("shared_128", 128, 4096, 1536, 24, "16,64", False, "bf16", "f32"),
        # a ragged prompt batch of a few requests
        _shared("shared_prompts", 2999, 4096, 1536, 6, "16,32", True, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "dispatch", "lora", "lora", "shared", "shared"])
    if op in ("route", "dispatch"):
        G = rng.choice([1, 1, 2, 4, 8, 16])
        per = _log(rng, 2, (512 if op == "route" else 128) // G)
        N = G * per
        topk_group = rng.randint(1, G)
        k = rng.randint(1, min(16, topk_group * per))
        B = _log(rng, 1, 16384 * 256 // max(N, 256)) if op == "route" else _log(rng, 1, 128)
        return _route("", B, N, k, rng.choice(["softmax", "sigmoid"]), G, topk_group, rng.choice(["max", "top2"]),
                      rng.random() < 0.6, rng.random() < 0.7, rng.choice([1.0, 2.5, 16.0]),
                      rng.choice(["f32", "bf16"]) if op == "route" else "f32", op=op)
    # (H and O in steps of the packed tiles)
    B = _log(rng, 1, 4096)
    H = 32 * _log(rng, 8, 128)
    R = _log(rng, 1, 32)
    ranks = ",".join(str(_log(rng, 1, 64)) for _ in range(rng.randint(1, 3)))
    runs = B > 256 and rng.random() < 0.7
    if op == "lora":
        x = rng.choice(["bf16", "bf16", "f32"])
        if x == "f32":
            B = min(B, 1024)
        return _lora("", B, H, 16 * _log(rng, 8, 256), R, ranks, runs, x, rng.choice(["bf16", "f32"]))
    y = rng.choice(["bf16", "f32"])
    return _shared("", min(B, 2048), H, 32 * _log(rng, 4, 48), R, ranks, runs, "bf16", y)


# --------------------------------------------------------------------------
# inputs (made from the seed alone)
# --------------------------------------------------------------------------
_T = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _rank_list(case):
    r = [int(v) for v in case["ranks"].split(",")]
    return [r[a % len(r)] for a in range(case["adapters"])]


def _adapter_ids(case, g):
    """Every adapter in turn, in shuffled order or as runs; every ninth entry of the turn has no adapter."""
    B, R = case["B"], case["adapters"]
    i = torch.arange(B, device=DEV)
    turn = i * (R + 1) // B if case["runs"] else i % (R + 1)
    ids = torch.where((turn == R) | ((i % 9 == 8) & (not case["runs"])), torch.full_like(turn, -1), turn)
    if not case["runs"]:
        ids = ids[torch.randperm(B, generator=g, device=DEV)]
    return ids.to(torch.int32)


def _pair(case, g, H, O):
    """One adapter (A, B, scale) for each entry of the table, as a trained one: A about 1/sqrt(H), B small."""
    out = []
    for a, r in enumerate(_rank_list(case)):
        out.append((_normal(g, (r, H), H ** -0.5, torch.bfloat16), _normal(g, (O, r), 0.2, torch.bfloat16),
                    0.25 + 0.125 * (a % 8)))
    return out


def _inputs(case, seed):
    g = _gen(seed)
    if case["op"] in ("route", "dispatch"):
        # router logits with a few favoured experts; a bias that balances part of it
        favour = torch.randn(case["N"], generator=g, device=DEV) * 0.7
        logits = (torch.randn(case["B"], case["N"], generator=g, device=DEV) * 1.3 + favour).to(_T[case["dtype"]])
        bias = (-0.1 * favour + 0.02 * torch.randn(case["N"], generator=g, device=DEV)) if case["bias"] else None
        return {"logits": logits, "bias": bias}
    B, H = case["B"], case["H"]
    d = {"x": _normal(g, (B, H), 1.0, _T[case["x"]]), "ids": _adapter_ids(case, g)}
    if case["op"] == "lora":
        d["w"] = _normal(g, (case["O"], H), 0.02, torch.bfloat16)
        d["adapters"] = _pair(case, g, H, case["O"])
    else:
        I = case["I"]
        d["gate"], d["up"] = (_normal(g, (I, H), 0.02, torch.bfloat16) for _ in range(2))
        d["down"] = _normal(g, (H, I), 0.02, torch.bfloat16)
        d["a_gate"], d["a_up"], d["a_down"] = _pair(case, g, H, I), _pair(case, g, H, I), _pair(case, g, I, H)
    return d


def _stack(case, adapters):
    """Adapters side by side for the plain form: A [sum r, H], B [O, sum r], the adapter and the scale of each row of A."""
    who = torch.tensor([a for a, (A, _, _) in enumerate(adapters) for _ in range(A.shape[0])], device=DEV,
                       dtype=torch.int32)
    scale = torch.tensor([s for A, _, s in adapters for _ in range(A.shape[0])], device=DEV)
    return {"A": torch.cat([A for A, _, _ in adapters]), "B": torch.cat([b for _, b, _ in adapters], 1).contiguous(),
            "who": who, "scale": scale}


def prepare(case, seed):
    d = _inputs(case, seed)
    st = {"case": case, **d}
    op = case["op"]
    if not own:
        for name in ("adapters", "a_gate", "a_up", "a_down"):
            if name in d:
                st[name] = _stack(case, d[name])
        return st
    import aware_expert_routing_amd as moe
    st["moe"] = moe
    if op in ("route", "dispatch"):
        B, N, k = case["B"], case["N"], case["k"]
        i32 = dict(device=DEV, dtype=torch.int32)
        st["route"] = {"idx": torch.empty(B, k, **i32), "w": torch.empty(B, k, device=DEV)}
        if op == "dispatch":
            T = torch.empty(1, **i32)
            st["disp"] = {"cnt": torch.empty(N, **i32), "offsets": torch.empty(N + 1, **i32),
                          "perm": torch.empty(B * k, **i32), "active": torch.empty(N, **i32), "T": T}
            st["sync"] = torch.zeros(1, **i32)
        return st
    B, H = case["B"], case["H"]
    top = max(_rank_list(case))

    def table(adapters, h, o):
        t = moe.LoraTable(len(adapters), h, o, top, DEV)
        for a, (A, b, s) in enumerate(adapters):
            t.publish(a, A, b, s)
        return t

    if op == "lora":
        O = case["O"]
        st["packed"] = moe.pack_weights(moe.MOE_W_BF16, d["w"])[0]
        st["table"] = table(d["adapters"], H, O)
        st["y"] = torch.empty(B, O, device=DEV, dtype=_T[case["y"]])
        st["ws"] = torch.empty(moe.lora_workspace_bytes(B, H, O, top, d["x"].dtype, st["y"].dtype), device=DEV,
                               dtype=torch.uint8)
    else:
        I = case["I"]
        st["shared"] = moe.ExpertTensors.pack(moe.MOE_W_BF16, d["gate"], d["up"], d["down"])
        st["tables"] = (table(d["a_gate"], H, I), table(d["a_up"], H, I), table(d["a_down"], I, H))
        st["y"] = torch.empty(B, H, device=DEV, dtype=_T[case["y"]])
        st["ws"] = torch.empty(moe.shared_ffn_workspace_bytes(B, H, I, top, d["x"].dtype, st["y"].dtype), device=DEV,
                               dtype=torch.uint8)
    return st


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _plain_route(case, logits, bias):
    B, N = logits.shape
    G, per, k = case["groups"], case["N"] // case["groups"], case["k"]
    l = logits.double()          # the order of close selection values is decided in 64 bits
    if case["score"] == "softmax":
        e = torch.exp(l - l.max(1, keepdim=True).values)
        s = e / e.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    choice = l if bias is None else s + bias.double()
    if G > 1:
        if case["group_score"] == "max" or per == 1:
            value = choice.view(B, G, per).max(2).values
        else:
            value = (s if bias is None else choice).view(B, G, per).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        keep = value.sort(dim=1, descending=True, stable=True).indices[:, :case["topk_group"]]
        mask = torch.zeros(B, G, device=logits.device, dtype=torch.bool).scatter_(1, keep, True)
        choice = torch.where(mask.repeat_interleave(per, 1), choice, torch.full_like(choice, -math.inf))
    idx = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.to(torch.int32), (w * case["scale"]).float()


def _plain_dispatch(idx, N):
    B, k = idx.shape
    flat = idx.reshape(-1).long()
    cnt = (flat[:, None] == torch.arange(N, device=idx.device)[None, :]).sum(0)
    offsets = torch.cat([torch.zeros_like(cnt[:1]), cnt.cumsum(0)])
    perm = flat.sort(stable=True).indices          # by (expert, token)
    e = torch.arange(N, device=idx.device)
    order = torch.where(cnt > 0, e, e + N).sort().values
    active = torch.where(order < N, order, torch.full_like(order, -1))
    return [v.to(torch.int32) for v in (cnt, offsets, perm, active, (cnt > 0).sum().reshape(1))]


def _plain_lora(x, w, t, ids):
    """x (32 bits) through w and the adapters: every adapter's rows at once, those of other tokens set to zero."""
    v = x @ t["A"].float().T
    v = v * ((ids[:, None] == t["who"][None, :]).float() * t["scale"])
    return x @ w.float().T + v @ t["B"].float().T


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        moe = st["moe"]
        if op == "route":
            return moe.route_grouped(st["logits"], case["k"], score=case["score"], bias=st["bias"],
                                     n_group=case["groups"], topk_group=case["topk_group"],
                                     group_score=case["group_score"], renorm=case["renorm"], scale=case["scale"],
                                     idx=st["route"]["idx"], w=st["route"]["w"])
        if op == "dispatch":
            r, d = moe.route_grouped_dispatch(st["logits"], case["k"], score=case["score"], bias=st["bias"],
                                              n_group=case["groups"], topk_group=case["topk_group"],
                                              group_score=case["group_score"], renorm=case["renorm"],
                                              scale=case["scale"], route=st["route"], disp=st["disp"],
                                              sync=st["sync"])
            return [r["idx"], r["w"], d["cnt"], d["offsets"], d["perm"], d["active"], d["T"]]
        if op == "lora":
            return moe.lora_linear(st["x"], st["packed"], st["table"], st["ids"], y=st["y"], ws=st["ws"])
        return moe.shared_ffn(st["x"], st["shared"], st["tables"], st["ids"], y=st["y"], ws=st["ws"])
    if op == "route":
        return _plain_route(case, st["logits"], st["bias"])
    if op == "dispatch":
        idx, w = _plain_route(case, st["logits"], st["bias"])
        return [idx, w] + _plain_dispatch(idx, case["N"])
    x = st["x"].float()
    if op == "lora":
        return _plain_lora(x, st["w"], st["adapters"], st["ids"]).to(_T[case["y"]])
    g = _plain_lora(x, st["gate"], st["a_gate"], st["ids"])
    u = _plain_lora(x, st["up"], st["a_up"], st["ids"])
    h = g / (1.0 + torch.exp(-g)) * u
    return _plain_lora(h, st["down"], st["a_down"], st["ids"]).to(_T[case["y"]])


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def _counts(case):
    """(adapters used, rows of A they have together, sum over tokens of their rank) of _adapter_ids."""
    B, R, ranks = case["B"], case["adapters"], _rank_list(case)
    tokens = [0] * R
    for i in range(B):
        turn = i * (R + 1) // B if case["runs"] else i % (R + 1)
        if turn < R and (case["runs"] or i % 9 != 8):
            tokens[turn] += 1
    used = [a for a in range(R) if tokens[a]]
    return sum(ranks[a] for a in used), sum(ranks[a] * tokens[a] for a in used)


def work(case):
    size = {"f32": 4, "bf16": 2}
    B = case["B"]
    if case["op"] in ("route", "dispatch"):
        N, k = case["N"], case["k"]
        out = B * k * 8
        if case["op"] == "dispatch":
            out += B * k * 4 + (3 * N + 2) * 4
        return {"bytes": B * N * size[case["dtype"]] + (N * 4 if case["bias"] else 0) + out, "flops": 8 * B * N}
    H = case["H"]
    rows, row_tokens = _counts(case)
    if case["op"] == "lora":
        O = case["O"]
        return {"bytes": O * H * 2 + rows * (H + O) * 2 + B * (H * size[case["x"]] + O * size[case["y"]] + 4),
                "flops": 2 * B * H * O + 2 * row_tokens * (H + O)}
    I = case["I"]
    return {"bytes": 3 * I * H * 2 + 3 * rows * (H + I) * 2 + B * (H * size[case["x"]] + H * size[case["y"]] + 4),
            "flops": 6 * B * H * I + 6 * row_tokens * (H + I)}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_linear(x, w, adapters, ids):
    y = x.matmul(w.double().t())
    for a, (A, b, s) in enumerate(adapters):
        at = (ids == a).nonzero().flatten()
        if at.numel():
            y[at] += s * x[at].matmul(A.double().t()).matmul(b.double().t())
    return y


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] in ("route", "dispatch"):
        # the weights of the experts the definition picks, in the order of their picking
        l = d["logits"].double()
        score = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
        pick = l.clone() if d["bias"] is None else score + d["bias"].double()
        rows = torch.arange(case["B"], device=DEV)
        per = case["N"] // case["groups"]
        if case["groups"] > 1:
            first, second = (pick if case["group_score"] == "max" or d["bias"] is not None else score).clone(), None
            by_group = first.view(case["B"], case["groups"], per)
            best = by_group.max(2)
            value = best.values.clone()
            if case["group_score"] == "top2" and per > 1:
                second = by_group.scatter(2, best.indices[:, :, None], -math.inf).max(2).values
                value = value + second
            left = value
            allowed = torch.zeros(case["B"], case["groups"], dtype=torch.bool, device=DEV)
            for _ in range(case["topk_group"]):
                j = left.argmax(1)
                allowed[rows, j] = True
                left[rows, j] = -math.inf
            pick = pick.masked_fill(~allowed[:, torch.arange(case["N"], device=DEV) // per], -math.inf)
        w = []
        for _ in range(case["k"]):
            e = pick.argmax(1)
            w.append(score[rows, e])
            pick[rows, e] = -math.inf
        w = torch.stack(w, 1)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        w = w * case["scale"]
        return (None, w) if case["op"] == "route" else [None, w, None, None, None, None, None]
    x = d["x"].double()
    if case["op"] == "lora":
        return _exact_linear(x, d["w"], d["adapters"], d["ids"])
    g = _exact_linear(x, d["gate"], d["a_gate"], d["ids"])
    u = _exact_linear(x, d["up"], d["a_up"], d["ids"])
    return _exact_linear(g * torch.sigmoid(g) * u, d["down"], d["a_down"], d["ids"])
