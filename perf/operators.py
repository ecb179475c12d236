"""Workloads of the serving operators around the tree verification, with their plain forms.

A hybrid model (Gated DeltaNet layers with attention layers between them) that serves with
tree speculative decoding needs, next to the verification and the commit of a draft tree:

  prefill       the gated delta rule over whole prompts (ragged batch, states in a pool)
  decode_step   the gated delta rule for one token a sequence (no draft to verify)
  attend        attention of draft trees (or single tokens) over a paged cache whose first
                part, the prefix, is shared by every sequence of the batch
  cache_append  the accepted rows (or a prompt's) written to the pages of their sequences

`listed()` are workloads worth timing, `draw()` more of the same ranges, `prepare()` makes the
inputs, `run()` is one call, `exact()` the same in 64 bits, `work()` what a call has to move
and compute.  With `own` false, `run()` evaluates the operators with elementary torch
operations in 32 bits; with `own` true it calls the library.
"""

import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}
_ES = {BF16: 2, F32: 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one short prompt, 16 qk heads shared by 32 v heads: the latency of a first token
        dict(name="prefill-512", op="prefill", B=1, lo=512, hi=512, Hqk=16, Hv=32, dk=128, dv=128,
             dtype=BF16),
        # a batch of prompts of very different lengths, as a scheduler packs them
        dict(name="prefill-ragged", op="prefill", B=16, lo=17, hi=2048, Hqk=16, Hv=32, dk=128,
             dv=128, dtype=BF16),
        # one long document
        dict(name="prefill-32k", op="prefill", B=1, lo=32768, hi=32768, Hqk=16, Hv=32, dk=128,
             dv=128, dtype=BF16),
        # the 32-bit variant at small, unequal head sizes
        dict(name="prefill-f32", op="prefill", B=3, lo=1, hi=201, Hqk=2, Hv=4, dk=32, dv=48,
             dtype=F32),
        # one sequence's next token: launch latency
        dict(name="step-1", op="decode_step", B=1, Hqk=16, Hv=32, dk=128, dv=128, dtype=BF16),
        # a full serving batch: 512 MB of states read and written
        dict(name="step-256", op="decode_step", B=256, Hqk=16, Hv=32, dk=128, dv=128, dtype=BF16),
        # one sequence's next token over a short cache: launch latency
        dict(name="attend-1", op="attend", B=1, n_lo=1, n_hi=1, prefix=0, c_lo=300, c_hi=300,
             Hq=32, Hkv=8, D=128, page=16, dtype=BF16),
        # parallel samples of one long prompt, a token each: the cache of the prompt is shared
        dict(name="attend-shared-64", op="attend", B=64, n_lo=1, n_hi=1, prefix=32768, c_lo=1,
             c_hi=512, Hq=32, Hkv=8, D=128, page=64, dtype=BF16),
        # the serving batch of the tree verification: 32 trees of 128 nodes, a common system
        # prompt, and a conversation of its own for each
        dict(name="attend-trees-32", op="attend", B=32, n_lo=128, n_hi=128, prefix=1024, c_lo=256,
             c_hi=4096, Hq=32, Hkv=8, D=128, page=64, dtype=BF16),
        # the 32-bit variant: ragged trees, pages of 24 rows
        dict(name="attend-f32", op="attend", B=3, n_lo=1, n_hi=40, prefix=77, c_lo=1, c_hi=200,
             Hq=6, Hkv=2, D=64, page=24, dtype=F32),
        # the accepted paths of the serving batch, up to 24 nodes each
        dict(name="append-paths-32", op="cache_append", B=32, n_lo=128, n_hi=128, path=24, c_lo=1,
             c_hi=4096, Hkv=8, D=128, page=64, dtype=BF16),
        # the keys and values of a batch of prompts
        dict(name="append-prompts", op="cache_append", B=16, n_lo=17, n_hi=4096, path=0, c_lo=1,
             c_hi=64, Hkv=8, D=128, page=64, dtype=BF16),
    ]


def _log_int(r, lo, hi):
    return min(hi, max(lo, int(round(math.exp(r.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _cost(case):
    w = work(case)
    rate = 1.9e15 if case["dtype"] == BF16 and case.get("dk", 128) == case.get("dv", 128) else 2e13
    return max(w["bytes"] / 6.8e12, w["flops"] / rate)


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode_step", "attend", "attend", "attend",
                     "cache_append"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        f32 = rng.random() < 0.2
        dtype = F32 if f32 else BF16
        if op in ("prefill", "decode_step"):
            Hqk = rng.choice([1, 2, 4, 8, 16])
            case = dict(op=op, B=_log_int(rng, 1, 16 if op == "prefill" else 256), Hqk=Hqk,
                        Hv=Hqk * rng.choice([1, 2, 2, 4]), dk=128, dv=128, dtype=dtype)
            if f32 or rng.random() < 0.15:
                case.update(dk=rng.choice([16, 32, 64, 96, 128]), dv=rng.choice([32, 48, 64, 128]))
            if op == "prefill":
                hi = _log_int(rng, 1, 2048 if case["dk"] != 128 or f32 else 32768)
                case.update(lo=_log_int(rng, 1, hi), hi=hi)
        else:
            Hkv = rng.choice([1, 2, 4, 8])
            n_hi = 1 if rng.random() < 0.35 else _log_int(rng, 1, 256)
            c_hi = _log_int(rng, 1, 256 if f32 else 8192)
            case = dict(op=op, B=_log_int(rng, 1, 64), n_lo=_log_int(rng, 1, n_hi), n_hi=n_hi,
                        c_lo=_log_int(rng, 1, c_hi), c_hi=c_hi, Hkv=Hkv,
                        D=rng.choice([64, 128, 128, 128]), page=rng.choice([16, 24, 32, 64, 128]),
                        dtype=dtype)
            if f32 or rng.random() < 0.1:
                case.update(D=rng.choice([16, 48, 80, 96]))
            if op == "attend":
                case.update(Hq=Hkv * rng.choice([1, 2, 3, 4, 8]),
                            prefix=0 if rng.random() < 0.25 else _log_int(
                                rng, 1, 512 if f32 else 32768))
            else:
                case.update(path=rng.choice([0, _log_int(rng, 1, 24)]))
                if case["path"] == 0:
                    case.update(n_hi=_log_int(rng, n_hi, 4096))
        # (the plain forms work on padded batches: what they hold stays within tens of GB)
        if op == "prefill":
            held = case["B"] * case["hi"] * case["Hv"] / (2 << 20)
        else:
            held = (case["B"] * case.get("Hq", 0) * case.get("n_hi", 0)
                    * (case.get("prefix", 0) + case.get("c_hi", 0)) / 1e9)
        if _cost(case) <= most and held <= 1:
            return case


def _lens(n, lo, hi, key):
    """n lengths between lo and hi, spread over their logarithm; the first is hi."""
    r = random.Random("%s %d %d %d" % (key, n, lo, hi))
    return [hi] + [_log_int(r, max(lo, 1), max(hi, 1)) for _ in range(n - 1)]


def _paths(case):
    r = random.Random("path %d %d" % (case["B"], case["path"]))
    return [min(n, r.randint(1, case["path"])) for n in _lens(case["B"], case["n_lo"],
                                                              case["n_hi"], "nodes")]


def work(case):
    B, es = case["B"], _ES[case["dtype"]]
    if case["op"] in ("prefill", "decode_step"):
        T = sum(_lens(B, case["lo"], case["hi"], "tokens")) if case["op"] == "prefill" else B
        Hqk, Hv, dk, dv = case["Hqk"], case["Hv"], case["dk"], case["dv"]
        return {"bytes": T * ((2 * Hqk * dk + 2 * Hv * dv) * es + 8 * Hv) + 8 * B * Hv * dk * dv,
                "flops": 6 * T * Hv * dk * dv}
    nodes = _lens(B, case["n_lo"], case["n_hi"], "nodes")
    ctx = _lens(B, case["c_lo"], case["c_hi"], "context")
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "cache_append":
        rows = sum(_paths(case)) if case["path"] else sum(nodes)
        return {"bytes": 4 * rows * Hkv * D * es, "flops": 0}
    Hq, T = case["Hq"], sum(nodes)
    return {"bytes": 2 * T * Hq * D * es + 4 * T * Hq + 2 * T * Hkv * D * es
            + 2 * (case["prefix"] + sum(ctx)) * Hkv * D * es,
            "flops": 4 * Hq * D * sum(n * (case["prefix"] + c + max(1, n // 8))
                                      for n, c in zip(nodes, ctx))}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _trees(nodes, r):
    """parent[] of one draft tree a sequence: each node hangs off one of the 8 before it."""
    return [p for n in nodes for p in [-1] + [i - 1 - r.randrange(min(i, 8)) for i in range(1, n)]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    dt, B = _DT[case["dtype"]], case["B"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dt)

    if case["op"] in ("prefill", "decode_step"):
        Hqk, Hv, dk, dv = case["Hqk"], case["Hv"], case["dk"], case["dv"]
        lens = _lens(B, case["lo"], case["hi"], "tokens") if case["op"] == "prefill" else [1] * B
        T = sum(lens)
        unit = [torch.nn.functional.normalize(torch.randn(T, Hqk, dk, generator=g, device="cuda"),
                                              dim=-1).to(dt) for _ in range(2)]
        # decays from heads that remember thousands of tokens to heads that remember a few
        rate = torch.exp(torch.empty(Hv, device="cuda").uniform_(math.log(2e-3), 0.0, generator=g))
        la = -rate * torch.rand(T, Hv, generator=g, device="cuda").add_(0.5)
        beta = torch.sigmoid(torch.randn(T, Hv, generator=g, device="cuda"))
        slots = list(range(B + 2))
        r.shuffle(slots)
        pool = torch.randn(B + 2, Hv, dk, dv, generator=g, device="cuda").mul_(0.1)
        return dict(case=case, q=unit[0], k=unit[1], v=normal(T, Hv, dv), log_alpha=la, beta=beta,
                    cu=_ints(_cu(lens)), N_max=max(lens), pool=pool, slot=_ints(slots[:B]),
                    pool_out=pool.clone(), o=torch.empty(T, Hv, dv, dtype=dt, device="cuda"))

    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    nodes = _lens(B, case["n_lo"], case["n_hi"], "nodes")
    ctx = _lens(B, case["c_lo"], case["c_hi"], "context")
    T, cu = sum(nodes), _cu(nodes)
    spare = max(nodes) if case["op"] == "cache_append" else 0
    width = -(-(max(ctx) + spare) // page)
    n_prefix = -(-case.get("prefix", 0) // page)
    held = [-(-(c + spare) // page) for c in ctx]
    order = torch.randperm(n_prefix + sum(held) + 3, generator=g, device="cuda").int()
    first = _ints([n_prefix + s for s in _cu(held)[:B]])[:, None]
    cols = torch.arange(width, device="cuda", dtype=torch.int32)[None]
    table = torch.where(cols < _ints(held)[:, None], order[torch.clamp(
        first + cols, max=order.numel() - 1).long()], -1)
    st = dict(case=case, k=normal(T, Hkv, D), v=normal(T, Hkv, D), cu=_ints(cu), N_max=max(nodes),
              k_cache=normal(order.numel(), page, Hkv, D),
              v_cache=normal(order.numel(), page, Hkv, D), table=table.contiguous(),
              ctx=_ints(ctx))
    parents = _trees(nodes, r)
    if case["op"] == "attend":
        st.update(q=normal(T, case["Hq"], D, scale=1.5), parent=_ints(parents),
                  prefix_pages=order[:n_prefix].contiguous(),
                  o=torch.empty(T, case["Hq"], D, dtype=dt, device="cuda"),
                  lse=torch.empty(T, case["Hq"], device="cuda"))
        return st
    st.update(path=None, path_len=None, new_len=torch.empty(B, dtype=torch.int32, device="cuda"))
    if case["path"]:
        paths = []
        for b, n in enumerate(_paths(case)):
            # a root-to-node path of at most n nodes of sequence b's tree
            at, walk = r.randrange(nodes[b]), []
            while at >= 0:
                walk.append(at)
                at = parents[cu[b] + at]
            walk = walk[::-1][:n]
            paths.append(walk + [-1] * (case["path"] - len(walk)))
        st.update(path=_ints(paths), path_len=_ints([sum(x >= 0 for x in p) for p in paths]))
    return st


# ---------------------------------------------------------------------------
# one call
# ---------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if not own:
        return _PLAIN[op](st)
    import gated_deltanet_tree_gdn_gb300 as gt
    if op == "prefill":
        return gt.prefill(st["q"], st["k"], st["v"], st["log_alpha"], st["beta"], st["cu"],
                          st["pool"], state_slot=st["slot"], N_max=st["N_max"],
                          pool_out=st["pool_out"], o=st["o"])
    if op == "decode_step":
        return gt.decode_step(st["q"], st["k"], st["v"], st["log_alpha"], st["beta"], st["pool"],
                              state_slot=st["slot"], pool_out=st["pool_out"], o=st["o"])
    if op == "attend":
        return gt.attend(st["q"], st["k"], st["v"], st["parent"], st["cu"], st["k_cache"],
                         st["v_cache"], st["table"], st["ctx"], prefix_pages=st["prefix_pages"],
                         prefix_len=st["case"]["prefix"], N_max=st["N_max"], o=st["o"],
                         lse=st["lse"])
    new_len = gt.cache_append(st["k"], st["v"], st["cu"], st["k_cache"], st["v_cache"],
                              st["table"], st["ctx"], path=st["path"], path_len=st["path_len"],
                              N_max=st["N_max"], new_len=st["new_len"])
    return st["k_cache"], st["v_cache"], new_len


def _rows(st, width):
    """Row numbers [B, width] of the packed rows of each sequence, and which of them it has."""
    start, stop = st["cu"][:-1, None].long(), st["cu"][1:, None].long()
    at = start + torch.arange(width, device="cuda")[None]
    return torch.clamp(at, max=int(st["k"].shape[0]) - 1), at < stop


def _plain_prefill(st):
    """The gated delta rule in chunks of 64 tokens: inside a chunk the writes solve a unit lower
    triangular system, between chunks the state is carried."""
    case, C = st["case"], 64
    L = -(-st["N_max"] // C) * C
    rows, has = _rows(st, L)
    G = case["Hv"] // case["Hqk"]

    def chunks(x, fill):  # [T, H, d] -> [B, chunks, H, C, d]
        y = torch.where(has[..., None, None], x[rows].float(), fill)
        return y.unflatten(1, (L // C, C)).transpose(2, 3)

    q = chunks(st["q"], 0.0).repeat_interleave(G, dim=2)
    k = chunks(st["k"], 0.0).repeat_interleave(G, dim=2)
    v = chunks(st["v"], 0.0)
    g = chunks(st["log_alpha"][..., None], 0.0).cumsum(dim=3)
    beta = chunks(st["beta"][..., None], 0.0)
    low = torch.ones(C, C, device="cuda").tril()
    # (the mask comes before the exponential: above the diagonal its argument is positive)
    decay = torch.exp((g - g.transpose(3, 4)) * low) * low
    kk = k @ k.transpose(3, 4)
    X = (beta * decay * kk).tril(-1)
    Y = decay * (q @ k.transpose(3, 4))
    del decay, kk
    inv = torch.eye(C, device="cuda").expand_as(X).clone()  # (I + X)^-1, a row at a time
    for i in range(1, C):
        inv[..., i, :i] = -(X[..., i:i + 1, :i] @ inv[..., :i, :i])[..., 0, :]
    W = inv @ (beta * torch.exp(g) * k)
    U0 = inv @ (beta * v)
    del inv, X
    last = g[..., -1:, :]
    q = q * torch.exp(g)
    k = k * torch.exp(last - g)
    S = st["pool"][st["slot"].long()]
    o = torch.empty_like(v)
    for c in range(L // C):
        U = U0[:, c] - W[:, c] @ S
        o[:, c] = q[:, c] @ S + Y[:, c] @ U
        S = torch.exp(last[:, c]) * S + k[:, c].transpose(2, 3) @ U
    st["pool_out"].index_copy_(0, st["slot"].long(), S)
    o = o.transpose(2, 3).flatten(1, 2)
    return o[has].to(st["o"].dtype), st["pool_out"]


def _plain_step(st):
    G = st["case"]["Hv"] // st["case"]["Hqk"]
    q = st["q"].float().repeat_interleave(G, dim=1)
    k = st["k"].float().repeat_interleave(G, dim=1)
    S = torch.exp(st["log_alpha"])[..., None, None] * st["pool"][st["slot"].long()]
    u = st["beta"][..., None] * (st["v"].float() - (k[:, :, None] @ S)[:, :, 0])
    S = S + k[..., None] * u[:, :, None]
    st["pool_out"].index_copy_(0, st["slot"].long(), S)
    return (q[:, :, None] @ S)[:, :, 0].to(st["o"].dtype), st["pool_out"]


def _plain_attend(st):
    case, N = st["case"], st["N_max"]
    Hkv, D, page, P = case["Hkv"], case["D"], case["page"], case["prefix"]
    G = case["Hq"] // Hkv
    rows, has = _rows(st, N)
    q = st["q"][rows].float().unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4) / math.sqrt(D)
    kp, vp = (x[st["prefix_pages"].long()].flatten(0, 1)[:P].float().transpose(0, 1)
              for x in (st["k_cache"], st["v_cache"]))  # [Hkv, P, D]
    kc, vc = (x[st["table"].clamp(min=0).long()].flatten(1, 2).float().transpose(1, 2)
              for x in (st["k_cache"], st["v_cache"]))  # [B, Hkv, C, D]
    kn, vn = (x[rows].float().transpose(1, 2) for x in (st["k"], st["v"]))  # [B, Hkv, N, D]
    # the nodes on each node's root-to-node path: the closure of the parent relation
    par = torch.where(has, st["parent"][rows].long(), -1)
    on = torch.eye(N, device="cuda") + (par[..., None] == torch.arange(N, device="cuda")).float()
    for _ in range(max(1, (N - 1).bit_length())):
        on = ((on @ on) > 0).float()
    at = torch.arange(kc.shape[2], device="cuda")
    in_ctx = at < st["ctx"][:, None]
    B = q.shape[0]
    s = torch.cat([(q.transpose(0, 1).flatten(1, 3) @ kp.transpose(1, 2)).unflatten(
        1, (B, G, N)).transpose(0, 1),
        (q @ kc.transpose(2, 3)[:, :, None]).masked_fill(~in_ctx[:, None, None, None], -math.inf),
        (q @ kn.transpose(2, 3)[:, :, None]).masked_fill(on[:, None, None] == 0, -math.inf)],
        dim=-1)  # [B, Hkv, G, N, P + C + N]
    top = s.amax(dim=-1, keepdim=True)
    s = torch.exp(s - top)
    total = s.sum(dim=-1, keepdim=True)
    pp, pc, pn = s.split([P, kc.shape[2], N], dim=-1)
    o = (pp.transpose(0, 1).flatten(1, 3) @ vp).unflatten(1, (B, G, N)).transpose(0, 1)
    vc = vc.masked_fill(~in_ctx[:, None, :, None], 0.0)
    o = (o + pc @ vc[:, :, None] + pn @ vn[:, :, None]) / total
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[has].to(st["o"].dtype)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)[has]
    return o, lse


def _plain_append(st):
    page = st["case"]["page"]
    rows, has = _rows(st, st["N_max"])
    if st["path"] is not None:
        j = torch.arange(st["path"].shape[1], device="cuda")
        has = j < st["path_len"][:, None]
        rows = st["cu"][:-1, None].long() + st["path"].clamp(min=0).long()
    count = has.sum(dim=1)
    at = st["ctx"][:, None].long() + torch.arange(rows.shape[1], device="cuda")
    pages = st["table"].long().gather(1, torch.clamp(at // page, max=st["table"].shape[1] - 1))
    where = (pages * page + at % page)[has]
    for cache, x in ((st["k_cache"], st["k"]), (st["v_cache"], st["v"])):
        cache.flatten(0, 1).index_copy_(0, where, x[rows[has]])
    st["new_len"].copy_(st["ctx"] + count)
    return st["k_cache"], st["v_cache"], st["new_len"]


_PLAIN = dict(prefill=_plain_prefill, decode_step=_plain_step, attend=_plain_attend,
              cache_append=_plain_append)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("prefill", "decode_step"):
        return _exact_rule(st)
    if case["op"] == "attend":
        return _exact_attend(st)
    k, v = st["k_cache"].double(), st["v_cache"].double()
    cu, ctx, table = st["cu"].tolist(), st["ctx"].tolist(), st["table"].tolist()
    for b in range(case["B"]):
        new = list(range(cu[b + 1] - cu[b]))
        if st["path"] is not None:
            new = st["path"][b, :int(st["path_len"][b])].tolist()
        spots = [ctx[b] + j for j in range(len(new))]
        to = [table[b][p // case["page"]] for p in spots], [p % case["page"] for p in spots]
        fro = [cu[b] + i for i in new]
        k[to] = st["k"][fro].double()
        v[to] = st["v"][fro].double()
        ctx[b] += len(new)
    return k, v, None


def _exact_rule(st):
    """S <- a (I - b k k^T) S + b k v^T and o = S^T q, token by token.  Sequences are taken
    longest first, so that those still running are the leading ones."""
    case = st["case"]
    step = case["op"] == "decode_step"
    cu = list(range(case["B"] + 1)) if step else st["cu"].tolist()
    lens = [b - a for a, b in zip(cu, cu[1:])]
    by_len = sorted(range(case["B"]), key=lambda b: -lens[b])
    slots = st["slot"].long()[by_len]
    S = st["pool"].double()[slots]
    heads = torch.arange(case["Hv"], device="cuda") // (case["Hv"] // case["Hqk"])
    start = torch.tensor([cu[b] for b in by_len], device="cuda")
    o = torch.empty(st["o"].shape, dtype=torch.float64, device="cuda")
    a, beta = torch.exp(st["log_alpha"].double()), st["beta"].double()
    live = case["B"]
    for t in range(max(lens)):
        while lens[by_len[live - 1]] <= t:
            live -= 1
        i = start[:live] + t
        k, q = st["k"][i].double()[:, heads], st["q"][i].double()[:, heads]
        Sl = S[:live]
        Sl *= a[i][..., None, None]
        err = st["v"][i].double() - torch.einsum("bhk,bhkv->bhv", k, Sl)
        Sl += torch.einsum("bhk,bhv->bhkv", k, beta[i][..., None] * err)
        o[i] = torch.einsum("bhk,bhkv->bhv", q, Sl)
    out = st["pool_out"].double()
    out[slots] = S
    return o, out


def _exact_attend(st):
    case = st["case"]
    page, P, Hkv = case["page"], case["prefix"], case["Hkv"]
    cu, ctx, parent = st["cu"].tolist(), st["ctx"].tolist(), st["parent"].tolist()
    o = torch.empty(st["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["lse"].shape, dtype=torch.float64, device="cuda")
    pk, pv = (x[st["prefix_pages"].long()].flatten(0, 1)[:P] for x in (st["k_cache"],
                                                                      st["v_cache"]))
    for b in range(case["B"]):
        own_rows, n = slice(cu[b], cu[b + 1]), cu[b + 1] - cu[b]
        pages = st["table"][b, :-(-ctx[b] // page)].long()
        K, V = (torch.cat([p, c[pages].flatten(0, 1)[:ctx[b]], x[own_rows]])
                for p, c, x in ((pk, st["k_cache"], st["k"]), (pv, st["v_cache"], st["v"])))
        sees = torch.zeros(n, P + ctx[b] + n, dtype=torch.bool)
        sees[:, :P + ctx[b]] = True
        for i in range(n):
            up = parent[cu[b] + i]
            if up >= 0:
                sees[i] = sees[up]
            sees[i, P + ctx[b] + i] = True
        bias = torch.zeros(sees.shape, dtype=torch.float64).masked_fill(~sees, -math.inf).cuda()
        for h in range(Hkv):
            q = st["q"][own_rows].unflatten(1, (Hkv, -1))[:, h].double()  # [n, G, D]
            s = torch.einsum("ngd,md->ngm", q, K[:, h].double()) / math.sqrt(case["D"])
            s = s + bias[:, None]
            z = torch.logsumexp(s, dim=-1)
            lse[own_rows].unflatten(1, (Hkv, -1))[:, h] = z
            o[own_rows].unflatten(1, (Hkv, -1))[:, h] = torch.exp(s - z[..., None]) @ V[:, h].double()
    return o, lse
