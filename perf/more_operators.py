"""Workloads of the operators in front of a hybrid model's attention, with their plain forms.

What a layer's projection gives becomes what the attention over a paged cache (and the gated
delta rule) takes:

  tree_positions     where the nodes of a draft tree, or the rows of a prompt, stand in their
                     sequence: behind the shared prefix and the context, at the node's depth
  norm_rope          queries and keys normalised for each head (root mean square with weights,
                     or to unit length) and rotated by their rows' positions, in one pass
  cache_append_rope  the same for rows that join the cache: keys normalised and rotated on their
                     way to their sequences' pages, values copied beside them, queries rotated

`listed()` are workloads worth timing, `draw()` more of the same ranges, `prepare()` makes the
inputs, `run()` is one call, `exact()` the same in 64 bits, `work()` what a call has to move
and compute.  With `own` false, `run()` evaluates the operators with elementary torch
operations in 32 bits (angles in 64); with `own` true it calls the library.
"""

import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}
_ES = {BF16: 2, F32: 4}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

# R: how many elements of a head are rotated; half: element i with i + R / 2, else 2 i with 2 i + 1
# rows: how the inputs lie: "dense", "fused" (columns of one projection's output), "gated" (each
#       query head of that output is followed by its gate)
# far:  positions start anywhere below it; len: consecutive rows of one sequence
# stretch: None, "linear" or "yarn": positions past those of the training, and by how much

def listed():
    return [
        # the serving batch of the tree verification: 32 trees of 128 nodes
        dict(name="positions-trees-32", op="tree_positions", B=32, lo=128, hi=128, tree=True,
             prefix=1024, ctx=4096),
        # many small and large trees together
        dict(name="positions-trees-256", op="tree_positions", B=256, lo=1, hi=1024, tree=True,
             prefix=0, ctx=131072),
        # the next token of one sequence: launch latency
        dict(name="rope-token-1", op="norm_rope", T=1, len=1, Hq=32, Hkv=8, D=128, R=128, half=True,
             norm="rms", rows="fused", far=4096, stretch=None, dtype=BF16),
        # the serving batch's 32 trees of 128 nodes, straight from the projection
        dict(name="rope-trees-32", op="norm_rope", T=4096, len=128, Hq=32, Hkv=8, D=128, R=128,
             half=True, norm="rms", rows="fused", far=5120, stretch=None, dtype=BF16),
        # a long document of a model with gated attention that rotates a quarter of each head,
        # behind far positions of a stretched context
        dict(name="rope-document", op="norm_rope", T=32768, len=32768, Hq=32, Hkv=8, D=128, R=32,
             half=True, norm="rms", rows="gated", far=1 << 20, stretch="yarn", dtype=BF16),
        # rotation alone, neighbouring elements in pairs, an odd number of rows
        dict(name="rope-interleaved", op="norm_rope", T=8191, len=117, Hq=16, Hkv=16, D=128, R=128,
             half=False, norm=None, rows="dense", far=32768, stretch="linear", dtype=BF16),
        # the keys and queries of the gated delta rule: unit length, no positions
        dict(name="unit-prompt", op="norm_rope", T=16384, len=1024, Hq=16, Hkv=16, D=128, R=0,
             half=True, norm="unit", rows="fused", far=1, stretch=None, dtype=BF16),
        # the 32-bit variant at odd sizes: 20 of 80 elements, 3 query heads a key head
        dict(name="rope-f32", op="norm_rope", T=1001, len=77, Hq=6, Hkv=2, D=80, R=20, half=True,
             norm="rms", rows="dense", far=8192, stretch=None, dtype=F32),
        # the next token of one sequence, straight into its page
        dict(name="append-token-1", op="cache_append_rope", B=1, lo=1, hi=1, c_lo=300, c_hi=300,
             prefix=0, Hq=32, Hkv=8, D=128, R=128, half=True, norm="rms", rows="fused", page=64,
             keep=False, stretch=None, dtype=BF16),
        # a token of each sequence of a full batch behind a shared prompt
        dict(name="append-tokens-128", op="cache_append_rope", B=128, lo=1, hi=1, c_lo=1, c_hi=2048,
             prefix=32768, Hq=32, Hkv=8, D=128, R=128, half=True, norm="rms", rows="fused", page=64,
             keep=False, stretch="yarn", dtype=BF16),
        # a batch of prompts: their keys and values into the pages and, for their own causal
        # attention, beside them
        dict(name="append-prompts-16", op="cache_append_rope", B=16, lo=17, hi=4096, c_lo=1, c_hi=64,
             prefix=1024, Hq=32, Hkv=8, D=128, R=64, half=True, norm="rms", rows="fused", page=64,
             keep=True, stretch=None, dtype=BF16),
        # the 32-bit variant: pairs of neighbours, no norm, pages of 24 rows, keys and values alone
        dict(name="append-f32", op="cache_append_rope", B=3, lo=1, hi=201, c_lo=1, c_hi=100, prefix=77,
             Hq=0, Hkv=4, D=48, R=32, half=False, norm=None, rows="dense", page=24, keep=False,
             stretch=None, dtype=F32),
    ]


def _log_int(r, lo, hi):
    return min(hi, max(lo, int(round(math.exp(r.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tree_positions", "norm_rope", "norm_rope", "norm_rope", "cache_append_rope",
                     "cache_append_rope"])
    most = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    while True:
        if op == "tree_positions":
            tree = rng.random() < 0.7
            hi = _log_int(rng, 1, 1024 if tree else 32768)
            case = dict(op=op, B=_log_int(rng, 1, 256), lo=_log_int(rng, 1, hi), hi=hi, tree=tree,
                        prefix=rng.choice([0, _log_int(rng, 1, 32768)]), ctx=_log_int(rng, 1, 1 << 20))
        else:
            D = rng.choice([64, 128, 128, 128, 16, 48, 80, 96, 112])
            case = dict(op=op, Hkv=rng.choice([1, 2, 4, 8, 16]), D=D,
                        R=rng.choice([D, D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)]),
                        half=rng.random() < 0.6, norm=rng.choice(["rms", "rms", "unit", None]),
                        stretch=rng.choice([None, None, "linear", "yarn"]),
                        rows=rng.choice(["dense", "fused", "gated"]),
                        dtype=F32 if rng.random() < 0.2 else BF16)
            case["Hq"] = case["Hkv"] * rng.choice([1, 2, 3, 4, 8])
            if op == "norm_rope":
                T = _log_int(rng, 1, 32768)
                case.update(T=T, len=_log_int(rng, 1, T), far=_log_int(rng, 1, 1 << 20))
                if case["norm"] and rng.random() < 0.2:
                    case.update(R=0)
            else:
                hi, c_hi = _log_int(rng, 1, 4096), _log_int(rng, 1, 2048)
                case.update(B=_log_int(rng, 1, 128), lo=_log_int(rng, 1, hi), hi=hi, c_hi=c_hi,
                            c_lo=_log_int(rng, 1, c_hi), page=rng.choice([16, 24, 32, 64, 128]),
                            prefix=rng.choice([0, _log_int(rng, 1, 1 << 20)]),
                            keep=rng.random() < 0.4)
                if rng.random() < 0.2:
                    case.update(Hq=0)
        if work(case)["bytes"] <= most:
            return case


def _lens(n, lo, hi, key):
    """n lengths between lo and hi, spread over their logarithm; the first is hi."""
    r = random.Random("%s %d %d %d" % (key, n, lo, hi))
    return [hi] + [_log_int(r, lo, hi) for _ in range(n - 1)]


def work(case):
    if case["op"] == "tree_positions":
        T = sum(_lens(case["B"], case["lo"], case["hi"], "rows"))
        return {"bytes": (8 if case["tree"] else 4) * T + 8 * case["B"], "flops": 0}
    one = case["D"] * _ES[case["dtype"]]
    per_head = (3 * case["R"] if case["R"] else 0) + (4 * case["D"] if case["norm"] else 0)
    if case["op"] == "norm_rope":
        T, H = case["T"], case["Hq"] + case["Hkv"]
        return {"bytes": 2 * T * H * one + (4 * T if case["R"] else 0), "flops": T * H * per_head}
    T = sum(_lens(case["B"], case["lo"], case["hi"], "rows"))
    return {"bytes": T * (2 * case["Hq"] + (6 if case["keep"] else 4) * case["Hkv"]) * one
            + 16 * case["B"], "flops": T * (case["Hq"] + case["Hkv"]) * per_head}


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


def _frequencies(R, stretch):
    """Radians a position of each pair (64 bits), and what the rotated part is multiplied by."""
    base, i = 1e6, torch.arange(0, R, 2, dtype=torch.float64, device="cuda")
    f = base ** (-i / R) if R else i
    if stretch == "linear":
        return f / 8.0, 1.0
    if stretch == "yarn":
        # pairs that turn often within the trained length keep their speed, those that hardly
        # turn are slowed by the factor, the ones between are blended
        factor, trained = 32.0, 32768
        at = [R * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base))
              for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
        slow = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return f * (1.0 - slow) + f / factor * slow, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _heads(case, T, g):
    """q, k, v [T, heads, D] as the projection leaves them."""
    dt, Hq, Hkv, D = _DT[case["dtype"]], case["Hq"], case["Hkv"], case["D"]
    gate = 2 if case["rows"] == "gated" else 1
    wide = torch.empty(T, (gate * Hq + 2 * Hkv) * D, dtype=dt, device="cuda")
    wide.copy_(torch.randn(wide.shape, generator=g, device="cuda"))
    wide *= 1.5
    q, k, v = wide.split([gate * Hq * D, Hkv * D, Hkv * D], dim=1)
    q = q.unflatten(1, (Hq, gate * D))[..., :D] if Hq else None
    k, v = k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))
    if case["rows"] == "dense":
        q, k, v = q.contiguous() if Hq else None, k.contiguous(), v.contiguous()
    return q, k, v


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    if case["op"] == "tree_positions":
        lens = _lens(case["B"], case["lo"], case["hi"], "rows")
        # each node hangs off one of the 8 before it
        parents = [p for n in lens for p in [-1] + [i - 1 - int(r.random() * min(i, 8))
                                                    for i in range(1, n)]] if case["tree"] else None
        return dict(case=case, cu=_ints(_cu(lens)), N_max=max(lens),
                    parent=_ints(parents) if case["tree"] else None,
                    ctx=_ints([r.randint(0, case["ctx"]) for _ in lens]),
                    positions=torch.empty(sum(lens), dtype=torch.int32, device="cuda"))
    Hq, Hkv, D, R = case["Hq"], case["Hkv"], case["D"], case["R"]
    lens = None if case["op"] == "norm_rope" else _lens(case["B"], case["lo"], case["hi"], "rows")
    T = case["T"] if lens is None else sum(lens)
    q, k, v = _heads(case, T, g)
    inv_freq, scale = _frequencies(R, case["stretch"])
    st = dict(case=case, q=q, k=k, inv_freq=inv_freq, scale=scale,
              # turns a position, in units of 2^-64
              freq=(inv_freq / (2 * math.pi) * 2.0 ** 64).round().long() if R else None,
              wq=None, wk=None, q_out=None, k_out=None, v_out=None)
    if case["norm"] == "rms":
        st["wq"], st["wk"] = (torch.randn(D, generator=g, device="cuda").mul_(0.2).add_(1.0)
                              for _ in range(2))
    if Hq:
        st["q_out"] = torch.empty(T, Hq, D, dtype=_DT[case["dtype"]], device="cuda")
    if lens is None:
        start = [r.randrange(case["far"]) for _ in range(-(-T // case["len"]))]
        at = torch.arange(T, device="cuda")
        st.update(k_out=torch.empty(T, Hkv, D, dtype=_DT[case["dtype"]], device="cuda"),
                  positions=(_ints(start)[at // case["len"]] + at % case["len"]).int())
        return st
    ctx, page = _lens(case["B"], case["c_lo"], case["c_hi"], "context"), case["page"]
    held = [-(-(c + n) // page) for c, n in zip(ctx, lens)]
    order = torch.randperm(sum(held) + 3, generator=g, device="cuda").int()
    cols = torch.arange(max(held), device="cuda", dtype=torch.int32)[None]
    table = torch.where(cols < _ints(held)[:, None], order[torch.clamp(
        _ints(_cu(held)[:-1])[:, None] + cols, max=order.numel() - 1).long()], -1)
    if case["keep"]:
        st["k_out"], st["v_out"] = (torch.empty(T, Hkv, D, dtype=_DT[case["dtype"]], device="cuda")
                                    for _ in range(2))
    caches = [torch.randn(order.numel(), page, Hkv, D, generator=g, device="cuda").to(
        _DT[case["dtype"]]) for _ in range(2)]
    st.update(v=v, cu=_ints(_cu(lens)), N_max=max(lens), table=table.contiguous(), ctx=_ints(ctx),
              k_cache=caches[0], v_cache=caches[1],
              new_len=torch.empty(case["B"], dtype=torch.int32, device="cuda"))
    return st


# ---------------------------------------------------------------------------
# one call
# ---------------------------------------------------------------------------

def run(st):
    case = st["case"]
    if not own:
        return _PLAIN[case["op"]](st)
    import gated_deltanet_tree_gdn_gb300 as gt
    if case["op"] == "tree_positions":
        return gt.tree_positions(st["parent"], st["cu"], context_len=st["ctx"],
                                 prefix_len=case["prefix"], N_max=st["N_max"],
                                 positions=st["positions"])
    if case["op"] == "norm_rope":
        return gt.norm_rope(st["q"], st["k"], st["positions"] if case["R"] else None, st["freq"],
                            interleaved=not case["half"], rope_scale=st["scale"],
                            norm=case["norm"], q_weight=st["wq"], k_weight=st["wk"], eps=EPS,
                            q_out=st["q_out"], k_out=st["k_out"])
    q_out, new_len = gt.cache_append_rope(
        st["q"], st["k"], st["v"], st["cu"], st["k_cache"], st["v_cache"], st["table"], st["ctx"],
        st["freq"], prefix_len=case["prefix"], interleaved=not case["half"],
        rope_scale=st["scale"], norm=case["norm"], q_weight=st["wq"], k_weight=st["wk"], eps=EPS,
        q_out=st["q_out"], k_out=st["k_out"], v_out=st["v_out"], N_max=st["N_max"],
        new_len=st["new_len"])
    return q_out, st["k_out"], st["v_out"], st["k_cache"], st["v_cache"], new_len


def _plain_positions(st):
    """Depths by doubling: every node adds its ancestor's count and jumps to that one's."""
    rows = torch.arange(st["positions"].shape[0], device="cuda")
    seq = torch.searchsorted(st["cu"][1:].long(), rows, right=True)
    first = st["cu"].long()[seq]
    if st["parent"] is None:
        depth = rows - first
    else:
        up = st["parent"].long()
        depth = (up >= 0).long()
        up = torch.where(up >= 0, up + first, rows)
        for _ in range(st["N_max"].bit_length()):
            depth = depth + torch.where(up != rows, depth[up], 0)
            up = up[up]
    return (depth + st["ctx"].long()[seq] + st["case"]["prefix"]).int()


def _plain_heads(x, w, positions, st):
    """Head rows [T, H, D] normalised and rotated, in 32 bits."""
    case, R, y = st["case"], st["case"]["R"], x.float()
    if case["norm"]:
        square = (y * y).sum(dim=-1, keepdim=True)
        y = y / torch.sqrt((square / case["D"] if case["norm"] == "rms" else square) + EPS)
        if w is not None:
            y = y * w
    if R:
        angle = positions.double()[:, None] * st["inv_freq"]
        cos, sin = ((f(angle) * st["scale"]).float()[:, None] for f in (torch.cos, torch.sin))
        a, b = ((y[..., :R // 2], y[..., R // 2:R]) if case["half"] else
                (y[..., 0:R:2], y[..., 1:R:2]))
        pair = a * cos - b * sin, b * cos + a * sin
        turned = torch.cat(pair, dim=-1) if case["half"] else torch.stack(pair, dim=-1).flatten(-2)
        y = torch.cat([turned, y[..., R:]], dim=-1)
    return y.to(x.dtype)


def _plain_norm_rope(st):
    return (_plain_heads(st["q"], st["wq"], st["positions"], st),
            _plain_heads(st["k"], st["wk"], st["positions"], st))


def _plain_append(st):
    page = st["case"]["page"]
    rows = torch.arange(st["k"].shape[0], device="cuda")
    seq = torch.searchsorted(st["cu"][1:].long(), rows, right=True)
    at = st["ctx"].long()[seq] + rows - st["cu"].long()[seq]
    positions = at + st["case"]["prefix"]
    where = st["table"].long()[seq, at // page] * page + at % page
    k = _plain_heads(st["k"], st["wk"], positions, st)
    st["k_cache"].flatten(0, 1).index_copy_(0, where, k)
    st["v_cache"].flatten(0, 1).index_copy_(0, where, st["v"])
    q = None if st["q"] is None else _plain_heads(st["q"], st["wq"], positions, st)
    new_len = st["ctx"] + (st["cu"][1:] - st["cu"][:-1])
    own_rows = (k, st["v"].clone(memory_format=torch.contiguous_format)) if st["case"]["keep"] else (None, None)
    return q, *own_rows, st["k_cache"], st["v_cache"], new_len


_PLAIN = dict(tree_positions=_plain_positions, norm_rope=_plain_norm_rope,
              cache_append_rope=_plain_append)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tree_positions":
        cu, ctx, out = st["cu"].tolist(), st["ctx"].tolist(), []
        parent = None if st["parent"] is None else st["parent"].tolist()
        for b, first in enumerate(cu[:-1]):
            depth = []
            for t in range(cu[b + 1] - first):
                up = t - 1 if parent is None else parent[first + t]
                depth.append(0 if up < 0 else depth[up] + 1)
            out += [case["prefix"] + ctx[b] + d for d in depth]
        return _ints(out)
    if case["op"] == "norm_rope":
        return tuple(_exact_rows(x, w, st["positions"].tolist(), st)
                     for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])))
    cu, ctx, table = st["cu"].tolist(), st["ctx"].tolist(), st["table"].tolist()
    positions, pages, spots = [], [], []
    for b in range(case["B"]):
        for j in range(cu[b + 1] - cu[b]):
            positions.append(case["prefix"] + ctx[b] + j)
            pages.append(table[b][(ctx[b] + j) // case["page"]])
            spots.append((ctx[b] + j) % case["page"])
    k = _exact_rows(st["k"], st["wk"], positions, st)
    k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
    to = torch.tensor(pages, device="cuda"), torch.tensor(spots, device="cuda")
    k_cache[to], v_cache[to] = k, st["v"].double()
    q = None if st["q"] is None else _exact_rows(st["q"], st["wq"], positions, st)
    return q, *((k, st["v"].double()) if case["keep"] else (None, None)), k_cache, v_cache, None


def _exact_rows(x, w, positions, st):
    """Each pair as a complex number, turned by e^(i angle)."""
    case, R = st["case"], st["case"]["R"]
    y = x.to(torch.float64)
    if case["norm"] == "rms":
        y = y * torch.rsqrt(y.square().mean(dim=-1, keepdim=True) + EPS)
    elif case["norm"] == "unit":
        y = y * torch.rsqrt(y.square().sum(dim=-1, keepdim=True) + EPS)
    if w is not None:
        y = y * w.double()
    if not R:
        return y
    out = y.clone()
    first = torch.arange(R // 2, device="cuda") * (1 if case["half"] else 2)
    second = first + (R // 2 if case["half"] else 1)
    angle = torch.outer(torch.tensor(positions, dtype=torch.float64, device="cuda"), st["inv_freq"])
    turned = torch.complex(y[..., first], y[..., second]) * torch.polar(
        torch.full_like(angle, st["scale"]), angle)[:, None]
    out[..., first], out[..., second] = turned.real, turned.imag
    return out
