"""Speculative decoding of a small hybrid model: Gated DeltaNet and attention layers in turn.

    python examples/hybrid_serving.py

Every sequence shares a system prompt.  It is read once: `prefill` leaves its states, and
`cache_append` its keys and values on pages that all sequences then see as their prefix.  The
sequences' own prompts follow as one ragged batch.  After that a round drafts a tree of tokens
below each sequence's next one (`build_topw`), runs it through the model (`verify_packed` and
`attend`, which change nothing), and keeps the path that the model itself would have taken
(`commit_packed` for the states, `cache_append` for the keys and values).  Every third round
nothing is drafted, and the next token is run alone (`decode_step`, `attend` of one row,
`cache_append`).

The weights are random.  At the end the kept tokens are run through the model from nothing, in
one `prefill` and one causal `attend` a layer, and must give the same logits.
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_tree_gdn_gb300 as gt  # noqa: E402

VOCAB, WIDTH, LAYERS = 16, 256, 4          # even layers: Gated DeltaNet, odd: attention
HQK, HV, DK = 2, 4, 128                    # its heads (dk = dv)
HQ, HKV, D = 8, 2, 64                      # the attention's
PAGE, PAGES_EACH = 16, 16                  # pages of a sequence's own context
NODES, CANDIDATES, DEPTH = 24, 4, 6        # a draft tree


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """The layers' products around the operators; `rule` and `attention` are given by the call."""

    def __init__(self, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            x = torch.randn(*shape, device="cuda", generator=gen) / math.sqrt(shape[0])
            return x.bfloat16()

        self.embed = weight(VOCAB, WIDTH) * 4
        self.head = weight(WIDTH, VOCAB)
        self.layers = []
        for i in range(LAYERS):
            if i % 2 == 0:
                sizes = [HQK * DK, HQK * DK, HV * DK, HV, HV]
                out = HV * DK
            else:
                sizes = [HQ * D, HKV * D, HKV * D]
                out = HQ * D
            self.layers.append((weight(WIDTH, sum(sizes)), sizes, weight(out, WIDTH)))

    def run(self, tokens, rule, attention):
        """Logits of the rows' next tokens [T, VOCAB]."""
        x = self.embed[tokens.long()].float()
        T = x.shape[0]
        for i, (w_in, sizes, w_out) in enumerate(self.layers):
            y = torch.nn.functional.rms_norm(x, (WIDTH,)).bfloat16() @ w_in
            y = [p.contiguous() for p in y.split(sizes, dim=1)]
            if i % 2 == 0:
                unit = lambda z: torch.nn.functional.normalize(  # noqa: E731
                    z.view(T, HQK, DK).float(), dim=-1).bfloat16()
                log_alpha = -0.2 * torch.nn.functional.softplus(y[3].float())
                o = rule(i, unit(y[0]), unit(y[1]), y[2].view(T, HV, DK), log_alpha,
                         torch.sigmoid(y[4].float()))
            else:
                o = attention(i, y[0].view(T, HQ, D), y[1].view(T, HKV, D), y[2].view(T, HKV, D))
            x = x + (o.reshape(T, -1) @ w_out).float()
        return torch.nn.functional.rms_norm(x, (WIDTH,)).bfloat16().float() @ self.head.float()


class Server:
    """States, pages and lengths of a batch of sequences behind one system prompt."""

    def __init__(self, model, system_prompt, batch):
        self.model, self.B = model, batch
        self.prefix_len = len(system_prompt)
        n_prefix = -(-self.prefix_len // PAGE)
        # pages in an order of their own: the prefix's, then each sequence's
        pages = torch.randperm(n_prefix + batch * PAGES_EACH, device="cuda").int()
        self.prefix_pages = pages[:n_prefix].contiguous()
        self.table = pages[n_prefix:].view(batch, PAGES_EACH).contiguous()
        self.context_len = ints([0] * batch)
        self.caches = {i: [torch.zeros(len(pages), PAGE, HKV, D, dtype=torch.bfloat16, device="cuda")
                           for _ in range(2)] for i in range(1, LAYERS, 2)}
        self.states = {i: torch.zeros(batch, HV, DK, DK, device="cuda") for i in range(0, LAYERS, 2)}
        # the system prompt, once: sequence 0's state, given to all of them
        cu, none = ints([0, self.prefix_len]), ints([0])

        def rule(i, *qkvab):
            return gt.prefill(*qkvab, cu, self.states[i], pool_out=self.states[i])[0]

        def attention(i, q, k, v):
            o, _ = gt.attend(q, k, v, None, cu, *self.caches[i], self.prefix_pages[None], none)
            gt.cache_append(k, v, cu, *self.caches[i], self.prefix_pages[None], none)
            return o

        model.run(ints(system_prompt), rule, attention)
        for s in self.states.values():
            s[1:] = s[:1]

    def attend(self, i, q, k, v, parent, cu, rows):
        return gt.attend(q, k, v, parent, cu, *self.caches[i], self.table, self.context_len,
                         prefix_pages=self.prefix_pages, prefix_len=self.prefix_len,
                         N_max=rows)[0]

    def append(self, i, k, v, cu, rows, **path):
        return gt.cache_append(k, v, cu, *self.caches[i], self.table, self.context_len, N_max=rows,
                               **path)

    def prompts(self, lists):
        """The sequences' prompts as one ragged batch; the logits behind each one's last token."""
        lens = [len(x) for x in lists]
        ends = [sum(lens[:b + 1]) for b in range(self.B)]
        cu, rows, kept = ints([0] + ends), max(lens), []

        def rule(i, *qkvab):
            return gt.prefill(*qkvab, cu, self.states[i], N_max=rows, pool_out=self.states[i])[0]

        def attention(i, q, k, v):
            o = self.attend(i, q, k, v, None, cu, rows)
            kept.append(self.append(i, k, v, cu, rows))
            return o

        logits = self.model.run(ints(sum(lists, [])), rule, attention)
        self.context_len = kept[-1]
        return logits[ints(ends).long() - 1]

    def step(self, tokens):
        """One token of each sequence."""
        cu, kept = ints(list(range(self.B + 1))), []

        def rule(i, *qkvab):
            return gt.decode_step(*qkvab, self.states[i], pool_out=self.states[i])[0]

        def attention(i, q, k, v):
            o = self.attend(i, q, k, v, None, cu, 1)
            kept.append(self.append(i, k, v, cu, 1))
            return o

        logits = self.model.run(tokens, rule, attention)
        self.context_len = kept[-1]
        return logits

    def draft(self, seed):
        """A tree of NODES tokens a sequence: candidates at random, built best first."""
        gen = torch.Generator(device="cuda").manual_seed(seed)
        order = torch.rand(self.B, NODES, VOCAB, device="cuda", generator=gen).argsort(-1)
        cand = order[..., :CANDIDATES]
        logp = torch.log_softmax(torch.randn(self.B, NODES, CANDIDATES, device="cuda",
                                             generator=gen), -1).sort(-1, descending=True)[0]
        parent, index, _, built = gt.build_topw(logp.contiguous(), CANDIDATES, DEPTH)
        return parent, cand, index, built

    def tree(self, following, seed):
        """Drafts a tree below each sequence's next token, runs it, and keeps the path that the
        model takes.  Returns the drafted tokens kept and the logits behind them."""
        parent, cand, index, built = (x.cpu() for x in self.draft(seed))
        tokens, parents, lens = [], [], built.tolist()
        for b, n in enumerate(lens):
            for t in range(n):  # (node 0 is the next token itself)
                p = int(parent[b, t])
                tokens.append(following[b] if t == 0 else int(cand[b, p, int(index[b, t])]))
                parents.append(p)
        starts = [sum(lens[:b]) for b in range(self.B + 1)]
        cu, par, rows, rule_kept, attn_kept = ints(starts), ints(parents), max(lens), {}, {}

        def rule(i, q, k, v, log_alpha, beta):
            o, U = gt.verify_packed(q, k, v, log_alpha, beta, par, cu, self.states[i], N_max=rows)
            rule_kept[i] = (U, k, log_alpha)
            return o

        def attention(i, q, k, v):
            attn_kept[i] = (k, v)
            return self.attend(i, q, k, v, par, cu, rows)

        below = self.model.run(ints(tokens), rule, attention)
        # greedy: follow the model's own choice while the tree has it
        choice, paths = below.argmax(-1).tolist(), []
        for b in range(self.B):
            path = [0]
            while True:
                want = choice[starts[b] + path[-1]]
                child = [t for t in range(lens[b])
                         if parents[starts[b] + t] == path[-1] and tokens[starts[b] + t] == want]
                if not child:
                    break
                path += child[:1]
            paths.append(path)
        taken = [[tokens[starts[b] + t] for t in path[1:]] for b, path in enumerate(paths)]
        last = below[ints([starts[b] + path[-1] for b, path in enumerate(paths)]).long()]
        path_len = ints([len(x) for x in paths])
        path = ints([x + [-1] * (DEPTH - len(x)) for x in paths])
        for i, (U, k, log_alpha) in rule_kept.items():
            gt.commit_packed(path, path_len, U, k, log_alpha, cu, self.states[i],
                             pool_out=self.states[i], parent=par, N_max=rows)
        for i, (k, v) in attn_kept.items():
            kept = self.append(i, k, v, cu, rows, path=path, path_len=path_len)
        self.context_len = kept
        return taken, last


def whole(model, lists):
    """The logits behind each list of tokens, from nothing."""
    lens = [len(x) for x in lists]
    ends = [sum(lens[:b + 1]) for b in range(len(lists))]
    cu = ints([0] + ends)
    no_cache = torch.zeros(1, PAGE, HKV, D, dtype=torch.bfloat16, device="cuda")

    def rule(i, *qkvab):
        return gt.prefill(*qkvab, cu, torch.zeros(len(lists), HV, DK, DK, device="cuda"))[0]

    def attention(i, q, k, v):
        return gt.attend(q, k, v, None, cu, no_cache, no_cache,
                         torch.zeros(len(lists), 1, dtype=torch.int32, device="cuda"),
                         ints([0] * len(lists)))[0]

    return model.run(ints(sum(lists, [])), rule, attention)[ints(ends).long() - 1]


def serve(batch=6, rounds=6, seed=0):
    """Serves a batch; returns the tokens of each sequence, how many of them were drafted, and
    how far the served logits are from those of the whole sequences (relative 2-norm)."""
    gen = torch.Generator().manual_seed(seed)
    some = lambda n: torch.randint(VOCAB, (n,), generator=gen).tolist()  # noqa: E731
    system, prompts = some(75), [some(5 + 17 * b) for b in range(batch)]
    model = Model(seed)
    server = Server(model, system, batch)
    logits = server.prompts(prompts)
    tokens, drafted = [system + p for p in prompts], 0
    for r in range(rounds):
        following = logits.argmax(-1).tolist()
        if r % 3 < 2:
            taken, logits = server.tree(following, 100 * seed + r)
        else:
            taken, logits = [[]] * batch, server.step(ints(following))
        for b in range(batch):
            tokens[b] += [following[b]] + taken[b]
            drafted += len(taken[b])
    want = whole(model, tokens)
    return tokens, drafted, float((logits - want).norm() / want.norm())


if __name__ == "__main__":
    tokens, drafted, far = serve()
    for b, t in enumerate(tokens):
        print("sequence %d: %d tokens, the last %s" % (b, len(t), t[-12:]))
    print("%d tokens came from drafts; served and whole logits differ by %.1e" % (drafted, far))
