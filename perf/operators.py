"""The training-step operators around the DSpark loss, as measured cases.

Three operators stand beside the fused draft-vocabulary loss:

- linear cross entropy: the cross entropy of ``hidden @ weight.T`` over the whole
  vocabulary, with its gradients, the logits never kept;
- the scaled embedding lookup, and its gradient summed over sorted token ids;
- the global norm of many gradient tensors, and their clipping.

Each case is one pass.  Where ``own`` is false the pass is written in elementary torch
operations in 32 bits (64 for long sums), rounded once; where it is true it makes the
calls a training program makes of this package.
"""

import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
IGNORE = -100


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # --- linear cross entropy.  `rows` hidden rows, `ignored` of them carry no label.
        # One anchor block of a short draft on a small vocabulary: launch latency.
        dict(name="lce_block", op="lce", rows=56, ignored=9, vocab=8192, hidden=512, mode="train",
             weighted=True, z_alpha=0.0),
        # One sequence's last tokens scored against the full vocabulary: the head is read once.
        dict(name="lce_score_few", op="lce", rows=7, ignored=0, vocab=151936, hidden=4096, mode="score",
             weighted=False, z_alpha=0.0),
        # The recipe micro-batch, 4 x 16 blocks of 7, masked to prefixes: head and drafter trained.
        dict(name="lce_recipe_train", op="lce", rows=448, ignored=205, vocab=151936, hidden=4096, mode="train",
             weighted=True, z_alpha=0.0),
        # Odd sizes throughout: rows, vocabulary and hidden size end inside tiles; z-loss on.
        dict(name="lce_odd", op="lce", rows=1021, ignored=100, vocab=32003, hidden=1000, mode="train",
             weighted=False, z_alpha=1e-4),
        # The head is frozen (shared with the target): only the hidden rows get a gradient.
        dict(name="lce_frozen_head", op="lce", rows=1792, ignored=192, vocab=151936, hidden=4096, mode="frozen",
             weighted=True, z_alpha=0.0),
        # A large batch, nearly every row labelled.
        dict(name="lce_large_train", op="lce", rows=8192, ignored=301, vocab=151936, hidden=4096, mode="train",
             weighted=False, z_alpha=0.0),
        # --- embedding.  The tokens of the recipe micro-batch, looked up and scaled.
        dict(name="embed_recipe", op="embed", rows=448, vocab=151936, width=4096, dtype="bf16", dropped=45),
        # A long batch of tokens through a wide table.
        dict(name="embed_long", op="embed", rows=32749, vocab=151936, width=4096, dtype="bf16", dropped=0),
        # The gradient of a low-rank previous-token table from one micro-batch of 8192 rows.
        dict(name="embed_grad_rank", op="embed_grad", rows=8192, vocab=151936, width=256, dtype="bf16",
             grad="f32", dropped=800),
        # The gradient of a wide table from a long batch; token counts fall off as 1/rank.
        dict(name="embed_grad_long", op="embed_grad", rows=32749, vocab=151936, width=4096, dtype="bf16",
             grad="bf16", dropped=0),
        # --- clipping.  The auxiliary heads' gradients: two tables, a projection and a bias.
        dict(name="clip_heads", op="clip", sizes="heads", count=4, low=1, high=1, bf16=0.0, over=True),
        # Many tensors of a small drafter, most of them short, of both types.
        dict(name="clip_many", op="clip", sizes="spread", count=201, low=1, high=300000, bf16=0.5, over=True),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["lce", "lce", "embed", "embed_grad", "clip"])
    if op == "lce":
        rows, width = _log(rng, 1, 8192), 8 * _log(rng, 8, 512)
        return dict(op=op, rows=rows, ignored=int(rows * rng.choice([0.0, 0.1, 0.5]) * rng.random()),
                    vocab=_log(rng, 500, 151936), hidden=width, mode=rng.choice(["train", "train", "frozen", "score"]),
                    weighted=rng.random() < 0.5, z_alpha=rng.choice([0.0, 0.0, 1e-4]))
    if op in ("embed", "embed_grad"):
        rows = _log(rng, 1, 32768)
        case = dict(op=op, rows=rows, vocab=_log(rng, 100, 151936), width=8 * _log(rng, 8, 512),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), dropped=int(rows * rng.choice([0.0, 0.2]) * rng.random()))
        if op == "embed_grad":
            case["grad"] = rng.choice(["f32", "bf16"])
        return case
    return dict(op=op, sizes="spread", count=_log(rng, 1, 300), low=1, high=_log(rng, 1000, 400000),
                bf16=rng.choice([0.0, 0.5, 1.0]), over=rng.random() < 0.7)


def _sizes(case):
    """The element counts of a clipping case's tensors."""
    if case["sizes"] == "heads":
        return [151936 * 256, 151936 * 256, 4096 + 256, 1]
    r = random.Random(case["count"] * 1000003 + case["high"])
    return [_log(r, case["low"], case["high"]) for _ in range(case["count"])]


def _kinds(case):
    r = random.Random(case["count"])
    return ["bf16" if r.random() < case["bf16"] else "f32" for _ in range(case["count"])]


# ---------------------------------------------------------------------- inputs
def _tokens(gen, rows, vocab):
    """Token ids whose counts fall off as 1/rank, the ranks spread over the vocabulary."""
    u = torch.rand(rows, generator=gen, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * torch.log(torch.tensor(float(vocab), device="cuda", dtype=torch.float64))).long() - 1
    return (rank.clamp(0, vocab - 1) * 40503) % vocab


def _views(buckets, sizes, kinds):
    at, views = dict.fromkeys(buckets, 0), []
    for n, k in zip(sizes, kinds):
        views.append(buckets[k][at[k]:at[k] + n])
        at[k] += n
    return views


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] == "lce":
        r, v, h = case["rows"], case["vocab"], case["hidden"]
        weight = (rand(v, h) * (3.0 / h ** 0.5)).to(torch.bfloat16)
        targets = torch.randint(0, v, (r,), generator=gen, device="cuda")
        known = (torch.rand(r, 1, generator=gen, device="cuda") < 0.5).float()
        # half the rows point towards their label, as a half-trained drafter's do
        s["hidden_rows"] = (rand(r, h) + known * weight[targets].float()).to(torch.bfloat16)
        targets[torch.randperm(r, generator=gen, device="cuda")[:case["ignored"]]] = IGNORE
        s["weight"], s["targets"] = weight, targets
        s["row_weight"] = torch.exp(-(torch.arange(r, device="cuda") % 7).float() / 4.0) if case["weighted"] else None
        if own:
            from speculative_decoding_draft_vocab_b200 import torch_api
            s["call"] = torch_api.LinearCE(s["hidden_rows"], weight, targets, row_weight=s["row_weight"],
                                           ignore_index=IGNORE, z_alpha=case["z_alpha"],
                                           dhidden=case["mode"] != "score", dweight=case["mode"] == "train")
    elif case["op"] in ("embed", "embed_grad"):
        r, v, d, t = case["rows"], case["vocab"], case["width"], DTYPES[case["dtype"]]
        s["ids"] = _tokens(gen, r, v)
        s["valid"] = None
        if case["dropped"]:
            s["valid"] = torch.ones(r, dtype=torch.uint8, device="cuda")
            s["valid"][torch.randperm(r, generator=gen, device="cuda")[:case["dropped"]]] = 0
        s["scale"] = d ** 0.5
        if case["op"] == "embed":
            s["table"] = (rand(v, d) * 0.02).to(t)
        else:
            s["dout"] = rand(r, d).to(t)
        if own:
            from speculative_decoding_draft_vocab_b200 import torch_api
            if case["op"] == "embed":
                s["call"] = torch_api.Embedding(s["ids"], s["table"], scale=s["scale"], valid=s["valid"])
            else:
                s["call"] = torch_api.EmbeddingGrad(s["ids"], s["dout"], v, scale=s["scale"], valid=s["valid"],
                                                    dtype=DTYPES[case["grad"]])
    else:
        sizes, kinds = _sizes(case), _kinds(case)
        # each type's tensors lie back to back in one bucket, wherever that puts their first elements
        s["buckets"] = {k: rand(sum(n for n, x in zip(sizes, kinds) if x == k)).to(DTYPES[k])
                        for k in sorted(set(kinds))}
        s["kinds"] = kinds
        s["grads"] = _views(s["buckets"], sizes, kinds)
        expect = sum(sizes) ** 0.5
        s["max_norm"] = 0.3 * expect if case["over"] else 4.0 * expect
        if own:
            from speculative_decoding_draft_vocab_b200 import torch_api
            s["clipped"] = {k: torch.empty_like(b) for k, b in s["buckets"].items()}
            s["call"] = torch_api.GradClip(s["grads"], s["max_norm"], outs=_views(s["clipped"], sizes, kinds))
    return s


# ------------------------------------------------------------------------ one pass
def _lce_plain(s):
    keep = s["targets"] != IGNORE
    w = keep.float() if s["row_weight"] is None else keep * s["row_weight"]
    t = torch.where(keep, s["targets"], 0)
    hidden, weight = s["hidden_rows"].float(), s["weight"].float()
    z = hidden @ weight.T
    top = z.max(dim=1, keepdim=True).values
    p = torch.exp(z - top)
    total = p.sum(dim=1, keepdim=True)
    lse = (torch.log(total) + top)[:, 0]
    ce = lse - z.gather(1, t[:, None])[:, 0]
    del z
    num = (w.double() * (ce.double() + s["z_alpha"] * lse.double() ** 2)).sum().float()
    out = dict(loss_num=num, num_tokens=keep.sum(), ce_rows=torch.where(keep, ce, 0.0),
               lse_rows=torch.where(keep, lse, 0.0))
    if s["mode"] == "score":
        return out
    p *= (w * (1.0 + 2.0 * s["z_alpha"] * lse))[:, None] / total
    p.scatter_add_(1, t[:, None], -w[:, None])
    out["dhidden"] = (p @ weight).to(torch.bfloat16)
    if s["mode"] == "train":
        out["dweight"] = (p.T @ hidden).to(torch.bfloat16)
    return out


def _embed_plain(s):
    x = s["table"][s["ids"]].float() * s["scale"]
    if s["valid"] is not None:
        x = torch.where(s["valid"][:, None] != 0, x, 0.0)
    return x.to(s["table"].dtype)


def _embed_grad_plain(s):
    x = s["dout"].float() * s["scale"]
    if s["valid"] is not None:
        x = torch.where(s["valid"][:, None] != 0, x, 0.0)
    total = torch.zeros(s["vocab"], s["width"], device="cuda").index_add_(0, s["ids"], x)
    return total.to(DTYPES[s["grad"]])


def _clip_plain(s):
    sq = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum()
    norm = sq.sqrt().float()
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    coef = torch.where(torch.isfinite(norm), coef, 1.0)
    clipped = [(g.float() * coef).to(g.dtype) for g in s["grads"]]
    return dict(norm=norm, coef=coef, grads={k: torch.cat([c for c, x in zip(clipped, s["kinds"]) if x == k])
                                             for k in s["buckets"]})


def run(state):
    if own:
        call = state["call"]
        if state["op"] == "lce":
            call.forward()
            out = dict(loss_num=call.loss_num[0], num_tokens=call.num_tokens[0], ce_rows=call.ce_rows,
                       lse_rows=call.lse_rows)
            if state["mode"] != "score":
                call.backward()
                out["dhidden"] = call.dhidden
                if state["mode"] == "train":
                    out["dweight"] = call.dweight
            return out
        call.launch()
        if state["op"] == "clip":
            return dict(norm=call.norm[0], coef=call.coef[0], grads=state["clipped"])
        return call.out
    return {"lce": _lce_plain, "embed": _embed_plain, "embed_grad": _embed_grad_plain,
            "clip": _clip_plain}[state["op"]](state)


# ---------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "lce":
        r, v, h = case["rows"], case["vocab"], case["hidden"]
        n = r - case["ignored"]
        products = {"score": 1, "frozen": 2, "train": 3}[case["mode"]]
        moved = 2 * n * h + 2 * v * h + 8 * r + 8 * r  # labelled hidden rows, head, labels, row outputs
        moved += (2 * r * h if products > 1 else 0) + (2 * v * h if products > 2 else 0)
        return dict(bytes=moved, flops=2 * n * v * h * products)
    if case["op"] in ("embed", "embed_grad"):
        es = 2 if case["dtype"] == "bf16" else 4
        kept = case["rows"] - case["dropped"]
        if case["op"] == "embed":
            return dict(bytes=8 * case["rows"] + (kept + case["rows"]) * case["width"] * es,
                        flops=kept * case["width"])
        gs = 2 if case["grad"] == "bf16" else 4
        return dict(bytes=8 * case["rows"] + kept * case["width"] * es + case["vocab"] * case["width"] * gs,
                    flops=2 * kept * case["width"])
    sizes, kinds = _sizes(case), _kinds(case)
    moved = sum(n * (2 if k == "bf16" else 4) for n, k in zip(sizes, kinds))
    return dict(bytes=2 * moved, flops=3 * sum(sizes))  # read once, written once


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lce":
        return _lce_exact(s)
    if case["op"] == "embed":
        rows = s["table"].index_select(0, s["ids"]).double().mul_(s["scale"])
        return rows if s["valid"] is None else rows.masked_fill_((s["valid"] == 0).unsqueeze(1), 0.0)
    if case["op"] == "embed_grad":
        kept = torch.arange(case["rows"], device="cuda") if s["valid"] is None else s["valid"].nonzero().flatten()
        table = torch.zeros(case["vocab"], case["width"], dtype=torch.float64, device="cuda")
        for part in kept.split(4096):
            table.index_add_(0, s["ids"][part], s["dout"][part].double(), alpha=s["scale"])
        return table
    norm = sum(float(b.double().pow(2).sum()) for b in s["buckets"].values()) ** 0.5
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    one = lambda x: torch.tensor(x, dtype=torch.float64, device="cuda")  # noqa: E731
    return dict(norm=one(norm), coef=one(coef), grads={k: b.double() * coef for k, b in s["buckets"].items()})


def _lce_exact(s):
    """Rows in bands, each band over the whole vocabulary at once."""
    r, h = s["hidden_rows"].shape
    weight = s["weight"].double()
    zero = lambda *n: torch.zeros(*n, dtype=torch.float64, device="cuda")  # noqa: E731
    ce, lse, dh = zero(r), zero(r), zero(r, h)
    dw = zero(*weight.shape) if s["mode"] == "train" else None
    num = zero(1)
    kept = (s["targets"] != IGNORE).nonzero().flatten()
    for rows in kept.split(1024):
        x, t = s["hidden_rows"][rows].double(), s["targets"][rows]
        z = torch.matmul(x, weight.transpose(0, 1))
        l = torch.logsumexp(z, dim=1)
        c = l - z[torch.arange(rows.numel(), device="cuda"), t]
        a = torch.ones_like(l) if s["row_weight"] is None else s["row_weight"][rows].double()
        ce[rows], lse[rows] = c, l
        num += (a * (c + s["z_alpha"] * l * l)).sum()
        if s["mode"] == "score":
            continue
        g = torch.exp(z - l[:, None]) * (1.0 + 2.0 * s["z_alpha"] * l)[:, None]
        g[torch.arange(rows.numel(), device="cuda"), t] -= 1.0
        g *= a[:, None]
        dh[rows] = torch.matmul(g, weight)
        if dw is not None:
            dw.addmm_(g.transpose(0, 1), x)
    out = dict(loss_num=num[0], num_tokens=None, ce_rows=ce, lse_rows=lse)
    if s["mode"] != "score":
        out["dhidden"] = dh
        if dw is not None:
            out["dweight"] = dw
    return out
