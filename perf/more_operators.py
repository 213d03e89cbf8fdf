"""A full cache, shared and thinned out: measured cases.

Four operators around the paged latent cache of a decode step, each in its plain
form (elementary torch operations) and as the call that a user makes of the
library:

  shared   decode of a batch whose requests begin with the same long prefix: the
           prefix's pages are read and multiplied once for all of them
  mass     the attention weight that a step's queries gave each cached token,
           summed over heads and added to what earlier steps gave
  select   which tokens stay when a request's cache is cut to a budget: the
           first and the newest ones, and of the others those of most weight
  compact  the rows of the tokens that stay, moved to the front of the request's
           pages in every layer, and their weights with them

Sizes are those of the library's workloads (128 heads, or a tensor-parallel
rank's 16; 512 + 64 latent dims; contexts of one to 131,072 tokens).
"""
import math
import random

import torch

own = False

ROW, LORA = 576, 512
SCALE = 1.0 / math.sqrt(192.0)
KV_SCALE = 0.037


def listed():
    return [
        # a few short requests behind one short system prompt, a tensor-parallel rank's heads: the smallest step
        dict(name="shared_4x16", op="shared", batch=4, heads=16, page=16, shared=512, tails="1,17,64,200"),
        # a data-parallel rank's 20 requests, every head, half of their context in common
        dict(name="shared_20x128", op="shared", batch=20, heads=128, page=64, shared=2048, tails="64-2048"),
        # a node's 159 requests on a tensor-parallel rank, a long prompt in common
        dict(name="shared_159x16", op="shared", batch=159, heads=16, page=64, shared=4096, tails="16-1024"),
        # a rank that serves many requests of one very long prompt, every head
        dict(name="shared_64x128", op="shared", batch=64, heads=128, page=128, shared=8192, tails="1-777"),
        # one short request, every head
        dict(name="mass_1", op="mass", lens="201", heads=128, page=64, fp8=False, decay=1.0),
        # a data-parallel rank's step, every head, older steps fading
        dict(name="mass_20x4096", op="mass", lens=",".join(["4096"] * 20), heads=128, page=64, fp8=False, decay=0.99),
        # one very long request beside short ones, E4M3 cache, a tensor-parallel rank's heads
        dict(name="mass_e4m3_long", op="mass", lens="131072,1024,1024,1024,1024,1024,1024,1024", heads=16, page=64, fp8=True, decay=1.0),
        # short requests cut to a small budget
        dict(name="select_short", op="select", lens="2,18,65,201", budget=32, sink=4, recent=8),
        # a rank's requests cut to half
        dict(name="select_20x4096", op="select", lens=",".join(["4096"] * 20), budget=2048, sink=4, recent=512),
        # one very long request beside short ones
        dict(name="select_long", op="select", lens="131072,1024,1024,1024,1024,1024,1024,1024", budget=16001, sink=64, recent=1000),
        # one layer of a rank's requests cut to half
        dict(name="compact_20x4096", op="compact", lens=",".join(["4096"] * 20), budget=2048, sink=4, recent=512, layers=1, page=64, fp8=False),
        # several layers of ragged contexts held in E4M3
        dict(name="compact_e4m3_8_layers", op="compact", lens="8191,100,4097,2600,6000,5001,777,3333", budget=3001, sink=16, recent=333, layers=8,
             page=32, fp8=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _text(values):
    return ",".join(str(v) for v in values)


def _ints(text):
    return [int(v) for v in text.split(",")]


def _tails(case):
    """Tokens of each request behind the shared ones: a list, or one drawn from a range."""
    if "-" not in case["tails"]:
        return _ints(case["tails"])
    low, high = (int(v) for v in case["tails"].split("-"))
    rng = random.Random(case["batch"] * 131 + case["shared"])
    return [_log(rng, max(low, 1), high) for _ in range(case["batch"])]


def draw(rng):
    op = rng.choice(["shared", "shared", "mass", "mass", "select", "compact"])
    heads, page = rng.choice([1, 8, 16, 32, 64, 128]), rng.choice([16, 32, 64, 128, 256])
    if op == "shared":
        batch = min(_log(rng, 1, 256), 8192 // heads)
        shared = -(-_log(rng, 64, 8192) // page) * page
        high = _log(rng, 4, 2048)
        while batch * high > 64 * 1024:
            high //= 2
        return dict(op=op, batch=batch, heads=heads, page=page, shared=shared, tails="%d-%d" % (rng.randint(1, high), high))
    most = rng.choice([256, 4096, 131072])
    lens = [_log(rng, 1, most) for _ in range(rng.randint(1, 32))]
    while len(lens) > 1 and sum(lens) > 80000:
        lens.pop()
    if op == "mass":
        return dict(op=op, lens=_text(lens), heads=heads, page=page, fp8=rng.random() < 0.5, decay=rng.choice([1.0, 0.9]))
    sink, recent = rng.choice([0, 1, 4, 64]), _log(rng, 1, 512)
    budget = sink + recent + _log(rng, 1, max(2, max(lens)))
    if op == "select":
        return dict(op=op, lens=_text(lens), budget=budget, sink=sink, recent=recent)
    return dict(op=op, lens=_text(lens), budget=budget, sink=sink, recent=recent, layers=rng.choice([1, 1, 2, 4]), page=page, fp8=rng.random() < 0.5)


def _pages(lens, page, gen, first=0):
    """A block table over a shuffled pool with a quarter more pages than needed; each request's first
    `first` entries are left out (-1)."""
    need = [max(0, -(-n // page) - first) for n in lens]
    blocks = max(1, first + math.ceil(1.25 * sum(need)))
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, first + max(need))), -1, dtype=torch.int32, device="cuda")
    at = first
    for b, n in enumerate(need):
        table[b, first:first + n] = order[at:at + n]
        at += n
    return table, order[:first].contiguous(), blocks


def _lens(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _e4m3(x):
    return (x.float() / KV_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 29)

    def normal(*shape, by=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * by).to(torch.bfloat16)

    s = dict(op=case["op"])
    if case["op"] == "shared":
        B, H, page, shared = case["batch"], case["heads"], case["page"], case["shared"]
        lens = [shared + n for n in _tails(case)]
        table, shared_table, blocks = _pages(lens, page, gen, shared // page)
        s.update(q=normal(B, H, ROW), cache=normal(blocks, page, ROW), block_table=table, shared_table=shared_table, shared_blocks=_lens([shared // page]),
                 seq_lens=_lens(lens), shared=shared, longest=max(lens), out=torch.empty(B, H, LORA, dtype=torch.bfloat16, device="cuda"),
                 lse=torch.empty(B, H, dtype=torch.float32, device="cuda"), workspace=None)
        if own:
            import mla_latent_cache_decode_gb300 as mla
            s["workspace"] = mla.make_shared_workspace(B, H)
        return s
    lens = _ints(case["lens"])
    B, longest = len(lens), max(lens)
    s.update(seq_lens=_lens(lens), longest=longest)
    if case["op"] == "mass":
        H = case["heads"]
        table, _, blocks = _pages(lens, case["page"], gen)
        s.update(q=normal(B, H, ROW), cache=normal(blocks, case["page"], ROW), block_table=table, scale=None, decay=case["decay"],
                 before=torch.rand(B, longest, generator=gen, device="cuda") ** 8, mass=torch.zeros(B, longest, device="cuda"))
        if case["fp8"]:
            s["cache"], s["scale"] = _e4m3(s["cache"]), KV_SCALE
        # the step's own log-sum-exps, as its decode leaves them
        lse = torch.empty(B, H, device="cuda")
        for b, n in enumerate(lens):
            at = torch.arange(n, device="cuda")
            rows = s["cache"].view(-1, ROW)[table[b, at // case["page"]].long() * case["page"] + at % case["page"]]
            rows = rows.float() if s["scale"] is None else rows.view(torch.float8_e4m3fn).float() * KV_SCALE
            lse[b] = torch.logsumexp(s["q"][b].float() @ rows.T * SCALE, 1)
        s["lse"] = lse
        return s
    # weights as they come: most of them small, a few large, and tokens that nothing has looked at yet
    mass = torch.exp(2.0 * torch.randn(B, longest, generator=gen, device="cuda") - 3.0)
    mass *= torch.rand(B, longest, generator=gen, device="cuda") < 0.9
    s.update(mass=mass, sink=case["sink"], recent=case["recent"], keep=torch.empty(B, case["budget"], dtype=torch.int32, device="cuda"),
             new_lens=torch.empty(B, dtype=torch.int32, device="cuda"))
    if case["op"] == "compact":
        table, _, blocks = _pages(lens, case["page"], gen)
        chosen = _plain_select(s)
        s.update(keep=chosen["keep"], new_lens=chosen["new_lens"], block_table=table, fp8=case["fp8"],
                 cache=torch.stack([normal(blocks, case["page"], ROW) for _ in range(case["layers"])]))
        if case["fp8"]:
            s["cache"] = _e4m3(s["cache"])
    return s


# ------------------------------------------------------------------- plain forms

def _gather(s, first=0):
    """Every request's rows from token `first` on, padded to the longest: fp32 [B, tokens, 576], and which are real."""
    page = s["cache"].shape[1]
    at = torch.arange(first, max(first + 1, s["longest"]), device="cuda")
    real = at < s["seq_lens"][:, None]
    blocks = torch.where(real, s["block_table"][:, (at // page).clamp(max=s["block_table"].shape[1] - 1)], 0).long()
    rows = s["cache"].view(-1, ROW)[blocks * page + at % page]
    if s.get("scale") is not None:
        return rows.view(torch.float8_e4m3fn).float() * s["scale"], real
    return rows.float(), real


def _plain_shared(s):
    B, H, _ = s["q"].shape
    q = s["q"].float() * SCALE
    prefix = s["cache"][s["shared_table"].long()].reshape(-1, ROW)[:s["shared"]].float()
    rows, real = _gather(s, s["shared"])
    x = torch.matmul(q.view(-1, ROW), prefix.T).view(B, H, -1)
    y = torch.matmul(q, rows.transpose(1, 2)).masked_fill_(~real[:, None], -math.inf)
    top = torch.maximum(x.amax(2), y.amax(2))[..., None]
    x, y = (x - top).exp_(), (y - top).exp_()
    total = x.sum(2) + y.sum(2)
    out = torch.matmul(x.view(B * H, -1), prefix[:, :LORA]).view(B, H, LORA) + torch.matmul(y, rows[..., :LORA])
    return {"out": (out / total[..., None]).to(torch.bfloat16), "lse": top[..., 0] + total.log()}


def _plain_mass(s):
    rows, real = _gather(s)
    x = torch.matmul(s["q"].float() * SCALE, rows.transpose(1, 2))
    given = (x - s["lse"][..., None]).exp_().sum(1)
    return {"mass": torch.where(real, s["decay"] * s["before"] + given, 0.0)}


def _plain_select(s):
    n, budget = s["seq_lens"][:, None].long(), s["keep"].shape[1]
    at = torch.arange(s["longest"], device="cuda")
    safe = (at < s["sink"]) | (at >= n - s["recent"])
    x = torch.where(safe, math.inf, s["mass"]).masked_fill(at >= n, -math.inf)
    order = torch.sort(x, dim=1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(1, order, at.expand_as(order))
    kept = (rank < budget) & (at < n)
    place = kept.cumsum(1) - 1
    keep = torch.full((len(x), budget + 1), -1, dtype=torch.int64, device="cuda")
    keep.scatter_(1, torch.where(kept, place, budget), torch.where(kept, at, -1))
    return {"keep": keep[:, :budget].to(torch.int32), "new_lens": kept.sum(1).to(torch.int32)}


def _plain_compact(s):
    page = s["cache"].shape[2]
    j = torch.arange(s["keep"].shape[1], device="cuda")
    b, j = torch.nonzero(j < s["new_lens"][:, None], as_tuple=True)
    t = s["keep"][b, j].long()
    source = s["block_table"][b, t // page].long() * page + t % page
    target = s["block_table"][b, j // page].long() * page + j % page
    rows = s["cache"].view(len(s["cache"]), -1, ROW)
    rows[:, target] = rows[:, source]
    moved = s["mass"][b, t]
    at = torch.arange(s["longest"], device="cuda")
    s["mass"].masked_fill_(at < s["seq_lens"][:, None], 0.0)
    s["mass"][b, j] = moved
    return {"cache": s["cache"].view(torch.float8_e4m3fn) if s["fp8"] else s["cache"], "mass": s["mass"]}


_PLAIN = {"shared": _plain_shared, "mass": _plain_mass, "select": _plain_select, "compact": _plain_compact}


def _own(s):
    import mla_latent_cache_decode_gb300 as mla
    if s["op"] == "shared":
        mla.mla_decode_shared(s["q"], s["cache"], s["shared_table"], s["shared_blocks"], s["block_table"], s["seq_lens"], SCALE, s["out"], s["lse"],
                              workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "mass":
        if s["scale"] is None:
            mla.mla_attention_mass(s["q"], s["cache"], s["block_table"], s["seq_lens"], SCALE, s["lse"], s["mass"], previous=s["before"], decay=s["decay"])
        else:
            mla.mla_attention_mass_fp8(s["q"], s["cache"], s["block_table"], s["seq_lens"], SCALE, s["lse"], s["mass"], previous=s["before"],
                                       decay=s["decay"], kv_scale=s["scale"])
        return {"mass": s["mass"]}
    if s["op"] == "select":
        mla.mla_evict_select(s["mass"], s["seq_lens"], s["keep"], s["new_lens"], sink=s["sink"], recent=s["recent"])
        return {"keep": s["keep"], "new_lens": s["new_lens"]}
    if s["fp8"]:
        mla.mla_cache_compact_fp8(s["cache"], s["block_table"], s["keep"], s["seq_lens"], s["new_lens"], mass=s["mass"])
        return {"cache": s["cache"].view(torch.float8_e4m3fn), "mass": s["mass"]}
    mla.mla_cache_compact(s["cache"], s["block_table"], s["keep"], s["seq_lens"], s["new_lens"], mass=s["mass"])
    return {"cache": s["cache"], "mass": s["mass"]}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "shared":
        B, H, P, tails = case["batch"], case["heads"], case["shared"], _tails(case)
        return {"bytes": (P + sum(tails)) * ROW * 2 + B * H * (ROW + LORA) * 2 + B * H * 4,
                "flops": 2 * H * (B * P + sum(tails)) * (ROW + LORA)}
    lens = _ints(case["lens"])
    if case["op"] == "mass":
        H = case["heads"]
        return {"bytes": sum(lens) * (ROW * (1 if case["fp8"] else 2) + 8) + len(lens) * H * (ROW * 2 + 4), "flops": 2 * sum(lens) * H * ROW}
    kept = [min(n, case["budget"]) for n in lens]
    if case["op"] == "select":
        return {"bytes": 4 * sum(lens) + 4 * len(lens) * case["budget"], "flops": sum(lens)}
    # rows in front of the first token that goes do not move: about those of the tokens kept for being first
    moved = sum(max(0, k - case["sink"]) for n, k in zip(lens, kept) if k < n)
    return {"bytes": 2 * case["layers"] * moved * ROW * (1 if case["fp8"] else 2) + 4 * sum(kept) + 8 * sum(kept) + 4 * sum(lens), "flops": 0}


# ------------------------------------------------------------- definition, 64 bits

def _rows64(s, b, n, first_table=None):
    page = s["cache"].shape[1]
    pages = s["block_table"][b, :-(-n // page)].long()
    if first_table is not None:
        pages = torch.cat([first_table.long(), pages[len(first_table):]])
    rows = s["cache"][pages].reshape(-1, ROW)[:n]
    return rows.double() if s.get("scale") is None else rows.view(torch.float8_e4m3fn).double() * s["scale"]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "shared":
        out, lse = s["out"].double(), s["lse"].double()
        for b, n in enumerate(_tails(case)):
            rows = _rows64(s, b, case["shared"] + n, s["shared_table"])
            x = (s["q"][b].double() @ rows.T) * SCALE
            lse[b] = torch.logsumexp(x, 1)
            out[b] = torch.softmax(x, 1) @ rows[:, :LORA]
        return {"out": out, "lse": lse}
    lens = _ints(case["lens"])
    if case["op"] == "mass":
        mass = torch.zeros(s["mass"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            x = (s["q"][b].double() @ _rows64(s, b, n).T) * SCALE
            mass[b, :n] = case["decay"] * s["before"][b, :n].double() + torch.exp(x - s["lse"][b].double()[:, None]).sum(0)
        return {"mass": mass}
    if case["op"] == "select":
        keep = torch.full(s["keep"].shape, -1, dtype=torch.int32)
        new = []
        for b, (n, row) in enumerate(zip(lens, s["mass"].cpu().tolist())):
            # the newest and the first ones, then the others from the most weight down, the earlier one first
            fixed = [t for t in range(n) if t < case["sink"] or t >= n - case["recent"]]
            others = sorted((t for t in range(n) if case["sink"] <= t < n - case["recent"]), key=lambda t: -row[t])
            chosen = sorted((fixed + others)[:case["budget"]])
            keep[b, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
            new.append(len(chosen))
        return {"keep": keep.cuda(), "new_lens": _lens(new)}
    cache, mass = s["cache"], s["mass"].double()
    cache = cache.view(torch.float8_e4m3fn).double() if case["fp8"] else cache.double()
    before, weights, page = cache.clone(), mass.clone(), case["page"]
    for b, (n, k) in enumerate(zip(lens, s["new_lens"].tolist())):
        kept = s["keep"][b, :k].long()
        mass[b, :n] = 0
        mass[b, :k] = weights[b, kept]
        for i in range(0, k, page):
            t = kept[i:i + page]
            cache[:, int(s["block_table"][b, i // page]), :len(t)] = before[:, s["block_table"][b, t // page].long(), t % page]
    return {"cache": cache, "mass": mass}
