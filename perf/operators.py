"""The prompt side of multi-head latent attention, as measured cases.

Three operators that stand around a paged latent cache when prompts are taken
in, each in its plain form (elementary torch operations) and as the call that a
user makes of the library:

  append   the new tokens' latent rows: the 512 latent dims normalised, the 64
           shared key dims rotated, both stored into the paged cache (bf16 or
           E4M3), and every head's 64 rotary query dims rotated beside them
  expand   cached rows of each request back to per-head keys and values through
           the absorption weights W_UK and W_UV
  attend   attention of the prompts' queries over those keys and values, ragged
           over requests, causal at the end of each context or not

Sizes are those of the library's workloads (128 heads, or a tensor-parallel
rank's 16; 512 + 64 latent dims; contexts of one to some thousand tokens).
"""
import math

import torch

own = False

NOPE, ROPE, LORA, VDIM, ROW = 128, 64, 512, 128, 576
SCALE = 1.0 / math.sqrt(NOPE + ROPE)
EPS = 1e-6
MAX_POSITION = 131072


def listed():
    return [
        # one request's newest token: the smallest call, between two layers of a decode step
        dict(name="append_1", op="append", tokens=1, heads=128, page=64, fp8=False, pairs="adjacent", norm=True),
        # the 20 requests of a data-parallel rank, one new token each, E4M3 cache
        dict(name="append_20_e4m3", op="append", tokens=20, heads=128, page=64, fp8=True, pairs="adjacent", norm=True),
        # a prompt chunk of odd length, with the rotation in two halves
        dict(name="append_8191", op="append", tokens=8191, heads=128, page=64, fp8=False, pairs="halves", norm=True),
        # four short requests on small pages
        dict(name="expand_short", op="expand", lens="2,18,65,201", heads=128, page=16, fp8=False),
        # a tensor-parallel rank's 16 heads over ragged contexts
        dict(name="expand_16_heads", op="expand", lens="4096,1,777,2048,129,4000", heads=16, page=64, fp8=False),
        # two full prompts, every head
        dict(name="expand_2x4096", op="expand", lens="4096,4096", heads=128, page=64, fp8=False),
        # contexts held in E4M3, one of them odd
        dict(name="expand_e4m3", op="expand", lens="1500,3001", heads=128, page=32, fp8=True),
        # short prompts, one of them a single token
        dict(name="attend_short", op="attend", q_lens="1,17,64,200", kv_lens="1,17,64,200", heads=128, causal=True),
        # a few new tokens on long contexts, a tensor-parallel rank's heads
        dict(name="attend_few_on_long", op="attend", q_lens="5,1,3", kv_lens="8000,4097,6000", heads=16, causal=True),
        # a prompt's next chunk on the context it already has
        dict(name="attend_chunk", op="attend", q_lens="512,300", kv_lens="7680,2347", heads=128, causal=True),
        # ragged prompts of a tensor-parallel rank, every key visible
        dict(name="attend_16_heads_full", op="attend", q_lens="2048,100,1333,511", kv_lens="2048,700,1333,3000", heads=16, causal=False),
        # one long prompt, every head: the largest
        dict(name="attend_8192", op="attend", q_lens="8192", kv_lens="8192", heads=128, causal=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _text(values):
    return ",".join(str(v) for v in values)


def _ints(text):
    return [int(v) for v in text.split(",")]


def draw(rng):
    op = rng.choice(["append", "expand", "attend", "attend"])
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=rng.choice([1, 8, 16, 32, 64, 128]), page=rng.choice([16, 32, 64, 128, 256]),
                    fp8=rng.random() < 0.5, pairs=rng.choice(["adjacent", "halves"]), norm=rng.random() < 0.8)
    heads = rng.choice([1, 8, 16, 32, 64, 128])
    if op == "expand":
        lens = [_log(rng, 1, 4096) for _ in range(rng.randint(1, 8))]
        while sum(lens) > 8192:
            lens.pop()
        return dict(op=op, lens=_text(lens), heads=heads, page=rng.choice([16, 32, 64, 128, 256]), fp8=rng.random() < 0.5)
    causal = rng.random() < 0.75
    q_lens, kv_lens, n, top = [], [], rng.randint(1, 6), rng.choice([64, 1024, 4096, 8192])
    for _ in range(n):
        q = _log(rng, 1, top)
        q_lens.append(q)
        # the prompt alone, on a context that is there already, or (rarely) more queries than keys: some rows see none
        kind = rng.random()
        kv_lens.append(q if kind < 0.5 else min(8192, q + _log(rng, 1, 4096)) if kind < 0.95 else _log(rng, 1, q))
    # no more padded scores (the plain form holds them all) and no more work than the largest listed case
    most = 8192 * 8192 * 128
    while len(q_lens) > 1 and (len(q_lens) * max(q_lens) * max(kv_lens) * heads > most or 2 * _visible(q_lens, kv_lens, causal) * heads > most):
        q_lens.pop()
        kv_lens.pop()
    causal = causal or 2 * _visible(q_lens, kv_lens, False) * heads > most
    return dict(op=op, q_lens=_text(q_lens), kv_lens=_text(kv_lens), heads=heads, causal=causal)


def _offsets(lens, device="cuda"):
    o = [0]
    for n in lens:
        o.append(o[-1] + n)
    return torch.tensor(o, dtype=torch.int32, device=device)


def _pages(lens, page, gen):
    """A block table over a shuffled pool with a quarter more pages than needed."""
    need = [-(-n // page) for n in lens]
    blocks = max(1, math.ceil(1.25 * sum(need)))
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, blocks


def _rope_table():
    """cos and sin of position / 10000^(i/32), i < 32: fp32 [positions, 64], cosines first."""
    freq = 10000.0 ** (-torch.arange(ROPE // 2, dtype=torch.float64, device="cuda") / (ROPE // 2))
    angle = torch.arange(MAX_POSITION, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 17)

    def normal(*shape, by=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * by).to(torch.bfloat16)

    H = case["heads"]
    if case["op"] == "append":
        T, page = case["tokens"], case["page"]
        blocks = max(2, math.ceil(1.25 * T / page))
        cache = normal(blocks, page, ROW)
        q = normal(T, H, NOPE + ROPE)
        s = dict(kv=normal(T, ROW, by=2.0), q_pe=q[..., NOPE:], q_pe_out=torch.empty(T, H, ROPE, dtype=torch.bfloat16, device="cuda"),
                 positions=torch.randint(0, MAX_POSITION, (T,), generator=gen, device="cuda"), table=_rope_table(),
                 slots=torch.randperm(blocks * page, generator=gen, device="cuda")[:T],
                 weight=(1 + 0.1 * torch.randn(LORA, generator=gen, device="cuda")).to(torch.bfloat16) if case["norm"] else None,
                 adjacent=case["pairs"] == "adjacent", cache=cache, scale=None)
        if case["fp8"]:
            s["cache"], s["scale"] = cache.float().to(torch.float8_e4m3fn).view(torch.uint8), 0.037
    elif case["op"] == "expand":
        lens = _ints(case["lens"])
        table, blocks = _pages(lens, case["page"], gen)
        total = sum(lens)
        cache = normal(blocks, case["page"], ROW)
        s = dict(offsets=_offsets(lens), block_table=table, cache=cache, scale=None, w_uk=normal(H, NOPE, LORA, by=LORA ** -0.5),
                 w_uv=normal(H, LORA, VDIM, by=LORA ** -0.5), k_nope=torch.empty(total, H, NOPE, dtype=torch.bfloat16, device="cuda"),
                 v=torch.empty(total, H, VDIM, dtype=torch.bfloat16, device="cuda"), k_pe=torch.empty(total, ROPE, dtype=torch.bfloat16, device="cuda"))
        if case["fp8"]:
            s["cache"], s["scale"] = (cache.float() / 0.037).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), 0.037
    else:
        q_lens, kv_lens = _ints(case["q_lens"]), _ints(case["kv_lens"])
        Tq, Tk = sum(q_lens), sum(kv_lens)
        q = normal(Tq, H, NOPE + ROPE, by=1.5)
        s = dict(q_nope=q[..., :NOPE], q_pe=normal(Tq, H, ROPE, by=1.5), k_nope=normal(Tk, H, NOPE), k_pe=normal(Tk, ROPE), v=normal(Tk, H, VDIM),
                 q_offsets=_offsets(q_lens), kv_offsets=_offsets(kv_lens), max_q=max(q_lens), max_kv=max(kv_lens), causal=case["causal"],
                 out=torch.empty(Tq, H, VDIM, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(Tq, H, dtype=torch.float32, device="cuda"),
                 workspace=torch.empty(32 << 20, dtype=torch.uint8, device="cuda"))
    s["op"] = case["op"]
    return s


# ------------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, adjacent):
    """Each pair (a, b) of x [..., 64] turned by its angle: (a cos - b sin, b cos + a sin)."""
    if adjacent:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    x = s["kv"].float()
    latent, key = x[:, :LORA], x[:, LORA:]
    if s["weight"] is not None:
        latent = latent * torch.rsqrt((latent * latent).mean(1, keepdim=True) + EPS) * s["weight"].float()
    row = s["table"][s["positions"]]
    cos, sin = row[:, :ROPE // 2], row[:, ROPE // 2:]
    rows = torch.cat([latent, _rotate(key, cos, sin, s["adjacent"])], 1)
    q_pe = _rotate(s["q_pe"].float(), cos[:, None], sin[:, None], s["adjacent"]).to(torch.bfloat16)
    if s["scale"] is None:
        s["cache"].view(-1, ROW)[s["slots"]] = rows.to(torch.bfloat16)
        return {"cache": s["cache"], "q_pe": q_pe}
    codes = (rows * (1.0 / s["scale"])).clamp(-448, 448).to(torch.float8_e4m3fn)
    s["cache"].view(-1, ROW)[s["slots"]] = codes.view(torch.uint8)
    return {"cache": s["cache"].view(torch.float8_e4m3fn), "q_pe": q_pe}


def _plain_expand(s):
    offsets, page = s["offsets"].long(), s["cache"].shape[1]
    at = torch.arange(s["k_pe"].shape[0], device="cuda")
    b = torch.searchsorted(offsets, at, right=True) - 1
    pos = at - offsets[b]
    slot = s["block_table"][b, pos // page].long() * page + pos % page
    rows = s["cache"].view(-1, ROW)[slot]
    rows = rows.float() if s["scale"] is None else rows.view(torch.float8_e4m3fn).float() * s["scale"]
    latent = rows[:, :LORA]
    k = torch.matmul(latent, s["w_uk"].float().flatten(0, 1).T).view(-1, s["w_uk"].shape[0], NOPE)
    v = torch.matmul(latent, s["w_uv"].float().transpose(0, 1).flatten(1)).view(-1, s["w_uv"].shape[0], VDIM)
    return {"k_nope": k.to(torch.bfloat16), "v": v.to(torch.bfloat16), "k_pe": rows[:, LORA:].to(torch.bfloat16)}


def _plain_attend(s):
    qo, ko = s["q_offsets"].long(), s["kv_offsets"].long()
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_kv"], device="cuda")
    nq, nk = qo.diff()[:, None], ko.diff()[:, None]
    at_q = (qo[:-1, None] + i).clamp(max=s["q_pe"].shape[0] - 1)
    at_k = (ko[:-1, None] + j).clamp(max=s["k_pe"].shape[0] - 1)
    # requests padded to the longest: [batch, heads, tokens, dims]
    qn, qp = s["q_nope"].float()[at_q].transpose(1, 2), s["q_pe"].float()[at_q].transpose(1, 2)
    kn, kp = s["k_nope"].float()[at_k].transpose(1, 2), s["k_pe"].float()[at_k][:, None]
    scores = torch.matmul(qn, kn.transpose(2, 3))
    scores += torch.matmul(qp, kp.transpose(2, 3))
    scores *= SCALE
    seen = (j < nk)[:, None, :]
    if s["causal"]:
        seen = seen & (j <= i[:, None] + (nk - nq)[:, :, None])
    scores.masked_fill_(~seen[:, None], -math.inf)
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    scores -= top
    scores.exp_()
    total = scores.sum(3, keepdim=True)
    out = torch.matmul(scores, s["v"].float()[at_k].transpose(1, 2)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    real = i < nq
    return {"out": out.transpose(1, 2)[real].to(torch.bfloat16), "lse": lse.transpose(1, 2)[real]}


_PLAIN = {"append": _plain_append, "expand": _plain_expand, "attend": _plain_attend}


def _own(s):
    import mla_latent_cache_decode_gb300 as mla
    if s["op"] == "append":
        if s["scale"] is None:
            mla.mla_rope_append(s["kv"], s["positions"], s["table"], s["slots"], s["cache"], norm_weight=s["weight"], eps=EPS, interleaved=s["adjacent"],
                                q_pe=s["q_pe"], q_pe_out=s["q_pe_out"])
            return {"cache": s["cache"], "q_pe": s["q_pe_out"]}
        mla.mla_rope_append_fp8(s["kv"], s["positions"], s["table"], s["slots"], s["cache"], kv_scale=s["scale"], norm_weight=s["weight"], eps=EPS,
                                interleaved=s["adjacent"], q_pe=s["q_pe"], q_pe_out=s["q_pe_out"])
        return {"cache": s["cache"].view(torch.float8_e4m3fn), "q_pe": s["q_pe_out"]}
    if s["op"] == "expand":
        if s["scale"] is None:
            mla.mla_expand_kv(s["cache"], s["block_table"], s["offsets"], s["w_uk"], s["w_uv"], s["k_nope"], s["v"], s["k_pe"])
        else:
            mla.mla_expand_kv_fp8(s["cache"], s["block_table"], s["offsets"], s["w_uk"], s["w_uv"], s["k_nope"], s["v"], s["k_pe"], kv_scale=s["scale"])
        return {"k_nope": s["k_nope"], "v": s["v"], "k_pe": s["k_pe"]}
    mla.mla_prefill(s["q_nope"], s["q_pe"], s["k_nope"], s["k_pe"], s["v"], s["q_offsets"], s["kv_offsets"], SCALE, s["out"], s["lse"],
                    causal=s["causal"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------------- work

def _visible(q_lens, kv_lens, causal):
    """Pairs of a query and a key it sees."""
    n = 0
    for q, k in zip(q_lens, kv_lens):
        rows = min(q, k)  # causal: query i sees keys up to k - q + i, so the first q - k see none
        n += q * k if not causal else rows * (k - rows) + rows * (rows + 1) // 2
    return n


def work(case):
    H = case["heads"]
    if case["op"] == "append":
        T, element = case["tokens"], 1 if case["fp8"] else 2
        rotary = 2 * T * H * ROPE * 2
        return {"bytes": T * (ROW * 2 + ROW * element + 8 + 8 + ROPE * 4) + rotary + (LORA * 2 if case["norm"] else 0),
                "flops": T * (4 * LORA if case["norm"] else 0) + 3 * T * (H + 1) * ROPE}
    if case["op"] == "expand":
        T, element = sum(_ints(case["lens"])), 1 if case["fp8"] else 2
        return {"bytes": T * ROW * element + H * LORA * (NOPE + VDIM) * 2 + T * (H * (NOPE + VDIM) + ROPE) * 2,
                "flops": 2 * T * H * LORA * (NOPE + VDIM)}
    q_lens, kv_lens = _ints(case["q_lens"]), _ints(case["kv_lens"])
    Tq, Tk = sum(q_lens), sum(kv_lens)
    return {"bytes": Tq * H * (NOPE + ROPE + VDIM) * 2 + Tq * H * 4 + Tk * (H * (NOPE + VDIM) + ROPE) * 2,
            "flops": 2 * _visible(q_lens, kv_lens, case["causal"]) * H * (NOPE + ROPE + VDIM)}


# ------------------------------------------------------------- definition, 64 bits

def _turn64(x, angle_cos, angle_sin, adjacent):
    z = x.view(*x.shape[:-1], 32, 2) if adjacent else torch.stack(x.split(32, -1), -1)
    turned = torch.view_as_complex(z.contiguous()) * torch.complex(angle_cos, angle_sin)
    pair = torch.view_as_real(turned)
    return pair.flatten(-2) if adjacent else torch.cat([pair[..., 0], pair[..., 1]], -1)


def _e4m3_nearest(x):
    """The E4M3 value nearest to x (64 bits), ties to the even one, within +-448."""
    power = torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 1
    step = torch.ldexp(torch.ones_like(x), power - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        x = s["kv"].double()
        latent = x[:, :LORA]
        if s["weight"] is not None:
            latent = s["weight"].double() * latent / torch.sqrt(latent.square().sum(1, keepdim=True) / LORA + EPS)
        cos, sin = s["table"].double()[s["positions"]].split(32, 1)
        rows = torch.cat([latent, _turn64(x[:, LORA:], cos, sin, s["adjacent"])], 1)
        if s["scale"] is None:
            cache = s["cache"].double()
        else:
            cache, rows = s["cache"].view(torch.float8_e4m3fn).double(), _e4m3_nearest(rows / s["scale"])
        cache.view(-1, ROW).index_copy_(0, s["slots"], rows)
        return {"cache": cache, "q_pe": _turn64(s["q_pe"].double(), cos[:, None], sin[:, None], s["adjacent"])}
    if case["op"] == "expand":
        page = s["cache"].shape[1]
        rows = []
        for b, n in enumerate(_ints(case["lens"])):
            pages = s["cache"][s["block_table"][b, :-(-n // page)].long()]
            rows.append(pages.reshape(-1, ROW)[:n])
        rows = torch.cat(rows)
        rows = rows.double() if s["scale"] is None else rows.view(torch.float8_e4m3fn).double() * s["scale"]
        latent = rows[:, :LORA]
        k, v = (torch.empty(len(rows), case["heads"], n, dtype=torch.float64, device="cuda") for n in (NOPE, VDIM))
        for h in range(case["heads"]):
            k[:, h] = latent @ s["w_uk"][h].double().T
            v[:, h] = latent @ s["w_uv"][h].double()
        return {"k_nope": k, "v": v, "k_pe": rows[:, LORA:]}
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    k_pe = s["k_pe"].double()
    q0 = k0 = 0
    for nq, nk in zip(_ints(case["q_lens"]), _ints(case["kv_lens"])):
        for h in range(case["heads"]):
            for a in range(0, nq, 1024):
                n = min(1024, nq - a)
                at = slice(q0 + a, q0 + a + n)
                last = nk - nq + a + n if case["causal"] else nk  # keys that any of these rows sees
                if last <= 0:
                    continue
                q = torch.cat([s["q_nope"][at, h].double(), s["q_pe"][at, h].double()], 1) * SCALE
                k = torch.cat([s["k_nope"][k0:k0 + last, h].double(), k_pe[k0:k0 + last]], 1)
                x = q @ k.T
                if case["causal"]:
                    x += torch.full_like(x, -math.inf).triu_(nk - nq + a + 1)
                lse[at, h] = torch.logsumexp(x, 1)
                out[at, h] = torch.softmax(x, 1).nan_to_num_() @ s["v"][k0:k0 + last, h].double()
        q0, k0 = q0 + nq, k0 + nk
    return {"out": out, "lse": lse}
