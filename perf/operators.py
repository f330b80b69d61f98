"""Cases of the target model's attention operators around the verify step: what is timed, and what it must equal.

Three operators run once a layer when a target model scores drafted windows:

* ``rotary``     rotates the first ``rot`` elements of every head of x [tokens, heads, d] by the token's position;
* ``append``     rotates the new keys (and the queries) and writes keys and values into a paged cache;
* ``attention``  attends a window of new tokens of every request over its paged cache, causal, each request's window
                 ending at its cache length.

A frequency table is fp32 [rot / 2, 2]: the frequency in turns per position as an unevaluated sum high + low.

``run`` computes the plain form (elementary torch operations in fp32, rounded once) or, with ``own`` set, calls the
framework's operators.  The plain form reduces angles in fp64 before taking fp32 sines, because position * frequency in
fp32 is off by 1e-2 radians at the positions of long contexts.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
DEV = "cuda"


# ---------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # the queries of one drafted window (8 tokens) on their own: latency only
        dict(name="rotary one window", op="rotary", dtype="bf16", tokens=8, heads=32, d=128, rot=128,
             interleaved=False, inverse=False, pos=4096, stretch=1.0),
        # backward of a partial rotation in the interleaved layout, fp32, odd token count, a training micro-batch
        dict(name="rotary partial gradient", op="rotary", dtype="f32", tokens=1021, heads=24, d=64, rot=32,
             interleaved=True, inverse=True, pos=1021, stretch=1.0),
        # queries and keys of long prompts at stretched positions
        dict(name="rotary long prompts", op="rotary", dtype="bf16", tokens=16384, heads=40, d=128, rot=128,
             interleaved=False, inverse=False, pos=131072, stretch=8.0),
        # single tokens of a few requests: plain decoding, latency only
        dict(name="append single tokens", op="append", dtype="f16", batch=7, win_lo=1, win_hi=1, len_lo=100, len_hi=900,
             hq=14, hkv=2, d=64, rot=64, interleaved=True, page=16, heads_first=False, stretch=1.0),
        # drafted windows of the ragged verify step: 256 requests, 2048 tokens or so
        dict(name="append verify windows", op="append", dtype="bf16", batch=256, win_lo=1, win_hi=15, len_lo=128,
             len_hi=1024, hq=32, hkv=8, d=128, rot=128, interleaved=False, page=16, heads_first=False, stretch=4.0),
        # whole prompts, half of each head rotated, heads-first pages
        dict(name="append prompts", op="append", dtype="bf16", batch=5, win_lo=1001, win_hi=4097, len_lo=4099, len_hi=8191,
             hq=32, hkv=8, d=128, rot=64, interleaved=False, page=64, heads_first=True, stretch=1.0),
        # one token of one short request: the smallest call
        dict(name="attend one token", op="attention", dtype="f16", batch=1, win_lo=1, win_hi=1, len_lo=333, len_hi=333,
             hq=8, hkv=2, d=64, page=16, window=0, heads_first=False),
        # plain decoding of a batch with ragged lengths
        dict(name="attend single tokens", op="attention", dtype="bf16", batch=64, win_lo=1, win_hi=1, len_lo=256,
             len_hi=8192, hq=32, hkv=8, d=128, page=16, window=0, heads_first=False),
        # the ragged verify step's windows (256 requests of 16-token blocks cut to about 2048 tokens)
        dict(name="attend verify windows", op="attention", dtype="bf16", batch=256, win_lo=1, win_hi=15, len_lo=128,
             len_hi=4096, hq=32, hkv=8, d=128, page=32, window=0, heads_first=False),
        # 8-token blocks over very long contexts, few requests: the cache read is split over its length
        dict(name="attend long contexts", op="attention", dtype="bf16", batch=4, win_lo=8, win_hi=8, len_lo=65536,
             len_hi=131072, hq=64, hkv=8, d=128, page=64, window=0, heads_first=True),
        # chunks of long prompts over what the cache holds already: arithmetic counts
        dict(name="attend prompt chunks", op="attention", dtype="bf16", batch=2, win_lo=2048, win_hi=2048, len_lo=8192,
             len_hi=16384, hq=32, hkv=8, d=128, page=64, window=0, heads_first=False),
        # ragged whole prompts with narrow heads, one query head per key head, sliding window
        dict(name="attend sliding window", op="attention", dtype="f16", batch=5, win_lo=301, win_hi=2003, len_lo=301,
             len_hi=2003, hq=16, hkv=16, d=64, page=16, window=512, heads_first=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attention", "attention"])
    if op == "rotary":
        d = rng.choice([64, 80, 128])
        heads = rng.randint(1, 64)
        tokens = min(_log(rng, 1, 16384), 16384 * 40 * 128 // (heads * d) // 2)
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), tokens=tokens, heads=heads, d=d,
                    rot=rng.choice([d, d // 2, 32]), interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5,
                    pos=_log(rng, 64, 131072), stretch=rng.choice([1.0, 1.0, 4.0, 8.0]))
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    kind = rng.choice(["single", "windows", "windows", "prompts"])
    batch = _log(rng, 1, 8 if kind == "prompts" else 256)
    win = {"single": (1, 1), "windows": (1, rng.randint(1, 16)), "prompts": (17, _log(rng, 64, 4096))}[kind]
    len_hi = max(win[1], _log(rng, 16, 65536 if op == "attention" else 8192))
    case = dict(op=op, dtype=rng.choice(["bf16", "f16"]), batch=batch, win_lo=win[0], win_hi=win[1],
                len_lo=max(win[1], len_hi // rng.choice([1, 2, 8])), len_hi=len_hi, hq=hq, hkv=hkv, d=d, page=page,
                heads_first=rng.random() < 0.3)
    if op == "append":
        case.update(rot=rng.choice([d, d // 2]), interleaved=rng.random() < 0.5, stretch=rng.choice([1.0, 4.0]))
    else:
        case.update(window=rng.choice([0, 0, 0, 127, 1024]))
    while _too_large(case):                       # fewer requests first, then shorter ones
        if case["batch"] > 1:
            case["batch"] = (case["batch"] + 1) // 2
        else:
            case["len_hi"] = max(case["win_hi"], case["len_hi"] * 3 // 4)
            case["len_lo"] = max(case["win_hi"], min(case["len_lo"], case["len_hi"]))
            if case["len_hi"] == case["win_hi"]:
                case["win_hi"] = case["len_hi"] = case["len_lo"] = max(case["win_lo"], case["win_hi"] * 3 // 4)
    return case


def _too_large(c):
    cache = 2 * c["batch"] * c["len_hi"] * c["hkv"] * c["d"] * 2
    scores = c["batch"] * c["hq"] * c["win_hi"] * c["len_hi"] * 4
    flops = work(c)["flops"] if c["op"] == "attention" else 0
    return cache > 1.0e9 or (c["op"] == "attention" and (scores > 4.0e9 or flops > 4.0e11))


def _spread(lo, hi, n, step):
    """n whole numbers over [lo, hi] in a fixed scattered order, even over their logarithm, the ends among them."""
    if n == 1:
        return [hi]
    f = [((i * step) % 1.0) for i in range(n)]
    f[0], f[-1] = 0.0, 1.0
    return [min(hi, max(lo, int(round(math.exp(math.log(lo) + x * (math.log(hi) - math.log(lo))))))) for x in f]


def _shape(case):
    """Window and cache lengths of a case's requests."""
    wins = _spread(case["win_lo"], case["win_hi"], case["batch"], 0.6180339887)
    lens = _spread(case["len_lo"], case["len_hi"], case["batch"], 0.4142135624)
    return wins, [max(n, w) for n, w in zip(lens, wins)]


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _frequencies(rot, stretch):
    """Turns per position of each pair, base 10000; stretched: slow pairs slowed down by `stretch`, fast ones kept."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if stretch != 1.0:
        turns = 4096 * f / (2 * math.pi)                      # turns over the length the model was trained on
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        f = f * keep + f / stretch * (1 - keep)
    f = f / (2 * math.pi)
    high = f.to(torch.float32)
    return torch.stack([high, (f - high.double()).to(torch.float32)], dim=1).contiguous().to(DEV)


def _randn(g, *shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _cache(case, g, lens, dtype):
    """Key and value pages (NHD order, or views of heads-first storage) and a scattered page table."""
    page, hkv, d, batch = case["page"], case["hkv"], case["d"], case["batch"]
    per = [-(-n // page) for n in lens]
    n_pages = sum(per) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV, dtype=torch.int64)
    table = torch.zeros((batch, max(per)), dtype=torch.int32, device=DEV)
    flat = torch.tensor([b * max(per) + j for b in range(batch) for j in range(per[b])], device=DEV)
    table.view(-1)[flat] = order[: sum(per)].to(torch.int32)
    dims = (n_pages, hkv, page, d) if case["heads_first"] else (n_pages, page, hkv, d)
    k, v = (torch.empty(dims, dtype=dtype, device=DEV) for _ in range(2))
    for t in (k, v):
        t.copy_(torch.randn(dims, generator=g, device=DEV, dtype=dtype if dtype != torch.float32 else torch.float32))
    if case["heads_first"]:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    return k, v, table


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "rotary":
        # x: the query heads of a packed projection output, so tokens are a larger stride apart
        packed = _randn(g, case["tokens"], case["heads"] + 2, case["d"], dtype=dtype)
        start = torch.randint(0, case["pos"], (case["tokens"],), generator=g, device=DEV, dtype=torch.int32)
        return dict(case=case, x=packed[:, : case["heads"]], positions=start,
                    freq=_frequencies(case["rot"], case["stretch"]), mscale=1.0 + 0.1 * math.log(case["stretch"]))
    wins, lens = _shape(case)
    qo = [0]
    for n in wins:
        qo.append(qo[-1] + n)
    state = dict(case=case, wins=wins, lens=lens,
                 qo_indptr=torch.tensor(qo, dtype=torch.int32, device=DEV),
                 kv_len=torch.tensor(lens, dtype=torch.int32, device=DEV))
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    state["k_pages"], state["v_pages"], state["table"] = _cache(case, g, lens, dtype)
    if case["op"] == "append":
        packed = _randn(g, qo[-1], hq + 2 * hkv, d, dtype=dtype)      # one projection's output
        state.update(q=packed[:, :hq], k=packed[:, hq:hq + hkv], v=packed[:, hq + hkv:],
                     freq=_frequencies(case["rot"], case["stretch"]), mscale=1.0 + 0.1 * math.log(case["stretch"]))
    else:
        state["q"] = _randn(g, qo[-1], hq, d, dtype=dtype, scale=1.5)
    return state


# ---------------------------------------------------------------------------------------------------------------
# One pass: the plain form, or the framework's operators
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "rotary":
        return _plain_rotate(state["x"], state["positions"], state["freq"], case["interleaved"],
                             -1.0 if case["inverse"] else 1.0, state["mscale"])
    return _plain_append(state, case) if case["op"] == "append" else _plain_attend(state, case)


def _own(state, case):
    from speculative_decoding_verification_rows_gb300 import sv

    if case["op"] == "rotary":
        return sv.rotary(state["x"], state["positions"], state["freq"], interleaved=case["interleaved"],
                         inverse=case["inverse"], mscale=state["mscale"])
    if case["op"] == "append":
        q = sv.kv_append(state["k"], state["v"], state["k_pages"], state["v_pages"], state["table"],
                         state["qo_indptr"], state["kv_len"], freq=state["freq"], interleaved=case["interleaved"],
                         mscale=state["mscale"], q=state["q"])
        return dict(q=q, k_pages=state["k_pages"], v_pages=state["v_pages"])
    if "ws" not in state:
        state["ws"] = sv.Workspace(DEV)
    out = sv.paged_attention(state["q"], state["k_pages"], state["v_pages"], state["table"], state["qo_indptr"],
                             state["kv_len"], max_window=case["win_hi"], scale=case["d"] ** -0.5,
                             window=case["window"], ws=state["ws"])
    return dict(out=out.out, lse=out.lse)


def _plain_rotate(x, positions, freq, interleaved, sign, mscale):
    rot = 2 * freq.shape[0]
    turns = positions.double()[:, None] * (freq[:, 0].double() + freq[:, 1].double())
    angle = (2 * math.pi * (turns - turns.round())).float()[:, None, :]
    c, s = torch.cos(angle) * mscale, torch.sin(angle) * (sign * mscale)
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([turned, y[..., rot:]], dim=-1).to(x.dtype)


def _request_of(qo_indptr, tokens):
    t = torch.arange(tokens, device=qo_indptr.device, dtype=torch.int32)
    return torch.searchsorted(qo_indptr, t, right=True) - 1, t


def _plain_append(state, case):
    qo, kv_len, page = state["qo_indptr"], state["kv_len"], case["page"]
    r, t = _request_of(qo, state["q"].shape[0])
    pos = kv_len[r] - qo[r + 1] + t
    where = state["table"][r, pos // page].long(), (pos % page).long()
    turn = lambda x: _plain_rotate(x, pos, state["freq"], case["interleaved"], 1.0, state["mscale"])  # noqa: E731
    state["k_pages"].index_put_(where, turn(state["k"]))
    state["v_pages"].index_put_(where, state["v"])
    return dict(q=turn(state["q"]), k_pages=state["k_pages"], v_pages=state["v_pages"])


def _plain_attend(state, case):
    q, qo, kv_len, table = state["q"], state["qo_indptr"], state["kv_len"], state["table"]
    hq, hkv, d, batch, n = case["hq"], case["hkv"], case["d"], case["batch"], case["win_hi"]
    keys = table.shape[1] * case["page"]
    count = qo[1:] - qo[:-1]
    i = torch.arange(n, device=q.device, dtype=torch.int32)
    tok = (qo[:-1, None] + i).clamp(max=q.shape[0] - 1).long()
    rows = q[tok].float().view(batch, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    k = state["k_pages"][table.long()].flatten(1, 2).permute(0, 2, 3, 1).float()
    s = torch.matmul(rows, k).view(batch, hkv, hq // hkv, n, keys)
    del k
    s *= d ** -0.5
    pos = (kv_len - count)[:, None] + i
    j = torch.arange(keys, device=q.device, dtype=torch.int32)
    hidden = j > pos[..., None]
    if case["window"]:
        hidden |= j <= pos[..., None] - case["window"]
    s.masked_fill_(hidden[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s -= torch.where(m == -math.inf, 0.0, m)
    s.exp_()
    total = s.sum(-1, keepdim=True)
    v = state["v_pages"][table.long()].flatten(1, 2).permute(0, 2, 1, 3).float()
    o = torch.matmul(s.view(batch, hkv, -1, keys), v).view(batch, hkv, hq // hkv, n, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(batch, n, hq, d)
    lse = (m + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(batch, n, hq)
    r, t = _request_of(qo, q.shape[0])
    at = (t - qo[r]).long()
    return dict(out=o[r, at].to(q.dtype), lse=lse[r, at])


# ---------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    size = SIZES[case["dtype"]]
    if case["op"] == "rotary":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["d"] * size + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    wins, lens = _shape(case)
    tokens, hq, hkv, d = sum(wins), case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        return {"bytes": 2 * tokens * (hq + 2 * hkv) * d * size + 4 * tokens, "flops": 3 * tokens * (hq + hkv) * case["rot"]}
    window = case["window"]
    pairs = keys = 0
    for w, n in zip(wins, lens):
        first = n - w                                        # position of the window's first token
        if not window:
            pairs += w * first + w * (w + 1) // 2
            keys += n
        else:
            short = max(0, min(w, window - 1 - first))       # tokens that still see fewer than `window` keys
            pairs += short * first + short * (short + 1) // 2 + (w - short) * window
            keys += min(n, w + window - 1)
    return {"bytes": (2 * keys * hkv + 2 * tokens * hq) * d * size + 4 * tokens * hq, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rotary":
        return _turned64(state["x"], state["positions"], state["freq"], case["interleaved"],
                         -1 if case["inverse"] else 1, state["mscale"])
    if case["op"] == "append":
        return _append64(state, case)
    return _attend64(state, case)


def _turned64(x, positions, freq, interleaved, sign, mscale):
    """Every pair as a complex number times mscale * exp(i * sign * 2 pi * position * frequency)."""
    rot = 2 * freq.shape[0]
    f = freq.double().sum(1)
    turn = torch.polar(torch.full((1,), mscale, dtype=torch.float64, device=x.device),
                       torch.remainder(positions.double()[:, None] * f, 1.0) * (sign * 2 * math.pi))[:, None]
    out = x.double().clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(out[..., first], out[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _append64(state, case):
    page, at = case["page"], 0
    pages = state["table"].tolist()
    positions = [n - w + i for w, n in zip(state["wins"], state["lens"]) for i in range(w)]
    positions = torch.tensor(positions, device=DEV)
    q, k = (_turned64(state[x], positions, state["freq"], case["interleaved"], 1, state["mscale"]) for x in "qk")
    kp, vp, v = state["k_pages"].double(), state["v_pages"].double(), state["v"].double()
    for b, (w, n) in enumerate(zip(state["wins"], state["lens"])):
        p = n - w
        while p < n:                                         # one page at a time
            m = min(page - p % page, n - p)
            kp[pages[b][p // page], p % page: p % page + m] = k[at: at + m]
            vp[pages[b][p // page], p % page: p % page + m] = v[at: at + m]
            p, at = p + m, at + m
    return dict(q=q, k_pages=kp, v_pages=vp)


def _attend64(state, case):
    hq, hkv, d, window = case["hq"], case["hkv"], case["d"], case["window"]
    out = torch.zeros((state["q"].shape[0], hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((state["q"].shape[0], hq), -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (w, n) in enumerate(zip(state["wins"], state["lens"])):
        pages = state["table"][b, : -(-n // case["page"])].long()
        k = state["k_pages"][pages].flatten(0, 1)[:n]
        v = state["v_pages"][pages].flatten(0, 1)[:n]
        p = torch.arange(n - w, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)
        seen = (j <= p) & ((j > p - window) if window else True)
        for h in range(hq):
            kv = h // (hq // hkv)
            s = state["q"][at: at + w, h].double() @ k[:, kv].double().T / math.sqrt(d)
            s = torch.where(seen, s, -math.inf)
            lse[at: at + w, h] = torch.logsumexp(s, -1)
            out[at: at + w, h] = torch.softmax(s, -1) @ v[:, kv].double()
        at += w
    return dict(out=out, lse=lse)
