"""Cases and plain forms of the serving operators around a shared, paged latent cache.

Two sets, each used by a serving loop next to the decode step:

* a prompt prefix that a whole batch shares, expanded once into per-head keys and values
  (``expand``), attended to by every request of the step at once (``attend``), and joined
  with the decode over each request's own tokens in front of the output projection
  (``project``);
* a cache that outgrows its budget: the attention weight that each cached token received,
  summed over heads and query tokens and accumulated over steps (``weigh``), and the
  eviction that keeps the heaviest tokens and closes the gaps (``evict``).

``own`` selects the framework's calls; otherwise ``run`` computes the same in elementary
torch operations in fp32, rounded once to the output's type.
"""
import math

import torch

own = False

PAGE = 64
THETA = 10000.0
# heads, model width, latent width, rotary width, content width and value width per head
V2 = dict(d=5120, d_c=512, d_r=64, d_n=128, d_v=128)
TINY = dict(d=256, d_c=64, d_r=16, d_n=32, d_v=32)
DIMS = {"v2": V2, "tiny": TINY}


def listed():
    return [
        # a long system prompt or few-shot prefix admitted once, before its batch is served
        dict(name="expand_8192", op="expand", dims="v2", heads=128, length=8192, cache="bf16"),
        # a short prefix with an odd end, from the block-scaled fp8 cache
        dict(name="expand_1000_fp8block", op="expand", dims="v2", heads=128, length=1000,
             cache="fp8_e4m3_b128"),
        # the smallest call: one fp32 request of the tiny shape, two pages of prefix
        dict(name="attend_tiny_f32", op="attend", dims="tiny", heads=16, batch=1, q_len=1, length=128),
        # one decode step of 128 requests behind one long prefix
        dict(name="attend_b128_8192", op="attend", dims="v2", heads=128, batch=128, q_len=1, length=8192),
        # speculative decoding: four query tokens of each request
        dict(name="attend_b64_q4_4096", op="attend", dims="v2", heads=128, batch=64, q_len=4, length=4096),
        # the end of the attention block of a step: join prefix and own tokens, project
        dict(name="project_32", op="project", dims="v2", heads=128, rows=32),
        # the same for a large speculative batch (256 requests x 2 tokens)
        dict(name="project_512", op="project", dims="v2", heads=128, rows=512),
        # weights of a decode step's keys, at the ordinary serving size
        dict(name="weigh_b32_4096", op="weigh", dims="v2", heads=128, batch=32, q_len=1, shortest=4096,
             longest=4096, cache="bf16", decay=1.0),
        # few long contexts
        dict(name="weigh_b4_long", op="weigh", dims="v2", heads=128, batch=4, q_len=1, shortest=32768,
             longest=131072, cache="bf16", decay=0.9),
        # a per-tensor fp8 cache, odd ragged lengths
        dict(name="weigh_b64_fp8", op="weigh", dims="v2", heads=128, batch=64, q_len=1, shortest=1000,
             longest=8192, cache="fp8_e4m3", decay=1.0),
        # halve every request's cache in place
        dict(name="evict_b32_in_place", op="evict", dims="v2", batch=32, shortest=4096, longest=4096,
             cache="bf16", budget=2048, sinks=4, recent=256, in_place=True),
        # ragged requests of a large batch into new pages; the short ones stay whole
        dict(name="evict_b256_ragged", op="evict", dims="v2", batch=256, shortest=512, longest=8192,
             cache="bf16", budget=1500, sinks=4, recent=64, in_place=False),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["expand", "attend", "attend", "project", "weigh", "weigh", "evict"])
    tiny = rng.random() < 0.15
    dims = "tiny" if tiny else "v2"
    heads = 16 if tiny else rng.choice([16, 32, 64, 128, 128])
    cache = "f32" if tiny else rng.choice(["bf16", "bf16", "fp8_e4m3", "fp8_e4m3_b128"])
    if op == "expand":
        return dict(op=op, dims=dims, heads=heads, length=_log(rng, 1, 1024 if tiny else 8192), cache=cache)
    if op == "attend":
        q_len = rng.choice([1, 1, 1, 2, 4])
        batch = _log(rng, 1, 128 // q_len)
        return dict(op=op, dims=dims, heads=heads, batch=batch, q_len=q_len,
                    length=_log(rng, 1, 1024 if tiny else 8192))
    if op == "project":
        return dict(op=op, dims=dims, heads=heads, rows=_log(rng, 1, 512))
    if op == "weigh":
        batch, q_len = _log(rng, 1, 64), rng.choice([1, 1, 2, 4])
        longest = _log(rng, 64, 1024 if tiny else min(131072, 262144 // (batch * q_len)))
        return dict(op=op, dims=dims, heads=heads, batch=batch, q_len=q_len,
                    shortest=rng.randint(q_len, longest), longest=longest, cache=cache,
                    decay=rng.choice([0.0, 0.9, 1.0]))
    batch = _log(rng, 1, 128)
    longest = _log(rng, 64, 1024 if tiny else min(65536, 262144 // batch))
    budget = rng.randint(16, longest)
    recent = rng.randint(0, budget // 4)
    return dict(op=op, dims=dims, batch=batch, shortest=rng.randint(1, longest), longest=longest,
                cache=cache, budget=budget, sinks=rng.randint(0, min(8, budget - recent)),
                recent=recent, in_place=rng.random() < 0.5)


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _ints(g, lo, hi, shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _act(case):
    return torch.float32 if case["dims"] == "tiny" else torch.bfloat16


def _pages(n):
    return -(-n // PAGE)


def _spread(case):
    """The batch's lengths, the longest first: even over [shortest, longest]."""
    lo, hi = case["shortest"], case["longest"]
    return [hi] + [lo + int((hi - lo + 1) * (i * 0.6180339887498949 % 1)) for i in range(1, case["batch"])]


def _lengths(case, g):
    lens = torch.tensor(_spread(case), dtype=torch.int32, device="cuda")
    return lens[torch.randperm(case["batch"], generator=g, device="cuda")].contiguous()


def _tables(g, counts, width):
    """Block tables [len(counts)][width] over one shuffled pool, and the pool's size. Entries
    behind a request's last page are -1."""
    counts = torch.as_tensor(counts, device="cuda", dtype=torch.int64)
    total = int(counts.sum())
    perm = torch.randperm(total + 3, generator=g, device="cuda")[:total]
    at = torch.arange(width, device="cuda")[None, :]
    first = torch.cumsum(counts, 0) - counts
    used = at < counts[:, None]
    table = torch.where(used, perm[torch.clamp(first[:, None] + at, max=max(total - 1, 0))], -1)
    return table.to(torch.int32).contiguous(), total + 3


def _cache(case, g, num_pages, m):
    """A filled cache pool [num_pages][64][row] and its per-tensor scale: N(0, 1) latents and
    rotary keys in the cache's own format (random rows: the rotation keeps their distribution)."""
    rows, kind = num_pages * PAGE, case["cache"]
    D = m["d_c"] + m["d_r"]
    if kind in ("f32", "bf16"):
        t = torch.float32 if kind == "f32" else torch.bfloat16
        return torch.randn((rows, D), generator=g, device="cuda", dtype=t).view(num_pages, PAGE, D), 1.0
    if kind == "fp8_e4m3":
        scale = 5.25 / 448.0
        x = torch.randn((rows, D), generator=g, device="cuda") / scale
        return x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(num_pages, PAGE, D), scale
    c = torch.randn((rows, m["d_c"] // 128, 128), generator=g, device="cuda")
    s = c.abs().amax(-1) / 448.0
    codes = (c / s[..., None]).clamp_(-448, 448).to(torch.float8_e4m3fn)
    k = torch.randn((rows, m["d_r"]), generator=g, device="cuda").to(torch.bfloat16)
    row = torch.cat([codes.view(torch.uint8).view(rows, -1), s.view(torch.uint8), k.view(torch.uint8)], 1)
    return row.view(num_pages, PAGE, -1).contiguous(), 1.0


def _config(case, m, scale=1.0, heads=None):
    import mla_latent_kv_04_gb300 as M

    class Dims:
        num_heads, d_model, d_latent = heads or case.get("heads", 128), m["d"], m["d_c"]
        d_rope, d_nope, d_v, page_size = m["d_r"], m["d_n"], m["d_v"], PAGE
    act = "f32" if case["dims"] == "tiny" else "bf16"
    return M, M.make_config(Dims, act, case.get("cache", act), cache_scale=scale, rope_theta=THETA)


def prepare(case, seed):
    g, m, act = _gen(seed), DIMS[case["dims"]], _act(case)
    s = dict(case=case, m=m)
    if case["op"] == "expand":
        H, L = case["heads"], case["length"]
        s["table"], n = _tables(g, [_pages(L)], _pages(L))
        s["table"] = s["table"][0].contiguous()
        s["cache"], s["scale"] = _cache(case, g, n, m)
        s["W_UK"] = _normal(g, (m["d_c"], H * m["d_n"]), act, m["d_c"] ** -0.5)
        s["W_UV"] = _normal(g, (m["d_c"], H * m["d_v"]), act, m["d_c"] ** -0.5)
        s["keys"] = torch.empty((H, L, m["d_n"]), dtype=act, device="cuda")
        s["values"] = torch.empty((H, L, m["d_v"]), dtype=act, device="cuda")
        s["k_pe"] = torch.empty((L, m["d_r"]), dtype=act, device="cuda")
    elif case["op"] == "attend":
        H, L, B, q = case["heads"], case["length"], case["batch"], case["q_len"]
        s["keys"] = _normal(g, (H, L, m["d_n"]), act)
        s["values"] = _normal(g, (H, L, m["d_v"]), act)
        s["k_pe"] = _normal(g, (L, m["d_r"]), act)
        s["q_nope"] = _normal(g, (B, q, H, m["d_n"]), act)
        s["q_pe"] = _normal(g, (B, q, H, m["d_r"]), act)
        s["lens"] = _ints(g, q, 4096, (B,))
        s["u"] = torch.empty((B, q, H, m["d_v"]), dtype=act, device="cuda")
        s["lse"] = torch.empty((B, q, H), dtype=torch.float32, device="cuda")
    elif case["op"] == "project":
        H, R = case["heads"], case["rows"]
        s["o_lat"] = _normal(g, (R, H, m["d_c"]), act, 0.05)
        s["u_prefix"] = _normal(g, (R, H, m["d_v"]), act, 0.05)
        s["lse"] = 7.0 + torch.randn((R, H), generator=g, device="cuda")
        s["lse_prefix"] = 8.0 + torch.randn((R, H), generator=g, device="cuda")
        s["W_UV"] = _normal(g, (m["d_c"], H * m["d_v"]), act, m["d_c"] ** -0.5)
        s["W_O"] = _normal(g, (H * m["d_v"], m["d"]), act, (H * m["d_v"]) ** -0.5)
        s["out"] = torch.empty((R, m["d"]), dtype=act, device="cuda")
    elif case["op"] == "weigh":
        H, B, q = case["heads"], case["batch"], case["q_len"]
        s["lens"] = _lengths(case, g)
        width = _pages(case["longest"])
        s["table"], n = _tables(g, -(-s["lens"].long() // PAGE), width)
        s["cache"], s["scale"] = _cache(case, g, n, m)
        s["q_lat"] = _normal(g, (B, q, H, m["d_c"] + m["d_r"]), act, 0.6)
        # the decode's LSE of these heads: that of independent N(0, sd^2) scores
        norm = s["q_lat"].float().square().sum(-1) / (m["d_n"] + m["d_r"])
        s["lse"] = (torch.log(s["lens"].float())[:, None, None] + 0.5 * norm).contiguous()
        s["weights"] = torch.rand((B, width * PAGE), generator=g, device="cuda")
    else:
        B = case["batch"]
        s["lens"] = _lengths(case, g)
        width, budget = _pages(case["longest"]), case["budget"]
        counts = -(-s["lens"].long() // PAGE)
        if case["in_place"]:
            s["table"], n = _tables(g, counts, width)
            s["new_table"] = s["table"]
        else:
            kept = -(-s["lens"].long().clamp(max=budget) // PAGE)
            both, n = _tables(g, torch.cat([counts, kept]), width)
            s["table"] = both[:B].contiguous()
            s["new_table"] = both[B:, : _pages(min(budget, case["longest"]))].contiguous()
        s["cache"], s["scale"] = _cache(case, g, n, m)
        # accumulated weights: a heavy tail, and one token in twenty that never had any
        w = torch.exp(1.5 * torch.randn((B, width * PAGE), generator=g, device="cuda"))
        s["weights"] = w * (torch.rand(w.shape, generator=g, device="cuda") > 0.05)
        s["new_weights"] = torch.zeros((B, s["new_table"].shape[1] * PAGE), device="cuda")
        s["kept"] = torch.empty((B, budget), dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty((B,), dtype=torch.int32, device="cuda")
    if own:
        M, s["cfg"] = _config(case, m, s.get("scale", 1.0))
        need = 0
        if case["op"] == "attend":
            need = M.mla_prefix_attend_workspace_size(s["cfg"], case["batch"], case["q_len"], case["length"])
        elif case["op"] == "project":
            need = M.mla_output_proj_prefix_workspace_size(s["cfg"], case["rows"])
        s["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms

def _rows(raw, kind, m, scale):
    """Latent and rotary parts of raw cache rows [...][row], in fp32."""
    if kind in ("f32", "bf16"):
        x = raw.float()
        return x[..., : m["d_c"]], x[..., m["d_c"]:]
    if kind == "fp8_e4m3":
        x = raw.view(torch.float8_e4m3fn).float() * scale
        return x[..., : m["d_c"]], x[..., m["d_c"]:]
    c, n = m["d_c"], m["d_c"] // 128
    codes = raw[..., :c].contiguous().view(torch.float8_e4m3fn).float()
    s = raw[..., c: c + 4 * n].contiguous().view(torch.float32)
    x = (codes.unflatten(-1, (n, 128)) * s[..., None]).flatten(-2)
    return x, raw[..., c + 4 * n:].contiguous().view(torch.bfloat16).float()


def _turn(x, pos, m):
    """Pairs (2k, 2k + 1) of x turned by pos * theta^(-2k / d_r); pos broadcasts over x's
    leading dimensions. The angles are formed in fp64 (far positions)."""
    k = torch.arange(m["d_r"] // 2, device=x.device, dtype=torch.float64)
    a = pos.double()[..., None] * THETA ** (-2.0 * k / m["d_r"])
    sn, cs = torch.sin(a).float(), torch.cos(a).float()
    p = x.unflatten(-1, (-1, 2))
    x0, x1 = p[..., 0], p[..., 1]
    return torch.stack([x0 * cs - x1 * sn, x0 * sn + x1 * cs], -1).flatten(-2)


def _gather(cache, table):
    """The rows of every request, [B][pages * 64][row] (unused table entries give page 0)."""
    return cache[table.long().clamp(min=0)].flatten(1, 2)


def _plain_expand(s):
    m, H = s["m"], s["case"]["heads"]
    L = s["case"]["length"]
    c, k = _rows(_gather(s["cache"], s["table"][None])[0, :L], s["case"]["cache"], m, s["scale"])
    act = s["W_UK"].dtype
    keys = (c @ s["W_UK"].float()).view(L, H, -1).transpose(0, 1)
    values = (c @ s["W_UV"].float()).view(L, H, -1).transpose(0, 1)
    return keys.to(act).contiguous(), values.to(act).contiguous(), k.to(act)


def _plain_attend(s):
    m, c = s["m"], s["case"]
    B, q, H = c["batch"], c["q_len"], c["heads"]
    pos = c["length"] + s["lens"].long()[:, None] - q + torch.arange(q, device="cuda")
    q_pe = _turn(s["q_pe"].float(), pos[:, :, None].expand(B, q, H), m).reshape(B * q, H, -1)
    score = torch.einsum("rhd,hld->hrl", s["q_nope"].float().reshape(B * q, H, -1), s["keys"].float())
    score = score + torch.einsum("rhd,ld->hrl", q_pe, s["k_pe"].float())
    score = score * (m["d_n"] + m["d_r"]) ** -0.5
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    u = (p @ s["values"].float()) / total
    lse = (top + torch.log(total))[..., 0]
    act = s["q_nope"].dtype
    return (u.transpose(0, 1).reshape(B, q, H, -1).to(act).contiguous(),
            lse.transpose(0, 1).reshape(B, q, H).contiguous())


def _plain_project(s):
    m, H, R = s["m"], s["case"]["heads"], s["case"]["rows"]
    W_UV = s["W_UV"].float().view(m["d_c"], H, -1)
    u = torch.einsum("rhc,chv->rhv", s["o_lat"].float(), W_UV)
    a = 1.0 / (1.0 + torch.exp(s["lse_prefix"] - s["lse"]))[..., None]
    u = a * u + (1.0 - a) * s["u_prefix"].float()
    return (u.reshape(R, -1) @ s["W_O"].float()).to(s["W_O"].dtype)


def _plain_weigh(s):
    m, case = s["m"], s["case"]
    q, lens = case["q_len"], s["lens"].long()
    c, k = _rows(_gather(s["cache"], s["table"]), case["cache"], m, s["scale"])
    ql = s["q_lat"].float()
    B, _, H, _ = ql.shape
    x = torch.cat([c, k], -1)
    score = (ql.reshape(B, q * H, -1) @ x.transpose(1, 2)).view(B, q, H, -1) * (m["d_n"] + m["d_r"]) ** -0.5
    j = torch.arange(score.shape[-1], device="cuda")
    sees = j <= (lens[:, None] - q + torch.arange(q, device="cuda"))[:, :, None]
    p = torch.where(sees[:, :, None], torch.exp(score - s["lse"][..., None]), 0.0)
    mass = p.sum((1, 2))
    old = torch.where(j < (lens - q)[:, None], s["weights"], 0.0)
    s["weights"].copy_(torch.where(j < lens[:, None], case["decay"] * old + mass, s["weights"]))
    return s["weights"]


def _order(s):
    """kept [B][budget] (-1 behind the end) and the new lengths."""
    case, lens = s["case"], s["lens"].long()
    w, budget, sinks, recent = s["weights"], case["budget"], case["sinks"], case["recent"]
    j = torch.arange(w.shape[1], device="cuda")
    live = j < lens[:, None]
    sure = live & ((j < sinks) | (j >= (lens - recent)[:, None]) | (lens <= budget)[:, None])
    key = torch.where(sure, math.inf, torch.where(live, w, -math.inf))
    first = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :budget]
    new = lens.clamp(max=budget)
    at = torch.arange(first.shape[1], device="cuda")
    first = torch.where(at < new[:, None], first, w.shape[1]).sort(1).values
    kept = torch.full((w.shape[0], budget), -1, device="cuda", dtype=torch.int32)
    kept[:, : first.shape[1]] = torch.where(at < new[:, None], first, -1).to(torch.int32)
    return kept, new


def _parts(s):
    """The cache pool as the values it holds."""
    cache, kind, m = s["cache"], s["case"]["cache"], s["m"]
    if kind in ("f32", "bf16"):
        return cache
    if kind == "fp8_e4m3":
        return cache.view(torch.float8_e4m3fn)
    c, n = m["d_c"], m["d_c"] // 128
    return [cache[..., :c].contiguous().view(torch.float8_e4m3fn),
            cache[..., c: c + 4 * n].contiguous().view(torch.float32),
            cache[..., c + 4 * n:].contiguous().view(torch.bfloat16)]


def _plain_evict(s):
    m, case, kind = s["m"], s["case"], s["case"]["cache"]
    kept, new = _order(s)
    b, i = torch.nonzero(kept >= 0, as_tuple=True)
    j = kept[b, i].long()
    src = s["table"].long()[b, j // PAGE] * PAGE + j % PAGE
    dst = s["new_table"].long()[b, i // PAGE] * PAGE + i % PAGE
    flat = s["cache"].view(-1, s["cache"].shape[-1])
    raw = flat[src]
    _, k = _rows(raw, kind, m, s["scale"])
    k = _turn(k, i - j, m)
    if kind == "fp8_e4m3":
        k = torch.where((i == j)[:, None], raw[:, m["d_c"]:],
                        (k / s["scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        raw[:, m["d_c"]:] = k
    elif kind == "fp8_e4m3_b128":
        raw[:, m["d_c"] + m["d_c"] // 32:] = k.to(torch.bfloat16).view(torch.uint8)
    else:
        raw[:, m["d_c"]:] = k.to(raw.dtype)
    flat[dst] = raw
    s["new_weights"][b, i] = s["weights"][b, j]
    s["kept"].copy_(kept)
    s["new_lens"].copy_(new)
    return s["kept"], s["new_lens"], s["new_weights"], _parts(s)


PLAIN = {"expand": _plain_expand, "attend": _plain_attend, "project": _plain_project,
         "weigh": _plain_weigh, "evict": _plain_evict}


# ------------------------------------------------------------------------------- one pass

def _own(s):
    import mla_latent_kv_04_gb300 as M

    c, cfg = s["case"], s["cfg"]
    if c["op"] == "expand":
        M.mla_prefix_expand(cfg, s["W_UK"], s["W_UV"], s["cache"], s["table"], c["length"], s["keys"],
                            s["values"], s["k_pe"])
        return s["keys"], s["values"], s["k_pe"]
    if c["op"] == "attend":
        M.mla_prefix_attend(cfg, s["q_nope"], s["q_pe"], s["keys"], s["values"], s["k_pe"], s["lens"],
                            s["u"], s["lse"], s["ws"])
        return s["u"], s["lse"]
    if c["op"] == "project":
        M.mla_output_proj_prefix(cfg, s["o_lat"], s["lse"], s["u_prefix"], s["lse_prefix"], s["W_UV"],
                                 s["W_O"], s["out"], s["ws"])
        return s["out"]
    if c["op"] == "weigh":
        M.mla_key_weights(cfg, s["q_lat"], s["lse"], s["cache"], s["table"], s["lens"], s["weights"],
                          decay=c["decay"])
        return s["weights"]
    M.mla_evict_cache(cfg, s["weights"], s["lens"], s["table"], s["cache"], c["budget"], s["kept"],
                      s["new_lens"], new_block_table=s["new_table"], new_weights=s["new_weights"],
                      sinks=c["sinks"], recent=c["recent"])
    return s["kept"], s["new_lens"], s["new_weights"], _parts(s)


def run(s):
    return _own(s) if own else PLAIN[s["case"]["op"]](s)


# ------------------------------------------------------------------------------- work

def _row_bytes(kind, m):
    size = {"f32": 4, "bf16": 2, "fp8_e4m3": 1}
    if kind in size:
        return (m["d_c"] + m["d_r"]) * size[kind]
    return m["d_c"] + m["d_c"] // 32 + 2 * m["d_r"]


def work(case):
    m = DIMS[case["dims"]]
    a = 4 if case["dims"] == "tiny" else 2
    H = case.get("heads", 128)
    if case["op"] == "expand":
        L, n = case["length"], H * (m["d_n"] + m["d_v"])
        return {"bytes": L * _row_bytes(case["cache"], m) + a * (m["d_c"] * n + L * n + L * m["d_r"]),
                "flops": 2 * L * m["d_c"] * n}
    if case["op"] == "attend":
        L, R = case["length"], case["batch"] * case["q_len"]
        d = m["d_n"] + m["d_r"]
        return {"bytes": a * (L * (H * (m["d_n"] + m["d_v"]) + m["d_r"]) + R * H * (d + m["d_v"])) + 4 * R * H,
                "flops": 2 * R * H * L * (d + m["d_v"])}
    if case["op"] == "project":
        R = case["rows"]
        return {"bytes": a * (R * H * (m["d_c"] + m["d_v"]) + m["d_c"] * H * m["d_v"] + H * m["d_v"] * m["d"]
                              + R * m["d"]) + 8 * R * H,
                "flops": 2 * R * H * m["d_v"] * (m["d_c"] + m["d"])}
    lens = _spread(case)
    n = sum(lens)
    if case["op"] == "weigh":
        q = case["q_len"]
        return {"bytes": n * (_row_bytes(case["cache"], m) + (8 if case["decay"] else 4))
                + case["batch"] * q * H * (a * (m["d_c"] + m["d_r"]) + 4),
                "flops": 2 * n * q * H * (m["d_c"] + m["d_r"])}
    keep = sum(min(x, case["budget"]) for x in lens)
    # in place, a request within its budget and the first tokens of the others stay where they are
    stay = sum(x if x <= case["budget"] else case["sinks"] for x in lens) if case["in_place"] else 0
    return {"bytes": n * 4 + (keep - stay) * 2 * _row_bytes(case["cache"], m) + keep * 8,
            "flops": 3 * (keep - stay) * m["d_r"]}


# ------------------------------------------------------------------------------- 64 bits

def _exact_rows(case, m, raw, scale):
    """c [n][d_c] and k [n][d_r] of raw rows, in fp64."""
    kind, dc = case["cache"], m["d_c"]
    if kind in ("f32", "bf16"):
        x = raw.double()
        return x[:, :dc], x[:, dc:]
    if kind == "fp8_e4m3":
        # the scale as the library holds it: fp32
        x = raw.contiguous().view(torch.float8_e4m3fn).to(torch.float32).double() * float(torch.tensor(scale, dtype=torch.float32))
        return x[:, :dc], x[:, dc:]
    c = raw[:, :dc].contiguous().view(torch.float8_e4m3fn).to(torch.float32).double()
    sc = raw[:, dc: dc + dc // 32].contiguous().view(torch.float32).double()
    return (c * sc.repeat_interleave(128, 1),
            raw[:, dc + dc // 32:].contiguous().view(torch.bfloat16).double())


def _exact_turn(z, angle_pos, m):
    """The complex form of the rotation: pairs as complex numbers times e^(i pos theta_k)."""
    inv = torch.tensor([THETA ** (-2.0 * k / m["d_r"]) for k in range(m["d_r"] // 2)], dtype=torch.float64,
                       device=z.device)
    c = torch.view_as_complex(z.double().reshape(*z.shape[:-1], -1, 2).contiguous())
    a = angle_pos.double().unsqueeze(-1) * inv
    return torch.view_as_real(c * torch.complex(torch.cos(a), torch.sin(a))).reshape(z.shape)


def exact(case, seed):
    s = prepare(case, seed)
    m = s["m"]
    root = math.sqrt(m["d_n"] + m["d_r"])
    if case["op"] == "expand":
        L, H = case["length"], case["heads"]
        raw = torch.cat([s["cache"][p] for p in s["table"].tolist()])[:L]
        c, k = _exact_rows(case, m, raw, s["scale"])
        K = torch.stack([c @ s["W_UK"][:, h * m["d_n"]: (h + 1) * m["d_n"]].double() for h in range(H)])
        V = torch.stack([c @ s["W_UV"][:, h * m["d_v"]: (h + 1) * m["d_v"]].double() for h in range(H)])
        return K, V, k
    if case["op"] == "attend":
        B, q, H, L = case["batch"], case["q_len"], case["heads"], case["length"]
        t = torch.arange(q, device="cuda").repeat(B)
        pos = L + s["lens"].long().repeat_interleave(q) - q + t
        u, lse = [], []
        for h in range(H):
            qn = s["q_nope"][:, :, h].double().reshape(B * q, -1)
            qr = _exact_turn(s["q_pe"][:, :, h].reshape(B * q, -1), pos, m)
            z = (qn @ s["keys"][h].double().T + qr @ s["k_pe"].double().T) / root
            l = torch.logsumexp(z, 1)
            u.append(torch.exp(z - l[:, None]) @ s["values"][h].double())
            lse.append(l)
        return torch.stack(u, 1).reshape(B, q, H, -1), torch.stack(lse, 1).reshape(B, q, H)
    if case["op"] == "project":
        R, H = case["rows"], case["heads"]
        top = torch.maximum(s["lse"], s["lse_prefix"]).double()
        ea, eb = torch.exp(s["lse"].double() - top), torch.exp(s["lse_prefix"].double() - top)
        out = torch.zeros((R, m["d"]), dtype=torch.float64, device="cuda")
        for h in range(H):
            v = slice(h * m["d_v"], (h + 1) * m["d_v"])
            own_u = s["o_lat"][:, h].double() @ s["W_UV"][:, v].double()
            u = (ea[:, h, None] * own_u + eb[:, h, None] * s["u_prefix"][:, h].double()) / (ea + eb)[:, h, None]
            out += u @ s["W_O"][v].double()
        return out
    lens = s["lens"].tolist()
    if case["op"] == "weigh":
        out, q = s["weights"].double().clone(), case["q_len"]
        for b, n in enumerate(lens):
            raw = torch.cat([s["cache"][p] for p in s["table"][b, : _pages(n)].tolist()])[:n]
            x = torch.cat(_exact_rows(case, m, raw, s["scale"]), 1)
            mass = torch.zeros(n, dtype=torch.float64, device="cuda")
            for t in range(q):
                e = n - q + t + 1
                z = x[:e] @ s["q_lat"][b, t].double().T / root
                mass[:e] += torch.exp(z - s["lse"][b, t].double()).sum(1)
            old = out[b, :n].clone()
            old[n - q:] = 0
            out[b, :n] = float(case["decay"]) * old + mass if case["decay"] else mass
        return out
    # the eviction: what is kept and copied has one right answer; the turned keys have values
    B, budget = case["batch"], case["budget"]
    kept = torch.full((B, budget), -1, dtype=torch.int32)
    pool = s["cache"].reshape(-1, s["cache"].shape[-1]).clone()
    D0 = m["d_c"] + (m["d_c"] // 32 if case["cache"] == "fp8_e4m3_b128" else 0)
    weights = s["weights"].cpu().numpy()
    old_table, new_table = s["table"].cpu().tolist(), s["new_table"].cpu().tolist()
    new_w = s["new_weights"].double()
    rows_from, rows_to, shift = [], [], []
    for b, n in enumerate(lens):
        if n <= budget:
            keep = list(range(n))
        else:
            inner = range(case["sinks"], n - case["recent"])
            best = sorted(inner, key=lambda j: (-weights[b, j], j))[: budget - case["sinks"] - case["recent"]]
            keep = list(range(case["sinks"])) + sorted(best) + list(range(n - case["recent"], n))
        kept[b, : len(keep)] = torch.tensor(keep, dtype=torch.int32)
        new_w[b, : len(keep)] = s["weights"][b, torch.tensor(keep, device="cuda")].double()
        rows_from += [old_table[b][j // PAGE] * PAGE + j % PAGE for j in keep]
        rows_to += [new_table[b][i // PAGE] * PAGE + i % PAGE for i in range(len(keep))]
        shift += [i - j for i, j in enumerate(keep)]
    src, dst = torch.tensor(rows_from, device="cuda"), torch.tensor(rows_to, device="cuda")
    new_lens = torch.tensor([min(n, budget) for n in lens], dtype=torch.int32)
    raw = pool[src]
    _, k = _exact_rows(case, m, raw, s["scale"])
    k = _exact_turn(k, torch.tensor(shift, device="cuda"), m)
    if case["cache"] in ("f32", "bf16"):
        wide = pool.double()
        wide[dst] = torch.cat([raw[:, :D0].double(), k], 1)
        return kept, new_lens, new_w, wide.view(s["cache"].shape)
    pool[dst] = raw
    shape = (s["cache"].shape[0], PAGE, -1)
    if case["cache"] == "fp8_e4m3":
        wide = pool.view(torch.float8_e4m3fn).to(torch.float32).double()
        scale = float(torch.tensor(s["scale"], dtype=torch.float32))
        wide[dst, D0:] = (k / scale).clamp(-448, 448)
        return kept, new_lens, new_w, wide.view(shape)
    keys = pool[:, D0:].contiguous().view(torch.bfloat16).double()
    keys[dst] = k
    return kept, new_lens, new_w, [
        pool[:, : m["d_c"]].contiguous().view(torch.float8_e4m3fn).to(torch.float32).double().view(shape),
        pool[:, m["d_c"]: D0].contiguous().view(torch.float32).double().view(shape), keys.view(shape)]
