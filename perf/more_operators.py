"""Cases and plain forms of the operators that cut what a decode step reads.

Two sets, for the two streams of a step:

* the cache: a summary of each 64-token page (``keys``), the attention that a query's heads would
  pay to each page by those summaries (``score``), the pages that a query keeps (``select``) and the
  attention over their tokens alone (``attend``);
* the weights: 4-bit codes with a power of two for every 32 elements of the summed dimension, and
  back (``quantise``), and the product with them (``project``).

``own`` selects the framework's calls; otherwise ``run`` computes the same in elementary torch
operations in fp32, rounded once to the output's type.
"""
import math

import torch

own = False

PAGE = 64
# heads' model width, latent width, rotary width, content width and value width per head
V2 = dict(d=5120, d_c=512, d_r=64, d_n=128, d_v=128)
TINY = dict(d=256, d_c=64, d_r=16, d_n=32, d_v=32)
DIMS = {"v2": V2, "tiny": TINY}


def listed():
    return [
        # summaries of freshly cached prompts, every page of every request
        dict(name="keys_prompt_b32_4096", op="keys", dims="v2", batch=32, shortest=4096, longest=4096,
             cache="bf16", new=4096),
        # one speculative step of a large ragged batch: the pages that got two new tokens
        dict(name="keys_step_b256", op="keys", dims="v2", batch=256, shortest=512, longest=8192,
             cache="fp8_e4m3_b128", new=2),
        # a decode step's page scores at the ordinary serving size
        dict(name="score_b32_32768", op="score", dims="v2", heads=128, batch=32, q_len=1, shortest=32768,
             longest=32768),
        # few long contexts, two query tokens each
        dict(name="score_b4_long_q2", op="score", dims="v2", heads=128, batch=4, q_len=2, shortest=32768,
             longest=131072),
        # 64 of 512 pages for every request of a decode step
        dict(name="select_b32_512", op="select", dims="v2", batch=32, q_len=1, shortest=32768, longest=32768,
             budget=64, sinks=1, recent=2),
        # a large ragged batch with long contexts
        dict(name="select_b128_2048", op="select", dims="v2", batch=128, q_len=2, shortest=4096, longest=131072,
             budget=128, sinks=1, recent=4),
        # a decode step over 64 pages of each of 32 long requests
        dict(name="attend_b32_64", op="attend", dims="v2", heads=128, batch=32, q_len=1, shortest=32768,
             longest=32768, cache="bf16", budget=64),
        # a ragged speculative batch on a per-tensor fp8 cache, some requests shorter than the budget
        dict(name="attend_b64_q2_fp8", op="attend", dims="v2", heads=128, batch=64, q_len=2, shortest=1000,
             longest=16384, cache="fp8_e4m3", budget=96),
        # the smallest call: one weight of the tiny fp32 shape
        dict(name="quantise_tiny_f32", op="quantise", act="f32", K=1024, N=256),
        # the folded output projection's weights, once at load
        dict(name="quantise_folded", op="quantise", act="bf16", K=65536, N=5120),
        # the folded output projection of a decode step
        dict(name="project_32_folded", op="project", act="bf16", K=65536, N=5120, rows=32),
        # the unfolded one for a large speculative batch (256 requests x 2 tokens)
        dict(name="project_512", op="project", act="bf16", K=16384, N=5120, rows=512),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


# the weights of the attention block: folded and plain output, queries, latent and rotary key
WEIGHTS = [(65536, 5120), (16384, 5120), (16384, 5120), (5120, 1536), (1536, 16384), (5120, 8192), (5120, 576)]


def draw(rng):
    op = rng.choice(["keys", "score", "score", "select", "attend", "attend", "quantise", "project", "project"])
    tiny = rng.random() < 0.15
    dims = "tiny" if tiny else "v2"
    heads = 16 if tiny else rng.choice([16, 32, 64, 128, 128])
    cache = "f32" if tiny else rng.choice(["bf16", "bf16", "fp8_e4m3", "fp8_e4m3_b128"])
    if op == "keys":
        batch = _log(rng, 1, 128)
        longest = _log(rng, 8, 4096 if tiny else min(65536, 131072 // batch))
        shortest = rng.randint(1, longest)
        return dict(op=op, dims=dims, batch=batch, shortest=shortest, longest=longest, cache=cache,
                    new=rng.choice([1, 1, 2, rng.randint(1, shortest), longest]))
    if op in ("score", "select"):
        q_len = rng.choice([1, 1, 1, 2, 4])
        batch = _log(rng, 1, 32 // q_len if op == "score" else 128)
        longest = _log(rng, 64, 4096 if tiny else min(131072, (1 << 20) // (batch * q_len)))
        c = dict(op=op, dims=dims, batch=batch, q_len=q_len, shortest=rng.randint(q_len, longest),
                 longest=longest)
        if op == "score":
            return dict(c, heads=heads)
        budget = _log(rng, 1, max(1, longest // PAGE))
        recent = rng.randint(1, max(1, budget // 4))
        return dict(c, budget=budget, sinks=rng.randint(0, min(4, budget - recent)), recent=recent)
    if op == "attend":
        q_len = rng.choice([1, 1, 1, 2, 4])
        batch = _log(rng, 1, 64 // q_len)
        budget = _log(rng, 1, 16 if tiny else min(128, 8192 // (batch * q_len)))
        longest = _log(rng, 64, 4096 if tiny else 32768)
        # (the tensor-core kernel of the decode has 128 heads; the others are for small sizes)
        return dict(op=op, dims=dims, heads=16 if tiny else 128, batch=batch, q_len=q_len,
                    shortest=rng.randint(q_len, longest), longest=longest, cache=cache, budget=budget)
    if tiny or rng.random() < 0.3:
        K, N = 32 * _log(rng, 1, 128), _log(rng, 1, 2048)
        act = rng.choice(["f32", "bf16"])
        rows = _log(rng, 1, 64)
    else:
        (K, N), act, rows = rng.choice(WEIGHTS), "bf16", _log(rng, 1, 512)
        if K == 65536:
            rows = min(rows, 128)
    c = dict(op=op, act=act, K=K, N=N)
    return c if op == "quantise" else dict(c, rows=rows)


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _dtype(case):
    if "act" in case:
        return torch.float32 if case["act"] == "f32" else torch.bfloat16
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


def _tables(g, lens, width):
    """A block table [batch][width] over one shuffled pool, and the pool's size. Entries behind a
    request's last page are -1."""
    counts = -(-lens.long() // PAGE)
    total = int(counts.sum())
    perm = torch.randperm(total + 3, generator=g, device="cuda")[:total]
    at = torch.arange(width, device="cuda")[None, :]
    first = torch.cumsum(counts, 0) - counts
    table = torch.where(at < counts[:, None], perm[torch.clamp(first[:, None] + at, max=max(total - 1, 0))], -1)
    return table.to(torch.int32).contiguous(), total + 3


def _cache(case, g, num_pages, m):
    """A filled cache pool [num_pages][64][row] and its per-tensor scale: N(0, 1) latents and
    rotary keys in the cache's own format."""
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


def _config(case, scale=1.0):
    import mla_latent_kv_04_gb300 as M

    m = DIMS[case.get("dims", "v2")]

    class Dims:
        num_heads, d_model, d_latent = case.get("heads", 128), m["d"], m["d_c"]
        d_rope, d_nope, d_v, page_size = m["d_r"], m["d_n"], m["d_v"], PAGE
    act = "f32" if _dtype(case) == torch.float32 else "bf16"
    return M, M.make_config(Dims, act, case.get("cache", act), cache_scale=scale)


def _visible(case, lens):
    """Pages that query token t of request b sees, [batch][q_len]."""
    t = torch.arange(case["q_len"], device="cuda")
    return (lens.long()[:, None] - case["q_len"] + t) // PAGE + 1


def prepare(case, seed):
    g, act, op = _gen(seed), _dtype(case), case["op"]
    s = dict(case=case, scale=1.0)
    if op in ("quantise", "project"):
        K, N = case["K"], case["N"]
        W = _normal(g, (K, N), act, K ** -0.5)
        nt, kt = -(-N // 128), -(-K // 128)
        if op == "quantise":
            s["W"] = W
            s["codes"] = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty((nt, kt, 32, 4, 4), dtype=torch.uint8, device="cuda")
            s["back"] = torch.empty_like(W)
        else:
            code, e = _codes(W.float())
            del W
            code = code.t().contiguous()                       # [N][K]
            s["codes"] = code[:, 0::2] | (code[:, 1::2] << 4)
            byte = torch.full((nt * 128, kt * 4), 127, dtype=torch.uint8, device="cuda")
            byte[:N, : K // 32] = (e + 127).to(torch.uint8).t()
            # [row tile][4][32][column group][4] -> [row tile][column group][32][4][4]
            s["scales"] = byte.view(nt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous()
            s["x"] = _normal(g, (case["rows"], K), act, 0.05)
            s["out"] = torch.empty((case["rows"], N), dtype=act, device="cuda")
        if own:
            M, s["cfg"] = _config(case)
            need = M.mla_mx4_project_workspace_size(s["cfg"], K, N, case["rows"]) if op == "project" else 0
            s["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        return s
    m = s["m"] = DIMS[case["dims"]]
    D, B = m["d_c"] + m["d_r"], case["batch"]
    s["lens"] = _lengths(case, g)
    width = _pages(case["longest"])
    if op == "select":
        # attention mass of pages: a heavy tail, and one page in ten that got exactly none
        sc = torch.exp(2.0 * torch.randn((B, case["q_len"], width), generator=g, device="cuda"))
        s["scores"] = sc * (torch.rand(sc.shape, generator=g, device="cuda") > 0.1)
        s["pages"] = torch.empty((B, case["q_len"], case["budget"]), dtype=torch.int32, device="cuda")
    else:
        s["table"], n = _tables(g, s["lens"], width)
    if op in ("keys", "attend"):
        s["cache"], s["scale"] = _cache(case, g, n, m)
    if op == "keys":
        s["keys"] = _normal(g, (n, D), act)
    if op in ("score", "attend"):
        q = case["q_len"]
        s["q_lat"] = _normal(g, (B, q, case["heads"], D), act, 0.6)
    if op == "score":
        s["keys"] = _normal(g, (n, D), act, 0.4)
        s["scores"] = torch.zeros((B, q, width), device="cuda")
    if op == "attend":
        # the first page, the query's own and a random choice between them, ascending
        seen = _visible(case, s["lens"])
        at = torch.arange(max(width, case["budget"]), device="cuda")
        r = torch.rand((B, q, at.numel()), generator=g, device="cuda")
        r = torch.where((at == 0) | (at == seen[..., None] - 1), 2.0 + at, r)
        r = torch.where(at < seen[..., None], r, -1.0)
        best = r.sort(-1, descending=True).indices[..., : case["budget"]]
        keep = torch.arange(best.shape[-1], device="cuda") < seen[..., None]
        best = torch.where(keep, best, 1 << 30).sort(-1).values
        s["pages"] = torch.where(best < (1 << 30), best, -1).to(torch.int32).contiguous()
        s["out"] = torch.empty((B, q, case["heads"], m["d_c"]), dtype=act, device="cuda")
        s["lse"] = torch.empty((B, q, case["heads"]), dtype=torch.float32, device="cuda")
    if own:
        M, s["cfg"] = _config(case, s["scale"])
        need = 0
        if op == "score":
            need = M.mla_page_scores_workspace_size(s["cfg"], B, q, width)
        elif op == "attend":
            need = M.mla_decode_pages_workspace_size(s["cfg"], B, q, s["pages"].shape[2])
        s["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _codes(W):
    """4-bit codes [K][N] (bit 3 the sign) and exponents [K / 32][N] of fp32 weights: the exponent is
    that of the block's largest magnitude, rounded to two significant bits, less 2."""
    K, N = W.shape
    b = W.view(K // 32, 32, N)
    top = b.abs().amax(1)
    e = (((top.view(torch.int32) + (1 << 21)) >> 23) - 129).clamp(-127, 125)
    y = (b.abs() * torch.exp2(-e.float())[:, None]).view(K, N)
    code = torch.zeros((K, N), dtype=torch.uint8, device=W.device)
    for edge, even in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                       (5.0, False)):
        code += (y >= edge) if even else (y > edge)      # half-way values go to the even code
    return code | (torch.signbit(W).to(torch.uint8) << 3), e


def _weights(code, e, dtype=torch.float32):
    """Values of codes [K][N] under exponents [K / 32][N]."""
    g = torch.tensor(GRID + tuple(-v for v in GRID), dtype=dtype, device=code.device)
    v = g[code.int()].view(e.shape[0], 32, -1)
    return (v * torch.exp2(e.to(dtype))[:, None]).view(code.shape)


def _unpack(s):
    """Codes [K][N] and exponents [K / 32][N] of packed weights."""
    K, N = s["case"]["K"], s["case"]["N"]
    code = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).view(N, K).t()
    nt, kt = s["scales"].shape[:2]
    byte = s["scales"].permute(0, 3, 2, 1, 4).reshape(nt * 128, kt * 4)
    return code, byte[:N, : K // 32].t().int() - 127


def _plain_quantise(s):
    return _weights(*_codes(s["W"].float())).to(s["W"].dtype)


def _plain_project(s):
    return (s["x"].float() @ _weights(*_unpack(s))).to(s["x"].dtype)


def _rows(raw, kind, m, scale):
    """The values of raw cache rows [...][row], in fp32."""
    if kind in ("f32", "bf16"):
        return raw.float()
    if kind == "fp8_e4m3":
        return raw.view(torch.float8_e4m3fn).float() * scale
    c, n = m["d_c"], m["d_c"] // 128
    codes = raw[..., :c].contiguous().view(torch.float8_e4m3fn).float()
    s = raw[..., c: c + 4 * n].contiguous().view(torch.float32)
    x = (codes.unflatten(-1, (n, 128)) * s[..., None]).flatten(-2)
    return torch.cat([x, raw[..., c + 4 * n:].contiguous().view(torch.bfloat16).float()], -1)


def _plain_keys(s):
    case, lens = s["case"], s["lens"].long()
    first = (lens - case["new"]).clamp(min=0) // PAGE
    at = torch.arange(s["table"].shape[1], device="cuda")
    b, p = torch.nonzero((at >= first[:, None]) & (at * PAGE < lens[:, None]), as_tuple=True)
    page = s["table"].long()[b, p]
    n = (lens[b] - p * PAGE).clamp(max=PAGE)
    x = _rows(s["cache"][page], case["cache"], s["m"], s["scale"])
    x = torch.where((torch.arange(PAGE, device="cuda") < n[:, None])[..., None], x, 0.0)
    s["keys"][page] = (x.sum(1) / n[:, None]).to(s["keys"].dtype)
    return s["keys"]


def _plain_score(s):
    case, m, lens = s["case"], s["m"], s["lens"].long()
    B, q, H = case["batch"], case["q_len"], case["heads"]
    k = s["keys"].float()[s["table"].long().clamp(min=0)]                    # [B][pages][D]
    z = s["q_lat"].float().reshape(B, q * H, -1) @ k.transpose(1, 2) * (m["d_n"] + m["d_r"]) ** -0.5
    z = z.view(B, q, H, -1)
    see = lens[:, None] - q + torch.arange(q, device="cuda") + 1             # tokens that (b, t) sees
    at = torch.arange(z.shape[-1], device="cuda")
    count = (see[..., None] - at * PAGE).clamp(0, PAGE).float()              # [B][q][pages]
    z = torch.where(count[:, :, None] > 0, z, -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True)) * count[:, :, None]
    mass = (e / e.sum(-1, keepdim=True)).sum(2)
    s["scores"].copy_(torch.where(count > 0, mass, s["scores"]))
    return s["scores"]


def _plain_select(s):
    case = s["case"]
    seen, w = _visible(case, s["lens"])[..., None], s["scores"].shape[-1]
    budget = case["budget"]
    at = torch.arange(w, device="cuda")
    live = at < seen
    sure = live & ((at < case["sinks"]) | (at >= seen - case["recent"]) | (seen <= budget))
    key = torch.where(sure, math.inf, torch.where(live, s["scores"], -math.inf))
    first = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    kept = torch.arange(first.shape[-1], device="cuda") < seen
    first = torch.where(kept, first, w).sort(-1).values
    s["pages"].fill_(-1)
    s["pages"][..., : first.shape[-1]] = torch.where(first < w, first, -1).to(torch.int32)
    return s["pages"]


def _plain_attend(s):
    case, m, lens = s["case"], s["m"], s["lens"].long()
    B, q, H, n = case["batch"], case["q_len"], case["heads"], s["pages"].shape[2]
    pages = s["pages"].long()
    ids = torch.gather(s["table"].long()[:, None].expand(B, q, -1), 2, pages.clamp(min=0))
    see = lens[:, None] - q + torch.arange(q, device="cuda") + 1
    pos = pages[..., None] * PAGE + torch.arange(PAGE, device="cuda")
    live = ((pages[..., None] >= 0) & (pos < see[..., None, None])).view(B, q, n * PAGE)
    out, lse = [], []
    for b in range(B):                                                       # (a request's rows at a time)
        x = _rows(s["cache"][ids[b]], case["cache"], m, s["scale"]).flatten(1, 2)    # [q][n * 64][D]
        x = torch.where(live[b, ..., None], x, 0.0)
        z = s["q_lat"][b].float() @ x.transpose(1, 2) * (m["d_n"] + m["d_r"]) ** -0.5
        z = torch.where(live[b, :, None], z, -math.inf)
        top = z.amax(-1, keepdim=True)
        p = torch.exp(z - top)
        total = p.sum(-1, keepdim=True)
        out.append(p @ x[..., : m["d_c"]] / total)
        lse.append((top + torch.log(total))[..., 0])
    return torch.stack(out).to(s["q_lat"].dtype), torch.stack(lse)


PLAIN = {"keys": _plain_keys, "score": _plain_score, "select": _plain_select, "attend": _plain_attend,
         "quantise": _plain_quantise, "project": _plain_project}


# ------------------------------------------------------------------------------- one pass

def _own(s):
    import mla_latent_kv_04_gb300 as M

    c, cfg = s["case"], s["cfg"]
    if c["op"] == "keys":
        M.mla_page_keys(cfg, s["cache"], s["table"], s["lens"], s["keys"], new_tokens=c["new"])
        return s["keys"]
    if c["op"] == "score":
        M.mla_page_scores(cfg, s["q_lat"], s["keys"], s["table"], s["lens"], s["scores"], s["ws"])
        return s["scores"]
    if c["op"] == "select":
        M.mla_select_pages(cfg, s["scores"], s["lens"], s["pages"], sinks=c["sinks"], recent=c["recent"])
        return s["pages"]
    if c["op"] == "attend":
        M.mla_decode_pages(cfg, s["q_lat"], s["cache"], s["table"], s["lens"], s["pages"], s["out"], s["lse"],
                           s["ws"])
        return s["out"], s["lse"]
    if c["op"] == "quantise":
        M.mla_mx4_quantize(cfg, s["W"], s["codes"], s["scales"])
        M.mla_mx4_dequantize(cfg, s["codes"], s["scales"], s["back"])
        return s["back"]
    M.mla_mx4_project(cfg, s["x"], s["codes"], s["scales"], s["out"], s["ws"])
    return s["out"]


def run(s):
    return _own(s) if own else PLAIN[s["case"]["op"]](s)


# ------------------------------------------------------------------------------- work

def _row_bytes(kind, m):
    size = {"f32": 4, "bf16": 2, "fp8_e4m3": 1}
    if kind in size:
        return (m["d_c"] + m["d_r"]) * size[kind]
    return m["d_c"] + m["d_c"] // 32 + 2 * m["d_r"]


def work(case):
    a = 4 if _dtype(case) == torch.float32 else 2
    op = case["op"]
    if op in ("quantise", "project"):
        K, N = case["K"], case["N"]
        packed = N * (K // 2) + N * (K // 32)
        if op == "quantise":
            return {"bytes": packed + 2 * a * K * N, "flops": 2 * K * N}
        R = case["rows"]
        return {"bytes": packed + a * R * (K + N), "flops": 2 * R * K * N}
    m, lens = DIMS[case["dims"]], _spread(case)
    D = m["d_c"] + m["d_r"]
    if op == "keys":
        rows = sum(n - max(0, n - case["new"]) // PAGE * PAGE for n in lens)
        pages = sum(_pages(n) - max(0, n - case["new"]) // PAGE for n in lens)
        return {"bytes": rows * _row_bytes(case["cache"], m) + a * pages * D, "flops": rows * D}
    q = case["q_len"]
    if op == "attend":
        rows, read, budget = 0, 0.0, case["budget"]
        for n in lens:
            for t in range(q):
                see = n - q + t + 1
                seen = _pages(see)
                rows += see if seen <= budget else (budget - 1) * PAGE + see - (seen - 1) * PAGE
            # a page on the lists of several query tokens of a request has to be read once: the
            # expected union of the random lists (first and last page on all of them)
            seen = _pages(n)
            if seen <= budget:
                read += n
            else:
                share = max(0, budget - 2) / (seen - 2) if seen > 2 else 0.0
                read += (min(budget, 2) - 1) * PAGE + n - (seen - 1) * PAGE + (seen - 2) * (1 - (1 - share) ** q) * PAGE
        H = case["heads"]
        return {"bytes": int(read) * _row_bytes(case["cache"], m) + case["batch"] * q * H * (a * (D + m["d_c"]) + 4),
                "flops": 2 * rows * H * (D + m["d_c"])}
    seen = sum(_pages(n - q + t + 1) for n in lens for t in range(q))
    if op == "score":
        H, most = case["heads"], sum(_pages(n) for n in lens)
        return {"bytes": a * D * (most + case["batch"] * q * H) + 4 * seen, "flops": 2 * seen * H * D}
    return {"bytes": 4 * seen + 4 * case["batch"] * q * case["budget"], "flops": seen}


# ------------------------------------------------------------------------------- 64 bits

def _exact_rows(case, m, raw, scale):
    """The values of raw rows [n][row], in fp64."""
    kind, dc = case["cache"], m["d_c"]
    if kind in ("f32", "bf16"):
        return raw.double()
    if kind == "fp8_e4m3":
        # the scale as the library holds it: fp32
        held = float(torch.tensor(scale, dtype=torch.float32))
        return raw.contiguous().view(torch.float8_e4m3fn).to(torch.float32).double() * held
    c = raw[:, :dc].contiguous().view(torch.float8_e4m3fn).to(torch.float32).double()
    sc = raw[:, dc: dc + dc // 32].contiguous().view(torch.float32).double()
    return torch.cat([c * sc.repeat_interleave(128, 1),
                      raw[:, dc + dc // 32:].contiguous().view(torch.bfloat16).double()], 1)


def _nearest(y):
    """|y| in [0, 8) to the nearest of GRID in fp64; half-way values to the neighbour of even index."""
    unit = torch.where(y < 2.0, 0.5, torch.where(y < 4.0, 1.0, 2.0))
    return (torch.round(y / unit) * unit).clamp(max=6.0)     # (round: half to even)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        K, N = case["K"], case["N"]
        out = torch.empty((K, N), device="cuda")             # (fp32 holds every such value)
        for k in range(0, K, 32):
            w = s["W"][k: k + 32].double()
            top = w.abs().amax(0)
            frac, ex = torch.frexp(top)                      # top = frac 2^ex, frac in [1/2, 1)
            e = ex - 1 - 2 + (frac >= 0.875).int()           # two significant bits: 0.875 rounds up to 1
            unit = torch.exp2(torch.where(top > 0, e, 0).double().clamp(-127, 125))
            out[k: k + 32] = torch.copysign(_nearest(w.abs() / unit) * unit, w)
        return out
    if op == "project":
        K, N = case["K"], case["N"]
        grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device="cuda")
        out = torch.empty((case["rows"], N), dtype=torch.float64, device="cuda")
        x = s["x"].double()
        for n0 in range(0, N, 128):
            c = s["codes"][n0: n0 + 128]
            r = c.shape[0]
            w = torch.empty((r, K), dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = grid[(c & 15).long()], grid[(c >> 4).long()]
            sc = torch.stack([s["scales"][n0 // 128, :, i % 32, i // 32].reshape(-1)[: K // 32] for i in range(r)])
            w = w.view(r, -1, 32) * torch.exp2(sc.double() - 127.0)[..., None]
            out[:, n0: n0 + r] = x @ w.view(r, K).T
        return out
    m, B = s["m"], case["batch"]
    lens, root = s["lens"].tolist(), math.sqrt(m["d_n"] + m["d_r"])
    if op == "keys":
        out = s["keys"].double()
        for b, n in enumerate(lens):
            p0 = max(0, n - case["new"]) // PAGE
            ids = s["table"][b, p0: _pages(n)].long()
            x = _exact_rows(case, m, s["cache"][ids].flatten(0, 1), s["scale"]).view(len(ids), PAGE, -1)
            out[ids] = x.mean(1)
            last = n - (_pages(n) - 1) * PAGE
            out[ids[-1]] = x[-1, :last].mean(0)
        return out
    q = case["q_len"]
    if op == "select":
        scores = s["scores"].cpu().numpy()
        pages = torch.full((B, q, case["budget"]), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            for t in range(q):
                seen = _pages(n - q + t + 1)
                keep = list(range(seen))
                if seen > case["budget"]:
                    inner = range(case["sinks"], seen - case["recent"])
                    best = sorted(inner, key=lambda p: (-scores[b, t, p], p))
                    best = best[: case["budget"] - case["sinks"] - case["recent"]]
                    keep = sorted(list(range(case["sinks"])) + best + list(range(seen - case["recent"], seen)))
                pages[b, t, : len(keep)] = torch.tensor(keep, dtype=torch.int32)
        return pages
    if op == "score":
        out = s["scores"].double()
        for b, n in enumerate(lens):
            k = s["keys"][s["table"][b, : _pages(n)].long()].double()
            for t in range(q):
                see = n - q + t + 1
                seen = _pages(see)
                count = torch.full((seen,), float(PAGE), dtype=torch.float64, device="cuda")
                count[-1] = see - (seen - 1) * PAGE
                z = s["q_lat"][b, t].double() @ k[:seen].T / root + torch.log(count)
                out[b, t, :seen] = torch.softmax(z, 1).sum(0)
        return out
    out = torch.empty((B, q, case["heads"], m["d_c"]), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, q, case["heads"]), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        for t in range(q):
            see = n - q + t + 1
            keep = [p for p in s["pages"][b, t].tolist() if p >= 0]
            ids = s["table"][b, torch.tensor(keep, device="cuda")].long()
            x = _exact_rows(case, m, s["cache"][ids].flatten(0, 1), s["scale"])
            pos = (torch.tensor(keep, device="cuda")[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()
            x = x[pos < see]
            z = s["q_lat"][b, t].double() @ x.T / root
            lse[b, t] = torch.logsumexp(z, 1)
            out[b, t] = torch.softmax(z, 1) @ x[:, : m["d_c"]]
    return out, lse
