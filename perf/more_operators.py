"""Cases of the paged KV cache: norms, rotation and the writing of new keys and values into their pages,
attention of any number of new rows per request over the pages, and the commit that keeps or drops rows.

The sizes are those of this repository's workloads (synth/configs.py and the cases beside this file):
16 query heads on 4 KV heads of 256 bf16 (and 4 on 2 of 64 fp32), 1..8 verify rows per request, 1..32
requests, contexts of 15,360 and 63,488 positions, prompts in chunks; pages of 16 to 256 positions.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
# Rows: either B requests of R rows each (a verify pass; ragged: of which a request runs 1..R) or `lens`
# rows of each request (prompts and chunks of prompts, single tokens among them). past: positions in the
# cache before them (ragged or lens: different ones for each request). page: positions a page. prefix:
# positions of a shared prefix outside the pages, which the rotation counts.
def listed():
    wide = dict(q_heads=16, kv_heads=4, dim=256, dtype="bf16")
    small = dict(q_heads=4, kv_heads=2, dim=64, dtype="f32", page=16)
    return [
        # one small fp32 request's two verify rows, the whole head rotated, no norms: launch latency
        dict(small, name="append_tiny_f32_1x2", op="append", B=1, R=2, ragged=False, past=256,
             prefix=0, rot=64, pairs="half", norm=False, scaled=False),
        # a verify pass of 32 requests at mixed widths after a shared prompt, a quarter of each head
        # rotated, with norms
        dict(wide, name="append_verify_32x8", op="append", B=32, R=8, ragged=True, past=700,
             prefix=15360, page=64, rot=64, pairs="half", norm=True, scaled=False),
        # prompts of very different lengths in one call (empty, one token, odd ones), pairs side by side
        dict(name="append_ragged", op="append", lens="0,1,77,1000,2311", past=500, prefix=0,
             q_heads=16, kv_heads=8, dim=128, dtype="bf16", page=16, rot=128, pairs="interleaved",
             norm=True, scaled=False),
        # a long prompt's 15K tokens at once, frequencies scaled for a long context: most bytes
        dict(wide, name="append_prompt_15360", op="append", lens="15360", past=0, prefix=0, page=128,
             rot=64, pairs="half", norm=True, scaled=True),
        # greedy decoding of one small fp32 request: one draft of one kept
        dict(small, name="commit_tiny_f32_1x2", op="commit", B=1, R=2, ragged=False, past=256, layers=1),
        # 32 requests at mixed widths, twelve attention layers
        dict(wide, name="commit_32x8", op="commit", B=32, R=8, ragged=True, past=200, page=64, layers=12),
        # two rows of one small fp32 request: launch latency
        dict(small, name="attn_tiny_f32_1x2", op="attn", B=1, R=2, ragged=False, past=256),
        # greedy decoding of one long request (2 verify rows)
        dict(wide, name="attn_1x2_63488", op="attn", B=1, R=2, ragged=False, past=63488, page=64),
        # 32 requests at mixed widths, each with its own 15K or less: most bytes
        dict(wide, name="attn_verify_32x8_15360", op="attn", B=32, R=8, ragged=True, past=15360, page=64),
        # prompts of very different lengths from their start, and one token, in one call
        dict(name="attn_ragged", op="attn", lens="0,1,77,1000,2311", past=500, q_heads=16, kv_heads=8,
             dim=128, dtype="bf16", page=16),
        # a chunk of a prompt beside 31 requests that decode single tokens
        dict(wide, name="attn_chunk_beside_tokens", op="attn", lens="1000" + ",1" * 31, past=4000,
             page=128),
        # the last chunk of a 63K prompt: the most arithmetic
        dict(wide, name="attn_chunk_2048_over_61440", op="attn", lens="2048", past=61440, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "commit", "attn", "attn", "attn"])
    dim = rng.choice([64, 128, 256, 256])
    kv_heads = rng.choice([1, 2, 4, 8]) if dim < 256 else rng.choice([1, 2, 4])
    group = rng.choice([1, 2, 4, 6]) if kv_heads < 4 else rng.choice([1, 2, 4])
    case = dict(op=op, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                dtype="bf16" if rng.random() < 0.85 else "f32", page=rng.choice([16, 32, 64, 128, 256]))
    if op == "commit":
        case.update(B=_log_int(rng, 1, 32), R=rng.randint(1, 8), ragged=rng.random() < 0.5,
                    past=_log_int(rng, 1, 300), layers=rng.randint(1, 12))
        return case
    if op == "append":
        case.update(rot=rng.choice([dim, dim, dim // 2, dim // 4, 0]),
                    pairs=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.6,
                    scaled=rng.random() < 0.3, prefix=rng.choice([0, 0, _log_int(rng, 1, 60000)]))
    if rng.random() < 0.5:
        B = _log_int(rng, 1, 32)
        past = _log_int(rng, 1, 900 if op == "append" else 60000 if B == 1 else 15000)
        case.update(B=B, R=rng.randint(1, 8), ragged=rng.random() < 0.5, past=past)
    else:
        n = rng.choice([1, 1, 2, 3, 5])
        lens = [_log_int(rng, 1, (8000 if op == "append" else 4000) // n) for _ in range(n)]
        if n > 2 and rng.random() < 0.5:
            lens[rng.randrange(n)] = 0
        case.update(lens=",".join(str(x) for x in lens), past=rng.choice([0, _log_int(rng, 1, 12000)]))
    if op == "attn" and case["dtype"] == "f32":  # fp32 caches are small ones
        case["past"] = min(case["past"], 20000 // len(_own_of(case)))
    return case


def _own_of(case):
    """Rows of the call that each request owns."""
    if "lens" in case:
        return [int(x) for x in case["lens"].split(",")]
    return [case["R"]] * case["B"]


def _rows_of(case):
    """Rows that each request runs: all it owns, or a spread over 1..R."""
    if "lens" in case or not case["ragged"]:
        return _own_of(case)
    return [1 + (5 * b + 3) % case["R"] for b in range(case["B"])]


def _past_of(case):
    """Positions in the cache before the call's rows."""
    n, past = len(_own_of(case)), case["past"]
    if "lens" in case or case["ragged"]:
        return [past - (37 * b) % (past // 2 + 1) for b in range(n)]
    return [past] * n


def _kept_of(case):
    """Of a commit: the rows each request keeps, 1..rows."""
    return [1 + (3 * b + 1) % n for b, n in enumerate(_rows_of(case))]


def _elem(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    e, Hq, Hkv, D = _elem(case), case["q_heads"], case["kv_heads"], case["dim"]
    rows, past = _rows_of(case), _past_of(case)
    if case["op"] == "append":
        T = sum(rows)
        return dict(bytes=2 * T * (Hq + 2 * Hkv) * D * e,
                    flops=T * (Hq + Hkv) * (3 * D * case["norm"] + 3 * case["rot"]))
    if case["op"] == "commit":
        gone = sum(n - m for n, m in zip(rows, _kept_of(case)))
        return dict(bytes=gone * case["layers"] * 2 * Hkv * D * e + 84 * len(rows), flops=0)
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(rows, past))
    kv = sum(p + n for n, p in zip(rows, past) if n)
    return dict(bytes=2 * kv * Hkv * D * e + 2 * sum(rows) * Hq * D * e, flops=4 * pairs * Hq * D)


# ------------------------------------------------------------------------------------- inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def _i64(a):
    return torch.tensor(a, dtype=torch.int64, device=DEV)


def _frequencies(case):
    """[rot / 2] fp32 and the factor on cos and sin. Scaled: slow pairs turn eight times slower, fast
    ones as before, those between in part."""
    half = case["rot"] // 2
    f = 1e6 ** (-np.arange(half) / max(half, 1))
    if not case["scaled"]:
        return f.astype(np.float32), 1.0
    turns = 8192 * f / (2 * math.pi)
    keep = np.clip((turns - 1) / 31, 0, 1)
    return (f * (keep + (1 - keep) / 8)).astype(np.float32), 0.1 * math.log(8) + 1


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    Hq, Hkv, D, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    own_rows, rows, past = _own_of(case), _rows_of(case), _past_of(case)
    B, T, layers = len(rows), sum(own_rows), case.get("layers", 1)

    def rnd(*shape):  # in pieces: a long cache in fp32 at once would be several GB
        out = torch.empty(shape, dtype=_dt(case), device=DEV)
        flat = out.view(-1)
        for i in range(0, flat.numel(), 1 << 26):
            n = min(1 << 26, flat.numel() - i)
            flat[i:i + n] = torch.randn(n, generator=g, device=DEV)
        return out

    # the requests' pages lie in the pool in any order; a table row ends in entries that are not in use
    need = [-(-(p + n) // page) for n, p in zip(own_rows, past)]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max(need) + 2), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s = dict(case=case, table=table, k_pages=rnd(layers, pool, page, Hkv * D),
             v_pages=rnd(layers, pool, page, Hkv * D), past=_i64(past), kv_len=_i64(past),
             cu_rows=_i32(np.concatenate([[0], np.cumsum(own_rows)]).tolist()),
             n_rows=_i32(rows) if rows != own_rows else None)
    if case["op"] == "commit":
        acc = np.zeros((B, 16), dtype=np.int32)   # spec_accept_out: status, n_accept, n_emit, ...
        acc[:, 1], acc[:, 2] = np.array(_kept_of(case)) - 1, _kept_of(case)
        s.update(acc=torch.from_numpy(acc).to(DEV), k=_i32([n - 1 for n in rows]),
                 status=torch.zeros(B, dtype=torch.int32, device=DEV))
    elif case["op"] == "append":
        # q, k and v as column ranges of one row per token, as one projection leaves them
        mixed = rnd(T, (Hq + 2 * Hkv) * D)
        f, factor = _frequencies(case)
        s.update(mixed=mixed, q=mixed[:, :Hq * D], k=mixed[:, Hq * D:(Hq + Hkv) * D],
                 v=mixed[:, (Hq + Hkv) * D:], inv_freq=torch.from_numpy(f).to(DEV), rot_scale=factor,
                 q_out=torch.zeros((T, Hq * D), dtype=_dt(case), device=DEV))
        s["pos"] = s["past"] + case["prefix"] if case["prefix"] else None
        for n in ("q_norm", "k_norm"):
            s[n] = 1 + 0.2 * torch.randn(D, generator=g, device=DEV) if case["norm"] else None
    else:
        # queries a little longer than unit variance: the softmax then has some heavy positions
        s.update(q=(rnd(T, Hq * D).float() * 1.5).to(_dt(case)),
                 out=torch.zeros((T, Hq * D), dtype=_dt(case), device=DEV))
    if own:
        s.update(_handle(s))
    return s


# ------------------------------------------------------------------- the framework's operators
def _handle(s):
    """The cache's description, the operator's description and the workspace a program keeps."""
    import mtp_speculative_decoding_spec_gb300 as spec
    case, e = s["case"], _elem(s["case"])
    c = spec.spec_paged_cache()
    c.dtype = spec.SPEC_BF16 if case["dtype"] == "bf16" else spec.SPEC_F32
    c.layers, c.kv_heads, c.head_dim = s["k_pages"].shape[0], case["kv_heads"], case["dim"]
    c.page_size, c.n_pages = case["page"], s["k_pages"].shape[1]
    c.k_pages, c.v_pages = s["k_pages"].data_ptr(), s["v_pages"].data_ptr()
    c.layer_stride, c.page_stride = s["k_pages"].stride(0) * e, s["k_pages"].stride(1) * e
    c.page_table, c.table_stride = s["table"].data_ptr(), s["table"].stride(0)
    c.max_pages, c.kv_len = s["table"].shape[1], s["kv_len"].data_ptr()
    if case["op"] == "commit":
        return dict(cache=c)
    T = s["q"].shape[0]
    if case["op"] == "append":
        d = spec.spec_append_desc()
        d.q_heads, d.norm_eps = case["q_heads"], EPS
        for n in ("q", "k", "v"):
            setattr(d, n, s[n].data_ptr())
            setattr(d, n + "_stride", s["mixed"].stride(0))
        d.q_out, d.q_out_stride = s["q_out"].data_ptr(), s["q_out"].stride(0)
        if case["norm"]:
            d.q_norm, d.k_norm = s["q_norm"].data_ptr(), s["k_norm"].data_ptr()
        d.rot_dim, d.rot_interleaved = case["rot"], case["pairs"] == "interleaved"
        d.inv_freq, d.rot_scale = s["inv_freq"].data_ptr(), s["rot_scale"]
        if case["prefix"]:
            d.pos = s["pos"].data_ptr()
        return dict(cache=c, desc=d)
    d = spec.spec_paged_attn_desc()
    d.q_heads, d.scale = case["q_heads"], case["dim"] ** -0.5
    d.q, d.q_stride = s["q"].data_ptr(), s["q"].stride(0)
    d.out, d.out_stride = s["out"].data_ptr(), s["out"].stride(0)
    n = spec.spec_paged_attention_workspace_bytes(len(s["past"]), T, c, d)
    return dict(cache=c, desc=d, ws=torch.zeros(max(n, 256), dtype=torch.uint8, device=DEV))


def _run_own(s):
    import mtp_speculative_decoding_spec_gb300 as spec
    case, B = s["case"], s["past"].numel()
    if case["op"] == "commit":
        s["kv_len"].copy_(s["past"])  # so that every pass commits the same cycle
        spec.spec_paged_commit(B, s["cache"], s["acc"], s["k"], s["status"])
        return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], kv_len=s["kv_len"], status=s["status"])
    T = s["q"].shape[0]
    if case["op"] == "append":
        spec.spec_paged_append(B, s["cu_rows"], T, s["cache"], 0, s["desc"], s["n_rows"])
        return dict(q=s["q_out"], k_pages=s["k_pages"], v_pages=s["v_pages"])
    spec.spec_paged_attention(B, s["cu_rows"], T, s["cache"], 0, s["desc"], s["n_rows"], s["ws"])
    return dict(out=s["out"])


def run(s):
    if own:
        return _run_own(s)
    return dict(append=_plain_append, commit=_plain_commit, attn=_plain_attn)[s["case"]["op"]](s)


# ------------------------------------------------------------------------------- plain forms
def _rows(s):
    """Of the rows that run: their number in the call, request and position."""
    r = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.bucketize(r, s["cu_rows"][1:].long(), right=True)
    at = r - s["cu_rows"].long()[b]
    if s["n_rows"] is not None:
        runs = at < s["n_rows"][b]
        r, b, at = r[runs], b[runs], at[runs]
    return r, b, s["past"][b] + at


def _plain_append(s):
    """x w / sqrt(mean(x^2) + eps), its first `rot` dims turned by pos * inv_freq; K and V to their
    pages. Angles are formed in 64 bits: at a position of 60,000 fp32 would be off by 2e-3."""
    case = s["case"]
    D, rot, page = case["dim"], case["rot"], case["page"]
    r, b, pos = _rows(s)
    angle = (pos + case["prefix"])[:, None].double() * s["inv_freq"].double()[None]
    cos, sin = ((t.float() * s["rot_scale"])[:, None] for t in (torch.cos(angle), torch.sin(angle)))

    def turned(x, w):
        x = x[r].float().view(r.numel(), -1, D)
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * w
        y, part = x.clone(), x[..., :rot]
        a, c = (part[..., :rot // 2], part[..., rot // 2:]) if case["pairs"] == "half" else \
            (part[..., 0::2], part[..., 1::2])
        ya, yc = a * cos - c * sin, c * cos + a * sin
        y[..., :rot] = torch.cat([ya, yc], dim=-1) if case["pairs"] == "half" else \
            torch.stack([ya, yc], dim=-1).flatten(-2)
        return y.view(r.numel(), -1).to(_dt(case))

    s["q_out"][r] = turned(s["q"], s["q_norm"])
    at = s["table"][b, pos // page].long()
    s["k_pages"][0][at, pos % page] = turned(s["k"], s["k_norm"])
    s["v_pages"][0][at, pos % page] = s["v"][r]
    return dict(q=s["q_out"], k_pages=s["k_pages"], v_pages=s["v_pages"])


def _plain_commit(s):
    """Rows past the kept ones become zero in every layer, and the lengths the kept rows' more."""
    page = s["case"]["page"]
    keep = s["acc"][:, 2].long()
    r = torch.arange(s["case"]["R"], device=DEV)[None]
    gone = (r >= keep[:, None]) & (r <= s["k"][:, None])
    pos = (s["past"][:, None] + r).clamp(max=s["table"].shape[1] * page - 1)
    at, within = torch.gather(s["table"], 1, pos // page).long(), pos % page
    for pages in (s["k_pages"], s["v_pages"]):
        pages[:, at[gone], within[gone]] = 0
    return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], kv_len=s["past"] + keep,
                status=torch.zeros_like(s["status"]))


def _plain_attn(s):
    """softmax(scale q.k) v over the pages of the request up to the row itself, request by request and KV
    head by KV head; zero where a request does not run a row."""
    case = s["case"]
    Hq, Hkv, D, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    G, scale = Hq // Hkv, D ** -0.5
    out = torch.zeros((s["q"].shape[0], Hkv, G, D), device=DEV)
    q = s["q"].view(-1, Hkv, G, D)
    no = torch.full((), -math.inf, device=DEV)
    first = 0
    for b, (n, most, past) in enumerate(zip(_rows_of(case), _own_of(case), _past_of(case))):
        L = past + n
        at = s["table"][b, :-(-L // page)].long()
        pos = torch.arange(L, device=DEV)
        step = max(1, (1 << 28) // max(1, L * G))  # rows at once: scores of a gigabyte
        for h in range(Hkv if n else 0):
            k, v = (s[x][0].view(-1, page, Hkv, D)[at, :, h].reshape(-1, D)[:L].float()
                    for x in ("k_pages", "v_pages"))
            for i in range(0, n, step):
                rows = torch.arange(i, min(n, i + step), device=DEV)
                z = torch.matmul(q[first + i:first + i + rows.numel(), h].float().reshape(-1, D), k.T)
                z = z.view(rows.numel(), G, L) * scale
                z = torch.where(pos[None, None] <= (past + rows)[:, None, None], z, no)
                p = torch.exp(z - z.amax(dim=-1, keepdim=True))
                o = torch.matmul(p.view(-1, L), v).view(rows.numel(), G, D)
                out[first + i:first + i + rows.numel(), h] = o / p.sum(dim=-1, keepdim=True)
        first += most
    return dict(out=out.view(-1, Hq * D).to(_dt(case)))


# --------------------------------------------------------------------- 64 bits, by definition
def exact(case, seed):
    s = prepare(case, seed)
    D, page, rows = case["dim"], case["page"], _rows_of(case)
    if case["op"] == "commit":
        pools = [s["k_pages"].double(), s["v_pages"].double()]
        for b, (n, m) in enumerate(zip(rows, _kept_of(case))):
            for p in range(_past_of(case)[b] + m, _past_of(case)[b] + n):
                for pool in pools:
                    pool[:, int(s["table"][b, p // page]), p % page] = 0
        kept = [p + m for p, m in zip(_past_of(case), _kept_of(case))]
        return dict(k_pages=pools[0], v_pages=pools[1], kv_len=_i64(kept),
                    status=torch.zeros_like(s["status"]))
    first = np.concatenate([[0], np.cumsum(_own_of(case))]).tolist()
    if case["op"] == "attn":
        Hq, Hkv = case["q_heads"], case["kv_heads"]
        G = Hq // Hkv
        out = torch.zeros((s["q"].shape[0], Hq, D), dtype=torch.float64, device=DEV)
        for b, n in enumerate(rows):
            L = _past_of(case)[b] + n
            pages = s["table"][b, :(L + page - 1) // page].long()
            for h in range(Hq if n else 0):
                cols = slice(h // G * D, (h // G + 1) * D)
                k, v = (s[x][0][pages][:, :, cols].double().flatten(0, 1)[:L]
                        for x in ("k_pages", "v_pages"))
                for i in range(0, n, 256):
                    at = torch.arange(i, min(n, i + 256), device=DEV)
                    x = s["q"][first[b] + at][:, h * D:(h + 1) * D].double()
                    z = torch.einsum("rd,pd->rp", x, k) / math.sqrt(D)
                    later = torch.arange(L, device=DEV)[None] > (L - n + at)[:, None]
                    z = z.masked_fill(later, -math.inf)
                    out[first[b] + at, h] = torch.softmax(z, dim=1) @ v
        return dict(out=out.flatten(1))
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    q_out = s["q_out"].double()
    half = case["rot"] // 2
    left = torch.arange(half, device=DEV) * (1 if case["pairs"] == "half" else 2)
    right = left + (half if case["pairs"] == "half" else 1)
    for b, n in enumerate(rows):
        if n == 0:
            continue
        at = torch.arange(first[b], first[b] + n, device=DEV)
        pos = _past_of(case)[b] + torch.arange(n, device=DEV)
        angle = (pos + case["prefix"]).double()[:, None] * s["inv_freq"].double()
        turn = torch.exp(1j * angle) * s["rot_scale"]

        def spun(x, w):
            x = x[at].double().unflatten(1, (-1, D))
            if w is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()
            if half:
                z = torch.complex(x[..., left], x[..., right]) * turn[:, None]
                x = x.clone()
                x[..., left], x[..., right] = z.real, z.imag
            return x.flatten(1)

        q_out[at] = spun(s["q"], s["q_norm"])
        pages, within = s["table"][b].long()[pos // page], pos % page
        k_pages[0, pages, within] = spun(s["k"], s["k_norm"])
        v_pages[0, pages, within] = s["v"][at].double()
    return dict(q=q_out, k_pages=k_pages, v_pages=v_pages)
