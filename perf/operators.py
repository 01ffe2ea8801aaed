"""Cases of the trunk's token mixers that a verify cycle runs before the LM head: the gated delta
rule over the recurrent layers (the rows of a verify pass, and a prompt's chunks) and attention of
the verify rows over a shared prefix and each request's own KV cache.

The sizes are those of this repository's workloads (synth/configs.py): recurrent state of 16 heads
x [128, 128] fp32 (and 2 x [16, 16]), one attention layer of 4 KV heads x 256 bf16 (and 2 x 64
fp32), 1..8 verify rows per request, 1..32 requests, contexts of 15,360 and 63,488 positions.
"""

import math

import numpy as np
import torch

own = False

CHUNK = 64
DEV = "cuda"


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one small fp32 request, the state committed by replay: launch latency
        dict(name="rows_tiny_f32_1x1", op="rows", B=1, R=1, heads=2, key_heads=2, dk=16, dv=16,
             dtype="f32", mode="replay", ragged=False),
        # a verify pass of width 8 over one recurrent layer, the live state a slot: latency
        dict(name="rows_index_1x8", op="rows", B=1, R=8, heads=16, key_heads=16, dk=128, dv=128,
             dtype="bf16", mode="index", ragged=False),
        # 32 requests at mixed widths; only the replay inputs are written
        dict(name="rows_replay_32x8", op="rows", B=32, R=8, heads=16, key_heads=8, dk=128, dv=128,
             dtype="bf16", mode="replay", ragged=True),
        # 32 requests at mixed widths, the state snapshotted after every row: most bytes
        dict(name="rows_snapshot_32x8", op="rows", B=32, R=8, heads=16, key_heads=16, dk=128,
             dv=128, dtype="bf16", mode="snapshot", ragged=True),
        # prompts of very different lengths in one call: empty, one token, odd ones
        dict(name="prefill_ragged", op="prefill", lens="0,1,77,1000,2311", heads=16, key_heads=8,
             dk=128, dv=128, dtype="bf16", init=True),
        # one 15K prompt from an empty state
        dict(name="prefill_1x15360", op="prefill", lens="15360", heads=16, key_heads=16, dk=128,
             dv=128, dtype="bf16", init=False),
        # one 63K prompt continued from a state: the longest chain
        dict(name="prefill_1x63488", op="prefill", lens="63488", heads=16, key_heads=16, dk=128,
             dv=128, dtype="bf16", init=True),
        # two rows of one small fp32 request, no shared prefix: launch latency
        dict(name="attn_tiny_f32_1x2", op="attn", B=1, R=2, q_heads=4, kv_heads=2, dim=64,
             prefix=0, cap=512, base=256, dtype="f32", ragged=False),
        # greedy decoding of one long request (2 verify rows), all of it in its own cache
        dict(name="attn_1x2_own_63488", op="attn", B=1, R=2, q_heads=16, kv_heads=4, dim=256,
             prefix=0, cap=65536, base=63488, dtype="bf16", ragged=False),
        # single-token decoding of 8 samples of one long prompt, odd suffix lengths
        dict(name="attn_8x1_prefix_63488", op="attn", B=8, R=1, q_heads=16, kv_heads=4, dim=256,
             prefix=63488, cap=2048, base=1333, dtype="bf16", ragged=True),
        # 32 requests at mixed widths over one 15K prompt, a few of them sharing only part of it
        dict(name="attn_32x8_prefix_15360", op="attn", B=32, R=8, q_heads=16, kv_heads=4, dim=256,
             prefix=15360, cap=1024, base=700, dtype="bf16", ragged=True),
        # the same batch over a 63K prompt: the most arithmetic
        dict(name="attn_32x8_prefix_63488", op="attn", B=32, R=8, q_heads=16, kv_heads=4, dim=256,
             prefix=63488, cap=1024, base=700, dtype="bf16", ragged=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rows", "prefill", "attn"])
    if op == "rows":
        dk, dv = rng.choice([(128, 128), (128, 128), (64, 128), (16, 16), (96, 64)])
        key_heads = rng.choice([1, 2, 4, 8, 16])
        heads = min(16, key_heads * rng.choice([1, 1, 2, 4]))
        return dict(op=op, B=_log_int(rng, 1, 32), R=rng.randint(1, 8), heads=heads,
                    key_heads=min(key_heads, heads), dk=dk, dv=dv,
                    dtype=rng.choice(["bf16", "bf16", "f32"]),
                    mode=rng.choice(["snapshot", "replay", "index"]), ragged=rng.random() < 0.5)
    if op == "prefill":
        n = rng.choice([1, 1, 2, 3, 5])
        lens = [_log_int(rng, 1, 40000 // n) for _ in range(n)]
        if n > 2 and rng.random() < 0.5:
            lens[rng.randrange(n)] = 0
        key_heads = rng.choice([4, 8, 16])
        return dict(op=op, lens=",".join(str(x) for x in lens),
                    heads=min(16, key_heads * rng.choice([1, 2])), key_heads=key_heads, dk=128,
                    dv=rng.choice([128, 128, 64]), dtype="bf16", init=rng.random() < 0.5)
    dim = rng.choice([64, 128, 256, 256])
    kv_heads = rng.choice([1, 2, 4])
    group = rng.choice([1, 2, 4, 6] if kv_heads < 4 else [1, 2, 4])
    B = _log_int(rng, 1, 32)
    base = _log_int(rng, 1, 65000 if B == 1 else 4000)
    return dict(op=op, B=B, R=rng.randint(1, 8), q_heads=kv_heads * group,
                kv_heads=kv_heads, dim=dim, prefix=rng.choice([0, _log_int(rng, 1, 60000)]),
                cap=base + 8 + rng.randint(0, 200), base=base,
                dtype="bf16" if rng.random() < 0.85 or B * base > 20000 else "f32",
                ragged=rng.random() < 0.5)


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _rows_of(case):
    """Rows each request runs: R, or a spread over 1..R."""
    B, R = case["B"], case["R"]
    return [1 + (5 * b + 3) % R if case["ragged"] else R for b in range(B)]


def _own_of(case):
    """Positions of each request's own cache before this cycle's rows."""
    return [case["base"] - (37 * b) % (case["base"] // 2 + 1) if case["ragged"] else case["base"]
            for b in range(case["B"])]


def _prefix_of(case):
    """Positions of the shared prefix each request attends to: all, or now and then a part."""
    P = case["prefix"]
    return [P - (P // 3 + 5 * b) % (P + 1) if case["ragged"] and b % 8 == 5 else P
            for b in range(case["B"])]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rows":
        H, Hk, dk, dv = case["heads"], case["key_heads"], case["dk"], case["dv"]
        rows, st = sum(_rows_of(case)), 4 * H * dk * dv
        io = rows * ((2 * Hk * dk + 2 * H * dv) * e + 8 * H)
        if case["mode"] == "snapshot":    # the state in, the state before the cycle and per row out
            states = 2 * case["B"] + rows
        elif case["mode"] == "index":
            states = case["B"] + rows
        else:                             # the state in and out, the steps out
            states = 2 * case["B"]
            io += rows * 4 * H * (1 + dk + dv)
        return dict(bytes=io + states * st, flops=rows * H * dk * dv * 7)
    if case["op"] == "prefill":
        H, Hk, dk, dv = case["heads"], case["key_heads"], case["dk"], case["dv"]
        T, n = sum(_lens(case)), len(_lens(case))
        st = 4 * H * dk * dv * n * (2 if case["init"] else 1)
        return dict(bytes=T * ((2 * Hk * dk + 2 * H * dv) * e + 8 * H) + st,
                    flops=T * H * dk * dv * 7)
    Hq, Hkv, D, B = case["q_heads"], case["kv_heads"], case["dim"], case["B"]
    rows, own_len, pre = _rows_of(case), _own_of(case), _prefix_of(case)
    pairs = sum(n * (pre[b] + own_len[b]) + n * (n + 1) // 2 for b, n in enumerate(rows))
    kv = max(pre) + sum(own_len[b] + n for b, n in enumerate(rows))
    return dict(bytes=2 * kv * Hkv * D * e + 2 * sum(rows) * Hq * D * e, flops=4 * pairs * Hq * D)


# ------------------------------------------------------------------------------------- inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _delta_inputs(case, rows, g):
    """q, k, v as column ranges of one row per token (as a convolution over them leaves them),
    unit-norm keys and queries, decays that keep a token for ten to a few hundred steps."""
    H, Hk, dk, dv = case["heads"], case["key_heads"], case["dk"], case["dv"]
    n = max(rows, 1)
    qk = torch.randn((n, 2 * Hk, dk), generator=g, device=DEV)
    qk = qk / qk.norm(dim=-1, keepdim=True)
    v = torch.randn((n, H * dv), generator=g, device=DEV)
    mixed = torch.cat([qk.reshape(n, -1), v], dim=1).to(_dt(case))[:rows]
    gate = torch.randn((n, H), generator=g, device=DEV)
    head = torch.rand((1, H), generator=g, device=DEV)
    log_decay = -torch.exp(-5.5 + 3.5 * head) * torch.nn.functional.softplus(gate + 0.5)
    beta = torch.sigmoid(torch.randn((n, H), generator=g, device=DEV))
    return dict(mixed=mixed, q=mixed[:, :Hk * dk], k=mixed[:, Hk * dk:2 * Hk * dk],
                v=mixed[:, 2 * Hk * dk:], log_decay=log_decay[:rows].contiguous(),
                beta=beta[:rows].contiguous(), scale=dk ** -0.5)


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def _i64(a):
    return torch.tensor(a, dtype=torch.int64, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case=case)
    if case["op"] == "rows":
        B, R, H, dk, dv = case["B"], case["R"], case["heads"], case["dk"], case["dv"]
        s.update(_delta_inputs(case, B * R, g))
        n_slots = R + 1
        s["n_rows"] = _i32(_rows_of(case)) if case["ragged"] else None
        s["live"] = torch.randn((B, 1, H, dk, dv), generator=g, device=DEV) * 0.3
        s["live_slot"] = _i32([(3 * b + 1) % n_slots for b in range(B)])
        n = 1 if case["mode"] == "replay" else n_slots
        s["slots"] = torch.zeros((B, n_slots, 1, H, dk, dv), device=DEV)
        if case["mode"] == "index":
            s["slots"][torch.arange(B, device=DEV), s["live_slot"].long()] = s["live"]
        if n == 1:
            s["step_a"] = torch.zeros((B, R, 1, H), device=DEV)
            s["step_b"] = torch.zeros((B, R, 1, H, dk), device=DEV)
            s["step_c"] = torch.zeros((B, R, 1, H, dv), device=DEV)
        s["out"] = torch.zeros((B * R, H * dv), dtype=_dt(case), device=DEV)
    elif case["op"] == "prefill":
        lens, H, dk, dv = _lens(case), case["heads"], case["dk"], case["dv"]
        T = sum(lens)
        s.update(_delta_inputs(case, T, g))
        s["cu_rows"] = _i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
        s["init"] = torch.randn((len(lens), 1, H, dk, dv), generator=g, device=DEV) * 0.3 \
            if case["init"] else None
        s["live"] = torch.zeros((len(lens), 1, H, dk, dv), device=DEV)
        s["out"] = torch.zeros((T, H * dv), dtype=_dt(case), device=DEV)
    else:
        B, R, Hq, Hkv, D = case["B"], case["R"], case["q_heads"], case["kv_heads"], case["dim"]
        P, cap = case["prefix"], case["cap"]

        def rnd(*shape):  # in pieces: a long cache in fp32 at once would be several GB
            out = torch.empty(shape, dtype=_dt(case), device=DEV)
            flat = out.view(-1)
            for i in range(0, flat.numel(), 1 << 26):
                n = min(1 << 26, flat.numel() - i)
                flat[i:i + n] = torch.randn(n, generator=g, device=DEV)
            return out

        # queries a little longer than unit variance: the softmax then has some heavy positions
        s["q"] = (rnd(B * R, Hq * D).float() * 1.5).to(_dt(case))
        s["prefix_kv"] = rnd(2, P, Hkv * D) if P else None
        s["cache"] = rnd(B, 1, 2, cap, Hkv * D)
        s["kv_len"] = _i64(_own_of(case))
        s["prefix_len"] = _i64(_prefix_of(case)) if P else None
        s["n_rows"] = _i32(_rows_of(case)) if case["ragged"] else None
        s["out"] = torch.zeros((B * R, Hq * D), dtype=_dt(case), device=DEV)
    if own:
        s.update(_handle(s))
    return s


# ------------------------------------------------------------------- the framework's operators
def _handle(s):
    """The state description, the operator's description and the workspace a program keeps."""
    import mtp_speculative_decoding_spec_gb300 as spec
    case = s["case"]
    wdt = spec.SPEC_BF16 if case["dtype"] == "bf16" else spec.SPEC_F32
    st = spec.spec_state_desc()
    if case["op"] in ("rows", "prefill"):
        st.rec_layers, st.rec_heads, st.rec_dk, st.rec_dv = 1, case["heads"], case["dk"], case["dv"]
        st.rec_live = s["live"].data_ptr()
        d = spec.spec_delta_desc()
        d.dtype, d.key_heads, d.scale = wdt, case["key_heads"], s["scale"]
        for f in ("q", "k", "v"):
            setattr(d, f, s[f].data_ptr())
            setattr(d, f + "_stride", s["mixed"].stride(0))
        d.log_decay, d.beta = s["log_decay"].data_ptr(), s["beta"].data_ptr()
        d.out, d.out_stride = s["out"].data_ptr(), s["out"].stride(0)
        if case["op"] == "prefill":
            n = spec.spec_delta_prefill_workspace_bytes(s["mixed"].shape[0], len(_lens(case)), st)
            return dict(st=st, desc=d, ws=torch.zeros(max(n, 256), dtype=torch.uint8, device=DEV))
        st.rec_slots, st.n_slots = s["slots"].data_ptr(), case["R"] + 1
        st.live_slot = s["live_slot"].data_ptr()
        if case["mode"] == "replay":
            st.step_a, st.step_b = s["step_a"].data_ptr(), s["step_b"].data_ptr()
            st.step_c = s["step_c"].data_ptr()
        mode = {"snapshot": spec.SPEC_COMMIT_SNAPSHOT, "replay": spec.SPEC_COMMIT_REPLAY,
                "index": spec.SPEC_COMMIT_INDEX}[case["mode"]]
        return dict(st=st, desc=d, mode=mode)
    e = 2 if case["dtype"] == "bf16" else 4
    st.kv, st.kv_layers, st.kv_capacity = s["cache"].data_ptr(), 1, case["cap"]
    st.kv_row_bytes = case["kv_heads"] * case["dim"] * e
    st.kv_request_stride = 2 * case["cap"] * st.kv_row_bytes
    st.kv_len = s["kv_len"].data_ptr()
    d = spec.spec_attn_desc()
    d.dtype, d.q_heads, d.kv_heads, d.head_dim = wdt, case["q_heads"], case["kv_heads"], case["dim"]
    d.q, d.q_stride = s["q"].data_ptr(), s["q"].stride(0)
    d.out, d.out_stride, d.scale = s["out"].data_ptr(), s["out"].stride(0), case["dim"] ** -0.5
    if case["prefix"]:
        d.prefix_k, d.prefix_v = s["prefix_kv"][0].data_ptr(), s["prefix_kv"][1].data_ptr()
        d.prefix_capacity, d.prefix_stride = case["prefix"], case["kv_heads"] * case["dim"]
        d.prefix_len = s["prefix_len"].data_ptr()
    n = spec.spec_prefix_attention_workspace_bytes(case["B"], case["R"], st, d)
    return dict(st=st, desc=d, ws=torch.zeros(max(n, 256), dtype=torch.uint8, device=DEV))


def _run_own(s):
    import mtp_speculative_decoding_spec_gb300 as spec
    case = s["case"]
    if case["op"] == "rows":
        spec.spec_delta_rows(case["B"], case["R"], s["st"], 0, s["mode"], s["desc"], s["n_rows"])
        if case["mode"] == "replay":
            return dict(out=s["out"], start=s["slots"][:, 0], step_a=s["step_a"],
                        step_b=s["step_b"], step_c=s["step_c"])
        return dict(out=s["out"], slots=s["slots"])
    if case["op"] == "prefill":
        spec.spec_delta_prefill(len(_lens(case)), s["cu_rows"], s["mixed"].shape[0], s["st"], 0,
                                s["desc"], s["init"], s["ws"])
        return dict(out=s["out"], state=s["live"])
    spec.spec_prefix_attention(case["B"], case["R"], s["st"], 0, s["desc"], s["n_rows"], s["ws"])
    return dict(out=s["out"])


def run(s):
    if own:
        return _run_own(s)
    return dict(rows=_plain_rows, prefill=_plain_prefill, attn=_plain_attn)[s["case"]["op"]](s)


# ------------------------------------------------------------------------------- plain forms
def _heads_of(s, name, heads, dim):
    """[rows, heads, dim] fp32 of a column range, key heads repeated for the value heads."""
    case = s["case"]
    x = s[name].float().reshape(-1, heads, dim)
    return x.repeat_interleave(case["heads"] // heads, dim=1)


def _plain_rows(s):
    """S <- a S + k u^T with u = beta (v - (a S)^T k), o = scale S^T q, row by row."""
    case = s["case"]
    B, R, H, dk, dv = case["B"], case["R"], case["heads"], case["dk"], case["dv"]
    q = _heads_of(s, "q", case["key_heads"], dk).view(B, R, H, dk)
    k = _heads_of(s, "k", case["key_heads"], dk).view(B, R, H, dk)
    v = s["v"].float().reshape(B, R, H, dv)
    a = torch.exp(s["log_decay"]).view(B, R, H)
    beta = s["beta"].view(B, R, H)
    S = s["live"][:, 0]
    runs = torch.ones((B, R), dtype=torch.bool, device=DEV) if s["n_rows"] is None else \
        torch.arange(R, device=DEV)[None] < s["n_rows"][:, None]
    states, outs, us = [], [], []
    for r in range(R):
        D = a[:, r, :, None, None] * S
        u = beta[:, r, :, None] * (v[:, r] - torch.matmul(k[:, r, :, None], D)[:, :, 0])
        S = D + k[:, r, :, :, None] * u[:, :, None]
        o = torch.matmul(q[:, r, :, None], S)[:, :, 0] * s["scale"]
        on = runs[:, r, None, None]
        outs.append(torch.where(on, o, torch.zeros((), device=DEV)))
        us.append(torch.where(on, u, torch.zeros((), device=DEV)))
        if case["mode"] != "replay":
            states.append(S)
    out = torch.stack(outs, dim=1).to(_dt(case)).reshape(B * R, H * dv)
    if case["mode"] == "replay":
        on = runs[:, :, None, None]
        zero = torch.zeros((), device=DEV)
        return dict(out=out, start=s["live"], step_a=torch.where(on, a[:, :, None], zero),
                    step_b=torch.where(on[..., None], k[:, :, None], zero),
                    step_c=torch.stack(us, dim=1)[:, :, None])
    # row r's state goes to slot r + 1, or that many slots after the live one; the rest stay
    slots = torch.zeros_like(s["slots"])
    b = torch.arange(B, device=DEV)
    first = s["live_slot"].long() if case["mode"] == "index" else torch.zeros_like(b)
    slots[b, first] = s["live"]
    for r in range(R):
        at = (first + r + 1) % (R + 1)
        slots[b, at, 0] = torch.where(runs[:, r, None, None, None], states[r], slots[b, at, 0])
    return dict(out=out, slots=slots)


def _plain_prefill(s):
    """The same recurrence by chunks of 64 tokens. With G the running sum of the log decays in a
    chunk, A[i, j] = beta_i exp(G_i - G_j) k_i.k_j (j < i) and T = (I + A)^-1:
    u = T (beta v) - T (beta exp(G) k) S, o = scale (exp(G) q S + (exp(G_i - G_j) q_i.k_j)_{j<=i} u),
    S <- exp(G_last) S + (exp(G_last - G) k)^T u. Shorter requests are filled up with tokens of no
    decay and beta 0, which leave the state as it is."""
    case = s["case"]
    lens, H, dk, dv, C = _lens(case), case["heads"], case["dk"], case["dv"], CHUNK
    B, N = len(lens), max(1, -(-max(lens) // CHUNK))
    lens_t = torch.diff(s["cu_rows"].long())
    t = torch.arange(N * C, device=DEV)
    row = (s["cu_rows"][:-1, None].long() + t[None]).clamp(max=max(sum(lens) - 1, 0))
    live = t[None] < lens_t[:, None]

    def chunks(x, fill):  # [rows, H, n] -> [B, H, N, C, n]
        y = torch.where(live[:, :, None, None], x[row], torch.full((), fill, device=DEV))
        return y.view(B, N, C, H, -1).permute(0, 3, 1, 2, 4)

    q = chunks(_heads_of(s, "q", case["key_heads"], dk), 0.0)
    k = chunks(_heads_of(s, "k", case["key_heads"], dk), 0.0)
    v = chunks(s["v"].float().reshape(-1, H, dv), 0.0)
    G = torch.cumsum(chunks(s["log_decay"][:, :, None], 0.0)[..., 0], dim=-1)
    beta = chunks(s["beta"][:, :, None], 0.0)
    i = torch.arange(C, device=DEV)
    lower = i[:, None] >= i[None]
    decay = torch.exp(torch.where(lower, G[..., :, None] - G[..., None, :],
                                  torch.full((), -math.inf, device=DEV)))
    kt = k.transpose(-1, -2)
    T = torch.where(lower & (i[:, None] != i[None]), -beta * decay * torch.matmul(k, kt),
                    torch.zeros((), device=DEV))
    for r in range(1, C):  # forward substitution: row r of (I + A)^-1 from the rows above it
        T[..., r, :r] = T[..., r, :r] + torch.matmul(T[..., r, None, :r], T[..., :r, :r])[..., 0, :]
    T = T + torch.eye(C, device=DEV)
    u0 = torch.matmul(T, beta * v)
    w = torch.matmul(T, beta * torch.exp(G)[..., None] * k)
    attn = decay * torch.matmul(q, kt)
    qd = q * torch.exp(G)[..., None]
    kd = (k * torch.exp(G[..., -1:] - G)[..., None]).transpose(-1, -2)
    last = torch.exp(G[..., -1])[..., None, None]
    S = s["init"][:, 0] if s["init"] is not None else torch.zeros((B, H, dk, dv), device=DEV)
    o = torch.empty((B, H, N, C, dv), device=DEV)
    for n in range(N):
        u = u0[:, :, n] - torch.matmul(w[:, :, n], S)
        o[:, :, n] = torch.matmul(qd[:, :, n], S) + torch.matmul(attn[:, :, n], u)
        S = last[:, :, n] * S + torch.matmul(kd[:, :, n], u)
    o = (o * s["scale"]).permute(0, 2, 3, 1, 4).reshape(B, N * C, H * dv)
    return dict(out=o[live].to(_dt(case)), state=S[:, None])


def _plain_attn(s):
    """softmax(scale q.k) v over the request's part of the shared prefix and its own cache up to
    the row itself; zero where a request does not run the row."""
    case = s["case"]
    B, R, Hq, Hkv, D = case["B"], case["R"], case["q_heads"], case["kv_heads"], case["dim"]
    G, P, scale = Hq // Hkv, case["prefix"], D ** -0.5
    q = s["q"].float().reshape(B, R, Hkv, G, D).permute(2, 0, 1, 3, 4)     # [Hkv, B, R, G, D]
    most = case["base"] + R
    cache = s["cache"][:, 0, :, :most].float().reshape(B, 2, most, Hkv, D).permute(1, 3, 0, 2, 4)
    no = torch.full((), -math.inf, device=DEV)
    zero = torch.zeros((), device=DEV)
    pos = torch.arange(most, device=DEV)
    r = torch.arange(R, device=DEV)
    sees = pos[None, None] <= (s["kv_len"][:, None] + r[None])[:, :, None]      # [B, R, most]
    own_s = torch.matmul(q.reshape(Hkv, B, R * G, D), cache[0].transpose(-1, -2)) * scale
    own_s = torch.where(sees[None, :, :, None], own_s.view(Hkv, B, R, G, most), no)
    top = own_s.amax(dim=-1, keepdim=True)
    if P:
        kp, vp = s["prefix_kv"].float().reshape(2, P, Hkv, D).permute(0, 2, 1, 3)
        pre_s = torch.matmul(q.reshape(Hkv, B * R * G, D), kp.transpose(-1, -2))
        pre_s = pre_s.view(Hkv, B, R, G, P) * scale
        if case["ragged"]:
            has = torch.arange(P, device=DEV)[None] < s["prefix_len"][:, None]
            pre_s = torch.where(has[None, :, None, None], pre_s, no)
        top = torch.maximum(top, pre_s.amax(dim=-1, keepdim=True))
    own_p = torch.exp(own_s - top)
    total = own_p.sum(dim=-1, keepdim=True)
    o = torch.matmul(own_p.view(Hkv, B, R * G, most), cache[1]).view(Hkv, B, R, G, D)
    if P:
        pre_p = torch.exp(pre_s - top)
        total = total + pre_p.sum(dim=-1, keepdim=True)
        o = o + torch.matmul(pre_p.view(Hkv, B * R * G, P), vp).view(Hkv, B, R, G, D)
    o = (o / total).permute(1, 2, 0, 3, 4)
    if s["n_rows"] is not None:
        o = torch.where((r[None] < s["n_rows"][:, None])[:, :, None, None, None], o, zero)
    return dict(out=o.reshape(B * R, Hq * D).to(_dt(case)))


# --------------------------------------------------------------------- 64 bits, by definition
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(s)
    H, Hk, dk, dv = case["heads"], case["key_heads"], case["dk"], case["dv"]
    per = H // Hk
    head = [h // per for h in range(H)]

    def step(S, t):
        """One token of every request: S in 64 bits, t = the rows of the inputs."""
        k = s["k"][t].double().view(-1, Hk, dk)[:, head]
        q = s["q"][t].double().view(-1, Hk, dk)[:, head]
        v = s["v"][t].double().view(-1, H, dv)
        a = s["log_decay"][t].double().exp()
        S = S * a[:, :, None, None]
        u = (v - torch.einsum("bhi,bhij->bhj", k, S)) * s["beta"][t].double()[:, :, None]
        S = S + torch.einsum("bhi,bhj->bhij", k, u)
        return S, torch.einsum("bhi,bhij->bhj", q, S) * s["scale"], a, k, u

    if case["op"] == "rows":
        B, R, n = case["B"], case["R"], _rows_of(case)
        out = torch.zeros((B, R, H * dv), dtype=torch.float64, device=DEV)
        slots = torch.zeros((B, R + 1, 1, H, dk, dv), dtype=torch.float64, device=DEV)
        sa = torch.zeros((B, R, 1, H), dtype=torch.float64, device=DEV)
        sb = torch.zeros((B, R, 1, H, dk), dtype=torch.float64, device=DEV)
        sc = torch.zeros((B, R, 1, H, dv), dtype=torch.float64, device=DEV)
        for b in range(B):
            at = int(s["live_slot"][b]) if case["mode"] == "index" else 0
            S = s["live"][b].double()
            slots[b, at, 0] = S[0]
            for r in range(n[b]):
                S, o, a, k, u = step(S, torch.tensor([b * R + r], device=DEV))
                out[b, r], sa[b, r, 0], sb[b, r, 0], sc[b, r, 0] = o.view(-1), a[0], k[0], u[0]
                slots[b, (at + r + 1) % (R + 1), 0] = S[0]
        out = out.view(B * R, H * dv)
        if case["mode"] == "replay":
            return dict(out=out, start=slots[:, 0], step_a=sa, step_b=sb, step_c=sc)
        return dict(out=out, slots=slots)
    lens, cu = _lens(case), s["cu_rows"].tolist()
    out = torch.zeros((sum(lens), H * dv), dtype=torch.float64, device=DEV)
    state = torch.zeros((len(lens), 1, H, dk, dv), dtype=torch.float64, device=DEV)
    if s["init"] is not None:
        state[:] = s["init"]
    for b, n in enumerate(lens):
        S = state[b].clone()
        for t in range(cu[b], cu[b] + n):
            S, o, _, _, _ = step(S, slice(t, t + 1))
            out[t] = o.view(-1)
        state[b] = S
    return dict(out=out, state=state)


def _exact_attn(s):
    case = s["case"]
    B, R, Hq, Hkv, D = case["B"], case["R"], case["q_heads"], case["kv_heads"], case["dim"]
    G, P = Hq // Hkv, case["prefix"]
    out = torch.zeros((B, R, Hq, D), dtype=torch.float64, device=DEV)
    q = s["q"].double().view(B, R, Hq, D)
    for b, n in enumerate(_rows_of(case)):
        p, m = _prefix_of(case)[b], _own_of(case)[b]
        kv = s["cache"][b, 0, :, :m + n].double().view(2, m + n, Hkv, D)
        if p and P:
            kv = torch.cat([s["prefix_kv"][:, :p].double().view(2, p, Hkv, D), kv], dim=1)
        for h in range(Hkv):
            k, v = kv[0, :, h], kv[1, :, h]
            z = q[b, :n, h * G:(h + 1) * G].reshape(n * G, D) @ k.T / math.sqrt(D)
            reach = kv.shape[1] - n + torch.arange(n, device=DEV).repeat_interleave(G)
            z[torch.arange(kv.shape[1], device=DEV)[None] > reach[:, None]] = -math.inf
            out[b, :n, h * G:(h + 1) * G] = (torch.softmax(z, dim=1) @ v).view(n, G, D)
    return dict(out=out.view(B * R, Hq * D))
