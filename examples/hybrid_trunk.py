"""A small hybrid trunk (gated delta layers and one attention layer, random weights) decoding a batch
of requests that share a prompt, speculatively: the trunk's token mixers, the LM head with greedy
acceptance and the commit, all of a cycle on one stream.

    python examples/hybrid_trunk.py [--requests 8] [--prompt 1000] [--drafts 3] [--tokens 64] [--paged]

What a cycle runs (R = drafts + 1 verify rows a request):
    spec_delta_rows          each delta layer, from the request's live slot into the slots after it
    spec_prefix_attention    the attention layer, over the shared prompt and the request's own cache
    spec_lmhead_verify, spec_accept (one launch up to 8 rows), spec_commit_rollback: the engine
and the prompt once: spec_delta_prefill per delta layer. With --paged the attention layer's keys and
values lie in pages, of which the requests share those that the prompt fills, and queries and keys are
rotated by their positions:
    spec_paged_append, spec_paged_attention    in place of spec_prefix_attention
    spec_paged_commit                          beside spec_commit_rollback, by the engine
Embedding, projections, norms and the
prompt's own attention are plain torch. The drafts here are the tokens of a run without drafts, each
wrong with a given probability, so that cycles accept and roll back; greedy decoding must then give
the tokens of that run.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mtp_speculative_decoding_spec_gb300 as spec  # noqa: E402
from mtp_speculative_decoding_spec_gb300.engine import SpecVerifyEngine  # noqa: E402


class HybridTrunk:
    def __init__(self, requests, rows, capacity, dtype=torch.bfloat16, d=512, vocab=4096,
                 delta_layers=3, heads=8, key_heads=4, dk=128, dv=128, q_heads=8, kv_heads=2,
                 head_dim=128, mode="index", seed=0, device="cuda", paged=False, page=16, rot=0):
        self.B, self.R, self.cap, self.dt, self.dev = requests, rows, capacity, dtype, device
        self.L, self.H, self.Hk, self.dk, self.dv = delta_layers, heads, key_heads, dk, dv
        self.Hq, self.Hkv, self.D = q_heads, kv_heads, head_dim
        self.wdt = spec.SPEC_BF16 if dtype == torch.bfloat16 else spec.SPEC_F32
        self.mode = {"snapshot": spec.SPEC_COMMIT_SNAPSHOT, "replay": spec.SPEC_COMMIT_REPLAY,
                     "index": spec.SPEC_COMMIT_INDEX}[mode]
        g = torch.Generator(device=device).manual_seed(seed)

        def w(*shape, scale=None):
            return (torch.randn(shape, generator=g, device=device) *
                    (scale or shape[0] ** -0.5)).to(dtype)

        self.embed, self.head = w(vocab, d, scale=1.0), w(vocab, d, scale=2 * d ** -0.5)
        qkv = 2 * key_heads * dk + heads * dv
        self.delta = [dict(qkv=w(d, qkv), g=w(d, heads), b=w(d, heads), o=w(heads * dv, d))
                      for _ in range(delta_layers)]
        self.attn = dict(q=w(d, q_heads * head_dim), k=w(d, kv_heads * head_dim),
                         v=w(d, kv_heads * head_dim), o=w(q_heads * head_dim, d))
        # the state that the commit keeps: recurrent slots, and the attention layer's own caches
        n_slots, z = rows + 1, torch.zeros
        self.live = z((requests, delta_layers, heads, dk, dv), device=device)
        self.slots = z((requests, n_slots, delta_layers, heads, dk, dv), device=device)
        self.live_slot = z(requests, dtype=torch.int32, device=device)
        self.steps = [z((requests, rows, delta_layers, heads, n), device=device)
                      for n in (1, dk, dv)]
        self.cache = z((requests, 1, 2, capacity, kv_heads * head_dim), dtype=dtype, device=device)
        self.kv_len = z(requests, dtype=torch.int64, device=device)
        st = self.st = spec.spec_state_desc()
        st.rec_layers, st.rec_heads, st.rec_dk, st.rec_dv = delta_layers, heads, dk, dv
        st.n_slots, st.rec_live, st.rec_slots = n_slots, self.live.data_ptr(), self.slots.data_ptr()
        st.live_slot = self.live_slot.data_ptr()
        st.step_a, st.step_b, st.step_c = (t.data_ptr() for t in self.steps)
        e = self.cache.element_size()
        st.kv, st.kv_layers, st.kv_capacity = self.cache.data_ptr(), 1, capacity
        st.kv_row_bytes = kv_heads * head_dim * e
        st.kv_request_stride = self.cache.stride(0) * e
        st.kv_len = self.kv_len.data_ptr()
        self.paged, self.page, self.rot = paged, page, rot
        if paged:
            st.kv, st.kv_layers = None, 0
            self.cu = torch.arange(requests + 1, dtype=torch.int32, device=device)
            self.inv_freq = 10000.0 ** (-torch.arange(0, max(rot, 2), 2, device=device).float() / max(rot, 2))
        self.prefix = None
        self.ws = torch.zeros(256, dtype=torch.uint8, device=device)

    # ------------------------------------------------------------------ pieces of the trunk
    def _norm(self, x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(self.dt)

    def _delta_inputs(self, w, h):
        """q, k, v (unit-norm keys and queries) as column ranges of one row per token."""
        mixed = h @ w["qkv"]
        n = 2 * self.Hk * self.dk
        qk = mixed[:, :n].float().view(-1, 2 * self.Hk, self.dk)
        mixed[:, :n] = torch.nn.functional.normalize(qk, dim=-1).view(-1, n).to(self.dt)
        g = -torch.nn.functional.softplus((h @ w["g"]).float() - 3)
        beta = torch.sigmoid((h @ w["b"]).float())
        out = torch.empty((h.shape[0], self.H * self.dv), dtype=self.dt, device=self.dev)
        d = spec.spec_delta_desc()
        d.dtype, d.key_heads, d.scale = self.wdt, self.Hk, self.dk ** -0.5
        e = mixed.element_size()
        d.q, d.k = mixed.data_ptr(), mixed.data_ptr() + self.Hk * self.dk * e
        d.v = mixed.data_ptr() + n * e
        d.q_stride = d.k_stride = d.v_stride = mixed.stride(0)
        d.log_decay, d.beta = g.data_ptr(), beta.data_ptr()
        d.out, d.out_stride = out.data_ptr(), out.stride(0)
        return d, out, (mixed, g, beta)  # the last keeps what d points to

    def _attn_desc(self, q, out):
        d = spec.spec_attn_desc()
        d.dtype, d.q_heads, d.kv_heads, d.head_dim = self.wdt, self.Hq, self.Hkv, self.D
        d.q, d.q_stride, d.out, d.out_stride = q.data_ptr(), q.stride(0), out.data_ptr(), out.stride(0)
        d.scale = self.D ** -0.5
        if self.prefix is not None:
            d.prefix_k, d.prefix_v = self.prefix[0].data_ptr(), self.prefix[1].data_ptr()
            d.prefix_capacity, d.prefix_stride = self.prefix.shape[1], self.prefix.stride(1)
        return d

    # ------------------------------------------------------------------ the paged cache
    def _pages(self, T):
        """A cache whose requests share the T // page pages that a prompt of T fills, and have pages of
        their own for its rest and for `capacity` positions more."""
        shared, own = T // self.page, -(-(T % self.page + self.cap) // self.page)
        n = shared + self.B * own
        self.kv_pages = torch.zeros((2, n, self.page, self.Hkv * self.D), dtype=self.dt,
                                    device=self.dev)
        mine = shared + torch.arange(self.B * own, dtype=torch.int32, device=self.dev).view(self.B, own)
        self.table = torch.cat([torch.arange(shared, dtype=torch.int32, device=self.dev).expand(
            self.B, shared), mine], 1).contiguous()
        c = self.pc = spec.spec_paged_cache()
        c.dtype, c.layers, c.kv_heads, c.head_dim = self.wdt, 1, self.Hkv, self.D
        c.page_size, c.n_pages, c.max_pages = self.page, n, shared + own
        c.k_pages, c.v_pages = self.kv_pages[0].data_ptr(), self.kv_pages[1].data_ptr()
        c.page_stride = self.kv_pages.stride(1) * self.kv_pages.element_size()
        c.layer_stride = n * c.page_stride
        c.page_table, c.table_stride = self.table.data_ptr(), shared + own
        c.kv_len = self.kv_len.data_ptr()
        return shared

    def _append(self, B, rows, k, v, q=None):
        """New rows, `rows` of each of B requests: keys and values to their pages, queries rotated."""
        d = spec.spec_append_desc()
        d.k, d.v, d.k_stride, d.v_stride = k.data_ptr(), v.data_ptr(), k.stride(0), v.stride(0)
        if q is not None:
            d.q_heads, d.q, d.q_stride = self.Hq, q.data_ptr(), q.stride(0)
            d.q_out, d.q_out_stride = d.q, d.q_stride
        d.rot_dim, d.inv_freq, d.rot_scale = self.rot, self.inv_freq.data_ptr(), 1.0
        spec.spec_paged_append(B, self.cu[:B + 1] * rows, B * rows, self.pc, 0, d)

    def _attend(self, rows, q, out):
        d = spec.spec_paged_attn_desc()
        d.q_heads, d.scale = self.Hq, self.D ** -0.5
        d.q, d.q_stride, d.out, d.out_stride = q.data_ptr(), q.stride(0), out.data_ptr(), out.stride(0)
        n = spec.spec_paged_attention_workspace_bytes(self.B, self.B * rows, self.pc, d)
        if n > self.ws.numel():
            self.ws = torch.zeros(n, dtype=torch.uint8, device=self.dev)
        spec.spec_paged_attention(self.B, self.cu * rows, self.B * rows, self.pc, 0, d, None, self.ws)

    # ------------------------------------------------------------------ prompt and cycles
    def prefill(self, prompt):
        """The prompt (a list of tokens) once for all requests; every request starts after it."""
        T = len(prompt)
        x = self.embed[torch.tensor(prompt, device=self.dev)]
        state = torch.zeros_like(self.live[:1])
        st = spec.spec_state_desc()
        for f, _ in st._fields_:
            setattr(st, f, getattr(self.st, f))
        st.rec_live = state.data_ptr()
        cu = torch.tensor([0, T], dtype=torch.int32, device=self.dev)
        ws = torch.empty(spec.spec_delta_prefill_workspace_bytes(T, 1, st), dtype=torch.uint8,
                         device=self.dev)
        for layer, w in enumerate(self.delta):
            d, out, keep = self._delta_inputs(w, self._norm(x))
            spec.spec_delta_prefill(1, cu, T, st, layer, d, None, ws)
            x = x + out @ w["o"]
        h, w = self._norm(x), self.attn
        self.kv_len.zero_()
        if self.paged:
            shared = self._pages(T) * self.page
            k, v = h @ w["k"], h @ w["v"]
            if shared:
                self._append(1, shared, k, v)  # by request 0, on the pages that all have
                self.kv_len.fill_(shared)
            rest = T - shared
            if rest:
                self._append(self.B, rest, k[shared:].repeat(self.B, 1), v[shared:].repeat(self.B, 1))
                n = torch.full((self.B,), rest, dtype=torch.int32, device=self.dev)
                spec.spec_paged_commit(self.B, self.pc, None, n)
        else:
            self.prefix = torch.stack([h @ w["k"], h @ w["v"]])
        # the attention layer is the last: no later layer reads the prompt's outputs of it
        self.slots.zero_()
        self.slots[:, 0] = state
        self.live.copy_(state.expand_as(self.live))
        self.live_slot.zero_()
        self.cache.zero_()

    def verify_rows(self, tokens):
        """Hidden rows [B * R, d] of the verify rows tokens [B, R] (R at most the trunk's rows)."""
        B, R = tokens.shape
        x = self.embed[tokens.reshape(-1)]
        for layer, w in enumerate(self.delta):
            d, out, keep = self._delta_inputs(w, self._norm(x))
            spec.spec_delta_rows(B, R, self.st, layer, self.mode, d)
            x = x + out @ w["o"]
        h, w = self._norm(x), self.attn
        if self.paged:
            q = h @ w["q"]
            self._append(B, R, h @ w["k"], h @ w["v"], q)
            out = torch.empty_like(q)
            self._attend(R, q, out)
            return self._norm(x + out @ w["o"])
        at = self.kv_len[:, None] + torch.arange(R, device=self.dev)[None]
        b = torch.arange(B, device=self.dev)[:, None].expand(B, R)
        for i, name in enumerate("kv"):
            self.cache[:, 0, i].index_put_((b, at), (h @ w[name]).view(B, R, -1))
        q = h @ w["q"]
        out = torch.empty_like(q)
        d = self._attn_desc(q, out)
        n = spec.spec_prefix_attention_workspace_bytes(B, R, self.st, d)
        if n > self.ws.numel():
            self.ws = torch.zeros(n, dtype=torch.uint8, device=self.dev)
        spec.spec_prefix_attention(B, R, self.st, 0, d, None, self.ws)
        return self._norm(x + out @ w["o"])


def decode(trunk, prompt, n_tokens, drafts_of=None, drafts=0):
    """Greedy decoding of every request from the token after the prompt on. drafts_of(b, done, k):
    request b's drafts for the tokens from `done` on. Returns the tokens and the number of cycles."""
    B, k = trunk.B, drafts
    eng = SpecVerifyEngine(trunk.head, trunk.wdt, trunk.head.shape[0], trunk.head.shape[1], 1, B,
                           k + 1, k, want_q_logits=False, fuse_greedy=B * (k + 1) <= 8,
                           device=trunk.dev)
    trunk.prefill(prompt[:-1])
    eng.attach_state(trunk.st, trunk.mode)
    if trunk.paged:
        eng.attach_paged(trunk.pc)
    eng.set_requests(temps=[0.0] * B, k=[k] * B)
    tokens, cycles = [[] for _ in range(B)], 0
    last = [prompt[-1] + b for b in range(B)]  # each request goes its own way
    while min(len(t) for t in tokens) < n_tokens:
        rows = torch.tensor([[last[b]] + (drafts_of(b, len(tokens[b]), k) if k else [])
                             for b in range(B)])
        if k:
            eng.drafts.copy_(rows[:, 1:].int())
        eng.verify_cycle(trunk.verify_rows(rows.to(trunk.dev)))
        res = eng.out.cpu().numpy().view(spec.ACCEPT_OUT_DTYPE)
        assert (res["status"] == spec.REQ_OK).all()
        for b in range(B):
            tokens[b] += [int(t) for t in res["tokens"][b][:res["n_emit"][b]]]
            last[b] = tokens[b][-1]
        cycles += 1
    return [t[:n_tokens] for t in tokens], cycles


def noisy_drafts(tokens, vocab, wrong, seed=0):
    """Drafts that follow `tokens`, each replaced by a random token with probability `wrong`."""
    g = torch.Generator().manual_seed(seed)

    def of(b, done, k):
        out = []
        for i in range(k):
            right = tokens[b][done + i] if done + i < len(tokens[b]) else 0
            bad = float(torch.rand(1, generator=g)) < wrong
            out.append(int(torch.randint(vocab, (1,), generator=g)) if bad else right)
        return out

    return of


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--wrong", type=float, default=0.3)
    ap.add_argument("--mode", choices=("snapshot", "replay", "index"), default="index")
    ap.add_argument("--paged", action="store_true")
    a = ap.parse_args()
    trunk = HybridTrunk(a.requests, a.drafts + 1, a.tokens + 16, mode=a.mode, paged=a.paged,
                        rot=64 if a.paged else 0)
    g = torch.Generator().manual_seed(1)
    prompt = torch.randint(2000, (a.prompt,), generator=g).tolist()
    plain, n0 = decode(trunk, prompt, a.tokens)
    drafted, n1 = decode(trunk, prompt, a.tokens, noisy_drafts(plain, 4096, a.wrong), a.drafts)
    same = sum(x == y for p, d in zip(plain, drafted) for x, y in zip(p, d))
    print(f"{a.requests} requests x {a.tokens} tokens: {n0} cycles without drafts, {n1} with "
          f"{a.drafts} drafts each ({a.tokens / n1:.2f} tokens a cycle for the slowest request); "
          f"{same} of {a.requests * a.tokens} tokens the same")


if __name__ == "__main__":
    main()
