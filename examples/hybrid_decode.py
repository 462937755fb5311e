#!/usr/bin/env python3
"""Serving a small hybrid decoder: state-space layers and attention layers in turn, random
weights, requests that come, grow and end.

Every step goes through the library as a serving loop would: the page step takes and frees
cache pages and maps the step's tokens to slots, the norm and rotation of q and k write the
cache, attention reads it, and the SSD scan carries its state.  A step of one token a
request copies nothing to the host: lengths, tables and slots stay on the device.

A request that the free pages do not cover is refused for the step: its tokens are in no
cache and change no state, and the loop offers them again in the next one.

  python examples/hybrid_decode.py [--steps 12] [--cache bf16|f8] [--pages 20] [--check]

--check recomputes every request from scratch in fp64 (dense causal attention, the
sequential recurrence) and prints how far the served hidden states are from that.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_s6_amd as lib  # noqa: E402

D, LAYERS, VOCAB = 256, 4, 512
H, HK, HD, ROT = 8, 2, 64, 32                # attention: query and kv heads, their size, rotated part
SH, SP, SN = 8, 32, 64                       # state-space: heads, head size, state
PAGE, MAX_PAGES = 16, 8
EPS = 1e-6


def weights(device, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: (torch.randn(s, generator=g) / math.sqrt(s[-1])).to(device)  # noqa: E731
    w = {"embed": r(VOCAB, D) * math.sqrt(D), "layers": []}
    for i in range(LAYERS):
        if i % 2 == 0:
            w["layers"].append({"in": r(SH * SP + 2 * SN + SH, D), "out": r(D, SH * SP),
                                "A_log": torch.linspace(0.0, 2.0, SH).to(device), "D": torch.ones(SH, device=device),
                                "dt_bias": torch.full((SH,), -2.0, device=device)})
        else:
            w["layers"].append({"in": r((H + 2 * HK) * HD, D), "out": r(D, H * HD),
                                "wq": 1 + 0.1 * r(HD), "wk": 1 + 0.1 * r(HD)})
    w["inv_freq"] = (1e4 ** (-torch.arange(ROT // 2, dtype=torch.float64) / (ROT // 2))).float().to(device)
    return w


def rms(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def split_ssm(u):
    """Projected rows (..., SH*SP + 2*SN + SH) as x, B, C (bf16) and dt (fp32)."""
    x, b, c, dt = u.split([SH * SP, SN, SN, SH], -1)
    bf = lambda t, *s: t.unflatten(-1, s).to(torch.bfloat16).contiguous()  # noqa: E731
    return bf(x, SH, SP), bf(b, 1, SN), bf(c, 1, SN), dt.float().contiguous()


class Server:
    """A batch of places for requests, their pages, and each layer's cache or state."""

    def __init__(self, batch, n_pages, cache="bf16", device="cuda:0"):
        self.dev, self.w = torch.device(device), weights(device)
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)  # noqa: E731
        self.held, self.table = i32(batch), i32(batch, MAX_PAGES)
        self.free_ring = torch.arange(n_pages, dtype=torch.int32, device=device)
        self.ring = torch.tensor([0, n_pages], dtype=torch.int32, device=device)
        self.f8 = cache == "f8"
        self.cache_scale = 0.05 if self.f8 else 1.0
        self.layers = []
        for i in range(LAYERS):
            if i % 2 == 0:
                self.layers.append(torch.zeros((batch, SH, SP, SN), device=device))
            else:
                kv = torch.zeros((2, n_pages, PAGE, HK, HD), dtype=torch.bfloat16, device=device)
                self.layers.append(kv.to(torch.float8_e4m3fn) if self.f8 else kv)

    def step(self, hold, tokens, one_each):
        """Requests are to hold `hold` (batch,) int32 tokens: 0 ends one, and the grown ones'
        new tokens stand in `tokens` one request after the other (one_each: one of each
        request).  Returns the hidden states of the new tokens and the step's maps.  A prompt is
        a growth of many tokens.  A refused request (m["len"] is not what it was to hold) keeps its
        pages and its states, and the hidden states of its tokens mean nothing."""
        grown = self.held
        m = lib.ssm_kv_pages_step(self.held, hold, self.table, self.free_ring, self.ring, page_size=PAGE,
                                  n_tokens=len(tokens))
        self.held, self.ring = m["len"], m["ring"]
        request = m["request"].long()
        held = m["slots"] >= 0                                       # (not of a refused request)
        # a row of attention for each token; none of a refused one, whose further pages it does not have
        table, lens = self.table[request], torch.where(held, m["positions"] + 1, 0).int()
        x = self.w["embed"][tokens]
        for w, state in zip(self.w["layers"], self.layers):
            u = rms(x) @ w["in"].T
            x = x + (self.ssm(w, u, state, None if one_each else m["starts"].tolist(), grown, held) if "A_log" in w else
                     self.attention(w, u, state, m, table, lens)) @ w["out"].T
        return x, m

    def attention(self, w, u, kv, m, table, lens):
        u = u.to(torch.bfloat16)
        q, k, v = (t.unflatten(-1, (-1, HD)) for t in u.split([H * HD, HK * HD, HK * HD], -1))
        s = self.cache_scale
        q = lib.ssm_qk_norm_rope_cache_fwd(q, k, v, w["wq"], w["wk"], self.w["inv_freq"], m["positions"], m["slots"],
                                           kv[0], kv[1], eps=EPS, k_scale=s, v_scale=s)
        o = lib.ssm_paged_attn_decode_fwd(q, kv[0], kv[1], table, lens, scale=HD ** -0.5, k_scale=s, v_scale=s)
        return o.flatten(1).float()

    def ssm(self, w, u, state, starts, grown, held):
        """One call for all requests where each has one new token (starts is None), else a call
        for each of them.  A refused request's tokens are steps of no length, which leave its state as it is."""
        x, b, c, dt = split_ssm(u)
        dt = torch.where(held[:, None], dt, -1e4)       # softplus: 0
        scan = lambda s, h, t: lib.ssd_chunk_scan_fwd(  # noqa: E731
            x[s].view(h.shape[0], t, SH, SP), dt[s].view(-1, t, SH), w["dt_bias"], w["A_log"], b[s].view(-1, t, 1, SN),
            c[s].view(-1, t, 1, SN), w["D"], h, h_final=h)[0]
        n = len(u)
        if starts is None:
            state.mul_((grown > 0)[:, None, None, None])                    # a new request starts from zero
            return scan(slice(0, n), state, 1).flatten(1).view(n, -1)
        y = torch.empty((n, SH * SP), device=self.dev)
        for r in range(len(state)):
            lo, hi = starts[r], starts[r + 1]
            if hi > lo:
                h = state[r:r + 1].contiguous() * (grown[r] > 0)
                y[lo:hi] = scan(slice(lo, hi), h, hi - lo).view(hi - lo, -1)
                state[r] = h[0]
        return y


def recompute(w, tokens, cache_scale=None):
    """Hidden states of one request's tokens in fp64, with dense attention and the sequential
    recurrence; bf16 and 8-bit where the served path stores them."""
    bf = lambda t: t.to(torch.bfloat16).double()  # noqa: E731
    x = w["embed"][tokens].double()
    T = len(tokens)
    for lw in w["layers"]:
        u = rms(x) @ lw["in"].double().T
        if "A_log" in lw:
            xs, b, c, dt = u.split([SH * SP, SN, SN, SH], -1)
            xs, b, c = bf(xs).unflatten(-1, (SH, SP)), bf(b), bf(c)
            dt = torch.nn.functional.softplus(dt + lw["dt_bias"].double())
            h, ys = torch.zeros((SH, SP, SN), dtype=torch.float64, device=x.device), []
            for t in range(T):
                h = torch.exp(-dt[t] * lw["A_log"].double().exp())[:, None, None] * h \
                    + dt[t][:, None, None] * xs[t][:, :, None] * b[t]
                ys.append(h @ c[t] + lw["D"].double()[:, None] * xs[t])
            y = torch.stack(ys).flatten(1)
        else:
            q, k, v = (bf(t).unflatten(-1, (-1, HD)) for t in u.split([H * HD, HK * HD, HK * HD], -1))
            th = torch.arange(T, device=x.device).double()[:, None, None] * w["inv_freq"].double()

            def turned(t, weight):
                t = rms(t) * weight.double()
                a, z = t[..., :ROT // 2], t[..., ROT // 2:ROT]
                return bf(torch.cat([a * th.cos() - z * th.sin(), z * th.cos() + a * th.sin(), t[..., ROT:]], -1))

            q, k = turned(q, lw["wq"]), turned(k, lw["wk"])
            if cache_scale:
                k, v = ((t / cache_scale).float().to(torch.float8_e4m3fn).double() * cache_scale for t in (k, v))
            k, v = (t.repeat_interleave(H // HK, 1) for t in (k, v))
            s = torch.einsum("qhd,khd->hqk", q, k) * HD ** -0.5
            s = s.masked_fill(torch.ones((T, T), device=x.device).triu(1).bool(), -math.inf)
            y = torch.einsum("hqk,khd->qhd", s.softmax(-1), v).flatten(1)
        x = x + y @ lw["out"].double().T
    return x


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--cache", choices=("bf16", "f8"), default="bf16")
    ap.add_argument("--pages", type=int, default=20)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    batch = 4
    sv = Server(batch, n_pages=a.pages, cache=a.cache)
    g = torch.Generator().manual_seed(1)
    draw = lambda n: torch.randint(VOCAB, (n,), generator=g).tolist()  # noqa: E731
    said = [[] for _ in range(batch)]                    # what each place's request holds
    new = [draw(n) for n in (21, 1, 34, 16)]             # and what comes to it next: a prompt, or a token
    hidden = [[] for _ in range(batch)]
    worst = 0.0

    def check(r):
        got = torch.cat(hidden[r])
        want = recompute(sv.w, torch.tensor(said[r], device=sv.dev), sv.cache_scale if sv.f8 else None)
        return float((got.double() - want).norm() / want.norm())

    for step in range(a.steps + 1):
        hold = [len(s) + len(n) if n else 0 for s, n in zip(said, new)]          # nothing new: it ends
        x, m = sv.step(torch.tensor(hold, dtype=torch.int32, device=sv.dev),
                       torch.tensor([t for n in new for t in n], device=sv.dev), one_each=all(len(n) == 1 for n in new))
        # next: the likeliest token of each request (of a refused one, the same again); the second one
        # ends after five steps and its place goes to a new prompt the step after
        starts, held = m["starts"].tolist(), sv.held.tolist()
        logits = x @ sv.w["embed"].T
        for r, part in enumerate(x.split([len(n) for n in new])):
            if not new[r]:
                said[r], hidden[r], new[r] = [], [], draw(19)
            elif held[r] == hold[r]:
                said[r], hidden[r] = said[r] + new[r], hidden[r] + [part]
                new[r] = [int(logits[starts[r + 1] - 1].argmax())]
            if step == 5 and r == 1:
                if a.check and said[r]:
                    worst = max(worst, check(r))
                new[r] = []
        print(f"step {step}: {starts[-1]} new tokens, held {held}, free pages {int(sv.ring[1])}, "
              f"refused {int(m['denied'])}", flush=True)
    if a.check:
        worst = max([worst] + [check(r) for r in range(batch) if said[r]])
        print(f"hidden states served and recomputed in fp64 differ by {worst:.2e} of their norm")
    return worst


if __name__ == "__main__":
    main()
