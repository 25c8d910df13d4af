"""The operators for rotary models and models with capped scores, measured.

Five operators of a head-split layer, in their plain form (elementary torch
operations in fp32) and, with ``own`` set, through the package's entry points:

  rope      the rotary position embedding of queries and keys, one or several
            position axes, and its gradient (``rope_qk``);
  append    new tokens into both caches with the rotation of K and q applied
            on the way (``append_kv_rope``);
  decode    one new token per sequence, scores capped by a tanh, over
            contiguous, paged, 8- and 4-bit caches (``decode_attn_capped``);
  prefill   a chunk of prompt tokens, scores capped (``prefill_chunk_capped``);
  mix       a training step of the gated mix: the forward pass that keeps what
            the backward pass needs, then dq, dk, dv and dalpha
            (``gated_mix_train``, ``gated_mix_grad``).

``listed()`` gives the cases that are timed, ``draw(rng)`` more of the same
ranges, ``prepare(case, seed)`` a case's device state, ``run(state)`` one pass,
``exact(case, seed)`` the same outputs from the definitions in fp64, and
``work(case)`` the bytes and operations a pass cannot do without.
"""

import math

import torch

own = False

SINK, RECENT, PAGE = 16, 64, 64


# --------------------------------------------------------------------- cases

def listed():
    return [
        # q and k of one 4,096-token chunk at the end of a 128K prompt, rotated before its pre-fill
        dict(name="rope_prompt", op="rope", batch=1, hq=32, hkv=8, d=128, dtype="bf16", T=4096, rot=128, axes=1,
             layout="halves", inverse=False, start=126976, factor=1.0),
        # the gradient of q and k in a training step on image or video tokens: three axes, fp32, odd length,
        # part of each head rotated
        dict(name="rope_video_grad", op="rope", batch=2, hq=16, hkv=4, d=128, dtype="fp32", T=1021, rot=96, axes=3,
             layout="pairs", inverse=True, start=0, factor=1.0),
        # the append of one decode step: 64 sequences, paged caches (the smallest calls: latency counts)
        dict(name="append_step_b64_paged", op="append", batch=64, hq=32, hkv=32, r=8, d=128, dtype="bf16", T=1,
             rot=128, axes=1, layout="halves", paged=True, lo=200, hi=2000, capacity=2048, factor=1.0),
        # a chunk appended to a long contiguous cache, yarn-like factor on the angles' cosines
        dict(name="append_chunk_4k", op="append", batch=1, hq=32, hkv=8, r=4, d=128, dtype="bf16", T=4096, rot=128,
             axes=1, layout="halves", paged=False, lo=61440, hi=61440, capacity=65536, factor=1.2),
        # a ragged batch of short image prompts in fp32, head dimension 64, three axes, odd length
        dict(name="append_ragged_fp32", op="append", batch=3, hq=8, hkv=8, r=2, d=64, dtype="fp32", T=333, rot=64,
             axes=3, layout="halves", paged=False, lo=0, hi=700, capacity=1200, factor=1.0),
        # one token of one long sequence, grouped heads: the latency of a chat at 128K
        dict(name="decode_gqa_128k", op="decode", batch=1, hq=32, hkv=8, r=4, d=128, dtype="bf16", quant="none",
             paged=False, lo=131072, hi=131072, cap=50.0, gain=3.0),
        # a serving batch of uneven lengths over pages
        dict(name="decode_b64_paged", op="decode", batch=64, hq=32, hkv=32, r=8, d=128, dtype="bf16", quant="none",
             paged=True, lo=4096, hi=32768, cap=30.0, gain=3.0),
        # the smallest batch over a 4-bit cache
        dict(name="decode_gqa_32k_int4", op="decode", batch=1, hq=32, hkv=8, r=4, d=128, dtype="bf16", quant="int4",
             paged=False, lo=32711, hi=32711, cap=50.0, gain=3.0),
        # the last chunk of a 32K prompt
        dict(name="prefill_gqa_32k_last", op="prefill", batch=1, hq=32, hkv=8, r=4, d=128, dtype="bf16", c=4096,
             lo=28672, hi=28672, chunk_mode=False, cap=50.0, gain=3.0),
        # two short uneven prompts in fp32, head dimension 64, odd chunk
        dict(name="prefill_ragged_fp32", op="prefill", batch=2, hq=8, hkv=4, r=2, d=64, dtype="fp32", c=333, lo=77,
             hi=900, chunk_mode=False, cap=20.0, gain=3.0),
        # head identification on one 4,096-token sequence of a grouped layer, forward and backward
        dict(name="mix_step_gqa_4k", op="mix", batch=1, hq=32, hkv=8, d=128, dtype="bf16", n=4096, cap=50.0, gain=3.0),
        # the same on two short sequences in fp32, head dimension 64, odd length, without a cap
        dict(name="mix_step_fp32_odd", op="mix", batch=2, hq=8, hkv=8, d=64, dtype="fp32", n=509, cap=0.0, gain=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "prefill", "mix"])
    fast = rng.random() < 0.7                       # bf16 with head dimension 128, or the rest
    d = 128 if fast else rng.choice([64, 128])
    dtype = "bf16" if fast else rng.choice(["bf16", "fp32", "fp32"])
    hq, hkv = rng.choice([(32, 8), (32, 32), (16, 8), (8, 1), (8, 4), (8, 8)])
    heads = dict(hq=hq, hkv=hkv, d=d, dtype=dtype)
    rot = rng.choice([d, d, d // 2, 3 * d // 4])
    turn = dict(rot=rot, axes=rng.choice([1, 1, 3]), layout=rng.choice(["halves", "pairs"]),
                factor=rng.choice([1.0, 1.0, 1.2]))
    cap = rng.choice([20.0, 30.0, 50.0])
    gain = rng.choice([1.0, 3.0])
    if op == "rope":
        return dict(op=op, batch=rng.choice([1, 2, 3]), T=_log(rng, 1, 1365), inverse=rng.random() < 0.4,
                    start=_log(rng, 1, 1000000), **heads, **turn)
    if op == "append":
        batch, T = rng.choice([1, 2, 5, 16]), _log(rng, 1, 250)
        lo = rng.randint(0, 300)
        hi = rng.randint(lo, 1500)
        return dict(op=op, batch=batch, r=rng.randint(0, hkv), T=T, paged=rng.random() < 0.5, lo=lo, hi=hi,
                    capacity=-(-(hi + T) // PAGE) * PAGE, **heads, **turn)
    if op == "decode":
        batch = rng.choice([1, 1, 2, 8, 16])
        hi = _log(rng, 1, 131072 // batch)
        quant = rng.choice(["none", "none", "int8", "int4"]) if d == 128 and dtype == "bf16" else "none"
        return dict(op=op, batch=batch, r=rng.randint(1, min(8, hkv)), quant=quant,
                    paged=quant == "none" and rng.random() < 0.5, lo=rng.randint(1, hi), hi=hi, cap=cap, gain=gain,
                    **heads)
    if op == "prefill":
        c, batch = _log(rng, 1, 2048 if fast else 300), rng.choice([1, 1, 2])
        hi = _log(rng, 1, 16384 if fast else 1000)
        return dict(op=op, batch=batch, r=rng.randint(0, min(4, hkv)), c=c, lo=rng.randint(0, hi), hi=hi,
                    chunk_mode=rng.random() < 0.3, cap=cap, gain=gain, **heads)
    return dict(op=op, batch=rng.choice([1, 1, 2]), n=_log(rng, 1, 2048 if fast else 300),
                cap=rng.choice([0.0, cap]), gain=gain, **heads)


# ----------------------------------------------------------- what cases imply

def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _partition(c):
    """Retrieval KV heads spread over the layer; block order: retrieval heads, then streaming heads."""
    hkv, r = c["hkv"], c["r"]
    ret = sorted({(i * hkv) // r for i in range(r)}) if r else []
    return ret + [h for h in range(hkv) if h not in ret], r


def _lengths(c):
    b, lo, hi = c["batch"], c["lo"], c["hi"]
    return [lo + (hi - lo) * ((7 * i) % b) // max(b - 1, 1) for i in range(b)] if b > 1 else [hi]


def _sections(c):
    n = c["rot"] // 2
    return [n] if c["axes"] == 1 else [n // 4, 3 * n // 8, n - n // 4 - 3 * n // 8]


def _elem(c):
    return 2 if c["dtype"] == "bf16" else 4


def _lambda_pairs(n):
    w = SINK + RECENT
    return n * (n + 1) // 2 if n <= w else w * (w + 1) // 2 + (n - w) * w


def work(case):
    c, op, e = case, case["op"], _elem(case)
    B, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
    if op == "rope":
        n = B * c["T"]
        table = 2 * c["rot"] + 4 * (c["axes"] * n if c["axes"] > 1 else B)
        return dict(bytes=2 * n * (hq + hkv) * d * e + table, flops=3 * n * (hq + hkv) * c["rot"])
    if op == "append":
        n, r = B * c["T"], c["r"]
        new = sum(sum(1 for t in range(c["T"]) if L + t < SINK or t >= c["T"] - RECENT) for L in _lengths(c))
        written = 2 * (n * r + new * (hkv - r)) * d * e
        return dict(bytes=n * (2 * hq + 2 * hkv) * d * e + written, flops=3 * n * (hq + hkv) * c["rot"])
    if op == "decode":
        row = {"none": d * e, "int8": d + 4, "int4": d // 2 + 4}[c["quant"]]
        S, Ls = hkv - c["r"], _lengths(c)
        ring = sum(min(L, SINK + RECENT) for L in Ls)
        kept = 2 * (sum(Ls) * c["r"] * row + ring * S * d * e)
        return dict(bytes=kept + 2 * B * hq * d * e, flops=4 * d * (hq // hkv) * (sum(Ls) * c["r"] + ring * S))
    if op == "prefill":
        C, r, S, Ls = c["c"], c["r"], hkv - c["r"], _lengths(c)
        ring = [min(L, SINK + RECENT) for L in Ls]
        full = sum(C * L + C * (C + 1) // 2 for L in Ls)
        if c["chunk_mode"]:
            stream = sum(C * x + C * (C + 1) // 2 for x in ring)
        else:
            stream = sum(_lambda_pairs(L + C) - _lambda_pairs(L) for L in Ls)
        moved = B * C * (2 * hq + 2 * hkv) + 2 * (sum(Ls) * r + sum(ring) * S)
        return dict(bytes=moved * d * e, flops=4 * d * (hq // hkv) * (full * r + stream * S))
    n = c["n"]
    full, lam = n * (n + 1) // 2, _lambda_pairs(n)
    # forward: Q K^T and P V of the causal mask, P V of the sink and recent tokens; backward: five products
    flops = 2 * d * B * hq * (2 * full + lam + 5 * full)
    # q, k, v, dout in; out, dq, dk, dv out
    return dict(bytes=B * n * d * e * (4 * hq + 4 * hkv), flops=flops)


# --------------------------------------------------------------------- inputs

def _randn(g, shape, dtype, std=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(0.0, std, generator=g)


def _inv_freq(c):
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
    return torch.pow(500000.0, -2.0 * i / c["rot"]).float()


def _positions(c, g):
    """Positions of the tokens on three axes (time, height, width of 16 x 16 patches), or None: the cache's own."""
    if c["axes"] == 1:
        return None
    i = torch.arange(c["T"], device="cuda")
    base = torch.randint(0, 1000, (c["batch"], 1), generator=g, device="cuda") + c.get("start", 0)
    pos = torch.stack([base + i // 256, base + (i // 16) % 16, base + i % 16])
    return pos.to(torch.int32).contiguous()


def _caches(c, g, st, lengths, capacity):
    """Both caches of a layer that has taken `lengths` tokens."""
    B, r, d, dt = c["batch"], c["r"], c["d"], _dtype(c)
    S, W = c["hkv"] - r, SINK + RECENT
    quant, paged = c.get("quant", "none"), c.get("paged", False)
    st["page_table"] = None
    if quant == "int8":
        capacity = -(-capacity // 64) * 64
        st["k_full"] = _randn(g, (B, r, capacity, d), torch.float32, 40.0).round_().clamp_(-127, 127).to(torch.int8)
        st["v_full"] = _randn(g, (B, r, capacity // 64, d, 64), torch.float32, 40.0).round_().clamp_(-127, 127).to(torch.int8)
    elif quant == "int4":
        capacity = -(-capacity // 64) * 64
        nib = lambda shape: (_randn(g, shape, torch.float32, 2.6).round_().clamp_(-7, 7) + 8).to(torch.uint8)  # noqa: E731
        ks, vs = (B, r, capacity, 64), (B, r, capacity // 64, 4096)
        st["k_full"], st["v_full"] = nib(ks) | (nib(ks) << 4), nib(vs) | (nib(vs) << 4)
    elif paged:
        per = -(-capacity // PAGE)
        capacity = per * PAGE
        st["page_table"] = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
        st["k_full"] = _randn(g, (B * per, r, PAGE, d), dt)
        st["v_full"] = _randn(g, (B * per, r, PAGE, d), dt)
    else:
        st["k_full"] = _randn(g, (B, r, capacity, d), dt)
        st["v_full"] = _randn(g, (B, r, capacity, d), dt)
    st["k_scale"] = st["v_scale"] = None
    if quant != "none":
        step = 1.0 / (40.0 if quant == "int8" else 2.6)
        for name in ("k_scale", "v_scale"):
            st[name] = torch.empty((B, r, capacity), device="cuda").uniform_(0.5 * step, 1.5 * step, generator=g)
    st["capacity"] = capacity
    st["k_ring"], st["v_ring"] = _randn(g, (B, S, W, d), dt), _randn(g, (B, S, W, d), dt)
    L = torch.tensor(lengths, dtype=torch.int64, device="cuda")[:, None]
    st["ring_pos"] = _slot_positions(L).to(torch.int32).contiguous()
    st["seq_len"] = L[:, 0].to(torch.int32).contiguous()
    st["start_len"] = st["seq_len"].clone()


def _slot_positions(L):
    """The position that each ring slot holds after L tokens ([B, 1]); -1 where it holds none."""
    s = torch.arange(SINK + RECENT, device=L.device)[None, :]
    back = (L - 1 - s) % RECENT                      # slot s holds the last p < L with p = s modulo `recent`
    p = torch.where(s < SINK, s, L - 1 - back)
    return torch.where((p < L) & ((s < SINK) | (p >= SINK)), p, torch.full_like(p, -1))


def prepare(case, seed):
    c = dict(case)
    op, B, hq, hkv, d, dt = c["op"], c["batch"], c["hq"], c["hkv"], c["d"], _dtype(c)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    st = dict(case=c)
    gain = c.get("gain", 1.0)
    if op in ("rope", "append"):
        T = c["T"]
        st["q"], st["k"] = _randn(g, (B, T, hq, d), dt), _randn(g, (B, T, hkv, d), dt)
        st["q_out"] = torch.empty_like(st["q"])
        st["inv_freq"], st["pos"] = _inv_freq(c), _positions(c, g)
    if op == "rope":
        st["k_out"] = torch.empty_like(st["k"])
        st["seq_len"] = torch.full((B,), c["start"], dtype=torch.int32, device="cuda")
    elif op == "append":
        st["v"] = _randn(g, (B, c["T"], hkv, d), dt)
        _caches(c, g, st, _lengths(c), c["capacity"])
    elif op == "decode":
        st["q"] = _randn(g, (B, hq, d), dt, gain)
        st["out"] = torch.empty_like(st["q"])
        _caches(c, g, st, _lengths(c), c["hi"])
    elif op == "prefill":
        C = c["c"]
        st["q"], st["k"], st["v"] = _randn(g, (B, C, hq, d), dt, gain), _randn(g, (B, C, hkv, d), dt), _randn(g, (B, C, hkv, d), dt)
        st["out"] = torch.empty_like(st["q"])
        _caches(c, g, st, _lengths(c), max(c["hi"], 1))
    else:
        n = c["n"]
        st["q"], st["k"], st["v"] = _randn(g, (B, n, hq, d), dt, gain), _randn(g, (B, n, hkv, d), dt), _randn(g, (B, n, hkv, d), dt)
        st["dout"] = _randn(g, (B, n, hq, d), dt)
        st["alpha"] = torch.empty(hkv, device="cuda").uniform_(0.0, 1.0, generator=g)
        if hkv > 2:                                  # a gate at its start and a closed one
            st["alpha"][0], st["alpha"][-1] = 1.0, 0.0
        st["out"], st["dq"] = torch.empty_like(st["q"]), torch.empty_like(st["q"])
        st["dk"], st["dv"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
        st["dalpha"] = torch.empty_like(st["alpha"])
    if own:
        _handles(c, st)
    return st


def _handles(c, st):
    """The descriptors and workspaces that a program keeps."""
    from head_split_kv_b200 import duo
    st["duo"] = duo
    op, hkv = c["op"], c["hkv"]
    perm, r = _partition(c) if "r" in c else (list(range(hkv)), hkv)
    quant = {"none": duo.KV_PLAIN, "int8": duo.KV_INT8, "int4": duo.KV_INT4}[c.get("quant", "none")]
    desc = duo.desc_init(c["batch"], c["hq"], hkv, c["d"], duo.BF16 if c["dtype"] == "bf16" else duo.FP32, perm, r,
                         sink=SINK, recent=RECENT, page_size=PAGE if c.get("paged") else 0, kv_quant=quant,
                         stream_prefill=duo.STREAM_CHUNK if c.get("chunk_mode") else duo.STREAM_LAMBDA)
    st["desc"] = desc
    st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op in ("rope", "append"):
        st["rope"] = duo.rope_init(c["rot"], st["inv_freq"], sections=_sections(c), factor=c["factor"], pos=st["pos"],
                                   layout=duo.ROPE_HALVES if c["layout"] == "halves" else duo.ROPE_PAIRS)
    if op in ("append", "decode", "prefill"):
        st["counters"] = torch.zeros(duo.STATE_COUNTER_WORDS, dtype=torch.int32, device="cuda")
        ptr = lambda x: 0 if x is None else x.data_ptr()  # noqa: E731
        st["state"] = duo.KVState(
            k_full=ptr(st["k_full"]), v_full=ptr(st["v_full"]), page_table=ptr(st["page_table"]),
            capacity=st["capacity"], max_pages=st["capacity"] // PAGE if c.get("paged") else 0,
            n_pages=st["k_full"].shape[0] if c.get("paged") else 0, k_ring=ptr(st["k_ring"]), v_ring=ptr(st["v_ring"]),
            ring_pos=ptr(st["ring_pos"]), seq_len=ptr(st["seq_len"]), counters=ptr(st["counters"]),
            status=ptr(st["status"]), k_scale=ptr(st["k_scale"]), v_scale=ptr(st["v_scale"]))
    if op == "decode":
        st["ws"] = duo.Workspace(desc, duo.OP_DECODE, st["capacity"])
    elif op == "prefill":
        st["ws"] = duo.Workspace(desc, duo.OP_PREFILL, c["c"], state=st["state"])
    elif op == "mix":
        saved, work_bytes = duo.gated_mix_saved_bytes(desc, c["n"]), duo.gated_mix_grad_workspace_bytes(desc, c["n"])
        st["saved"] = torch.empty(max(saved, 16), dtype=torch.uint8, device="cuda")
        st["grad_ws"] = torch.empty(max(work_bytes, 16), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------------ run

def run(st):
    op = st["case"]["op"]
    if own:
        return _RUN_OWN[op](st["duo"], st["case"], st)
    return _RUN_PLAIN[op](st["case"], st)


def _own_rope(duo, c, st):
    duo.rope_qk(st["desc"], st["rope"], st["q"], st["k"], st["q_out"], st["k_out"], c["T"], seq_len=st["seq_len"],
                inverse=c["inverse"])
    return dict(q=st["q_out"], k=st["k_out"])


def _own_append(duo, c, st):
    st["seq_len"].copy_(st["start_len"])             # so that every pass appends the same tokens
    duo.append_kv_rope(st["desc"], st["state"], st["rope"], st["q"], st["k"], st["v"], st["q_out"], c["T"])
    return _append_outputs(st)


def _own_decode(duo, c, st):
    duo.decode_attn_capped(st["desc"], st["state"], c["cap"], st["q"], st["out"], st["ws"].ptr, st["ws"].nbytes)
    return st["out"]


def _own_prefill(duo, c, st):
    duo.prefill_chunk_capped(st["desc"], st["state"], c["cap"], st["q"], st["k"], st["v"], c["c"], st["out"],
                             st["ws"].ptr, st["ws"].nbytes)
    return st["out"]


def _own_mix(duo, c, st):
    duo.gated_mix_train(st["desc"], st["alpha"], c["cap"], st["q"], st["k"], st["v"], c["n"], st["out"], st["saved"],
                        st["saved"].numel(), st["status"])
    duo.gated_mix_grad(st["desc"], st["alpha"], c["cap"], st["q"], st["k"], st["v"], c["n"], st["saved"],
                       st["saved"].numel(), st["dout"], st["dq"], st["dk"], st["dv"], st["dalpha"], st["grad_ws"],
                       st["grad_ws"].numel(), st["status"])
    # the gates' gradient comes in fp32; an optimiser takes every gradient in the layer's type
    return {**{k: st[k] for k in ("out", "dq", "dk", "dv")}, "dalpha": st["dalpha"].to(_dtype(c))}


def _append_outputs(st):
    return {k: st[k] for k in ("q_out", "k_full", "v_full", "k_ring", "v_ring", "ring_pos", "seq_len")}


# ---- plain forms

def _token_positions(c, st):
    """[axes, B, T] int64."""
    if st["pos"] is not None:
        return st["pos"].long()
    return (st["seq_len"].long()[:, None] + torch.arange(c["T"], device="cuda")[None, :])[None]


def _axis_of_pair(c):
    """The axis that turns each pair of channels."""
    i, s = torch.arange(c["rot"] // 2, device="cuda"), _sections(c)
    return (i >= s[0]).long() + (i >= s[0] + s[1]).long() if c["axes"] > 1 else torch.zeros_like(i)


def _cos_sin(c, st):
    """cos and sin of every (sequence, token, pair), the angles in fp64: [B, T, 1, rot / 2] fp32."""
    pos = _token_positions(c, st)[_axis_of_pair(c)].permute(1, 2, 0)          # [B, T, rot / 2]
    ang = pos.double() * st["inv_freq"].double()
    return torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]


def _rotate(c, x, cos, sin):
    rot, f = c["rot"], c["factor"]
    sin = -sin if c.get("inverse") else sin
    y = x.float().clone()
    if c["layout"] == "halves":
        a, b = y[..., : rot // 2].clone(), y[..., rot // 2: rot].clone()
        y[..., : rot // 2], y[..., rot // 2: rot] = (a * cos - b * sin) * f, (b * cos + a * sin) * f
    else:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = (a * cos - b * sin) * f, (b * cos + a * sin) * f
    return y.to(x.dtype)


def _plain_rope(c, st):
    cos, sin = _cos_sin(c, st)
    return dict(q=_rotate(c, st["q"], cos, sin), k=_rotate(c, st["k"], cos, sin))


def _plain_append(c, st):
    st["seq_len"].copy_(st["start_len"])
    B, T, r = c["batch"], c["T"], c["r"]
    cos, sin = _cos_sin(c, st)
    st["q_out"] = _rotate(c, st["q"], cos, sin)
    perm = torch.tensor(_partition(c)[0], device="cuda")
    k, v = _rotate(c, st["k"], cos, sin)[:, :, perm], st["v"][:, :, perm]      # block order
    L = st["seq_len"].long()[:, None]
    p = L + torch.arange(T, device="cuda")                                     # [B, T] cache positions
    seq = torch.arange(B, device="cuda")[:, None].expand(B, T)
    for_full, for_ring = (lambda x: x[:, :, :r]), (lambda x: x[:, :, r:])
    if st["page_table"] is None:
        st["k_full"][seq, :, p], st["v_full"][seq, :, p] = for_full(k), for_full(v)
    else:
        page = st["page_table"].long()[seq, p // PAGE]
        st["k_full"][page, :, p % PAGE], st["v_full"][page, :, p % PAGE] = for_full(k), for_full(v)
    held = _slot_positions(L + T)                                              # [B, W]
    t = held - L
    new = (t >= 0)
    rows = torch.arange(B, device="cuda")[:, None]
    pick = t.clamp(0, T - 1)
    put = lambda ring, x: torch.where(new[:, None, :, None], for_ring(x)[rows, pick].transpose(1, 2), ring)  # noqa: E731
    st["k_ring"].copy_(put(st["k_ring"], k))
    st["v_ring"].copy_(put(st["v_ring"], v))
    st["ring_pos"].copy_(held)
    st["seq_len"].add_(T)
    return _append_outputs(st)


def _int4_places():
    """Byte and nibble of every feature of a K row, and of every (token, feature) of a 64-token V tile."""
    f = torch.arange(128, device="cuda")
    e = f % 8                                         # byte c of a word holds features (0, 2), (4, 6), (1, 3), (5, 7)
    k_byte = 16 * (f // 32) + 4 * ((f % 32) // 8) + 2 * (e % 2) + e // 4
    k_high = (e // 2) % 2
    t = torch.arange(64, device="cuda")[:, None]
    v_byte = 1024 * (t // 16) + 128 * (f // 16) + 16 * (f % 8) + 4 * ((t % 8) // 2) + 2 * (t % 2) + (t % 16) // 8
    v_high = ((f % 16) // 8).expand(64, 128)
    return k_byte, k_high, v_byte, v_high


def _cached_rows(c, st, n):
    """The first n rows of the full cache as fp32 [B, r, n, d]."""
    kf, vf, B, r, d = st["k_full"], st["v_full"], c["batch"], c["r"], c["d"]
    quant = c.get("quant", "none")
    if quant == "int8":
        t = torch.arange(64, device="cuda")
        # tokens of a 16-group in the order 0 1 8 9 2 3 10 11 4 5 12 13 6 7 14 15
        col = t // 16 * 16 + ((t % 8) // 2) * 4 + ((t % 16) // 8) * 2 + t % 2
        k, v = kf.float(), vf[..., col].float().transpose(-1, -2).reshape(B, r, -1, d)
    elif quant == "int4":
        kb, kh, vb, vh = _int4_places()
        k = ((kf[..., kb].int() >> (4 * kh)) & 15).float() - 8.0
        v = ((vf[..., vb.reshape(-1)].int() >> (4 * vh.reshape(-1))) & 15).float() - 8.0
        v = v.view(B, r, -1, d)
    elif st["page_table"] is not None:
        pages = st["page_table"].long()[:, : -(-n // PAGE)]
        rows = lambda x: x[pages].transpose(1, 2).reshape(B, r, -1, d)  # noqa: E731
        k, v = rows(kf).float(), rows(vf).float()
    else:
        k, v = kf[:, :, :n].float(), vf[:, :, :n].float()
    k, v = k[:, :, :n], v[:, :, :n]
    if quant != "none":
        k, v = k * st["k_scale"][:, :, :n, None], v * st["v_scale"][:, :, :n, None]
    return k, v


def _capped(s, cap):
    return cap * torch.tanh(s / cap) if cap else s


def _attend(q, k, v, seen, cap, scale):
    """q [B, H, G, n, d], k and v [B, H, m, d], seen [B, 1, 1, n, m]: softmax over what is seen; an empty row is 0."""
    s = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).view(*q.shape[:4], -1) * scale
    s = _capped(s, cap).masked_fill_(~seen, -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
    total = s.sum(-1, keepdim=True)
    out = torch.matmul(s.flatten(2, 3), v).view(q.shape)
    return out / torch.where(total > 0, total, torch.ones_like(total))


def _to_model_order(c, ret, stream):
    """[B, r, G, n, d] and [B, S, G, n, d] in block order -> [B, n, Hq, d] in model order."""
    perm = torch.tensor(_partition(c)[0], device="cuda")
    both = torch.cat([ret, stream], 1)[:, torch.argsort(perm)]                 # [B, Hkv, G, n, d]
    return both.flatten(1, 2).transpose(1, 2).to(_dtype(c))


def _plain_decode(c, st):
    B, r, d, hkv = c["batch"], c["r"], c["d"], c["hkv"]
    scale, n = 1.0 / math.sqrt(d), c["hi"]
    perm = torch.tensor(_partition(c)[0], device="cuda")
    q = st["q"].float().view(B, hkv, -1, 1, d)[:, perm]
    L = st["seq_len"].long()
    k, v = _cached_rows(c, st, n)
    seen = torch.arange(n, device="cuda")[None, :] < L[:, None]
    ret = _attend(q[:, :r], k, v, seen[:, None, None, None], c["cap"], scale)
    held = (st["ring_pos"] >= 0)[:, None, None, None]
    stream = _attend(q[:, r:], st["k_ring"].float(), st["v_ring"].float(), held, c["cap"], scale)
    return _to_model_order(c, ret, stream)[:, 0]


def _plain_prefill(c, st):
    B, r, d, hkv, C = c["batch"], c["r"], c["d"], c["hkv"], c["c"]
    scale, n = 1.0 / math.sqrt(d), c["hi"]
    perm = torch.tensor(_partition(c)[0], device="cuda")
    q = st["q"].float().view(B, C, hkv, -1, d).permute(0, 2, 3, 1, 4)[:, perm]
    kx, vx = (st[x].float().transpose(1, 2)[:, perm] for x in ("k", "v"))
    L = st["seq_len"].long()[:, None]
    i = torch.arange(C, device="cuda")
    k, v = _cached_rows(c, st, n)
    key = torch.cat([torch.arange(n, device="cuda").expand(B, n), L + i], 1)   # [B, n + C] positions
    real = torch.cat([torch.arange(n, device="cuda") < L, torch.ones(B, C, dtype=torch.bool, device="cuda")], 1)
    P = (L + i)[:, :, None]                                                    # [B, C, 1] query positions
    seen = real[:, None] & (key[:, None] <= P)
    ret = _attend(q[:, :r], torch.cat([k, kx[:, :r]], 2), torch.cat([v, vx[:, :r]], 2), seen[:, None, None], c["cap"], scale)
    key = torch.cat([st["ring_pos"].long(), L + i], 1)
    near = key[:, None] >= (L - RECENT)[:, None] if c["chunk_mode"] else P - key[:, None] < RECENT
    seen = (key >= 0)[:, None] & (key[:, None] <= P) & ((key[:, None] < SINK) | near)
    stream = _attend(q[:, r:], torch.cat([st["k_ring"].float(), kx[:, r:]], 2), torch.cat([st["v_ring"].float(), vx[:, r:]], 2),
                     seen[:, None, None], c["cap"], scale)
    return _to_model_order(c, ret, stream)


def _plain_mix(c, st):
    B, d, hq, hkv, n, cap = c["batch"], c["d"], c["hq"], c["hkv"], c["n"], c["cap"]
    scale, G = 1.0 / math.sqrt(d), hq // hkv
    q, do = (st[x].float().transpose(1, 2) for x in ("q", "dout"))             # [B, Hq, n, d]
    k, v = (st[x].float().transpose(1, 2).repeat_interleave(G, 1) for x in ("k", "v"))
    a = st["alpha"].repeat_interleave(G)[None, :, None, None]
    i = torch.arange(n, device="cuda")
    causal = i[:, None] >= i[None, :]
    lam = causal & ((i[None, :] < SINK) | (i[:, None] - i[None, :] < RECENT))
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    slope = None
    if cap:
        t = torch.tanh(s.div_(cap))
        s, slope = t * cap, 1.0 - t * t
    pc = torch.softmax(s.masked_fill(~causal, -math.inf), -1)
    ps = torch.softmax(s.masked_fill_(~lam, -math.inf), -1)
    oc, os_ = torch.matmul(pc, v), torch.matmul(ps, v)
    out = a * oc + (1.0 - a) * os_
    dc, ds = (do * oc).sum(-1, keepdim=True), (do * os_).sum(-1, keepdim=True)
    dalpha = (dc - ds).view(B, hkv, G, n).sum((0, 2, 3))
    pc, ps = pc.mul_(a), ps.mul_(1.0 - a)
    dv = torch.matmul((pc + ps).transpose(-1, -2), do)
    dp = torch.matmul(do, v.transpose(-1, -2))
    g = pc.mul_(dp - dc).add_(ps.mul_(dp.sub_(ds)))
    g = (g * slope if cap else g).mul_(scale)
    dq, dk = torch.matmul(g, k), torch.matmul(g.transpose(-1, -2), q)
    rows = lambda x: x.transpose(1, 2).contiguous().to(_dtype(c))  # noqa: E731
    group = lambda x: rows(x.view(B, hkv, G, n, d).sum(2))  # noqa: E731
    return dict(out=rows(out), dq=rows(dq), dk=group(dk), dv=group(dv), dalpha=dalpha.to(_dtype(c)))


_RUN_PLAIN = dict(rope=_plain_rope, append=_plain_append, decode=_plain_decode, prefill=_plain_prefill, mix=_plain_mix)
_RUN_OWN = dict(rope=_own_rope, append=_own_append, decode=_own_decode, prefill=_own_prefill, mix=_own_mix)


# ---------------------------------------------------------------------- exact

def exact(case, seed):
    """run()'s outputs from the definitions in fp64, head by head."""
    c, st = dict(case), prepare(case, seed)
    with torch.no_grad():
        return _EXACT[c["op"]](c, st)


def _turned(c, st, x, sign):
    """Each pair of channels as a complex number times factor * e^(i angle), fp64."""
    rot, T = c["rot"], c["T"]
    which = [a for a, n in enumerate(_sections(c)) for _ in range(n)]
    if st["pos"] is None:
        pos = torch.stack([st["seq_len"].double() + t for t in range(T)], 1)[..., None].expand(-1, -1, rot // 2)
    else:
        pos = torch.stack([st["pos"][a].double() for a in which], -1)
    turn = torch.polar(torch.full_like(pos, c["factor"]), sign * pos * st["inv_freq"].double())[:, :, None]
    y = x.double().clone()
    if c["layout"] == "halves":
        z = torch.complex(y[..., : rot // 2], y[..., rot // 2: rot]) * turn
        y[..., :rot] = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2).contiguous()) * turn
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    return y


def _exact_rope(c, st):
    sign = -1.0 if c["inverse"] else 1.0
    return dict(q=_turned(c, st, st["q"], sign), k=_turned(c, st, st["k"], sign))


def _exact_append(c, st):
    q, k, T = _turned(c, st, st["q"], 1.0), _turned(c, st, st["k"], 1.0), c["T"]
    perm, r = _partition(c)
    full = [st["k_full"].double(), st["v_full"].double()]
    ring = [st["k_ring"].double(), st["v_ring"].double()]
    ring_pos = st["ring_pos"].clone()
    for b, L in enumerate(_lengths(c)):
        p = torch.arange(L, L + T, device="cuda")
        keep = [t for t in range(T) if L + t < SINK or t >= T - RECENT]
        slots = [L + t if L + t < SINK else SINK + (L + t - SINK) % RECENT for t in keep]
        slot, kept = torch.tensor(slots, device="cuda"), torch.tensor(keep, device="cuda")
        ring_pos[b, slot] = (L + kept).to(torch.int32)
        for i, x in enumerate((k[b], st["v"][b].double())):
            for s, h in enumerate(perm):
                if s >= r:
                    ring[i][b, s - r, slot] = x[kept, h]
                elif st["page_table"] is None:
                    full[i][b, s, p] = x[:, h]
                else:
                    full[i][st["page_table"][b].long()[p // PAGE], s, p % PAGE] = x[:, h]
    seq_len = st["start_len"] + T
    return dict(q_out=q, k_full=full[0], v_full=full[1], k_ring=ring[0], v_ring=ring[1], ring_pos=ring_pos, seq_len=seq_len)


def _exact_heads(q, k, v, seen, cap, scale):
    """q [n, d], k and v [m, d] in fp64; seen [n, m] or None."""
    s = (q @ k.T) * scale
    s = torch.tanh(s / cap) * cap if cap else s
    if seen is not None:
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
    w = torch.exp(s - torch.logsumexp(s, -1, keepdim=True))
    return w @ v, w


def _exact_cached(c, st, b, s, n):
    """Rows 0..n-1 of sequence b, retrieval slot s, in fp64."""
    if c.get("quant", "none") == "none":
        if st["page_table"] is None:
            return st["k_full"][b, s, :n].double(), st["v_full"][b, s, :n].double()
        at = torch.arange(n, device="cuda")
        page = st["page_table"][b].long()[at // PAGE]
        return st["k_full"][page, s, at % PAGE].double(), st["v_full"][page, s, at % PAGE].double()
    t, f = torch.arange(n, device="cuda"), torch.arange(128, device="cuda")
    if c["quant"] == "int8":
        order = torch.tensor([0, 1, 8, 9, 2, 3, 10, 11, 4, 5, 12, 13, 6, 7, 14, 15], device="cuda")
        col = (t % 64) // 16 * 16 + torch.argsort(order)[t % 16]
        k, v = st["k_full"][b, s, :n].double(), st["v_full"][b, s][t // 64, :, col].double()
    else:
        pair = torch.tensor([0, 2, 0, 2, 1, 3, 1, 3], device="cuda")           # byte of each of 8 features
        high = torch.tensor([0, 0, 1, 1, 0, 0, 1, 1], device="cuda")
        raw = st["k_full"][b, s, :n].long()[:, f // 8 * 4 + pair[f % 8]]
        k = (torch.where(high[f % 8] == 1, raw // 16, raw % 16) - 8).double()
        u = t % 64
        at = (1024 * (u // 16) + 4 * (u % 8 // 2) + u % 2 * 2 + u % 16 // 8)[:, None] + (128 * (f // 16) + 16 * (f % 8))[None]
        raw = st["v_full"][b, s].long()[(t // 64)[:, None], at]
        v = (torch.where((f % 16 >= 8)[None], raw // 16, raw % 16) - 8).double()
    return k * st["k_scale"][b, s, :n, None].double(), v * st["v_scale"][b, s, :n, None].double()


def _exact_decode(c, st):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    (perm, r), G, scale = _partition(c), c["hq"] // c["hkv"], c["d"] ** -0.5
    for b, L in enumerate(_lengths(c)):
        for s, h in enumerate(perm):
            if s < r:
                k, v = _exact_cached(c, st, b, s, L)
            else:
                n = min(L, SINK + RECENT)                                      # every slot below is held
                k, v = st["k_ring"][b, s - r, :n].double(), st["v_ring"][b, s - r, :n].double()
            out[b, h * G: h * G + G] = _exact_heads(st["q"][b, h * G: h * G + G].double(), k, v, None, c["cap"], scale)[0]
    return out


def _exact_prefill(c, st):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    (perm, r), G, scale, C = _partition(c), c["hq"] // c["hkv"], c["d"] ** -0.5, c["c"]
    for b, L in enumerate(_lengths(c)):
        P = torch.arange(L, L + C, device="cuda")[:, None]
        for s, h in enumerate(perm):
            kx, vx = st["k"][b, :, h].double(), st["v"][b, :, h].double()
            if s < r:
                k, v = _exact_cached(c, st, b, s, L)
                key = torch.arange(L + C, device="cuda")[None]
                seen = key <= P
            else:
                n = min(L, SINK + RECENT)
                k, v = st["k_ring"][b, s - r, :n].double(), st["v_ring"][b, s - r, :n].double()
                key = torch.cat([st["ring_pos"][b, :n].long(), P[:, 0]])[None]
                old = (L if c["chunk_mode"] else P + 1) - RECENT               # the oldest token that is recent
                seen = (key <= P) & ((key < SINK) | (key >= old))
            k, v = torch.cat([k, kx]), torch.cat([v, vx])
            for g in range(h * G, h * G + G):
                out[b, :, g] = _exact_heads(st["q"][b, :, g].double(), k, v, seen, c["cap"], scale)[0]
    return out


def _exact_mix(c, st):
    G, n, cap, scale = c["hq"] // c["hkv"], c["n"], c["cap"], c["d"] ** -0.5
    i = torch.arange(n, device="cuda")
    masks = [i[:, None] >= i[None]]
    masks.append(masks[0] & ((i < SINK)[None] | (i[:, None] - i[None] < RECENT)))
    out, dq = (torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    dk, dv = (torch.zeros(st["k"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    dalpha = torch.zeros(c["hkv"], dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        for h in range(c["hq"]):
            j = h // G
            q, do = st["q"][b, :, h].double(), st["dout"][b, :, h].double()
            k, v = st["k"][b, :, j].double(), st["v"][b, :, j].double()
            a = st["alpha"][j].double()
            dp = do @ v.T
            grad = torch.zeros(n, n, dtype=torch.float64, device="cuda")
            for seen, share, sign in ((masks[0], a, 1.0), (masks[1], 1.0 - a, -1.0)):
                o, w = _exact_heads(q, k, v, seen, cap, scale)
                out[b, :, h] += share * o
                dalpha[j] += sign * (do * o).sum()
                dv[b, :, j] += share * (w.T @ do)
                grad += share * w * (dp - (w * dp).sum(-1, keepdim=True))
            if cap:
                grad *= 1.0 - torch.tanh((q @ k.T) * scale / cap) ** 2
            dq[b, :, h] = grad @ k * scale
            dk[b, :, j] += grad.T @ q * scale
    return dict(out=out, dq=dq, dk=dk, dv=dv, dalpha=dalpha)


_EXACT = dict(rope=_exact_rope, append=_exact_append, decode=_exact_decode, prefill=_exact_prefill, mix=_exact_mix)
