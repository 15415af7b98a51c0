"""Cases that measure the operators of the 8-bit paged cache and of its bounded special stream.

Four operators, each with a plain form in elementary torch operations:

* ``append``   a frame's K/V rows stored as e4m3 codes with one power-of-two scale per
               (token, head): every block of the model, then the frame is rolled back, so
               that the next pass takes the same slots.
* ``attend``   softmax(q K^T / sqrt(D)) V over the visible keys of such a cache, for one
               query row, a frame of them or several frames of them.
* ``weigh``    the attention weight that each special token received from the query rows,
               summed over rows and heads and added to a running total (a second pass over
               K with the rows' log-sum-exps).
* ``evict``    one frame-step of a special stream held at a fixed budget: the frame is
               appended to every block and the special tokens of least weight leave, their
               slots filled by the survivors from behind the budget.

``prepare`` draws K, V and q from the seed.  The plain form keeps what the cache would hold
(codes and scales); the framework's form keeps a cache that took the same frames.
"""
from __future__ import annotations

import math

import torch

own = False

HEADROOM = 16
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # append: one frame of a 16-head stream through its 24 blocks, and the largest frame
        dict(name="append_frame", op="append", L=24, B=1, H=16, D=64, P=256, S=6, ps=256),
        dict(name="append_high_res", op="append", L=24, B=1, H=16, D=64, P=999, S=6, ps=1024),
        dict(name="append_streams_d128", op="append", L=12, B=4, H=8, D=128, P=256, S=6, ps=256),
        # attend: a small stream whose call is all latency; one row and the six special rows over
        # the cache of a 10,000-frame stream; a frame over it; a large frame; four streams
        dict(name="attend_small", op="attend", B=1, H=4, D=64, P=16, S=2, ps=16, sc=2, w=4, frames=12, rows=18, lse=True),
        dict(name="attend_one_row_10k", op="attend", B=1, H=16, D=64, P=256, S=6, ps=256, sc=8, w=64, frames=10000,
             rows=1, lse=False),
        dict(name="attend_frame_10k", op="attend", B=1, H=16, D=64, P=256, S=6, ps=256, sc=8, w=64, frames=10000,
             rows=262, lse=False),
        dict(name="attend_high_res", op="attend", B=1, H=16, D=64, P=999, S=6, ps=1024, sc=8, w=32, frames=2000,
             rows=1005, lse=True),
        dict(name="attend_streams_d128", op="attend", B=4, H=8, D=128, P=256, S=6, ps=256, sc=4, w=128, frames=5000,
             rows=262, lse=False),
        # weigh: the special tokens of 200 frames, and of 10,000 frames
        dict(name="weigh_200_bf16", op="weigh", cache="bf16", B=1, H=16, D=64, P=256, S=6, ps=256, sc=8, w=64,
             frames=200, rows=262),
        dict(name="weigh_10k", op="weigh", cache="e4m3", B=1, H=16, D=64, P=256, S=6, ps=256, sc=8, w=64,
             frames=10000, rows=262),
        # evict: budgets of 200 and of 5,000 frames' special tokens, 24 blocks
        dict(name="evict_1200_bf16", op="evict", cache="bf16", L=24, H=16, D=64, P=256, S=6, ps=256, keep=1200, recent=16),
        dict(name="evict_30000", op="evict", cache="e4m3", L=24, H=16, D=64, P=256, S=6, ps=256, keep=30000, recent=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "weigh", "evict"])
    D = rng.choice([64, 128])
    H = rng.choice([1, 2, 3, 4, 8, 12, 16]) if D == 64 else rng.choice([1, 2, 4, 5, 8])
    P = _log_int(rng, 1, 999)
    S = _log_int(rng, 1, 32)
    ps = max(P, S, rng.choice([16, 64, 100, 256, 512, 1000]))
    if op == "append":
        return dict(op=op, L=rng.randint(1, 24), B=rng.randint(1, 4), H=H, D=D, P=P, S=S, ps=ps)
    if op == "evict":
        S = _log_int(rng, 1, 16)
        frames = _log_int(rng, 40, 2000)
        return dict(op=op, cache=rng.choice(["e4m3", "e4m3", "bf16", "f32"]), L=rng.randint(1, 16), H=H, D=D, P=P, S=S,
                    ps=ps, keep=S * frames, recent=rng.randint(1, 32))
    B = rng.randint(1, 4)
    sc, w = rng.randint(0, 8), rng.randint(1, 40)
    frames = _log_int(rng, 1, 3000)
    rows = min(rng.choice([1, 2, S, P + S, _log_int(rng, 1, 1005)]), 64 * (P + S))
    # no dearer than the largest listed case: query rows x visible keys x heads x dims, all streams
    while B * rows * _visible(P, S, sc, w, frames) * H * D > 4.5e10:
        frames = max(1, frames // 2)
        rows = max(1, rows // 2)
    if op == "attend":
        return dict(op=op, B=B, H=H, D=D, P=P, S=S, ps=ps, sc=sc, w=w, frames=frames, rows=rows, lse=rng.random() < 0.5)
    return dict(op=op, cache=rng.choice(["e4m3", "e4m3", "bf16", "f32"]), B=B, H=H, D=D, P=P, S=S, ps=ps, sc=sc, w=w,
                frames=frames, rows=rows)


def _visible(P, S, sc, w, frames):
    return P * min(frames, sc + w) + S * frames


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=None, dtype=torch.bfloat16):
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16)
    return (x if scale is None else x * scale).to(dtype)


def _head_scale(g, *shape):
    """A scale of its own for each head (last axis but one), as trained heads have."""
    return (torch.rand(*shape, 1, generator=g, device="cuda") * 1.25 + 0.5).to(torch.bfloat16)


def _stream_inputs(c, seed):
    """K/V of the visible patch rows [B, frames kept, P, H, D], of every special row
    [B, frames * S, H, D], and the query rows [B * rows, H, D]."""
    g = _gen(seed)
    B, H, D, P, S = c["B"], c["H"], c["D"], c["P"], c["S"]
    dtype = torch.float32 if c.get("cache") == "f32" else torch.bfloat16
    kept = min(c["frames"], c["sc"] + c["w"])
    hs = _head_scale(g, 3, 1, 1, H)
    return dict(kp=_randn(g, B, kept, P, H, D, scale=hs[0], dtype=dtype), vp=_randn(g, B, kept, P, H, D, scale=hs[1], dtype=dtype),
                ks=_randn(g, B, c["frames"] * S, H, D, scale=hs[0][0], dtype=dtype),
                vs=_randn(g, B, c["frames"] * S, H, D, scale=hs[1][0], dtype=dtype),
                q=_randn(g, B * c["rows"], H, D, scale=hs[2][0], dtype=dtype))


def _visible_kv(x):
    """[B, N, H, D] of K and of V: patch rows of the frames kept, then the special rows."""
    B, H, D = x["ks"].shape[0], x["ks"].shape[2], x["ks"].shape[3]
    return (torch.cat([x["kp"].reshape(B, -1, H, D), x["ks"]], 1), torch.cat([x["vp"].reshape(B, -1, H, D), x["vs"]], 1))


# ---------------------------------------------------------------- plain forms

def _quantise(x):
    """e4m3 codes of rows [..., D] and their scale bytes [...]: the smallest power of two s with
    amax / s <= 448 (byte b stands for 2^(b - 127); 0 for a row of zeros), code = x / s rounded once."""
    y = x.float()
    amax = y.abs().amax(-1)
    f, e = torch.frexp(amax)
    b = torch.where(amax > 0, (e - 9 + (f > 0.875).int() + 127).clamp(0, 254), torch.zeros_like(e))
    codes = torch.ldexp(y, (127 - b).unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, b.to(torch.uint8)


def _dequantise(codes, b):
    return torch.ldexp(codes.float(), (b.int() - 127).unsqueeze(-1))


def _attend(q, k, v, scale):
    """out [B, R, H, D] and lse [B, R, H] of softmax(q k^T scale) v; k, v [B, N, H, D], 32 bits."""
    s = torch.matmul(q.permute(0, 2, 1, 3), k.permute(0, 2, 3, 1)).mul_(scale)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)).div_(total)
    return o.permute(0, 2, 1, 3), (m + total.log()).squeeze(-1).permute(0, 2, 1)


def _weigh(q, k, lse, scale):
    """Sum over rows and heads of exp(q k^T scale - lse): [B, n]; q [B, R, H, D], k [B, n, H, D], lse [B, R, H]."""
    s = torch.matmul(q.permute(0, 2, 1, 3), k.permute(0, 2, 3, 1)).mul_(scale)
    return s.sub_(lse.permute(0, 2, 1).unsqueeze(-1)).exp_().sum((1, 2))


def _plain_append(st):
    P = st["case"]["P"]
    codes, b = _quantise(torch.stack([st["k"], st["v"]], 2))      # [L, B, 2, T, H, D]
    b = b.transpose(-1, -2)                                       # scales lie [H][token]
    return [x.unbind(1) for x in (codes[:, :, :, :P], b[..., :P], codes[:, :, :, P:], b[..., P:])]


def _plain_attend(st):
    c = st["case"]
    k, v = _dequantise(st["k"], st["kb"]), _dequantise(st["v"], st["vb"])
    q = st["q"].float().view(c["B"], c["rows"], c["H"], c["D"])
    o, lse = _attend(q, k, v, 1 / math.sqrt(c["D"]))
    o = o.reshape(st["q"].shape).to(torch.bfloat16)
    return [o, lse.reshape(-1, c["H"])] if c["lse"] else o


def _plain_weigh(st):
    c = st["case"]
    k = _dequantise(st["k"], st["kb"]) if c["cache"] == "e4m3" else st["k"].float()
    q = st["q"].float().view(c["B"], c["rows"], c["H"], c["D"])
    st["weights"] += _weigh(q, k, st["lse"].view(c["B"], c["rows"], c["H"]), 1 / math.sqrt(c["D"]))
    return st["weights"]


def _plain_evict(st):
    c = st["case"]
    P, S, ps, keep = c["P"], c["S"], c["ps"], c["keep"]
    n, arrived = keep + S, st["frames"] * S
    st["frames"] += 1
    kv = torch.stack([st["k"], st["v"]], 1)                     # [L, 2, T, H, D]
    if c["cache"] == "e4m3":
        kv, b = _quantise(kv)
        st["patch_scales"] = b[:, :, :P].transpose(-1, -2).contiguous()
    st["patch"] = kv[:, :, :P].contiguous()
    at = st["iota"][keep:n]
    raw, kv = (st["pool"].view(torch.uint8), kv.view(torch.uint8)) if c["cache"] == "e4m3" else (st["pool"], kv)
    raw[:, at // ps, :, at % ps] = kv[:, :, P:].permute(2, 0, 1, 3, 4)
    if c["cache"] == "e4m3":
        st["scales"][:, at // ps, :, :, at % ps] = b[:, :, P:].permute(2, 0, 1, 3)
    st["weights"][keep:n] = 0
    st["ids"][keep:n] = arrived + st["iota"][:S]
    # the S tokens of least weight leave, the first of equals; the newest frames' are kept
    guarded = st["ids"][:n] >= arrived + S - c["recent"] * S
    order = torch.sort(torch.where(guarded, math.inf, st["weights"][:n]), stable=True).indices
    gone = order[:S].sort().values                                # S positions, ascending
    leaves = (st["iota"][keep:n, None] == gone).any(1)
    src = st["iota"][keep:n][torch.sort(leaves.int(), stable=True).indices]  # survivors behind the budget first
    dst = torch.where(gone < keep, gone, src)                     # what leaves behind the budget stays where it is
    raw[:, dst // ps, :, dst % ps] = raw[:, src // ps, :, src % ps]
    if c["cache"] == "e4m3":
        st["scales"][:, dst // ps, :, :, dst % ps] = st["scales"][:, src // ps, :, :, src % ps]
    st["weights"][dst] = st["weights"][src]
    st["ids"][dst] = st["ids"][src]
    return _evict_outputs(st)


def _evict_outputs(st):
    keep = st["case"]["keep"]
    return [st["ids"][:keep], st["weights"][:keep], st["pool"]] + ([st["scales"]] if st["case"]["cache"] == "e4m3" else [])


# ---------------------------------------------------------------- states

def _own_cache(c, blocks, sc, w, frames, dtype):
    """A cache of the framework with its pools (one tensor [blocks, bytes]) and workspace."""
    import streaming_paged_kv_two_gb300 as spk
    cfg, keep = spk.make_config(
        num_blocks=blocks, num_streams=c.get("B", 1), num_heads=c["H"], head_dim=c["D"], page_size=c["ps"],
        patches_per_frame=c["P"], specials_per_frame=c["S"], scale_frames=sc, sliding_window=w,
        max_patch_pages=sc + w + HEADROOM, max_special_pages=-(-frames * c["S"] // c["ps"]),
        max_query_frames=-(-c.get("rows", 1) // (c["P"] + c["S"])),
        dtype={"e4m3": spk.SPK_E4M3, "bf16": spk.SPK_BF16, "f32": spk.SPK_F32}[dtype])
    pool_bytes, ws_bytes = spk.required_bytes(cfg)
    pools = torch.empty(blocks, pool_bytes, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(ws_bytes, dtype=torch.uint8, device="cuda")
    return spk.Cache(cfg, list(pools), keep), pools, ws


def _page_views(c, pools, first, pages, all_pages, dtype):
    """Codes [L, pages, 2, ps, H, D] of pages [first, first + pages) of every pool, and their
    scale bytes [L, pages, 2, H, ps] where the cache has them."""
    t = {"e4m3": torch.float8_e4m3fn, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    ps, H, D = c["ps"], c["H"], c["D"]
    end = all_pages * 2 * ps * H * D * (torch.tensor([], dtype=t).element_size())
    codes = pools[:, :end].view(t).view(pools.shape[0], all_pages, 2, ps, H, D)[:, first:first + pages]
    if dtype != "e4m3":
        return codes, None
    row = -(-ps // 128) * 128
    at = -(-end // 256) * 256
    scales = pools[:, at:at + all_pages * 2 * H * row].view(pools.shape[0], all_pages, 2, H, row)
    return codes, scales[:, first:first + pages, ..., :ps]


def _fill(c, cache, x, dtype):
    """The stream's frames appended one by one, as it would have seen them (block 0)."""
    B, P, S, sc, w = c["B"], c["P"], c["S"], c["sc"], c["w"]
    T, frames = P + S, c["frames"]
    st = torch.cuda.current_stream()
    kept = x["kp"].shape[1]
    step = max(1, min(500, (1 << 30) // (T * c["H"] * c["D"] * 4)))
    for s in range(B):
        for f0 in range(0, frames, step):
            n = min(step, frames - f0)
            f = torch.arange(f0, f0 + n, device="cuda")
            # frames the window has lost bring any patch rows; frames still visible bring their own
            at = torch.where(f < sc, f, (f - frames + kept).clamp(min=0))
            kv = torch.cat([torch.stack([x["kp"][s, at], x["vp"][s, at]], 1),
                            torch.stack([x["ks"][s].view(frames, S, c["H"], c["D"])[f0:f0 + n],
                                         x["vs"][s].view(frames, S, c["H"], c["D"])[f0:f0 + n]], 1)], 2)
            step_bytes = kv.stride(1) * kv.element_size()
            base = kv.data_ptr()
            for i in range(n):
                p = base + 2 * i * step_bytes
                cache.append_frame(s, 0, p, p + step_bytes, st)
                cache.evict_frames(s)
            torch.cuda.synchronize()


def prepare(case, seed):
    c = dict(case)
    return {"append": _prepare_append, "attend": _prepare_stream, "weigh": _prepare_stream, "evict": _prepare_evict}[c["op"]](c, seed)


def _prepare_append(c, seed):
    g = _gen(seed)
    L, B, T, H, D = c["L"], c["B"], c["P"] + c["S"], c["H"], c["D"]
    hs = _head_scale(g, 2, 1, 1, 1, H)
    st = dict(case=c, k=_randn(g, L, B, T, H, D, scale=hs[0]), v=_randn(g, L, B, T, H, D, scale=hs[1]))
    if own:
        cache, pools, ws = _own_cache(c, L, 4, 4, 4, "e4m3")
        msp, patch = cache.cfg.max_special_pages, B * (8 + HEADROOM)
        codes, b = _page_views(c, pools, 0, patch + B * msp, patch + B * msp, "e4m3")
        where = []
        for s in range(B):
            cache.append_frame(s, 0, st["k"][0, s], st["v"][0, s], torch.cuda.current_stream())
            where.append((cache.get_frame_targets(s)[0], patch + s * msp))  # its patch page, its first special page
            cache.rollback_frame(s)
        st.update(cache=cache, pools=pools, ws=ws, views=[
            [codes[:, p, :, :c["P"]] for p, _ in where], [b[:, p, ..., :c["P"]] for p, _ in where],
            [codes[:, p, :, :c["S"]] for _, p in where], [b[:, p, ..., :c["S"]] for _, p in where]])
    return st


def _prepare_stream(c, seed):
    x = _stream_inputs(c, seed)
    dtype = c.get("cache", "e4m3")
    B, rows, H, D = c["B"], c["rows"], c["H"], c["D"]
    st = dict(case=c, q=x["q"])
    k, v = _visible_kv(x)
    n = c["frames"] * c["S"]
    if c["op"] == "weigh":
        st["lse"], st["weights"] = _row_lse(c, x["q"], k, dtype), torch.rand(B, n, generator=_gen(seed + 1), device="cuda")
    if own:
        cache, pools, ws = _own_cache(c, 1, c["sc"], c["w"], c["frames"], dtype)
        _fill(c, cache, x, dtype)
        cap = cache.cfg.max_special_pages * c["ps"]
        st.update(cache=cache, pools=pools, ws=ws, out=torch.empty_like(x["q"]),
                  row_lse=torch.empty(B * rows, H, device="cuda"))
        if c["op"] == "weigh":
            st["buffer"] = torch.zeros(B, cap, device="cuda")
            st["ids"] = torch.zeros(B, cap, dtype=torch.int32, device="cuda")
            cache.track_specials(st["buffer"], st["ids"], torch.cuda.current_stream())
            st["buffer"][:, :n] = st["weights"]
            st["weights"] = st["buffer"][:, :n]
        cache.plan_rows(rows, ws, torch.cuda.current_stream())
        return st
    if c["op"] == "weigh":
        k = k[:, -n:]
        if dtype == "e4m3":
            st["k"], st["kb"] = _quantise(k)
        else:
            st["k"] = k.contiguous()
        return st
    st["k"], st["kb"] = _quantise(k)
    st["v"], st["vb"] = _quantise(v)
    return st


def _row_lse(c, q, k, dtype):
    """Natural log of the sum over the visible keys of exp(q k^T / sqrt(D)), in 64 bits: [B * rows, H]."""
    k = _dequantise(*_quantise(k)) if dtype == "e4m3" else k
    q = q.view(c["B"], c["rows"], c["H"], c["D"])
    out = [torch.logsumexp(torch.matmul(q[:, :, h].double(), k[:, :, h].double().transpose(1, 2)) / math.sqrt(c["D"]), -1)
           for h in range(c["H"])]
    return torch.stack(out, -1).float().reshape(-1, c["H"])


def _prepare_evict(c, seed):
    g = _gen(seed)
    L, T, H, D, P, S, ps, keep = c["L"], c["P"] + c["S"], c["H"], c["D"], c["P"], c["S"], c["ps"], c["keep"]
    dtype = {"f32": torch.float32}.get(c["cache"], torch.bfloat16)
    hs = _head_scale(g, 2, 1, 1, H)
    frames, n = keep // S, keep + S
    msp = -(-n // ps)
    held = [_randn(g, L, keep, H, D, scale=hs[i], dtype=dtype) for i in (0, 1)]
    st = dict(case=c, frames=frames, k=_randn(g, L, T, H, D, scale=hs[0], dtype=dtype),
              v=_randn(g, L, T, H, D, scale=hs[1], dtype=dtype), iota=torch.arange(n, device="cuda"))
    weights = torch.rand(keep, generator=g, device="cuda")
    if own:
        cache, pools, ws = _own_cache(dict(c, B=1), L, 8, 64, frames + 1, c["cache"])
        stream = torch.cuda.current_stream()
        st.update(cache=cache, pools=pools, ws=ws, weights=torch.zeros(msp * ps, device="cuda"),
                  ids=torch.zeros(msp * ps, dtype=torch.int32, device="cuda"))
        cache.track_specials(st["weights"], st["ids"], stream)
        patch = torch.zeros(P, H, D, dtype=dtype, device="cuda")
        for f in range(frames):
            rows = torch.cat([patch.expand(2, L, P, H, D), torch.stack([h[:, f * S:(f + 1) * S] for h in held])], 2)
            for b in range(L):
                cache.append_frame(0, b, rows[0, b], rows[1, b], stream)
            cache.evict_frames(0)
        torch.cuda.synchronize()
        pages = 72 + HEADROOM + msp
        st["pool"], st["scales"] = _page_views(c, pools, 72 + HEADROOM, msp, pages, c["cache"])
    else:
        at = st["iota"][:keep]
        kv = torch.stack(held, 1)                                 # [L, 2, keep, H, D]
        t = {"e4m3": torch.uint8, "bf16": torch.bfloat16, "f32": torch.float32}[c["cache"]]
        pool = torch.zeros(L, msp, 2, ps, H, D, dtype=t, device="cuda")
        if c["cache"] == "e4m3":
            kv, b = _quantise(kv)
            st["scales"] = torch.zeros(L, msp, 2, H, ps, dtype=torch.uint8, device="cuda")
            st["scales"][:, at // ps, :, :, at % ps] = b.permute(2, 0, 1, 3)
            kv = kv.view(torch.uint8)
        pool[:, at // ps, :, at % ps] = kv.permute(2, 0, 1, 3, 4)
        st["pool"] = pool.view(torch.float8_e4m3fn) if c["cache"] == "e4m3" else pool
        st["weights"] = torch.zeros(msp * ps, device="cuda")
        st["ids"] = torch.zeros(msp * ps, dtype=torch.int32, device="cuda")
        st["ids"][:keep] = at
    st["weights"][:keep] = weights
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "weigh": _plain_weigh, "evict": _plain_evict}[c["op"]](st)
    return {"append": _own_append, "attend": _own_attend, "weigh": _own_weigh, "evict": _own_evict}[c["op"]](st)


def _own_append(st):
    cache, stream = st["cache"], torch.cuda.current_stream()
    for b in range(st["case"]["L"]):
        for s in range(st["case"]["B"]):
            cache.append_frame(s, b, st["k"][b, s], st["v"][b, s], stream)
    for s in range(st["case"]["B"]):
        cache.rollback_frame(s)
    return st["views"]


def _own_attend(st):
    stream = torch.cuda.current_stream()
    if st["case"]["lse"]:
        st["cache"].run_attention_lse(0, st["q"], st["out"], st["row_lse"], st["ws"], stream)
        return [st["out"], st["row_lse"]]
    st["cache"].run_attention(0, st["q"], st["out"], st["ws"], stream)
    return st["out"]


def _own_weigh(st):
    st["cache"].accumulate_weights(0, st["q"], st["lse"], st["ws"], torch.cuda.current_stream())
    return st["weights"]


def _own_evict(st):
    cache, c, stream = st["cache"], st["case"], torch.cuda.current_stream()
    for b in range(c["L"]):
        cache.append_frame(0, b, st["k"][b], st["v"][b], stream)
    cache.evict_frames(0)
    cache.evict_specials(0, c["keep"], c["recent"], st["ws"], stream)
    return _evict_outputs(st)


# ---------------------------------------------------------------- work and 64-bit values

def work(c):
    H, D = c["H"], c["D"]
    if c["op"] == "append":
        rows = c["L"] * c["B"] * (c["P"] + c["S"]) * H
        return {"bytes": 2 * rows * (2 * D + D + 1), "flops": 2 * rows * 2 * D}
    if c["op"] == "evict":
        size = {"e4m3": D + 1, "bf16": 2 * D, "f32": 4 * D}[c["cache"]]
        read = 4 * D if c["cache"] == "f32" else 2 * D
        rows = c["L"] * (c["P"] + c["S"]) * H
        moved = c["L"] * c["S"] * H
        return {"bytes": 2 * rows * (read + size) + 4 * moved * size + 8 * (c["keep"] + c["S"]), "flops": 0}
    if c["op"] == "attend":
        n = _visible(c["P"], c["S"], c["sc"], c["w"], c["frames"])
        return {"bytes": c["B"] * H * (2 * n * (D + 1) + c["rows"] * (4 * D + (4 if c["lse"] else 0))),
                "flops": 4 * c["B"] * c["rows"] * n * H * D}
    n = c["frames"] * c["S"]
    size = {"e4m3": D + 1, "bf16": 2 * D, "f32": 4 * D}[c["cache"]]
    qsize = 4 * D if c["cache"] == "f32" else 2 * D
    return {"bytes": c["B"] * (H * (n * size + c["rows"] * (qsize + 4)) + 8 * n), "flops": 2 * c["B"] * c["rows"] * n * H * D}


def _held(x):
    """What the 8-bit cache holds of rows [..., D], in 64 bits: the nearest e4m3 multiple (ties to
    even) of the smallest power of two that keeps the row within 448, and that power's exponent."""
    y = x.double()
    amax = y.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.ceil(torch.log2(amax.clamp(min=1e-300) / E4M3_MAX)), torch.full_like(amax, -127.0))
    e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, e)
    e = torch.where((amax > 0) & (amax <= E4M3_MAX * torch.exp2(e - 1)), e - 1, e).clamp(min=-127)
    u = y * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(u / step) * step, e


def exact(case, seed):
    c = dict(case)
    H, D = c["H"], c["D"]
    if c["op"] == "append":
        g = _gen(seed)
        L, B, T, P = c["L"], c["B"], c["P"] + c["S"], c["P"]
        hs = _head_scale(g, 2, 1, 1, 1, H)
        k = _randn(g, L, B, T, H, D, scale=hs[0])
        v = _randn(g, L, B, T, H, D, scale=hs[1])
        held = torch.stack([_held(t)[0] for t in (k, v)], 2)
        return [held[:, :, :, :P].unbind(1), None, held[:, :, :, P:].unbind(1), None]
    if c["op"] == "evict":
        return None
    x = _stream_inputs(c, seed)
    dtype = c.get("cache", "e4m3")
    q = x["q"].view(c["B"], c["rows"], H, D)
    out = torch.empty(c["B"], c["rows"], H, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(c["B"], c["rows"], H, dtype=torch.float64, device="cuda")
    n = c["frames"] * c["S"]
    weights = torch.rand(c["B"], n, generator=_gen(seed + 1), device="cuda").double()
    for b in range(c["B"]):
        for h in range(H):
            ks, vs = (torch.cat([x[p][b, :, :, h].reshape(-1, D), x[t][b, :, h]]) for p, t in (("kp", "ks"), ("vp", "vs")))
            if dtype == "e4m3":
                (ks, ek), (vs, ev) = _held(ks), _held(vs)
                ks, vs = ks * torch.exp2(ek), vs * torch.exp2(ev)
            s = q[b, :, h].double() @ ks.double().T / math.sqrt(D)
            lse[b, :, h] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[b, :, h, None])
            out[b, :, h] = p @ vs.double()
            if c["op"] == "weigh":
                weights[b] += torch.exp(s[:, -n:] - lse[b, :, h, None].float().double()).sum(0)
    if c["op"] == "weigh":
        return weights
    out, lse = out.reshape(-1, H, D), lse.reshape(-1, H)
    return [out, lse] if c["lse"] else out
