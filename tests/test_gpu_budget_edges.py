"""GPU tests of the budgeted special stream and of the 8-bit cache where the calls meet unusual
state: reported timeouts, infinite keys, long records, evictions of many streams."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
import workloads as wl  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def work(**kw):
    base = dict(name="edges", num_blocks=1, num_streams=1, num_heads=2, head_dim=64, page_size=256,
                patches_per_frame=200, specials_per_frame=6, scale_frames=1, sliding_window=2,
                frames=6, dtype="bf16", value_scale=1.0)
    base.update(kw)
    return wl.Workload(**base)


def harness(w, kind, **kw):
    from budget_harness import Stream
    return Stream(w, kind, **kw)


# ---------------------------------------------------------------- accumulated weights

@pytest.mark.parametrize("kind", ["e4m3", "bf16", "f32"])
def test_a_reported_timeout_adds_nothing(kind):
    """The status word as a wait that gave up leaves it (set from the host): the running totals stay
    as they are until the report has been read."""
    from budget_harness import to_device
    import streaming_paged_kv_two_gb300 as spk
    w = work(frames=8)
    h = harness(w, kind)
    h.track()
    for f in range(w.frames):
        h.append(f)
    n = w.frames * w.specials_per_frame
    q = h.queries(6, 1)
    h.cache.plan_rows(6, h.ws, h.st)
    lse = torch.from_numpy(h.oracle(0, q, 6)[1].astype(np.float32)).cuda()
    qd = to_device(q, h.w.dtype)
    h.weights[:, :n] = 0.5
    h.ws.view(torch.int32)[0] = 1
    h.cache.accumulate_weights(0, qd, lse, h.ws, h.st)
    torch.cuda.synchronize()
    assert torch.equal(h.weights[:, :n], torch.full_like(h.weights[:, :n], 0.5))
    with pytest.raises(spk.SpkError) as e:
        h.status()
    assert e.value.code == spk.SPK_ERR_DEVICE_TIMEOUT
    h.cache.accumulate_weights(0, qd, lse, h.ws, h.st)
    torch.cuda.synchronize()
    assert float(h.weights[:, :n].min()) > 0.5
    assert h.status() == 0
    h.close()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [1, 6, 206, 402])
def test_keys_of_minus_infinite_score_weigh_nothing(kind, D, rows):
    """A special key with an infinite element that every query row meets with the other sign: its
    scores are -inf, its weight is 0 (and it is the first to leave), whatever rows the last tile lacks."""
    from budget_harness import to_device
    w = work(frames=8, head_dim=D)
    h = harness(w, kind, max_query_frames=2)
    P = w.patches_per_frame

    def kv(f):
        def rows_of(s, b):
            k, v = wl.frame_kv(w, s, b, f)
            k = wl.bf16_bits_to_f32(k)
            if f == 3:
                k[P + 2, :, 5] = np.inf
            return (wl.f32_to_bf16_bits(k), v) if kind == "bf16" else (k, wl.bf16_bits_to_f32(v))
        return rows_of

    h.track()
    for f in range(w.frames):
        h.append(f, kv(f))
    q = wl.to_f64(h.queries(rows, 4), h.w.dtype).astype(np.float32)
    q[:, :, 5] = -np.abs(q[:, :, 5]) - np.float32(0.25)
    q = wl.f32_to_bf16_bits(q) if kind == "bf16" else q
    k, v = h.visible(0, 0)
    with np.errstate(invalid="ignore"):
        _, lse = oracle.attend(wl.to_f64(q, h.w.dtype), k, v)
    assert np.isfinite(lse).all()
    h.cache.plan_rows(rows, h.ws, h.st)
    h.cache.accumulate_weights(0, to_device(q, h.w.dtype), torch.from_numpy(lse.astype(np.float32)).cuda(), h.ws, h.st)
    torch.cuda.synchronize()
    n = w.frames * w.specials_per_frame
    got = h.weights[0, :n].cpu().numpy()
    dead = 3 * w.specials_per_frame + 2
    assert got[dead] == 0 and np.isfinite(got).all()
    exact = oracle.key_weights(wl.to_f64(q, h.w.dtype), np.stack([r[0] for r in h.special[(0, 0)]]), lse)
    # a score of at most 20 in fp32 (its D roundings, the log-sum-exp's and the exponential's)
    live = np.arange(n) != dead
    assert np.abs(got[live] / exact[live] - 1).max() <= (2 * D + 64) * 2.0 ** -24 * 20
    assert h.evict(0, n - 1, 0)[dead] == n - 1
    assert h.status() == 0
    h.close()


def weight_bounds(q, k, lse, e4m3):
    """(exact sum, bound of its error) per key: q [R, H, D], k [n, H, D], lse [R, H] in 64 bits.

    A term exp(s - lse) is off by the fp32 rounding of its exponent: the score's (D + 8 roundings of the
    absolute sum of its products, twice: product and scaling), the log-sum-exp's (twice), 2^-20 for the
    exponential and its argument.  An 8-bit cache's q is two e4m3 values under a power of two that puts
    the row's largest value at 224 or more, or up to 16 times lower where the rows of the head share one: an
    element of more than 2^-10 of the head's largest is exact, another is off by half a step of 2^-9 of
    what the head's largest is at least 224 of.  The sum adds a rounding for each of its levels."""
    R, H, D = q.shape
    rows, big = np.abs(q).max(-1), np.abs(q).max((0, 2))                      # [R, H], [H]
    apart = (rows > 0) & (rows < big * 2.0 ** -5)
    ref = np.where(apart.any(0), rows, big)                                   # [R, H]: whose 224 counts
    loss = np.where(np.abs(q) < ref[..., None] * 2.0 ** -9, ref[..., None] * 2.0 ** -10 / 224, 0.0) if e4m3 else 0 * q
    total, bound = np.zeros(len(k)), np.zeros(len(k))
    for h in range(H):
        p = np.exp(q[:, h] @ k[:, h].T / np.sqrt(D) - lse[:, h, None])        # [R, n]
        ds = ((np.abs(q[:, h]) * (2 * (D + 8) * 2.0 ** -24) + loss[:, h]) @ np.abs(k[:, h]).T) / np.sqrt(D)
        total += p.sum(0)
        bound += (p * (ds + np.abs(lse[:, h, None]) * 2.0 ** -22 + 2.0 ** -20)).sum(0)
    return total, bound + total * (R / 16 + 40 + H) * 2.0 ** -24


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("rows,D", [(8, 64), (8, 128), (150, 64), (150, 128)])
def test_weights_of_long_records(kind, rows, D):
    """Records long enough that each of the two CTAs of a (stream, head) walks its ring of 128-key tiles
    several times with every warpgroup (some 25 tiles), pages that end inside a tile, and a stream that holds far fewer tokens than the others."""
    from budget_harness import to_device
    w = work(num_streams=4, num_heads=16, head_dim=D, frames=80, specials_per_frame=61, patches_per_frame=90,
             page_size=200, sliding_window=1)
    h = harness(w, kind)
    h.track()
    for f in range(w.frames):
        h.append(f)
    h.weights[1, :w.frames * 61] = torch.rand(w.frames * 61, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    h.evict(1, 700, 2)
    g = np.random.default_rng(rows)
    q = h.queries(rows, rows, 1.5)
    lse = g.uniform(2, 6, (4 * rows, 16)).astype(np.float32)
    before = h.weights.clone()
    h.cache.plan_rows(rows, h.ws, h.st)
    h.cache.accumulate_weights(0, to_device(q, "bf16"), torch.from_numpy(lse).cuda(), h.ws, h.st)
    assert h.status() == 0
    for s in range(4):
        n = len(h.special[(s, 0)])
        assert n == (700 if s == 1 else 4880)
        assert torch.equal(h.weights[s, n:], before[s, n:])       # behind the last token: untouched
        at = np.unique(np.concatenate([np.arange(n - 140, n), g.integers(0, n, 400)]))
        k = np.stack([h.special[(s, 0)][i][0] for i in at])
        r = slice(s * rows, (s + 1) * rows)
        exact, bound = weight_bounds(wl.to_f64(q[r], "bf16"), k, lse[r].astype(np.float64), kind == "e4m3")
        was = before[s].double().cpu().numpy()[at]
        got = h.weights[s].double().cpu().numpy()[at]
        worst = (np.abs(got - was - exact) / (bound + (was + exact) * 2.0 ** -24)).max()
        assert worst <= 1, (s, worst)
    h.close()


@pytest.mark.parametrize("kind", ["e4m3", "bf16", "f32"])
@pytest.mark.parametrize("rows,D", [(769, 64), (800, 64), (1600, 64), (385, 128), (800, 128)])
def test_weights_of_more_rows_than_one_pass_holds(kind, rows, D):
    from budget_harness import to_device
    w = work(num_streams=2, num_heads=3, head_dim=D, frames=9, specials_per_frame=64, patches_per_frame=16, page_size=100)
    h = harness(w, kind, max_query_frames=20)
    h.track()
    for f in range(w.frames):
        h.append(f)
    q = h.queries(rows, rows, 1.5)
    x = wl.to_f64(q, h.w.dtype).astype(np.float32)
    x[:rows // 2] *= np.float32(4)                       # the passes' largest values differ
    q = wl.f32_to_bf16_bits(x) if kind != "f32" else x
    lse = np.random.default_rng(rows).uniform(20, 24, (2 * rows, 3)).astype(np.float32)
    h.cache.plan_rows(rows, h.ws, h.st)
    h.cache.accumulate_weights(0, to_device(q, h.w.dtype), torch.from_numpy(lse).cuda(), h.ws, h.st)
    assert h.status() == 0
    for s in range(2):
        n = len(h.special[(s, 0)])
        r = slice(s * rows, (s + 1) * rows)
        k = np.stack([x[0] for x in h.special[(s, 0)]])
        exact, bound = weight_bounds(wl.to_f64(q[r], h.w.dtype), k, lse[r].astype(np.float64), kind == "e4m3")
        worst = (np.abs(h.weights[s, :n].double().cpu().numpy() - exact) / bound).max()
        assert worst <= 1, (s, worst)
    h.close()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("big", [2.0 ** 5, 2.0 ** 9, 2.0 ** 13])
def test_a_row_far_above_the_others_takes_nothing_from_them(D, big):
    """One query row of a head far larger than the rest (and a row of zeros): the others' terms are as
    exact as they are without it."""
    from budget_harness import to_device
    w = work(head_dim=D, num_heads=2, frames=40)
    h = harness(w, "e4m3")
    h.track()
    for f in range(w.frames):
        h.append(f)
    rows = 70
    q = wl.to_f64(h.queries(rows, 3), "bf16").astype(np.float32)
    q[33, 1] *= np.float32(big)
    q[50] = 0
    q = wl.f32_to_bf16_bits(q)
    x = wl.to_f64(q, "bf16")
    lse = np.full((rows, 2), 5.0)
    lse[33, 1] = 1e5 if big > 2.0 ** 9 else 5e4 if big > 32 else 500.0       # (its own terms are 0)
    h.cache.plan_rows(rows, h.ws, h.st)
    h.cache.accumulate_weights(0, to_device(q, "bf16"), torch.from_numpy(lse.astype(np.float32)).cuda(), h.ws, h.st)
    k = np.stack([r[0] for r in h.special[(0, 0)]])
    exact, bound = weight_bounds(x, k, lse, True)
    worst = (np.abs(h.weights[0, :len(k)].double().cpu().numpy() - exact) / bound).max()
    assert worst <= 1, worst
    assert h.status() == 0
    h.close()


# ---------------------------------------------------------------- eviction

def test_evictions_of_many_streams_do_not_wait_for_the_gpu():
    """One plan and five evictions, twice over, queued behind a kernel that runs for a good while:
    the calls return before it has ended, and give what they give on an idle GPU."""
    w = work(num_streams=5, frames=4, patches_per_frame=8, page_size=16)
    h = harness(w, "e4m3")
    h.track()
    for f in range(w.frames):
        h.append(f)
    n = w.frames * w.specials_per_frame
    h.weights[:, :n] = torch.arange(n, device="cuda", dtype=torch.float32)
    torch.cuda.synchronize()
    for keep in (20, 15):
        done = torch.cuda.Event()
        torch.cuda._sleep(1_000_000_000)
        done.record()
        h.cache.plan(h.ws, h.st)
        for s in range(w.num_streams):
            h.cache.evict_specials(s, keep, 0, h.ws, h.st)
        assert not done.query()
        torch.cuda.synchronize()
        # the lowest positions have the least weight: the newest tokens are left
        assert [sorted(x) for x in h.ids[:, :keep].tolist()] == [list(range(n - keep, n))] * w.num_streams
    h.close()


def test_eviction_over_more_pages_than_one_launch_lists():
    from test_gpu_budget import check_pool
    w = work(num_blocks=2, num_heads=1, frames=1100, specials_per_frame=4, patches_per_frame=2, page_size=4)
    h = harness(w, "e4m3")
    h.track()
    for f in range(w.frames):
        h.append(f)
    n = w.frames * w.specials_per_frame
    g = np.random.default_rng(2)
    for keep in (4100, 4001, 90):
        n = len(h.special[(0, 0)])
        h.weights[0, :n] = torch.from_numpy(g.random(n).astype(np.float32)).cuda()
        h.evict(0, keep, 3)
        check_pool(h, 0, keep)
    h.close()


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [3, 8, 16, 31, 136, 206])
def test_a_nan_stays_where_it_is(D, rows):
    """A NaN or an infinity in a query row stays in that row and head, a NaN element of V in its dim of
    its head; everything else is the oracle's."""
    from budget_harness import check_attention
    w = work(head_dim=D, frames=5)
    h = harness(w, "e4m3", splits=2)

    def kv(f):
        def rows_of(s, b):
            k, v = wl.frame_kv(w, s, b, f)
            v = v.copy()
            if f == 4:               # (frames 0, 3 and 4 are visible)
                v[17, 1, 9] = 0x7FC0
            return k, v
        return rows_of

    for f in range(w.frames):
        h.append(f, kv(f))
    q = h.queries(rows, 3)
    bad = sorted({0, rows // 2, rows - 1})
    for i, r in enumerate(bad):
        q[r, 0, 5] = (0x7FC0, 0x7F80, 0xFF80)[i]         # NaN, inf, -inf
    h.cache.plan_rows(rows, h.ws, h.st)
    out, lse = h.attend(0, q)
    clean = q.copy()
    clean[bad, 0, 5] = 0
    assert np.isnan(out[bad, 0]).all() and not np.isfinite(lse[bad, 0]).any()
    assert np.isnan(out[:, 1, 9]).all()
    # the rest against an oracle that has neither
    for key, (k, v) in list(h.patch.items()):
        h.patch[key] = (k, np.nan_to_num(v))
    o, l, a, ds, flushed = h.oracle(0, clean, rows)
    got_o, got_l = out.copy(), lse.copy()
    got_o[bad, 0], got_l[bad, 0] = o[bad, 0], l[bad, 0]
    got_o[:, 1, 9] = o[:, 1, 9]
    check_attention((got_o, got_l), (o, l, a, ds, flushed), "e4m3", f"{rows} rows")
    assert h.status() == 0
    h.close()


# ---------------------------------------------------------------- workspace

@pytest.mark.parametrize("kind,heads,splits", [("e4m3", 1, 256), ("e4m3", 1, 0), ("e4m3", 16, 256), ("bf16", 2, 32), ("f32", 2, 32)])
def test_calls_stay_inside_the_workspace(kind, heads, splits):
    """Attention of every planned size with as many splits as it takes, weights and an eviction, in a
    workspace of exactly the stated size: what lies behind it is not written."""
    from budget_harness import check_attention, to_device
    w = work(num_heads=heads, frames=300, specials_per_frame=64, patches_per_frame=16, page_size=64)
    h = harness(w, kind, splits=splits, max_query_frames=3)
    guard = torch.full((h.ws.numel() + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    h.ws = guard[:h.ws.numel()]
    h.ws.zero_()
    h.track()
    for f in range(w.frames):
        h.append(f)
    for rows in (1, 32, 33, 80, 81, 240):
        q = h.queries(rows, rows)
        h.cache.plan_rows(rows, h.ws, h.st)
        got = h.attend(0, q)
        if rows in (1, 80, 240):
            check_attention(got, h.oracle(0, q, rows), kind, f"{rows} rows")
        lse = torch.from_numpy(got[1].astype(np.float32)).cuda()
        h.cache.accumulate_weights(0, to_device(q, h.w.dtype), lse, h.ws, h.st)
    h.evict(0, 10000, 2)
    assert h.status() == 0
    assert bool((guard[h.ws.numel():] == 0xA5).all())
    h.close()


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_pages_past_four_gigabytes(kind, monkeypatch):
    """The stream's special pages at the end of a pool of 5.5 (bf16: 11) GB: attention, weights and an
    eviction address them and their scales."""
    import budget_harness
    from budget_harness import check_attention, to_device
    from test_gpu_budget import check_pool
    import streaming_paged_kv_two_gb300 as spk

    def config(w, splits, max_query_frames):
        pages = 1300
        return spk.make_config(
            num_blocks=1, num_streams=1, num_heads=16, head_dim=128, page_size=1024,
            patches_per_frame=w.patches_per_frame, specials_per_frame=w.specials_per_frame,
            scale_frames=w.scale_frames, sliding_window=w.sliding_window, max_patch_pages=8, max_special_pages=pages,
            dtype=spk.SPK_BF16, splits_per_stream=splits, max_query_frames=max_query_frames,
            special_page_order=list(range(8 + pages - 1, 7, -1)))

    monkeypatch.setattr(budget_harness, "spk_config_for", config)
    w = work(num_heads=16, head_dim=128, frames=25, specials_per_frame=64, page_size=1024)
    h = harness(w, kind)
    assert h.pools[0].numel() > 2 ** 32
    h.track()
    for f in range(w.frames):
        h.append(f)
    for rows in (1, 40):
        q = h.queries(rows, rows)
        h.cache.plan_rows(rows, h.ws, h.st)
        got = h.attend(0, q)
        check_attention(got, h.oracle(0, q, rows), kind, f"{rows} rows")
    n = w.frames * 64
    lse = np.full((40, 16), 6.0, np.float32)
    h.cache.accumulate_weights(0, to_device(q, "bf16"), torch.from_numpy(lse).cuda(), h.ws, h.st)
    exact, bound = weight_bounds(wl.to_f64(q, "bf16"), np.stack([r[0] for r in h.special[(0, 0)]]), lse.astype(np.float64),
                                 kind == "e4m3")
    assert (np.abs(h.weights[0, :n].double().cpu().numpy() - exact) / bound).max() <= 1
    h.evict(0, 1100, 2)
    check_pool(h, 0)
    assert h.status() == 0
    h.close()


# ---------------------------------------------------------------- builds

def test_a_build_with_other_register_counts_serves_the_8_bit_cache(tmp_path):
    """The many-row kernel plans each role's registers for the count that its launch bounds give here.
    A build that comes to another count (here: the plan names fewer) still creates caches and computes
    the same attention."""
    import os
    import shutil
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    pkg = tmp_path / "streaming_paged_kv_two_gb300"
    shutil.copytree(os.path.join(root, "streaming_paged_kv_two_gb300"), pkg,
                    ignore=shutil.ignore_patterns("_build", "*.so", "__pycache__"))
    shutil.copytree(os.path.join(root, "include"), tmp_path / "include")
    src = pkg / "csrc" / "spk_attn_e4m3_tc.cu"
    text = src.read_text()
    assert text.count("kRegs = D == 64 ? 72 : 96;") == 1
    src.write_text(text.replace("kRegs = D == 64 ? 72 : 96;", "kRegs = D == 64 ? 64 : 88;"))
    script = """
import streaming_paged_kv_two_gb300 as spk
assert spk.LIB_PATH.startswith(%r), spk.LIB_PATH
from test_gpu_budget_edges import harness, work
from budget_harness import check_attention
for D in (64, 128):
    w = work(head_dim=D)
    h = harness(w, "e4m3")
    for f in range(w.frames):
        h.append(f)
    q = h.queries(206, D)
    h.cache.plan_rows(206, h.ws, h.st)
    check_attention(h.attend(0, q), h.oracle(0, q, 206), "e4m3")
    assert h.status() == 0
    h.close()
""" % str(tmp_path)
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(tmp_path), os.path.join(root, "tests"), root]))
    for cmd in ([sys.executable, str(pkg / "build.py")], [sys.executable, "-c", script]):
        r = subprocess.run(cmd, env=env, cwd=tmp_path, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stdout + r.stderr
