"""Host-side tests (no GPU) of the 8-bit cache and of the budgeted special stream: sizes,
refusals, bookkeeping of evictions, and pins of their oracle."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
import workloads as wl

spk = pytest.importorskip("streaming_paged_kv_two_gb300")
torch = pytest.importorskip("torch")


def make(dtype=None, **over):
    args = dict(num_blocks=1, num_streams=1, num_heads=2, head_dim=64, page_size=16, patches_per_frame=10,
                specials_per_frame=3, scale_frames=1, sliding_window=2, max_patch_pages=8, max_special_pages=6,
                dtype=spk.SPK_E4M3 if dtype is None else dtype)
    args.update(over)
    return spk.make_config(**args)


def refused(code, call, *args):
    with pytest.raises(spk.SpkError) as e:
        call(*args)
    assert e.value.code == code, e.value


# ---------------------------------------------------------------- oracle pins

def test_rounding_to_e4m3_is_torchs():
    x = np.concatenate([np.linspace(-448, 448, 20001), 2.0 ** np.linspace(-14, 8.8, 5001),
                        np.arange(0, 64) * 2.0 ** -11, [0.0, -0.0]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(oracle.round_e4m3(x), want)


def test_scale_is_the_smallest_power_of_two_that_fits():
    assert oracle.quantise(np.array([[448.0]]))[1][0] == 127
    assert oracle.quantise(np.array([[448.0 * (1 + 2 ** -20)]]))[1][0] == 128
    assert oracle.quantise(np.array([[0.0, 0.0]]))[1][0] == 0
    assert oracle.quantise(np.array([[np.inf, 1.0]]))[1][0] == 119          # 1 <= 448 * 2^-8
    assert oracle.held(np.array([[np.inf, 1.0]]))[0, 0] == 448 * 2.0 ** -8
    x = np.random.default_rng(1).standard_normal((50, 64))
    h = oracle.held(x)
    amax = np.abs(x).max(-1, keepdims=True)
    assert np.all(np.abs(h - x) <= np.maximum(np.abs(x) * 2.0 ** -4, amax / 224 * 2.0 ** -10))


def test_eviction_by_hand():
    w = [5, 1, 4, 1, 3, 1, 9]
    # three of least weight are at 1, 3, 5: the survivors behind 4 (position 4 and 6) fill 1 and 3
    assert oracle.evict(w, range(7), 4, 100) == [0, 4, 2, 6]
    # ties: the lowest positions leave first
    assert oracle.evict([1, 1, 1, 1], range(4), 2, 100) == [2, 3]
    # recent tokens are kept whatever their weight; NaN weighs most
    assert oracle.evict([1, 0, np.nan, 0, 0], range(5), 3, 3) == [3, 4, 2]
    assert oracle.evict(w, range(7), 7, 0) == list(range(7))


def test_key_weights_sum_to_rows_times_heads():
    g = np.random.default_rng(0)
    q, k, v = (g.standard_normal((n, 2, 64)) for n in (5, 9, 9))
    _, lse = oracle.attend(q, k, v)
    assert np.isclose(oracle.key_weights(q, k, lse).sum(), 5 * 2)


# ---------------------------------------------------------------- sizes

def test_pool_bytes_hold_codes_and_scales():
    cfg, _ = make(page_size=200, patches_per_frame=150, max_patch_pages=3, max_special_pages=4)
    pool, _ = spk.required_bytes(cfg)
    codes = 7 * 2 * 200 * 2 * 64
    assert pool == -(-codes // 256) * 256 + 7 * 2 * 2 * 256       # rows of 200 scale bytes padded to 256
    half = spk.required_bytes(make(spk.SPK_BF16, page_size=200, patches_per_frame=150, max_patch_pages=3,
                                   max_special_pages=4)[0])[0]
    assert half == 2 * codes


def test_workspace_covers_one_row_over_many_splits():
    small = spk.required_bytes(make(num_heads=1)[0])[1]
    assert small >= 256 * 13 * 64 * 4     # 256 splits of one head


def test_workspace_of_many_query_frames_is_not_sized_for_many_splits():
    """Up to 256 splits serve calls of few rows: the partials of 64 frames' rows are those of 32 splits."""
    frames = dict(num_heads=1, patches_per_frame=256, specials_per_frame=6, page_size=256, max_query_frames=64)
    e4m3, bf16 = (spk.required_bytes(make(t, **frames)[0])[1] for t in (spk.SPK_E4M3, spk.SPK_BF16))
    assert e4m3 <= bf16 + (1 << 20)
    frames.update(num_heads=4, head_dim=128, patches_per_frame=999, page_size=1024)
    e4m3, bf16 = (spk.required_bytes(make(t, **frames)[0])[1] for t in (spk.SPK_E4M3, spk.SPK_BF16))
    assert e4m3 <= bf16 + (1 << 20)


@pytest.mark.parametrize("dtype", [spk.SPK_E4M3, spk.SPK_BF16, spk.SPK_F32])
def test_workspace_holds_no_scratch_of_its_own_for_the_budget(dtype):
    """A longer special stream adds plan tables (8 bytes a chunk); its weights' and evictions' scratch
    (4 bytes a head and 8 a token) lies over the partials."""
    size = dict(num_heads=16, patches_per_frame=256, specials_per_frame=6, page_size=256)
    short, long = (spk.required_bytes(make(dtype, max_special_pages=n, **size)[0])[1] for n in (1, 235))
    assert long - short <= 234 * 8 * (4 if dtype == spk.SPK_E4M3 else 2) + 512


def test_splits_follow_the_planned_rows():
    """200 forced splits: as many as eight heads may have (608 / 8) for up to two frames' rows, as many as
    the partials hold (10,240 rows a stream and head: 32 splits of eight frames) for more.  One head
    may have them all (3 patch and 188 special pages): its partials hold 77,824 rows."""
    cfg, _ = make(num_heads=8, patches_per_frame=30, specials_per_frame=10, page_size=64, max_special_pages=200,
                  splits_per_stream=200, max_query_frames=8)
    one, _ = make(num_heads=1, patches_per_frame=30, specials_per_frame=10, page_size=64, max_special_pages=200,
                  splits_per_stream=200, max_query_frames=8)
    for cfg, wanted in ((cfg, ((1, 76), (40, 76), (80, 76), (160, 64), (320, 32))), (one, ((1, 191), (320, 191)))):
        c = spk.Cache(cfg)
        for _ in range(1200):
            c.append_frame(0, 0)
            c.evict_frames(0)
        for rows, splits in wanted:
            c.plan_rows(rows)
            assert c.get_plan_info()["num_splits"] == splits, rows


# ---------------------------------------------------------------- refusals and bookkeeping

@pytest.mark.parametrize("dtype", [spk.SPK_E4M3, spk.SPK_BF16, spk.SPK_F32])
def test_plan_rows_limits(dtype):
    c = spk.Cache(make(dtype, max_query_frames=2)[0])
    refused(spk.SPK_ERR_BAD_STATE, c.plan_rows, 1)                 # no frame yet
    c.append_frame(0, 0)
    for rows in (0, -1, 27):
        refused(spk.SPK_ERR_INVALID_ARG, c.plan_rows, rows)
    for rows in (1, 13, 26):
        c.plan_rows(rows)
        assert c.get_plan_host()["qo_indptr"] == [0, rows]
    c.plan()
    assert c.get_plan_host()["qo_indptr"] == [0, 13]


def test_calls_on_a_bookkeeping_only_cache_are_refused():
    c = spk.Cache(make()[0])
    c.append_frame(0, 0)
    c.plan()
    refused(spk.SPK_ERR_INVALID_ARG, c.run_attention_lse, 0, 256, 256, 256, 256)
    refused(spk.SPK_ERR_INVALID_ARG, c.run_attention_lse, 0, 256, 256, 258, 256)   # lse alignment
    refused(spk.SPK_ERR_INVALID_ARG, c.run_attention_lse, 0, 256, 256, None, 256)
    refused(spk.SPK_ERR_INVALID_ARG, c.accumulate_weights, 0, 256, 256, 256)
    refused(spk.SPK_ERR_INVALID_ARG, c.track_specials, 256, 256)
    refused(spk.SPK_ERR_INVALID_ARG, c.read_scales, 0, 0, 256)
    refused(spk.SPK_ERR_INVALID_ARG, c.evict_specials, 0, 1, 0, 256)
    c.track_specials(None, None)


def test_evict_specials_refusals():
    c = spk.Cache(make(num_blocks=2)[0])
    for _ in range(3):
        c.append_frame(0, 0)
    refused(spk.SPK_ERR_INVALID_ARG, c.evict_specials, 0, 0, 0)
    refused(spk.SPK_ERR_INVALID_ARG, c.evict_specials, 1, 4, 0)
    refused(spk.SPK_ERR_INVALID_ARG, c.evict_specials, 0, 4, -1)
    refused(spk.SPK_ERR_INVALID_ARG, c.evict_specials, 0, 5, 2)    # 2 frames hold 6 tokens
    refused(spk.SPK_ERR_BAD_STATE, c.evict_specials, 0, 6, 2)      # block 1 of the frame is missing
    c.append_frame(0, 1)
    c.evict_specials(0, 6, 2)
    assert c.get_stats(0)["special_tokens"] == 6


def test_evict_specials_bookkeeping():
    c = spk.Cache(make(page_size=16, max_special_pages=2)[0])
    for f in range(10):
        c.append_frame(0, 0)
        c.evict_frames(0)
    refused(spk.SPK_ERR_OUT_OF_SPECIAL_PAGES, c.append_frame, 0, 0)  # 30 of 32 slots
    c.evict_specials(0, 30, 0)                                      # nothing to do: the plan-less state stays
    assert c.get_frame_targets(0)[1][0][0] >= 0
    c.evict_specials(0, 16, 1)
    st = c.get_stats(0)
    assert st["special_tokens"] == 16 and st["frame_count"] == 10
    assert [t for t, _ in c.get_frame_targets(0)[1]] == [-1, -1, -1]
    refused(spk.SPK_ERR_BAD_STATE, c.rollback_frame, 0)
    refused(spk.SPK_ERR_BAD_STATE, c.get_plan_host)
    c.plan()
    plan = c.get_plan_host()
    assert plan["last_page_len"] == [16] and len(plan["indices"]) == 3 + 1
    c.append_frame(0, 0)                                            # the freed page is taken again
    assert [s for _, s in c.get_frame_targets(0)[1]] == [0, 1, 2]
    c.rollback_frame(0)
    assert c.get_stats(0)["special_tokens"] == 16
    for _ in range(200):                                            # a budget holds for ever
        c.append_frame(0, 0)
        c.evict_frames(0)
        c.evict_specials(0, 16, 1)
    assert c.get_stats(0)["special_tokens"] == 16 and c.get_stats(0)["frame_count"] == 210
    c.reset()
    assert c.get_stats(0)["special_tokens"] == 0
    c.append_frame(0, 0)
    assert [s for _, s in c.get_frame_targets(0)[1]] == [0, 1, 2]


def test_plan_before_and_after_eviction_lists_the_survivors_pages():
    c = spk.Cache(make(page_size=16, max_special_pages=6, special_page_order=[13, 8, 10, 9, 12, 11])[0])
    for f in range(16):                                             # 48 tokens: pages 13, 8, 10
        c.append_frame(0, 0)
        c.evict_frames(0)
    c.plan()
    assert c.get_plan_host()["indices"][-3:] == [13, 8, 10]
    c.evict_specials(0, 17, 0)
    c.plan()
    p = c.get_plan_host()
    assert p["indices"][-2:] == [13, 8] and p["last_page_len"] == [1]
    for f in range(6):                                              # 35 tokens: the third page is 10 again
        c.append_frame(0, 0)
        c.evict_frames(0)
    c.plan()
    assert c.get_plan_host()["indices"][-3:] == [13, 8, 10]
