"""Tile maps of starts that fall back or leave the range: which sequences are passed over, that the walk stays
within the split buffers, and what the attention calls make of such maps."""
import numpy as np
import pytest
import torch

from load_balanced_paged_02_gb300 import _build
from load_balanced_paged_02_gb300 import binding as hb
import _tiles as tl


def taken(starts, num_tokens, q_len=1):
    """(first row, rows) of every sequence, (None, 0) where it is passed over: starts that decrease or leave
    [0, num_tokens], or a begin before the end of an earlier sequence whose starts do neither."""
    got, ends = [], 0
    for a, b in zip(starts, starts[1:]):
        a, b = a * q_len, b * q_len
        in_order = 0 <= a <= b <= num_tokens
        got.append((a, b - a) if in_order and a >= ends else (None, 0))
        if in_order:
            ends = max(ends, b)
    return got


def walk_of(mode, seqs, lens, T):
    """Per sequence: tiles and units (two per tile, one per block)."""
    got = []
    for (_, n), L in zip(seqs, lens):
        if n == 0 or (mode == 1 and L <= 0):
            got.append((0, 0))
            continue
        tiles, units = -(-n // T), 0
        for i in range(tiles):
            end = L if mode == 1 else max(0, L - n + min(n, T * (i + 1)))
            units += 2 + (-(-end // 128) if mode == 1 else max(1, -(-end // 128)))
        got.append((tiles, units))
    return got


def bad_starts(rng, S, num_tokens):
    """Starts in order, with some of them replaced by ones that fall back or leave the range."""
    st = sorted(int(x) for x in rng.integers(0, num_tokens + 1, S + 1))
    for _ in range(int(rng.integers(1, max(2, S // 3)))):
        at = int(rng.integers(0, S + 1))
        st[at] = int(rng.choice([0, num_tokens, num_tokens + 9, -3, int(rng.integers(0, num_tokens + 1))]))
    return st


def alternating(S, num_tokens):
    return [0 if s % 2 == 0 else num_tokens for s in range(S + 1)]


def test_the_rule_keeps_split_rows_in_bounds():
    """On the CPU: with the rule above, the last split row that a prefix map names lies within
    hpc_prefix_split_rows; with every sequence judged by its own two starts it would not."""
    _build.build()
    L, rng = hb.lib(), np.random.default_rng(1)
    over = 0
    for rep in range(400):
        B, q_len, hkv, ctas = int(rng.integers(1, 300)), int(rng.integers(1, 9)), int(rng.integers(1, 9)), int(rng.integers(2, 200))
        S = int(rng.integers(1, 60))
        st = alternating(S, B) if rep % 4 == 0 else bad_starts(rng, S, B)
        rows = L.hpc_prefix_split_rows(S, B, q_len, hkv, ctas)
        for T in (32, 64):
            seqs = taken(st, B * q_len, q_len)
            assert sum(n for _, n in seqs) <= B * q_len
            per_head = sum(t for t, _ in walk_of(1, seqs, [100] * S, T))
            assert (per_head * hkv + ctas // (T // 32)) * T * 8 <= rows
            alone = [((a * q_len, (b - a) * q_len) if 0 <= a <= b <= B else (None, 0)) for a, b in zip(st, st[1:])]
            over += (sum(t for t, _ in walk_of(1, alone, [100] * S, T)) * hkv + ctas // (T // 32)) * T * 8 > rows
    assert over > 100


def plan_of(mode, st, lens, num_tokens, hkv, ctas, T, q_len):
    if mode == 0:
        return hb.hpc_prefill_plan(tl.i32(st), tl.i32(lens), num_tokens, hkv, 1000, num_ctas=ctas, tile_tokens=T)
    return hb.hpc_prefix_plan(tl.i32(st), tl.i32(lens), num_tokens // q_len, hkv, 1000, q_len=q_len, num_ctas=ctas, tile_tokens=T)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [32, 64])
@pytest.mark.parametrize("mode", [0, 1])
def test_maps(mode, T):
    """The map alone: sequences, tiles and units before each, the header and every worker's start."""
    rng = np.random.default_rng(2 + mode)
    for rep in range(60):
        S = int(rng.integers(1, 50)) if rep < 50 else int(rng.integers(1020, 2100))
        q_len = int(rng.integers(1, 9)) if mode == 1 else 1
        B = int(rng.integers(1, 400))
        hkv, ctas = int(rng.integers(1, 9)), int(rng.integers(2, 200))
        st = alternating(S, B) if rep % 5 == 0 else bad_starts(rng, S, B)
        if rep >= 55:  # in order up to the second thousand of sequences
            st[:1030] = sorted(min(max(x, 0), B) for x in st[:1030])
        lens = [int(x) for x in rng.integers(0, 700, S)]
        plan = plan_of(mode, st, lens, B * q_len, hkv, ctas, T, q_len)
        words = plan.words().cpu().numpy()
        seqs = taken(st, B * q_len, q_len)
        walk = walk_of(mode, seqs, lens, T)
        workers = ctas // (T // 32)
        per_head = sum(u for _, u in walk)
        bucket = max(-(-per_head * hkv // workers), 1)
        bad = 16 if any(a is None for a, _ in seqs) else 0
        assert list(words[:16]) == [per_head, 0, bucket, 0, -(-per_head * hkv // bucket), S, hkv, workers, B * q_len, mode,
                                    sum(t for t, _ in walk), q_len, bad, T, 0, 0], f"header {rep}"
        at = 16 + 8 * (workers + 1)
        rows, tiles, units = words[at:at + 4 * S].reshape(S, 4), 0, 0
        before = words[at + 4 * S:at + 4 * S + 2 * (S + 1)].view(np.int64)
        for s, ((a, n), (t, u)) in enumerate(zip(seqs, walk)):
            assert list(rows[s][1:]) == [n, lens[s], tiles] and (a is None or rows[s][0] == a), f"map {rep}, sequence {s}"
            assert s == 0 or rows[s][0] >= rows[s - 1][0], f"map {rep}: first rows fall at {s}"
            assert before[s] == units
            tiles, units = tiles + t, units + u
        assert before[S] == units
        start = words[16:at].reshape(workers + 1, 8)
        for j in range(workers + 1):
            g = j * bucket
            if g >= per_head * hkv:
                assert list(start[j]) == [hkv] + [0] * 7
                continue
            s = int(np.searchsorted(before, g % per_head, side="right")) - 1
            assert list(start[j][:2]) == [g // per_head, s] and list(start[j][4:]) == list(rows[s])


@pytest.mark.gpu
def test_tile_numbers_of_many_rows():
    """200 groups that each claim all of 1024 requests: the first has them, the rest are passed over."""
    st = alternating(200, 1024)
    plan = hb.hpc_prefix_plan(tl.i32(st), tl.i32([64] * 200), 1024, 1, 1, num_ctas=152, tile_tokens=32)
    assert plan.words()[10].item() == 32 and hb.hpc_tile_read_error(plan) == 16


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [32, 64])
def test_prompts_of_such_starts(tile):
    """Each row of a sequence that is not passed over is that sequence's; the others keep their bits."""
    rng = np.random.default_rng(7)
    for st in ([0, 20, 5, 40, 60], [0, 60, 0, 60, 0], [30, 10, 20, 15, 60], [-1, 20, 61, 40, 50]):
        lens = [70, 20, 100, 33]
        c = tl.make_cache([lens], 1, "bf16", 5)
        q = tl.make_q((60, 8, 128), 6)
        out, lse = torch.full_like(q, 7.0), torch.full((60, 8), 7.0, device="cuda")
        _, _, plan = hb.prefill(q, c["k_cache"], c["v_cache"], c["tables"][0], tl.i32(st), tl.i32(lens), out=out, out_lse=lse,
                                num_ctas=int(rng.integers(2, 20)), tile_tokens=tile)
        assert hb.hpc_tile_read_error(plan) == 16
        seen = torch.zeros(60, dtype=torch.bool)
        for b, (a, n) in enumerate(taken(st, 60)):
            if n == 0:
                continue
            seen[a:a + n] = True
            ref = tl.attend(q[a:a + n], c["k"][0][b], c["v"][0][b], [max(0, lens[b] - n + i + 1) for i in range(n)])
            tl.check_rows(out[a:a + n], lse[a:a + n], ref, False, f"starts {st}, sequence {b}")
        assert bool((out.cpu()[~seen] == 7).all()) and bool((lse.cpu()[~seen] == 7).all())


@pytest.mark.gpu
def test_prefix_attention_of_such_starts():
    """Groups that each claim the whole batch: the split buffers behind the last row keep their bits."""
    B, S, hkv, ctas = 64, 40, 2, 20
    plens = [200] * S
    c = tl.make_cache([plens], hkv, "bf16", 9)
    q = tl.make_q((B, 8 * hkv, 128), 10)
    for tile in (32, 64):
        plan = hb.hpc_prefix_plan(tl.i32(alternating(S, B)), tl.i32(plens), B, hkv, c["tables"][0].shape[1], num_ctas=ctas, tile_tokens=tile)
        rows = hb._prefix_rows(plan)
        po = torch.full((rows + 256, 128), 7.0, device="cuda")
        pl = torch.full((rows + 256,), 7.0, device="cuda")
        hb.hpc_prefix_attn(q, c["k_cache"], c["v_cache"], c["tables"][0], plan, po[:rows], pl[:rows])
        assert hb.hpc_tile_read_error(plan) == 16
        assert bool((po[rows:] == 7).all()) and bool((pl[rows:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [32, 64])
@pytest.mark.parametrize("q_len", [1, 2])
def test_groups_beside_passed_over_ones_keep_their_prefix(q_len, tile):
    """A merged row finds its group's prefix whatever groups around it are passed over."""
    own, hkv = [5, 64, 0, 130, 17, 1, 70, 9], 1
    for st in ([0, 4, 99, 4, 8], [0, 3, 1, 3, 8], [-2, 0, 5, 2, 8], [2, 2, 6, 0, 6], [0, 8, 0, 8, 0], [4, 0, 4, 4, 9]):
        plens = [200, 128, 70, 300]
        c = tl.make_cache([own, plens], hkv, "bf16", 21)
        q = tl.make_q((8, 8, 128) if q_len == 1 else (8, q_len, 8, 128), 22)
        out, lse, pplan, plan = hb.decode_shared_prefix(q, c["k_cache"], c["v_cache"], c["tables"][0], tl.i32(own), c["tables"][1],
                                                        tl.i32(plens), tl.i32(st), tile_tokens=tile, prefix_num_ctas=6)
        assert hb.hpc_tile_read_error(pplan) == 16 and hb.hpc_decode_read_error(plan) == 0
        groups = taken(st, 8)
        for b in range(8):
            k, v, p = c["k"][0][b], c["v"][0][b], 0
            for g, (a, n) in enumerate(groups):
                if n and a <= b < a + n:
                    k, v, p = torch.cat([c["k"][1][g], k]), torch.cat([c["v"][1][g], v]), plens[g]
            ref = tl.attend(q[b].reshape(q_len, 8, 128), k, v, [p + max(0, own[b] - q_len + i + 1) for i in range(q_len)])
            tl.check_rows(out[b].reshape(q_len, 8, 128), lse[b].reshape(q_len, 8), ref, False, f"starts {st}, request {b}")


@pytest.mark.gpu
def test_lengths_at_the_end_of_31_bits():
    """On the map alone: a tile's last limit, up to 64 past the last key, must not pass 2^31 - 1."""
    lens = [2147483647, 2147483392, 2147483391, 2147483393]
    plan = hb.hpc_prefill_plan(tl.i32([0, 3, 6, 9, 12]), tl.i32(lens), 12, 1, 1 << 26, num_ctas=4, tile_tokens=32)
    assert hb.hpc_tile_read_error(plan) == 4
    rows = plan.words()[16 + 8 * 5:16 + 8 * 5 + 16].view(4, 4)
    assert rows[:, 2].tolist() == [2147483392, 2147483392, 2147483391, 2147483392]
    plan = hb.hpc_prefill_plan(tl.i32([0, 3]), tl.i32([2147483392]), 3, 1, 1 << 26, num_ctas=4, tile_tokens=32)
    assert hb.hpc_tile_read_error(plan) == 0 and plan.words()[0].item() == 2 + 2147483392 // 128
