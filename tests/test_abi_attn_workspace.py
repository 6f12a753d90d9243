"""The workspace of prompt attention: room for the rows whose keys are shared out, and no more (CPU)."""
import pytest

KV_OP_ATTN_PROMPT = 7
MAX_SHARES = 16


@pytest.fixture(scope="module")
def lib():
    from kv_cache_compression_obs_gb300.build import build
    build()
    from kv_cache_compression_obs_gb300 import api
    return api.library_handle()


# B, Hq, Hkv, Tq, Tk, d, packed sequences, rows of a head that are shared out at most.  152 items are one
# round; an item is 128 rows of two heads, or 256 rows of one head where a KV head has an odd number of them.
CASES = [
    (1, 32, 8, 3712, 32768, 128, 0, 128),     # 29 tiles of 16 items: the last of them
    (1, 32, 8, 2560, 32768, 128, 0, 128),     # 20 tiles
    (1, 32, 8, 2000, 32001, 128, 0, 7 * 128),  # 16 tiles: one round is 9 and a half of them
    (4, 32, 8, 600, 8000, 64, 0, 2 * 128),     # 20 tiles of four batch rows
    (1, 7, 1, 12000, 90000, 64, 0, 5 * 256),   # 47 tiles of 7 items of 256 rows; two rounds are 43
    (1, 32, 8, 16, 32768, 128, 0, 16),        # few rows: all of them, and not whole tiles
    (1, 4, 2, 2048, 2048, 128, 8, 2048),      # packed: no more than the tokens
    (1, 32, 8, 20, 40000, 128, 20, 20),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_room_for_the_shared_rows_alone(lib, case):
    B, Hq, Hkv, Tq, Tk, d, n_seq, rows = case
    got = lib.kv_workspace_size(KV_OP_ATTN_PROMPT, B, Hq, Hkv, Tk, d, Tq, n_seq)
    assert got <= MAX_SHARES * rows * Hq * (4 * d + 8) + 32
    if got:  # at least two shares
        assert got > 2 * min(rows, 16) * Hq * (4 * d + 8)


@pytest.mark.parametrize("Tq", list(range(300, 6000, 257)))
def test_a_chunk_never_takes_more_than_a_round(lib, Tq):
    """Only the last, partial round is shared out: n < 152 items of 256 rows in s shares.  Shares are taken
    where their rounds pay, ceil(n s / 152) (256 / s + 2) < 0.85 (256 + 2) with 256 key tiles, so
    n s < 152 * 0.85 * 258 / (256 / s + 2) <= 12.2 * 152 for s <= 16."""
    got = lib.kv_workspace_size(KV_OP_ATTN_PROMPT, 1, 32, 8, 32768, 128, Tq, 0)
    assert got <= 12.2 * 152 * 256 * (4 * 128 + 8) + 32
