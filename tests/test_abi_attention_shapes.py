"""Shapes that the attention takes and refuses (no GPU needed)."""
import pytest

from test_abi_attention import A, _attend, _need

SHARED = dict(group_starts=A, shared_lens=A)


@pytest.mark.parametrize("kw", [
    dict(seqs=1024, tokens=9215, max_q_len=8192, q_heads=32, kv_heads=8, max_pages=8192, max_kv_len=131072),
    dict(seqs=4096, tokens=20479, max_q_len=16384, q_heads=32, kv_heads=8, max_pages=1024, max_kv_len=16384),
    dict(seqs=4096, tokens=16384, max_q_len=4, q_heads=32, kv_heads=8, max_pages=2048, max_kv_len=32768, groups=4096, max_shared_len=16384),
    dict(seqs=65536, tokens=65535, max_q_len=65535, q_heads=1024, kv_heads=1024, head_dim=64, max_pages=64, max_kv_len=1024, groups=65536,
         max_shared_len=512),
    dict(seqs=65536, tokens=65536, max_q_len=1, q_heads=32, kv_heads=8, page_size=1024, max_pages=1 << 20, max_kv_len=1 << 30),
    dict(seqs=65536, tokens=65535, max_q_len=1, q_heads=1023, kv_heads=1023, page_size=1024, max_pages=1 << 20, max_kv_len=1 << 30),
    dict(seqs=1, tokens=1 << 20, max_q_len=1 << 20, q_heads=63, kv_heads=21, page_size=64, max_pages=1 << 18, max_kv_len=1 << 17)],
    ids=["chunk", "prompts", "groups", "heads", "tokens", "pairs", "prompt"])
def test_products_of_bounds(kw):
    """What is laid out goes by the rows that there are: sequences times the longest one's rows may be any number."""
    need = _need(**{k: v for k, v in kw.items() if k not in SHARED})
    assert 16 <= need <= 1 << 38
    assert _attend(**kw, **(SHARED if "groups" in kw else {}), scratch_bytes=need - 1) == 4


def test_scratch_past_what_a_card_has():
    """Rows times pieces of 1024 pages: 2^38 bytes and no more."""
    kw = dict(seqs=1, tokens=1 << 20, max_q_len=1 << 20, q_heads=32, kv_heads=8, head_dim=128, page_size=16, max_pages=1 << 16)
    most = _need(**kw, max_kv_len=15 * 16384 - 15)
    assert 0 < most <= 1 << 38
    assert _need(**kw, max_kv_len=16 * 16384) == 0 and _attend(**kw, max_kv_len=16 * 16384, scratch_bytes=1 << 40) == 2
