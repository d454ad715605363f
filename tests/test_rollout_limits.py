"""nvfp4_kv_attention's limits on its sizes, as include/fp4q/rollout.h states
them: refused on the host as a shape, with no workspace asked for (no GPU
needed; nothing here launches a kernel)."""
import fp4_block_quantization_amd as fq
from test_rollout_host import A4, SHAPE, attend


def need(**kw):
    a = dict(page=16, heads=2, dim=64, batch=2, t=1, q_heads=4, max_pages=3, ppages=0, groups=0)
    a.update(kw)
    return fq.rollout_lib().nvfp4_kv_attention_workspace_bytes(*a.values())


def refused(**kw):
    prefix = dict(ptable=A4, plens=A4, offs=A4) if kw.get("groups") else {}
    given = dict(kw, q_stride=kw.get("q_heads", 4) * kw.get("dim", 64), **prefix)
    return attend(**given) == SHAPE and need(**kw) == 0


def test_more_query_rows_than_one_launch_takes_are_accepted():
    # an ordinary prefill: 64 prompts of 4096 tokens and 64 heads, 2^24 rows
    assert need(batch=64, t=4096, q_heads=64, max_pages=256, ppages=2, groups=1) > 2 ** 24 * 64 * 4


def test_query_rows_past_31_bits():
    assert refused(batch=2, t=1 << 28, q_heads=4)
    assert need(batch=1, t=1 << 28, q_heads=4, heads=4, ppages=1, groups=1) > 0
    assert refused(batch=65536)
    assert refused(groups=65536, ppages=1)


def test_room_of_the_tables_past_31_bits():
    # 2^24 tiles of 64 tokens a table, read by 64 x 2 items: 2^31
    assert refused(batch=64, max_pages=1 << 26)
    assert need(batch=63, max_pages=1 << 26) > 0
    # as a prefix: groups of 1024 x 2 rows, 128 or 64 blocks of 16 rows and two heads each
    wide = dict(q_heads=4, t=1024, max_pages=1, ppages=1 << 26)
    assert refused(batch=2, groups=1, **wide)
    assert need(batch=2, groups=1, **dict(wide, ppages=1 << 20)) > 0
