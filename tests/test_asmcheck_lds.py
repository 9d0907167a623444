"""The static check's rule for loads from memory straight to LDS, on
hand-written snippets whose verdict is known."""

import textwrap

import pytest

from moe_grouped_precision_amd import asmcheck, build


def _check(tmp_path, body, lds=True):
    src = tmp_path / "k.s"
    src.write_text("kern:\n" + textwrap.dedent(body) + "\ts_endpgm\n")
    return asmcheck.check(str(src), lds=lds)


PREFIX = """
        global_load_lds_dwordx4 v[10:11], off
        global_load_dwordx4 v[0:3], v12, s[2:3]
        global_load_dwordx4 v[4:7], v12, s[2:3]
"""


def test_wait_that_covers_the_load(tmp_path):
    body = PREFIX + """
        s_waitcnt vmcnt(2)
        s_barrier
        ds_read_b128 v[20:23], v13
    """
    assert _check(tmp_path, body) == []


@pytest.mark.parametrize("use", ["s_barrier", "ds_read_b128 v[20:23], v13", "ds_load_b32 v20, v13"])
@pytest.mark.parametrize("wait", ["", "s_waitcnt vmcnt(3)", "s_waitcnt lgkmcnt(0)"])
def test_wait_that_leaves_it_pending(tmp_path, use, wait):
    body = PREFIX + f"""
        {wait}
        {use}
    """
    assert any("load to LDS pending" in f for f in _check(tmp_path, body))
    assert not any("load to LDS pending" in f for f in _check(tmp_path, body, lds=False))


def test_one_load_fewer_on_one_path(tmp_path):
    # the count holds on the long path only
    body = """
        global_load_lds_dwordx4 v[10:11], off
        global_load_dwordx4 v[0:3], v12, s[2:3]
        s_cbranch_scc1 .Lskip
        global_load_dwordx4 v[4:7], v12, s[2:3]
    .Lskip:
        s_waitcnt vmcnt(2)
        s_barrier
    """
    assert any("load to LDS pending" in f for f in _check(tmp_path, body))


def test_loads_in_a_loop_and_the_buffer_form(tmp_path):
    body = """
    .Lloop:
        buffer_load_dwordx4 v10, s[4:7], 0 offen lds
        s_cbranch_scc1 .Lloop
        global_load_dwordx4 v[0:3], v12, s[2:3]
        s_waitcnt vmcnt({})
        s_barrier
    """
    assert _check(tmp_path, body.format(1)) == []
    assert any("load to LDS pending" in f for f in _check(tmp_path, body.format(2)))


def test_stores_count_as_operations(tmp_path):
    body = """
        global_load_lds_dwordx4 v[10:11], off
        global_store_short v[14:15], v16, off
        s_waitcnt vmcnt(1)
        s_barrier
    """
    assert _check(tmp_path, body) == []


def test_matvec_is_built_under_the_rule():
    assert build.ASM_CHECKED["matvec.hip"] is True
