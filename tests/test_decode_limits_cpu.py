"""What the decode calls ask for and refuse, without a GPU: workspaces, and arrays that may not share memory."""
import ctypes

import pytest

import filtered_int8_ann_b200 as st
from filtered_int8_ann_b200 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return st.lib()


def attend_bytes(lib, T, R, max_q, max_len, heads=8, group=4, dim=128):
    need = ctypes.c_int64(-1)
    c = st._KvCache(None, None, None, None, 1, heads, 16, dim)
    return lib.st_kv_attend_workspace(ctypes.byref(c), T, heads * group, R, max_q, max_len, ctypes.byref(need)), need.value


@pytest.mark.parametrize("T,R,max_q,max_len,group", [
    (2517, 4, 2048, 8192, 4), (8192 + 63, 64, 8192, 65536, 4), (8192 + 63, 64, 8192, 131072, 8), (8200, 16, 2048, 131072, 4),
    (8192 + 999, 1000, 8192, 65536, 4), (70000, 3, 35000, 200000, 1)])
def test_attend_workspace_of_mixed_batches(lib, T, R, max_q, max_len, group):
    """Beside prompts, rows of up to 32 columns (query tokens x heads per cache head) need parts for those columns alone,
    however many tokens the prompts have: 128 MiB of them, or one for each 2048 cached tokens."""
    heads, part = 8, 4 * (128 + 2)
    status, need = attend_bytes(lib, T, R, max_q, max_len, group=group)
    assert status == st.ST_OK
    status, prompts = attend_bytes(lib, T, 1, max_q, max_len, group=group)  # (one row of so many columns is a prompt)
    assert status == st.ST_OK
    assert need - prompts <= max(128 << 20, R * heads * 32 * -(-max_len // 2048) * part)


def test_attend_workspace_of_single_tokens(lib):
    """Tokens behind the last row's take no part."""
    assert attend_bytes(lib, 64, 64, 1, 16384) == attend_bytes(lib, 5000, 64, 1, 16384)


@pytest.mark.parametrize("T,R,max_q,max_len,heads,group", [
    (2**31 - 1, 1, 2**20, 2**31 - 1, 1, 65535), (2**31 - 1, 7, 2**20, 2**31 - 1, 1000, 65), (2**31 - 1, 32768, 33, 2**31 - 1, 1024, 1),
    (2**31 - 1, 32768, 2**20, 2**27, 15, 4369), (2**30, 1, 2**20, 2**30, 4, 16380)])
def test_attend_workspace_that_no_memory_holds(lib, T, R, max_q, max_len, heads, group):
    """Sizes whose workspace would be more than 2^48 bytes (and more than 64 bits count) are refused."""
    assert T * heads * group * -(-max_len // 16384) * 4 * 130 > 2**48
    assert attend_bytes(lib, T, R, max_q, max_len, heads, group) == (st.ST_ERR_UNSUPPORTED, 0)
