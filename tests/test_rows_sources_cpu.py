"""What no run can show about the row operators' kernels, read off their sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int2_kv_cache_append_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["attn_rows.cu", "attn_rows_tc.cu", "attn_rows_lanes.cu"])
def test_attention_reads_the_calls_own_results_by_plain_loads(name):
    """These kernels start while the query rotation still writes, so the
    read-only data path is not for what they load themselves (the cache, which
    nobody writes during the call, is loaded in rows_tc.cuh)."""
    code = _code(name)
    assert "qrot" in code or "load_queries" in code
    assert "__ldg" not in code



@pytest.mark.parametrize("name,first_read", [("attn_rows_tc.cu", "load_queries<"), ("attn_rows_lanes.cu", "a.qrot")])
def test_attention_beside_its_predecessor_acquires_the_queries(name, first_read):
    """The kernel that does not wait for the one before it takes the queries
    from that one's release, with a barrier behind it, before it reads them."""
    code = _code(name)
    acquire = code.index("a.beside && !ready_wait(a.ready")
    assert acquire < code.index("__syncthreads()") < code.index(first_read)
