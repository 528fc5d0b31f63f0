"""A wait for stores that other CTAs of the cluster make with st.async, read with plain loads after it, acquires at
cluster scope; the default scope orders them only against this CTA's own threads.  Hardware delivers the data before
the count either way, so no run can show the difference: the sources are read instead."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "precision_quantized_attention_b200", "csrc")


def _read(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name", [n for n in sorted(os.listdir(CSRC)) if n.endswith(".cu")])
def test_waits_for_peers_stores_acquire_at_cluster_scope(name):
    s = _read(name)
    barriers = {b for call in re.findall(r"st_async_v4\((.*?)\);", s, re.S) for b in re.findall(r"BAR\((\w+)", call)}
    assert (name == "gemm_int8.cu") == bool(barriers)
    for b in barriers:
        waits = re.findall(r"(mbar_\w+(?:<\w+>)?)\(BAR\(%s\b" % b, s)
        waits = [w for w in waits if "wait" in w]
        assert waits and set(waits) == {"mbar_wait<true>"}


def test_the_cluster_wait_names_its_scope():
    s = _read("sm100_ptx.cuh")
    body = s[s.index("bool mbar_try_wait_cluster"):]
    assert "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64" in body[:body.index("return ok")]
    wait = s[s.index("template <bool CLUSTER = false>"):]
    assert re.search(r"CLUSTER \? mbar_try_wait_cluster\(bar, parity\) : mbar_try_wait\(bar, parity\)", wait[:1200])
