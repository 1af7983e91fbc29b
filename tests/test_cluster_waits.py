"""Memory scopes of the waits in the kernel sources.  A wait that another block
of the cluster ends (by st.async into this block's shared memory) has to acquire
at cluster scope for that block's data to be visible: an order that no run can be
relied on to miss, so it is checked in the source.  Needs no GPU."""
import os
import re

from linear_attention_feature_gb300 import build as labuild


def source(name):
    with open(os.path.join(labuild.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_waits_for_cluster_maps_acquire_at_cluster_scope():
    # the only barrier that other blocks complete is the one that send_map counts on
    text = source("la_recurrence.cuh")
    sent = re.findall(r"send_map<V>\(.*?&(\w+)\[", text)
    assert sent and set(sent) == {"maps_in"}
    waits = re.findall(r"\bwait_for(<\w+>)?\(&(\w+)", text)
    assert sorted(b for _, b in waits) == ["full", "maps_in", "state_in"]
    for scope, bar in waits:
        assert (scope == "<true>") == (bar in sent), (bar, scope)
    body = text[text.index("bool wait_for("):]
    assert re.search(r"kCluster \? tc::mbar_try_wait_cluster_ns", body)
    ptx = source("la_tc_ptx.cuh")
    form = ptx[ptx.index("bool mbar_try_wait_cluster_ns"):]
    assert "mbarrier.try_wait.parity.acquire.cluster.shared::cta" in form[:form.index("return")]


def test_no_other_kernel_receives_data_from_another_block():
    for path in labuild.sources() + [os.path.join(labuild.CSRC, "la_tc_ptx.cuh")]:
        text = source(os.path.basename(path))
        assert "st.async" not in text and "multicast" not in text, path
