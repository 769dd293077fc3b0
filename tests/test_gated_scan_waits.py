"""The waits of the recurrence's cluster exchange, in the source: what other blocks of a cluster
send (st.async, counted by `low` and `high`) is released at cluster scope and has to be acquired at
that scope.  Nothing on a GPU shows a missing scope reliably, so the text is looked at."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_ssm_sequence_b200",
                   "csrc", "gated_scan.cu")


def test_maps_of_other_blocks_are_acquired_at_cluster_scope():
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    waits = re.findall(r"(\w+)(<\w+>)?\(\s*&(?:x\.)?(low|high|full)\[", text)
    waits = [w for w in waits if "wait" in w[0]]
    assert {w[2] for w in waits} == {"low", "high", "full"}
    for name, source, bar in waits:
        assert (name, source) == ("wait_bar", "<kOwnLoads>" if bar == "full" else "<kClusterMaps>"), bar
    # kClusterMaps waits, first poll and slow path alike, go through the one form with this scope
    assert text.count("mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64") == 1
    assert re.search(r"S == kClusterMaps \? try_wait_cluster\(bar, parity\) : tc::mbar_try_wait\(bar, parity\)", text)
    assert text.count("tc::mbar_try_wait(") == 1 and text.count("try_wait<S>(bar, parity)") == 2
