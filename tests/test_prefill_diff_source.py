"""What the kernels' sources must hold to, and no run can show: the memory model's order
between the two CTAs of a cluster, and copies that stay within a CTA."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_167_gb300", "csrc")


def code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"/\*.*?\*/", " ", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", " ", text)


def waits(text):
    """(wait, its barrier's expression) of every call."""
    return re.findall(r"\b(mbar_wait\w*)\((\w+)", text)


def test_waits_for_the_other_cta_acquire_at_cluster_scope():
    """Barriers that another CTA completes (an arrival, a commit or a store of its own) are
    waited for with an acquire at cluster scope: at the CTA's scope, the default, nothing
    orders the reads behind the wait after what the other CTA wrote."""
    text = code("pa_prefill_diff.cu")
    assert ".acquire.cluster." in text
    remote = {"barUnit", "my_full", "my_norm"}
    seen = waits(text)
    for name in remote:
        kinds = {kind for kind, bar in seen if bar == name}
        assert kinds == {"mbar_wait_cluster"}, f"{name}: {sorted(kinds)}"


def test_no_load_is_multicast():
    """The library runs on every GPU of a machine and takes any pool's address: no tensor or
    bulk copy in it writes to several CTAs.  (A commit that arrives on several is no copy.)"""
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".cpp", ".h")):
            joined = re.sub(r'"\s*"', "", code(name))          # string literals of one instruction
            copies = [line for line in re.findall(r"cp\.async\.bulk[\w.:]*", joined) if "multicast" in line]
            assert not copies, f"{name}: {copies}"
