"""The weight gradient's barriers join the two CTAs of a pair: what its source
says about the scope of every arrival and wait, read on the CPU (a weaker scope
would be a race, which no run on a GPU has to show)."""
import os
import re

from zero_distributed_optimizer_gb300 import build as libbuild


def _instructions(name):
    with open(os.path.join(libbuild.CSRC, "wgrad.cu")) as f:
        text = re.sub(r'"\s*\n\s*"', "", f.read())  # adjacent pieces of one string
    return re.findall(re.escape(name) + r"[\w.:]*", text)


def test_waits_acquire_at_the_clusters_scope():
    waits = _instructions("mbarrier.try_wait") + _instructions("mbarrier.test_wait")
    assert waits and all(".acquire.cluster." in w for w in waits), waits


def test_arrivals_on_the_other_ctas_barriers_release_at_the_clusters_scope():
    """By a release of their own, or by a release fence of that scope directly
    before a relaxed arrival."""
    with open(os.path.join(libbuild.CSRC, "wgrad.cu")) as f:
        text = re.sub(r'(\\n\\t)?"\s*\n\s*"', "", f.read())
    arrivals = re.findall(r"([\w.:]*);?(mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*)", text)
    assert arrivals
    for before, arrival in arrivals:
        fenced = ".relaxed.cluster." in arrival and before.startswith("fence.release.") and before.endswith(".cluster")
        assert ".release.cluster." in arrival or fenced, (before, arrival)
