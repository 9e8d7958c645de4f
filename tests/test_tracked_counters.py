"""The HBM counters that bench.py reports beside its timings are of the delta kernels as they are: each tracked summary holds the
hash of their present sources. (A change of delta.hip, delta_mfma.hip or delta_common.h makes them stale: helpers of
other kernels have a place elsewhere.)"""
import os
import re

import bench

PROFILES = os.path.join(bench.ROOT, "profiles")


def test_each_counter_summary_is_of_the_present_delta_kernels():
    names = [n for n in sorted(os.listdir(PROFILES)) if n.startswith("pmc_traffic_")]
    assert names
    for name in names:
        fields = dict(re.findall(r"^(\w+):\s*(.+?)\s*$", open(os.path.join(PROFILES, name)).read(), flags=re.M))
        assert fields["kernel_source_sha256"] == bench.delta_source_sha256(), name
        traffic, source = bench.measured_traffic(name[len("pmc_traffic_"):-len(".md")], fields["kernel"])
        assert traffic is not None and traffic > 0, (name, source)
