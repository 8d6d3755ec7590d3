"""The recorded counters of the k-quant and TQ4_1S kernels are attached to a benchmark line while
the sources they were captured with are unchanged. Those sources hold nothing of the
decode-step operators, so that work on these leaves the record standing. CPU only."""
import json
import os
import re

from conftest import ROOT

OWN = re.compile(r"kq_add_rmsnorm_q8_1|kq_swiglu_q8_1|kq_moe_route\b|matvec_g4|KQ_BF16|G4")


def test_recorded_sources_hold_no_decode_step_operators():
    with open(os.path.join(ROOT, "profiles", "ncu_sections.json")) as f:
        entries = dict(json.load(f)["sections"])
    with open(os.path.join(ROOT, "profiles", "ncu_traffic.json")) as f:
        entries.update(json.load(f))
    assert entries
    for name, e in entries.items():
        for src in e["sources"]:
            with open(os.path.join(ROOT, src)) as f:
                assert not OWN.search(f.read()), f"{name}: {src}"
