"""Every bounded wait of a call reports in the status word that the caller
gave.  (A wait that gives up cannot be brought about from outside, so this
looks at the sources.)  Host only."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_head_latent_absorbed_b200", "csrc")


def test_no_call_goes_through_an_entry_point_that_has_no_status():
    # mla_fold_wuk is for tests and takes no status: its kernel gets a null one
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        text = re.sub(r"//.*", "", open(path).read())
        calls = re.findall(r"(?<!int )\bmla_fold_wuk\s*\(", text)
        assert not calls, os.path.basename(path)
