"""rf_verify_draft's kernel remembers refused nodes only where children were chosen outright. The form with draft
probabilities never writes them, so it has no such array to read from."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ridge_map_kv_gb300", "csrc", "verify.cu")


def test_the_form_with_draft_probabilities_has_no_refused_nodes():
    code = re.sub(r"//[^\n]*", "", open(SRC).read())
    owners = re.findall(r"struct (\w+(?:<\w+>)?)[^{};]*\{([^{}]*)\}", code)
    assert [name for name, body in owners if re.search(r"\brefused\s*\[", body)] == ["VerifyRefused<false>"]
    # the kernel's shared memory takes it from there
    assert re.search(r"struct VerifyShared : VerifyRefused<kDraft>", code)
