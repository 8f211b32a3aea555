"""Layer operators at the edges of what they take, without a GPU."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "state_space_sequence_ssm_amd", "csrc")


# ---------------------------------------------------------------- the staging waves' order
def _body(text, name):
    """The body of the lambda `name` of a kernel."""
    i = text.index(f"auto {name} = [&](")
    i = text.index("{", i)
    depth, j = 0, i
    while True:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
        if depth == 0:
            return text[i:j]


@pytest.mark.parametrize("source,kernel", [("scan.hip", "scan_kernel"), ("scan_backward.hip", "reverse_kernel")])
def test_what_a_step_finishes_is_not_what_it_stages(source, kernel):
    """Between two barriers a staging wave finishes one tile and then stages another in
    the same half of LDS, while the other waves may still be finishing: no array is
    both read by the one and written by the other."""
    with open(os.path.join(CSRC, source)) as f:
        text = f.read()
    text = re.sub(r"//[^\n]*", "", text[text.index(f"void {kernel}("):])
    names = "dl|us|ds|bc|ys|o|gB|gA|wp|sdu"
    used = {k: set(re.findall(rf"&?(?:\bsh\.)?\b({names})\[", _body(text, k))) for k in ("finish", "stage")}
    assert used["stage"] >= {"dl", "us", "bc"} and used["finish"]
    assert not used["finish"] & used["stage"]
