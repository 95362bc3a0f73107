"""Host-only checks of the kernels' inline PTX."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "second_order_optimizer_shampoo_b200", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def statements(text):
    """The asm statements of a source."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[m.start():i]


@pytest.mark.parametrize("name", SOURCES)
def test_tensor_memory_loads_wait_in_their_own_statement(name):
    """A load's registers hold its values only behind tcgen05.wait::ld; in a
    statement of its own the wait does not keep register arithmetic behind it."""
    with open(os.path.join(CSRC, name)) as f:
        for asm in statements(f.read()):
            if "tcgen05.ld." in asm:
                assert "tcgen05.wait::ld" in asm, asm[:200]


@pytest.mark.parametrize("name", SOURCES)
def test_no_choice_is_made_for_a_fixed_number_of_sms(name):
    """Tile sizes and grids follow the device's own SM count: no constant stands in
    for it (a default that a query overwrites is not one)."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"\bconst(?:expr)?\s+\w+\s+(?:pairs|sms)\s*=\s*\d+", text)
