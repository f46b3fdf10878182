"""Loads that the library does not make, looked for in its sources: a tensor or bulk load that sends to
several blocks would read a peer's memory, where a caller's pointer names some, and may not be in
code that ranks of several GPUs run."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hyper_connection_mix_gb300", "csrc")


def statements():
    """(file, the string literals joined) of every asm statement."""
    for name in sorted(os.listdir(CSRC)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(((?:\s*\"(?:[^\"\\]|\\.)*\")+)", text):
            yield name, "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m.group(1)))


def test_no_copy_is_sent_to_several_blocks():
    found = [s for s in statements() if "cp.async.bulk" in s[1]]
    assert found, "no bulk copies found: has the form of the statements changed?"
    assert not [s for s in found if "multicast" in s[1]]
