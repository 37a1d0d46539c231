"""The sort by digits is a chain of kernels each of which reads the order that the one of the
digit before has written: behind its own griddep_wait."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "blackwell_tile_gemm_gb300", "csrc")


def code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def kernel(text, name):
    start = text.index(name + "(const RowsArgs p)")
    body = text[text.index("{", start):]
    return body[:body.index("\n}\n")]


def test_an_earlier_digits_order_is_read_behind_the_wait():
    text = code("group_rows.cu")
    # Only these two places read it: the key of a row, and the row itself.
    assert len(re.findall(r"p\.from\[", text)) == 2
    for name in ("count_rows_kernel", "place_rows_kernel"):
        body = kernel(text, name)
        first = min(body.index(x) for x in ("walk<kDigit>", "key_of<kDigit>", "p.from[")
                    if x in body)
        waits = [m.group(1) for m in re.finditer(r"^\s*(.*?)griddep_wait\(\);", body[:first], re.M)]
        assert waits, name
        # Unconditional, or wherever there is such an order.
        assert any(w.strip() == "" or "(kDigit && p.from != nullptr)" in w for w in waits), name
