"""What the launches of the dense feed-forward block read and write, and which
of them may run at the same time, read from the sources (no GPU needed).

A launch starts when all of the one before have said that it may.  An ordinary
one and one that reads what was written say so after everything before them is
over, one that runs beside says so at once; each ends after those before it."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_side_gb300",
                    "csrc")


def launches(name):
    """(mode, after, reads, writes) of a function's launches, in order."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "api.cu")).read())
    body = text[text.index(f"mok_status {name}("):]
    body = body[:body.index("\n}\n")]
    found, after, gates, outs = [], None, set(), set()
    for line in re.split(r";", body):
        if m := re.search(r"ffn_params\(ws, (\w+),", line):
            after, gates, outs = m.group(1), set(), set()
        elif m := re.search(r"p\.(h|u) = ", line):
            gates.add(m.group(1))
        elif m := re.search(r"p\.out\[\d\] = (?:\w+<[^>]*>\()?([^()]+)\)?\s*$", line):
            outs.add(m.group(1).strip())
        elif m := re.search(r"launch_ffn\((\w+), (.*)", line, re.S):
            reads = {o.strip() for o in re.findall(r"\{([^{},]+),", m.group(2))}
            mode = m.group(1)
            found.append((mode, after, reads | (gates if mode == "FFN_DA" else set()),
                          outs | (gates if mode == "FFN_GATE" else set())))
    return found


def faults(order):
    """What a launch touches that one which may still run beside it writes, or the other way round."""
    bad = []
    for i, (mode, after, reads, writes) in enumerate(order):
        if after != "FFN_BESIDE_IT":
            continue
        j = i - 1
        while order[j][1] == "FFN_BESIDE_IT":
            j -= 1
        for other, _, r, w in order[j:i]:
            bad += [(mode, other, t) for t in reads & w | writes & (r | w)]
    return bad


def test_launches_beside_each_other_share_nothing_that_is_written():
    for name, modes in (("ffn_forward", ["FFN_GATE", "FFN_OUT"]),
                        ("mok_ffn_backward", ["FFN_DA", "FFN_DW2", "FFN_DX", "FFN_DW13"])):
        order = launches(name)
        assert [m for m, *_ in order] == modes
        assert order[0][1] == "FFN_AFTER_ALL" and all(r and w for _, _, r, w in order), order
        assert not faults(order), faults(order)
        # every launch that is not beside the one before reads something that was written here
        written = set()
        for _, after, reads, writes in order:
            assert (after == "FFN_AFTER_ALL") == (not written) and (after != "FFN_READS_IT" or reads & written)
            written |= writes


def test_another_order_would_not_do():
    da, dw2, dx, dw13 = launches("mok_ffn_backward")
    assert {"s + L.dh", "s + L.du"} <= da[3] & dw13[2] & dx[2]
    assert faults([da, dw13, dw2, dx]) and faults([da, dw2, dw13, dx])


def test_what_a_launch_lets_start():
    """Its own wait stands before the word to the next launch; one beside another waits at its end."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "ffn.cu")).read())
    turn = text[text.index("void launch_in_turn("):]
    turn = turn[:turn.index("}")]
    assert turn.index("if (p.after == FFN_READS_IT) griddep_wait();") < turn.index("griddep_launch_dependents();")
    assert text.count("griddep_launch_dependents();") == 1
    assert len(re.findall(r"if \(p\.after == FFN_BESIDE_IT\) griddep_wait\(\);\n\}", text)) == 2
