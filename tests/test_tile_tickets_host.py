"""The tile kernels of the gated recurrence hand each block its next tile through shared
memory, by one thread, with one barrier of the block a tile where every tile is a group of
its own.  A warp that is held up after that barrier still has the ticket to read while
thread 0 may be as far as the next tile's.  Such a mix of two tiles cannot be provoked
reliably (and would leave a block's warps at different barriers), so the order is read off
the sources: in the loops as written, with only the barriers that every call passes, a
ticket's place is written again only behind a barrier that all its readers have passed."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_54_b200", "csrc")
KERNELS = [("ssm_gscan_tok.cu", "k_tok_fwd"), ("ssm_gscan_tok.cu", "k_tok_bwd"), ("ssm_gscan_rows.cu", "k_tiles_fwd"),
           ("ssm_gscan_rows.cu", "k_tiles_bwd")]


def _braced(src, start):
    """The text of the block whose opening brace is the first one from `start`."""
    first = at = src.index("{", start)
    depth = 0
    while True:
        depth += {"{": 1, "}": -1}.get(src[at], 0)
        at += 1
        if depth == 0:
            return src[first + 1:at - 1]


def _loop(path, kernel):
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, path)).read())
    body = _braced(src, re.search(r"\) %s\(GsParams p\)" % kernel, src).end())
    return _braced(body, body.index("for (int stg = 0;; stg ^= 1)"))


def _events(loop):
    """(kind, slot expression) of the loop's statements in order: write, read, barrier."""
    out = []
    depth = 0
    for line in loop.split("\n"):
        code = line.strip()
        write = re.search(r"hand_out\((sm\.ticket[^,]*),", code)
        read = re.match(r"const Taken next = (sm\.ticket[^;]*);", code)
        if write:
            out.append(("write", write.group(1)))
        elif read:
            out.append(("read", read.group(1)))
        elif depth == 0 and code.startswith("__syncthreads();"):  # neither in an if nor in a block
            out.append(("barrier", None))
        depth += line.count("{") - line.count("}")
    return out


def races(events, rounds=4):
    """Accesses to one slot of which one is a write, with no barrier between them, over some
    rounds of the loop; a thread's own accesses (the writer's of one round) aside."""
    trace = []
    for i in range(rounds):
        for kind, slot in events:
            trace.append((kind, slot and slot.replace("stg", str(i % 2)), i))
    found = []
    for a, (kind, slot, i) in enumerate(trace):
        if kind == "barrier":
            continue
        for kind2, slot2, j in trace[a + 1:]:
            if kind2 == "barrier":
                break
            if slot2 == slot and "write" in (kind, kind2):
                found.append((kind, kind2, slot, i, j))
    return found


@pytest.mark.parametrize("path,kernel", KERNELS)
def test_a_ticket_is_read_before_the_next_one_takes_its_place(path, kernel):
    events = _events(_loop(path, kernel))
    assert [k for k, _ in events].count("write") == 1 and [k for k, _ in events].count("read") == 1, events
    assert not races(events), (events, races(events))


def test_the_model_tells_one_place_from_two():
    one = [("write", "t"), ("barrier", None), ("read", "t")]
    assert races(one) and not races(one + [("barrier", None)])
    assert not races([(k, s and "t[stg]") for k, s in one])
    assert races([("write", "t[stg]"), ("read", "t[stg]"), ("barrier", None)])
