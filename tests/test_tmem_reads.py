"""Every tensor-memory load names its registers in the wait that completes it. A load's registers are defined,
as the compiler sees it, by the load itself; only a wait that takes them as operands keeps their uses behind it."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "indexer_top_sparse_paged_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))
CALL = re.compile(r"\btmem_ld(16|32|_wait)\(")


def calls(path):
    """(what, arguments split at the top level) of every load and wait, in source order."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for m in CALL.finditer(text):
        if re.search(r"__forceinline__ void $", text[:m.start()]):
            continue  # the definition
        depth, args, start = 1, [], m.end()
        for i in range(m.end(), len(text)):
            depth += text[i] in "([{"
            depth -= text[i] in ")]}"
            if (depth == 1 and text[i] == ",") or depth == 0:
                args.append(text[start:i].strip())
                start = i + 1
            if depth == 0:
                break
        yield m.group(1), [a for a in args if a]


def array(arg):
    return re.match(r"\w+", arg).group(0)


@pytest.mark.parametrize("path", [p for p in SOURCES if list(calls(p))], ids=os.path.basename)
def test_every_load_is_waited_for_by_name(path):
    open_loads = []
    for what, args in calls(path):
        if what != "_wait":
            assert len(args) == 2
            open_loads.append(array(args[1]))
            continue
        assert args and {array(a) for a in args} == set(open_loads), (path, args, open_loads)
        open_loads = []
    assert not open_loads
