"""Shared memory of the linear chunk kernel, from its source: what plain stores write before the
tensor copies start lies outside everything that those copies read or write. (Both sides meet at a
barrier only, and a barrier does not order plain stores before the copies' own.)"""

import re
from pathlib import Path

SRC = (Path(__file__).resolve().parent.parent / "gated_delta_rule_144_b200" / "csrc" /
       "kda_linear_chunk.cu").read_text()


def constants():
    """Integer constants of the file, evaluated in their order."""
    code = re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", SRC), flags=re.S)
    known = {}
    for body in re.findall(r"constexpr (?:int|uint32_t) ([^;()]*(?:\([^;]*\))?[^;]*);", code):
        for one in body.split(","):
            m = re.fullmatch(r"\s*(\w+)\s*=\s*(.+?)\s*", one, flags=re.S)
            if not m:
                continue
            expr = re.sub(r"(.+)\?(.+):(.+)", r"((\2) if (\1) else (\3))", m.group(2), flags=re.S)
            try:
                known[m.group(1)] = int(eval(expr.replace("/", "//"), {}, known))
            except (NameError, SyntaxError):
                pass   # depends on a template's argument
    return known


def test_the_slot_search_and_the_tensor_copies_share_nothing():
    c = constants()
    at = re.search(r"chunk_slot<!kOut>\(p, g, tid, reinterpret_cast<int\*>\(sm( \+ \w+)?\)", SRC)
    first = eval("0" + (at.group(1) or ""), {}, c)
    words = c.get("kFindInts", max(c["kSorted"], c["kThreads"] // 32 + 2))
    search = range(first, first + 4 * words)
    copies = [range(0, 2 * c["kStage"]), range(c["OFF_OUT"], c["OFF_OUT"] + c["kPanel"])]
    for x in copies:
        assert search.stop <= x.start or x.stop <= search.start, (search, x)
    assert search.stop <= c["OFF_BAR"] < c["kSmem"] <= 232448
    # every copy's place is one of those two
    for to in re.findall(r"tma_load_3d\((.+?),", SRC):
        assert re.fullmatch(r"st \+ (place\(m\)|ST_V)", to), to
    assert re.findall(r"tma_store_3d\(&maps\.o, (.+?),", SRC) == ["sb + OFF_OUT"]
